"""Refusals of the token log probabilities, the block norms and the adapters, which
come back before any CUDA call (the pointers here are never dereferenced), and the
64-bit gradients of their definitions against differences."""
import ctypes as C

import pytest

torch = pytest.importorskip("torch")
from tuning_refs import (INF, adapter, adapter_grad, logprobs, logprobs_grad, residual_norm,  # noqa: E402
                         residual_norm_grad)

P, L, Z, F = C.c_void_p, C.c_longlong, C.c_size_t, C.c_float
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    from quantized_expert_ffn_warp_gb300 import build, moe
    build.build()
    return moe.load_library()


def refused(lib, rc, code):
    return rc == code and lib.moe_last_error().decode() != ""


def overlaps(lib, rc):
    return rc == -1 and "overlap" in lib.moe_last_error().decode()


# ---------------------------------------------------------------- log probabilities

LP = dict(logits=0x100000, dtype=1, ld=1000, n=8, V=1000, targets=0x20000, top=5, logp=0x30000,
          ent=0x40000, stats=0x50000, ids=0x60000, tlp=0x70000, ws=0x80000, ws_bytes=None)


def token_logprobs(lib, **kw):
    a = dict(LP, **kw)
    size = a["ws_bytes"]
    if size is None:
        size = lib.moe_token_logprobs_workspace(a["n"], a["V"], a["dtype"], a["top"])
    return lib.moe_token_logprobs(P(a["logits"]), a["dtype"], L(a["ld"]), a["n"], a["V"],
                                  P(a["targets"]), a["top"], P(a["logp"]), P(a["ent"]),
                                  P(a["stats"]), P(a["ids"]), P(a["tlp"]), P(a["ws"]), Z(size),
                                  None)


def token_logprobs_grad(lib, **kw):
    a = dict(LP, dlogp=0x90000, dent=0xA0000, out=0x200000, ldd=1000)
    a.update(kw)
    return lib.moe_token_logprobs_grad(P(a["logits"]), a["dtype"], L(a["ld"]), a["n"], a["V"],
                                       P(a["targets"]), P(a["stats"]), P(a["ent"]), P(a["dlogp"]),
                                       P(a["dent"]), P(a["out"]), L(a["ldd"]), None)


LP_BOTH = [(dict(logits=None), -1), (dict(stats=None), -1), (dict(ent=None), -1),
           (dict(dtype=3), -2), (dict(dtype=-1), -2), (dict(n=0), -1), (dict(n=-4), -1),
           (dict(n=(1 << 26) + 1), -1), (dict(V=0), -1), (dict(V=(1 << 20) + 1, ld=1 << 21), -1),
           (dict(ld=999), -1), (dict(ld=(1 << 31) + 1), -1), (dict(logits=0x100001), -1),
           (dict(targets=0x20002), -1), (dict(stats=0x50004), -1), (dict(ent=0x40002), -1)]


@pytest.mark.parametrize("kw,code", LP_BOTH + [
    (dict(logp=None), -1), (dict(ids=None), -1), (dict(tlp=None), -1), (dict(top=-1), -1),
    (dict(top=33), -1), (dict(V=4, top=5), -1), (dict(V=100000, ld=100000, ws=None), -1),
    (dict(V=100000, ld=100000, ws_bytes=100), -1), (dict(V=100000, ld=100000, ws=0x80010), -1)])
def test_token_logprobs_refuses(lib, kw, code):
    assert refused(lib, token_logprobs(lib, **kw), code)


@pytest.mark.parametrize("kw,code", LP_BOTH + [
    (dict(out=None), -1), (dict(targets=None), -1), (dict(dlogp=None, dent=None), -1),
    (dict(ldd=999), -1), (dict(out=0x200001), -1), (dict(dlogp=0x90001), -1),
    (dict(dent=0xA0002), -1)])
def test_token_logprobs_grad_refuses(lib, kw, code):
    assert refused(lib, token_logprobs_grad(lib, **kw), code)


@pytest.mark.parametrize("kw,hit", [
    (dict(), False), (dict(logp=0x40000), True), (dict(ent=0x20000), True),
    (dict(stats=0x100000 + 1992), True), (dict(stats=0x100000 + 16000), False),
    (dict(stats=0x100000 + 2000, ld=2000, n=2), False), (dict(tlp=0x60000 + 156), True),
    (dict(tlp=0x60000 + 160), False), (dict(ws=0x20000, V=100000, ld=100000), True),
    (dict(targets=None, logp=0x40000), False), (dict(top=0, ids=0x40000, tlp=0x40000), False)])
def test_token_logprobs_overlaps(lib, kw, hit):
    rc = token_logprobs(lib, **kw)
    assert rc != 0 and overlaps(lib, rc) == hit


@pytest.mark.parametrize("kw,hit", [
    (dict(out=0x100000), False), (dict(out=0x100002), True), (dict(out=0x100000, ldd=1200), True),
    (dict(out=0x100000 + 16000), False), (dict(out=0x20000 - 1990), True), (dict(ent=0x200000), True),
    (dict(ent=0x200000, dent=None), False), (dict(out=0x100000 + 2000, ld=2000, ldd=2000), False),
    (dict(out=0x100000, n=1), False), (dict(out=0x100002, n=1), True)])
def test_token_logprobs_grad_overlaps(lib, kw, hit):
    rc = token_logprobs_grad(lib, **kw)
    assert rc != 0 and overlaps(lib, rc) == hit


def test_token_logprobs_workspace_sizes(lib):
    ws = lib.moe_token_logprobs_workspace
    assert ws(0, 8, 0, 0) == 0 and ws(1, 0, 0, 0) == 0 and ws(1, 1 << 21, 0, 0) == 0
    assert ws(1, 1 << 20, 3, 0) == 0 and ws(1, 1 << 20, 0, 33) == 0
    assert 0 < ws(1, 1 << 20, 0, 0) < ws(1, 1 << 20, 0, 1) == ws(1, 1 << 20, 0, 32)
    assert ws(1000, 1 << 20, 0, 32) == 0 and ws(1, 100, 0, 32) == 0


# ---------------------------------------------------------------- block norms

RN = dict(resid=0x100000, ld_resid=64, y=0x200000, ld_y=64, dtype=1, n=8, H=64, gain=0x10000,
          gate=0x20000, per_token=1, scale=1.0, next_gain=0x30000, eps=1e-6, out=0x300000, ld_out=64,
          xn=0x400000, ld_xn=64, stats=0x40000)


def norm(lib, **kw):
    a = dict(RN, **kw)
    return lib.moe_residual_norm(P(a["resid"]), L(a["ld_resid"]), P(a["y"]), L(a["ld_y"]),
                                 a["dtype"], a["n"], a["H"], P(a["gain"]), P(a["gate"]),
                                 a["per_token"], F(a["scale"]), P(a["next_gain"]), F(a["eps"]),
                                 P(a["out"]), L(a["ld_out"]), P(a["xn"]), L(a["ld_xn"]),
                                 P(a["stats"]), None)


def norm_grad(lib, **kw):
    a = dict(RN, dout=0x500000, ld_dout=64, dxn=0x600000, ld_dxn=64, dresid=0x700000, ld_dresid=64,
             dy=0x800000, ld_dy=64, dgain=0x50000, dgate=0x60000, dnext=0x70000, ws=0x900000,
             ws_bytes=None)
    a.update(kw)
    size = a["ws_bytes"]
    if size is None:
        size = lib.moe_residual_norm_grad_workspace(a["n"], a["H"])
    return lib.moe_residual_norm_grad(
        P(a["dout"]), L(a["ld_dout"]), P(a["dxn"]), L(a["ld_dxn"]), P(a["out"]), L(a["ld_out"]),
        P(a["y"]), L(a["ld_y"]), P(a["stats"]), a["dtype"], a["n"], a["H"], P(a["gain"]),
        P(a["gate"]), a["per_token"], F(a["scale"]), P(a["next_gain"]), P(a["dresid"]),
        L(a["ld_dresid"]), P(a["dy"]), L(a["ld_dy"]), P(a["dgain"]), P(a["dgate"]), P(a["dnext"]),
        P(a["ws"]), Z(size), None)


RN_BOTH = [(dict(y=None), -1), (dict(stats=None), -1), (dict(dtype=2), -2), (dict(n=0), -1),
           (dict(n=(1 << 26) + 1), -1), (dict(H=0), -1), (dict(H=60), -1), (dict(H=16392), -1),
           (dict(next_gain=None), -1), (dict(scale=NAN), -1), (dict(scale=INF), -1),
           (dict(ld_y=56), -1), (dict(ld_y=65), -1), (dict(y=0x200008), -1), (dict(gain=0x10002), -1),
           (dict(gate=0x20001), -1), (dict(gate=0x20002, per_token=0), -1), (dict(stats=0x40004), -1),
           (dict(ld_out=(1 << 31) + 8), -1)]


@pytest.mark.parametrize("kw,code", RN_BOTH + [
    (dict(resid=None), -1), (dict(out=None), -1), (dict(eps=-1.0), -1), (dict(eps=NAN), -1),
    (dict(eps=INF), -1), (dict(xn=0x400004), -1), (dict(ld_resid=48), -1)])
def test_residual_norm_refuses(lib, kw, code):
    assert refused(lib, norm(lib, **kw), code)


@pytest.mark.parametrize("kw,code", RN_BOTH + [
    (dict(out=None), -1), (dict(dresid=None), -1), (dict(dy=None), -1), (dict(ws=None), -1),
    (dict(ws_bytes=64), -1), (dict(ws=0x900004), -1), (dict(dout=None, dxn=None), -1),
    (dict(gain=None), -1), (dict(gate=None), -1), (dict(dxn=None), -1), (dict(dgain=0x50002), -1),
    (dict(ld_dxn=32), -1)])
def test_residual_norm_grad_refuses(lib, kw, code):
    assert refused(lib, norm_grad(lib, **kw), code)


@pytest.mark.parametrize("kw,hit", [
    (dict(), False), (dict(out=0x100000), False), (dict(out=0x100000, ld_out=128), True),
    (dict(out=0x200000), True), (dict(out=0x100010), True), (dict(xn=0x300000), True),
    (dict(xn=0x100000), True), (dict(xn=None, ld_xn=0), False), (dict(stats=0x300000), True),
    (dict(stats=0x10000), True), (dict(out=0x100080, ld_out=128, ld_resid=128), False),
    (dict(out=0x100000, n=1), False), (dict(xn=0x30000, n=1), True)])
def test_residual_norm_overlaps(lib, kw, hit):
    rc = norm(lib, **kw)
    assert rc != 0 and overlaps(lib, rc) == hit


@pytest.mark.parametrize("kw,hit", [
    (dict(), False), (dict(dresid=0x500000), False), (dict(dresid=0x600000), True),
    (dict(dy=0x500000), True), (dict(dy=0x200000), True), (dict(dgain=0x60000), True),
    (dict(dgate=0x20000), True), (dict(dgain=0x50000, dnext=0x50000 + 252), True),
    (dict(dnext=0x50000 + 256), False), (dict(ws=0x500000), True),
    # nothing is summed over the tokens: the workspace is not used
    (dict(ws=0x500000, dgain=None, dnext=None), False),
    # without dxn, out and next_gain are not read
    (dict(dxn=None, dnext=None, out=0x800000), False)])
def test_residual_norm_grad_overlaps(lib, kw, hit):
    rc = norm_grad(lib, **kw)
    assert rc != 0 and overlaps(lib, rc) == hit


def test_residual_norm_grad_workspace_sizes(lib):
    ws = lib.moe_residual_norm_grad_workspace
    assert ws(0, 64) == 0 and ws(4, 60) == 0 and ws(4, 16392) == 0
    assert ws(4, 64) == 4 * 64 * 8 and ws(1 << 26, 8) > ws(4096, 8) > 0


# ---------------------------------------------------------------- adapters

AD = dict(x=0x100000, ldx=64, dtype=1, n=8, K=64, N=48, ids=0x10000, L=3, r=16, A=0x200000,
          B=0x300000, scale=0x20000, base=0x400000, ldb=48, out=0x500000, ldo=48, h=0x600000,
          ws=0x700000, ws_bytes=None)


def adapters(lib, **kw):
    a = dict(AD, **kw)
    size = a["ws_bytes"]
    if size is None:
        size = lib.moe_adapter_workspace(a["n"], a["L"], a["r"], a["K"], a["N"])
    return lib.moe_adapter(P(a["x"]), L(a["ldx"]), a["dtype"], a["n"], a["K"], a["N"], P(a["ids"]),
                           a["L"], a["r"], P(a["A"]), P(a["B"]), P(a["scale"]), P(a["base"]),
                           L(a["ldb"]), P(a["out"]), L(a["ldo"]), P(a["h"]), P(a["ws"]), Z(size),
                           None)


def adapters_grad(lib, **kw):
    a = dict(AD, dy=0x800000, lddy=48, ldb=64, dx=0x500000, lddx=64, dA=0x900000, dB=0xA00000)
    a.update(kw)
    size = a["ws_bytes"]
    if size is None:
        size = lib.moe_adapter_workspace(a["n"], a["L"], a["r"], a["K"], a["N"])
    return lib.moe_adapter_grad(P(a["dy"]), L(a["lddy"]), P(a["x"]), L(a["ldx"]), P(a["h"]),
                                a["dtype"], a["n"], a["K"], a["N"], P(a["ids"]), a["L"], a["r"],
                                P(a["A"]), P(a["B"]), P(a["scale"]), P(a["base"]), L(a["ldb"]),
                                P(a["dx"]), L(a["lddx"]), P(a["dA"]), P(a["dB"]), P(a["ws"]),
                                Z(size), None)


AD_BOTH = [(dict(x=None), -1), (dict(ids=None), -1), (dict(A=None), -1), (dict(B=None), -1),
           (dict(ws=None), -1), (dict(dtype=2), -2), (dict(n=0), -1), (dict(n=(1 << 20) + 1), -1),
           (dict(L=0), -1), (dict(L=1025), -1), (dict(r=0), -1), (dict(r=12), -1), (dict(r=136), -1),
           (dict(K=0), -1), (dict(N=0), -1), (dict(K=(1 << 20) + 1, ldx=1 << 21), -1),
           (dict(N=(1 << 20) + 1), -1), (dict(ldx=63), -1), (dict(x=0x100001), -1),
           (dict(ids=0x10002), -1), (dict(A=0x200008), -1), (dict(B=0x300002), -1),
           (dict(scale=0x20002), -1), (dict(ldb=40), -1), (dict(ws=0x700010), -1),
           (dict(ws_bytes=100), -1), (dict(ldb=(1 << 31) + 1), -1)]


@pytest.mark.parametrize("kw,code", AD_BOTH + [
    (dict(out=None), -1), (dict(out=0x500001), -1), (dict(ldo=47), -1), (dict(h=0x600001), -1)])
def test_adapter_refuses(lib, kw, code):
    assert refused(lib, adapters(lib, **kw), code)


@pytest.mark.parametrize("kw,code", AD_BOTH + [
    (dict(dy=None), -1), (dict(h=None), -1), (dict(dx=None, dA=None, dB=None), -1),
    (dict(h=0x600008), -1), (dict(dA=0x900008), -1), (dict(dB=0xA00002), -1), (dict(lddy=47), -1),
    (dict(lddx=63), -1), (dict(dy=0x800001), -1)])
def test_adapter_grad_refuses(lib, kw, code):
    assert refused(lib, adapters_grad(lib, **kw), code)


@pytest.mark.parametrize("kw,hit", [
    (dict(), False), (dict(out=0x400000), False), (dict(out=0x400000, ldo=64), True),
    (dict(out=0x400002), True), (dict(out=0x100000), True), (dict(out=0x200000), True),
    (dict(out=0x300000 + 3 * 16 * 48 * 2), False), (dict(out=0x300000 + 3 * 16 * 48 * 2 - 2), True),
    (dict(h=0x100000), True), (dict(h=0x10000), True), (dict(h=None), False),
    (dict(ws=0x100000), True), (dict(ws=0x10000), True), (dict(out=0x400000, n=1), False)])
def test_adapter_overlaps(lib, kw, hit):
    rc = adapters(lib, **kw)
    assert rc != 0 and overlaps(lib, rc) == hit


@pytest.mark.parametrize("kw,hit", [
    (dict(), False), (dict(dx=0x400000), False), (dict(dx=0x100000), True),
    (dict(dx=0x100000, dA=None, x=None), False), (dict(dA=0x200000), True), (dict(dB=0x900010), True),
    (dict(dB=0x600000), True), (dict(h=None, dB=None, dA=0x600000), False),
    # base is read for dx only
    (dict(dx=None, dA=0x400000), False), (dict(ws=0x800000), True)])
def test_adapter_grad_overlaps(lib, kw, hit):
    rc = adapters_grad(lib, **kw)
    assert rc != 0 and overlaps(lib, rc) == hit


def test_adapter_workspace_sizes(lib):
    ws = lib.moe_adapter_workspace
    for bad in ((0, 1, 8, 8, 8), (1, 0, 8, 8, 8), (1, 1, 4, 8, 8), (1, 1, 8, 0, 8), (1, 1, 8, 8, 0),
                (1, 1025, 8, 8, 8), (1, 1, 136, 8, 8), (1 << 21, 1, 8, 8, 8)):
        assert ws(*bad) == 0
    assert ws(1, 1, 8, 8, 8) > 0 and ws(64, 4, 16, 8, 65536) == ws(64, 4, 16, 65536, 8)
    assert ws(64, 4, 16, 65536, 8) >= ws(64, 4, 16, 8, 8)


# ---------------------------------------------------------------- the binding

def test_binding_refuses_wrong_tensors():
    from quantized_expert_ffn_warp_gb300 import moe
    logits, t = torch.zeros((4, 10)), torch.zeros(4, dtype=torch.int32)
    x = torch.zeros((4, 64), dtype=torch.float16)
    fwd = dict(stats=torch.zeros((4, 2)), entropy=torch.zeros(4))
    w = torch.zeros((2, 8, 64), dtype=torch.float16)
    for call in (lambda: moe.token_logprobs(logits, t),                 # no GPU tensors
                 lambda: moe.token_logprobs(logits[0], t),
                 lambda: moe.token_logprobs(logits.double(), t),
                 lambda: moe.token_logprobs(logits, t.long()),
                 lambda: moe.token_logprobs(logits, t[:3]),
                 lambda: moe.token_logprobs(logits, t, top=-1),
                 lambda: moe.token_logprobs(logits.t(), t),
                 lambda: moe.token_logprobs_grad(logits, None, fwd, torch.zeros(4)),
                 lambda: moe.token_logprobs_grad(logits, t, fwd, torch.zeros(3)),
                 lambda: moe.token_logprobs_grad(logits, t, fwd, torch.zeros(4).half()),
                 lambda: moe.residual_norm(x, x),
                 lambda: moe.residual_norm(x, x[:, :32]),
                 lambda: moe.residual_norm(x, x, gate=torch.zeros(4, dtype=torch.float16)),
                 lambda: moe.residual_norm(x, x, gate=torch.zeros((4, 2), dtype=torch.float16)),
                 lambda: moe.residual_norm(x, x, gain=torch.zeros(64)),
                 lambda: moe.residual_norm_grad(x, x, x, x, torch.zeros((4, 2))),
                 lambda: moe.residual_norm_grad(x, None, None, x, torch.zeros((4, 1))),
                 lambda: moe.adapter(x, t, w, w.transpose(1, 2).contiguous()),
                 lambda: moe.adapter(x, t, w[0], w),
                 lambda: moe.adapter(x, t.long(), w, w.transpose(1, 2).contiguous()),
                 lambda: moe.adapter(x, t, w.float(), w.transpose(1, 2).contiguous()),
                 lambda: moe.adapter(x, t, w, w.transpose(1, 2)),
                 lambda: moe.adapter_grad(x, x, x, t, w, w.transpose(1, 2).contiguous()),
                 lambda: moe.adapter_grad(x, x[:, :32], x[:, :8].contiguous(), t, w,
                                          w.transpose(1, 2).contiguous())):
        with pytest.raises(moe.MoeError):
            call()


# ---------------------------------------------------------------- gradients by differences

def differences(f, x, step=1e-5):
    """Central differences of the number f(x) in every entry of x."""
    g = torch.zeros_like(x)
    for i in range(x.numel()):
        d = torch.zeros_like(x).view(-1)
        d[i] = step
        d = d.view_as(x)
        g.view(-1)[i] = (f(x + d) - f(x - d)) / (2 * step)
    return g


def test_logprobs_gradient_against_differences():
    torch.manual_seed(1)
    l = torch.randn((4, 6), dtype=torch.float64)
    targets = torch.tensor([0, 5, -1, 3])
    wl, we = torch.randn(4, dtype=torch.float64), torch.randn(4, dtype=torch.float64)

    def loss(x):
        r = logprobs(x, targets)
        return (wl * r["logp"]).sum() + (we * r["entropy"]).sum()
    want = differences(loss, l)
    got, _ = logprobs_grad(l, targets, logprobs(l, targets), wl, we)
    # central differences: a third derivative of order 1 times step^2, 2^-53 / step
    assert (got - want).abs().max() < 1e-8


@pytest.mark.parametrize("gate", [(3, 1), (8,), None])
@pytest.mark.parametrize("gain", [True, False])
def test_residual_norm_gradients_against_differences(gate, gain):
    torch.manual_seed(2)
    f = torch.float64
    x = dict(resid=torch.randn((3, 8), dtype=f), y=torch.randn((3, 8), dtype=f),
             gain=torch.rand(8, dtype=f) + 0.5 if gain else None,
             gate=torch.rand(gate, dtype=f) if gate else None,
             next_gain=torch.rand(8, dtype=f) + 0.5)
    wo, wx = torch.randn((3, 8), dtype=f), torch.randn((3, 8), dtype=f)

    def forward(**kw):
        a = dict(x, **kw)
        return residual_norm(a["resid"], a["y"], a["gain"], a["gate"], 0.75, a["next_gain"], 1e-3)
    r = forward()
    got, _ = residual_norm_grad(wo, wx, r["out"], x["y"], r["stats"], x["gain"], x["gate"], 0.75,
                                x["next_gain"])
    for name, g in got.items():
        def loss(v):
            q = forward(**{name[1:]: v})
            return (wo * q["out"]).sum() + (wx * q["xn"]).sum()
        assert (g - differences(loss, x[name[1:]])).abs().max() < 1e-7, name


@pytest.mark.parametrize("scaled", [True, False])
def test_adapter_gradients_against_differences(scaled):
    torch.manual_seed(3)
    f = torch.float64
    import tuning_refs
    tuning_refs.PAIR[f], tuning_refs.TINY[f] = 0.0, 0.0
    ids = torch.tensor([1, 0, -1, 1, 5])
    x = dict(x=torch.randn((5, 6), dtype=f), A=torch.randn((3, 2, 6), dtype=f),
             B=torch.randn((3, 4, 2), dtype=f), base=torch.randn((5, 4), dtype=f))
    scale = torch.rand(3, dtype=f) if scaled else None
    wo = torch.randn((5, 4), dtype=f)

    def forward(**kw):
        a = dict(x, **kw)
        return adapter(a["x"], ids, a["A"], a["B"], scale, a["base"])
    h = forward()[1][0]
    got = adapter_grad(wo, x["x"], h, ids, x["A"], x["B"], scale, None)
    for name, (g, _) in got.items():
        def loss(v):
            return (wo * forward(**{name[1:]: v})[0][0]).sum()
        # the loss is of second order in each argument: differences are off by roundings
        assert (g - differences(loss, x[name[1:]], 1e-3)).abs().max() < 1e-9, name
