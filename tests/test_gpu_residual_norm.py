"""Block norms and their gradients against 64-bit definitions; the bounds are
derived in tuning_refs.py."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from tuning_refs import DT, H, half_step, residual_norm, residual_norm_grad  # noqa: E402

EPS = 1e-6


def _moe():
    from quantized_expert_ffn_warp_gb300 import moe
    return moe


def batch(n, hid, dtype, seed, gate="token", gain=True, next_gain=True, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[dtype]

    def rows(scale):
        wide = torch.randn((n, hid + pad), device="cuda", generator=g) * scale
        return wide.to(dt)[:, :hid]
    shape = {"token": (n, 1), "channel": (hid,), None: None}[gate]
    ga = None if shape is None else torch.randn(shape, device="cuda", generator=g).to(dt)

    def vector():
        return (torch.rand(hid, device="cuda", generator=g) + 0.5).to(dt)
    return dict(resid=rows(2.0), y=rows(0.5), gain=vector() if gain else None, gate=ga,
                next_gain=vector() if next_gain else None), rows


def check_forward(a, scale, got=None, eps=EPS):
    moe = _moe()
    got = moe.residual_norm(**a, scale=scale, eps=eps) if got is None else got
    ref = residual_norm(a["resid"], a["y"], a["gain"], a["gate"], scale, a["next_gain"], eps)
    dt = a["y"].dtype
    assert ((got["out"].double() - ref["out"]).abs()
            <= ref["out_err"] + half_step(ref["out"], dt)).all()
    assert ((got["stats"][:, 0].double() - ref["stats"][:, 0]).abs()
            <= 24 * H * ref["stats"][:, 0]).all()
    if a["next_gain"] is None:
        assert "xn" not in got and (got["stats"][:, 1] == 1).all()
    else:
        assert ((got["xn"].double() - ref["xn"]).abs()
                <= ref["xn_err"] + half_step(ref["xn"], dt)).all()
        assert ((got["stats"][:, 1:].double() - ref["stats"][:, 1:]).abs() <= ref["r2_err"]).all()
    return got


def check_grad(a, fwd, dout, dxn, scale):
    moe = _moe()
    kw = dict(gain=a["gain"], gate=a["gate"], scale=scale, next_gain=a["next_gain"])
    got = moe.residual_norm_grad(dout, dxn, fwd["out"], a["y"], fwd["stats"], **kw)
    want, err = residual_norm_grad(dout, dxn, fwd["out"], a["y"], fwd["stats"], a["gain"],
                                   a["gate"], scale, a["next_gain"])
    assert got.keys() == want.keys()
    for k, w in want.items():
        assert got[k].shape == w.shape
        step = half_step(w, got[k].dtype) if got[k].dtype is not torch.float32 else H * w.abs()
        assert ((got[k].double() - w).abs() <= err[k] + step).all(), k
    return got


SHAPES = [(1, 8), (3, 16), (7, 264), (1, 4096), (2, 8192), (5, 8200), (3, 16384), (1000, 640),
          (77, 2048), (2000, 4096), (130000, 8)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n,hid", SHAPES)
@pytest.mark.parametrize("gate,gain,next_gain", [
    ("token", True, True), ("channel", True, True), (None, True, True), ("token", False, True),
    ("channel", False, False), (None, False, True), ("token", True, False), (None, False, False)])
def test_forward_and_gradient(n, hid, dtype, gate, gain, next_gain):
    a, rows = batch(n, hid, dtype, n + hid, gate, gain, next_gain)
    fwd = check_forward(a, 0.75)
    check_grad(a, fwd, rows(0.02), rows(0.02) if next_gain else None, 0.75)
    if next_gain:
        check_grad(a, fwd, None, rows(0.02), 0.75)
        check_grad(a, fwd, rows(1.0), None, 0.75)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n,hid", [(200, 8200), (1000, 12296), (305, 16384), (20000, 8200)])
def test_gradient_of_wide_rows(n, hid, dtype):
    """Many rows of two blocks each, with one sum a row and with two, on two streams."""
    moe = _moe()
    a, rows = batch(n, hid, dtype, n, "channel", pad=8)
    fwd = check_forward(a, 0.75)
    dout, dxn = rows(0.02), rows(0.02)
    got = check_grad(a, fwd, dout, dxn, 0.75)
    check_grad(a, fwd, dout, None, 0.75)
    kw = dict(gain=a["gain"], gate=a["gate"], scale=0.75, next_gain=a["next_gain"])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    again = [moe.residual_norm_grad(dout, dxn, fwd["out"], a["y"], fwd["stats"], **kw, stream=s)
             for _ in range(3) for s in streams]
    torch.cuda.synchronize()
    for r in again:
        for k, v in got.items():
            assert torch.equal(r[k], v), k


@pytest.mark.parametrize("n,hid,pad", [(5, 520, 8), (33, 1024, 1032), (1, 64, 64)])
def test_strided_rows_and_in_place(n, hid, pad):
    moe = _moe()
    a, rows = batch(n, hid, "bf16", 5, pad=pad)
    fwd = check_forward(a, 1.0)
    dout, dxn = rows(0.02), rows(0.02)
    check_grad(a, fwd, dout, dxn, 1.0)
    again = moe.residual_norm(**a, eps=EPS, out=a["resid"])
    assert again["out"] is a["resid"] and torch.equal(a["resid"], fwd["out"])
    assert torch.equal(again["xn"], fwd["xn"]) and torch.equal(again["stats"], fwd["stats"])


@pytest.mark.parametrize("n", [1, 3, 700])
def test_gradient_in_place_of_dout(n):
    """dresid written over dout, through the C call."""
    moe = _moe()
    a, rows = batch(n, 512, "fp16", 8)
    fwd = moe.residual_norm(**a, eps=EPS)
    dout, dxn = rows(0.02), rows(0.02)
    kw = dict(gain=a["gain"], gate=a["gate"], next_gain=a["next_gain"])
    want = moe.residual_norm_grad(dout, dxn, fwd["out"], a["y"], fwd["stats"], **kw)
    dy, dg = torch.empty_like(dout), torch.empty((n, 1), device="cuda")
    p = [t.data_ptr() for t in (dout, dxn, fwd["out"], a["y"])]
    rc = moe.load_library().moe_residual_norm_grad(
        p[0], 512, p[1], 512, p[2], 512, p[3], 512, fwd["stats"].data_ptr(), moe.MOE_FP16, n, 512,
        a["gain"].data_ptr(), a["gate"].data_ptr(), 1, 1.0, a["next_gain"].data_ptr(), p[0], 512,
        dy.data_ptr(), 512, None, dg.data_ptr(), None, None, 0,
        torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    assert torch.equal(dout, want["dresid"]) and torch.equal(dy, want["dy"])
    assert torch.equal(dg, want["dgate"])


@pytest.mark.parametrize("eps", [0.0, 1e-6, 4.0])
def test_zero_and_large_rows(eps):
    moe = _moe()
    a, rows = batch(6, 256, "bf16", 5)
    a["y"][0] = 0
    a["y"][1] *= 1e15
    a["resid"][2] *= 1e15
    a["resid"][3] = 0
    a["y"][3] = 0
    if eps:
        fwd = check_forward(a, 1.0, eps=eps)
        assert (fwd["xn"][3] == 0).all() and (fwd["out"][3] == 0).all()
        return
    got = moe.residual_norm(**a, eps=0.0)       # 0 / 0 is a NaN of its row alone
    assert torch.isnan(got["xn"][3]).all() and torch.isnan(got["out"][0]).all()
    assert torch.isfinite(got["xn"][[1, 2, 4, 5]]).all()


def test_values_that_are_not_finite_stay_in_their_row():
    moe = _moe()
    a, rows = batch(5, 1024, "fp16", 6)
    a["y"][1, 3] = float("nan")
    a["resid"][3, 1000] = float("inf")
    fwd = moe.residual_norm(**a, eps=EPS)
    assert torch.isnan(fwd["xn"][1]).all() and torch.isfinite(fwd["xn"][[0, 2, 4]]).all()
    assert fwd["out"][3, 1000] == float("inf")
    g = moe.residual_norm_grad(rows(0.02), rows(0.02), fwd["out"], a["y"], fwd["stats"],
                               gain=a["gain"], gate=a["gate"], next_gain=a["next_gain"])
    assert torch.isfinite(g["dy"][[0, 2, 4]]).all() and torch.isnan(g["dy"][1]).all()


def test_same_bits_on_other_streams_and_in_graphs():
    moe = _moe()
    n, hid = 900, 1280
    a, rows = batch(n, hid, "bf16", 7, gate="channel")
    dout, dxn = rows(0.02), rows(0.02)
    kw = dict(gain=a["gain"], gate=a["gate"], next_gain=a["next_gain"])

    def both(y, stream=None):
        f = moe.residual_norm(a["resid"], y, **kw, stream=stream)
        return f, moe.residual_norm_grad(dout, dxn, f["out"], y, f["stats"], **kw, stream=stream)

    def equal(x, y):
        return all(torch.equal(x[i][k], y[i][k]) for i in range(2) for k in x[i])
    first = both(a["y"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    again = both(a["y"], side)
    side.synchronize()
    assert equal(first, again)
    static, pool = a["y"].clone(), torch.cuda.graph_pool_handle()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            res = both(static)
        graphs.append((g, res))
    for turn in range(4):
        static.copy_(batch(n, hid, "bf16", 20 + turn)[0]["y"])
        g, res = graphs[turn % 2]
        g.replay()
        torch.cuda.synchronize()
        assert equal(res, both(static))


def test_offsets_beyond_32_bits():
    moe = _moe()
    n, hid = 140000, 16384
    a, _ = batch(8, hid, "bf16", 3)
    resid = torch.zeros((n, hid), dtype=torch.bfloat16, device="cuda")
    y = torch.zeros_like(resid)
    resid[-8:], y[-8:] = a["resid"], a["y"]
    kw = dict(gain=a["gain"], next_gain=a["next_gain"])
    small = moe.residual_norm(a["resid"], a["y"], **kw)
    big = moe.residual_norm(resid, y, **kw, out=resid)
    assert torch.equal(big["xn"][-8:], small["xn"]) and torch.equal(big["out"][-8:], small["out"])
    assert (big["xn"][:-8] == 0).all()


def test_refusals():
    moe = _moe()
    a, rows = batch(4, 64, "bf16", 1)
    for bad in (dict(gate=a["gate"][:, 0]), dict(y=a["y"].half()), dict(gain=a["gain"][:32]),
                dict(resid=a["resid"].cpu()), dict(out=a["y"]), dict(eps=-1.0),
                dict(scale=float("inf"))):
        with pytest.raises(moe.MoeError):
            moe.residual_norm(**dict(a, **bad))
    odd = torch.zeros((4, 68), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(moe.MoeError):
        moe.residual_norm(odd[:, 4:], a["y"])
    with pytest.raises(moe.MoeError):
        moe.residual_norm(odd[:, :60].contiguous(), odd[:, :60].contiguous())
