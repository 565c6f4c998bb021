"""A tuning step of a frozen 4-bit block with adapters, and a decode step, through the
library's calls as they are used together: norm, 4-bit products with the adapters of
several requests, gated residual with the next norm, vocabulary head, log
probabilities, and back.

The step is checked against automatic differentiation of the same model in 64 bits.
Between the loss and any gradient lie about twenty tensors of fp16, each rounded by half
a step (2^-11 relative) of unstructured error, which the norms and random matrices
behind it pass on at most doubled in the 2-norm: 20 * 2 * 2^-11.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
TOL = 20 * 2 * 2.0 ** -11
HID, INNER, VOCAB, RANK, COUNT, SCALE, EPS = 256, 512, 1003, 16, 3, 0.9, 1e-5


def _moe():
    from quantized_expert_ffn_warp_gb300 import moe
    return moe


def matrix(rows, cols, g):
    codes = torch.randint(0, 256, (rows, cols // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = ((torch.rand((rows, cols // 128), device="cuda", generator=g) + 0.5)
              * 0.2 / cols ** 0.5).half()
    zeros = torch.randint(6, 10, (rows, cols // 128), dtype=torch.uint8, device="cuda", generator=g)
    return codes, scales, zeros


def dense(w):
    q = torch.stack((w[0] & 15, w[0] >> 4), 2).flatten(1).double()
    return (q - w[2].double().repeat_interleave(128, 1)) * w[1].double().repeat_interleave(128, 1)


def model(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*s, scale=1.0):
        return (torch.randn(s, device="cuda", generator=g) * scale).half()
    reqs = torch.sort(torch.randint(-1, COUNT, (n,), device="cuda", generator=g)).values
    p = dict(resid=randn(n, HID), y=randn(n, HID, scale=0.5),
             up=matrix(INNER, HID, g), down=matrix(HID, INNER, g), head=matrix(VOCAB, HID, g),
             A1=randn(COUNT, RANK, HID, scale=HID ** -0.5), B1=randn(COUNT, INNER, RANK, scale=0.1),
             A2=randn(COUNT, RANK, INNER, scale=INNER ** -0.5), B2=randn(COUNT, HID, RANK, scale=0.1),
             g0=randn(HID, scale=0.2) + 1, g1=randn(HID, scale=0.2) + 1, g2=randn(HID, scale=0.2) + 1,
             g3=randn(HID, scale=0.2) + 1, gate=torch.sigmoid(randn(n, 1).float()).half(),
             gate2=torch.rand(HID, device="cuda", generator=g).half(),
             ids=reqs.to(torch.int32).contiguous(),
             scale=torch.rand(COUNT, device="cuda", generator=g) + 0.5,
             targets=torch.randint(-1, VOCAB, (n,), device="cuda", generator=g).to(torch.int32))
    p["weight"] = torch.rand(n, device="cuda", generator=g) / n
    return p


def forward(p, stream=None, top=0):
    moe = _moe()
    s = dict(stream=stream)
    a = moe.residual_norm(p["resid"], p["y"], gain=p["g0"], gate=p["gate"], scale=SCALE,
                          next_gain=p["g1"], eps=EPS, **s)
    up = moe.linear(a["xn"], *p["up"], **s)
    up, h1 = moe.adapter(a["xn"], p["ids"], p["A1"], p["B1"], p["scale"], base=up, out=up, **s)
    y = moe.linear(up, *p["down"], **s)
    y, h2 = moe.adapter(up, p["ids"], p["A2"], p["B2"], p["scale"], base=y, out=y, **s)
    b = moe.residual_norm(a["out"], y, gain=p["g2"], gate=p["gate2"], scale=SCALE,
                          next_gain=p["g3"], eps=EPS, **s)
    logits = moe.linear(b["xn"], *p["head"], **s)
    lp = moe.token_logprobs(logits, p["targets"], top=top, **s)
    return dict(a=a, up=up, h1=h1, y=y, h2=h2, b=b, logits=logits, lp=lp)


def backward(p, f, stream=None):
    moe = _moe()
    s = dict(stream=stream)
    dl = moe.token_logprobs_grad(f["logits"], p["targets"], f["lp"], -p["weight"], 0.01 * p["weight"],
                                 out=f["logits"], **s)
    dxn = moe.linear_input_grad(dl, *p["head"], **s)
    gb = moe.residual_norm_grad(None, dxn, f["b"]["out"], f["y"], f["b"]["stats"], gain=p["g2"],
                                gate=p["gate2"], scale=SCALE, next_gain=p["g3"], **s)
    dup = moe.linear_input_grad(gb["dy"], *p["down"], **s)
    g2 = moe.adapter_grad(gb["dy"], f["up"], f["h2"], p["ids"], p["A2"], p["B2"], p["scale"],
                          base=dup, out=dup, **s)
    dx = moe.linear_input_grad(dup, *p["up"], **s)
    g1 = moe.adapter_grad(dup, f["a"]["xn"], f["h1"], p["ids"], p["A1"], p["B1"], p["scale"],
                          base=dx, out=dx, **s)
    ga = moe.residual_norm_grad(gb["dresid"], dx, f["a"]["out"], p["y"], f["a"]["stats"],
                                gain=p["g0"], gate=p["gate"], scale=SCALE, next_gain=p["g1"], **s)
    return dict(A1=g1["dA"], B1=g1["dB"], A2=g2["dA"], B2=g2["dB"], g0=ga["dgain"],
                gate=ga["dgate"], g1=ga["dnext_gain"], g2=gb["dgain"], gate2=gb["dgate"],
                g3=gb["dnext_gain"], resid=ga["dresid"], y=ga["dy"])


def reference(p, names):
    """(loss terms, gradients) of the model in 64 bits by automatic differentiation."""
    v = {k: p[k].double().requires_grad_(True) for k in names}

    def rms(x):
        return x * (x.square().mean(1, keepdim=True) + EPS).rsqrt()

    def adapt(x, y, A, B):
        hot = torch.stack([(p["ids"] == a).double() * p["scale"][a].double() for a in range(COUNT)], 1)
        h = torch.einsum("tk,ark->tar", x, A)
        return y + torch.einsum("tar,ajr,ta->tj", h, B, hot)
    out = SCALE * v["resid"] + v["gate"] * v["g0"] * rms(v["y"])
    xn = v["g1"] * rms(out)
    up = adapt(xn, xn @ dense(p["up"]).t(), v["A1"], v["B1"])
    y = adapt(up, up @ dense(p["down"]).t(), v["A2"], v["B2"])
    out2 = SCALE * out + v["gate2"] * v["g2"] * rms(y)
    logits = (v["g3"] * rms(out2)) @ dense(p["head"]).t()
    lp = torch.log_softmax(logits, 1)
    on = p["targets"] >= 0
    given = lp.gather(1, p["targets"].clamp(min=0).long()[:, None])[:, 0] * on
    ent = -(lp.exp() * lp).sum(1)
    w = p["weight"].double()
    (-(w * given).sum() + 0.01 * (w * ent).sum()).backward()
    return given.detach(), ent.detach(), {k: t.grad for k, t in v.items()}


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("n", [5, 150, 700])
def test_tuning_step_against_automatic_differentiation(n):
    p = model(n, n)
    f = forward(p)
    lp, ent = f["lp"]["logp"], f["lp"]["entropy"]
    got = backward(p, f)
    given, entropy, want = reference(p, list(got))
    assert rel(lp, given) <= TOL and rel(ent, entropy) <= TOL
    for k, w in want.items():
        assert got[k].shape == w.shape
        assert rel(got[k], w) <= TOL, (k, rel(got[k], w))


def test_tuning_step_in_a_graph_on_another_stream():
    """The step captured once and replayed on other inputs gives the eager bits, beside
    the same step run eagerly on another stream."""
    p, q = model(300, 1), model(300, 2)
    live = {k: (v.clone() if torch.is_tensor(v) else v) for k, v in p.items()}
    backward(live, forward(live))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = backward(live, forward(live))
    side = torch.cuda.Stream()
    for src in (q, p):
        for k in ("resid", "y", "gate", "ids", "targets", "weight", "A1", "B2"):
            live[k].copy_(src[k])
        torch.cuda.synchronize()
        g.replay()
        eager = {k: (live[k] if k in ("resid", "y", "gate", "ids", "targets", "weight", "A1", "B2")
                     else p[k]) for k in p}
        want = backward(eager, forward(eager, side), side)
        side.synchronize()
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(res[k], want[k]), k


@pytest.mark.parametrize("n", [1, 4, 13])
def test_decode_step(n):
    """Single tokens of several requests: alternatives and log probabilities agree with
    the logits, and a token's result does not depend on its neighbours' adapters."""
    p = model(n, 30 + n)
    f = forward(p, top=5)
    l = f["logits"].double()
    lp = torch.log_softmax(l, 1)
    order = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :5]
    assert torch.equal(f["lp"]["top_ids"].long(), order)
    assert (f["lp"]["top_logp"].double() - lp.gather(1, order)).abs().max() <= 1e-4
    if n > 1:
        other = dict(p, ids=p["ids"].clone())
        other["ids"][1:] = (other["ids"][1:] + 1) % COUNT
        g = forward(other, top=5)
        assert torch.equal(g["logits"][0], f["logits"][0])
