"""Routing losses and their gradient against a 64-bit evaluation.

Tolerances (h = 2^-24, half an fp32 step): exp of a rounded difference d has a
relative error of at most (|d| + 4) h, with |d| below 100 wherever the result
matters; a sum of N terms in any order at most N h of the sum of magnitudes;
16-bit outputs add half a step of their type.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
H = 2.0 ** -24
INF = float("inf")


def _moe():
    from quantized_expert_ffn_warp_gb300 import moe
    return moe


def batch(n, E, k, seed, dtype=torch.float32, spread=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = (spread * torch.randn((n, E), device="cuda", generator=g)).to(dtype)
    idx = torch.topk(logits.float(), k, dim=1).indices.to(torch.int32).contiguous()
    sel = torch.gather(logits.float(), 1, idx.long())
    w = torch.softmax(sel, 1).contiguous()
    return logits, idx, w


def tensors(seq, mask, n):
    s = None if seq is None else torch.tensor(seq, dtype=torch.int32, device="cuda")
    m = None
    if mask is not None:
        g = torch.Generator(device="cuda").manual_seed(77)
        m = (torch.rand(n, device="cuda", generator=g) < mask).to(torch.uint8)
    return s, m


def reference(logits, idx, seq, mask):
    """dict as balance_loss gives it, in 64 bits, by the definition."""
    n, E = logits.shape
    k = idx.shape[1]
    seq = [0, n] if seq is None else seq.tolist()
    S = len(seq) - 1
    live = torch.zeros(n, dtype=torch.bool, device="cuda")
    for s in range(S):
        live[seq[s]:seq[s + 1]] = True
    if mask is not None:
        live &= mask != 0
    l = logits.double()
    lse = torch.where(live, torch.logsumexp(l, 1), 0.0)
    p = torch.where(live[:, None], torch.softmax(l, 1), 0.0)
    empty = live & (l == -INF).all(1)
    p[empty] = 0
    counts = torch.zeros((S, E), dtype=torch.int64)
    prob = torch.zeros((S, E), dtype=torch.float64, device="cuda")
    tokens, bal, parts = [], 0.0, 0
    for s in range(S):
        r = slice(seq[s], seq[s + 1])
        T = int(live[r].sum())
        tokens.append(T)
        ids = idx[r][live[r]].reshape(-1)
        ids = ids[(ids >= 0) & (ids < E)].long().cpu()
        counts[s] = torch.bincount(ids, minlength=E)
        if T:
            parts += 1
            prob[s] = p[r].sum(0) / T
            bal = bal + (counts[s].cuda().double() * E / (k * T) * prob[s]).sum()
    ltot = torch.where(empty, 0.0, lse)
    z = (ltot ** 2).sum() / max(sum(tokens), 1)
    bal = torch.as_tensor(bal, dtype=torch.float64, device="cuda") / max(parts, 1)
    return dict(loss=torch.stack((bal, z)), counts=counts.int().cuda(), prob=prob, lse=lse,
                tokens=torch.tensor(tokens, dtype=torch.int32, device="cuda"), p=p, live=live,
                parts=parts, empty=empty)


def reference_grad(logits, idx, ref, dloss, w, dw, seq):
    n, E = logits.shape
    k = idx.shape[1]
    seq = [0, n] if seq is None else seq.tolist()
    f, gs = torch.zeros((n, E), device="cuda").double(), torch.zeros(n, device="cuda").double()
    for s in range(len(seq) - 1):
        T = int(ref["tokens"][s])
        if T:
            f[seq[s]:seq[s + 1]] = ref["counts"][s].double() * E / (k * T)
            gs[seq[s]:seq[s + 1]] = dloss[0].double() / (ref["parts"] * T)
    p, lse = ref["p"], torch.where(ref["empty"], 0.0, ref["lse"])
    total = max(int(ref["tokens"].sum()), 1)
    dot = (f * p).sum(1, keepdim=True)
    zt = (2 * dloss[1].double() * lse / total)[:, None]
    g = p * ((f - dot) * gs[:, None] + zt)
    size = p * ((f + dot) * gs[:, None].abs() + zt.abs())
    if dw is not None:
        w, dw = w.double(), dw.double()
        d = w * (dw - (w * dw).sum(1, keepdim=True))
        dm = w * (dw.abs() + (w * dw.abs()).sum(1, keepdim=True))
        ok = (idx >= 0) & (idx < E) & ref["live"][:, None]
        at = torch.where(ok, idx, 0).long()
        g = g.scatter_add(1, at, torch.where(ok, d, 0.0))
        size = size.scatter_add(1, at, torch.where(ok, dm, 0.0))
    return g, size


def check_forward(got, ref, n, E):
    assert torch.equal(got["counts"], ref["counts"]) and torch.equal(got["tokens"], ref["tokens"])
    fin = torch.isfinite(ref["lse"])
    assert torch.equal(got["lse"][~fin].double(), ref["lse"][~fin])
    le, lg = ref["lse"][fin], got["lse"][fin].double()
    assert ((lg - le).abs() <= (104 + E) * H + 2 * H * le.abs()).all()
    terms = 104 + E + n
    assert ((got["prob"].double() - ref["prob"]).abs() <= terms * H * ref["prob"] + 1e-38).all()
    a, b = got["loss"].double(), ref["loss"]
    # a loss is a sum of non-negative terms; lse^2 doubles lse's relative error,
    # which cancellation near lse = 0 can raise: its absolute error enters
    lm = torch.where(fin, ref["lse"], 0.0).abs().max()
    assert (a[0] - b[0]).abs() <= (terms + 8) * H * b[0] + 1e-38
    assert (a[1] - b[1]).abs() <= (n + 16) * H * b[1] + 3 * lm * (104 + E + 2 * lm) * H


def check_grad(got, ref, size, E, dtype):
    err = (got.double() - ref).abs()
    tol = (2 * (104 + E) + 200) * H * size + 1e-38
    if dtype != torch.float32:
        tol = tol + torch.finfo(dtype).eps / 2 * ref.abs() + torch.finfo(dtype).smallest_normal * \
            torch.finfo(dtype).eps
    assert (err <= tol).all(), (err / tol).max()


CASES = [
    # n, E, k, offsets, share of tokens kept by the mask
    (1, 1, 1, None, None), (1, 8, 2, None, None), (7, 33, 32, None, None), (64, 64, 2, None, None),
    (5, 100, 3, [0, 0, 2, 2, 5, 5], None), (1000, 256, 8, [0, 999, 1000], 0.9),
    (777, 500, 4, [3, 3, 10, 500, 700], 0.5), (300, 1024, 8, None, 0.97),
    (130, 130, 5, [0, 130], 0.0), (3000, 16, 2, list(range(0, 3001, 30)), 0.8),
    (20000, 64, 6, [0, 1, 15000, 15000, 20000], None), (9, 3, 1, [9, 9], None),
]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("n,E,k,seq,keep", CASES)
def test_losses_and_gradient(n, E, k, seq, keep, dtype):
    moe = _moe()
    logits, idx, w = batch(n, E, k, n + E, DT[dtype])
    s, m = tensors(seq, keep, n)
    got = moe.balance_loss(logits, idx, s, m)
    ref = reference(logits, idx, s, m)
    check_forward(got, ref, n, E)
    dloss = torch.tensor([0.7, -0.3], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    dw = torch.randn((n, k), device="cuda", generator=g)
    for d in (None, dw):
        out = moe.balance_loss_grad(logits, idx, got, dloss, w, d, s, m)
        rg, size = reference_grad(logits, idx, ref, dloss, w, d, s)
        check_grad(out, rg, size, E, DT[dtype])
        assert (out[~ref["live"]] == 0).all()
    # strided rows, and the gradient in the logits' place
    wide = torch.full((n, E + 3), float("nan"), dtype=DT[dtype], device="cuda")
    wide[:, :E] = logits
    again = moe.balance_loss(wide[:, :E], idx, s, m)
    for key in got:
        assert torch.equal(again[key], got[key]), key
    inplace = moe.balance_loss_grad(wide[:, :E], idx, got, dloss, w, dw, s, m, out=wide[:, :E])
    assert torch.equal(inplace, out) and torch.isnan(wide[:, E:]).all()


def test_gradient_against_differences():
    """Central differences of the 64-bit losses in single logits, counts held:
    their error is the third-order term, below 1e-5 at a step of 1e-3."""
    moe = _moe()
    n, E, k = 12, 10, 2
    logits, idx, w = batch(n, E, k, 3)
    s, m = tensors([0, 5, 12], None, n)
    got = moe.balance_loss(logits, idx, s, m)
    dloss = torch.tensor([1.0, 0.5], device="cuda")
    dw = torch.linspace(-1, 1, n * k, device="cuda").view(n, k)
    grad = moe.balance_loss_grad(logits, idx, got, dloss, w, dw, s, m).double()

    def total(l):
        r = reference(l, idx, s, m)
        ws = torch.softmax(torch.gather(l.double(), 1, idx.long()), 1)
        return (r["loss"] * dloss.double()).sum() + (ws * dw.double()).sum()

    for t, e in [(0, 0), (3, 7), (4, int(idx[4, 0])), (5, int(idx[5, 1])), (11, 9)]:
        h = torch.zeros_like(logits, dtype=torch.float64)
        h[t, e] = 1e-3
        fd = (total(logits.double() + h) - total(logits.double() - h)) / 2e-3
        assert (fd - grad[t, e]).abs() <= 1e-5


def test_masked_experts_rows_and_ids():
    """-inf and lowest-value logits, rows of nothing but -inf, NaN in tokens
    that take no part, ids out of range and twice in a token."""
    moe = _moe()
    n, E, k = 40, 70, 4
    logits, idx, w = batch(n, E, k, 8)
    logits[:, 5] = -INF
    logits[3, 10:] = -INF
    logits[4] = -INF
    logits[4, 69] = 1.0
    logits[6] = -INF
    logits[7, 1:] = torch.finfo(torch.float32).min
    logits[20] = float("nan")
    logits[39] = INF
    idx[2] = 11
    idx[9] = torch.tensor([-1, E, 2 ** 31 - 1, 0])
    idx[10] = torch.tensor([69, 3, 69, 3])
    mask = torch.ones(n, dtype=torch.bool, device="cuda")
    mask[20] = False
    seq = torch.tensor([0, 8, 39], dtype=torch.int32, device="cuda")
    got = moe.balance_loss(logits, idx, seq, mask)
    ref = reference(logits, idx, seq, mask)
    check_forward(got, ref, n, E)
    dloss = torch.tensor([1.0, 1.0], device="cuda")
    dw = torch.linspace(-2, 1, n * k, device="cuda").view(n, k)
    out = moe.balance_loss_grad(logits, idx, got, dloss, w, dw, seq, mask)
    rg, size = reference_grad(logits, idx, ref, dloss, w, dw, seq)
    check_grad(out, rg, size, E, torch.float32)
    assert (out[20] == 0).all() and (out[39] == 0).all()
    # all that row 6 has is the gradient of its weights
    free = torch.ones(E, dtype=torch.bool, device="cuda")
    free[idx[6].long()] = False
    assert (out[6][free] == 0).all()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("n", [18, 600])
def test_rows_of_large_logits(n, dtype):
    """Rows of the type's lowest value (a mask that leaves nothing) and rows
    about large numbers, whose lse cannot hold log(sum): p is still the
    softmax of the logits as stored.  600 tokens run in many blocks."""
    moe = _moe()
    E, k, t = 96, 4, DT[dtype]
    logits, idx, w = batch(n, E, k, 21, torch.float32)
    top = torch.finfo(t).max
    base = [0.0, 60.0, 70.0, -70.0, 1e3, -1e3, 6e4, -6e4, 7e4, -1e5, 1e6, 1e9, -1e9, 1e20, -1e38,
            top, -top, 2e38]
    base = torch.tensor(base, device="cuda").clamp(-top, top)
    rows = base[torch.arange(n, device="cuda") % len(base)]
    logits = (logits + rows[:, None]).clamp(-top, top).to(t)
    logits[rows == -top] = -top
    small = rows.abs() <= 1e5
    for mask, dloss in ((None, [0.7, 0.0]), (small, [0.7, -0.3])):
        dloss = torch.tensor(dloss, device="cuda")
        got = moe.balance_loss(logits, idx, None, mask)
        ref = reference(logits, idx, None, mask)
        if mask is None:
            terms = 104 + E + n
            assert torch.isfinite(got["lse"]).all()
            assert ((got["prob"].double() - ref["prob"]).abs() <= terms * H * ref["prob"]).all()
            assert (got["loss"][0] - ref["loss"][0]).abs() <= (terms + 8) * H * ref["loss"][0]
            assert t == torch.float16 or got["loss"][1] == INF      # lse^2 above fp32
        else:
            check_forward(got, ref, n, E)
        out = moe.balance_loss_grad(logits, idx, got, dloss, None, None, None, mask)
        rg, size = reference_grad(logits, idx, ref, dloss, None, None, None)
        check_grad(out, rg, size, E, t)


def test_non_finite_logits_propagate():
    logits, idx, w = batch(6, 40, 2, 1)
    logits[2, 7] = float("nan")
    logits[3] = float("nan")
    logits[4, 1] = INF
    got = _moe().balance_loss(logits, idx)
    bad = torch.tensor([0, 0, 1, 1, 1, 0], dtype=torch.bool, device="cuda")
    assert torch.equal(torch.isnan(got["lse"]) | torch.isinf(got["lse"]), bad)
    assert torch.isnan(got["loss"]).all() and torch.isnan(got["prob"]).any()
    dloss = torch.ones(2, device="cuda")
    grad = _moe().balance_loss_grad(logits, idx, got, dloss)
    assert torch.equal(torch.isnan(grad).any(1), bad)


def test_same_bits_streams_and_graphs():
    moe = _moe()
    n, E, k = 5000, 256, 8
    logits, idx, w = batch(n, E, k, 1)
    s, m = tensors([0, 100, 2500, 5000], 0.9, n)
    dloss = torch.tensor([0.01, 0.001], device="cuda")
    dw = torch.ones((n, k), device="cuda")
    first = moe.balance_loss(logits, idx, s, m)
    grad = moe.balance_loss_grad(logits, idx, first, dloss, w, dw, s, m)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for st in streams * 2:
        with torch.cuda.stream(st):
            f = moe.balance_loss(logits, idx, s, m)
            got.append((f, moe.balance_loss_grad(logits, idx, f, dloss, w, dw, s, m)))
    torch.cuda.synchronize()
    for f, g in got:
        assert all(torch.equal(f[q], first[q]) for q in first) and torch.equal(g, grad)
    sl, si = logits.clone(), idx.clone()
    graphs = []
    for _ in range(2):              # two graphs, each with its own workspace
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            f = moe.balance_loss(sl, si, s, m)
            g = moe.balance_loss_grad(sl, si, f, dloss, w, dw, s, m)
        graphs.append((gr, f, g))
    l2, i2, _ = batch(n, E, k, 2)
    sl.copy_(l2)
    si.copy_(i2)
    torch.cuda.synchronize()
    for st, (gr, _, _) in zip(streams, graphs):
        with torch.cuda.stream(st):
            gr.replay()
    torch.cuda.synchronize()
    want = moe.balance_loss(l2, i2, s, m)
    wg = moe.balance_loss_grad(l2, i2, want, dloss, w, dw, s, m)
    for _, f, g in graphs:
        assert all(torch.equal(f[q], want[q]) for q in want) and torch.equal(g, wg)


def test_router_tuning_step():
    """The operators together, as a router behind a frozen 4-bit projection is
    tuned: project, route with the library's router, losses, the gradient back
    through the router and the projection, and the counts into the placement
    of the experts."""
    import numpy as np
    from quantized_expert_ffn_warp_gb300 import synth
    moe = _moe()
    H, E, k, n, K = 256, 16, 2, 24, 512
    g = torch.Generator(device="cuda").manual_seed(11)
    codes = torch.randint(0, 256, (H, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = (torch.rand((H, K // 128), device="cuda", generator=g) * 0.01 + 0.005).half()
    zeros = torch.randint(6, 10, (H, K // 128), dtype=torch.uint8, device="cuda", generator=g)
    spec = synth.LayerSpec("step", hidden=H, inter=256, n_experts=E, top_k=k, max_tokens=64)
    layer = moe.MoeLayer.from_packed(synth.make_layer(spec))
    x = (0.2 * torch.randn((n, K), device="cuda", generator=g)).half()
    h = moe.linear(x, codes, scales, zeros)
    r = layer.route_topk(h)
    logits = layer.router_logits(h)
    f = moe.balance_loss(logits, r["idx"])
    assert torch.equal(f["counts"][0], r["counts"])
    assert layer.forward_routed(h, r["idx"], r["w"]).isfinite().all()
    plan = moe.residency_plan(f["counts"].sum(0).cpu().numpy(), 4)
    counts = f["counts"].sum(0).cpu().numpy()
    assert sorted(counts[plan].tolist()) == sorted(np.sort(counts)[-4:].tolist())

    dloss = torch.tensor([1.0, 0.1], device="cuda")
    dw = torch.randn((n, k), device="cuda", generator=g)
    dl = moe.balance_loss_grad(logits, r["idx"], f, dloss, r["w"], dw)
    wr = torch.from_numpy(synth.make_layer(spec).router_w.view(np.float16).astype(np.float64)).cuda()
    dh = (dl.double() @ wr).half()
    dx = moe.linear_input_grad(dh, codes, scales, zeros)

    # the whole step in 64 bits through autograd, counts and ids held
    q = torch.stack((codes & 15, codes >> 4), 2).reshape(H, K).double()
    W = (q - zeros.double().repeat_interleave(128, 1)) * scales.double().repeat_interleave(128, 1)
    xr = x.double().requires_grad_()
    lr = (xr @ W.t()) @ wr.t()
    lse = torch.logsumexp(lr, 1)
    p = torch.exp(lr - lse[:, None])
    bal = (f["counts"][0].double() * E / (k * n) * p.mean(0)).sum()
    ws = torch.softmax(torch.gather(lr, 1, r["idx"].long()), 1)
    loss = dloss[0] * bal + dloss[1] * (lse ** 2).mean() + (ws * dw).sum()
    loss.backward()
    # three fp16 roundings (h, dh, dx) and that of the weights; h's moves the
    # logits by about 2^-11 of |h| |wr|, the losses' gradient no more than that
    rel = (dx.double() - xr.grad).norm() / xr.grad.norm()
    assert rel <= 16 * 2.0 ** -11
    layer.close()


@pytest.mark.parametrize("n,E,k,S", [(70000, 8, 2, 65535), (300000, 16, 4, 3), (4000, 1024, 32, 5),
                                     (256, 512, 8, 4), (257, 512, 8, 4), (256, 513, 8, 4)])
def test_largest_sizes(n, E, k, S):
    """The most segments, many tokens, the widest rows, and both sides of the
    one-launch limit."""
    moe = _moe()
    logits, idx, w = batch(n, E, k, 4)
    g = torch.Generator(device="cuda").manual_seed(4)
    cuts = torch.sort(torch.randint(0, n + 1, (S + 1,), device="cuda", generator=g)).values.int()
    cuts = cuts.contiguous()
    got = moe.balance_loss(logits, idx, cuts)
    t = torch.arange(n, device="cuda", dtype=torch.int32)
    seg = torch.searchsorted(cuts, t, right=True).long() - 1
    live = (seg >= 0) & (seg < S)
    p = torch.softmax(logits.double(), 1)
    T = torch.zeros(S, dtype=torch.int64, device="cuda").index_add_(
        0, seg[live], torch.ones_like(seg[live]))
    assert torch.equal(got["tokens"].long(), T)
    counts = torch.zeros(S * E, dtype=torch.int64, device="cuda")
    flat = (seg[:, None] * E + idx.long())[live].reshape(-1)
    counts.index_add_(0, flat, torch.ones_like(flat))
    assert torch.equal(got["counts"].long().flatten(), counts)
    prob = torch.zeros((S, E), dtype=torch.float64, device="cuda").index_add_(0, seg[live], p[live])
    prob /= T.clamp(min=1)[:, None]
    # a segment's sum: at most (tokens of a block per warp + warps + blocks) additions
    terms = 104 + E + n // 8 + 700
    assert ((got["prob"].double() - prob).abs() <= terms * H * prob + 1e-38).all()
    f = counts.view(S, E).double() * E / (k * T.clamp(min=1)[:, None])
    bal = (f * prob).sum() / (T > 0).sum()
    lse = torch.logsumexp(logits.double(), 1)
    z = (lse[live] ** 2).mean()
    loss = got["loss"].double()
    assert (loss[0] - bal).abs() <= 2 * terms * H * bal
    assert (loss[1] - z).abs() <= 2 * terms * H * z + 1e-5 * H * n
    dloss = torch.tensor([0.7, -0.3], device="cuda")
    dw = torch.ones((n, k), device="cuda") * torch.arange(k, device="cuda")
    out = moe.balance_loss_grad(logits, idx, got, dloss, w, dw, cuts).double()
    s = seg.clamp(0, S - 1)
    gs = 0.7 / ((T > 0).sum() * T.clamp(min=1)[s]).double() * live
    dot = (f[s] * p).sum(1, keepdim=True)
    zt = (-0.6 * lse / T.sum() * live)[:, None]
    ref = p * ((f[s] - dot) * gs[:, None] + zt)
    size = p * ((f[s] + dot) * gs[:, None].abs() + zt.abs())
    d = w.double() * (dw - (w.double() * dw).sum(1, keepdim=True)) * live[:, None]
    ref = ref.scatter_add(1, idx.long(), d)
    size = size.scatter_add(1, idx.long(), w.double() * (dw + (w.double() * dw).sum(1, keepdim=True)))
    assert ((out - ref).abs() <= (2 * (104 + E) + 200) * H * size + 1e-38).all()


def test_offsets_beyond_32_bits():
    """Rows far enough apart that element offsets pass 2^32."""
    moe = _moe()
    n, E, k = 600, 24, 3
    ld = (1 << 32) // (n - 1) + 64
    logits, idx, w = batch(n, E, k, 6, torch.bfloat16)
    far = torch.empty((n - 1) * ld + E, dtype=torch.bfloat16, device="cuda")
    rows = far.as_strided((n, E), (ld, 1))
    rows.copy_(logits)
    near, got = moe.balance_loss(logits, idx), moe.balance_loss(rows, idx)
    assert all(torch.equal(near[q], got[q]) for q in near)
    dloss = torch.ones(2, device="cuda")
    want = moe.balance_loss_grad(logits, idx, near, dloss, w, w)
    assert torch.equal(moe.balance_loss_grad(rows, idx, got, dloss, w, w, out=rows), want)


def test_slices_of_one_buffer():
    """Logits and their gradient as column slices of one buffer."""
    moe = _moe()
    n, E, k = 70, 40, 2
    logits, idx, w = batch(n, E, k, 4)
    dloss = torch.tensor([1.0, 0.5], device="cuda")
    want = moe.balance_loss_grad(logits, idx, moe.balance_loss(logits, idx), dloss)
    buf = torch.full((n, 2 * E + 6), 7.0, device="cuda")
    buf[:, :E] = logits
    left, right = buf[:, :E], buf[:, E + 3:2 * E + 3]
    moe.balance_loss_grad(left, idx, moe.balance_loss(left, idx), dloss, out=right)
    assert torch.equal(left, logits) and torch.equal(right, want)
    assert (buf[:, E:E + 3] == 7).all() and (buf[:, 2 * E + 3:] == 7).all()
    with pytest.raises(moe.MoeError):
        moe.balance_loss_grad(left, idx, moe.balance_loss(left, idx), dloss, out=buf[:, 3:E + 3])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("n,seq", [
    (5, [0, 0, 5]), (5, [0, 0]), (200, [0, 0, 0, 0, 200]), (7, [0, 0, 3, 3, 7]), (6, [0, 0, 0]),
    (9, [0, 0, 4]), (9, [2, 2, 9]), (300, [0, 0, 300]), (40, [0, 0, 0, 0, 0, 40])])
def test_leading_empty_segments(n, seq, dtype):
    """Empty segments in front of the first token are written like any other,
    whatever the output memory held: the C call on outputs full of a pattern,
    and the gradient that reads them."""
    moe = _moe()
    E, k, S = 40, 3, len(seq) - 1
    logits, idx, w = batch(n, E, k, n, DT[dtype])
    s, _ = tensors(seq, None, n)
    lib = moe.load_library()
    size = lib.moe_balance_workspace(n, E, S)
    spec = dict(loss=((2,), torch.float32), counts=((S, E), torch.int32),
                tokens=((S,), torch.int32), prob=((S, E), torch.float32),
                lse=((n,), torch.float32), ws=((size,), torch.uint8))
    out = {q: torch.empty(shape, dtype=t, device="cuda") for q, (shape, t) in spec.items()}
    for t in out.values():
        t.view(torch.uint8).fill_(0x5A)
    code = {"fp32": moe.MOE_FP32, "fp16": moe.MOE_FP16, "bf16": moe.MOE_BF16}[dtype]
    rc = lib.moe_balance_loss(logits.data_ptr(), code, E, n, E, idx.data_ptr(), k, s.data_ptr(), S,
                              None, *(out[q].data_ptr() for q in spec), size,
                              torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    ref = reference(logits, idx, s, None)
    check_forward(out, ref, n, E)
    dloss = torch.tensor([0.7, -0.3], device="cuda")
    dw = torch.linspace(-1, 1, n * k, device="cuda").view(n, k)
    for d in (None, dw):
        got = moe.balance_loss_grad(logits, idx, out, dloss, w, d, s)
        rg, size = reference_grad(logits, idx, ref, dloss, w, d, s)
        check_grad(got, rg, size, E, DT[dtype])
        assert (got[~ref["live"]] == 0).all()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("n,E,k", [(60000, 8, 4), (60001, 33, 1), (40000, 256, 8), (9000, 1024, 32)])
def test_successive_tokens_meet_in_the_same_experts(n, E, k, dtype):
    """Runs of tokens whose weights reach the same few experts, so that an entry
    of shared memory is written, read and cleared by different lanes from one
    token to the next: within the bounds, and the same bits every time."""
    moe = _moe()
    logits, _, _ = batch(n, E, k, 31, DT[dtype])
    g = torch.Generator(device="cuda").manual_seed(3)
    turn = torch.rand((n, k), device="cuda", generator=g).argsort(1)
    idx = (turn + E - k).to(torch.int32).contiguous()    # the last k experts in any order
    w = torch.softmax(torch.gather(logits.float(), 1, idx.long()), 1).contiguous()
    dw = torch.randn((n, k), device="cuda", generator=g)
    got = moe.balance_loss(logits, idx)
    dloss = torch.tensor([0.7, -0.3], device="cuda")
    first = moe.balance_loss_grad(logits, idx, got, dloss, w, dw)
    ref = reference(logits, idx, None, None)
    rg, size = reference_grad(logits, idx, ref, dloss, w, dw, None)
    check_grad(first, rg, size, E, DT[dtype])
    for _ in range(20):
        assert torch.equal(moe.balance_loss_grad(logits, idx, got, dloss, w, dw), first)


@pytest.mark.parametrize("k", [1, 4])
def test_gradient_without_ids(k):
    """Without top-k weights the ids are not read: the gradient with k alone is
    that with the ids, bit for bit, and that of the definition."""
    moe = _moe()
    n, E = 50, 24
    logits, idx, w = batch(n, E, k, 2)
    f = moe.balance_loss(logits, idx)
    dloss = torch.tensor([0.7, -0.3], device="cuda")
    got = moe.balance_loss_grad(logits, None, f, dloss, top_k=k)
    assert torch.equal(got, moe.balance_loss_grad(logits, idx, f, dloss))
    rg, size = reference_grad(logits, idx, reference(logits, idx, None, None), dloss, None, None,
                              None)
    check_grad(got, rg, size, E, torch.float32)
    for bad in (None, 0, 33, E + 1):
        with pytest.raises(moe.MoeError):
            moe.balance_loss_grad(logits, None, f, dloss, top_k=bad)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("dloss", [[INF, 0.0], [0.0, -INF], [float("nan"), 1.0], [1.0, float("nan")]])
def test_loss_gradients_that_are_not_finite(dloss, dtype):
    """An overflowed loss gradient stays in the tokens that take part: the
    others, and rows of nothing but -inf, get 0 (there: their weights'
    gradient)."""
    moe = _moe()
    n, E, k = 60, 70, 4
    logits, idx, w = batch(n, E, k, 12, DT[dtype])
    logits[6] = -INF
    mask = torch.ones(n, dtype=torch.bool, device="cuda")
    mask[::3] = False       # token 6 comes back below
    mask[6] = True
    seq = torch.tensor([0, 20, 20, 55], dtype=torch.int32, device="cuda")
    live = mask.clone()
    live[55:] = False
    f = moe.balance_loss(logits, idx, seq, mask)
    dloss = torch.tensor(dloss, device="cuda")
    dw = torch.linspace(-2, 1, n * k, device="cuda").view(n, k)
    plain = moe.balance_loss_grad(logits, idx, f, dloss, None, None, seq, mask)
    both = moe.balance_loss_grad(logits, idx, f, dloss, w, dw, seq, mask)
    for got in (plain, both):
        assert (got[~live] == 0).all()
        live[6] = False
        assert not torch.isfinite(got[live]).all(1).any()
        live[6] = True
    assert (plain[6] == 0).all()
    alone = moe.balance_loss_grad(logits, idx, f, torch.zeros_like(dloss), w, dw, seq, mask)
    assert torch.equal(both[6], alone[6]) and torch.isfinite(both[6]).all() and (both[6] != 0).any()


@pytest.mark.parametrize("n,E,S,dtype,top", [
    (1 << 26, 8, 1, "fp16", 10.3), (1 << 26, 8, 1, "bf16", 3.1), (1 << 24, 16, 5, "fp32", 7.7),
    (1 << 22, 300, 3, "bf16", 4.4), (1 << 20, 600, 1, "fp16", 5.3), (1 << 21, 1024, 200, "bf16", 2.2),
    (131070, 1024, 65535, "fp16", 6.1)])
def test_long_batches_of_equal_rows(n, E, S, dtype, top):
    """Equal terms round alike, so that a chain's error grows with its length:
    the bound here does not.  Of an fp32 sum it is 64 + 8 + 157 roundings (the
    span of a warp, the warps, the blocks) and up to 8 of folding; a term adds
    (1.3 |d| + 3) H twice for its exponential and the row's sum, E / 32 + 5 for
    that sum, 5 for the quotient, with |d| <= 2; lse^2 twice that of lse, whose
    logarithm is good to 12 H here, over lse >= 4."""
    moe = _moe()
    row = (torch.linspace(-1, 1, E, device="cuda") + top).to(DT[dtype])
    logits = row.expand(n, E).contiguous()
    idx = torch.full((n, 1), E - 1, dtype=torch.int32, device="cuda")
    seq = torch.linspace(0, n, S + 1, dtype=torch.float64).round().int().cuda()
    got = moe.balance_loss(logits, idx, seq if S > 1 else None)
    p, lse = torch.softmax(row.double(), 0), torch.logsumexp(row.double(), 0)
    chain, term = 64 + 8 + 157 + 8, 2 * 6 + E / 32 + 5 + 5
    assert torch.equal(got["tokens"].long(), (seq[1:] - seq[:-1]).long())
    assert ((got["prob"].double() - p).abs() <= (chain + term) * H * p).all()
    assert ((got["lse"].double() - lse).abs() <= (term + 12 + 2 * lse) * H).all()
    bal = E * p[E - 1]
    assert (got["loss"][0].double() - bal).abs() <= (chain + term + 16) * H * bal
    z = lse ** 2
    assert (got["loss"][1].double() - z).abs() <= (chain + 8 + 2 * ((term + 12) / lse + 2)) * H * z


def test_long_batches_with_infinite_squares():
    """lse^2 above fp32 is an infinity in loss[1], in long batches too, and
    NaN stays NaN."""
    moe = _moe()
    n, E, k = 1 << 20, 8, 2
    logits, idx, w = batch(n, E, k, 3)
    logits[::1000] = torch.finfo(torch.float32).min
    got = moe.balance_loss(logits, idx)
    ref = torch.softmax(logits.double(), 1).mean(0)
    assert got["loss"][1] == INF and torch.isfinite(got["loss"][0])
    assert ((got["prob"][0].double() - ref).abs() <= 400 * H * ref).all()
    logits[70000] = float("nan")
    got = moe.balance_loss(logits, idx)
    assert torch.isnan(got["loss"]).all() and torch.isnan(got["prob"]).all()
