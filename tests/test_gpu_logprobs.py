"""Token log probabilities and their gradient against 64-bit definitions; the
bounds are derived in tuning_refs.py."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from tuning_refs import DT, H, INF, half_step, logprob_bounds, logprobs, logprobs_grad  # noqa: E402


def _moe():
    from quantized_expert_ffn_warp_gb300 import moe
    return moe


def batch(n, V, dtype, seed, spread=2.5, pad=0, lead=0):
    """logits [n, V] of rows `pad` longer that start `lead` elements into a buffer."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    wide = (spread * torch.randn((n, V + pad + lead), device="cuda", generator=g)).to(DT[dtype])
    targets = torch.randint(-1, V + 1, (n,), device="cuda", generator=g).to(torch.int32)
    return wide[:, lead:lead + V], targets


def same(a, b):
    """Equal where not finite (NaN anywhere in place of NaN)."""
    bad = ~torch.isfinite(b)
    return torch.equal(torch.nan_to_num(a[bad], 7e30), torch.nan_to_num(b[bad].to(a.dtype), 7e30))


def check(logits, targets, top, got=None):
    got = _moe().token_logprobs(logits, targets, top=top) if got is None else got
    ref = logprobs(logits, targets, top)
    V = logits.shape[1]
    logsum, ent, lp = logprob_bounds(ref, V)
    fin = torch.isfinite(ref["stats"]).all(1)
    m = ref["stats"][:, 0]
    assert torch.equal(got["stats"][:, 0].double()[~torch.isnan(m)], m[~torch.isnan(m)])
    for name, bound in (("entropy", ent), ("stats", None), ("logp", None), ("top_logp", None)):
        if name not in ref:
            assert name not in got
            continue
        a, b = got[name].double(), ref[name]
        if name == "stats":
            a, b, bound = a[:, 1], b[:, 1], logsum
        elif name == "logp":
            bound = lp(b, torch.where(ref["on"], ref["d"].gather(1, ref["at"][:, None])[:, 0], 0.0))
        elif name == "top_logp":
            bound = lp(b, ref["d"].gather(1, ref["top_ids"].long())
                       ).amax(1, keepdim=True) if b.dim() == 1 else 4 * H * b.abs() + logsum[:, None]
        ok = torch.isfinite(b)
        assert ((a - b).abs()[ok] <= (bound.expand_as(b))[ok]).all(), name
        assert same(a, b), name
    if top:
        assert torch.equal(got["top_ids"], ref["top_ids"])
    del fin
    return got, ref


SIZES = [(1, 1), (1, 2), (3, 7), (2, 31), (5, 255), (700, 255), (4, 4095), (3, 4097), (1, 32003),
         (13, 32003), (650, 32003), (2, 131072), (1, 1048576), (70000, 3)]


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("n,V", SIZES)
@pytest.mark.parametrize("top", [0, 5, 32])
def test_sizes(n, V, dtype, top):
    logits, targets = batch(n, V, dtype, n + V)
    check(logits, targets, min(top, V))


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("pad,lead", [(1, 0), (3, 5), (64, 8), (13, 3)])
@pytest.mark.parametrize("n,V", [(1, 999), (6, 8191), (700, 1000)])
def test_strides_and_unaligned_rows(n, V, dtype, pad, lead):
    logits, targets = batch(n, V, dtype, n + V, pad=pad, lead=lead)
    check(logits, targets, 7)
    check(logits, None, 0)


@pytest.mark.parametrize("n", [3, 900])
@pytest.mark.parametrize("kind", ["ties", "rising", "falling", "few_values", "spikes", "zeros"])
def test_order_of_the_likeliest(n, kind):
    V = 9001
    g = torch.Generator(device="cuda").manual_seed(1)
    i = torch.arange(V, device="cuda", dtype=torch.float32)
    row = dict(ties=torch.zeros(V, device="cuda"), rising=i / 900, falling=-i / 900,
               few_values=torch.floor(i % 3), spikes=torch.where(i % 1500 == 1499, 5.0, 0.0),
               zeros=torch.where(i % 2 == 0, 0.0, -0.0))[kind]
    logits = row.repeat(n, 1)
    if kind == "few_values":
        logits = logits[:, torch.randperm(V, device="cuda", generator=g)].contiguous()
    targets = torch.full((n,), 17, dtype=torch.int32, device="cuda")
    for top in (1, 20, 32):
        check(logits, targets, top)
        check(logits.half(), targets, top)


@pytest.mark.parametrize("n", [2, 1000])
@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
def test_masked_rows_and_values_that_are_not_finite(n, dtype):
    V = 5003
    logits, targets = batch(n, V, dtype, 3)
    targets = targets.clamp(0, V - 1)
    logits = logits.clone()
    logits[0] = -INF
    logits[1, 1:] = -INF
    check(logits, targets, 9)
    logits[1, :4000] = -INF
    logits[1, 4001:] = -INF
    check(logits, targets, 32)
    logits[0] = torch.finfo(DT[dtype]).min       # a mask of the type's lowest value
    check(logits, targets, 9)
    logits[0, 77] = -3.0
    check(logits, targets, 9)
    logits[0] = torch.finfo(DT[dtype]).max
    check(logits, targets, 9)
    logits[0] = 1.0
    logits[0, 3] = float("nan")
    logits[1] = float("nan")
    got, ref = check(logits, targets, 9)
    assert torch.isnan(got["logp"][:2]).all() and torch.isnan(got["entropy"][:2]).all()
    logits[0, 3] = INF
    got = _moe().token_logprobs(logits, targets, top=2)
    assert got["top_ids"][0, 0] == 3 and torch.isnan(got["stats"][0, 1])
    assert torch.isfinite(got["logp"][2:]).all()


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("n,V,pad,lead", [(1, 1, 0, 0), (3, 31, 0, 0), (5, 999, 3, 5), (2, 131072, 0, 0),
                                          (700, 4097, 0, 0), (9, 32003, 61, 8), (70000, 5, 0, 0)])
@pytest.mark.parametrize("which", ["logp", "entropy", "both"])
def test_gradient(n, V, dtype, pad, lead, which):
    moe = _moe()
    logits, targets = batch(n, V, dtype, n + V, pad=pad, lead=lead)
    logits = logits.clone() if V < 4 else logits
    if V > 40:
        logits[:, V - 7:] = -INF
        logits[0] = -INF
    g = torch.Generator(device="cuda").manual_seed(5)
    dlogp = torch.randn(n, device="cuda", generator=g) if which != "entropy" else None
    dent = torch.randn(n, device="cuda", generator=g) if which != "logp" else None
    ref = logprobs(logits, targets)
    fwd = dict(stats=ref["stats"].float(), entropy=ref["entropy"].float())
    want, err = logprobs_grad(logits, targets, ref, dlogp, dent)
    got = moe.token_logprobs_grad(logits, targets, fwd, dlogp, dent)
    assert ((got.double() - want).abs() <= err + half_step(want, DT[dtype])).all()
    # in place, and into rows that lie otherwise
    room = torch.full((n, V + 3), 7.0, dtype=DT[dtype], device="cuda")
    moe.token_logprobs_grad(logits, targets, fwd, dlogp, dent, out=room[:, 1:V + 1])
    assert torch.equal(room[:, 1:V + 1], got) and (room[:, V + 1:] == 7).all()
    assert (room[:, 0] == 7).all()
    moe.token_logprobs_grad(logits, targets, fwd, dlogp, dent, out=logits)
    assert torch.equal(logits, got)


@pytest.mark.parametrize("n", [4, 800])
def test_gradient_of_positions_without_a_target(n):
    """Their rows are 0 whatever their logits and dlogp hold, without an entropy term."""
    moe = _moe()
    V = 1003
    logits, targets = batch(n, V, "bf16", 9)
    targets.zero_()
    targets[1], targets[2] = -1, V
    dlogp = torch.ones(n, device="cuda")
    dlogp[1] = float("nan")
    logits[1] = float("nan")
    fwd = moe.token_logprobs(logits, targets)
    got = moe.token_logprobs_grad(logits, targets, fwd, dlogp)
    assert (got[1:3] == 0).all() and torch.isfinite(got).all() and (got[0] != 0).any()
    assert (fwd["logp"][1:3] == 0).all()
    logits[0, 5] = float("nan")
    fwd = moe.token_logprobs(logits, targets)
    assert torch.isnan(moe.token_logprobs_grad(logits, targets, fwd, dlogp)[0]).all()


def test_offsets_beyond_32_bits():
    """More than 2^31 elements: the last rows."""
    moe = _moe()
    n, V = 36000, 65537
    logits = torch.zeros((n, V), dtype=torch.bfloat16, device="cuda")
    logits[-3:] = batch(3, V, "bf16", 2)[0]
    targets = torch.full((n,), 65536, dtype=torch.int32, device="cuda")
    got = moe.token_logprobs(logits, targets, top=3)
    tail = {k: v[-3:] for k, v in got.items()}
    check(logits[-3:], targets[-3:], 3, tail)
    assert torch.equal(got["top_ids"][0].cpu(), torch.arange(3, dtype=torch.int32))
    dlogp = torch.ones(n, device="cuda")
    part = moe.token_logprobs_grad(logits[-3:], targets[-3:], tail, dlogp[-3:])
    moe.token_logprobs_grad(logits, targets, got, dlogp, out=logits)
    assert torch.equal(logits[-3:], part)


@pytest.mark.parametrize("n,V", [(2, 32003), (700, 5000)])
def test_same_bits_on_other_streams_and_in_graphs(n, V):
    moe = _moe()
    logits, targets = batch(n, V, "bf16", 4)
    dlogp = torch.ones(n, device="cuda")
    first = moe.token_logprobs(logits, targets, top=8)
    grad = moe.token_logprobs_grad(logits, targets, first, dlogp, dlogp)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    again = moe.token_logprobs(logits, targets, top=8, stream=side)
    side.synchronize()
    for k in first:
        assert torch.equal(first[k], again[k]), k
    # two graphs over one pool, replayed in turn on other inputs
    graphs, outs = [], []
    pool = torch.cuda.graph_pool_handle()
    static = logits.clone()
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            f = moe.token_logprobs(static, targets, top=8)
            d = moe.token_logprobs_grad(static, targets, f, dlogp, dlogp)
        graphs.append(g)
        outs.append((f, d))
    for turn in range(3):
        other = batch(n, V, "bf16", 50 + turn)[0]
        static.copy_(other if turn < 2 else logits)
        g, (f, d) = graphs[turn % 2], outs[turn % 2]
        g.replay()
        torch.cuda.synchronize()
        want = moe.token_logprobs(static, targets, top=8)
        for k in want:
            assert torch.equal(f[k], want[k]), k
        assert torch.equal(d, moe.token_logprobs_grad(static, targets, want, dlogp, dlogp))
    assert torch.equal(d, grad)


def test_other_streams_tensors_and_refusals():
    moe = _moe()
    logits, targets = batch(4, 100, "fp32", 4)
    with pytest.raises(moe.MoeError):
        moe.token_logprobs(logits, targets.cpu())
    with pytest.raises(moe.MoeError):
        moe.token_logprobs(logits, targets, top=101)
    with pytest.raises(moe.MoeError):
        moe.token_logprobs(logits.t(), targets)
    fwd = moe.token_logprobs(logits, targets)
    with pytest.raises(moe.MoeError):
        moe.token_logprobs_grad(logits, targets, fwd)
    wide = torch.zeros((4, 150), device="cuda")
    with pytest.raises(moe.MoeError, match="overlap"):
        moe.token_logprobs_grad(wide[:, :100], targets, fwd, torch.ones(4, device="cuda"),
                                out=wide[:, 50:])
