"""Adapters where h and u, the products between the two matrices, are far from 1 in
size, have more bits than the activations' type, or are summed over very many tokens."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from tuning_refs import DT, H, half_step  # noqa: E402

INF = float("inf")


def _moe():
    from quantized_expert_ffn_warp_gb300 import moe
    return moe


# ---------------------------------------------------------------- values that are not finite

@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("rank", [8, 16, 24, 40, 72, 128])
@pytest.mark.parametrize("n", [3, 200])
def test_an_infinite_h_gives_infinite_results(n, rank, dtype):
    """Sums of +inf and positive terms are +inf, at ranks that the products pad too."""
    moe, dt = _moe(), DT[dtype]
    x = torch.ones((n, 64), dtype=dt, device="cuda")
    x[1, 5] = INF
    ids = torch.zeros(n, dtype=torch.int32, device="cuda")
    A = torch.full((1, rank, 64), 2.0 ** -6, dtype=dt, device="cuda")
    B = torch.full((1, 200, rank), 2.0 ** -4, dtype=dt, device="cuda")
    out, h = moe.adapter(x, ids, A, B)
    rest = [i for i in range(n) if i != 1]
    assert (h[1] == INF).all() and (h[rest] == 1).all()
    assert (out[1] == INF).all() and (out[rest] == rank / 16).all()
    dy = torch.ones((n, 200), dtype=dt, device="cuda")
    dy[1, 7] = INF
    got = moe.adapter_grad(dy, torch.ones_like(x), torch.ones_like(h), ids, A, B)
    assert (got["dx"][1] == INF).all() and (got["dx"][rest] == rank * 12.5 / 64).all()
    assert (got["dA"] == INF).all()
    assert (got["dB"][0, 7] == INF).all() and torch.isfinite(got["dB"][0, 8:]).all()


# ---------------------------------------------------------------- sizes

def rel(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


def limit(want, dtype, rows, n):
    """The rounding of the results themselves, and of fp32 sums over rows and tokens: an
    accumulation for every 16 terms, each off by at most a step 2 H of a partial sum that
    is at most about twice the result; the terms' own splits at most 4 H."""
    return rel(want.to(dtype), want) * 1.01 + (rows + n + 64) / 16 * 4 * H + 4 * H


def operands(n, cols, rows, rank, count, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + n)

    def randn(*s, scale=1.0):
        return (torch.randn(s, device="cuda", generator=g) * scale).to(DT[dtype])
    ids = torch.randint(0, count, (n,), device="cuda", generator=g).to(torch.int32)
    return randn, ids


def exact_grad(dy, x, ids, A, B, scale):
    f = torch.float64
    dx = torch.zeros(x.shape, dtype=f, device="cuda")
    dA = torch.zeros(A.shape, dtype=f, device="cuda")
    for a in range(len(A)):
        t = (ids == a).nonzero()[:, 0]
        u = scale[a].to(f) * (dy[t].to(f) @ B[a].to(f))
        dx[t] = u @ A[a].to(f)
        dA[a] = u.t() @ x[t].to(f)
    return dx, dA


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n,rows,size_dy,size_b,size_a", [
    (2048, 1024, 2e-2, 5e-2, 0.05), (2048, 1024, 1e-4, 1e-3, 30.0), (8192, 1024, 1e-4, 1e-4, 300.0),
    (8192, 4096, 1e-5, 1e-4, 1e3), (300, 1000, 3e-6, 1e-4, 3e3)])
def test_gradients_of_small_u(n, rows, size_dy, size_b, size_a, dtype):
    """The sizes that an adapter's first steps have under a mean loss: B starts at 0."""
    moe = _moe()
    cols, rank, count = 512, 16, 2
    randn, ids = operands(n, cols, rows, rank, count, dtype)
    x, dy = randn(n, cols), randn(n, rows, scale=size_dy)
    A, B = randn(count, rank, cols, scale=size_a), randn(count, rows, rank, scale=size_b)
    scale = torch.tensor([0.75, 2.0], device="cuda")
    h = torch.zeros((n, rank), dtype=x.dtype, device="cuda")
    got = moe.adapter_grad(dy, x, h, ids, A, B, scale)
    dx, dA = exact_grad(dy, x, ids, A, B, scale)
    assert rel(got["dA"], dA) <= limit(dA, x.dtype, rows, n)
    assert rel(got["dx"], dx) <= limit(dx, x.dtype, rows, rank)
    only = moe.adapter_grad(dy, x, h, ids, A, B, scale, input_grad=False)
    assert torch.equal(only["dA"], got["dA"]) and torch.equal(only["dB"], got["dB"])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("size_x,size_a,size_b", [(1e-4, 1e-3, 8.0), (1e-5, 1e-3, 100.0),
                                                  (1e-3, 1e-5, 1e3)])
def test_forward_of_small_h(size_x, size_a, size_b, dtype):
    moe = _moe()
    n, cols, rows, rank, count = 500, 1024, 384, 24, 3
    randn, ids = operands(n, cols, rows, rank, count, dtype)
    x, A = randn(n, cols, scale=size_x), randn(count, rank, cols, scale=size_a)
    B = randn(count, rows, rank, scale=size_b)
    scale = torch.tensor([1.0, 30.0, 200.0], device="cuda")
    out, _ = moe.adapter(x, ids, A, B, scale)
    at = ids.long()
    h = torch.einsum("tk,trk->tr", x.double(), A.double()[at])
    want = torch.einsum("tr,tjr->tj", h, B.double()[at]) * scale.double()[at][:, None]
    assert rel(out, want) <= limit(want, x.dtype, cols, rank)


def test_products_beyond_the_range_of_fp16():
    """h and u above 65504 whose results are within it."""
    moe = _moe()
    n, cols, rows, rank, count = 150, 1024, 2048, 16, 2
    randn, ids = operands(n, cols, rows, rank, count, "fp16")
    scale = torch.tensor([0.5, 2.0], device="cuda")
    x, dy = randn(n, cols, scale=1e-4), randn(n, rows, scale=300.0)
    A, B = randn(count, rank, cols, scale=1e-4), randn(count, rows, rank, scale=300.0)
    h = torch.zeros((n, rank), dtype=torch.float16, device="cuda")
    got = moe.adapter_grad(dy, x, h, ids, A, B, scale)
    dx, dA = exact_grad(dy, x, ids, A, B, scale)
    assert (dy.double() @ B[0].double()).abs().max() > 1e6 and dA.abs().max() < 65504
    assert rel(got["dA"], dA) <= limit(dA, x.dtype, rows, n)
    assert rel(got["dx"], dx) <= limit(dx, x.dtype, rows, rank)
    x, A = randn(n, cols, scale=300.0), randn(count, rank, cols, scale=300.0)
    B = randn(count, rows, rank, scale=1e-4)
    out, h = moe.adapter(x, ids, A, B, scale)
    at = ids.long()
    want = torch.einsum("tk,trk->tr", x.double(), A.double()[at])
    big = want.abs() > 70000        # what is kept of h is fp16
    assert big.any() and torch.equal(h[big].double(), INF * want[big].sign())
    want = torch.einsum("tr,tjr->tj", want, B.double()[at]) * scale.double()[at][:, None]
    assert rel(out, want) <= limit(want, x.dtype, cols, rank)


def test_tokens_of_unequal_size():
    """Every token's own result, and sums over tokens whose u differ by 2^24."""
    moe = _moe()
    n, cols, rows, rank = 600, 256, 512, 16
    randn, ids = operands(n, cols, rows, rank, 1, "fp16")
    size = 2.0 ** -(torch.arange(n, device="cuda") % 25)
    dy = (randn(n, rows).float() * size[:, None]).half()
    x = (randn(n, cols).float() * 1e-4 / size[:, None]).half()
    A, B, one = randn(1, rank, cols), randn(1, rows, rank, scale=0.01), torch.ones(1, device="cuda")
    h = torch.zeros((n, rank), dtype=torch.float16, device="cuda")
    got = moe.adapter_grad(dy, x, h, ids, A, B)
    dx, dA = exact_grad(dy, x, ids, A, B, one)
    assert rel(got["dA"], dA) <= limit(dA, x.dtype, rows, n)
    for i in range(25):
        assert rel(got["dx"][i::25], dx[i::25]) <= limit(dx[i::25], x.dtype, rows, rank)


# ---------------------------------------------------------------- bits

# What is left when the leading parts of h or u cancel.  h = a + b s + c s^2 (s = 2^-8; in
# fp16 a + b s with s = 2^-11) has 24 (22) bits; a second rank holds b, and base -a.  At most
# six roundings of sums below 4, 2^-21 each in the tensor cores and the epilogue.

def _parts(dtype, n):
    g = torch.Generator(device="cuda").manual_seed(7)
    step, s = (2.0 ** -7, 2.0 ** -8) if dtype == "bf16" else (2.0 ** -10, 2.0 ** -11)
    k = torch.randint(0, int(0.9 / step), (n, 3), device="cuda", generator=g)
    v = (1 + k * step).to(DT[dtype])
    return v, s, 2 if dtype == "bf16" else 1


TOL = 6 * 2.0 ** -21


@pytest.mark.parametrize("dtype,size", [("bf16", 1.0), ("bf16", 2.0 ** -30), ("fp16", 1.0),
                                        ("fp16", 2.0 ** -9)])
@pytest.mark.parametrize("rank", [8, 16, 32, 64, 128])
def test_h_and_u_keep_their_bits(dtype, size, rank):
    moe, n = _moe(), 700
    v, s, last = _parts(dtype, n)
    dt = v.dtype
    x = torch.zeros((n, 8), dtype=dt, device="cuda")
    x[:, :3] = v * size
    if last == 1:
        x[:, 2] = 0
    A = torch.zeros((1, rank, 8), dtype=dt, device="cuda")
    A[0, 0, :3] = torch.tensor([1.0, s, s * s if last == 2 else 0.0], device="cuda")
    if last == 2:
        A[0, 1, 1] = 1.0
    B = torch.zeros((1, 8, rank), dtype=dt, device="cuda")
    B[0, 0, 0], B[0, 0, 1] = 1.0, -s
    base = torch.zeros((n, 8), dtype=dt, device="cuda")
    base[:, 0] = -v[:, 0]
    ids = torch.zeros(n, dtype=torch.int32, device="cuda")
    scale = torch.tensor([1 / size], device="cuda")
    want = v[:, last].double() * s ** last
    out, _ = moe.adapter(x, ids, A, B, scale, base=base)
    assert ((out[:, 0].double() - want).abs() <= TOL + half_step(want, dt)).all()
    # the same through B and A backward
    h = torch.zeros((n, rank), dtype=dt, device="cuda")
    Bt, At = A.transpose(1, 2).contiguous(), B.transpose(1, 2).contiguous()
    got = moe.adapter_grad(x, base, h, ids, At, Bt, scale, base=base)
    assert ((got["dx"][:, 0].double() - want).abs() <= TOL + half_step(want, dt)).all()


@pytest.mark.parametrize("dtype,size", [("bf16", 1.0), ("fp16", 1.0), ("fp16", 2.0 ** -9)])
@pytest.mark.parametrize("rank", [8, 24, 64, 128])
def test_sums_over_tokens_keep_the_bits_of_u(dtype, size, rank):
    """Two tokens an adapter, whose u differ in the last part alone, and x = 1, -1."""
    moe, n = _moe(), 900
    v, s, last = _parts(dtype, n)
    dt = v.dtype
    dy = torch.zeros((n, 2, 8), dtype=dt, device="cuda")
    dy[:, :, :last] = (v * size)[:, None, :last]
    dy[:, 0, last] = v[:, last] * size
    B = torch.zeros((n, 8, rank), dtype=dt, device="cuda")
    B[:, :3, rank - 1] = torch.tensor([1.0, s, s * s], device="cuda").to(dt)
    x = torch.ones((n, 2, 16), dtype=dt, device="cuda")
    x[:, 1] = -1
    ids = torch.arange(n, device="cuda", dtype=torch.int32).repeat_interleave(2).contiguous()
    A = torch.zeros((n, rank, 16), dtype=dt, device="cuda")
    h = torch.zeros((2 * n, rank), dtype=dt, device="cuda")
    scale = torch.full((n,), 1 / size, device="cuda")
    got = moe.adapter_grad(dy.flatten(0, 1), x.flatten(0, 1), h, ids, A, B, scale)
    want = (v[:, last].double() * s ** last)[:, None].expand(n, 16)
    assert ((got["dA"][:, rank - 1].double() - want).abs() <= TOL + half_step(want, dt)).all()
    assert (got["dA"][:, :rank - 1] == 0).all()


# ---------------------------------------------------------------- long sums

@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n,rank", [(1 << 20, 8), (300001, 64), (150000, 128), (16385, 64), (16384, 24)])
def test_sums_over_very_many_tokens_of_one_sign(n, rank, dtype):
    """One of many loaded adapters has all tokens.  16384 tokens at most are one chain, 1024
    accumulations of 16 terms off by a step 2 H each; more are chains of 4096, 256 such
    accumulations each, and at most 257 sums of those, H each.  The lower parts of u are
    2^-8 and less of the first and so are their sums' errors."""
    moe, count = _moe(), 304
    g = torch.Generator(device="cuda").manual_seed(n)

    def part(*shape, top=1.0):
        return ((torch.rand(shape, device="cuda", generator=g) / 2 + 0.5) * top).to(DT[dtype])
    x, dy, h = part(n, 16), part(n, 24, top=2.0 ** -8), part(n, rank)
    A, B = part(count, rank, 16), part(count, 24, rank, top=0.25)
    ids = torch.full((n,), 5, dtype=torch.int32, device="cuda")
    got = moe.adapter_grad(dy, x, h, ids, A, B, input_grad=False)
    u = dy.double() @ B[5].double()
    for name, want in (("dA", u.t() @ x.double()), ("dB", dy.double().t() @ h.double())):
        v = got[name][5].double()
        err = (1024 * 2 * 1.01 + 32) * H * want
        assert ((v - want).abs() <= err + half_step(want, x.dtype)).all(), name
        got[name][5] = 0
        assert (got[name] == 0).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_long_contractions_of_one_sign(dtype):
    """A x over 2^20 columns in one piece, as many loaded adapters and some tokens have
    them.  Chains of 16384 columns are 1024 accumulations of 16 terms, off by a step 2 H
    each; 64 sums of those, H each."""
    moe, n, cols, count = _moe(), 160, 1 << 20, 304
    g = torch.Generator(device="cuda").manual_seed(1)
    x = (torch.rand((n, cols), device="cuda", generator=g) / 2 + 0.5).to(DT[dtype])
    A = torch.zeros((count, 8, cols), dtype=DT[dtype], device="cuda")
    A[7] = (torch.rand((8, cols), device="cuda", generator=g) / 2 + 0.5) * 2.0 ** -10
    B = torch.zeros((count, 8, 8), dtype=DT[dtype], device="cuda")
    B[7] = torch.eye(8, device="cuda")
    ids = torch.full((n,), 7, dtype=torch.int32, device="cuda")
    out, h = moe.adapter(x, ids, A, B)
    want = x.double() @ A[7].double().t()
    err = (1024 * 2 + 64 + 32) * H * want
    for got in (out, h):
        assert ((got.double() - want).abs() <= err + half_step(want, x.dtype)).all()


# ---------------------------------------------------------------- the same bits

@pytest.mark.parametrize("n", [5, 900])
def test_fp16_same_bits_on_streams_in_graphs_and_in_any_order(n):
    """Each token's and each adapter's power of two is found anew in every call."""
    moe = _moe()
    cols, rows, rank, count = 512, 768, 24, 5
    randn, ids = operands(n, cols, rows, rank, count, "fp16")
    A, B = randn(count, rank, cols, scale=0.05), randn(count, rows, rank, scale=1e-3)
    dy = randn(n, rows, scale=1e-4)

    def both(x, stream=None):
        out, h = moe.adapter(x, ids, A, B, stream=stream)
        g = moe.adapter_grad(dy, x, h, ids, A, B, stream=stream)
        only = moe.adapter_grad(dy, x, h, ids, A, B, input_grad=False, stream=stream)
        assert set(only) == {"dA", "dB"}
        return [out, h, g["dx"], g["dA"], g["dB"], only["dA"], only["dB"]]
    x = randn(n, cols)
    first = both(x)
    torch.cuda.synchronize()
    assert torch.equal(first[3], first[5]) and torch.equal(first[4], first[6])
    side = torch.cuda.Stream()
    again = both(x, side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, again))
    p = torch.randperm(n, device="cuda")
    out, h = moe.adapter(x[p].contiguous(), ids[p].contiguous(), A, B)
    assert torch.equal(out, first[0][p]) and torch.equal(h, first[1][p])
    static, pool, graphs = x.clone(), torch.cuda.graph_pool_handle(), []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            res = both(static)
        graphs.append((g, res))
    for turn in range(4):       # sizes that differ from call to call
        static.copy_(randn(n, cols, scale=(1.0, 1e-3, 100.0, 1e-5)[turn]))
        g, res = graphs[turn % 2]
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(res, both(static)))
