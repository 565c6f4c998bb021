"""4-bit products against a 64-bit evaluation of their formulas.

Tolerance of one output r = sum of the terms v (2^-24: half an fp32 step, u:
half a step of the output type, S = sum |v|):
  u |r|                     the rounding of the output
  u S                       the rounding of each weight (q - z) s to the
                            activations' type, where the kernel makes one
  (terms / 8 + 64) 2^-23 S  fp32 sums: an MMA adds 16 terms to the
                            accumulator with a few truncated steps, at most
                            one 2^-23 step of the sum each; splits add < 64
Independent roundings do not add up: over a whole output the relative 2-norm
error is that of the output rounding and of the weight rounding, each at most
u, so 2 u plus the fp32 part bounds it with a wide margin (their root mean
squares are u / sqrt 3).
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


def _moe():
    from quantized_expert_ffn_warp_gb300 import moe
    return moe


def matrix(rows, K, group, seed, scale=(0.005, 0.02)):
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = (torch.rand((rows, K // group), device="cuda", generator=g)
              * (scale[1] - scale[0]) + scale[0]).half()
    zeros = torch.randint(0, 16, (rows, K // group), dtype=torch.uint8, device="cuda", generator=g)
    q = torch.stack((codes & 15, codes >> 4), 2).reshape(rows, K).double()
    W = ((q - zeros.double().repeat_interleave(group, 1))
         * scales.double().repeat_interleave(group, 1))
    return (codes, scales, zeros, group), W


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=g) * scale).to(dtype)


def strided(t, pad, fill=float("nan")):
    wide = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device=t.device)
    wide[:, : t.shape[1]] = t
    return wide[:, : t.shape[1]]


def check(got, ref, S, terms, dtype):
    u = torch.finfo(dtype).eps / 2
    fp32 = (terms / 8 + 64) * 2.0 ** -23
    err = (got.double() - ref).abs()
    tol = u * ref.abs() * (1 + 4 * u) + (u + fp32) * S
    bad = err > tol
    assert not bad.any(), "%d of %d over the bound, worst %g of it" % (
        bad.sum(), bad.numel(), (err / tol).max())
    rel = (got.double() - ref).norm() / ref.norm()
    assert rel <= 2 * u + fp32 * (S.norm() / ref.norm()), rel


SIZES = [
    # n, rows, K, group
    (1, 1, 32, 32), (1, 16, 128, 128), (1, 17, 512, 128), (2, 1027, 544, 32), (3, 33, 1152, 128),
    (4, 130, 192, 64), (5, 15, 2048, 128), (7, 300, 4096, 64), (8, 256, 4224, 128),
    (9, 257, 640, 128), (16, 31, 1056, 32), (17, 129, 1024, 128), (33, 384, 1088, 64),
    (64, 1000, 512, 128), (65, 128, 8192, 128), (130, 515, 768, 32), (255, 136, 384, 128),
    (256, 640, 1024, 64), (300, 1031, 2048, 128), (513, 72, 96, 32), (1, 5003, 14336, 128),
]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("n,rows,K,group", SIZES)
def test_linear(n, rows, K, group, dtype):
    m, W = matrix(rows, K, group, seed=rows + K)
    x = randn((n, K), DT[dtype], n)
    bias, res = randn((rows,), DT[dtype], 3), randn((n, rows), DT[dtype], 4)
    ref, S = x.double() @ W.t(), x.double().abs() @ W.t().abs()
    check(_moe().linear(x, *m), ref, S, K, DT[dtype])
    ref, S = ref + bias.double() + res.double(), S + bias.double().abs() + res.double().abs()
    check(_moe().linear(x, *m, bias=bias, residual=res), ref, S, K + 2, DT[dtype])
    # strided rows: what lies between them is not read and stays as it was
    xs, out, rs = strided(x, 24), strided(torch.zeros_like(res), 5, 7.0), strided(res, 3)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _moe().linear(xs, *m, bias=bias, residual=rs, out=out, status=st)
    check(got, ref, S, K + 2, DT[dtype])
    assert got is out and st.item() == 0
    gap = out.as_strided((n, 5), (rows + 5, 1), rows)
    assert n == 1 or (gap[:-1] == 7).all()
    # the residual stream updated in place
    got = res.clone()
    _moe().linear(x, *m, bias=bias, residual=got, out=got)
    check(got, ref, S, K + 2, DT[dtype])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("n,rows,K,group", SIZES)
def test_linear_input_grad(n, rows, K, group, dtype):
    m, W = matrix(rows, K, group, seed=rows + K)
    dy = randn((n, rows), DT[dtype], n, 0.1)
    ref, S = dy.double() @ W, dy.double().abs() @ W.abs()
    check(_moe().linear_input_grad(dy, *m), ref, S, rows, DT[dtype])
    for pad in (8 - rows % 8, 3):       # rows on 16-byte boundaries, and on none
        out = strided(torch.zeros((n, K), dtype=DT[dtype], device="cuda"), 3, 7.0)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = _moe().linear_input_grad(strided(dy, pad), *m, out=out, status=st)
        check(got, ref, S, rows, DT[dtype])
        assert st.item() == 0
        gap = out.as_strided((n, 3), (K + 3, 1), K)
        assert n == 1 or (gap[:-1] == 7).all()


@pytest.mark.parametrize("dtype", list(DT))
def test_gradient_is_the_difference_quotient(dtype):
    """The product is linear in x: the difference of two products along v is
    <dx, v> of the gradient, up to the two roundings of the outputs."""
    n, rows, K = 4, 200, 512
    m, W = matrix(rows, K, 128, seed=1)
    x, v = randn((n, K), DT[dtype], 1), randn((n, K), DT[dtype], 2)
    dy = randn((n, rows), DT[dtype], 3)
    moe = _moe()
    xv = (x.double() + v.double()).to(DT[dtype])
    step = xv.double() - x.double()
    dx = moe.linear_input_grad(dy, *m).double()
    y1, y0 = moe.linear(xv, *m).double(), moe.linear(x, *m).double()
    u = torch.finfo(DT[dtype]).eps / 2
    lhs, rhs = (dy.double() * (y1 - y0)).sum(), (dx * step).sum()
    S = dy.double().abs() @ W.abs()
    tol = (u * (dy.double().abs() * (y1.abs() + y0.abs())).sum()
           + ((2 * u + 1e-4) * S * step.abs()).sum())
    assert (lhs - rhs).abs() <= tol


@pytest.mark.parametrize("n", [1, 8, 40, 300])
def test_values_out_of_the_ordinary(n):
    """Infinities and NaN of one token stay in that token; an overflowing sum
    becomes an infinity, as the formula's rounding has it."""
    rows, K = 150, 640
    m, W = matrix(rows, K, 128, seed=9)
    x = randn((n, K), torch.float16, 5)
    x[0, 3] = float("inf")
    if n > 1:
        x[1, 0] = float("nan")
        x[n - 1] = 60000.0
    y = _moe().linear(x, *m)
    ref = (x.double() @ W.t())
    clean = ref.half()
    assert torch.equal(torch.isnan(y), torch.isnan(clean))
    ok = ~torch.isnan(clean)
    # near the largest fp16 value rounding may go either way
    edge = ref.abs().sub(65520).abs() < 70
    assert torch.equal(torch.isinf(y)[ok & ~edge], torch.isinf(clean)[ok & ~edge])
    # the sign of an infinity is exact; a finite sum within its error bound
    # u S of zero may come out with either sign
    inf = ok & ~edge & torch.isinf(clean)
    assert torch.equal(torch.sign(y)[inf], torch.sign(clean)[inf])
    dy = randn((n, rows), torch.float16, 6)
    dy[0, rows - 1] = float("nan")
    dx = _moe().linear_input_grad(dy, *m)
    assert torch.isnan(dx[0]).all() and torch.isfinite(dx[1:]).all()


@pytest.mark.parametrize("n", [2, 24, 200])
def test_scales_of_zero_and_symmetric_extremes(n):
    """Scales of 0 give a zero product, codes and zero points at both ends of
    their range the exact products."""
    rows, K = 64, 256
    codes = torch.zeros((rows, K // 2), dtype=torch.uint8, device="cuda")
    codes[::2] = 0xFF
    scales = torch.full((rows, 2), 0.5, dtype=torch.float16, device="cuda")
    zeros = torch.zeros((rows, 2), dtype=torch.uint8, device="cuda")
    zeros[:, 1] = 15
    scales[5] = 0
    x = torch.ones((n, K), dtype=torch.float16, device="cuda")
    q = torch.where(torch.arange(rows, device="cuda") % 2 == 0, 15.0, 0.0)
    ref = 128 * 0.5 * (q + (q - 15))
    ref[5] = 0
    assert torch.equal(_moe().linear(x, codes, scales, zeros).float(),
                       ref.expand(n, rows).contiguous())
    dx = _moe().linear_input_grad(x[:, :rows].contiguous(), codes, scales, zeros)
    w = torch.where(torch.arange(K, device="cuda")[None] < 128, q[:, None], q[:, None] - 15) * 0.5
    w[5] = 0
    assert torch.equal(dx.float(), w.sum(0).expand(n, K).contiguous())


@pytest.mark.parametrize("n", [1, 12, 48, 600])
def test_same_bits_streams_and_graphs(n):
    """The same call gives the same bits: again, on another stream, two at
    once, and captured with new inputs under the replay."""
    moe = _moe()
    m, W = matrix(520, 1024, 128, seed=2)
    x, dy = randn((n, 1024), torch.bfloat16, 1), randn((n, 520), torch.bfloat16, 2)
    y, dx = moe.linear(x, *m), moe.linear_input_grad(dy, *m)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):
        for s in (s1, s2):
            outs.append((moe.linear(x, *m, out=torch.empty_like(y), stream=s),
                         moe.linear_input_grad(dy, *m, out=torch.empty_like(dx), stream=s)))
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, y) and torch.equal(b, dx)
    x2, dy2 = randn((n, 1024), torch.bfloat16, 3), randn((n, 520), torch.bfloat16, 4)
    sx, sdy = x.clone(), dy.clone()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        gy = moe.linear(sx, *m)
        gdx = moe.linear_input_grad(sdy, *m)
    sx.copy_(x2)
    sdy.copy_(dy2)
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(gy, moe.linear(x2, *m)) and torch.equal(gdx, moe.linear_input_grad(dy2, *m))


def test_refusals_on_device():
    moe = _moe()
    m, _ = matrix(64, 256, 128, seed=1)
    x = randn((3, 256), torch.float16, 1)
    for call in (lambda: moe.linear(x[:, 1:129], *m), lambda: moe.linear(x.float(), *m),
                 lambda: moe.linear(x.t(), *m), lambda: moe.linear(x[:0], *m),
                 lambda: moe.linear(x, m[0], m[1][:, :1], m[2], 128),
                 lambda: moe.linear(x, m[0].t(), m[1], m[2], 128),
                 lambda: moe.linear(x, *m, bias=x[0, :64].bfloat16()),
                 lambda: moe.linear(x, *m, residual=x[:2, :64]),
                 lambda: moe.linear(x, *m, out=torch.empty((3, 64), device="cuda")),
                 lambda: moe.linear(x, *m, out=x[:, :64]),
                 lambda: moe.linear_input_grad(x, *m)):
        with pytest.raises(moe.MoeError):
            call()


@pytest.mark.parametrize("n,rows,K,group", [
    (3, 48, 65536, 128), (20, 48, 65536, 64), (2, 1 << 20, 32, 32), (40, 1 << 20, 32, 32),
    (524280, 9, 32, 32), (8, 4864, 4352, 64), (5, 19500, 256, 128), (7, 40000, 1024, 32),
])
def test_largest_sizes(n, rows, K, group):
    """Both ends of every range: the longest rows, the most rows, the most
    tokens (dy with odd strides too), several row tiles per CTA."""
    moe = _moe()
    m, W = matrix(rows, K, group, seed=rows + K)
    x = randn((n, K), torch.float16, 1)
    S = x.double().abs() @ W.t().abs()
    check(moe.linear(x, *m), x.double() @ W.t(), S, K, torch.float16)
    dy = randn((n, rows), torch.float16, 2, 0.1)
    ref, S = dy.double() @ W, dy.double().abs() @ W.abs()
    check(moe.linear_input_grad(dy, *m), ref, S, rows, torch.float16)
    if rows % 8:
        check(moe.linear_input_grad(strided(dy, 8 - rows % 8), *m), ref, S, rows, torch.float16)


@pytest.mark.parametrize("n", [4, 12])
def test_offsets_beyond_32_bits(n):
    """Rows far enough apart that element offsets pass 2^32."""
    moe = _moe()
    rows, K = 40, 128
    ld = (1 << 32) // (n - 1) // 8 * 8 + 64
    m, W = matrix(rows, K, 128, seed=1)
    far = torch.empty((n - 1) * ld + K, dtype=torch.float16, device="cuda")
    other = torch.empty((n - 1) * ld + K, dtype=torch.float16, device="cuda")
    x = far.as_strided((n, K), (ld, 1))
    out = other.as_strided((n, rows), (ld, 1))
    x.copy_(randn((n, K), torch.float16, 1))
    got = moe.linear(x, *m, out=out)
    check(got, x.double() @ W.t(), x.double().abs() @ W.t().abs(), K, torch.float16)
    dx = far.as_strided((n, K), (ld, 1))
    want = got.double() @ W
    S = got.double().abs() @ W.abs()
    check(moe.linear_input_grad(got, *m, out=dx), want, S, rows, torch.float16)


def test_results_on_another_stream_are_that_streams_memory():
    """Outputs made for an explicit stream come from its pool: work still
    pending on the current stream cannot own them."""
    moe = _moe()
    m, W = matrix(256, 512, 128, seed=1)
    x = randn((4, 512), torch.float16, 1)
    want, dwant = moe.linear(x, *m), moe.linear_input_grad(x[:, :256].contiguous(), *m)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        junk = torch.full((4, 256), 7.0, dtype=torch.float16, device="cuda")
        busy = torch.randn(2048, 2048, device="cuda")
        for _ in range(4):
            busy = busy @ busy * 1e-3
        junk.mul_(2)            # pending behind the products on the current stream
        del junk
        y = moe.linear(x, *m, stream=side)
        side.synchronize()
        first = y.clone()
        torch.cuda.synchronize()
        assert torch.equal(first, want) and torch.equal(y, want)
    dx = moe.linear_input_grad(x[:, :256].contiguous(), *m, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(dx, dwant)


@pytest.mark.parametrize("n", [9, 40, 700])
def test_gradient_without_a_workspace(n):
    """Unaligned gradients through the C call without the workspace: the same
    product, several passes over the matrix."""
    moe = _moe()
    rows, K = 301, 640
    (codes, scales, zeros, group), W = matrix(rows, K, 128, seed=3)
    dy = randn((n, rows), torch.bfloat16, 2)
    dx = torch.empty((n, K), dtype=torch.bfloat16, device="cuda")
    rc = moe.load_library().moe_linear_input_grad(
        codes.data_ptr(), scales.data_ptr(), zeros.data_ptr(), rows, K, group, dy.data_ptr(), rows,
        n, moe.MOE_BF16, dx.data_ptr(), K, None, 0, None, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    check(dx, dy.double() @ W, dy.double().abs() @ W.abs(), rows, torch.bfloat16)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("n,rows,K,group", [
    (33, 6144, 4096, 64), (200, 4096, 4096, 32), (200, 4096, 4096, 64), (120, 4096, 4096, 128),
    (300, 4096, 2048, 32), (8, 4096, 14336, 64), (3, 9000, 4096, 32),
])
def test_pipelines_at_length(n, rows, K, group, dtype):
    """Long contractions back to back, where every ring turns over many times
    and all SMs compete for memory: each of 30 calls in turn over three sets
    of inputs is within the bounds, and the same inputs give the same bits."""
    moe = _moe()
    sets = []
    for i in range(3):
        m, W = matrix(rows, K, group, seed=i)
        x, dy = randn((n, K), DT[dtype], i), randn((n, rows), DT[dtype], 9 + i, 0.1)
        sets.append((m, x, dy, moe.linear(x, *m), moe.linear_input_grad(dy, *m)))
        check(sets[-1][3], x.double() @ W.t(), x.double().abs() @ W.t().abs(), K, DT[dtype])
        check(sets[-1][4], dy.double() @ W, dy.double().abs() @ W.abs(), rows, DT[dtype])
        del W
    again = [(moe.linear(sets[i % 3][1], *sets[i % 3][0]),
              moe.linear_input_grad(sets[i % 3][2], *sets[i % 3][0])) for i in range(30)]
    for i, (y, dx) in enumerate(again):
        assert torch.equal(y, sets[i % 3][3]) and torch.equal(dx, sets[i % 3][4]), i


@pytest.mark.parametrize("n", [3, 40, 300])
def test_slices_of_one_buffer(n):
    """Input, residual and output as column slices of one buffer."""
    moe = _moe()
    rows, K = 129, 256
    m, _ = matrix(rows, K, 128, seed=9)
    x, res, dy = (randn((n, w), torch.float16, n + w) for w in (K, rows, rows))
    want, dwant = moe.linear(x, *m, residual=res), moe.linear_input_grad(dy, *m)
    buf = torch.full((n, 680), 5.0, dtype=torch.float16, device="cuda")
    xs, rs, ys = buf[:, :K], buf[:, K:K + rows], buf[:, K + rows:K + 2 * rows]
    xs.copy_(x)
    rs.copy_(res)
    moe.linear(xs, *m, residual=rs, out=ys)
    assert torch.equal(xs, x) and torch.equal(rs, res) and torch.equal(ys, want)
    assert (buf[:, K + 2 * rows:] == 5).all()
    ds, xo = buf[:, 3:3 + rows], buf[:, 200:200 + K]
    buf.fill_(5.0)
    ds.copy_(dy)
    moe.linear_input_grad(ds, *m, out=xo)
    assert torch.equal(ds, dy) and torch.equal(xo, dwant)
    with pytest.raises(moe.MoeError):
        moe.linear_input_grad(ds, *m, out=buf[:, 130:130 + K])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("n", [2, 8, 24, 200])
@pytest.mark.parametrize("rows,K,group", [
    (33, 256, 128), (33, 256, 32), (64, 384, 128), (64, 288, 32), (95, 192, 64), (1, 32, 32)])
def test_infinite_scale_of_the_last_group(n, rows, K, group, dtype):
    """An infinite scale in the matrix's last group makes infinities where the
    formula does, and no NaN of the padding behind the last row and column."""
    moe = _moe()
    codes = torch.full((rows, K // 2), 0x99, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, K // group), 0.01, dtype=torch.float16, device="cuda")
    scales[-1, -1] = float("inf")
    zeros = torch.full((rows, K // group), 3, dtype=torch.uint8, device="cuda")
    y = moe.linear(torch.ones((n, K), dtype=DT[dtype], device="cuda"), codes, scales, zeros, group)
    dx = moe.linear_input_grad(torch.ones((n, rows), dtype=DT[dtype], device="cuda"), codes, scales,
                               zeros, group)
    inf = float("inf")
    assert (y[:, -1] == inf).all() and torch.isfinite(y[:, :-1]).all()
    assert (dx[:, K - group:] == inf).all() and torch.isfinite(dx[:, :K - group]).all()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("n,rows,K,group", [
    (2, 1 << 20, 32, 32), (8, 1 << 20, 128, 128), (40, 1 << 20, 32, 32), (300, 1 << 18, 64, 64),
    (3, 48, 65536, 128), (8, 2000, 65536, 32), (20, 48, 65536, 64), (300, 200, 65536, 128),
    (9, 5, 65536, 128), (1, 1 << 20, 256, 64), (524280, 9, 32, 32)])
def test_long_contractions_exactly(n, rows, K, group, dtype):
    """Activations of -1, 0 and 1, scales that are powers of two, so that every
    weight is exact and every partial sum a multiple of the least scale below
    2^24 of it: the output is the rounded exact sum, and a block that is left
    out, read twice or taken from elsewhere shows."""
    moe = _moe()
    g = torch.Generator(device="cuda").manual_seed(rows + K)
    codes = torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    zeros = torch.randint(0, 16, (rows, K // group), dtype=torch.uint8, device="cuda", generator=g)
    # |q - z| <= 15 and 2^20 terms: one scale over the longest contraction
    # (15 * 2^20 < 2^24), two where it is 2^16 long
    exps = torch.zeros((rows, K // group), dtype=torch.int32, device="cuda")
    if max(rows, K) <= 1 << 18:
        exps = torch.randint(0, 2, exps.shape, dtype=torch.int32, device="cuda", generator=g)
    scales = torch.ldexp(torch.full(exps.shape, 2.0 ** -6, device="cuda"), exps).half()
    q = torch.stack((codes & 15, codes >> 4), 2).reshape(rows, K).float()
    W = ((q - zeros.float().repeat_interleave(group, 1))
         * scales.float().repeat_interleave(group, 1))
    for call, width, w in ((moe.linear, K, W.t()), (moe.linear_input_grad, rows, W)):
        x = torch.randint(-1, 2, (n, width), device="cuda", generator=g).to(DT[dtype])
        assert width * 15 * (2 if exps.any() else 1) < 1 << 24
        ref = (x.double() @ w.double()).to(DT[dtype])
        got = call(x, codes, scales, zeros, group)
        assert torch.equal(got, ref), (got != ref).sum()
