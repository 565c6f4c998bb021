"""Adapters of many requests and their gradients against 64-bit definitions; the
bounds are derived in tuning_refs.py."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from tuning_refs import DT, adapter, adapter_grad, half_step  # noqa: E402


def _moe():
    from quantized_expert_ffn_warp_gb300 import moe
    return moe


def case(n, cols, rows, rank, count, dtype, seed=0, kind="random", scaled=True, base=True, pad=0,
         lead=0):
    g = torch.Generator(device="cuda").manual_seed(seed + n + cols + rows)
    dt = DT[dtype]

    def wide(w, scale=1.0):
        t = torch.randn((n, w + pad + lead), device="cuda", generator=g) * scale
        return t.to(dt)[:, lead:lead + w]
    ids = torch.randint(-1, count + 1, (n,), device="cuda", generator=g).to(torch.int32)
    if kind == "runs":
        ids = torch.sort(ids).values.flip(0).contiguous()
    elif kind == "one":
        ids[:] = count - 1
    elif kind == "none":
        ids[:] = torch.where(ids >= 0, -5, count + 7)
    return dict(x=wide(cols), ids=ids,
                A=(torch.randn((count, rank, cols), device="cuda", generator=g) / cols ** 0.5).to(dt),
                B=(torch.randn((count, rows, rank), device="cuda", generator=g) * 0.1).to(dt),
                scale=torch.rand(count, device="cuda", generator=g) + 0.5 if scaled else None,
                base=wide(rows) if base else None), wide


def check(c, wide, backward=True):
    moe = _moe()
    dt, n = c["x"].dtype, c["x"].shape[0]
    out, h = moe.adapter(**c)
    (ro, oe), (rh, he) = adapter(**c)
    assert ((out.double() - ro).abs() <= oe + half_step(ro, dt)).all()
    assert ((h.double() - rh).abs() <= he + half_step(rh, dt)).all()
    off = (c["ids"] < 0) | (c["ids"] >= c["A"].shape[0])
    assert (h[off] == 0).all()
    assert torch.equal(out[off], c["base"][off] if c["base"] is not None
                       else torch.zeros_like(out[off]))
    if not backward:
        return out, h
    dy = wide(c["B"].shape[1], 0.02)
    base = wide(c["A"].shape[2], 0.02) if c["base"] is not None else None
    a = (dy, c["x"], h, c["ids"], c["A"], c["B"], c["scale"], base)
    got = moe.adapter_grad(*a)
    for k, (w, e) in adapter_grad(*a).items():
        assert got[k].shape == w.shape
        assert ((got[k].double() - w).abs() <= e + half_step(w, dt)).all(), k
    return out, h, a, got


SIZES = [(1, 8, 8, 8, 1), (1, 2048, 2048, 16, 64), (3, 64, 96, 24, 2), (13, 2048, 512, 16, 64),
         (64, 512, 512, 32, 1), (65, 4096, 768, 64, 3), (200, 256, 1024, 40, 5),
         (333, 1000, 264, 128, 7), (300, 2048, 1024, 8, 3), (1500, 640, 520, 48, 1000),
         (4001, 320, 448, 64, 16), (2500, 1280, 96, 112, 2)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n,cols,rows,rank,count", SIZES)
@pytest.mark.parametrize("kind", ["random", "runs"])
def test_sizes(n, cols, rows, rank, count, dtype, kind):
    c, wide = case(n, cols, rows, rank, count, dtype, kind=kind)
    check(c, wide)


@pytest.mark.parametrize("kind", ["one", "none"])
@pytest.mark.parametrize("n", [1, 31, 700])
@pytest.mark.parametrize("scaled,base", [(True, False), (False, True), (False, False)])
def test_one_adapter_or_none(n, kind, scaled, base):
    c, wide = case(n, 384, 320, 16, 4, "bf16", kind=kind, scaled=scaled, base=base)
    out, h, a, got = check(c, wide)
    if kind == "none":
        assert (got["dA"] == 0).all() and (got["dB"] == 0).all()
    else:
        assert (got["dA"][:3] == 0).all() and (got["dB"][3] != 0).any()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n,cols,rows,rank,pad,lead", [
    (1, 1, 1, 8, 0, 0), (5, 33, 31, 8, 0, 0), (70, 1027, 999, 24, 0, 0), (150, 515, 2050, 64, 3, 5),
    (40, 256, 512, 16, 8, 8), (300, 100, 60, 128, 4, 4), (9, 4095, 32003, 32, 1, 0)])
def test_odd_widths_and_strides(n, cols, rows, rank, pad, lead, dtype):
    c, wide = case(n, cols, rows, rank, 3, dtype, pad=pad, lead=lead)
    check(c, wide)


@pytest.mark.parametrize("n,rows", [(20, 256), (500, 257)])
def test_in_place_and_parts(n, rows):
    """out over base, dx over its base, and each gradient by itself."""
    moe = _moe()
    c, wide = case(n, 512, rows, 16, 5, "bf16")
    out, h, a, got = check(c, wide)
    room = torch.full((n, rows + 40), 3.0, dtype=torch.bfloat16, device="cuda")
    room[:, 8:8 + rows] = c["base"]
    again, _ = moe.adapter(**dict(c, base=room[:, 8:8 + rows], out=room[:, 8:8 + rows]))
    assert torch.equal(again, out) and (room[:, :8] == 3).all() and (room[:, 8 + rows:] == 3).all()
    only = moe.adapter_grad(*a[:-1], base=None, input_grad=False)
    assert set(only) == {"dA", "dB"}
    assert torch.equal(only["dA"], got["dA"]) and torch.equal(only["dB"], got["dB"])
    dx = a[-1].clone()
    only = moe.adapter_grad(a[0], None, None, *a[3:7], base=dx, out=dx, weight_grad=False)
    assert set(only) == {"dx"} and only["dx"] is dx and torch.equal(dx, got["dx"])


@pytest.mark.parametrize("n", [7, 400])
def test_values_that_are_not_finite_stay_with_their_token(n):
    moe = _moe()
    c, wide = case(n, 256, 320, 16, 2, "fp16", kind="one")
    c["x"][3] = float("nan")
    c["x"][5, 0] = float("inf")
    out, h = moe.adapter(**c)
    rest = [i for i in range(n) if i not in (3, 5)]
    assert torch.isnan(out[3]).all() and torch.isfinite(out[rest]).all()
    assert not torch.isfinite(h[5]).any() and torch.isfinite(h[rest]).all()
    # an adapter's values reach its own tokens and gradients only
    c, wide = case(n, 256, 320, 16, 3, "bf16")
    c["A"][1], c["B"][1] = float("nan"), float("inf")
    dy = wide(320, 0.02)
    out, h = moe.adapter(**c)
    got = moe.adapter_grad(dy, c["x"], h, c["ids"], c["A"], c["B"], c["scale"])
    rest = c["ids"] != 1
    assert torch.isfinite(out[rest]).all() and torch.isfinite(got["dx"][rest]).all()
    for k in ("dA", "dB"):
        assert torch.isfinite(got[k][[0, 2]]).all()


@pytest.mark.parametrize("n", [5, 900])
def test_same_bits_on_other_streams_and_in_graphs(n):
    moe = _moe()
    c, wide = case(n, 1024, 768, 32, 6, "bf16")
    dy = wide(768, 0.02)

    def both(x, stream=None):
        out, h = moe.adapter(**dict(c, x=x), stream=stream)
        g = moe.adapter_grad(dy, x, h, c["ids"], c["A"], c["B"], c["scale"], stream=stream)
        return [out, h, g["dx"], g["dA"], g["dB"]]
    first = both(c["x"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    again = both(c["x"], side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, again))
    static, pool, graphs = c["x"].clone(), torch.cuda.graph_pool_handle(), []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            res = both(static)
        graphs.append((g, res))
    for turn in range(4):
        static.copy_(wide(1024))
        g, res = graphs[turn % 2]
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(res, both(static)))


def test_tokens_in_any_order_get_the_same_rows():
    """A token's result does not depend on the others of the call."""
    moe = _moe()
    c, _ = case(600, 512, 512, 16, 9, "bf16")
    out, h = moe.adapter(**c)
    p = torch.randperm(600, device="cuda")
    moved = dict(c, x=c["x"][p].contiguous(), ids=c["ids"][p].contiguous(),
                 base=c["base"][p].contiguous())
    o2, h2 = moe.adapter(**moved)
    assert torch.equal(o2, out[p]) and torch.equal(h2, h[p])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n,cols,rows,rank,count", [(2500, 777, 900, 24, 700),
                                                    (1900, 1024, 1000, 8, 1024),
                                                    (4000, 896, 520, 72, 400)])
def test_many_adapters_of_unequal_size(n, cols, rows, rank, count, dtype):
    # from one to several hundred tokens an adapter, many of them with none
    c, wide = case(n, cols, rows, rank, count, dtype)
    g = torch.Generator(device="cuda").manual_seed(n)
    c["ids"] = (torch.rand(n, device="cuda", generator=g) ** 6 * (count + 3)).int() - 1
    check(c, wide)


def test_offsets_beyond_32_bits():
    moe = _moe()
    n, rows = 70000, 32768
    c, _ = case(8, 64, rows, 8, 2, "bf16", kind="one")
    x = torch.zeros((n, 64), dtype=torch.bfloat16, device="cuda")
    base = torch.zeros((n, rows), dtype=torch.bfloat16, device="cuda")
    ids = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    x[-8:], base[-8:], ids[-8:] = c["x"], c["base"], c["ids"]
    small, _ = moe.adapter(**c)
    out, h = moe.adapter(x, ids, c["A"], c["B"], c["scale"], base=base, out=base)
    assert torch.equal(out[-8:], small) and (out[:-8] == 0).all()
    g = moe.adapter_grad(out, x, h, ids, c["A"], c["B"], c["scale"])
    want = adapter_grad(small, c["x"], h[-8:], c["ids"], c["A"], c["B"], c["scale"], None)
    for k, (w, e) in want.items():
        v = (g[k][-8:] if k == "dx" else g[k]).double()
        assert ((v - w).abs() <= e + half_step(w, small.dtype)).all(), k
    assert (g["dx"][:-8] == 0).all()


def test_refusals():
    moe = _moe()
    c, wide = case(4, 64, 32, 8, 2, "bf16")
    for bad in (dict(ids=c["ids"].cpu()), dict(ids=c["ids"][:3]), dict(A=c["A"][:, :4]),
                dict(B=c["B"].half()), dict(out=c["x"]), dict(scale=c["scale"].double()),
                dict(base=c["base"].t())):
        with pytest.raises(moe.MoeError):
            moe.adapter(**dict(c, **bad))
    odd = torch.zeros((2, 12, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(moe.MoeError, match="rank"):
        moe.adapter(c["x"], c["ids"], odd, odd.transpose(1, 2).contiguous())
