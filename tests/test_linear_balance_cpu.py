"""Refusals of the 4-bit products and the routing losses: argument errors come
back as status codes before any CUDA call, so they need no GPU (the pointers
here are never dereferenced)."""
import ctypes as C

import pytest

P, L, Z = C.c_void_p, C.c_longlong, C.c_size_t


@pytest.fixture(scope="module")
def lib():
    from quantized_expert_ffn_warp_gb300 import build, moe
    build.build()
    return moe.load_library()


LIN = dict(codes=0x10000, scales=0x20000, zeros=0x30000, rows=96, cols=256, group=128, x=0x40000,
           ldx=256, n=4, dtype=0, bias=None, residual=None, ldr=0, y=0x50000, ldy=96, status=None)


def linear(lib, **kw):
    a = dict(LIN, **kw)
    return lib.moe_linear(P(a["codes"]), P(a["scales"]), P(a["zeros"]), a["rows"], a["cols"],
                          a["group"], P(a["x"]), L(a["ldx"]), a["n"], a["dtype"], P(a["bias"]),
                          P(a["residual"]), L(a["ldr"]), P(a["y"]), L(a["ldy"]), P(a["status"]),
                          None)


def linear_grad(lib, **kw):
    a = dict(LIN, x=0x40000, ldx=96, y=0x50000, ldy=256, ws=None, ws_bytes=0)
    a.update(kw)
    return lib.moe_linear_input_grad(P(a["codes"]), P(a["scales"]), P(a["zeros"]), a["rows"],
                                     a["cols"], a["group"], P(a["x"]), L(a["ldx"]), a["n"],
                                     a["dtype"], P(a["y"]), L(a["ldy"]), P(a["ws"]), Z(a["ws_bytes"]),
                                     P(a["status"]), None)


BOTH = [
    (dict(codes=None), -1), (dict(scales=None), -1), (dict(zeros=None), -1), (dict(x=None), -1),
    (dict(y=None), -1), (dict(dtype=2), -2), (dict(dtype=-1), -2), (dict(group=16), -2),
    (dict(group=0), -2), (dict(rows=0), -1), (dict(rows=-5), -1), (dict(rows=(1 << 20) + 1), -1),
    (dict(cols=0), -1), (dict(cols=200), -1), (dict(cols=65536 + 128), -1), (dict(n=0), -1),
    (dict(n=-1), -1), (dict(n=(1 << 19) + 1), -1), (dict(ldx=88), -1), (dict(ldy=88), -1),
    (dict(ldy=(1 << 31) + 1), -1), (dict(codes=0x10008), -1), (dict(scales=0x20001), -1),
    (dict(y=0x50001), -1), (dict(status=0x60002), -1), (dict(y=0x40000), -1),
    (dict(y=0x40000 + 64), -1), (dict(group=64, cols=96), -1),
]


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(x=0x40008), -1), (dict(ldx=260), -1), (dict(bias=0x60001), -1),
    (dict(residual=0x60001, ldr=96), -1), (dict(residual=0x60000, ldr=95), -1),
    (dict(residual=0x50000 + 2, ldr=96), -1), (dict(residual=0x50000, ldr=100), -1),
])
def test_linear_refuses(lib, kw, code):
    assert linear(lib, **kw) == code and lib.moe_last_error().decode()


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(x=0x40001), -1),
    (dict(n=20, rows=95, ldx=95, ws=0x80008, ws_bytes=96 * 40), -1),
])
def test_linear_input_grad_refuses(lib, kw, code):
    assert linear_grad(lib, **kw) == code and lib.moe_last_error().decode()


BAL = dict(logits=0x10000, dtype=2, ld=64, n=8, E=64, idx=0x20000, k=2, seq=None, S=1, mask=None,
           loss=0x30000, counts=0x40000, tokens=0x50000, prob=0x60000, lse=0x70000, ws=0x80000,
           ws_bytes=None)


def balance(lib, **kw):
    a = dict(BAL, **kw)
    size = a["ws_bytes"]
    if size is None:
        size = lib.moe_balance_workspace(a["n"], a["E"], a["S"])
    return lib.moe_balance_loss(P(a["logits"]), a["dtype"], L(a["ld"]), a["n"], a["E"],
                                P(a["idx"]), a["k"], P(a["seq"]), a["S"], P(a["mask"]),
                                P(a["loss"]), P(a["counts"]), P(a["tokens"]), P(a["prob"]),
                                P(a["lse"]), P(a["ws"]), Z(size), None)


def balance_grad(lib, **kw):
    a = dict(BAL, dloss=0x90000, w=0xA0000, dw=0xB0000, out=0xC0000, ldd=64)
    a.update(kw)
    return lib.moe_balance_loss_grad(P(a["logits"]), a["dtype"], L(a["ld"]), a["n"], a["E"],
                                     P(a["idx"]), a["k"], P(a["seq"]), a["S"], P(a["mask"]),
                                     P(a["lse"]), P(a["counts"]), P(a["tokens"]), P(a["dloss"]),
                                     P(a["w"]), P(a["dw"]), P(a["out"]), L(a["ldd"]), None)


BATCH = [
    (dict(logits=None), -1), (dict(counts=None), -1), (dict(tokens=None), -1),
    (dict(lse=None), -1), (dict(dtype=3), -2), (dict(n=0), -1), (dict(E=0), -1),
    (dict(E=1025, ld=1025), -1), (dict(k=0), -1), (dict(k=33), -1), (dict(E=1, ld=64, k=2), -1),
    (dict(ld=63), -1), (dict(ld=(1 << 31) + 1), -1), (dict(S=0), -1), (dict(S=2), -1),
    (dict(S=65536, seq=0xD0000), -1), (dict(seq=0xD0002), -1), (dict(logits=0x10002), -1),
    (dict(idx=0x20002), -1), (dict(counts=0x40002), -1), (dict(lse=0x70002), -1),
]


@pytest.mark.parametrize("kw,code", BATCH + [
    (dict(idx=None), -1), (dict(loss=None), -1), (dict(prob=None), -1), (dict(ws=None), -1),
    (dict(ws=0x80080), -1), (dict(ws_bytes=0), -1), (dict(ws_bytes=1000), -1),
])
def test_balance_loss_refuses(lib, kw, code):
    assert balance(lib, **kw) == code and lib.moe_last_error().decode()


@pytest.mark.parametrize("kw,code", BATCH + [
    (dict(dloss=None), -1), (dict(out=None), -1), (dict(w=None), -1), (dict(idx=None), -1),
    (dict(ldd=63), -1), (dict(ldd=(1 << 31) + 1), -1), (dict(out=0x10000 + 64), -1),
    (dict(out=0x10000, ldd=128), -1), (dict(dloss=0x90001), -1), (dict(dw=0xB0002), -1),
    (dict(w=0xA0002), -1),
])
def test_balance_loss_grad_refuses(lib, kw, code):
    assert balance_grad(lib, **kw) == code and lib.moe_last_error().decode()


@pytest.mark.parametrize("at,overlaps", [
    (0, False), (64, False), (60, True), (136, False), (137, True), (-64, False), (-63, True),
    (4 * 200 + 64, False), (7 * 200 + 30, True), (7 * 200 + 64, False), (-7 * 200 - 64, False),
    (-7 * 200 - 63, True)])
def test_column_slices_of_one_buffer_do_not_overlap(lib, at, overlaps):
    """Rows of 64 in a buffer of stride 200, `at` elements from one slice to
    the other (0: in place).  What does not overlap is refused for its device."""
    rc = balance_grad(lib, logits=0x20000, out=0x20000 + 4 * at, ld=200, ldd=200, n=8)
    assert rc != 0 and ("overlap" in lib.moe_last_error().decode()) == overlaps


def test_linear_input_grad_workspace_sizes(lib):
    ws = lib.moe_linear_input_grad_workspace
    assert ws(96, 8, P(0x40002), L(97)) == 0 and ws(96, 20, P(0x40000), L(96)) == 0
    assert ws(97, 20, P(0x40000), L(97)) == 20 * 104 * 2
    assert ws(96, 20, P(0x40002), L(96)) == 20 * 96 * 2
    assert ws(0, 20, P(0x40002), L(97)) == 0 and ws(97, 1 << 20, P(0x40002), L(97)) == 0


def test_balance_workspace_sizes(lib):
    ws = lib.moe_balance_workspace
    assert ws(0, 8, 1) == 0 and ws(8, 0, 1) == 0 and ws(8, 8, 0) == 0 and ws(8, 1025, 1) == 0
    assert ws(8, 8, 65536) == 0
    assert 0 < ws(1, 1, 1) <= ws(64, 64, 1) <= ws(65536, 1024, 300)


def test_binding_refuses_wrong_tensors():
    """Shapes, types, strides and devices are checked before an address is
    taken: CPU tensors are refused like any other wrong tensor."""
    torch = pytest.importorskip("torch")
    from quantized_expert_ffn_warp_gb300 import moe
    codes = torch.zeros((8, 64), dtype=torch.uint8)
    scales, zeros = torch.zeros((8, 1), dtype=torch.float16), torch.zeros((8, 1), dtype=torch.uint8)
    x = torch.zeros((2, 128), dtype=torch.float16)
    for call in (lambda: moe.linear(x, codes, scales, zeros),
                 lambda: moe.linear(x, codes, scales, zeros, 48),
                 lambda: moe.linear(x, codes[0], scales, zeros),
                 lambda: moe.linear_input_grad(x[:, :8], codes, scales, zeros),
                 lambda: moe.balance_loss(x.float(), torch.zeros((2, 1), dtype=torch.int32)),
                 lambda: moe.balance_loss(x.float(), None),
                 lambda: moe.balance_loss(x.double(), torch.zeros((2, 1), dtype=torch.int32))):
        with pytest.raises(moe.MoeError):
            call()


def test_gradient_without_ids_needs_top_k(monkeypatch):
    """The counts' scale E / (k T) needs k: without ids it has to be given, and
    it reaches the library; with ids it has to agree with them."""
    torch = pytest.importorskip("torch")
    from quantized_expert_ffn_warp_gb300 import moe
    seen = []

    class Lib:
        def moe_balance_loss_grad(self, *a):
            seen.append((a[5], a[6]))
            return 0

    monkeypatch.setattr(moe, "load_library", Lib)
    monkeypatch.setattr(moe, "_raw_stream", lambda t, stream: 0)
    logits, idx = torch.zeros((6, 8)), torch.zeros((6, 3), dtype=torch.int32)
    fwd = dict(lse=torch.zeros(6), counts=torch.zeros((1, 8), dtype=torch.int32),
               tokens=torch.zeros(1, dtype=torch.int32))
    dloss = torch.zeros(2)
    with pytest.raises(moe.MoeError, match="top_k"):
        moe.balance_loss_grad(logits, None, fwd, dloss)
    with pytest.raises(moe.MoeError, match="top_k"):
        moe.balance_loss_grad(logits, idx, fwd, dloss, top_k=2)
    assert not seen
    moe.balance_loss_grad(logits, None, fwd, dloss, top_k=3)
    moe.balance_loss_grad(logits, idx, fwd, dloss)
    moe.balance_loss_grad(logits, idx, fwd, dloss, top_k=3)
    assert seen == [(None, 3), (idx.data_ptr(), 3), (idx.data_ptr(), 3)]


def _overlaps(lib, rc):
    return rc == -1 and "overlap" in lib.moe_last_error().decode()


W = 96 * 128          # bytes of the codes of LIN, of which y's 4 rows take 768


@pytest.mark.parametrize("kw,overlaps", [
    (dict(bias=0x50000), True), (dict(bias=0x50000 + 766), True), (dict(bias=0x50000 + 768), False),
    (dict(bias=0x50000 - 192), False), (dict(bias=0x50000 - 190), True),
    (dict(bias=0x50000 + 192, ldy=192), False), (dict(bias=0x50000 + 194, ldy=192), True),
    (dict(bias=0x50000 + 190, ldy=192), True), (dict(y=0x10000), True),
    (dict(y=0x10000 + W - 2), True), (dict(y=0x10000 + W), False), (dict(y=0x20000 + 382), True),
    (dict(y=0x20000 + 384), False), (dict(y=0x30000 - 766), True), (dict(y=0x30000 - 768), False),
    (dict(status=0x50000 + 764), True), (dict(status=0x50000 + 768), False)])
def test_linear_output_overlaps(lib, kw, overlaps):
    """y against the matrix, the bias and the status word; a bias may lie in the
    gaps between y's rows.  What does not overlap is refused for its device."""
    rc = linear(lib, **kw)
    assert rc != 0 and _overlaps(lib, rc) == overlaps


COPY = dict(n=20, rows=95, ldx=95, ws=0x80000, ws_bytes=96 * 40)


@pytest.mark.parametrize("kw,overlaps", [
    (dict(), False), (dict(ws=0x40000), True), (dict(ws=0x40000 + 3792), True),
    (dict(ws=0x40000 + 3808), False), (dict(ws=0x40000 - 96 * 40), False),
    (dict(ws=0x40000 - 96 * 40 + 16), True), (dict(ws=0x50000 + 16), True),
    (dict(ws=0x50000 + 20 * 512), False), (dict(ws=0x10000 + 95 * 128 - 16), True),
    (dict(ws=0x10000 + 95 * 128), False), (dict(ws=0x20000 + 368), True),
    (dict(ws=0x30000 + 176), True), (dict(ws=0x60000, status=0x60000 + 96 * 40 - 4), True),
    (dict(ws=0x60000, status=0x60000 + 96 * 40), False),
    # one that is too small, or not needed, is not used
    (dict(ws=0x40000, ws_bytes=96 * 40 - 1), False), (dict(ws=0x40000, ldx=96), False)])
def test_linear_input_grad_workspace_overlaps(lib, kw, overlaps):
    rc = linear_grad(lib, **dict(COPY, **kw))
    assert rc != 0 and _overlaps(lib, rc) == overlaps


@pytest.mark.parametrize("kw,overlaps", [
    (dict(), False), (dict(ws=0x10000), True), (dict(ws=0x10000 + 2048), False),
    (dict(ws=0x20000), True), (dict(ws=0x30000), True), (dict(ws=0x40000), True),
    (dict(ws=0x50000), True), (dict(ws=0x60000), True), (dict(ws=0x70000), True),
    (dict(ws=0x90000, mask=0x90000 + 7), True), (dict(ws=0x90000, seq=0x90004), True),
    (dict(lse=0x10000), True), (dict(lse=0x20000 + 60), True), (dict(lse=0x20000 + 64), False),
    (dict(prob=0x40000 + 252), True), (dict(prob=0x40000 + 256), False),
    (dict(loss=0x50000), True), (dict(tokens=0x30000 + 4), True), (dict(tokens=0x30000 + 8), False),
    (dict(lse=0x10000 + 256, ld=96), False), (dict(lse=0x10000 + 352, ld=96), False),
    (dict(lse=0x10000 + 356, ld=96), True), (dict(counts=0x10000 + 512, ld=192), False),
    (dict(counts=0x10000 + 516, ld=192), True)])
def test_balance_loss_overlaps(lib, kw, overlaps):
    """The workspace and the outputs against everything; an output may lie in
    the gaps between the logits' rows."""
    rc = balance(lib, **kw)
    assert rc != 0 and _overlaps(lib, rc) == overlaps


@pytest.mark.parametrize("shape", [(0,), (1,), ()])
def test_binding_refuses_offsets_without_a_segment(shape):
    torch = pytest.importorskip("torch")
    from quantized_expert_ffn_warp_gb300 import moe
    seq = torch.zeros(shape, dtype=torch.int32)
    logits, idx = torch.zeros((2, 4)), torch.zeros((2, 1), dtype=torch.int32)
    with pytest.raises(moe.MoeError, match="seq_offsets"):
        moe.balance_loss(logits, idx, seq)
    with pytest.raises(moe.MoeError, match="seq_offsets"):
        moe.balance_loss_grad(logits, idx, {}, torch.zeros(2), seq_offsets=seq)
