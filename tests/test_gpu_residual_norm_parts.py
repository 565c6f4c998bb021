"""Gradients of the block norms through one of their two results alone."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from test_gpu_residual_norm import batch  # noqa: E402


def _moe():
    from quantized_expert_ffn_warp_gb300 import moe
    return moe


@pytest.mark.parametrize("n,hid", [(5, 512), (700, 1024), (40, 16384)])
@pytest.mark.parametrize("gate,gain", [("token", True), ("channel", True), (None, False)])
def test_gradient_through_out_alone_reads_no_second_factor(n, hid, gate, gain):
    """Without dxn, whatever the factor of the next block's norm is: infinite for a row of
    zeros without eps, or a NaN."""
    moe = _moe()
    a, rows = batch(n, hid, "bf16", n, gate, gain)
    fwd = moe.residual_norm(**a, scale=0.75, eps=1e-6)
    kw = dict(gain=a["gain"], gate=a["gate"], scale=0.75, next_gain=a["next_gain"])
    dout = rows(0.02)
    want = moe.residual_norm_grad(dout, None, None, a["y"], fwd["stats"], **kw)
    stats = fwd["stats"].clone()
    stats[1, 1], stats[2, 1], stats[3, 1] = float("inf"), float("nan"), -float("inf")
    got = moe.residual_norm_grad(dout, None, None, a["y"], stats, **kw)
    assert got.keys() == want.keys()
    for k, w in want.items():
        assert torch.isfinite(w).all() and torch.equal(got[k], w), k


def test_gradient_through_out_alone_of_a_row_of_zeros():
    moe = _moe()
    a, rows = batch(6, 256, "fp16", 1)
    a["gain"] = a["gate"] = None        # out = resid + y
    a["resid"][2] = 0
    a["y"][2] = 0
    fwd = moe.residual_norm(**a, eps=0.0)
    assert torch.isinf(fwd["stats"][2, 1])
    dout = rows(0.02)
    got = moe.residual_norm_grad(dout, None, None, a["y"], fwd["stats"], next_gain=a["next_gain"])
    assert torch.equal(got["dresid"], dout) and torch.equal(got["dy"], dout)
