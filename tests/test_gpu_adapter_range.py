"""Adapters where h and u, the products between the two matrices, are not finite."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from tuning_refs import DT  # noqa: E402

INF = float("inf")


def _moe():
    from quantized_expert_ffn_warp_gb300 import moe
    return moe


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
