"""Token log probabilities where the largest logit of a row, or of
a thread's first values, is far from 0: the fill of a mask, or logits of any size.
The bounds are those of tuning_refs.py, derived there for every finite logit."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from test_gpu_logprobs import batch, check  # noqa: E402

FAR = [-1e10, 1e10, -3e9, -1e9, 1e20, -1e30, 2.0 ** 21, -(2.0 ** 99)]


def masked(logits, fill, where):
    """logits with `fill` in all columns, all but one, the first 8192 or the last."""
    logits = logits.clone()
    if where == "all":
        logits[:] = fill
    elif where == "but_one":
        keep = logits[:, 99].clone()
        logits[:] = fill
        logits[:, 99] = keep
    elif where == "first":
        logits[:, :8192] = fill
    else:
        logits[:, -1] = fill
    return logits


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("fill", FAR)
@pytest.mark.parametrize("where", ["all", "but_one", "first", "last"])
@pytest.mark.parametrize("n,V", [(2, 32003), (620, 32003), (620, 8001)])
def test_forward(n, V, dtype, fill, where):
    if where == "first" and V < 9000:
        pytest.skip("the columns are all of the row's")
    logits, targets = batch(n, V, dtype, 11)
    logits = masked(logits, fill, where)
    targets = targets.clamp(0, V - 1)
    targets[0], targets[1] = 99, V - 1
    check(logits, targets, 5)
    check(logits, targets, 0)
