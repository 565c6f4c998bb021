"""Token log probabilities and their gradient where the largest logit of a row, or of
a thread's first values, is far from 0: the fill of a mask, or logits of any size.
The bounds are those of tuning_refs.py, derived there for every finite logit."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from test_gpu_logprobs import batch, check  # noqa: E402
from tuning_refs import DT, H, half_step, logprobs, logprobs_grad  # noqa: E402

FAR = [-1e10, 1e10, -3e9, -1e9, 1e20, -1e30, 2.0 ** 21, -(2.0 ** 99)]


def _moe():
    from quantized_expert_ffn_warp_gb300 import moe
    return moe


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


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("fill", FAR)
@pytest.mark.parametrize("where", ["all", "but_one", "first", "last"])
@pytest.mark.parametrize("which", ["logp", "entropy", "both"])
@pytest.mark.parametrize("n,V", [(3, 32003), (300, 8193)])
def test_gradient(n, V, dtype, fill, where, which):
    logits, targets = batch(n, V, dtype, 12, pad=1)
    logits = masked(logits, fill, where)
    g = torch.Generator(device="cuda").manual_seed(5)
    dlogp = torch.randn(n, device="cuda", generator=g) if which != "entropy" else None
    dent = torch.randn(n, device="cuda", generator=g) if which != "logp" else None
    ref = logprobs(logits, targets)
    fwd = dict(stats=ref["stats"].float(), entropy=ref["entropy"].float())
    # where the largest logit m is far, l - m comes first: no term of m's own size in the
    # bound.  Elsewhere the rest of m log2 e behind its fp32 value is rounded at H^2 m, as
    # tuning_refs.py counts it (it shows where p = 1 and the entropy is 0: the gradient is 0).
    m = ref["stats"][:, 0]
    near = dict(ref, stats=torch.stack((torch.where(m.abs() > 2.0 ** 20, 0.0, m),
                                        ref["stats"][:, 1]), 1))
    want, err = logprobs_grad(logits, targets, near, dlogp, dent)
    got = _moe().token_logprobs_grad(logits, targets, fwd, dlogp, dent)
    assert ((got.double() - want).abs() <= err + half_step(want, DT[dtype])).all()
    _moe().token_logprobs_grad(logits, targets, fwd, dlogp, dent, out=logits)
    assert torch.equal(logits, got)


def test_a_row_of_gradients_sums_to_its_target_in_flat_rows():
    """sum_v p_v of a wide, flat row from the statistics that the gradient is given.

    Errors that all of a row's values share do not average out: of 2^x 4 H (2 units in
    the last place) for each value and 4 H for the row's factor; the rounded log2 e
    scales l - m, below 0.2 * 2^-25.  What differs from value to value (half a step
    of an argument below 32, 2^-20 ln 2 = 11.1 H, and two roundings) averages to below H
    over 160001 values.  10 H in all.  What is left of the row's constant
    (m + logsum) log2 e behind its fp32 value, at logsum log2 e > 16, is up to 11.1 H."""
    n, V = 512, 160001
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = 0.02 * torch.randn((n, V), device="cuda", generator=g)
    logits += torch.linspace(0.5, 4.0, n, device="cuda")[:, None]
    ref = logprobs(logits, None)
    stats = ref["stats"].float()
    assert (ref["stats"][:, 1] > 11.5).all()
    del ref
    targets = torch.zeros(n, dtype=torch.int32, device="cuda")
    ones = torch.ones(n, device="cuda")
    got = _moe().token_logprobs_grad(logits, targets, dict(stats=stats), ones)
    p = (logits.double() - stats[:, :1].double() - stats[:, 1:].double()).exp()
    want = p[:, 1:].sum(1)
    off = (got[:, 1:].double().sum(1) + want).abs() / want / H
    assert off.max() <= 10, off.max()
