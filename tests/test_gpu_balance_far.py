"""Balance loss and gradient where every logit of a row is far from zero, as a large negative number in masked places
leaves them: the probabilities go by the differences alone."""
import pytest
import torch

from test_gpu_balance_loss import built, check, config, inputs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E", [8, 130, 256])
def test_rows_far_from_zero(score, dtype, E):
    """Rows around +-c for c from 1e5 to past 1e30: all the same, and a step of the type apart in some places. The
    tolerances are those of any other logits (exponents beyond 90 have no probability left)."""
    T, k = 96, 2
    logits, idx, _, _ = inputs(T, E, k, dtype, seed=E)
    gen = torch.Generator(device="cuda").manual_seed(1)
    centres = [1e5, 1e6, 3e6, 1e7, 1e8, 1e9, 3e9, 1e10, 7e12, 1e20, 9e29, 2e30]
    row = 0
    for c in centres:
        for sign in (-1.0, 1.0):
            z = torch.full((E,), sign * c, dtype=dtype, device="cuda")
            logits[row] = z
            up = torch.nextafter(z.float(), torch.full_like(z.float(), float("inf"))).to(dtype)
            pick = torch.rand(E, generator=gen, device="cuda") < 0.3
            logits[row + 1] = torch.where(pick, up, z)
            row += 2
    check(config(T, E, k, score), logits, idx, None, None, score, torch.ones(1, device="cuda"))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("mask_value", [-1e4, -1e9, -1e10, -1e20, -3e29])
def test_rows_masked_with_a_large_number(score, mask_value):
    """A row whose experts are all masked is even; with one expert left it has all of the probability."""
    T, E, k = 40, 16, 2
    logits, idx, _, _ = inputs(T, E, k, torch.float32)
    logits[3] = mask_value
    logits[7, 1:] = mask_value
    out, d = check(config(T, E, k, score), logits, idx, None, None, score, torch.ones(1, device="cuda"))
    assert torch.isfinite(out["loss"]).all() and torch.isfinite(d).all()
    assert abs(float(out["mean_prob"].sum()) - 1) < 1e-5
