"""Edges of the 4-bit operators on the GPU."""
import pytest
import torch

import plain_fp4 as plain
import routing_dispatch_expert_gb300 as rde
from test_gpu_fp4 import built, rng  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("g", [1.0, 1e-2, 1e-4, 1e-6, 1e-10, 1e-16, 1e-19, 1e-30])
def test_quantize_numbers_far_past_the_scale(dtype, g):
    """NVFP4 blocks whose numbers are far beyond 6 * 448 g, up to the type's lowest and largest: the scale and the
    codes saturate, and keep their signs."""
    x = torch.randn(32, 64, generator=rng(1), device="cuda") * g
    x[:, ::7] *= 300
    for row, v in enumerate((1e3, 1e10, 1e15, 1e18, 1e20, 1e25, 1e29, 1e31, 1e35, 3e38)):
        x[row, 3], x[row, 20], x[row, 33], x[row, 34] = v, -v, v, -v / 2
    x = x.clamp(-3e38, 3e38).to(dtype)
    x[12, 5], x[12, 40] = torch.finfo(dtype).min, torch.finfo(dtype).max
    x[13] = torch.finfo(dtype).min
    gt = torch.tensor([g], device="cuda")
    q, s = rde.quantize_fp4(x, "nvfp4", gt)
    rq, rs = plain.quantize(x, "nvfp4", float(gt))
    assert torch.equal(s, rs)
    assert torch.equal(q, rq)
