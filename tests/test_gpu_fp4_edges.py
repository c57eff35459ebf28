"""Edges of the 4-bit operators on the GPU."""
import pytest
import torch

import plain_fp4 as plain
import routing_dispatch_expert_gb300 as rde
from test_gpu_fp4 import FORMATS, built, operand, product_tolerance, rng  # noqa: F401

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


def test_matmul_with_more_than_2_29_columns():
    """Every column of a product whose rows are longer than 2^31 bytes is written (11 GB of operands and output)."""
    N, K = (1 << 29) + 256, 32
    aq = torch.full((1, K // 2), 0x22, dtype=torch.uint8, device="cuda")  # ones
    bq = torch.full((N, K // 2), 0x22, dtype=torch.uint8, device="cuda")
    bq[0], bq[12345], bq[-1] = 0x44, 0x33, 0x55  # 2, 1.5 and 3
    one = lambda n: torch.full((n, 1), 127, dtype=torch.uint8, device="cuda")  # noqa: E731
    y = torch.full((1, N), float("nan"), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rde.matmul_fp4(aq, one(1), bq, one(N), "mxfp4", y=y, status=status)
    assert int(status) == 0
    assert (float(y[0, 0]), float(y[0, 12345]), float(y[0, -1])) == (64.0, 48.0, 96.0)
    assert int((y != 32).sum()) == 3


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(128, 7168, 512), (128, 9728, 256), (128, 9729, 256), (256, 4864, 288), (256, 4865, 288),
                                   (384, 3200, 256), (127, 9728, 256), (129, 4864, 256)])
def test_matmul_of_whole_row_tiles(fmt, M, N, K):
    """Whole 128-row tiles on both sides of where all narrow tiles run at once."""
    aq, a_s, ga, a = operand(M, K, fmt, 1)
    bq, b_s, gb, b = operand(N, K, fmt, 2, 0.02)
    ref, mag = a @ b.T, a.abs() @ b.abs().T
    for dtype in (torch.bfloat16, torch.float32):
        y = rde.matmul_fp4(aq, a_s, bq, b_s, fmt, ga, gb, dtype=dtype)
        assert (y.double() - ref).abs().sub(product_tolerance(ref, mag, K, dtype)).amax() <= 0


def rounded(v, dtype):
    """fp64 numbers rounded once, to nearest even, to a 16-bit type."""
    bits, least, most = {torch.bfloat16: (8, -133, torch.finfo(torch.bfloat16).max),
                         torch.float16: (11, -24, 65504.0)}[dtype]
    e = torch.frexp(v)[1] - bits  # the last bit of v's binade
    step = torch.pow(2.0, e.clamp(min=least).double())
    r = torch.round(v / step) * step
    return torch.where(r.abs() > most, torch.copysign(torch.full_like(r, float("inf")), r), r)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_dequantize_rounds_once(dtype):
    """code * scale * g for every code and scale, and matrix scales g for which rounding to fp32 first gives another
    16-bit number (found here by trying), and very small and large ones."""
    code = torch.arange(16, dtype=torch.uint8)
    q = (code.repeat(2)[::2] | code.repeat(2)[1::2] << 4).repeat(127, 1)  # a row: codes 0 .. 15 twice
    s = torch.arange(127, dtype=torch.uint8).unsqueeze(1).repeat(1, 2)
    unit = plain.values(q, s, "nvfp4", 1.0)
    gen = torch.Generator().manual_seed(4)
    tried = torch.rand(400000, generator=gen) + 0.5
    parts = torch.unique(torch.frexp(unit)[0].abs())  # the same up to a power of two
    v = tried.double().unsqueeze(1) * parts
    differ = tried[(v.float().to(dtype).double() != rounded(v, dtype)).any(1)].tolist()
    assert len(differ) > 5
    smallest = [float(torch.tensor(v)) for v in (3e-5, 1e-9, 1.37e-36, 5e-38, 3e-39, 2.7e-41, 1.1e30)]
    for g in differ[:40] + smallest:
        got = rde.dequantize_fp4(q.cuda(), s.cuda(), "nvfp4", torch.tensor([g], device="cuda"), dtype=dtype)
        assert torch.equal(got.cpu().double(), rounded(unit * g, dtype)), g


def test_a_wait_that_gives_up_is_reported_without_a_status_word():
    """The word that products without one record in: read and cleared, and untouched by products that end well."""
    aq, a_s, ga, _ = operand(40, 256, "nvfp4", 1)
    rde.matmul_fp4_status()
    y = rde.matmul_fp4(aq, a_s, aq, a_s, "nvfp4", ga, ga)
    assert rde.matmul_fp4_status() == 0
    cfg = rde.make_config(T=8, h=256, E=8, k=2, I=256, dtype="nvfp4")
    rde.selftest_wait_timeout(cfg, None, 1_000_000)  # about half a millisecond of SM clock
    assert torch.equal(rde.matmul_fp4(aq, a_s, aq, a_s, "nvfp4", ga, ga), y)
    assert rde.matmul_fp4_status() == rde.moe.MOE_STATUS_WAIT_TIMEOUT
    assert rde.matmul_fp4_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_matmul_of_very_long_rows(fmt):
    """2^25 + 32 elements a row, 131073 K blocks: whole numbers at both ends and at the seams, so that sums are exact."""
    K, M, N = (1 << 25) + 32, 3, 70
    one = 0x38 if fmt == "nvfp4" else 127
    scales = lambda n: torch.full((n, K // plain.BLOCK[fmt]), one, dtype=torch.uint8, device="cuda")  # noqa: E731
    aq = torch.zeros(M, K // 2, dtype=torch.uint8, device="cuda")
    bq = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    bq[:] = 0x24  # 2, 1, 2, 1 ..
    at = [0, 127, 128, 1 << 16, (1 << 24) - 1, K // 2 - 16, K // 2 - 1]  # bytes: elements 2 i and 2 i + 1
    for m in range(M):
        for i in at[:len(at) - m]:
            aq[m, i] = 0x42  # 1, 2
    y = rde.matmul_fp4(aq, scales(M), bq, scales(N), fmt, dtype=torch.float32)
    assert rde.matmul_fp4_status() == 0
    for m in range(M):
        assert (y[m] == 4.0 * (len(at) - m)).all()
