"""Scales of 8-bit products at the ends of fp32's range: the two scales of a block are
multiplied first, by the definition."""

import pytest

import strided_gemm_gb300 as sg
from tests.test_layers_gpu import clean_status, gen, torch  # noqa: F401
from tests.test_serving_gpu import status_is

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(70, 260, 384), (70, 260, 380), (300, 520, 640), (16, 1024, 2048), (70, 260, 75)])
@pytest.mark.parametrize("gb", [1, 128])
def test_products_of_scales(torch, M, N, K, gb):
    """Small whole numbers times powers of two: every step is exact, a subnormal product
    of scales among them, as long as it is a power of two and sums stay below 2^13 of it."""
    g = gen(torch, 6)
    f8 = torch.float8_e4m3fn

    def operand(rows):
        wide = torch.zeros(rows, K if K % 16 else K + 16, device="cuda").to(f8)[:, :K]       # 75: the kernel without maps
        wide.copy_(torch.randint(1, 3, (rows, K), generator=g, device="cuda").float().to(f8))
        return wide

    A, B = operand(M), operand(N)
    s, C = A.double() @ B.double().t(), torch.empty(M, N, device="cuda")

    def product(a, b, alpha):
        SA = torch.full((M, -(-K // 128)), 2.0 ** a, device="cuda")
        SB = torch.full((-(-N // gb), -(-K // 128)), 2.0 ** b, device="cuda")
        return sg.matmul_fp8(A, SA, B.t(), SB.t(), C, alpha=alpha)

    for a, b in ((-70, -55), (100, -100), (-126, 120), (55, 55), (-75, -70), (-100, -49)):
        alpha = 2.0 ** min(120, -(a + b))
        assert torch.equal(product(a, b, alpha).double(), alpha * 2.0 ** (a + b) * s), (a, b)
    assert bool((product(70, 70, 2.0 ** -100) == float("inf")).all())
    assert bool((product(-80, -80, 2.0 ** 120) == 0).all())
    status_is(0)
