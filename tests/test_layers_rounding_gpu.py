"""Roundings that the definitions of the operators around a layer's products fix:
outputs of 8-bit products rounded once, and sums of one sign over many rows."""

import pytest

import strided_gemm_gb300 as sg
from tests.test_layers_gpu import clean_status, gen, torch  # noqa: F401
from tests.test_serving_gpu import status_is

pytestmark = pytest.mark.gpu


# Tiles of every shape: pairs of CTAs, 128 columns, fewer, split along K, and a K that
# no tensor map takes.
ADDED = [(1, 700, 1000, 640), (1, 2600, 1032, 384), (1, 16, 2048, 2000), (2, 4, 6, 300), (2, 300, 264, 256), (1, 4099, 2560, 128),
         (1, 130, 100, 77)]


@pytest.mark.parametrize("size", ADDED)
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("gb", [1, 128])
def test_sums_added_to_c_are_rounded_once(torch, size, pad, gb):
    """C <- alpha S + C as one fused operation.  S is a whole number below 2^13 and C
    the rounded -alpha S, so that what is left, the product's rounding error, has at
    most 13 + 24 - 24 bits: exact in 64 bits and in fp32.  A subnormal C stays as it is
    when nothing is added to it."""
    batch, M, N, K = size
    g = gen(torch, M + N)
    f8 = torch.float8_e4m3fn

    def operand(rows):
        wide = torch.zeros(batch, rows, K if K % 16 else K + 16, device="cuda").to(f8)[..., :K]
        wide.copy_(torch.randint(-2, 3, (batch, rows, K), generator=g, device="cuda").float().to(f8))
        return wide

    A, B = operand(M), operand(N)
    SA = torch.ones(batch, M, -(-K // 128), device="cuda")
    SB = torch.ones(batch, -(-N // gb), -(-K // 128), device="cuda")
    s = A.double() @ B.double().transpose(1, 2)
    alpha = float(torch.tensor(1.0 / 3.0, dtype=torch.float32))

    def added_to(old, alpha):
        C = torch.empty(batch, M, N + pad, device="cuda")[..., :N]
        C.copy_(old)
        sg.matmul_fp8(A, SA, B.transpose(1, 2), SB.transpose(1, 2), C, alpha=alpha, accumulate=True)
        return C

    old = -(alpha * s).float()
    assert torch.equal(added_to(old, alpha).double(), alpha * s + old.double())
    tiny = torch.full((batch, M, N), 2.0 ** -140, device="cuda")
    assert torch.equal(added_to(tiny, 0.0), tiny)
    A.zero_()
    assert torch.equal(added_to(tiny, 1.0), tiny)
    status_is(0)


def gradient_of_ones(torch, t, tokens, heads, D):
    """(relative error of dweight, depth): x = 1 and dy = c for every element, so that
    dweight is rows c / sqrt(1 + eps)."""
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32}[t]
    x = torch.ones(1, 1, D, device="cuda", dtype=dt).expand(tokens, heads, D)
    dy = torch.full((1, 1, D), 1.1, device="cuda", dtype=dt).expand(tokens, heads, D)
    dx, dw = torch.empty(tokens, heads, D, device="cuda", dtype=dt), torch.empty(D, device="cuda")
    ws = torch.empty(sg.sbgemm_norm_rope_workspace_bytes([D]), device="cuda", dtype=torch.uint8)
    sg.norm_rope_backward([sg.RopeGrad(x, dy, dx, norm=D, dweight=dw)], None, None, workspace=ws)
    status_is(0)
    ref = tokens * heads * float(dy[0, 0, 0]) * (1 + 1e-6) ** -0.5
    return float((dw.double() - ref).abs().max()) / ref


@pytest.mark.parametrize("t,D", [("bf16", 33), ("fp32", 7), ("fp32", 300)])
def test_long_sums_of_one_sign_at_any_alignment(torch, t, D):
    """2^20 rows, some 3400 a CTA one behind the other: every addend is off by
    (D / 2 + 8) 2^-24 of itself as every normed element is, the CTAs' sums and the
    whole by a rounding each, and nothing grows with the rows."""
    assert gradient_of_ones(torch, t, 1 << 16, 16, D) <= (D / 2 + 10) * 2.0 ** -24


def test_long_sums_of_one_sign_in_vectors(torch):
    """Rows of 64 bf16 elements are 4 lanes' work, so that 64 groups of lanes a CTA and
    two CTAs an SM (less one) share them: that many additions, then 3 over a warp's
    groups and 8 over the warps."""
    tokens, heads, D = 1 << 16, 16, 64
    groups = (2 * torch.cuda.get_device_properties(0).multi_processor_count - 1) * 64
    depth = -(-tokens * heads // groups) + 3 + 8
    assert gradient_of_ones(torch, "bf16", tokens, heads, D) <= (D / 2 + 10 + depth) * 2.0 ** -24
