"""Operands whose rows overlap in memory (sliding windows), which the strides allow:
8-bit products, and latent attention's cache and queries."""

import pytest

import strided_gemm_gb300 as sg
from tests.test_layers_gpu import HALF, TINY, U, clean_status, gen, torch  # noqa: F401
from tests.test_serving_gpu import assert_within, attention_bound, attention_reference, status_is

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N", [(200, 140), (5, 300), (600, 520)])
def test_products_of_windows(torch, M, N):
    g = gen(torch, 8)
    f8, K = torch.float8_e4m3fn, 512
    A = torch.randn(16 * M + K, generator=g, device="cuda").to(f8).as_strided((M, K), (16, 1))
    B = torch.randn(32 * N + K, generator=g, device="cuda").to(f8).as_strided((N, K), (32, 1))
    SA, SB = torch.rand(M, 4, generator=g, device="cuda"), torch.rand(-(-N // 128), 4, generator=g, device="cuda")
    C = torch.empty(M, N, device="cuda")
    sg.matmul_fp8(A, SA, B.t(), SB.t(), C)
    va = A.double() * SA.double().repeat_interleave(128, 1)
    vb = B.double() * SB.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)
    ref, S = va @ vb.t(), va.abs() @ vb.abs().t()
    assert_within(torch, C, ref, (K + 12) * U * S + HALF["fp32"] * ref.abs() + TINY)
    status_is(0)


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("block", [16, 12])
def test_attention_over_windows(torch, shared, block):
    g = gen(torch, 9)
    S, H, R, P, pages, n = 3, 16, 512, 64, 12, 45
    D, i32 = R + P, dict(device="cuda", dtype=torch.int32)
    cache = torch.randn(pages * block * 64 + D, generator=g, device="cuda").bfloat16().as_strided(
        (pages, block, D), (block * 64, 64, 1))
    q = torch.randn(S * H * 64 + D, generator=g, device="cuda").bfloat16().as_strided((S, 1, H, D), (H * 64, H * 64, 64, 1))
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(S, 4)
    lens, o = torch.full((S,), n, **i32), torch.empty(S, 1, H, R, device="cuda", dtype=torch.bfloat16)
    if shared:
        ws = torch.empty(sg.sbgemm_latent_shared_workspace_bytes(S, 1, 1, H, R), device="cuda", dtype=torch.uint8)
        sg.latent_attention_shared(q, cache, table, lens, torch.tensor([0, S], **i32), torch.zeros(1, **i32), o, alpha=0.05,
                                   workspace=ws)
    else:
        ws = torch.empty(sg.sbgemm_latent_workspace_bytes(torch.cuda.current_device()), device="cuda", dtype=torch.uint8)
        sg.latent_attention_paged(q, cache, table, lens, o, alpha=0.05, workspace=ws)
    for s in range(S):
        kv = cache[table[s].long()].reshape(-1, D)[:n].double()
        keep = torch.ones(1, n, device="cuda", dtype=torch.bool)
        O, W, Z, sv = attention_reference(q[s].double().transpose(0, 1), kv, kv[:, :R], 0.05, keep)
        assert_within(torch, o[s].transpose(0, 1), O, attention_bound("bf16", D, n, O, W, Z, sv))
    status_is(0)
