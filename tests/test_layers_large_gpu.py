"""Operators around a layer's products on arrays of more than 2^31 elements: the
rows behind that many are compared with the same rows in arrays of their own."""

import math

import pytest

import strided_gemm_gb300 as sg
from tests.test_layers_gpu import Shared, clean_status, gen, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def same(torch, a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("group", [1, 128])
def test_quantise_many_elements(torch, group):
    M, K = 33024, 65664                                      # 2.17e9
    x = torch.empty(M, K, device="cuda", dtype=torch.bfloat16)
    x[-256:] = torch.randn(256, K, generator=gen(torch, 1), device="cuda").bfloat16()
    x[:-256] = 1.0
    y, s = torch.empty(M, K, device="cuda", dtype=torch.float8_e4m3fn), torch.empty(M // group, K // 128, device="cuda")
    sg.quantize_fp8(x, y, s)
    y2, s2 = torch.empty_like(y[-256:]), torch.empty(256 // group, K // 128, device="cuda")
    sg.quantize_fp8(x[-256:], y2, s2)
    assert same(torch, y[-256:], y2) and torch.equal(s[-(256 // group):], s2)
    assert bool((s[:100] == 1.0 / 448.0).all())


def test_product_with_many_outputs(torch):
    M, N, K = 66048, 32896, 128                              # 2.17e9
    g = gen(torch, 2)
    A, B = (torch.randn(n, K, generator=g, device="cuda").to(torch.float8_e4m3fn) for n in (M, N))
    SA, SB = torch.rand(M, 1, generator=g, device="cuda"), torch.rand(N // 128, 1, generator=g, device="cuda")
    C = torch.empty(M, N, device="cuda", dtype=torch.bfloat16)
    sg.matmul_fp8(A, SA, B.t(), SB.t(), C)
    last = torch.empty(512, N, device="cuda", dtype=torch.bfloat16)
    sg.matmul_fp8(A[-512:], SA[-512:], B.t(), SB.t(), last)
    assert same(torch, C[-512:], last)
    first = torch.empty(512, N, device="cuda", dtype=torch.bfloat16)
    sg.matmul_fp8(A[:512], SA[:512], B.t(), SB.t(), first)
    assert same(torch, C[:512], first)


def test_rotation_of_many_elements(torch):
    tokens, heads, D, n = 52480, 41, 1024, 100               # 2.2e9
    g = gen(torch, 3)
    x = torch.empty(tokens, heads, D, device="cuda", dtype=torch.bfloat16)
    x[:-n] = 0.5
    x[-n:] = torch.randn(n, heads, D, generator=g, device="cuda").bfloat16()
    pos = torch.randint(0, 1 << 30, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    w = torch.randn(D, generator=g, device="cuda").bfloat16()
    table = sg.rope_table(512)
    last = x[-n:].clone()
    sg.norm_rope([sg.RopePart(x, x, norm=D, weight=w)], pos, table)
    want = torch.empty_like(last)
    sg.norm_rope([sg.RopePart(last, want, norm=D, weight=w)], pos[-n:], table)
    assert same(torch, x[-n:], want)
    dx = torch.empty_like(last)
    sg.norm_rope_backward([sg.RopeGrad(x[-n:], x[-n:], dx, norm=D, weight=w)], pos[-n:], table)
    sg.norm_rope_backward([sg.RopeGrad(x, x, x, norm=D, weight=w)], pos, table)
    assert same(torch, x[-n:], dx)


def test_shared_in_a_long_cache(torch):
    c = Shared(torch, "bf16", [(700, 30, 1, 90)], 16, 1, 512, 64, 64)
    c.run()
    want = c.o.clone()
    pages, own = 60000, c.cache.shape[0]                     # 2.2e9 elements
    cache = torch.empty(pages, 64, 576, device="cuda", dtype=torch.bfloat16)
    cache[-own:] = c.cache
    c.table[c.table >= 0] += pages - own
    c.cache = cache
    c.o.fill_(math.nan)
    c.run()
    assert same(torch, c.o, want)
    c.check(torch)
