"""Norms, rotations and their gradients in place on arrays that lie side by side in
each head's place: queries and keys out of [tokens][heads][q | k | v]."""

import pytest

from tests.test_layers_gpu import Rope, clean_status, gen, torch  # noqa: F401
from tests.test_serving_gpu import assert_within, status_is

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("tokens", [1, 37])
@pytest.mark.parametrize("D", [64, 7])
def test_queries_and_keys_head_by_head_in_place(torch, t, tokens, D):
    heads = 5
    r = Rope(torch, t, tokens, D // 2 * 2, False, [(heads, D, D, 0), (heads, D, D, 0)])
    both = []
    for src in (r.x, r.dy):
        packed = torch.randn(tokens, heads, 3 * D, generator=gen(torch, 3), device="cuda").to(src[0].dtype)
        packed[..., :D], packed[..., D:2 * D] = src[0], src[1]
        both.append(packed)
    r.x, r.dy = ([p[..., :D], p[..., D:2 * D]] for p in both)
    values = [p[..., 2 * D:].clone() for p in both]
    want, grads = [r.reference(i) for i in range(2)], [r.gradient(i) for i in range(2)]
    dw = [torch.empty(D, device="cuda") for _ in range(2)]
    r.backward(r.dy, dw)
    r.forward(r.x)
    for i in range(2):
        assert_within(torch, r.x[i], *want[i])
        assert_within(torch, r.dy[i], *grads[i][:2])
        assert_within(torch, dw[i], *grads[i][2:])
    for p, v in zip(both, values):
        assert torch.equal(p[..., 2 * D:], v)
    status_is(0)
