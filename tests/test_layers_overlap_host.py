"""Which arrays of one call of the norms and rotations may lie in one another's
gaps: the host's check against every element's address.  No GPU: what passes the
check of overlaps is refused by the next one, which asks for a device."""

import random

import pytest

import strided_gemm_gb300 as sg
from tests.test_layers_host import A, B, C, D, E, F, OVERLAP, built, rope, rope_back, status  # noqa: F401

PAST = (sg.SBGEMM_ERR_CUDA, sg.SBGEMM_ERR_NOT_DEVICE_MEMORY)


def interleaved(tokens, heads, dim, order=(0, 1), **kw):
    """Queries and keys out of [tokens][heads][q | k | v], turned in place."""
    parts = []
    for i in order:
        at = A + 2 * i * dim
        parts.append((at, 3 * heads * dim, 3 * dim, at, 3 * heads * dim, 3 * dim, heads, dim, dim, 0, 0))
    return status(sg.sbgemm_norm_rope, sg.TYPE_BF16, parts, D, tokens, E, dim, **kw)


@pytest.mark.parametrize("tokens", [1, 8])
@pytest.mark.parametrize("heads", [1, 5, 16])
@pytest.mark.parametrize("order", [(0, 1), (1, 0), (2, 0), (0, 1, 2), (2, 1, 0)])
def test_heads_of_several_arrays_side_by_side(tokens, heads, order):
    assert interleaved(tokens, heads, 64, order) in PAST
    assert interleaved(tokens, heads, 64, (0, 0)) == OVERLAP


def test_gradients_of_arrays_side_by_side():
    rows = dict(x_token=16 * 192, x_head=192, dy=A, dy_token=16 * 192, dy_head=192, dx=A, dx_token=16 * 192, dx_head=192, x=B)
    beside = dict(x=B + 128, dy=A + 128, dx=A + 128)
    assert rope_back(part=rows, second=beside) in PAST
    assert rope_back(part=rows, second=dict(beside, dy=A + 126, dx=A + 126)) == OVERLAP


def elements(base, ts, hs, tokens, heads, dim):
    return {base + t * ts + h * hs + d for t in range(tokens) for h in range(heads) for d in range(dim)}


def test_the_check_against_every_address():
    """Random arrays in one stretch of memory: nothing that shares an element passes,
    and of arrays that do not, all with one token stride and one head stride whose
    parts of a token follow one another do."""
    rng = random.Random(4)
    passed = apart = 0
    for _ in range(6000):
        tokens, heads, dim = rng.randint(1, 4), rng.randint(1, 4), rng.randint(1, 6)
        heads2, dim2 = rng.randint(1, 4), rng.randint(1, 6)
        hs = dim + rng.randint(0, 8)
        hs2 = hs if rng.random() < 0.7 else dim2 + rng.randint(0, 8)
        ts = max(heads * hs, heads2 * hs2) + rng.choice([0, 0, 0, 1, 5, 40])
        ts2 = ts if rng.random() < 0.8 else ts + rng.randint(1, 5)
        off = rng.randint(-30, 30) if rng.random() < 0.8 else rng.randint(-2 * ts, 2 * ts)
        a, b = 1000, 1000 + off
        parts = [(F, ts, hs, A + 2 * a, ts, hs, heads, dim, 0, 0, 0), (F, ts2, hs2, A + 2 * b, ts2, hs2, heads2, dim2, 0, 0, 0)]
        one, two = elements(a, ts, hs, tokens, heads, dim), elements(b, ts2, hs2, tokens, heads2, dim2)
        if len(one) < tokens * heads * dim or len(two) < tokens * heads2 * dim2:
            continue
        st = status(sg.sbgemm_norm_rope, sg.TYPE_BF16, parts, 0, tokens, 0, 0)
        assert st in PAST or st == OVERLAP
        if one & two:
            assert st == OVERLAP, (parts, tokens)
        else:
            apart += 1
            passed += st != OVERLAP
    assert apart > 1000 and passed > 0.6 * apart, (passed, apart)


@pytest.mark.parametrize("want,at", [
    (OVERLAP, dict(dweight=A)), (OVERLAP, dict(dweight=A + 2 * 1024 * 7)), (OVERLAP, dict(dweight=B + 64)),
    (OVERLAP, dict(dweight=C)), (OVERLAP, dict(dweight=D)), (OVERLAP, dict(dweight=E + 28)), (OVERLAP, dict(dweight=F)),
    (None, dict(dweight=F + 4096)),
])
def test_the_gradient_of_a_part_without_heads_meets_nothing_of_the_others(want, at):
    """It is zeroed first: x, dy, dx, the weight, positions and steps of the others."""
    st = rope_back(part=dict(weight=D), second=dict(heads=0, weight=0, **at))
    assert st == want if want is not None else st in PAST
