"""Refusals of the operators around a layer's products that need no GPU: every
check of arguments comes before the first CUDA call, on addresses that nothing
reads.  And the tables of rotations against exact arithmetic."""

import ctypes
import math
from fractions import Fraction

import pytest

import strided_gemm_gb300 as sg
from strided_gemm_gb300 import build as sgbuild

BASE = 0x7F0000000000       # 256-byte aligned addresses, far apart, never dereferenced
A, B, C, D, E, F, G = (BASE + i * (1 << 36) for i in range(7))

INVALID, NULL, OVERLAP, UNSUPPORTED, OK = (
    sg.SBGEMM_ERR_INVALID_VALUE, sg.SBGEMM_ERR_NULL_POINTER, sg.SBGEMM_ERR_OUTPUT_OVERLAP,
    sg.SBGEMM_ERR_UNSUPPORTED, sg.SBGEMM_OK)


@pytest.fixture(scope="module", autouse=True)
def built():
    sgbuild.build()
    sg.load()


def status(f, *args, **kw):
    try:
        f(*args, **kw)
    except sg.SbgemmError as e:
        return e.status
    return sg.SBGEMM_OK


def matrix(**kw):
    a = dict(type=sg.TYPE_E4M3, group=1, data=A, row_stride=256, k_stride=1, batch_stride=0, scale=B,
             scale_row_stride=2, scale_k_stride=1, scale_batch_stride=0)
    a.update(kw)
    return sg.Fp8Matrix(**a)


def fp8(a=None, b=None, **kw):
    args = dict(A=matrix(**(a or {})), B=matrix(**{**dict(data=C, scale=D, group=128), **(b or {})}),
                type_c=sg.TYPE_BF16, C=E, rsC=64, csC=1, bsC=64 * 64, M=32, N=64, K=256, batch=2)
    args.update(kw)
    return status(sg.sbgemm_fp8, **args)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(type_c=sg.TYPE_E4M3)), (INVALID, dict(type_c=0)), (NULL, dict(A=None)), (NULL, dict(B=None)),
    (INVALID, dict(M=-1)), (INVALID, dict(K=-1)), (NULL, dict(C=0)), (INVALID, dict(C=E + 1)),
    (INVALID, dict(type_c=sg.TYPE_FP32, C=E + 2)),
    (INVALID, dict(a=dict(type=sg.TYPE_BF16))), (INVALID, dict(b=dict(type=6))), (INVALID, dict(a=dict(group=64))),
    (INVALID, dict(b=dict(group=0))), (NULL, dict(a=dict(data=0))), (NULL, dict(b=dict(scale=0))),
    (INVALID, dict(a=dict(scale=B + 2))), (INVALID, dict(a=dict(row_stride=1 << 62))),
    (OVERLAP, dict(bsC=0)), (OVERLAP, dict(rsC=63)), (OVERLAP, dict(C=A)), (OVERLAP, dict(C=B)), (OVERLAP, dict(C=C + 64)),
    (OVERLAP, dict(C=D)), (UNSUPPORTED, dict(M=1 << 31, batch=1, a=dict(row_stride=0, scale_row_stride=0))),
    (OK, dict(M=0)), (OK, dict(N=0)), (OK, dict(batch=0)),
    (OK, dict(K=0, accumulate=1, a=dict(data=0, scale=0), b=dict(data=0, scale=0))),
])
def test_fp8_refusals(want, kw):
    assert fp8(**kw) == want


def quantise(y=None, **kw):
    args = dict(type_x=sg.TYPE_BF16, X=C, rsX=256, csX=1, bsX=32 * 256,
                Y=matrix(**{**dict(batch_stride=32 * 256, scale_batch_stride=64), **(y or {})}), M=32, K=256, batch=2)
    args.update(kw)
    return status(sg.sbgemm_quantize_fp8, **args)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(type_x=sg.TYPE_E4M3)), (NULL, dict(Y=None)), (NULL, dict(X=0)), (INVALID, dict(X=C + 1)),
    (INVALID, dict(type_x=sg.TYPE_FP32, X=C + 2)), (INVALID, dict(K=-1)), (INVALID, dict(y=dict(group=2))),
    (INVALID, dict(y=dict(type=sg.TYPE_FP16))), (NULL, dict(y=dict(data=0))), (NULL, dict(y=dict(scale=0))),
    (OVERLAP, dict(y=dict(row_stride=255))), (OVERLAP, dict(y=dict(batch_stride=0))),
    (OVERLAP, dict(y=dict(scale_row_stride=1))), (OVERLAP, dict(y=dict(scale_batch_stride=0))),
    (OVERLAP, dict(y=dict(data=C))), (OVERLAP, dict(y=dict(scale=C + 128))), (OVERLAP, dict(y=dict(scale=A))),
    (OK, dict(M=0)), (OK, dict(K=0)), (OK, dict(batch=0)),
])
def test_quantise_refusals(want, kw):
    assert quantise(**kw) == want


def rope(part=None, second=None, **kw):
    p = dict(x=A, x_token=1024, x_head=64, y=B, y_token=1024, y_head=64, heads=16, D=64, norm=64, start=0, weight=C)
    p.update(part or {})
    parts = [tuple(p.values())]
    if second is not None:
        parts.append(tuple({**p, **second}.values()))
    args = dict(type=sg.TYPE_BF16, parts=parts, positions=D, tokens=8, steps=E, dims=64)
    args.update(kw)
    return status(sg.sbgemm_norm_rope, **args)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(type=sg.TYPE_E4M3)), (INVALID, dict(tokens=-1)), (INVALID, dict(dims=63)), (INVALID, dict(dims=-2)),
    (INVALID, dict(interleaved=2)), (INVALID, dict(dims=66)), (NULL, dict(positions=0)), (NULL, dict(steps=0)),
    (INVALID, dict(positions=D + 2)), (INVALID, dict(steps=E + 4)), (UNSUPPORTED, dict(tokens=1 << 31)),
    (INVALID, dict(part=dict(norm=65))), (INVALID, dict(part=dict(start=1))), (INVALID, dict(part=dict(heads=-1))),
    (INVALID, dict(part=dict(start=-1))), (UNSUPPORTED, dict(part=dict(D=4097, x_head=4097, y_head=4097))),
    (NULL, dict(part=dict(x=0))), (NULL, dict(part=dict(y=0))), (INVALID, dict(part=dict(x=A + 1))),
    (INVALID, dict(part=dict(weight=C + 1))), (OVERLAP, dict(part=dict(y_head=63))), (OVERLAP, dict(part=dict(y_token=1000))),
    (OVERLAP, dict(part=dict(y=A + 64))), (OVERLAP, dict(part=dict(y=A, y_head=128, y_token=2048))),
    (OVERLAP, dict(part=dict(y=C))), (OVERLAP, dict(part=dict(y=D))), (OVERLAP, dict(part=dict(y=E))),
    (OVERLAP, dict(second=dict(x=F))), (OVERLAP, dict(second=dict(y=A, x=F))),
    (INVALID, dict(part=dict(x_token=1 << 61))),
    (OK, dict(tokens=0)), (OK, dict(parts=[])), (OK, dict(part=dict(heads=0))), (OK, dict(part=dict(D=0, norm=0), dims=0)),
])
def test_rope_refusals(want, kw):
    assert rope(**kw) == want


def test_rope_takes_no_more_parts_than_it_has_room_for():
    part = (A, 1024, 64, B, 1024, 64, 16, 64, 64, 0, C)
    assert status(sg.sbgemm_norm_rope, sg.TYPE_BF16, [part] * 5, D, 8, E, 64) == INVALID


def rope_back(part=None, second=None, **kw):
    p = dict(x=A, x_token=1024, x_head=64, dy=B, dy_token=1024, dy_head=64, dx=C, dx_token=1024, dx_head=64, heads=16,
             D=64, norm=64, start=0, weight=D, dweight=0)
    p.update(part or {})
    parts = [tuple(p.values())]
    if second is not None:
        parts.append(tuple({**p, **second}.values()))
    args = dict(type=sg.TYPE_BF16, parts=parts, positions=E, tokens=8, steps=F, dims=64)
    args.update(kw)
    return status(sg.sbgemm_norm_rope_backward, **args)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(type=0)), (INVALID, dict(dims=1)), (NULL, dict(positions=0)), (NULL, dict(part=dict(x=0))),
    (NULL, dict(part=dict(dy=0))), (NULL, dict(part=dict(dx=0))), (INVALID, dict(part=dict(dweight=G + 2))),
    (INVALID, dict(workspace=G + 8, workspace_bytes=1 << 20)), (OVERLAP, dict(part=dict(dx=A + 64))),
    (OVERLAP, dict(part=dict(dx=B + 2))), (OVERLAP, dict(part=dict(dx=D))), (OVERLAP, dict(part=dict(dx=E))),
    (OVERLAP, dict(second=dict())), (INVALID, dict(part=dict(norm=70))),
    (OK, dict(tokens=0)), (OK, dict(parts=[])), (OK, dict(part=dict(heads=0))),
])
def test_rope_backward_refusals(want, kw):
    assert rope_back(**kw) == want


def test_packed_parts_do_not_count_as_overlapping():
    """Queries and keys side by side in one projection's rows, turned in place:
    past the checks of overlaps (the next one asks for a device)."""
    rows = dict(x_token=1280, y_token=1280, x=A, y=A)
    beside = dict(x=A + 2 * 1024, y=A + 2 * 1024, heads=4)
    past = (sg.SBGEMM_ERR_CUDA, sg.SBGEMM_ERR_NOT_DEVICE_MEMORY)
    assert rope(part=rows, second=beside) in past
    assert rope(part=rows, second=dict(beside, y=A + 2 * 1023)) == OVERLAP
    assert rope(part=rows, second=dict(beside, heads=5)) == OVERLAP          # reaches into the next token


def shared(**kw):
    a = dict(type=sg.TYPE_BF16, Q=A, hsQ=576, tsQ=16 * 576, bsQ=16 * 576, cache=B, rsC=576, psC=16 * 576,
             num_blocks=100, block_size=16, block_table=C, max_blocks=8, seq_lens=D, group_starts=F, prefix_lens=F + 4096,
             n_groups=2, O=E, hsO=512, tsO=16 * 512, bsO=16 * 512, q_len=1, heads=16, N=128, R=512, P=64, n_seqs=4,
             alpha=0.1, causal=1)
    a.update(kw)
    return status(sg.sbgemm_latent_attention_shared, **a)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(type=3)), (INVALID, dict(n_groups=-1)), (NULL, dict(group_starts=0)), (NULL, dict(prefix_lens=0)),
    (INVALID, dict(group_starts=F + 2)), (INVALID, dict(prefix_lens=F + 1)), (OVERLAP, dict(O=F)),
    (UNSUPPORTED, dict(n_groups=1 << 30)), (INVALID, dict(N=129)), (INVALID, dict(causal=2)), (NULL, dict(Q=0)),
    (UNSUPPORTED, dict(R=513)), (INVALID, dict(workspace=G + 16, workspace_bytes=1 << 20)), (OVERLAP, dict(bsO=0)),
    (OK, dict(n_seqs=0)), (OK, dict(heads=0)), (OK, dict(q_len=0)), (OK, dict(R=0)),
])
def test_shared_refusals(want, kw):
    assert shared(**kw) == want


def test_workspace_sizes_are_checked():
    n = ctypes.c_size_t(0)
    lib = sg.load()
    assert lib.sbgemm_latent_shared_workspace_bytes(0, -1, 1, 1, 16, 512, ctypes.byref(n)) == INVALID
    assert lib.sbgemm_latent_shared_workspace_bytes(0, 4, 1, 1, 16, 513, ctypes.byref(n)) == UNSUPPORTED
    assert lib.sbgemm_latent_shared_workspace_bytes(0, 4, 1, 1, 16, 512, None) == NULL
    assert lib.sbgemm_norm_rope_workspace_bytes(0, -1, ctypes.byref(n)) == INVALID
    assert lib.sbgemm_norm_rope_workspace_bytes(0, 5 * 4096, ctypes.byref(n)) == INVALID
    assert lib.sbgemm_norm_rope_workspace_bytes(0, 16, None) == NULL


def test_steps_are_exact_fractions_of_a_turn():
    f = sg.rope_frequencies(128, base=500000.0, factor=8.0, original=8192)
    assert len(f) == 64 and f[0] == 1.0 and f[-1] < 1e-5
    # pi to 60 digits: the phases at far positions stay within a step's rounding.
    pi = Fraction(31415926535897932384626433832795028841971693993751058209749, 10 ** 58)
    for x, step in zip(f, sg.rope_steps(f)):
        exact = Fraction(x) / (2 * pi)
        got = Fraction(step % 2 ** 64, 2 ** 64)
        # One rounding of the quotient to a double and one of 2 pi: 2^-52 relative.
        assert abs(got - exact) <= exact * Fraction(1, 2 ** 52) + Fraction(1, 2 ** 64)
    assert sg.rope_steps([2 * math.pi, math.pi, -math.pi / 2]) == [0, -2 ** 63, -2 ** 62]


def test_frequencies_by_parts():
    plain, far = sg.rope_frequencies(64), sg.rope_frequencies(64, factor=16.0, original=4096)
    assert far[0] == plain[0] and far[-1] == plain[-1] / 16.0
    assert all(a >= b >= a / 16.0 for a, b in zip(plain, far))


def test_torch_helpers_refuse_tensors():
    torch = pytest.importorskip("torch")
    e4 = torch.float8_e4m3fn
    x8, s = torch.zeros(4, 128).to(e4), torch.ones(4, 1)
    with pytest.raises(TypeError):
        sg.matmul_fp8(x8, s, x8.t(), s.t(), torch.zeros(4, 4))                   # on the CPU
    with pytest.raises(TypeError):
        sg.quantize_fp8(torch.zeros(4, 128), x8, s)
    with pytest.raises(TypeError):
        sg.quantize_fp8(torch.zeros(4, 128, dtype=torch.int32), x8, s)
    with pytest.raises(ValueError):
        sg.rope_table(3, device="cpu")
    with pytest.raises(ValueError):
        sg.rope_table(4, frequencies=[1.0], device="cpu")
    t = sg.rope_table(4, device="cpu")
    with pytest.raises(TypeError):
        sg.norm_rope([sg.RopePart(torch.zeros(2, 3, 8), torch.zeros(2, 3, 8))], torch.zeros(2, dtype=torch.int32), t)
    sg.norm_rope([], None, None)
    with pytest.raises(TypeError):
        sg.latent_attention_shared(torch.zeros(1, 1, 1, 576).bfloat16(), torch.zeros(4, 16, 576).bfloat16(),
                                   torch.zeros(1, 4, dtype=torch.int32), None, torch.zeros(2, dtype=torch.int32),
                                   torch.zeros(1, dtype=torch.int32), torch.zeros(1, 1, 1, 512).bfloat16(), 1.0)
