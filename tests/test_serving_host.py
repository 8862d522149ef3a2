"""Refusals of the 16-bit serving operators that need no GPU: every check of
arguments comes before the first CUDA call, on addresses that nothing reads."""

import ctypes
import glob
import os
import re

import pytest

import strided_gemm_gb300 as sg
from strided_gemm_gb300 import build as sgbuild
from strided_gemm_gb300 import serving

BASE = 0x7F0000000000       # 256-byte aligned addresses, far apart, never dereferenced
A, B, C, D, E, F, G = (BASE + i * (1 << 36) for i in range(7))


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


INVALID, NULL, OVERLAP, UNSUPPORTED, OK = (
    sg.SBGEMM_ERR_INVALID_VALUE, sg.SBGEMM_ERR_NULL_POINTER, sg.SBGEMM_ERR_OUTPUT_OVERLAP,
    sg.SBGEMM_ERR_UNSUPPORTED, sg.SBGEMM_OK)


def half(**kw):
    a = dict(type=sg.TYPE_BF16, A=A, rsA=64, csA=1, bsA=0, B=B, rsB=32, csB=1, bsB=0, C=C, rsC=32, csC=1, bsC=512,
             M=16, N=32, K=64, batch=2)
    a.update(kw)
    return status(sg.sbgemm_half, **a)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(type=0)), (INVALID, dict(type=3)), (INVALID, dict(M=-1)), (INVALID, dict(K=-1)),
    (NULL, dict(A=0)), (NULL, dict(B=0)), (NULL, dict(C=0)), (INVALID, dict(A=A + 1)), (INVALID, dict(C=C + 1)),
    (OVERLAP, dict(bsC=0)), (OVERLAP, dict(rsC=31)), (OVERLAP, dict(C=A)), (OVERLAP, dict(C=B + 64)),
    (INVALID, dict(rsA=1 << 60)), (UNSUPPORTED, dict(M=1 << 31, rsA=0, batch=1)),
    (OK, dict(M=0, A=0, B=0, C=0)), (OK, dict(batch=0)), (OK, dict(K=0, accumulate=1, A=0, B=0)),
])
def test_half_refusals(want, kw):
    assert half(**kw) == want


def paged(**kw):
    a = dict(type=sg.TYPE_BF16, Q=A, hsQ=576, tsQ=16 * 576, bsQ=16 * 576, cache=B, rsC=576, psC=16 * 576,
             num_blocks=100, block_size=16, block_table=C, max_blocks=8, seq_lens=D, O=E, hsO=512,
             tsO=16 * 512, bsO=16 * 512, q_len=1, heads=16, N=128, R=512, P=64, n_seqs=4, alpha=0.1, causal=1)
    a.update(kw)
    return status(sg.sbgemm_latent_attention_paged, **a)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(type=0)), (INVALID, dict(q_len=-1)), (INVALID, dict(N=-1)), (INVALID, dict(causal=2)),
    (INVALID, dict(N=129)), (INVALID, dict(num_blocks=0)), (INVALID, dict(block_size=0)),
    (INVALID, dict(max_blocks=0)), (UNSUPPORTED, dict(R=513)), (UNSUPPORTED, dict(P=129)),
    (UNSUPPORTED, dict(heads=1 << 31)), (UNSUPPORTED, dict(N=(1 << 31) - 64, max_blocks=1 << 30)),
    (NULL, dict(Q=0)), (NULL, dict(cache=0)), (NULL, dict(block_table=0)),
    (NULL, dict(O=0)), (INVALID, dict(Q=A + 1)), (INVALID, dict(block_table=C + 2)), (INVALID, dict(seq_lens=D + 1)),
    (OVERLAP, dict(hsO=256)), (OVERLAP, dict(bsO=0)), (OVERLAP, dict(O=B)), (OVERLAP, dict(O=A)), (OVERLAP, dict(O=D)),
    (INVALID, dict(workspace=F + 16, workspace_bytes=1 << 20)), (INVALID, dict(psC=1 << 60)),
    (OK, dict(n_seqs=0)), (OK, dict(heads=0)), (OK, dict(q_len=0)), (OK, dict(R=0)),
])
def test_paged_refusals(want, kw):
    assert paged(**kw) == want


def test_paged_reads_no_path_of_the_options():
    o = sg._Options()
    o.force_path = sg.PATH_TMA_TF32
    args = [sg.TYPE_BF16, A, 576, 576, 576, B, 576, 9216, 10, 16, C, 8, D, E, 512, 512, 512, 1, 1, 128, 512, 64, 1,
            0.1, 0, None]
    assert sg.load().sbgemm_latent_attention_paged(*args, ctypes.byref(o)) == UNSUPPORTED
    o.force_path, o.reserved[0] = sg.PATH_AUTO, 1
    assert sg.load().sbgemm_latent_attention_paged(*args, ctypes.byref(o)) == INVALID


def packed(**kw):
    a = dict(type=sg.TYPE_FP16, Q=A, hsQ=192, tsQ=4 * 192, total_q=10, K_nope=B, hsK=256, tsK=1024, K_rope=C, tsR=64,
             V=B + 256, hsV=256, tsV=1024, total_k=20, q_starts=D, k_starts=E, n_seqs=2, max_q=8, O=F, hsO=128,
             tsO=512, heads=4, Dn=128, P=64, Dv=128, alpha=0.1, causal=1)
    a.update(kw)
    return status(sg.sbgemm_latent_attention, **a)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(type=7)), (INVALID, dict(total_q=-1)), (INVALID, dict(Dn=0, P=0)), (INVALID, dict(causal=-1)),
    (UNSUPPORTED, dict(Dn=600)), (UNSUPPORTED, dict(Dv=513)), (UNSUPPORTED, dict(n_seqs=65536)),
    (NULL, dict(Q=0)), (NULL, dict(K_nope=0)), (NULL, dict(K_rope=0)), (NULL, dict(V=0)), (NULL, dict(O=0)),
    (NULL, dict(q_starts=0)), (NULL, dict(k_starts=0)), (INVALID, dict(q_starts=D + 2)), (INVALID, dict(V=B + 257)),
    (OVERLAP, dict(hsO=64)), (OVERLAP, dict(O=A)), (OVERLAP, dict(O=C)), (OVERLAP, dict(O=D)),
    (OK, dict(total_q=0)), (OK, dict(max_q=0)), (OK, dict(n_seqs=0)), (OK, dict(Dv=0)),
])
def test_packed_refusals(want, kw):
    assert packed(**kw) == want


def pool(**kw):
    p = serving._Pool()
    caches, sizes = kw.pop("caches", [A, B]), kw.pop("page_bytes", [16 * 64, 16 * 32])
    p.caches = (ctypes.c_void_p * len(caches))(*caches)
    p.page_bytes = (ctypes.c_int64 * len(sizes))(*sizes)
    p.n_caches = kw.pop("n_caches", len(caches))
    p.num_blocks, p.block_size, p.n_seqs, p.max_blocks = 100, 16, 8, 10
    p.ref_counts, p.block_table, p.seq_lens = C, C + 4096, C + 8192
    for k, v in kw.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(n_caches=-1)), (INVALID, dict(n_caches=65)), (INVALID, dict(num_blocks=0)),
    (INVALID, dict(block_size=0)), (INVALID, dict(page_bytes=[16 * 64, 16 * 24 + 8])),
    (INVALID, dict(page_bytes=[16 * 64, 16 * 8])), (INVALID, dict(page_bytes=[0, 512])),
    (INVALID, dict(caches=[A, B + 8])), (NULL, dict(caches=[A, None])), (OVERLAP, dict(caches=[A, A + 1024])),
    (NULL, dict(ref_counts=None)), (NULL, dict(block_table=None)), (NULL, dict(seq_lens=None)),
    (INVALID, dict(seq_lens=C + 8194)), (OVERLAP, dict(seq_lens=C + 4096)), (OVERLAP, dict(ref_counts=A)),
    (INVALID, dict(n_seqs=0)), (INVALID, dict(max_blocks=0)),
])
def test_pool_refusals(want, kw):
    p = ctypes.byref(pool(**kw))
    lib = sg.load()
    assert lib.sbgemm_pages_free(p, D, 4, None) == want
    assert lib.sbgemm_pages_fork(p, D, E, 4, None, None) == want
    assert lib.sbgemm_pages_compact(p, None, None, None) == want


def test_pool_requests():
    lib, p = sg.load(), ctypes.byref(pool())
    for f, args in ((lib.sbgemm_pages_copy, (D, -1, None, None)), (lib.sbgemm_pages_fork, (D, E, -1, None, None)),
                    (lib.sbgemm_pages_append, (D, E, -1, None, None, 0, None, None)),
                    (lib.sbgemm_pages_append, (D, E, 1, None, None, -1, None, None)),
                    (lib.sbgemm_pages_free, (D, -1, None)), (lib.sbgemm_pages_free, (D + 2, 1, None))):
        assert f(p, *args) == INVALID
    for f, args in ((lib.sbgemm_pages_copy, (None, 1, None, None)), (lib.sbgemm_pages_fork, (None, E, 1, None, None)),
                    (lib.sbgemm_pages_fork, (D, None, 1, None, None)), (lib.sbgemm_pages_free, (None, 1, None))):
        assert f(p, *args) == NULL
    for f, args in ((lib.sbgemm_pages_copy, (None, 0, None, None)),
                    (lib.sbgemm_pages_fork, (None, None, 0, None, None)),
                    (lib.sbgemm_pages_append, (None, None, 0, None, None, 0, None, None)),
                    (lib.sbgemm_pages_free, (None, 0, None))):
        assert f(p, *args) == OK
    assert lib.sbgemm_pages_free(None, D, 1, None) == NULL


def test_pages_workspace_bytes():
    b = sg.sbgemm_pages_workspace_bytes(1000, 10, 5)
    assert b >= 4 * (2 * 1000 + 10 + 1) and b % 256 == 0
    assert sg.sbgemm_pages_workspace_bytes(2000, 10, 5) > b
    with pytest.raises(sg.SbgemmError):
        sg.sbgemm_pages_workspace_bytes(-1, 10, 5)


def test_fastcall_statuses_match_ctypes(monkeypatch):
    """The fast-call module and ctypes give the same statuses, and the former
    refuses arguments it cannot convert."""
    if sg._fast is None:
        pytest.skip("the fast-call module is not built (no Python headers)")
    cases = [(half, dict(type=9)), (half, dict(C=A)), (half, dict(M=0)), (paged, dict(N=129)), (paged, dict(O=0)),
             (paged, dict(n_seqs=0)), (packed, dict(Dv=513)), (packed, dict(V=0)), (packed, dict(Dv=0))]
    fast = [f(**kw) for f, kw in cases]
    pages = [status(serving._pages_on, op, (A, B), (1024, 512 + bad), 100, 16, C, C + 4096, 8, 10, C + 8192, D, E, n,
                    (F, G) if op == 2 else (), (64, 32) if op == 2 else (), 4, 0, 0, 0)
             for op in range(5) for bad in (0, 8) for n in (0, -1)]
    monkeypatch.setattr(sg, "_fast", None)
    assert fast == [f(**kw) for f, kw in cases]
    assert pages == [status(serving._pages_on, op, (A, B), (1024, 512 + bad), 100, 16, C, C + 4096, 8, 10, C + 8192, D,
                            E, n, (F, G) if op == 2 else (), (64, 32) if op == 2 else (), 4, 0, 0, 0)
                     for op in range(5) for bad in (0, 8) for n in (0, -1)]


def test_fastcall_refuses_what_it_cannot_convert():
    if sg._fast is None:
        pytest.skip("the fast-call module is not built (no Python headers)")
    f = sg._fast
    for call in (lambda: f.half(1), lambda: f.paged(1), lambda: f.packed(1), lambda: f.pages(1),
                 lambda: f.half("1", A, 1, 1, 1, B, 1, 1, 1, C, 1, 1, 1, 0, 0, 0, 0, 1.0, 0, 0),
                 lambda: f.pages(0, [A], (1024,), 100, 16, 0, 0, 0, 0, 0, D, 0, 1, (), (), 0, 0, 0),
                 lambda: f.pages(0, (A, B), (1024,), 100, 16, 0, 0, 0, 0, 0, D, 0, 1, (), (), 0, 0, 0),
                 lambda: f.pages(0, (A,) * 65, (1024,) * 65, 100, 16, 0, 0, 0, 0, 0, D, 0, 1, (), (), 0, 0, 0),
                 lambda: f.pages(2, (A,), (1024,), 100, 16, C, C, 1, 1, C, D, E, 1, (), (), 0, 0, 0)):
        with pytest.raises(TypeError):
            call()


def test_torch_helpers_refuse_tensors():
    torch = pytest.importorskip("torch")
    bf, i32 = dict(dtype=torch.bfloat16), dict(dtype=torch.int32)
    x = torch.zeros(4, 8, **bf)
    with pytest.raises(TypeError):
        sg.matmul_half(x, x.t(), torch.zeros(4, 4, **bf))              # on the CPU
    with pytest.raises(TypeError):
        sg.matmul_half(x.float(), x.float().t(), torch.zeros(4, 4))
    with pytest.raises(TypeError):
        sg.latent_attention_paged(torch.zeros(1, 1, 1, 576, **bf), torch.zeros(4, 16, 576, **bf),
                                  torch.zeros(1, 4, **i32), None, torch.zeros(1, 1, 1, 512, **bf), 1.0)
    with pytest.raises(ValueError):
        sg.pages_copy([], torch.zeros(1, 2, **i32), workspace=None)
    with pytest.raises(TypeError):
        sg.pages_free([torch.zeros(4, 16, 8, **bf)], torch.zeros(4, **i32), torch.zeros(1, 4, **i32),
                      torch.zeros(1, **i32), torch.zeros(1, **i32))


def test_no_load_is_multicast():
    """Every TMA load lands in the shared memory of the CTA that asks for it (a
    pair's by its barrier's address): none is multicast over a cluster, since an
    operand may lie in another GPU's memory and the library serves runs of
    several ranks.  (Barrier arrivals over a pair are no loads.)"""
    files = [f for x in ("*.cu", "*.cuh", "*.cpp", "*.h") for f in glob.glob(os.path.join(sgbuild.CSRC, x))]
    assert len(files) > 20
    for f in files:
        with open(f) as fh:
            text = fh.read()
        # The strings of an asm statement, joined: an instruction may run over several.
        for statement in re.findall(r"\basm\b[^;]*?\((.*?)\);\n", text, re.S):
            code = "".join(re.findall(r'"([^"]*)"', statement))
            for instruction in re.split(r";|\\n", code):
                if "cp.async" in instruction:
                    assert "multicast" not in instruction, (os.path.basename(f), instruction)


def test_every_kernel_file_has_the_debug_build_check_its_addresses():
    """Kernels that touch a caller's operands check the addresses in the debug
    build (debug_check.cuh); the self-test and the status reader touch none."""
    for f in sorted(glob.glob(os.path.join(sgbuild.CSRC, "*.cu"))):
        with open(f) as fh:
            text = fh.read()
        if "__global__" in text and os.path.basename(f) not in ("selftest.cu", "status.cu",
                                                                             "attention_tc.cu"):
            assert "dbg_in_" in text, os.path.basename(f)
