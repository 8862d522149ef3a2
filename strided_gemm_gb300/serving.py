"""The 16-bit serving operators of libsbgemm: the strided product, latent
attention over a paged cache or over packed sequences, and the operations on a
cache's pages (include/sbgemm.h has each one's definition).

The sbgemm_* functions carry the C names and arguments; the others take torch
CUDA tensors, read strides from them, and run on the tensors' device and its
current stream unless a stream is given.  A non-zero status raises
SbgemmError; what only the device can see (block ids, lengths, page requests)
is reported by the next sbgemm_device_status.
"""

from __future__ import annotations

import ctypes

import strided_gemm_gb300 as _sg

_i64, _vp, _int, _f32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float
_size = ctypes.c_size_t


class _Pool(ctypes.Structure):
    _fields_ = [("caches", ctypes.POINTER(_vp)), ("page_bytes", ctypes.POINTER(_i64)),
                ("n_caches", _i64), ("num_blocks", _i64), ("block_size", _i64),
                ("ref_counts", _vp), ("block_table", _vp), ("n_seqs", _i64),
                ("max_blocks", _i64), ("seq_lens", _vp)]


def declare(lib) -> None:
    """Sets the argument types of the library's serving functions."""
    opt = ctypes.POINTER(_sg._Options)
    pool = ctypes.POINTER(_Pool)
    arguments = {
        "sbgemm_half": [_int] + [_vp, _i64, _i64, _i64] * 3 + [_i64] * 4 + [_f32, _int, _vp],
        "sbgemm_latent_attention_paged":
            [_int, _vp] + [_i64] * 3 + [_vp] + [_i64] * 4 + [_vp, _i64, _vp, _vp] + [_i64] * 9 +
            [_f32, _int, _vp, opt],
        "sbgemm_latent_workspace_bytes": [_int, ctypes.POINTER(_size)],
        "sbgemm_latent_attention":
            [_int, _vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _i64, _vp, _vp,
             _i64, _i64, _vp, _i64, _i64] + [_i64] * 4 + [_f32, _int, _vp],
        "sbgemm_pages_workspace_bytes": [_i64, _i64, _i64, ctypes.POINTER(_size)],
        "sbgemm_pages_copy": [pool, _vp, _i64, _vp, opt],
        "sbgemm_pages_fork": [pool, _vp, _vp, _i64, _vp, opt],
        "sbgemm_pages_append": [pool, _vp, _vp, _i64, ctypes.POINTER(_vp), ctypes.POINTER(_i64), _i64, _vp, opt],
        "sbgemm_pages_free": [pool, _vp, _i64, _vp],
        "sbgemm_pages_compact": [pool, _vp, _vp, opt],
    }
    for name, types in arguments.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = _int, types


def bind(fast, lib) -> None:
    """Hands the fast-call module (csrc/fastcall.c) the serving functions' addresses."""
    fast.bind_serving(*(ctypes.cast(getattr(lib, name), _vp).value for name in (
        "sbgemm_half", "sbgemm_latent_attention_paged", "sbgemm_latent_attention", "sbgemm_pages_copy",
        "sbgemm_pages_fork", "sbgemm_pages_append", "sbgemm_pages_free", "sbgemm_pages_compact")))


def _lib():
    return _sg._lib if _sg._lib is not None else _sg.load()


def _check(st: int, where: str) -> None:
    if st:
        raise _sg.SbgemmError(st, where)


# ---- the C functions ------------------------------------------------------------

def sbgemm_half(type, A, rsA, csA, bsA, B, rsB, csB, bsB, C, rsC, csC, bsC,
                M, N, K, batch, alpha=1.0, accumulate=0, stream=0) -> None:
    """C <- alpha*A*B (+C) on 16-bit operands (type: TYPE_BF16 or TYPE_FP16)."""
    lib = _lib()
    if _sg._fast is not None:
        st = _sg._fast.half(type, A, rsA, csA, bsA, B, rsB, csB, bsB, C, rsC, csC, bsC, M, N, K, batch, alpha,
                            accumulate, stream or 0)
    else:
        st = lib.sbgemm_half(type, A, rsA, csA, bsA, B, rsB, csB, bsB, C, rsC, csC, bsC,
                             M, N, K, batch, alpha, 1 if accumulate else 0, stream or None)
    if st:
        raise _sg.SbgemmError(st, "sbgemm_half")


def sbgemm_latent_attention_paged(type, Q, hsQ, tsQ, bsQ, cache, rsC, psC, num_blocks, block_size,
                                  block_table, max_blocks, seq_lens, O, hsO, tsO, bsO, q_len, heads, N,
                                  R, P, n_seqs, alpha, causal=0, stream=0, workspace: int = 0,
                                  workspace_bytes: int = 0) -> None:
    """Latent attention, absorbed form, over a paged cache of [c | k_rope] rows."""
    lib = _lib()
    o = _sg._opts_ref(_sg.MATH_FP32, _sg.PATH_AUTO, workspace, workspace_bytes, _sg.KSPLIT_ANY)
    if _sg._fast is not None:
        st = _sg._fast.paged(type, Q, hsQ, tsQ, bsQ, cache, rsC, psC, num_blocks, block_size, block_table,
                             max_blocks, seq_lens or 0, O, hsO, tsO, bsO, q_len, heads, N, R, P, n_seqs, alpha,
                             int(causal), stream or 0, o[2])
    else:
        st = lib.sbgemm_latent_attention_paged(
            type, Q, hsQ, tsQ, bsQ, cache, rsC, psC, num_blocks, block_size, block_table, max_blocks,
            seq_lens or None, O, hsO, tsO, bsO, q_len, heads, N, R, P, n_seqs, alpha, int(causal),
            stream or None, o[1])
    if st:
        raise _sg.SbgemmError(st, "sbgemm_latent_attention_paged")


def sbgemm_latent_workspace_bytes(device: int = 0) -> int:
    """Bytes of workspace with which latent_attention_paged splits keys freely."""
    n = _size(0)
    _check(_lib().sbgemm_latent_workspace_bytes(int(device), ctypes.byref(n)), "sbgemm_latent_workspace_bytes")
    return n.value


def sbgemm_latent_attention(type, Q, hsQ, tsQ, total_q, K_nope, hsK, tsK, K_rope, tsR, V, hsV, tsV, total_k,
                            q_starts, k_starts, n_seqs, max_q, O, hsO, tsO, heads, Dn, P, Dv, alpha,
                            causal=0, stream=0) -> None:
    """Latent attention, expanded form, over packed sequences."""
    lib = _lib()
    if _sg._fast is not None:
        st = _sg._fast.packed(type, Q, hsQ, tsQ, total_q, K_nope or 0, hsK, tsK, K_rope or 0, tsR, V or 0, hsV,
                              tsV, total_k, q_starts, k_starts, n_seqs, max_q, O, hsO, tsO, heads, Dn, P, Dv,
                              alpha, int(causal), stream or 0)
    else:
        st = lib.sbgemm_latent_attention(
            type, Q, hsQ, tsQ, total_q, K_nope or None, hsK, tsK, K_rope or None, tsR, V or None, hsV, tsV,
            total_k, q_starts, k_starts, n_seqs, max_q, O, hsO, tsO, heads, Dn, P, Dv, alpha, int(causal),
            stream or None)
    if st:
        raise _sg.SbgemmError(st, "sbgemm_latent_attention")


def sbgemm_pages_workspace_bytes(num_blocks: int, n_seqs: int, n: int) -> int:
    """Bytes of workspace for any page operation with up to n requests."""
    b = _size(0)
    _check(_lib().sbgemm_pages_workspace_bytes(int(num_blocks), int(n_seqs), int(n), ctypes.byref(b)),
           "sbgemm_pages_workspace_bytes")
    return b.value


# ---- torch helpers --------------------------------------------------------------
#
# A decode step's launches take a few microseconds on the GPU, so what these
# helpers spend on the host counts: shapes, strides and devices are read once
# each, and nothing is allocated or looked up that a call does not need.

_torch = None
_kinds: dict = {}
_raw_stream = _get_device = None


def _setup():
    global _torch, _raw_stream, _get_device
    import torch
    _kinds.update({torch.bfloat16: _sg.TYPE_BF16, torch.float16: _sg.TYPE_FP16})
    # The handle of a device's current stream without building a Stream object.
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda d: torch.cuda.current_stream(d).cuda_stream)
    _get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _torch = torch


def _kind(t, name):
    if _torch is None:
        _setup()
    k = _kinds.get(t.dtype)
    if k is None:
        raise TypeError(f"{name} must be a bfloat16 or float16 tensor")
    return k


def _device(t):
    d = t.get_device()
    if d < 0:
        raise TypeError("the tensors must be CUDA tensors")
    return d


def _same(t, name, dtype, dev):
    if t.dtype != dtype or t.get_device() != dev:
        raise TypeError(f"{name} must be a {dtype} tensor on cuda:{dev}")


def _ints(t, name, dev):
    """The address of an int32 array on the device."""
    if t.dtype != _torch.int32 or t.get_device() != dev:
        raise TypeError(f"{name} must be an int32 tensor on cuda:{dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _run(dev, stream, f, *args):
    """f(*args, stream handle) with the tensors' device as the current one."""
    if stream is None:
        stream = _raw_stream(dev)
    if _get_device() != dev:
        with _torch.cuda.device(dev):
            return f(*args, stream)
    return f(*args, stream)


def _workspace(ws, dev):
    if ws is None:
        return 0, 0
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("the workspace must be a contiguous tensor on the operands' device")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def matmul_half(A, B, C, alpha: float = 1.0, accumulate: bool = False, stream=None):
    """C <- alpha*A@B (+C) on torch CUDA bfloat16 or float16 tensors viewed as
    [batch, M, K], [batch, K, N] and [batch, M, N] (2-D means batch 1; A and B
    may have batch 1 to be shared), any strides.  Returns C."""
    A3, B3, C3 = (t if t.dim() == 3 else _sg._as3(t, n) for t, n in ((A, "A"), (B, "B"), (C, "C")))
    kind, dev, dtype = _kind(C3, "C"), _device(C3), C3.dtype
    _same(A3, "A", dtype, dev)
    _same(B3, "B", dtype, dev)
    batch, M, N = C3.shape
    nA, mA, K = A3.shape
    nB, kB, nN = B3.shape
    if mA != M or kB != K or nN != N:
        raise ValueError(f"shape mismatch: A{tuple(A3.shape)} B{tuple(B3.shape)} C{tuple(C3.shape)}")
    if (nA != batch and nA != 1) or (nB != batch and nB != 1):
        raise ValueError(f"batches {nA} of A and {nB} of B do not match {batch}")
    ba, ra, ca = A3.stride()
    bb, rb, cb = B3.stride()
    bc, rc, cc = C3.stride()
    _run(dev, stream, _half_on, kind, A3.data_ptr(), ra, ca, ba if nA == batch else 0,
         B3.data_ptr(), rb, cb, bb if nB == batch else 0, C3.data_ptr(), rc, cc, bc, M, N, K, batch, alpha,
         accumulate)
    return C


# The C functions with the stream last.
_half_on = sbgemm_half


def _paged_on(*args):
    sbgemm_latent_attention_paged(*args[:-3], args[-1], args[-3], args[-2])


_packed_on = sbgemm_latent_attention


def latent_attention_paged(Q, cache, block_table, seq_lens, O, alpha, causal: bool = True,
                           workspace=None, max_len=None, stream=None):
    """Latent attention, absorbed form: Q [n_seqs, q_len, heads, R + P] against
    the rows [c | k_rope] of cache [num_blocks, block_size, R + P] that
    block_table (int32 [n_seqs, max_blocks]) and seq_lens (int32 [n_seqs]; None
    for max_len everywhere) give each sequence; O [n_seqs, q_len, heads, R]
    receives the averaged c.  bfloat16 or float16, unit stride along the last
    axis.  max_len: the longest length (default: what the table can hold); a
    workspace of sbgemm_latent_workspace_bytes splits the keys over the GPU.
    Returns O."""
    kind, dev, dtype = _kind(O, "O"), _device(O), O.dtype
    _same(Q, "Q", dtype, dev)
    _same(cache, "cache", dtype, dev)
    table = _ints(block_table, "block_table", dev)
    if Q.dim() != 4 or O.dim() != 4 or cache.dim() != 3 or block_table.dim() != 2:
        raise ValueError("Q and O are 4-D, cache is 3-D, block_table is 2-D")
    n_seqs, q_len, heads, wide = Q.shape
    num_blocks, block_size, row = cache.shape
    n_o, q_o, h_o, R = O.shape
    n_t, max_blocks = block_table.shape
    if n_o != n_seqs or q_o != q_len or h_o != heads or row != wide or R > wide or n_t != n_seqs:
        raise ValueError(f"shape mismatch: Q{tuple(Q.shape)} cache{tuple(cache.shape)} "
                         f"block_table{tuple(block_table.shape)} O{tuple(O.shape)}")
    lens = 0
    if seq_lens is not None:
        lens = _ints(seq_lens, "seq_lens", dev)
        if tuple(seq_lens.shape) != (n_seqs,):
            raise ValueError(f"seq_lens must have shape ({n_seqs},)")
    bq, tq, hq, eq = Q.stride()
    bo, to, ho, eo = O.stride()
    pc, rc, ec = cache.stride()
    if (wide > 1 and (eq != 1 or ec != 1)) or (R > 1 and eo != 1):
        raise ValueError("Q, cache and O need unit stride along their last axis")
    N = max_blocks * block_size if max_len is None else int(max_len)
    ws, ws_bytes = _workspace(workspace, dev)
    _run(dev, stream, _paged_on, kind, Q.data_ptr(), hq, tq, bq, cache.data_ptr(), rc, pc, num_blocks,
         block_size, table, max_blocks, lens, O.data_ptr(), ho, to, bo, q_len, heads, N, R, wide - R, n_seqs,
         alpha, causal, ws, ws_bytes)
    return O


def latent_attention(Q, K_nope, K_rope, V, O, q_starts, k_starts, max_q, alpha, causal: bool = True,
                     stream=None):
    """Latent attention, expanded form, over packed sequences: Q [total_q,
    heads, Dn + P], K_nope [total_k, heads, Dn], K_rope [total_k, P] (shared by
    the heads), V [total_k, heads, Dv], O [total_q, heads, Dv]; sequence s has
    the rows q_starts[s]..q_starts[s+1] of Q and O and k_starts[s]..
    k_starts[s+1] of the keys (int32 [n_seqs + 1]), at most max_q queries.
    bfloat16 or float16, unit stride along the last axis.  Returns O."""
    kind, dev, dtype = _kind(O, "O"), _device(O), O.dtype
    for t, name in ((Q, "Q"), (K_nope, "K_nope"), (K_rope, "K_rope"), (V, "V")):
        _same(t, name, dtype, dev)
    qs, ks = _ints(q_starts, "q_starts", dev), _ints(k_starts, "k_starts", dev)
    total_q, heads, wide = Q.shape
    total_k, h_k, Dn = K_nope.shape
    n_v, h_v, Dv = V.shape
    n_r, P = K_rope.shape
    n_seqs = q_starts.numel() - 1
    if (h_k != heads or n_v != total_k or h_v != heads or n_r != total_k or wide != Dn + P or
            tuple(O.shape) != (total_q, heads, Dv) or k_starts.numel() != n_seqs + 1 or n_seqs < 0):
        raise ValueError(f"shape mismatch: Q{tuple(Q.shape)} K_nope{tuple(K_nope.shape)} "
                         f"K_rope{tuple(K_rope.shape)} V{tuple(V.shape)} O{tuple(O.shape)} "
                         f"q_starts{tuple(q_starts.shape)} k_starts{tuple(k_starts.shape)}")
    tq, hq, eq = Q.stride()
    tk, hk, ek = K_nope.stride()
    tr, er = K_rope.stride()
    tv, hv, ev = V.stride()
    to, ho, eo = O.stride()
    if ((eq != 1 and wide > 1) or (ek != 1 and Dn > 1) or (er != 1 and P > 1) or
            ((ev != 1 or eo != 1) and Dv > 1)):
        raise ValueError("Q, K_nope, K_rope, V and O need unit stride along their last axis")
    _run(dev, stream, _packed_on, kind, Q.data_ptr(), hq, tq, total_q, K_nope.data_ptr(), hk, tk,
         K_rope.data_ptr(), tr, V.data_ptr(), hv, tv, total_k, qs, ks, n_seqs, int(max_q), O.data_ptr(), ho, to,
         heads, Dn, P, Dv, alpha, causal)
    return O


_OPS = ("sbgemm_pages_copy", "sbgemm_pages_fork", "sbgemm_pages_append", "sbgemm_pages_free",
        "sbgemm_pages_compact")
_COPY, _FORK, _APPEND, _FREE, _COMPACT = range(5)


def _pages_on(op, caches, sizes, num_blocks, block_size, refs, table, n_seqs, max_blocks, lens, a, b, n, rows,
              strides, total, ws, ws_bytes, stream):
    """One page operation: the fast-call module's, or the same through ctypes."""
    lib = _lib()
    o = _sg._opts_ref(_sg.MATH_FP32, _sg.PATH_AUTO, ws, ws_bytes, _sg.KSPLIT_ANY)
    if _sg._fast is not None:
        st = _sg._fast.pages(op, caches, sizes, num_blocks, block_size, refs, table, n_seqs, max_blocks, lens,
                             a, b, n, rows, strides, total, stream, o[2])
    else:
        p = _Pool()
        p.caches, p.page_bytes = (_vp * len(caches))(*caches), (_i64 * len(sizes))(*sizes)
        p.n_caches, p.num_blocks, p.block_size = len(caches), num_blocks, block_size
        p.ref_counts, p.block_table, p.seq_lens = refs or None, table or None, lens or None
        p.n_seqs, p.max_blocks = n_seqs, max_blocks
        ref, s = ctypes.byref(p), stream or None
        if op == _COPY:
            st = lib.sbgemm_pages_copy(ref, a, n, s, o[1])
        elif op == _FORK:
            st = lib.sbgemm_pages_fork(ref, a, b, n, s, o[1])
        elif op == _APPEND:
            st = lib.sbgemm_pages_append(ref, a, b, n, (_vp * len(rows))(*rows), (_i64 * len(rows))(*strides),
                                         total, s, o[1])
        elif op == _FREE:
            st = lib.sbgemm_pages_free(ref, a, n, s)
        else:
            st = lib.sbgemm_pages_compact(ref, a or None, s, o[1])
    if st:
        raise _sg.SbgemmError(st, _OPS[op])


def _caches(caches):
    """(device, addresses, bytes a page, num_blocks, block_size) of a pool's
    caches [num_blocks, block_size, ...], contiguous, on one device."""
    if _torch is None:
        _setup()
    if not caches:
        raise ValueError("at least one cache gives the pool its block size")
    num_blocks, block_size = caches[0].shape[:2]
    dev = _device(caches[0])
    pointers, sizes = [], []
    for c in caches:
        shape = c.shape
        if c.get_device() != dev or not c.is_contiguous():
            raise TypeError("the caches must be contiguous CUDA tensors on one device")
        if len(shape) < 2 or shape[0] != num_blocks or shape[1] != block_size:
            raise ValueError("the caches must share [num_blocks, block_size]")
        pointers.append(c.data_ptr())
        sizes.append(c.numel() // num_blocks * c.element_size() if num_blocks else 0)
    return dev, tuple(pointers), tuple(sizes), num_blocks, block_size


def _books(ref_counts, block_table, seq_lens, num_blocks, dev):
    """(addresses of) ref_counts, block_table, n_seqs, max_blocks, seq_lens."""
    if block_table.dim() != 2:
        raise ValueError("block_table must be [n_seqs, max_blocks]")
    n_seqs, max_blocks = block_table.shape
    if ref_counts.numel() != num_blocks or seq_lens.numel() != n_seqs:
        raise ValueError(f"shape mismatch: ref_counts{tuple(ref_counts.shape)} for {num_blocks} blocks, "
                         f"block_table{tuple(block_table.shape)} seq_lens{tuple(seq_lens.shape)}")
    return (_ints(ref_counts, "ref_counts", dev), _ints(block_table, "block_table", dev), n_seqs, max_blocks,
            _ints(seq_lens, "seq_lens", dev))


def pages_copy(caches, pairs, workspace, stream=None) -> None:
    """Copies page pairs[k, 0] to page pairs[k, 1] (int32 [n, 2]) in every cache
    [num_blocks, block_size, ...] of the list."""
    dev, ptrs, sizes, num_blocks, block_size = _caches(caches)
    if pairs.dim() != 2 or pairs.shape[1] != 2:
        raise ValueError("pairs must be [n, 2]")
    _run(dev, stream, _pages_on, _COPY, ptrs, sizes, num_blocks, block_size, 0, 0, 0, 0, 0,
         _ints(pairs, "pairs", dev), 0, pairs.shape[0], (), (), 0, *_workspace(workspace, dev))


def pages_fork(caches, ref_counts, block_table, seq_lens, parents, children, workspace, stream=None) -> None:
    """Sequence children[k] becomes a copy of sequence parents[k] (int32 [n]):
    full pages shared, the rows of an unfinished last page copied."""
    dev, ptrs, sizes, num_blocks, block_size = _caches(caches)
    n = parents.numel()
    if children.numel() != n:
        raise ValueError("parents and children must have one length")
    _run(dev, stream, _pages_on, _FORK, ptrs, sizes, num_blocks, block_size,
         *_books(ref_counts, block_table, seq_lens, num_blocks, dev), _ints(parents, "parents", dev),
         _ints(children, "children", dev), n, (), (), 0, *_workspace(workspace, dev))


def pages_append(caches, ref_counts, block_table, seq_lens, seqs, starts, rows, workspace,
                 stream=None) -> None:
    """Sequence seqs[k] (int32 [n]) grows by the tokens starts[k]..starts[k+1]
    (int32 [n + 1]) of the rows [total, ...], one tensor a cache."""
    dev, ptrs, sizes, num_blocks, block_size = _caches(caches)
    n = seqs.numel()
    if starts.numel() != n + 1 or len(rows) != len(caches):
        raise ValueError("starts has one entry more than seqs, rows one tensor for each cache")
    total = rows[0].shape[0]
    pointers, strides = [], []
    for i, (r, c) in enumerate(zip(rows, caches)):
        shape = r.shape
        if r.get_device() != dev or r.dtype != c.dtype or shape[0] != total or shape[1:] != c.shape[2:]:
            raise ValueError(f"rows[{i}] must be {(total,) + tuple(c.shape[2:])} of its cache's type")
        if total and not r.is_contiguous() and not r[0].is_contiguous():
            raise ValueError(f"a token's row in rows[{i}] must be contiguous")
        pointers.append(r.data_ptr())
        strides.append(r.stride(0) * r.element_size())
    _run(dev, stream, _pages_on, _APPEND, ptrs, sizes, num_blocks, block_size,
         *_books(ref_counts, block_table, seq_lens, num_blocks, dev), _ints(seqs, "seqs", dev),
         _ints(starts, "starts", dev), n, tuple(pointers), tuple(strides), total, *_workspace(workspace, dev))


def pages_free(caches, ref_counts, block_table, seq_lens, seqs, stream=None) -> None:
    """Frees the sequences seqs (int32 [n]): their pages' counts fall by one and
    their lengths become 0."""
    dev, ptrs, sizes, num_blocks, block_size = _caches(caches)
    _run(dev, stream, _pages_on, _FREE, ptrs, sizes, num_blocks, block_size,
         *_books(ref_counts, block_table, seq_lens, num_blocks, dev), _ints(seqs, "seqs", dev), 0, seqs.numel(),
         (), (), 0, 0, 0)


def pages_compact(caches, ref_counts, block_table, seq_lens, workspace, moved=None, stream=None) -> None:
    """Moves the pages in use to the front of the pool, table entries and counts
    with them; moved (int32 [1], optional) receives how many moved."""
    dev, ptrs, sizes, num_blocks, block_size = _caches(caches)
    if moved is not None and moved.numel() < 1:
        raise ValueError("moved must hold one int32")
    _run(dev, stream, _pages_on, _COMPACT, ptrs, sizes, num_blocks, block_size,
         *_books(ref_counts, block_table, seq_lens, num_blocks, dev),
         0 if moved is None else _ints(moved, "moved", dev), 0, 0, (), (), 0, *_workspace(workspace, dev))
