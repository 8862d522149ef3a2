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


def _lib():
    return _sg._lib if _sg._lib is not None else _sg.load()


def _check(st: int, where: str) -> None:
    if st:
        raise _sg.SbgemmError(st, where)


# ---- the C functions ------------------------------------------------------------

def sbgemm_half(type, A, rsA, csA, bsA, B, rsB, csB, bsB, C, rsC, csC, bsC,
                M, N, K, batch, alpha=1.0, accumulate=0, stream=0) -> None:
    """C <- alpha*A*B (+C) on 16-bit operands (type: TYPE_BF16 or TYPE_FP16)."""
    _check(_lib().sbgemm_half(type, A, rsA, csA, bsA, B, rsB, csB, bsB, C, rsC, csC, bsC,
                              M, N, K, batch, alpha, 1 if accumulate else 0, stream or None), "sbgemm_half")


def sbgemm_latent_attention_paged(type, Q, hsQ, tsQ, bsQ, cache, rsC, psC, num_blocks, block_size,
                                  block_table, max_blocks, seq_lens, O, hsO, tsO, bsO, q_len, heads, N,
                                  R, P, n_seqs, alpha, causal=0, stream=0, workspace: int = 0,
                                  workspace_bytes: int = 0) -> None:
    """Latent attention, absorbed form, over a paged cache of [c | k_rope] rows."""
    o = _sg._opts_ref(_sg.MATH_FP32, _sg.PATH_AUTO, workspace, workspace_bytes, _sg.KSPLIT_ANY)
    _check(_lib().sbgemm_latent_attention_paged(
        type, Q, hsQ, tsQ, bsQ, cache, rsC, psC, num_blocks, block_size, block_table, max_blocks,
        seq_lens or None, O, hsO, tsO, bsO, q_len, heads, N, R, P, n_seqs, alpha, int(causal),
        stream or None, o[1]), "sbgemm_latent_attention_paged")


def sbgemm_latent_workspace_bytes(device: int = 0) -> int:
    """Bytes of workspace with which latent_attention_paged splits keys freely."""
    n = _size(0)
    _check(_lib().sbgemm_latent_workspace_bytes(int(device), ctypes.byref(n)), "sbgemm_latent_workspace_bytes")
    return n.value


def sbgemm_latent_attention(type, Q, hsQ, tsQ, total_q, K_nope, hsK, tsK, K_rope, tsR, V, hsV, tsV, total_k,
                            q_starts, k_starts, n_seqs, max_q, O, hsO, tsO, heads, Dn, P, Dv, alpha,
                            causal=0, stream=0) -> None:
    """Latent attention, expanded form, over packed sequences."""
    _check(_lib().sbgemm_latent_attention(
        type, Q, hsQ, tsQ, total_q, K_nope or None, hsK, tsK, K_rope or None, tsR, V or None, hsV, tsV,
        total_k, q_starts, k_starts, n_seqs, max_q, O, hsO, tsO, heads, Dn, P, Dv, alpha, int(causal),
        stream or None), "sbgemm_latent_attention")


def sbgemm_pages_workspace_bytes(num_blocks: int, n_seqs: int, n: int) -> int:
    """Bytes of workspace for any page operation with up to n requests."""
    b = _size(0)
    _check(_lib().sbgemm_pages_workspace_bytes(int(num_blocks), int(n_seqs), int(n), ctypes.byref(b)),
           "sbgemm_pages_workspace_bytes")
    return b.value


# ---- torch helpers --------------------------------------------------------------

def _type_of(t, name):
    import torch
    if t.dtype == torch.bfloat16:
        return _sg.TYPE_BF16
    if t.dtype == torch.float16:
        return _sg.TYPE_FP16
    raise TypeError(f"{name} must be a bfloat16 or float16 tensor")


def _same(ref, dtype, **tensors):
    """Every tensor on the CUDA device of `ref` and of the type asked for."""
    dev = ref.device
    if dev.type != "cuda":
        raise TypeError("the tensors must be CUDA tensors")
    for name, t in tensors.items():
        if t.dtype != dtype or t.device != dev:
            raise TypeError(f"{name} must be a {dtype} tensor on {dev}")


def _int32(ref, **tensors):
    import torch
    _same(ref, torch.int32, **tensors)
    for name, t in tensors.items():
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


class _On:
    """Runs the library's call with the tensors' device as the current one;
    gives the stream handle."""

    __slots__ = ("guard", "stream")

    def __init__(self, device, stream):
        import torch
        self.guard = None
        if device.index is not None and device.index != torch.cuda.current_device():
            self.guard = torch.cuda.device(device)
        self.stream = torch.cuda.current_stream(device).cuda_stream if stream is None else stream

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self.stream

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _workspace(ws, ref):
    if ws is None:
        return 0, 0
    if ws.device != ref.device or not ws.is_contiguous():
        raise ValueError("the workspace must be a contiguous tensor on the operands' device")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def matmul_half(A, B, C, alpha: float = 1.0, accumulate: bool = False, stream=None):
    """C <- alpha*A@B (+C) on torch CUDA bfloat16 or float16 tensors viewed as
    [batch, M, K], [batch, K, N] and [batch, M, N] (2-D means batch 1; A and B
    may have batch 1 to be shared), any strides.  Returns C."""
    A3, B3, C3 = _sg._as3(A, "A"), _sg._as3(B, "B"), _sg._as3(C, "C")
    kind = _type_of(C3, "C")
    _same(C3, C3.dtype, A=A3, B=B3)
    batch, M, N = C3.shape
    K = A3.shape[2]
    if A3.shape[1] != M or B3.shape[1] != K or B3.shape[2] != N:
        raise ValueError(f"shape mismatch: A{tuple(A3.shape)} B{tuple(B3.shape)} C{tuple(C3.shape)}")
    for t, n in ((A3, "A"), (B3, "B")):
        if t.shape[0] not in (1, batch):
            raise ValueError(f"{n} batch {t.shape[0]} does not match {batch}")
    ba, ra, ca = A3.stride()
    bb, rb, cb = B3.stride()
    bc, rc, cc = C3.stride()
    with _On(C3.device, stream) as s:
        sbgemm_half(kind, A3.data_ptr(), ra, ca, ba if A3.shape[0] == batch else 0,
                    B3.data_ptr(), rb, cb, bb if B3.shape[0] == batch else 0,
                    C3.data_ptr(), rc, cc, bc, M, N, K, batch, alpha, accumulate, s)
    return C


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
    kind = _type_of(O, "O")
    _same(O, O.dtype, Q=Q, cache=cache)
    if Q.dim() != 4 or O.dim() != 4 or cache.dim() != 3 or block_table.dim() != 2:
        raise ValueError("Q and O are 4-D, cache is 3-D, block_table is 2-D")
    n_seqs, q_len, heads, wide = Q.shape
    num_blocks, block_size, row = cache.shape
    R = O.shape[3]
    if tuple(O.shape[:3]) != (n_seqs, q_len, heads) or row != wide or R > wide or block_table.shape[0] != n_seqs:
        raise ValueError(f"shape mismatch: Q{tuple(Q.shape)} cache{tuple(cache.shape)} "
                         f"block_table{tuple(block_table.shape)} O{tuple(O.shape)}")
    _int32(O, block_table=block_table)
    if seq_lens is not None:
        _int32(O, seq_lens=seq_lens)
        if tuple(seq_lens.shape) != (n_seqs,):
            raise ValueError(f"seq_lens must have shape ({n_seqs},)")
    bq, tq, hq, eq = Q.stride()
    bo, to, ho, eo = O.stride()
    pc, rc, ec = cache.stride()
    if (wide > 1 and (eq != 1 or ec != 1)) or (R > 1 and eo != 1):
        raise ValueError("Q, cache and O need unit stride along their last axis")
    max_blocks = block_table.shape[1]
    N = max_blocks * block_size if max_len is None else int(max_len)
    ws, ws_bytes = _workspace(workspace, O)
    with _On(O.device, stream) as s:
        sbgemm_latent_attention_paged(kind, Q.data_ptr(), hq, tq, bq, cache.data_ptr(), rc, pc, num_blocks,
                                      block_size, block_table.data_ptr(), max_blocks,
                                      0 if seq_lens is None else seq_lens.data_ptr(),
                                      O.data_ptr(), ho, to, bo, q_len, heads, N, R, wide - R, n_seqs,
                                      alpha, causal, s, ws, ws_bytes)
    return O


def latent_attention(Q, K_nope, K_rope, V, O, q_starts, k_starts, max_q, alpha, causal: bool = True,
                     stream=None):
    """Latent attention, expanded form, over packed sequences: Q [total_q,
    heads, Dn + P], K_nope [total_k, heads, Dn], K_rope [total_k, P] (shared by
    the heads), V [total_k, heads, Dv], O [total_q, heads, Dv]; sequence s has
    the rows q_starts[s]..q_starts[s+1] of Q and O and k_starts[s]..
    k_starts[s+1] of the keys (int32 [n_seqs + 1]), at most max_q queries.
    bfloat16 or float16, unit stride along the last axis.  Returns O."""
    kind = _type_of(O, "O")
    _same(O, O.dtype, Q=Q, K_nope=K_nope, K_rope=K_rope, V=V)
    _int32(O, q_starts=q_starts, k_starts=k_starts)
    total_q, heads, wide = Q.shape
    total_k, _, Dn = K_nope.shape
    Dv, P = V.shape[2], K_rope.shape[1]
    n_seqs = q_starts.numel() - 1
    if (tuple(K_nope.shape[:2]) != (total_k, heads) or tuple(V.shape[:2]) != (total_k, heads) or
            K_rope.shape[0] != total_k or wide != Dn + P or tuple(O.shape) != (total_q, heads, Dv) or
            k_starts.numel() != n_seqs + 1 or n_seqs < 0):
        raise ValueError(f"shape mismatch: Q{tuple(Q.shape)} K_nope{tuple(K_nope.shape)} "
                         f"K_rope{tuple(K_rope.shape)} V{tuple(V.shape)} O{tuple(O.shape)} "
                         f"q_starts{tuple(q_starts.shape)} k_starts{tuple(k_starts.shape)}")
    tq, hq, eq = Q.stride()
    tk, hk, ek = K_nope.stride()
    tr, er = K_rope.stride()
    tv, hv, ev = V.stride()
    to, ho, eo = O.stride()
    if any(n > 1 and e != 1 for n, e in ((wide, eq), (Dn, ek), (P, er), (Dv, ev), (Dv, eo))):
        raise ValueError("Q, K_nope, K_rope, V and O need unit stride along their last axis")
    with _On(O.device, stream) as s:
        sbgemm_latent_attention(kind, Q.data_ptr(), hq, tq, total_q, K_nope.data_ptr(), hk, tk,
                                K_rope.data_ptr(), tr, V.data_ptr(), hv, tv, total_k,
                                q_starts.data_ptr(), k_starts.data_ptr(), n_seqs, int(max_q),
                                O.data_ptr(), ho, to, heads, Dn, P, Dv, alpha, causal, s)
    return O


def _pool(caches, ref_counts=None, block_table=None, seq_lens=None):
    """The C struct of a pool; every cache [num_blocks, block_size, ...] contiguous."""
    first = caches[0] if caches else ref_counts
    p = _Pool()
    n = len(caches)
    if n:
        num_blocks, block_size = first.shape[:2]
        pointers, sizes = (_vp * n)(), (_i64 * n)()
        for i, c in enumerate(caches):
            if c.device != first.device or c.device.type != "cuda" or not c.is_contiguous():
                raise TypeError("the caches must be contiguous CUDA tensors on one device")
            if c.dim() < 2 or c.shape[0] != num_blocks or c.shape[1] != block_size:
                raise ValueError("the caches must share [num_blocks, block_size]")
            pointers[i] = c.data_ptr()
            sizes[i] = c.numel() // num_blocks * c.element_size() if num_blocks else 0
        p.caches, p.page_bytes, p.n_caches = pointers, sizes, n
        p.num_blocks, p.block_size = num_blocks, block_size
    if ref_counts is not None:
        _int32(first, ref_counts=ref_counts, block_table=block_table, seq_lens=seq_lens)
        if not n:
            raise ValueError("at least one cache gives the pool its block size")
        if (tuple(ref_counts.shape) != (p.num_blocks,) or block_table.dim() != 2 or
                tuple(seq_lens.shape) != (block_table.shape[0],)):
            raise ValueError(f"shape mismatch: ref_counts{tuple(ref_counts.shape)} "
                             f"block_table{tuple(block_table.shape)} seq_lens{tuple(seq_lens.shape)}")
        p.ref_counts, p.block_table = ref_counts.data_ptr(), block_table.data_ptr()
        p.seq_lens = seq_lens.data_ptr()
        p.n_seqs, p.max_blocks = block_table.shape
    return p


def _pages_options(workspace, ref):
    ws, ws_bytes = _workspace(workspace, ref)
    return _sg._opts_ref(_sg.MATH_FP32, _sg.PATH_AUTO, ws, ws_bytes, _sg.KSPLIT_ANY)[1]


def pages_copy(caches, pairs, workspace, stream=None) -> None:
    """Copies page pairs[k, 0] to page pairs[k, 1] (int32 [n, 2]) in every cache
    [num_blocks, block_size, ...] of the list."""
    p = _pool(caches)
    _int32(caches[0], pairs=pairs)
    if pairs.dim() != 2 or pairs.shape[1] != 2:
        raise ValueError("pairs must be [n, 2]")
    o = _pages_options(workspace, pairs)
    with _On(pairs.device, stream) as s:
        _check(_lib().sbgemm_pages_copy(ctypes.byref(p), pairs.data_ptr(), pairs.shape[0], s or None, o),
               "sbgemm_pages_copy")


def pages_fork(caches, ref_counts, block_table, seq_lens, parents, children, workspace, stream=None) -> None:
    """Sequence children[k] becomes a copy of sequence parents[k] (int32 [n]):
    full pages shared, the rows of an unfinished last page copied."""
    p = _pool(caches, ref_counts, block_table, seq_lens)
    _int32(ref_counts, parents=parents, children=children)
    n = parents.numel()
    if children.numel() != n:
        raise ValueError("parents and children must have one length")
    o = _pages_options(workspace, ref_counts)
    with _On(ref_counts.device, stream) as s:
        _check(_lib().sbgemm_pages_fork(ctypes.byref(p), parents.data_ptr(), children.data_ptr(), n,
                                        s or None, o), "sbgemm_pages_fork")


def pages_append(caches, ref_counts, block_table, seq_lens, seqs, starts, rows, workspace,
                 stream=None) -> None:
    """Sequence seqs[k] (int32 [n]) grows by the tokens starts[k]..starts[k+1]
    (int32 [n + 1]) of the rows [total, ...], one tensor a cache."""
    p = _pool(caches, ref_counts, block_table, seq_lens)
    _int32(ref_counts, seqs=seqs, starts=starts)
    n, total = seqs.numel(), rows[0].shape[0]
    if starts.numel() != n + 1 or len(rows) != len(caches):
        raise ValueError("starts has one entry more than seqs, rows one tensor for each cache")
    pointers, strides = (_vp * len(rows))(), (_i64 * len(rows))()
    for i, (r, c) in enumerate(zip(rows, caches)):
        if r.device != c.device or r.dtype != c.dtype or r.shape != (total,) + tuple(c.shape[2:]):
            raise ValueError(f"rows[{i}] must be {(total,) + tuple(c.shape[2:])} of its cache's type")
        if total and not r[0].is_contiguous():
            raise ValueError(f"a token's row in rows[{i}] must be contiguous")
        pointers[i], strides[i] = r.data_ptr(), r.stride(0) * r.element_size()
    o = _pages_options(workspace, ref_counts)
    with _On(ref_counts.device, stream) as s:
        _check(_lib().sbgemm_pages_append(ctypes.byref(p), seqs.data_ptr(), starts.data_ptr(), n, pointers,
                                          strides, total, s or None, o), "sbgemm_pages_append")


def pages_free(caches, ref_counts, block_table, seq_lens, seqs, stream=None) -> None:
    """Frees the sequences seqs (int32 [n]): their pages' counts fall by one and
    their lengths become 0."""
    p = _pool(caches, ref_counts, block_table, seq_lens)
    _int32(ref_counts, seqs=seqs)
    with _On(ref_counts.device, stream) as s:
        _check(_lib().sbgemm_pages_free(ctypes.byref(p), seqs.data_ptr(), seqs.numel(), s or None),
               "sbgemm_pages_free")


def pages_compact(caches, ref_counts, block_table, seq_lens, workspace, moved=None, stream=None) -> None:
    """Moves the pages in use to the front of the pool, table entries and counts
    with them; moved (int32 [1], optional) receives how many moved."""
    p = _pool(caches, ref_counts, block_table, seq_lens)
    if moved is not None:
        _int32(ref_counts, moved=moved)
        if moved.numel() < 1:
            raise ValueError("moved must hold one int32")
    o = _pages_options(workspace, ref_counts)
    with _On(ref_counts.device, stream) as s:
        _check(_lib().sbgemm_pages_compact(ctypes.byref(p), 0 if moved is None else moved.data_ptr(),
                                           s or None, o), "sbgemm_pages_compact")
