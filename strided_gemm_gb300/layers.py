"""The operators around a layer's products: products of 8-bit floats with block
scales and the quantisation that feeds them, and norms of queries, keys and
latents with the rotation of their positions (include/sbgemm.h has each one's
definition).

As in serving.py, the sbgemm_* functions carry the C names and arguments; the
others take torch CUDA tensors, read strides from them, and run on the tensors'
device and its current stream unless a stream is given.
"""

from __future__ import annotations

import ctypes
import math

import strided_gemm_gb300 as _sg
from . import serving as _serving

_i64, _vp, _int, _f32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float
_size = ctypes.c_size_t


class Fp8Matrix(ctypes.Structure):
    """sbgemm_fp8_matrix: 8-bit data with fp32 scales, addresses and strides."""
    _fields_ = [("type", _int), ("group", _int), ("data", _vp), ("row_stride", _i64), ("k_stride", _i64),
                ("batch_stride", _i64), ("scale", _vp), ("scale_row_stride", _i64), ("scale_k_stride", _i64),
                ("scale_batch_stride", _i64)]


class _Part(ctypes.Structure):
    _fields_ = [("x", _vp), ("x_token", _i64), ("x_head", _i64), ("y", _vp), ("y_token", _i64), ("y_head", _i64),
                ("heads", _i64), ("D", _i64), ("norm", _i64), ("start", _i64), ("weight", _vp)]


class _Grad(ctypes.Structure):
    _fields_ = [("x", _vp), ("x_token", _i64), ("x_head", _i64), ("dy", _vp), ("dy_token", _i64),
                ("dy_head", _i64), ("dx", _vp), ("dx_token", _i64), ("dx_head", _i64), ("heads", _i64), ("D", _i64),
                ("norm", _i64), ("start", _i64), ("weight", _vp), ("dweight", _vp)]


def declare(lib) -> None:
    """Sets the argument types of the library's functions of this file."""
    opt, matrix = ctypes.POINTER(_sg._Options), ctypes.POINTER(Fp8Matrix)
    arguments = {
        "sbgemm_fp8": [matrix, matrix, _int, _vp] + [_i64] * 7 + [_f32, _int, _vp],
        "sbgemm_quantize_fp8": [_int, _vp, _i64, _i64, _i64, matrix, _i64, _i64, _i64, _vp],
        "sbgemm_norm_rope": [_int, ctypes.POINTER(_Part), _i64, _vp, _i64, _vp, _i64, _f32, _int, _f32, _vp],
        "sbgemm_norm_rope_backward": [_int, ctypes.POINTER(_Grad), _i64, _vp, _i64, _vp, _i64, _f32, _int, _f32,
                                      _int, _vp, opt],
        "sbgemm_norm_rope_workspace_bytes": [_int, _i64, ctypes.POINTER(_size)],
    }
    for name, types in arguments.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = _int, types


def bind(fast, lib) -> None:
    """Hands the fast-call module (csrc/fastcall.c) these functions' addresses."""
    fast.bind_layers(*(ctypes.cast(getattr(lib, name), _vp).value for name in (
        "sbgemm_latent_attention_shared", "sbgemm_fp8", "sbgemm_quantize_fp8", "sbgemm_norm_rope",
        "sbgemm_norm_rope_backward")))


def _lib():
    return _sg._lib if _sg._lib is not None else _sg.load()


def _check(st: int, where: str) -> None:
    if st:
        raise _sg.SbgemmError(st, where)


# ---- the C functions ------------------------------------------------------------

def _numbers(m):
    """An Fp8Matrix's fields in order."""
    return tuple(getattr(m, name) or 0 for name, _ in Fp8Matrix._fields_)


def _fp8(a, b, type_c, C, rsC, csC, bsC, M, N, K, batch, alpha, accumulate, stream) -> None:
    """sbgemm_fp8 of two tuples of Fp8Matrix's fields."""
    lib = _lib()
    if _sg._fast is not None:
        st = _sg._fast.fp8(*a, *b, type_c, C, rsC, csC, bsC, M, N, K, batch, alpha, accumulate, stream or 0)
    else:
        st = lib.sbgemm_fp8(ctypes.byref(Fp8Matrix(*a)), ctypes.byref(Fp8Matrix(*b)), type_c, C, rsC, csC, bsC, M, N, K,
                            batch, alpha, 1 if accumulate else 0, stream or None)
    if st:
        raise _sg.SbgemmError(st, "sbgemm_fp8")


def sbgemm_fp8(A, B, type_c, C, rsC, csC, bsC, M, N, K, batch, alpha=1.0, accumulate=0, stream=0) -> None:
    """C <- alpha*A*B (+C) on 8-bit matrices with block scales (Fp8Matrix)."""
    if A is None or B is None:
        raise _sg.SbgemmError(_sg.SBGEMM_ERR_NULL_POINTER, "sbgemm_fp8")
    _fp8(_numbers(A), _numbers(B), type_c, C, rsC, csC, bsC, M, N, K, batch, alpha, accumulate, stream)


def _quantize(type_x, X, rsX, csX, bsX, y, M, K, batch, stream) -> None:
    """sbgemm_quantize_fp8 into a tuple of Fp8Matrix's fields."""
    lib = _lib()
    if _sg._fast is not None:
        st = _sg._fast.quantize(type_x, X, rsX, csX, bsX, *y, M, K, batch, stream or 0)
    else:
        st = lib.sbgemm_quantize_fp8(type_x, X, rsX, csX, bsX, ctypes.byref(Fp8Matrix(*y)), M, K, batch, stream or None)
    if st:
        raise _sg.SbgemmError(st, "sbgemm_quantize_fp8")


def sbgemm_quantize_fp8(type_x, X, rsX, csX, bsX, Y, M, K, batch, stream=0) -> None:
    """Quantises X into the 8-bit matrix Y (Fp8Matrix), data and scales."""
    if Y is None:
        raise _sg.SbgemmError(_sg.SBGEMM_ERR_NULL_POINTER, "sbgemm_quantize_fp8")
    _quantize(type_x, X, rsX, csX, bsX, _numbers(Y), M, K, batch, stream)


def sbgemm_norm_rope(type, parts, positions, tokens, steps, dims, magnitude=1.0, interleaved=0, eps=1e-6,
                     stream=0) -> None:
    """Norm and rotation of the arrays that `parts` (sbgemm_rope_part tuples in
    the fields' order) describe."""
    lib = _lib()
    n = len(parts)
    if interleaved not in (0, 1) or n > _sg.MAX_ROPE_PARTS:
        st = _sg.SBGEMM_ERR_INVALID_VALUE
    elif _sg._fast is not None:
        st = _sg._fast.rope(type, tuple(parts), positions, tokens, steps, dims, magnitude, interleaved, eps, stream or 0)
    else:
        array = (_Part * max(1, n))(*(_Part(*p) for p in parts))
        st = lib.sbgemm_norm_rope(type, array, n, positions, tokens, steps, dims, magnitude, int(interleaved), eps,
                                  stream or None)
    if st:
        raise _sg.SbgemmError(st, "sbgemm_norm_rope")


def sbgemm_norm_rope_backward(type, parts, positions, tokens, steps, dims, magnitude=1.0, interleaved=0, eps=1e-6,
                              accumulate=0, stream=0, workspace: int = 0, workspace_bytes: int = 0) -> None:
    """The gradient of sbgemm_norm_rope (sbgemm_rope_grad tuples)."""
    lib = _lib()
    n = len(parts)
    o = _sg._opts_ref(_sg.MATH_FP32, _sg.PATH_AUTO, workspace, workspace_bytes, _sg.KSPLIT_ANY)
    if interleaved not in (0, 1) or n > _sg.MAX_ROPE_PARTS:
        st = _sg.SBGEMM_ERR_INVALID_VALUE
    elif _sg._fast is not None:
        st = _sg._fast.rope_back(type, tuple(parts), positions, tokens, steps, dims, magnitude, interleaved, eps,
                                 accumulate, stream or 0, o[2])
    else:
        array = (_Grad * max(1, n))(*(_Grad(*p) for p in parts))
        st = lib.sbgemm_norm_rope_backward(type, array, n, positions, tokens, steps, dims, magnitude, int(interleaved),
                                           eps, 1 if accumulate else 0, stream or None, o[1])
    if st:
        raise _sg.SbgemmError(st, "sbgemm_norm_rope_backward")


def sbgemm_norm_rope_workspace_bytes(norms, device: int | None = None) -> int:
    """Bytes of workspace for norm_rope_backward with these numbers of normed
    elements, one a part (or their sum), on `device` (default: the current one)."""
    if device is None:
        import torch
        device = torch.cuda.current_device()
    n = _size(0)
    total = sum(norms) if hasattr(norms, "__iter__") else int(norms)
    _check(_lib().sbgemm_norm_rope_workspace_bytes(int(device), int(total), ctypes.byref(n)),
           "sbgemm_norm_rope_workspace_bytes")
    return n.value


# ---- torch helpers --------------------------------------------------------------

_torch = None
_floats: dict = {}
_fp8s: dict = {}


def _setup():
    global _torch
    import torch
    _floats.update({torch.bfloat16: _sg.TYPE_BF16, torch.float16: _sg.TYPE_FP16, torch.float32: _sg.TYPE_FP32})
    _fp8s.update({torch.float8_e4m3fn: _sg.TYPE_E4M3, torch.float8_e5m2: _sg.TYPE_E5M2})
    if _serving._torch is None:
        _serving._setup()
    _torch = torch


def _float_kind(t, name):
    if _torch is None:
        _setup()
    k = _floats.get(t.dtype)
    if k is None:
        raise TypeError(f"{name} must be a bfloat16, float16 or float32 tensor")
    return k


def _group(rows, groups, name):
    """How many rows a scale covers, from the number of scales along them."""
    if groups == rows:
        return 1
    if groups == (rows + 127) // 128:
        return 128
    raise ValueError(f"{name} has {groups} scales for {rows} rows: one for each, or for each 128, is wanted")


def _view(t, name):
    """Shape and strides of a 2-D or 3-D tensor as [batch, rows, columns] (no
    view is made: that costs more than the rest of a call)."""
    s, st = t.shape, t.stride()
    if len(s) == 2:
        return 1, s[0], s[1], 0, st[0], st[1]
    if len(s) == 3:
        return s[0], s[1], s[2], st[0], st[1], st[2]
    raise ValueError(f"{name} must be 2-D or 3-D, got {tuple(s)}")


def _matrix(x, s, name, dev, turned, batch, rows, k):
    """Fp8Matrix's fields for a tensor of `rows` x `k` over the batch (turned: k x
    rows) with its scales laid out alike."""
    kind = _fp8s.get(x.dtype)
    if kind is None:
        raise TypeError(f"{name} must be a float8_e4m3fn or float8_e5m2 tensor")
    if s.dtype != _torch.float32:
        raise TypeError(f"the scales of {name} must be a float32 tensor")
    if x.get_device() != dev or s.get_device() != dev:
        raise TypeError(f"{name} and its scales must be on cuda:{dev}")
    n, r, c, bs, rs, cs = _view(x, name)
    ns, sr, sc, bss, rss, css = _view(s, f"the scale of {name}")
    if turned:
        r, c, rs, cs, sr, sc, rss, css = c, r, cs, rs, sc, sr, css, rss
    if (n != batch and n != 1) or ns != n or r != rows or c != k or sc != (k + 127) // 128:
        raise ValueError(f"shape mismatch: {name}{tuple(x.shape)} with scales {tuple(s.shape)} in a batch of {batch}")
    group = _group(rows, sr, f"the scale of {name}")
    if n != batch:
        bs = bss = 0
    return kind, group, x.data_ptr(), rs, cs, bs, s.data_ptr(), rss, css, bss


def matmul_fp8(A, A_scale, B, B_scale, C, alpha: float = 1.0, accumulate: bool = False, stream=None):
    """C <- alpha*A@B (+C) on torch CUDA float8 tensors viewed as [batch, M, K]
    and [batch, K, N] (2-D means batch 1; either may have batch 1 to be shared),
    any strides, with float32 scales A_scale [batch, M or ceil(M / 128),
    ceil(K / 128)] and B_scale [batch, ceil(K / 128), N or ceil(N / 128)]: one
    for each row, or each 128 of them, and 128 elements of K.  C: bfloat16,
    float16 or float32.  The tensor cores take operands with unit stride along
    K, so a weight [N, K] is passed as W.t() with W_scale.t().  Returns C."""
    kind = _float_kind(C, "C")
    dev = _serving._device(C)
    batch, M, N, bc, rc, cc = _view(C, "C")
    K = A.shape[-1]
    a = _matrix(A, A_scale, "A", dev, False, batch, M, K)
    b = _matrix(B, B_scale, "B", dev, True, batch, N, K)
    _serving._run(dev, stream, _fp8, a, b, kind, C.data_ptr(), rc, cc, bc, M, N, K, batch, alpha, accumulate)
    return C


def quantize_fp8(X, Y, scale, stream=None):
    """Quantises X [batch, M, K] (bfloat16, float16 or float32; 2-D means batch
    1; any strides, so X.t() is quantised along X's rows) into Y (float8, the
    same shape) with the scales [batch, M or ceil(M / 128), ceil(K / 128)].
    Returns (Y, scale)."""
    kind = _float_kind(X, "X")
    dev = _serving._device(X)
    batch, M, K, bx, rx, cx = _view(X, "X")
    y = _matrix(Y, scale, "Y", dev, False, batch, M, K)
    if Y.dim() != X.dim() or (batch > 1 and Y.shape[0] != batch):
        raise ValueError(f"shape mismatch: X{tuple(X.shape)} Y{tuple(Y.shape)}")
    _serving._run(dev, stream, _quantize, kind, X.data_ptr(), rx, cx, bx, y, M, K, batch)
    return Y, scale


class RopeTable:
    """The rotation of `dims` elements: a step of 2^-64 turns a position for each
    pair (int64 [dims / 2] on the device, read as unsigned), and the factor of
    cosine and sine."""

    def __init__(self, steps, magnitude: float = 1.0):
        self.steps, self.magnitude, self.dims = steps, float(magnitude), 2 * steps.numel()


def rope_steps(frequencies):
    """Frequencies in radians a position as steps of 2^-64 turns (signed 64-bit
    integers that mean the same modulo 2^64)."""
    out = []
    for f in frequencies:
        step = round(math.ldexp(f / (2 * math.pi), 64)) & (2 ** 64 - 1)
        out.append(step - 2 ** 64 if step >= 2 ** 63 else step)
    return out


def rope_frequencies(dims: int, base: float = 10000.0, factor: float = 1.0, original: int = 4096,
                     fast: float = 32.0, slow: float = 1.0):
    """base ** (-2 i / dims) radians a position for each pair i.  A factor above
    1 stretches the positions beyond `original` by parts (YaRN): a pair that
    turns less than `slow` times in `original` positions is slowed down by the
    factor, one that turns more than `fast` times is left alone, with a linear
    ramp over the pairs between."""
    f = [base ** (-2.0 * i / dims) for i in range(dims // 2)]
    if factor == 1.0:
        return f

    def pair(turns):
        return dims * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))

    lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), dims - 1)
    ramp = [min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0) for i in range(dims // 2)]
    return [x / factor * r + x * (1 - r) for x, r in zip(f, ramp)]


def rope_table(dims: int, base: float = 10000.0, factor: float = 1.0, original: int = 4096, fast: float = 32.0,
               slow: float = 1.0, magnitude: float | None = None, frequencies=None, device="cuda") -> RopeTable:
    """The table of `norm_rope` for `dims` rotated elements: rope_frequencies, or
    the given ones (radians a position, one a pair).  magnitude: default 1, and
    0.1 ln(factor) + 1 for a factor other than 1.  Made once, outside any graph
    capture."""
    import torch
    if dims < 0 or dims % 2:
        raise ValueError(f"dims must be even, got {dims}")
    f = rope_frequencies(dims, base, factor, original, fast, slow) if frequencies is None else \
        [float(x) for x in frequencies]
    if len(f) != dims // 2:
        raise ValueError(f"{dims // 2} frequencies are wanted, got {len(f)}")
    if magnitude is None:
        magnitude = 1.0 if factor == 1.0 else 0.1 * math.log(factor) + 1.0
    return RopeTable(torch.tensor(rope_steps(f), dtype=torch.int64, device=device), magnitude)


class RopePart:
    """One array of norm_rope: x and y [tokens, heads, D] (or [tokens, D]), unit
    stride along D; the first `norm` elements of a row are normed (weight [norm]
    of x's type, or None), those from `start` on are rotated.  y may be x."""
    __slots__ = ("x", "y", "norm", "weight", "start")

    def __init__(self, x, y, norm: int = 0, weight=None, start: int = 0):
        self.x, self.y, self.norm, self.weight, self.start = x, y, norm, weight, start


class RopeGrad:
    """One array of norm_rope_backward: x (None without a norm), dy and dx
    [tokens, heads, D] (or [tokens, D]), dweight float32 [norm] or None."""
    __slots__ = ("x", "dy", "dx", "norm", "weight", "dweight", "start")

    def __init__(self, x, dy, dx, norm: int = 0, weight=None, dweight=None, start: int = 0):
        self.x, self.dy, self.dx, self.norm, self.weight, self.dweight, self.start = (
            x, dy, dx, norm, weight, dweight, start)


def _rows(t, name, dtype, dev, tokens, shape=None):
    """(address, token stride, head stride, heads, D) of [tokens, heads, D] or [tokens, D]."""
    if t.dtype != dtype or t.get_device() != dev:
        raise TypeError(f"{name} must be a {dtype} tensor on cuda:{dev}")
    s, st = t.shape, t.stride()
    if len(s) == 2:
        s, st = (s[0], 1, s[1]), (st[0], s[1], st[1])
    if len(s) != 3 or s[0] != tokens or (shape is not None and tuple(s[1:]) != shape):
        raise ValueError(f"shape mismatch: {name}{tuple(t.shape)} for {tokens} tokens")
    if s[2] > 1 and st[2] != 1:
        raise ValueError(f"{name} needs unit stride along its last axis")
    return t.data_ptr(), st[0], st[1], s[1], s[2]


def _vector(t, name, n, dtype, dev):
    if t is None:
        return None
    if t.dtype != dtype or t.get_device() != dev:
        raise TypeError(f"{name} must be a {dtype} tensor on cuda:{dev}")
    if tuple(t.shape) != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of {n} elements")
    return t.data_ptr()


def _angles(positions, table, dev):
    """(positions, tokens or None, steps, dims, magnitude)"""
    if table is None or table.dims == 0:
        return 0, None, 0, 0, 1.0
    if table.steps.dtype != _torch.int64:
        raise TypeError("the table's steps must be an int64 tensor")
    if table.steps.get_device() != dev or not table.steps.is_contiguous():
        raise ValueError(f"the table must be contiguous on cuda:{dev}")
    if positions is None:
        raise TypeError("a rotation needs positions")
    if positions.dim() != 1:
        raise ValueError("positions must be [tokens]")
    return (_serving._ints(positions, "positions", dev), positions.shape[0], table.steps.data_ptr(), table.dims,
            table.magnitude)


_norm_rope_on = sbgemm_norm_rope


def norm_rope(parts, positions, table, interleaved: bool = False, eps: float = 1e-6, stream=None):
    """RMS norms and rotations of several arrays in one launch (RopePart each, up
    to MAX_ROPE_PARTS; one type, the same tokens): queries and keys, or query
    rope parts and latent rows of a cache.  positions: int32 [tokens]; table:
    rope_table (None for norms only).  Pairs are (i, i + dims / 2) of the rotated
    elements, or (2 i, 2 i + 1) when interleaved."""
    if not parts:
        return
    x0 = parts[0].x
    kind, dev = _float_kind(x0, "x"), _serving._device(x0)
    at, tokens, steps, dims, magnitude = _angles(positions, table, dev)
    if tokens is None:
        tokens = x0.shape[0]
    rows = []
    for p in parts:
        x, xt, xh, heads, D = _rows(p.x, "x", x0.dtype, dev, tokens)
        y, yt, yh, _, _ = _rows(p.y, "y", x0.dtype, dev, tokens, (heads, D))
        rows.append((x, xt, xh, y, yt, yh, heads, D, p.norm, p.start,
                     _vector(p.weight, "weight", p.norm, x0.dtype, dev)))
    _serving._run(dev, stream, _norm_rope_on, kind, rows, at, tokens, steps, dims, magnitude, bool(interleaved), eps)


def _norm_rope_backward_on(kind, rows, at, tokens, steps, dims, magnitude, interleaved, eps, accumulate, ws, ws_bytes,
                           stream):
    sbgemm_norm_rope_backward(kind, rows, at, tokens, steps, dims, magnitude, interleaved, eps, accumulate, stream, ws,
                              ws_bytes)


def norm_rope_backward(parts, positions, table, interleaved: bool = False, eps: float = 1e-6,
                       accumulate: bool = False, workspace=None, stream=None):
    """Gradients of norm_rope (RopeGrad each): dx, and dweight summed over tokens
    and heads, added to what is there when `accumulate`.  A workspace of
    sbgemm_norm_rope_workspace_bytes is needed when a dweight is wanted.  Without
    norms this is the inverse rotation."""
    if not parts:
        return
    d0 = parts[0].dy
    kind, dev = _float_kind(d0, "dy"), _serving._device(d0)
    at, tokens, steps, dims, magnitude = _angles(positions, table, dev)
    if tokens is None:
        tokens = d0.shape[0]
    rows = []
    for p in parts:
        dy, dt, dh, heads, D = _rows(p.dy, "dy", d0.dtype, dev, tokens)
        dx, gt, gh, _, _ = _rows(p.dx, "dx", d0.dtype, dev, tokens, (heads, D))
        x, xt, xh = None, 0, 0
        if p.norm:
            if p.x is None:
                raise TypeError("a normed part's gradient needs its x")
            x, xt, xh, _, _ = _rows(p.x, "x", d0.dtype, dev, tokens, (heads, D))
        rows.append((x, xt, xh, dy, dt, dh, dx, gt, gh, heads, D, p.norm, p.start,
                     _vector(p.weight, "weight", p.norm, d0.dtype, dev),
                     _vector(p.dweight, "dweight", p.norm, _torch.float32, dev)))
    ws, ws_bytes = _serving._workspace(workspace, dev)
    _serving._run(dev, stream, _norm_rope_backward_on, kind, rows, at, tokens, steps, dims, magnitude,
                  bool(interleaved), eps, accumulate, ws, ws_bytes)
