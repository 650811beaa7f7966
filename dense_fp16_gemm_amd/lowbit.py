"""Products with one operand held in 4 or 8 bits (``include/gemm_f16_lowbit.h``).

``W4Matrix``: a weight matrix in 4-bit codes with a scale for each group of
32, 64 or 128 weights of a row; ``gemm_nt_w4(a, w)`` is a @ w.T from one row
of a (one token) to long prompts.  ``Q8Matrix``: a matrix of activations in
8-bit codes with a scale for each 32 values of a row, kept from the forward to
the backward pass; ``gemm_tn_q8(dy, x)`` is dy.T @ x, a linear layer's weight
gradient.

As in the rest of the package, every arithmetic step runs in the library's HIP
kernels and torch gives device memory and streams only.  Each function works
on the current stream, or on `stream`: what it allocates then belongs to that
stream, and the tensors passed in are recorded on it, so that the caller may
drop them at once.  Like the rest of the package, none of them takes part in
autograd: what they return is cut off from the graph of tensors that require
gradients, and a torch.autograd.Function connects it.
"""
from __future__ import annotations

import ctypes

from . import GemmError, _check, gemm_f16_device_cus, load

# torch, and what the calls below use of it: bound with the first matrix, since
# importing this package does not import torch
torch = None


def _bind_torch() -> None:
    global torch, _f16, _int8, _int32, _empty, _current_device, _raw_stream, _lib
    import torch as t

    _f16, _int8, _int32, _empty = t.float16, t.int8, t.int32, t.empty_strided
    _lib = load()
    # without torch's check that CUDA is initialised (the operands are on a GPU),
    # and the raw handle without building a Stream object, where torch has these
    _current_device = getattr(t._C, "_cuda_getDevice", None) or t.cuda.current_device
    _raw_stream = getattr(t._C, "_cuda_getCurrentRawStream", None) or \
        (lambda index: t.cuda.current_stream(index).cuda_stream)
    torch = t


LOWBIT_DECODE, LOWBIT_STREAM, LOWBIT_TILE = 0, 1, 2
Q8_GROUP = 32
W4_GROUPS = (32, 64, 128)


class LowbitPlan(ctypes.Structure):
    """What a low-bit product runs (gemm_f16_lowbit_plan_t)."""
    _fields_ = [(name, ctypes.c_int32) for name in
                ("kernel", "block_m", "block_n", "waves", "splits", "grid")] + \
               [("workspace_bytes", ctypes.c_int64)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


def _declare(lib) -> None:
    """Argument types of the functions of gemm_f16_lowbit.h."""
    i64, i32, p = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p
    pi64, plan = ctypes.POINTER(i64), ctypes.POINTER(LowbitPlan)
    for name, args in {
        "gemm_f16_w4_sizes": [i64, i64, i32, pi64, pi64],
        "gemm_f16_w4_quantize": [i64, i64, i32, p, p, p, p],
        "gemm_f16_w4_pack": [i64, i64, i32, p, p, p, p, p],
        "gemm_f16_w4_dequantize": [i64, i64, i32, p, p, p, p],
        "gemm_f16_nt_w4_plan": [i64, i64, i64, i32, i32, plan],
        "gemm_f16_nt_w4": [i64, i64, i64, i32, p, p, p, p, p, i64, p],
        "gemm_f16_q8_quantize": [i64, i64, p, p, p, p],
        "gemm_f16_q8_dequantize": [i64, i64, p, p, p, p],
        "gemm_f16_tn_q8_plan": [i64, i64, i64, i32, plan],
        "gemm_f16_tn_q8": [i64, i64, i64, p, p, p, p, p, i64, p],
    }.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int


# ---- C ABI, same names -----------------------------------------------------
def gemm_f16_w4_sizes(N: int, K: int, group: int) -> tuple[int, int]:
    """(bytes of words, bytes of scales) of an [N, K] matrix in W4 storage."""
    words, scales = ctypes.c_int64(), ctypes.c_int64()
    _check(load().gemm_f16_w4_sizes(N, K, group, ctypes.byref(words), ctypes.byref(scales)),
           "gemm_f16_w4_sizes")
    return words.value, scales.value


def gemm_f16_w4_quantize(N: int, K: int, group: int, W: int, words: int, scales: int,
                         stream: int = 0) -> None:
    _check(load().gemm_f16_w4_quantize(N, K, group, W, words, scales, stream),
           "gemm_f16_w4_quantize")


def gemm_f16_w4_pack(N: int, K: int, group: int, codes: int, in_scales: int, words: int,
                     scales: int, stream: int = 0) -> None:
    _check(load().gemm_f16_w4_pack(N, K, group, codes, in_scales, words, scales, stream),
           "gemm_f16_w4_pack")


def gemm_f16_w4_dequantize(N: int, K: int, group: int, words: int, scales: int, W: int,
                           stream: int = 0) -> None:
    _check(load().gemm_f16_w4_dequantize(N, K, group, words, scales, W, stream),
           "gemm_f16_w4_dequantize")


def gemm_f16_nt_w4_plan(M: int, N: int, K: int, group: int, num_cus: int) -> LowbitPlan:
    plan = LowbitPlan()
    _check(load().gemm_f16_nt_w4_plan(M, N, K, group, num_cus, ctypes.byref(plan)),
           "gemm_f16_nt_w4_plan")
    return plan


def gemm_f16_nt_w4(M: int, N: int, K: int, group: int, A: int, words: int, scales: int, C: int,
                   workspace: int = 0, workspace_bytes: int = 0, stream: int = 0) -> None:
    _check(load().gemm_f16_nt_w4(M, N, K, group, A, words, scales, C, workspace, workspace_bytes,
                                 stream), "gemm_f16_nt_w4")


def gemm_f16_q8_quantize(R: int, N: int, X: int, codes: int, scales: int, stream: int = 0) -> None:
    _check(load().gemm_f16_q8_quantize(R, N, X, codes, scales, stream), "gemm_f16_q8_quantize")


def gemm_f16_q8_dequantize(R: int, N: int, codes: int, scales: int, X: int,
                           stream: int = 0) -> None:
    _check(load().gemm_f16_q8_dequantize(R, N, codes, scales, X, stream),
           "gemm_f16_q8_dequantize")


def gemm_f16_tn_q8_plan(M: int, N: int, K: int, num_cus: int) -> LowbitPlan:
    plan = LowbitPlan()
    _check(load().gemm_f16_tn_q8_plan(M, N, K, num_cus, ctypes.byref(plan)),
           "gemm_f16_tn_q8_plan")
    return plan


def gemm_f16_tn_q8(M: int, N: int, K: int, A: int, codes: int, scales: int, C: int,
                   workspace: int = 0, workspace_bytes: int = 0, stream: int = 0) -> None:
    _check(load().gemm_f16_tn_q8(M, N, K, A, codes, scales, C, workspace, workspace_bytes, stream),
           "gemm_f16_tn_q8")


# ---- the two forms -----------------------------------------------------------
class W4Matrix:
    """An [n, k] matrix in W4 storage: words int32 [ceil(n / 16), ceil(k / 128),
    64, 4] and scales fp16 [ceil(n / 16), 128 ceil(k / 128) / group, 16], as
    quantize_w4() and pack_w4() make them.  The tensors are kept, not copied.
    One that was saved is checked as a new one is, so it is read back onto a GPU
    (torch.load's map_location)."""

    __slots__ = ("words", "scales", "n", "k", "group")

    def __init__(self, words, scales, n: int, k: int, group: int):
        if torch is None:
            _bind_torch()
        if group not in W4_GROUPS:
            raise ValueError(f"group must be one of {W4_GROUPS}, not {group!r}")
        if n < 0 or k < 0:
            raise ValueError(f"negative size: n={n}, k={k}")
        if words.dtype != torch.int32 or scales.dtype != torch.float16:
            raise TypeError("words must be torch.int32 and scales torch.float16")
        words_shape, scales_shape = _w4_shapes(n, k, group)
        if tuple(words.shape) != words_shape or tuple(scales.shape) != scales_shape:
            raise ValueError(f"words{tuple(words.shape)} and scales{tuple(scales.shape)} are not "
                             f"those of a {n} x {k} matrix with groups of {group}")
        if not words.is_cuda or words.device != scales.device:
            raise ValueError("words and scales must be on the same GPU")
        if not (words.is_contiguous() and scales.is_contiguous()):
            raise ValueError("words and scales must be contiguous")
        self._set(words, scales, int(n), int(k), int(group))

    def _set(self, words, scales, n, k, group):
        self.words, self.scales, self.n, self.k, self.group = words, scales, n, k, group
        return self

    def __reduce__(self):
        return type(self), (self.words, self.scales, self.n, self.k, self.group)

    @property
    def shape(self) -> tuple[int, int]:
        return self.n, self.k

    @property
    def device(self):
        return self.words.device

    @property
    def nbytes(self) -> int:
        return self.words.numel() * 4 + self.scales.numel() * 2

    def __repr__(self) -> str:
        return f"W4Matrix({self.n} x {self.k}, group={self.group}, device={self.device})"


def _w4_shapes(n: int, k: int, group: int) -> tuple[tuple, tuple]:
    nb, kt = -(-n // 16), -(-k // 128)
    return (nb, kt, 64, 4), (nb, 128 * kt // group, 16)


class Q8Matrix:
    """An [r, n] matrix in Q8 storage: codes int8 [r, 32 ceil(n / 32)] and
    scales fp16 [r, ceil(n / 32)], as quantize_q8() makes them.  The tensors
    are kept, not copied; a range of rows of both is a Q8Matrix too.  Saved and
    read back as a W4Matrix is."""

    __slots__ = ("codes", "scales", "r", "n")

    def __init__(self, codes, scales, n: int):
        if torch is None:
            _bind_torch()
        if n < 0:
            raise ValueError(f"negative size: n={n}")
        if codes.dtype != torch.int8 or scales.dtype != torch.float16:
            raise TypeError("codes must be torch.int8 and scales torch.float16")
        groups = -(-n // Q8_GROUP)
        if codes.dim() != 2 or codes.shape[1] != Q8_GROUP * groups or \
                tuple(scales.shape) != (codes.shape[0], groups):
            raise ValueError(f"codes{tuple(codes.shape)} and scales{tuple(scales.shape)} are not "
                             f"those of a matrix with {n} columns")
        if not codes.is_cuda or codes.device != scales.device:
            raise ValueError("codes and scales must be on the same GPU")
        if not (codes.is_contiguous() and scales.is_contiguous()):
            raise ValueError("codes and scales must be contiguous")
        self._set(codes, scales, int(codes.shape[0]), int(n))

    def _set(self, codes, scales, r, n):
        self.codes, self.scales, self.r, self.n = codes, scales, r, n
        return self

    def __reduce__(self):
        return type(self), (self.codes, self.scales, self.n)

    @property
    def shape(self) -> tuple[int, int]:
        return self.r, self.n

    @property
    def device(self):
        return self.codes.device

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel() * 2

    def __repr__(self) -> str:
        return f"Q8Matrix({self.r} x {self.n}, device={self.device})"


# ---- torch convenience -------------------------------------------------------
# A call for one token is a few microseconds on the GPU, so the path to it is
# kept short: few Python calls, one into the library, no wrapper objects, no
# device switch where the device is current.
def _is_matrix(x, dtype) -> bool:
    return x.dtype is dtype and x.dim() == 2 and x.is_cuda and x.is_contiguous()


def _refuse(x, dtype, what: str):
    """Raises what is wrong with an x that is not _is_matrix(x, dtype)."""
    if x.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}")
    if x.dim() != 2:
        raise ValueError(f"{what} must be a matrix")
    if not x.is_cuda:
        raise ValueError(f"{what} must be on a GPU")
    raise ValueError(f"{what} must be contiguous (row-major)")


def _call(index, stream, fn, *args) -> None:
    """fn(*args, stream) on device `index`."""
    s = _raw_stream(index) if stream is None else stream.cuda_stream
    if index == _current_device():
        status = fn(*args, s)
    else:
        with torch.cuda.device(index):
            status = fn(*args, s)
    if status:
        raise GemmError(status, fn.__name__)


def _new(on, stream, shape, dtype):
    """Memory on the device of `on` that belongs to the stream it will be used on."""
    if stream is None:
        return on.new_empty(shape, dtype=dtype)
    if stream.device != on.device:
        raise ValueError(f"stream is on {stream.device}, the operands on {on.device}")
    with torch.cuda.stream(stream):
        return on.new_empty(shape, dtype=dtype)


def _new_rows(on, stream, rows, cols, dtype):
    """_new() of a matrix, by torch's quickest way."""
    if stream is None:
        return _empty((rows, cols), (cols, 1), dtype=dtype, device=on.device)
    return _new(on, stream, (rows, cols), dtype)


def _new_w4(on, stream, n: int, k: int, group: int) -> W4Matrix:
    if group not in W4_GROUPS:
        raise ValueError(f"group must be one of {W4_GROUPS}, not {group!r}")
    group = int(group)
    words, scales = _w4_shapes(n, k, group)
    q = W4Matrix.__new__(W4Matrix)
    if stream is not None:
        return q._set(_new(on, stream, words, torch.int32), _new(on, stream, scales, _f16), n, k, group)
    device, kt, groups = on.device, words[1], scales[1]
    return q._set(_empty(words, (256 * kt, 256, 4, 1), dtype=_int32, device=device),
                  _empty(scales, (16 * groups, 16, 1), dtype=_f16, device=device), n, k, group)


def _record(stream, *tensors) -> None:
    """Tensors of other streams, used on `stream`: not to be reused before it is done."""
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _output(out, on, stream, shape):
    if out is None:
        return _new_rows(on, stream, *shape, _f16)
    if stream is not None and stream.device != on.device:
        raise ValueError(f"stream is on {stream.device}, the operands on {on.device}")
    if out.dtype != _f16 or tuple(out.shape) != shape or not out.is_contiguous() or \
            out.device != on.device:
        raise ValueError(f"out must be a contiguous float16 {list(shape)} tensor on {on.device}")
    return out


def quantize_w4(w, group: int = 128, stream=None) -> W4Matrix:
    """w [N, K] fp16 in 4-bit codes, a scale for each `group` weights of a row."""
    if torch is None:
        _bind_torch()
    if not _is_matrix(w, _f16):
        _refuse(w, _f16, "w")
    n, k = w.shape
    q = _new_w4(w, stream, n, k, group)
    _call(w.get_device(), stream, _lib.gemm_f16_w4_quantize, n, k, q.group, w.data_ptr(),
          q.words.data_ptr(), q.scales.data_ptr())
    if stream is not None:
        _record(stream, w)
    return q


def pack_w4(codes, scales, group: int = 128, stream=None) -> W4Matrix:
    """A W4Matrix from another quantiser's codes [N, K] int8 in -8..7 and scales
    [N, ceil(K / group)] fp16, weight = code * scale.  Scales are rounded to 8
    significant bits, by up to 2^-8 of their value; a group that cannot be held
    (a code out of range, a scale that is not finite or is rounded to 65536, a
    weight past 65504) becomes NaN."""
    if torch is None:
        _bind_torch()
    if not _is_matrix(codes, _int8):
        _refuse(codes, _int8, "codes")
    if not _is_matrix(scales, _f16):
        _refuse(scales, _f16, "scales")
    n, k = codes.shape
    q = _new_w4(codes, stream, n, k, group)
    if tuple(scales.shape) != (n, -(-k // group)):
        raise ValueError(f"scales{tuple(scales.shape)} do not fit codes{tuple(codes.shape)} in "
                         f"groups of {group}")
    if codes.device != scales.device:
        raise ValueError("codes and scales must be on the same GPU")
    _call(codes.get_device(), stream, _lib.gemm_f16_w4_pack, n, k, q.group, codes.data_ptr(),
          scales.data_ptr(), q.words.data_ptr(), q.scales.data_ptr())
    if stream is not None:
        _record(stream, codes, scales)
    return q


def dequantize_w4(w: W4Matrix, out=None, stream=None):
    """The [n, k] fp16 matrix that w stands for, exactly."""
    if not isinstance(w, W4Matrix):
        raise TypeError("w must be a W4Matrix")
    words = w.words
    if not words.is_cuda:
        raise ValueError("w must be on a GPU")
    out = _output(out, words, stream, (w.n, w.k))
    _call(words.get_device(), stream, _lib.gemm_f16_w4_dequantize, w.n, w.k, w.group,
          words.data_ptr(), w.scales.data_ptr(), out.data_ptr())
    if stream is not None:
        _record(stream, words, w.scales, out)
    return out


def quantize_q8(x, stream=None) -> Q8Matrix:
    """x [R, N] fp16 in 8-bit codes, a scale for each 32 values of a row."""
    if torch is None:
        _bind_torch()
    if not _is_matrix(x, _f16):
        _refuse(x, _f16, "x")
    r, n = x.shape
    groups = -(-n // Q8_GROUP)
    codes = _new_rows(x, stream, r, groups * Q8_GROUP, _int8)
    scales = _new_rows(x, stream, r, groups, _f16)
    _call(x.get_device(), stream, _lib.gemm_f16_q8_quantize, r, n, x.data_ptr(),
          codes.data_ptr(), scales.data_ptr())
    if stream is not None:
        _record(stream, x)
    return Q8Matrix.__new__(Q8Matrix)._set(codes, scales, r, n)


def dequantize_q8(x: Q8Matrix, out=None, stream=None):
    """The [r, n] fp16 matrix that x stands for, exactly."""
    if not isinstance(x, Q8Matrix):
        raise TypeError("x must be a Q8Matrix")
    codes = x.codes
    if not codes.is_cuda:
        raise ValueError("x must be on a GPU")
    out = _output(out, codes, stream, (x.r, x.n))
    _call(codes.get_device(), stream, _lib.gemm_f16_q8_dequantize, x.r, x.n, codes.data_ptr(),
          x.scales.data_ptr(), out.data_ptr())
    if stream is not None:
        _record(stream, codes, x.scales, out)
    return out


# workspace bytes of a product, per (planner, sizes, device): a repeated call
# costs a dictionary lookup
_workspace_bytes: dict = {}


def _plan_workspace(key) -> int:
    """The bytes that key[0](*key[1:-1], compute units of device key[-1]) plans."""
    with torch.cuda.device(key[-1]):
        need = key[0](*key[1:-1], gemm_f16_device_cus()).workspace_bytes
    if len(_workspace_bytes) >= 1024:
        _workspace_bytes.clear()
    _workspace_bytes[key] = need
    return need


def _workspace(need, on, workspace, stream):
    """(tensor, its address, its bytes)."""
    if workspace is None:
        workspace = _empty((need,), (1,), dtype=torch.uint8, device=on.device) if stream is None \
            else _new(on, stream, (need,), torch.uint8)
        return workspace, workspace.data_ptr(), need
    if not workspace.is_cuda or workspace.device != on.device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the operands' device")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def gemm_nt_w4(a, w: W4Matrix, out=None, workspace=None, stream=None):
    """C = a @ W.T for a [M, K] fp16 and W [N, K] in 4 bits, fp16 [M, N]
    (gemm_f16_nt_w4).  The workspace that some sizes need (see
    gemm_f16_nt_w4_plan) is allocated with torch unless `workspace` is given.
    More than 48 rows want an a that is 16-byte aligned, as torch's own tensors
    are, or a K that is not a multiple of 8 (for which rows are copied): others
    take several times as long."""
    if not isinstance(w, W4Matrix):
        raise TypeError("w must be a W4Matrix")
    if not _is_matrix(a, _f16):
        _refuse(a, _f16, "a")
    m, k = a.shape
    n, words = w.n, w.words
    if k != w.k:
        raise ValueError(f"shape mismatch: a{tuple(a.shape)} w{w.shape}")
    index = a.get_device()
    if index != words.get_device():
        raise ValueError("a and w must be on the same GPU")
    out = _output(out, a, stream, (m, n))
    key = (gemm_f16_nt_w4_plan, m, n, k, w.group, index)
    need = _workspace_bytes.get(key)
    if need is None:
        need = _plan_workspace(key)
    ws, ws_ptr, ws_bytes = None, 0, 0
    if need or workspace is not None:
        ws, ws_ptr, ws_bytes = _workspace(need, a, workspace, stream)
    _call(index, stream, _lib.gemm_f16_nt_w4, m, n, k, w.group, a.data_ptr(), words.data_ptr(),
          w.scales.data_ptr(), out.data_ptr(), ws_ptr, ws_bytes)
    if stream is not None:
        _record(stream, a, words, w.scales, out, ws)
    return out


def gemm_tn_q8(a, x: Q8Matrix, out=None, workspace=None, stream=None):
    """C = a.T @ X for a [K, M] fp16 and X [K, N] in 8 bits, fp16 [M, N]
    (gemm_f16_tn_q8): with a the gradient of a linear layer's output and X its
    kept input, the gradient of its [M, N] weight.  Workspace as for
    gemm_nt_w4."""
    if not isinstance(x, Q8Matrix):
        raise TypeError("x must be a Q8Matrix")
    if not _is_matrix(a, _f16):
        _refuse(a, _f16, "a")
    k, m = a.shape
    n, codes = x.n, x.codes
    if k != x.r:
        raise ValueError(f"shape mismatch: a{tuple(a.shape)} x{x.shape}")
    index = a.get_device()
    if index != codes.get_device():
        raise ValueError("a and x must be on the same GPU")
    out = _output(out, a, stream, (m, n))
    key = (gemm_f16_tn_q8_plan, m, n, k, index)
    need = _workspace_bytes.get(key)
    if need is None:
        need = _plan_workspace(key)
    ws, ws_ptr, ws_bytes = None, 0, 0
    if need or workspace is not None:
        ws, ws_ptr, ws_bytes = _workspace(need, a, workspace, stream)
    _call(index, stream, _lib.gemm_f16_tn_q8, m, n, k, a.data_ptr(), codes.data_ptr(),
          x.scales.data_ptr(), out.data_ptr(), ws_ptr, ws_bytes)
    if stream is not None:
        _record(stream, a, codes, x.scales, out, ws)
    return out
