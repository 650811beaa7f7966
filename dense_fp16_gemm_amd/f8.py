"""Products in 8-bit floating point (``include/gemm_f16_f8.h``).

``F8Matrix``: a matrix, or a stack of them, in e4m3 codes with a power of two
for each 128 values of a row (block 1) or each 128 x 128 values (block 128).
``quantize_f8(x)`` makes one from fp16, or one of the transpose;
``gemm_nt_f8(a, w)`` is a @ w.T from one row of a (one token) to a training
step, and with transposed forms a linear layer's gradients.

The conventions are those of ``lowbit``: every arithmetic step runs in the
library's HIP kernels, calls work on the current stream or on `stream`, results
take no part in autograd.
"""
from __future__ import annotations

import ctypes

from . import _check, gemm_f16_device_cus, load, lowbit
from .lowbit import LowbitPlan, _call, _new, _output, _record, _refuse, _workspace

# bound with the first matrix, as in lowbit
torch = None

F8_GROUP = 128
F8_BLOCKS = (1, 128)


def _bind_torch() -> None:
    global torch, _f16, _f8, _uint8, _empty, _lib
    if lowbit.torch is None:
        lowbit._bind_torch()
    t = lowbit.torch
    _f16, _f8, _uint8, _empty = t.float16, t.float8_e4m3fn, t.uint8, t.empty_strided
    _lib = load()
    torch = t


def _declare(lib) -> None:
    """Argument types of the functions of gemm_f16_f8.h."""
    i64, i32, p = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p
    pi64, plan = ctypes.POINTER(i64), ctypes.POINTER(LowbitPlan)
    for name, args in {
        "gemm_f16_f8_sizes": [i64, i64, i64, i32, pi64, pi64],
        "gemm_f16_f8_quantize": [i64, i64, i64, i32, i32, p, p, p, p],
        "gemm_f16_f8_dequantize": [i64, i64, i64, i32, p, p, p, p],
        "gemm_f16_nt_f8_plan": [i64, i64, i64, i32, i32, i32, plan],
        "gemm_f16_nt_f8": [i64, i64, i64, p, p, i32, p, p, p, p, i64, p],
        "gemm_f16_nt_f8_x": [i64, i64, i64, p, i32, p, p, p, p, i64, p],
        "gemm_f16_nt_f8_experts_plan": [i64, i64, i64, i64, i32, i32, i32, plan],
        "gemm_f16_nt_f8_experts": [i64, i64, i64, i64, i32, p, p, p, p, p, p, p, p, i64, p],
        "gemm_f16_nt_f8_experts_x": [i64, i64, i64, i64, i32, p, p, p, p, p, p, p, i64, p],
        "gemm_f16_f8_experts_columns": [i64, i64, pi64],
        "gemm_f16_f8_quantize_experts": [i64, i64, i64, i32, p, p, p, p, p, p],
        "gemm_f16_nt_f8_experts_grad_plan": [i64, i64, i64, i64, i32, plan],
        "gemm_f16_nt_f8_experts_grad": [i64, i64, i64, i64, p, p, p, p, p, p, p],
    }.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int


# ---- C ABI, same names -----------------------------------------------------
def gemm_f16_f8_sizes(count: int, R: int, K: int, block: int) -> tuple[int, int]:
    """(bytes of codes, bytes of scales) of `count` [R, K] matrices in F8 storage."""
    codes, scales = ctypes.c_int64(), ctypes.c_int64()
    _check(load().gemm_f16_f8_sizes(count, R, K, block, ctypes.byref(codes), ctypes.byref(scales)),
           "gemm_f16_f8_sizes")
    return codes.value, scales.value


def gemm_f16_f8_quantize(count: int, R: int, K: int, block: int, transposed: bool, X: int,
                         codes: int, scales: int, stream: int = 0) -> None:
    _check(load().gemm_f16_f8_quantize(count, R, K, block, transposed, X, codes, scales, stream),
           "gemm_f16_f8_quantize")


def gemm_f16_f8_dequantize(count: int, R: int, K: int, block: int, codes: int, scales: int,
                           X: int, stream: int = 0) -> None:
    _check(load().gemm_f16_f8_dequantize(count, R, K, block, codes, scales, X, stream),
           "gemm_f16_f8_dequantize")


def gemm_f16_nt_f8_plan(M: int, N: int, K: int, b_block: int, a_f16: bool,
                        num_cus: int) -> LowbitPlan:
    plan = LowbitPlan()
    _check(load().gemm_f16_nt_f8_plan(M, N, K, b_block, a_f16, num_cus, ctypes.byref(plan)),
           "gemm_f16_nt_f8_plan")
    return plan


def gemm_f16_nt_f8(M: int, N: int, K: int, a_codes: int, a_scales: int, b_block: int,
                   b_codes: int, b_scales: int, C: int, workspace: int = 0,
                   workspace_bytes: int = 0, stream: int = 0) -> None:
    _check(load().gemm_f16_nt_f8(M, N, K, a_codes, a_scales, b_block, b_codes, b_scales, C,
                                 workspace, workspace_bytes, stream), "gemm_f16_nt_f8")


def gemm_f16_nt_f8_x(M: int, N: int, K: int, X: int, b_block: int, b_codes: int, b_scales: int,
                     C: int, workspace: int = 0, workspace_bytes: int = 0,
                     stream: int = 0) -> None:
    _check(load().gemm_f16_nt_f8_x(M, N, K, X, b_block, b_codes, b_scales, C, workspace,
                                   workspace_bytes, stream), "gemm_f16_nt_f8_x")


# ---- storage -----------------------------------------------------------------
def _f8_shapes(count: tuple, r: int, k: int, block: int) -> tuple[tuple, tuple]:
    return count + (r, -(-k // 128) * 128), count + (-(-k // 512), -(-r // block), 4)


class F8Matrix:
    """An [r, k] matrix, or a stack [e, r, k], in F8 storage: codes
    float8_e4m3fn [.., r, 128 ceil(k / 128)], zero past k, and scales uint8 [..,
    ceil(k / 512), ceil(r / block), 4] (exponents + 127; the four of a row are
    those of neighbouring groups of 128 columns), as quantize_f8() makes them.
    The tensors are kept, not copied.  Saved and read back as a W4Matrix is."""

    __slots__ = ("codes", "scales", "k", "block")

    def __init__(self, codes, scales, k: int, block: int):
        if torch is None:
            _bind_torch()
        if block not in F8_BLOCKS:
            raise ValueError(f"block must be one of {F8_BLOCKS}, not {block!r}")
        if k < 0:
            raise ValueError(f"negative size: k={k}")
        if codes.dtype != _f8 or scales.dtype != _uint8:
            raise TypeError("codes must be torch.float8_e4m3fn and scales torch.uint8")
        if codes.dim() not in (2, 3) or \
                (tuple(codes.shape), tuple(scales.shape)) != \
                _f8_shapes(tuple(codes.shape[:-2]), codes.shape[-2], k, block):
            raise ValueError(f"codes{tuple(codes.shape)} and scales{tuple(scales.shape)} are not "
                             f"those of a matrix with {k} columns and blocks of {block}")
        if not codes.is_cuda or codes.device != scales.device:
            raise ValueError("codes and scales must be on the same GPU")
        if not (codes.is_contiguous() and scales.is_contiguous()):
            raise ValueError("codes and scales must be contiguous")
        self._set(codes, scales, int(k), int(block))

    def _set(self, codes, scales, k, block):
        self.codes, self.scales, self.k, self.block = codes, scales, k, block
        return self

    # stored with the codes as bytes: pickle by itself reads no float8 tensor back
    def __getstate__(self):
        return self.codes.view(_uint8), self.scales, self.k, self.block

    def __setstate__(self, state):
        if torch is None:
            _bind_torch()
        codes, scales, k, block = state
        self.__init__(codes.view(_f8), scales, k, block)

    @property
    def shape(self) -> tuple:
        return tuple(self.codes.shape[:-1]) + (self.k,)

    @property
    def device(self):
        return self.codes.device

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()

    def __repr__(self) -> str:
        size = " x ".join(map(str, self.shape))
        return f"F8Matrix({size}, block={self.block}, device={self.device})"


def _new_f8(on, stream, count: tuple, r: int, k: int, block: int) -> F8Matrix:
    codes, scales = _f8_shapes(count, r, k, block)
    q = F8Matrix.__new__(F8Matrix)
    if stream is not None or count:
        return q._set(_new(on, stream, codes, _f8), _new(on, stream, scales, _uint8), k, block)
    # by torch's quickest way
    device, blocks = on.device, scales[1]
    return q._set(_empty(codes, (codes[1], 1), dtype=_f8, device=device),
                  _empty(scales, (4 * blocks, 4, 1), dtype=_uint8, device=device), k, block)


def quantize_f8(x, block: int = 1, transposed: bool = False, stream=None) -> F8Matrix:
    """x [R, K] (or [E, R, K]) fp16 in e4m3 with a scale for each 128 values of a
    row (block 1) or each 128 x 128 (block 128).  transposed: the transpose's
    form [K, R], whose groups of 128 run along R."""
    if torch is None:
        _bind_torch()
    if block not in F8_BLOCKS:
        raise ValueError(f"block must be one of {F8_BLOCKS}, not {block!r}")
    if x.dtype is not _f16 or not x.is_cuda or not x.is_contiguous() or x.dim() not in (2, 3):
        _refuse_stack(x, "x")
    count, (r, k) = tuple(x.shape[:-2]), x.shape[-2:]
    if transposed:
        r, k = k, r
    q = _new_f8(x, stream, count, r, k, int(block))
    _call(x.get_device(), stream, _lib.gemm_f16_f8_quantize, count[0] if count else 1, r, k,
          q.block, bool(transposed), x.data_ptr(), q.codes.data_ptr(), q.scales.data_ptr())
    if stream is not None:
        _record(stream, x)
    return q


def _refuse_stack(x, what: str):
    """Raises what is wrong with an x that is no fp16 matrix or stack of them."""
    if x.dtype != _f16:
        raise TypeError(f"{what} must be {_f16}")
    if x.dim() not in (2, 3):
        raise ValueError(f"{what} must be a matrix or a stack of matrices")
    if not x.is_cuda:
        raise ValueError(f"{what} must be on a GPU")
    raise ValueError(f"{what} must be contiguous (row-major)")


def dequantize_f8(x: F8Matrix, out=None, stream=None):
    """The fp16 matrix (or stack) that x stands for, each value rounded to fp16."""
    if not isinstance(x, F8Matrix):
        raise TypeError("x must be an F8Matrix")
    codes = x.codes
    if not codes.is_cuda:
        raise ValueError("x must be on a GPU")
    shape = x.shape
    out = _new(codes, stream, shape, _f16) if out is None else _output(out, codes, stream, shape)
    count = shape[0] if len(shape) == 3 else 1
    _call(codes.get_device(), stream, _lib.gemm_f16_f8_dequantize, count, shape[-2], x.k, x.block,
          codes.data_ptr(), x.scales.data_ptr(), out.data_ptr())
    if stream is not None:
        _record(stream, codes, x.scales, out)
    return out


# ---- products ------------------------------------------------------------------
# workspace bytes of a product, per (planner, sizes, device): a repeated call
# costs a dictionary lookup
_workspace_bytes: dict = {}


def _planned(key) -> int:
    """The bytes that key[0](*key[1:-1], compute units of device key[-1]) plans."""
    need = _workspace_bytes.get(key)
    if need is None:
        with torch.cuda.device(key[-1]):
            need = key[0](*key[1:-1], gemm_f16_device_cus()).workspace_bytes
        if len(_workspace_bytes) >= 1024:
            _workspace_bytes.clear()
        _workspace_bytes[key] = need
    return need


def _operand(a, what: str) -> bool:
    """Whether a, a product's first operand, is an fp16 matrix (to be quantised)
    and not in F8; raises what else it is."""
    if isinstance(a, F8Matrix):
        if a.block != 1 or a.codes.dim() != 2:
            raise ValueError(f"{what} must be a matrix with blocks of 1")
        return False
    if a.dtype is not _f16 or a.dim() != 2 or not a.is_cuda or not a.is_contiguous():
        _refuse(a, _f16, what)
    return True


def gemm_nt_f8(a, w: F8Matrix, out=None, workspace=None, stream=None):
    """C = a @ W.T, fp16 [M, N], for a [M, K] in F8 with block 1, or in fp16 and
    quantised in the call, and W [N, K] in F8 (gemm_f16_nt_f8).  With w =
    quantize_f8(W, 128) that is a linear layer; its input's gradient is
    gemm_nt_f8(dy, quantize_f8(W, 128, transposed=True)) and its weight's
    gemm_nt_f8(quantize_f8(dy, transposed=True), quantize_f8(x, transposed=True)).
    The workspace that some calls need (see gemm_f16_nt_f8_plan) is allocated
    with torch unless `workspace` is given."""
    if not isinstance(w, F8Matrix):
        raise TypeError("w must be an F8Matrix")
    codes = w.codes
    if codes.dim() != 2:
        raise ValueError("w must be one matrix")
    f16 = _operand(a, "a")
    first = a if f16 else a.codes
    m, k = first.shape[0], a.shape[1]
    n = codes.shape[0]
    if k != w.k:
        raise ValueError(f"shape mismatch: a{tuple(a.shape)} w{w.shape}")
    index = first.get_device()
    if index < 0 or index != codes.get_device():
        raise ValueError("a and w must be on the same GPU")
    out = _output(out, first, stream, (m, n))
    need = _planned((gemm_f16_nt_f8_plan, m, n, k, w.block, f16, index))
    ws, ws_ptr, ws_bytes = None, 0, 0
    if need or workspace is not None:
        ws, ws_ptr, ws_bytes = _workspace(need, first, workspace, stream)
    if f16:
        _call(index, stream, _lib.gemm_f16_nt_f8_x, m, n, k, a.data_ptr(), w.block,
              codes.data_ptr(), w.scales.data_ptr(), out.data_ptr(), ws_ptr, ws_bytes)
    else:
        _call(index, stream, _lib.gemm_f16_nt_f8, m, n, k, first.data_ptr(), a.scales.data_ptr(),
              w.block, codes.data_ptr(), w.scales.data_ptr(), out.data_ptr(), ws_ptr, ws_bytes)
    if stream is not None:
        _record(stream, first, None if f16 else a.scales, codes, w.scales, out, ws)
    return out
