"""Layers of experts: routing, the experts' products, and their combination
(``include/gemm_f16_experts.h`` and ``include/gemm_f16_f8.h``).

    r = route(gemm_nt(x, w_router), 8)             # each token's experts and weights
    h = gemm_nt_f8_experts(x, w_up, r, gather=True)  # a row for each of its choices
    y = gemm_nt_f8_experts(act(h), w_down, r)
    out = combine_experts(y, r)                    # and their weighted sum

Rows of h and y stand in the order of r: by expert.  Nothing here waits for the
GPU: which rows an expert has is read on the device, so that each call can be
captured into a graph whose replays route anew.  The conventions are those of
``lowbit``.
"""
from __future__ import annotations

import ctypes

from . import _check, f8, load
from .f8 import F8Matrix, LowbitPlan, _operand, _planned
from .lowbit import _call, _new, _new_rows, _output, _record, _refuse, _workspace

torch = None

ROUTE_SCORES = {"softmax": 0, "sigmoid": 1}


def _bind_torch() -> None:
    global torch, _f16, _f32, _int32, _uint8, _empty, _lib
    f8._bind_torch()
    t = f8.torch
    _f16, _f32, _int32, _uint8, _empty = t.float16, t.float32, t.int32, t.uint8, t.empty_strided
    _lib = load()
    torch = t


def _declare(lib) -> None:
    """Argument types of the functions of gemm_f16_experts.h."""
    i64, i32, p, d = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_double
    for name, args in {
        "gemm_f16_route_workspace": [i64, i64, i32, ctypes.POINTER(i64)],
        "gemm_f16_route": [i64, i64, i32, i32, i32, i32, i32, i32, d, p, i32, p, p, p, p, p, p, p,
                           i64, p],
        "gemm_f16_route_backward": [i64, i64, i32, i32, i32, d, p, i32, p, p, p, p, p],
        "gemm_f16_combine": [i64, i32, i64, p, p, p, p, p],
        "gemm_f16_combine_backward": [i64, i32, i64, p, p, p, p, p, p, p, p],
    }.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int


# ---- C ABI, same names -----------------------------------------------------
def gemm_f16_nt_f8_experts_plan(S: int, E: int, N: int, K: int, top: int, a_f16: bool,
                                num_cus: int) -> LowbitPlan:
    plan = LowbitPlan()
    _check(load().gemm_f16_nt_f8_experts_plan(S, E, N, K, top, a_f16, num_cus,
                                              ctypes.byref(plan)), "gemm_f16_nt_f8_experts_plan")
    return plan


def gemm_f16_nt_f8_experts(S: int, E: int, N: int, K: int, top: int, a_codes: int, a_scales: int,
                           w_codes: int, w_scales: int, rows: int, offsets: int, C: int,
                           workspace: int = 0, workspace_bytes: int = 0, stream: int = 0) -> None:
    _check(load().gemm_f16_nt_f8_experts(S, E, N, K, top, a_codes, a_scales, w_codes, w_scales,
                                         rows, offsets, C, workspace, workspace_bytes, stream),
           "gemm_f16_nt_f8_experts")


def gemm_f16_nt_f8_experts_x(S: int, E: int, N: int, K: int, top: int, X: int, w_codes: int,
                             w_scales: int, rows: int, offsets: int, C: int, workspace: int = 0,
                             workspace_bytes: int = 0, stream: int = 0) -> None:
    _check(load().gemm_f16_nt_f8_experts_x(S, E, N, K, top, X, w_codes, w_scales, rows, offsets, C,
                                           workspace, workspace_bytes, stream),
           "gemm_f16_nt_f8_experts_x")


def gemm_f16_f8_experts_columns(S: int, E: int) -> int:
    """Columns that S rows of E experts may take, each expert's padded to 128s."""
    columns = ctypes.c_int64()
    _check(load().gemm_f16_f8_experts_columns(S, E, ctypes.byref(columns)),
           "gemm_f16_f8_experts_columns")
    return columns.value


def gemm_f16_f8_quantize_experts(S: int, E: int, R: int, top: int, X: int, rows: int,
                                 offsets: int, codes: int, scales: int, stream: int = 0) -> None:
    _check(load().gemm_f16_f8_quantize_experts(S, E, R, top, X, rows, offsets, codes, scales,
                                               stream), "gemm_f16_f8_quantize_experts")


def gemm_f16_nt_f8_experts_grad_plan(S: int, E: int, M: int, N: int, num_cus: int) -> LowbitPlan:
    plan = LowbitPlan()
    _check(load().gemm_f16_nt_f8_experts_grad_plan(S, E, M, N, num_cus, ctypes.byref(plan)),
           "gemm_f16_nt_f8_experts_grad_plan")
    return plan


def gemm_f16_nt_f8_experts_grad(S: int, E: int, M: int, N: int, a_codes: int, a_scales: int,
                                b_codes: int, b_scales: int, offsets: int, C: int,
                                stream: int = 0) -> None:
    _check(load().gemm_f16_nt_f8_experts_grad(S, E, M, N, a_codes, a_scales, b_codes, b_scales,
                                              offsets, C, stream), "gemm_f16_nt_f8_experts_grad")


def gemm_f16_route_workspace(T: int, E: int, top: int) -> int:
    need = ctypes.c_int64()
    _check(load().gemm_f16_route_workspace(T, E, top, ctypes.byref(need)),
           "gemm_f16_route_workspace")
    return need.value


def gemm_f16_route(T: int, E: int, top: int, scores: int, groups: int, top_groups: int,
                   group_max: bool, renormalize: bool, scale: float, logits: int,
                   logits_f32: bool, bias: int, experts: int, weights: int, rows: int,
                   places: int, offsets: int, workspace: int = 0, workspace_bytes: int = 0,
                   stream: int = 0) -> None:
    _check(load().gemm_f16_route(T, E, top, scores, groups, top_groups, group_max, renormalize,
                                 scale, logits, logits_f32, bias, experts, weights, rows, places,
                                 offsets, workspace, workspace_bytes, stream), "gemm_f16_route")


def gemm_f16_route_backward(T: int, E: int, top: int, scores: int, renormalize: bool,
                            scale: float, logits: int, logits_f32: bool, experts: int,
                            weights: int, dweights: int, dlogits: int, stream: int = 0) -> None:
    _check(load().gemm_f16_route_backward(T, E, top, scores, renormalize, scale, logits,
                                          logits_f32, experts, weights, dweights, dlogits, stream),
           "gemm_f16_route_backward")


def gemm_f16_combine(T: int, top: int, N: int, y: int, weights: int, places: int, out: int,
                     stream: int = 0) -> None:
    _check(load().gemm_f16_combine(T, top, N, y, weights, places, out, stream),
           "gemm_f16_combine")


def gemm_f16_combine_backward(T: int, top: int, N: int, dout: int, y: int, weights: int,
                              rows: int, places: int, dy: int, dweights: int,
                              stream: int = 0) -> None:
    _check(load().gemm_f16_combine_backward(T, top, N, dout, y, weights, rows, places, dy,
                                            dweights, stream), "gemm_f16_combine_backward")


# ---- routing -------------------------------------------------------------------
class Routing:
    """What route() returns for T tokens, `top` choices each, and E experts:

    experts int32 [T, top], -1 where there is none; weights fp32 [T, top]
    rows    int32 [T top]  the slot (token * top + choice) at each position, by
                           expert; -1 from offsets[E] on
    places  int32 [T, top] each slot's position, -1 for no expert
    offsets int32 [E + 1]  where each expert's positions begin (their differences
                           are the experts' loads)

    and how the weights come from the logits (scores, renormalize, scale), for
    route_backward().  The tensors are kept, not copied.  Those that route() makes
    are, but for the weights, parts of one allocation: whoever keeps or saves one of them
    (not a clone() of it) keeps all four.  Saved and read back as a W4Matrix is."""

    __slots__ = ("experts", "weights", "rows", "places", "offsets", "scores", "renormalize",
                 "scale")

    def __init__(self, experts, weights, rows, places, offsets, scores: str = "softmax",
                 renormalize: bool = True, scale: float = 1.0):
        if torch is None:
            _bind_torch()
        if scores not in ROUTE_SCORES:
            raise ValueError(f"scores must be one of {tuple(ROUTE_SCORES)}, not {scores!r}")
        if experts.dtype != _int32 or rows.dtype != _int32 or places.dtype != _int32 or \
                offsets.dtype != _int32 or weights.dtype != _f32:
            raise TypeError("experts, rows, places and offsets must be torch.int32 and weights "
                            "torch.float32")
        if experts.dim() != 2 or experts.shape[1] < 1 or weights.shape != experts.shape or \
                places.shape != experts.shape or tuple(rows.shape) != (experts.numel(),) or \
                offsets.dim() != 1 or offsets.numel() < 2:
            raise ValueError("experts, weights and places must be [tokens, top], rows [tokens * "
                             "top] and offsets [experts + 1]")
        for x in (experts, weights, rows, places, offsets):
            if not x.is_cuda or x.device != experts.device:
                raise ValueError("a routing's tensors must be on the same GPU")
            if not x.is_contiguous():
                raise ValueError("a routing's tensors must be contiguous")
        self._set(experts, weights, rows, places, offsets, scores, bool(renormalize), float(scale))

    def _set(self, experts, weights, rows, places, offsets, scores, renormalize, scale):
        self.experts, self.weights, self.rows = experts, weights, rows
        self.places, self.offsets = places, offsets
        self.scores, self.renormalize, self.scale = scores, renormalize, scale
        return self

    def __reduce__(self):
        return type(self), (self.experts, self.weights, self.rows, self.places, self.offsets,
                            self.scores, self.renormalize, self.scale)

    @property
    def tokens(self) -> int:
        return self.experts.shape[0]

    @property
    def top(self) -> int:
        return self.experts.shape[1]

    @property
    def n_experts(self) -> int:
        return self.offsets.shape[0] - 1

    @property
    def slots(self) -> int:
        return self.rows.shape[0]

    @property
    def device(self):
        return self.experts.device

    def __repr__(self) -> str:
        return (f"Routing({self.tokens} tokens, {self.top} of {self.n_experts} experts, "
                f"device={self.device})")


def _logits(x):
    if x.dtype is not _f16 and x.dtype is not _f32:
        raise TypeError("logits must be torch.float16 or torch.float32")
    if x.dim() != 2 or not x.is_cuda or not x.is_contiguous():
        _refuse(x, x.dtype, "logits")


# workspace bytes of route() by (tokens, experts, top)
_route_bytes: dict = {}


def route(logits, top: int, scores: str = "softmax", bias=None, groups: int = 1,
          top_groups: int = 1, group_score: str = "top2", renormalize: bool = True,
          scale: float = 1.0, stream=None) -> Routing:
    """Chooses each token's `top` experts from its logits [T, E] (fp16 or fp32)
    and orders the rows by expert (gemm_f16_route).

    Scores are the logits' softmax or sigmoid; experts are chosen by score + bias
    (fp32 [E]), where groups > 1 among those of the top_groups groups that score
    highest (by their two best experts, group_score "top2", or their best,
    "max"); ties go to the lowest index.  Weights are the scores without the
    bias, divided by their sum where `renormalize`, times `scale`.  An expert
    whose logit is -inf is not chosen: a row of them has experts -1, weights 0."""
    if torch is None:
        _bind_torch()
    _logits(logits)
    t, e = logits.shape
    if scores not in ROUTE_SCORES:
        raise ValueError(f"scores must be one of {tuple(ROUTE_SCORES)}, not {scores!r}")
    if group_score not in ("top2", "max"):
        raise ValueError(f"group_score must be 'top2' or 'max', not {group_score!r}")
    if not 1 <= e <= 1024 or not 1 <= top <= min(e, 32):
        raise ValueError(f"top must be from 1 to 32 and experts from top to 1024, not {top} of {e}")
    if not 1 <= groups <= 64 or e % groups or not 1 <= top_groups <= groups:
        raise ValueError(f"{e} experts do not stand in {groups} groups (at most 64) of which "
                         f"{top_groups} can be taken")
    if bias is not None and (bias.dtype != _f32 or tuple(bias.shape) != (e,) or
                             bias.device != logits.device or not bias.is_contiguous()):
        raise ValueError(f"bias must be a contiguous float32 [{e}] tensor on {logits.device}")
    top, index = int(top), logits.get_device()
    # one allocation for experts, rows, places and offsets, as tensors of their own (views
    # of one cost the host 1 us more); the weights, of another type, apart, since torch
    # saves no tensors of two types that share memory
    slots = t * top
    size = 3 * slots + e + 1
    if stream is None:
        memory = _empty((size,), (1,), dtype=_int32, device=logits.device)
        weights = _empty((t, top), (top, 1), dtype=_f32, device=logits.device)
    else:
        memory = _new(logits, stream, (size,), _int32)
        weights = _new(logits, stream, (t, top), _f32)
    experts, rows, places, offsets = memory.unsafe_split_with_sizes((slots, slots, slots, e + 1))
    experts, places = experts.view(t, top), places.view(t, top)
    key = (t, e, top)
    need = _route_bytes.get(key)
    if need is None:
        if len(_route_bytes) >= 1024:
            _route_bytes.clear()
        need = _route_bytes[key] = gemm_f16_route_workspace(t, e, top)
    ws = None if not need else _new(logits, stream, (need,), _uint8) if stream is not None else \
        _empty((need,), (1,), dtype=_uint8, device=logits.device)
    at, each = memory.data_ptr(), 4 * slots
    _call(index, stream, _lib.gemm_f16_route, t, e, top, ROUTE_SCORES[scores], groups, top_groups,
          group_score == "max", bool(renormalize), scale, logits.data_ptr(),
          logits.dtype is _f32, 0 if bias is None else bias.data_ptr(), at, weights.data_ptr(),
          at + each, at + 2 * each, at + 3 * each, 0 if ws is None else ws.data_ptr(), need)
    if stream is not None:
        _record(stream, logits, bias, ws)
    return Routing.__new__(Routing)._set(experts, weights, rows, places, offsets, scores,
                                         bool(renormalize), float(scale))


def _routing(r):
    if not isinstance(r, Routing):
        raise TypeError("routing must be a Routing")
    if not r.experts.is_cuda:
        raise ValueError("routing must be on a GPU")


def route_backward(logits, routing: Routing, dweights, stream=None):
    """The gradient of the logits (their type) from that of routing.weights, fp32
    [T, top] (gemm_f16_route_backward).  The choice and the bias have none."""
    _routing(routing)
    _logits(logits)
    if tuple(logits.shape) != (routing.tokens, routing.n_experts) or \
            logits.device != routing.device:
        raise ValueError(f"logits{tuple(logits.shape)} are not those of {routing!r}")
    if dweights.dtype != _f32 or dweights.shape != routing.experts.shape or \
            dweights.device != routing.device or not dweights.is_contiguous():
        raise ValueError(f"dweights must be a contiguous float32 {list(routing.experts.shape)} "
                         f"tensor on {routing.device}")
    out = _new_rows(logits, stream, *logits.shape, logits.dtype)
    _call(logits.get_device(), stream, _lib.gemm_f16_route_backward, routing.tokens,
          routing.n_experts, routing.top, ROUTE_SCORES[routing.scores], routing.renormalize,
          routing.scale, logits.data_ptr(), logits.dtype is _f32, routing.experts.data_ptr(),
          routing.weights.data_ptr(), dweights.data_ptr(), out.data_ptr())
    if stream is not None:
        _record(stream, logits, routing.experts, routing.weights, dweights)
    return out


# ---- the experts' products -------------------------------------------------------
def gemm_nt_f8_experts(a, w: F8Matrix, routing: Routing, gather: bool = False, out=None,
                       workspace=None, stream=None):
    """Row p of C [T top, N], fp16, is a's row times the transpose of its expert's
    W [N, K] (gemm_f16_nt_f8_experts).  a, in F8 with block 1 or in fp16 and
    quantised in the call, is [T top, K] in the routing's order; with `gather` it
    is [T, K], the tokens, and each row is taken for each of its choices.  w:
    quantize_f8 of [E, N, K] with block 128.  With w quantised transposed and the
    gradients of C for a, C is the gradient of the rows, and combine_experts(...,
    weighted=False) adds up those of a token.  Rows past the last expert's
    are 0."""
    _routing(routing)
    if not isinstance(w, F8Matrix):
        raise TypeError("w must be an F8Matrix")
    codes = w.codes
    e, top = routing.n_experts, routing.top
    if codes.dim() != 3 or w.block != 128 or codes.shape[0] != e:
        raise ValueError(f"w must be a stack of {e} matrices with blocks of 128")
    f16 = _operand(a, "a")
    first = a if f16 else a.codes
    slots, n, k = routing.slots, codes.shape[1], a.shape[1]
    if k != w.k or first.shape[0] != (routing.tokens if gather else slots):
        raise ValueError(f"shape mismatch: a{tuple(a.shape)} w{w.shape} {routing!r} "
                         f"gather={gather}")
    index = first.get_device()
    if index < 0 or index != codes.get_device() or index != routing.rows.get_device():
        raise ValueError("a, w and routing must be on the same GPU")
    out = _output(out, first, stream, (slots, n))
    if not gather:
        top = 0
    need = _planned((gemm_f16_nt_f8_experts_plan, slots, e, n, k, top, f16, index))
    ws, ws_ptr, ws_bytes = None, 0, 0
    if need or workspace is not None:
        ws, ws_ptr, ws_bytes = _workspace(need, first, workspace, stream)
    rows, offsets = routing.rows, routing.offsets
    if f16:
        _call(index, stream, _lib.gemm_f16_nt_f8_experts_x, slots, e, n, k, top, a.data_ptr(),
              codes.data_ptr(), w.scales.data_ptr(), rows.data_ptr(), offsets.data_ptr(),
              out.data_ptr(), ws_ptr, ws_bytes)
    else:
        _call(index, stream, _lib.gemm_f16_nt_f8_experts, slots, e, n, k, top, first.data_ptr(),
              a.scales.data_ptr(), codes.data_ptr(), w.scales.data_ptr(), rows.data_ptr(),
              offsets.data_ptr(), out.data_ptr(), ws_ptr, ws_bytes)
    if stream is not None:
        _record(stream, first, None if f16 else a.scales, codes, w.scales, rows, offsets, out, ws)
    return out


def quantize_f8_experts(x, routing: Routing, gather: bool = False, stream=None) -> F8Matrix:
    """x [T top, R] fp16 in the routing's order (or with `gather` [T, R], the
    tokens) in the transposed form [R, columns] that gemm_nt_f8_experts_grad
    takes: an expert's rows are columns from a multiple of 128 on, with zeros up
    to the next; columns past the last expert's are not written."""
    _routing(routing)
    if not (x.dtype is _f16 and x.dim() == 2 and x.is_cuda and x.is_contiguous()):
        _refuse(x, _f16, "x")
    if x.shape[0] != (routing.tokens if gather else routing.slots):
        raise ValueError(f"shape mismatch: x{tuple(x.shape)} {routing!r} gather={gather}")
    index = x.get_device()
    if index != routing.rows.get_device():
        raise ValueError("x and routing must be on the same GPU")
    s, e, r = routing.slots, routing.n_experts, x.shape[1]
    q = f8._new_f8(x, stream, (), r, 128 * (s // 128 + min(e, s)), 1)
    _call(index, stream, _lib.gemm_f16_f8_quantize_experts, s, e, r, routing.top if gather else 0,
          x.data_ptr(), routing.rows.data_ptr(), routing.offsets.data_ptr(), q.codes.data_ptr(),
          q.scales.data_ptr())
    if stream is not None:
        _record(stream, x, routing.rows, routing.offsets)
    return q


def gemm_nt_f8_experts_grad(dy: F8Matrix, x: F8Matrix, routing: Routing, out=None, stream=None):
    """Each expert's dY.T @ X, fp16 [E, N, K], for dy [N, columns] and x [K,
    columns] as quantize_f8_experts makes them: the gradient of its [N, K]
    weight (gemm_f16_nt_f8_experts_grad).  0 for an expert without rows."""
    _routing(routing)
    s, e = routing.slots, routing.n_experts
    columns = 128 * (s // 128 + min(e, s))
    for q, what in ((dy, "dy"), (x, "x")):
        if not isinstance(q, F8Matrix):
            raise TypeError(f"{what} must be an F8Matrix")
        if q.codes.dim() != 2 or q.block != 1 or q.k != columns:
            raise ValueError(f"{what} must be what quantize_f8_experts makes for {routing!r}")
    first = dy.codes
    index = first.get_device()
    if index < 0 or index != x.codes.get_device() or index != routing.offsets.get_device():
        raise ValueError("dy, x and routing must be on the same GPU")
    m, n = first.shape[0], x.codes.shape[0]
    shape = (e, m, n)
    out = _new(first, stream, shape, _f16) if out is None else _output(out, first, stream, shape)
    _call(index, stream, _lib.gemm_f16_nt_f8_experts_grad, s, e, m, n, first.data_ptr(),
          dy.scales.data_ptr(), x.codes.data_ptr(), x.scales.data_ptr(),
          routing.offsets.data_ptr(), out.data_ptr())
    if stream is not None:
        _record(stream, first, dy.scales, x.codes, x.scales, routing.offsets, out)
    return out


# ---- combination -------------------------------------------------------------------
def _rows_of(y, routing, what):
    if not (y.dtype is _f16 and y.dim() == 2 and y.is_cuda and y.is_contiguous()):
        _refuse(y, _f16, what)
    if y.shape[0] != routing.slots:
        raise ValueError(f"shape mismatch: {what}{tuple(y.shape)} {routing!r}")
    if y.get_device() != routing.places.get_device():
        raise ValueError(f"{what} and routing must be on the same GPU")


def combine_experts(y, routing: Routing, weighted: bool = True, out=None, stream=None):
    """out [T, N], fp16: each token's sum over its choices of weight times its row
    of y [T top, N] fp16 (gemm_f16_combine); all weights 1 with weighted=False.
    A choice without an expert adds its weight times 0."""
    _routing(routing)
    _rows_of(y, routing, "y")
    t, n = routing.tokens, y.shape[1]
    out = _output(out, y, stream, (t, n))
    _call(y.get_device(), stream, _lib.gemm_f16_combine, t, routing.top, n, y.data_ptr(),
          routing.weights.data_ptr() if weighted else 0, routing.places.data_ptr(), out.data_ptr())
    if stream is not None:
        _record(stream, y, routing.weights, routing.places, out)
    return out


def combine_experts_backward(dout, y, routing: Routing, weighted: bool = True, stream=None):
    """(dy fp16 [T top, N], dweights fp32 [T, top]) from dout [T, N] fp16, the
    gradient of combine_experts(y, routing) (gemm_f16_combine_backward).  With
    weighted=False all weights are 1, y may be None and dweights is None."""
    _routing(routing)
    if not (dout.dtype is _f16 and dout.dim() == 2 and dout.is_cuda and dout.is_contiguous()):
        _refuse(dout, _f16, "dout")
    t, n = routing.tokens, dout.shape[1]
    if dout.shape[0] != t:
        raise ValueError(f"shape mismatch: dout{tuple(dout.shape)} {routing!r}")
    index = dout.get_device()
    if index != routing.places.get_device():
        raise ValueError("dout and routing must be on the same GPU")
    dweights = None
    if weighted:
        _rows_of(y, routing, "y")
        if y.shape[1] != n:
            raise ValueError(f"shape mismatch: dout{tuple(dout.shape)} y{tuple(y.shape)}")
        dweights = _new_rows(dout, stream, t, routing.top, _f32)
    dy = _new_rows(dout, stream, routing.slots, n, _f16)
    _call(index, stream, _lib.gemm_f16_combine_backward, t, routing.top, n, dout.data_ptr(),
          y.data_ptr() if weighted else 0, routing.weights.data_ptr() if weighted else 0,
          routing.rows.data_ptr(), routing.places.data_ptr(), dy.data_ptr(),
          dweights.data_ptr() if weighted else 0)
    if stream is not None:
        _record(stream, dout, y if weighted else None, routing.weights, routing.rows,
                routing.places)
    return dy, dweights
