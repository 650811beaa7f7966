"""Plain 64-bit references for the 8-bit floating point operands and for
routing to experts (no library code)."""
from __future__ import annotations

import numpy as np


def code_values() -> np.ndarray:
    """The number that each of the 256 codes stands for."""
    c = np.arange(256)
    e, m = c >> 3 & 15, c & 7
    v = np.where(e > 0, np.ldexp(8.0 + m, e - 10), np.ldexp(m * 1.0, -9))
    v[(c & 127) == 127] = np.nan
    return np.where(c >= 128, -v, v)


def scale_of(largest: np.ndarray) -> np.ndarray:
    """Exponents: the smallest e >= -32 with 448 2^e >= largest, found by trying."""
    e = np.full(largest.shape, -32)
    for k in range(-31, 10):
        e = np.where(448.0 * 2.0 ** (k - 1) < largest, k, e)
    return e


def round_codes(q: np.ndarray) -> np.ndarray:
    """|q| <= 448 rounded to the nearest e4m3 number, ties to even: a multiple of
    2^-9 below 2^-6, else of an eighth of its leading bit."""
    _, e = np.frexp(np.maximum(np.abs(q), 2.0 ** -6))
    place = np.ldexp(1.0, e - 4)
    return np.rint(q / place) * place


def encode(x: np.ndarray, block: int):
    """(values q float64 [R, Kp], exponents int [ceil(R / block), Kp / 128]) of x [R, K]."""
    r, k = x.shape
    rp, kp = -(-r // block) * block, -(-k // 128) * 128
    v = np.zeros((rp, kp))
    v[:r, :k] = x.astype(np.float64)
    finite = np.where(np.isfinite(v), np.abs(v), 0.0).reshape(rp // block, block, kp // 128, 128)
    e = scale_of(finite.max(axis=(1, 3)))
    s = np.repeat(np.repeat(np.ldexp(1.0, e), block, 0), 128, 1)
    v = np.where(np.isfinite(v), v, np.nan)
    return round_codes(v / s)[:r], e


def stored_scales(e: np.ndarray) -> np.ndarray:
    """uint8 [ceil(groups / 4), blocks, 4] of exponents [blocks, groups]; bytes of
    absent groups are 0."""
    blocks, groups = e.shape
    full = np.zeros((blocks, -(-groups // 4) * 4), dtype=np.int64)
    full[:, :groups] = e + 127
    return full.reshape(blocks, -1, 4).transpose(1, 0, 2).astype(np.uint8)


def values(q: np.ndarray, e: np.ndarray, block: int, k: int) -> np.ndarray:
    s = np.repeat(np.repeat(np.ldexp(1.0, e), block, 0), 128, 1)[: q.shape[0]]
    return (q * s)[:, :k]


def quantized(x: np.ndarray, block: int) -> np.ndarray:
    """What x stands for once quantised, in 64 bits."""
    q, e = encode(x, block)
    return values(q, e, block, x.shape[1])


def product_bound(abs_sum: np.ndarray, exact: np.ndarray, k: int) -> np.ndarray:
    """How far a correct product may be from the exact sum.

    The matrix units add eight neighbouring products at a time, each cut towards
    zero at 2^-13 of the largest one's leading bit: less than 8 * 2^-13 of the
    largest for each eight, at most 2^-10 of the sum of magnitudes in all.  A
    path to a result passes K / 8 sums of eight and some to join partial sums
    (64 waves and ranges at most), each a rounding of at most 2^-23 (cut, not
    rounded).  Rounding to fp16 is half a step: 2^-11 of the value, or 2^-25
    among the subnormals."""
    before = abs_sum * (2.0 ** -10 + (k / 8 + 64) * 2.0 ** -23)
    return before + (np.abs(exact) + before) * 2.0 ** -11 + 2.0 ** -25


# ---- routing -------------------------------------------------------------------
def scores_of(x: np.ndarray, kind: str) -> np.ndarray:
    with np.errstate(all="ignore"):
        if kind == "sigmoid":
            return 1.0 / (1.0 + np.exp(-x))
        top = np.where(np.isneginf(x), -1e300, x).max(1, keepdims=True)
        p = np.where(np.isneginf(x), 0.0, np.exp(x - top))
        total = p.sum(1, keepdims=True)
        return p / np.where(total > 0, total, 1.0)


def route(logits: np.ndarray, top: int, kind="softmax", bias=None, groups=1, top_groups=1,
          group_score="top2", renormalize=True, scale=1.0):
    """(experts, weights float64) token by token."""
    x = logits.astype(np.float64)
    t, e = x.shape
    experts, weights = np.full((t, top), -1), np.zeros((t, top))
    s = scores_of(x, kind)
    for i in range(t):
        c = s[i] + (0.0 if bias is None else bias.astype(np.float64))
        if np.isnan(x[i]).any() or np.isnan(np.where(np.isneginf(x[i]), 0, c)).any() or \
                (kind == "softmax" and np.isposinf(x[i]).any()):
            weights[i] = np.nan
            continue
        c = np.where(np.isneginf(x[i]), -np.inf, c)
        if groups > 1:
            per = e // groups
            score = []
            for g in range(groups):
                best = sorted((v for v in c[g * per:(g + 1) * per] if v != -np.inf), reverse=True)
                take = best[:2] if group_score == "top2" else best[:1]
                score.append(sum(take) if take else -np.inf)
            kept = sorted((g for g in range(groups) if score[g] != -np.inf),
                          key=lambda g: (-score[g], g))[:top_groups]
            for g in range(groups):
                if g not in kept:
                    c[g * per:(g + 1) * per] = -np.inf
        order = sorted((j for j in range(e) if c[j] != -np.inf), key=lambda j: (-c[j], j))[:top]
        w = np.array([s[i, j] for j in order])
        if renormalize and len(order):
            w = w / (w.sum() + 1e-20)
        experts[i, :len(order)] = order
        weights[i, :len(order)] = scale * w
    return experts, weights


def order(experts: np.ndarray, e: int):
    """(rows, places, offsets), slot by slot."""
    flat = experts.reshape(-1)
    rows, places = np.full(flat.size, -1), np.full(flat.size, -1)
    offsets = np.zeros(e + 1, dtype=np.int64)
    at = 0
    for k in range(e):
        offsets[k] = at
        for slot in np.nonzero(flat == k)[0]:
            rows[at], places[slot] = slot, at
            at += 1
    offsets[e] = at
    return rows, places.reshape(experts.shape), offsets


def weights_of(x: np.ndarray, experts: np.ndarray, kind, renormalize, scale) -> np.ndarray:
    """The weights as a function of the logits, for chosen experts."""
    s = scores_of(x, kind)
    w = np.where(experts >= 0, np.take_along_axis(s, np.maximum(experts, 0), 1), 0.0)
    if renormalize:
        w = w / (w.sum(1, keepdims=True) + 1e-20)
    return scale * w


def route_gradient(x: np.ndarray, experts: np.ndarray, dw: np.ndarray, kind, renormalize, scale):
    """By the formula, with each derivative written as a matrix."""
    t, e = x.shape
    s = scores_of(x, kind)
    out = np.zeros((t, e))
    for i in range(t):
        on = np.nonzero(experts[i] >= 0)[0]
        chosen = experts[i, on]
        v = s[i, chosen]
        if renormalize:
            total = v.sum() + 1e-20
            dwdv = scale * (np.eye(len(on)) / total - v[:, None] / total ** 2)   # [weight, score]
        else:
            dwdv = scale * np.eye(len(on))
        with np.errstate(all="ignore"):
            if kind == "sigmoid":
                dsdx = np.diag(s[i] / (1.0 + np.exp(x[i])))
            else:
                dsdx = np.diag(s[i]) - np.outer(s[i], s[i])
        dsdx[np.isneginf(x[i])] = 0.0
        dsdx[:, np.isneginf(x[i])] = 0.0
        out[i] = dw[i, on] @ dwdv @ dsdx[chosen]
    return out
