"""Plain 64-bit references for the 4-bit and 8-bit forms (no library code).

Quantising follows the definition in gemm_f16_lowbit.h with exact arithmetic:
scales are looked up in the ascending list of all admissible ones, and every
quotient of an fp16 number and a scale is a float64 quotient, whose rounding
error (2^-53) is far below its distance from a tie unless it is one, and then
it is exact.
"""
from __future__ import annotations

import numpy as np

W4 = dict(bits=8, top=7, most=9344.0)
Q8 = dict(bits=4, top=127, most=576.0)


def scales_list(bits: int, most: float) -> np.ndarray:
    few = np.arange(1, 2 ** bits) * 2.0 ** -24
    more = [m * 2.0 ** e for e in range(-23, 10) for m in range(2 ** (bits - 1), 2 ** bits)]
    all_ = np.unique(np.concatenate([few, more]))
    return all_[all_ <= most]


def encode(x: np.ndarray, group: int, bits: int, top: int, most: float):
    """(codes int64 [R, groups * group], scales float64 [R, groups]) of fp16 x."""
    rows, cols = x.shape
    groups = -(-cols // group)
    v = np.zeros((rows, groups * group))
    v[:, :cols] = x.astype(np.float64)
    v = v.reshape(rows, groups, group)
    bad = ~np.isfinite(v).all(-1)
    v = np.where(bad[..., None], 0.0, v)
    s_all = scales_list(bits, most)
    at = np.minimum(np.searchsorted(s_all * top, np.abs(v).max(-1)), len(s_all) - 1)
    s = s_all[at]
    q = np.rint(v / s[..., None])
    q = np.clip(q, -top, top)
    q = np.where(np.abs(q * s[..., None]) > 65504, q - np.sign(q), q)
    q[bad] = 0
    s = np.where(bad, np.nan, s)
    return q.astype(np.int64).reshape(rows, -1), s


def values(codes: np.ndarray, scales: np.ndarray, group: int, cols: int) -> np.ndarray:
    rows = codes.shape[0]
    v = codes.reshape(rows, -1, group).astype(np.float64) * scales.astype(np.float64)[..., None]
    return v.reshape(rows, -1)[:, :cols]


def w4_words(codes: np.ndarray) -> np.ndarray:
    """int32 words [Nb, Kt, 64, 4] of codes [N, K] in -8..7, one weight at a time."""
    n, k = codes.shape
    nb, kt = -(-n // 16), -(-k // 128)
    full = np.zeros((nb * 16, kt * 128), dtype=np.int64)
    full[:n, :k] = codes
    rows, cols = np.indices(full.shape)
    lane = cols % 32 // 8 * 16 + rows % 16
    word = ((rows // 16 * kt + cols // 128) * 64 + lane) * 4 + cols % 128 // 32
    shift = cols % 2 * 16 + cols % 8 // 2 * 4
    out = np.zeros(nb * kt * 256, dtype=np.uint64)
    np.bitwise_or.at(out, word.ravel(), ((full + 8).astype(np.uint64) << shift.astype(np.uint64)).ravel())
    return out.astype(np.uint32).view(np.int32).reshape(nb, kt, 64, 4)


def w4_scales(scales: np.ndarray, n: int, k: int, group: int, pad: float) -> np.ndarray:
    """[Nb, 128 Kt / group, 16] from [N, ceil(K / group)]; absent ones are `pad`."""
    nb, kt = -(-n // 16), -(-k // 128)
    full = np.full((nb * 16, kt * 128 // group), pad)
    full[:n, :scales.shape[1]] = scales
    return full.reshape(nb, 16, -1).transpose(0, 2, 1)


def round8(s: np.ndarray) -> np.ndarray:
    """fp16 numbers to 8 significant bits, to nearest with ties to even."""
    s = s.astype(np.float64)
    with np.errstate(all="ignore"):
        m, e = np.frexp(s)
        return np.where(np.isfinite(s), np.ldexp(np.rint(np.ldexp(m, 8)), e - 8), s)


def product_bound(a_abs_sum: np.ndarray, exact: np.ndarray, k: int) -> np.ndarray:
    """How far a correct kernel's fp16 result may be from the exact sum.

    The operands' products are exact in fp32: scale times code is an fp16
    number, and two of those make 22 significant bits.  A path to a result
    passes at most 8 fp32 additions for each MFMA of 32 products, K / 4 in all,
    and some to join partial sums (8 waves and 64 ranges: 72; more ranges leave
    each a smaller share of the K / 4), each a rounding of at most 2^-24 of the
    sum of magnitudes.
    The K / 32 more is room that no kernel needs (one that scaled the sum of a
    group of codes would).  Rounding to fp16 is half a step: 2^-11 of the
    value, or 2^-25 among the subnormals."""
    fp32 = (k / 4 + k / 32 + 72) * 2.0 ** -24 * a_abs_sum
    return fp32 + (np.abs(exact) + fp32) * 2.0 ** -11 + 2.0 ** -25
