"""CPU oracle of the operators on 8-bit activations, in fp64 numpy.

A row of values r * p_k gets codes rnd(R p_k / P), P = max|p|, nearest code with
ties to even, R = 127 (int8) or 448 (E4M3), and the scale fp32(r P / R). The
fp64 quotient is rounded to 47 bits first, so that a true tie whose p and P are
themselves rounded is a tie. Rows of zeros: scale 0, codes 0. Rows with an infinity or NaN, or a scale past
fp32: scale NaN, codes 0.
"""
from __future__ import annotations

import numpy as np

from .rtq_oracle import decode_f8

TOP = {"q8": 127.0, "f8": 448.0}


def nearest_e4m3(t: np.ndarray) -> np.ndarray:
    """fp64 values of magnitude up to 448 -> the codes of the nearest E4M3 values, ties to the even code."""
    a = np.abs(t)
    grid = decode_f8(np.arange(0x7F, dtype=np.uint8))       # codes 0 .. 0x7E, ascending, 448 the last
    middle = (grid[1:] + grid[:-1]) / 2                     # exact
    low = np.searchsorted(middle, a, side="left")           # middles strictly below a
    tie = (low < len(middle)) & (a == middle[np.minimum(low, len(middle) - 1)])
    code = np.where(tie & (low % 2 == 1), low + 1, low)
    return (code | (np.signbit(t).astype(np.int64) << 7)).astype(np.uint8)


def to_47_bits(t: np.ndarray) -> np.ndarray:
    """fp64 values rounded to 47 significant bits, halves away from zero."""
    return ((t.view(np.uint64) + np.uint64(32)) & ~np.uint64(63)).view(np.float64)


def codes_and_scale(p: np.ndarray, r, fmt: str):
    """p fp64 [M, K], r fp64 [M] or 1: (codes int8 / uint8 [M, K], scale fp32 [M])."""
    p = np.asarray(p, np.float64)
    R = TOP[fmt]
    with np.errstate(all="ignore"):
        P = np.max(np.abs(p), axis=1)                       # NaN propagates
        scale = (P * r / R).astype(np.float32)
        fine = np.isfinite(scale)
        live = fine & (P > 0)
        t = to_47_bits(np.where(live[:, None], R * p / P[:, None], 0.0))
    if fmt == "q8":
        codes = np.rint(t).astype(np.int8)
    else:
        codes = nearest_e4m3(t)
    return codes, np.where(fine, scale, np.float32(np.nan)).astype(np.float32)


def round_to(v: np.ndarray, dtype: str) -> np.ndarray:
    """fp32 values rounded once to the stream's type, as fp32."""
    v = np.asarray(v, np.float32)
    if dtype == "fp32":
        return v
    if dtype == "fp16":
        with np.errstate(over="ignore"):
            return v.astype(np.float16).astype(np.float32)
    b = v.view(np.uint32)
    up = ((b >> 16) & 1) + np.uint32(0x7FFF)
    out = ((b + up) & np.uint32(0xFFFF0000)).view(np.float32)
    return np.where(np.isnan(v), v, out)


def rms_norm_parts(x, residual, weight, eps: float, dtype: str):
    """(h, p, r): the fp32 rows that are normalised, p = h * weight in fp64, the factor r [M]."""
    with np.errstate(all="ignore"):
        h = np.asarray(x, np.float32)
        if residual is not None:
            h = round_to(h + np.asarray(residual, np.float32), dtype)
        d = h.astype(np.float64)
        r = 1.0 / np.sqrt(np.mean(d * d, axis=1) + float(np.float32(eps)))
        return h, d * np.asarray(weight, np.float64), r


def silu_mul(a, b) -> np.ndarray:
    a = np.asarray(a, np.float64)
    with np.errstate(all="ignore"):
        return a / (1.0 + np.exp(-a)) * np.asarray(b, np.float64)


def gemm_a8(x, sx, w, sw, bias, fmt: str):
    """(y, size): the product in fp64, and sum_k |x w| with its scales, which its roundings go by."""
    value = (lambda c: np.asarray(c, np.float64)) if fmt == "q8" else (lambda c: np.asarray(decode_f8(c), np.float64))
    xv, wv = value(x), value(w)
    s = np.asarray(sx, np.float64)[:, None] * (1.0 if sw is None else np.asarray(sw, np.float64)[None, :])
    y = xv @ wv.T * s
    size = np.abs(xv) @ np.abs(wv).T * np.abs(s)
    return (y if bias is None else y + np.asarray(bias, np.float64)), size
