"""Plain numpy forms of the int8 lm_head and sampling operators, in 64 bits.

Written from the operators' definitions; they share no code with the library.
"""
from bisect import bisect_left, bisect_right
from fractions import Fraction
from itertools import accumulate

import numpy as np


def bf16_to_f32(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32)


def f32_to_bf16(x):
    """bf16 bits of float32 values, round to nearest even; infinities kept, NaN as 0x7fc0."""
    x = np.ascontiguousarray(x, np.float32)
    u = x.view(np.uint32)
    r = ((u + ((u >> 16) & 1) + 0x7FFF) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), r)


def quantize(x):
    """(codes int8, scale f32): both quotients are 64-bit ones rounded to f32, which are the
    correctly rounded f32 quotients (53 >= 2 * 24 + 2 bits)."""
    x = np.asarray(x, np.float64)
    top = np.abs(x).max(1)
    fine = np.isfinite(top)
    with np.errstate(invalid="ignore", over="ignore"):
        scale = np.where(fine, (np.where(fine, top, 0.0) / 127.0).astype(np.float32), np.float32(np.nan))
        s = scale.astype(np.float64)[:, None]
        some = fine[:, None] & (s > 0)
        ratio = np.divide(x, s, out=np.zeros_like(x), where=some & np.isfinite(x)).astype(np.float32)
    return np.clip(np.rint(ratio), -127, 127).astype(np.int8), scale.astype(np.float32)


def product(a, sa, w, sw):
    """float32 values before the output rounding: the exact integer sum, rounded to f32,
    times the two scales with one rounding each."""
    acc = np.empty((a.shape[0], w.shape[0]), np.int64)
    for n in range(0, w.shape[0], 4096):  # every partial sum is an integer below 2^53
        acc[:, n:n + 4096] = np.matmul(a.astype(np.float64), w[n:n + 4096].astype(np.float64).T).astype(np.int64)
    with np.errstate(invalid="ignore", over="ignore", under="ignore"):
        return acc.astype(np.float32) * sa.astype(np.float32)[:, None] * sw.astype(np.float32)[None, :]


def sample_row(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, allowed=None):
    """(id, probability) of one row; logits and settings are taken as the f32 values they are."""
    l = np.asarray(logits, np.float64)
    u, temperature, top_p, min_p = (float(np.float32(v)) for v in (u, temperature, top_p, min_p))
    if not (0 <= u < 1 and 0 <= temperature < np.inf and top_k >= 0 and 0 < top_p <= 1 and 0 <= min_p <= 1):
        return -1, 0.0
    live = ~np.isnan(l) & (l > -np.inf)
    if allowed is not None:
        live &= np.asarray(allowed, bool)
    ids = np.flatnonzero(live)
    if ids.size == 0:
        return -1, 0.0
    order = ids[np.lexsort((ids, -l[ids]))]
    M = l[order[0]]
    if temperature == 0:
        return int(order[0]), 1.0
    with np.errstate(invalid="ignore", over="ignore", under="ignore"):
        w = np.where(l[order] == M, 1.0, np.exp((l[order] - M) / temperature))
    n = min(order.size, top_k) if top_k > 0 else order.size
    # sums and products of the 64-bit weights without any rounding, as integers of 2^-200
    units = [int(x) for x in w * 2.0 ** 200]
    before = [0] + list(accumulate(units))
    keep = np.arange(order.size) < n
    if top_p < 1:
        goal = Fraction(top_p) * before[n]
        keep &= np.arange(order.size) < bisect_left(before, goal)
    keep &= w >= min_p
    kept = sorted((int(i), x) for i, x in zip(order[keep], np.array(units, object)[keep]))
    sums = list(accumulate(x for _, x in kept))
    j = min(bisect_right(sums, Fraction(u) * sums[-1]), len(kept) - 1)
    return kept[j][0], float(Fraction(kept[j][1], sums[-1]))


def pack_allowed(mask):
    """bool [..., V] -> int32 words [..., ceil(V / 32)], bit v % 32 of word v / 32."""
    mask = np.asarray(mask, bool)
    V = mask.shape[-1]
    padded = np.zeros(mask.shape[:-1] + (-(-V // 32) * 32,), bool)
    padded[..., :V] = mask
    return np.ascontiguousarray(np.packbits(padded, axis=-1, bitorder="little")).view(np.int32)
