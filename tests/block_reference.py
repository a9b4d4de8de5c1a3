"""Plain float64 / integer references of the operators that keep state per
block (8-bit float caches, key bounds, chosen blocks) and of the device's block
tables, and the error bound the attention tests use.  numpy only; nothing of
the library is used here."""
from __future__ import annotations

import math

import numpy as np

MIN_EXP = -96
BF16_PARTS = 2.0 ** -18              # see attend()


def e4m3_values() -> np.ndarray:
    """The value of each e4m3 code (NaN for the two NaN codes)."""
    v = np.zeros(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = math.nan if e == 15 and m == 7 else (-x if s else x)
    return v


E4M3 = e4m3_values()
_POS = E4M3[:127]                     # 0 .. 448, ascending


def e4m3_encode(x) -> np.ndarray:
    """Nearest e4m3 code (ties to even), |x| <= 448 after rounding."""
    x = np.asarray(x, np.float64)
    a = np.abs(x)
    hi = np.minimum(np.searchsorted(_POS, a), 126)
    lo = np.maximum(hi - 1, 0)
    dh, dl = np.abs(_POS[hi] - a), np.abs(a - _POS[lo])
    code = np.where(dl < dh, lo, np.where(dl > dh, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code + np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def exponent(amax: float, top: float) -> int:
    """The least e >= MIN_EXP with amax <= top * 2^e."""
    e = MIN_EXP
    if amax > 0:
        e = max(MIN_EXP, math.frexp(amax)[1] - 12)
        while amax > top * 2.0 ** e:
            e += 1
    return e


def runs(slots, bs):
    """(first token, block, offset, rows) of every run of neighbouring new rows of a block."""
    out = []
    t, T = 0, len(slots)
    while t < T:
        s = int(slots[t])
        if s < 0:
            t += 1
            continue
        n = 1
        while t + n < T and (s % bs) + n < bs and int(slots[t + n]) == s + n:
            n += 1
        out.append((t, s // bs, s % bs, n))
        t += n
    return out


def append_f8(x, slots, bs, codes, scales):
    """x [T, H, D] float; codes uint8 [NB, H, bs, D], scales [NB, H] updated in place."""
    x = np.asarray(x, np.float64)
    for t, b, off, n in runs(slots, bs):
        for h in range(x.shape[1]):
            rows = x[t:t + n, h]
            e = exponent(float(np.abs(rows).max()), 448.0)
            if off > 0:
                old = max(MIN_EXP, math.frexp(float(scales[b, h]))[1] - 1 if scales[b, h] > 0 else MIN_EXP)
                if e > old:
                    codes[b, h, :off] = e4m3_encode(E4M3[codes[b, h, :off]] * 2.0 ** (old - e))
                e = max(e, old)
            codes[b, h, off:off + n] = e4m3_encode(rows * 2.0 ** -e)
            scales[b, h] = 2.0 ** e


def append_bounds(k, slots, bs, bounds, exps):
    """k [T, H, D]; bounds int8 [NB, H, 2, D], exps int32 [NB, H] updated in place."""
    k = np.asarray(k, np.float64)
    for t, b, off, n in runs(slots, bs):
        for h in range(k.shape[1]):
            rows = k[t:t + n, h]
            e = exponent(float(np.abs(rows).max()), 127.0)
            old = int(exps[b, h])
            if off > 0:
                e = max(e, old)
            lo, hi = np.floor(rows.min(0) * 2.0 ** -e), np.ceil(rows.max(0) * 2.0 ** -e)
            if off > 0:
                was = bounds[b, h].astype(np.float64) * 2.0 ** (old - e)
                lo, hi = np.minimum(lo, np.floor(was[0])), np.maximum(hi, np.ceil(was[1]))
            bounds[b, h, 0], bounds[b, h, 1] = lo, hi
            exps[b, h] = e


def choose(q, ids, bounds, exps, kvh, budget):
    """q [G, D] of one (sequence, KV head), ids its blocks: the chosen indices, ascending."""
    n = len(ids)
    if n <= budget:
        return np.arange(n)
    q = np.asarray(q, np.float64)
    qi = np.rint(q * 2.0 ** -exponent(float(np.abs(q).max()), 127.0)).astype(np.int64)
    lo, hi = bounds[ids, kvh, 0].astype(np.int64), bounds[ids, kvh, 1].astype(np.int64)
    # sum_d max(qi_d lo_d, qi_d hi_d) for lo <= hi; written by the sign of qi, which also says
    # what bounds the wrong way round give
    s = np.where(qi[:, None] > 0, qi[:, None] * hi[None], qi[:, None] * lo[None]).sum(2).max(0)
    score = s.astype(np.float64) * np.exp2(exps[ids, kvh].astype(np.float64))
    order = np.lexsort((np.arange(n - 1), -score[:n - 1]))
    return np.sort(np.concatenate([order[:budget - 1], [n - 1]]))


def attend(q, k, v, scale, weight=2.0 ** -22):
    """q [G, D], k and v [n, D] (float64): softmax(scale q k^T) v, zeros if n = 0; and the
    error bound of an fp32 kernel.

    The bound, per element.  The kernel's products are exact; a score is a sum of D / 16 MMA
    accumulations in fp32, each off by at most 2^-22 of the sum of magnitudes
    a = max_t scale sum_d |q_d k_td| (an MMA may truncate), plus its roundings to the log2
    domain: (D / 16 + 4) 2^-22 a in all.  A weight is off by that, relatively, plus 2^-22 for
    the exponential and `weight` for its two 16-bit parts (2^-22 for fp16; bf16 parts have 8
    bits each, the second off by half a step of the first one's rest: 2^-18); the sum over n
    rows by an accumulation for each 16 rows and a dozen for joining states, 2^-22 each.
    Numerator and denominator are both off by as much, so the quotient by twice that of
    max |v|."""
    if k.shape[0] == 0:
        return np.zeros_like(q), 0.0
    s = scale * (q @ k.T)
    w = np.exp(s - s.max(1, keepdims=True))
    a = scale * (np.abs(q) @ np.abs(k).T).max()
    D, n = k.shape[1], k.shape[0]
    tol = 2.0 * (2.0 ** -22 * ((D / 16 + 4) * a + n / 16 + 15) + weight) * np.abs(v).max()
    return (w @ v) / w.sum(1, keepdims=True), tol


def reserve(free, lens, new, tables, bs):
    """Device reservation, one sequence after another; `free` (list, top last), lens and tables
    updated in place.  Returns the slots."""
    slots = []
    for b in range(len(lens)):
        for _ in range(int(new[b])):
            p = int(lens[b])
            if p % bs == 0:
                tables[b, p // bs] = free.pop()
            slots.append(int(tables[b, p // bs]) * bs + p % bs)
            lens[b] += 1
    return slots
