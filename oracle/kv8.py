"""Plain statement of the paged 8-bit cache (test infrastructure): the format by its bits,
appending block by block, attention and eviction in 64 bits.

Written from the definitions in include/cp.h with numpy; it shares no code with the
CUDA library.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 16
NAN = 0x7f


def decode(code):
    """e4m3 bytes -> values (64 bits): sign, exponent of bias 7, three bits of mantissa."""
    c = np.asarray(code).astype(np.int64)
    e, m = (c >> 3) & 15, (c & 7).astype(np.float64)
    v = np.where(e > 0, np.ldexp(1 + m / 8, e - 7), np.ldexp(m / 8, -6))
    v = np.where((c & 0x7f) == NAN, math.nan, v)
    return np.where(c & 0x80, -v, v)


POSITIVE = decode(np.arange(NAN))       # the 127 magnitudes, ascending


def encode(x):
    """Values -> the nearest e4m3 bytes, ties to the even one, held within +-448; infinities and
    NaN become NaN."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.where(np.isfinite(x), np.abs(x), 0), 448.0)
    hi = np.clip(np.searchsorted(POSITIVE, a), 1, NAN - 1)
    lo = hi - 1
    dl, dh = a - POSITIVE[lo], POSITIVE[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = code | np.where(np.signbit(x), 0x80, 0)
    return np.where(np.isfinite(x), code, NAN).astype(np.uint8)


def scale_of(x):
    """2^e, e the smallest integer in [-40, 60] with amax <= 448 2^e over the finite values of x."""
    f = np.abs(np.asarray(x, np.float64))
    top = f[np.isfinite(f)].max(initial=0.0)
    e = -40
    while e < 60 and top > math.ldexp(448.0, e):
        e += 1
    return math.ldexp(1.0, e)


def append(cache, scales, pages, lens, k, v, n_new=None):
    """Rows k, v [B, n, Hkv, D] into cache [P, Hkv, 2, page, D] uint8 and scales [P, Hkv, 2, page / 16]."""
    page = cache.shape[3]
    B, n, H, _ = k.shape
    for b in range(B):
        m = n if n_new is None else min(max(int(n_new[b]), 0), n)
        a, z = int(lens[b]), int(lens[b]) + m
        for first in range(a // BLOCK * BLOCK, z, BLOCK):
            lo, hi = max(first, a), min(first + BLOCK, z)
            p, at = pages[b, first // page], first % page
            for h in range(H):
                for w, x in enumerate((k, v)):
                    new = np.asarray(x[b, lo - a:hi - a, h], np.float64)
                    s = scale_of(new)
                    row = cache[p, h, w, at:at + BLOCK]
                    if lo > first:
                        old = float(scales[p, h, w, at // BLOCK])
                        s = max(s, old)
                        if s > old:
                            row[:lo - first] = encode(decode(row[:lo - first]) * (old / s))
                    row[lo - first:hi - first] = encode(new / s)
                    scales[p, h, w, at // BLOCK] = s


def read(cache, scales, pages, b, h, slots):
    """Values of the slots: k, v [len(slots), D]."""
    page = cache.shape[3]
    slots = np.asarray(slots, np.int64)
    p, at = pages[b, slots // page], slots % page
    return [decode(cache[p, h, w, at]) * scales[p, h, w, at // BLOCK].astype(np.float64)[:, None] for w in (0, 1)]


def sees(limit, window, sinks):
    """Slots that a row of that limit sees."""
    if window <= 0 or limit <= window:
        return np.arange(max(limit, 0))
    low = limit - window
    return np.concatenate([np.arange(min(sinks, low)), np.arange(low, limit)])


def attend(q, k, v, vs, scale):
    """One query row against keys k and values v [L, D] (vs: each value row's scale) in 64 bits: out, lse,
    the weights, and what an output may be off by: weights in fp16 (2^-11 of themselves, or 2^-32 of the largest
    product of weight and scale), scores as fp32 sums of D exact products."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    if not len(k):
        return np.zeros(v.shape[-1]), -math.inf, np.zeros(0), np.zeros(v.shape[-1]), 0.0
    s = scale * (k @ q)
    top = s.max()
    p = np.exp(s - top)
    z = p.sum()
    p /= z
    ds = scale * (np.abs(k) @ np.abs(q)).max() * (q.size + 8) * 2.0 ** -23 + 2.0 ** -20
    rel = 2.0 ** -11 + 2 * ds + (len(k) / 16 + 40) * 2.0 ** -23
    err = rel * (p @ np.abs(v)) + 2.0 ** -32 * (p * vs).max() * (np.abs(v) / vs[:, None]).sum(0)
    return p @ v, top + math.log(z), p, err, ds + 2.0 ** -21 + 2.0 ** -22 * abs(top + math.log(z))


def evict(mass, length, budget, first, last):
    """The slots that stay of one kv head: ascending."""
    m = np.where(np.isnan(mass[:length]), np.finfo(np.float64).max, np.asarray(mass[:length], np.float64))
    m = np.where(np.isposinf(mass[:length]), np.finfo(np.float64).max / 2, m)
    forced = (np.arange(length) < first) | (np.arange(length) >= length - last)
    m = np.where(forced, math.inf, m)
    order = np.argsort(-m, kind="stable")
    return np.sort(order[:min(budget, length)])


def moved(cache, scales, pages, b, h, w, slots):
    """Codes and scales of the rows of `slots` in a block-wise row of their own: codes [n, D], scales [blocks]."""
    page = cache.shape[3]
    slots = np.asarray(slots, np.int64)
    p, at = pages[b, slots // page], slots % page
    code, s = cache[p, h, w, at], scales[p, h, w, at // BLOCK].astype(np.float64)
    out, tops = np.zeros_like(code), []
    for i in range(0, len(slots), BLOCK):
        top = s[i:i + BLOCK].max()
        tops.append(top)
        f = (s[i:i + BLOCK] / top)[:, None]
        out[i:i + BLOCK] = np.where(f == 1, code[i:i + BLOCK], encode(decode(code[i:i + BLOCK]) * f))
    return out, np.array(tops)
