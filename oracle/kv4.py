"""Plain numpy statement of the paged 4-bit cache (test infrastructure): the
byte format, rotation and quantisation in the fp32 steps that define them, and
attention and page selection in 64 bits.

Written from the definitions in include/cp.h, one element at a time; it shares
no code with the CUDA library.
"""
from __future__ import annotations

import numpy as np

F32, F16 = np.float32, np.float16
K_NIBBLE = (0, 4, 1, 5, 2, 6, 3, 7)   # nibble of element o of an 8-element run


def places(D: int):
    """Of token t and element d in a 16-token block of 20 D bytes: the byte and
    shift of the K code and of the V code, and the byte of the K scale and of the
    V scale (the minima: 2 and 4 bytes on).  Six [16, D] int arrays."""
    ng = D // 32
    kb, ks, km, vb, vs, vm = (np.zeros((16, D), np.int64) for _ in range(6))
    for t in range(16):
        hf, c, lo = t // 8, t % 8 // 2, t % 2
        for d in range(D):
            gr, r = d // 32, d % 32
            nib = K_NIBBLE[r % 8]
            kb[t, d] = t * D // 2 + (r // 8 * ng + gr) * 4 + nib // 2
            ks[t, d] = 4 * (nib % 2)
            km[t, d] = 8 * D + 4 * (t * ng + gr)
            word = 2 * (hf * 32 * ng + (r // 4 * 4 + c) * ng + gr) + lo
            vb[t, d] = 10 * D + 2 * word + r % 4 // 2
            vs[t, d] = 4 * (r % 2)
            vm[t, d] = 18 * D + 8 * ((4 * hf + c) * ng + gr) + 2 * lo
    return kb, ks, km, vb, vs, vm


def quantise(x):
    """fp32 rows [..., D] -> codes, scale and minimum (fp16) per element."""
    x = np.asarray(x, F32)
    g = x.reshape(*x.shape[:-1], -1, 32)
    bad = ~np.isfinite(g).all(-1, keepdims=True)
    y = np.clip(np.where(bad, F32(0), g), F32(-65408), F32(65408))
    lo, hi = y.min(-1, keepdims=True), y.max(-1, keepdims=True)
    s = ((hi - lo) * F32(1 / 15)).astype(F16)
    m = lo.astype(F16)
    sf, mf = s.astype(F32), m.astype(F32)
    code = np.rint((y - mf) / np.where(sf > 0, sf, F32(1)))
    code = np.clip(np.where(sf > 0, code, F32(0)), 0, 15).astype(np.uint8)
    s, m = np.where(bad, F16(0), s), np.where(bad, F16(np.nan), m)
    code = np.where(bad, np.uint8(0), code)
    shape = x.shape
    return code.reshape(shape), *(np.broadcast_to(z, g.shape).reshape(shape) for z in (s, m))


def rotate(x, cos, sin, interleaved):
    """x [..., D] fp32, cos and sin [..., rot / 2]: every product and sum rounded."""
    x = np.asarray(x, F32).copy()
    h = cos.shape[-1]
    a, b = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
    x1, x2 = x[..., a].copy(), x[..., b].copy()
    x[..., a] = x1 * cos - x2 * sin
    x[..., b] = x2 * cos + x1 * sin
    return x


def bf16(x):
    """fp32 values rounded to bf16 (nearest even), as fp32."""
    u = np.ascontiguousarray(x, F32).view(np.uint32)
    r = ((u + 0x7fff + ((u >> 16) & 1)) & np.uint32(0xffff0000)).view(F32)
    return np.where(np.isfinite(x), r, x).astype(F32)


def write(cache, pages, b, h, slot, k, v):
    """One token's rows (fp32, rotated) into cache [P, Hkv, page, w] uint8."""
    P, Hkv, page, w = cache.shape
    D = w // 5 * 4
    kb, ks, km, vb, vs, vm = places(D)
    block = cache[pages[b, slot // page], h].reshape(-1)[slot % page // 16 * 20 * D:][:20 * D]
    t = slot % 16
    for x, at, sh, meta, step in ((k, kb, ks, km, 2), (v, vb, vs, vm, 4)):
        code, s, m = quantise(x)
        for d in range(D):
            keep = 0x0f if sh[t, d] else 0xf0
            block[at[t, d]] = (block[at[t, d]] & keep) | (code[d] << sh[t, d])
        for d in range(0, D, 32):
            block[meta[t, d]:meta[t, d] + 2] = s[d:d + 1].view(np.uint8)
            block[meta[t, d] + step:meta[t, d] + step + 2] = m[d:d + 1].view(np.uint8)


def read(cache, pages, b, h, slots):
    """Values of the slots (exact in fp32 up to its one rounding): k, v [len(slots), D] in fp32."""
    P, Hkv, page, w = cache.shape
    D = w // 5 * 4
    kb, ks, km, vb, vs, vm = places(D)
    out = np.zeros((2, len(slots), D), F32)
    for i, slot in enumerate(slots):
        block = cache[pages[b, slot // page], h].reshape(-1)[slot % page // 16 * 20 * D:][:20 * D]
        half = np.ascontiguousarray(block).view(F16)
        t = slot % 16
        for x, at, sh, meta, step in ((0, kb, ks, km, 1), (1, vb, vs, vm, 2)):
            code = (block[at[t]] >> sh[t].astype(np.uint8)) & 15
            out[x, i] = code.astype(F32) * half[meta[t] // 2].astype(F32) + half[meta[t] // 2 + step].astype(F32)
    return out[0], out[1]


def attend(q, k, v, scale):
    """One query row against keys k, v [L, D] in 64 bits: out, lse, and
    sum p |v| (what roundings of p and v are relative to)."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    if not len(k):
        return np.zeros(v.shape[-1]), -np.inf, np.zeros(v.shape[-1])
    s = scale * (k @ q)
    top = s.max()
    p = np.exp(s - top)
    z = p.sum()
    return p @ v / z, top + np.log(z), p @ np.abs(v) / z


def select(q, lo, hi, n_sel, keep_first, keep_last):
    """Pages (of the len(lo) that a row sees) by the bound; q [heads, D], lo and hi
    [pages, D]; ascending, -1 behind."""
    n = len(lo)
    q, lo, hi = (np.asarray(x, np.float64) for x in (q, lo, hi))
    score = np.maximum(q[:, None] * lo, q[:, None] * hi).sum(-1).max(0) if n else np.zeros(0)
    score = np.where(np.isnan(score), np.inf, score)
    forced = (np.arange(n) < keep_first) | (np.arange(n) >= n - keep_last)
    order = sorted(range(n), key=lambda i: (not forced[i], -score[i], i))
    take = sorted(order[:n_sel])
    return np.array(take + [-1] * (n_sel - len(take)), np.int32)
