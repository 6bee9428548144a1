"""The paged 4-bit cache on the GPU, against the plain statement in oracle/kv4.py.

Append and read-back are compared bit for bit.  Attention is held to bounds
counted from its roundings: with A = sum p |v| / sum p of a row,
  - the weight p of a token is rounded to fp16 (2^-11 relative; below fp16's
    normal range by at most 2^-25 of a weight whose reference is at least one
    2^-8th of the largest), V's value to fp16 (2^-11, 2^-25 below the normal
    range): (2^-11 + 2^-11) A and small terms,
  - fp32 accumulation: at most one rounding of 2^-23 (the tensor core may truncate)
    per 16 tokens and per join,
  - the output's own rounding to bf16: its 8 bits put neighbours at [1, 2) 2^-7 apart,
    so half a step is up to 2^-8 relative.
lse: a score is a sum of D / 32 groups, each an fp32 sum of exact products; with
B = scale sum_d (s code + |m|) |q| it is off by at most 2^-19 B, and exponent and
logarithm by a few 2^-22 of the terms.
"""
import math

import numpy as np
import pytest
import torch

from context_parallelism_02_gb300 import _lib, api, inputs
from oracle import kv4 as o

pytestmark = pytest.mark.gpu
I32 = torch.int32


def rope(max_pos, rot):
    ang = np.arange(max_pos)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)


def table(rng, B, M, spare=3):
    """A page table in random order and the pool's size."""
    P = B * M + spare
    return rng.permutation(P)[:B * M].reshape(B, M).astype(np.int32), P


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).cuda()


def ok():
    torch.cuda.synchronize()
    assert api.cp_get_error() == 0


def rows(rng, dtype, *shape):
    x = rng.standard_normal(shape).astype(np.float32)
    return o.bf16(x) if dtype == torch.bfloat16 else x


APPEND = [  # B, n, Hq, Hkv, D, page, rot, interleaved, dtype, fused, ragged
    (1, 1, 4, 2, 128, 64, 128, False, torch.bfloat16, False, False),
    (3, 1, 8, 1, 64, 16, 64, False, torch.bfloat16, True, True),
    (2, 37, 2, 2, 128, 16, 64, False, torch.float32, False, True),
    (2, 150, 3, 1, 64, 32, 32, True, torch.bfloat16, True, False),
    (1, 300, 2, 2, 64, 128, 64, False, torch.float32, True, False),
    (4, 70, 2, 1, 128, 256, 96, False, torch.bfloat16, False, True),
    (2, 65, 1, 1, 128, 64, 0, False, torch.bfloat16, False, True),
    (1, 33, 2, 1, 128, 32, 128, True, torch.float32, False, False),
]


@pytest.mark.parametrize("B,n,Hq,Hkv,D,page,rot,inter,dtype,fused,ragged", APPEND)
def test_append_bytes(cuda_dev, B, n, Hq, Hkv, D, page, rot, inter, dtype, fused, ragged):
    rng = np.random.default_rng(B * 1000 + n)
    lens = np.array([(17 * b * b + 5 * b) % 90 if B > 1 else 41 for b in range(B)], np.int32)
    n_new = np.array([(n - 7 * b) % (n + 1) for b in range(B)], np.int32) if ragged else None
    M = (int(lens.max()) + n + page - 1) // page
    pages, P = table(rng, B, M)
    cache = rng.integers(0, 256, (P, Hkv, page, D // 4 * 5), dtype=np.uint8)
    summ = o.bf16(rng.standard_normal((P, Hkv, 2, D)))
    q, k, v = (rows(rng, dtype, B, n, h, D) for h in (Hq, Hkv, Hkv))
    pos = rng.integers(0, 500, (B, n)).astype(np.int32) if n % 2 else None
    cos, sin = rope(500, rot) if rot else (None, None)
    if fused:
        x = torch.cat([dev(t, dtype).flatten(2) for t in (q, k, v)], -1)
        gq, gk, gv = (t.unflatten(-1, (-1, D)) for t in x.split([Hq * D, Hkv * D, Hkv * D], -1))
    else:
        gq, gk, gv = (dev(t, dtype) for t in (q, k, v))
    gc, gs = dev(cache), dev(summ, torch.bfloat16)
    got_q = api.kv4_append(gk, gv, gc, dev(pages), dev(lens), cos=None if cos is None else dev(cos),
                           sin=None if sin is None else dev(sin), q=gq, n_new=None if n_new is None else dev(n_new),
                           positions=None if pos is None else dev(pos), summary=gs, interleaved=inter)
    ok()
    want_q = np.zeros_like(q)
    for b in range(B):
        m = n if n_new is None else int(n_new[b])
        for j in range(m):
            slot = int(lens[b]) + j
            at = slot if pos is None else int(pos[b, j])
            kk, qq = k[b, j], q[b, j]
            if rot:
                kk, qq = o.rotate(kk, cos[at], sin[at], inter), o.rotate(qq, cos[at], sin[at], inter)
            want_q[b, j] = o.bf16(qq) if dtype == torch.bfloat16 else qq
            for h in range(Hkv):
                o.write(cache, pages, b, h, slot, kk[h], v[b, j, h])
                box = summ[pages[b, slot // page], h]
                r = o.bf16(kk[h])
                fresh = slot % page == 0
                box[0] = r if fresh else np.minimum(box[0], r)
                box[1] = r if fresh else np.maximum(box[1], r)
    np.testing.assert_array_equal(got_q.float().cpu().numpy(), want_q)
    np.testing.assert_array_equal(gc.cpu().numpy(), cache)
    np.testing.assert_array_equal(gs.float().cpu().numpy(), summ)


def test_append_one_by_one_equals_at_once(cuda_dev):
    rng = np.random.default_rng(5)
    B, n, H, D, page = 2, 45, 2, 128, 16
    pages, P = table(rng, B, 4)
    k, v = (dev(rows(rng, torch.bfloat16, B, n, H, D), torch.bfloat16) for _ in range(2))
    cos, sin = (dev(x) for x in rope(64, D))
    pools = [(torch.zeros(P, H, page, 160, dtype=torch.uint8, device="cuda"),
              torch.zeros(P, H, 2, D, dtype=torch.bfloat16, device="cuda")) for _ in range(2)]
    lens = dev(np.array([0, 19], np.int32))
    api.kv4_append(k, v, pools[0][0], dev(pages), lens, cos, sin, summary=pools[0][1])
    for j in range(n):
        api.kv4_append(k[:, j:j + 1], v[:, j:j + 1], pools[1][0], dev(pages), lens + j, cos, sin, summary=pools[1][1])
    ok()
    for x, y in zip(*pools):
        assert torch.equal(x, y)


def test_append_values_that_are_not_finite_or_too_large(cuda_dev):
    D, page = 64, 16
    k = torch.zeros(1, 4, 1, D)
    k[0, 0, 0, 3] = math.nan
    k[0, 1, 0, 40] = -math.inf
    k[0, 2, 0, :] = torch.linspace(-1e30, 1e30, D)
    k[0, 3] = 2.5                              # a constant group: scale 0
    v = k.flip(1).contiguous()
    pages, lens = dev(np.array([[0]], np.int32)), dev(np.array([0], np.int32))
    cache, summ = api.kv4_cache(1, 1, page, D, summary=True)
    api.kv4_append(k.cuda(), v.cuda(), cache, pages, lens, summary=summ)
    gk, gv = api.kv4_gather(cache, pages, lens + 4, 4, dtype=torch.float32)
    ok()
    assert torch.equal(gk.flip(1).isnan(), gv.isnan())
    x = gk[0, :, 0].cpu()
    assert x[0, :32].isnan().all() and (x[0, 32:] == 0).all()
    assert x[1, 32:].isnan().all() and (x[1, :32] == 0).all()
    # -65408 is an fp16 (a multiple of 32); + 15 roundings of the scale, at most 4 each
    assert (x[2, :31] == -65408).all() and x[2].abs().max() <= 65408 + 15 * 4 + 16 and (x[3] == 2.5).all()
    s = summ[0, 0].float().cpu()               # a key that is not finite opens its elements' range
    assert s[0, 3] == -math.inf and s[1, 3] == math.inf and s[0, 40] == -math.inf and s[1, 40] == math.inf


def test_append_codes_on_exact_halves(cuda_dev):
    """Values half way between two codes go to the even one, as the quotient does: bf16 values meet such halves."""
    rng = np.random.default_rng(18)
    D, page = 128, 16
    v = rng.integers(0, 31, (1, 64, 2, D)).astype(np.float32) * 0.5     # s = 1 where 0 and 15 are in the group
    v[..., ::32], v[..., 1::32] = 0.0, 15.0
    v *= np.exp2(rng.integers(-6, 7, (1, 64, 2, 1))).astype(np.float32)
    k = o.bf16(rng.standard_normal((1, 64, 2, D)) * 3)
    pages, P = table(rng, 1, 4)
    cache = np.zeros((P, 2, page, D // 4 * 5), np.uint8)
    gc = dev(cache)
    api.kv4_append(dev(k, torch.bfloat16), dev(v, torch.bfloat16), gc, dev(pages), dev(np.array([0], np.int32)))
    ok()
    for t in range(64):
        for h in range(2):
            o.write(cache, pages, 0, h, t, k[0, t, h], v[0, t, h])
    np.testing.assert_array_equal(gc.cpu().numpy(), cache)


def test_attn_of_the_largest_values_is_finite(cuda_dev):
    """Values of both signs at the end of the range in one group: s code + m stays below fp16's overflow (65520)."""
    D = 64
    v = (torch.ones(1, 8, 1, D, device="cuda") * 1e30).cumprod(-1).clamp(max=1e30)
    v[..., ::2] *= -1
    v[0, 1] *= 0.5e-30 * 65408                    # other scales, whose roundings go other ways
    v[0, 2] = v[0, 0].sign() * 65000
    cache, lens = api.kv4_cache(1, 1, 16, D), dev(np.array([0], np.int32))
    pages = dev(np.array([[0]], np.int32))
    api.kv4_append(torch.zeros_like(v), v, cache, pages, lens)
    q = torch.zeros(1, 1, 1, D, dtype=torch.bfloat16, device="cuda")
    out, _ = api.kv4_attn(q, cache, pages, lens + 8)
    ok()
    assert torch.isfinite(out).all()


GATHER = [(1, 1, 1, 128, 64), (2, 100, 2, 64, 16), (3, 77, 1, 128, 32), (2, 300, 2, 64, 256)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,count,Hkv,D,page", GATHER)
def test_gather(cuda_dev, B, count, Hkv, D, page, dtype):
    rng = np.random.default_rng(count)
    M = (count + 60 + page - 1) // page
    pages, P = table(rng, B, M)
    k, v = (rows(rng, torch.float32, B, M * page, Hkv, D) for _ in range(2))
    cache = torch.zeros(P, Hkv, page, D // 4 * 5, dtype=torch.uint8, device="cuda")
    api.kv4_append(dev(k), dev(v), cache, dev(pages), dev(np.zeros(B, np.int32)))
    start = np.array([(13 * b) % 40 + (b > 0) for b in range(B)], np.int32)
    lens = np.array([count + int(start[b]) - (0, 5, count // 2)[b] for b in range(B)], np.int32)
    for st in (None, start):
        gk, gv = api.kv4_gather(cache, dev(pages), dev(lens), count, start=None if st is None else dev(st), dtype=dtype)
        ok()
        host = cache.cpu().numpy()
        for b in range(B):
            s0 = 0 if st is None else int(st[b])
            m = max(0, min(count, int(lens[b]) - s0))
            for h in range(Hkv):
                for got, want in zip((gk, gv), o.read(host, pages, b, h, range(s0, s0 + m))):
                    want = o.bf16(want) if dtype == torch.bfloat16 else want
                    np.testing.assert_array_equal(got[b, :m, h].float().cpu().numpy(), want)
                    assert (got[b, m:, h] == 0).all()


def fill(rng, B, L, Hkv, D, page, shift=True):
    """A pool holding L tokens of each sequence; what is behind them is NaN."""
    M = (L + page - 1) // page + 1
    pages, P = table(rng, B, M)
    k, v = (rows(rng, torch.bfloat16, B, max(L, 1), Hkv, D) for _ in range(2))
    if shift:
        k += 0.5
        v -= 1.25
    cache = torch.full((P, Hkv, page, D // 4 * 5), 255, dtype=torch.uint8, device="cuda")
    summ = torch.full((P, Hkv, 2, D), math.nan, dtype=torch.bfloat16, device="cuda")
    if L:
        api.kv4_append(dev(k, torch.bfloat16), dev(v, torch.bfloat16), cache, dev(pages),
                       dev(np.zeros(B, np.int32)), summary=summ)
    return cache, summ, pages


def check_attn(out, lse, q, cache, pages, limits, scale, slots_of=None):
    """Every row against the oracle; limits [B, n]."""
    host = cache.cpu().numpy()
    B, n, Hq, D = q.shape
    Hkv = host.shape[1]
    got, glse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(B):
        for h in range(Hkv):
            top = int(limits[b].max())
            kk, vv = o.read(host, pages, b, h, range(top))
            for j in range(n):
                lim = int(limits[b, j])
                at = np.arange(lim) if slots_of is None else np.array([s for s in slots_of(b, j, h) if s < lim], int)
                for x in range(h * Hq // Hkv, (h + 1) * Hq // Hkv):
                    want, z, a = o.attend(q[b, j, x], kk[at], vv[at], scale)
                    # 2^-25: a weight or value below fp16's normal range; references lag by up to 2^8
                    tol = (2 * 2.0 ** -11 + (len(at) / 16 + 32) * 2.0 ** -23) * a \
                        + len(at) * 2.0 ** -25 * np.abs(vv[at]).max(initial=0) + 2.0 ** -25
                    if out.dtype == torch.bfloat16:
                        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
                    err = np.abs(got[b, j, x] - want)
                    assert (err <= tol).all(), (b, j, x, lim, float((err / tol).max()))
                    if not len(at):
                        assert glse[b, x, j] == -np.inf
                        continue
                    size = scale * (np.abs(q[b, j, x]) @ (np.abs(kk[at]).max(0) + 8.0))
                    assert abs(glse[b, x, j] - z) <= 2.0 ** -19 * size + 2.0 ** -20 * (abs(z) + 1), \
                        (b, j, x, lim, glse[b, x, j], z)


ATTN = [  # lens, n, Hq, Hkv, D, page
    ([1], 1, 1, 1, 128, 64),
    ([0, 1, 15, 16, 17], 1, 4, 2, 128, 16),
    ([33, 64, 100, 0, 31], 1, 8, 1, 64, 32),
    ([700, 3], 1, 14, 2, 128, 64),
    ([513, 260], 1, 16, 1, 64, 128),
    ([300, 7, 1], 2, 6, 2, 128, 16),
    ([129, 40], 5, 8, 2, 64, 64),
    ([1000], 3, 20, 1, 128, 256),
    ([90, 2], 16, 4, 1, 64, 16),
    ([2500, 1100, 4], 1, 4, 4, 128, 64),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,n,Hq,Hkv,D,page", ATTN)
def test_attn(cuda_dev, lens, n, Hq, Hkv, D, page, causal):
    rng = np.random.default_rng(sum(lens) + n)
    B = len(lens)
    cache, _, pages = fill(rng, B, max(lens), Hkv, D, page)
    lens = np.array(lens, np.int32)
    # behind a sequence's own length: NaN rows, and table entries that name no page
    for b in range(B):
        m = max(lens) - lens[b]
        if m:
            nan = torch.full((1, int(m), Hkv, D), math.nan, dtype=torch.bfloat16, device="cuda")
            api.kv4_append(nan, nan, cache, dev(pages[b:b + 1]), dev(lens[b:b + 1]))
    used = np.where(np.arange(pages.shape[1]) * page < lens[:, None], pages, -1).astype(np.int32)
    q = rows(rng, torch.bfloat16, B, n, Hq, D)
    q[:, -1, 0] *= 6.0                                   # one row with a sharp softmax
    q = o.bf16(q)                                        # what the kernel gets
    out, lse = api.kv4_attn(dev(q, torch.bfloat16), cache, dev(used), dev(lens), causal=causal)
    f32 = torch.empty(B, n, Hq, D, device="cuda")
    api.kv4_attn(dev(q, torch.bfloat16), cache, dev(used), dev(lens), causal=causal, scale=0.3, out=f32)
    out2, lse2 = api.kv4_attn(dev(q, torch.bfloat16), cache, dev(used), dev(lens), causal=causal)
    ok()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    lim = lens[:, None] - (n - 1) + np.arange(n) if causal else np.repeat(lens[:, None], n, 1)
    lim = np.maximum(lim, 0)
    check_attn(out, lse, q, cache, pages, lim, 1 / math.sqrt(D))
    _, lse3 = api.kv4_attn(dev(q, torch.bfloat16), cache, dev(used), dev(lens), causal=causal, scale=0.3, out=f32)
    ok()
    check_attn(f32, lse3, q, cache, pages, lim, 0.3)


def test_attn_visible_counts_and_empty_rows(cuda_dev):
    rng = np.random.default_rng(8)
    cache, _, pages = fill(rng, 2, 200, 2, 128, 32)
    vis = np.array([[0, 200, 5, -4, 31], [1, 999, 16, 17, 100]], np.int32)
    lens = np.array([200, 150], np.int32)
    q = rows(rng, torch.bfloat16, 2, 5, 6, 128)
    out, lse = api.kv4_attn(dev(q, torch.bfloat16), cache, dev(pages), dev(lens), vis=dev(vis))
    ok()
    check_attn(out, lse, q, cache, pages, np.clip(vis, 0, lens[:, None]), 1 / math.sqrt(128))
    assert (out[0, 0] == 0).all() and lse[0, :, 0].isinf().all()


@pytest.mark.parametrize("D,group", [(64, 2), (128, 5)])
def test_attn_unseen_tokens_that_are_not_finite(cuda_dev, D, group):
    """A later token whose key and value are not finite reaches only the rows that see it."""
    rng = np.random.default_rng(9)
    cache, _, pages = fill(rng, 1, 40, 1, D, 16)
    q = rows(rng, torch.bfloat16, 1, 4, group, D)
    bad = torch.full((1, 1, 1, D), math.inf, dtype=torch.bfloat16, device="cuda")
    good = torch.ones_like(bad)
    lens = dev(np.array([40], np.int32))
    ref, rlse = api.kv4_attn(dev(q, torch.bfloat16), cache, dev(pages), lens)
    for k, v in ((bad, bad), (good, bad), (bad, good)):
        trial = cache.clone()
        api.kv4_append(k, v, trial, dev(pages), lens - 2)        # slot 38: rows 0 and 1 do not see it
        out, lse = api.kv4_attn(dev(q, torch.bfloat16), trial, dev(pages), lens)
        ok()
        if k is bad and v is bad:
            assert torch.isfinite(lse[..., :2]).all()
        assert torch.equal(lse[..., :2], rlse[..., :2])
        # other order of the sums: twice the bound, 2 (2^-11 + 2^-11) A with A <= 6, and the bf16 step
        assert (out[0, :2].float() - ref[0, :2].float()).abs().max() <= 4 * 2.0 ** -11 * 6 + 2 * 2.0 ** -8 * 4
        assert out[0, 2:].isnan().all()


def test_attn_bad_pages_and_lengths_are_reported_and_skipped(cuda_dev):
    rng = np.random.default_rng(10)
    cache, _, pages = fill(rng, 2, 96, 1, 64, 32)
    q = rows(rng, torch.bfloat16, 2, 1, 2, 64)
    gq = dev(q, torch.bfloat16)
    lens = np.array([96, 96], np.int32)
    for wrong in (-1, cache.shape[0], 2 ** 31 - 1, -2 ** 31):
        p = pages.copy()
        p[0, 1] = wrong
        out, lse = api.kv4_attn(gq, cache, dev(p), dev(lens))
        torch.cuda.synchronize()
        assert api.cp_get_error() == _lib.CP_ECACHE and api.cp_get_error() == 0
        keep = [s for s in range(96) if s // 32 != 1]
        check_attn(out, lse, q, cache, pages, lens[:, None], 0.125, lambda b, j, h: keep if b == 0 else range(96))
        api.kv4_gather(cache, dev(p), dev(lens), 96)
        torch.cuda.synchronize()
        assert api.cp_get_error() == _lib.CP_ECACHE
        before = cache.clone()
        k = torch.ones(2, 1, 1, 64, device="cuda")
        api.kv4_append(k, k, cache, dev(p), dev(np.array([40, 40], np.int32)))
        torch.cuda.synchronize()
        assert api.cp_get_error() == _lib.CP_ECACHE
        changed = (before != cache).flatten(1).any(1).nonzero().flatten().tolist()
        assert changed == [int(pages[1, 1])]
        cache.copy_(before)
    for wrong, seen in ((-5, 0), (129, 128), (2 ** 31 - 1, 128)):
        gl = dev(np.array([wrong, 96], np.int32))
        full, _, fp = fill(np.random.default_rng(11), 2, 128, 1, 64, 32)
        out, lse = api.kv4_attn(gq, full, dev(fp[:, :4]), gl)
        torch.cuda.synchronize()
        assert api.cp_get_error() == _lib.CP_ECACHE
        check_attn(out, lse, q, full, fp, np.array([[seen], [96]]), 0.125)
        k = torch.ones(2, 1, 1, 64, device="cuda")
        before = full.clone()
        api.kv4_append(k, k, full, dev(fp[:, :4]), gl)
        torch.cuda.synchronize()
        assert api.cp_get_error() == _lib.CP_ECACHE
        changed = (before != full).flatten(1).any(1).nonzero().flatten().tolist()
        assert changed == [int(fp[1, 3])]


def test_append_position_outside_the_table(cuda_dev):
    cache = torch.zeros(2, 1, 16, 80, dtype=torch.uint8, device="cuda")
    pages, lens = dev(np.array([[0, 1]], np.int32)), dev(np.array([14], np.int32))
    k = torch.ones(1, 4, 1, 64, device="cuda")
    cos, sin = (dev(x) for x in rope(16, 64))
    q = api.kv4_append(k, k, cache, pages, lens, cos, sin, q=k)
    torch.cuda.synchronize()
    assert api.cp_get_error() == _lib.CP_ECACHE
    assert (cache[1] == 0).all() and (cache[0] != 0).any() and (q[0, 2:] == 0).all() and (q[0, :2] != 0).any()
    pos = dev(np.array([[0, -1, 15, 16]], np.int32))
    cache.zero_()
    q = api.kv4_append(k, k, cache, pages, lens, cos, sin, q=k, positions=pos)
    torch.cuda.synchronize()
    assert api.cp_get_error() == _lib.CP_ECACHE
    assert (q[0, [1, 3]] == 0).all() and (q[0, [0, 2]] != 0).any(-1).all()


@pytest.mark.parametrize("n,Hq,Hkv,D,page", [(1, 4, 2, 128, 16), (3, 8, 1, 64, 32), (2, 20, 1, 128, 64)])
def test_attn_selected_pages(cuda_dev, n, Hq, Hkv, D, page):
    rng = np.random.default_rng(n * 7)
    L = 5 * page + 9
    cache, _, pages = fill(rng, 2, L, Hkv, D, page)
    lens = np.array([L, 2 * page], np.int32)
    sel = np.full((2, n, Hkv, 5), -1, np.int32)
    for j in range(n):
        for h in range(Hkv):
            sel[0, j, h] = rng.permutation([0, 2, 5, 3, -1])
            sel[1, j, h] = [1, -1, -1, 0, 1] if j == 0 else -1        # page 1 twice; no page at all
    q = rows(rng, torch.bfloat16, 2, n, Hq, D)
    out, lse = api.kv4_attn(dev(q, torch.bfloat16), cache, dev(pages), dev(lens), sel=dev(sel))
    ok()
    lim = np.maximum(lens[:, None] - (n - 1) + np.arange(n), 0)

    def slots(b, j, h):
        return [p * page + t for p in sel[b, j, h] if p >= 0 for t in range(page)]
    check_attn(out, lse, q, cache, pages, lim, 1 / math.sqrt(D), slots)
    sel[1, 0, 0, 2] = 2                                               # behind the sequence
    sel[0, 0, 0, 0] = 2 ** 31 - 1
    keep = [p for p in sel[0, 0, 0, 1:] if p >= 0]
    out, lse = api.kv4_attn(dev(q, torch.bfloat16), cache, dev(pages), dev(lens), sel=dev(sel))
    torch.cuda.synchronize()
    assert api.cp_get_error() == _lib.CP_ECACHE
    sel[1, 0, 0, 2] = sel[0, 0, 0, 0] = -1
    check_attn(out, lse, q, cache, pages, lim, 1 / math.sqrt(D), slots)
    assert sorted(keep) == sorted(p for p in sel[0, 0, 0] if p >= 0)


SELECT = [  # pages that hold tokens, n, Hq, Hkv, D, page, n_sel, first, last
    ([1, 0, 3], 1, 2, 1, 64, 16, 4, 1, 1),
    ([40, 17], 1, 8, 2, 128, 64, 5, 1, 1),
    ([700, 300], 1, 4, 1, 64, 16, 64, 2, 3),
    ([60], 3, 24, 2, 128, 32, 7, 0, 0),
    ([1200], 1, 3, 3, 64, 128, 1, 0, 1),
]


@pytest.mark.parametrize("counts,n,Hq,Hkv,D,page,n_sel,first,last", SELECT)
@pytest.mark.parametrize("ties", [False, True])
def test_select(cuda_dev, counts, n, Hq, Hkv, D, page, n_sel, first, last, ties):
    """Small integers: every bound is exact in fp32, so the pages must be equal; with few different ones, ties."""
    rng = np.random.default_rng(len(counts) + n + ties)
    B, M = len(counts), max(counts) + 2
    pages, P = table(rng, B, M)
    lens = np.array([c * page - (c * 5) % page for c in counts], np.int32)
    box = rng.integers(-1 if ties else -60, 2 if ties else 61, (P, Hkv, 2, D)).astype(np.float32)
    box = np.sort(box, 2)
    if ties:
        box[:, :, :, 2:] = 0
    q = rng.integers(-8, 9, (B, n, Hq, D)).astype(np.float32)
    sel = api.kv4_select(dev(q, torch.bfloat16), dev(box, torch.bfloat16), dev(pages), dev(lens), page, n_sel,
                         keep_first=first, keep_last=last)
    ok()
    got = sel.cpu().numpy()
    for b in range(B):
        for j in range(n):
            lim = max(0, int(lens[b]) - (n - 1) + j)
            m = -(-lim // page)
            for h in range(Hkv):
                r = Hq // Hkv
                t = box[pages[b, :m], h]
                want = o.select(q[b, j, h * r:(h + 1) * r], t[:, 0], t[:, 1], n_sel, first, last)
                np.testing.assert_array_equal(got[b, j, h], want)


def test_select_scores_that_are_not_numbers_come_first(cuda_dev):
    rng = np.random.default_rng(4)
    box = rng.standard_normal((50, 1, 2, 64)).astype(np.float32)
    box[33, 0, :, 5] = math.nan
    box[20, 0, 0, 7], box[20, 0, 1, 7] = -math.inf, math.inf
    pages = np.arange(50, dtype=np.int32)[None]
    q = rows(rng, torch.bfloat16, 1, 1, 2, 64)
    sel = api.kv4_select(dev(q, torch.bfloat16), dev(box, torch.bfloat16), dev(pages), dev(np.array([800], np.int32)), 16,
                         4)
    ok()
    assert sel.flatten().tolist()[:1] == [0] and {20, 33, 49} < set(sel.flatten().tolist())


def test_prefill_then_decode_equals_ring_attention(cuda_dev):
    """A prompt through ring attention and into the cache; the next tokens over the
    cache against ring attention on the rows that the cache gives back."""
    rng = np.random.default_rng(12)
    S, new, Hq, Hkv, D, page = 512, 8, 8, 2, 128, 64
    cos, sin = (dev(x) for x in rope(S, D))
    q, k, v = (dev(rows(rng, torch.bfloat16, 1, S, h, D), torch.bfloat16) for h in (Hq, Hkv, Hkv))
    pages, P = table(rng, 1, S // page)
    cache, summ = api.kv4_cache(P, Hkv, page, D, summary=True)
    gp = dev(pages)
    L = S - new
    api.kv4_append(k[:, :L], v[:, :L], cache, gp, dev(np.array([0], np.int32)), cos, sin, summary=summ)
    qs = api.kv4_append(k[:, L:], v[:, L:], cache, gp, dev(np.array([L], np.int32)), cos, sin, q=q[:, L:], summary=summ)
    lens = dev(np.array([S], np.int32))
    kr, vr = api.kv4_gather(cache, gp, lens, S)
    qr = api.kv4_append(k, v, torch.empty_like(cache), gp, dev(np.array([0], np.int32)), cos, sin, q=q)
    assert torch.equal(qr[:, L:], qs)
    ref, rlse = api.ring_attn_fwd(qr, kr, vr, 4, inputs.ZIGZAG, True)
    out, lse = api.kv4_attn(qs, cache, gp, lens)
    every = api.kv4_select(qs, summ, gp, lens, page, S // page)
    out2, lse2 = api.kv4_attn(qs, cache, gp, lens, sel=every)
    ok()
    # the ring gets k and v rounded to bf16 (2^-8 relative each) and rounds its weights (2^-8)
    s = float(qr.float().abs().max() * kr.float().abs().max() * D / math.sqrt(D))
    assert (lse - rlse[..., L:]).abs().max() <= 1e-3 + 2.0 ** -8 * min(s, 8.0)
    for x in (out, out2):
        assert (x.float() - ref[:, L:].float()).abs().max() <= 2e-2
    assert (lse - lse2).abs().max() <= 1e-5
    # context-parallel: four ranks hold a quarter of the slots each; partials joined by log-sum-exp
    outs, lses = [], []
    for r in range(4):
        part, _ = api.kv4_cache(P, Hkv, page, D, summary=True)
        lo, hi = r * S // 4, (r + 1) * S // 4
        pos = torch.arange(lo, hi, dtype=I32, device="cuda")[None]
        zero = dev(np.array([0], np.int32))
        api.kv4_append(k[:, lo:hi], v[:, lo:hi], part, gp, zero, cos, sin, positions=pos)
        vis = (torch.arange(L, S, device="cuda", dtype=I32) + 1 - lo).clamp(0, S // 4)[None].contiguous()
        f32 = torch.empty(1, new, Hq, D, device="cuda")
        _, z = api.kv4_attn(qs, part, gp, zero + S // 4, vis=vis, out=f32)
        outs.append(f32.reshape(-1, D))
        lses.append(z.transpose(1, 2).reshape(-1))
    joined, jlse = api.lse_merge_n(torch.stack(outs), torch.stack(lses).contiguous())
    ok()
    assert (jlse.reshape(new, Hq).T - lse[0]).abs().max() <= 1e-5
    assert (joined.reshape(1, new, Hq, D) - out.float()).abs().max() <= 2.0 ** -8 * 4 + 4 * 2.0 ** -11 * 4


def test_streams_and_graph_replay(cuda_dev):
    """A decode step captured once and replayed as the cache grows, and the same on another stream."""
    rng = np.random.default_rng(13)
    B, Hq, Hkv, D, page, steps = 2, 4, 2, 64, 16, 40
    pages, P = table(rng, B, 4)
    k, v, q = (dev(rows(rng, torch.bfloat16, steps, B, 1, h, D), torch.bfloat16) for h in (Hkv, Hkv, Hq))
    cos, sin = (dev(x) for x in rope(64, D))

    def pools():
        return [x.zero_() for x in api.kv4_cache(P, Hkv, page, D, summary=True)] + [
            torch.tensor([0, 3], dtype=I32, device="cuda")]

    def step(pool, kk, vv, qq):
        cache, summ, lens = pool
        qr = api.kv4_append(kk, vv, cache, gp, lens, cos, sin, q=qq, summary=summ)
        lens += 1
        sel = api.kv4_select(qr, summ, gp, lens, page, 2)
        return api.kv4_attn(qr, cache, gp, lens) + api.kv4_attn(qr, cache, gp, lens, sel=sel)
    gp = dev(pages)
    eager = pools()
    want = [[t.clone() for t in step(eager, k[i], v[i], q[i])] for i in range(steps)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = pools()
        got = [[t.clone() for t in step(other, k[i], v[i], q[i])] for i in range(steps)]
    side.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    pool = pools()
    ik, iv, iq = k[0].clone(), v[0].clone(), q[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(pool, ik, iv, iq)
    fresh = pools()
    for x, y in zip(pool, fresh):
        x.copy_(y)
    for i in range(steps):
        ik.copy_(k[i]), iv.copy_(v[i]), iq.copy_(q[i])
        graph.replay()
        assert all(torch.equal(x, y) for x, y in zip(want[i], outs)), i
    ok()


def test_offsets_past_32_bits(cuda_dev):
    """A pool of more than 4 GiB, its tokens at the far end."""
    page, Hkv, D = 256, 8, 128
    per = Hkv * page * 160
    P = (1 << 32) // per + 40
    cache = torch.empty(P, Hkv, page, 160, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(14)
    pages = np.array([[P - 1, P - 3], [P - 20, 0]], np.int32)
    k, v = (rows(rng, torch.bfloat16, 2, 300, Hkv, D) for _ in range(2))
    zero = dev(np.zeros(2, np.int32))
    api.kv4_append(dev(k, torch.bfloat16), dev(v, torch.bfloat16), cache, dev(pages), zero)
    small, sp = torch.empty(4, Hkv, page, 160, dtype=torch.uint8, device="cuda"), np.array([[0, 1], [2, 3]], np.int32)
    api.kv4_append(dev(k, torch.bfloat16), dev(v, torch.bfloat16), small, dev(sp), zero)
    q = dev(rows(rng, torch.bfloat16, 2, 1, 16, D), torch.bfloat16)
    a, b = api.kv4_attn(q, cache, dev(pages), zero + 300), api.kv4_attn(q, small, dev(sp), zero + 300)
    c, d = api.kv4_gather(cache, dev(pages), zero + 300, 300), api.kv4_gather(small, dev(sp), zero + 300, 300)
    ok()
    for x, y in zip(a + c, b + d):
        assert torch.equal(x, y)


def test_attn_long_and_ragged_batches_cut_across_blocks(cuda_dev):
    """Lengths over four orders of magnitude in one batch: pieces of items in many blocks, joined.  Against the
    fp32 read-back in 64 bits on the GPU, with check_attn's bounds."""
    rng = np.random.default_rng(15)
    for D, Hq, Hkv, page, n, lens in ((128, 8, 2, 64, 1, [9000, 1, 0, 40, 3000, 17, 12345]),
                                      (64, 24, 2, 16, 2, [5, 20000, 33, 2])):
        B, L = len(lens), max(lens)
        cache, _, pages = fill(rng, B, L, Hkv, D, page)
        q = rows(rng, torch.bfloat16, B, n, Hq, D)
        gl = dev(np.array(lens, np.int32))
        kr, vr = api.kv4_gather(cache, dev(pages), gl, L, dtype=torch.float32)
        f32 = torch.empty(B, n, Hq, D, device="cuda")
        _, lse = api.kv4_attn(dev(q, torch.bfloat16), cache, dev(pages), gl, out=f32)
        ok()
        for b in range(B):
            for j in range(n):
                m = max(0, lens[b] - n + 1 + j)
                if not m:
                    assert (f32[b, j] == 0).all() and (lse[b, :, j] == -math.inf).all()
                    continue
                for x in range(Hq):
                    k, v = (t[b, :m, x * Hkv // Hq].double() for t in (kr, vr))
                    s = k @ torch.from_numpy(q[b, j, x]).double().cuda() / math.sqrt(D)
                    z = s.logsumexp(0)
                    p = (s - z).exp()
                    tol = (2.0 ** -10 + (m / 16 + 32) * 2.0 ** -23) * (p @ v.abs()) + m * 2.0 ** -25 * v.abs().max()
                    assert ((f32[b, j, x] - p @ v).abs() <= tol).all()
                    size = float(np.abs(q[b, j, x]) @ (k.abs().amax(0).cpu().numpy() + 8)) / math.sqrt(D)
                    assert abs(lse[b, x, j] - z) <= 2.0 ** -19 * size + 2.0 ** -20 * (abs(z) + 1)


def test_attn_value_that_is_not_a_number_is_not_lost_between_blocks(cuda_dev):
    """A whole block of tokens whose keys are NaN: every row that sees it is NaN, wherever the pieces are cut."""
    rng = np.random.default_rng(16)
    cache, _, pages = fill(rng, 1, 5000, 1, 128, 16)
    nan = torch.full((1, 16, 1, 128), math.nan, dtype=torch.bfloat16, device="cuda")
    q = dev(rows(rng, torch.bfloat16, 1, 1, 4, 128), torch.bfloat16)
    for at in (0, 16, 2048, 4976):
        trial = cache.clone()
        api.kv4_append(nan, nan, trial, dev(pages), dev(np.array([at], np.int32)))
        out, lse = api.kv4_attn(q, trial, dev(pages), dev(np.array([5000], np.int32)))
        ok()
        assert out.isnan().all() and lse.isnan().all()



def reference(q, kr, vr, limits, scale):
    """q [B, n, Hq, D], kr and vr [B, L, Hkv, D] fp32, limits [B, n]: out, lse and sum p |v| in 64 bits."""
    B, n, Hq, D = q.shape
    L, Hkv = kr.shape[1:3]
    k, v = (t.double().repeat_interleave(Hq // Hkv, 2) for t in (kr, vr))
    s = torch.einsum("bnhd,blhd->bhnl", q.double(), k) * scale
    s = s.masked_fill(torch.arange(L, device=q.device) >= limits.to(q.device)[:, None, :, None], -math.inf)
    z = s.logsumexp(-1)
    p = torch.exp(s - z.masked_fill(z == -math.inf, 0.0)[..., None])
    return torch.einsum("bhnl,blhd->bnhd", p, v), z, torch.einsum("bhnl,blhd->bnhd", p, v.abs())


def check_reference(out, lse, q, kr, vr, limits, scale):
    """The bounds of check_attn, for whole batches."""
    want, z, a = reference(q, kr, vr, limits, scale)
    L = kr.shape[1]
    tol = (2.0 ** -10 + (L / 16 + 32) * 2.0 ** -23) * a + L * 2.0 ** -25 * vr.abs().max().double() + 2.0 ** -25
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    assert ((out.double() - want).abs() <= tol).all()
    empty = z == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    size = scale * q.double().abs().sum(-1).amax() * (kr.abs().amax() + 8).double()
    assert ((lse.double() - z).masked_fill(empty, 0.0).abs()
            <= 2.0 ** -19 * size + 2.0 ** -20 * (z.masked_fill(empty, 0.0).abs() + 1)).all()


@pytest.mark.parametrize("B,n,Hq,Hkv,D,page,L", [(70, 1, 4, 2, 64, 16, 300), (300, 1, 2, 1, 128, 32, 90),
                                                 (1, 200, 8, 2, 64, 64, 700), (3, 33, 10, 5, 128, 16, 150),
                                                 (2, 1, 128, 1, 128, 64, 900)])
def test_attn_many_sequences_many_rows(cuda_dev, B, n, Hq, Hkv, D, page, L):
    rng = np.random.default_rng(B + n)
    lens = rng.integers(0, L + 1, B).astype(np.int32)
    lens[-1] = L
    if B > 40:
        lens[35:40] = 0
    M = -(-L // page)
    pages, P = table(rng, B, M)
    cache = torch.full((P, Hkv, page, D // 4 * 5), 255, dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(n)
    k, v = (torch.randn(B, L, Hkv, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    api.kv4_append(k, v, cache, dev(pages), dev(np.zeros(B, np.int32)), n_new=dev(lens))
    q = torch.randn(B, n, Hq, D, generator=g, device="cuda").bfloat16()
    out, lse = api.kv4_attn(q, cache, dev(pages), dev(lens))
    kr, vr = api.kv4_gather(cache, dev(pages), dev(lens), L, dtype=torch.float32)
    ok()
    lim = torch.from_numpy(np.maximum(lens[:, None] - (n - 1) + np.arange(n), 0))
    check_reference(out, lse, q, kr, vr, lim, 1 / math.sqrt(D))


@pytest.mark.parametrize("B,Hkv,pages_of_64,n", [(1, 1, 11, 2), (1, 1, 13, 2), (19, 4, 30, 2), (19, 4, 33, 2), (160, 1, 2, 2),
                                                 (40, 4, 16, 2), (40, 4, 17, 2), (50, 4, 9, 5), (90, 4, 3, 5), (230, 2, 3, 1)])
def test_attn_on_both_sides_of_a_block_per_item(cuda_dev, B, Hkv, pages_of_64, n):
    """Table sizes and item counts around the choice between a block per item and stretches, ragged lengths in both;
    a bounded wait in a block that joins in shared memory."""
    L = pages_of_64 * 64
    rng = np.random.default_rng(L)
    lens = rng.integers(0, L + 1, B).astype(np.int32)
    lens[0] = L
    pages, P = table(rng, B, pages_of_64)
    cache = torch.full((P, Hkv, 64, 160), 255, dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(L)
    k, v = (torch.randn(B, L, Hkv, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
    api.kv4_append(k, v, cache, dev(pages), dev(np.zeros(B, np.int32)), n_new=dev(lens))
    q = torch.randn(B, n, 3 * Hkv, 128, generator=g, device="cuda").bfloat16()
    out, lse = api.kv4_attn(q, cache, dev(pages), dev(lens))
    kr, vr = api.kv4_gather(cache, dev(pages), dev(lens), L, dtype=torch.float32)
    ok()
    lim = torch.from_numpy(np.maximum(lens[:, None] - (n - 1) + np.arange(n), 0))
    check_reference(out, lse, q, kr, vr, lim, 1 / math.sqrt(128))
    try:
        api.cp_debug_set_wait_limit(1)
        api.kv4_attn(q, cache, dev(pages), dev(lens))
        torch.cuda.synchronize()
        assert api.cp_get_error() == _lib.CP_ETIMEOUT
    finally:
        api.cp_debug_set_wait_limit(0)
    again, _ = api.kv4_attn(q, cache, dev(pages), dev(lens))
    ok()
    assert torch.equal(out, again)


def test_attn_sizes_of_scores_and_queries(cuda_dev):
    """Queries from 2^-100 to 2^40 in one tile, rows of zeros, keys of 2^-10 to 2^8: each row scaled by itself."""
    rng = np.random.default_rng(19)
    D, L = 128, 200
    pages, P = table(rng, 1, 4)
    cache = torch.full((P, 1, 64, 160), 255, dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(1, L, 1, D, generator=g, device="cuda") for _ in range(2))
    k *= torch.exp2(torch.randint(-10, 9, (1, L, 1, 1), generator=g, device="cuda").float())
    lens = dev(np.array([L], np.int32))
    api.kv4_append(k, v, cache, dev(pages), lens - L)
    q = torch.randn(1, 1, 8, D, generator=g, device="cuda")
    for i, e in enumerate((-100, -30, -8, 0, 3, 20, 40)):
        q[0, 0, i] *= 2.0 ** e
    q[0, 0, 7] = 0
    q = q.bfloat16()
    out, lse = api.kv4_attn(q, cache, dev(pages), lens)
    kr, vr = api.kv4_gather(cache, dev(pages), lens, L, dtype=torch.float32)
    ok()
    for i in range(8):   # by row: the bound of lse is relative to the row's own scores
        check_reference(out[:, :, i:i + 1], lse[:, i:i + 1], q[:, :, i:i + 1], kr, vr, torch.tensor([[L]]), 1 / math.sqrt(D))


def test_attn_query_rows_that_are_not_finite(cuda_dev):
    """A row of q with an infinity, a NaN or a magnitude beyond 2^110 is NaN; the other rows of its tile are what they were."""
    rng = np.random.default_rng(25)
    cache, _, pages = fill(rng, 1, 300, 1, 128, 64)
    q = dev(rows(rng, torch.bfloat16, 1, 1, 8, 128), torch.bfloat16)
    lens = dev(np.array([300], np.int32))
    want, wlse = api.kv4_attn(q, cache, dev(pages), lens)
    bad = q.clone()
    bad[0, 0, 1, 5], bad[0, 0, 4, 100], bad[0, 0, 6] = math.inf, math.nan, 2.0 ** 112
    out, lse = api.kv4_attn(bad, cache, dev(pages), lens)
    ok()
    for i in range(8):
        if i in (1, 4, 6):
            assert out[0, 0, i].isnan().all() and lse[0, i].isnan().all()
        else:
            assert torch.equal(out[0, 0, i], want[0, 0, i]) and torch.equal(lse[0, i], wlse[0, i])


def test_append_rotates_q_in_place(cuda_dev):
    rng = np.random.default_rng(20)
    cos, sin = (dev(x) for x in rope(64, 128))
    pages, lens = dev(np.array([[0]], np.int32)), dev(np.array([3], np.int32))
    q, k = (dev(rows(rng, torch.bfloat16, 1, 20, h, 128), torch.bfloat16) for h in (12, 1))
    cache = api.kv4_cache(1, 1, 64, 128)
    want = api.kv4_append(k, k, cache, pages, lens, cos, sin, q=q)
    got = api.kv4_append(k, k, cache, pages, lens, cos, sin, q=q, q_out=q)
    ok()
    assert got is q and torch.equal(got, want)


@pytest.mark.parametrize("count,n_sel", [(1030, 100), (2100, 64), (9000, 333), (70000, 50)])
def test_select_over_many_pages(cuda_dev, count, n_sel):
    """Every number of keys per thread, ties among them; small integers, so that every bound is exact."""
    rng = np.random.default_rng(count)
    box = np.sort(rng.integers(-40, 41, (count, 1, 2, 64)).astype(np.float32), 2)
    box[rng.integers(0, count, count // 3)] = box[7]
    pages = rng.permutation(count).astype(np.int32)[None]
    q = rng.integers(-8, 9, (1, 1, 3, 64)).astype(np.float32)
    sel = api.kv4_select(dev(q, torch.bfloat16), dev(box, torch.bfloat16), dev(pages),
                         dev(np.array([count * 16 - 3], np.int32)), 16, n_sel)
    ok()
    t = box[pages[0], 0]
    np.testing.assert_array_equal(sel.cpu().numpy()[0, 0, 0], o.select(q[0, 0], t[:, 0], t[:, 1], n_sel, 1, 1))


def test_select_reports_bad_pages_and_lengths(cuda_dev):
    rng = np.random.default_rng(21)
    box = dev(np.sort(rng.standard_normal((20, 1, 2, 64)), 2).astype(np.float32), torch.bfloat16)
    q = dev(rows(rng, torch.bfloat16, 1, 1, 2, 64), torch.bfloat16)
    pages = np.arange(20, dtype=np.int32)[None].copy()
    pages[0, 5] = 20
    sel = api.kv4_select(q, box, dev(pages), dev(np.array([320], np.int32)), 16, 4)
    torch.cuda.synchronize()
    assert api.cp_get_error() == _lib.CP_ECACHE
    assert ((sel >= 0) & (sel < 20)).all()
    pages[0, 5] = 5
    for length in (-1, 2 ** 31 - 1):
        sel = api.kv4_select(q, box, dev(pages), dev(np.array([length], np.int32)), 16, 4)
        torch.cuda.synchronize()
        assert api.cp_get_error() == _lib.CP_ECACHE
        assert (sel < 20).all()


def test_calls_on_two_streams_and_two_graphs_at_once(cuda_dev):
    """Calls that overlap have workspaces of their own (each call takes one, a captured one its graph's)."""
    rng = np.random.default_rng(22)
    work = []
    for i in range(2):
        cache, summ, pages = fill(rng, 3, 3000, 2, 128, 64)
        q = dev(rows(rng, torch.bfloat16, 3, 1, 8, 128), torch.bfloat16)
        lens = dev(np.array([3000, 17, 1234], np.int32))

        def step(q=q, cache=cache, summ=summ, pages=dev(pages), lens=lens):
            sel = api.kv4_select(q, summ, pages, lens, 64, 5)
            return [sel, *api.kv4_attn(q, cache, pages, lens), *api.kv4_attn(q, cache, pages, lens, sel=sel)]
        work.append((step, [t.clone() for t in step()]))
    ok()
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs = []
    for (step, _), s in zip(work, streams):
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs = step()
        graphs.append((graph, outs))
    for _ in range(20):
        got = []
        for (step, _), s in zip(work, streams):
            with torch.cuda.stream(s):
                got.append(step())
        torch.cuda.synchronize()
        for (_, want), g in zip(work, got):
            assert all(torch.equal(x, y) for x, y in zip(want, g))
        for (graph, outs), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for (_, want), (_, outs) in zip(work, graphs):
            assert all(torch.equal(x, y) for x, y in zip(want, outs))
    ok()


def test_stream_argument(cuda_dev):
    """Every call on a stream that is not the current one."""
    rng = np.random.default_rng(23)
    cache, summ, pages = fill(rng, 1, 500, 1, 64, 32)
    q = dev(rows(rng, torch.bfloat16, 1, 1, 4, 64), torch.bfloat16)
    lens, gp = dev(np.array([500], np.int32)), dev(pages)
    k = dev(rows(rng, torch.bfloat16, 1, 1, 1, 64), torch.bfloat16)

    def step(cache, summ, stream):
        qr = api.kv4_append(k, k, cache, gp, lens, q=q, summary=summ, stream=stream)
        sel = api.kv4_select(qr, summ, gp, lens, 32, 3, stream=stream)
        return [sel, *api.kv4_attn(qr, cache, gp, lens, sel=sel, stream=stream),
                *api.kv4_gather(cache, gp, lens, 501, stream=stream)]
    want = step(cache.clone(), summ.clone(), None)
    ok()
    side = torch.cuda.Stream()
    c, s = cache.clone(), summ.clone()
    side.wait_stream(torch.cuda.current_stream())
    got = step(c, s, side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_binding_refusals_on_the_gpu(cuda_dev):
    D = 64
    cache, summ = api.kv4_cache(4, 2, 16, D, summary=True)
    pages, lens = dev(np.array([[0, 1]], np.int32)), dev(np.array([3], np.int32))
    k = torch.zeros(1, 2, 2, D, device="cuda")
    q = torch.zeros(1, 1, 4, D, dtype=torch.bfloat16, device="cuda")
    bad = [
        lambda: api.kv4_append(k, k, cache, pages, lens.long()),
        lambda: api.kv4_append(k, k, cache, pages.cpu(), lens),
        lambda: api.kv4_append(k, k, cache, pages[0], lens),
        lambda: api.kv4_append(k[:, :, :1], k[:, :, :1], cache, pages, lens),
        lambda: api.kv4_append(k, k.bfloat16(), cache, pages, lens),
        lambda: api.kv4_append(k.transpose(2, 3), k.transpose(2, 3), cache, pages, lens),
        lambda: api.kv4_append(k.transpose(2, 3).contiguous().transpose(2, 3), k, cache, pages, lens),
        lambda: api.kv4_append(k, k, cache, pages, lens, cos=torch.zeros(5, 32, device="cuda")),
        lambda: api.kv4_append(k, k, cache, pages, lens, n_new=dev(np.zeros(2, np.int32))),
        lambda: api.kv4_append(k, k, cache, pages, lens, positions=dev(np.zeros((1, 3), np.int32))),
        lambda: api.kv4_append(k, k, cache, pages, lens, q_out=k),
        lambda: api.kv4_append(k, k, cache, pages, lens, summary=summ[:2]),
        lambda: api.kv4_gather(cache, pages, lens, 4, start=lens.float()),
        lambda: api.kv4_gather(cache, pages, lens, 4, k=k),
        lambda: api.kv4_attn(q.float(), cache, pages, lens),
        lambda: api.kv4_attn(q[..., :32], cache, pages, lens),
        lambda: api.kv4_attn(q, cache[:, :, ::2], pages, lens),
        lambda: api.kv4_attn(q, cache, pages, lens, vis=dev(np.zeros((1, 2), np.int32))),
        lambda: api.kv4_attn(q, cache, pages, lens, sel=dev(np.zeros((1, 1, 1, 2), np.int32))),
        lambda: api.kv4_attn(q, cache, pages, lens, out=q.half()),
        lambda: api.kv4_attn(q, cache, pages, lens, lse=torch.zeros(1, 1, 4, device="cuda")),
        lambda: api.kv4_attn(q, cache, pages, lens, workspace=torch.empty(64, dtype=torch.uint8, device="cuda")),
        lambda: api.kv4_attn(q[:, :, :3].contiguous(), cache, pages, lens),
        lambda: api.kv4_select(q, summ, pages, lens, 16, 0),
        lambda: api.kv4_select(q, summ, pages, lens, 16, 2, keep_first=2, keep_last=1),
        lambda: api.kv4_select(q, summ, pages, lens, 24, 2),
        lambda: api.kv4_select(q, summ, pages, lens, 16, 2, sel=dev(np.zeros((1, 1, 2, 3), np.int32))),
    ]
    before = cache.clone()
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, _lib.CpError)):
            call()
            raise AssertionError(i)
    ok()
    assert torch.equal(before, cache)
    for call, error in ((lambda: api.kv4_gather(cache, pages, lens, "4"), TypeError),
                        (lambda: api.kv4_gather(cache, pages, lens, 1 << 40), ValueError),
                        (lambda: api.kv4_gather(cache, pages, lens, -1), _lib.CpError),
                        (lambda: api.kv4_attn(q, cache, pages, lens, scale="x"), TypeError),
                        (lambda: api.kv4_attn(q, cache, pages, lens, vis=3), ValueError),
                        (lambda: api.kv4_attn(q, cache, pages, None), ValueError),
                        (lambda: api.kv4_select(q, summ, pages, lens, 16, 1 << 33), ValueError)):
        with pytest.raises(error):
            call()
    # rows that do not start on 16 bytes
    x = torch.zeros(1, 2, 2 * D + 2, device="cuda", dtype=torch.bfloat16)[..., :2 * D].unflatten(-1, (2, D))
    with pytest.raises(_lib.CpError):
        api.kv4_append(x, x, cache, pages, lens)
    # nothing to do
    assert api.kv4_append(k[:, :0], k[:, :0], cache, pages, lens) is None
    out, lse = api.kv4_attn(q[:0], cache, pages[:0], lens[:0])
    assert out.shape == (0, 1, 4, D) and lse.shape == (0, 4, 1)
    gk, _ = api.kv4_gather(cache, pages, lens, 0)
    assert gk.shape == (1, 0, 2, D)
    out, lse = api.kv4_attn(q, cache, pages[:, :0].contiguous(), lens * 0)      # no pages at all
    ok()
    assert (out == 0).all() and lse.isinf().all()


def test_attn_bounded_wait(cuda_dev):
    """A wait that runs out ends the kernel with CP_ETIMEOUT, its copies landed; the next call is whole again."""
    rng = np.random.default_rng(17)
    cache, _, pages = fill(rng, 2, 9000, 2, 128, 64)
    q = dev(rows(rng, torch.bfloat16, 2, 1, 8, 128), torch.bfloat16)
    lens = dev(np.array([9000, 9000], np.int32))
    want = api.kv4_attn(q, cache, dev(pages), lens)
    ok()
    try:
        api.cp_debug_set_wait_limit(1)
        api.kv4_attn(q, cache, dev(pages), lens)
        torch.cuda.synchronize()
        assert api.cp_get_error() == _lib.CP_ETIMEOUT
    finally:
        api.cp_debug_set_wait_limit(0)
    got = api.kv4_attn(q, cache, dev(pages), lens)
    ok()
    assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_capture_behind_memsets_copies_and_joined_streams(cuda_dev):
    """The calls captured behind nodes of every kind: a kernel, a memset, a copy, two streams at once, nothing."""
    rng = np.random.default_rng(24)
    cache, summ, pages = fill(rng, 2, 700, 1, 64, 16)
    q, k = (dev(rows(rng, torch.bfloat16, 2, 1, h, 64), torch.bfloat16) for h in (3, 1))
    gp, lens = dev(pages), dev(np.array([650, 321], np.int32))

    def call(q):
        qr = api.kv4_append(k, k, cache, gp, lens, q=q, summary=summ)
        sel = api.kv4_select(qr, summ, gp, lens, 16, 4)
        return [qr, sel, *api.kv4_attn(qr, cache, gp, lens, sel=sel), *api.kv4_gather(cache, gp, lens, 60)]
    want = [t.clone() for t in call(q)]
    ok()
    src, buf, side = q.clone(), torch.empty_like(q), torch.cuda.Stream()
    for kind in ("nothing", "kernel", "memset", "copy", "streams"):
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            x = src
            if kind == "kernel":
                x = src + 0
            if kind == "memset":
                torch.zeros(1 << 16, device="cuda")
            if kind == "copy":
                buf.copy_(src)
                x = buf
            if kind == "streams":
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    buf.copy_(src * 1)
                y = src * 1
                torch.cuda.current_stream().wait_stream(side)
                x = buf
            outs = call(x)
            if kind == "streams":
                outs.append(y)
        for _ in range(3):
            buf.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(g, w) for g, w in zip(outs, want)), kind
    ok()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D,page,inter", [(64, 16, False), (128, 64, True)])
def test_page_ranges_bound_the_scores(cuda_dev, D, page, inter, dtype):
    """The largest q.k that a page's range allows, against the keys that attention reads: they pass it at most by the
    bf16 rounding of the range (2^-8 of an element's extremes) and by the quantisation of the key (half a step; the scale's
    rounding, 15 codes of 2^-11 of it; the minimum's, 2^-11 of it; below fp16's normal range 2^-25 in place of 2^-11)."""
    rng = np.random.default_rng(26)
    L, H, rot = 5 * page, 2, D
    pages, P = table(rng, 1, 5)
    k = rng.standard_normal((1, L, H, D)) * np.exp2(rng.integers(-6, 7, (1, L, H, 1))) + rng.standard_normal((1, 1, H, D)) * 8
    k = k.astype(np.float32)
    k = o.bf16(k) if dtype == torch.bfloat16 else k
    cos, sin = rope(L, rot)
    cache, summ = api.kv4_cache(P, H, page, D, summary=True)
    zero = dev(np.array([0], np.int32))
    api.kv4_append(dev(k, dtype), dev(k, dtype), cache, dev(pages), zero, dev(cos), dev(sin), summary=summ, interleaved=inter)
    kr, _ = api.kv4_gather(cache, dev(pages), zero + L, L, dtype=torch.float32)
    ok()
    turned = o.rotate(k[0], cos[:, None], sin[:, None], inter)                           # [L, H, D] fp32, as the append has it
    _, s, m = (x.astype(np.float64) for x in o.quantise(turned))
    slack = s * (0.5 + 15 * 2.0 ** -11) + 2.0 ** -11 * np.abs(m) + 16 * 2.0 ** -25 + 2.0 ** -22 * np.abs(turned)
    q = rng.standard_normal((200, D))
    box = summ.double().cpu().numpy()[pages[0]]                                            # [5, H, 2, D]
    read = kr[0].double().cpu().numpy().reshape(5, page, H, D)
    slack, turned = slack.reshape(5, page, H, D), turned.astype(np.float64).reshape(5, page, H, D)
    for p in range(5):
        for h in range(H):
            lo, hi = box[p, h]
            bound = np.maximum(q * lo, q * hi).sum(-1)                                     # [200]
            edge = np.abs(q) @ (2.0 ** -8 * np.maximum(np.abs(lo), np.abs(hi)))
            assert (q @ turned[p, :, h].T <= (bound + edge)[:, None]).all()
            assert (q @ read[p, :, h].T <= (bound + edge)[:, None] + np.abs(q) @ slack[p, :, h].T).all()
