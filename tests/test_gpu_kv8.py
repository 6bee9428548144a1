"""The paged 8-bit cache on the GPU, against the plain statement in oracle/kv8.py: appended, read back, moved and
selected bit for bit, attention within the bounds that attend() counts from its roundings."""
import math
import threading

import numpy as np
import pytest
import torch

from context_parallelism_02_gb300 import _lib, api
from oracle import kv8 as o
from oracle import window as ow

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")
BF16, F32 = torch.bfloat16, torch.float32


def ok():
    torch.cuda.synchronize()
    assert api.cp_get_error() == 0


def table(g, B, M, spare=3):
    P = B * M + spare
    return torch.randperm(P, generator=g, device="cuda")[:B * M].reshape(B, M).int(), P


def pool(seed, B, L, Hkv, D, page, width=None, junk=True):
    """Sequences of L tokens, appended; what is not written holds NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    M = -(-L // page)
    used, P = table(g, B, M)
    cache, scales = api.kv8_cache(P, Hkv, page, D)
    cache.fill_(0x7f if junk else 0)
    scales.fill_(math.nan if junk else 0)
    pages = torch.full((B, width or M), -1, **I32)
    pages[:, :M] = used
    k, v = (torch.randn(B, L, Hkv, D, generator=g, device="cuda") * torch.exp(torch.randn(B, L, 1, 1, generator=g, device="cuda"))
            for _ in range(2))
    api.kv8_append(k.bfloat16(), v.bfloat16(), cache, scales, pages, torch.zeros(B, **I32))
    return cache, scales, pages, g


def same_codes(a, b):
    """Equal bytes, any NaN for a NaN."""
    nan = ((a & 0x7f) == 0x7f) & ((b & 0x7f) == 0x7f)
    assert ((a == b) | nan).all()


APPEND = [  # B, n, Hkv, D, page, dtype, strided, ragged
    (1, 1, 2, 128, 64, BF16, False, False),
    (3, 1, 1, 64, 16, BF16, True, True),
    (5, 16, 2, 128, 16, F32, False, False),
    (2, 37, 2, 128, 16, F32, True, True),
    (2, 150, 3, 64, 32, BF16, True, False),
    (1, 300, 2, 64, 128, F32, False, False),
    (4, 70, 1, 128, 256, BF16, False, True),
]


@pytest.mark.parametrize("B,n,H,D,page,dtype,strided,ragged", APPEND)
def test_append_bytes(cuda_dev, B, n, H, D, page, dtype, strided, ragged):
    rng = np.random.default_rng(B * 1000 + n)
    g = torch.Generator(device="cuda").manual_seed(n)
    lens = np.array([(17 * b * b + 5 * b) % 90 if B > 1 else 41 for b in range(B)], np.int32)
    n_new = np.array([(n - 7 * b) % (n + 1) for b in range(B)], np.int32) if ragged else None
    pages, P = table(g, B, (int(lens.max()) + n + page - 1) // page)
    cache = rng.integers(0, 127, (P, H, 2, page, D), dtype=np.uint8) | (rng.integers(0, 2, (P, H, 2, page, D), dtype=np.uint8) << 7)
    scales = (2.0 ** rng.integers(-8, 2, (P, H, 2, page // 16))).astype(np.float32)
    # rows of several sizes: blocks whose scale grows, stays, and codes below the normal range
    x = torch.randn(B, n, 3, H, D, generator=g, device="cuda") * torch.exp(3 * torch.randn(B, n, 1, 1, 1, generator=g, device="cuda"))
    x = x.to(dtype)
    k, v = (x[:, :, 0], x[:, :, 2]) if strided else (x[:, :, 0].contiguous(), x[:, :, 2].contiguous())
    gc, gs = torch.from_numpy(cache).cuda(), torch.from_numpy(scales).cuda()
    api.kv8_append(k, v, gc, gs, pages, torch.from_numpy(lens).cuda(), n_new=None if n_new is None else torch.from_numpy(n_new).cuda())
    ok()
    o.append(cache, scales, pages.cpu().numpy(), lens, k.double().cpu().numpy(), v.double().cpu().numpy(), n_new)
    np.testing.assert_array_equal(gs.cpu().numpy(), scales)
    same_codes(gc.cpu().numpy(), cache)


def test_append_one_by_one_equals_at_once(cuda_dev):
    """Values of one power of ten: no code leaves the normal range when a scale grows, so how tokens came does not show."""
    g = torch.Generator(device="cuda").manual_seed(5)
    B, n, H, D, page = 2, 45, 2, 128, 16
    pages, P = table(g, B, 4)
    k, v = ((torch.rand(B, n, H, D, generator=g, device="cuda") + 0.1) * (1 - 2 * (torch.rand(B, n, H, D, generator=g, device="cuda") < 0.5)
                                                                          .float()) for _ in range(2))
    pools = [(torch.zeros(P, H, 2, page, D, dtype=torch.uint8, device="cuda"), torch.zeros(P, H, 2, page // 16, device="cuda")) for _ in range(2)]
    lens = torch.tensor([0, 16], **I32)
    api.kv8_append(k, v, *pools[0], pages, lens)
    for j in range(n):
        api.kv8_append(k[:, j:j + 1], v[:, j:j + 1], *pools[1], pages, lens + j)
    ok()
    assert all(torch.equal(x, y) for x, y in zip(*pools))


def test_values_that_are_not_finite_too_large_or_too_small(cuda_dev):
    D, page, n = 64, 16, 64
    k = torch.zeros(1, n, 1, D, device="cuda")
    k[0, 3, 0, 5], k[0, 4, 0, 6], k[0, 5, 0, 7], k[0, 6, 0, 8] = math.nan, math.inf, -math.inf, 3.0
    k[0, 16:32] = torch.linspace(-3e38, 3e38, D, device="cuda")          # beyond 448 2^60
    k[0, 32:48, 0, :] = 1e-30                                            # below the smallest scale's codes
    # the last block: all zero
    v = k.flip(1).contiguous()
    cache, scales = api.kv8_cache(4, 1, page, D)
    pages, lens = torch.arange(4, **I32)[None], torch.zeros(1, **I32)
    api.kv8_append(k, v, cache, scales, pages, lens)
    gk, gv = api.kv8_gather(cache, scales, pages, lens + n, n, dtype=F32)
    ok()
    c, s = np.zeros(cache.shape, np.uint8), np.zeros(scales.shape, np.float32)
    o.append(c, s, pages.cpu().numpy(), [0], k.double().cpu().numpy(), v.double().cpu().numpy())
    np.testing.assert_array_equal(scales.cpu().numpy(), s)
    same_codes(cache.cpu().numpy(), c)
    want_k, want_v = o.read(c, s, pages.cpu().numpy(), 0, 0, range(n))
    np.testing.assert_array_equal(gk[0, :, 0].double().cpu().numpy(), want_k)
    np.testing.assert_array_equal(gv[0, :, 0].double().cpu().numpy(), want_v)
    assert gk[0, 3, 0, 5].isnan() and gk[0, 4, 0, 6].isnan() and gk[0, 6, 0, 8] == 3
    # (the linspace overflows to values that are not finite; these are not)
    big = torch.full((1, 16, 1, D), 3e38, device="cuda")
    api.kv8_append(big, -big, cache, scales, pages, lens)
    gk, gv = api.kv8_gather(cache, scales, pages, lens + 16, 16, dtype=F32)
    ok()
    assert (gk == 448 * 2.0 ** 60).all() and (gv == -448 * 2.0 ** 60).all() and (scales[0] == 2.0 ** 60).all()


def test_gather_ranges(cuda_dev):
    B, L, H, D, page = 3, 200, 2, 128, 32
    cache, scales, pages, g = pool(1, B, L, H, D, page)
    lens = torch.tensor([200, 97, 0], **I32)
    start = torch.tensor([150, 0, 5], **I32)
    for dtype in (BF16, F32):
        k, v = api.kv8_gather(cache, scales, pages, lens, 77, start=start, dtype=dtype)
        ok()
        for b in range(B):
            m = max(0, min(77, int(lens[b] - start[b])))
            for h in range(H):
                want = o.read(cache.cpu().numpy(), scales.cpu().numpy(), pages.cpu().numpy(), b, h, range(int(start[b]), int(start[b]) + m))
                for x, y in zip((k, v), want):
                    np.testing.assert_array_equal(x[b, :m, h].double().cpu().numpy(), y)
                    assert (x[b, m:, h] == 0).all()


def check_attn(q, cache, scales, pages, lens, out, lse, limits, window, sinks, scale=None, mass=None, rows=None, wide=False):
    """Every row (b, j, head) against the cache's values; limits [B][n]."""
    c, s, t = cache.cpu().numpy(), scales.cpu().numpy(), pages.cpu().numpy()
    B, n, Hq, D = q.shape
    H = cache.shape[1]
    scale = scale or D ** -0.5
    unit = 2.0 ** -24 if out.dtype == F32 else 2.0 ** -8
    weights = {}
    for b in range(B):
        for h in range(H):
            kk, vv = o.read(c, s, t, b, h, range(int(lens[b])))
            sl = np.arange(int(lens[b]))
            vs = s[t[b, sl // cache.shape[3]], h, 1, sl % cache.shape[3] // 16].astype(np.float64)
            for j in range(n):
                at = o.sees(min(max(int(limits[b][j]), 0), int(lens[b])), window, sinks)
                for x in range(h * Hq // H, (h + 1) * Hq // H):
                    ref, z, p, err, ez = o.attend(q[b, j, x].double().cpu().numpy(), kk[at], vv[at], vs[at], scale)
                    got = out[b, j, x].double().cpu().numpy()
                    if not len(at):
                        assert (got == 0).all() and lse[b, x, j] == -math.inf
                        continue
                    d = np.abs(got - ref) - (err + unit * np.abs(ref) + unit * err)
                    assert d.max() <= 0, (b, j, x, d.max(), len(at))
                    assert abs(lse[b, x, j].item() - z) <= ez, (b, j, x)
                    w = weights.setdefault((b, h), [np.zeros(int(lens[b])), np.zeros(int(lens[b])), np.zeros(int(lens[b]), bool)])
                    w[0][at] += p
                    w[1][at] += p * 4 * ez
                    w[2][at] = True
    if mass is not None:
        before, after = mass
        for b in range(B):
            for h in range(H):
                want = before[b, h].double().cpu().numpy()
                err = np.abs(want) * 2.0 ** -23
                touched = np.zeros(len(want), bool)
                if (b, h) in weights:
                    w = weights[b, h]
                    m = len(w[0])
                    want[:m] += w[0]
                    err[:m] += w[1] + (np.abs(want[:m]) + w[0]) * 2.0 ** -22
                    touched[:m] = w[2]
                got = after[b, h].double().cpu().numpy()
                assert (np.abs(got - want) <= err)[touched].all()
                assert np.array_equal(got[~touched], before[b, h].double().cpu().numpy()[~touched])


ATTN = [  # lens, n, Hq, Hkv, D, page, window, sinks, mass, fp32 out
    ([1], 1, 1, 1, 64, 16, 0, 0, True, False),
    ([15, 16, 17], 1, 4, 2, 128, 16, 0, 0, True, False),
    ([500], 1, 8, 2, 128, 64, 0, 0, False, True),
    ([700, 3, 0, 64], 1, 8, 8, 64, 32, 0, 0, True, False),
    ([2000, 1999], 3, 6, 2, 128, 128, 0, 0, True, False),
    ([300, 33], 5, 16, 2, 64, 16, 0, 0, True, True),          # 40 rows: three tiles
    ([257], 2, 17, 1, 128, 256, 0, 0, True, False),           # 34 rows of one kv head
    ([9000], 1, 4, 1, 128, 64, 0, 0, True, False),            # stretches and the join
    ([6000, 50, 4100], 1, 8, 4, 64, 16, 0, 0, False, False),
    ([2500, 40], 1, 4, 2, 128, 16, 100, 4, True, False),      # windows: blocks are skipped between
    ([2500, 40, 5], 4, 4, 2, 128, 64, 33, 20, True, True),
    ([5000] * 3, 1, 8, 8, 128, 32, 1024, 0, False, False),
    ([1000], 3, 2, 1, 64, 16, 1, 0, True, False),
    ([1000], 3, 2, 1, 64, 16, 1, 64, True, False),
    ([300], 2, 4, 4, 64, 16, 290, 64, True, False),           # window and sinks meet
    ([3000, 700], 1, 4, 4, 128, 64, 5000, 4, False, False),   # a window beyond the context
    ([400] * 40, 1, 8, 4, 64, 16, 0, 0, True, False),         # more items than SMs
    ([512, 1, 300] * 20, 1, 16, 8, 128, 16, 0, 0, True, False),   # more than run at once, of a short table
]


@pytest.mark.parametrize("lens,n,Hq,H,D,page,window,sinks,want_mass,f32", ATTN)
def test_attention(cuda_dev, lens, n, Hq, H, D, page, window, sinks, want_mass, f32):
    B, L = len(lens), max(lens)
    cache, scales, pages, g = pool(B + L, B, L, H, D, page)
    # what lies behind the lengths may hold anything
    q = torch.randn(B, n, Hq, D, generator=g, device="cuda").bfloat16()
    gl = torch.tensor(lens, **I32)
    out = torch.empty(q.shape, dtype=F32 if f32 else BF16, device="cuda")
    mass = torch.rand(B, H, pages.shape[1] * page, generator=g, device="cuda") if want_mass else None
    before = mass.clone() if want_mass else None
    _, lse = api.kv8_attn(q, cache, scales, pages, gl, window=window, sinks=sinks, mass=mass, out=out)
    ok()
    limits = [[x - (n - 1) + j for j in range(n)] for x in lens]
    check_attn(q, cache, scales, pages, lens, out, lse, limits, window, sinks, mass=(before, mass) if want_mass else None)


@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3)])
@pytest.mark.parametrize("mode", ["vis", "all"])
def test_attention_under_vis_and_without_causality(cuda_dev, mode, window, sinks):
    lens, n, page = [700, 130, 0], 3, 32
    cache, scales, pages, g = pool(3, 3, 700, 2, 64, page)
    q = torch.randn(3, n, 4, 64, generator=g, device="cuda").bfloat16()
    vis = [[700, 0, 51], [-5, 500, 1], [3, 0, 1]]
    kw = dict(vis=torch.tensor(vis, **I32)) if mode == "vis" else dict(causal=False)
    mass = torch.zeros(3, 2, pages.shape[1] * page, device="cuda")
    out, lse = api.kv8_attn(q, cache, scales, pages, torch.tensor(lens, **I32), window=window, sinks=sinks, mass=mass, **kw)
    ok()
    limits = vis if mode == "vis" else [[x] * n for x in lens]
    check_attn(q, cache, scales, pages, lens, out, lse, limits, window, sinks, mass=(torch.zeros_like(mass), mass))


@pytest.mark.parametrize("size", [1e-20, 1.0, 1e6])
def test_blocks_of_very_different_scales(cuda_dev, size):
    """V's scales range over 2^60: the product of weight and scale is what is rounded, whichever is small."""
    B, L, H, D, page = 1, 320, 1, 64, 16
    g = torch.Generator(device="cuda").manual_seed(4)
    k, v = (torch.randn(B, L, H, D, generator=g, device="cuda") for _ in range(2))
    v *= size * torch.exp2((torch.arange(L, device="cuda") // 16 * 7 % 41 - 30).float())[None, :, None, None]
    k *= torch.exp2((torch.arange(L, device="cuda") // 16 % 5 - 2).float())[None, :, None, None]
    cache, scales = api.kv8_cache(L // page, H, page, D)
    pages, lens = torch.arange(L // page, **I32)[None], torch.tensor([L], **I32)
    api.kv8_append(k, v, cache, scales, pages, lens * 0)
    q = 4 * torch.randn(B, 1, 2, D, generator=g, device="cuda").bfloat16()
    out = torch.empty(q.shape, device="cuda")
    _, lse = api.kv8_attn(q, cache, scales, pages, lens, out=out)
    ok()
    check_attn(q, cache, scales, pages, [L], out, lse, [[L]], 0, 0)


@pytest.mark.parametrize("top", [1e-30, 1e-3, 300.0])
def test_sizes_of_q(cuda_dev, top):
    cache, scales, pages, g = pool(8, 1, 900, 2, 128, 64)
    q = (torch.randn(1, 1, 8, 128, generator=g, device="cuda") * top).bfloat16()
    q[0, 0, 3] = 0
    out, lse = api.kv8_attn(q, cache, scales, pages, torch.tensor([900], **I32))
    ok()
    check_attn(q, cache, scales, pages, [900], out, lse, [[900]], 0, 0)


@pytest.mark.parametrize("what", ["k", "v"])
def test_nan_reaches_only_the_rows_that_see_it(cuda_dev, what):
    """Four drafted tokens with a window: NaN in slots that some rows see, none sees, and all see."""
    L, n, page, W, K = 400, 4, 16, 40, 3
    cache, scales, pages, g = pool(9, 1, L, 1, 64, page)
    clean = cache.clone()
    q = torch.randn(1, n, 2, 64, generator=g, device="cuda").bfloat16()
    lens = torch.tensor([L], **I32)
    w = "kv".index(what)
    for slot in (0, 2, 3, 17, 200, L - n - W, L - n - W + 2, L - 20, L - 3, L - 1):
        cache.copy_(clean)
        cache[pages[0, slot // page], 0, w, slot % page, 5] = 0xff
        out, lse = api.kv8_attn(q, cache, scales, pages, lens, window=W, sinks=K)
        want, wl = api.kv8_attn(q, clean, scales, pages, lens, window=W, sinks=K)
        ok()
        for j in range(n):
            if slot in o.sees(L - n + 1 + j, W, K):
                assert out[0, j, :, 5].isnan().all()
                assert out[0, j].isnan().all() == (what == "k") and lse[0, :, j].isnan().all() == (what == "k")
            else:
                assert torch.equal(out[0, j], want[0, j]) and torch.equal(lse[0, :, j], wl[0, :, j]), (slot, j)
    cache.copy_(clean)
    scales[pages[0, 5]] = math.nan                       # a block that nobody sees
    out, lse = api.kv8_attn(q, cache, scales, pages, lens, window=W, sinks=K)
    assert torch.equal(out, want) and torch.equal(lse, wl)


def test_pages_out_of_the_window_are_not_read(cuda_dev):
    """They may have gone back to the pool."""
    lens = torch.tensor([3000, 900], **I32)
    cache, scales, pages, g = pool(10, 2, 3000, 2, 64, 32)
    q = torch.randn(2, 2, 4, 64, generator=g, device="cuda").bfloat16()
    want = api.kv8_attn(q, cache, scales, pages, lens, window=200, sinks=5)
    gone = pages.clone()
    gone[0, 1:(3000 - 1 - 200) // 32] = -7
    gone[1, 1:(900 - 1 - 200) // 32] = 1 << 30
    got = api.kv8_attn(q, cache, scales, gone, lens, window=200, sinks=5)
    ok()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_window_agrees_with_the_prompts_attention(cuda_dev):
    """The single-token form on the rows that the cache holds: window_attn_fwd's last rows."""
    S, W, K, H, Hq, D, page = 700, 150, 6, 2, 4, 128, 32
    cache, scales, pages, g = pool(11, 1, S, H, D, page)
    lens = torch.tensor([S], **I32)
    k, v = api.kv8_gather(cache, scales, pages, lens, S)
    q = torch.randn(1, 5, Hq, D, generator=g, device="cuda").bfloat16()
    out, lse = api.kv8_attn(q, cache, scales, pages, lens, window=W, sinks=K)
    ref, z = api.window_attn_fwd(q, k, v, W, K)
    ok()
    o2, zr, eo, ez = ow.forward(q, k, v, W, K)
    ow.within(ref, o2, eo, "prompt")
    ow.within(out, o2, eo, "cache")
    assert (lse - z).abs().max() <= 2e-5


EVICT = [  # lens, H, D, page, budget, first, last
    ([1], 1, 64, 16, 1, 0, 0),
    ([50, 7, 0, 16], 2, 128, 16, 16, 2, 3),
    ([1000, 999, 333], 2, 64, 32, 333, 0, 0),
    ([500], 3, 128, 256, 100, 50, 50),
    ([500, 200], 1, 64, 64, 77, 4, 70),
    ([9000, 5000], 2, 64, 64, 2000, 4, 64),        # clusters
    ([70000], 1, 64, 128, 1234, 4, 500),
    ([300] * 70, 4, 64, 16, 65, 1, 8),
]


@pytest.mark.parametrize("lens,H,D,page,budget,first,last", EVICT)
@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
def test_evict(cuda_dev, lens, H, D, page, budget, first, last, kind):
    B, L = len(lens), max(lens)
    g = torch.Generator(device="cuda").manual_seed(L + B)
    M, To = -(-L // page), -(-budget // page) + 1
    order, P = table(g, B, M + To)
    cache = torch.randint(0, 127, (P, H, 2, page, D), dtype=torch.uint8, generator=g, device="cuda")
    scales = torch.exp2(torch.randint(-6, 3, (P, H, 2, page // 16), generator=g, device="cuda").float())
    pages, to = order[:, :M].contiguous(), order[:, M:].contiguous()
    mass = torch.exp(2 * torch.randn(B, H, M * page, generator=g, device="cuda"))
    if kind == "ties":
        mass = (mass * 2).round() / 2
        mass[:, :, ::7] = -0.0
    if kind == "odd":
        mass[:, :, 5::40] = math.nan
        mass[:, :, 6::90] = math.inf
        mass[:, :, 3::11] *= -1
    was = cache.clone(), scales.clone()
    gl = torch.tensor(lens, **I32)
    kept, lens_to, mass_to = api.kv8_evict(cache, scales, pages, gl, mass, to, budget, first, last)
    k, v = api.kv8_gather(cache, scales, to, lens_to, budget)
    ok()
    assert lens_to.tolist() == [min(x, budget) for x in lens]
    c, s, t, mm = was[0].cpu().numpy(), was[1].cpu().numpy(), pages.cpu().numpy(), mass.cpu().numpy()
    gc, gs = cache.cpu().numpy(), scales.cpu().numpy()
    for b in range(B):
        for h in range(H):
            want = o.evict(mm[b, h], lens[b], budget, first, last)
            n = len(want)
            np.testing.assert_array_equal(kept[b, h].cpu().numpy(), np.concatenate([want, np.full(budget - n, -1)]))
            np.testing.assert_array_equal(mass_to[b, h, :n].cpu().numpy(), mm[b, h, want])
            assert (mass_to[b, h, n:] == 0).all()
            if (b + h) % 3 or not n:
                continue                                           # the rows of a third of the heads
            for w, x in enumerate((k, v)):
                code, tops = o.moved(c, s, t, b, h, w, want)
                val = o.decode(code) * np.repeat(tops, 16)[:n, None]
                np.testing.assert_array_equal(x[b, :n, h].double().cpu().numpy(), val)
            assert (k[b, n:, h] == 0).all()
    # nothing else is written
    mine = torch.zeros(P, dtype=torch.bool, device="cuda")
    mine[to.flatten().long()] = True
    assert torch.equal(cache[~mine], was[0][~mine]) and torch.equal(scales[~mine], was[1][~mine])
    used = (torch.tensor([min(x, budget) for x in lens], device="cuda")[:, None] > torch.arange(To, device="cuda") * page)
    assert torch.equal(cache[to[~used].long()], was[0][to[~used].long()])


def test_evict_of_rows_too_long_for_shared_memory(cuda_dev):
    """A table of over 400000 slots: keys are read from memory in every round."""
    page, D, L, budget = 256, 64, 410000, 900
    M, To = -(-L // page), 4
    g = torch.Generator(device="cuda").manual_seed(1)
    cache = torch.randint(0, 127, (M + To, 1, 2, page, D), dtype=torch.uint8, generator=g, device="cuda")
    scales = torch.ones(M + To, 1, 2, page // 16, device="cuda")
    pages, to = torch.arange(M, **I32)[None], torch.arange(M, M + To, **I32)[None]
    mass = (torch.rand(1, 1, M * page, generator=g, device="cuda") * 5000).round()
    kept, lens_to, mass_to = api.kv8_evict(cache, scales, pages, torch.tensor([L], **I32), mass, to, budget, 3, 10)
    ok()
    want = o.evict(mass[0, 0].cpu().numpy(), L, budget, 3, 10)
    np.testing.assert_array_equal(kept[0, 0].cpu().numpy(), want)
    np.testing.assert_array_equal(mass_to[0, 0, :budget].cpu().numpy(), mass[0, 0].cpu().numpy()[want])
    i = torch.from_numpy(want).cuda()
    assert torch.equal(cache[to[0].long()].permute(1, 2, 0, 3, 4).reshape(2, -1, D)[:, :budget],
                       cache[:M].permute(1, 2, 0, 3, 4).reshape(2, -1, D)[:, i])


def test_a_run_with_eviction(cuda_dev):
    """Prompt, steps that accumulate weights, eviction, more steps: every step against attention over what the
    cache holds, and the accumulated weights against their sum."""
    B, S, H, Hq, D, page, budget = 2, 190, 2, 4, 64, 16, 96
    g = torch.Generator(device="cuda").manual_seed(21)
    M, To = 14, 8
    order, P = table(g, B, M + To)
    cache, scales = api.kv8_cache(P, H, page, D)
    pages, to = order[:, :M].contiguous(), order[:, M:].contiguous()
    r = lambda n, h: torch.randn(B, n, h, D, generator=g, device="cuda").bfloat16()  # noqa: E731
    q, k, v = r(S, Hq), r(S, H), r(S, H)
    out, lse = api.window_attn_fwd(q, k, v, S)               # the prompt itself
    o1, z1, eo, ez = ow.forward(q, k, v, S, 0)
    ow.within(out, o1, eo, "prompt")
    lens = torch.zeros(B, **I32)
    api.kv8_append(k, v, cache, scales, pages, lens)
    lens += S
    mass = torch.zeros(B, H, M * page, device="cuda")
    for step in range(12):
        q, k, v = r(1, Hq), r(1, H), r(1, H)
        api.kv8_append(k, v, cache, scales, pages, lens)
        lens += 1
        before = mass.clone()
        out, lse = api.kv8_attn(q, cache, scales, pages, lens, mass=mass)
        ok()
        check_attn(q, cache, scales, pages, lens.tolist(), out, lse, [[int(x)] for x in lens], 0, 0, mass=(before, mass))
        assert abs(float((mass - before).sum()) - B * Hq) <= 1e-3   # each row's weights sum to 1
        if step == 5:
            kept, lens, mass = api.kv8_evict(cache, scales, pages, lens, mass, to, budget, keep_first=2, keep_last=8)
            pages = to
            assert lens.tolist() == [budget] * B and (kept[:, :, :2] == torch.tensor([0, 1], device="cuda")).all()
    assert lens.tolist() == [budget + 6] * B


def test_captured_steps_replay(cuda_dev):
    """A captured step (append, attention with weights, eviction, read-back) follows the lengths on the device."""
    B, H, D, page = 2, 2, 128, 32
    g = torch.Generator(device="cuda").manual_seed(30)

    def fresh():
        order = torch.arange(B * 24, **I32).reshape(B, 24)
        cache, scales = api.kv8_cache(B * 24, H, page, D)
        cache.zero_(), scales.zero_()
        t = dict(cache=cache, scales=scales, pages=order[:, :16].contiguous(), to=order[:, 16:].contiguous(),
                 lens=torch.tensor([300, 77], **I32), mass=torch.zeros(B, H, 16 * page, device="cuda"))
        gg = torch.Generator(device="cuda").manual_seed(31)
        k = torch.randn(B, 400, H, D, generator=gg, device="cuda")
        api.kv8_append(k, k.flip(1), t["cache"], t["scales"], t["pages"], torch.zeros(B, **I32))
        return t
    q = torch.randn(B, 1, 4, D, generator=g, device="cuda").bfloat16()
    k = torch.randn(B, 1, H, D, generator=g, device="cuda").bfloat16()

    def step(t):
        api.kv8_append(k, k, t["cache"], t["scales"], t["pages"], t["lens"])
        t["lens"] += 1
        outs = list(api.kv8_attn(q, t["cache"], t["scales"], t["pages"], t["lens"], mass=t["mass"]))
        outs += api.kv8_attn(q, t["cache"], t["scales"], t["pages"], t["lens"], window=50, sinks=4)
        outs += api.kv8_evict(t["cache"], t["scales"], t["pages"], t["lens"], t["mass"], t["to"], 60, 2, 5)
        outs += api.kv8_gather(t["cache"], t["scales"], t["to"], outs[-2], 60)
        return outs
    a, b = fresh(), fresh()
    step(b)                                                   # warm
    b = fresh()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = step(b)
    for t, v in fresh().items():
        b[t].copy_(v)
    for _ in range(4):
        want = step(a)
        graph.replay()
        ok()
        assert all(torch.equal(x, y) for x, y in zip(want, got))
        assert all(torch.equal(a[n], b[n]) for n in a)


def test_other_stream_and_threads(cuda_dev):
    """Two threads, each with a stream, a pool and steps of its own, as one after the other."""
    want, got, errors = {}, {}, []

    def steps(i, into):
        cache, scales, pages, g = pool(40 + i, 2, 2000, 2, 64, 32, width=70)
        to = torch.arange(cache.shape[0], **I32)[None].repeat(2, 1)[:, :0]
        extra, es = api.kv8_cache(cache.shape[0] + 16, 2, 32, 64)
        extra[:cache.shape[0]].copy_(cache), es[:cache.shape[0]].copy_(scales)
        to = (torch.arange(16, **I32) + cache.shape[0]).reshape(2, 8)
        q = torch.randn(2, 1, 4, 64, generator=g, device="cuda").bfloat16()
        lens = torch.tensor([1900, 300 + i], **I32)
        mass = torch.zeros(2, 2, 70 * 32, device="cuda")
        outs = []
        for _ in range(20):
            k = torch.randn(2, 1, 2, 64, generator=g, device="cuda").bfloat16()
            api.kv8_append(k, k, extra, es, pages, lens)
            lens += 1
            outs += [*api.kv8_attn(q, extra, es, pages, lens, mass=mass), mass.clone(),
                     *api.kv8_evict(extra, es, pages, lens, mass, to, 250, 1, 9)]
        torch.cuda.current_stream().synchronize()
        into[i] = outs

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                steps(i, got)
        except Exception as e:   # shown by the main thread
            errors.append(e)
    for i in range(2):
        steps(i, want)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    ok()
    assert not errors
    for i in range(2):
        assert all(torch.equal(x, y) for x, y in zip(want[i], got[i]))


def test_given_stream_and_buffers(cuda_dev):
    """stream= and buffers of the caller's own with any contents give the same; what lies around them stays."""
    B, L, page = 2, 600, 32
    cache, scales, pages, g = pool(50, B, L, 2, 64, page)
    lens = torch.tensor([600, 211], **I32)
    q = torch.randn(B, 2, 4, 64, generator=g, device="cuda").bfloat16()
    mass0 = torch.rand(B, 2, pages.shape[1] * page, generator=g, device="cuda")
    m1, m2 = mass0.clone(), mass0.clone()
    out, lse = api.kv8_attn(q, cache, scales, pages, lens, mass=m1)
    ok()
    s = torch.cuda.Stream()
    need = api.kv8_attn_workspace(B, 2, 4, 2, 64, page, pages.shape[1], True)
    ws = torch.full((need + 512,), 255, dtype=torch.uint8, device="cuda")
    mine, z = torch.full_like(out, math.nan), torch.full_like(lse, math.nan)
    torch.cuda.synchronize()
    got = api.kv8_attn(q, cache, scales, pages, lens, mass=m2, out=mine, lse=z, workspace=ws[256:256 + need], stream=s)
    s.synchronize()
    assert got[0] is mine or got[0].data_ptr() == mine.data_ptr()
    assert torch.equal(mine, out) and torch.equal(z, lse) and torch.equal(m1, m2)
    assert (ws[:256] == 255).all() and (ws[-256:] == 255).all()
    k, v = api.kv8_gather(cache, scales, pages, lens, 70, start=lens - 60, stream=s)
    s.synchronize()
    k2, v2 = torch.full_like(k, math.nan), torch.full_like(v, math.nan)
    api.kv8_gather(cache, scales, pages, lens, 70, start=lens - 60, k=k2, v=v2)
    ok()
    assert torch.equal(k, k2) and torch.equal(v, v2) and (k2[:, 60:] == 0).all()


def test_tables_wider_than_the_sequences(cuda_dev):
    """A table for a far longer context takes other kernels, not other results (but for the order of sums)."""
    lens = torch.tensor([500, 64, 1, 0], **I32)
    outs = []
    for width in (8, 4000):
        cache, scales, pages, g = pool(60, 4, 500, 2, 128, 64, width)
        q = torch.randn(4, 1, 6, 128, generator=g, device="cuda").bfloat16()
        out, lse = api.kv8_attn(q, cache, scales, pages, lens)
        ok()
        check_attn(q, cache, scales, pages, lens.tolist(), out, lse, [[int(x)] for x in lens], 0, 0)


def test_bad_pages_lengths_and_slots_are_reported(cuda_dev):
    """They are skipped and recorded; neighbours stay as they are."""
    H, D, page = 1, 64, 16
    cache, scales, pages, g = pool(70, 1, 64, H, D, page)
    k = torch.randn(1, 20, H, D, generator=g, device="cuda").bfloat16()
    q = torch.randn(1, 1, 2, D, generator=g, device="cuda").bfloat16()
    was = cache.clone()
    bad = pages.clone()
    bad[0, 2] = cache.shape[0]
    one = torch.tensor([64], **I32)
    mass = torch.zeros(1, H, 64, device="cuda")
    spare = [p for p in range(cache.shape[0]) if p not in pages[0].tolist()]
    to = torch.tensor([[cache.shape[0] + 3, -1]], **I32)
    calls = [lambda: api.kv8_append(k, k, cache, scales, bad, torch.tensor([32], **I32)),
             lambda: api.kv8_append(k, k, cache, scales, pages, torch.tensor([60], **I32)),      # slots behind the table
             lambda: api.kv8_append(k, k, cache, scales, pages, torch.tensor([-3], **I32)),
             lambda: api.kv8_gather(cache, scales, bad, one, 64),
             lambda: api.kv8_gather(cache, scales, pages, one, 8, start=torch.tensor([-4], **I32)),
             lambda: api.kv8_attn(q, cache, scales, bad, one),
             lambda: api.kv8_attn(q, cache, scales, pages, one * 2),
             # (slots 44 to 63: the bad page's last ones among them)
             lambda: api.kv8_evict(cache, scales, bad, one, mass, torch.tensor([spare[:2]], **I32), 20, keep_last=20),
             lambda: api.kv8_evict(cache, scales, pages, one, mass, to, 20)]
    for i, call in enumerate(calls):
        call()
        torch.cuda.synchronize()
        assert api.cp_get_error() == _lib.CP_ECACHE, i
    assert torch.equal(cache[spare[2:]], was[spare[2:]])


def test_wait_that_runs_out(cuda_dev):
    """The bounded waits' failure path: a status, and the next call works."""
    for L in (9000, 300):
        cache, scales, pages, g = pool(80, 1, L, 1, 128, 64)
        q = torch.randn(1, 1, 2, 128, generator=g, device="cuda").bfloat16()
        lens = torch.tensor([L], **I32)
        want = api.kv8_attn(q, cache, scales, pages, lens)
        ok()
        api.cp_debug_set_wait_limit(1)
        try:
            api.kv8_attn(q, cache, scales, pages, lens)
            torch.cuda.synchronize()
            assert api.cp_get_error() == _lib.CP_ETIMEOUT
        finally:
            api.cp_debug_set_wait_limit(0)
        got = api.kv8_attn(q, cache, scales, pages, lens)
        ok()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_a_pool_beyond_32_bits(cuda_dev):
    """Rows and scales past 2^32 bytes of the pool."""
    H, D, page = 8, 128, 256
    P = 9000                                                     # 4.7 GB
    cache, scales = api.kv8_cache(P, H, page, D)
    pages = torch.tensor([[P - 1, 3, P - 2]], **I32)
    to = torch.tensor([[P - 5]], **I32)
    g = torch.Generator(device="cuda").manual_seed(90)
    n = 700
    k, v = (torch.randn(1, n, H, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    lens = torch.tensor([n], **I32)
    api.kv8_append(k, v, cache, scales, pages, lens * 0)
    q = torch.randn(1, 1, H, D, generator=g, device="cuda").bfloat16()
    mass = torch.zeros(1, H, 3 * page, device="cuda")
    out, lse = api.kv8_attn(q, cache, scales, pages, lens, mass=mass)
    kept, lt, mt = api.kv8_evict(cache, scales, pages, lens, mass, to, 200)
    gk, gv = api.kv8_gather(cache, scales, to, lt, 200)
    fk, fv = api.kv8_gather(cache, scales, pages, lens, n)
    ok()
    small = torch.stack([cache[p] for p in pages[0].tolist()]), torch.stack([scales[p] for p in pages[0].tolist()])
    t = torch.tensor([[0, 1, 2]], **I32)
    check_attn(q, small[0], small[1], t, [n], out, lse, [[n]], 0, 0)
    for h in range(H):
        i = kept[0, h].long()
        assert (gk[0, :, h].double() - fk[0, i, h].double()).abs().max() <= 2.0 ** -3 * fk.abs().max()
        assert torch.equal(mt[0, h, :200], mass[0, h, i])


def test_refusals(cuda_dev):
    cache, scales, pages, g = pool(95, 2, 64, 2, 64, 16)
    lens = torch.tensor([64, 64], **I32)
    k = torch.randn(2, 1, 2, 64, device="cuda").bfloat16()
    q = torch.randn(2, 1, 4, 64, device="cuda").bfloat16()
    mass = torch.zeros(2, 2, 64, device="cuda")
    for kw in (dict(k=k.half(), v=k.half()), dict(k=k[..., :32].contiguous(), v=k[..., :32].contiguous()), dict(v=k.float()),
               dict(k=k.transpose(2, 3), v=k.transpose(2, 3)), dict(cache=cache[0]), dict(cache=cache.float()), dict(scales=scales[:, :1]),
               dict(scales=scales.double()), dict(pages=pages.long()), dict(pages=pages[:1]), dict(lens=lens[:1]), dict(lens=lens.cpu()),
               dict(n_new=lens.long()), dict(k=k.cpu(), v=k.cpu())):
        a = dict(k=k, v=k, cache=cache, scales=scales, pages=pages, lens=lens - 1) | kw
        with pytest.raises(ValueError):
            api.kv8_append(**a)
    for kw in (dict(q=q.float()), dict(q=q[0]), dict(q=q[..., :32].contiguous()), dict(mass=mass[..., :32]), dict(mass=mass.double()),
               dict(out=q.half()), dict(lse=torch.empty(2, 4, 2, device="cuda")), dict(vis=lens), dict(workspace=torch.empty(9).cuda()[::2])):
        a = dict(q=q, cache=cache, scales=scales, pages=pages, lens=lens) | kw
        with pytest.raises(ValueError):
            api.kv8_attn(**a)
    for kw in (dict(window=-1), dict(sinks=-2), dict(scale=math.nan), dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(api.CpError):
            api.kv8_attn(q, cache, scales, pages, lens, **kw)
    to = torch.zeros(2, 1, **I32)
    for kw in (dict(mass=mass[:1]), dict(pages_to=to[:1]), dict(pages_to=to.long()), dict(kept=to), dict(lens_to=lens.long()),
               dict(mass_to=mass)):
        a = dict(cache=cache, scales=scales, pages=pages, lens=lens, mass=mass, pages_to=to, budget=10) | kw
        with pytest.raises(ValueError):
            api.kv8_evict(**a)
    for kw in (dict(budget=0), dict(budget=17), dict(keep_first=-1), dict(keep_first=6, keep_last=6)):
        with pytest.raises(api.CpError):
            api.kv8_evict(**(dict(cache=cache, scales=scales, pages=pages, lens=lens, mass=mass, pages_to=to, budget=10) | kw))
    with pytest.raises(ValueError):
        api.kv8_gather(cache, scales, pages, lens, 4, dtype=torch.float16)
    with pytest.raises(api.CpError):
        api.kv8_gather(cache, scales, pages, lens, -1)


def test_no_gradient(cuda_dev):
    """Inputs that require gradients are taken; what comes back requires none, as the documentation says."""
    cache, scales, pages, g = pool(96, 1, 100, 1, 64, 16)
    k, q = (torch.randn(1, 1, h, 64, generator=g, device="cuda").bfloat16().requires_grad_() for h in (1, 2))
    lens = torch.tensor([40], **I32)
    api.kv8_append(k, k, cache, scales, pages, lens)
    out, lse = api.kv8_attn(q, cache, scales, pages, lens)
    ok()
    assert not (out.requires_grad or lse.requires_grad)
    for f in (api.kv8_append, api.kv8_gather, api.kv8_attn):
        assert "radient" in f.__doc__


def test_a_bad_page_adds_no_mass_and_moves_as_zeros(cuda_dev):
    """Slots of a page that is not there: their mass stays, and what is kept of them is 0."""
    H, D, page, L = 2, 64, 16, 80
    cache, scales, pages, _ = pool(3, 1, L, H, D, page)
    lens = torch.tensor([L], **I32)
    bad = pages.clone()
    bad[0, 1] = cache.shape[0] + 5
    q = torch.randn(1, 1, 4, D, device=cuda_dev).bfloat16()
    mass = torch.full((1, H, pages.shape[1] * page), 2.0, device=cuda_dev)
    ws = torch.full((api.kv8_attn_workspace(1, 1, 4, H, D, page, pages.shape[1], True),), 0x7f, dtype=torch.uint8, device=cuda_dev)
    out, lse = api.kv8_attn(q, cache, scales, bad, lens, mass=mass, workspace=ws)
    assert api.cp_get_error() == _lib.CP_ECACHE
    # (2 plus a weight below 2^-23 is 2: the weights of the other slots show in their sum, 160 roundings of 2^-23)
    assert torch.isfinite(out).all() and (mass[..., 16:32] == 2).all() and (mass >= 2).all()
    assert abs(float((mass[..., :L] - 2).sum()) - 4) < 1e-4
    spare = [p for p in range(cache.shape[0]) if p not in pages.flatten().tolist()][:2]
    mass.zero_()
    mass[..., 16:32] = 1
    kept, _, _ = api.kv8_evict(cache, scales, bad, lens, mass, torch.tensor([spare], **I32), 20)
    assert api.cp_get_error() == _lib.CP_ECACHE
    assert kept[0, 0].tolist() == [0, 1, 2, 3, *range(16, 32)]
    assert not (cache[spare[0], :, :, 4:16] & 0x7f).any() and torch.isfinite(scales[spare]).all()


def test_attention_refuses_to_write_over_q(cuda_dev):
    cache, scales, pages, _ = pool(5, 1, 64, 2, 64, 16)
    q = torch.randn(1, 1, 4, 64, device=cuda_dev).bfloat16()
    with pytest.raises(api.CpError) as e:
        api.kv8_attn(q, cache, scales, pages, torch.tensor([64], **I32), out=q)
    assert e.value.code == _lib.CP_EINVAL


def test_evict_refuses_to_write_what_it_reads(cuda_dev):
    H, D, page, L = 2, 64, 16, 64
    cache, scales, pages, _ = pool(4, 2, L, H, D, page)
    lens = torch.full((2,), L, **I32)
    mass = torch.rand(2, H, pages.shape[1] * page, device=cuda_dev)
    with pytest.raises(api.CpError) as e:                  # more than pages_to hold, and than memory would
        api.kv8_evict(cache, scales, pages, lens, mass, pages.flip(1).contiguous(), 2 ** 31 - 1)
    assert e.value.code == _lib.CP_EINVAL
    for kw in (dict(lens_to=lens), dict(mass_to=mass)):
        with pytest.raises(api.CpError) as e:
            api.kv8_evict(cache, scales, pages, lens, mass, pages.flip(1).contiguous(), 16, **kw)
        assert e.value.code == _lib.CP_EINVAL
