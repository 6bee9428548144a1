"""The 8-bit cache where a call meets its limits: blocks that no row sees and rows of q that are not finite, windows
and wide tiles through stretches and join, many rows with weights."""
import math

import numpy as np
import pytest
import torch

from context_parallelism_02_gb300 import api
from oracle import kv8 as o
from test_gpu_kv8 import F32, I32, check_attn, ok, pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan, float(np.uint32(0x7f7f7f7f).view(np.float32)), -1.0, 0.0])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3)])
@pytest.mark.parametrize("L", [300, 9000])
def test_scales_of_blocks_that_no_row_sees(cuda_dev, value, window, sinks, L):
    """Under vis every block below the length is read: the scales of those that no row sees (pages reserved or reused,
    not written) may hold anything.  Short tables and stretches with their join."""
    n, H, Hq, D, page = 2, 2, 4, 64, 16
    cache, scales, pages, g = pool(12, 1, L, H, D, page)
    q = torch.randn(1, n, Hq, D, generator=g, device="cuda").bfloat16()
    vis, lens = [[L // 2, L // 2 - 7]], torch.tensor([L], **I32)
    seen = np.unique(np.concatenate([o.sees(x, window, sinks) for x in vis[0]]))
    hidden = sorted(set(range(-(-L // page))) - set(seen // page))
    assert len(hidden) > 4
    bad = scales.clone()
    bad[pages[0, hidden].long()] = value
    got = []
    for s in (scales, bad):
        mass = torch.zeros(1, H, pages.shape[1] * page, device="cuda")
        out, lse = api.kv8_attn(q, cache, s, pages, lens, window=window, sinks=sinks, vis=torch.tensor(vis, **I32), mass=mass)
        ok()
        got.append((out, lse, mass))
    assert torch.isfinite(got[0][0]).all()
    assert all(torch.equal(x, y) for x, y in zip(*got))


@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 2)])
@pytest.mark.parametrize("L", [1, 20, 300, 9000])
def test_rows_of_q_with_an_infinity(cuda_dev, L, window, sinks):
    """One infinite element makes every score an infinity of its token's sign there (or NaN): the row, its lse and
    the weights of what it sees are NaN, also where all its scores are -infinity.  Other rows are as they were."""
    H, Hq, D, page = 2, 8, 64, 16
    cache, scales, pages, g = pool(13, 1, L, H, D, page)
    cache[pages[0].long(), :, 0] &= 0x7f                        # keys without a sign
    k = cache[pages[0].long(), :, 0].view(torch.float8_e4m3fn).float()
    assert not (k < 0).any()
    q = torch.randn(1, 1, Hq, D, generator=g, device="cuda").bfloat16()
    lens = torch.tensor([L], **I32)
    at = torch.from_numpy(o.sees(L, window, sinks)).cuda()
    kk, vv = o.read(cache.cpu().numpy(), scales.cpu().numpy(), pages.cpu().numpy(), 0, 0, at.cpu().numpy())
    vs = scales.cpu().numpy()[pages.cpu().numpy()[0, at.cpu().numpy() // page], 0, 1, at.cpu().numpy() % page // 16]
    clean = api.kv8_attn(q, cache, scales, pages, lens, window=window, sinks=sinks)
    for element, value in ((5, math.inf), (5, -math.inf), (63, -math.inf)):
        bad = q.clone()
        bad[0, 0, 1, element] = value
        mass = torch.zeros(1, H, pages.shape[1] * page, device="cuda")
        out, lse = api.kv8_attn(bad, cache, scales, pages, lens, window=window, sinks=sinks, mass=mass)
        ok()
        assert out[0, 0, 1].isnan().all() and lse[0, 1].isnan()
        assert mass[0, 0, at].isnan().all() and int(mass[0, 0].isnan().sum()) == len(at)
        assert torch.equal(out[0, 0, 4:], clean[0][0, 0, 4:]) and torch.equal(lse[0, 4:], clean[1][0, 4:])   # the other kv head's
        for x in (0, 2, 3):                                     # those that share its tile
            ref, z, _, err, ez = o.attend(q[0, 0, x].double().cpu().numpy(), kk, vv, vs.astype(np.float64), D ** -0.5)
            d = np.abs(out[0, 0, x].double().cpu().numpy() - ref) - (err + 2.0 ** -8 * (np.abs(ref) + err))
            assert d.max() <= 0 and abs(lse[0, x].item() - z) <= ez


def attention(lens, n, Hq, H, D, page, window, sinks, want_mass, seed, f32=False):
    """One call against the definition, with a workspace of its own that has other things around it."""
    B = len(lens)
    cache, scales, pages, g = pool(seed, B, max(lens), H, D, page)
    q = torch.randn(B, n, Hq, D, generator=g, device="cuda").bfloat16()
    mass = torch.rand(B, H, pages.shape[1] * page, generator=g, device="cuda") if want_mass else None
    before = mass.clone() if want_mass else None
    need = api.kv8_attn_workspace(B, n, Hq, H, D, page, pages.shape[1], want_mass)
    ws = torch.full((need + 512,), 0x5a, dtype=torch.uint8, device="cuda")
    out = torch.empty(q.shape, dtype=F32, device="cuda") if f32 else None
    out, lse = api.kv8_attn(q, cache, scales, pages, torch.tensor(lens, **I32), window=window, sinks=sinks, mass=mass, out=out,
                            workspace=ws[256:256 + need])
    ok()
    assert (ws[:256] == 0x5a).all() and (ws[256 + need:] == 0x5a).all()
    limits = [[x - (n - 1) + j for j in range(n)] for x in lens]
    check_attn(q, cache, scales, pages, lens, out, lse, limits, window, sinks, mass=(before, mass) if want_mass else None)


# lens, n, Hq, Hkv, D, page, window, sinks, mass.  An item has more blocks than a block of warps takes by itself, so
# warps' stretches begin and end at all of its blocks: among the sinks, at the gap behind them, in the window.
WINDOWS = [
    ([5000, 3000, 1030], 1, 8, 8, 128, 32, 1024, 4, False),
    ([5000, 900, 40], 3, 8, 4, 64, 16, 800, 70, True),
    ([4000, 4001], 2, 8, 2, 128, 64, 1000, 300, True),
    ([2600] * 30, 1, 8, 8, 64, 16, 1100, 20, False),          # more items than SMs
    ([6000, 6000, 17], 6, 8, 2, 64, 128, 1500, 33, True),     # 24 rows: two tiles of 16
    ([6000], 1, 1, 1, 128, 16, 3000, 1, True),
    ([2300 - 45 * i for i in range(50)], 1, 16, 8, 128, 16, 1100, 20, False),   # few pieces an item: joined by a warp per row
    ([1900 - 30 * i for i in range(50)], 2, 16, 8, 64, 32, 1040, 33, True),
]


@pytest.mark.parametrize("case", WINDOWS)
def test_windows_with_sinks_through_stretches_and_join(cuda_dev, case):
    attention(*case, seed=20 + len(case[0]))


# D = 64 with tiles of 16 rows: the workspace has room for three blocks of warps an SM
WIDE = [
    ([16384, 16000], 4, 16, 4, 64, 64, 0, 0, False),          # as many warps as fit at once
    ([1040] * 24, 5, 16, 4, 64, 16, 0, 0, False),             # 20 rows, 192 items
    ([5000, 700, 3], 3, 16, 4, 64, 16, 0, 0, True),           # 12 rows
    ([9000], 2, 16, 2, 64, 256, 0, 0, True),
]


@pytest.mark.parametrize("case", WIDE)
def test_many_rows_of_64_elements_through_stretches_and_join(cuda_dev, case):
    attention(*case, seed=40 + len(case[0]), f32=len(case[0]) == 1)


# more rows of a kv head than the weights' kernel takes at a time (64): lengths with stretches of slots that all rows see
# whole, and ends, windows and short sequences where they do not
MANY_ROWS = [
    ([2500, 1100], 5, 17, 1, 64, 32, 0, 0, True),             # 85 rows, no multiple of four
    ([2500, 1100], 5, 17, 1, 64, 32, 700, 5, True),
    ([3000, 70, 1], 8, 32, 2, 128, 64, 0, 0, True),           # 128 rows
    ([3000, 70, 1], 8, 32, 2, 128, 64, 1200, 40, True),
    ([400], 9, 29, 1, 64, 16, 0, 0, True),                    # 261 rows, a block of warps per item
]


@pytest.mark.parametrize("case", MANY_ROWS)
def test_weights_of_many_rows(cuda_dev, case):
    attention(*case, seed=60 + len(case[0]))


def test_widths_of_the_table_agree(cuda_dev):
    """A table for a far longer context takes other kernels: results differ by their roundings, each within what it may be off."""
    lens, H, Hq, D, page = [500, 64, 1, 0, 333], 2, 6, 128, 64
    got = []
    for width in (8, 4000):
        cache, scales, pages, g = pool(60, 5, 500, H, D, page, width)
        q = torch.randn(5, 1, Hq, D, generator=g, device="cuda").bfloat16()
        out = torch.empty(q.shape, dtype=F32, device="cuda")
        got.append((out, api.kv8_attn(q, cache, scales, pages, torch.tensor(lens, **I32), out=out)[1]))
    ok()
    c, s, t = cache.cpu().numpy(), scales.cpu().numpy(), pages.cpu().numpy()
    (a, za), (b, zb) = got
    for i, L in enumerate(lens):
        for x in range(Hq):
            if not L:
                assert not a[i].any() and not b[i].any() and torch.equal(za[i], zb[i])
                continue
            h, at = x * H // Hq, np.arange(L)
            kk, vv = o.read(c, s, t, i, h, at)
            ref, z, _, err, ez = o.attend(q[i, 0, x].double().cpu().numpy(), kk, vv, s[t[i, at // page], h, 1, at % page // 16].astype(np.float64),
                                          D ** -0.5)
            d = (a[i, 0, x].double() - b[i, 0, x].double()).abs().cpu().numpy()
            assert (d <= 2 * (err + 2.0 ** -24 * (np.abs(ref) + err))).all() and abs(za[i, x] - zb[i, x]).item() <= 2 * ez


def test_a_prompts_last_tokens_say_what_is_evicted(cuda_dev):
    """Prompt, append, the weights that its last tokens give to all, eviction, a step: the queries of a prompt as rows of kv8_attn."""
    B, S, n, H, Hq, D, page, budget = 2, 700, 24, 2, 8, 64, 32, 200
    g = torch.Generator(device="cuda").manual_seed(70)
    M, To = -(-S // page), -(-budget // page) + 1
    order = torch.randperm(B * (M + To), generator=g, device="cuda").int().reshape(B, -1)
    pages, to = order[:, :M].contiguous(), order[:, M:].contiguous()
    cache, scales = api.kv8_cache(B * (M + To), H, page, D)
    q, k, v = (torch.randn(B, S, h, D, generator=g, device="cuda").bfloat16() for h in (Hq, H, H))
    api.kv8_append(k, v, cache, scales, pages, torch.zeros(B, **I32))
    lens, mass = torch.full((B,), S, **I32), torch.zeros(B, H, M * page, device="cuda")
    last = q[:, -n:].contiguous()
    out, lse = api.kv8_attn(last, cache, scales, pages, lens, mass=mass)
    ok()
    check_attn(last, cache, scales, pages, [S] * B, out, lse, [[S - n + 1 + j for j in range(n)]] * B, 0, 0, mass=(torch.zeros_like(mass), mass))
    assert abs(float(mass.double().sum()) - B * n * Hq) <= 1e-3 * B * n * Hq
    kept, lens_to, mass_to = api.kv8_evict(cache, scales, pages, lens, mass, to, budget, keep_first=4, keep_last=n)
    for b in range(B):
        for h in range(H):
            np.testing.assert_array_equal(kept[b, h].cpu().numpy(), o.evict(mass[b, h].cpu().numpy(), S, budget, 4, n))
    api.kv8_append(k[:, :1], v[:, :1], cache, scales, to, lens_to)
    lens_to += 1
    before = mass_to.clone()
    out, lse = api.kv8_attn(last[:, :1].contiguous(), cache, scales, to, lens_to, mass=mass_to)
    ok()
    check_attn(last[:, :1].contiguous(), cache, scales, to, [budget + 1] * B, out, lse, [[budget + 1]] * B, 0, 0, mass=(before, mass_to))


@pytest.mark.parametrize("n", [1, 40])
def test_sequences_without_new_tokens_need_no_pages(cuda_dev, n):
    """A padded batch whose idle sequences have lengths of before and no pages: nothing is written, read or reported for them."""
    H, D, page = 2, 64, 16
    cache, scales, pages, g = pool(14, 3, 100, H, D, page)
    was, were = cache.clone(), scales.clone()
    k = torch.randn(3, n, H, D, generator=g, device="cuda").bfloat16()
    pages[1:] = -1
    api.kv8_append(k, k, cache, scales, pages, torch.tensor([0, 37, 99], **I32), n_new=torch.tensor([n, 0, -2], **I32))
    ok()
    mine = torch.zeros(cache.shape[0], dtype=torch.bool, device="cuda")
    mine[pages[0].long()] = True
    assert torch.equal(cache[~mine], was[~mine])
    assert torch.equal(scales[~mine].nan_to_num(-1), were[~mine].nan_to_num(-1))


def test_evict_of_rows_that_just_fit_shared_memory(cuda_dev):
    """A cluster of eight blocks with 195 KB of keys each."""
    page, D, L, budget = 256, 64, 390000, 1000
    M, To = -(-L // page), 4
    g = torch.Generator(device="cuda").manual_seed(2)
    cache = torch.randint(0, 127, (M + To, 1, 2, page, D), dtype=torch.uint8, generator=g, device="cuda")
    scales = torch.ones(M + To, 1, 2, page // 16, device="cuda")
    pages, to = torch.arange(M, **I32)[None], torch.arange(M, M + To, **I32)[None]
    mass = torch.rand(1, 1, M * page, generator=g, device="cuda")
    kept, _, mass_to = api.kv8_evict(cache, scales, pages, torch.tensor([L], **I32), mass, to, budget, 3, 10)
    ok()
    want = o.evict(mass[0, 0].cpu().numpy(), L, budget, 3, 10)
    np.testing.assert_array_equal(kept[0, 0].cpu().numpy(), want)
    np.testing.assert_array_equal(mass_to[0, 0, :budget].cpu().numpy(), mass[0, 0].cpu().numpy()[want])


@pytest.mark.parametrize("L", [1, 40, 9000])
def test_scores_below_the_range_of_fp32(cuda_dev, L):
    """Scores that overflow to -infinity: a row of nothing else is an empty one, (0, -inf), and adds no weight."""
    H, Hq, D, page = 1, 4, 64, 16
    g = torch.Generator(device="cuda").manual_seed(15)
    pages, P = torch.randperm(-(-L // page), generator=g, device="cuda").int()[None], -(-L // page)
    cache, scales = api.kv8_cache(P, H, page, D)
    k = torch.full((1, L, H, D), 1e12, device="cuda")
    api.kv8_append(k, torch.ones_like(k), cache, scales, pages, torch.zeros(1, **I32))
    q = torch.randn(1, 1, Hq, D, generator=g, device="cuda").mul(1e-13).bfloat16()
    q[0, 0, 1] = -3e38
    mass, lens = torch.zeros(1, H, P * page, device="cuda"), torch.tensor([L], **I32)
    out, lse = api.kv8_attn(q, cache, scales, pages, lens, mass=mass)
    ok()
    assert not out[0, 0, 1].any() and lse[0, 1] == -math.inf
    # all keys are alike: the other rows give each 1 / L, to the roundings of the sums, (L / 16 + 40) 2^-23, and of e^(s - lse)
    assert (mass[0, 0, :L] * L / (Hq - 1) - 1).abs().max() <= (L / 16 + 40) * 2.0 ** -23 + 2.0 ** -18 and not mass[0, 0, L:].any()
    assert (out[0, 0, [0, 2, 3]].float() - 1).abs().max() <= 2.0 ** -7
