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
