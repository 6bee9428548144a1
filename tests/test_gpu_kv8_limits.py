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
