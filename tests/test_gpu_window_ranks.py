"""Windowed attention of ranks that hold a part of the rows each, of many sinks, and rows whose scores are all -infinity."""
import math

import pytest
import torch

from context_parallelism_02_gb300 import api
from oracle import window as ref
from test_gpu_window import BF16, F32, UNIT, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D,W", [(64, 1), (128, 1), (128, 3)])
def test_a_row_whose_scores_are_all_minus_infinity(cuda_dev, dtype, D, W):
    """It sees keys, so it is no empty row: its lse is NaN as its output is, and a merge does not drop it."""
    S, H = 300, 2
    q, k, v, do = make((1, S, S, H, 1, D, W, 0), dtype, cuda_dev)
    k[..., 7] = k[..., 7].abs() + 0.5
    o, z, eo, ez = ref.forward(q, k, v, W, 0, None, UNIT[dtype])
    for at in (0, 1, 130, S - 1):
        bad = q.clone()
        bad[0, at, 1, 7] = -math.inf
        out, lse = api.window_attn_fwd(bad, k, v, W)
        rest = torch.ones(S, H, dtype=torch.bool, device=cuda_dev)
        rest[at, 1] = False
        assert out[0, at, 1].isnan().all() and lse[0, 1, at].isnan()
        ref.within(out[0][rest], o[0][rest], eo[0][rest], "out")
        ref.within(lse[0].T[rest], z[0].T[rest], ez[0].T[rest], "lse")
        rows = lambda z: z.transpose(1, 2).float().contiguous()  # noqa: E731
        merged, zm = api.lse_merge(out.float(), rows(lse), torch.ones_like(out.float()), torch.zeros_like(rows(lse)))
        assert merged[0, at, 1].isnan().all() and zm[0, at, 1].isnan()
        dq, dk, dv = api.window_attn_bwd(bad, k, v, out, lse, do, W)
        assert api.cp_get_error() == 0
        assert dq[0, at, 1].isnan().all() and dv[0, max(0, at - W + 1):at + 1].isnan().all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(3, 2048, 2048, 8, 8, 64, 1, 1500), (4, 1000, 1300, 16, 8, 128, 100, 900)])
def test_so_many_sinks_that_their_pieces_are_few(cuda_dev, dtype, shape):
    """The rows behind the window go in fewer and longer pieces than a window's units are."""
    check(shape, dtype, *make(shape, dtype, cuda_dev))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("S,Hq,Hkv,D,W,K,cuts", [(1200, 4, 2, 64, 200, 5, (0, 300, 600, 900, 1200)),
                                                 (1000, 2, 2, 128, 130, 70, (0, 64, 65, 500, 1000)),
                                                 (700, 4, 1, 64, 1, 0, (0, 350, 700))])
def test_ranks_behind_their_halo_make_up_the_whole_gradient(cuda_dev, dtype, S, Hq, Hkv, D, W, K, cuts):
    """Each rank's k and v are the sinks' rows, the window - 1 rows before its shard and the shard.  Its dQ rows are the
    whole's, and dK and dV, sent back to where the rows came from and added up, too: each rank's within what its own call may
    be off, and so their sum within the sum of that."""
    q, k, v, do = make((2, S, S, Hq, Hkv, D, W, K), dtype, cuda_dev)
    whole, _ = ref.backward(q, k, v, do, W, K, None, UNIT[dtype])
    sums = [torch.zeros_like(x) for x in whole]
    errs = [torch.zeros_like(x) for x in whole]
    for a, b in zip(cuts, cuts[1:]):
        lo = max(0, a - W + 1)
        rows = torch.cat([torch.arange(min(K, lo)), torch.arange(lo, b)]).to(cuda_dev)
        mine = torch.arange(a, b, device=cuda_dev)
        args = [q[:, mine].contiguous(), k[:, rows].contiguous(), v[:, rows].contiguous()]
        out, lse = api.window_attn_fwd(*args, W, K)
        got = api.window_attn_bwd(*args, out, lse, do[:, mine].contiguous(), W, K)
        assert api.cp_get_error() == 0
        _, err = ref.backward(*args, do[:, mine], W, K, None, UNIT[dtype])
        for i, at in enumerate((mine, rows, rows)):
            sums[i].index_add_(1, at, got[i].double())
            errs[i].index_add_(1, at, err[i])
    for name, x, y, e in zip(("dq", "dk", "dv"), sums, whole, errs):
        ref.within(x, y, e, name)
