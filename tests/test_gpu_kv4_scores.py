"""kv4_attn at the ends of the score and weight range: scores so large that neighbouring floats lie 16 apart, and
long tails of small weights behind one large one."""
import math

import numpy as np
import pytest
import torch

from context_parallelism_02_gb300 import api

pytestmark = pytest.mark.gpu


def cached(k, v, page=64):
    """A pool holding the rows k, v [1, L, H, D]; its table and length."""
    L, H, D = k.shape[1:]
    M = -(-L // page)
    cache = api.kv4_cache(M, H, page, D)
    pages = torch.arange(M, dtype=torch.int32, device="cuda")[None]
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.kv4_append(k, v, cache, pages, lens)
    return cache, pages, lens + L


@pytest.mark.parametrize("L", [700, 6000])
@pytest.mark.parametrize("D,group", [(64, 1), (64, 9), (128, 4), (128, 16)])
def test_scores_whose_neighbours_are_far_apart(cuda_dev, D, group, L):
    """Scores of 2^27 + 16 i: 8 more than an odd multiple of 16 rounds to the next one, so a score that is 16 above the
    reference must not pass for one within 8 of it.  Values of 1: whatever the weights, the output is 1."""
    scale = float(np.float32(1) / np.float32(1.44269504088896340736))      # its product with log2(e) rounds to 1
    k = torch.zeros(1, L, 1, D, device="cuda")
    k[..., :32] = 1.0
    # one q element of 2^27, one of 16: scores in powers of two are 2^27 + 16 (1, 2 or 3) in runs of 32 tokens
    k[..., 32:64] = (torch.arange(L, device="cuda") // 32 % 3 + 1).float()[None, :, None, None]
    q = torch.zeros(1, 1, group, D, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 2.0 ** 27
    q[..., 32] = 16.0
    cache, pages, lens = cached(k.bfloat16(), torch.ones_like(k).bfloat16())
    out, lse = api.kv4_attn(q, cache, pages, lens, scale=scale)
    torch.cuda.synchronize()
    assert api.cp_get_error() == 0
    assert (out == 1).all()
    # the largest score 2^27 + 48, in fp32 (spacing 8 in natural units: one for the score, one for the sum)
    assert (lse.double() - (2.0 ** 27 + 48) * math.log(2)).abs().max() <= 3 * 8
