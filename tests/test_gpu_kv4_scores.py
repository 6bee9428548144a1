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


def exact(q, k, v, scale):
    """One kv head in 64 bits: q [R, D], k and v [L, D]; out, lse, sum p |v| and scale sum |q| |k| (largest over the tokens)."""
    q, k, v = (t.double() for t in (q, k, v))
    s = scale * q @ k.T
    z = s.logsumexp(-1)
    p = (s - z[:, None]).exp()
    return p @ v, z, p @ v.abs(), (scale * q.abs() @ k.abs().T).amax(-1)


def close(out, lse, q, k, v, scale):
    """fp32 outputs [R, D] within what the roundings allow.  With A = sum p |v|: weights and values to fp16, 2^-11 of
    themselves each; a weight below fp16's normal range 2^-25, and the row's largest is at least 2^7, so 2^-32 of it; a value
    there 2^-25; fp32 accumulation 2^-23 per 16 tokens and per join; a score is off by up to 2^-19 of scale sum |q| |k|,
    which moves a weight and the sum by that."""
    want, z, a, b = exact(q, k, v, scale)
    L = k.shape[0]
    rel = 2.0 ** -10 + 2.0 ** -22 + (L / 16 + 32) * 2.0 ** -23 + 2 * 2.0 ** -19 * b[:, None]
    top = (scale * q.double() @ k.double().T).amax(-1, keepdim=True)
    largest = (top - z[:, None]).exp()                       # the largest weight of a row
    tol = rel * a + L * 2.0 ** -32 * largest * v.abs().max().double() + 2.0 ** -25
    err = (out.double() - want).abs()
    assert (err <= tol).all(), float((err / tol).max())
    assert ((lse.double() - z).abs() <= 2.0 ** -19 * b + 2.0 ** -20 * (z.abs() + 1)).all()


@pytest.mark.parametrize("L,Hkv", [(640, 1), (4096, 2), (16384, 8)])
@pytest.mark.parametrize("D,group", [(64, 2), (128, 4), (64, 12)])
@pytest.mark.parametrize("gap", [12.0, 20.0, 24.0, 26.5, 30.0])
def test_long_tail_behind_large_scores(cuda_dev, D, group, L, Hkv, gap):
    """Every 64th token's score lies 2^gap above the others' and its value is 0: the output is the tail's."""
    g = torch.Generator(device="cuda").manual_seed(int(gap * 2) + L)
    scale = math.log(2)                                      # scores in powers of two: k's first element
    k = torch.zeros(1, L, Hkv, D, device="cuda")
    # constant groups of multiples of 2^-6 below 64: exact in fp16, and exactly what the cache holds
    k[..., :32] = torch.randint(0, 64, (1, L, Hkv, 1), generator=g, device="cuda") / 64.0
    sink = torch.arange(L, device="cuda") % 64 == 37
    k[:, sink] = 0
    k[:, sink, :, :32] = gap + 1.0
    v = 1 + torch.randint(0, 64, (1, L, Hkv, 1), generator=g, device="cuda").float() / 64 + torch.zeros(D, device="cuda")
    v[:, sink] = 0
    q = torch.zeros(1, 1, group * Hkv, D, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    cache, pages, lens = cached(k, v)
    kr, vr = api.kv4_gather(cache, pages, lens, L, dtype=torch.float32)
    assert torch.equal(kr, k) and torch.equal(vr, v)
    out = torch.empty(1, 1, group * Hkv, D, device="cuda")
    _, lse = api.kv4_attn(q, cache, pages, lens, scale=scale, out=out)
    torch.cuda.synchronize()
    assert api.cp_get_error() == 0
    for h in range(Hkv):
        want = exact(q[0, 0, h * group:(h + 1) * group], k[0, :, h], v[0, :, h], scale)[0]
        got = out[0, 0, h * group:(h + 1) * group]
        # values of 1 to 2 are fp16, and the scores are exact: a tail weight of 2^-t of the sink's, at most 2^(7 - t)
        # beside 2^7 for the sink, is off by 2^-11 or, below 2^-14, by 2^(t - 32) of itself; t <= gap + 1; and the fp32
        # sums of weights and of values
        t = 2.0 ** -11 + 2.0 ** (gap + 1 - 32) + 2 * (L / 16 + 32) * 2.0 ** -23
        assert ((got.double() - want).abs() <= t * want).all(), float(((got.double() - want).abs() / (t * want)).max())
        close(got, lse[0, h * group:(h + 1) * group, 0], q[0, 0, h * group:(h + 1) * group], k[0, :, h], v[0, :, h], scale)


@pytest.mark.parametrize("L", [500, 5000, 40000])
@pytest.mark.parametrize("D,group,size", [(64, 3, 0.2), (128, 8, 1.0), (128, 5, 4.0)])
def test_error_does_not_grow_with_the_length(cuda_dev, D, group, size, L):
    """Random rows, flat to sharp softmax, against the bound counted from the roundings."""
    g = torch.Generator(device="cuda").manual_seed(L + D)
    k, v = (torch.randn(1, L, 2, D, generator=g, device="cuda") for _ in range(2))
    q = (torch.randn(1, 1, 2 * group, D, generator=g, device="cuda") * size).bfloat16()
    cache, pages, lens = cached(k, v)
    kr, vr = api.kv4_gather(cache, pages, lens, L, dtype=torch.float32)
    out = torch.empty(1, 1, 2 * group, D, device="cuda")
    _, lse = api.kv4_attn(q, cache, pages, lens, out=out)
    torch.cuda.synchronize()
    assert api.cp_get_error() == 0
    for h in range(2):
        at = slice(h * group, (h + 1) * group)
        close(out[0, 0, at], lse[0, at, 0], q[0, 0, at], kr[0, :, h], vr[0, :, h], D ** -0.5)
