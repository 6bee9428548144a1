"""Forms of the kv4 calls that the documentation allows: selection under vis and without causality, buffers of the
caller's own with any contents, wide tables, one process calling from two threads."""
import math
import threading

import numpy as np
import pytest
import torch

from context_parallelism_02_gb300 import api
from oracle import kv4 as o

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


def pool(seed, B, L, Hkv, D, page, width=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    M = -(-L // page)
    P = B * M + 1
    cache, summ = api.kv4_cache(P, Hkv, page, D, summary=True)
    pages = torch.full((B, width or M), -1, **I32)
    pages[:, :M] = torch.randperm(P, generator=g, device="cuda")[:B * M].reshape(B, M).int()
    k, v = (torch.randn(B, L, Hkv, D, generator=g, device="cuda") for _ in range(2))
    api.kv4_append(k, v, cache, pages, torch.zeros(B, **I32), summary=summ)
    return cache, summ, pages, g


def done():
    torch.cuda.synchronize()
    assert api.cp_get_error() == 0


@pytest.mark.parametrize("mode", ["vis", "all"])
@pytest.mark.parametrize("D,page,Hq,Hkv,n,n_sel,first,last", [(64, 16, 6, 2, 3, 5, 1, 2), (128, 256, 4, 4, 2, 2, 0, 0),
                                                              (64, 32, 17, 1, 4, 40, 3, 1)])
def test_select_under_vis_and_without_causality(cuda_dev, mode, D, page, Hq, Hkv, n, n_sel, first, last):
    """Small integers: bounds are exact, so the pages must be equal; attention over them, against the read-back."""
    rng = np.random.default_rng(D + n)
    B, M = 2, 12
    L = M * page
    cache, _, pages, _ = pool(1, B, L, Hkv, D, page)
    P = cache.shape[0]
    box = np.sort(rng.integers(-30, 31, (P, Hkv, 2, D)).astype(np.float32), 2)
    q = rng.integers(-8, 9, (B, n, Hq, D)).astype(np.float32)
    lens = np.array([L, L // 2 + 3], np.int32)
    vis = rng.integers(-2, L + 40, (B, n)).astype(np.int32)
    vis[0, 0], vis[1, 0] = 0, 1
    gq = torch.from_numpy(q).cuda().bfloat16()
    kw = dict(vis=torch.from_numpy(vis).cuda()) if mode == "vis" else dict(causal=False)
    gl = torch.from_numpy(lens).cuda()
    sel = api.kv4_select(gq, torch.from_numpy(box).cuda().bfloat16(), pages, gl, page, n_sel, keep_first=first, keep_last=last,
                         **kw)
    gq2 = (gq / 16).contiguous()
    f32 = torch.empty(B, n, Hq, D, device="cuda")
    _, lse = api.kv4_attn(gq2, cache, pages, gl, sel=sel, out=f32, **kw)
    kr, vr = api.kv4_gather(cache, pages, gl, L, dtype=torch.float32)
    done()
    got, table, r = sel.cpu().numpy(), pages.cpu().numpy(), Hq // Hkv
    for b in range(B):
        for j in range(n):
            lim = int(np.clip(vis[b, j], 0, lens[b])) if mode == "vis" else int(lens[b])
            m = -(-lim // page)
            for h in range(Hkv):
                t = box[table[b, :m], h]
                want = o.select(q[b, j, h * r:(h + 1) * r], t[:, 0], t[:, 1], n_sel, first, last)
                np.testing.assert_array_equal(got[b, j, h], want)
                at = [p * page + s for p in want if p >= 0 for s in range(page) if p * page + s < lim]
                kk, vv = kr[b, at, h].cpu().numpy(), vr[b, at, h].cpu().numpy()
                for x in range(h * r, (h + 1) * r):
                    ref, z, a = o.attend(gq2[b, j, x].float().cpu().numpy(), kk, vv, D ** -0.5)
                    if not at:
                        assert (f32[b, j, x] == 0).all() and lse[b, x, j] == -math.inf
                        continue
                    # weights and values rounded to fp16, fp32 sums; a score off by 2^-19 of its terms
                    e = 2.0 ** -19 * D ** -0.5 * float(np.abs(gq2[b, j, x].float().cpu().numpy()) @ np.abs(kk).max(0))
                    tol = (2.0 ** -10 + 2 * e + (len(at) / 16 + 32) * 2.0 ** -23) * a + 2.0 ** -25 * (1 + len(at) * 2.0 ** -7)
                    assert (np.abs(f32[b, j, x].double().cpu().numpy() - ref) <= tol).all()
                    assert abs(lse[b, x, j].item() - z) <= e + 2.0 ** -20 * (abs(z) + 1)


@pytest.mark.parametrize("B,L", [(1, 9000), (5, 3000), (3, 500)])
def test_buffers_of_the_callers_own(cuda_dev, B, L):
    """Workspaces, outputs and lists that hold NaN or old numbers before the call."""
    cache, summ, pages, g = pool(2, B, L, 2, 128, 64)
    lens = torch.tensor([L - 41 * b for b in range(B)], **I32)
    q = torch.randn(B, 1, 8, 128, generator=g, device="cuda").bfloat16()
    sel = api.kv4_select(q, summ, pages, lens, 64, 4)
    out, lse = api.kv4_attn(q, cache, pages, lens)
    ws = torch.full((api.kv4_attn_workspace(128),), 255, dtype=torch.uint8, device="cuda")
    ws2 = torch.full((api.kv4_select_workspace(B, 1, 2, pages.shape[1]),), 255, dtype=torch.uint8, device="cuda")
    sel2 = torch.full_like(sel, 99)
    assert api.kv4_select(q, summ, pages, lens, 64, 4, sel=sel2, workspace=ws2) is not None
    mine, z = torch.full_like(out, math.nan), torch.full_like(lse, math.nan)
    api.kv4_attn(q, cache, pages, lens, out=mine, lse=z, workspace=ws)
    done()
    assert torch.equal(sel, sel2) and torch.equal(mine, out) and torch.equal(z, lse)
    k, v = api.kv4_gather(cache, pages, lens, 70, start=lens - 60)
    k2, v2 = torch.full_like(k, math.nan), torch.full_like(v, math.nan)
    api.kv4_gather(cache, pages, lens, 70, start=lens - 60, k=k2, v=v2)
    done()
    assert torch.equal(k, k2) and torch.equal(v, v2) and (k2[:, 60:] == 0).all()


@pytest.mark.parametrize("lens", [[500], [3000, 17, 1, 0], [64] * 40])
def test_tables_wider_than_the_sequences(cuda_dev, lens):
    """A table for a far longer context takes other kernels, not other results: both against the read-back."""
    B, L = len(lens), max(lens)
    gl = torch.tensor(lens, **I32)
    outs = []
    for width in (-(-L // 64), 5000):
        cache, summ, pages, g = pool(3, B, L, 2, 128, 64, width)
        q = torch.randn(B, 2, 6, 128, generator=g, device="cuda").bfloat16()
        f32 = torch.empty(B, 2, 6, 128, device="cuda")
        _, lse = api.kv4_attn(q, cache, pages, gl, out=f32)
        sel = api.kv4_select(q, summ, pages, gl, 64, 3)
        kr, vr = api.kv4_gather(cache, pages, gl, L, dtype=torch.float32)
        done()
        for b, m in enumerate(lens):
            for j in range(2):
                lim = max(0, m - 1 + j)
                if not lim:
                    assert (f32[b, j] == 0).all() and (lse[b, :, j] == -math.inf).all()
                    continue
                for x in range(6):
                    ref, z, a = o.attend(q[b, j, x].float().cpu().numpy(), kr[b, :lim, x // 3].cpu().numpy(),
                                         vr[b, :lim, x // 3].cpu().numpy(), 128 ** -0.5)
                    tol = (2.0 ** -10 + 2.0 ** -13 + (lim / 16 + 32) * 2.0 ** -23) * a + 2.0 ** -25 * (1 + lim * 2.0 ** -7)
                    assert (np.abs(f32[b, j, x].double().cpu().numpy() - ref) <= tol).all()
                    assert abs(lse[b, x, j].item() - z) <= 2.0 ** -14
        outs.append((sel, kr, vr))
    assert all(torch.equal(x, y) for x, y in zip(*outs))


def test_calls_from_two_threads(cuda_dev):
    """Two threads, each with a stream, a pool and a sequence of steps of its own."""
    want, got, errors = {}, {}, []

    def steps(i, into):
        cache, summ, pages, g = pool(10 + i, 2, 2000, 2, 64, 32)
        q = torch.randn(2, 1, 4, 64, generator=g, device="cuda").bfloat16()
        lens = torch.tensor([1900, 300 + i], **I32)
        outs = []
        for _ in range(25):
            k = torch.randn(2, 1, 2, 64, generator=g, device="cuda").bfloat16()
            qr = api.kv4_append(k, k, cache, pages, lens, q=q, summary=summ)
            lens += 1
            sel = api.kv4_select(qr, summ, pages, lens, 32, 6)
            outs += [sel, *api.kv4_attn(qr, cache, pages, lens), *api.kv4_attn(qr, cache, pages, lens, sel=sel)]
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
    done()
    assert not errors
    for i in range(2):
        assert all(torch.equal(x, y) for x, y in zip(want[i], got[i]))


def test_no_gradient(cuda_dev):
    """Inputs that require gradients are taken; what comes back requires none, as the documentation says."""
    cache, summ, pages, g = pool(5, 1, 100, 1, 64, 16)
    k, q = (torch.randn(1, 1, h, 64, generator=g, device="cuda").bfloat16().requires_grad_() for h in (1, 2))
    lens = torch.tensor([40], **I32)
    qr = api.kv4_append(k, k, cache, pages, lens, q=q, summary=summ)
    out, lse = api.kv4_attn(q, cache, pages, lens)
    done()
    assert torch.equal(qr, q) and not (qr.requires_grad or out.requires_grad or lse.requires_grad)
    for f in (api.kv4_append, api.kv4_gather, api.kv4_attn):
        assert "radient" in f.__doc__
