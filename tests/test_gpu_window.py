"""Windowed attention with sinks on the GPU against the definition in 64 bits."""
import itertools

import pytest
import torch

from context_parallelism_02_gb300 import _lib, api
from oracle import window as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
UNIT = {BF16: 2.0 ** -8, F32: 2.0 ** -24}

# B, Sq, Sk, Hq, Hkv, D, window, sinks: rows and windows around the tiles of 64, 128 and
# 256, windows of one token and beyond the prompt, sinks that share the first tile (up to
# 64), that have tiles of their own, that meet the window and that cover everything, chunks
SHAPES = [
    (1, 1, 1, 1, 1, 64, 1, 0),
    (1, 1, 1000, 2, 1, 128, 300, 4),
    (1, 64, 64, 1, 1, 64, 16, 0),
    (2, 128, 128, 2, 1, 128, 32, 4),
    (1, 129, 129, 2, 2, 128, 128, 1),
    (1, 300, 300, 2, 2, 128, 100, 16),
    (2, 513, 700, 4, 2, 64, 77, 20),
    (1, 640, 640, 1, 1, 128, 127, 17),
    (1, 1000, 1000, 3, 1, 128, 1, 1),
    (1, 1000, 1000, 2, 1, 64, 2, 0),
    (1, 1000, 1000, 2, 1, 128, 2000, 3),
    (1, 777, 777, 2, 2, 128, 129, 65),
    (1, 900, 1200, 2, 1, 64, 200, 130),
    (1, 1500, 1500, 2, 1, 64, 256, 600),
    (1, 700, 700, 1, 1, 128, 90, 5000),
    (1, 100, 2000, 4, 4, 128, 513, 64),
    (1, 2048, 2048, 8, 2, 128, 500, 64),
]


def make(shape, dtype, dev, seed=0):
    B, Sq, Sk, Hq, Hkv, D, _, _ = shape
    g = torch.Generator(device=dev).manual_seed(seed + 7 * Sq + Sk)
    r = lambda s, h: torch.randn(B, s, h, D, generator=g, device=dev).to(dtype)  # noqa: E731
    return r(Sq, Hq), r(Sk, Hkv), r(Sk, Hkv), r(Sq, Hq)


def check(shape, dtype, q, k, v, do, scale=None):
    W, K = shape[-2:]
    out, lse = api.window_attn_fwd(q, k, v, W, K, scale)
    grads = api.window_attn_bwd(q, k, v, out, lse, do, W, K, scale)
    assert api.cp_get_error() == 0
    o, z, eo, ez = ref.forward(q, k, v, W, K, scale, UNIT[dtype])
    ref.within(out, o, eo, "out")
    ref.within(lse, z, ez, "lse")
    want, err = ref.backward(q, k, v, do, W, K, scale, UNIT[dtype])
    for name, x, y, e in zip(("dq", "dk", "dv"), grads, want, err):
        ref.within(x, y, e, name)
    return out, lse, grads


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_gradients(cuda_dev, shape, dtype):
    check(shape, dtype, *make(shape, dtype, cuda_dev))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scale(cuda_dev, dtype):
    shape = (1, 260, 260, 2, 1, 64, 70, 4)
    check(shape, dtype, *make(shape, dtype, cuda_dev), scale=0.31)


def test_window_beyond_the_prompt_is_causal_attention(cuda_dev):
    """The plain ring call gives the same values but for the order of sums."""
    shape = (1, 1024, 1024, 4, 2, 128, 1 << 40, 0)
    q, k, v, do = make(shape, BF16, cuda_dev)
    out, lse, grads = check(shape, BF16, q, k, v, do)
    o2, z2 = api.ring_attn_fwd(q, k, v, 1, 0, True)
    assert (lse - z2).abs().max() <= 1e-5
    assert (out.float() - o2.float()).abs().max() <= 2.0 ** -6 * o2.float().abs().max()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_chunks_make_up_the_whole(cuda_dev, dtype):
    """A prompt in chunks, each with its sinks, halo and own rows alone as k and v."""
    S, W, K = 1200, 150, 7
    q, k, v, _ = make((1, S, S, 4, 2, 128, W, K), dtype, cuda_dev)
    whole, lse = api.window_attn_fwd(q, k, v, W, K)
    o, z, eo, ez = ref.forward(q, k, v, W, K, None, UNIT[dtype])
    ref.within(whole, o, eo, "whole")
    for a, b in ((0, 100), (100, 500), (500, 501), (501, 1200)):
        lo = max(0, a - W + 1)
        rows = torch.cat([torch.arange(min(K, lo)), torch.arange(lo, b)]).to(cuda_dev)
        out, zc = api.window_attn_fwd(q[:, a:b].contiguous(), k[:, rows].contiguous(), v[:, rows].contiguous(), W, K)
        ref.within(out, o[:, a:b], eo[:, a:b], (a, b))
        ref.within(zc, z[..., a:b], ez[..., a:b], (a, b))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_repeats_bit_for_bit(cuda_dev, dtype):
    shape = (2, 900, 900, 4, 1, 64, 100, 6)
    q, k, v, do = make(shape, dtype, cuda_dev)
    runs = []
    for _ in range(2):
        out, lse = api.window_attn_fwd(q, k, v, 100, 6)
        runs.append((out, lse, *api.window_attn_bwd(q, k, v, out, lse, do, 100, 6)))
    assert all(torch.equal(a, b) for a, b in zip(*runs))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_units_of_one_block(cuda_dev, dtype):
    """Few blocks, each with many units of work: the barriers' running phases."""
    shape = (1, 1000, 1000, 6, 3, 128, 200, 4)
    q, k, v, do = make(shape, dtype, cuda_dev)
    plain = api.window_attn_fwd(q, k, v, 200, 4)
    api.cp_debug_set_grid_limit(2)
    try:
        few = api.window_attn_fwd(q, k, v, 200, 4)
        torch.cuda.synchronize()
    finally:
        api.cp_debug_set_grid_limit(0)
    assert all(torch.equal(a, b) for a, b in zip(plain, few))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_buffers_of_the_caller_and_their_neighbours(cuda_dev, dtype):
    """Outputs in the middle of larger buffers: what lies around them stays."""
    shape = (2, 200, 331, 4, 2, 64, 60, 5)
    q, k, v, do = make(shape, dtype, cuda_dev)

    def guarded(like):
        big = torch.full((like.numel() + 512,), 7.0, dtype=like.dtype, device=cuda_dev)
        return big, big[256:256 + like.numel()].view(like.shape)
    lse0 = torch.empty(2, 4, 200, device=cuda_dev)
    bufs = [guarded(t) for t in (q, lse0, q, k, v)]
    out, lse, dq, dk, dv = (b[1] for b in bufs)
    assert api.window_attn_fwd(q, k, v, 60, 5, out=out, lse=lse)[0] is out
    n = api.window_attn_bwd_workspace(2, 4, 2, 200, 331, 64, 60, 5, dtype)
    ws = torch.full((n + 512,), 77, dtype=torch.uint8, device=cuda_dev)
    api.window_attn_bwd(q, k, v, out, lse, do, 60, 5, dq=dq, dk=dk, dv=dv, workspace=ws[256:256 + n])
    torch.cuda.synchronize()
    for big, _ in bufs:
        assert (big[:256] == 7).all() and (big[-256:] == 7).all()
    assert (ws[:256] == 77).all() and (ws[-256:] == 77).all()
    want, err = ref.backward(q, k, v, do, 60, 5, None, UNIT[dtype])
    for x, y, e in zip((dq, dk, dv), want, err):
        ref.within(x, y, e, "gradient")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_on_a_stream_and_captured(cuda_dev, dtype):
    shape = (1, 500, 500, 2, 1, 128, 120, 4)
    q, k, v, do = make(shape, dtype, cuda_dev)
    want = api.window_attn_fwd(q, k, v, 120, 4)
    want += api.window_attn_bwd(q, k, v, *want, do, 120, 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = api.window_attn_fwd(q, k, v, 120, 4, stream=s)
    got += api.window_attn_bwd(q, k, v, *got, do, 120, 4, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    g = torch.cuda.CUDAGraph()
    ins = [t.clone() for t in (q, k, v, do)]
    with torch.cuda.graph(g):
        o, z = api.window_attn_fwd(*ins[:3], 120, 4)
        gr = api.window_attn_bwd(*ins[:3], o, z, ins[3], 120, 4)
    for t in ins:
        t.normal_()
    g.replay()
    fresh = api.window_attn_fwd(*ins[:3], 120, 4)
    fresh += api.window_attn_bwd(*ins[:3], *fresh, ins[3], 120, 4)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((o, z, *gr), fresh))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradients_against_differences(cuda_dev, dtype):
    """sum(dout * out) of the definition changes along random directions as the gradients say."""
    shape = (1, 150, 180, 2, 1, 64, 40, 5)
    q, k, v, do = make(shape, dtype, cuda_dev)
    out, lse = api.window_attn_fwd(q, k, v, 40, 5)
    grads = api.window_attn_bwd(q, k, v, out, lse, do, 40, 5)
    errs = ref.backward(q, k, v, do, 40, 5, None, UNIT[dtype])[1]
    h = 1e-4
    for i, (x, g, e) in enumerate(zip((q, k, v), grads, errs)):
        d = torch.randn_like(x.double())
        f = []
        for sign in (1, -1):
            args = [t.double() for t in (q, k, v)]
            args[i] = args[i] + sign * h * d
            f.append(float((do.double() * ref.forward(*args, 40, 5)[0]).sum()))
        diff = (f[0] - f[1]) / (2 * h)
        # third derivatives times h^2: 1e-8 of terms of order one per element
        assert abs(diff - float((g.double() * d).sum())) <= float((e * d.abs()).sum()) + 1e-6 * x.numel() ** 0.5


def test_lse_merges_with_other_parts(cuda_dev):
    """Two windows over disjoint keys: the parts joined by lse_merge are the whole."""
    S, D = 256, 64
    q, k, v, _ = make((1, S, S, 2, 2, D, S, 0), F32, cuda_dev)
    near, zn = api.window_attn_fwd(q, k, v, 64, 0)
    see = ref.visible(S, S, S, 0, cuda_dev) & ~ref.visible(S, S, 64, 0, cuda_dev)
    Q, K, V = (ref.heads(t, 2) for t in (q, k, v))
    s = (Q @ K.transpose(-1, -2) / D ** 0.5).masked_fill(~see, -torch.inf)
    zf = s.logsumexp(-1)
    far = (torch.exp(s - zf.masked_fill(zf == -torch.inf, 0)[..., None]) @ V).permute(0, 2, 1, 3).float().contiguous()
    rows = lambda z: z.transpose(1, 2).float().contiguous()  # noqa: E731
    out, z = api.lse_merge(near, rows(zn), far, rows(zf))
    o, zr, eo, ez = ref.forward(q, k, v, S, 0, None, 2.0 ** -22)
    ref.within(out, o, eo, "out")
    ref.within(z.transpose(1, 2), zr, ez + 1e-6, "lse")


def test_refusals(cuda_dev):
    q, k, v, do = make((1, 64, 64, 2, 1, 64, 8, 0), BF16, cuda_dev)
    out, lse = api.window_attn_fwd(q, k, v, 8)
    for bad in (dict(window=0), dict(window=-3), dict(window=8, sinks=-1), dict(window=8, scale=float("nan"))):
        with pytest.raises(api.CpError) as e:
            api.window_attn_fwd(q, k, v, **bad)
        assert e.value.code == _lib.CP_EINVAL
        with pytest.raises(api.CpError):
            api.window_attn_bwd(q, k, v, out, lse, do, **bad)
    with pytest.raises(api.CpError):                       # more rows than keys
        api.window_attn_fwd(q, k[:, :32].contiguous(), v[:, :32].contiguous(), 8)
    with pytest.raises(api.CpError):
        api.window_attn_fwd(q[..., :32].contiguous(), k[..., :32].contiguous(), v[..., :32].contiguous(), 8)
    with pytest.raises(api.CpError):                       # a workspace that is too small
        api.window_attn_bwd(q, k, v, out, lse, do, 8, workspace=torch.empty(64, dtype=torch.uint8, device=cuda_dev))
    for args in ((q.half(), k.half(), v.half()), (q, k.float(), v), (q[:, ::2], k, v), (q, k, v[:, :32].contiguous()),
                 (q[0], k, v), (q.cpu(), k, v), (q, k.cpu(), v)):
        with pytest.raises(ValueError):
            api.window_attn_fwd(*args, 8)
    for kw in (dict(out=out.float()), dict(out=out[:, :32]), dict(lse=lse.double()), dict(lse=lse[:, :1])):
        with pytest.raises(ValueError):
            api.window_attn_fwd(q, k, v, 8, **kw)
    with pytest.raises(api.CpError):                       # outputs over inputs
        api.window_attn_fwd(q, k, v, 8, out=q)
    for kw in (dict(dq=q), dict(dq=do), dict(dk=v), dict(dk=k), dict(dv=k)):
        with pytest.raises(api.CpError):
            api.window_attn_bwd(q, k, v, out, lse, do, 8, **kw)
    both = torch.empty_like(k)
    with pytest.raises(api.CpError):
        api.window_attn_bwd(q, k, v, out, lse, do, 8, dk=both, dv=both)
    for kw in (dict(dq=k), dict(dk=q), dict(dv=v.float())):
        with pytest.raises(ValueError):
            api.window_attn_bwd(q, k, v, out, lse, do, 8, **kw)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_nothing_to_do(cuda_dev, dtype):
    """No batch, no rows: empty results, and keys that no row sees have gradients of zero."""
    z = lambda *s: torch.zeros(*s, dtype=dtype, device=cuda_dev)  # noqa: E731
    out, lse = api.window_attn_fwd(z(0, 5, 2, 64), z(0, 9, 2, 64), z(0, 9, 2, 64), 4)
    assert out.shape == (0, 5, 2, 64) and lse.shape == (0, 2, 5)
    q, k = z(2, 0, 2, 64), torch.randn(2, 9, 2, 64, device=cuda_dev).to(dtype)
    out, lse = api.window_attn_fwd(q, k, k, 4)
    dq, dk, dv = api.window_attn_bwd(q, k, k, out, lse, q, 4)
    assert dq.numel() == 0 and not dk.any() and not dv.any()


@pytest.mark.parametrize("dtype,D", list(itertools.product([F32, BF16], [64, 128])))
def test_misaligned_to_32_bytes(cuda_dev, dtype, D):
    """Outputs that start on a 16-byte boundary that is no 32-byte one."""
    q, k, v, _ = make((1, 200, 200, 2, 1, D, 50, 3), dtype, cuda_dev)
    e = 16 // q.element_size()
    out = torch.empty(q.numel() + e, dtype=dtype, device=cuda_dev)[e:].view(q.shape)
    api.window_attn_fwd(q, k, v, 50, 3, out=out)
    assert torch.equal(out, api.window_attn_fwd(q, k, v, 50, 3)[0])


@pytest.mark.parametrize("shape", [(1, 1000, 1000, 6, 3, 128, 200, 4), (2, 200, 2000, 4, 2, 64, 130, 300),
                                   (1, 300, 900, 2, 1, 128, 1, 70)])
def test_backward_with_many_units_of_one_block(cuda_dev, shape):
    """Few blocks with many units each, units without any row among them."""
    q, k, v, do = make(shape, BF16, cuda_dev)
    W, K = shape[-2:]
    out, lse = api.window_attn_fwd(q, k, v, W, K)
    plain = api.window_attn_bwd(q, k, v, out, lse, do, W, K)
    api.cp_debug_set_grid_limit(2)
    try:
        few = api.window_attn_bwd(q, k, v, out, lse, do, W, K)
        assert api.cp_get_error() == 0
    finally:
        api.cp_debug_set_grid_limit(0)
    assert all(torch.equal(a, b) for a, b in zip(plain, few))


BADS = [float("nan"), float("inf")]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", BADS)
@pytest.mark.parametrize("shape", [(1, 200, 700, 2, 1, 64, 100, 4), (2, 300, 900, 4, 2, 128, 130, 70), (1, 129, 500, 2, 2, 128, 1, 0)])
def test_keys_that_no_row_sees_may_hold_anything(cuda_dev, shape, dtype, bad):
    """A chunk whose earlier rows, outside windows and sinks, are not finite."""
    B, Sq, Sk, Hq, Hkv, D, W, K = shape
    q, k, v, do = make(shape, dtype, cuda_dev)
    unseen = ~ref.visible(Sq, Sk, W, K, cuda_dev).any(0)
    assert unseen.sum() > 100
    clean = [t.masked_fill(unseen[None, :, None, None], 0) for t in (k, v)]
    for which in (0, 1, 2):
        kk, vv = (t.clone() for t in clean)
        if which != 1:
            kk[:, unseen] = bad
        if which != 0:
            vv[:, unseen] = -bad
        out, lse = api.window_attn_fwd(q, kk, vv, W, K)
        grads = api.window_attn_bwd(q, kk, vv, out, lse, do, W, K)
        assert api.cp_get_error() == 0
        o, z, eo, ez = ref.forward(q, *clean, W, K, None, UNIT[dtype])
        ref.within(out, o, eo, "out")
        ref.within(lse, z, ez, "lse")
        want, err = ref.backward(q, *clean, do, W, K, None, UNIT[dtype])
        for name, x, y, e in zip(("dq", "dk", "dv"), grads, want, err):
            ref.within(x, y, e, name)
        assert not grads[1][:, unseen].any() and not grads[2][:, unseen].any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", BADS)
def test_padding_behind_the_rows_may_hold_anything(cuda_dev, dtype, bad):
    shape = (2, 520, 520, 4, 2, 128, 90, 4)
    q, k, v, _ = make(shape, dtype, cuda_dev)
    o, z, eo, ez = ref.forward(q, k, v, 90, 4, None, UNIT[dtype])
    for n in (1, 130, 300, 519):
        qq, kk, vv = (t.clone() for t in (q, k, v))
        for t in (qq, kk, vv):
            t[:, n:] = bad
        out, lse = api.window_attn_fwd(qq, kk, vv, 90, 4)
        assert api.cp_get_error() == 0
        ref.within(out[:, :n], o[:, :n], eo[:, :n], n)
        ref.within(lse[..., :n], z[..., :n], ez[..., :n], n)
        assert not torch.isfinite(out[:, n:]).any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("at", [0, 150, 383, 699])
def test_a_row_that_is_not_finite_reaches_the_gradients_of_its_keys_alone(cuda_dev, dtype, at):
    shape = (1, 700, 700, 4, 2, 64, 60, 5)
    q, k, v, do = make(shape, dtype, cuda_dev)
    out, lse = api.window_attn_fwd(q, k, v, 60, 5)
    see = ref.visible(700, 700, 60, 5, cuda_dev)[at]
    gone = do.clone()
    gone[:, at] = 0
    want, err = ref.backward(q, k, v, gone, 60, 5, None, UNIT[dtype])
    broken = do.clone()
    broken[:, at] = float("nan")
    dq, dk, dv = api.window_attn_bwd(q, k, v, out, lse, broken, 60, 5)
    assert api.cp_get_error() == 0
    rest = torch.arange(700, device=cuda_dev) != at
    ref.within(dq[:, rest], want[0][:, rest], err[0][:, rest], "dq")
    ref.within(dk[:, ~see], want[1][:, ~see], err[1][:, ~see], "dk")
    ref.within(dv[:, ~see], want[2][:, ~see], err[2][:, ~see], "dv")
    assert dq[:, at].isnan().all() and dk[:, see].isnan().all() and dv[:, see].isnan().all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", BADS)
@pytest.mark.parametrize("which", ["q", "k", "v"])
def test_one_row_that_is_not_finite(cuda_dev, dtype, bad, which):
    """A row of q, k or v with NaN or infinities throughout: rows that see it are not finite (for q, k: their lse
    as well), rows that do not are as without it, and so are the gradients of what no such row sees."""
    S, at, W, K = 500, 260, 70, 5
    shape = (1, S, S, 4, 2, 64, W, K)
    q, k, v, do = make(shape, dtype, cuda_dev)
    o, z, eo, ez = ref.forward(q, k, v, W, K, None, UNIT[dtype])
    see = ref.visible(S, S, W, K, cuda_dev)
    hit = see[:, at] if which != "q" else torch.arange(S, device=cuda_dev) == at    # rows
    broken = [t.clone() for t in (q, k, v)]
    broken["qkv".index(which)][:, at] = bad
    out, lse = api.window_attn_fwd(*broken, W, K)
    ref.within(out[:, ~hit], o[:, ~hit], eo[:, ~hit], "out")
    ref.within(lse[..., ~hit], z[..., ~hit], ez[..., ~hit], "lse")
    assert not torch.isfinite(out[:, hit]).any()
    if which == "v":
        ref.within(lse, z, ez, "lse")
    else:
        assert lse[..., hit].isnan().all()
    far = ~see[hit].any(0)                                    # keys that no such row sees
    gone = do.clone()
    gone[:, hit] = 0
    want, err = ref.backward(q, k, v, gone, W, K, None, UNIT[dtype])
    dq, dk, dv = api.window_attn_bwd(*broken, out, lse, do, W, K)
    assert api.cp_get_error() == 0
    ref.within(dq[:, ~hit], want[0][:, ~hit], err[0][:, ~hit], "dq")
    ref.within(dk[:, far], want[1][:, far], err[1][:, far], "dk")
    ref.within(dv[:, far], want[2][:, far], err[2][:, far], "dv")
    assert dq[:, hit].isnan().all()


@pytest.mark.parametrize("S,W,K", [(1500, 2, 0), (1500, 3, 1), (1500, 17, 0), (1500, 63, 0), (1500, 64, 0), (1500, 8, 30),
                                   (300, 300, 0), (1200, 1200, 0)])
def test_gradients_of_rows_that_see_few_keys(cuda_dev, S, W, K):
    """dQ and dK are off by two roundings to bf16, of dS and of the result, each as large as the other relative to
    the norm, and independent: sqrt(2) of one of them.  What out's rounding leaves in Delta adds at most 2^-9 sqrt(sum P^2)
    of the rows' share, sum P^2 about e / 64 where 64 keys are seen: sqrt(2 + e / 64) = 1.43; 1.5 leaves 5 % for the
    spread of norms over 10^5 elements."""
    q, k, v, do = make((2, S, S, 4, 2, 64, W, K), BF16, cuda_dev)
    out, lse = api.window_attn_fwd(q, k, v, W, K)
    grads = api.window_attn_bwd(q, k, v, out, lse, do, W, K)
    for x, y in zip(grads[:2], ref.backward(q, k, v, do, W, K)[0]):
        assert (x.double() - y).norm() <= 1.5 * (y.bfloat16().double() - y).norm()
