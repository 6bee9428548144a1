"""Windowed attention where a call meets its limits: tensors past 2^32 elements, tile coordinates under the checking
build, waits that run out, two calls at once."""
import threading

import pytest
import torch

from context_parallelism_02_gb300 import CP_ETIMEOUT, _lib, api, build
from oracle import window as ref
from test_gpu_window import BF16, F32, SHAPES, UNIT, check, make

pytestmark = pytest.mark.gpu


def both(q, k, v, do, W, K):
    out, lse = api.window_attn_fwd(q, k, v, W, K)
    return (out, lse, *api.window_attn_bwd(q, k, v, out, lse, do, W, K))


@pytest.fixture(scope="module")
def debug_bounds(cuda_dev):
    build.build(debug_bounds=True)
    with _lib.variant("debug_bounds") as lib:
        assert api.cp_get_error() == 0
        yield lib


@pytest.mark.parametrize("shape", SHAPES)
def test_in_bounds(debug_bounds, cuda_dev, shape):
    """The checking build records a tile coordinate or row outside its tensor as CP_EBOUNDS: there is none."""
    args = make(shape, BF16, cuda_dev)
    plain = check(shape, BF16, *args)
    api.cp_debug_set_grid_limit(3)
    try:
        few = both(*args, *shape[-2:])
        assert api.cp_get_error() == 0
    finally:
        api.cp_debug_set_grid_limit(0)
    assert all(torch.equal(a, b) for a, b in zip((plain[0], plain[1], *plain[2]), few))


@pytest.mark.parametrize("shape", [(1, 2048, 2048, 2, 2, 128, 300, 4), (2, 700, 1500, 4, 2, 64, 130, 200)])
def test_waits_that_run_out(cuda_dev, shape):
    """A status, no hang, and the next call works."""
    q, k, v, do = make(shape, BF16, cuda_dev)
    W, K = shape[-2:]
    want = both(q, k, v, do, W, K)
    assert api.cp_get_error() == 0
    for call in (lambda: api.window_attn_fwd(q, k, v, W, K),
                 lambda: api.window_attn_bwd(q, k, v, want[0], want[1], do, W, K)):
        api.cp_debug_set_wait_limit(1)
        try:
            call()
            assert api.cp_get_error() == CP_ETIMEOUT
        finally:
            api.cp_debug_set_wait_limit(0)
    got = both(q, k, v, do, W, K)
    assert api.cp_get_error() == 0
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("dtype,B,S,Hq,Hkv,D", [(BF16, 9, 65536, 64, 8, 128), (F32, 17, 65536, 32, 4, 128)])
def test_tensors_beyond_2_32_elements(cuda_dev, dtype, B, S, Hq, Hkv, D):
    """The last rows of the last batch and kv head, whose keys are the sinks and the window before them."""
    W, K, n = 500, 70, 300
    g = torch.Generator(device=cuda_dev).manual_seed(5)

    def draw(H):
        x = torch.empty(B, S, H, D, dtype=dtype, device=cuda_dev)
        for b in range(B):
            x[b] = torch.randn(S, H, D, generator=g, device=cuda_dev)
        return x
    q, k, v, do = draw(Hq), draw(Hkv), draw(Hkv), draw(Hq)
    assert q.numel() > 2 ** 32
    out, lse, dq, dk, dv = both(q, k, v, do, W, K)
    assert api.cp_get_error() == 0
    grp = Hq // Hkv
    keys = torch.cat([torch.arange(K), torch.arange(S - n - W + 1, S)]).to(cuda_dev)
    rows = lambda t: t[-1:, -n:, -grp:].contiguous()  # noqa: E731
    cols = lambda t: t[-1:, keys][:, :, -1:].contiguous()  # noqa: E731
    args = rows(q), cols(k), cols(v)
    o, z, eo, ez = ref.forward(*args, W, K, None, UNIT[dtype])
    ref.within(rows(out), o, eo, "out")
    ref.within(lse[-1:, -grp:, -n:], z, ez, "lse")
    want, err = ref.backward(*args, rows(do), W, K, None, UNIT[dtype])
    ref.within(rows(dq), want[0], err[0], "dq")
    for x, y, e in zip((dk, dv), want[1:], err[1:]):          # keys that only these rows see
        ref.within(x[-1:, -n:, -1:], y[:, -n:], e[:, -n:], "dk, dv")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_two_threads_on_streams_of_their_own(cuda_dev, dtype):
    shapes = [(1, 900, 900, 4, 2, 128, 200, 4), (2, 500, 800, 2, 1, 64, 90, 70)]
    args = [make(s, dtype, cuda_dev) for s in shapes]
    want = [both(*a, *s[-2:]) for a, s in zip(args, shapes)]
    torch.cuda.synchronize()
    wrong = []

    def run(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                got = both(*args[i], *shapes[i][-2:])
                s.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(want[i], got)):
                    wrong.append(i)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and api.cp_get_error() == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_tensors_that_are_not_finite_throughout(cuda_dev, bad):
    """Nothing finite is left to compute, and 2^33 visible pairs are not computed one by one."""
    shape = (2, 16384, 16384, 64, 8, 64, 8192, 4)
    q, k, v, do = make(shape, BF16, cuda_dev)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for which in range(4):
        ins = [q, k, v, do]
        ins[which] = torch.full_like(ins[which], bad)
        start.record()
        got = both(*ins, 8192, 4)
        end.record()
        assert api.cp_get_error() == 0
        assert start.elapsed_time(end) < 500
        assert not any(torch.isfinite(t).all() for t in got[2:4])
