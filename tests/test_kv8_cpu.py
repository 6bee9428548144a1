"""The paged 8-bit cache without a GPU: the oracle's format against torch's, the C ABI's refusals (every
check comes before the first CUDA call) and the binding's."""
import inspect
import math

import numpy as np
import pytest
import torch

from context_parallelism_02_gb300 import _lib, api
from oracle import kv8 as o

FAKE = 1 << 20   # never touched: the checks come first


def test_codes_are_torchs_e4m3():
    every = torch.arange(256, dtype=torch.uint8)
    want = every.view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(o.decode(every.numpy()), want)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(4000) * 2.0 ** rng.integers(-14, 9, 4000), o.POSITIVE,
                        (o.POSITIVE[1:] + o.POSITIVE[:-1]) / 2]).clip(-448, 448).astype(np.float32)
    got = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(o.encode(x), got)
    np.testing.assert_array_equal(o.encode([1e9, -1e9, math.inf, math.nan]), [0x7e, 0xfe, 0x7f, 0x7f])


def test_scale_is_the_smallest_power_of_two():
    assert o.scale_of([0.0]) == 2.0 ** -40 and o.scale_of([448.0]) == 1 and o.scale_of([448.5]) == 2
    assert o.scale_of([math.nan, -3.5, math.inf]) == 2.0 ** -7 and o.scale_of([1e300]) == 2.0 ** 60


def append(**kw):
    a = dict(k=FAKE, v=FAKE, cache=FAKE, scales=FAKE, pages=FAKE, lens=FAKE, n_new=None, strides=None, B=1, n=4, Hkv=2,
             D=128, P=8, page=64, M=4, dtype=1) | kw
    return _lib.load().kv8_append(*a.values(), None)


def gather(**kw):
    a = dict(cache=FAKE, scales=FAKE, pages=FAKE, lens=FAKE, start=None, k=FAKE, v=FAKE, B=1, count=4, Hkv=2, D=128, P=8,
             page=64, M=4, dtype=1) | kw
    return _lib.load().kv8_gather(*a.values(), None)


def attn(**kw):
    a = dict(q=FAKE, cache=FAKE, scales=FAKE, pages=FAKE, lens=FAKE, vis=None, out=FAKE, lse=FAKE, mass=None, B=1, n=1, Hq=8,
             Hkv=2, D=128, P=8, page=64, M=4, window=0, sinks=0, causal=1, out_dtype=1, scale=-1.0, ws=FAKE,
             bytes=1 << 40) | kw
    return _lib.load().kv8_attn(*a.values(), None)


def evict(**kw):
    a = dict(cache=FAKE, scales=FAKE, pages=FAKE, lens=FAKE, mass=FAKE, to=FAKE, kept=FAKE, lens_to=FAKE, mass_to=None, B=1,
             Hkv=2, D=128, P=8, page=64, M=4, max_to=2, budget=100, first=4, last=16) | kw
    return _lib.load().kv8_evict(*a.values(), None)


CALLS = [append, gather, attn, evict]


@pytest.mark.parametrize("call", CALLS)
def test_shared_refusals(call):
    bad = _lib.CP_EINVAL
    for kw in (dict(B=-1), dict(Hkv=0), dict(P=-1), dict(M=-1), dict(cache=None), dict(cache=FAKE + 8), dict(scales=None),
               dict(scales=FAKE + 2), dict(pages=None), dict(pages=FAKE + 2), dict(lens=None), dict(lens=FAKE + 1)):
        assert call(**kw) == bad, kw
    for kw in (dict(D=96), dict(D=32), dict(page=8), dict(page=48), dict(page=512), dict(M=2 ** 26, page=64)):
        assert call(**kw) == _lib.CP_EUNSUPPORTED, kw
    assert call(B=0) == _lib.CP_OK


def test_refusals_of_each_call():
    bad, no = _lib.CP_EINVAL, _lib.CP_EUNSUPPORTED
    for kw in (dict(n=-1), dict(k=None), dict(v=None), dict(k=FAKE + 8), dict(v=FAKE + 4), dict(n_new=FAKE + 2)):
        assert append(**kw) == bad, kw
    assert append(dtype=2) == no and append(n=0) == _lib.CP_OK
    assert append(B=2 ** 30, n=2 ** 30) == no
    strides = np.array([512, 128, 4, 512, 128, 4], np.int64)     # rows of 4 elements apart: not 16 bytes
    assert append(strides=strides.ctypes.data) == bad
    for kw in (dict(count=-1), dict(k=None), dict(v=FAKE + 8), dict(start=FAKE + 2)):
        assert gather(**kw) == bad, kw
    assert gather(dtype=2) == no and gather(count=0) == _lib.CP_OK
    for kw in (dict(q=None), dict(q=FAKE + 8), dict(out=None), dict(out=FAKE + 8), dict(lse=None), dict(mass=FAKE + 2),
               dict(n=-1), dict(Hq=9), dict(causal=2), dict(window=-1), dict(sinks=-1), dict(scale=math.nan), dict(ws=None),
               dict(ws=FAKE + 8), dict(bytes=100), dict(vis=FAKE + 2)):
        assert attn(**kw) == bad, kw
    assert attn(out_dtype=2) == no and attn(n=0) == _lib.CP_OK
    L = _lib.load()
    need = L.kv8_attn_workspace(1, 1, 8, 2, 128, 64, 4, 1)
    plain = L.kv8_attn_workspace(1, 1, 8, 2, 128, 64, 4, 0)
    assert need == plain + 2 * 4 * 256 * 4                       # 4 rows a slot and kv head
    assert attn(mass=FAKE, bytes=need - 1) == bad and attn(bytes=plain - 1) == bad
    assert L.kv8_attn_workspace(1, 1, 8, 2, 96, 64, 4, 1) == 0 and L.kv8_attn_workspace(1, 1, 9, 2, 128, 64, 4, 1) == 0
    for kw in (dict(to=None), dict(kept=None), dict(lens_to=None), dict(mass=None), dict(mass=FAKE + 2), dict(mass_to=FAKE + 2),
               dict(budget=0), dict(budget=129), dict(first=-1), dict(last=-1), dict(first=90, last=11), dict(max_to=-1),
               dict(max_to=1)):
        assert evict(**kw) == bad, kw


def test_binding_refuses_cpu_tensors_and_documents():
    x = torch.zeros(1, 1, 1, 64)
    i = torch.zeros(1, dtype=torch.int32)
    c = torch.zeros(1, 1, 2, 16, 64, dtype=torch.uint8)
    with pytest.raises(ValueError):
        api.kv8_append(x, x, c, i, i[None], i)
    with pytest.raises(ValueError):
        api.kv8_attn(x.bfloat16(), c, i, i[None], i)
    for D, page in ((96, 16), (64, 24)):
        with pytest.raises(api.CpError):
            api.kv8_cache(4, 2, page, D)
    for f in (api.kv8_append, api.kv8_gather, api.kv8_attn, api.kv8_evict, api.window_attn_fwd, api.window_attn_bwd):
        assert f.__doc__ and "stream" in inspect.signature(f).parameters
