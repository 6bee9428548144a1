"""The paged 4-bit cache without a GPU: the oracle's format against itself, the C
ABI's refusals (every check comes before the first CUDA call) and the binding's."""
import ctypes

import numpy as np
import pytest
import torch

from context_parallelism_02_gb300 import _lib, api
from oracle import kv4 as o

FAKE = 1 << 20   # never touched: the checks come first


@pytest.mark.parametrize("D", [64, 128])
def test_block_places_cover_every_byte_once(D):
    kb, ks, km, vb, vs, vm = o.places(D)
    nibbles = sorted([2 * b + s // 4 for b, s in zip(kb.ravel(), ks.ravel())] +
                     [2 * b + s // 4 for b, s in zip(vb.ravel(), vs.ravel())])
    meta = set()
    for at, step in ((km, 2), (vm, 4)):
        for x in np.unique(at):
            meta |= {x, x + 1, x + step, x + step + 1}
    assert len(meta) == 4 * D
    codes = [n for b in range(20 * D) if b not in meta for n in (2 * b, 2 * b + 1)]
    assert nibbles == codes


@pytest.mark.parametrize("D", [64, 128])
def test_oracle_write_read_round_trip(D):
    rng = np.random.default_rng(3)
    page = 32
    cache = rng.integers(0, 256, (3, 2, page, D // 4 * 5), dtype=np.uint8)
    pages = np.array([[2, 0]], np.int32)
    rows = rng.standard_normal((2, 40, D)).astype(np.float32)
    for t in range(40):
        o.write(cache, pages, 0, 1, t, rows[0, t], rows[1, t])
    for got, x in zip(o.read(cache, pages, 0, 1, range(40)), rows):
        code, s, m = o.quantise(x)
        np.testing.assert_array_equal(got, code.astype(np.float32) * s.astype(np.float32) + m.astype(np.float32))
        # half a step, and the roundings of the scale (15 codes of it) and of the minimum
        step = s.astype(np.float64)
        assert (np.abs(got - x) <= step * (0.5 + 15 * 2.0 ** -11) + np.abs(x).max() * 2.0 ** -11).all()


def test_bf16_rounding():
    x = np.array([1.0, 1.00390625, 1.01171875, -3.0e38, 0.0], np.float32)
    np.testing.assert_array_equal(o.bf16(x), torch.tensor(x).bfloat16().float().numpy())


def append(**kw):
    a = dict(k=FAKE, v=FAKE, q=FAKE, q_out=FAKE, cache=FAKE, summary=None, pages=FAKE, lens=FAKE, n_new=None,
             positions=None, cos=FAKE, sin=FAKE, strides=None, B=1, n=4, Hq=8, Hkv=2, D=128, P=8, page=64, M=4,
             rot=128, inter=0, max_pos=100, dtype=1)
    a.update(kw)
    return _lib.load().kv4_append(*a.values(), None)


def gather(**kw):
    a = dict(cache=FAKE, pages=FAKE, lens=FAKE, start=None, k=FAKE, v=FAKE, B=1, count=4, Hkv=2, D=128, P=8, page=64,
             M=4, dtype=1)
    a.update(kw)
    return _lib.load().kv4_gather(*a.values(), None)


def attn(**kw):
    a = dict(q=FAKE, cache=FAKE, pages=FAKE, lens=FAKE, vis=None, sel=None, out=FAKE, lse=FAKE, B=1, n=1, Hq=8,
             Hkv=2, D=128, P=8, page=64, M=4, n_sel=0, causal=1, out_dtype=1, scale=-1.0, ws=FAKE, bytes=1 << 40)
    a.update(kw)
    return _lib.load().kv4_attn(*a.values(), None)


def select(**kw):
    a = dict(q=FAKE, summary=FAKE, pages=FAKE, lens=FAKE, vis=None, sel=FAKE, B=1, n=1, Hq=8, Hkv=2, D=128, P=8,
             page=64, M=4, n_sel=4, causal=1, first=1, last=1, ws=FAKE, bytes=1 << 40)
    a.update(kw)
    return _lib.load().kv4_select(*a.values(), None)


@pytest.mark.parametrize("call", [append, gather, attn, select])
def test_refusals_shared(cplib, call):
    assert call(B=0) == _lib.CP_OK
    assert call(B=-1) == _lib.CP_EINVAL
    assert call(Hkv=0) == _lib.CP_EINVAL
    assert call(P=-1) == _lib.CP_EINVAL
    assert call(M=-1) == _lib.CP_EINVAL
    assert call(D=96) == _lib.CP_EUNSUPPORTED
    for page in (0, 8, 48, 512):
        assert call(page=page) == _lib.CP_EUNSUPPORTED
    assert call(pages=None) == _lib.CP_EINVAL
    assert call(lens=None) == _lib.CP_EINVAL
    assert call(pages=FAKE + 2) == _lib.CP_EINVAL
    assert call(lens=FAKE + 1) == _lib.CP_EINVAL


def test_append_refusals(cplib):
    E, U = _lib.CP_EINVAL, _lib.CP_EUNSUPPORTED
    assert append(n=0) == _lib.CP_OK
    assert append(n=-1) == E
    for name in ("k", "v", "cache", "cos", "sin"):
        assert append(**{name: None}) == E
    for name in ("k", "v", "q", "q_out", "cache", "summary", "cos", "sin"):
        assert append(**{name: FAKE + 8}) == E
    assert append(n_new=FAKE + 2) == E and append(positions=FAKE + 2) == E
    assert append(q=None) == E and append(q_out=None) == E           # q and q_out go together
    assert append(Hq=7) == E and append(Hq=0) == E
    for rot in (-16, 8, 144, 100):
        assert append(rot=rot) == E
    assert append(inter=2) == E
    assert append(max_pos=-1) == E
    assert append(dtype=2) == U
    strides = lambda *s: ctypes.cast((ctypes.c_int64 * 9)(*s), ctypes.c_void_p)
    ok = [4096, 1024, 128] * 3
    for i in range(9):
        assert append(strides=strides(*ok[:i], 4, *ok[i + 1:])) == E  # rows off a 16-byte boundary
        assert append(strides=strides(*ok[:i], -128, *ok[i + 1:])) == E


def test_gather_refusals(cplib):
    E = _lib.CP_EINVAL
    assert gather(count=0) == _lib.CP_OK
    assert gather(count=-1) == E
    for name in ("cache", "k", "v"):
        assert gather(**{name: None}) == E
        assert gather(**{name: FAKE + 8}) == E
    assert gather(start=FAKE + 1) == E
    assert gather(dtype=3) == _lib.CP_EUNSUPPORTED


def test_attn_refusals(cplib):
    E = _lib.CP_EINVAL
    assert attn(n=0) == _lib.CP_OK
    assert attn(n=-1) == E
    for name in ("q", "cache", "out", "lse", "ws"):
        assert attn(**{name: None}) == E
    for name in ("q", "cache", "out", "ws"):
        assert attn(**{name: FAKE + 8}) == E
    assert attn(lse=FAKE + 2) == E and attn(vis=FAKE + 2) == E
    assert attn(Hq=7) == E and attn(Hq=0) == E
    assert attn(causal=2) == E
    assert attn(out_dtype=2) == _lib.CP_EUNSUPPORTED
    assert attn(scale=float("nan")) == E
    assert attn(n_sel=3) == E                       # a count without a list
    assert attn(sel=FAKE, n_sel=0) == E
    assert attn(sel=FAKE + 2, n_sel=3) == E
    assert attn(sel=FAKE, n_sel=(1 << 26) + 1) == _lib.CP_EUNSUPPORTED
    L = _lib.load()
    assert L.kv4_attn_workspace(96) == 0
    for D in (64, 128):
        need = L.kv4_attn_workspace(D)
        assert need > 0 and attn(D=D, bytes=need - 1) == E


def test_select_refusals(cplib):
    E = _lib.CP_EINVAL
    assert select(n=0) == _lib.CP_OK
    for name in ("q", "summary", "sel", "ws"):
        assert select(**{name: None}) == E
    for name in ("q", "summary", "ws"):
        assert select(**{name: FAKE + 8}) == E
    assert select(n_sel=0) == E
    assert select(first=-1) == E and select(last=-1) == E
    assert select(n_sel=4, first=3, last=2) == E
    assert select(first=2 ** 31 - 1, last=2 ** 31 - 1) == E
    L = _lib.load()
    need = L.kv4_select_workspace(1, 1, 2, 4)
    assert need >= 32 and select(bytes=need - 1) == E
    assert L.kv4_select_workspace(-1, 1, 2, 4) == 0
    assert L.kv4_select_workspace(2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1) == 0


def test_error_code_has_a_message(cplib):
    assert _lib.strerror(_lib.CP_ECACHE) not in (_lib.strerror(-99), _lib.strerror(_lib.CP_EBOUNDS))


def test_binding_refuses_host_tensors_and_bad_shapes():
    k = torch.zeros(1, 2, 2, 64)
    cache = torch.zeros(4, 2, 16, 80, dtype=torch.uint8)
    pages, lens = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        api.kv4_append(k, k, cache, pages, lens)
    with pytest.raises(ValueError):
        api.kv4_append(k, k[:, :1], cache, pages, lens)
    with pytest.raises(ValueError):
        api.kv4_append(k.half(), k.half(), cache, pages, lens)
    with pytest.raises(ValueError):
        api.kv4_gather(cache, pages, lens, 4)
    with pytest.raises(ValueError):
        api.kv4_gather(cache, pages, lens, 4, dtype=torch.float16)
    with pytest.raises(ValueError):
        api.kv4_attn(k.bfloat16(), cache, pages, lens)
    with pytest.raises(ValueError):
        api.kv4_attn(k.bfloat16()[0], cache, pages, lens)
    with pytest.raises(ValueError):
        api.kv4_select(k.bfloat16(), torch.zeros(4, 2, 2, 64, dtype=torch.bfloat16), pages, lens, 16, 2)
    for D, page in ((96, 16), (64, 24)):
        with pytest.raises(_lib.CpError):
            api.kv4_cache(4, 2, page, D)


def test_sizes_whose_products_pass_64_bits_are_refused(cplib):
    """Rows with strides of 0 and an empty pool need no memory, so sizes alone must not wrap a launch's counts."""
    U, most = _lib.CP_EUNSUPPORTED, 2 ** 31 - 1
    zero = ctypes.cast((ctypes.c_int64 * 9)(), ctypes.c_void_p)
    for B, n, H in ((most, most, most), (1 << 20, most, most), (most, 1, most), (256, (1 << 31) - 128, 1 << 30)):
        assert append(B=B, n=n, Hkv=H, q=None, q_out=None, strides=zero, P=0) == U
        assert append(B=B, n=n, Hkv=1, Hq=H, strides=zero, P=0) == U
        assert gather(B=B, count=n, Hkv=H, P=0) == U
        assert attn(B=B, n=n, Hkv=H, Hq=H, P=0) == U
        assert attn(B=B, n=n, Hkv=1, Hq=H, P=0, sel=FAKE, n_sel=4) == U
        assert select(B=B, n=n, Hkv=H, Hq=H, P=0) == U
