"""Windowed attention and the 8-bit cache without a GPU: what a call needs and what it refuses to write over."""
import pytest

from context_parallelism_02_gb300 import _lib

F32, BF16 = 0, 1


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,Hq,Hkv,S,W,K", [(1, 8, 8, 131072, 128, 65536), (1, 32, 8, 32768, 1024, 16384), (2, 4, 4, 65536, 1, 65535),
                                            (1, 1, 1, 1048576, 16, 300000), (1, 8, 1, 8192, 64, 100), (4, 8, 8, 16384, 1024, 4)])
def test_workspace_of_many_sinks(B, Hq, Hkv, S, W, K, dtype):
    """The sinks' partial gradients in fp32 pass what K and V would take in it only by what fills the SMs: Delta,
    three times K (the slot of the window's units and pieces as long as K), and 4 x 152 units and one more per tile."""
    D = 128
    tile = 128 if dtype == BF16 else 32
    need = _lib.load().window_attn_bwd_workspace(B, Hq, Hkv, S, S, D, W, K, dtype)
    tiles = -(-K // tile) * B * Hkv
    assert need <= 256 + B * Hq * S * 4 + max(3 * B * Hkv * S * D * 4, (4 * 152 + 2 * tiles) * tile * 2 * D * 4) + 256


def pointers(names):
    """Addresses a GB apart: never touched, every call below is refused first."""
    return {n: (i + 1) << 30 for i, n in enumerate(names)}


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_windowed_attention_refuses_outputs_over_what_it_reads(dtype):
    """By its first bytes or its last ones: q and its like have B Sq Hq D elements, k B Sk Hkv D."""
    B, Hq, Hkv, Sq, Sk, D = 2, 4, 2, 64, 100, 64
    size = 4 if dtype == F32 else 2
    nq, nk, nz = B * Sq * Hq * D * size, B * Sk * Hkv * D * size, B * Hq * Sq * 4
    L = _lib.load()

    def fwd(**kw):
        p = pointers(["q", "k", "v", "out", "lse"]) | kw
        return L.window_attn_fwd(*p.values(), B, Hq, Hkv, Sq, Sk, D, 8, 2, dtype, -1.0, None)

    need = L.window_attn_bwd_workspace(B, Hq, Hkv, Sq, Sk, D, 8, 2, dtype)
    names = ["q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv"]

    def bwd(ws=1 << 40, **kw):
        p = pointers(names) | kw
        return L.window_attn_bwd(*p.values(), B, Hq, Hkv, Sq, Sk, D, 8, 2, dtype, -1.0, ws, need, None)
    at = pointers(["q", "k", "v", "out", "lse"])
    read = dict(q=nq, k=nk, v=nk)
    for name, mine in (("out", nq), ("lse", nz)):
        for other, n in (read | {"lse" if name == "out" else "out": nz if name == "out" else nq}).items():
            assert fwd(**{name: at[other] + n - 16}) == _lib.CP_EINVAL, (name, other)
            assert fwd(**{name: at[other] - mine + 16}) == _lib.CP_EINVAL, (name, other)
    at = pointers(names)
    read = dict(q=nq, k=nk, v=nk, out=nq, lse=nz, dout=nq)
    wrote = dict(dq=nq, dk=nk, dv=nk)
    for name, mine in wrote.items():
        for other, n in (read | {w: x for w, x in wrote.items() if w != name}).items():
            assert bwd(**{name: at[other] + n - 16}) == _lib.CP_EINVAL, (name, other)
            assert bwd(**{name: at[other] - mine + 16}) == _lib.CP_EINVAL, (name, other)
    for other, n in (read | wrote).items():
        assert bwd(ws=at[other] + n - 16) == bwd(ws=at[other] - need + 16) == _lib.CP_EINVAL, other


def refused(call, wrote, read):
    """Every output, moved over the end of each other buffer and over its beginning."""
    at = pointers([*wrote, *read])
    for name, mine in wrote.items():
        for other, n in (read | {w: x for w, x in wrote.items() if w != name}).items():
            assert call(at | {name: at[other] + n - 16}) == _lib.CP_EINVAL, (name, other)
            assert call(at | {name: at[other] - mine + 16}) == _lib.CP_EINVAL, (name, other)


def test_the_8_bit_cache_refuses_outputs_over_what_it_reads():
    B, n, Hq, H, D, P, page, M, to, budget = 8, 8, 6, 2, 64, 20, 32, 5, 3, 70
    L = _lib.load()
    pool = dict(cache=P * H * 2 * page * D, scales=P * H * 2 * page // 16 * 4)
    tables = dict(pages=B * M * 4, lens=B * 4)
    mass, rows = B * H * M * page * 4, B * n * H * D * 4

    def append(p):
        return L.kv8_append(p["k"], p["v"], p["cache"], p["scales"], p["pages"], p["lens"], p["n_new"], None, B, n, H, D, P, page, M,
                            F32, None)
    refused(append, pool, tables | dict(k=rows, v=rows, n_new=B * 4))

    def gather(p):
        return L.kv8_gather(p["cache"], p["scales"], p["pages"], p["lens"], p["start"], p["k"], p["v"], B, n, H, D, P, page, M, F32, None)
    refused(gather, dict(k=rows, v=rows), pool | tables | dict(start=B * 4))
    need = L.kv8_attn_workspace(B, n, Hq, H, D, page, M, 1)

    def attn(p):
        return L.kv8_attn(p["q"], p["cache"], p["scales"], p["pages"], p["lens"], p["vis"], p["out"], p["lse"], p["mass"], B, n, Hq, H,
                          D, P, page, M, 0, 0, 1, F32, -1.0, p["ws"], need, None)
    heads = B * n * Hq
    refused(attn, dict(out=heads * D * 4, lse=heads * 4, mass=mass, ws=need), pool | tables | dict(q=heads * D * 2, vis=B * n * 4))

    def evict(p):
        return L.kv8_evict(p["cache"], p["scales"], p["pages"], p["lens"], p["mass"], p["to"], p["kept"], p["lens_to"], p["mass_to"], B,
                           H, D, P, page, M, to, budget, 2, 8, None)
    refused(evict, dict(kept=B * H * budget * 4, lens_to=B * 4, mass_to=B * H * to * page * 4), pool | tables | dict(mass=mass, to=B * to * 4))
