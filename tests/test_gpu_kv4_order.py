"""The cache's kernels behind a kernel that lets them start early and writes what they
read late: nothing may be read before that kernel is complete."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from context_parallelism_02_gb300 import api, build

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))
DELAY_NS = 40000   # several times what a call of these sizes takes


@pytest.fixture(scope="module")
def late_copy(cuda_dev, tmp_path_factory):
    """copy(dst, src): dst = src on the current stream, by a kernel that triggers its dependents first."""
    lib = str(tmp_path_factory.mktemp("late_copy") / "late_copy.so")
    subprocess.run([build.nvcc(), *build.ARCH, "-O2", "-shared", "-Xcompiler", "-fPIC", "-cudart", "static",
                    os.path.join(HERE, "late_copy.cu"), "-o", lib], check=True, capture_output=True, text=True)
    call = ctypes.CDLL(lib).late_copy
    call.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint, ctypes.c_void_p]

    def copy(dst, src):
        assert dst.is_contiguous() and src.is_contiguous() and dst.nbytes == src.nbytes
        assert call(dst.data_ptr(), src.data_ptr(), dst.nbytes, DELAY_NS, torch.cuda.current_stream().cuda_stream) == 0
    return copy


def make(seed, B, L, Hq, Hkv, D, page, width):
    """A filled pool, a query token per sequence, and the table, with `width` entries a sequence."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    M = -(-L // page)
    P = B * M + 2
    cache, summ = api.kv4_cache(P, Hkv, page, D, summary=True)
    cache.zero_()
    summ.zero_()
    pages = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    pages[:, :M] = torch.randperm(P, generator=g, device="cuda")[:B * M].reshape(B, M).int()
    k, v = (torch.randn(B, L, Hkv, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    api.kv4_append(k, v, cache, pages, torch.zeros(B, dtype=torch.int32, device="cuda"), summary=summ)
    q = torch.randn(B, 1, Hq, D, generator=g, device="cuda").bfloat16()
    return cache, summ, pages, q


def behind(late_copy, name, tensors, call, stale):
    """call(tensors) with tensors[name] written late over `stale`, eagerly and captured, equals the call on settled data."""
    right = tensors[name].clone()
    settled = {n: t.clone() for n, t in tensors.items()}
    want = [t.clone() for t in call(settled)] + [settled["cache"].clone()]
    late = {n: t.clone() for n, t in tensors.items()}

    def run():
        late_copy(late[name], right)
        return list(call(late))
    torch.cuda.synchronize()
    for _ in range(3):
        late[name].copy_(stale)
        late["cache"].copy_(tensors["cache"] if name != "cache" else stale)
        torch.cuda.synchronize()
        got = run()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got + [late["cache"]], want)), name
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(3):
        late[name].copy_(stale)
        late["cache"].copy_(tensors["cache"] if name != "cache" else stale)
        for t in got:
            t.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got + [late["cache"]], want)), name
    assert api.cp_get_error() == 0


# sequences, their capacity, entries of a table row: one long sequence and a ragged batch that are cut into
# stretches and joined, and a short table with a block per item
SHAPES = [(1, 9000, 141), (5, 3000, 60), (3, 500, 8)]


@pytest.mark.parametrize("B,L,width", SHAPES)
def test_attn_lengths_written_late(late_copy, B, L, width):
    """Stale lengths cut the batch in other places than the true ones: a join by them takes other parts."""
    cache, _, pages, q = make(1, B, L, 8, 2, 128, 64, width)
    lens = torch.tensor([L - 37 * b for b in range(B)], dtype=torch.int32, device="cuda")
    stale = torch.tensor([(100 + 613 * b) % L for b in range(B)], dtype=torch.int32, device="cuda")
    for old in (stale, torch.zeros_like(lens)):
        behind(late_copy, "lens", dict(lens=lens, cache=cache), lambda t: api.kv4_attn(q, t["cache"], pages, t["lens"]), old)


def test_decode_step_of_lengths_written_late(late_copy):
    """A whole decode step behind the late lengths: append, their increment, selection, attention, read-back."""
    B, L, page = 3, 2500, 64
    cache, summ, pages, q = make(2, B, L, 4, 2, 64, page, 45)
    g = torch.Generator(device="cuda").manual_seed(3)
    k = torch.randn(B, 1, 2, 64, generator=g, device="cuda").bfloat16()

    def step(t):
        api.kv4_append(k, k, t["cache"], pages, t["lens"], summary=t["summary"])
        t["lens"] += 1
        sel = api.kv4_select(q, t["summary"], pages, t["lens"], page, 6)
        return [sel, *api.kv4_attn(q, t["cache"], pages, t["lens"]), *api.kv4_attn(q, t["cache"], pages, t["lens"], sel=sel),
                *api.kv4_gather(t["cache"], pages, t["lens"], 20, start=t["lens"] - 10)]
    lens = torch.tensor([2400, 63, 1000], dtype=torch.int32, device="cuda")

    def fresh():
        return dict(cache=cache.clone(), summary=summ.clone(), lens=lens.clone())
    a, b = fresh(), fresh()
    for _ in range(4):
        torch.cuda.synchronize()
        want = step(a)
        torch.cuda.synchronize()
        late_copy(b["lens"], (a["lens"] - 1).contiguous())
        got = step(b)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert all(torch.equal(a[n], b[n]) for n in a)
    assert api.cp_get_error() == 0


@pytest.mark.parametrize("name", ["q", "pages", "lens", "vis", "sel", "cache"])
@pytest.mark.parametrize("B,L,width", SHAPES)
def test_attn_inputs_written_late(late_copy, name, B, L, width):
    cache, _, pages, q = make(4, B, L, 8, 2, 128, 64, width)
    rng = np.random.default_rng(5)
    M = -(-L // 64)
    sel = torch.from_numpy(np.stack([rng.permutation(M)[:4] for _ in range(B * 2)]).astype(np.int32)).cuda().reshape(B, 1, 2, 4)
    tensors = dict(q=q, pages=pages, lens=torch.full((B,), L, dtype=torch.int32, device="cuda"), cache=cache,
                   vis=torch.full((B, 1), L - 5, dtype=torch.int32, device="cuda"), sel=sel.contiguous())
    stale = dict(q=-q, pages=pages.roll(1, 1).clamp(min=0), lens=tensors["lens"] // 3, vis=tensors["vis"] // 2, sel=sel.flip(-1) * 0,
                 cache=cache.flip(0))[name].contiguous()

    def call(t):
        out = api.kv4_attn(t["q"], t["cache"], t["pages"], t["lens"], vis=t["vis"])
        return out if name != "sel" else api.kv4_attn(t["q"], t["cache"], t["pages"], t["lens"], vis=t["vis"], sel=t["sel"])
    behind(late_copy, name, tensors, call, stale)


@pytest.mark.parametrize("name", ["q", "summary", "pages", "lens"])
def test_select_inputs_written_late(late_copy, name):
    cache, summ, pages, q = make(6, 2, 3000, 4, 2, 64, 16, 190)
    tensors = dict(q=q, summary=summ, pages=pages, lens=torch.tensor([3000, 1200], dtype=torch.int32, device="cuda"), cache=cache[:1])
    stale = dict(q=-q, summary=-summ, pages=pages.roll(1, 1).clamp(min=0), lens=tensors["lens"] // 3)[name].contiguous()
    behind(late_copy, name, tensors, lambda t: [api.kv4_select(t["q"], t["summary"], t["pages"], t["lens"], 16, 9)], stale)


@pytest.mark.parametrize("name", ["k", "v", "q", "cos", "sin", "positions", "n_new", "pages", "lens"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_inputs_written_late(late_copy, name, dtype):
    B, n, H, D, page = 2, 90, 2, 64, 32
    g = torch.Generator(device="cuda").manual_seed(7)
    q, k, v = (torch.randn(B, n, h, D, generator=g, device="cuda").to(dtype) for h in (4, H, H))
    cos, sin = (torch.rand(400, D // 2, generator=g, device="cuda") for _ in range(2))
    P = 2 * 8
    pages = torch.randperm(P, generator=g, device="cuda").reshape(B, 8).int()
    i32 = dict(dtype=torch.int32, device="cuda")
    tensors = dict(k=k, v=v, q=q, cos=cos, sin=sin, positions=torch.randint(0, 400, (B, n), generator=g, **i32),
                   n_new=torch.tensor([n, 51], **i32), pages=pages, lens=torch.tensor([40, 77], **i32),
                   cache=torch.zeros(P, H, page, D // 4 * 5, dtype=torch.uint8, device="cuda"))
    stale = dict(tensors, positions=tensors["positions"].flip(0), n_new=tensors["n_new"] // 2, pages=pages.flip(1),
                 lens=tensors["lens"] // 2)[name]
    stale = (-stale if stale.is_floating_point() else stale).contiguous()
    behind(late_copy, name, tensors,
           lambda t: [api.kv4_append(t["k"], t["v"], t["cache"], t["pages"], t["lens"], t["cos"], t["sin"], q=t["q"],
                                     positions=t["positions"], n_new=t["n_new"])], stale)


@pytest.mark.parametrize("name", ["cache", "pages", "lens", "start"])
def test_gather_inputs_written_late(late_copy, name):
    cache, _, pages, _ = make(8, 2, 500, 2, 2, 128, 16, 32)
    i32 = dict(dtype=torch.int32, device="cuda")
    tensors = dict(cache=cache, pages=pages, lens=torch.tensor([500, 123], **i32), start=torch.tensor([17, 3], **i32))
    stale = dict(cache=cache.flip(0), pages=pages.roll(1, 1).clamp(min=0), lens=tensors["lens"] // 3,
                 start=tensors["start"] * 2)[name].contiguous()
    behind(late_copy, name, tensors, lambda t: list(api.kv4_gather(t["cache"], t["pages"], t["lens"], 300, start=t["start"])), stale)
