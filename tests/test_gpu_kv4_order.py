"""The cache's kernels behind a kernel that lets them start early and writes what they
read late: nothing may be read before that kernel is complete."""
import ctypes
import math
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
