"""The 8-bit cache's kernels behind a kernel that lets them start early and writes what they read late: nothing
may be read before that kernel is complete."""
import pytest
import torch

from context_parallelism_02_gb300 import api
from tests.test_gpu_kv4_order import late_copy  # noqa: F401 - a fixture

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


def make(seed, B, L, Hq, H, D, page, width):
    g = torch.Generator(device="cuda").manual_seed(seed)
    M = -(-L // page)
    P = B * M + 2
    cache, scales = api.kv8_cache(P + 4 * B, H, page, D)
    cache.zero_(), scales.fill_(1)
    pages = torch.full((B, width), -1, **I32)
    pages[:, :M] = torch.randperm(P, generator=g, device="cuda")[:B * M].reshape(B, M).int()
    to = (torch.arange(4 * B, **I32) + P).reshape(B, 4)
    k, v = (torch.randn(B, L, H, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    api.kv8_append(k, v, cache, scales, pages, torch.zeros(B, **I32))
    return dict(cache=cache, scales=scales, pages=pages, to=to, q=torch.randn(B, 1, Hq, D, generator=g, device="cuda").bfloat16(),
                k=k[:, :1].contiguous(), lens=torch.tensor([L - 37 * b for b in range(B)], **I32),
                mass=torch.rand(B, H, width * page, generator=g, device="cuda"))


def behind(late_copy, name, tensors, call, stale):  # noqa: F811
    """call(tensors) with tensors[name] written late over `stale`, eagerly and captured, equals the call on settled data."""
    right = tensors[name].clone()
    kept = [n for n in ("cache", "scales", "mass") if n != name]
    settled = {n: t.clone() for n, t in tensors.items()}
    want = [t.clone() for t in call(settled)] + [settled[n].clone() for n in kept]
    late = {n: t.clone() for n, t in tensors.items()}

    def reset():
        for n in kept:
            late[n].copy_(tensors[n])
        late[name].copy_(stale)
        torch.cuda.synchronize()

    def run():
        late_copy(late[name], right)
        return list(call(late))
    for _ in range(3):
        reset()
        got = run()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got + [late[n] for n in kept], want)), name
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(3):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got + [late[n] for n in kept], want)), name
    assert api.cp_get_error() == 0


# one long sequence and a ragged batch that are cut into stretches and joined, a short table with a block per item
SHAPES = [(1, 9000, 141), (5, 3000, 60), (3, 500, 8)]


def stale_of(t, name):
    if name in ("lens",):
        return t[name] // 3
    if name == "pages":
        return t[name].roll(1, 1).clamp(min=0)
    if name == "to":
        return t[name].flip(1)
    if name == "cache":
        return t[name].flip(0)
    return -t[name] if name != "scales" else t[name] * 4


@pytest.mark.parametrize("name", ["q", "pages", "lens", "cache", "scales", "mass"])
@pytest.mark.parametrize("B,L,width", SHAPES)
def test_attn_inputs_written_late(late_copy, name, B, L, width):  # noqa: F811
    t = make(4, B, L, 8, 2, 128, 64, width)

    def call(t):
        got = [*api.kv8_attn(t["q"], t["cache"], t["scales"], t["pages"], t["lens"], mass=t["mass"])]
        return got + [*api.kv8_attn(t["q"], t["cache"], t["scales"], t["pages"], t["lens"], window=300, sinks=5), t["mass"].clone()]
    behind(late_copy, name, t, call, stale_of(t, name).contiguous())


@pytest.mark.parametrize("name", ["k", "pages", "lens", "scales"])
def test_append_inputs_written_late(late_copy, name):  # noqa: F811
    t = make(5, 3, 700, 4, 2, 64, 32, 24)
    t["lens"] = torch.tensor([690, 5, 40], **I32)

    def call(t):
        api.kv8_append(t["k"], t["k"], t["cache"], t["scales"], t["pages"], t["lens"])
        return [*api.kv8_gather(t["cache"], t["scales"], t["pages"], t["lens"] + 1, 20, start=(t["lens"] - 5))]
    behind(late_copy, name, t, call, stale_of(t, name).contiguous())


@pytest.mark.parametrize("name", ["pages", "lens", "cache", "scales", "mass", "to"])
@pytest.mark.parametrize("B,L,width", SHAPES)
def test_evict_inputs_written_late(late_copy, name, B, L, width):  # noqa: F811
    t = make(6, B, L, 4, 2, 64, 64, width)

    def call(t):
        kept, lens, mass = api.kv8_evict(t["cache"], t["scales"], t["pages"], t["lens"], t["mass"], t["to"], 200, 2, 30)
        return [kept, lens, mass, *api.kv8_gather(t["cache"], t["scales"], t["to"], lens, 200)]
    behind(late_copy, name, t, call, stale_of(t, name).contiguous())


@pytest.mark.parametrize("lens", [[2400, 63, 1000], [300, 20, 500]])
def test_a_step_of_lengths_written_late(late_copy, lens):  # noqa: F811
    """A whole decode step behind the late lengths: append, their increment, attention with weights, eviction, read-back."""
    t = make(2, 3, max(lens) + 8, 4, 2, 64, 64, 45)
    a = {n: x.clone() for n, x in t.items()}
    b = {n: x.clone() for n, x in t.items()}
    for x in (a, b):
        x["lens"].copy_(torch.tensor(lens, **I32))

    def step(t):
        api.kv8_append(t["k"], t["k"], t["cache"], t["scales"], t["pages"], t["lens"])
        t["lens"] += 1
        got = [*api.kv8_attn(t["q"], t["cache"], t["scales"], t["pages"], t["lens"], mass=t["mass"])]
        got += api.kv8_evict(t["cache"], t["scales"], t["pages"], t["lens"], t["mass"], t["to"], 250, 2, 30)
        return got + [*api.kv8_gather(t["cache"], t["scales"], t["to"], got[-2], 250)]
    for _ in range(4):
        torch.cuda.synchronize()
        want = step(a)
        torch.cuda.synchronize()
        right = (a["lens"] - 1).contiguous()
        b["lens"].copy_(right // 2)
        torch.cuda.synchronize()
        late_copy(b["lens"], right)
        got = step(b)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert all(torch.equal(a[n], b[n]) for n in a)
    assert api.cp_get_error() == 0
