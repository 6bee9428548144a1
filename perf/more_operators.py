"""Cases and plain forms of attention with a bounded reach and of the 8-bit cache.

Long contexts at bounded cost.  Training and prefill: attention with a sliding
window and a few first tokens that stay visible (``fwd``, and ``train`` with its
gradients).  Serving: a paged cache in 8 bits with a power-of-two scale per block
of 16 tokens, kv head and K or V (``append``: write new tokens, and read them back;
``attn``: attention of a few query tokens over the cache, whole or with a window and
first tokens, and the weight that every cached token got), and the cache cut down
to the tokens of the largest accumulated weight (``evict``).

Cache: [n_pages, Hkv, 2 (K, V), page, D] codes in e4m3, scales fp32
[n_pages, Hkv, 2, page / 16]; value = scale * code.  A block's scale is 2^e, e the
smallest integer in [-40, 60] with amax <= 448 * 2^e over its tokens.  Tokens that
join a block can raise its scale; the older codes are then rounded to it.
"""
import math

import torch

own = False

DEV = "cuda"
BLK = 16                                 # tokens that share a scale
E_MIN, E_MAX = -40, 60                   # exponents of a scale


def listed():
    return [
        # the next chunk of a prompt that is prefilled in chunks, behind its window: latency
        dict(name="fwd_chunk", op="fwd", B=1, Sq=1000, Sk=2027, Hq=32, Hkv=8, D=128, window=1024, sinks=4, dtype="bf16"),
        # a whole prompt of 32768 tokens, 32 query heads on 8 kv heads
        dict(name="fwd_32k", op="fwd", B=1, Sq=32768, Sk=32768, Hq=32, Hkv=8, D=128, window=4096, sinks=4, dtype="bf16"),
        # one layer's attention of a training step
        dict(name="train_16k", op="train", B=1, Sq=16384, Sk=16384, Hq=16, Hkv=16, D=128, window=1024, sinks=4,
             dtype="bf16"),
        # a small check run in full precision, odd sizes
        dict(name="train_f32_odd", op="train", B=2, Sq=1001, Sk=1001, Hq=6, Hkv=2, D=64, window=200, sinks=5, dtype="f32"),
        # one new token of each conversation of a batch: latency
        dict(name="append_one_token", op="append", B=16, n=1, Hkv=8, D=128, page=64, past=32767, dtype="bf16",
             fused=False, ragged=False),
        # the whole prompt after a prefill, k and v as views of one projection's output
        dict(name="append_prompt_32k", op="append", B=1, n=32768, Hkv=8, D=128, page=64, past=0, dtype="bf16",
             fused=True, ragged=False),
        # one token over a short context: latency
        dict(name="attn_short_512", op="attn", B=1, n=1, L=512, Hq=32, Hkv=8, D=128, page=64, window=0, sinks=0,
             mass=False, ragged=False),
        # a serving batch of 32k contexts
        dict(name="attn_16x32k", op="attn", B=16, n=1, L=32768, Hq=32, Hkv=8, D=128, page=64, window=0, sinks=0,
             mass=False, ragged=False),
        # a ragged serving batch, lengths from 1 to 8192, of a model with a window and first tokens
        dict(name="attn_window_64x8k", op="attn", B=64, n=1, L=8192, Hq=32, Hkv=8, D=128, page=16, window=1024, sinks=4,
             mass=False, ragged=True),
        # four drafted tokens over contexts that will be cut down: the weights are accumulated
        dict(name="attn_mass_8x16k", op="attn", B=8, n=4, L=16384, Hq=16, Hkv=8, D=64, page=32, window=0, sinks=0,
             mass=True, ragged=False),
        # one conversation of 65536 tokens cut down to a quarter
        dict(name="evict_64k", op="evict", B=1, L=65536, budget=16384, first=4, last=512, Hkv=8, D=128, page=64,
             ragged=False),
        # a ragged batch cut down to 1000 tokens each; some need no cut
        dict(name="evict_16x8k", op="evict", B=16, L=8192, budget=1000, first=4, last=64, Hkv=8, D=128, page=16, ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["fwd", "train", "append", "attn", "attn", "evict"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8])
    page = rng.choice([16, 32, 64, 128])
    if op in ("fwd", "train"):
        f32 = rng.random() < 0.2
        Hq = Hkv * rng.choice([1, 1, 2, 3, 4])
        B = rng.choice([1, 1, 2, 3])
        most = 2048 if f32 else 65536 if op == "fwd" else 16384     # rows of the batch
        Sk = _log(rng, 16, most // B)
        Sq = rng.choice([Sk, Sk, max(1, Sk // 3), _log(rng, 1, Sk)]) if op == "fwd" else Sk
        pairs = (1 << 26) if f32 else (1 << 32) if op == "fwd" else (1 << 28)
        # a row that sees itself alone has no gradient of q and k: nothing to compare
        least = 1 if op == "fwd" else 2
        window = _log(rng, least, max(least, min(2 * Sk, pairs // (B * Sq * Hq))))
        return dict(op=op, B=B, Sq=Sq, Sk=Sk, Hq=Hq, Hkv=Hkv, D=D, window=window,
                    sinks=rng.choice([0, 1, 4, 4, 7, 64, 200]), dtype="f32" if f32 else "bf16")
    if op == "append":
        B = _log(rng, 1, 128)
        return dict(op=op, B=B, n=_log(rng, 1, max(1, 16384 // B)), Hkv=Hkv, D=D, page=page, past=_log(rng, 1, 8192) - 1,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), fused=rng.random() < 0.5, ragged=rng.random() < 0.5)
    if op == "attn":
        B = _log(rng, 1, 64)
        window = rng.choice([0, 0, _log(rng, 1, 8192)])
        return dict(op=op, B=B, n=rng.choice([1, 1, 1, 1, 2, 5, 8]), L=_log(rng, 16, 524288 // max(B, 4)),
                    Hq=Hkv * rng.choice([1, 2, 4, 4, 7, 8]), Hkv=Hkv, D=D, page=page, window=window,
                    sinks=rng.choice([0, 4, 64]) if window else 0, mass=rng.random() < 0.3, ragged=rng.random() < 0.5)
    B = _log(rng, 1, 32)
    L = _log(rng, 16, 131072 // max(B, 2))
    budget = _log(rng, 2, L + 10)
    first = rng.choice([0, 1, 4])
    return dict(op=op, B=B, L=L, budget=budget, first=min(first, budget // 2), last=rng.choice([0, budget // 8, budget // 2]),
                Hkv=Hkv, D=D, page=page, ragged=rng.random() < 0.5)


# --- the cache format, in elementary operations ------------------------------------------------------


def _scale_of(amax):
    """2^e with e the smallest integer in range such that amax <= 448 2^e."""
    m, e = torch.frexp(amax)                                      # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = e - 9 + (m > 0.875).to(e.dtype)
    e = torch.where(amax > 0, e, E_MIN).clamp(E_MIN, E_MAX)
    return torch.ldexp(torch.ones_like(amax), e)


def _codes(x, scale):
    """x / scale rounded to e4m3 (nearest even), held within +-448."""
    return (x / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _pack(x):
    """[..., page, D] fp32 -> codes like x, scales [..., page / 16]."""
    b = x.unflatten(-2, (-1, BLK))
    s = _scale_of(b.abs().amax((-1, -2)))
    return _codes(b, s[..., None, None]).flatten(-3, -2), s


def _values(codes, scales):
    """Codes [..., page, D] and scales [..., page / 16] -> values, fp32."""
    return codes.float() * scales.repeat_interleave(BLK, -1).unsqueeze(-1)


def _read(cache, scales, pages):
    """Pages [B, M] -> k, v [B, Hkv, M page, D] fp32."""
    B, M = pages.shape
    at = pages.long().clamp(min=0)
    x = _values(cache.view(torch.float8_e4m3fn)[at], scales[at])                  # [B, M, Hkv, 2, page, D]
    k, v = x.permute(3, 0, 2, 1, 4, 5).flatten(3, 4).unbind(0)
    return k, v


# --- inputs -------------------------------------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 2654435761 % (1 << 31) + 29)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _spread(case, lo, hi):
    """The batch's lengths: all `hi`, or spread evenly over the logarithm of [lo, hi]."""
    B = case["B"]
    if not case["ragged"] or B == 1:
        return [hi] * B
    return [max(lo, min(hi, int(lo * (hi / lo) ** (i / (B - 1))))) for i in range(B - 1)] + [hi]


def _lens(case, g, lo, hi):
    x = torch.tensor(_spread(case, lo, hi), dtype=torch.int32, device=DEV)
    return x[torch.randperm(x.numel(), generator=g, device=DEV)].contiguous()


def _pool(case, g, M, extra=0, content=True):
    """A pool with room for B sequences of M pages and `extra` pages more for each, its pages in random order."""
    B, Hkv, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    P = B * (M + extra) + 3
    cache = torch.zeros(P, Hkv, 2, page, D, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(P, Hkv, 2, page // BLK, device=DEV)
    order = torch.randperm(P, generator=g, device=DEV)[:B * (M + extra)].reshape(B, M + extra).to(torch.int32)
    if content:
        step = max(1, (1 << 26) // (Hkv * page * D))
        # tokens differ in size (a first token is often small, some are large), and so do channels
        chan = torch.exp(0.7 * _randn(g, Hkv, 2, 1, D))
        for a in range(0, P, step):                               # a slab at a time: a pool of several GB
            p = min(P, a + step) - a
            x = _randn(g, p, Hkv, 2, page, D) * torch.exp(0.3 * _randn(g, p, Hkv, 2, page, 1)) * chan
            x[:, :, 0] *= 0.6
            c, scales[a:a + p] = _pack(x.bfloat16().float())
            cache[a:a + p] = c.view(torch.uint8)
    return cache, scales, order[:, :M].contiguous(), order[:, M:].contiguous()


def _unused(pages, lens, page):
    """Entries behind a sequence's last page name no page."""
    used = torch.arange(pages.shape[1], device=DEV) * page < lens.unsqueeze(1)
    return torch.where(used, pages, -1).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    op, B, Hkv, D = case["op"], case["B"], case["Hkv"], case["D"]
    if op in ("fwd", "train"):
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s.update(q=_randn(g, B, case["Sq"], case["Hq"], D).to(dt), k=_randn(g, B, case["Sk"], Hkv, D).to(dt),
                 v=_randn(g, B, case["Sk"], Hkv, D).to(dt))
        if op == "train":
            s.update(dout=_randn(g, B, case["Sq"], case["Hq"], D).to(dt))
        return s
    page = case["page"]
    if op == "append":
        n, past = case["n"], case["past"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        cache, scales, pages, _ = _pool(case, g, -(-(past + n) // page), content=False)
        lens = _lens(case, g, max(1, past // 2), past) if past else torch.zeros(B, dtype=torch.int32, device=DEV)
        # the block that the new tokens join holds the tokens before them
        at = (lens.long() - 1).clamp(min=0) // page
        old = pages.gather(1, at.unsqueeze(1)).squeeze(1).long()
        c, sc = _pack(_randn(g, B, Hkv, 2, page, D).bfloat16().float())
        cache[old], scales[old] = c.view(torch.uint8), sc
        n_new = _lens(case, g, 1, n) if case["ragged"] else None
        if case["fused"]:
            x = _randn(g, B, n, 3 * Hkv * D).to(dt)               # q's share lies between, and is not cached
            k, _, v = (t.unflatten(-1, (-1, D)) for t in x.split(Hkv * D, -1))
        else:
            k, v = (_randn(g, B, n, Hkv, D).to(dt) for _ in range(2))
        s.update(k=k, v=v, cache=cache, scales=scales, pages=pages, lens=lens, n_new=n_new,
                 after=(lens + (n if n_new is None else n_new)).int())
        return s
    M = -(-case["L"] // page)
    if op == "attn":
        n = case["n"]
        cache, scales, pages, _ = _pool(case, g, M)
        lens = _lens(case, g, min(n, case["L"]), case["L"])
        s.update(cache=cache, scales=scales, pages=_unused(pages, lens, page), lens=lens,
                 q=_randn(g, B, n, case["Hq"], D).bfloat16())
        if case["mass"]:
            s.update(mass=torch.exp(2 * _randn(g, B, Hkv, M * page)) / 16)
        return s
    cache, scales, pages, to = _pool(case, g, M, extra=-(-case["budget"] // page))
    lens = _lens(case, g, max(1, case["L"] // 16), case["L"])
    mass = torch.exp(2 * _randn(g, B, Hkv, M * page)) / 16
    mass = torch.where(torch.rand(mass.shape, generator=g, device=DEV) < 0.1, 0.0, mass)   # never looked at
    s.update(cache=cache, scales=scales, pages=_unused(pages, lens, page), lens=lens, mass=mass, to=to)
    return s


# --- one pass -----------------------------------------------------------------------------------------


def _chunk(s, i0, i1):
    """Keys that the query rows [i0, i1) reach, and which of them each row sees."""
    off = s["Sk"] - s["Sq"]
    lo = max(0, i0 + off - s["window"] + 1)
    keys = torch.cat([torch.arange(min(s["sinks"], lo), device=DEV), torch.arange(lo, i1 + off, device=DEV)])
    pos = torch.arange(i0 + off, i1 + off, device=DEV).unsqueeze(1)
    return keys, (keys <= pos) & ((keys > pos - s["window"]) | (keys < s["sinks"]))


def _run_window(s):
    B, Sq, Hq, Hkv, D = s["B"], s["Sq"], s["Hq"], s["Hkv"], s["D"]
    scale = 1.0 / math.sqrt(D)
    q = s["q"].float().reshape(B, Sq, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)   # [B, Hkv, R, Sq, D]
    k, v = (s[x].float().permute(0, 2, 1, 3).unsqueeze(2) for x in ("k", "v"))    # [B, Hkv, 1, Sk, D]
    train = s["op"] == "train"
    out, lse = torch.empty_like(q), torch.empty(q.shape[:-1], device=DEV)
    if train:
        do = s["dout"].float().reshape(B, Sq, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)
        dq, dk, dv = torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(v)
    step = max(64, min(Sq, max(s["window"], 1024), (1 << 28) // (B * Hq * (2 * min(s["window"], s["Sk"]) + s["sinks"]))))
    for i0 in range(0, Sq, step):                                 # all scores at once are too many for long rows
        i1 = min(Sq, i0 + step)
        keys, seen = _chunk(s, i0, i1)
        kc, vc, qc = k[..., keys, :], v[..., keys, :], q[..., i0:i1, :]
        x = torch.where(seen, (qc @ kc.transpose(-1, -2)) * scale, -math.inf)
        top = x.amax(-1, keepdim=True)
        p = torch.exp(x - top)
        z = p.sum(-1, keepdim=True)
        p = p / z
        o = p @ vc
        out[..., i0:i1, :] = o
        lse[..., i0:i1] = (top + torch.log(z)).squeeze(-1)
        if train:
            g = do[..., i0:i1, :]
            ds = p * (g @ vc.transpose(-1, -2) - (g * o).sum(-1, keepdim=True)) * scale
            dq[..., i0:i1, :] = ds @ kc
            dk.index_add_(3, keys, (ds.transpose(-1, -2) @ qc).sum(2, keepdim=True))
            dv.index_add_(3, keys, (p.transpose(-1, -2) @ g).sum(2, keepdim=True))
    dt = s["q"].dtype

    def rows(x):
        return x.permute(0, 3, 1, 2, 4).reshape(B, x.shape[3], -1, D).to(dt)
    got = dict(out=rows(out), lse=lse.reshape(B, Hq, Sq))
    return got | dict(dq=rows(dq), dk=rows(dk), dv=rows(dv)) if train else got


def _run_append(s):
    B, n, Hkv, D, page = s["B"], s["n"], s["Hkv"], s["D"], s["page"]
    lens, end = s["lens"].long(), s["after"].long()
    # the blocks that the new tokens touch: held values of the older tokens, rows of the new ones
    T = (n + BLK - 2) // BLK + 1
    blk = (lens // BLK).unsqueeze(1) + torch.arange(T, device=DEV)                # [B, T]
    hit = blk * BLK < end.unsqueeze(1)
    per = page // BLK
    phys = s["pages"].gather(1, (blk // per).clamp(max=s["pages"].shape[1] - 1)).long()
    codes = s["cache"].view(torch.float8_e4m3fn).unflatten(3, (per, BLK))         # [P, Hkv, 2, per, 16, D]
    held, held_s = codes[phys, :, :, blk % per], s["scales"][phys, :, :, blk % per]   # [B, T, Hkv, 2, 16, D], [B, T, Hkv, 2]
    slot = blk.unsqueeze(2) * BLK + torch.arange(BLK, device=DEV)                 # [B, T, 16]
    new = (slot >= lens[:, None, None]) & (slot < end[:, None, None])
    row = (slot - lens[:, None, None]).clamp(0, n - 1).flatten(1)
    x = torch.stack([s["k"], s["v"]], 3).float()                                  # [B, n, Hkv, 2, D]
    x = x[torch.arange(B, device=DEV).unsqueeze(1), row].unflatten(1, (T, BLK)).permute(0, 1, 3, 4, 2, 5)
    mask = new[:, :, None, None, :, None]
    older = (blk * BLK < lens.unsqueeze(1))[..., None, None]
    top = _scale_of(torch.where(mask, x.abs(), 0.0).amax((-1, -2)))
    scale = torch.where(older, torch.maximum(held_s, top), top)
    grown = torch.where(older, held_s / scale, 1.0)[..., None, None]
    made = torch.where(mask, _codes(x, scale[..., None, None]).float(), (held.float() * grown))
    made = made.to(torch.float8_e4m3fn)
    cache8 = s["cache"].unflatten(3, (per, BLK))
    cache8[phys[hit], :, :, (blk % per)[hit]] = made.view(torch.uint8)[hit]
    s["scales"][phys[hit], :, :, (blk % per)[hit]] = scale[hit]
    # read back
    val = (made.float() * scale[..., None, None]).permute(0, 1, 4, 2, 3, 5).flatten(1, 2)   # [B, T 16, Hkv, 2, D]
    j = torch.arange(n, device=DEV)
    back = (lens % BLK).unsqueeze(1) + j
    val = val[torch.arange(B, device=DEV).unsqueeze(1), back]
    val = torch.where((j < (end - lens).unsqueeze(1))[..., None, None, None], val, 0.0).bfloat16()
    return dict(k=val[..., 0, :].contiguous(), v=val[..., 1, :].contiguous())


def _seen(s, L):
    """Whether token j of the batch sees slot l: [B, n, L]."""
    slot = torch.arange(L, device=DEV)
    limit = (s["lens"].long().unsqueeze(1) - (s["n"] - 1) + torch.arange(s["n"], device=DEV)).unsqueeze(-1)
    see = slot < limit
    return see & ((slot >= limit - s["window"]) | (slot < s["sinks"])) if s["window"] else see


def _run_attn(s):
    B, n, Hq, Hkv, D = s["B"], s["n"], s["Hq"], s["Hkv"], s["D"]
    k, v = _read(s["cache"], s["scales"], s["pages"])                             # [B, Hkv, L, D]
    see = _seen(s, k.shape[2])
    live = see.any(1)[:, None, :, None]
    k, v = torch.where(live, k, 0.0), torch.where(live, v, 0.0)                   # what nobody sees may hold anything
    q = s["q"].float().reshape(B, n, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).flatten(2, 3)   # [B, Hkv, R n, D]
    x = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    x = torch.where(see.unsqueeze(1).repeat(1, 1, Hq // Hkv, 1), x, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = torch.exp(x - top)
    z = p.sum(-1, keepdim=True)
    p = p / torch.where(z > 0, z, 1.0)
    out = (p @ v).unflatten(2, (Hq // Hkv, n)).permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)
    got = dict(out=out.bfloat16(), lse=(top + torch.log(z)).squeeze(-1).reshape(B, Hq, n))
    return got | dict(mass=s["mass"] + p.sum(2)) if s["mass"] is not False else got


def _run_evict(s):
    B, Hkv, D, page, budget = s["B"], s["Hkv"], s["D"], s["page"], s["budget"]
    lens = s["lens"].long()
    L = s["mass"].shape[-1]
    slot = torch.arange(L, device=DEV)
    there = (slot < lens.unsqueeze(1)).unsqueeze(1)
    forced = ((slot < s["first"]) | (slot >= (lens - s["last"]).unsqueeze(1))).unsqueeze(1)
    key = torch.where(there, torch.where(forced, math.inf, s["mass"]), -math.inf)
    n = min(budget, L)
    at = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :n]
    at = torch.where(at < lens[:, None, None], at, L).sort(-1).values             # ascending, L: none
    kept = torch.full((B, Hkv, budget), -1, dtype=torch.int32, device=DEV)
    kept[..., :n] = torch.where(at < L, at, -1)
    # rows of the kept slots, block by block of their new places
    cap = s["to"].shape[1] * page
    src = torch.full((B, Hkv, cap), -1, device=DEV)
    src[..., :n] = kept[..., :n].long()
    some, src = src >= 0, src.clamp(min=0)
    b = torch.arange(B, device=DEV)[:, None, None]
    h = torch.arange(Hkv, device=DEV)[None, :, None]
    phys = s["pages"].long()[b, src // page].clamp(min=0)
    codes = s["cache"][phys, h, :, src % page].view(torch.float8_e4m3fn).float()  # [B, Hkv, cap, 2, D]
    sc = s["scales"][phys, h, :, src % page // BLK]                               # [B, Hkv, cap, 2]
    new = torch.where(some.unsqueeze(-1), sc, 0.0).unflatten(2, (-1, BLK)).amax(3).repeat_interleave(BLK, 2)
    made = torch.where(some[..., None, None], codes * (sc / new.clamp(min=1e-30)).unsqueeze(-1), 0.0).to(torch.float8_e4m3fn)
    # into the new pages
    ph = s["to"].long()
    full = made.view(torch.uint8).unflatten(2, (-1, page)).permute(0, 2, 1, 4, 3, 5)        # [B, M, Hkv, 2, page, D]
    s["cache"][ph] = full.contiguous()
    s["scales"][ph] = new[:, :, ::BLK].unflatten(2, (-1, page // BLK)).permute(0, 2, 1, 4, 3).contiguous()
    value = (made.float() * new.unsqueeze(-1))[:, :, :budget].bfloat16().permute(3, 0, 2, 1, 4)
    mass = torch.zeros(B, Hkv, cap, device=DEV)
    mass[..., :] = torch.where(some, s["mass"].gather(2, src), 0.0)
    return dict(kept=kept, lens=lens.clamp(max=budget).int(), mass=mass, k=value[0].contiguous(), v=value[1].contiguous())


def run(s):
    op = s["op"]
    if own:
        from context_parallelism_02_gb300 import api
        if op == "fwd":
            out, lse = api.window_attn_fwd(s["q"], s["k"], s["v"], s["window"], s["sinks"])
            return dict(out=out, lse=lse)
        if op == "train":
            out, lse = api.window_attn_fwd(s["q"], s["k"], s["v"], s["window"], s["sinks"])
            dq, dk, dv = api.window_attn_bwd(s["q"], s["k"], s["v"], out, lse, s["dout"], s["window"], s["sinks"])
            return dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv)
        if op == "append":
            api.kv8_append(s["k"], s["v"], s["cache"], s["scales"], s["pages"], s["lens"], n_new=s["n_new"])
            k, v = api.kv8_gather(s["cache"], s["scales"], s["pages"], s["after"], s["n"], start=s["lens"])
            return dict(k=k, v=v)
        if op == "attn":
            mass = s["mass"].clone() if s["mass"] is not False else None
            out, lse = api.kv8_attn(s["q"], s["cache"], s["scales"], s["pages"], s["lens"], window=s["window"],
                                    sinks=s["sinks"], mass=mass)
            return dict(out=out, lse=lse) if mass is None else dict(out=out, lse=lse, mass=mass)
        kept, lens, mass = api.kv8_evict(s["cache"], s["scales"], s["pages"], s["lens"], s["mass"], s["to"], s["budget"],
                                         keep_first=s["first"], keep_last=s["last"])
        k, v = api.kv8_gather(s["cache"], s["scales"], s["to"], lens, s["budget"])
        return dict(kept=kept, lens=lens, mass=mass, k=k, v=v)
    if op in ("fwd", "train"):
        return _run_window(s)
    return dict(append=_run_append, attn=_run_attn, evict=_run_evict)[op](s)


def _pairs(case):
    """(query row, key) pairs of one head that are not masked."""
    whole = case["window"] + case["sinks"]                        # keys that a row sees from position `whole` - 1 on
    at, end = case["Sk"] - case["Sq"], case["Sk"]
    cut = min(max(at, whole), end)
    return (cut - at) * (at + 1 + cut) // 2 + (end - cut) * whole


def work(case):
    op, B, Hkv, D = case["op"], case["B"], case["Hkv"], case["D"]
    if op in ("fwd", "train"):
        e = 2 if case["dtype"] == "bf16" else 4
        q, kv, Hq = B * case["Sq"] * case["Hq"] * D * e, B * case["Sk"] * Hkv * D * e, case["Hq"]
        lse = B * Hq * case["Sq"] * 4
        n = _pairs(case) * B * Hq * D
        if op == "fwd":
            return dict(bytes=2 * q + 2 * kv + lse, flops=4 * n)
        return dict(bytes=4 * q + 4 * kv + lse, flops=14 * n)
    if op == "append":
        tokens = sum(_spread(case, 1, case["n"])) * Hkv
        e = 2 if case["dtype"] == "bf16" else 4
        # read the rows, write the codes; read them back as bf16
        return dict(bytes=tokens * (2 * D * e + 2 * D + 2 * D) + case["B"] * case["n"] * Hkv * 4 * D, flops=tokens * 4 * D)
    if op == "attn":
        n, Hq = case["n"], case["Hq"]
        seen = sum(min(x, case["window"] + n - 1 + case["sinks"]) if case["window"] else x
                   for x in _spread(case, min(n, case["L"]), case["L"])) * Hkv
        io = B * n * Hq * (4 * D + 4)
        return dict(bytes=seen * (2 * D + 8 / BLK + (8 if case["mass"] else 0)) + io, flops=seen * n * (Hq // Hkv) * 4 * D)
    lens = _spread(case, max(1, case["L"] // 16), case["L"])
    kept = sum(min(x, case["budget"]) for x in lens) * Hkv
    # the weights read, the kept rows moved and read back as bf16
    return dict(bytes=sum(lens) * Hkv * 4 + kept * (2 * 2 * D + 12 + 2 * D) + case["B"] * case["budget"] * Hkv * 4 * D, flops=0)


# --- the definitions in 64 bits -----------------------------------------------------------------------


def _exact_window(s):
    """Row blocks of one head at a time; the gradients by differentiating the definition."""
    B, Sq, Sk, Hq, Hkv, D, W = (s[x] for x in ("B", "Sq", "Sk", "Hq", "Hkv", "D", "window"))
    train = s["op"] == "train"
    out = torch.empty(B, Sq, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.empty(B, Hq, Sq, dtype=torch.float64, device=DEV)
    grads = [torch.zeros(s[x].shape, dtype=torch.float64, device=DEV) for x in ("q", "k", "v")] if train else None
    step = 1024 if W > 512 else 512
    with torch.set_grad_enabled(train):
        for b in range(B):
            for h in range(Hq):
                kv = h // (Hq // Hkv)
                for r0 in range(0, Sq, step):
                    r1 = min(Sq, r0 + step)
                    first, last = max(0, r0 + Sk - Sq - W + 1), r1 + Sk - Sq
                    near = torch.arange(first, last, device=DEV)
                    col = torch.cat([torch.arange(0, min(first, s["sinks"]), device=DEV), near])
                    q = s["q"][b, r0:r1, h].double().requires_grad_(train)
                    k = s["k"][b, :, kv].double()[col].requires_grad_(train)
                    v = s["v"][b, :, kv].double()[col].requires_grad_(train)
                    at = torch.arange(r0, r1, device=DEV)[:, None] + (Sk - Sq)
                    hidden = (col[None] > at) | ((at - col[None] >= W) & (col[None] >= s["sinks"]))
                    x = (torch.einsum("id,jd->ij", q, k) / math.sqrt(D)).masked_fill(hidden, -math.inf)
                    y = torch.einsum("ij,jd->id", torch.softmax(x, -1), v)
                    out[b, r0:r1, h] = y.detach()
                    lse[b, h, r0:r1] = torch.logsumexp(x.detach(), -1)
                    if train:
                        gq, gk, gv = torch.autograd.grad(y, (q, k, v), s["dout"][b, r0:r1, h].double())
                        grads[0][b, r0:r1, h] += gq
                        grads[1][b, :, kv].index_add_(0, col, gk)
                        grads[2][b, :, kv].index_add_(0, col, gv)
    got = dict(out=out, lse=lse)
    return got | dict(zip(("dq", "dk", "dv"), grads)) if train else got


def _e4m3(x):
    """x (64 bits) rounded to the nearest e4m3 value, ties to the even one."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -60))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _scale64(amax):
    e = torch.full_like(amax, E_MIN)
    for t in range(E_MIN, E_MAX):
        e = torch.where(amax > 448 * 2.0 ** t, t + 1.0, e)
    return torch.exp2(e)


def _code64(byte):
    """The value of an e4m3 byte by its bits."""
    b = byte.to(torch.int64)
    e, m = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e > 0, (1 + m / 8) * torch.exp2(e.double() - 7), m / 8 * 2.0 ** -6)
    return torch.where(b >= 128, -mag, mag)


def _slots64(s, b, h, count):
    """k, v [count, D] of the sequence's first slots."""
    page = s["page"]
    slot = torch.arange(count, device=DEV)
    ph = s["pages"][b].long()[slot // page]
    return [_code64(s["cache"][ph, h, w, slot % page]) * s["scales"][ph, h, w, slot % page // BLK].double().unsqueeze(-1)
            for w in (0, 1)]


def _exact_append(s):
    B, n, Hkv, D = s["B"], s["n"], s["Hkv"], s["D"]
    got = [torch.zeros(B, n, Hkv, D, dtype=torch.float64, device=DEV) for _ in range(2)]
    for b in range(B):
        a, z = int(s["lens"][b]), int(s["after"][b])
        for w, x in enumerate((s["k"], s["v"])):
            rows = x[b, :z - a].double().transpose(0, 1)                          # [Hkv, new, D]
            first = min(z, -(-a // BLK) * BLK) if a % BLK else a
            if a % BLK:                                                           # the block that they join
                ph, o = int(s["pages"][b, a // s["page"]]), a % s["page"] // BLK
                sc = torch.maximum(s["scales"][ph, :, w, o].double(), _scale64(rows[:, :first - a].abs().amax((1, 2))))
                got[w][b, :first - a] = (_e4m3(rows[:, :first - a] / sc[:, None, None]) * sc[:, None, None]).transpose(0, 1)
            rest = rows[:, first - a:]
            m = -(-rest.shape[1] // BLK)
            if m:
                pad = torch.zeros(Hkv, m * BLK, D, dtype=torch.float64, device=DEV)
                pad[:, :rest.shape[1]] = rest
                pad = pad.reshape(Hkv, m, BLK * D)
                sc = _scale64(pad.abs().amax(-1, keepdim=True))
                val = (_e4m3(pad / sc) * sc).reshape(Hkv, m * BLK, D)[:, :rest.shape[1]]
                got[w][b, first - a:z - a] = val.transpose(0, 1)
    return dict(k=got[0], v=got[1])


def _exact_attn(s):
    B, n, Hq, Hkv, D = s["B"], s["n"], s["Hq"], s["Hkv"], s["D"]
    out = torch.zeros(B, n, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, Hq, n), -math.inf, dtype=torch.float64, device=DEV)
    mass = s["mass"].double() if s["mass"] is not False else None
    for b in range(B):
        L = int(s["lens"][b])
        for h in range(Hkv):
            k, v = _slots64(s, b, h, L)
            for j in range(n):
                limit = L - n + 1 + j
                use = torch.zeros(L, dtype=torch.bool, device=DEV)
                use[max(0, limit - s["window"]) if s["window"] else 0:max(0, limit)] = True
                use[:max(0, min(s["sinks"], limit))] = True
                rows = slice(h * Hq // Hkv, (h + 1) * Hq // Hkv)
                if bool(use.any()):
                    at = use.nonzero().squeeze(1)
                    x = s["q"][b, j, rows].double() @ k[at].T / math.sqrt(D)
                    z = torch.logsumexp(x, -1, keepdim=True)
                    p = torch.exp(x - z)
                    out[b, j, rows], lse[b, rows, j] = p @ v[at], z.squeeze(-1)
                    if mass is not None:
                        mass[b, h, at] += p.sum(0)
    return dict(out=out, lse=lse) if mass is None else dict(out=out, lse=lse, mass=mass)


def _exact_evict(s):
    B, Hkv, D, budget, page = s["B"], s["Hkv"], s["D"], s["budget"], s["page"]
    cap = s["to"].shape[1] * page
    kept = torch.full((B, Hkv, budget), -1, dtype=torch.int32, device=DEV)
    mass = torch.zeros(B, Hkv, cap, dtype=torch.float64, device=DEV)
    got = [torch.zeros(B, budget, Hkv, D, dtype=torch.float64, device=DEV) for _ in range(2)]
    for b in range(B):
        L = int(s["lens"][b])
        n = min(L, budget)
        for h in range(Hkv):
            m = s["mass"][b, h, :L].double().clone()
            m[:s["first"]] = math.inf
            m[max(0, L - s["last"]):] = math.inf
            top = torch.sort(m, descending=True, stable=True).indices[:n]
            take = torch.sort(top).values
            kept[b, h, :n] = take.int()
            mass[b, h, :n] = s["mass"][b, h, take].double()
            ph = s["pages"][b].long()[take // page]
            for w in (0, 1):
                code = _code64(s["cache"][ph, h, w, take % page])
                sc = s["scales"][ph, h, w, take % page // BLK].double()
                big = torch.zeros(-(-n // BLK) * BLK, dtype=torch.float64, device=DEV)
                big[:n] = sc
                big = big.reshape(-1, BLK).amax(1).repeat_interleave(BLK)[:n, None]
                got[w][b, :n, h] = _e4m3(code * sc[:, None] / big) * big
    return dict(kept=kept, lens=s["lens"].clamp(max=budget).int(), mass=mass, k=got[0], v=got[1])


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("fwd", "train"):
        return _exact_window(s)
    return dict(append=_exact_append, attn=_exact_attn, evict=_exact_evict)[op](s)
