"""Cases and plain forms of the paged 4-bit cache operators.

A long prompt is prefilled by ring attention; its keys and values then live in
a paged cache that holds them in 4 bits, and decoding reads that cache once per
token.  The operators: ``append`` (rotate q and k, quantise k and v, write them
into pages, and read the written rows back as the rows that ring attention
takes), ``gather`` (a range of cached tokens back as BSHD), ``attn`` (attention
of a few query tokens over the whole cache) and ``sparse`` (pages selected per
query by a bound on q.k, then attention over those pages).

Cache format, per page and kv head, in blocks of 16 tokens of 20 D bytes:
K codes [8 D], K scale/minimum pairs in fp16 [D / 32 per token], V codes [8 D],
V scales and minima; a group of 32 neighbouring d shares a scale and a minimum,
value = scale * code + minimum.
"""
import math

import torch

own = False

DEV = "cuda"
G = 32                                   # elements that share a scale and a minimum
K_ORDER = (0, 2, 4, 6, 1, 3, 5, 7)       # nibble e of a K word holds element K_ORDER[e] of its 8


def listed():
    return [
        # one new token of one conversation: pure latency
        dict(name="append_one_token", op="append", B=1, n=1, Hq=32, Hkv=8, D=128, page=64, past=32767, dtype="bf16",
             rot=128, interleaved=False, fused=False, summary=True, ragged=False),
        # the whole prompt after a ring prefill of 32768 tokens, q/k/v as views of one projection's output
        dict(name="append_prompt_32k", op="append", B=1, n=32768, Hq=32, Hkv=8, D=128, page=64, past=0, dtype="bf16",
             rot=128, interleaved=False, fused=True, summary=True, ragged=False),
        # padded batch of odd chunks, fp32 inputs, partial interleaved rotation, small pages
        dict(name="append_ragged_fp32", op="append", B=7, n=1001, Hq=6, Hkv=2, D=64, page=16, past=300, dtype="f32",
             rot=32, interleaved=True, fused=False, summary=False, ragged=True),
        # a short context read back for the next chunk's ring step
        dict(name="gather_1k", op="gather", B=1, count=1024, Hkv=8, D=128, page=64, dtype="bf16"),
        # a 32k context of four sequences read back
        dict(name="gather_4x32k", op="gather", B=4, count=32768, Hkv=8, D=128, page=64, dtype="bf16"),
        # one token over a short context: latency
        dict(name="attn_short_512", op="attn", B=1, n=1, L=512, Hq=32, Hkv=8, D=128, page=64, ragged=False),
        # ragged serving batch, lengths from 1 to 8192
        dict(name="attn_ragged_64x8k", op="attn", B=64, n=1, L=8192, Hq=32, Hkv=8, D=128, page=16, ragged=True),
        # one token over the long prompt, one query head per kv head
        dict(name="attn_long_128k", op="attn", B=1, n=1, L=131072, Hq=8, Hkv=8, D=128, page=64, ragged=False),
        # a serving batch of 32k contexts
        dict(name="attn_16x32k", op="attn", B=16, n=1, L=32768, Hq=32, Hkv=8, D=128, page=64, ragged=False),
        # eight drafted tokens checked at once, causal among themselves
        dict(name="attn_draft_8_tokens", op="attn", B=4, n=8, L=16384, Hq=16, Hkv=4, D=64, page=32, ragged=True),
        # one token over the long prompt, 64 of 2048 pages
        dict(name="sparse_long_128k", op="sparse", B=1, n=1, L=131072, Hq=32, Hkv=8, D=128, page=64, n_sel=64,
             ragged=False),
        # the same in a ragged batch, 64 of up to 1024 pages
        dict(name="sparse_16x32k", op="sparse", B=16, n=1, L=32768, Hq=32, Hkv=8, D=128, page=32, n_sel=64,
             ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "gather", "attn", "attn", "sparse"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        B = _log(rng, 1, 128)
        n = _log(rng, 1, max(1, 16384 // B))
        return dict(op=op, B=B, n=n, Hq=Hkv * rng.choice([1, 2, 3, 4, 8]), Hkv=Hkv, D=D, page=page,
                    past=_log(rng, 1, 8192) - 1, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    rot=rng.choice([D, D, D // 2]), interleaved=rng.random() < 0.3, fused=rng.random() < 0.5,
                    summary=rng.random() < 0.5, ragged=rng.random() < 0.5)
    if op == "gather":
        B = _log(rng, 1, 16)
        return dict(op=op, B=B, count=_log(rng, 1, 131072 // B), Hkv=Hkv, D=D, page=page,
                    dtype=rng.choice(["bf16", "f32"]))
    if op == "attn":
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, n=rng.choice([1, 1, 1, 1, 2, 5, 8, 16]), L=_log(rng, 16, 524288 // max(B, 4)),
                    Hq=Hkv * rng.choice([1, 2, 4, 4, 7, 8, 16]), Hkv=Hkv, D=D, page=page, ragged=rng.random() < 0.5)
    B = _log(rng, 1, 16)
    return dict(op=op, B=B, n=rng.choice([1, 1, 1, 2, 3]), L=_log(rng, 2048, 524288 // max(B, 4)),
                Hq=Hkv * rng.choice([1, 2, 4, 8]), Hkv=Hkv, D=D, page=page, n_sel=_log(rng, 8, 64),
                ragged=rng.random() < 0.5)


# --- the cache format, in elementary operations ------------------------------------------------------


def _quantise(x):
    """codes (uint8), scale and minimum (fp16) of groups of 32 along the last axis of x (fp32)."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // G, G)
    lo, hi = g.amin(-1), g.amax(-1)
    s = ((hi - lo) / 15.0).half()
    m = lo.half()
    sf = s.float().unsqueeze(-1)
    code = torch.where(sf > 0, (g - m.float().unsqueeze(-1)) / torch.where(sf > 0, sf, 1.0), 0.0)
    return code.round().clamp(0, 15).to(torch.uint8).reshape(x.shape), s, m


def _nibbles(codes):
    """Last axis of nibbles (even first) -> bytes."""
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _pack(k, v):
    """[..., 16, D] fp32 blocks of k and v -> [..., 20 D] bytes."""
    lead, D = k.shape[:-2], k.shape[-1]
    ng = D // G
    kc, ks, km = _quantise(k)
    vc, vs, vm = _quantise(v)
    # K codes: token, c (8-element run of the group), group, nibble e
    kc = kc.reshape(*lead, 16, ng, 4, 8)[..., list(K_ORDER)].transpose(-3, -2)
    kb = _nibbles(kc).reshape(*lead, 8 * D)
    kmeta = torch.stack([ks, km], -1).contiguous().view(torch.uint8).reshape(*lead, 64 * ng)
    # V codes: token = half * 8 + 2 c + low, d = 32 group + 4 g + e -> half, g, c, group, low, e
    nl = len(lead)
    vc = vc.reshape(*lead, 2, 4, 2, ng, 8, 4).permute(*range(nl), nl, nl + 4, nl + 1, nl + 3, nl + 2, nl + 5)
    vb = _nibbles(vc).reshape(*lead, 8 * D)
    # V scales and minima: half, c, group, (scale, minimum), low
    vmeta = torch.stack([vs, vm], -2).reshape(*lead, 2, 4, 2, 2, ng)      # half, c, low, which, group
    vmeta = vmeta.permute(*range(nl), nl, nl + 1, nl + 4, nl + 3, nl + 2).contiguous()
    vmeta = vmeta.view(torch.uint8).reshape(*lead, 64 * ng)
    return torch.cat([kb, kmeta, vb, vmeta], -1)


def _unpack(b):
    """[..., 20 D] bytes -> k, v [..., 16, D] fp32."""
    lead, D = b.shape[:-1], b.shape[-1] // 20
    ng, nl = D // G, b.dim() - 1

    def codes(x):
        return torch.stack([x & 15, x >> 4], -1).reshape(*x.shape[:-1], 2 * x.shape[-1])

    def half(x):
        return x.contiguous().view(torch.float16).float()
    kb, kmeta, vb, vmeta = b.split([8 * D, 64 * ng, 8 * D, 64 * ng], -1)
    inv = sorted(range(8), key=lambda e: K_ORDER[e])
    kc = codes(kb).reshape(*lead, 16, 4, ng, 8)[..., inv].transpose(-3, -2)          # token, group, c, element
    kmeta = half(kmeta).reshape(*lead, 16, ng, 1, 2)
    k = kc.float().reshape(*lead, 16, ng, 4, 8) * kmeta[..., 0:1] + kmeta[..., 1:2]
    vc = codes(vb).reshape(*lead, 2, 8, 4, ng, 2, 4).permute(*range(nl), nl, nl + 2, nl + 4, nl + 3, nl + 1, nl + 5)
    vmeta = half(vmeta).reshape(*lead, 2, 4, ng, 2, 2).permute(*range(nl), nl, nl + 1, nl + 4, nl + 2, nl + 3)
    v = vc.float() * vmeta[..., 0].unsqueeze(-1).unsqueeze(-1) + vmeta[..., 1].unsqueeze(-1).unsqueeze(-1)
    return k.reshape(*lead, 16, D), v.reshape(*lead, 16, D)


def _read(cache, pages):
    """Cache pages [...] of the pool -> k, v [..., Hkv, page, D] fp32."""
    P, Hkv, page, w = cache.shape
    b = cache[pages.long()].reshape(*pages.shape, Hkv, page // 16, 16 * w)
    k, v = _unpack(b)
    return k.reshape(*pages.shape, Hkv, page, -1), v.reshape(*pages.shape, Hkv, page, -1)


# --- inputs -------------------------------------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 2654435761 % (1 << 31) + 17)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _lens(case, g, lo, hi):
    """Lengths of the batch: all `hi`, or spread over [lo, hi] with one of each end."""
    B = case["B"]
    if not case["ragged"]:
        return torch.full((B,), hi, dtype=torch.int32, device=DEV)
    u = torch.rand(B, generator=g, device=DEV)
    x = torch.exp(math.log(lo) + u * (math.log(hi + 1) - math.log(lo))).floor().clamp(lo, hi)
    x[B // 2] = lo
    x[0] = hi
    return x.to(torch.int32)


def _pool(case, g, L, content=True):
    """A pool with room for B sequences of L tokens, its pages in random order, and the page table."""
    B, Hkv, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    M = -(-L // page)
    P = B * M + 3
    cache = torch.zeros(P, Hkv, page, D + D // 4, dtype=torch.uint8, device=DEV)
    summary = torch.zeros(P, Hkv, 2, D, dtype=torch.bfloat16, device=DEV)
    if content:
        for a in range(0, P, max(1, (1 << 25) // (Hkv * page * D))):   # a slab at a time: a pool of several GB
            p = min(P, a + max(1, (1 << 25) // (Hkv * page * D))) - a
            # the tokens of a page have something in common, as neighbouring tokens do
            k = (_randn(g, p, Hkv, page, D) + 0.7 * _randn(g, p, Hkv, 1, D)).bfloat16().float()
            v = _randn(g, p, Hkv, page, D).bfloat16().float()
            cache[a:a + p] = _pack(k.reshape(p, Hkv, page // 16, 16, D),
                                   v.reshape(p, Hkv, page // 16, 16, D)).reshape(p, Hkv, page, -1)
            summary[a:a + p] = torch.stack([k.amin(2), k.amax(2)], 2).bfloat16()
    order = torch.randperm(P, generator=g, device=DEV)[:B * M]
    return cache, summary, order.reshape(B, M).to(torch.int32)


def _unused(pages, lens, page):
    """Entries behind a sequence's last page name no page."""
    used = torch.arange(pages.shape[1], device=DEV) * page < lens.unsqueeze(1)
    return torch.where(used, pages, -1).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    op, B, Hkv, D, page = case["op"], case["B"], case["Hkv"], case["D"], case["page"]
    s = dict(case)
    if op == "append":
        n, Hq, R = case["n"], case["Hq"], case["rot"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        lens = _lens(case, g, max(1, case["past"] // 2), max(1, case["past"]))
        lens = lens if case["past"] else torch.zeros_like(lens)
        cache, summary, pages = _pool(case, g, case["past"] + n, content=False)
        n_new = _lens(case, g, 1, n) if case["ragged"] else None
        if case["fused"]:
            x = _randn(g, B, n, (Hq + 2 * Hkv) * D).to(dt)
            q, k, v = (t.unflatten(-1, (-1, D)) for t in x.split([Hq * D, Hkv * D, Hkv * D], -1))
        else:
            q, k, v = (_randn(g, B, n, h, D).to(dt) for h in (Hq, Hkv, Hkv))
        top = case["past"] + n
        ang = torch.arange(top, dtype=torch.float64, device=DEV).unsqueeze(1) * (
            10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=DEV) / R))
        s.update(q=q, k=k, v=v, cache=cache, summary=summary if case["summary"] else None, pages=pages, lens=lens,
                 n_new=n_new, after=lens + (n if n_new is None else n_new), cos=ang.cos().float(), sin=ang.sin().float())
        return s
    if op == "gather":
        cache, _, pages = _pool(case, g, case["count"])
        lens = torch.full((B,), case["count"], dtype=torch.int32, device=DEV)
        s.update(cache=cache, pages=pages, lens=lens)
        return s
    n = case["n"]
    cache, summary, pages = _pool(case, g, case["L"])
    lens = _lens(case, g, max(n, 1), max(n, case["L"])) if op == "attn" else _lens(case, g, case["L"] // 8, case["L"])
    lens = lens.clamp(max=case["L"])
    s.update(cache=cache, summary=summary, pages=_unused(pages, lens, page), lens=lens,
             q=_randn(g, B, n, case["Hq"], D).bfloat16())
    return s


# --- one pass -----------------------------------------------------------------------------------------


def _rotate(x, cos, sin, R, interleaved):
    x = x.float()
    r = x[..., :R]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :R // 2], r[..., R // 2:])
    y1, y2 = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([y1, y2], -1).flatten(-2) if interleaved else torch.cat([y1, y2], -1)
    return torch.cat([y, x[..., R:]], -1)


def _run_append(s):
    B, n, Hkv, D, page, R = s["B"], s["n"], s["Hkv"], s["D"], s["page"], s["rot"]
    j = torch.arange(n, device=DEV)
    pos = s["lens"].long().unsqueeze(1) + j                                       # [B, n]
    live = torch.ones_like(pos, dtype=torch.bool) if s["n_new"] is None else j < s["n_new"].unsqueeze(1)
    cos, sin = s["cos"][pos.clamp(max=s["cos"].shape[0] - 1)].unsqueeze(2), s["sin"][
        pos.clamp(max=s["cos"].shape[0] - 1)].unsqueeze(2)
    q = _rotate(s["q"], cos, sin, R, s["interleaved"]).to(s["q"].dtype)
    q = torch.where(live[..., None, None], q, 0)
    k = _rotate(s["k"], cos, sin, R, s["interleaved"])
    v = s["v"].float()
    # the pages that the new tokens touch, unpacked into bytes of single values, changed, and packed again
    M = s["pages"].shape[1]
    P = s["cache"].shape[0]
    first = s["lens"].long() // page
    T = (n + page - 2) // page + 1
    lp = first.unsqueeze(1) + torch.arange(T, device=DEV)                         # [B, T] pages touched
    end = s["lens"].long() + (n if s["n_new"] is None else s["n_new"].long())
    hit = lp * page < end.unsqueeze(1)
    phys = torch.where(hit, s["pages"].gather(1, lp.clamp(max=M - 1)).long(), P)
    slot = lp.unsqueeze(2) * page + torch.arange(page, device=DEV)                # [B, T, page]
    new = (slot >= s["lens"].long()[:, None, None]) & (slot < end[:, None, None])
    row = (slot - s["lens"].long()[:, None, None]).clamp(0, n - 1)
    at = row.reshape(B, T * page, 1, 1).expand(B, T * page, Hkv, D)

    def paged(x):
        return x.gather(1, at).reshape(B, T, page, Hkv, D).transpose(2, 3)        # [B, T, Hkv, page, D]
    kn, vn = paged(k), paged(v)
    held = s["cache"][phys.clamp(max=P - 1)]                                      # [B, T, Hkv, page, w]
    w = held.shape[-1]
    mask = new[:, :, None, :, None].expand(B, T, Hkv, page, D)
    ones = torch.where(mask, 1.0, 0.0)
    blocks = (B, T, Hkv, page // 16, 16, D)
    fresh = _pack(kn.reshape(blocks), vn.reshape(blocks))
    own_bits = _mask_bytes(ones.reshape(blocks))
    merged = torch.where(own_bits, fresh, held.reshape(B, T, Hkv, page // 16, 16 * w))
    s["cache"][phys[hit]] = merged.reshape(B, T, Hkv, page, w)[hit]
    out = dict(q=q)
    if s["summary"] is not None:
        kb = kn.bfloat16().float()
        lo = torch.where(mask, kb, math.inf).amin(3)
        hi = torch.where(mask, kb, -math.inf).amax(3)
        old = s["summary"][phys.clamp(max=P - 1)].float()
        kept = (lp * page < s["lens"].long().unsqueeze(1))[:, :, None, None]      # older tokens in the page
        lo = torch.where(kept, torch.minimum(lo, old[:, :, :, 0]), lo)
        hi = torch.where(kept, torch.maximum(hi, old[:, :, :, 1]), hi)
        s["summary"][phys[hit]] = torch.stack([lo, hi], 3).bfloat16()[hit]
        out["summary"] = s["summary"]
    kh, vh = _read(s["cache"], phys.clamp(max=P - 1))                             # [B, T, Hkv, page, D]
    back = (pos - (first * page).unsqueeze(1)).reshape(B, n, 1, 1).expand(B, n, Hkv, D)
    for name, x in (("k", kh), ("v", vh)):
        x = x.transpose(2, 3).reshape(B, T * page, Hkv, D).gather(1, back)
        out[name] = torch.where(live[..., None, None], x, 0.0).bfloat16()
    return out


def _mask_bytes(ones):
    """[..., 16, D] of 1 and 0 (equal over a token) -> [..., 20 D], whether the byte is that token's."""
    lead, D, nl = ones.shape[:-2], ones.shape[-1], ones.dim() - 2
    t = ones[..., 0] > 0                                                          # [..., 16]
    ng = D // G
    kb = t.unsqueeze(-1).expand(*lead, 16, D // 2).reshape(*lead, 8 * D)
    km = t.unsqueeze(-1).expand(*lead, 16, 4 * ng).reshape(*lead, 64 * ng)
    h = t.reshape(*lead, 2, 1, 4, 1, 2, 1).expand(*lead, 2, 8, 4, ng, 2, 2).reshape(*lead, 8 * D)
    m = t.reshape(*lead, 2, 4, 1, 1, 2, 1).expand(*lead, 2, 4, ng, 2, 2, 2).reshape(*lead, 64 * ng)
    return torch.cat([kb, km, h, m], -1)


def _attend(q, k, v, seen):
    """q [B, n, Hkv, R, D], k and v [B, n or 1, Hkv, L, D], seen [B, n, 1 or Hkv, 1, L] -> out, lse."""
    s = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(q.shape[-1]))
    s = torch.where(seen, s, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    lse = torch.log(total) + top
    out = (p @ v) / torch.where(total > 0, total, 1.0)
    return out, lse.squeeze(-1)


def _finish(s, out, lse):
    B, n, Hq, D = s["q"].shape
    return out.reshape(B, n, Hq, D).bfloat16(), lse.reshape(B, n, Hq).transpose(1, 2).contiguous()


def _limits(s):
    n = s["n"]
    return s["lens"].long().unsqueeze(1) - (n - 1) + torch.arange(n, device=DEV)  # [B, n] slots that a row sees


def _run_attn(s):
    B, n, Hq, Hkv, D, page = s["B"], s["n"], s["Hq"], s["Hkv"], s["D"], s["page"]
    k, v = _read(s["cache"], s["pages"].clamp(min=0))                             # [B, M, Hkv, page, D]
    L = k.shape[1] * page
    k, v = (x.transpose(1, 2).reshape(B, 1, Hkv, L, D) for x in (k, v))
    R = Hq // Hkv
    # rows of a kv head: token-major, then head of the group
    q = s["q"].float().reshape(B, 1, n, Hkv, R, D).transpose(2, 3).reshape(B, 1, Hkv, n * R, D)
    seen = torch.arange(L, device=DEV) < _limits(s).reshape(B, n, 1, 1).expand(B, n, R, 1).reshape(B, 1, 1, n * R, 1)
    out, lse = _attend(q, k, v, seen)
    out = out.reshape(B, Hkv, n, R, D).transpose(1, 2)
    return _finish(s, out, lse.reshape(B, Hkv, n, R).transpose(1, 2))


def _run_sparse(s):
    B, n, Hq, Hkv, D, page = s["B"], s["n"], s["Hq"], s["Hkv"], s["D"], s["page"]
    M = s["pages"].shape[1]
    q = s["q"].reshape(B, n, Hkv, Hq // Hkv, D)
    # 64 bits: which page comes last among the selected hangs on small differences
    box = s["summary"][s["pages"].clamp(min=0).long()].double().transpose(1, 2).unsqueeze(1)   # [B, 1, Hkv, M, 2, D]
    qd = q.double()
    score = (qd.clamp(max=0) @ box[..., 0, :].transpose(-1, -2) +
             qd.clamp(min=0) @ box[..., 1, :].transpose(-1, -2)).amax(3)                       # [B, n, Hkv, M]
    limit = _limits(s).clamp(min=0)
    count = ((limit + page - 1) // page)[..., None, None]
    idx = torch.arange(M, device=DEV)
    score = torch.where((idx < 1) | (idx >= count - 1), math.inf, score)
    score = torch.where(idx < count, score, -math.inf)
    N = s["n_sel"]
    order = score.sort(dim=-1, descending=True, stable=True)
    sel = order.indices[..., :N]
    real = order.values[..., :N] > -math.inf                                                   # [B, n, Hkv, N]
    phys = s["pages"].clamp(min=0).long()[:, None, None].expand(B, n, Hkv, M).gather(-1, sel)
    P, _, _, w = s["cache"].shape
    rows = s["cache"].reshape(P * Hkv, page // 16, 16 * w)[phys * Hkv + torch.arange(Hkv, device=DEV)[:, None]]
    k, v = (x.reshape(B, n, Hkv, sel.shape[-1] * page, D) for x in _unpack(rows))
    slot = (sel.unsqueeze(-1) * page + torch.arange(page, device=DEV)).reshape(B, n, Hkv, 1, -1)
    seen = (slot < limit[..., None, None, None]) & real.unsqueeze(-1).expand(*real.shape, page).reshape(B, n, Hkv, 1, -1)
    out, lse = _attend(q.float(), k, v, seen)
    return _finish(s, out, lse)


def _run_gather(s):
    B, n, Hkv, D = s["B"], s["count"], s["Hkv"], s["D"]
    dt = torch.bfloat16 if s["dtype"] == "bf16" else torch.float32
    k, v = _read(s["cache"], s["pages"])
    return [x.transpose(2, 3).reshape(B, -1, Hkv, D)[:, :n].to(dt).contiguous() for x in (k, v)]


def run(state):
    s = state
    if own:
        from context_parallelism_02_gb300 import api
        if s["op"] == "append":
            q = api.kv4_append(s["k"], s["v"], s["cache"], s["pages"], s["lens"], s["cos"], s["sin"], q=s["q"],
                               n_new=s["n_new"], summary=s["summary"], interleaved=s["interleaved"])
            k, v = api.kv4_gather(s["cache"], s["pages"], s["after"], s["n"], start=s["lens"])
            out = dict(q=q, k=k, v=v)
            if s["summary"] is not None:
                out["summary"] = s["summary"]
            return out
        if s["op"] == "gather":
            return list(api.kv4_gather(s["cache"], s["pages"], s["lens"], s["count"],
                                       dtype=torch.bfloat16 if s["dtype"] == "bf16" else torch.float32))
        if s["op"] == "attn":
            return api.kv4_attn(s["q"], s["cache"], s["pages"], s["lens"])
        sel = api.kv4_select(s["q"], s["summary"], s["pages"], s["lens"], s["page"], s["n_sel"])
        return api.kv4_attn(s["q"], s["cache"], s["pages"], s["lens"], sel=sel)
    return dict(append=_run_append, gather=_run_gather, attn=_run_attn, sparse=_run_sparse)[s["op"]](s)


# --- what a pass cannot do without --------------------------------------------------------------------


def work(case):
    op, B, Hkv, D, page = case["op"], case["B"], case["Hkv"], case["D"], case["page"]
    token = Hkv * (D + D // 4)                        # bytes of a cached token, k and v
    if op == "gather":
        return dict(bytes=B * case["count"] * (token + 2 * Hkv * D * (2 if case["dtype"] == "bf16" else 4)),
                    flops=4 * B * case["count"] * Hkv * D)
    n, Hq = case["n"], case["Hq"]
    mean = 1.0
    if case["ragged"]:                                # lengths spread over their logarithm
        hi = {"append": n, "attn": case["L"] if op == "attn" else 0}.get(op, case.get("L", 0))
        lo = {"append": 1, "attn": min(n, hi)}.get(op, max(1, hi // 8))
        mean = (hi - lo) / (hi * math.log(hi / lo)) if hi > lo else 1.0
    if op == "append":
        e = 2 if case["dtype"] == "bf16" else 4
        rows = B * n * mean
        return dict(bytes=rows * (2 * Hkv * D * e + 2 * Hq * D * e + 4 * case["rot"] + token + 2 * Hkv * D * 2),
                    flops=rows * (3 * (Hq + Hkv) * case["rot"] + 8 * Hkv * D))
    io = B * n * Hq * (4 * D + 4)
    L = case["L"] * mean
    if op == "attn":
        return dict(bytes=B * L * token + io, flops=4.0 * D * Hq * B * n * L)
    picked = min(L, case["n_sel"] * page)
    return dict(bytes=B * (L / page) * Hkv * 4 * D + B * n * picked * token + io,
                flops=4.0 * D * Hq * B * n * (picked + L / page))


# --- the definitions in 64 bits -----------------------------------------------------------------------


def _places(D):
    """For token t and element d of a block: byte and shift of the codes of k and v, and the half-word
    (from the block's start) of their scale; the minimum is `step` half-words on."""
    ng = D // G
    kb, ks, vb, vs, km, vm = ([[0] * D for _ in range(16)] for _ in range(6))
    for t in range(16):
        half, c, low = t // 8, t % 8 // 2, t % 2
        for d in range(D):
            gr, r = divmod(d, G)
            e = K_ORDER.index(r % 8)
            kb[t][d], ks[t][d] = t * (D // 2) + r // 8 * 4 * ng + gr * 4 + e // 2, e % 2 * 4
            km[t][d] = (8 * D + t * 4 * ng + gr * 4) // 2
            e = r % 4
            vb[t][d] = 8 * D + 64 * ng + half * 128 * ng + (r // 4 * 4 + c) * 4 * ng + gr * 4 + low * 2 + e // 2
            vs[t][d] = e % 2 * 4
            vm[t][d] = (16 * D + 64 * ng + ((half * 4 + c) * ng + gr) * 8) // 2 + low
    return [torch.tensor(x, device=DEV) for x in (kb, ks, km, vb, vs, vm)]


def _decode64(blocks, D):
    """[N, 20 D] bytes -> k, v [N, 16, D] in 64 bits."""
    kb, ks, km, vb, vs, vm = _places(D)
    meta = blocks.contiguous().view(torch.float16)
    k = (blocks[:, kb] >> ks.to(torch.uint8) & 15).double() * meta[:, km].double() + meta[:, km + 1].double()
    v = (blocks[:, vb] >> vs.to(torch.uint8) & 15).double() * meta[:, vm].double() + meta[:, vm + 2].double()
    return k, v


def _tokens64(s, pages, h):
    """Slots of the pages [m] of one kv head: k, v [m * page, D]."""
    page, D = s["page"], s["D"]
    blocks = s["cache"][pages.long(), h].reshape(-1, 20 * D)
    parts = [_decode64(b, D) for b in blocks.split(4096)]
    return [torch.cat([p[i] for p in parts]).reshape(-1, D) for i in (0, 1)]


def _exact_rows(s, b, j, h, slots, k, v, out, lse):
    R = s["Hq"] // s["Hkv"]
    limit = int(s["lens"][b]) - (s["n"] - 1) + j
    see = slots < limit
    x = s["q"][b, j, h * R:(h + 1) * R].double() @ k.T / math.sqrt(s["D"])
    x = x.masked_fill(~see, -math.inf)
    z = torch.logsumexp(x, -1)
    w = torch.exp(x - z.masked_fill(z == -math.inf, 0.0).unsqueeze(-1))
    out[b, j, h * R:(h + 1) * R] = w @ v
    lse[b, h * R:(h + 1) * R, j] = z


def exact(case, seed):
    s = prepare(case, seed)
    op, B, Hkv, D, page = s["op"], s["B"], s["Hkv"], s["D"], s["page"]
    if op == "gather":
        k = torch.empty(B, s["count"], Hkv, D, dtype=torch.float64, device=DEV)
        v = torch.empty_like(k)
        for b in range(B):
            for h in range(Hkv):
                kk, vv = _tokens64(s, s["pages"][b], h)
                k[b, :, h], v[b, :, h] = kk[:s["count"]], vv[:s["count"]]
        return [k, v]
    n, Hq = s["n"], s["Hq"]
    if op == "append":
        return _exact_append(s)
    out = torch.zeros(B, n, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, Hq, n), -math.inf, dtype=torch.float64, device=DEV)
    for b in range(B):
        L = int(s["lens"][b])
        pages = s["pages"][b, :-(-L // page)]
        for h in range(Hkv):
            if op == "attn":
                k, v = _tokens64(s, pages, h)
                slots = torch.arange(k.shape[0], device=DEV)
                for j in range(n):
                    _exact_rows(s, b, j, h, slots, k, v, out, lse)
                continue
            box = s["summary"][pages.long(), h].double()                       # [m, 2, D]
            for j in range(n):
                limit = L - (n - 1) + j
                m = -(-limit // page)
                q = s["q"][b, j, h * Hq // Hkv:(h + 1) * Hq // Hkv].double()
                bound = torch.maximum(q[:, None] * box[None, :m, 0], q[:, None] * box[None, :m, 1]).sum(-1).amax(0)
                bound[0] = bound[m - 1] = math.inf
                take = torch.argsort(-bound, stable=True)[:s["n_sel"]]
                k, v = _tokens64(s, pages[take], h)
                slots = (take[:, None] * page + torch.arange(page, device=DEV)).reshape(-1)
                _exact_rows(s, b, j, h, slots, k, v, out, lse)
    return out, lse


def _exact_append(s):
    B, n, Hkv, D, page, R = s["B"], s["n"], s["Hkv"], s["D"], s["page"], s["rot"]
    live = torch.arange(n, device=DEV) < (s["after"] - s["lens"]).unsqueeze(1)
    at = (s["lens"].long().unsqueeze(1) + torch.arange(n, device=DEV)).clamp(max=s["cos"].shape[0] - 1)
    turn = torch.complex(s["cos"].double(), s["sin"].double())[at].unsqueeze(2)

    def rotated(x):
        x = x.double()
        if s["interleaved"]:
            z = torch.view_as_complex(x[..., :R].reshape(*x.shape[:-1], R // 2, 2).contiguous()) * turn
            y = torch.view_as_real(z).reshape(*x.shape[:-1], R)
        else:
            z = torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous()) * turn
            y = torch.cat([z.real, z.imag], -1)
        return torch.cat([y, x[..., R:]], -1) * live[..., None, None]

    def held(x):
        g = x.reshape(*x.shape[:-1], D // G, G)
        low = g.min(-1, keepdim=True).values
        step = ((g.max(-1, keepdim=True).values - low) / 15).half().double()
        low = low.half().double()
        code = torch.where(step > 0, (g - low) / step.clamp(min=1e-30), 0.0).round().clamp(0, 15)
        return (code * step + low).reshape(x.shape)
    k = rotated(s["k"])
    out = dict(q=rotated(s["q"]), k=held(k), v=held(s["v"].double() * live[..., None, None]))
    if s["summary"] is not None:
        box = s["summary"].double()
        for b in range(B):
            a, m = int(s["lens"][b]), int(s["after"][b])
            for p in range(a // page, -(-m // page)):
                rows = k[b, max(0, p * page - a):(p + 1) * page - a]
                rows = rows[:m - a - max(0, p * page - a)]
                lo, hi = rows.amin(0), rows.amax(0)
                i = int(s["pages"][b, p])
                if p * page < a:
                    lo, hi = torch.minimum(lo, box[i, :, 0]), torch.maximum(hi, box[i, :, 1])
                box[i, :, 0], box[i, :, 1] = lo, hi
        out["summary"] = box
    return out
