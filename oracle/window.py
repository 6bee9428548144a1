"""Windowed attention with sinks in 64 bits, its gradients by the formulas, and how far
kernels of given roundings may be from them (test infrastructure)."""
import math

import torch


def visible(Sq, Sk, window, sinks, device="cpu"):
    p = torch.arange(Sq, device=device)[:, None] + Sk - Sq
    j = torch.arange(Sk, device=device)[None]
    return (j <= p) & ((j > p - window) | (j < sinks))


def heads(x, Hq):
    """[B, S, H, D] -> [B, Hq, S, D] in 64 bits, kv heads repeated."""
    return x.double().permute(0, 2, 1, 3).repeat_interleave(Hq // x.shape[2], 1)


def forward(q, k, v, window, sinks, scale=None, unit=2.0 ** -8):
    """out [B, Sq, Hq, D], lse [B, Hq, Sq] and bounds of what a kernel may be off that rounds
    weights and outputs by `unit` of themselves (half a step) and sums in fp32."""
    Hq, D = q.shape[2], q.shape[3]
    scale = scale or 1 / math.sqrt(D)
    Q, K, V = heads(q, Hq), heads(k, Hq), heads(v, Hq)
    see = visible(q.shape[1], k.shape[1], window, sinks, q.device)
    s = (Q @ K.transpose(-1, -2) * scale).masked_fill(~see, -math.inf)
    lse = s.logsumexp(-1)
    p = torch.exp(s - lse[..., None])
    out = p @ V
    # a score is a sum of D products in fp32, and its exponential good to 2^-21: a relative
    # error of each weight, and of their sum
    ds = score_error(Q, K, scale, see)
    rel = unit + 2 * ds + 2.0 ** -20
    e_out = rel * (p @ V.abs()) + unit * out.abs()
    e_lse = ds.squeeze(-1) + 2.0 ** -21 + 2.0 ** -23 * lse.abs()
    rows = lambda x: x.permute(0, 2, 1, 3)  # noqa: E731
    return rows(out), lse, rows(e_out), e_lse


def score_error(Q, K, scale, see):
    """Largest error of a row's visible scores: (D + 4) half steps of fp32 on sum |q k|, [B, H, Sq, 1]."""
    mag = (Q.abs() @ K.abs().transpose(-1, -2) * scale).masked_fill(~see, 0).amax(-1, keepdim=True)
    return (Q.shape[-1] + 4) * 2.0 ** -24 * mag


def backward(q, k, v, dout, window, sinks, scale=None, unit=2.0 ** -8):
    """(dq, dk, dv) and their bounds, for a kernel that also rounds dS by `unit` of itself and
    takes Delta from the rounded out."""
    Hq, Hkv, D = q.shape[2], k.shape[2], q.shape[3]
    scale = scale or 1 / math.sqrt(D)
    Q, K, V, G = heads(q, Hq), heads(k, Hq), heads(v, Hq), heads(dout, Hq)
    see = visible(q.shape[1], k.shape[1], window, sinks, q.device)
    s = (Q @ K.transpose(-1, -2) * scale).masked_fill(~see, -math.inf)
    p = torch.softmax(s, -1)
    out = p @ V
    dp = G @ V.transpose(-1, -2)
    delta = (G * out).sum(-1, keepdim=True)
    ds = p * (dp - delta)
    grads = [ds @ K * scale, ds.transpose(-1, -2) @ Q * scale, p.transpose(-1, -2) @ G]
    es = 2 * score_error(Q, K, scale, see) + 2.0 ** -19
    e_out = (unit + es) * (p @ V.abs()) + unit * out.abs()
    fp = (D + 4) * 2.0 ** -24
    e_delta = (G.abs() * (e_out + fp * out.abs())).sum(-1, keepdim=True)
    e_ds = (unit + es) * ds.abs() + p * (e_delta + fp * (G.abs() @ V.abs().transpose(-1, -2)))
    e_p = (unit + es) * p
    n = 2.0 ** -24 * 2 * q.shape[1]                  # the sums over rows and keys, in fp32
    errs = [scale * ((e_ds + n * ds.abs()) @ K.abs()), scale * ((e_ds + n * ds.abs()).transpose(-1, -2) @ Q.abs()),
            (e_p + n * p).transpose(-1, -2) @ G.abs()]

    def rows(x, h):
        x = x.unflatten(1, (h, -1)).sum(2)
        return x.permute(0, 2, 1, 3)
    grads = [rows(g, h) for g, h in zip(grads, (Hq, Hkv, Hkv))]
    errs = [rows(e, h) + unit * g.abs() for e, h, g in zip(errs, (Hq, Hkv, Hkv), grads)]
    return grads, errs


def within(got, ref, err, what):
    got = got.double()
    assert torch.isfinite(got).all(), what
    over = (got - ref).abs() - err
    worst = int(over.argmax())
    assert over.max() <= 0, (what, "off by", float((got - ref).abs().flatten()[worst]), "may be",
                             float(err.flatten()[worst]), "at", worst, "value", float(ref.flatten()[worst]))
