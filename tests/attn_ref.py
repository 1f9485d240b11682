"""Softmax attention in 64 bits, and how far a result may be off.

A result may be off by what its kernel's roundings can add up to, taken from the values themselves in 64 bits:
  u    half a step of the tensors' type (bf16 2^-8, fp32 2^-24), for each rounding to it: the probabilities and ds before
       their second product (bf16 only), and the stored result;
  w    2^-24 of fp32 arithmetic: a sum of n products is off by at most (n + 2) w of the sum of their magnitudes;
  e    the relative error of a probability: its score's error (the sum over d, the scale, the subtraction, each relative to
       the magnitudes) and exp2's own 2 ulp, doubled for the normaliser.
"""
import math

import torch

DEVICE = "cpu"
W = 2.0 ** -24


def half_step(T):
    return torch.finfo(T).eps / 2


def attend(q, k, v, scale, first=0, causal=True, do=None, T=torch.bfloat16):
    """q [n, H, d] (token `first` on) over k [L, G, d] and v [L, G, dv]; every result as (value, how far off it may be):
    o [n, H, dv], lse [H, n] and with do dq, dk, dv."""
    q, k, v = (t.to(DEVICE).double() for t in (q, k, v))
    do = do.to(DEVICE).double() if do is not None else None
    n, H, d = q.shape
    L, G, width = v.shape
    r, u = H // G, half_step(T)
    inner = u if T != torch.float32 else 0.0        # rounding of p and ds before the second product
    o, to = (torch.zeros(n, H, width, dtype=torch.float64, device=DEVICE) for _ in range(2))
    lse, tl = (torch.zeros(H, n, dtype=torch.float64, device=DEVICE) for _ in range(2))
    dq, tq = torch.zeros_like(q), torch.zeros_like(q)
    dk, tk = torch.zeros_like(k), torch.zeros_like(k)
    dv, tv = torch.zeros_like(v), torch.zeros_like(v)
    hidden = torch.zeros(n, L, dtype=torch.bool, device=DEVICE)
    if causal:
        hidden = torch.arange(L, device=DEVICE) > first + torch.arange(n, device=DEVICE)[:, None]
    for h in range(H):
        g = h // r
        Q, K, V = q[:, h], k[:, g], v[:, g]
        s = (Q @ K.T * scale).masked_fill(hidden, -math.inf)
        size = (Q.abs() @ K.abs().T * abs(scale)).masked_fill(hidden, 0)     # magnitudes in a score
        if L == 0:
            lse[h] = -math.inf
            continue
        top = s.amax(-1, keepdim=True)
        base = torch.where(top == -math.inf, torch.zeros_like(top), top)
        p = torch.exp(s - base)
        total = p.sum(-1, keepdim=True)
        p = p / torch.where(total == 0, torch.ones_like(total), total)
        lse[h] = (base + torch.log(total)).squeeze(-1)
        o[:, h] = p @ V
        # a score's error: d products, two scalings, the subtraction of the maximum; exp2 2 ulp
        es = (d + 6) * W * size.amax(-1, keepdim=True) + 4 * W * base.abs()
        e = 2 * es + (L + 8) * W
        tl[h] = (es.squeeze(-1) + (L + 8) * W + 4 * W * torch.where(lse[h].isfinite(), lse[h].abs(), torch.zeros_like(lse[h])))
        to[:, h] = (inner * (1 + u) + e + (L + 2) * W) * (p @ V.abs()) + u * o[:, h].abs() * (1 + u)
        if do is None:
            continue
        D = do[:, h]
        dp = D @ V.T
        delta = (D * o[:, h]).sum(-1, keepdim=True)
        ds = p * (dp - delta)
        # o is read as stored, with its own error
        tdelta = (D.abs() * to[:, h]).sum(-1, keepdim=True) + (width + 2) * W * (D.abs() * o[:, h].abs()).sum(-1, keepdim=True)
        tdp = (width + 2) * W * (D.abs() @ V.abs().T)
        tds = p * (tdelta + tdp) * (1 + inner + e) + (inner * (1 + u) + e + 4 * W) * ds.abs()
        grow = 1 + (L + n + 4) * W
        dq[:, h] = ds @ K * scale
        tq[:, h] = abs(scale) * grow * (tds @ K.abs()) + (L + 4) * W * abs(scale) * (ds.abs() @ K.abs())
        dk[:, g] += ds.T @ Q * scale
        tk[:, g] += abs(scale) * grow * (tds.T @ Q.abs()) + (r * n + 4) * W * abs(scale) * (ds.abs().T @ Q.abs())
        dv[:, g] += p.T @ D
        tv[:, g] += ((inner * (1 + u) + e) * p).T @ D.abs() + (r * n + 4) * W * (p.T @ D.abs())
    if do is None:
        return (o, to), (lse, tl)
    done = [(x, t * (1 + u) + u * x.abs()) for x, t in ((dq, tq), (dk, tk), (dv, tv))]
    return (o, to), (lse, tl), *done


def check(got, want, name):
    value, bound = want
    got = got.detach().to(value.device).double()
    assert got.shape == value.shape, (name, got.shape, value.shape)
    if not value.numel():
        return
    same = got == value                                   # infinities
    off = torch.where(same, torch.zeros_like(value), (got - value).abs())
    bad = ~(off <= bound + 1e-30)
    if bad.any():
        at = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{name}{list(at)}: {got[at].item()} for {value[at].item()}, off by {off[at].item():.3g}, "
                             f"allowed {bound[at].item():.3g}; {int(bad.sum())} of {bad.numel()}")
