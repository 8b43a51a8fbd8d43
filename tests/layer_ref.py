"""fp64 definitions (torch, CPU or GPU tensors) of the rotary embedding with
head norms and of attention with windows, sinks and shared prefixes, and the
error bounds the kernels are held to.  Shares no code with the CUDA path."""
import math

import torch


def rope_frequencies(rot, base=10000.0, scaling="none", factor=1.0, original_length=0, beta_fast=32.0, beta_slow=1.0):
    """(radians per position [rot/2] fp64, gain)."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = torch.exp(-2.0 * i / rot * math.log(base))
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        dims = [rot * math.log(original_length / (b * 2 * math.pi)) / (2 * math.log(base)) for b in (beta_fast, beta_slow)]
        low, high = max(math.floor(dims[0]), 0), min(math.ceil(dims[1]), rot - 1)
        ramp = ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def rope(x, weight, norm, eps, positions, freq, gain, rot, layout):
    """(y, bound) of [T, H, d]: bound = absolute error of an fp32 evaluation,
    before the output's rounding.  The norm's mean of d squares and its root
    are off by at most (d + 4) 2^-24, in practice far less; the angle by
    pi 2^-24 (a 32-bit fraction of a turn rounded to fp32), sine and cosine by
    2^-22; two products and a sum by 3 * 2^-24: together below 2^-17 of
    (|a| + |b|) for d <= 128."""
    x = x.double()
    if norm:
        x = x * (x.square().mean(-1, keepdim=True) + eps).rsqrt()
        if weight is not None:
            x = x * weight.double()
    t = positions.double()[:, None] * freq.to(x.device)
    c, s = (t.cos() * gain)[:, None], (t.sin() * gain)[:, None]
    y, b = x.clone(), x.abs().clone()
    if layout == "half":
        ia, ib = torch.arange(rot // 2), torch.arange(rot // 2, rot)
    else:
        ia, ib = torch.arange(0, rot, 2), torch.arange(1, rot, 2)
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    b[..., ia] = b[..., ib] = (x[..., ia].abs() + x[..., ib].abs()) * max(1.0, gain)
    return y, b * 2.0 ** -17


def attend(q, k, v, seen, scale):
    """(o, lse, o_bound, lse_bound) of rows q [n, H_q, d] over keys k, v
    [m, H_kv, d] with seen [n, m]: fp64 softmax; rows that see nothing get 0
    and -inf.

    Bounds: a score's d products are exact in fp32 and summed in fp32, off by
    at most d 2^-24 scale sum|q k|; the exponent's product and difference and
    the exp2 by 2^-22 (|s| + |m| + 1); a weight is rounded to bf16 (2^-8 of
    it) before it meets its value, the output once more (2^-8); sums of m
    terms in fp32 by 2^-24 m in the worst case, counted with m <= 2^11
    (pairwise and blocked sums stay far below)."""
    n, H_q, d = q.shape
    G = H_q // k.shape[1]
    if k.shape[0] == 0:  # no key at all: one that nobody sees
        k, v, seen = k.new_zeros(1, *k.shape[1:]), v.new_zeros(1, *v.shape[1:]), seen.new_zeros(n, 1)
    q, k, v = q.double(), k.double(), v.double()
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    # masked rows may hold anything: they take no part
    used = seen.any(0)
    kk = torch.where(used[:, None, None], kk, torch.zeros_like(kk))
    vv = torch.where(used[:, None, None], vv, torch.zeros_like(vv))
    s = torch.einsum("nhd,mhd->hnm", q, kk) * scale
    mag = torch.einsum("nhd,mhd->hnm", q.abs(), kk.abs()) * scale
    s = s.masked_fill(~seen, -math.inf)
    empty = ~seen.any(1)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(empty, torch.zeros_like(lse), lse)[..., None])
    top = torch.where(seen, s.abs(), torch.zeros_like(s)).amax(-1, keepdim=True)
    ds = torch.where(seen, mag * d * 2.0 ** -24, torch.zeros_like(s)) + 2.0 ** -22 * (2 * top + 1) + 2.0 ** -13
    o = torch.einsum("hnm,mhd->nhd", p, vv)
    # each weight is off by 2^-8 and its exponent's error, the sum it is
    # divided by by the exponents' errors
    w = torch.einsum("hnm,mhd->nhd", p * (2.0 ** -8 + 2 * ds), vv.abs())
    w = w + torch.einsum("hnm,hnm->hn", p, ds).T[..., None] * o.abs()
    bound = w * 1.01 + o.abs() * 2.0 ** -8
    lse_bound = torch.where(empty, torch.zeros_like(lse), (p * ds).sum(-1)) + 2.0 ** -21 * lse.abs().nan_to_num(posinf=0.0) + 2.0 ** -20
    return o, lse.T, bound, lse_bound.T


def seen_packed(pos_q, pos_k, window, sinks):
    i, j = pos_q[:, None], pos_k[None]
    ok = j <= i
    if window:
        ok = ok & ((i - j < window) | (j < sinks))
    return ok
