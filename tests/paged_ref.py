"""fp64 definitions (torch, CPU or GPU tensors) of a cache held in 4 bits and of
decoding attention over it, and the error bounds the kernels are held to.
Shares no code with the CUDA path."""
import math

import torch

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
E4M3 = [m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:-1]


def nearest(grid, x):
    """Place in `grid` of the number nearest to each x >= 0; of two as near the even place."""
    grid = torch.tensor(grid, dtype=torch.float64, device=x.device)
    far = (x[..., None] - grid).abs()
    best = far.amin(-1, keepdim=True)
    place = torch.arange(len(grid), device=x.device)
    tie = torch.where(far == best, place % 2, 2)  # the even one of the nearest
    return tie.argmin(-1)


def hold(x, g):
    """Codes [..., d] (0..15) and scale bytes [..., d/16] of x [..., H, d] fp64 under head scales g [H]."""
    b = x.unflatten(-1, (-1, 16))
    g = g.double()[:, None]
    top = b.abs().amax(-1)
    bad = ~torch.isfinite(b).all(-1)
    s = nearest(E4M3, torch.where(bad, torch.zeros_like(top), top / (6 * g)).clamp_max(448.0))
    sg = torch.tensor(E4M3, dtype=torch.float64, device=x.device)[s] * g
    t = torch.where(sg[..., None] > 0, b.abs() / sg[..., None].clamp_min(1e-300), torch.zeros_like(b)).nan_to_num(0.0)
    code = nearest(E2M1, t.clamp_max(6.0)) + torch.where(b < 0, 8, 0)
    return code.flatten(-2), torch.where(bad, 0x7f, s)


def stands_for(code, scale, g):
    """fp64 values of codes [..., H, d] with scale bytes [..., H, d/16] under g [H]."""
    e2 = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=code.device)
    e4 = torch.tensor(E4M3 + [math.nan], dtype=torch.float64, device=code.device)
    e4 = torch.cat([e4, -e4])
    x = e2[code.long()].unflatten(-1, (-1, 16)) * e4[scale.long()][..., None]
    return x.flatten(-2) * g.double()[:, None]


def unpack(pages, page_size, d):
    """(key codes, key scales, value codes, value scales) [n_pages, page_size, H, ...] of pages uint8 [n_pages, H, ...]."""
    n, H = pages.shape[:2]
    p = pages.view(n, H, page_size // 16, 18 * d)
    kc = p[..., : 8 * d].reshape(n, H, -1, d // 2)
    vc = p[..., 8 * d: 16 * d].reshape(n, H, -1, 2, d // 16, 8, 8).permute(0, 1, 2, 3, 5, 4, 6).reshape(n, H, -1, d // 2)
    ks = p[..., 16 * d: 17 * d].reshape(n, H, -1, d // 16)
    vs = p[..., 17 * d:].reshape(n, H, -1, d // 16, 16).transpose(-1, -2).reshape(n, H, -1, d // 16)
    out = []
    for c, s in ((kc, ks), (vc, vs)):
        c = torch.stack([c & 15, c >> 4], -1).flatten(-2)
        out += [c.transpose(1, 2), s.transpose(1, 2)]
    return out


def pack(kc, ks, vc, vs):
    """Pages uint8 [n_pages, H, ...] of codes [n_pages, page_size, H, d] and scales [..., d/16]."""
    n, ps, H, d = kc.shape
    flat = []
    for c in (kc, vc):
        c = c.transpose(1, 2).to(torch.uint8)
        flat.append((c[..., 0::2] | (c[..., 1::2] << 4)).view(n, H, ps // 16, 16, d // 2))
    flat[1] = flat[1].view(n, H, ps // 16, 2, 8, d // 16, 8).transpose(-3, -2)
    ks, vs = (s.transpose(1, 2).to(torch.uint8).reshape(n, H, ps // 16, 16, d // 16) for s in (ks, vs))
    flat += [ks, vs.transpose(-1, -2)]
    return torch.cat([x.reshape(n, H, ps // 16, -1) for x in flat], -1).view(n, H, -1).contiguous()


def attend(q, k, v, length, window, sinks, scale, softcap=None, slopes=None, hidden=None):
    """(o, lse, o_bound, lse_bound) of the new tokens q [Lq, H_q, d] of a request over its keys
    and values [length, H, d] fp64; hidden [length]: keys on no page.

    Bounds: q and k meet exactly (8 and 6 bits) and are summed in fp32 by the
    tensor cores, counted with d 2^-23 of sum|q k|; the factor of a score has
    three roundings, tanh, the bias and its sum a few more, the exponent's
    difference and exp2 2^-22 each: 2^-20 (2 |s| + |bias| + 1) together.  A weight
    is rounded to 11 bits (2^-11 of it), or by 2^-32 of the reference's weight,
    which a key of the row has; the output to bf16 (2^-8); sums of m terms in fp32
    by 2^-24 m in the worst case, counted with m <= 2^10 (lanes sum parts)."""
    Lq, H_q, d = q.shape
    H = k.shape[1]
    G = H_q // H
    i = length - Lq + torch.arange(Lq, device=q.device)[:, None]
    j = torch.arange(length, device=q.device)[None]
    seen = j <= i
    if window:
        seen = seen & ((i - j < window) | (j < sinks))
    if hidden is not None:
        seen = seen & ~hidden[None]
    o = torch.zeros(Lq, H_q, d, dtype=torch.float64, device=q.device)
    lse = torch.full((Lq, H_q), -math.inf, dtype=torch.float64, device=q.device)
    if length == 0:
        return o, lse, o.clone(), torch.zeros_like(lse)
    used = seen.any(0)[:, None, None]
    k, v = torch.where(used, k, torch.zeros_like(k)), torch.where(used, v, torch.zeros_like(v))
    q = q.double()
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    s = torch.einsum("nhd,mhd->hnm", q, kk) * scale
    mag = torch.einsum("nhd,mhd->hnm", q.abs(), kk.abs()) * scale
    if softcap:
        s = softcap * torch.tanh(s / softcap)
    bias = torch.zeros_like(s)
    if slopes is not None:
        bias = slopes.double()[:, None, None] * (i - j)[None]
        s = s - bias
    s = s.masked_fill(~seen, -math.inf)
    empty = ~seen.any(1)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(empty, torch.zeros_like(lse), lse)[..., None])
    size = torch.where(seen, s.abs() + bias.abs(), torch.zeros_like(s))
    ds = torch.where(seen, mag * d * 2.0 ** -23, torch.zeros_like(s)) + 2.0 ** -20 * (2 * size.amax(-1, keepdim=True) + 1) + 2.0 ** -14
    o = torch.einsum("hnm,mhd->nhd", p, vv)
    w = torch.einsum("hnm,mhd->nhd", p * (2.0 ** -11 + 2 * ds), vv.abs())
    w = w + torch.einsum("hnm,hnm->hn", p, ds).T[..., None] * o.abs()
    w = w + 2.0 ** -32 * vv.abs().sum(0)
    o_bound = w * 1.01 + o.abs() * 2.0 ** -8
    lse_bound = torch.where(empty, torch.zeros_like(lse), (p * ds).sum(-1)) + 2.0 ** -21 * lse.abs().nan_to_num(posinf=0.0)
    return o, lse.T, o_bound, lse_bound.T
