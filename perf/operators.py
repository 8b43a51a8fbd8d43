"""Operators of the receiver's recomputed layers and of its decoding, as measured.

Three operators stand around the attention-map path:

- ``rope``: the RMS norm of every query and key head and the rotary position
  embedding in one pass (what a sender or receiver layer does before its
  scores are formed);
- ``window``: attention over packed sequences with a sliding window and a few
  first tokens that stay visible, whole prompts, prefill chunks over a prefix,
  and single tokens over a cache (the receiver's first r layers, which it
  computes itself);
- ``prefix``: decoding attention of a batch whose requests share one long
  prefix and have a short cache each of their own.

``run`` computes them with elementary torch operations in fp32, or, where
``own`` is true, through the package's public entry points.  ``exact`` is the
definition in fp64.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # one decoded token of a 32-query-head, 8-KV-head receiver: pure latency
        dict(name="rope_token", op="rope", T=1, hq=32, hkv=8, d=128, rot=128, layout="half", norm=True,
             scaling="none", factor=1.0, orig=0, base=10000.0, start=4096, dtype="bf16"),
        # a decode step of 64 requests far into a stretched context, part of the head rotated
        dict(name="rope_batch", op="rope", T=64, hq=24, hkv=8, d=128, rot=64, layout="interleaved", norm=True,
             scaling="yarn", factor=8.0, orig=32768, base=1000000.0, start=250000, dtype="bf16"),
        # fp32 heads of 64, odd length, rotation only
        dict(name="rope_f32", op="rope", T=4099, hq=24, hkv=8, d=64, rot=64, layout="half", norm=False,
             scaling="linear", factor=4.0, orig=0, base=10000.0, start=0, dtype="f32"),
        # a long prompt of the 40-head sender
        dict(name="rope_prompt", op="rope", T=16384, hq=40, hkv=40, d=128, rot=128, layout="half", norm=True,
             scaling="none", factor=1.0, orig=0, base=1000000.0, start=0, dtype="bf16"),
        # eight packed prompts of uneven length, a window of 1024 and 4 sinks
        dict(name="window_packed", op="window", lens="1024,1,2311,640,77,1500,3001,1111", begin=0, hq=32, hkv=8,
             d=128, window=1024, sinks=4),
        # a whole prompt without a window: the receiver's recomputed layers
        dict(name="window_causal", op="window", lens="8192", begin=0, hq=32, hkv=8, d=128, window=0, sinks=0),
        # a long prompt with a wide window
        dict(name="window_long", op="window", lens="16384", begin=0, hq=24, hkv=8, d=128, window=4096, sinks=64),
        # a prefill chunk of 300 tokens over a cached prefix of 16000
        dict(name="window_chunk", op="window", lens="16300", begin=16000, hq=32, hkv=8, d=128, window=0, sinks=0),
        # a decode step of 32 requests, uneven caches, window and sinks
        dict(name="window_decode", op="decode", n=32, lq=1, cap=16384, prefix=0, hq=32, hkv=8, d=128,
             window=4096, sinks=4),
        # two requests over a short shared prompt: latency
        dict(name="prefix_small", op="decode", n=2, lq=1, cap=128, prefix=1000, hq=24, hkv=8, d=128, window=0,
             sinks=0),
        # a decode step of 64 requests over a 16k shared prompt
        dict(name="prefix_batch", op="decode", n=64, lq=1, cap=512, prefix=16384, hq=32, hkv=8, d=128, window=0,
             sinks=0),
        # 200 requests, two new tokens each, over a 32k shared prompt
        dict(name="prefix_large", op="decode", n=200, lq=2, cap=700, prefix=32767, hq=24, hkv=8, d=128, window=0,
             sinks=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "window", "window", "decode", "prefix"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 8])
    if op == "rope":
        return dict(op="rope", T=_log(rng, 1, 16384), hq=hq, hkv=hkv, d=d,
                    rot=rng.choice([d, d, d // 2, d // 4, 2 * rng.randint(3, d // 2)]),
                    layout=rng.choice(["half", "interleaved"]), norm=rng.random() < 0.7,
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]), factor=rng.choice([2.0, 4.0, 8.0]),
                    orig=rng.choice([4096, 32768]), base=rng.choice([10000.0, 1000000.0]),
                    start=_log(rng, 1, 1000000), dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "window":
        total = _log(rng, 16, 8192)
        n = rng.randint(1, min(9, total))
        cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        begin = 0
        if rng.random() < 0.3:  # one sequence, a chunk at its end
            lens = [total]
            begin = total - min(total, _log(rng, 1, 1024))
        return dict(op="window", lens=",".join(str(x) for x in lens), begin=begin, hq=hq, hkv=hkv, d=d,
                    window=rng.choice([0, _log(rng, 1, 8192), _log(rng, 1, 1024)]),
                    sinks=rng.choice([0, 1, 4, _log(rng, 1, 300)]))
    if op == "decode":
        return dict(op="decode", n=_log(rng, 1, 64), lq=rng.choice([1, 1, 2, 4]), cap=_log(rng, 1, 16384), prefix=0,
                    hq=hq, hkv=hkv, d=d, window=rng.choice([0, _log(rng, 1, 4096)]), sinks=rng.choice([0, 4, 64]))
    return dict(op="decode", n=_log(rng, 1, 200), lq=rng.choice([1, 1, 2, 3]), cap=_log(rng, 1, 700),
                prefix=_log(rng, 1, 32768), hq=hq, hkv=hkv, d=d, window=0, sinks=0)


# ------------------------------------------------------------------ inputs --
def _seqlens(case):
    return [int(x) for x in case["lens"].split(",")]


def _cache_lens(case, seed):
    """Cache lengths spread evenly over 1..cap, dealt to the requests by the seed."""
    n, cap = case["n"], case["cap"]
    lens = [1 + (cap - 1) * (2 * r + 1) // (2 * n) for r in range(n)]
    random.Random(seed).shuffle(lens)
    return lens


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]

    def rnd(*shape, dt=torch.bfloat16, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dt)

    s = dict(case=case)
    if case["op"] == "rope":
        T, dt = case["T"], _DT[case["dtype"]]
        # the queries and keys of a fused projection: rows of q, k and v heads
        qkv = rnd(T, (hq + 2 * hkv) * d, dt=dt)
        s["q"] = qkv[:, : hq * d].view(T, hq, d)
        s["k"] = qkv[:, hq * d : (hq + hkv) * d].view(T, hkv, d)
        s["pos"] = (torch.arange(T, device=dev) + case["start"] + seed % 7).to(torch.int32)
        s["wq"] = (1.0 + 0.1 * torch.randn(d, generator=g, device=dev)).to(dt) if case["norm"] else None
        s["wk"] = (1.0 + 0.1 * torch.randn(d, generator=g, device=dev)).to(dt) if case["norm"] else None
        s["freq"] = torch.tensor(_frequencies(case), dtype=torch.float64, device=dev)
        if own:
            from cross_model_attention_gb300 import mapflow
            s["plan"] = mapflow.RotaryPlan(case["rot"], base=case["base"], layout=case["layout"],
                                           scaling=case["scaling"], factor=case["factor"],
                                           original_length=case["orig"])
        return s
    if case["op"] == "window":
        lens = _seqlens(case)
        T = sum(lens)
        s["q"], s["k"], s["v"] = rnd(T, hq, d, std=1.5), rnd(T, hkv, d), rnd(T, hkv, d)
        s["seq"] = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens)).to(dev)
        s["at"] = torch.cat([torch.arange(x) for x in lens]).to(dev)
        s["o"] = torch.zeros_like(s["q"])
        if own:
            from cross_model_attention_gb300 import mapflow
            cu = [0]
            for x in lens:
                cu.append(cu[-1] + x)
            s["plan"] = mapflow.WindowAttention(cu, hq, hkv, d, window=case["window"] or None, sinks=case["sinks"],
                                                q_begin=[case["begin"]] if case["begin"] else None)
        return s
    n, lq, cap, P = case["n"], case["lq"], case["cap"], case["prefix"]
    s["q"] = rnd(n, lq, hq, d, std=1.5)
    s["k"], s["v"] = rnd(n, cap, hkv, d), rnd(n, cap, hkv, d)
    s["kp"] = rnd(P, hkv, d) if P else None
    s["vp"] = rnd(P, hkv, d) if P else None
    s["lens"] = torch.tensor(_cache_lens(case, seed), dtype=torch.int32, device=dev)
    s["o"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(n, lq, hq, dtype=torch.float32, device=dev)
    if own:
        from cross_model_attention_gb300 import mapflow
        s["plan"] = mapflow.CacheAttention(n, lq, cap, hq, hkv, d, window=case["window"] or None,
                                           sinks=case["sinks"], prefix_len=P)
    return s


# --------------------------------------------------------------------- run --
def run(s):
    case = s["case"]
    if case["op"] == "rope":
        if own:
            q, k = s["plan"].apply(s["q"], s["k"], s["pos"], q_weight=s["wq"], k_weight=s["wk"], eps=1e-6)
            return {"q": q, "k": k}
        return {"q": _rope(s["q"], s["wq"], s), "k": _rope(s["k"], s["wk"], s)}
    if case["op"] == "window":
        if own:
            s["plan"].attend(s["q"], s["k"], s["v"], o=s["o"])
            return s["o"][case["begin"]:]
        return _packed(s)
    if own:
        s["plan"].attend(s["q"], s["k"], s["v"], s["lens"], k_prefix=s["kp"], v_prefix=s["vp"], o=s["o"],
                         lse=s["lse"])
        return {"o": s["o"], "lse": s["lse"]}
    return _cached(s)


def _frequencies(case):
    """Radians per position of each rotated pair, stretched for long contexts."""
    rot, base, f = case["rot"], case["base"], case["factor"]
    if case["scaling"] == "ntk" and rot > 2:
        base = base * f ** (rot / (rot - 2.0))
    plain = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if case["scaling"] == "linear":
        return [x / f for x in plain]
    if case["scaling"] == "yarn":
        def dim_of(turns):
            return rot * math.log(case["orig"] / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
        low, high = max(math.floor(dim_of(32.0)), 0), min(math.ceil(dim_of(1.0)), rot - 1)
        out = []
        for i, x in enumerate(plain):
            r = min(1.0, max(0.0, (i - low) / max(high - low, 1e-3)))
            out.append(x / f * r + x * (1.0 - r))
        return out
    return plain


def _gain(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "yarn" else 1.0


def _rope(x, w, s):
    case, dt = s["case"], x.dtype
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    rot = case["rot"]
    turn = (s["pos"].double()[:, None] * s["freq"]).remainder(2.0 * math.pi)  # far positions: angles in 64 bits
    cos = (turn.cos() * _gain(case)).float()[:, None]
    sin = (turn.sin() * _gain(case)).float()[:, None]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if case["layout"] == "interleaved" else \
        (x[..., : rot // 2], x[..., rot // 2 : rot])
    y, z = a * cos - b * sin, b * cos + a * sin
    first = torch.stack([y, z], -1).flatten(-2) if case["layout"] == "interleaved" else torch.cat([y, z], -1)
    return torch.cat([first, x[..., rot:]], -1).to(dt)


def _weights(s, hidden):
    """Rows' maxima, exp(score - maximum) and their sums; a row that sees nothing has weights of zero."""
    s = s.masked_fill_(hidden, float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = m.masked_fill(m == float("-inf"), 0.0)
    p = s.sub_(m).exp_()
    return m, p, p.sum(-1, keepdim=True)


def _packed(s):
    case = s["case"]
    b, hq, hkv, d = case["begin"], case["hq"], case["hkv"], case["d"]
    q, k, v = s["q"][b:], s["k"], s["v"]
    n, G = q.shape[0], hq // hkv
    qf = q.float().view(n, hkv, G, d).permute(1, 2, 0, 3).reshape(hkv, G * n, d)
    sc = (qf @ k.float().permute(1, 2, 0)).view(hkv, G, n, -1).mul_(1.0 / math.sqrt(d))
    i, j = s["at"][b:, None], s["at"][None]
    seen = (s["seq"][b:, None] == s["seq"][None]) & (j <= i)
    if case["window"]:
        seen &= (i - j < case["window"]) | (j < case["sinks"])
    _, p, l = _weights(sc, ~seen)
    o = (p.view(hkv, G * n, -1) @ v.float().permute(1, 0, 2)).view(hkv, G, n, d) / l
    return o.permute(2, 0, 1, 3).reshape(n, hq, d).to(q.dtype)


def _cached(s):
    case, q = s["case"], s["q"]
    n, lq, cap, P = case["n"], case["lq"], case["cap"], case["prefix"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    G = hq // hkv
    qf = q.float().view(n, lq, hkv, G, d).permute(2, 0, 3, 1, 4) * (1.0 / math.sqrt(d))  # [hkv, n, G, lq, d]
    qf = qf.reshape(hkv, n, G * lq, d)
    sc = (qf @ s["k"].float().permute(2, 0, 3, 1)).reshape(hkv, n, G, lq, cap)
    j = torch.arange(cap, device=q.device)
    i = (s["lens"].long()[:, None] - lq + torch.arange(lq, device=q.device))[:, None, :, None]  # last row: the newest key
    seen = j <= i
    if case["window"]:
        seen = seen & ((i - j < case["window"]) | (j < case["sinks"]))
    sc = sc.masked_fill_(~seen, float("-inf"))
    if P:
        pre = (qf.reshape(hkv, n * G * lq, d) @ s["kp"].float().permute(1, 2, 0)).reshape(hkv, n, G, lq, P)
        sc = torch.cat([pre, sc], -1)
    m, p, l = _weights(sc, torch.zeros((), dtype=torch.bool, device=q.device))
    o = p[..., P:].reshape(hkv, n, G * lq, cap) @ s["v"].float().permute(2, 0, 1, 3)
    if P:
        o += (p[..., :P].reshape(hkv, n * G * lq, P) @ s["vp"].float().permute(1, 0, 2)).view(hkv, n, G * lq, d)
    o = o.reshape(hkv, n, G, lq, d) / l.clamp_min(1e-30)
    lse = (m + l.log()).squeeze(-1)
    return {"o": o.permute(1, 3, 0, 2, 4).reshape(n, lq, hq, d).to(q.dtype),
            "lse": lse.permute(1, 3, 0, 2).reshape(n, lq, hq)}


# -------------------------------------------------------------------- work --
def _seen(i, window, sinks):
    """Keys that the row at position i sees."""
    if not window or i < window:
        return i + 1
    return window + min(sinks, i - window + 1)


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "rope":
        e = 4 if case["dtype"] == "f32" else 2
        values = case["T"] * (hq + hkv) * d
        return {"bytes": 2 * e * values + 4 * case["T"], "flops": 8 * values}
    if case["op"] == "window":
        lens, b = _seqlens(case), case["begin"]
        pairs = sum(_seen(i, case["window"], case["sinks"]) for x in lens for i in range(b, x))
        rows = sum(lens) - b
        # keys that no row sees are not read: before the chunk's window
        keys = sum(lens)
        if b and case["window"]:
            first = max(0, b - case["window"] + 1)
            keys = keys - first + min(first, case["sinks"])
        return {"bytes": 2 * (2 * rows * hq * d + 2 * keys * hkv * d), "flops": 4 * d * hq * pairs}
    n, lq, P = case["n"], case["lq"], case["prefix"]
    lens = _cache_lens(case, 0)
    pairs = keys = 0
    for x in lens:
        if x:
            at = [i for i in range(x - lq, x) if i >= 0]
            pairs += sum(_seen(i, case["window"], case["sinks"]) for i in at)
            lo = max(0, at[0] - case["window"] + 1) if case["window"] else 0
            keys += x - lo + min(lo, case["sinks"])
    pairs += n * lq * P
    return {"bytes": 2 * (2 * n * lq * hq * d + 2 * (keys + P) * hkv * d) + 4 * n * lq * hq + 4 * n,
            "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------- exact --
def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "rope":
        th = s["pos"].to(f64)[:, None] * s["freq"][None]
        half, rot = case["rot"] // 2, case["rot"]
        if case["layout"] == "interleaved":
            ia, ib = torch.arange(0, rot, 2), torch.arange(1, rot, 2)
        else:
            ia, ib = torch.arange(half), torch.arange(half, rot)
        out = {}
        for name, w in (("q", s["wq"]), ("k", s["wk"])):
            x = s[name].to(f64)
            if w is not None:
                x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.to(f64)
            z = torch.complex(x[..., ia], x[..., ib]) * torch.polar(torch.full_like(th, _gain(case)), th)[:, None]
            y = x.clone()
            y[..., ia], y[..., ib] = z.real, z.imag
            out[name] = y
        return out
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    G = hq // hkv
    if case["op"] == "window":
        b, lens = case["begin"], _seqlens(case)
        if 4.0 * d * hq * sum((x - b) * x for x in lens) > 8e12:
            return None
        o = torch.zeros(sum(lens) - b, hq, d, dtype=f64, device=s["q"].device)
        t0 = 0
        for x in lens:
            for h in range(hq):
                for r0 in range(b, x, 4096):
                    r1 = min(x, r0 + 4096)
                    k = s["k"][t0:t0 + x, h // G].to(f64)
                    v = s["v"][t0:t0 + x, h // G].to(f64)
                    sc = s["q"][t0 + r0:t0 + r1, h].to(f64) @ k.T / math.sqrt(d)
                    i = torch.arange(r0, r1, device=sc.device)[:, None]
                    j = torch.arange(x, device=sc.device)[None]
                    hide = j > i
                    if case["window"]:
                        hide = hide | ((j <= i - case["window"]) & (j >= case["sinks"]))
                    o[t0 + r0 - b:t0 + r1 - b, h] = torch.softmax(sc.masked_fill(hide, -math.inf), -1) @ v
            t0 += x
        return o
    n, lq, P = case["n"], case["lq"], case["prefix"]
    if 4.0 * d * hq * n * lq * (P + case["cap"]) > 2e12:
        return None
    o = torch.zeros(n, lq, hq, d, dtype=f64, device=s["q"].device)
    lse = torch.full((n, lq, hq), -math.inf, dtype=f64, device=s["q"].device)
    kp = s["kp"].to(f64) if P else None
    vp = s["vp"].to(f64) if P else None
    for r, x in enumerate(_cache_lens(case, seed)):
        k, v = s["k"][r, :x].to(f64), s["v"][r, :x].to(f64)
        if P:
            k, v = torch.cat([kp, k]), torch.cat([vp, v])
        for t in range(lq):
            at = x - lq + t
            j = torch.arange(-P, x, device=k.device)
            keep = (j < 0) | (j <= at)  # the whole prefix, then the cache up to the row
            if case["window"]:
                keep &= (j > at - case["window"]) | (j < case["sinks"])
            kk, vv = k[keep], v[keep]
            if kk.shape[0] == 0:
                continue
            sc = torch.einsum("hgd,jhd->hgj", s["q"][r, t].to(f64).view(hkv, G, d), kk) / math.sqrt(d)
            lse[r, t] = torch.logsumexp(sc, -1).reshape(hq)
            o[r, t] = torch.einsum("hgj,jhd->hgd", torch.softmax(sc, -1), vv).reshape(hq, d)
    return {"o": o, "lse": lse}
