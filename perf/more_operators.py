"""Operators of a paged cache of keys and values, as measured.

- ``append``: a step's keys (their head norm and rotary embedding applied on the
  way) and values into the pages of their sequences, in bf16 or in 4 bits;
- ``read``: tokens of a paged cache back as bf16 rows, which attention over a
  chunk and its cached prefix takes.  An ``append`` case reads its tokens back,
  as a prefill chunk does, so that what the cache holds comes out as values;
- ``attend``: decoding attention over a cache held in 4 bits, with windows, first
  tokens that stay visible, scores capped by a tanh and a bias by distance.

4 bits: 16 neighbouring dimensions of a token's head share a scale s in e4m3,
s = max |x| / (6 g) rounded to nearest even, at most 448, and a value is held as
the e2m1 number (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) nearest to
x / (s g), ties to even, at most 6; it stands for that number times s g, where g
is a scale per head.  In memory: 16 tokens of a head are 18 d bytes, the keys'
codes [16][d/2] (even dimensions in the low bits), the values' [2][d/16][8][8],
the keys' scales [16][d/16], the values' [d/16][16].

``run`` computes them with elementary torch operations, or, where ``own`` is
true, through the package's public entry points.  ``exact`` is the definition in
fp64.
"""
import math
import random

import torch

own = False

_EPS = 1e-6


# ------------------------------------------------------------------- cases --
def listed():
    rope = dict(rot=128, layout="half", scaling="none", factor=1.0, orig=0, base=1000000.0)
    return [
        # one decoded token of an 8-KV-head receiver: pure latency
        dict(name="append_token", op="append", n=1, T=1, start=777, shift=0, pad=0, ps=64, hkv=8, d=128, fmt="fp4",
             norm=True, scales=False, **rope),
        # a decode step of 64 requests far into a stretched context, of a batch with 6 unused places
        dict(name="append_batch", op="append", n=64, T=64, start=500, shift=250000, pad=6, ps=16, hkv=8, d=128,
             fmt="fp4", norm=True, scales=True, rot=64, layout="interleaved", scaling="yarn", factor=8.0, orig=32768,
             base=1000000.0),
        # five uneven prompts of an 8-KV-head receiver, with head norms
        dict(name="append_prompt", op="append", n=5, T=16384, start=0, shift=0, pad=0, ps=64, hkv=8, d=128, fmt="fp4",
             norm=True, scales=True, **rope),
        # a prefill chunk into a bf16 cache of the 40-head sender, rotation only
        dict(name="append_bf16", op="append", n=2, T=4099, start=300, shift=0, pad=0, ps=128, hkv=40, d=128,
             fmt="bf16", norm=False, scales=False, **rope),
        # a short cached prompt of heads of 64
        dict(name="read_short", op="read", n=1, T=333, ps=16, hkv=8, d=64, scales=True),
        # the cached prefixes of three chunks, uneven
        dict(name="read_prefix", op="read", n=3, T=32000, ps=64, hkv=8, d=128, scales=True),
        # one request with a short context: latency
        dict(name="attend_one", op="attend", n=1, lq=1, cap=1000, ps=64, hq=32, hkv=8, d=128, window=0, sinks=0,
             softcap=0.0, slopes=False, scales=False, empty=False),
        # a decode step of 32 requests with a window and 4 sinks
        dict(name="attend_window", op="attend", n=32, lq=1, cap=16384, ps=64, hq=32, hkv=8, d=128, window=4096,
             sinks=4, softcap=0.0, slopes=False, scales=True, empty=False),
        # four very long contexts of a 24-query-head receiver
        dict(name="attend_long", op="attend", n=4, lq=1, cap=131072, ps=128, hq=24, hkv=8, d=128, window=0, sinks=0,
             softcap=0.0, slopes=False, scales=True, empty=False),
        # many short requests of 40 heads of 64 without groups, small pages, unused places in the batch
        dict(name="attend_many", op="attend", n=256, lq=1, cap=1024, ps=16, hq=40, hkv=40, d=64, window=0, sinks=0,
             softcap=0.0, slopes=False, scales=True, empty=True),
        # three drafted tokens each, capped scores and a bias by distance
        dict(name="attend_capped", op="attend", n=24, lq=3, cap=6000, ps=32, hq=32, hkv=8, d=128, window=0, sinks=0,
             softcap=50.0, slopes=True, scales=True, empty=False),
        # eight drafted tokens of eight heads a group: many rows over each key
        dict(name="attend_drafts", op="attend", n=8, lq=8, cap=8000, ps=64, hq=64, hkv=8, d=128, window=0, sinks=0,
             softcap=0.0, slopes=False, scales=True, empty=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "read", "attend", "attend", "attend"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8, 8])
    ps = rng.choice([16, 32, 64, 128, 48])
    if op == "append":
        T = _log(rng, 1, 16384)
        return dict(op="append", n=min(T, _log(rng, 1, 64)), T=T, start=rng.choice([0, rng.randint(0, 700)]),
                    shift=rng.choice([0, _log(rng, 1, 1000000)]), pad=rng.choice([0, 0, min(T - 1, rng.randint(0, 9))]),
                    ps=ps, hkv=hkv, d=d, fmt=rng.choice(["fp4", "fp4", "bf16"]), norm=rng.random() < 0.6,
                    scales=rng.random() < 0.6, rot=rng.choice([d, d, d // 2, d // 4, 2 * rng.randint(3, d // 2)]),
                    layout=rng.choice(["half", "half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]), factor=rng.choice([2.0, 4.0, 8.0]),
                    orig=rng.choice([4096, 32768]), base=rng.choice([10000.0, 1000000.0]))
    if op == "read":
        T = _log(rng, 1, 32000)
        return dict(op="read", n=min(T, _log(rng, 1, 32)), T=T, ps=ps, hkv=hkv, d=d, scales=rng.random() < 0.6)
    G = rng.choice([1, 2, 3, 4, 5, 8])
    n = _log(rng, 1, 256)
    cap = min(_log(rng, 1, 65536), (1 << 27) // (n * hkv * d))
    return dict(op="attend", n=n, lq=rng.choice([1, 1, 1, 2, 4, 8]), cap=max(1, cap), ps=ps, hq=hkv * G, hkv=hkv, d=d,
                window=rng.choice([0, 0, _log(rng, 1, 4096)]), sinks=rng.choice([0, 4, 70]),
                softcap=rng.choice([0.0, 0.0, 30.0, 50.0]), slopes=rng.random() < 0.3, scales=rng.random() < 0.6,
                empty=rng.random() < 0.3)


# ------------------------------------------------------------------ inputs --
def _split(case):
    """New or cached tokens of each sequence: uneven, every one at least 1."""
    n, T = case["n"], case["T"] - case.get("pad", 0)
    n = min(n, T)
    cuts = [0] + sorted(random.Random(n * 7919 + T).sample(range(1, T), n - 1)) + [T]
    return [b - a for a, b in zip(cuts, cuts[1:])]


def _cache_lens(case, seed):
    """Cache lengths spread evenly over 1..cap, dealt to the requests by the seed; some requests unused."""
    n, cap = case["n"], case["cap"]
    lens = [1 + (cap - 1) * (2 * r + 1) // (2 * n) for r in range(n)]
    random.Random(seed).shuffle(lens)
    return [0 if case["empty"] and r % 7 == 3 else x for r, x in enumerate(lens)]


def _pages(mp, n, ps, hkv, d, g, dev):
    """(table [n][mp] of pages in no order, pages that it takes and a few more)."""
    count = n * mp + 3
    table = torch.randperm(count, generator=g, device=dev)[: n * mp].to(torch.int32).view(n, mp)
    return table, count


def _head_scales(case, g, dev):
    if not case["scales"]:
        return None, None
    h = case["hkv"]
    return tuple(torch.exp(0.7 * torch.randn(h, generator=g, device=dev)) for _ in range(2))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    ps, hkv, d = case["ps"], case["hkv"], case["d"]

    def rnd(*shape, dt=torch.bfloat16, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dt)

    s = dict(case=case)
    s["k_scale"], s["v_scale"] = _head_scales(case, g, dev)
    if case["op"] == "attend":
        n, lq, hq = case["n"], case["lq"], case["hq"]
        mp = -(-case["cap"] // ps)
        s["table"], count = _pages(mp, n, ps, hkv, d, g, dev)
        s["pages"] = _filled(count, s, rnd)
        s["lens"] = torch.tensor(_cache_lens(case, seed), dtype=torch.int32, device=dev)
        s["q"] = rnd(n, lq, hq, d, std=1.5)
        s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, hq + 1, device=dev) / hq) if case["slopes"] else None
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(n, lq, hq, dtype=torch.float32, device=dev)
    else:
        lens = _split(case)
        start = case.get("start", 0)
        mp = -(-(start + max(lens)) // ps)
        s["table"], count = _pages(mp, len(lens), ps, hkv, d, g, dev)
        T, pad = case["T"], case.get("pad", 0)
        # which sequence a token belongs to (-1: none) and its place there
        seq = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens))
        at = torch.cat([torch.arange(x) for x in lens]) + start
        s["seq"] = torch.cat([seq, torch.full((pad,), -1)]).to(torch.int32).to(dev)
        s["at"] = torch.cat([at, torch.zeros(pad, dtype=torch.int64)]).to(torch.int32).to(dev)
        s["ko"] = torch.zeros(T, hkv, d, dtype=torch.bfloat16, device=dev)
        s["vo"] = torch.zeros(T, hkv, d, dtype=torch.bfloat16, device=dev)
        if case["op"] == "read":
            s["pages"] = _filled(count, s, rnd)
        else:
            # the keys and values of a fused projection
            kv = rnd(T, 2 * hkv * d)
            s["k"] = kv[:, : hkv * d].view(T, hkv, d)
            s["v"] = kv[:, hkv * d :].view(T, hkv, d)
            s["w"] = (1.0 + 0.1 * torch.randn(d, generator=g, device=dev)).to(torch.bfloat16) if case["norm"] else None
            s["pos"] = s["at"] + case["shift"]
            s["freq"] = torch.tensor(_frequencies(case), dtype=torch.float64, device=dev)
            if case["fmt"] == "fp4":
                s["pages"] = torch.zeros(count, hkv, ps // 16 * 18 * d, dtype=torch.uint8, device=dev)
            else:
                s["kp"] = torch.zeros(count, ps, hkv, d, dtype=torch.bfloat16, device=dev)
                s["vp"] = torch.zeros(count, ps, hkv, d, dtype=torch.bfloat16, device=dev)
    if own:
        from cross_model_attention_gb300 import mapflow
        if "pages" in s:
            s["cache"] = mapflow.PagedCache.fp4(s["pages"], ps, d, k_scale=s["k_scale"], v_scale=s["v_scale"])
        else:
            s["cache"] = mapflow.PagedCache.bf16(s["kp"], s["vp"])
        if case["op"] == "append":
            s["rope"] = mapflow.RotaryPlan(case["rot"], base=case["base"], layout=case["layout"],
                                           scaling=case["scaling"], factor=case["factor"],
                                           original_length=case["orig"])
    return s


def _filled(count, s, rnd):
    """4-bit pages of `count` pages of random keys and values."""
    case = s["case"]
    ps, hkv, d = case["ps"], case["hkv"], case["d"]
    parts = []
    for scale, std in ((s["k_scale"], 1.0), (s["v_scale"], 0.7)):
        x = rnd(count, hkv, ps // 16, 16, d, std=std).float()
        parts.append(_held(x, torch.ones(hkv, device=x.device) if scale is None else scale, (1, hkv, 1, 1, 1)))
    (kc, ks), (vc, vs) = parts
    vc = vc.view(count, hkv, ps // 16, 2, 8, d // 16, 8).transpose(-3, -2)
    flat = [kc, vc, ks, vs.transpose(-1, -2)]
    return torch.cat([x.reshape(count, hkv, ps // 16, -1) for x in flat], -1).view(count, hkv, -1)


# --------------------------------------------------------------------- run --
def run(s):
    case = s["case"]
    if case["op"] == "attend":
        if own:
            s["cache"].attend(s["q"], s["table"], s["lens"], window=case["window"] or None, sinks=case["sinks"],
                              softcap=case["softcap"] or None, slopes=s["slopes"], o=s["o"], lse=s["lse"])
            return {"o": s["o"], "lse": s["lse"]}
        return _attend(s)
    if own:
        if case["op"] == "append":
            s["cache"].append(s["k"], s["v"], s["seq"], s["at"], s["table"], rope=s["rope"], positions=s["pos"],
                              k_weight=s["w"], eps=_EPS)
        s["cache"].read(s["seq"], s["at"], s["table"], k=s["ko"], v=s["vo"])
        return {"k": s["ko"], "v": s["vo"]}
    if case["op"] == "append":
        _append(s)
    return _read(s)


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
        ramp = [min(1.0, max(0.0, (i - low) / max(high - low, 1e-3))) for i in range(rot // 2)]
        return [x / f * r + x * (1.0 - r) for x, r in zip(plain, ramp)]
    return plain


def _gain(case):
    # (the table's gain is a 32-bit number)
    return float(torch.tensor(0.1 * math.log(case["factor"]) + 1.0)) if case["scaling"] == "yarn" else 1.0


def _held(x, g, shape):
    """x [..., d] in 4 bits: (bytes of two codes [..., d/2], e4m3 scales as bytes [..., d/16])."""
    g = g.to(x.dtype).view(shape)
    b = x.unflatten(-1, (-1, 16))
    sc = (b.abs().amax(-1) / (6.0 * g)).clamp_max(448.0).float().to(torch.float8_e4m3fn)
    sg = (sc.to(x.dtype) * g).unsqueeze(-1)
    t = torch.where(sg > 0, b.abs() / sg, 0.0)
    code = torch.zeros_like(t, dtype=torch.uint8)
    code += (t > 0.25).to(torch.uint8) + (t >= 0.75) + (t > 1.25) + (t >= 1.75) + (t > 2.5) + (t >= 3.5) + (t > 5.0)
    code |= (b < 0).to(torch.uint8) << 3
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), sc.view(torch.uint8)


def _values(codes, scales, g, shape):
    """What bytes of codes [..., d/2] with scales [..., d/16] stand for, fp32."""
    lut = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    lut = torch.cat([lut, -lut])
    x = torch.stack([lut[(codes & 15).long()], lut[(codes >> 4).long()]], -1).flatten(-2)
    x = (x.unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2)
    return x if g is None else x * g.view(shape)


def _rotated(s, dt):
    case = s["case"]
    x = s["k"].to(dt)
    if s["w"] is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS) * s["w"].to(dt)
    rot = case["rot"]
    turn = (s["pos"].double()[:, None] * s["freq"]).remainder(2.0 * math.pi)  # far positions: angles in 64 bits
    cos = (turn.cos() * _gain(case)).to(dt)[:, None]
    sin = (turn.sin() * _gain(case)).to(dt)[:, None]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if case["layout"] == "interleaved" else \
        (x[..., : rot // 2], x[..., rot // 2 : rot])
    y, z = a * cos - b * sin, b * cos + a * sin
    first = torch.stack([y, z], -1).flatten(-2) if case["layout"] == "interleaved" else torch.cat([y, z], -1)
    return torch.cat([first, x[..., rot:]], -1)


def _places(s):
    """Of the tokens that belong to a sequence: which they are, their page and their place in it."""
    ps = s["case"]["ps"]
    t = torch.nonzero(s["seq"] >= 0).squeeze(-1)
    at = s["at"][t].long()
    return t, s["table"][s["seq"][t].long(), at // ps].long(), at % ps


def _bytes(s, page, o):
    """Where in `pages` the tokens' bytes are: keys' and values' codes, keys' and values' scales, each [t][hkv][...]."""
    hkv, d, ps = s["case"]["hkv"], s["case"]["d"], s["case"]["ps"]
    dev = page.device
    h = torch.arange(hkv, device=dev)
    base = (((page[:, None] * hkv + h) * (ps // 16) + o[:, None] // 16) * (18 * d))[..., None]
    i = (o % 16)[:, None, None]
    j, b = torch.arange(d // 2, device=dev), torch.arange(d // 16, device=dev)
    return (base + i * (d // 2) + j,
            base + 8 * d + (i // 8) * (4 * d) + (j // 8) * 64 + (i % 8) * 8 + j % 8,
            base + 16 * d + i * (d // 16) + b,
            base + 17 * d + b * 16 + i)


def _append(s):
    case = s["case"]
    t, page, o = _places(s)
    if case["fmt"] == "bf16":
        s["kp"][page, o] = _rotated(s, torch.float32)[t].to(torch.bfloat16)
        s["vp"][page, o] = s["v"][t]
        return
    one = torch.ones(case["hkv"], device=t.device)
    shape = (1, case["hkv"], 1, 1)
    # 64 bits: a value next to the border between two codes has to find its side
    kc, ks = _held(_rotated(s, torch.float64)[t], one if s["k_scale"] is None else s["k_scale"].double(), shape[:3])
    vc, vs = _held(s["v"][t].double(), one if s["v_scale"] is None else s["v_scale"].double(), shape[:3])
    flat = s["pages"].view(-1)
    ikc, ivc, iks, ivs = _bytes(s, page, o)
    flat[ikc], flat[ivc], flat[iks], flat[ivs] = kc, vc, ks, vs


def _read(s):
    case = s["case"]
    t, page, o = _places(s)
    k, v = torch.zeros_like(s["ko"]), torch.zeros_like(s["vo"])
    if case.get("fmt") == "bf16":
        k[t], v[t] = s["kp"][page, o], s["vp"][page, o]
        return {"k": k, "v": v}
    flat = s["pages"].view(-1)
    ikc, ivc, iks, ivs = _bytes(s, page, o)
    shape = (1, case["hkv"], 1)
    k[t] = _values(flat[ikc], flat[iks], s["k_scale"], shape).to(torch.bfloat16)
    v[t] = _values(flat[ivc], flat[ivs], s["v_scale"], shape).to(torch.bfloat16)
    return {"k": k, "v": v}


def _attend(s):
    case = s["case"]
    n, lq, hq, hkv, d, ps = case["n"], case["lq"], case["hq"], case["hkv"], case["d"], case["ps"]
    G, mp = hq // hkv, s["table"].shape[1]
    nb = ps // 16
    # the requests' pages, [n][hkv][mp * nb][18 d] bytes, and the values in them
    raw = s["pages"][s["table"].long()].view(n, mp, hkv, nb, 18 * d).transpose(1, 2).reshape(n, hkv, mp * nb, 18 * d)
    shape = (1, hkv, 1, 1, 1)
    K = _values(raw[..., : 8 * d].unflatten(-1, (16, d // 2)), raw[..., 16 * d : 17 * d].unflatten(-1, (16, d // 16)),
                s["k_scale"], shape).reshape(n, hkv, mp * ps, d)
    vc = raw[..., 8 * d : 16 * d].unflatten(-1, (2, d // 16, 8, 8)).transpose(-3, -2).flatten(-4)
    V = _values(vc.unflatten(-1, (16, d // 2)), raw[..., 17 * d :].unflatten(-1, (d // 16, 16)).transpose(-1, -2).contiguous(),
                s["v_scale"], shape).reshape(n, hkv, mp * ps, d)
    q = s["q"].float().view(n, lq, hkv, G, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, G * lq, d) * (1.0 / math.sqrt(d))
    sc = (q @ K.transpose(-1, -2)).view(n, hkv, G, lq, mp * ps)
    if case["softcap"]:
        sc = torch.tanh_(sc.div_(case["softcap"])).mul_(case["softcap"])
    j = torch.arange(mp * ps, device=q.device)
    i = (s["lens"].long()[:, None] - lq + torch.arange(lq, device=q.device))[:, None, None, :, None]
    if s["slopes"] is not None:
        sc -= s["slopes"].view(1, hkv, G, 1, 1) * (i - j)
    seen = j <= i
    if case["window"]:
        seen = seen & ((i - j < case["window"]) | (j < case["sinks"]))
    sc = sc.masked_fill_(~seen, float("-inf"))
    m = sc.amax(-1, keepdim=True)
    m = m.masked_fill(m == float("-inf"), 0.0)
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p.view(n, hkv, G * lq, -1) @ V).view(n, hkv, G, lq, d) / l.clamp_min(1e-30)
    lse = (m + l.log()).squeeze(-1)
    return {"o": o.permute(0, 3, 1, 2, 4).reshape(n, lq, hq, d).to(torch.bfloat16),
            "lse": lse.permute(0, 3, 1, 2).reshape(n, lq, hq)}


# -------------------------------------------------------------------- work --
def _seen(i, window, sinks):
    """Keys that the row at position i sees."""
    if not window or i < window:
        return i + 1
    return window + min(sinks, i - window + 1)


def work(case):
    hkv, d = case["hkv"], case["d"]
    held = 9 * d // 8  # bytes of a token's key and value of one head in 4 bits: 2 (d / 2 + d / 16)
    if case["op"] == "attend":
        n, lq, hq = case["n"], case["lq"], case["hq"]
        pairs = keys = 0
        for x in _cache_lens(case, 0):
            at = [i for i in range(x - lq, x) if i >= 0]
            pairs += sum(_seen(i, case["window"], case["sinks"]) for i in at)
            lo = max(0, at[0] - case["window"] + 1) if case["window"] and at else 0
            keys += x - lo + min(lo, case["sinks"])
        return {"bytes": keys * hkv * held + n * lq * hq * (4 * d + 4) + 4 * n + 4 * keys // case["ps"],
                "flops": 4 * d * hq * pairs}
    values = (case["T"] - case.get("pad", 0)) * hkv * d  # of keys, and as many of values
    rows = 2 * 2 * values
    cached = values * 9 // 8 if case.get("fmt", "fp4") == "fp4" else rows
    if case["op"] == "read":
        return {"bytes": cached + rows + 8 * case["T"], "flops": 2 * 2 * values}
    return {"bytes": 2 * rows + cached + 12 * case["T"], "flops": 20 * values}


# ------------------------------------------------------------------- exact --
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
_E4M3 = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]


def _nearest(grid, x):
    """Places in `grid` (ascending, from 0) of the numbers nearest to x >= 0, the even place of two as near."""
    grid = torch.tensor(grid, dtype=torch.float64, device=x.device)
    up = torch.bucketize(x, grid).clamp(1, len(grid) - 1)
    below, above = x - grid[up - 1], grid[up] - x
    lower = (below < above) | ((below == above) & (up % 2 == 1))
    return torch.where(lower, up - 1, up)


def _rounded(x, g):
    """The 4-bit value of each of x [t, hkv, d] under head scales g (or None), fp64."""
    g = torch.ones(x.shape[1], device=x.device) if g is None else g
    g = g.double()[None, :, None, None]
    b = x.double().reshape(*x.shape[:2], -1, 16)
    e4, e2 = (torch.tensor(v, dtype=torch.float64, device=x.device) for v in (_E4M3, _E2M1))
    sc = e4[_nearest(_E4M3, b.abs().amax(-1, keepdim=True) / (6.0 * g))] * g
    t = torch.where(sc > 0, b.abs() / sc.clamp_min(1e-300), torch.zeros_like(b))
    return (torch.sign(b) * e2[_nearest(_E2M1, t)] * sc).reshape(x.shape)


def _decoded(code, scale, dev):
    """fp64 values of codes 0..15 with e4m3 scales given as bytes of the same shape."""
    e2 = torch.tensor(_E2M1 + [-v for v in _E2M1], dtype=torch.float64, device=dev)
    e4 = torch.tensor(_E4M3, dtype=torch.float64, device=dev)
    return e2[code.long()] * e4[scale.long()]


def _block_of(pages, d):
    """Keys and values [..., 16 tokens, d] of 16-token blocks [..., 18 d] of bytes, fp64, without the heads' scales."""
    dev = pages.device
    tok, dim = torch.arange(16, device=dev)[:, None], torch.arange(d, device=dev)[None]
    kb = pages[..., tok * (d // 2) + dim // 2]
    vb = pages[..., 8 * d + (tok // 8) * 4 * d + (dim // 16) * 64 + (tok % 8) * 8 + (dim % 16) // 2]
    ks = pages[..., 16 * d + tok * (d // 16) + dim // 16]
    vs = pages[..., 17 * d + (dim // 16) * 16 + tok]
    nib = 4 * (dim % 2)
    return _decoded((kb >> nib) & 15, ks, dev), _decoded((vb >> nib) & 15, vs, dev)


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    hkv, d, ps = case["hkv"], case["d"], case["ps"]
    dev = s["table"].device
    if case["op"] == "append":
        x = s["k"].to(f64)
        if s["w"] is not None:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + _EPS) * s["w"].to(f64)
        th = s["pos"].to(f64)[:, None] * s["freq"][None]
        half, rot = case["rot"] // 2, case["rot"]
        if case["layout"] == "interleaved":
            ia, ib = torch.arange(0, rot, 2), torch.arange(1, rot, 2)
        else:
            ia, ib = torch.arange(half), torch.arange(half, rot)
        z = torch.complex(x[..., ia], x[..., ib]) * torch.polar(torch.full_like(th, _gain(case)), th)[:, None]
        y = x.clone()
        y[..., ia], y[..., ib] = z.real, z.imag
        v = s["v"].to(f64)
        if case["fmt"] == "fp4":
            y, v = _rounded(y, s["k_scale"]), _rounded(v, s["v_scale"])
        used = (s["seq"] >= 0)[:, None, None]
        return {"k": torch.where(used, y, 0.0), "v": torch.where(used, v, 0.0)}
    gk = (torch.ones(hkv, device=dev) if s["k_scale"] is None else s["k_scale"]).to(f64)
    gv = (torch.ones(hkv, device=dev) if s["v_scale"] is None else s["v_scale"]).to(f64)

    def tokens(r, x):
        """Keys and values [hkv, x, d] of the first x tokens of sequence r."""
        raw = s["pages"][s["table"][r, : -(-x // ps)].long()].view(-1, hkv, ps // 16, 18 * d)
        out = []
        for part, gs in zip(_block_of(raw, d), (gk, gv)):
            out.append(part.permute(1, 0, 2, 3, 4).reshape(hkv, -1, d)[:, :x] * gs[:, None, None])
        return out
    if case["op"] == "read":
        lens = _split(case)
        ks, vs = zip(*(tokens(r, x) for r, x in enumerate(lens)))
        return {"k": torch.cat(ks, 1).transpose(0, 1), "v": torch.cat(vs, 1).transpose(0, 1)}
    n, lq, hq = case["n"], case["lq"], case["hq"]
    G = hq // hkv
    o = torch.zeros(n, lq, hq, d, dtype=f64, device=dev)
    lse = torch.full((n, lq, hq), -math.inf, dtype=f64, device=dev)
    for r, x in enumerate(_cache_lens(case, seed)):
        if x == 0:
            continue
        k, v = tokens(r, x)
        sc = torch.einsum("tkgd,kjd->kgtj", s["q"][r].to(f64).view(lq, hkv, G, d), k) / math.sqrt(d)
        if case["softcap"]:
            sc = case["softcap"] * torch.tanh(sc / case["softcap"])
        far = (x - lq + torch.arange(lq, device=dev))[:, None] - torch.arange(x, device=dev)[None]
        if s["slopes"] is not None:
            sc = sc - s["slopes"].to(f64).view(hkv, G, 1, 1) * far
        hide = far < 0
        if case["window"]:
            hide = hide | ((far >= case["window"]) & (torch.arange(x, device=dev)[None] >= case["sinks"]))
        sc = sc.masked_fill(hide, -math.inf)
        lse[r] = torch.logsumexp(sc, -1).permute(2, 0, 1).reshape(lq, hq)
        p = torch.softmax(sc, -1).nan_to_num(0.0)  # a row that sees nothing
        o[r] = torch.einsum("kgtj,kjd->tkgd", p, v).reshape(lq, hq, d)
    return {"o": o, "lse": lse}
