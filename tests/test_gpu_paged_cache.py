"""A paged cache, appended to, read back and attended over, against the fp64
definitions of tests/paged_ref.py."""
import math
import threading

import pytest
import torch

from cross_model_attention_gb300 import mapflow
from tests import layer_ref
from tests import paged_ref as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "a GPU is needed"
    return torch.device("cuda", torch.cuda.current_device())


def _rnd(g, dev, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device=dev) * std).to(BF)


def _gen(dev, seed=0):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


def _scales(g, dev, H, on=True):
    return torch.exp(0.7 * torch.randn(H, generator=g, device=dev)) if on else None


def _pages(dev, n, H, ps, d, byte=0xff):
    """Pages of nothing that is finite: scales of NaN."""
    return torch.full((n, H, ps // 16 * 18 * d), byte, dtype=torch.uint8, device=dev)


def _tokens(lens, dev, start=0):
    seq = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens)).to(torch.int32).to(dev)
    at = torch.cat([torch.arange(x) for x in lens]).to(torch.int32).to(dev) + start
    return seq, at.to(torch.int32)


def _slots(seq, at, table, ps):
    return table[seq.long(), at.long() // ps].long(), at.long() % ps


def _rotated(k, w, norm, pos, rope, layout, rot, **kw):
    """fp64 keys and the bound of their fp32 evaluation."""
    if rope is None:
        y = k.double()
        if norm:
            y = y * (y.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
            if w is not None:
                y = y * w.double()
        return y, k.double().abs() * 2.0 ** -17
    f, gain = layer_ref.rope_frequencies(rot, **kw)
    return layer_ref.rope(k, w, norm, 1e-6, pos, f, float(torch.tensor(gain)), rot, layout)


def _check_held(pages, ps, d, page, o, y, v, gk, gv):
    """The pages hold exactly what the definition says of y and v [T, H, d]; a zero's sign is free."""
    kc, ks, vc, vs = (x[page, o].long() for x in ref.unpack(pages, ps, d))
    H = y.shape[1]
    one = torch.ones(H, device=y.device)
    for code, scale, x, g in ((kc, ks, y, gk), (vc, vs, v.double(), gv)):
        want_c, want_s = ref.hold(x, one if g is None else g)
        assert torch.equal(scale, want_s)
        fine = (want_s != 0x7f).repeat_interleave(16, -1)
        same = (code == want_c) | ((code & 7 == 0) & (want_c & 7 == 0)) | ~fine
        assert same.all(), (~same).nonzero()[:5]


ROPES = [None, dict(rot=128, layout="half", base=1e6), dict(rot=128, layout="interleaved", base=1e4),
         dict(rot=64, layout="half", base=1e4, scaling="linear", factor=4.0),
         dict(rot=64, layout="interleaved", base=1e6, scaling="yarn", factor=8.0, original_length=32768),
         dict(rot=20, layout="half", base=1e4), dict(rot=32, layout="half", base=1e6),
         dict(rot=6, layout="interleaved", base=1e4), dict(rot=48, layout="half", base=1e4, scaling="ntk", factor=2.0)]


@pytest.mark.parametrize("case", range(36))
def test_append_holds_what_the_definition_says(dev, case):
    g = _gen(dev, case)
    kw = ROPES[case % len(ROPES)]
    norm, d = case % 2 == 0, 64 if case % 3 == 0 else 128
    H, ps = (1, 8, 3, 2)[case % 4], (16, 64, 48, 128)[case // 9]
    lens = ([1], [5, 37, 1, 20], [129, 64], [300, 1, 1, 2, 16, 17])[case % 4]
    T = sum(lens)
    seq, at = _tokens(lens, dev, start=7 if case % 5 == 0 else 0)
    mp = (max(lens) + 7 + ps - 1) // ps
    table = torch.randperm(len(lens) * mp + 2, generator=g, device=dev)[: len(lens) * mp].to(torch.int32).view(-1, mp)
    pages = _pages(dev, len(lens) * mp + 2, H, ps, d)
    gk, gv = _scales(g, dev, H, case % 3 != 1), _scales(g, dev, H, case % 3 == 1)
    kv = _rnd(g, dev, T, 2 * H * d)  # parts of one projection
    k, v = kv[:, : H * d].view(T, H, d), kv[:, H * d:].view(T, H, d)
    w = (1 + 0.1 * torch.randn(d, generator=g, device=dev)).to(BF) if norm and case % 4 else None
    pos = (at + (0, 1000003, 77)[case % 3]).to(torch.int32)
    plan = None
    if kw is not None:
        kw = dict(kw, rot=min(kw["rot"], d))
        plan = mapflow.RotaryPlan(kw["rot"], **{a: b for a, b in kw.items() if a != "rot"})
    cache = mapflow.PagedCache.fp4(pages, ps, d, k_scale=gk, v_scale=gv)
    before = pages.clone()
    cache.append(k, v, seq, at, table, rope=plan, positions=pos if plan else None, k_weight=w, norm=norm)
    if kw is None:
        y, _ = _rotated(k, w, norm, None, None, None, None)
    else:
        y, _ = _rotated(k, w, norm, pos, plan, kw["layout"], kw["rot"],
                        **{a: b for a, b in kw.items() if a not in ("rot", "layout")})
    page, o = _slots(seq, at, table, ps)
    _check_held(pages, ps, d, page, o, y, v, gk, gv)
    # nothing else was written
    kept = torch.ones(pages.shape[0], ps, dtype=torch.bool, device=dev)
    kept[page, o] = False
    for a, b in zip(ref.unpack(pages, ps, d), ref.unpack(before, ps, d)):
        assert torch.equal(a[kept], b[kept])
    # and it is read back as the values it stands for, rounded once
    ko, vo = cache.read(seq, at, table)
    one = torch.ones(H, device=dev)
    kc, ks, vc, vs = (x[page, o] for x in ref.unpack(pages, ps, d))
    for got, c, s, gs in ((ko, kc, ks, gk), (vo, vc, vs, gv)):
        want = ref.stands_for(c, s, one if gs is None else gs)
        assert torch.allclose(got.double(), want, rtol=2.0 ** -8 + 2.0 ** -23, atol=0)


@pytest.mark.parametrize("d", [64, 128])
def test_values_on_the_border_between_two_codes(dev, d):
    # integers and halves with scales of few bits: most quotients are exact, many are ties
    g = _gen(dev, d)
    T, H = 777, 4
    k = (torch.randint(-24, 25, (T, H, d), generator=g, device=dev) / 4).to(BF)
    v = (torch.randint(-56, 57, (T, H, d), generator=g, device=dev) / 2).to(BF)
    for gs in (None, torch.tensor([0.5, 1.0, 1.5, 0.75], device=dev)):
        pages = _pages(dev, 8, H, 128, d)
        seq, at = _tokens([T], dev)
        table = torch.arange(8, dtype=torch.int32, device=dev)[None]
        cache = mapflow.PagedCache.fp4(pages, 128, d, k_scale=gs, v_scale=gs)
        cache.append(k, v, seq, at, table)
        page, o = _slots(seq, at, table, 128)
        _check_held(pages, 128, d, page, o, k.double(), v, gs, gs)


def test_zeros_small_large_and_not_finite(dev):
    d, H, T = 128, 2, 9
    g = _gen(dev, 5)
    x = _rnd(g, dev, T, H, d)
    x[0] = 0
    x[1] *= 1e-30
    x[2] *= 1e30
    x[3, 0, 17] = math.inf
    x[4, 1, 90] = math.nan
    x[5, 0, 3] = -math.inf
    x[6, :, 32:64] = 0
    pages = _pages(dev, 2, H, 16, d, byte=0)
    seq, at = _tokens([T], dev)
    table = torch.tensor([[1]], dtype=torch.int32, device=dev)
    cache = mapflow.PagedCache.fp4(pages, 16, d)
    cache.append(x, x.clone(), seq, at, table)
    page, o = _slots(seq, at, table, 16)
    _check_held(pages, 16, d, page, o, x.double(), x, None, None)
    k, v = cache.read(seq, at, table)
    bad = torch.zeros_like(x, dtype=torch.bool)
    bad[3, 0, 16:32] = bad[4, 1, 80:96] = bad[5, 0, :16] = True
    assert torch.equal(k.isnan(), bad) and torch.equal(v.isnan(), bad)
    # with norm and rotary: rows of huge values are normed like any, a row's infinity makes its pairs NaN
    plan = mapflow.RotaryPlan(128)
    cache.append(x, x.clone(), seq, at, table, rope=plan, norm=True)
    y, _ = _rotated(x, None, True, at, plan, "half", 128)
    kc, ks, _, _ = (z[page, o].long() for z in ref.unpack(pages, 16, d))
    fine = [0, 1, 2, 6, 7, 8]
    want_c, want_s = ref.hold(y, torch.ones(H, device=dev))
    assert torch.equal(ks[fine], want_s[fine])
    assert ((kc == want_c) | ((kc & 7 == 0) & (want_c & 7 == 0)))[fine].all()
    for t, h in ((3, 0), (4, 1), (5, 0)):
        assert torch.equal(ks[t, h] == 0x7f, want_s[t, h] == 0x7f)
    assert not (ks[3, 1] == 0x7f).any()


def test_tokens_that_are_left_out(dev):
    d, H, ps, T = 64, 3, 16, 12
    g = _gen(dev, 9)
    k, v = _rnd(g, dev, T, H, d), _rnd(g, dev, T, H, d)
    #                    none                past   negative     page -1  page 99
    seq = torch.tensor([0, -1, 1, 0, 2, 7, 0, 1, 1, 0, 1, -5], dtype=torch.int32, device=dev)
    at = torch.tensor([0, 3, 31, 32, 0, 0, -1, 5, 20, 40, 1 << 30, 0], dtype=torch.int32, device=dev)
    table = torch.tensor([[2, 0], [99, 1]], dtype=torch.int32, device=dev)
    used = [0, 2, 8]  # (0, 0) on page 2, (1, 31) and (1, 20) on page 1
    pages = _pages(dev, 4, H, ps, d, byte=0x11)
    cache = mapflow.PagedCache.fp4(pages, ps, d)
    before = pages.clone()
    cache.append(k, v, seq, at, table)
    pg, o = torch.tensor([2, 1, 1], device=dev), torch.tensor([0, 15, 4], device=dev)
    _check_held(pages, ps, d, pg, o, k[used].double(), v[used], None, None)
    kept = torch.ones(4, ps, dtype=torch.bool, device=dev)
    kept[pg, o] = False
    for a, b in zip(ref.unpack(pages, ps, d), ref.unpack(before, ps, d)):
        assert torch.equal(a[kept], b[kept])
    ko, vo = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    cache.read(seq, at, table, k=ko, v=vo)
    rest = [i for i in range(T) if i not in used]
    assert (ko[rest] == 7).all() and (vo[rest] == 7).all() and (ko[used] != 7).any()
    # the same for bf16 rows
    kp, vp = torch.full((4, ps, H, d), 5.0, dtype=BF, device=dev), torch.full((4, ps, H, d), 5.0, dtype=BF, device=dev)
    rows = mapflow.PagedCache.bf16(kp, vp)
    rows.append(k, v, seq, at, table)
    assert torch.equal(kp[pg, o], k[used]) and torch.equal(vp[pg, o], v[used])
    assert (kp[kept] == 5).all() and (vp[kept] == 5).all()
    ko, vo = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    rows.read(seq, at, table, k=ko, v=vo)
    assert torch.equal(ko[used], k[used]) and (ko[rest] == 7).all() and (vo[rest] == 7).all()


@pytest.mark.parametrize("case", range(9))
def test_append_bf16(dev, case):
    g = _gen(dev, 100 + case)
    kw = ROPES[case]
    norm, d, H = case % 2 == 1, 64 if case % 3 == 0 else 128, 5
    lens, ps = [33, 1, 70], 37
    T = sum(lens)
    seq, at = _tokens(lens, dev)
    table = torch.tensor([[4, 0], [1, 6], [3, 5]], dtype=torch.int32, device=dev)
    kp = torch.zeros(7, ps, 2, H, d, dtype=BF, device=dev)[:, :, 0]  # tokens further apart than their heads
    vp = torch.zeros(7, ps, H, d, dtype=BF, device=dev)
    k, v = _rnd(g, dev, T, H, d), _rnd(g, dev, T, H, d)
    pos = (at + 12345).to(torch.int32)
    plan = None
    if kw is not None:
        kw = dict(kw, rot=min(kw["rot"], d))
        plan = mapflow.RotaryPlan(kw["rot"], **{a: b for a, b in kw.items() if a != "rot"})
    cache = mapflow.PagedCache.bf16(kp, vp)
    cache.append(k, v, seq, at, table, rope=plan, positions=pos if plan else None, norm=norm)
    kw = kw or {}
    y, bound = _rotated(k, None, norm, pos, plan, kw.get("layout"), kw.get("rot"),
                        **{a: b for a, b in kw.items() if a not in ("rot", "layout")})
    page, o = _slots(seq, at, table, ps)
    assert ((kp[page, o].double() - y).abs() <= y.abs() * 2.0 ** -8 + bound * 1.01).all()
    assert torch.equal(vp[page, o], v)
    ko, vo = cache.read(seq, at, table)
    assert torch.equal(ko, kp[page, o]) and torch.equal(vo, v)
    if plan is not None:  # as the rotary layer has them, and without `positions` at the places
        # (each within y 2^-8 + bound of y, so within twice that of each other)
        _, kr = plan.apply(k.clone(), k, pos, norm=norm)
        assert ((ko.double() - kr.double()).abs() <= 2 * (y.abs() * 2.0 ** -8 + bound * 1.01)).all()
        cache.append(k, v, seq, at, table, rope=plan, norm=norm)
        again = cache.read(seq, at, table)[0]
        cache.append(k, v, seq, at, table, rope=plan, positions=at, norm=norm)
        assert torch.equal(cache.read(seq, at, table)[0], again) and not torch.equal(ko, again)


# --------------------------------------------------------------- attention --
def _world(dev, seed, n, H, d, ps, lens, scales=True, spare=2):
    """Pages of random keys and values for n requests, NaN wherever no key is; the table names
    no page past a request's keys."""
    g = _gen(dev, seed)
    mp = max(1, max((x + ps - 1) // ps for x in lens))
    need = [(x + ps - 1) // ps for x in lens]
    ids = torch.randperm(sum(need) + spare, generator=g, device=dev)
    table = torch.full((n, mp), -7, dtype=torch.int32, device=dev)
    c = 0
    for r, x in enumerate(need):
        table[r, :x] = ids[c: c + x].to(torch.int32)
        c += x
    gk, gv = _scales(g, dev, H, scales), _scales(g, dev, H, scales)
    one = torch.ones(H, device=dev)
    N = sum(need) + spare
    kc, vc = (torch.randint(0, 16, (N, ps, H, d), generator=g, device=dev) for _ in range(2))
    ks, vs = (torch.randint(0x28, 0x38, (N, ps, H, d // 16), generator=g, device=dev) for _ in range(2))
    alive = torch.zeros(N, ps, dtype=torch.bool, device=dev)
    for r, x in enumerate(lens):
        j = torch.arange(x, device=dev)
        alive[table[r].long()[j // ps], j % ps] = True
    ks[~alive], vs[~alive] = 0x7f, 0x7f
    pages = ref.pack(kc, ks, vc, vs)
    k = ref.stands_for(kc, ks, one if gk is None else gk * 0.2)
    v = ref.stands_for(vc, vs, one if gv is None else gv)
    if gk is not None:
        gk = gk * 0.2
    lens_t = torch.tensor(lens, dtype=torch.int32, device=dev)

    def keys(r, x=None):
        j = torch.arange(lens[r] if x is None else x, device=dev)
        at = table[r].long()[j // ps], j % ps
        return k[at], v[at]
    return g, pages, table, lens_t, gk, gv, keys


def _check_attend(dev, q, lens, keys, o, lse, window, sinks, scale, softcap, slopes, which=None, hidden=None):
    for r in range(len(lens)) if which is None else which:
        k, v = keys(r)
        wo, wl, bo, bl = ref.attend(q[r], k, v, lens[r], window, sinks, scale, softcap, slopes,
                                    None if hidden is None else hidden(r))
        got, got_l = o[r].double(), lse[r].double()
        assert torch.isfinite(got).all(), r
        assert ((got - wo).abs() <= bo + 1e-30).all(), (r, ((got - wo).abs() - bo).max())
        empty = wl == -math.inf
        assert torch.equal(got_l == -math.inf, empty)
        assert ((got_l - wl).abs() <= bl)[~empty].all(), (r, ((got_l - wl).abs() - bl)[~empty].max())


EDGES = [0, 1, 15, 16, 17, 31, 32, 33, 47, 63, 64, 65, 127, 128, 129, 200, 500]
ATTEND = [
    # d, G, H, Lq, ps, lens, window, sinks, softcap, slopes, scales
    (128, 4, 8, 1, 64, EDGES, 0, 0, None, False, True),
    (64, 4, 3, 1, 16, EDGES, 0, 0, None, False, False),
    (128, 1, 5, 1, 32, EDGES, 0, 0, 20.0, False, True),
    (64, 1, 40, 1, 48, EDGES, 0, 0, None, True, True),
    (128, 8, 2, 1, 128, EDGES, 33, 5, None, False, True),
    (128, 3, 2, 3, 16, EDGES, 0, 0, 30.0, True, True),       # 9 rows
    (64, 5, 2, 3, 64, EDGES, 64, 70, None, False, True),      # 15 rows
    (128, 8, 2, 8, 64, EDGES, 0, 0, None, False, False),     # 64 rows
    (64, 16, 1, 8, 32, EDGES, 100, 1, 10.0, True, True),      # 128 rows
    (128, 128, 1, 1, 64, [700, 3], 0, 0, None, False, True),
    (128, 1, 1, 128, 64, [700, 100, 128], 0, 0, None, False, True),
    (128, 4, 2, 1, 64, EDGES, 1, 0, None, False, True),
    (128, 4, 2, 2, 64, EDGES, 1, 1, None, False, True),
    (128, 2, 2, 4, 16, EDGES, 40, 200, None, False, True),   # sinks that meet the window
    (128, 4, 1, 1, 64, [20000], 0, 0, None, False, True),    # one unit over all SMs
    (64, 2, 1, 5, 128, [30001], 0, 0, 40.0, True, True),
    (128, 4, 8, 1, 64, [9000, 1, 0, 4000, 12, 0, 0, 700], 0, 0, None, False, True),
    (128, 4, 8, 1, 64, [9000, 1, 0, 4000, 12, 0, 0, 700], 513, 33, None, True, True),
    (128, 6, 8, 2, 32, [5000, 4999, 1, 70], 0, 0, None, False, True),
]


@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attend(dev, case):
    d, G, H, Lq, ps, lens, window, sinks, softcap, slopes, scales = ATTEND[case]
    n = len(lens)
    g, pages, table, lens_t, gk, gv, keys = _world(dev, case, n, H, d, ps, lens, scales)
    cache = mapflow.PagedCache.fp4(pages, ps, d, k_scale=gk, v_scale=gv)
    q = _rnd(g, dev, n, Lq, H * G, d, std=1.5)
    sl = 2.0 ** (-8.0 * torch.arange(1, H * G + 1, device=dev) / (H * G)) if slopes else None
    lse = torch.empty(n, Lq, H * G, dtype=torch.float32, device=dev)
    o = cache.attend(q, table, lens_t, window=window or None, sinks=sinks, softcap=softcap, slopes=sl, lse=lse)
    _check_attend(dev, q, lens, keys, o, lse, window, sinks, d ** -0.5, softcap, sl)
    for r, x in enumerate(lens):  # rows that see nothing
        for t in range(max(0, Lq - x)):
            assert (o[r, t] == 0).all() and (lse[r, t] == -math.inf).all()
    again = cache.attend(q, table, lens_t, window=window or None, sinks=sinks, softcap=softcap, slopes=sl)
    assert torch.equal(again, o)


def test_attend_many_requests(dev):
    # more requests than threads, most of them unused, and tokens further apart than their heads
    n, H, G, d, ps = 2500, 2, 4, 64, 16
    lens = [0] * n
    for i in range(0, n, 37):
        lens[i] = 1 + (i * 13) % 150
    g, pages, table, lens_t, gk, gv, keys = _world(dev, 3, n, H, d, ps, lens)
    cache = mapflow.PagedCache.fp4(pages, ps, d, k_scale=gk, v_scale=gv)
    wide = _rnd(g, dev, n, 1, 2 * H * G, d)
    q = wide[:, :, : H * G]
    o = torch.full((n, 1, H * G + 8, d), 3.0, dtype=BF, device=dev)
    lse = torch.empty(n, 1, H * G, dtype=torch.float32, device=dev)
    cache.attend(q, table, lens_t, o=o[:, :, : H * G], lse=lse, scale=0.3)
    used = [i for i in range(n) if lens[i]]
    _check_attend(dev, q, lens, keys, o[:, :, : H * G], lse, 0, 0, 0.3, None, None, which=used)
    idle = torch.tensor([i for i in range(n) if not lens[i]], device=dev)
    assert (o[idle][:, :, : H * G] == 0).all() and (lse[idle] == -math.inf).all()
    assert (o[:, :, H * G:] == 3).all()


def test_attend_of_lengths_past_the_table_and_below_zero(dev):
    lens = [64, 40, 33]
    g, pages, table, lens_t, gk, gv, keys = _world(dev, 8, 3, 2, 128, 32, lens)
    cache = mapflow.PagedCache.fp4(pages, 32, 128, k_scale=gk, v_scale=gv)
    q = _rnd(g, dev, 3, 1, 8, 128)
    o = cache.attend(q, table, torch.tensor([1 << 30, -5, 33], dtype=torch.int32, device=dev))
    want = cache.attend(q, table, torch.tensor([64, 0, 33], dtype=torch.int32, device=dev))
    assert torch.equal(o, want) and (o[1] == 0).all()


def test_keys_on_no_page_are_hidden(dev):
    lens, ps = [300, 200, 64], 16
    g, pages, table, lens_t, gk, gv, keys = _world(dev, 11, 3, 2, 128, ps, lens)
    ids = table.clone()
    ids[0, 3], ids[0, 18], ids[1, 0], ids[2, :] = -1, pages.shape[0], 1 << 30, -2
    cache = mapflow.PagedCache.fp4(pages, ps, 128, k_scale=gk, v_scale=gv)
    q = _rnd(g, dev, 3, 2, 8, 128)
    lse = torch.empty(3, 2, 8, dtype=torch.float32, device=dev)
    o = cache.attend(q, ids, lens_t, lse=lse)

    def hidden(r):
        page = ids[r].long()[torch.arange(lens[r], device=dev) // ps]
        return (page < 0) | (page >= pages.shape[0])
    _check_attend(dev, q, lens, keys, o, lse, 0, 0, 128 ** -0.5, None, None, hidden=hidden)
    assert (o[2] == 0).all()


def test_pages_before_a_window_may_be_given_back(dev):
    lens, ps, window, sinks = [1000, 517], 16, 100, 20
    g, pages, table, lens_t, gk, gv, keys = _world(dev, 12, 2, 2, 64, ps, lens)
    q = _rnd(g, dev, 2, 3, 4, 64)
    cache = mapflow.PagedCache.fp4(pages, ps, 64, k_scale=gk, v_scale=gv)
    lse = torch.empty(2, 3, 4, dtype=torch.float32, device=dev)
    ids, gone = table.clone(), pages.clone()
    for r, x in enumerate(lens):
        first, last = -(-sinks // ps), (x - 3 - window + 1) // ps
        gone[table[r, first:last].long()] = 0xff  # others' by now
        ids[r, first:last] = -1
    o = mapflow.PagedCache.fp4(gone, ps, 64, k_scale=gk, v_scale=gv).attend(q, ids, lens_t, window=window, sinks=sinks, lse=lse)
    _check_attend(dev, q, lens, keys, o, lse, window, sinks, 64 ** -0.5, None, None)
    assert torch.equal(o, cache.attend(q, table, lens_t, window=window, sinks=sinks))


def test_what_is_not_finite_stays_where_it_is_seen(dev):
    lens, ps = [100, 90, 80], 16
    g, pages, table, lens_t, gk, gv, keys = _world(dev, 13, 3, 2, 128, ps, lens, scales=False)
    cache = mapflow.PagedCache.fp4(pages, ps, 128)
    q = _rnd(g, dev, 3, 2, 8, 128)
    clean = cache.attend(q, table, lens_t)
    kc, ks, vc, vs = ref.unpack(pages, ps, 128)
    ks[table[1, 2].long(), 5, 1, 3] = 0x7f      # a key of request 1, head 1
    vs[table[0, 1].long(), 9, 0, 2] = 0x7f      # a value of request 0, head 0, dimensions 32..47
    q[2, 0, 6, 77] = math.inf
    q[2, 1, 1, 3] = math.nan
    bad = mapflow.PagedCache.fp4(ref.pack(kc, ks, vc, vs), ps, 128).attend(q, table, lens_t)
    nan = torch.zeros_like(bad, dtype=torch.bool)
    nan[1, :, 4:] = nan[0, :, :4, 32:48] = nan[2, 0, 6] = nan[2, 1, 1] = True
    assert torch.equal(bad.isnan(), nan)
    assert torch.equal(bad[~nan], clean[~nan])


@pytest.mark.parametrize("size", [1e-20, 1.0, 1e20])
def test_rows_of_any_size(dev, size):
    lens = [200, 77]
    g, pages, table, lens_t, gk, gv, keys = _world(dev, 14, 2, 2, 64, 32, lens)
    cache = mapflow.PagedCache.fp4(pages, 32, 64, k_scale=gk, v_scale=gv)
    q = (torch.randn(2, 1, 6, 64, generator=g, device=dev) * size).to(BF)
    lse = torch.empty(2, 1, 6, dtype=torch.float32, device=dev)
    o = cache.attend(q, table, lens_t, scale=0.125 / size, lse=lse)
    _check_attend(dev, q, lens, keys, o, lse, 0, 0, 0.125 / size, None, None)


def test_rising_scores_move_the_reference(dev):
    # each tile's scores are far above the last one's, then far below
    d, ps, x = 64, 64, 1024
    kc = torch.full((16, ps, 1, d), 2, device=dev)
    ks = torch.zeros(16, ps, 1, d // 16, dtype=torch.long, device=dev)
    step = torch.arange(x, device=dev)
    size = torch.where(step < 600, step // 8, (x - step) // 8)
    ks[step // ps, step % ps, 0, :] = size[:, None].clamp(0, 0x7e)
    g = _gen(dev, 15)
    vc, vs = torch.randint(0, 16, (16, ps, 1, d), generator=g, device=dev), torch.full((16, ps, 1, d // 16), 0x38, device=dev)
    pages = ref.pack(kc, ks, vc, vs)
    one = torch.ones(1, device=dev)
    k, v = ref.stands_for(kc, ks, one).reshape(x, 1, d), ref.stands_for(vc, vs, one).reshape(x, 1, d)
    table = torch.arange(16, dtype=torch.int32, device=dev)[None]
    q = torch.ones(1, 1, 2, d, dtype=BF, device=dev)
    q[:, :, 1] = -1
    lse = torch.empty(1, 1, 2, dtype=torch.float32, device=dev)
    o = mapflow.PagedCache.fp4(pages, ps, d).attend(q, table, torch.tensor([x], dtype=torch.int32, device=dev), lse=lse)
    _check_attend(dev, q, [x], lambda r: (k, v), o, lse, 0, 0, d ** -0.5, None, None)


def test_offsets_past_32_bits(dev):
    # 2.1 million pages of 2304 bytes, 4.8 GB, tokens on the first and the last
    n, ps, d = 2100000, 16, 128
    pages = torch.zeros(n, 1, 18 * d, dtype=torch.uint8, device=dev)
    cache = mapflow.PagedCache.fp4(pages, ps, d)
    g = _gen(dev, 16)
    k, v = _rnd(g, dev, 32, 1, d), _rnd(g, dev, 32, 1, d)
    seq, at = _tokens([32], dev)
    table = torch.tensor([[n - 1, 0]], dtype=torch.int32, device=dev)
    cache.append(k, v, seq, at, table)
    few = _pages(dev, 2, 1, ps, d, byte=0)
    small = mapflow.PagedCache.fp4(few, ps, d)
    near = torch.tensor([[1, 0]], dtype=torch.int32, device=dev)
    small.append(k, v, seq, at, near)
    assert torch.equal(pages[n - 1], few[1]) and torch.equal(pages[0], few[0])
    a, b = cache.read(seq, at, table), small.read(seq, at, near)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    q = _rnd(g, dev, 1, 1, 4, d)
    lens = torch.tensor([32], dtype=torch.int32, device=dev)
    assert torch.equal(cache.attend(q, table, lens), small.attend(q, near, lens))


# ------------------------------------------------------------ as it is used --
def test_prompt_chunk_and_decoding_together(dev):
    """Prompts into the cache, a chunk over what it holds, then decoded tokens: q from the
    rotary layer, keys on the way into the cache, attention over pages or read-back rows."""
    g = _gen(dev, 20)
    H, G, d, ps, n = 2, 4, 128, 64, 3
    plan = mapflow.RotaryPlan(d, base=1e6)
    gk, gv = _scales(g, dev, H), _scales(g, dev, H)
    first, chunk = [200, 65, 130], [100, 1, 40]
    full = [a + b for a, b in zip(first, chunk)]
    mp = 6
    table = torch.randperm(n * mp, generator=g, device=dev).to(torch.int32).view(n, mp)
    pages = _pages(dev, n * mp, H, ps, d)
    cache = mapflow.PagedCache.fp4(pages, ps, d, k_scale=gk, v_scale=gv)
    w = (1 + 0.1 * torch.randn(d, generator=g, device=dev)).to(BF)
    seq, at = _tokens(full, dev)
    T = sum(full)
    q, k, v = _rnd(g, dev, T, H * G, d), _rnd(g, dev, T, H, d), _rnd(g, dev, T, H, d)
    late = torch.cat([torch.arange(x) >= a for a, x in zip(first, full)]).to(dev)
    for part in (~late, late):  # the prompts, then a chunk of each
        cache.append(k[part], v[part], seq[part], at[part], table, rope=plan, k_weight=w)
    qr, _ = plan.apply(q, None, at, q_weight=w)
    y, _ = _rotated(k, w, True, at, plan, "half", d, base=1e6)
    code, s = ref.hold(y, gk)
    kh = ref.stands_for(code, s, gk)
    code, s = ref.hold(v.double(), gv)
    vh = ref.stands_for(code, s, gv)
    # the chunk over the cached prompt
    cu = [0]
    for x in full:
        cu.append(cu[-1] + x)
    kr, vr = cache.read(seq, at, table)
    o = mapflow.WindowAttention(cu, H * G, H, d, q_begin=first).attend(qr, kr, vr)
    for r, (a, x) in enumerate(zip(first, full)):
        rows = slice(cu[r] + a, cu[r + 1])
        i, j = torch.arange(a, x, device=dev), torch.arange(x, device=dev)
        keys = slice(cu[r], cu[r + 1])
        wo, _, bo, _ = layer_ref.attend(qr[rows], kr[keys], vr[keys], layer_ref.seen_packed(i, j, 0, 0), d ** -0.5)
        assert ((o[rows].double() - wo).abs() <= bo).all()
    # the last token of each by decoding over the pages: the same rows but for the rounding of read-back rows
    last = torch.tensor([c - 1 for c in cu[1:]], device=dev)
    lens = torch.tensor(full, dtype=torch.int32, device=dev)
    lse = torch.empty(n, 1, H * G, dtype=torch.float32, device=dev)
    dec = cache.attend(qr[last][:, None], table, lens, lse=lse)
    _check_attend(dev, qr[last][:, None], full, lambda r: (kh[cu[r]:cu[r + 1]], vh[cu[r]:cu[r + 1]]), dec, lse, 0, 0,
                  d ** -0.5, None, None)
    # read-back rows have 2^-8 of each key and value: scores off by 2^-8 sum|q k| / sqrt(d) < 0.25, so o by far less than o itself
    assert (dec[:, 0].double() - o[last].double()).norm() < 0.05 * o[last].double().norm()


def test_bf16_rows_are_the_caches_of_cache_attention(dev):
    g = _gen(dev, 21)
    n, cap, H, G, d = 4, 90, 2, 3, 64
    plan = mapflow.RotaryPlan(32)
    kp, vp = torch.zeros(n, cap, H, d, dtype=BF, device=dev), torch.zeros(n, cap, H, d, dtype=BF, device=dev)
    cache = mapflow.PagedCache.bf16(kp, vp)
    own = torch.arange(n, dtype=torch.int32, device=dev)[:, None]
    lens = [50, 1, 89, 17]
    seq, at = _tokens(lens, dev)
    k, v = _rnd(g, dev, sum(lens), H, d), _rnd(g, dev, sum(lens), H, d)
    cache.append(k, v, seq, at, own, rope=plan)
    # a decoded token of each
    k1, v1, q1 = _rnd(g, dev, n, H, d), _rnd(g, dev, n, H, d), _rnd(g, dev, n, 1, H * G, d)
    step = torch.tensor(lens, dtype=torch.int32, device=dev)
    cache.append(k1, v1, own[:, 0].contiguous(), step, own, rope=plan)
    o = mapflow.CacheAttention(n, 1, cap, H * G, H, d).attend(q1, kp, vp, step + 1)
    for r, x in enumerate(lens):
        kk, vv = kp[r, : x + 1], vp[r, : x + 1]
        wo, _, bo, _ = layer_ref.attend(q1[r], kk, vv, torch.ones(1, x + 1, dtype=torch.bool, device=dev), d ** -0.5)
        assert ((o[r].double() - wo).abs() <= bo).all()
        assert torch.equal(vv[-1], v1[r])


def test_a_captured_step_follows_lengths_and_pages(dev):
    g, mp = _gen(dev, 22), 20
    big = torch.zeros(3 * mp, 2, 18 * 128, dtype=torch.uint8, device=dev)
    cache = mapflow.PagedCache.fp4(big, 16, 128)
    plan = mapflow.RotaryPlan(128)
    ids = torch.arange(3 * mp, dtype=torch.int32, device=dev).view(3, mp)
    seq = torch.arange(3, dtype=torch.int32, device=dev)
    k, v, q = _rnd(g, dev, 3, 2, 128), _rnd(g, dev, 3, 2, 128), _rnd(g, dev, 3, 1, 8, 128)
    at, lens = torch.zeros(3, dtype=torch.int32, device=dev), torch.zeros(3, dtype=torch.int32, device=dev)
    o1, o2 = torch.empty_like(q), torch.empty_like(q)

    def step(o):
        cache.append(k, v, seq, at, ids, rope=plan)
        cache.attend(q, ids, lens, o=o)
    step(o1)  # (warm: the kernels' attributes are set before a capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(o1)
    twin = torch.zeros_like(big)
    other = mapflow.PagedCache.fp4(twin, 16, 128)
    perm = torch.randperm(3 * mp, generator=g, device=dev).to(torch.int32).view(3, mp)
    for x in range(100):
        k.copy_(_rnd(g, dev, 3, 2, 128))
        v.copy_(_rnd(g, dev, 3, 2, 128))
        q.copy_(_rnd(g, dev, 3, 1, 8, 128))
        at.fill_(x)
        lens.fill_(x + 1)
        if x == 50:  # from here on another sequence's pages
            ids.copy_(ids.flip(0))
            perm = perm.flip(0).contiguous()
        graph.replay()
        other.append(k, v, seq, at, perm, rope=plan)
        other.attend(q, perm, lens, o=o2)
        assert torch.equal(o1, o2), x
    assert torch.isfinite(o1).all() and o1.any()


def test_streams_and_calls_at_once(dev):
    lens = [900, 20, 3000]
    g, pages, table, lens_t, gk, gv, keys = _world(dev, 23, 3, 2, 128, 64, lens)
    cache = mapflow.PagedCache.fp4(pages, 64, 128, k_scale=gk, v_scale=gv)
    qs = [_rnd(g, dev, 3, 1, 8, 128) for _ in range(6)]
    want = [cache.attend(q, table, lens_t) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [torch.empty_like(q) for q in qs]
    for rep in range(5):
        for i, q in enumerate(qs):
            cache.attend(q, table, lens_t, o=got[i], stream=streams[i % 3])
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
            a.zero_()
    seq, at = _tokens(lens, dev)
    a = cache.read(seq, at, table)
    torch.cuda.synchronize()
    b = cache.read(seq, at, table, stream=streams[0])
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_bindings_refuse(dev):
    g, pages, table, lens_t, gk, gv, keys = _world(dev, 24, 2, 2, 64, 16, [20, 30])
    cache = mapflow.PagedCache.fp4(pages, 16, 64, k_scale=gk, v_scale=gv)
    q = _rnd(g, dev, 2, 1, 4, 64)
    x = _rnd(g, dev, 2, 2, 64)
    seq = torch.zeros(2, dtype=torch.int32, device=dev)
    bad = [lambda: cache.attend(q.float(), table, lens_t), lambda: cache.attend(q[:1], table, lens_t),
           lambda: cache.attend(q, table.long(), lens_t), lambda: cache.attend(q, table[:1], lens_t),
           lambda: cache.attend(q, table, lens_t.long()), lambda: cache.attend(q, table.cpu(), lens_t),
           lambda: cache.attend(q, table, lens_t, window=0), lambda: cache.attend(q, table, lens_t, sinks=-1),
           lambda: cache.attend(q, table, lens_t, softcap=0.0), lambda: cache.attend(q, table, lens_t, softcap=float("nan")),
           lambda: cache.attend(q, table, lens_t, slopes=torch.ones(2, device=dev)), lambda: cache.attend(q, table, lens_t, o=q),
           lambda: cache.attend(q, table, lens_t, scale=0.0), lambda: cache.attend(q[:, 0], table, lens_t),
           lambda: cache.attend(q.expand(2, 1, 4, 64)[..., ::2], table, lens_t),
           lambda: cache.attend(_rnd(g, dev, 2, 65, 4, 64), table, lens_t),
           lambda: cache.append(x, x.float(), seq, seq, table), lambda: cache.append(x, x, seq.long(), seq, table),
           lambda: cache.append(x, x, seq, seq[:1], table), lambda: cache.append(x, x, seq, seq, table.t()),
           lambda: cache.append(x, x, seq, seq, table, positions=seq),
           lambda: cache.append(x, x, seq, seq, table, rope=mapflow.RotaryPlan(128)),
           lambda: cache.append(x, x, seq, seq, table, k_weight=torch.ones(64, device=dev)),
           lambda: cache.read(seq, seq, table, k=x, v=x), lambda: cache.read(seq, seq, table, k=x[:1]),
           lambda: mapflow.PagedCache.fp4(pages[:, :, :-1], 16, 64), lambda: mapflow.PagedCache.fp4(pages, 16, 64, k_scale=gk[:1]),
           lambda: mapflow.PagedCache.bf16(x[None], x[None].float()),
           lambda: mapflow.PagedCache.bf16(x[None], x[None].clone()).attend(q, table, lens_t)]
    for i, call in enumerate(bad):
        with pytest.raises((mapflow.MapFlowError, TypeError)):
            call()
            pytest.fail(f"call {i} was taken")
    torch.cuda.synchronize()


@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_begin_between_32_bytes(dev, d):
    """Rows at odd multiples of 16 bytes give what rows at even ones give."""
    g, H, ps, T = _gen(dev, 25 + d), 3, 16, 75
    width = H * d + 8

    def odd(T, heads):
        return torch.zeros(T, heads * d + 8, dtype=BF, device=dev)[:, 8:].view(T, heads, d)

    assert odd(2, H).data_ptr() % 32 == 16 and odd(2, H).stride(0) == width
    k, v, q = _rnd(g, dev, T, H, d), _rnd(g, dev, T, H, d), _rnd(g, dev, 5, 1, 2 * H, d)
    ko, vo, qo = odd(T, H), odd(T, H), odd(5, 2 * H)
    ko.copy_(k), vo.copy_(v), qo.copy_(q[:, 0])
    seq, at = _tokens([20, 1, 16, 30, 8], dev)
    table = torch.randperm(10, generator=g, device=dev).to(torch.int32).view(5, 2)
    lens = torch.tensor([20, 1, 16, 30, 8], dtype=torch.int32, device=dev)
    for layout, rot in (("half", d), ("interleaved", 32), ("half", 20)):
        plan = mapflow.RotaryPlan(rot, layout=layout)
        held = []
        for kk, vv in ((k, v), (ko, vo), (k, vo)):
            pages = torch.zeros(10, H, 18 * d, dtype=torch.uint8, device=dev)
            mapflow.PagedCache.fp4(pages, ps, d).append(kk, vv, seq, at, table, rope=plan, norm=True)
            held.append(pages)
        assert torch.equal(held[0], held[1]) and torch.equal(held[0], held[2])
        cache = mapflow.PagedCache.fp4(held[0], ps, d)
        want, got = cache.read(seq, at, table), cache.read(seq, at, table, k=odd(T, H), v=odd(T, H))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        o = odd(5, 2 * H)[:, None]
        assert torch.equal(cache.attend(qo[:, None], table, lens, o=o), cache.attend(q, table, lens))
        rows = []
        for kk, vv, make in ((k, v, None), (ko, vo, None), (k, v, odd)):
            if make is None:
                ck, cv = (torch.zeros(10, ps, H, d, dtype=BF, device=dev) for _ in range(2))
            else:
                ck, cv = (make(10 * ps, H).unflatten(0, (10, ps)) for _ in range(2))
            c = mapflow.PagedCache.bf16(ck, cv)
            c.append(kk, vv, seq, at, table, rope=plan, norm=True)
            rows.append((ck, cv, *c.read(seq, at, table), *c.read(seq, at, table, k=odd(T, H), v=odd(T, H))))
        for other in rows[1:]:
            assert all(torch.equal(a, b) for a, b in zip(rows[0], other))
        assert torch.equal(rows[0][2], rows[0][4]) and torch.equal(rows[0][3], v) and torch.equal(rows[0][5], v)


def test_pages_that_requests_share(dev):
    lens = [900, 900, 900]
    g, pages, table, lens_t, gk, gv, keys = _world(dev, 30, 3, 2, 128, 64, lens)
    cache = mapflow.PagedCache.fp4(pages, 64, 128, k_scale=gk, v_scale=gv)
    q = _rnd(g, dev, 3, 1, 8, 128)
    table[1:, :9] = table[0, :9]  # one prompt's pages in all three
    table[2, 11] = table[2, 10]   # and one page twice in a request
    copies = pages[table.long().flatten()].contiguous()
    own = torch.arange(table.numel(), dtype=torch.int32, device=dev).view_as(table)
    o = cache.attend(q, table, lens_t)
    assert torch.equal(o, mapflow.PagedCache.fp4(copies, 64, 128, k_scale=gk, v_scale=gv).attend(q, own, lens_t))
    assert torch.equal(o[:, 0, 0].isfinite(), torch.ones_like(o[:, 0, 0], dtype=torch.bool))


def test_two_graphs_replayed_at_once(dev):
    lens = [5000, 20, 3000]
    g, pages, table, lens_t, gk, gv, keys = _world(dev, 31, 3, 2, 128, 64, lens)
    cache = mapflow.PagedCache.fp4(pages, 64, 128, k_scale=gk, v_scale=gv)
    qs = [_rnd(g, dev, 3, 1, 8, 128) for _ in range(2)]
    want = [cache.attend(q, table, lens_t) for q in qs]
    got = [torch.zeros_like(q) for q in qs]
    torch.cuda.synchronize()
    graphs = []
    for q, o in zip(qs, got):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(4):
                cache.attend(q, table, lens_t, o=o)
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for o in got:
            o.zero_()
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("captured", [False, True])
def test_steps_in_a_row_follow_each_other(dev, captured):
    """A step's attention sees what the append before it wrote, and no step's
    append overtakes the attention or the reading before it."""
    g, H, d, n, steps = _gen(dev, 32), 8, 128, 40, 24
    k, v = _rnd(g, dev, steps, n, H, d), _rnd(g, dev, steps, n, H, d)
    q = _rnd(g, dev, n, 1, 4 * H, d)
    table = torch.arange(2 * n, dtype=torch.int32, device=dev).view(n, 2)
    seq = torch.arange(n, dtype=torch.int32, device=dev)
    at = [torch.full((n,), x % 18, dtype=torch.int32, device=dev) for x in range(steps)]  # the last ones over the first
    lens = [torch.full((n,), min(x + 1, 18), dtype=torch.int32, device=dev) for x in range(steps)]
    pages = torch.zeros(2 * n, H, 18 * d, dtype=torch.uint8, device=dev)
    cache = mapflow.PagedCache.fp4(pages, 16, d)
    plan = mapflow.RotaryPlan(d)
    o = [torch.zeros_like(q) for _ in range(steps)]
    rows = [(torch.zeros_like(k[0]), torch.zeros_like(k[0])) for _ in range(steps)]

    def run(wait):
        for x in range(steps):
            cache.append(k[x], v[x], seq, at[x], table, rope=plan, norm=True)
            wait()
            cache.attend(q, table, lens[x], o=o[x])
            wait()
            cache.read(seq, at[x], table, *rows[x])
            wait()

    run(torch.cuda.synchronize)
    want = [t.clone() for t in o + [a for r in rows for a in r] + [pages]]
    graph = None
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(lambda: None)
    for _ in range(5):
        for t in o + [a for r in rows for a in r] + [pages]:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay() if captured else run(lambda: None)
        torch.cuda.synchronize()
        for a, b in zip(o + [a for r in rows for a in r] + [pages], want):
            assert torch.equal(a, b)


def test_threads_on_one_stream(dev):
    """Calls of several threads on the default stream, which share its workspace."""
    lens = [5000, 20, 3000]
    g, pages, table, lens_t, gk, gv, keys = _world(dev, 33, 3, 2, 128, 64, lens)
    cache = mapflow.PagedCache.fp4(pages, 64, 128, k_scale=gk, v_scale=gv)
    qs = [_rnd(g, dev, 3, lq, 8, 128) for lq in (1, 1, 2, 8)]
    want = [cache.attend(q, table, lens_t) for q in qs]
    got = [[torch.zeros_like(q) for _ in range(100)] for q in qs]
    torch.cuda.synchronize()

    def work(q, out):
        for o in out:
            cache.attend(q, table, lens_t, o=o)

    threads = [threading.Thread(target=work, args=a) for a in zip(qs, got)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(o, b) for o in a)


def test_reading_into_given_and_new_tensors(dev):
    g, pages, table, lens_t, gk, gv, keys = _world(dev, 34, 2, 3, 64, 16, [20, 33])
    cache = mapflow.PagedCache.fp4(pages, 16, 64, k_scale=gk, v_scale=gv)
    seq, at = _tokens([20, 33], dev)
    seq[4] = -1
    k, v = cache.read(seq, at, table)
    assert k.is_contiguous() and v.is_contiguous() and (k[4] == 0).all() and (v[4] == 0).all() and k[5].any()
    for given in ({"k"}, {"v"}, {"k", "v"}):
        own = {name: torch.full_like(k, 7.0) for name in given}
        got = cache.read(seq, at, table, **own)
        for name, a, b in zip("kv", got, (k, v)):
            assert name not in own or a is own[name]
            assert (a[4] == (7 if name in own else 0)).all()
            assert torch.equal(a[:4], b[:4]) and torch.equal(a[5:], b[5:])
    empty = cache.read(seq[:0], at[:0], table)
    assert empty[0].shape == empty[1].shape == (0, 3, 64)


@pytest.mark.parametrize("layout,rot", [("half", 64), ("interleaved", 64), ("half", 20)])
def test_append_of_more_heads_than_32_at_once(dev, layout, rot):
    """A prompt long enough for a group of lanes to take all 40 heads of a token."""
    g, H, d, ps, T = _gen(dev, 35 + rot), 40, 64, 64, 5000
    k, v = _rnd(g, dev, T, H, d), _rnd(g, dev, T, H, d)
    seq, at = _tokens([T], dev)
    table = torch.randperm((T + ps - 1) // ps, generator=g, device=dev).to(torch.int32)[None]
    gk, gv = _scales(g, dev, H), _scales(g, dev, H)
    pages = _pages(dev, table.shape[1], H, ps, d)
    cache = mapflow.PagedCache.fp4(pages, ps, d, k_scale=gk, v_scale=gv)
    cache.append(k, v, seq, at, table, rope=mapflow.RotaryPlan(rot, layout=layout), norm=True)
    y, _ = _rotated(k, None, True, at, True, layout, rot)
    _check_held(pages, ps, d, *_slots(seq, at, table, ps), y, v, gk, gv)


@pytest.mark.parametrize("d,lq", [(128, 1), (64, 3), (128, 3)])
def test_biases_that_rise_either_way(dev, d, lq):
    """Slopes of both signs: the heaviest key is the newest or the oldest, and the reference moves along."""
    lens = [1500, 64, 333]
    g, pages, table, lens_t, gk, gv, keys = _world(dev, 36 + d + lq, 3, 2, d, 32, lens)
    cache = mapflow.PagedCache.fp4(pages, 32, d, k_scale=gk, v_scale=gv)
    q = _rnd(g, dev, 3, lq, 8, d, std=1.5)
    slopes = torch.tensor([0.5, -0.5, 3.0, -3.0, 0.01, -0.01, 0.0, 40.0], device=dev)
    lse = torch.empty(3, lq, 8, dtype=torch.float32, device=dev)
    for cap in (None, 30.0, 1e5):
        o = cache.attend(q, table, lens_t, softcap=cap, slopes=slopes, lse=lse)
        _check_attend(dev, q, lens, keys, o, lse, 0, 0, d ** -0.5, cap, slopes)
    o = cache.attend(q, table, lens_t, window=100, sinks=40, slopes=slopes, lse=lse)
    _check_attend(dev, q, lens, keys, o, lse, 100, 40, d ** -0.5, None, slopes)


@pytest.mark.parametrize("d", [64, 128])
def test_quotients_beside_a_border(dev, d):
    """Head scales that put a block's scale, or a value's code, within fp32's rounding of the
    border between two: the exact quotient decides (a tie only where it lies on it)."""
    H, T, ps = 256, 48, 16
    rng = torch.Generator().manual_seed(40 + d)
    draw = lambda *shape: torch.rand(*shape, generator=rng, dtype=torch.float64)  # noqa: E731
    x = (draw(T, H, d) * 2 - 1) * 0.5
    g = torch.empty(H, dtype=torch.float64)
    codes = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
    for h in range(H):
        top = float((0.5 + draw(1) * 8).to(BF).double())
        if h % 2 == 0:    # top / (6 g) beside the middle of two scales
            m = float(torch.ldexp(17.0 + 2 * torch.floor(draw(1) * 8), torch.floor(draw(1) * 9) - 7))
            g[h] = (torch.tensor(top / (6 * m), dtype=torch.float64)).float().double()
            x[:, h] *= top / 8
            x[:, h, ::16] = top
        else:             # a value over s g beside the middle of two codes
            s = float(torch.ldexp(8.0 + torch.floor(draw(1) * 8), torch.floor(draw(1) * 9) - 6))
            c = codes[int(draw(1) * 7)].item()
            g[h] = torch.tensor(top / (s * c), dtype=torch.float64).float().double()
            x[:, h] *= 4 * s * g[h]
            x[:, h, ::16] = 6 * s * g[h]
            x[:, h, 5::16] = top
            x[:, h, 9::16] = -top
    x, gs = x.to(BF).to(dev), g.float().to(dev)
    pages = _pages(dev, T // ps, H, ps, d)
    cache = mapflow.PagedCache.fp4(pages, ps, d, k_scale=gs, v_scale=gs)
    seq, at = _tokens([T], dev)
    table = torch.arange(T // ps, dtype=torch.int32, device=dev)[None]
    cache.append(x, x, seq, at, table)
    page, o = _slots(seq, at, table, ps)
    _check_held(pages, ps, d, page, o, x.double(), x, gs, gs)
    # rotated and normed dimensions beside such ones, in the same rows
    plan = mapflow.RotaryPlan(32)
    cache.append(x, x, seq, at, table, rope=plan)
    y, _ = _rotated(x, None, False, at, plan, "half", 32)
    _check_held(pages, ps, d, page, o, y, x, gs, gs)


@pytest.mark.parametrize("layout,rot", [("half", 128), ("half", 64), ("interleaved", 128), ("half", 20), ("interleaved", 6)])
def test_position_zero_turns_nothing(dev, layout, rot):
    g = _gen(dev, 50 + rot)
    T, H, d, ps = 333, 3, 128, 16
    k = (torch.randint(-24, 25, (T, H, d), generator=g, device=dev) / 4).to(BF)
    v = _rnd(g, dev, T, H, d)
    seq, at = _tokens([T], dev)
    table = torch.arange((T + ps - 1) // ps, dtype=torch.int32, device=dev)[None]
    page, o = _slots(seq, at, table, ps)
    zero = torch.zeros(T, dtype=torch.int32, device=dev)
    some = torch.where(at % 3 == 0, zero, at)
    for gs in (None, torch.tensor([0.5, 1.1, 3.0], device=dev)):
        for pos in (zero, some):
            pages = _pages(dev, table.shape[1], H, ps, d)
            cache = mapflow.PagedCache.fp4(pages, ps, d, k_scale=gs, v_scale=gs)
            cache.append(k, v, seq, at, table, rope=mapflow.RotaryPlan(rot, layout=layout), positions=pos)
            y, _ = _rotated(k, None, False, pos, True, layout, rot)
            _check_held(pages, ps, d, page, o, y, v, gs, gs)
            if pos is zero:
                assert torch.equal(y, k.double())
