"""Appending to a paged cache at the ends of its inputs' ranges: what is not
finite, gains below zero, small eps, head scales of any size."""
import math

import pytest
import torch

from cross_model_attention_gb300 import mapflow
from tests import layer_ref
from tests import paged_ref as ref
from tests.test_gpu_paged_cache import BF, _check_attend, _check_held, _gen, _pages, _rnd, _slots, _tokens, _world

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "a GPU is needed"
    return torch.device("cuda", torch.cuda.current_device())


def _rows(dev, k, at, ps=16, **kw):
    """k [T, H, d] as a bf16 cache holds them, at the places `at` of one sequence."""
    T, H, d = k.shape
    n = (T + ps - 1) // ps
    kp, vp = (torch.full((n, ps, H, d), 5.0, dtype=BF, device=dev) for _ in range(2))
    cache = mapflow.PagedCache.bf16(kp, vp)
    table = torch.arange(n, dtype=torch.int32, device=dev)[None]
    cache.append(k, k.clone(), torch.zeros_like(at), at, table, **kw)
    return kp.view(-1, H, d)[:T]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout,rot", [(None, 0), ("half", 32), ("half", 20), ("interleaved", 32), ("interleaved", 6)])
@pytest.mark.parametrize("norm", [False, True])
def test_bf16_dimensions_that_are_not_turned(dev, d, layout, rot, norm):
    g, T, H = _gen(dev, 60 + d + rot), 19, 3
    k = _rnd(g, dev, T, H, d)
    k[1, 0, 40] = math.inf       # dimensions past every rotated part, at either end of a pair of
    k[2, 1, 41] = -math.inf      # neighbours, of chunks of 8 and of halves
    k[3, 2, 48] = math.nan
    k[4, 0, 63] = math.inf
    k[5, 1, d - 1] = math.inf
    k[6, :, rot:] = -0.0
    _, at = _tokens([T], dev)
    w = (1 + 0.1 * torch.randn(d, generator=g, device=dev)).to(BF) if norm else None
    plan = mapflow.RotaryPlan(rot, layout=layout) if layout else None
    got = _rows(dev, k, at, rope=plan, norm=norm, k_weight=w)[..., rot:]
    if not norm:
        want = k[..., rot:]
        assert torch.equal(got.isnan(), want.isnan())
        bits = lambda x: x.nan_to_num(7.0, math.inf, -math.inf).contiguous().view(torch.int16)  # noqa: E731
        assert torch.equal(bits(got), bits(want))
        return
    # a row's infinity leaves 0 beside itself, its NaN nothing
    y = k.double() * (k.double().square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w.double()
    want = y[..., rot:]
    assert torch.equal(got.isnan(), want.isnan())
    assert ((got.double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -17))[~want.isnan()].all()
    assert torch.equal(got[6].signbit(), torch.ones_like(got[6], dtype=torch.bool))


@pytest.mark.parametrize("layout,rot", [(None, 0), ("half", 128), ("half", 20), ("interleaved", 128)])
def test_bf16_rows_whose_squares_pass_the_range(dev, layout, rot):
    """Squares past fp32's range make a row 0, as in the rotary layer, whatever the weights."""
    g, T, H, d = _gen(dev, 61), 9, 2, 128
    k = _rnd(g, dev, T, H, d)
    k[2:6] = torch.where(k[2:6] > 0, 3e38, -3e38).to(BF)
    w = torch.full((d,), 4.0, dtype=BF, device=dev)
    _, at = _tokens([T], dev)
    plan = mapflow.RotaryPlan(rot, layout=layout) if layout else None
    got = _rows(dev, k, at, rope=plan, norm=True, k_weight=w)
    assert (got[2:6] == 0).all() and torch.isfinite(got).all() and (got[:2] != 0).any()
    if plan is not None:
        _, want = plan.apply(k.clone(), k, at, norm=True, q_weight=w, k_weight=w)
        assert (want[2:6] == 0).all()


@pytest.mark.parametrize("gain", [-1000.0, -1.5, -0.25, 64.0])
@pytest.mark.parametrize("layout,rot", [("half", 120), ("half", 128), ("interleaved", 128)])
def test_gains_of_either_sign(dev, gain, layout, rot):
    g, T, H, d, ps = _gen(dev, 62), 16384, 8, 128, 64
    k, v = _rnd(g, dev, T, H, d, std=0.05), _rnd(g, dev, T, H, d)
    seq, at = _tokens([T], dev)
    table = torch.arange(T // ps, dtype=torch.int32, device=dev)[None]
    pages = _pages(dev, T // ps, H, ps, d)
    plan = mapflow.RotaryPlan(rot, layout=layout)
    plan.gain = gain
    mapflow.PagedCache.fp4(pages, ps, d).append(k, v, seq, at, table, rope=plan)
    f, _ = layer_ref.rope_frequencies(rot)
    y, _ = layer_ref.rope(k, None, False, 0.0, at, f, gain, rot, layout)
    _check_held(pages, ps, d, *_slots(seq, at, table, ps), y, v, None, None)


@pytest.mark.parametrize("eps", [1e-40, 1e-36, 1e-25])
@pytest.mark.parametrize("layout,rot", [(None, 0), ("half", 128), ("half", 20), ("interleaved", 64)])
def test_small_eps(dev, eps, layout, rot):
    """Rows of zeros stay zeros and rows of tiny values are normed, down to an eps below fp32's normal numbers."""
    g, T, H, d, ps = _gen(dev, 63), 64, 3, 128, 16
    k, v = _rnd(g, dev, T, H, d), _rnd(g, dev, T, H, d)
    eps = float(torch.tensor(eps, dtype=torch.float32))
    k[5:9] = 0
    k[9:30] = (k[9:30].float() * 3 * eps ** 0.5).to(BF)     # squares about eps
    k[30:40] = (k[30:40].float() * 0.01 * eps ** 0.5).to(BF)
    seq, at = _tokens([T], dev)
    plan = mapflow.RotaryPlan(rot, layout=layout) if layout else None
    if plan is None:
        y = k.double() * (k.double().square().mean(-1, keepdim=True) + eps).rsqrt()
    else:
        f, gain = layer_ref.rope_frequencies(rot)
        y, _ = layer_ref.rope(k, None, True, eps, at, f, gain, rot, layout)
    table = torch.arange(T // ps, dtype=torch.int32, device=dev)[None]
    pages = _pages(dev, T // ps, H, ps, d)
    mapflow.PagedCache.fp4(pages, ps, d).append(k, v, seq, at, table, rope=plan, norm=True, eps=eps)
    _check_held(pages, ps, d, *_slots(seq, at, table, ps), y, v, None, None)
    got = _rows(dev, k, at, rope=plan, norm=True, eps=eps)
    assert (got[5:9] == 0).all() and torch.isfinite(got).all()
    # (a square is off by 2^-150 at most, which is 2^-17 of 1e-40)
    assert ((got.double() - y).abs() <= y.abs() * 2.0 ** -8 + 2.0 ** -15 * y.abs().amax(-1, keepdim=True)).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout,rot", [(None, 0), ("half", 64), ("half", 20), ("interleaved", 32)])
def test_head_scales_at_the_ends_of_their_range(dev, d, layout, rot):
    g, T, ps = _gen(dev, 64 + d), 80, 16
    lo, hi = 2.0 ** -64, 2.0 ** 64
    gk = torch.tensor([lo, 1.37 * lo, hi, hi / 1.37, 1.0, lo, hi], device=dev)
    size = torch.tensor([lo, lo, hi, hi, 1.0, 1e37, 1e-37], dtype=torch.float64, device=dev)  # of a head's values
    H = len(gk)
    k, v = ((torch.randn(T, H, d, generator=g, device=dev, dtype=torch.float64) * size[:, None]).to(BF) for _ in range(2))
    # scales of a block from 2^-9 to 448, zeros among them
    mult = 2.0 ** torch.randint(-9, 9, (T, 1, d // 16, 1), generator=g, device=dev).float()
    few = torch.arange(H, device=dev)[:, None] < 5
    k, v = (torch.where(few, (x.float().unflatten(-1, (-1, 16)) * mult).flatten(-2).to(BF), x) for x in (k, v))
    k[7], v[8] = 0, 0
    seq, at = _tokens([T], dev)
    table = torch.arange(T // ps, dtype=torch.int32, device=dev)[None]
    plan = mapflow.RotaryPlan(rot, layout=layout) if layout else None
    y = k.double()
    if plan is not None:
        f, gain = layer_ref.rope_frequencies(rot)
        y, _ = layer_ref.rope(k, None, False, 0.0, at, f, gain, rot, layout)
    pages = _pages(dev, T // ps, H, ps, d)
    cache = mapflow.PagedCache.fp4(pages, ps, d, k_scale=gk, v_scale=gk)
    cache.append(k, v, seq, at, table, rope=plan)
    page, o = _slots(seq, at, table, ps)
    kc, ks, vc, vs = (x[page, o].long() for x in ref.unpack(pages, ps, d))
    for code, scale, x, gs in ((kc, ks, y, gk), (vc, vs, v.double(), gk)):
        want_c, want_s = ref.hold(x, gs)
        assert torch.equal(scale, want_s)
        assert ((code == want_c) | ((code & 7 == 0) & (want_c & 7 == 0))).all()
    vo = cache.read(seq, at, table)[1]
    want = ref.stands_for(vc, vs, gk)
    assert torch.allclose(vo.double(), want, rtol=2.0 ** -8 + 2.0 ** -23, atol=0)


def test_head_scales_out_of_their_range_hold_nan(dev):
    g, T, d, ps = _gen(dev, 65), 33, 128, 16
    bad = [0.0, -1.0, 2.0 ** -64 * 0.999, 1e-37, 1e-42, 2.0 ** 64 * 1.001, 1e38, math.inf, -math.inf, math.nan]
    gk = torch.tensor([1.0] + bad + [2.0 ** 64], device=dev)
    H = len(gk)
    k, v = _rnd(g, dev, T, H, d), _rnd(g, dev, T, H, d)
    k[3], v[4] = 0, 0
    k[5], v[6] = 1e30, 1e30
    seq, at = _tokens([T], dev)
    table = torch.arange(3, dtype=torch.int32, device=dev)[None]
    for plan, norm in ((None, False), (mapflow.RotaryPlan(d), True), (mapflow.RotaryPlan(20), False),
                       (mapflow.RotaryPlan(32, layout="interleaved"), True)):
        pages = _pages(dev, 3, H, ps, d, byte=0)
        cache = mapflow.PagedCache.fp4(pages, ps, d, k_scale=gk, v_scale=gk)
        cache.append(k, v, seq, at, table, rope=plan, norm=norm)
        page, o = _slots(seq, at, table, ps)
        _, ks, _, vs = (x[page, o].long() for x in ref.unpack(pages, ps, d))
        for s in (ks, vs):
            assert (s[:, 1:-1] == 0x7f).all() and (s[:, 0] != 0x7f).all() and (s[:, -1] != 0x7f).all()
        for x in cache.read(seq, at, table):
            assert x[:, 1:-1].isnan().all() and torch.isfinite(x[:, 0]).all() and torch.isfinite(x[:, -1]).all()


@pytest.mark.parametrize("d,lq", [(128, 1), (64, 3)])
@pytest.mark.parametrize("e", [-64, 64])
def test_attention_under_head_scales_at_the_ends(dev, d, lq, e):
    lens = [700, 33, 5000]
    g, pages, table, lens_t, gk, gv, keys = _world(dev, 66 + d, 3, 2, d, 32, lens, scales=False)
    one = torch.ones(2, device=dev)
    cache = mapflow.PagedCache.fp4(pages, 32, d, k_scale=one * 2.0 ** e, v_scale=one * 2.0 ** -e)
    q = _rnd(g, dev, 3, lq, 8, d, std=1.5)
    lse = torch.empty(3, lq, 8, dtype=torch.float32, device=dev)
    scale = d ** -0.5 * 2.0 ** -e
    o = cache.attend(q, table, lens_t, scale=scale, lse=lse)
    plain = mapflow.PagedCache.fp4(pages, 32, d).attend(q, table, lens_t)
    assert torch.equal(o.double(), plain.double() * 2.0 ** -e)

    def far(r):
        k, v = keys(r)
        return k * 2.0 ** e, v
    _check_attend(dev, q, lens, far, (o.double() * 2.0 ** e), lse, 0, 0, scale, None, None)


@pytest.mark.parametrize("size,gain,still", [(2.0 ** 45, 1.0, False), (2.0 ** 60, -0.3, False), (1.0, 1.5, True)])
@pytest.mark.parametrize("layout,rot", [("half", 128), ("half", 20), ("interleaved", 128), ("half", 64)])
def test_signs_of_values_that_are_small_beside_others(dev, layout, rot, size, gain, still):
    """A value within the error of its block's largest, or of its pair's other block's, but past a
    code of its own block: its sign counts."""
    g, T, H, d, ps = _gen(dev, 67), 4096, 8, 128, 16
    k, v = _rnd(g, dev, T, H, d, std=size), _rnd(g, dev, T, H, d)
    seq, at = _tokens([T], dev)
    pos = at
    if still:  # (nothing is turned, the products with the gain round: blocks of very different sizes side by side)
        pos = torch.zeros_like(at)
        wide = 2.0 ** torch.randint(0, 23, (T, 1, d // 16, 1), generator=g, device=dev).float()
        k = (k.float().unflatten(-1, (-1, 16)) * wide).flatten(-2).to(BF)
    table = torch.arange(T // ps, dtype=torch.int32, device=dev)[None]
    pages = _pages(dev, T // ps, H, ps, d)
    plan = mapflow.RotaryPlan(rot, layout=layout)
    plan.gain = gain
    mapflow.PagedCache.fp4(pages, ps, d).append(k, v, seq, at, table, rope=plan, positions=pos)
    f, _ = layer_ref.rope_frequencies(rot)
    y, _ = layer_ref.rope(k, None, False, 0.0, pos, f, float(torch.tensor(gain)), rot, layout)
    _check_held(pages, ps, d, *_slots(seq, at, table, ps), y, v, None, None)
