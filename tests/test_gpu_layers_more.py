"""More GPU tests of the rotary embedding and of window, cache and prefix
attention: values that are not finite, lost blocks, many empty slots."""
import math

import numpy as np
import pytest
import torch

from cross_model_attention_gb300 import mapflow
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU test selected on a machine without a GPU"


def rnd(seed, *shape, dt=BF, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)


# ------------------------------------------------ values that are not finite --
def reach_is(got, want, sees, may):
    """Rows that see the value are not finite, rows that it may not reach are as without it."""
    assert not torch.isfinite(got[sees]).all(-1).any()
    assert torch.equal(got[~may], want[~may])
    assert (sees & ~may).sum() == 0


@pytest.mark.parametrize("L,begin,H_q,H_kv,d,window,sinks,at,bad", [
    (700, 0, 2, 2, 64, None, 0, 300, math.nan),
    (700, 0, 2, 2, 128, 16, 0, 300, math.nan),     # later rows of the pair no longer see it
    (700, 0, 2, 2, 128, 16, 0, 505, math.inf),     # seen from two pairs
    (700, 0, 8, 2, 128, 40, 3, 250, -math.inf),    # 32 tokens to a tile
    (700, 0, 8, 2, 64, 40, 3, 1, math.nan),        # a sink: every later row sees it
    (900, 100, 6, 2, 128, 50, 0, 200, math.nan),   # pairs begin at the chunk's first row
    (5000, 4900, 4, 2, 128, 300, 0, 4950, math.nan),  # partial results that are joined
])
def test_reach_of_a_value_packed(L, begin, H_q, H_kv, d, window, sinks, at, bad):
    G, pair = H_q // H_kv, 2 * (128 // (H_q // H_kv))
    q, k, v = rnd(0, L, H_q, d), rnd(1, L, H_kv, d), rnd(2, L, H_kv, d)
    plan = mapflow.WindowAttention([0, L], H_q, H_kv, d, window=window, sinks=sinks, q_begin=[begin] if begin else None)
    want = plan.attend(q, k, v)[begin:]
    v2, head = v.clone(), 1
    v2[at, head, 5] = bad
    got = plan.attend(q, k, v2)[begin:]
    plan.status()
    i = torch.arange(begin, L, device="cuda")
    row = ref.seen_packed(i, torch.tensor([at], device="cuda"), window, sinks)[:, 0]
    pairs = (i - begin) // pair
    near = torch.isin(pairs, pairs[row])
    mine = torch.arange(H_q, device="cuda") // G == head
    reach_is(got, want, row[:, None] & mine, near[:, None] & mine)
    k2 = k.clone()  # a key reaches nothing but the rows that see it
    k2[at, head, 5] = bad
    got = plan.attend(q, k2, v)[begin:]
    hit = row[:, None] & mine
    assert torch.equal(got[~hit], want[~hit])


@pytest.mark.parametrize("lens,Lq,H_q,H_kv,d,window,sinks,P,at,bad", [
    ([300, 200], 2, 4, 2, 128, 16, 0, 0, 284, math.nan),   # hidden from the second new token
    ([300, 200], 4, 40, 40, 64, None, 0, 0, 299, math.inf),  # 32 of 40 heads to a tile
    ([2000, 200], 1, 32, 8, 128, None, 0, 0, 1500, math.nan),
    ([60, 3, 0], 2, 8, 2, 128, None, 0, 500, 59, math.nan),
])
def test_reach_of_a_value_cached(lens, Lq, H_q, H_kv, d, window, sinks, P, at, bad):
    n, cap, G = len(lens), max(lens), H_q // H_kv
    HG = min(H_kv, 128 // (Lq * G))
    q, k, v = rnd(0, n, Lq, H_q, d), rnd(1, n, cap, H_kv, d), rnd(2, n, cap, H_kv, d)
    pre = dict(k_prefix=rnd(3, P, H_kv, d), v_prefix=rnd(4, P, H_kv, d)) if P else {}
    plan = mapflow.CacheAttention(n, Lq, cap, H_q, H_kv, d, window=window, sinks=sinks, prefix_len=P)
    dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = plan.attend(q, k, v, dl, **pre)
    v2, head = v.clone(), H_kv - 1
    v2[0, at, head, 7] = bad
    got = plan.attend(q, k, v2, dl, **pre)
    plan.status()
    row = ref.seen_packed(torch.arange(lens[0] - Lq, lens[0], device="cuda"), torch.tensor([at], device="cuda"),
                          window, sinks)[:, 0]
    kv = torch.arange(H_q, device="cuda") // G
    sees, may = (torch.zeros(n, Lq, H_q, dtype=torch.bool, device="cuda") for _ in range(2))
    sees[0] = row[:, None] & (kv == head)
    may[0] = (kv // HG == head // HG)[None]
    reach_is(got, want, sees, may)
    k2 = k.clone()
    k2[0, at, head, 7] = bad
    assert torch.equal(plan.attend(q, k2, v, dl, **pre)[~sees], want[~sees])


# --------------------------------------------------------------- empty slots --
def slots_case(n, used, cap, H_q=2, H_kv=1, d=64, seed=0):
    """A plan of n requests of which `used` (request -> keys) have any."""
    q = rnd(seed, n, 1, H_q, d)
    k, v = rnd(seed + 1, n, cap, H_kv, d), rnd(seed + 2, n, cap, H_kv, d)
    lens = torch.zeros(n, dtype=torch.int32)
    for r, x in used.items():
        lens[r] = x
    plan = mapflow.CacheAttention(n, 1, cap, H_q, H_kv, d)
    return plan, q, k, v, lens.cuda()


@pytest.mark.parametrize("n", [8191, 8192, 8193, 16384, 65537, 70001, 131073, 300001])
def test_cache_slots_past_the_map(n):
    """The map of used slots has a bit for one, or from 8193 requests on for 8, 16, 32 or 64 of them."""
    rng = np.random.default_rng(n)
    edges = [0, 7, 8, 63, 64, 127, 128, 2047, 2048, n // 2, n - 65, n - 64, n - 9, n - 8, n - 1]
    used = {int(r): int(rng.integers(1, 9)) for r in list(rng.integers(0, n, 200)) + edges}
    plan, q, k, v, lens = slots_case(n, used, 8, seed=1)
    lse = torch.zeros(n, 1, 2, device="cuda")
    o = plan.attend(q, k, v, lens, lse=lse)
    plan.status()
    some = torch.tensor(sorted(used), device="cuda")
    none = torch.ones(n, dtype=torch.bool, device="cuda")
    none[some] = False
    assert (o[none] == 0).all() and torch.isneginf(lse[none]).all()
    # the used ones at once: rows of one sequence each, other requests' keys hidden
    mine = torch.arange(len(some), device="cuda")
    seen = (mine[:, None] == mine.repeat_interleave(8)[None]) & \
        (torch.arange(8, device="cuda").repeat(len(some))[None] < lens[some][:, None])
    want, wl, bo, bl = ref.attend(q[some, 0], k[some].flatten(0, 1), v[some].flatten(0, 1), seen, 64 ** -0.5)
    assert ((o[some, 0].double() - want).abs() <= bo).all()
    assert ((lse[some, 0].double() - wl).abs() <= bl).all()


def test_empty_slots_past_the_map_cost_little():
    """100000 slots of which the first and last 300 are used: 0.3 ms, where a
    walk over the others one by one would take more than 20 ms.  (3 ms: eight
    times what the lengths and the launch take.)"""
    n = 100000
    used = {r: 600 for r in [*range(297), *range(n - 300, n)]}
    plan, q, k, v, lens = slots_case(n, used, 600)
    o = torch.empty_like(q)
    times = []
    for _ in range(6):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        plan.attend(q, k, v, lens, o=o)
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    plan.status()
    assert min(times) < 3.0
    for r in (0, 296, n - 300, n - 1):
        want, _, bo, _ = ref.attend(q[r], k[r], v[r], torch.ones(1, 600, dtype=torch.bool, device="cuda"), 64 ** -0.5)
        assert ((o[r].double() - want).abs() <= bo).all()
    assert (o[297:n - 300] == 0).all()


# --------------------------------------------------------------- lost blocks --
def marks(m, H_kv, d):
    """Values of m keys that are 1 in a column of 16 keys' own (d such groups
    apart) and 0 elsewhere: a row's outputs are sums of its weights, so that 16
    keys (one step of the second product) that are lost, or counted twice, show
    however long the row is."""
    v = torch.zeros(m, H_kv, d, dtype=BF, device="cuda")
    j = torch.arange(m, device="cuda")
    v[j, :, j // 16 % d] = 1
    return v


def check_marks(o, q, k, v, seen, what):
    """o against fp64, within bounds that every whole group of 16 visible keys exceeds."""
    n, H_q, d = q.shape
    m, G = k.shape[0], H_q // k.shape[1]
    want, _, bound, _ = ref.attend(q, k, v, seen, d ** -0.5)
    over = (o.double() - want).abs() - bound
    assert (over <= 0).all(), f"{what}: {over.max().item()} over the bound"
    s = torch.einsum("nhd,mhd->nhm", q.double(), k.double().repeat_interleave(G, 1)) * d ** -0.5
    p = torch.softmax(s.masked_fill(~seen[:, None], -math.inf), -1)
    column = v[:, 0].argmax(-1)[::16]
    groups = len(column)
    pad = groups * 16 - m
    weight = torch.nn.functional.pad(p, (0, pad)).view(n, H_q, groups, 16).sum(-1)
    whole = torch.nn.functional.pad(seen, (0, pad)).view(n, groups, 16).all(-1)
    seen_by = whole[:, None].expand_as(weight)
    assert (weight > bound[..., column])[seen_by].all(), what


@pytest.mark.parametrize("lens,Lq,cap,H_q,H_kv,d,window,sinks,P", [
    ([9000, 20000, 1, 15000], 1, 20000, 32, 8, 128, None, 0, 0),
    ([20000, 3, 15000], 1, 20000, 16, 8, 64, None, 0, 0),
    ([12000] * 12, 2, 12000, 8, 8, 128, 5000, 130, 0),
    ([6000], 1, 6000, 2, 1, 128, None, 0, 0),
    ([900, 3000], 1, 3000, 32, 8, 128, None, 0, 20000),
    ([(r * 997) % 3000 + 1 for r in range(70)], 1, 3000, 8, 2, 128, None, 0, 9000),
    ([7] * 50, 3, 8, 6, 2, 64, None, 0, 3333),
])
def test_cache_loses_no_keys(lens, Lq, cap, H_q, H_kv, d, window, sinks, P):
    n = len(lens)
    q, k = rnd(0, n, Lq, H_q, d, std=0.5), rnd(1, n, cap, H_kv, d)
    kp = rnd(2, P, H_kv, d) if P else None
    every = marks(P + cap, H_kv, d)
    v, vp = every[P:].repeat(n, 1, 1, 1), every[:P].contiguous() if P else None
    plan = mapflow.CacheAttention(n, Lq, cap, H_q, H_kv, d, window=window, sinks=sinks, prefix_len=P)
    o = plan.attend(q, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"), kp, vp)
    plan.status()
    for r, L in enumerate(lens):
        seen = ref.seen_packed(torch.arange(L - Lq, L, device="cuda"), torch.arange(L, device="cuda"), window, sinks)
        kk = k[r, :L]
        if P:
            kk = torch.cat([kp, kk])
            seen = torch.cat([torch.ones(Lq, P, dtype=torch.bool, device="cuda"), seen], 1)
        check_marks(o[r], q[r], kk, every[:P + L], seen, f"request {r}")


@pytest.mark.parametrize("L,begin,H_q,H_kv,d,window,sinks", [
    (6000, 5999, 32, 8, 128, None, 0),
    (6000, 5900, 8, 2, 64, None, 0),
    (9000, 8950, 4, 2, 128, 4500, 7),
    (4100, 0, 4, 1, 128, 1024, 4),
    (5000, 0, 2, 2, 64, None, 0),
])
def test_packed_loses_no_keys(L, begin, H_q, H_kv, d, window, sinks):
    q, k, v = rnd(0, L, H_q, d, std=0.5), rnd(1, L, H_kv, d), marks(L, H_kv, d)
    plan = mapflow.WindowAttention([0, L], H_q, H_kv, d, window=window, sinks=sinks, q_begin=[begin])
    o = plan.attend(q, k, v)
    plan.status()
    for r0 in range(begin, L, 500):
        r1 = min(L, r0 + 500)
        seen = ref.seen_packed(torch.arange(r0, r1, device="cuda"), torch.arange(r1, device="cuda"), window, sinks)
        check_marks(o[r0:r1], q[r0:r1], k[:r1], v[:r1], seen, f"rows {r0} to {r1}")
