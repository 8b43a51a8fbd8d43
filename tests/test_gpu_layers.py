"""GPU tests of the rotary embedding with head norms, window attention with
sinks and shared-prefix attention, against fp64 definitions (layer_ref)."""
import math
import threading

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


def close(got, want, bound, what):
    got = got.double()
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() - bound
    assert (over <= 0).all(), f"{what}: {over.max().item()} over the bound"


# ------------------------------------------------------------------ rotary --
def check_rope(T, H_q, H_k, d, rot, layout, dt, norm, scaling="none", start=0, seed=0, weights=True):
    freq, gain = ref.rope_frequencies(rot, 10000.0, scaling, 4.0, 4096)
    plan = mapflow.RotaryPlan(rot, 10000.0, layout, scaling, 4.0, 4096)
    qkv = rnd(seed, T, (H_q + 2 * H_k) * d, dt=dt)
    q, k = qkv[:, :H_q * d].view(T, H_q, d), qkv[:, H_q * d:(H_q + H_k) * d].view(T, H_k, d)
    pos = (start + torch.randperm(T, generator=torch.Generator().manual_seed(seed))).to(torch.int32).cuda()
    wq = rnd(seed + 1, d, dt=dt) if norm and weights else None
    wk = rnd(seed + 2, d, dt=dt) if norm and weights else None
    before = qkv.clone()
    qo, ko = plan.apply(q, k, pos, q_weight=wq, k_weight=wk, eps=1e-6, norm=norm)
    assert torch.equal(before, qkv)
    for x, w, y, name in ((q, wq, qo, "q"), (k, wk, ko, "k")):
        want, bound = ref.rope(x, w, norm, 1e-6, pos, freq, gain, rot, layout)
        close(y, want, bound + want.abs() * torch.finfo(dt).eps / 2, name)
    return plan, q, k, pos, wq, wk, qo, ko


@pytest.mark.parametrize("T,H_q,H_k,d,rot,layout,dt,norm,scaling", [
    (1, 32, 8, 128, 128, "half", BF, True, "none"),
    (1, 1, 1, 64, 64, "interleaved", BF, False, "none"),
    (67, 24, 8, 128, 64, "interleaved", BF, True, "yarn"),
    (130, 3, 1, 64, 32, "half", BF, True, "linear"),
    (33, 5, 5, 128, 20, "half", BF, True, "none"),           # pairs inside 16-byte chunks
    (33, 5, 5, 64, 6, "half", torch.float32, True, "ntk"),
    (19, 2, 2, 128, 2, "half", BF, False, "none"),
    (19, 2, 2, 64, 2, "interleaved", torch.float32, True, "none"),
    (1025, 40, 40, 128, 128, "half", BF, True, "none"),
    (4099, 24, 8, 64, 64, "half", torch.float32, False, "linear"),
    (9000, 1, 1, 64, 64, "half", BF, True, "none"),          # few heads: many tokens per CTA
    (2000, 1, 1, 128, 96, "half", torch.float32, True, "yarn"),
])
def test_rope(T, H_q, H_k, d, rot, layout, dt, norm, scaling):
    check_rope(T, H_q, H_k, d, rot, layout, dt, norm, scaling)


def test_rope_far_positions():
    # fp32 angles would be off by 2^-24 of 2e9 radians: hundreds of turns
    check_rope(64, 4, 2, 128, 128, "half", torch.float32, False, start=2_000_000_000)
    check_rope(64, 4, 2, 128, 128, "interleaved", torch.float32, False, start=-500_000)


def test_rope_norm_without_weights_and_zero_rows():
    check_rope(17, 4, 2, 128, 128, "half", BF, True, weights=False)
    plan = mapflow.RotaryPlan(128)
    q = torch.zeros(3, 2, 128, dtype=BF, device="cuda")
    qo, ko = plan.apply(q, None, torch.arange(3, dtype=torch.int32, device="cuda"), norm=True)
    assert ko is None and torch.equal(qo, q)


@pytest.mark.parametrize("rot,layout", [(128, "half"), (20, "half"), (64, "interleaved")])
def test_rope_in_place_and_strided_out(rot, layout):
    plan, q, k, pos, wq, wk, qo, ko = check_rope(301, 6, 2, 128, rot, layout, BF, True, seed=3)
    buf = torch.full((301, 1200), 7.0, dtype=BF, device="cuda")
    out = buf[:, 8:8 + 768].view(301, 6, 128)
    plan.apply(q, k, pos, wq, wk, q_out=out, k_out=buf[:, 800:1056].view(301, 2, 128))
    assert torch.equal(out, qo) and torch.equal(buf[:, 800:1056].view(301, 2, 128), ko)
    assert (buf[:, :8] == 7).all() and (buf[:, 776:800] == 7).all() and (buf[:, 1056:] == 7).all()
    plan.apply(q, k, pos, wq, wk, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko)


def test_rope_of_no_tokens_and_other_streams_tables():
    plan = mapflow.RotaryPlan(128)
    q = torch.empty(0, 4, 128, dtype=BF, device="cuda")
    qo, ko = plan.apply(q, q[:, :2], torch.empty(0, dtype=torch.int32, device="cuda"), norm=True)
    assert qo.shape == (0, 4, 128) and ko.shape == (0, 2, 128)


def test_rope_many_tokens_uneven_heads():
    # several heads to a group, shares of q and k that do not divide evenly
    check_rope(9001, 40, 8, 64, 64, "half", BF, True, seed=2)
    check_rope(9001, 7, 3, 128, 96, "interleaved", torch.float32, True, seed=3)
    check_rope(3001, 13, 40, 128, 20, "half", BF, True, seed=4)


def test_rope_refuses_overlap_and_wrong_tensors():
    plan = mapflow.RotaryPlan(64)
    buf = rnd(0, 20, 4, 64)
    pos = torch.arange(10, dtype=torch.int32, device="cuda")
    q, k = buf[:10], buf[10:]
    for kw in (dict(q_out=buf[5:15]), dict(k_out=q), dict(q_out=torch.empty(9, 4, 64, dtype=BF, device="cuda"))):
        with pytest.raises(mapflow.MapFlowError):
            plan.apply(q, k, pos, **kw)
    for bad in (pos.long(), pos[:9], pos.cpu()):
        with pytest.raises(mapflow.MapFlowError):
            plan.apply(q, k, bad)
    with pytest.raises(mapflow.MapFlowError):
        plan.apply(q, k, pos, q_weight=torch.ones(64, device="cuda"))
    with pytest.raises(mapflow.MapFlowError):
        plan.apply(q.transpose(0, 1), None, pos[:4])


# --------------------------------------------------------- packed attention --
def check_packed(lens, H_q, H_kv, d, window=None, sinks=0, begin=None, seed=0, qstd=1.5, scale=None):
    T = sum(lens)
    cu = np.concatenate([[0], np.cumsum(lens)])
    q, k, v = rnd(seed, T, H_q, d, std=qstd), rnd(seed + 1, T, H_kv, d), rnd(seed + 2, T, H_kv, d)
    plan = mapflow.WindowAttention(cu, H_q, H_kv, d, window=window, sinks=sinks, q_begin=begin)
    o = torch.full((T, H_q, d), 3.0, dtype=BF, device="cuda")
    lse = torch.full((T, H_q), 3.0, device="cuda")
    plan.attend(q, k, v, o=o, lse=lse, scale=scale)
    plan.status()
    for s, L in enumerate(lens):
        a, b = int(cu[s]), begin[s] if begin else 0
        assert (o[a:a + b] == 3).all() and (lse[a:a + b] == 3).all()
        for r0 in range(b, L, 512):  # rows of a sequence, some at a time
            r1 = min(L, r0 + 512)
            seen = ref.seen_packed(torch.arange(r0, r1, device="cuda"), torch.arange(L, device="cuda"), window, sinks)
            want, wl, bo, bl = ref.attend(q[a + r0:a + r1], k[a:a + L], v[a:a + L], seen, scale or d ** -0.5)
            close(o[a + r0:a + r1], want, bo, f"o of sequence {s}")
            close(lse[a + r0:a + r1], wl, bl, f"lse of sequence {s}")
    return plan, q, k, v, o, lse


@pytest.mark.parametrize("lens,H_q,H_kv,d,window,sinks", [
    ([1], 1, 1, 64, None, 0),
    ([1], 8, 8, 128, 1, 0),
    ([127], 2, 2, 128, None, 0),
    ([128, 129], 4, 2, 128, None, 0),
    ([300, 1, 77, 16, 130], 6, 2, 128, 50, 3),
    ([257, 640], 5, 1, 64, 128, 4),
    ([513], 8, 1, 128, 100, 130),            # sinks across a block's end
    ([700], 24, 8, 64, 200, 0),
    ([1000, 0, 37], 3, 3, 128, 1, 1),        # each row sees itself and the first token
    ([900], 4, 4, 64, 2000, 5),              # window longer than the sequence
    ([260], 128, 1, 128, None, 0),           # one token per tile
    ([500, 321], 8, 2, 128, 64, 64),         # sinks and windows that end with a half block, and one past it
    ([700, 450], 4, 2, 64, 129, 65),
    ([385, 64, 65, 63], 4, 4, 128, 190, 1),
    ([90], 100, 1, 64, 17, 2),               # tiles with spare rows
])
def test_packed(lens, H_q, H_kv, d, window, sinks):
    check_packed(lens, H_q, H_kv, d, window, sinks)


def test_packed_many_heads_and_long():
    check_packed([2600, 511], 40, 40, 128, None, 0, seed=5)
    check_packed([4100], 32, 8, 128, 1024, 4, seed=6)


@pytest.mark.parametrize("lens,begin,H_q,H_kv,window,sinks", [
    ([6000], [5999], 32, 8, None, 0),        # a single row: cut over many CTAs, one tile
    ([6000], [5900], 8, 2, None, 0),         # tile pairs and a lone tile
    ([5000, 300, 40], [4990, 300, 3], 4, 4, None, 0),
    ([9000], [8950], 4, 2, 4500, 7),
])
def test_packed_chunks(lens, begin, H_q, H_kv, window, sinks):
    check_packed(lens, H_q, H_kv, 128, window, sinks, begin=begin)
    check_packed(lens, H_q, H_kv, 64, window, sinks, begin=begin, seed=9)


def test_packed_rows_16_bytes_off_a_sector():
    T, H_q, H_kv, d = 300, 4, 2, 64
    q, k, v = rnd(0, T, H_q, d), rnd(1, T, H_kv, d), rnd(2, T, H_kv, d)
    plan = mapflow.WindowAttention([0, T], H_q, H_kv, d)
    want = plan.attend(q, k, v)
    wide = torch.zeros(T, H_q * d + 8, dtype=BF, device="cuda")
    o = wide[:, 8:].view(T, H_q, d)
    plan.attend(q, k, v, o=o)
    assert torch.equal(o, want) and (wide[:, :8] == 0).all()


def test_packed_mixed_runs():
    # pairs, lone tiles whole and cut, and a long chunk in one plan
    lens = [3000, 20, 500, 1, 9000, 64, 0, 129]
    begin = [0, 0, 490, 0, 8990, 0, 0, 1]
    for d in (64, 128):
        check_packed(lens, 8, 2, d, None, 0, begin=begin, seed=d)
        check_packed(lens, 6, 2, d, 700, 9, begin=begin, seed=d + 1)


def test_packed_large_scores_and_scale():
    check_packed([300], 4, 2, 128, None, 0, qstd=40.0)        # references move often, weights near one-hot
    check_packed([300], 4, 2, 64, 64, 2, scale=0.5)


def test_packed_garbage_elsewhere_reaches_nothing():
    lens = [150, 333, 70]
    plan, q, k, v, o, lse = check_packed(lens, 4, 2, 128, 64, 2)
    for s in (0, 1, 2):
        qq, kk, vv = q.clone(), k.clone(), v.clone()
        keep = torch.zeros(sum(lens), dtype=torch.bool, device="cuda")
        keep[sum(lens[:s]):sum(lens[:s + 1])] = True
        for x in (qq, kk, vv):
            x[~keep] = float("nan")
        got = plan.attend(qq, kk, vv)
        assert torch.equal(got[keep], o[keep])


def test_packed_chunk_without_sight_of_old_keys():
    # keys before every row's window (sinks apart) may hold anything
    lens, begin = [2000], [1500]
    plan, q, k, v, o, lse = check_packed(lens, 4, 2, 128, 256, 5, begin=begin)
    k[5:1500 - 255] = float("nan")
    v[5:1500 - 255] = float("inf")
    got = plan.attend(q, k, v)
    assert torch.equal(got[1500:], o[1500:])


def test_packed_strided_and_repeatable():
    lens, H_q, H_kv, d = [400, 77], 8, 2, 128
    T = sum(lens)
    qkv = rnd(4, T, (H_q + 2 * H_kv) * d)
    q = qkv[:, :H_q * d].view(T, H_q, d)
    k = qkv[:, H_q * d:(H_q + H_kv) * d].view(T, H_kv, d)
    v = qkv[:, (H_q + H_kv) * d:].view(T, H_kv, d)
    plan = mapflow.WindowAttention([0, 400, 477], H_q, H_kv, d)
    wide = torch.zeros(T, H_q * d + 64, dtype=BF, device="cuda")
    o = wide[:, 32:32 + H_q * d].view(T, H_q, d)
    plan.attend(q, k, v, o=o)
    want = plan.attend(q.contiguous(), k.contiguous(), v.contiguous())
    assert torch.equal(o, want)
    assert (wide[:, :32] == 0).all() and (wide[:, -32:] == 0).all()
    for _ in range(3):
        assert torch.equal(plan.attend(q, k, v), want)


# ---------------------------------------------------------- cache attention --
def check_cache(lens, Lq, cap, H_q, H_kv, d, window=None, sinks=0, P=0, n_max=None, seed=0, junk=float("nan")):
    n = len(lens)
    q = rnd(seed, n, Lq, H_q, d, std=1.5)
    k, v = rnd(seed + 1, n, cap, H_kv, d), rnd(seed + 2, n, cap, H_kv, d)
    kp, vp = (rnd(seed + 3, P, H_kv, d), rnd(seed + 4, P, H_kv, d)) if P else (None, None)
    for r, L in enumerate(lens):  # past a cache's keys: anything
        k[r, max(0, min(L, cap)):] = junk
        v[r, max(0, min(L, cap)):] = junk
    plan = mapflow.CacheAttention(n_max or n, Lq, cap, H_q, H_kv, d, window=window, sinks=sinks, prefix_len=P)
    dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    lse = torch.empty(n, Lq, H_q, device="cuda")
    o = plan.attend(q, k, v, dl, kp, vp, lse=lse)
    plan.status()
    for r, L in enumerate(lens):
        L = max(0, min(L, cap))
        kk, vv = k[r, :L], v[r, :L]
        seen = ref.seen_packed(torch.arange(L - Lq, L, device="cuda"), torch.arange(L, device="cuda"), window, sinks)
        if P:
            kk, vv = torch.cat([kp, kk]), torch.cat([vp, vv])
            seen = torch.cat([torch.ones(Lq, P, dtype=torch.bool, device="cuda"), seen], 1)
        want, wl, bo, bl = ref.attend(q[r], kk, vv, seen, d ** -0.5)
        close(o[r], want, bo, f"o of request {r}")
        none = ~seen.any(1)
        assert torch.isneginf(lse[r][none]).all() and (o[r][none] == 0).all()
        close(lse[r][~none], wl[~none], bl[~none], f"lse of request {r}")
    return plan, q, k, v, dl, kp, vp, o, lse


@pytest.mark.parametrize("lens,Lq,cap,H_q,H_kv,d,window,sinks", [
    ([1], 1, 1, 1, 1, 64, None, 0),
    ([5], 1, 16, 8, 2, 128, None, 0),
    ([0, 1, 127, 128, 129, 500], 1, 500, 8, 2, 128, None, 0),
    ([0, 0], 1, 10, 4, 2, 64, None, 0),
    ([3, 0, 1, 40], 4, 64, 6, 2, 128, None, 0),        # fewer keys than new tokens
    ([300, 17, 299], 5, 300, 5, 1, 64, 33, 2),
    ([2000, 1, 777, 1500], 1, 2048, 32, 8, 128, 500, 4),
    ([2000, 900], 2, 2000, 24, 8, 128, 256, 300),      # more sinks than a block
    ([40, 41, 42], 32, 64, 4, 1, 128, None, 0),        # 128 rows of one request
    ([63, 64, 65, 191, 192, 193, 320], 1, 320, 8, 2, 128, None, 0),
    ([400, 193, 130, 129, 66], 1, 400, 8, 2, 64, 64, 1),
    ([400, 350, 260, 129, 66], 2, 400, 4, 2, 128, 127, 64),
    ([-5, 99], 1, 64, 2, 1, 128, None, 0),             # lengths held to the capacity
    ([6000], 1, 6000, 2, 1, 128, None, 0),             # one request over every CTA
])
def test_cache(lens, Lq, cap, H_q, H_kv, d, window, sinks):
    check_cache(lens, Lq, cap, H_q, H_kv, d, window, sinks)


@pytest.mark.parametrize("lens,Lq,cap,H_q,H_kv,d,P", [
    ([1], 1, 4, 1, 1, 64, 1),
    ([0, 0, 0], 1, 4, 8, 2, 128, 130),                 # the prefix alone
    ([10, 3], 2, 16, 24, 8, 128, 1000),                # one lone tile
    ([1, 5, 9, 0] * 20, 1, 9, 4, 1, 64, 500),          # 80 tokens of 4 heads: a pair and a lone tile
    ([200, 1] * 33, 1, 200, 8, 8, 128, 257),
    ([7] * 50, 3, 8, 6, 2, 128, 3333),
    ([60] * 64, 1, 64, 32, 8, 128, 4097),
])
def test_shared_prefix(lens, Lq, cap, H_q, H_kv, d, P):
    check_cache(lens, Lq, cap, H_q, H_kv, d, P=P)


def test_cache_long_runs():
    # tens of key blocks per CTA, the ring's stages used many times over
    check_cache([9000, 20000, 1, 15000], 1, 20000, 32, 8, 128)
    check_cache([20000, 3, 15000], 1, 20000, 16, 8, 64)
    check_cache([12000] * 12, 2, 12000, 8, 8, 128, 5000, 130)


def test_cache_many_requests_and_head_groups():
    rng = np.random.default_rng(0)
    check_cache([int(x) for x in rng.integers(0, 41, 600)], 1, 40, 4, 2, 64)
    check_cache([int(x) for x in rng.integers(0, 300, 40)], 4, 300, 40, 40, 128)      # 3 heads to a tile, 14 tiles
    check_cache([int(x) for x in rng.integers(0, 300, 30)], 3, 300, 44, 11, 64, 100, 7)  # last tile part full
    check_cache([int(x) for x in rng.integers(0, 500, 300)], 1, 500, 24, 8, 128, P=2000)
    check_cache([100, 0, 33], 1, 128, 1024, 1024, 64)


@pytest.mark.parametrize("n,P", [(1, 20000), (3, 9000), (70, 9000)])
def test_prefix_and_long_caches(n, P):
    rng = np.random.default_rng(n)
    check_cache([int(x) for x in rng.integers(1, 3000, n)], 1, 3000, 32, 8, 128, P=P)


def test_cache_fewer_requests_than_planned_and_garbage():
    plan, q, k, v, dl, kp, vp, o, lse = check_cache([30, 2, 64], 1, 64, 8, 2, 128, P=300, n_max=9)
    got = plan.attend(q[:2], k[:2], v[:2], dl[:2], kp, vp)
    # other cuts of the same keys: both are within the bounds of the truth
    for r in range(2):
        L = int(dl[r])
        kk, vv = torch.cat([kp, k[r, :L]]), torch.cat([vp, v[r, :L]])
        want, _, bo, _ = ref.attend(q[r], kk, vv, torch.ones(1, 300 + L, dtype=torch.bool, device="cuda"), 128 ** -0.5)
        close(got[r], want, bo, f"request {r}")
    # another request's keys reach nobody else
    k2, v2 = k.clone(), v.clone()
    k2[1] = v2[1] = float("nan")
    got = plan.attend(q, k2, v2, dl, kp, vp)
    assert torch.equal(got[0], o[0]) and torch.equal(got[2], o[2])
    # a strided cache: the first heads of a wider one
    wide = torch.full((3 * 64, 4 * 128), float("nan"), dtype=BF, device="cuda")
    kw = wide[:, :256].view(3, 64, 2, 128)
    kw.copy_(k)
    assert torch.equal(plan.attend(q, kw, v, dl, kp, vp), o)


def test_scores_that_are_not_numbers_stay_so():
    """A query or a key that is NaN makes the rows that use it NaN, whole or
    joined from partial results, and no other row."""
    plan, q, k, v, o, lse = check_packed([700], 4, 2, 128)[:6]
    chunk, cq, ck, cv, co, cl = check_packed([5000], 4, 2, 128, begin=[4990])
    for p, x, y, z, at in ((plan, q, k, v, 650), (chunk, cq, ck, cv, 4995)):
        want = p.attend(x, y, z)
        x2, got, gl = x.clone(), torch.zeros_like(x), torch.zeros(x.shape[:2], device="cuda")
        x2[at, 1] = float("nan")
        p.attend(x2, y, z, o=got, lse=gl)
        lo = 4990 if p is chunk else 0
        hit = torch.zeros(x.shape[:2], dtype=torch.bool, device="cuda")
        hit[at, 1] = True
        assert torch.isnan(got[hit]).all() and torch.isnan(gl[hit]).all()
        assert torch.equal(got[lo:][~hit[lo:]], want[lo:][~hit[lo:]]) and not torch.isnan(gl[lo:][~hit[lo:]]).any()
    for P in (0, 1000):
        plan, q, k, v, dl, kp, vp, o, lse = check_cache([300, 1, 0, 40], 2, 300, 8, 2, 128, P=P)
        q2, gl = q.clone(), torch.empty_like(lse)
        q2[0, 1, 3] = q2[1, 1, 0] = q2[3, 0, 7] = float("nan")
        hit = torch.isnan(q2).any(-1)
        got = plan.attend(q2, k, v, dl, kp, vp, lse=gl)
        assert torch.isnan(got[hit]).all() and torch.isnan(gl[hit]).all()
        assert torch.equal(got[~hit], o[~hit]) and torch.equal(gl[~hit], lse[~hit])


def test_offsets_past_32_bits():
    """Rows 2^26 and caches 2^31 values apart."""
    T, H_q, H_kv, d, ld = 40, 4, 2, 128, 1 << 26
    buf = torch.empty(T * ld, dtype=BF, device="cuda")
    wide = buf.view(T, ld)
    q, k, v, o = (wide[:, a:a + n * d].view(T, n, d) for a, n in ((0, H_q), (1024, H_kv), (2048, H_kv), (4096, H_q)))
    q0, k0, v0 = rnd(0, T, H_q, d), rnd(1, T, H_kv, d), rnd(2, T, H_kv, d)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    rope = mapflow.RotaryPlan(d)
    q.copy_(q0), k.copy_(k0), v.copy_(v0)
    rope.apply(q, k, pos, norm=True, q_out=q, k_out=k)
    q1, k1 = rope.apply(q0, k0, pos, norm=True)
    assert torch.equal(q, q1) and torch.equal(k, k1)
    plan = mapflow.WindowAttention([0, T], H_q, H_kv, d)
    plan.attend(q, k, v, o=o)
    plan.status()
    assert torch.equal(o, plan.attend(q1, k1, v0))
    # (the last request's cache begins 2^31 + 2^30 values in)
    n, cap = 4, (1 << 30) // (H_kv * d)
    kc, vc = (torch.empty(n, cap, H_kv, d, dtype=BF, device="cuda") for _ in range(2))
    lens = torch.tensor([0, 0, 0, T], dtype=torch.int32, device="cuda")
    kc[3, :T], vc[3, :T] = k0, v0
    dec = mapflow.CacheAttention(n, 1, cap, H_q, H_kv, d)
    qd = rnd(5, n, 1, H_q, d)
    got = dec.attend(qd, kc, vc, lens)
    dec.status()
    small = mapflow.CacheAttention(n, 1, T, H_q, H_kv, d)
    ks, vs = (x[:, :T].contiguous() for x in (kc, vc))
    want, _, bo, _ = ref.attend(qd[3], ks[3], vs[3], torch.ones(1, T, dtype=torch.bool, device="cuda"), d ** -0.5)
    close(got[3], want, bo, "far cache")
    assert (got[:3] == 0).all() and (small.attend(qd, ks, vs, lens)[:3] == 0).all()


@pytest.mark.parametrize("P", [0, 300])
def test_cache_mostly_unused_slots(P):
    for n, used in ((256, (0, 31, 32, 200, 255)), (8300, (0, 8000, 8191, 8192, 8250, 8299)), (300, (299,))):
        lens = [0] * n
        for i, r in enumerate(used):
            lens[r] = 40 - 3 * i
        check_cache(lens, 1, 40, 2, 1, 64, P=P)


def test_workspace_grows_with_requests_not_with_their_keys():
    # units + CTAs runs at most, two streams of a tile's 32 rows each
    for n, cap, P in ((1, 8192, 0), (512, 8192, 0), (512, 8, 32768)):
        plan = mapflow.CacheAttention(n, 1, cap, 32, 8, 128, prefix_len=P)
        pairs = -(-n * 4 // 256) if P else 0
        rows = 2 * (n + 160) * 32 + 2 * (pairs * 8 + 160) * 128 * (P > 0)
        assert plan._workspace_bytes(n) <= rows * (128 * 4 + 8) + 8 * (n + 8 * pairs) + 1024


def test_cache_refusals():
    plan = mapflow.CacheAttention(4, 1, 32, 4, 2, 64, prefix_len=16)
    q, k, v = rnd(0, 4, 1, 4, 64), rnd(1, 4, 32, 2, 64), rnd(2, 4, 32, 2, 64)
    kp, vp = rnd(3, 16, 2, 64), rnd(4, 16, 2, 64)
    lens = torch.full((4,), 9, dtype=torch.int32, device="cuda")
    good = plan.attend(q, k, v, lens, kp, vp)
    bad = [dict(k_prefix=None), dict(k_prefix=kp[:15]), dict(lens=lens.long()), dict(lens=lens.cpu()),
           dict(lens=lens[:3]), dict(q=q.float()), dict(q=q[:, :, :2]), dict(k_cache=k[:, :16]),
           dict(k_cache=k[:3]), dict(o=q), dict(o=good[:3]), dict(scale=0.0), dict(scale=-1.0),
           dict(scale=float("nan")), dict(lse=torch.empty(4, 1, 4, device="cuda", dtype=torch.float64)),
           dict(q=torch.cat([q, q]), k_cache=torch.cat([k, k]), v_cache=torch.cat([v, v]), lens=torch.cat([lens, lens]))]
    for kw in bad:
        args = dict(q=q, k_cache=k, v_cache=v, lens=lens, k_prefix=kp, v_prefix=vp)
        args.update(kw)
        with pytest.raises(mapflow.MapFlowError):
            plan.attend(**args)
    assert torch.equal(plan.attend(q, k, v, lens, kp, vp), good)
    lone = mapflow.CacheAttention(4, 1, 32, 4, 2, 64)
    with pytest.raises(mapflow.MapFlowError):
        lone.attend(q, k, v, lens, kp, vp)
    packed = mapflow.WindowAttention([0, 8], 4, 2, 64)
    x = rnd(5, 8, 4, 64)
    y = rnd(6, 8, 2, 64)
    with pytest.raises(mapflow.MapFlowError):
        packed.attend(x, y, y, o=x)
    with pytest.raises(mapflow.MapFlowError):
        packed.attend(x[:7], y[:7], y[:7])


def test_cache_follows_lens_in_a_captured_graph():
    n, cap, P = 3, 300, 200
    plan = mapflow.CacheAttention(n, 1, cap, 8, 2, 128, prefix_len=P)
    q, k, v = rnd(0, n, 1, 8, 128), rnd(1, n, cap, 2, 128), rnd(2, n, cap, 2, 128)
    kp, vp = rnd(3, P, 2, 128), rnd(4, P, 2, 128)
    lens = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    o = torch.empty_like(q)
    plan.attend(q, k, v, lens, kp, vp, o=o)
    torch.cuda.synchronize()
    g, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.attend(q, k, v, lens, kp, vp, o=o)
    o2 = torch.empty_like(q)
    q2 = rnd(9, n, 1, 8, 128)
    with torch.cuda.graph(g2):
        plan.attend(q2, k, v, lens, kp, vp, o=o2)
    side = torch.cuda.Stream()
    for ln in ([300, 0, 7], [128, 129, 1]):
        lens.copy_(torch.tensor(ln, dtype=torch.int32))
        want, want2 = plan.attend(q, k, v, lens, kp, vp), plan.attend(q2, k, v, lens, kp, vp)
        torch.cuda.synchronize()
        g.replay()                       # two graphs of one plan at the same time
        with torch.cuda.stream(side):
            g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(o2, want2)


def test_streams():
    lens = [600, 300]
    plan, q, k, v, o, lse = check_packed(lens, 4, 2, 128, 200, 3)
    chunk, cq, ck, cv, co, _ = check_packed([5000], 4, 2, 128, begin=[4990])
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for i in range(12):
        s = streams[i % 3]
        got.append((plan.attend(q, k, v, stream=s), chunk.attend(cq, ck, cv, stream=s)))
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a, o) and torch.equal(b[4990:], co[4990:])
    rp = mapflow.RotaryPlan(128)
    pos = torch.arange(900, dtype=torch.int32, device="cuda")
    want, _ = rp.apply(q, None, pos)
    torch.cuda.synchronize()
    got, _ = rp.apply(q, None, pos, stream=streams[0])
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_threads():
    """Two threads use the same plans on streams of their own."""
    plan, q, k, v, dl, kp, vp, o, lse = check_cache([30, 2, 64, 0], 1, 64, 8, 2, 128, P=300)
    chunk, cq, ck, cv, co, _ = check_packed([5000], 4, 2, 128, begin=[4990])
    torch.cuda.synchronize()
    wrong = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(30):
                a, b = plan.attend(q, k, v, dl, kp, vp), chunk.attend(cq, ck, cv)
                s.synchronize()
                if not (torch.equal(a, o) and torch.equal(b[4990:], co[4990:])):
                    wrong.append(1)

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_layers_together():
    """A receiver layer as it is served: rotary and norms on a fused
    projection, window attention over the prompt, then decode steps over the
    cache; every decode step equals the packed attention's row."""
    T, steps, H_q, H_kv, d, W, S = 200, 6, 8, 2, 128, 64, 4
    N = T + steps
    qkv = rnd(1, N, (H_q + 2 * H_kv) * d)
    q, k = qkv[:, :H_q * d].view(N, H_q, d), qkv[:, H_q * d:(H_q + H_kv) * d].view(N, H_kv, d)
    v = qkv[:, (H_q + H_kv) * d:].view(N, H_kv, d)
    wq, wk = rnd(2, d), rnd(3, d)
    rope = mapflow.RotaryPlan(d, 1e6)
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    qr, kr = rope.apply(q, k, pos, wq, wk)
    whole = mapflow.WindowAttention([0, N], H_q, H_kv, d, window=W, sinks=S).attend(qr, kr, v)
    prompt = mapflow.WindowAttention([0, T], H_q, H_kv, d, window=W, sinks=S)
    q0, k0 = rope.apply(q[:T], k[:T], pos[:T], wq, wk)
    assert torch.equal(prompt.attend(q0, k0, v[:T]), whole[:T])
    kc = torch.full((1, 256, H_kv, d), float("nan"), dtype=BF, device="cuda")
    vc = kc.clone()
    kc[0, :T], vc[0, :T] = k0, v[:T]
    dec = mapflow.CacheAttention(1, 1, 256, H_q, H_kv, d, window=W, sinks=S)
    for t in range(T, N):
        q1, k1 = rope.apply(q[t:t + 1], k[t:t + 1], pos[t:t + 1], wq, wk)
        assert torch.equal(q1[0], qr[t]) and torch.equal(k1[0], kr[t])
        kc[0, t], vc[0, t] = k1[0], v[t]
        o = dec.attend(q1[None], kc, vc, torch.tensor([t + 1], dtype=torch.int32, device="cuda"))
        lo = t - W + 1
        seen = ref.seen_packed(torch.tensor([t], device="cuda"), torch.arange(t + 1, device="cuda"), W, S)
        want, _, bo, _ = ref.attend(q1, kc[0, :t + 1], vc[0, :t + 1], seen, d ** -0.5)
        close(o[0], want, bo, f"step {t}")
        close(whole[t:t + 1], want, bo, f"row {t}")
        assert lo > S


def test_rows_of_the_reused_layers_path():
    """The compressor takes what the rotary call gives: with p = 1 and an
    identity head map its retrieval is the packed attention of the same q, k."""
    T, H, d = 320, 4, 128
    q, k, v = rnd(1, T, H, d), rnd(2, T, H, d), rnd(3, T, H, d)
    qr, kr = mapflow.RotaryPlan(d).apply(q, k, torch.arange(T, dtype=torch.int32, device="cuda"), norm=True)
    bsr = mapflow.BSR(1, T, H, 64, [0, T])
    bsr.compress(0, qr, kr, 1.0)
    o = torch.empty(1, T, H, d, dtype=BF, device="cuda")
    bsr.retrieve(torch.eye(H, device="cuda")[None], v[None], o, [0])
    mine = mapflow.WindowAttention([0, T], H, H, d).attend(qr, kr, v)
    ex = bsr.export(0)
    seen = ref.seen_packed(torch.arange(T, device="cuda"), torch.arange(T, device="cuda"), None, 0)
    want, wl, bo, bl = ref.attend(qr, kr, v, seen, d ** -0.5)
    close(mine, want, bo, "attention")
    # the compressor's row statistics are the same softmax
    lse = torch.empty(T, H, device="cuda")
    mapflow.WindowAttention([0, T], H, H, d).attend(qr, kr, v, lse=lse)
    close(ex["row_max"].T + ex["row_sum"].T.log(), wl, bl + 2.0 ** -20 * wl.abs(), "statistics")
    # (and the retrieval stores its weights as bf16 before the product too)
    close(o[0], want, bo * 2, "retrieval at p = 1")
    bsr.close()
