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
