"""GPU tests of plans of the rotary and attention layers that are dropped
while their kernels may still run, or while a stream is captured."""
import pytest
import torch

from cross_model_attention_gb300 import mapflow

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


def test_rotary_plan_dropped_behind_a_call_on_another_stream():
    """The table's memory must not be handed out again while the call waits."""
    side = torch.cuda.Stream()
    q, pos = rnd(0, 500, 8, 128), torch.arange(500, dtype=torch.int32, device="cuda")
    want, _ = mapflow.RotaryPlan(128).apply(q, None, pos)
    torch.cuda.synchronize()
    for _ in range(3):
        plan = mapflow.RotaryPlan(128)
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # about 10 ms
        got, _ = plan.apply(q, None, pos, stream=side)
        del plan
        junk = [torch.full((64,), -1, dtype=torch.int64, device="cuda") for _ in range(64)]
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        del junk, got


def test_rotary_plan_dropped_during_a_capture():
    side = torch.cuda.Stream()
    q, pos = rnd(0, 50, 8, 128), torch.arange(50, dtype=torch.int32, device="cuda")
    old, kept = mapflow.RotaryPlan(128), mapflow.RotaryPlan(128)
    want, _ = kept.apply(q, None, pos)
    old.apply(q, None, pos, stream=side)
    torch.cuda.synchronize()
    g, out = torch.cuda.CUDAGraph(), torch.zeros_like(q)
    with torch.cuda.graph(g):
        kept.apply(q, None, pos, q_out=out)
        del old
        with torch.cuda.stream(side):  # not part of the capture
            other = mapflow._capturing(torch.cuda.current_device())
    assert other and not mapflow._capturing(torch.cuda.current_device())
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    del kept
    assert not mapflow._parked


def test_attention_plans_dropped_during_a_capture():
    side = torch.cuda.Stream()
    q, k, v = rnd(0, 5000, 4, 64), rnd(1, 5000, 2, 64), rnd(2, 5000, 2, 64)
    lens = torch.tensor([4000], dtype=torch.int32, device="cuda")

    def plans():
        return (mapflow.WindowAttention([0, 5000], 4, 2, 64, q_begin=[4990]),
                mapflow.CacheAttention(1, 1, 5000, 4, 2, 64))

    def call(a, b, **kw):
        return a.attend(q, k, v, **kw)[4990:], b.attend(q[None, :1], k[None], v[None], lens, **kw)
    kept, old = plans(), plans()
    want = call(*kept)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        got = call(*old)  # still to run when the plans go
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g.capture_begin()  # (torch.cuda.graph would wait for the device)
        out = call(*kept)
        del old
        assert len(mapflow._parked) == 2
        g.capture_end()
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    for x, y, z in zip(got, want, out):
        assert torch.equal(x, y) and torch.equal(z, y)
    del kept
    assert not mapflow._parked


def test_compressed_state_dropped_during_a_capture():
    T, H, d = 256, 4, 128
    q, k, v = rnd(1, T, H, d), rnd(2, T, H, d), rnd(3, 1, T, H, d)
    bsr = mapflow.BSR(1, T, H, 64, [0, T])
    bsr.compress(0, q, k, 0.95)
    o, x = torch.empty_like(v), torch.zeros(8, device="cuda")
    bsr.retrieve(torch.eye(H, device="cuda")[None], v, o, [0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x += 1
        del bsr
        assert len(mapflow._parked) == 1
    g.replay()
    assert (x == 1).all()
    mapflow.BSR(1, T, H, 64, [0, T]).close()
    assert not mapflow._parked
