"""Plans of the rotary and attention layers that are dropped while their
kernels may still run (host side, no GPU needed)."""
import weakref

import pytest

from cross_model_attention_gb300 import build as build_mod
from cross_model_attention_gb300 import mapflow

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    build_mod.build()


@pytest.fixture
def gpu(monkeypatch):
    """A stand-in for the GPU's state: the waits for it, and whether a stream is captured."""
    class State:
        waits, capturing, watch = [], False, None

    state = State()
    state.waits = []
    monkeypatch.setattr(torch.cuda, "synchronize", lambda dev=None: state.waits.append(
        (dev, state.watch is not None and state.watch() is not None)))
    monkeypatch.setattr(mapflow, "_capturing", lambda gpu: state.capturing, raising=False)
    if hasattr(mapflow, "_parked"):
        monkeypatch.setattr(mapflow, "_parked", [])
    return state


def rotary(home):
    """A plan whose table stands on the CPU, with a library call that does nothing."""
    plan = mapflow.RotaryPlan(64, device="cpu")
    plan._home = home
    plan._call = lambda *args: 0
    return plan


def call(plan, stream):
    q = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    return plan._apply(stream, -1, mapflow.MF_DTYPE_BF16, q, None, torch.arange(3, dtype=torch.int32), None, None,
                       1e-6, None, None, None)


def test_rotary_table_outlives_calls_on_other_streams(gpu):
    plan = rotary(home=5)
    gpu.watch = weakref.ref(plan.turns)
    call(plan, 5)
    call(plan, 9)
    del plan
    assert gpu.waits == [(-1, True)]  # one wait, with the table still there
    assert gpu.watch() is None


def test_rotary_table_of_one_stream_needs_no_wait(gpu):
    plan = rotary(home=5)
    gpu.watch = weakref.ref(plan.turns)
    call(plan, 5)
    del plan
    assert gpu.waits == [] and gpu.watch() is None


def test_rotary_plan_dropped_during_a_capture(gpu):
    plan, other = rotary(home=5), rotary(home=5)
    gpu.watch = weakref.ref(plan.turns)
    call(plan, 9)
    call(other, 9)
    gpu.capturing = True
    del plan
    assert gpu.waits == [] and gpu.watch() is not None  # neither waited for nor given back
    gpu.capturing = False
    del other
    assert len(gpu.waits) == 2 and all(alive for _, alive in gpu.waits[:1]) and gpu.watch() is None


def test_a_failed_wait_keeps_the_table(gpu, monkeypatch):
    plan = rotary(home=5)
    gpu.watch = weakref.ref(plan.turns)
    call(plan, 9)

    def fails(dev=None):
        raise RuntimeError("not permitted")
    monkeypatch.setattr(torch.cuda, "synchronize", fails)
    del plan
    assert gpu.watch() is not None
