"""Plans of the rotary and attention layers, and compressed states, that are
dropped while their kernels may still run (host side, no GPU needed)."""
import ctypes
import os
import subprocess
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
        waits, capturing, watch, running = [], False, None, False

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
    # and does not keep what is released after it
    done = []
    mapflow._release(0, lambda: done.append(1))
    assert done == [1] and gpu.watch() is not None
    monkeypatch.setattr(torch.cuda, "synchronize", lambda dev=None: None)
    mapflow._release_parked()
    assert gpu.watch() is None


# ------------------------------- the library's host code on a fake runtime --
@pytest.fixture(scope="module")
def host(tmp_path_factory):
    """mf_attn.cu's host code linked with stand-ins for the CUDA runtime."""
    return fake_library(tmp_path_factory, "mf_attn.cu")


def fake_library(tmp_path_factory, source, *flags):
    here = os.path.dirname(os.path.abspath(__file__))
    out = str(tmp_path_factory.mktemp("fake") / "libfake.so")
    cuda = os.path.dirname(os.path.dirname(build_mod._nvcc()))
    cmd = ["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wl,-Bsymbolic,-z,lazy", *flags, "-I", os.path.join(cuda, "include"),
           "-x", "c++", os.path.join(build_mod.CSRC, source), os.path.join(here, "fake_cuda.cpp"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    dlopen = ctypes.CDLL(None).dlopen  # (ctypes itself would ask for every function, called or not)
    dlopen.restype, dlopen.argtypes = ctypes.c_void_p, [ctypes.c_char_p, ctypes.c_int]
    handle = dlopen(out.encode(), os.RTLD_LAZY)
    assert handle
    lib = ctypes.CDLL(out, handle=handle)
    lib.fake_log.restype = ctypes.c_char_p
    return lib


P = 1 << 30  # aligned addresses, far apart, that host checks never follow
NO_ALLOC = (mapflow.ALLOC_FN(), mapflow.FREE_FN(), None)


def plan_of(host, form, device=0):
    host.fake_device(device)
    h = ctypes.c_void_p()
    if form == "packed":
        cu = (ctypes.c_int32 * 2)(0, 5000)
        rc = host.mf_attn_create_packed(ctypes.byref(h), cu, None, 1, 4, 2, 64, 0, 0, *NO_ALLOC)
    else:
        rc = host.mf_attn_create_cache(ctypes.byref(h), 2, 1, 64, 0, 4, 2, 64, 0, 0, *NO_ALLOC)
    assert rc == mapflow.MF_OK
    host.fake_log()
    return h


def attend(host, h, form):
    i64, f32, vp = ctypes.c_int64, ctypes.c_float, ctypes.c_void_p
    if form == "packed":
        a = [vp(P), i64(256), vp(2 * P), i64(128), vp(3 * P), i64(128), vp(4 * P), i64(256), None]
        return host.mf_attn_packed(h, *a, mapflow.MF_DTYPE_BF16, f32(1), vp(5 * P), i64(1 << 30), None)
    a = [vp(P), i64(256), vp(2 * P), i64(128), vp(3 * P), i64(128), vp(6 * P), None, i64(0), None, i64(0), vp(4 * P),
         i64(256), None]
    return host.mf_attn_cached(h, 2, *a, mapflow.MF_DTYPE_BF16, f32(1), vp(5 * P), i64(1 << 30), None)


FORMS = ["packed", "cache"]


@pytest.mark.parametrize("form", FORMS)
def test_destroy_waits_for_the_plans_own_device(host, form):
    h = plan_of(host, form, device=1)
    host.fake_device(3)
    host.mf_attn_destroy(h)
    did = host.fake_log().decode().split()
    assert did[0] == "sync1" and set(did[1:]) == {"free1", "unpin1"}
    assert host.fake_current() == 3


@pytest.mark.parametrize("form", FORMS)
def test_calls_under_another_device_are_refused(host, form):
    h = plan_of(host, form, device=1)
    before = host.fake_launches()
    host.fake_device(0)
    assert attend(host, h, form) == mapflow.MF_ERR_ARG
    assert host.mf_attn_status(h, None) == mapflow.MF_ERR_ARG
    assert host.fake_launches() == before
    host.fake_device(1)
    assert attend(host, h, form) == mapflow.MF_OK and host.mf_attn_status(h, None) == mapflow.MF_OK
    assert host.fake_launches() > before
    host.mf_attn_destroy(h)


@pytest.mark.parametrize("form", FORMS)
def test_destroy_without_a_wait_frees_nothing(host, form):
    """A wait that a stream capture refuses leaves the tables to the kernels that may read them."""
    h = plan_of(host, form)
    host.fake_sync_returns(900)  # cudaErrorStreamCaptureUnsupported
    host.mf_attn_destroy(h)
    host.fake_sync_returns(0)
    assert host.fake_log().decode().split() == ["sync0"]
    h = plan_of(host, form)
    host.fake_sync_returns(700)  # any other error: nothing runs any more
    host.mf_attn_destroy(h)
    host.fake_sync_returns(0)
    assert "free0" in host.fake_log().decode().split()


@pytest.mark.parametrize("cls", [mapflow.WindowAttention, mapflow.CacheAttention, mapflow.BSR])
def test_plans_and_states_dropped_during_a_capture(gpu, monkeypatch, cls):
    gone = []

    class Lib:
        mf_attn_destroy = mf_bsr_destroy = staticmethod(gone.append)
    monkeypatch.setattr(mapflow, "load_library", lambda: Lib)

    class Plan(cls):
        def __del__(self):
            if gpu.running:  # (a failure leaves plans that are none)
                super().__del__()

    def plan(handle):
        p = Plan.__new__(Plan)
        p.handle, p._keep, p._gpu = handle, (), 0
        return p
    monkeypatch.setattr(gpu, "running", True)
    a, b, c = plan(1), plan(2), plan(3)
    a.close()
    a.close()
    assert gone == [1]
    gpu.capturing = True
    del b
    assert gone == [1]
    gpu.capturing = False
    c.close()
    assert sorted(gone) == [1, 2, 3]


@pytest.fixture(scope="module")
def host_bsr(tmp_path_factory):
    """mf_api.cu's host code linked with stand-ins for the CUDA runtime."""
    return fake_library(tmp_path_factory, "mf_api.cu", "-DFAKE_RUNTIME_ONLY")


def bsr_of(host, device=0):
    host.fake_device(device)
    h = ctypes.c_void_p()
    cu = (ctypes.c_int32 * 2)(0, 300)
    assert host.mf_bsr_create(ctypes.byref(h), 2, 300, 4, 64, 1, cu, 1, *NO_ALLOC) == mapflow.MF_OK
    host.fake_log()
    return h


def test_bsr_destroy_waits_for_its_own_device(host_bsr):
    h = bsr_of(host_bsr, device=1)
    host_bsr.fake_device(3)
    host_bsr.mf_bsr_destroy(h)
    did = host_bsr.fake_log().decode().split()
    assert did[0] == "sync1" and set(did[1:]) == {"free1", "sync1", "unpin1"}
    assert host_bsr.fake_current() == 3


def test_bsr_destroy_without_a_wait_frees_nothing(host_bsr):
    h = bsr_of(host_bsr)
    host_bsr.fake_sync_returns(900)  # cudaErrorStreamCaptureUnsupported
    host_bsr.mf_bsr_destroy(h)
    host_bsr.fake_sync_returns(0)
    assert host_bsr.fake_log().decode().split() == ["sync0"]
