"""The paged cache's host code: what may share memory in its calls (no GPU
needed: a stand-in for the CUDA runtime)."""
import ctypes
import os

import pytest

from cross_model_attention_gb300 import mapflow
from tests import test_paged_cache as base
from tests.test_layer_lifetimes import fake_library

E, PTR = mapflow, base.PTR
OK, ARG = E.MF_OK, E.MF_ERR_ARG


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    """mf_cache_api.cu's host code linked with stand-ins for the CUDA runtime and the launchers."""
    here = os.path.dirname(os.path.abspath(__file__))
    lib = fake_library(tmp_path_factory, "mf_cache_api.cu", os.path.join(here, "fake_paged.cpp"))
    full = mapflow.load_library()
    for name in ("mf_cache_append", "mf_cache_read", "mf_attn_paged", "mf_attn_paged_workspace"):
        getattr(lib, name).argtypes = getattr(full, name).argtypes
    lib.mf_last_error.restype = ctypes.c_char_p
    return lib


# 10 pages of 64 tokens of 8 heads of 128: their bytes, and where a call of
# test_paged_cache.py's defaults has its tensors (PTR times a number each)
PAGES = 10 * 64 // 16 * 8 * 18 * 128
LAST = PTR + PAGES - 16


def _refused(host, call, cache, name, **kw):
    before = host.fake_paged_launches()
    assert call(host, cache, **kw) == ARG, kw
    assert host.fake_paged_launches() == before
    said = host.mf_last_error().decode()
    assert "share" in said and name in said, said


def _taken(host, call, cache, **kw):
    before = host.fake_paged_launches()
    assert call(host, cache, **kw) == OK, (kw, host.mf_last_error())
    assert host.fake_paged_launches() == before + 1


def _need(host, Lq=1, H_q=32, H=8, d=128):
    n = ctypes.c_int64()
    assert host.mf_attn_paged_workspace(Lq, H_q, H, d, ctypes.byref(n)) == OK
    return n.value


def test_attention_takes_tensors_that_are_apart(host):
    need, c = _need(host), base._cache()
    _taken(host, base._attend, c)
    _taken(host, base._attend, c, lse=10 * PTR, slopes=11 * PTR)
    # side by side, to the byte; more workspace than is needed is not looked at
    end = PTR + PAGES
    _taken(host, base._attend, c, o=end, lse=end + 3 * 8192, ws=PTR - (need + 255) // 256 * 256, ws_bytes=need)
    _taken(host, base._attend, c, ws=PTR - (need + 255) // 256 * 256, ws_bytes=1 << 40)
    # rows of q and of o beside each other in one tensor
    _taken(host, base._attend, c, ld_q=8192, o=3 * PTR + 8192, ld_o=8192)
    scales = base._cache(k_scale=12 * PTR, v_scale=12 * PTR)  # (one for both)
    _taken(host, base._attend, scales)


@pytest.mark.parametrize("name,size,kw", [
    ("o", 3 * 8192, lambda x: dict(o=x)), ("lse", 3 * 32 * 4, lambda x: dict(lse=x)), ("workspace", 0, lambda x: dict(ws=x))])
def test_attention_refuses_outputs_over_its_inputs(host, name, size, kw):
    size = size or (_need(host) + 255) // 256 * 256
    k_scale, v_scale = 12 * PTR, 13 * PTR
    c = base._cache(k_scale=k_scale, v_scale=v_scale)
    inputs = dict(pages=(PTR, PAGES), q=(3 * PTR, 3 * 8192), lens=(5 * PTR, 12), table=(7 * PTR, 48), k_scale=(k_scale, 32),
                  v_scale=(v_scale, 32), slopes=(11 * PTR, 128))
    for other, (a, n) in inputs.items():
        step = 256 if name == "workspace" else 16
        for x in (a, a - size + step, a + (n - 1) // step * step):
            _refused(host, base._attend, c, name, slopes=11 * PTR, **kw(x))
        for x in (a - size, a + -(-n // step) * step):
            _taken(host, base._attend, c, slopes=11 * PTR, **kw(x))


def test_attention_refuses_outputs_over_each_other(host):
    need = (_need(host) + 255) // 256 * 256
    c = base._cache()
    for lse in (4 * PTR, 4 * PTR + 3 * 8192 - 4, 4 * PTR - 3 * 128 + 4):
        _refused(host, base._attend, c, "lse", lse=lse)
    for ws in (4 * PTR, 4 * PTR + 3 * 8192 - 256, 4 * PTR - need + 256):
        _refused(host, base._attend, c, "workspace", ws=ws)
    for lse in (9 * PTR, 9 * PTR + 4096):
        _refused(host, base._attend, c, "workspace", lse=lse)


FORMS = [dict(), dict(format=base.BF16)]


@pytest.mark.parametrize("form", FORMS)
def test_append_refuses_a_cache_over_what_it_reads(host, form):
    for at, size in ([(PTR, PAGES)] if not form else [(PTR, 640 * 2048), (2 * PTR, 640 * 2048)]):
        c = base._cache(**form)
        inputs = dict(seq=20, at=20, table=32, positions=20, turns=512, k_weight=256)
        for name, n in inputs.items():
            key = "w" if name == "k_weight" else name
            more = dict(norm=1) if key == "w" else {}
            for x in (at, at + size - 16, at - n // 16 * 16 + 16 - (16 if n % 16 else 0)):
                _refused(host, base._append, c, name, **{key: x}, **more)
            for x in (at + size, at - -(-n // 16) * 16):
                _taken(host, base._append, c, **{key: x}, **more)
    for name in ("k_scale", "v_scale"):
        _refused(host, base._append, base._cache(**{name: LAST}), name)
        _taken(host, base._append, base._cache(**{name: LAST + 16}))


def test_read_refuses_outputs_over_its_inputs(host):
    for out, name in (("k", "k_out"), ("v", "v_out")):
        for other, n in (("seq", 20), ("at", 20), ("table", 32)):
            x = {"k": 3, "v": 4}[out] * PTR
            for at in (x, x + 5 * 2048 - 4, x - n + 4):
                _refused(host, base._read, base._cache(), name, **{other: at})
            _taken(host, base._read, base._cache(), **{other: x + 5 * 2048})
            _taken(host, base._read, base._cache(), **{other: x - n})
        for scale in ("k_scale", "v_scale"):
            _refused(host, base._read, base._cache(**{scale: x + 64}), name)
    _taken(host, base._read, base._cache(), k=3 * PTR, ld_k=2048, v=3 * PTR + 2048, ld_v=2048)
