"""More host-side tests of the rotary and attention layers (no GPU needed)."""
import numpy as np
import pytest

from cross_model_attention_gb300 import build as build_mod
from cross_model_attention_gb300 import mapflow

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    build_mod.build()


class Seen(Exception):
    pass


@pytest.fixture
def ask(monkeypatch):
    """Makes a plan as far as the library's create call and returns the integers it got."""
    class Lib:
        mf_attn_packed = mf_attn_cached = None

        @staticmethod
        def mf_attn_create_packed(out, cu, qb, *rest):
            raise Seen(rest[:6])

        @staticmethod
        def mf_attn_create_cache(out, *rest):
            raise Seen(rest[:9])
    monkeypatch.setattr(mapflow, "load_library", lambda: Lib)
    monkeypatch.setattr(mapflow, "_torch_allocator", lambda: (None, None))

    def run(cls, *args, **kw):
        with pytest.raises(Seen) as e:
            cls(*args, **kw)
        return e.value.args[0]
    return run


@pytest.mark.parametrize("far", [2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 1, 2 ** 63, 10 ** 30])
def test_windows_and_sinks_past_32_bits_hide_nothing(ask, far):
    got = ask(mapflow.WindowAttention, [0, 9], 4, 2, 64, window=far, sinks=far)
    assert got == (1, 4, 2, 64, 2 ** 31 - 1, 2 ** 31 - 1)
    got = ask(mapflow.CacheAttention, 2, 1, 9, 4, 2, 64, window=far, sinks=far)
    assert got == (2, 1, 9, 0, 4, 2, 64, 2 ** 31 - 1, 2 ** 31 - 1)
    assert ask(mapflow.WindowAttention, [0, 9], 4, 2, 64)[4:] == (0, 0)


def refused(make):
    with pytest.raises(mapflow.MapFlowError) as e:
        make()
    assert e.value.code == mapflow.MF_ERR_ARG


@pytest.mark.parametrize("name", ["n", "Lq", "capacity", "prefix_len", "H_q", "H_kv", "d"])
@pytest.mark.parametrize("extra", [2 ** 31, 2 ** 32])
def test_sizes_past_32_bits_are_refused(name, extra):
    a = dict(n=1, Lq=1, capacity=8, prefix_len=0, H_q=4, H_kv=2, d=64)
    a[name] += extra
    refused(lambda: mapflow.CacheAttention(**a))
    if name in ("H_q", "H_kv", "d"):
        refused(lambda: mapflow.WindowAttention([0, 9], a["H_q"], a["H_kv"], a["d"]))


def test_offsets_past_32_bits_are_refused():
    for cu in ([0, 2 ** 32 + 5], np.array([0, 2 ** 32 + 5]), np.array([0, 2 ** 31])):
        refused(lambda: mapflow.WindowAttention(cu, 4, 2, 64))
    refused(lambda: mapflow.WindowAttention([0, 9], 4, 2, 64, q_begin=np.array([2 ** 32])))
    refused(lambda: mapflow.WindowAttention([0, 9], 4, 2, 64, sinks=-1))
    refused(lambda: mapflow.mf_rope_frequencies(2 ** 32 + 64))
    refused(lambda: mapflow.mf_rope_frequencies(64, scaling="yarn", factor=2.0, original_length=2 ** 32 + 4096))
