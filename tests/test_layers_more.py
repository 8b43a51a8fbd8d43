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
    for cu in ([0, 2 ** 32 + 5], np.array([0, 2 ** 32 + 5]), np.array([0, 2 ** 31]), np.array([-2 ** 63, 9])):
        refused(lambda: mapflow.WindowAttention(cu, 4, 2, 64))
    refused(lambda: mapflow.WindowAttention([0, 9], 4, 2, 64, q_begin=np.array([2 ** 32])))
    refused(lambda: mapflow.WindowAttention([0, 9], 4, 2, 64, sinks=-1))
    refused(lambda: mapflow.mf_rope_frequencies(2 ** 32 + 64))
    refused(lambda: mapflow.mf_rope_frequencies(64, scaling="yarn", factor=2.0, original_length=2 ** 32 + 4096))


@pytest.mark.parametrize("rot,base", [(128, 10000.0), (128, 1e6), (96, 500000.0), (20, 10000.0), (2, 10000.0)])
def test_table_entries_are_off_by_their_fp64_rounding_alone(rot, base):
    """Against 50 digits.  The exponent x = 2 i / rot is rounded (ln(base) x 2^-53
    of the power), the power is off by at most one step (2^-52), 2 pi and the
    division by half a step each (2^-53), and the entry is rounded to a whole."""
    from decimal import Decimal, getcontext
    getcontext().prec = 50
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510")
    turns, _ = mapflow.mf_rope_frequencies(rot, base)
    ln = Decimal(base).ln()
    for i, t in enumerate(turns):
        x = Decimal(2 * i) / rot
        want = (-x * ln).exp() / two_pi * 2 ** 64
        bound = want * (4 + ln * x) / 2 ** 53 + Decimal("0.5")
        assert abs(int(t) - want) <= bound, i
        # as an angle at the farthest position: what the header says
        assert abs(int(t) - want) / 2 ** 64 * two_pi * 2 ** 31 < Decimal("1e-6") + two_pi / 2 ** 34, i


def test_by_parts_scaling_leaves_pair_0():
    """Also where every pair turns less than beta_slow times in the original length."""
    plain, _ = mapflow.mf_rope_frequencies(64)
    for length in (1, 4, 100, 4096):
        t, _ = mapflow.mf_rope_frequencies(64, scaling="yarn", factor=4.0, original_length=length)
        assert t[0] == plain[0] and (t <= plain).all()
    t, _ = mapflow.mf_rope_frequencies(64, scaling="yarn", factor=4.0, original_length=4)
    np.testing.assert_allclose(t[1:].astype(np.float64), plain[1:] / 4.0, rtol=1e-14)
