"""Rotary embedding with head norms, window attention with sinks and
shared-prefix attention: host-side refusals (no GPU needed)."""
import ctypes

import numpy as np
import pytest

from cross_model_attention_gb300 import build as build_mod
from cross_model_attention_gb300 import mapflow
from tests import layer_ref as ref

E = mapflow
PTR = 1 << 20  # an aligned address that host checks never follow


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return mapflow.load_library()


@pytest.mark.parametrize("rot,base,scaling,factor,orig", [
    (128, 10000.0, "none", 1.0, 0), (64, 1e6, "linear", 4.0, 0), (2, 10000.0, "ntk", 2.0, 0),
    (96, 10000.0, "ntk", 8.0, 0), (128, 1e6, "yarn", 8.0, 32768), (20, 10000.0, "yarn", 2.0, 17)])
def test_frequencies(lib, rot, base, scaling, factor, orig):
    turns, gain = mapflow.mf_rope_frequencies(rot, base, scaling, factor, orig)
    f, g = ref.rope_frequencies(rot, base, scaling, factor, orig)
    got = turns.astype(np.float64) * 2.0 ** -64 * 2 * np.pi
    # a pow and a handful of fp64 operations on each side; the table's 64-bit
    # fraction is rounded to half a unit, 2^-65 of a turn
    np.testing.assert_allclose(got, f.numpy(), rtol=1e-14, atol=2.0 ** -65 * 2 * np.pi)
    assert abs(gain - g) <= 2.0 ** -24 * g


@pytest.mark.parametrize("kw", [
    dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=-2), dict(base=1.0), dict(base=float("inf")),
    dict(base=float("nan")), dict(scaling="linear", factor=0.5), dict(scaling="linear", factor=float("inf")),
    dict(scaling="yarn", factor=2.0), dict(scaling="yarn", factor=2.0, original_length=64, beta_slow=0.0),
    dict(scaling="yarn", factor=2.0, original_length=64, beta_fast=1.0, beta_slow=2.0), dict(scaling="other")])
def test_frequencies_refuse(lib, kw):
    args = dict(rot_dim=64)
    args.update(kw)
    with pytest.raises(mapflow.MapFlowError) as ei:
        mapflow.mf_rope_frequencies(**args)
    assert ei.value.code == E.MF_ERR_ARG


def _rope(lib, **kw):
    a = dict(q=PTR, ld_q=512, q_out=2 * PTR, ld_qo=512, k=3 * PTR, ld_k=256, k_out=4 * PTR, ld_ko=256, wq=None,
             wk=None, norm=0, eps=1e-6, pos=5 * PTR, turns=6 * PTR, rot=128, layout=0, gain=1.0,
             dtype=E.MF_DTYPE_BF16, T=10, H_q=4, H_k=2, d=128)
    a.update(kw)
    f = ctypes.c_float
    return lib.mf_qk_norm_rope(a["q"], a["ld_q"], a["q_out"], a["ld_qo"], a["k"], a["ld_k"], a["k_out"], a["ld_ko"],
                               a["wq"], a["wk"], a["norm"], f(a["eps"]), a["pos"], a["turns"], a["rot"], a["layout"],
                               f(a["gain"]), a["dtype"], a["T"], a["H_q"], a["H_k"], a["d"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), E.MF_ERR_ARG), (dict(q_out=None), E.MF_ERR_ARG), (dict(k=None), E.MF_ERR_ARG),
    (dict(pos=None), E.MF_ERR_ARG), (dict(turns=None), E.MF_ERR_ARG),
    (dict(pos=7 * PTR + 2), E.MF_ERR_ARG), (dict(turns=7 * PTR + 4), E.MF_ERR_ARG), (dict(q=PTR + 8), E.MF_ERR_ARG),
    (dict(ld_q=511), E.MF_ERR_ARG), (dict(ld_q=516), E.MF_ERR_ARG), (dict(ld_k=248), E.MF_ERR_ARG),
    (dict(rot=0), E.MF_ERR_ARG), (dict(rot=5), E.MF_ERR_ARG), (dict(rot=130), E.MF_ERR_ARG),
    (dict(layout=2), E.MF_ERR_ARG), (dict(norm=2), E.MF_ERR_ARG), (dict(norm=1, eps=0.0), E.MF_ERR_ARG),
    (dict(norm=1, eps=float("nan")), E.MF_ERR_ARG), (dict(wq=7 * PTR), E.MF_ERR_ARG), (dict(wq=7 * PTR + 2, norm=1), E.MF_ERR_ARG),
    (dict(gain=float("inf")), E.MF_ERR_ARG), (dict(dtype=3), E.MF_ERR_ARG), (dict(T=-1), E.MF_ERR_ARG),
    (dict(H_q=0), E.MF_ERR_ARG), (dict(H_k=-1), E.MF_ERR_ARG), (dict(d=96), E.MF_ERR_UNSUPPORTED),
    (dict(q_out=PTR + 1024), E.MF_ERR_ARG),            # shifted over q
    (dict(q_out=PTR, ld_qo=520), E.MF_ERR_ARG),        # q's memory with another stride
    (dict(k_out=PTR), E.MF_ERR_ARG),                   # over q
    (dict(k_out=2 * PTR), E.MF_ERR_ARG),               # over q_out
    (dict(ld_q=768, ld_qo=768, q_out=PTR + 512, k=PTR + 1024, ld_k=768), E.MF_ERR_ARG),
])
def test_rope_refuses(lib, kw, code):
    assert _rope(lib, **kw) == code
    assert lib.mf_last_error().decode()


def test_rope_of_no_tokens_is_a_no_op(lib):
    assert _rope(lib, T=0, q=None, q_out=None, k=None, k_out=None) == E.MF_OK


def _packed(lib, cu=(0, 100), qb=None, H_q=4, H_kv=2, d=128, window=0, sinks=0, alloc=None, free=None):
    h = ctypes.c_void_p()
    cu = np.asarray(cu, np.int32)
    qb = None if qb is None else np.asarray(qb, np.int32)
    A, F = alloc or mapflow.ALLOC_FN(), free or mapflow.FREE_FN()
    return lib.mf_attn_create_packed(ctypes.byref(h), cu.ctypes.data, None if qb is None else qb.ctypes.data,
                                     len(cu) - 1, H_q, H_kv, d, window, sinks, A, F, None)


@pytest.mark.parametrize("kw,code", [
    (dict(cu=[0, 100, 50]), E.MF_ERR_ARG), (dict(cu=[1, 100]), E.MF_ERR_ARG), (dict(cu=[0, 0]), E.MF_ERR_ARG),
    (dict(cu=[0]), E.MF_ERR_ARG), (dict(H_q=3, H_kv=2), E.MF_ERR_ARG), (dict(H_kv=0), E.MF_ERR_ARG),
    (dict(d=96), E.MF_ERR_UNSUPPORTED), (dict(H_q=258, H_kv=2), E.MF_ERR_UNSUPPORTED),
    (dict(H_q=2048, H_kv=2048), E.MF_ERR_UNSUPPORTED), (dict(window=-1), E.MF_ERR_ARG),
    (dict(sinks=-1), E.MF_ERR_ARG), (dict(qb=[101]), E.MF_ERR_ARG), (dict(qb=[-1]), E.MF_ERR_ARG),
    (dict(qb=[100]), E.MF_ERR_ARG), (dict(cu=[0, (1 << 29) + 1]), E.MF_ERR_UNSUPPORTED),
    (dict(cu=[0, (1 << 26) + 1]), E.MF_ERR_UNSUPPORTED),
    (dict(cu=[i << 26 for i in range(8)] + [(7 << 26) + 5], H_q=64, H_kv=64), E.MF_ERR_UNSUPPORTED),  # 2^27 runs
    (dict(alloc=mapflow.ALLOC_FN(lambda n, c, s: None)), E.MF_ERR_ARG)])
def test_packed_plan_refuses(lib, kw, code):
    assert _packed(lib, **kw) == code
    assert lib.mf_last_error().decode()


@pytest.mark.parametrize("kw,code", [
    (dict(n=0), E.MF_ERR_ARG), (dict(Lq=0), E.MF_ERR_ARG), (dict(cap=0), E.MF_ERR_ARG), (dict(P=-1), E.MF_ERR_ARG),
    (dict(P=10, window=5), E.MF_ERR_UNSUPPORTED), (dict(P=10, sinks=5), E.MF_ERR_UNSUPPORTED),
    (dict(Lq=65), E.MF_ERR_UNSUPPORTED), (dict(n=70000, cap=70000), E.MF_ERR_UNSUPPORTED),
    (dict(n=1 << 22), E.MF_ERR_UNSUPPORTED), (dict(cap=(1 << 26) + 1), E.MF_ERR_UNSUPPORTED),
    (dict(P=(1 << 26) + 1), E.MF_ERR_UNSUPPORTED),
    (dict(d=32), E.MF_ERR_UNSUPPORTED), (dict(H_q=5), E.MF_ERR_ARG)])
def test_cache_plan_refuses(lib, kw, code):
    a = dict(n=2, Lq=1, cap=64, P=0, H_q=4, H_kv=2, d=128, window=0, sinks=0)
    a.update(kw)
    h = ctypes.c_void_p()
    rc = lib.mf_attn_create_cache(ctypes.byref(h), a["n"], a["Lq"], a["cap"], a["P"], a["H_q"], a["H_kv"], a["d"],
                                  a["window"], a["sinks"], mapflow.ALLOC_FN(), mapflow.FREE_FN(), None)
    assert rc == code
    assert lib.mf_last_error().decode()


def test_null_handles(lib):
    f = ctypes.c_float
    n = ctypes.c_int64()
    assert lib.mf_attn_create_packed(None, None, None, 1, 1, 1, 64, 0, 0, mapflow.ALLOC_FN(), mapflow.FREE_FN(),
                                     None) == E.MF_ERR_ARG
    assert lib.mf_attn_create_cache(None, 1, 1, 1, 0, 1, 1, 64, 0, 0, mapflow.ALLOC_FN(), mapflow.FREE_FN(),
                                    None) == E.MF_ERR_ARG
    assert lib.mf_attn_packed(None, None, 0, None, 0, None, 0, None, 0, None, 1, f(1), None, 0, None) == E.MF_ERR_ARG
    assert lib.mf_attn_cached(None, 1, None, 0, None, 0, None, 0, None, None, 0, None, 0, None, 0, None, 1, f(1),
                              None, 0, None) == E.MF_ERR_ARG
    assert lib.mf_attn_workspace(None, 1, ctypes.byref(n)) == E.MF_ERR_ARG
    assert lib.mf_attn_status(None, None) == E.MF_ERR_ARG
    lib.mf_attn_destroy(None)


def test_bindings_refuse_what_the_library_cannot_see(lib):
    torch = pytest.importorskip("torch")
    with pytest.raises(mapflow.MapFlowError):
        mapflow.RotaryPlan(64, layout="other", device="cpu")
    plan = mapflow.RotaryPlan(64, device="cpu")
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(mapflow.MapFlowError):  # not on a GPU
        plan.apply(x, x.clone(), torch.zeros(4, dtype=torch.int32))
    with pytest.raises(TypeError):
        plan.apply(x.half(), None, torch.zeros(4, dtype=torch.int32))
    for kw in (dict(window=0), dict(window=-3), dict(q_begin=[0, 0])):
        with pytest.raises(mapflow.MapFlowError):
            mapflow.WindowAttention([0, 4], 2, 2, 64, **kw)
    with pytest.raises(mapflow.MapFlowError):
        mapflow.CacheAttention(1, 1, 4, 2, 2, 64, window=0)
