"""A paged cache and attention over it in 4 bits: host-side refusals (no GPU
needed), and the definitions that the GPU tests compare with."""
import ctypes

import pytest

from cross_model_attention_gb300 import build as build_mod
from cross_model_attention_gb300 import mapflow
from tests import paged_ref as ref

E = mapflow
PTR = 1 << 30  # an aligned address that host checks never follow
BF16, FP4 = mapflow.MF_CACHE_BF16, mapflow.MF_CACHE_FP4


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return mapflow.load_library()


def _cache(**kw):
    a = dict(format=FP4, page_size=64, H=8, d=128, n_pages=10, k=PTR, v=None, ld_k=0, ld_v=0, k_scale=None, v_scale=None)
    if kw.get("format") == BF16:
        a.update(v=2 * PTR, ld_k=1024, ld_v=1024)
    a.update(kw)
    return mapflow.CacheStruct(**a)


CACHES = [
    (dict(format=2), E.MF_ERR_ARG), (dict(format=-1), E.MF_ERR_ARG), (dict(d=96), E.MF_ERR_UNSUPPORTED),
    (dict(H=0), E.MF_ERR_ARG), (dict(H=1025), E.MF_ERR_ARG), (dict(page_size=0), E.MF_ERR_ARG),
    (dict(page_size=24), E.MF_ERR_ARG), (dict(page_size=-16), E.MF_ERR_ARG), (dict(n_pages=0), E.MF_ERR_ARG),
    (dict(n_pages=1 << 31), E.MF_ERR_ARG), (dict(k=None), E.MF_ERR_ARG), (dict(k=PTR + 8), E.MF_ERR_ARG),
    (dict(v=PTR), E.MF_ERR_ARG), (dict(k_scale=PTR + 2), E.MF_ERR_ARG), (dict(v_scale=PTR + 1), E.MF_ERR_ARG),
    (dict(format=BF16, v=None), E.MF_ERR_ARG), (dict(format=BF16, ld_k=1016), E.MF_ERR_ARG),
    (dict(format=BF16, ld_v=1028), E.MF_ERR_ARG), (dict(format=BF16, k_scale=3 * PTR), E.MF_ERR_ARG)]


def _append(lib, cache, **kw):
    a = dict(k=3 * PTR, ld_k=1024, v=4 * PTR, ld_v=1024, T=5, seq=5 * PTR, at=6 * PTR, table=7 * PTR, ld_table=4, n_seqs=2,
             max_pages=4, positions=None, turns=8 * PTR, rot=128, layout=0, gain=1.0, w=None, norm=0, eps=1e-6)
    a.update(kw)
    return lib.mf_cache_append(None if cache is None else ctypes.addressof(cache), a["k"], a["ld_k"], a["v"], a["ld_v"],
                               a["T"], a["seq"], a["at"], a["table"], a["ld_table"], a["n_seqs"], a["max_pages"],
                               a["positions"], a["turns"], a["rot"], a["layout"], a["gain"], a["w"], a["norm"], a["eps"],
                               None)


def _read(lib, cache, **kw):
    a = dict(T=5, seq=5 * PTR, at=6 * PTR, table=7 * PTR, ld_table=4, n_seqs=2, max_pages=4, k=3 * PTR, ld_k=1024,
             v=4 * PTR, ld_v=1024)
    a.update(kw)
    return lib.mf_cache_read(None if cache is None else ctypes.addressof(cache), a["T"], a["seq"], a["at"], a["table"],
                             a["ld_table"], a["n_seqs"], a["max_pages"], a["k"], a["ld_k"], a["v"], a["ld_v"], None)


def _attend(lib, cache, **kw):
    a = dict(n=3, Lq=1, H_q=32, q=3 * PTR, ld_q=4096, table=7 * PTR, ld_table=4, max_pages=4, lens=5 * PTR, o=4 * PTR,
             ld_o=4096, lse=None, slopes=None, softcap=0.0, window=0, n_sink=0, scale=0.1, ws=9 * PTR, ws_bytes=1 << 40)
    a.update(kw)
    return lib.mf_attn_paged(None if cache is None else ctypes.addressof(cache), a["n"], a["Lq"], a["H_q"], a["q"],
                             a["ld_q"], a["table"], a["ld_table"], a["max_pages"], a["lens"], a["o"], a["ld_o"], a["lse"],
                             a["slopes"], a["softcap"], a["window"], a["n_sink"], a["scale"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,code", CACHES)
def test_bad_caches_are_refused(lib, kw, code):
    c = _cache(**kw)
    for call in (_append, _read, _attend):
        got = call(lib, c)
        if call is _attend and kw.get("format") == BF16 and got == E.MF_ERR_UNSUPPORTED:
            continue
        assert got == code, call
        assert lib.mf_last_error().decode()


TABLES = [(dict(table=None), E.MF_ERR_ARG), (dict(table=7 * PTR + 2), E.MF_ERR_ARG), (dict(ld_table=3), E.MF_ERR_ARG),
          (dict(max_pages=0), E.MF_ERR_ARG), (dict(ld_table=(1 << 32) + 1), E.MF_ERR_UNSUPPORTED),
          (dict(max_pages=(1 << 20) + 1, ld_table=1 << 21), E.MF_ERR_UNSUPPORTED)]


@pytest.mark.parametrize("kw,code", TABLES + [
    (dict(T=-1), E.MF_ERR_ARG), (dict(n_seqs=0), E.MF_ERR_ARG), (dict(seq=None), E.MF_ERR_ARG), (dict(at=None), E.MF_ERR_ARG),
    (dict(seq=5 * PTR + 1), E.MF_ERR_ARG), (dict(k=None), E.MF_ERR_ARG), (dict(v=None), E.MF_ERR_ARG),
    (dict(k=3 * PTR + 8), E.MF_ERR_ARG), (dict(ld_k=1016), E.MF_ERR_ARG), (dict(ld_v=1028), E.MF_ERR_ARG),
    (dict(rot=-2), E.MF_ERR_ARG), (dict(rot=5), E.MF_ERR_ARG), (dict(rot=130), E.MF_ERR_ARG), (dict(layout=2), E.MF_ERR_ARG),
    (dict(turns=None), E.MF_ERR_ARG), (dict(turns=PTR + 4), E.MF_ERR_ARG), (dict(positions=PTR + 2), E.MF_ERR_ARG),
    (dict(gain=float("nan")), E.MF_ERR_ARG), (dict(norm=2), E.MF_ERR_ARG), (dict(norm=1, eps=0.0), E.MF_ERR_ARG),
    (dict(norm=1, eps=float("inf")), E.MF_ERR_ARG), (dict(w=PTR), E.MF_ERR_ARG), (dict(w=PTR + 2, norm=1), E.MF_ERR_ARG),
    (dict(k=PTR + 4096), E.MF_ERR_ARG), (dict(v=PTR - 4096), E.MF_ERR_ARG)])
def test_append_refuses(lib, kw, code):
    assert _append(lib, _cache(), **kw) == code
    assert lib.mf_last_error().decode()
    assert _append(lib, None) == E.MF_ERR_ARG


@pytest.mark.parametrize("kw,code", TABLES + [
    (dict(T=-1), E.MF_ERR_ARG), (dict(n_seqs=0), E.MF_ERR_ARG), (dict(seq=None), E.MF_ERR_ARG), (dict(at=6 * PTR + 3), E.MF_ERR_ARG),
    (dict(k=None), E.MF_ERR_ARG), (dict(v=4 * PTR + 4), E.MF_ERR_ARG), (dict(ld_k=1016), E.MF_ERR_ARG),
    (dict(k=PTR), E.MF_ERR_ARG), (dict(v=3 * PTR), E.MF_ERR_ARG), (dict(v=3 * PTR + 1024), E.MF_ERR_ARG)])
def test_read_refuses(lib, kw, code):
    assert _read(lib, _cache(), **kw) == code
    assert lib.mf_last_error().decode()
    assert _read(lib, None) == E.MF_ERR_ARG


def test_a_bf16_cache_apart_from_what_goes_in(lib):
    c = _cache(format=BF16)
    assert _append(lib, c, k=PTR + 2048) == E.MF_ERR_ARG
    assert _append(lib, c, v=2 * PTR) == E.MF_ERR_ARG
    assert _read(lib, c, k=2 * PTR + 64 * 2048) == E.MF_ERR_ARG
    assert _append(lib, _cache(format=BF16, v=PTR + 1024)) == E.MF_ERR_ARG  # its keys over its values


@pytest.mark.parametrize("kw,code", TABLES + [
    (dict(n=-1), E.MF_ERR_ARG), (dict(n=(1 << 20) + 1), E.MF_ERR_UNSUPPORTED), (dict(Lq=0), E.MF_ERR_ARG),
    (dict(H_q=12), E.MF_ERR_ARG), (dict(H_q=0), E.MF_ERR_ARG), (dict(H_q=2048), E.MF_ERR_UNSUPPORTED),
    (dict(Lq=33), E.MF_ERR_UNSUPPORTED), (dict(lens=None), E.MF_ERR_ARG), (dict(lens=PTR + 2), E.MF_ERR_ARG),
    (dict(lse=PTR + 2), E.MF_ERR_ARG), (dict(slopes=PTR + 1), E.MF_ERR_ARG), (dict(q=None), E.MF_ERR_ARG),
    (dict(o=None), E.MF_ERR_ARG), (dict(ld_q=4088), E.MF_ERR_ARG), (dict(ld_o=4100), E.MF_ERR_ARG),
    (dict(o=3 * PTR), E.MF_ERR_ARG), (dict(window=-1), E.MF_ERR_ARG), (dict(n_sink=-1), E.MF_ERR_ARG),
    (dict(scale=0.0), E.MF_ERR_ARG), (dict(scale=float("nan")), E.MF_ERR_ARG), (dict(softcap=-1.0), E.MF_ERR_ARG),
    (dict(softcap=float("inf")), E.MF_ERR_ARG), (dict(softcap=float("nan")), E.MF_ERR_ARG), (dict(ws=None), E.MF_ERR_ARG),
    (dict(softcap=1e-20, scale=1e15), E.MF_ERR_ARG), (dict(softcap=1e20, scale=1e-15), E.MF_ERR_ARG),
    (dict(ws=9 * PTR + 128), E.MF_ERR_ARG)])
def test_attend_refuses(lib, kw, code):
    assert _attend(lib, _cache(), **kw) == code
    assert lib.mf_last_error().decode()
    assert _attend(lib, None) == E.MF_ERR_ARG


def test_attention_takes_a_4_bit_cache(lib):
    assert _attend(lib, _cache(format=BF16)) == E.MF_ERR_UNSUPPORTED


def test_nothing_to_do_is_a_no_op(lib):
    assert _append(lib, _cache(), T=0, k=None, v=None, seq=None, at=None, table=None) == E.MF_OK
    assert _read(lib, _cache(), T=0, k=None, v=None, seq=None, at=None, table=None) == E.MF_OK
    assert _attend(lib, _cache(), n=0, q=None, o=None, table=None, lens=None, ws=None) == E.MF_OK


@pytest.mark.parametrize("args", [(0, 4, 2, 64), (1, 5, 2, 64), (1, 4, 2, 96), (65, 4, 2, 64), (1, 2048, 1024, 64)])
def test_workspace_refuses(lib, args):
    n = ctypes.c_int64()
    assert lib.mf_attn_paged_workspace(*args, ctypes.byref(n)) in (E.MF_ERR_ARG, E.MF_ERR_UNSUPPORTED)
    assert lib.mf_attn_paged_workspace(1, 4, 2, 64, None) == E.MF_ERR_ARG


def test_bindings_refuse_what_the_library_cannot_see(lib):
    torch = pytest.importorskip("torch")
    u8 = torch.zeros(2, 4, 18 * 64, dtype=torch.uint8)
    with pytest.raises(mapflow.MapFlowError):  # not on a GPU
        mapflow.PagedCache.fp4(u8, 16, 64)
    for args in ((u8, 24, 64), (u8, 16, 96), (u8, 0, 64), (u8.view(-1), 16, 64)):
        with pytest.raises(mapflow.MapFlowError):
            mapflow.PagedCache.fp4(*args)
    x = torch.zeros(2, 16, 4, 64, dtype=torch.bfloat16)
    for args in ((x, x.clone()), (x[0], x[0])):
        with pytest.raises(mapflow.MapFlowError):
            mapflow.PagedCache.bf16(*args)


def test_the_definition_by_hand():
    torch = pytest.importorskip("torch")
    one = torch.ones(1)
    x = torch.zeros(1, 32, dtype=torch.float64)
    x[0, 0] = 6.0  # scale 1: values are their own codes, halves between go to the even code
    x[0, 1:8] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    x[0, 8:12] = torch.tensor([-0.2500001, -4.9999, -5.0001, 0.74])
    code, s = ref.hold(x, one)
    assert s[0].tolist() == [0x38, 0]
    assert code[0, :12].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 9, 14, 15, 1]
    assert code[0, 16:].tolist() == [0] * 16
    assert ref.E4M3[0x38] == 1.0 and ref.E4M3[0x7e] == 448.0 and ref.E4M3[1] == 2.0 ** -9
    # a scale between 1 and 1.125 is rounded to the nearest, to even at the middle
    for top, byte in ((6.374, 0x38), (6.375, 0x38), (6.376, 0x39), (7.125, 0x3a), (1e6, 0x7e), (0.005, 0), (0.0059, 1)):
        y = torch.zeros(1, 16, dtype=torch.float64)
        y[0, 3] = -top
        assert ref.hold(y, one)[1][0, 0] == byte
    # a head's scale: the same codes for values of its size
    c3, s3 = ref.hold(3.0 * x, 3.0 * one)
    assert torch.equal(c3, code) and torch.equal(s3, s)
    x[0, 20] = float("nan")
    assert ref.hold(x, one)[1].tolist() == [[0x38, 0x7f]]


def test_packing_and_unpacking():
    torch = pytest.importorskip("torch")
    g = torch.Generator().manual_seed(1)
    for d, ps in ((64, 16), (128, 48)):
        kc, vc = (torch.randint(0, 16, (3, ps, 2, d), generator=g) for _ in range(2))
        ks, vs = (torch.randint(0, 256, (3, ps, 2, d // 16), generator=g) for _ in range(2))
        pages = ref.pack(kc, ks, vc, vs)
        assert pages.shape == (3, 2, ps // 16 * 18 * d)
        for a, b in zip((kc, ks, vc, vs), ref.unpack(pages, ps, d)):
            assert torch.equal(a, b.long())
        # token 9 of piece 0, head 1: its value's dimension 35 and that block's scale
        piece = pages[2, 1, : 18 * d]
        assert (int(piece[8 * d + 4 * d + 2 * 64 + 1 * 8 + 1]) >> 4) == int(vc[2, 9, 1, 35])
        assert int(piece[17 * d + 2 * 16 + 9]) == int(vs[2, 9, 1, 2])
        assert (int(piece[9 * (d // 2) + 17]) >> 4) == int(kc[2, 9, 1, 35])
        assert int(piece[16 * d + 9 * (d // 16) + 2]) == int(ks[2, 9, 1, 2])


@pytest.mark.parametrize("kw", [
    dict(n=1 << 20, max_pages=1 << 10, ld_table=1 << 10),                        # 2^20 requests of 2^16 keys
    dict(n=1 << 10, max_pages=1 << 20, ld_table=1 << 20),                        # 2^10 of 2^26
    dict(n=1 << 14, max_pages=1 << 15, ld_table=1 << 15, Lq=32, H_q=1024, ld_q=1 << 17, ld_o=1 << 17,  # 2^30 tiles of
         cache=dict(H=256))])                                                    # 256 heads of 8 groups of 16 rows
def test_more_keys_than_a_call_counts_are_refused(lib, kw):
    kw = dict(kw)
    c = _cache(**kw.pop("cache", {}))
    assert _attend(lib, c, **dict(kw, q=1 << 44, o=1 << 45)) == E.MF_ERR_UNSUPPORTED
    assert "too many keys" in lib.mf_last_error().decode()


def test_calls_with_their_arguments_in_one_piece(lib):
    """The struct forms check and refuse as the plain calls do, field by field."""
    good, bad = _cache(), _cache(d=96)

    def append(cache=good, k=3 * PTR, ld_k=1024, v=4 * PTR, ld_v=1024, seq=5 * PTR, at=6 * PTR, table=7 * PTR, ld_table=4,
               positions=0, turns=8 * PTR, w=0, gain=1.0, eps=1e-6, T=5, n_seqs=2, max_pages=4, rot=128, layout=0, norm=0):
        return lib.mf_cache_append_args(mapflow._append_args(
            ctypes.addressof(cache), k, ld_k, v, ld_v, seq, at, table, ld_table, positions, turns, w, 0, gain, eps, T, n_seqs,
            max_pages, rot, layout, norm))

    def read(cache=good, seq=5 * PTR, at=6 * PTR, table=7 * PTR, ld_table=4, k=3 * PTR, ld_k=1024, v=4 * PTR, ld_v=1024, T=5,
             n_seqs=2, max_pages=4):
        return lib.mf_cache_read_args(mapflow._read_args(ctypes.addressof(cache), seq, at, table, ld_table, k, ld_k, v, ld_v,
                                                         0, T, n_seqs, max_pages, 0))

    def attend(cache=good, q=3 * PTR, ld_q=4096, table=7 * PTR, ld_table=4, lens=5 * PTR, o=4 * PTR, ld_o=4096, lse=0, slopes=0,
               ws=9 * PTR, ws_bytes=1 << 40, softcap=0.0, scale=0.1, n=3, Lq=1, H_q=32, max_pages=4, window=0, n_sink=0):
        return lib.mf_attn_paged_args(mapflow._paged_args(
            ctypes.addressof(cache), q, ld_q, table, ld_table, lens, o, ld_o, lse, slopes, ws, ws_bytes, 0, softcap, scale, n,
            Lq, H_q, max_pages, window, n_sink))

    def fails(call, word, code=E.MF_ERR_ARG, **kw):
        assert call(**kw) == code, (word, kw)
        assert word in lib.mf_last_error().decode(), (word, lib.mf_last_error())

    assert append(T=0) == read(T=0) == attend(n=0) == E.MF_OK
    for call in (append, read, attend):
        fails(call, "d = 96", E.MF_ERR_UNSUPPORTED, cache=bad)
        fails(call, "max_pages", max_pages=0)
        fails(call, "table", table=0)
        fails(call, "table", ld_table=3)
    for call in (append, read):
        for name in ("seq", "at"):
            fails(call, name, **{name: 0})
            fails(call, name, **{name: PTR + 1})
        fails(call, "k", k=0), fails(call, "v", v=0), fails(call, "k", ld_k=1016), fails(call, "v", ld_v=1028)
        fails(call, "T must", T=-1)
        fails(call, "no rows", n_seqs=0)
    fails(append, "positions", positions=PTR + 2), fails(append, "turns", turns=0), fails(append, "k_weight", w=PTR + 2, norm=1)
    fails(append, "weight without", w=PTR), fails(append, "gain", gain=float("inf")), fails(append, "gain", gain=1e300)
    fails(append, "eps", norm=1, eps=0.0), fails(append, "eps", norm=1, eps=1e300), fails(append, "rot_dim", rot=7)
    fails(append, "layout", layout=2), fails(append, "norm", norm=2)
    fails(attend, "q", q=0), fails(attend, "q", ld_q=4088), fails(attend, "lens", lens=0), fails(attend, "o", o=0)
    fails(attend, "o", ld_o=4100), fails(attend, "lse", lse=PTR + 2), fails(attend, "slopes", slopes=PTR + 1)
    fails(attend, "workspace", ws=0), fails(attend, "softcap", softcap=-1.0), fails(attend, "softcap", softcap=1e300)
    fails(attend, "scale", scale=0.0), fails(attend, "scale", scale=1e300), fails(attend, "n must", n=-1)
    fails(attend, "Lq", Lq=0), fails(attend, "H_q", H_q=12), fails(attend, "window", window=-1), fails(attend, "n_sink", n_sink=-1)
    for call in (lib.mf_cache_append_args, lib.mf_cache_read_args, lib.mf_attn_paged_args):
        assert call(None) == E.MF_ERR_ARG
