"""Refusals of the C ABI's calls over a cache of 8 bits, which come before anything touches a GPU."""

import ctypes

import pytest

from test_serving_abi import BAD_CACHES, Pages

P = ctypes.c_void_p
ARG = -1


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_draft_stream_gb300 import build
    from speculative_decoding_draft_stream_gb300.nanospec import load_library

    return load_library(build.build())


class Scales(ctypes.Structure):
    _fields_ = ([(n, P) for n in ("k", "v")] +
                [(f"{t}_{n}", ctypes.c_int64) for t in "kv" for n in ("layer", "page", "head")])


def cache(**kw):
    a = dict(k=16, v=16, k_layer=65536, k_page=4096, k_head=2048, k_token=128, v_layer=65536, v_page=4096, v_head=2048,
             v_token=128, layers=2, pages=16, heads=2, page_size=16, row_bytes=128, max_seqs=4, table_ld=8, table=16,
             lengths=16, refs=16)
    a.update(kw)
    return ctypes.byref(Pages(**a))


def scales(**kw):
    a = dict(k=8, v=16, k_layer=512, k_page=32, k_head=16, v_layer=512, v_page=32, v_head=16)
    a.update(kw)
    return ctypes.byref(Scales(**a))


def calls(lib, c, s):
    yield lib.ns_pages_extend_scaled(c, s, P(16), P(16), 1, P(16), 1 << 40, None)
    yield lib.ns_pages_compact_scaled(c, s, P(16), P(16), P(16), 4, P(16), 1, None)
    yield lib.ns_pages_copy_scaled(c, s, P(16), P(16), 1, None)
    yield lib.ns_pages_write_scaled(c, s, 0, P(16), P(16), 1, P(16), P(16), 0, 256, 128, 256, 128, 4, None)
    yield lib.ns_pages_read(c, s, 0, P(16), P(16), 1, P(16), P(16), 0, 256, 128, 256, 128, 4, None)


@pytest.mark.parametrize("kw", BAD_CACHES + [dict(row_bytes=96), dict(row_bytes=256), dict(page_size=12)])
def test_a_bad_cache_is_refused(lib, kw):
    assert all(r == ARG for r in calls(lib, cache(**kw), scales()))


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(k=12), dict(v=20), dict(k_layer=4), dict(k_page=1),
                                dict(k_head=12), dict(v_layer=2), dict(v_page=4), dict(v_head=9)])
def test_bad_exponents_are_refused(lib, kw):
    assert all(r == ARG for r in calls(lib, cache(), scales(**kw)))


def test_no_exponents_are_refused_where_they_are_needed(lib):
    c = cache()
    assert lib.ns_pages_extend_scaled(c, None, P(16), P(16), 1, P(16), 1 << 40, None) == ARG
    assert lib.ns_pages_compact_scaled(c, None, P(16), P(16), P(16), 4, P(16), 1, None) == ARG
    assert lib.ns_pages_copy_scaled(c, None, P(16), P(16), 1, None) == ARG
    assert lib.ns_pages_write_scaled(c, None, 0, P(16), P(16), 1, P(16), P(16), 0, 256, 128, 256, 128, 4, None) == ARG


@pytest.mark.parametrize("f", ["write", "read"])
def test_bad_rows_are_refused(lib, f):
    def call(**kw):
        a = dict(layer=0, seqs=16, cu=16, n=1, k=16, v=16, dtype=0, kt=256, kh=128, vt=256, vh=128, tokens=4)
        a.update(kw)
        g = lib.ns_pages_write_scaled if f == "write" else lib.ns_pages_read
        return g(cache(), scales(), a["layer"], P(a["seqs"]), P(a["cu"]), a["n"], P(a["k"]), P(a["v"]), a["dtype"],
                 a["kt"], a["kh"], a["vt"], a["vh"], a["tokens"], None)

    for kw in (dict(layer=-1), dict(layer=2), dict(seqs=None), dict(cu=None), dict(seqs=18), dict(cu=17), dict(n=-1),
               dict(n=8193), dict(k=None), dict(v=None), dict(k=24), dict(v=8), dict(dtype=2), dict(dtype=-1),
               dict(kt=8), dict(kh=4), dict(vt=24), dict(vh=2), dict(tokens=-1)):
        assert call(**kw) == ARG, kw
    assert call(tokens=0, k=None) == 0 and call(n=0, seqs=None) == 0


def attend(lib, **kw):
    a = dict(q=16, dtype=0, B=1, n=1, hq=8, hkv=2, dim=64, qs=512, qt=512, qh=64, k=16, v=16, pages=4, page=16,
             kp=2048, kh=1024, kt=64, vp=2048, vh=1024, vt=64, ke=8, ve=8, kep=32, keh=16, vep=32, veh=16, table=16,
             ld=4, seqs=1, lengths=16, ids=16, mask=None, scale=0.125, most=0, out=16, lse=16, ws=16, bytes=1 << 40)
    a.update(kw)
    return lib.ns_attend_paged_scaled(
        P(a["q"]), a["dtype"], a["B"], a["n"], a["hq"], a["hkv"], a["dim"], a["qs"], a["qt"], a["qh"], P(a["k"]),
        P(a["v"]), a["pages"], a["page"], a["kp"], a["kh"], a["kt"], a["vp"], a["vh"], a["vt"], P(a["ke"]), P(a["ve"]),
        a["kep"], a["keh"], a["vep"], a["veh"], P(a["table"]), a["ld"], a["seqs"], P(a["lengths"]), P(a["ids"]),
        P(a["mask"]), ctypes.c_float(a["scale"]), a["most"], P(a["out"]), P(a["lse"]), P(a["ws"]), a["bytes"], None)


@pytest.mark.parametrize("kw", [
    dict(ke=None), dict(ve=None), dict(ke=4), dict(ve=12), dict(kep=4), dict(keh=1), dict(vep=2), dict(veh=12),
    dict(kp=2056), dict(kh=8), dict(kt=72), dict(vp=8), dict(vh=24), dict(vt=8), dict(dtype=2), dict(dim=96),
    dict(page=4), dict(k=8), dict(scale=0.0), dict(n=65), dict(ld=1 << 27),
])
def test_attention_refuses(lib, kw):
    assert attend(lib, **kw) == ARG


def test_attention_of_nothing_is_done(lib):
    assert attend(lib, B=0, ke=None) == 0
