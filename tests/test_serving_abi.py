"""Refusals of the serving operators' C ABI, which come before anything touches a GPU."""

import ctypes
import os

import pytest

P = ctypes.c_void_p
ARG = -1


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_draft_stream_gb300 import build
    from speculative_decoding_draft_stream_gb300.nanospec import load_library

    return load_library(build.build())


def prompt(lib, **kw):
    a = dict(q=16, k=16, v=16, dtype=0, tokens=10, hq=8, hkv=2, dim=64, qt=512, qh=64, kt=128, kh=64, vt=128, vh=64,
             cu=16, n=1, most=10, scale=0.125, out=16, lse=16)
    a.update(kw)
    return lib.ns_attend_prompt(P(a["q"]), P(a["k"]), P(a["v"]), a["dtype"], a["tokens"], a["hq"], a["hkv"], a["dim"],
                                a["qt"], a["qh"], a["kt"], a["kh"], a["vt"], a["vh"], P(a["cu"]), a["n"], a["most"],
                                ctypes.c_float(a["scale"]), P(a["out"]), P(a["lse"]), None)


def paged(lib, **kw):
    a = dict(q=16, dtype=0, B=1, n=1, hq=8, hkv=2, dim=64, qs=512, qt=512, qh=64, k=16, v=16, pages=4, page=16,
             kp=2048, kh=1024, kt=64, vp=2048, vh=1024, vt=64, table=16, ld=4, seqs=1, lengths=16, ids=16, mask=None,
             scale=0.125, most=0, out=16, lse=16, ws=16, bytes=1 << 40)
    a.update(kw)
    return lib.ns_attend_paged(P(a["q"]), a["dtype"], a["B"], a["n"], a["hq"], a["hkv"], a["dim"], a["qs"], a["qt"],
                               a["qh"], P(a["k"]), P(a["v"]), a["pages"], a["page"], a["kp"], a["kh"], a["kt"],
                               a["vp"], a["vh"], a["vt"], P(a["table"]), a["ld"], a["seqs"], P(a["lengths"]),
                               P(a["ids"]), P(a["mask"]), ctypes.c_float(a["scale"]), a["most"], P(a["out"]),
                               P(a["lse"]), P(a["ws"]), a["bytes"], None)


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(dim=96), dict(dim=0), dict(hq=9), dict(hkv=0), dict(hq=0), dict(tokens=-1), dict(n=-1),
    dict(most=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(q=None), dict(k=None), dict(v=None), dict(cu=None), dict(out=None), dict(q=18), dict(k=24), dict(v=8),
    dict(out=20), dict(lse=18), dict(cu=18), dict(qt=516), dict(qh=0), dict(kt=-128), dict(kh=0), dict(vt=4),
    dict(vh=1 << 39),
])
def test_prompt_refuses(lib, kw):
    assert prompt(lib, **kw) == ARG


@pytest.mark.parametrize("kw", [dict(tokens=0), dict(n=0), dict(most=0)])
def test_prompt_of_nothing_is_done(lib, kw):
    assert prompt(lib, **kw) == 0


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(dim=32), dict(hq=7), dict(B=-1), dict(B=4097), dict(n=0), dict(n=65), dict(pages=0),
    dict(page=4), dict(page=24), dict(page=2048), dict(ld=0), dict(seqs=0), dict(ld=1 << 27), dict(most=-1),
    dict(scale=0.0), dict(scale=float("nan")), dict(q=None), dict(k=None), dict(v=None), dict(table=None),
    dict(lengths=None), dict(ids=None), dict(out=None), dict(ws=None), dict(q=18), dict(k=24), dict(v=24),
    dict(mask=20), dict(ws=24), dict(lse=18), dict(out=18), dict(out=20), dict(out=24), dict(qs=511), dict(qt=3), dict(qh=1), dict(kp=2049), dict(kh=4),
    dict(kt=2), dict(vp=12), dict(vh=12), dict(vt=12),
])
def test_paged_refuses(lib, kw):
    assert paged(lib, **kw) == ARG


def test_paged_of_nothing_is_done(lib):
    assert paged(lib, B=0) == 0


def test_workspaces_of_bad_calls_are_nothing(lib):
    for a in ((-1, 1, 8, 2, 64), (4097, 1, 8, 2, 64), (1, 0, 8, 2, 64), (1, 65, 8, 2, 64), (1, 1, 8, 3, 64), (1, 1, 8, 2, 80)):
        assert lib.ns_attend_paged_workspace(*a) == 0


class Pages(ctypes.Structure):
    _fields_ = ([(n, P) for n in ("k", "v")] +
                [(f"{t}_{n}", ctypes.c_int64) for t in "kv" for n in ("layer", "page", "head", "token")] +
                [(n, ctypes.c_int32) for n in ("layers", "pages", "heads", "page_size", "row_bytes", "max_seqs",
                                               "table_ld")] +
                [(n, P) for n in ("table", "lengths", "refs")])


def cache(**kw):
    a = dict(k=16, v=16, k_layer=65536, k_page=4096, k_head=2048, k_token=128, v_layer=65536, v_page=4096, v_head=2048,
             v_token=128, layers=2, pages=16, heads=2, page_size=16, row_bytes=128, max_seqs=4, table_ld=8, table=16,
             lengths=16, refs=16)
    a.update(kw)
    return ctypes.byref(Pages(**a))


BAD_CACHES = [
    dict(k=None), dict(v=None), dict(table=None), dict(lengths=None), dict(refs=None), dict(k=8), dict(v=24),
    dict(table=18), dict(k_layer=8), dict(k_page=4), dict(k_head=8), dict(v_token=8), dict(layers=0), dict(pages=0),
    dict(heads=0), dict(page_size=0), dict(row_bytes=0), dict(row_bytes=24), dict(max_seqs=0), dict(table_ld=0),
]


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_pages_refuse_a_bad_cache(lib, kw):
    c = cache(**kw)
    assert lib.ns_pages_truncate(c, P(16), P(16), 1, None) == ARG
    assert lib.ns_pages_fork(c, P(16), P(16), 1, None) == ARG
    assert lib.ns_pages_extend(c, P(16), P(16), 1, P(16), 1 << 40, None) == ARG
    assert lib.ns_pages_write(c, 0, P(16), P(16), 1, P(16), P(16), 256, 128, 256, 128, 4, None) == ARG
    assert lib.ns_pages_compact(c, P(16), P(16), P(16), 4, P(16), 1, None) == ARG
    assert lib.ns_pages_copy(c, P(16), P(16), 1, None) == ARG
    assert lib.ns_pages_workspace(c, 1) == 0


def test_pages_refuse_bad_calls(lib):
    c = cache()
    many = 8193
    assert lib.ns_pages_truncate(None, P(16), P(16), 1, None) == ARG
    assert lib.ns_pages_truncate(c, None, P(16), 1, None) == ARG
    for n in (-1, many):
        assert lib.ns_pages_truncate(c, P(16), P(16), n, None) == ARG
        assert lib.ns_pages_fork(c, P(16), P(16), n, None) == ARG
        assert lib.ns_pages_extend(c, P(16), P(16), n, P(16), 1 << 40, None) == ARG
        assert lib.ns_pages_compact(c, P(16), P(16), P(16), 4, P(16), n, None) == ARG
    assert lib.ns_pages_fork(c, P(16), None, 1, None) == ARG
    assert lib.ns_pages_extend(c, P(16), None, 1, P(16), 1 << 40, None) == ARG
    assert lib.ns_pages_extend(c, P(16), P(16), 1, None, 1 << 40, None) == ARG
    assert lib.ns_pages_extend(c, P(16), P(16), 1, P(16), 8, None) == ARG
    for layer in (-1, 2):
        assert lib.ns_pages_write(c, layer, P(16), P(16), 1, P(16), P(16), 256, 128, 256, 128, 4, None) == ARG
    assert lib.ns_pages_write(c, 0, P(16), P(16), 1, P(16), P(16), 250, 128, 256, 128, 4, None) == ARG
    assert lib.ns_pages_write(c, 0, P(16), P(16), 1, P(20), P(16), 256, 128, 256, 128, 4, None) == ARG
    assert lib.ns_pages_write(c, 0, P(16), P(16), 1, P(16), P(16), 256, 128, 256, 128, -1, None) == ARG
    assert lib.ns_pages_compact(c, P(16), None, P(16), 4, P(16), 1, None) == ARG
    assert lib.ns_pages_copy(c, P(16), None, 1, None) == ARG
    for f in (lib.ns_pages_truncate, lib.ns_pages_fork, lib.ns_pages_copy):
        assert f(c, None, None, 0, None) == 0


@pytest.mark.parametrize("kw", [
    dict(logits=None), dict(dtype=3), dict(rows=-1), dict(V=0), dict(ld=9), dict(t=0.0), dict(t=-1.0),
    dict(t=float("nan")), dict(n_ids=-1), dict(n_ids=2, ids=None), dict(n_ids=2, lp=None), dict(k=-1), dict(k=33),
    dict(k=3, top=None), dict(k=3, toplp=None),
])
def test_logprobs_refuse(lib, kw):
    a = dict(logits=16, dtype=2, rows=2, V=10, ld=10, t=1.0, ids=16, n_ids=1, k=2, lp=16, ent=16, lse=16, top=16, toplp=16)
    a.update(kw)
    assert lib.ns_token_logprobs(P(a["logits"]), a["dtype"], a["rows"], a["V"], a["ld"], ctypes.c_float(a["t"]),
                                 P(a["ids"]), a["n_ids"], a["k"], P(a["lp"]), P(a["ent"]), P(a["lse"]), P(a["top"]),
                                 P(a["toplp"]), None) == ARG


def test_header_and_python_have_the_same_limits():
    from speculative_decoding_draft_stream_gb300 import serving

    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "nanospec_ops.h")).read()
    for name in ("MAX_NEW", "MAX_ATTEND_SEQS", "MAX_ALTERNATIVES", "MAX_PAGE_SEQS"):
        assert f"#define NS_{name} {getattr(serving, name)}" in text
    for name in ("NO_PAGES", "BAD_SEQ", "SHARED_PAGE"):
        assert f"#define NS_FLAG_{name} {getattr(serving, 'FLAG_' + name):#x}u" in text


@pytest.mark.parametrize("off", [1, 2, 3])
def test_pages_refuse_integers_off_their_boundary(lib, off):
    c, a, x = cache(), P(16), P(16 + off)
    assert lib.ns_pages_truncate(c, x, a, 1, None) == ARG
    assert lib.ns_pages_truncate(c, a, x, 1, None) == ARG
    assert lib.ns_pages_fork(c, x, a, 1, None) == ARG
    assert lib.ns_pages_fork(c, a, x, 1, None) == ARG
    assert lib.ns_pages_extend(c, x, a, 1, a, 1 << 40, None) == ARG
    assert lib.ns_pages_extend(c, a, x, 1, a, 1 << 40, None) == ARG
    assert lib.ns_pages_write(c, 0, x, a, 1, a, a, 256, 128, 256, 128, 4, None) == ARG
    assert lib.ns_pages_write(c, 0, a, x, 1, a, a, 256, 128, 256, 128, 4, None) == ARG
    for place in range(4):
        args = [a, a, a, a]
        args[place] = x
        assert lib.ns_pages_compact(c, args[0], args[1], args[2], 4, args[3], 1, None) == ARG
    assert lib.ns_pages_copy(c, x, a, 1, None) == ARG
    assert lib.ns_pages_copy(c, a, x, 1, None) == ARG


@pytest.mark.parametrize("place", range(6))
@pytest.mark.parametrize("off", [1, 2, 3])
def test_logprobs_refuse_words_off_their_boundary(lib, place, off):
    w = [P(16 + off if i == place else 16) for i in range(6)]  # ids, log probabilities, entropy, lse, top ids, theirs
    assert lib.ns_token_logprobs(P(16), 2, 2, 10, 10, ctypes.c_float(1.0), w[0], 1, 2, *w[1:], None) == ARG


@pytest.mark.parametrize("t", [1e-45, 2.9e-39, 3e-39, 4.2e-39, float("inf")])
def test_logprobs_refuse_temperatures_whose_inverse_overflows(lib, t):
    """The kernels work in powers of two: log2(e) / T has to be finite, not 1 / T alone."""
    w = [P(16)] * 6
    assert lib.ns_token_logprobs(P(16), 2, 2, 10, 10, ctypes.c_float(t), w[0], 1, 2, *w[1:], None) == ARG


@pytest.mark.parametrize("kw", [dict(ld=(1 << 27) - 8), dict(ld=(1 << 28) - 31, page=8)])
def test_paged_refuses_tables_whose_last_tile_ends_past_31_bits(lib, kw):
    assert paged(lib, **kw) == ARG
