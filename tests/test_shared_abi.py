"""Refusals of ns_attend_shared, which come before anything touches a GPU."""

import ctypes

import pytest

P = ctypes.c_void_p
ARG = -1


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_draft_stream_gb300 import build
    from speculative_decoding_draft_stream_gb300.nanospec import load_library

    return load_library(build.build())


def shared(lib, **kw):
    a = dict(q=16, dtype=0, B=4, n=2, hq=8, hkv=2, dim=64, qs=1024, qt=512, qh=64, k=16, v=16, pages=4, page=16,
             kp=2048, kh=1024, kt=64, vp=2048, vh=1024, vt=64, table=16, ld=4, seqs=4, lengths=16, ids=16, groups=16,
             G=2, mask=None, scale=0.125, most=0, out=16, lse=16, ws=16, bytes=1 << 40)
    a.update(kw)
    return lib.ns_attend_shared(
        P(a["q"]), a["dtype"], a["B"], a["n"], a["hq"], a["hkv"], a["dim"], a["qs"], a["qt"], a["qh"], P(a["k"]),
        P(a["v"]), a["pages"], a["page"], a["kp"], a["kh"], a["kt"], a["vp"], a["vh"], a["vt"], P(a["table"]), a["ld"],
        a["seqs"], P(a["lengths"]), P(a["ids"]), P(a["groups"]), a["G"], P(a["mask"]), ctypes.c_float(a["scale"]),
        a["most"], P(a["out"]), P(a["lse"]), P(a["ws"]), a["bytes"], None)


@pytest.mark.parametrize("kw", [
    dict(groups=None), dict(groups=18), dict(G=0), dict(G=-1), dict(G=513), dict(qs=1536), dict(dtype=2), dict(dim=96),
    dict(page=12), dict(k=8), dict(n=65, qs=65 * 512), dict(hq=9), dict(scale=float("nan")), dict(ws=None),
])
def test_shared_refuses(lib, kw):
    assert shared(lib, **kw) == ARG


def test_shared_of_nothing_is_done(lib):
    assert shared(lib, B=0, G=0, groups=None) == 0
    assert shared(lib, B=0) == 0


def test_workspaces_of_bad_calls_are_nothing(lib):
    for a in ((-1, 1, 1, 8, 2, 64), (4097, 1, 1, 8, 2, 64), (4, 0, 1, 8, 2, 64), (4, 513, 1, 8, 2, 64),
              (4, 1, 0, 8, 2, 64), (4, 1, 65, 8, 2, 64), (4, 1, 1, 8, 3, 64), (4, 1, 1, 8, 2, 80)):
        assert lib.ns_attend_shared_workspace(*a) == 0
