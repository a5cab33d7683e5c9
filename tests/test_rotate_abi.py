"""Refusals of ns_norm_rotate, which come before anything touches a GPU."""

import ctypes

import pytest

P = ctypes.c_void_p
ARG = -1


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_draft_stream_gb300 import build
    from speculative_decoding_draft_stream_gb300.nanospec import load_library

    return load_library(build.build())


def rotate(lib, **kw):
    a = dict(q=16, k=16, dtype=0, tokens=10, hq=8, hkv=2, dim=64, qt=512, qh=64, kt=128, kh=64, pos=16, freq=16,
             rotary=64, neighbours=0, qw=16, kw=16, eps=1e-6, qo=16, ko=16, qot=512, qoh=64, kot=128, koh=64)
    a.update(kw)
    return lib.ns_norm_rotate(P(a["q"]), P(a["k"]), a["dtype"], a["tokens"], a["hq"], a["hkv"], a["dim"], a["qt"],
                              a["qh"], a["kt"], a["kh"], P(a["pos"]), P(a["freq"]), a["rotary"], a["neighbours"],
                              P(a["qw"]), P(a["kw"]), ctypes.c_float(a["eps"]), P(a["qo"]), P(a["ko"]), a["qot"],
                              a["qoh"], a["kot"], a["koh"], None)


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(dim=96), dict(tokens=-1), dict(hq=0), dict(hkv=-1), dict(hq=65536), dict(rotary=-16),
    dict(rotary=24), dict(rotary=80), dict(eps=float("nan")), dict(eps=float("inf")), dict(eps=-1.0), dict(q=None),
    dict(k=None), dict(qo=None), dict(ko=None), dict(pos=None), dict(freq=None), dict(q=8), dict(k=24), dict(qo=24),
    dict(ko=8), dict(pos=18), dict(freq=20), dict(qw=24), dict(kw=8), dict(qt=516), dict(qh=4), dict(kt=12),
    dict(kh=1), dict(qot=516), dict(qoh=4), dict(kot=12), dict(koh=1),
])
def test_rotate_refuses(lib, kw):
    assert rotate(lib, **kw) == ARG


def test_rotation_of_nothing_is_done(lib):
    assert rotate(lib, tokens=0, q=None, pos=None) == 0
