"""norm_rotate against its formula in 64 bits.

Tolerance.  With u the type's half step (2^-8 bf16, 2^-11 fp16): the sum of D
squares, the root and two products leave y off by (D / 2 + 6) 2^-24 of itself;
a cosine or sine is off by 2^-21 (its own rounding, an angle of up to half a
turn rounded to 24 bits, and 2^-33 turns), and by position * f * 2^-52 for the
product that the reference rounds; a' = a cos - b sin adds three roundings:
   |error| <= (|y_a| + |y_b|) (2^-21 + (D / 2 + 10) 2^-24 + p f 2^-52) + u |a'|
and half of fp16's smallest step, 2^-25.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
UNIT = {BF16: 2.0 ** -8, F16: 2.0 ** -11}


@pytest.fixture(scope="module")
def ns():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import speculative_decoding_draft_stream_gb300 as p
    from speculative_decoding_draft_stream_gb300 import build

    build.build()
    p.ops_error(clear=True)
    return p


def freqs(R, base=10000.0):
    return (base ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).cuda()


def formula(x, weight, pos, inv, eps, neighbours):
    """(rows, bound on their error) in 64 bits."""
    dt, D, h = x.dtype, x.shape[-1], inv.numel()
    y, p, f = x.double().cpu(), pos.double().cpu()[:, None, None], inv.cpu()
    if eps is not None:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt()
        if weight is not None:
            y = y * weight.double().cpu()
    out, size = y.clone(), torch.zeros_like(y)
    far = torch.zeros_like(y)
    ia = torch.arange(h) * 2 if neighbours else torch.arange(h)
    ib = ia + 1 if neighbours else ia + h
    a, b, t = y[..., ia], y[..., ib], p * f
    out[..., ia], out[..., ib] = a * t.cos() - b * t.sin(), b * t.cos() + a * t.sin()
    size[..., ia] = size[..., ib] = a.abs() + b.abs()
    far[..., ia] = far[..., ib] = (t.abs() * 2.0 ** -52).expand_as(a)
    rel = (D / 2 + 10) * 2.0 ** -24
    tol = size * (2.0 ** -21 + far) + torch.maximum(size, y.abs()) * rel + UNIT[dt] * out.abs() * (1 + rel)
    return out, tol + (2.0 ** -25 if dt == F16 else 0.0)


def check(got, want, what):
    out, tol = want
    over = (got.double().cpu() - out).abs() - tol
    assert over.numel() == 0 or over.max() <= 0, f"{what}: off by {over.max():.3g} more than its bound"


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("D,R", [(128, 128), (128, 64), (64, 64), (64, 16), (128, 0), (128, 112)])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("T,hq,hkv", [(1, 32, 8), (7, 5, 1), (513, 12, 4)])
@pytest.mark.parametrize("norm", [False, True])
def test_formula(ns, dt, D, R, neighbours, T, hq, hkv, norm):
    g = torch.Generator(device="cuda").manual_seed(T + D + R)
    qkv = torch.randn(T, hq + 2 * hkv, D, generator=g, device="cuda").to(dt)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hkv]
    pos = torch.randint(0, 100000, (T,), generator=g, device="cuda", dtype=torch.int32)
    inv = freqs(R) if R else torch.empty(0, dtype=torch.float64, device="cuda")
    w = [(1 + torch.randn(D, generator=g, device="cuda")).to(dt) for _ in range(2)] if norm else [None, None]
    eps = 1e-5 if norm else None
    a, b = ns.norm_rotate(q, k, pos, inv, q_weight=w[0], k_weight=w[1], eps=eps, neighbours=neighbours)
    check(a, formula(q, w[0], pos, inv, eps, neighbours), "q")
    check(b, formula(k, w[1], pos, inv, eps, neighbours), "k")


@pytest.mark.parametrize("p0", [0, 1, -7, 1 << 20, (1 << 31) - 5, -(1 << 31)])
def test_far_positions(ns, p0):
    x = torch.randn(5, 3, 128, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(F16)
    pos = torch.tensor([max(-(1 << 31), min((1 << 31) - 1, p0 + i)) for i in range(5)], dtype=torch.int32,
                       device="cuda")
    for inv in (freqs(128, 500000.0), freqs(128) * 7.5, -freqs(128), torch.full((64,), 1e-12, dtype=torch.float64).cuda()):
        got, none = ns.norm_rotate(x, None, pos, inv)
        assert none is None
        check(got, formula(x, None, pos, inv, None, False), f"{p0}")


def test_no_weight_zero_rows_and_values_that_are_not_finite(ns):
    x = torch.randn(4, 2, 64, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(BF16)
    x[1, 0] = 0
    x[2, 1, 3] = float("inf")
    x[3, 0, 40] = float("nan")
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    got, _ = ns.norm_rotate(x, None, pos, freqs(64), eps=1e-6)
    assert (got[1, 0] == 0).all()
    assert torch.isnan(got[3, 0]).all() and torch.isnan(got[2, 1, 3]) and torch.isfinite(got[2, 0]).all()
    fine = torch.ones(4, 2, dtype=torch.bool)
    fine[2, 1] = fine[3, 0] = False
    out, tol = formula(x, None, pos, freqs(64), 1e-6, False)
    assert ((got.double().cpu() - out).abs() <= tol)[fine].all()


@pytest.mark.parametrize("T", [3, 4000])
def test_in_place_over_a_fused_projection_and_strided_outputs(ns, T):
    g = torch.Generator(device="cuda").manual_seed(3)
    qkv = torch.randn(T, 12, 128, generator=g, device="cuda").to(BF16)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") + 77
    inv, was = freqs(64), qkv.clone()
    want = ns.norm_rotate(qkv[:, :8], qkv[:, 8:10], pos, inv, eps=1e-6)
    wide = torch.zeros(T, 20, 128, dtype=BF16, device="cuda")
    a, b = wide[:, 1:9], wide[:, 15:17]
    r = ns.norm_rotate(qkv[:, :8], qkv[:, 8:10], pos, inv, eps=1e-6, q_out=a, k_out=b)
    assert r[0] is a and r[1] is b and torch.equal(a, want[0]) and torch.equal(b, want[1])
    assert (wide[:, 0] == 0).all() and (wide[:, 9:15] == 0).all() and (wide[:, 17:] == 0).all()
    q, k = qkv[:, :8], qkv[:, 8:10]
    ns.norm_rotate(q, k, pos, inv, eps=1e-6, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(qkv[:, 10:], was[:, 10:])


def test_heads_before_tokens_no_tokens_and_another_stream(ns):
    g = torch.Generator(device="cuda").manual_seed(4)
    q = torch.randn(8, 100, 64, generator=g, device="cuda").to(F16).transpose(0, 1)
    pos = torch.arange(100, dtype=torch.int32, device="cuda")
    want, _ = ns.norm_rotate(q.contiguous(), None, pos, freqs(64))
    out = torch.empty(8, 100, 64, dtype=F16, device="cuda").transpose(0, 1)
    ns.norm_rotate(q, None, pos, freqs(64), q_out=out)
    assert torch.equal(out, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, none = ns.norm_rotate(q, None, pos, freqs(64), stream=s)
    s.synchronize()
    assert torch.equal(got, want) and none is None
    a, b = ns.norm_rotate(q[:0], q[:0, :2], pos[:0], freqs(64))
    assert a.shape == (0, 8, 64) and b.shape == (0, 2, 64)


def test_replayed_from_a_graph(ns):
    g = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randn(60, 8, 128, generator=g, device="cuda").to(BF16)
    pos, inv = torch.arange(60, dtype=torch.int32, device="cuda"), freqs(128)
    out = torch.empty_like(q)
    ns.norm_rotate(q, None, pos, inv, eps=1e-6, q_out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ns.norm_rotate(q, None, pos, inv, eps=1e-6, q_out=out)
    q.mul_(-0.5), pos.add_(1000)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ns.norm_rotate(q, None, pos, inv, eps=1e-6)[0])


def test_refusals(ns):
    q = torch.zeros(4, 2, 64, dtype=BF16, device="cuda")
    pos, inv = torch.zeros(4, dtype=torch.int32, device="cuda"), freqs(64)
    w = torch.ones(64, dtype=BF16, device="cuda")
    bad = [
        lambda: ns.norm_rotate(q.float(), None, pos, inv),
        lambda: ns.norm_rotate(q.cpu(), None, pos, inv),
        lambda: ns.norm_rotate(q[..., :32], None, pos, inv[:16]),
        lambda: ns.norm_rotate(q, q.half(), pos, inv),
        lambda: ns.norm_rotate(q, q[:3], pos, inv),
        lambda: ns.norm_rotate(q, None, pos.long(), inv),
        lambda: ns.norm_rotate(q, None, pos[:3], inv),
        lambda: ns.norm_rotate(q, None, pos, inv.float()),
        lambda: ns.norm_rotate(q, None, pos, inv[:4]),
        lambda: ns.norm_rotate(q, None, pos, freqs(80)),
        lambda: ns.norm_rotate(q, None, pos, inv, q_weight=w),
        lambda: ns.norm_rotate(q, None, pos, inv, q_weight=w.float(), eps=1e-6),
        lambda: ns.norm_rotate(q, None, pos, inv, q_weight=w[:32], eps=1e-6),
        lambda: ns.norm_rotate(q, None, pos, inv, eps=-1e-6),
        lambda: ns.norm_rotate(q, None, pos, inv, q_out=torch.empty(4, 3, 64, dtype=BF16, device="cuda")),
        lambda: ns.norm_rotate(q, None, pos, inv, q_out=torch.empty(4, 1, 64, dtype=BF16, device="cuda").expand(4, 2, 64)),
        lambda: ns.norm_rotate(q.clone().requires_grad_(), None, pos, inv),
        lambda: ns.norm_rotate(q.transpose(1, 2), None, pos, inv),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    odd = torch.zeros(4 * 128 + 4, dtype=BF16, device="cuda")[4:].view(4, 2, 64)  # off a 16-byte boundary
    with pytest.raises(ns.NanoSpecError):
        ns.norm_rotate(odd, None, pos, inv)
    with torch.no_grad():
        ns.norm_rotate(q.clone().requires_grad_(), None, pos, inv)
    assert ns.ops_error() == 0
