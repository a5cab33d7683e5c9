"""token_logprobs against log-softmax in 64 bits.

Tolerance: with z = x / T, d = z - max z: rounding of 1 / T and of the product
move d by 2^-22 |d| at most, the exponential by 2^-21; the fp32 sums of n
terms in chains of n / 256 or fewer by (n / 256 + 64) 2^-24.  So log S is
within e = (n / 256 + 64) 2^-24 + 2^-20 + 2^-22 D, D the entropy-weighted |d|
(at most 90 before its terms vanish: e takes 90), log p within e + 2^-22 |d|,
lse within that plus 2^-22 |max z|, the entropy within 2 e (1 + entropy).
"""

import math

import pytest
import torch

from serving_ref import check

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def ns():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import speculative_decoding_draft_stream_gb300 as p
    from speculative_decoding_draft_stream_gb300 import build

    build.build()
    p.ops_error(clear=True)
    return p


def reference(x, ids, k, T):
    """x [rows, V] on the CPU; rows without NaN and +inf, some of them perhaps all -inf."""
    z = x.double() / T
    rows, V = z.shape
    m = z.amax(-1, keepdim=True)
    empty = torch.isinf(m.squeeze(1))
    d = torch.where(empty[:, None], torch.full_like(z, -math.inf), z - torch.where(torch.isinf(m), 0.0, m))
    p = torch.exp(d)
    s = p.sum(-1)
    ls = torch.where(empty, 0.0, torch.log(s.clamp_min(1e-300)))
    lp = d - ls[:, None]
    ent = ls - torch.where(p > 0, p * d, 0.0).sum(-1) / s.clamp_min(1e-300)
    lse = torch.where(empty, -math.inf, m.squeeze(1) + ls)
    order = torch.sort(x.float() + 0.0, dim=-1, descending=True, stable=True).indices[:, :k]
    top = torch.full((rows, k), -1, dtype=torch.int32)
    top[:, :min(k, V)] = order.to(torch.int32)
    tlp = torch.full((rows, k), -math.inf, dtype=torch.float64)
    tlp[:, :min(k, V)] = lp.gather(1, order)
    e = (V / 256 + 64) * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * 90
    off = lambda v: e + 2.0 ** -22 * torch.where(torch.isinf(v), 0.0, v).abs()  # noqa: E731
    want = lp.gather(1, ids.long().clamp(0, V - 1)) if ids is not None else torch.empty(rows, 0)
    if ids is not None:
        want = torch.where((ids >= 0) & (ids < V), want, math.nan)
    return {"logprobs": (want, off(torch.nan_to_num(want))), "entropy": (torch.where(empty, 0.0, ent), 2 * e * (1 + ent.abs())),
            "lse": (lse, off(lse)), "top_ids": top, "top_logprobs": (tlp, off(tlp))}


def run(ns, x, ids, k, T=1.0, flags=0, device_x=None):
    dx = x.cuda() if device_x is None else device_x
    r = ns.token_logprobs(dx, None if ids is None else ids.cuda(), k, temperature=T)
    w = reference(x, ids, k, T)
    assert r.top_ids.cpu().equal(w["top_ids"]), "top ids"
    for name in ("logprobs", "entropy", "lse", "top_logprobs"):
        want, tol = w[name]
        check(getattr(r, name), want, tol, name)
    assert ns.ops_error(clear=True) == flags


def make(rows, V, dtype, seed, std=2.0):
    g = torch.Generator()
    g.manual_seed(seed)
    x = torch.randn((rows, V), generator=g) * std
    x[:, V // 2] += 8.0
    ids = torch.randint(0, V, (rows, 3), generator=g, dtype=torch.int32)
    return x.to(dtype), ids


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("V", [1, 2, 3, 5, 31, 33, 255, 1000, 1027, 4099, 8192, 20011, 70001])
def test_vocabulary_sizes(ns, dtype, V):
    x, ids = make(3, V, dtype, V)
    run(ns, x, ids, min(10, V))
    run(ns, x, ids, 32, T=0.7)


@pytest.mark.parametrize("rows", [1, 2, 37, 160, 700])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_row_counts(ns, rows, dtype):
    """One CTA, or a cluster of two, four or eight, for a row."""
    x, ids = make(rows, 34000, dtype, rows)
    run(ns, x, ids, 5, T=1.3)


@pytest.mark.parametrize("k", [0, 1, 2, 7, 31, 32])
def test_alternatives(ns, k):
    x, ids = make(4, 50021, F32, k)
    run(ns, x, ids, k)
    run(ns, x, None, k)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_rows_off_16_byte_boundaries(ns, dtype):
    for V in (9, 1001, 40003):
        for shift in (1, 2, 3, 5, 7):
            x, ids = make(5, V, dtype, V + shift)
            wide = torch.full((5, V + 13), float("nan"), dtype=dtype, device="cuda")
            view = wide[:, shift:shift + V]
            view.copy_(x)
            run(ns, x, ids, 6, device_x=view)


def test_ties_go_to_the_lower_id(ns):
    for V in (40, 3000, 60000):
        x = torch.zeros(3, V)
        x[1, ::3] = -0.0
        x[2] = torch.randint(0, 4, (V,), generator=torch.Generator().manual_seed(V)).float()
        ids = torch.zeros(3, 1, dtype=torch.int32)
        run(ns, x, ids, 32)
        run(ns, x.to(BF16), ids, 9)


def test_sorted_rows(ns):
    V = 30000
    up = torch.arange(V).float() / 1000
    x = torch.stack([up, up.flip(0), -up])
    run(ns, x, torch.zeros(3, 1, dtype=torch.int32), 32)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_masked_logits(ns, dtype):
    """-inf and the type's lowest value as masks: probability 0; a row with nothing left."""
    for V in (50, 9000, 40000):
        x, ids = make(5, V, dtype, V)
        x[0, : V // 2] = -math.inf
        x[1] = -math.inf
        x[2, 1:] = torch.finfo(dtype).min
        x[3] = -math.inf
        x[3, V - 1] = 2.0
        x[4, ::2] = torch.finfo(dtype).min
        ids[0, 0], ids[3, 0] = 0, V - 1
        run(ns, x, ids, 4)


def test_large_magnitudes(ns):
    x, ids = make(3, 5000, F32, 1)
    x[0] *= 1e4
    x[1] += 3e5
    x[2] = 3e38
    run(ns, x, ids, 5)


def test_rows_with_nan_or_inf(ns):
    x, ids = make(4, 30000, F32, 2)
    x[0, 17] = math.nan
    x[1, 29999] = math.inf
    x[2] = math.nan
    r = ns.token_logprobs(x.cuda(), ids.cuda(), 4)
    for i in (0, 1, 2):
        for t in (r.lse, r.entropy, r.logprobs):
            assert torch.isnan(t[i]).all()
    w = reference(x[3:], ids[3:], 4, 1.0)
    check(r.logprobs[3:], *w["logprobs"], "a row beside them")
    order = torch.sort(torch.nan_to_num(x[0], nan=-math.inf), descending=True, stable=True).indices[:4]
    assert r.top_ids[0].cpu().equal(order.to(torch.int32))
    assert r.top_ids[1, 0] == 29999 and (r.top_ids[2] == -1).all()


def test_ids_out_of_range(ns):
    x, ids = make(3, 1000, F32, 3)
    ids[0, 1] = -1
    run(ns, x, ids, 2)
    ids[1, 0], ids[2, 2] = 1000, -2
    run(ns, x, ids, 2, flags=0x1)


def test_many_ids(ns):
    x, _ = make(2, 4097, F16, 4)
    ids = torch.randint(0, 4097, (2, 1000), dtype=torch.int32, generator=torch.Generator().manual_seed(5))
    run(ns, x, ids, 1)


def test_offsets_past_32_bits(ns):
    V, rows = 1024, 9
    step = (1 << 32) // 8 + 8
    buf = torch.empty(step * 8 + V, dtype=BF16, device="cuda")
    view = buf.as_strided((rows, V), (step, 1))
    x, ids = make(rows, V, BF16, 6)
    view.copy_(x)
    run(ns, x, ids, 3, device_x=view)


def test_other_stream_and_repeats(ns):
    x, ids = make(20, 50000, F32, 7)
    dx, di = x.cuda(), ids.cuda()
    a = ns.token_logprobs(dx, di, 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        b = ns.token_logprobs(dx, di, 8, stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_refusals(ns):
    x = torch.zeros(4, 100, device="cuda")
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    for f in (lambda: ns.token_logprobs(x.double(), ids), lambda: ns.token_logprobs(x, ids.long()),
              lambda: ns.token_logprobs(x, ids[:3]), lambda: ns.token_logprobs(x, ids, 33),
              lambda: ns.token_logprobs(x.t(), None), lambda: ns.token_logprobs(x.cpu(), None),
              lambda: ns.token_logprobs(x[0], None), lambda: ns.token_logprobs(x, ids, -1)):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: ns.token_logprobs(x, ids, temperature=0.0), lambda: ns.token_logprobs(x, ids, temperature=-1.0),
              lambda: ns.token_logprobs(x, ids, temperature=math.nan),
              lambda: ns.token_logprobs(x[:, :0], None),
              lambda: ns.token_logprobs(x[:1].expand(4, 100), None)):
        with pytest.raises(ns.NanoSpecError):
            f()
    assert ns.token_logprobs(x[:0], ids[:0], 3).top_ids.shape == (0, 3)


@pytest.mark.parametrize("t", [4.3e-39, 1e-38, 1e-30, 1e30, 1e37])
def test_extreme_temperatures(ns, t):
    """One token has all the probability, or each the same; nothing is NaN."""
    x = torch.tensor([[1.0, 3.0, -2.0, 0.5], [0.0, -1.0, -1.0, -3.0]])
    ids = torch.tensor([[1, 0], [0, 3]], dtype=torch.int32)
    r = ns.token_logprobs(x.cuda(), ids.cuda(), 1, temperature=t)
    assert not any(torch.isnan(v.float()).any() for v in r) and r.top_ids[:, 0].tolist() == [1, 0]
    if t < 1:
        assert r.logprobs[:, 0].tolist() == [0.0, 0.0] and r.entropy.tolist() == [0.0, 0.0]
        assert (r.logprobs[:, 1] < -1e29).all()
    else:
        assert (r.logprobs.cpu() + math.log(4)).abs().max() < 1e-6 and (r.entropy.cpu() - math.log(4)).abs().max() < 1e-6
