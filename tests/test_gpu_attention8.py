"""attend_paged over a cache of 8 bits against softmax attention in 64 bits over what the codes stand for.

Tolerance, beside serving_ref's (u sum p |v| for the probabilities' rounding, with the larger of the type's u and
fp16's): probabilities that carry the values' scales are kept in fp16 with the largest p_j 2^ve_j at 2^8, so one is off
by at most 2^-25 there, 2^-33 of that largest, times its code (at most 448): 2^-33 * 448 * n * max p_j 2^ve_j in all.
A query in fp16, its largest element at 1 or above, is off by 2^-25 of that element: the score by
2^-25 max |q| sum |k| scale.

Beyond 16 rows in fp16 the values' scales are in the values: keys and values are codes times their power of two in
fp16, off by at most 2^-25 (half a step below 2^-14, where it cannot hold them), and probabilities are kept 2^6 times
larger, so that one (relative to the largest, at most 1) is off by at most 2^-25 2^-6.  So a score is off by
2^-25 sum |q| scale, and an output by 2^-31 sum |v| over the keys that it sees, and 2^-25 sum p = 2^-25.
"""

import random

import pytest
import torch

from serving8_ref import E4M3, quantise, values
from serving_ref import attend_rows, check

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def ns():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import speculative_decoding_draft_stream_gb300 as p
    from speculative_decoding_draft_stream_gb300 import build

    build.build()
    p.ops_error(clear=True)
    return p


def tree(n, rng):
    words = []
    for i in range(n):
        parent = rng.randrange(-1, i) if i else -1
        words.append((1 << i) | (words[parent] if parent >= 0 else 0))
    return words


def signed(w):
    return w - (1 << 64) if w >= 1 << 63 else w


def run(ns, lens, n, hq, hkv, d, dtype, page, seed, mask=None, layout="plain", sizes=1.0, max_len=0, spoil=None,
        scale=None, qstd=1.0):
    """mask: None, "tree", or a list of words for each sequence; sizes: how far the rows' sizes spread; spoil(codes_k,
    exps_k, codes_v, exps_v, row): changes pool rows, row(b, p) being where position p of sequence b lies."""
    g = torch.Generator().manual_seed(seed)
    rng = random.Random(seed)
    B = len(lens)
    held = [-(-x // page) for x in lens]
    pages = sum(held) + 3
    order = list(range(pages))
    rng.shuffle(order)
    table = torch.full((B + 2, max(held + [1]) + 1), -1, dtype=torch.int32)
    seqs = rng.sample(range(B + 2), B)
    at = 0
    for b in range(B):
        table[seqs[b], :held[b]] = torch.tensor(order[at:at + held[b]], dtype=torch.int32)
        at += held[b]
    lengths = torch.zeros(B + 2, dtype=torch.int32)
    lengths[seqs] = torch.tensor(lens, dtype=torch.int32)
    pool = []
    for _ in range(2):
        x = torch.randn(pages, hkv, page, d, generator=g).double()
        x *= torch.exp(sizes * torch.randn(pages, hkv, page, 1, generator=g).double())
        c, e = quantise(x.clamp(-60000, 60000))
        pool += [c.float().to(E4M3), e]
    # what lies behind a sequence's end may be anything
    def row(b, p):
        return order[sum(held[:b]) + p // page], p % page
    for b in range(B):
        for p in range(lens[b], held[b] * page):
            i, r = row(b, p)
            for c, e in (pool[:2], pool[2:]):
                c.view(torch.uint8)[i, :, r] = 0x7f
                e[i, :, r] = 255
    if spoil is not None:
        spoil(*pool, row)
    q = (torch.randn(B, n, hq, d, generator=g) * qstd).to(dtype)
    words = None
    if mask == "tree":
        words = [tree(n, rng) for _ in range(B)]
    elif mask is not None:
        words = mask
    dk, ke, dv, ve = pool
    if layout == "plain":
        dk, dv, gke, gve, gq = dk.cuda(), dv.cuda(), ke.cuda(), ve.cuda(), q.cuda()
    else:  # tokens before heads, exponents in wider pages, queries as slices
        dk, dv = (t.view(torch.uint8).transpose(1, 2).contiguous().cuda().transpose(1, 2).view(E4M3) for t in (dk, dv))
        wide = torch.full((pages, hkv + 3, page + 8), 255, dtype=torch.uint8)
        wide[:, 1:hkv + 1, :page] = ke
        gke = wide.cuda()[:, 1:hkv + 1, :page]
        gve = ve.transpose(0, 1).contiguous().cuda().transpose(0, 1)
        gq = torch.cat([q, q], 2).cuda()[:, :, :hq]
        if layout == "odd":  # queries that TMA cannot fetch
            gq = torch.cat([q, q[..., :2]], -1).cuda()[..., :d]
    m = None if words is None else torch.tensor([[signed(w) for w in r] for r in words], dtype=torch.int64).cuda()
    scale = d ** -0.5 if scale is None else scale
    out, lse = ns.attend_paged(gq, dk, dv, table.cuda(), lengths.cuda(), torch.tensor(seqs, dtype=torch.int32).cuda(),
                               mask=m, scale=scale, max_len=max_len, k_exp=gke, v_exp=gve)
    assert out.dtype == dtype and out.shape == q.shape
    out, lse = out.cpu(), lse.cpu()
    grp = hq // hkv
    k_all, v_all = values(pool[0].float(), ke), values(pool[2].float(), ve)
    for b in range(B):
        L = lens[b]
        at = [row(b, p) for p in range(L)]
        ip, ir = [i for i, _ in at], [r for _, r in at]
        sees = torch.ones(n, L, dtype=torch.bool)
        for i in range(n):
            for j in range(n):
                p = L - n + j
                if 0 <= p < L:
                    sees[i, p] = j <= i if words is None else bool(words[b][i] >> j & 1)
        for h in range(hkv):
            k, v = k_all[ip, h, ir] if L else k_all[:0, 0, 0], v_all[ip, h, ir] if L else v_all[:0, 0, 0]
            vs = torch.exp2(ve[ip, h, ir].double() - 127) if L else torch.zeros(0).double()
            for x in range(grp):
                hh = h * grp + x
                qq = q[b, :, hh]
                wild = (sees.double() @ torch.isnan(k).any(-1).double()) > 0 if L else torch.zeros(n, dtype=torch.bool)
                o, z, to, tz = attend_rows(qq, torch.nan_to_num(k), v, sees, scale)
                if L:
                    fine = torch.nan_to_num(k)
                    more = 2.0 ** -25 * scale * qq.double().abs().amax(-1) * fine.abs().sum(-1).max()
                    p = torch.where(sees, torch.exp((qq.double() @ fine.T) * scale - z.nan_to_num(neginf=0.0)[:, None]), 0.0)
                    big = (p * torch.nan_to_num(vs)).amax(-1)
                    pv = p @ torch.nan_to_num(v).abs()
                    if dtype == F16 and n * grp > 16:
                        more = more + 2.0 ** -25 * scale * qq.double().abs().sum(-1)
                        to = to + 2.0 ** -31 * (sees.double() @ torch.nan_to_num(v).abs()) + 2.0 ** -25
                    tz = tz + more
                    to = to + 2 * more[:, None] * pv + (2.0 ** -33 * 448 * L) * big[:, None]
                o[wild], z[wild] = float("nan"), float("nan")
                check(out[b, :, hh], o, to, f"out of sequence {b} head {hh}")
                check(lse[b, :, hh], z, tz, f"lse of sequence {b} head {hh}")
    assert ns.ops_error() == 0


EDGES = [1, 2, 7, 8, 9, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257, 700]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,mask", [(1, None), (4, "tree"), (17, "tree")])
def test_lengths(ns, dtype, d, n, mask):
    run(ns, [x + n - 1 for x in EDGES] + [n], n, 4, 1, d, dtype, 16, n + d, mask)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (7, 1), (14, 2), (8, 8), (16, 1), (12, 4), (32, 1), (33, 1), (130, 1)])
@pytest.mark.parametrize("n", [1, 3])
def test_heads(ns, hq, hkv, n):
    run(ns, [70, n, 301], n, hq, hkv, 128, BF16, 16, 2)
    run(ns, [70, n, 301], n, hq, hkv, 64, F16, 16, 3)


@pytest.mark.parametrize("page", [8, 32, 128, 1024])
@pytest.mark.parametrize("n", [1, 40])
def test_pages(ns, page, n):
    run(ns, [n + 2, 1025, 333, 2100], n, 8, 2, 128, BF16, page, page + n, "tree")
    run(ns, [n + 2, 1025, 333, 2100], n, 8, 2, 64, F16, page, page + n + 1)


@pytest.mark.parametrize("layout", ["strided", "odd"])
@pytest.mark.parametrize("n", [1, 5, 33])
def test_strides(ns, layout, n):
    run(ns, [200, 64, 515], n, 8, 2, 128, BF16, 16, 4, "tree", layout)
    run(ns, [200, 64, 515], n, 8, 2, 64, F16, 16, 5, None, layout)


@pytest.mark.parametrize("dtype,lens,n,hq,hkv,d", [
    (BF16, [5000], 1, 32, 8, 128), (F16, [9001], 1, 12, 4, 64), (F16, [33000], 1, 28, 4, 128),
    (BF16, [30000, 17], 2, 4, 1, 128), (BF16, [4000] * 3 + [11] * 40, 1, 28, 4, 128), (F16, [1300] * 20, 1, 32, 8, 64),
    (BF16, [3000, 70, 1500], 60, 8, 2, 128), (F16, [2000, 64], 64, 8, 8, 64), (BF16, [20000], 60, 4, 1, 128),
])
def test_longer(ns, dtype, lens, n, hq, hkv, d):
    """Clusters of both sizes, the line of tiles with its joins, and blocks of rows."""
    run(ns, lens, n, hq, hkv, d, dtype, 16, len(lens) + n, "tree" if n > 1 else None, max_len=max(lens))


@pytest.mark.parametrize("n", [1, 20])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_rows_of_very_different_sizes(ns, n, dtype):
    """A value row's size spreads over e^+-12: probabilities alone would not say which keys count."""
    run(ns, [300, 1030], n, 8, 2, 128, dtype, 16, 7, "tree", sizes=3.0, qstd=0.02)
    run(ns, [300, 1030], n, 8, 2, 64, dtype, 16, 8, "tree", sizes=3.0, qstd=0.02)


@pytest.mark.parametrize("n", [1, 20])
def test_exponents_at_their_ends(ns, n):
    """Values at 2^-40 and 2^40 of theirs, the small ones with nearly all the probability, or none."""
    def spoil(ck, ek, cv, ev, row):
        ev[:] = 87
        for p in (3, 90, 150):
            i, r = row(0, p)
            ev[i, :, r] = 167
            ck.view(torch.uint8)[i, :, r] = 0
    run(ns, [260], n, 4, 1, 128, BF16, 16, 9, None, sizes=0.0, spoil=spoil, qstd=3.0)

    def zeros(ck, ek, cv, ev, row):  # rows of zeros, as they are written
        for c, e in ((ck, ek), (cv, ev)):
            c.view(torch.uint8)[:, :, ::2] = 0
            e[:, :, ::2] = 87
    run(ns, [260, 40], n, 4, 1, 128, F16, 16, 10, None, spoil=zeros)

    def small(ck, ek, cv, ev, row):
        ek[:] = 87
        ev[:] = 87
    run(ns, [260, 40], n, 4, 1, 64, BF16, 16, 11, None, spoil=small)


@pytest.mark.parametrize("n", [1, 20])
@pytest.mark.parametrize("d", [64, 128])
def test_queries_of_any_size(ns, n, d):
    run(ns, [260], n, 4, 1, d, BF16, 16, 12, None, qstd=2.0 ** -100, scale=1.0)
    run(ns, [260], n, 4, 1, d, BF16, 16, 13, None, qstd=2.0 ** 90, scale=2.0 ** -93)
    run(ns, [260], n, 4, 1, d, F16, 16, 14, None, qstd=2.0 ** -13, scale=2.0 ** 9)


@pytest.mark.parametrize("n,hq", [(3, 4), (20, 4), (40, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_are_not_finite(ns, n, hq, d):
    """Keys and values with exponent 255 and codes that are NaN reach the rows that see them and no others; a value
    does not reach the log-sum-exp."""
    L = 200
    words = [[(1 << i) if i % 3 else 0 for i in range(n)], [(1 << (i + 1)) - 1 for i in range(n)]]

    def spoil(ck, ek, cv, ev, row):
        i, r = row(0, L - n + 2)
        ev[i, :, r] = 255
        i, r = row(0, L - n + 1)
        ek[i, 0, r] = 255
        i, r = row(1, L - 1)
        cv.view(torch.uint8)[i, 0, r, 5] = 0x7f
        cv.view(torch.uint8)[i, 0, r, d - 1] = 0xff
    run(ns, [L, L], n, hq, 1, d, BF16, 16, 15, words, spoil=spoil)


def test_rows_that_see_nothing(ns):
    for n in (1, 20):
        words = [[0] * n, [0 if i % 2 else 1 for i in range(n)]]
        run(ns, [n, n], n, 4, 2, 64, BF16, 8, 16, words)
    q = torch.randn(2, 3, 4, 64, device="cuda").to(BF16)
    k = torch.zeros(4, 2, 16, 64, dtype=torch.uint8, device="cuda").view(E4M3)
    e = torch.full((4, 2, 16), 127, dtype=torch.uint8, device="cuda")
    z = torch.zeros(2, dtype=torch.int32, device="cuda")
    out, lse = ns.attend_paged(q, k, k, torch.full((2, 2), -1, dtype=torch.int32, device="cuda"), z,
                               torch.arange(2, dtype=torch.int32, device="cuda"), k_exp=e, v_exp=e)
    assert (out == 0).all() and (lse == -float("inf")).all() and ns.ops_error() == 0


@pytest.mark.parametrize("n", [1, 40])
def test_bad_pages_and_sequences(ns, n):
    """No row sees the positions of a page that is not there; a sequence out of range gives zeros."""
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(3, n, 8, 64, generator=g, device="cuda").to(BF16)
    cache = ns.KvPages.new(1, 40, 2, 16, 64, 3, 12, scaled=True)
    lens = torch.tensor([150, 150, 150], dtype=torch.int32, device="cuda")
    seqs = torch.arange(3, dtype=torch.int32, device="cuda")
    cache.extend(seqs, lens)
    k, v = (torch.randn(450, 2, 64, generator=g, device="cuda").to(BF16) for _ in range(2))
    cu = torch.tensor([0, 150, 300, 450], dtype=torch.int32, device="cuda")
    cache.write(0, seqs, cu, k, v)
    cache.table[1, 2] = 40
    cache.table[1, 4] = -5
    out, lse = cache.attend(0, q, torch.tensor([0, 1, 7], dtype=torch.int32, device="cuda"))
    assert ns.ops_error(clear=True) == ns.FLAG_BAD_ID | ns.FLAG_BAD_SEQ
    assert (out[2] == 0).all() and (lse[2] == -float("inf")).all()
    for b in range(2):
        kk, vv = (values(*quantise(t[150 * b:150 * (b + 1)].cpu())) for t in (k, v))
        seen = torch.ones(n, 150, dtype=torch.bool)
        seen[:, 150 - n:] = torch.ones(n, n, dtype=torch.bool).tril()
        if b == 1:
            seen[:, 32:48] = seen[:, 64:80] = False
        for h in range(8):
            o, z, to, tz = attend_rows(q[b, :, h].cpu(), kk[:, h // 4], vv[:, h // 4], seen, 0.125)
            check(out[b, :, h], o, to * 1.01, "out")
            check(lse[b, :, h], z, tz + 1e-5, "lse")


def test_same_bits_again_and_in_a_graph(ns):
    g = torch.Generator(device="cuda").manual_seed(4)
    for n, lens in ((1, [700, 33, 20000]), (60, [900, 100, 64])):
        cache = ns.KvPages.new(2, 1400, 4, 16, 128, 3, 1300, scaled=True)
        seqs, L = torch.arange(3, dtype=torch.int32, device="cuda"), torch.tensor(lens, dtype=torch.int32, device="cuda")
        cache.extend(seqs, L)
        T = sum(lens)
        k = torch.randn(T, 4, 128, generator=g, device="cuda").to(F16)
        cu = torch.tensor([0, lens[0], lens[0] + lens[1], T], dtype=torch.int32, device="cuda")
        cache.write(1, seqs, cu, k, k.flip(0))
        q = torch.randn(3, n, 28, 128, generator=g, device="cuda").to(F16)
        kw = {"max_len": max(lens)}
        a, al = cache.attend(1, q, seqs, **kw)
        b, bl = cache.attend(1, q, seqs, **kw)
        assert torch.equal(a, b) and torch.equal(al, bl)
        out = torch.empty_like(a)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            cache.attend(1, q, seqs, out=out, **kw)
        for _ in range(2):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, a)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        c, _ = cache.attend(1, q, seqs, stream=s, **kw)
        s.synchronize()
        assert torch.equal(c, a)
    assert ns.ops_error() == 0


def test_refusals(ns):
    cache = ns.KvPages.new(1, 4, 2, 16, 64, 2, 2, scaled=True)
    seqs = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 1, 4, 64, dtype=BF16, device="cuda")
    k, v, ke, ve = cache.k[0], cache.v[0], cache.k_exp[0], cache.v_exp[0]
    rest = (cache.table, cache.lengths, seqs)
    bad = [
        lambda: ns.attend_paged(q, k, v, *rest),
        lambda: ns.attend_paged(q, k, v, *rest, k_exp=ke),
        lambda: ns.attend_paged(q, k, v, *rest, v_exp=ve),
        lambda: ns.attend_paged(q, k.to(BF16), v.to(BF16), *rest, k_exp=ke, v_exp=ve),
        lambda: ns.attend_paged(q, k, v, *rest, k_exp=ke.int(), v_exp=ve),
        lambda: ns.attend_paged(q, k, v, *rest, k_exp=ke[:3], v_exp=ve),
        lambda: ns.attend_paged(q, k, v, *rest, k_exp=ke, v_exp=ve[:, :1]),
        lambda: ns.attend_paged(q, k, v, *rest, k_exp=ke.cpu(), v_exp=ve),
        lambda: ns.attend_paged(q, k, v, *rest, k_exp=ke.transpose(1, 2).contiguous().transpose(1, 2), v_exp=ve),
        lambda: ns.attend_paged(q.float(), k, v, *rest, k_exp=ke, v_exp=ve),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            f()
            pytest.fail(f"call {i} was not refused")
    off = torch.zeros(4 * 2 * 16 + 4, dtype=torch.uint8, device="cuda")[4:].view(4, 2, 16)  # off an 8-byte boundary
    with pytest.raises(ns.NanoSpecError):
        ns.attend_paged(q, k, v, *rest, k_exp=off, v_exp=ve)
    assert ns.ops_error() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_values_beyond_fp16(ns, d):
    """A value row of 448 * 2^10 among ones, all with the same weight: as it is for up to 16 rows, and where it is made an
    fp16 (20 rows in fp16) 65504.  Sums of at most 64 terms are exact enough: u for a weight, u for the output."""
    L, page = 64, 16
    x = torch.ones(4, 1, page, d, dtype=torch.float64)
    x[0, 0, 3] = 448.0 * 2 ** 10
    cv, ev = quantise(x)
    ck, ek = quantise(torch.zeros_like(x))
    pool = [c.float().to(E4M3).cuda() for c in (ck, cv)]
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    one = torch.tensor([L], dtype=torch.int32, device="cuda")
    for dtype, n, top in ((BF16, 1, 448.0 * 2 ** 10), (BF16, 20, 448.0 * 2 ** 10), (F16, 1, 448.0 * 2 ** 10), (F16, 20, 65504.0)):
        q = torch.zeros(1, n, 1, d, dtype=dtype, device="cuda")
        out, _ = ns.attend_paged(q, *pool, table, one, one - L, k_exp=ek.cuda(), v_exp=ev.cuda())
        seen = torch.arange(L - n + 1, L + 1, dtype=torch.float64)
        want = ((seen - 1 + top) / seen)[:, None].expand(n, d)
        u = torch.finfo(dtype).eps
        assert torch.allclose(out[0, :, 0].cpu().double(), want, rtol=1.1 * u, atol=0), (dtype, n)
    assert ns.ops_error() == 0
