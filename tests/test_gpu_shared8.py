"""attend_shared over a cache of 8 bits against softmax attention in 64 bits over what the codes stand for: trees, rows
that are not finite, pages out of range, strides, malformed groups.

Tolerance: serving_ref's (probabilities rounded to the queries' type, keys and values as they are), which holds for bf16,
where a code times its power of two is exact.  In fp16 keys and values are off by at most 2^-25 (half a step below 2^-14),
and a probability, kept 2^6 times larger and at most 1, by 2^-25 2^-6: a score by 2^-25 scale sum |q|, and an output by
twice that times sum p |v|, by 2^-31 sum |v| over the keys that it sees, and by 2^-25 sum p = 2^-25."""

import random

import pytest
import torch

from serving8_ref import E4M3, quantise, values
from serving_ref import attend_rows, check
from test_gpu_shared import BF16, F16, i32, ns, signed, tree  # noqa: F401

pytestmark = pytest.mark.gpu


def run(ns, prompts, tails, n, hq, hkv, d, dtype, page, seed, mask=None, layout="plain", sizes=0.5, spoil=None,  # noqa: F811
        gone=(), groups=None, flags=0, wide=True):
    """As test_gpu_shared's run, over codes; spoil(codes_k, exps_k, codes_v, exps_v, row)."""
    g = torch.Generator().manual_seed(seed)
    rng = random.Random(seed)
    seq_of = [(i, p, t) for i, (p, ts) in enumerate(zip(prompts, tails)) for t in ts]
    lens = [p + t for _, p, t in seq_of]
    B, held = len(lens), [-(-(p + t) // page) for _, p, t in seq_of]
    pages = sum(held) + 3
    order = list(range(pages))
    rng.shuffle(order)
    rows, taken, at = [], {}, 0
    for b, (i, p, _) in enumerate(seq_of):
        if i not in taken:
            taken[i] = order[at:at + p // page]
            at += p // page
        own = held[b] - p // page
        rows.append(taken[i] + order[at:at + own])
        at += own
    table = torch.full((B + 2, (1 << 20) // page if wide else max(held) + 1), -1, dtype=torch.int32)
    lengths = torch.zeros(B + 2, dtype=torch.int32)
    seqs = rng.sample(range(B + 2), B)
    missing = [torch.zeros(x, dtype=torch.bool) for x in lens]
    for b in range(B):
        table[seqs[b], :held[b]] = torch.tensor(rows[b], dtype=torch.int32)
        lengths[seqs[b]] = lens[b]
    for b, slot in gone:
        for c in range(B):  # every sequence with that page
            if slot < held[c] and rows[c][slot] == rows[b][slot]:
                table[seqs[c], slot] = pages + 5
                missing[c][slot * page:(slot + 1) * page] = True
    pool = []
    for _ in range(2):
        x = torch.randn(pages, hkv, page, d, generator=g).double()
        x *= torch.exp(sizes * torch.randn(pages, hkv, page, 1, generator=g).double())
        c, e = quantise(x.clamp(-60000, 60000))
        pool += [c.float().to(E4M3), e]

    def row(b, p):
        return rows[b][p // page], p % page
    for b in range(B):  # what lies behind a sequence's end may be anything
        for p in range(lens[b], held[b] * page):
            i, r = row(b, p)
            for c, e in (pool[:2], pool[2:]):
                c.view(torch.uint8)[i, :, r] = 0x7f
                e[i, :, r] = 255
    if spoil is not None:
        spoil(*pool, row)
    q = torch.randn(B, n, hq, d, generator=g).to(dtype)
    words = [tree(n, rng) for _ in range(B)] if mask == "tree" else mask
    dk, ke, dv, ve = pool
    if layout == "plain":
        dk, dv, gke, gve, gq = dk.cuda(), dv.cuda(), ke.cuda(), ve.cuda(), q.cuda()
    else:  # tokens before heads, exponents in wider pages and heads before pages, queries as slices
        dk, dv = (t.view(torch.uint8).transpose(1, 2).contiguous().cuda().transpose(1, 2).view(E4M3) for t in (dk, dv))
        wider = torch.full((pages, hkv + 3, page + 8), 255, dtype=torch.uint8)
        wider[:, 1:hkv + 1, :page] = ke
        gke = wider.cuda()[:, 1:hkv + 1, :page]
        gve = ve.transpose(0, 1).contiguous().cuda().transpose(0, 1)
        gq = torch.cat([q, q], 2).cuda()[:, :, :hq]
    m = None if words is None else torch.tensor([[signed(w) for w in r] for r in words], dtype=torch.int64).cuda()
    cu = [0]
    for t in tails:
        cu.append(cu[-1] + len(t))
    out, lse = ns.attend_shared(gq, dk, dv, table.cuda(), lengths.cuda(), i32(seqs), i32(cu if groups is None else groups),
                                mask=m, k_exp=gke, v_exp=gve)
    assert ns.ops_error(clear=True) == (flags | (ns.FLAG_BAD_ID if gone else 0))
    out, lse = out.cpu(), lse.cpu()
    k_all, v_all = values(dk.cpu().float(), ke), values(dv.cpu().float(), ve)
    for b in range(B):
        L = lens[b]
        at = [row(b, p) for p in range(L)]
        ip, ir = [i for i, _ in at], [r for _, r in at]
        sees = torch.ones(n, L, dtype=torch.bool)
        for i in range(n):
            for j in range(n):
                if 0 <= L - n + j < L:
                    sees[i, L - n + j] = j <= i if words is None else bool(words[b][i] >> j & 1)
        sees &= ~missing[b]
        for h in range(hkv):
            k, v = k_all[ip, h, ir], v_all[ip, h, ir]
            wild = (sees.double() @ torch.isnan(k).any(-1).double()) > 0
            for x in range(hq // hkv):
                hh = h * (hq // hkv) + x
                qq = q[b, :, hh]
                o, z, to, tz = attend_rows(qq, torch.nan_to_num(k), v, sees, d ** -0.5)
                if dtype == F16:
                    size = torch.nan_to_num(v).abs()
                    more = 2.0 ** -25 * d ** -0.5 * qq.double().abs().sum(-1)
                    to = to + 2 * more[:, None] * size.amax() + 2.0 ** -31 * (sees.double() @ size) + 2.0 ** -25
                    tz = tz + more
                o[wild], z[wild] = float("nan"), float("nan")
                check(out[b, :, hh], o, to, f"out of sequence {b} head {hh}")
                check(lse[b, :, hh], z, tz, f"lse of sequence {b} head {hh}")


SHAPES = [(1, 8, 2), (5, 8, 2), (20, 8, 2), (30, 4, 1), (9, 14, 1), (64, 2, 1)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d,page", [(64, 8), (128, 16), (128, 256)])
@pytest.mark.parametrize("n,hq,hkv", SHAPES)
def test_trees(ns, dtype, d, page, n, hq, hkv):  # noqa: F811
    """One row tile (few tokens to a group) and two."""
    run(ns, [700, 150], [[n, n + 40, n + 7], [n, n + 3]], n, hq, hkv, d, dtype, page, n + d, "tree")
    run(ns, [520], [[n + i for i in range(9)]], n, hq, hkv, d, dtype, page, n + d, "tree")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 3, 20])
def test_strides(ns, dtype, d, n):  # noqa: F811
    run(ns, [600, 130], [[n, n + 200, n + 9], [n + 1, n]], n, 8, 2, d, dtype, 16, n, "tree" if n > 1 else None, "strided")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n", [1, 20])
def test_rows_of_very_different_sizes(ns, dtype, n):  # noqa: F811
    run(ns, [600], [[n, n + 140, n + 9]], n, 8, 2, 128, dtype, 16, 30 + n, "tree" if n > 1 else None, sizes=2.0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,members", [(3, 3), (20, 3), (20, 9)])
def test_rows_that_are_not_finite(ns, d, n, members):  # noqa: F811
    """Exponents of 255 and codes that are NaN among new tokens and behind the prefix reach the rows that see them alone; a
    value does not reach the log-sum-exp."""
    L = 300
    words = [[((1 << i) if i % 3 else 0) if b % 2 else (1 << (i + 1)) - 1 for i in range(n)] for b in range(members)]

    def spoil(ck, ek, cv, ev, row):
        i, r = row(0, L + 2)  # (the first member's new tokens are L ..)
        ev[i, :, r] = 255
        i, r = row(1, L + 1)
        ek[i, :, r] = 255
        i, r = row(1, L + 2)
        cv.view(torch.uint8)[i, :, r, 5] = 0x7f
        cv.view(torch.uint8)[i, :, r, d - 1] = 0xff
        i, r = row(2, L + 1)
        ck.view(torch.uint8)[i, :, r, 7] = 0x7f
    run(ns, [L], [[n] * members], n, 4, 1, d, BF16, 16, n, words, spoil=spoil)


@pytest.mark.parametrize("n", [1, 20])
def test_rows_of_the_prefix_that_are_not_finite(ns, n):  # noqa: F811
    """A value that is NaN is NaN in everyone's columns, a key in everyone's whole row, of its own head alone."""
    def value(ck, ek, cv, ev, row):
        i, r = row(0, 200)
        cv.view(torch.uint8)[i, 0, r, 9] = 0xff
        i, r = row(0, 70)
        ev[i, 1, r] = 255

    def key(ck, ek, cv, ev, row):
        i, r = row(0, 255)
        ek[i, 0, r] = 255
    for spoil in (value, key):
        run(ns, [300], [[n, n + 1, n + 150]], n, 4, 2, 128, BF16, 16, n, spoil=spoil)


def test_pages_out_of_range(ns):  # noqa: F811
    for dtype in (BF16, F16):
        run(ns, [600], [[5, 70, 200]], 1, 4, 1, 128, dtype, 16, 14, gone=[(0, 3), (1, 38)])
        run(ns, [600], [[65, 70, 200]], 40, 2, 1, 64, dtype, 32, 15, "tree", gone=[(0, 4), (2, 22)])
        run(ns, [600], [[65, 70, 200, 20]], 20, 4, 1, 128, dtype, 8, 16, "tree", gone=[(0, 0), (1, 80)])


@pytest.mark.parametrize("n", [1, 8, 30])
def test_groups_that_are_not_as_they_should_be(ns, n):  # noqa: F811
    tails = [[n, n + 2], [n + 3], [n + 4, n + 5]]
    for groups in ([0, 3, 2, 5], [1, 2, 3, 5], [0, 2, 3, 4], [0, 9, 9, 5], [0, -1, 3, 5]):
        run(ns, [300, 300, 140], tails, n, 4, 1, 64, BF16, 16, 10, groups=groups, flags=ns.FLAG_BAD_SEQ)
    run(ns, [300, 300, 140], tails, n, 4, 1, 64, BF16, 16, 10, groups=[0, 5])


def test_rows_that_see_nothing(ns):  # noqa: F811
    n = 20
    words = [[0] * n, [1 << i for i in range(n)], [0 if i % 2 else (1 << (i + 1)) - 1 for i in range(n)]]
    run(ns, [0], [[n, n, n]], n, 4, 1, 64, BF16, 8, 11, words)
    run(ns, [256], [[n, n, n + 7]], n, 4, 1, 128, F16, 8, 12, words)
