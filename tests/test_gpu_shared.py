"""attend_shared against softmax attention in 64 bits, with the tolerances of attend_paged (a row's parts are joined in
fp32 as that call's are)."""

import random

import pytest
import torch

from serving8_ref import quantise, values
from serving_ref import attend_rows, check, with_wild_values

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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def tree(n, rng):
    words = []
    for i in range(n):
        parent = rng.randrange(-1, i) if i else -1
        words.append((1 << i) | (words[parent] if parent >= 0 else 0))
    return words


def signed(w):
    return w - (1 << 64) if w >= 1 << 63 else w


def run(ns, prompts, tails, n, hq, hkv, d, dtype, page, seed, mask=None, layout="plain", spoil=None, gone=(),
        groups=None, flags=0, max_len=0, wide=True):
    """prompts[g]: positions that group g's members begin with; tails[g]: what each of them holds behind, new tokens
    included.  mask: None, "tree" or words of each sequence.  spoil(k, v, row): changes pool rows, row(b, p) being
    where position p of sequence b lies.  gone: (sequence, slot) whose page is out of range.  wide: a table for 2^20
    positions, by which a call of few rows shares, however short its sequences are."""
    g = torch.Generator().manual_seed(seed)
    rng = random.Random(seed)
    seq_of = [(i, p, t) for i, (p, ts) in enumerate(zip(prompts, tails)) for t in ts]
    lens = [p + t for _, p, t in seq_of]
    B = len(lens)
    held = [-(-x // page) for x in lens]
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
    table = torch.full((B + 2, (1 << 20) // page if wide else max(held + [1]) + 1), -1, dtype=torch.int32)
    seqs = rng.sample(range(B + 2), B)
    lengths = torch.zeros(B + 2, dtype=torch.int32)
    missing = [[False] * x for x in lens]
    for b in range(B):
        table[seqs[b], :held[b]] = torch.tensor(rows[b], dtype=torch.int32)
        lengths[seqs[b]] = lens[b]
    for b, slot in gone:
        for c in range(B):  # every sequence with that page
            if slot < held[c] and rows[c][slot] == rows[b][slot]:
                table[seqs[c], slot] = pages + 5
                missing[c][slot * page:(slot + 1) * page] = [True] * len(missing[c][slot * page:(slot + 1) * page])
    k, v = (torch.randn(pages, hkv, page, d, generator=g).to(dtype) for _ in range(2))

    def row(b, p):
        return rows[b][p // page], p % page
    if spoil is not None:
        spoil(k, v, row)
    q = torch.randn(B, n, hq, d, generator=g).to(dtype)
    words = [tree(n, rng) for _ in range(B)] if mask == "tree" else mask
    if layout == "plain":
        dk, dv, dq = k.cuda(), v.cuda(), q.cuda()
    else:
        dk, dv = (t.transpose(1, 2).contiguous().cuda().transpose(1, 2) for t in (k, v))
        dq = torch.cat([q, q], 2).cuda()[:, :, :hq]
    m = None if words is None else torch.tensor([[signed(w) for w in r] for r in words], dtype=torch.int64).cuda()
    cu = [0]
    for t in tails:
        cu.append(cu[-1] + len(t))
    out, lse = ns.attend_shared(dq, dk, dv, table.cuda(), lengths.cuda(), i32(seqs), i32(cu if groups is None else groups),
                                mask=m, max_len=max_len)
    assert out.dtype == dtype and out.shape == q.shape
    assert ns.ops_error(clear=True) == (flags | (ns.FLAG_BAD_ID if gone else 0))
    out, lse = out.cpu(), lse.cpu()
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
        sees &= ~torch.tensor(missing[b], dtype=torch.bool)
        for h in range(hkv):
            kk, vv = k[ip, h, ir], v[ip, h, ir]
            for x in range(hq // hkv):
                hh = h * (hq // hkv) + x
                o, z, to, tz = attend_rows(q[b, :, hh], kk, torch.where(torch.isfinite(vv), vv, 0.0), sees,
                                           d ** -0.5)
                o = with_wild_values(o, vv, sees)
                check(out[b, :, hh], o, to, f"out of sequence {b} head {hh}")
                check(lse[b, :, hh], z, tz, f"lse of sequence {b} head {hh}")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("prompt", [1, 100, 127, 128, 129, 383, 384, 1000])
def test_prompt_lengths(ns, dtype, d, prompt):
    run(ns, [prompt], [[1, 5, 200, 30]], 1, 8, 2, d, dtype, 16, prompt + d)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (7, 1), (14, 2), (8, 8), (16, 1), (32, 8), (28, 4), (33, 1), (130, 1)])
@pytest.mark.parametrize("n", [1, 3])
def test_heads(ns, hq, hkv, n):
    run(ns, [300, 140], [[n, 20, n + 1], [n + 300, 9 + n]], n, hq, hkv, 128, BF16, 16, 2)


@pytest.mark.parametrize("page", [8, 32, 128, 1024])
@pytest.mark.parametrize("n,mask", [(1, None), (40, "tree")])
def test_pages(ns, page, n, mask):
    run(ns, [2100], [[n, n + 100, n + 1100]], n, 4, 1, 64, F16, page, page, mask)


@pytest.mark.parametrize("n,mask", [(2, None), (17, "tree"), (60, "tree"), (64, None)])
def test_new_tokens(ns, n, mask):
    run(ns, [700, 260], [[n, n + 3, 200 + n], [n + 1] * 4], n, 8, 2, 128, BF16, 16, n, mask)
    run(ns, [700, 260], [[n, n + 3, 200 + n], [n + 1] * 4], n, 12, 4, 64, F16, 16, n, mask, layout="strided")


@pytest.mark.parametrize("n", [1, 60])
def test_calls_that_do_not_share(ns, n):
    """Few keys in all, or many rows: attend_paged's kernels, with the groups looked at all the same."""
    run(ns, [700, 260], [[n, n + 3, 200 + n], [n + 1] * 4], n, 8, 2, 128, BF16, 16, 20, wide=False)
    run(ns, [300, 300, 140], [[n, n + 1], [n + 2], [n, n]], n, 4, 1, 64, BF16, 16, 10, groups=[0, 3, 2, 5],
        flags=ns.FLAG_BAD_SEQ, wide=False)


def test_many_members_and_groups(ns):
    """Rows of a group over several items; groups of one; prompts that share nothing whole."""
    run(ns, [520], [[1 + i % 7 for i in range(100)]], 1, 4, 1, 128, BF16, 16, 3)
    run(ns, [520, 60, 1030, 140], [[9], [3, 4], [1] * 20, [2, 2, 2]], 1, 8, 2, 128, F16, 16, 4)
    run(ns, [140] * 40, [[1, 2]] * 40, 1, 2, 1, 64, BF16, 16, 5)


def test_long_prefix(ns):
    """A prefix over many CTAs: dozens of parts to a row."""
    run(ns, [9000], [[1, 2, 150]], 1, 4, 1, 128, BF16, 64, 6, max_len=9150)
    run(ns, [5000], [[60, 61, 64]], 60, 2, 1, 64, BF16, 16, 7, "tree")


def test_empty_groups_and_empty_sequences(ns):
    run(ns, [0, 300, 0, 300], [[], [1, 4], [], [2, 2, 2]], 1, 4, 1, 64, BF16, 16, 8)
    run(ns, [0, 260], [[0, 0], [1, 1]], 1, 4, 1, 64, F16, 16, 9)  # sequences that hold nothing


def test_groups_that_are_not_as_they_should_be(ns):
    for groups in ([0, 3, 2, 5], [1, 2, 3, 5], [0, 2, 3, 4], [0, 9, 9, 5], [0, -1, 3, 5]):
        run(ns, [300, 300, 140], [[1, 2], [3], [4, 5]], 1, 4, 1, 64, BF16, 16, 10, groups=groups,
            flags=ns.FLAG_BAD_SEQ)
    run(ns, [300, 300, 140], [[1, 2], [3], [4, 5]], 1, 4, 1, 64, BF16, 16, 10, groups=[0, 5])  # as they should not be, yet right


def test_rows_that_see_nothing_and_masks(ns):
    n = 20
    words = [[0] * n, [1 << i for i in range(n)], [(1 << (i + 1)) - 1 for i in range(n)]]
    run(ns, [0], [[n, n, n]], n, 4, 1, 64, BF16, 8, 11, words)
    run(ns, [256], [[n, n, n + 7]], n, 4, 1, 64, BF16, 8, 12, words)


@pytest.mark.parametrize("d", [64, 128])
def test_values_that_are_not_finite(ns, d):
    """In the prefix everyone sees them; among new tokens only the rows that the mask lets; behind the end no one."""
    n, L = 20, 300

    def spoil(k, v, row):
        i, r = row(0, 5)
        v[i, 0, r, 3] = float("inf")
        i, r = row(0, L + n - 2)
        v[i, 0, r, 7] = float("nan")
        i, r = row(1, L + n - 1)
        v[i, 0, r, d - 1] = -float("inf")
        i, r = row(1, L + n - 1)
        if r + 1 < 16:
            v[i, 0, r + 1:] = float("nan")
            k[i, 0, r + 1:] = float("nan")
    run(ns, [L], [[n, n]], n, 4, 1, d, BF16, 16, 13, "tree", spoil=spoil)


def test_pages_out_of_range(ns):
    run(ns, [600], [[5, 70, 200]], 1, 4, 1, 128, BF16, 16, 14, gone=[(0, 3), (1, 38)])
    run(ns, [600], [[65, 70, 200]], 40, 2, 1, 64, F16, 32, 15, "tree", gone=[(0, 4), (2, 22)])


def test_sequences_out_of_range_end_their_groups_sharing(ns):
    g = torch.Generator(device="cuda").manual_seed(1)
    cache = ns.KvPages.new(1, 100, 2, 16, 64, 4, 1 << 16)
    cache.extend(i32([0]), i32([300]))
    cache.k.normal_(generator=g), cache.v.normal_(generator=g)
    cache.fork(i32([0, 0]), i32([1, 2]))
    q = torch.randn(4, 1, 8, 64, generator=g, device="cuda").to(BF16)
    out, lse = cache.attend(0, q, i32([0, 1, 9, 2]), groups=i32([0, 4]))
    assert ns.ops_error(clear=True) == ns.FLAG_BAD_SEQ
    assert (out[2] == 0).all() and (lse[2] == -float("inf")).all()
    want, wl = cache.attend(0, q[[0, 1, 3]], i32([0, 1, 2]))
    assert torch.allclose(out[[0, 1, 3]].float(), want.float(), rtol=2 ** -7, atol=2 ** -7)
    assert torch.allclose(lse[[0, 1, 3]], wl, rtol=0, atol=1e-4) and ns.ops_error() == 0


def test_after_a_fork_twice_the_same_bits_and_from_a_graph(ns):
    g = torch.Generator(device="cuda").manual_seed(2)
    cache = ns.KvPages.new(2, 400, 4, 16, 128, 10, 1 << 16)
    cache.k.normal_(generator=g), cache.v.normal_(generator=g)
    own, kids = i32([0, 1]), list(range(2, 10))
    cache.extend(own, i32([700, 333]))
    cache.fork(i32([0] * 4 + [1] * 4), i32(kids))
    cache.extend(i32(kids), i32([1, 5, 9, 60, 1, 2, 3, 4]))
    seqs, groups = i32(kids), i32([0, 4, 8])
    q = torch.randn(8, 1, 28, 128, generator=g, device="cuda").to(BF16)
    a, al = cache.attend(1, q, seqs, groups=groups)
    b, bl = cache.attend(1, q, seqs, groups=groups)
    assert torch.equal(a, b) and torch.equal(al, bl)
    w, wl = cache.attend(1, q, seqs)
    assert (a.float() - w.float()).norm() / w.float().norm() < 0.01 and (al - wl).abs().max() < 1e-4
    out = torch.empty_like(a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.attend(1, q, seqs, groups=groups, out=out)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c, _ = cache.attend(1, q, seqs, groups=groups, stream=s)
    s.synchronize()
    assert torch.equal(c, a)
    need = ns.load_library().ns_attend_shared_workspace(8, 2, 1, 28, 4, 128)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    c, _ = cache.attend(1, q, seqs, groups=groups, workspace=ws)
    assert torch.equal(c, a)
    # two calls at once, each with its own workspace
    outs = []
    for st in (s, torch.cuda.Stream()):
        st.wait_stream(torch.cuda.current_stream())
        for _ in range(4):
            outs.append(cache.attend(1, q, seqs, groups=groups, stream=st)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(x, a) for x in outs) and ns.ops_error() == 0


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d,page", [(64, 8), (128, 16), (128, 64)])
@pytest.mark.parametrize("n", [1, 5, 20])
def test_eight_bits(ns, dtype, d, page, n):
    """A cache of 8 bits, its members after a fork, against what its codes stand for (test_gpu_attention8's bounds beyond
    16 rows)."""
    g = torch.Generator().manual_seed(n + d)
    prompts, tails = [700, 150], [[n, n + 40, n + 7], [n, n + 3]]
    kids = [(i, t) for i, ts in enumerate(tails) for t in ts]
    cache = ns.KvPages.new(2, 400, 2, page, d, 7, (1 << 20) // page, scaled=True)
    for t in (cache.k, cache.v):
        t.view(torch.uint8).fill_(0x7f)  # what no row stands on may be anything
    cache.k_exp.fill_(255), cache.v_exp.fill_(255)
    rows = {}

    def write(seq, count, upto):
        cu = torch.tensor([0, count], dtype=torch.int32, device="cuda")
        k, v = ((torch.randn(count, 2, d, generator=g) * torch.exp(torch.randn(count, 2, 1, generator=g))).to(dtype)
                for _ in range(2))
        cache.write(1, i32([seq]), cu, k.cuda(), v.cuda())
        rows[seq] = [torch.cat((a, values(*quantise(b)))) for a, b in zip(rows.get(seq, [torch.empty(0, 2, d).double()] * 2),
                                                                          (k, v))]

    cache.extend(i32([0, 1]), i32(prompts))
    for i, p in enumerate(prompts):
        write(i, p, p)
    cache.fork(i32([i for i, _ in kids]), i32(list(range(2, 7))))
    cache.extend(i32(list(range(2, 7))), i32([t for _, t in kids]))
    for b, (i, t) in enumerate(kids):
        rows[2 + b] = list(rows[i])
        write(2 + b, t, t)
    hq = 8
    q = torch.randn(5, n, hq, d, generator=g).to(dtype)
    out, lse = cache.attend(1, q.cuda(), i32(list(range(2, 7))), groups=i32([0, 3, 5]))
    assert ns.ops_error() == 0
    out, lse = out.cpu(), lse.cpu()
    for b in range(5):
        k, v = rows[2 + b]
        L = len(k)
        sees = torch.ones(n, L, dtype=torch.bool)
        sees[:, L - n:] = torch.ones(n, n, dtype=torch.bool).tril()
        for h in range(hq):
            kk, vv = k[:, h // 4], v[:, h // 4]
            o, z, to, tz = attend_rows(q[b, :, h], kk, vv, sees, d ** -0.5)
            if dtype == F16:
                more = 2.0 ** -25 * d ** -0.5 * q[b, :, h].double().abs().sum(-1)
                to = to + 2 * more[:, None] * vv.abs().amax() + 2.0 ** -31 * (sees.double() @ vv.abs()) + 2.0 ** -25
                tz = tz + more
            check(out[b, :, h], o, to, f"out of {b} head {h}")
            check(lse[b, :, h], z, tz, f"lse of {b} head {h}")


def test_refusals(ns):
    cache = ns.KvPages.new(1, 8, 2, 16, 64, 4, 2)
    q, seqs = torch.zeros(4, 2, 4, 64, dtype=BF16, device="cuda"), i32([0, 1, 2, 3])
    args = (cache.k[0], cache.v[0], cache.table, cache.lengths, seqs)
    groups = i32([0, 2, 4])
    call = lambda q=q, groups=groups, **kw: ns.attend_shared(q, *args, groups, **kw)
    bad = [
        lambda: call(groups=i32([])),
        lambda: call(groups=i32([0])),
        lambda: call(groups=i32([[0, 4]])),
        lambda: call(groups=groups.long()),
        lambda: call(groups=groups.cpu()),
        lambda: call(groups=i32([0] * 514)),
        lambda: call(q=torch.zeros(4, 3, 4, 64, dtype=BF16, device="cuda")[:, :2]),
        lambda: call(q=q.float()),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            f()
            pytest.fail(f"call {i} was not refused")
    for f in (lambda: call(q=torch.zeros(4 * 2 * 4 * 64 + 4, dtype=BF16, device="cuda")[4:].view(4, 2, 4, 64)),
              lambda: call(workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ns.NanoSpecError):
            f()
    none = ns.attend_shared(q[:0], *args[:4], seqs[:0], i32([0]))
    assert none[0].shape == (0, 2, 4, 64)
    assert ns.ops_error() == 0


@pytest.mark.parametrize("n,hq", [(1, 4), (3, 4), (60, 4)])
def test_many_sequences_that_do_not_share(ns, n, hq):
    """Calls of few keys whose items are too many for clusters (and of many rows): the groups are looked at there too."""
    tails = [[n, n + 1]] * 20
    run(ns, [140] * 20, tails, n, hq, 2, 64, BF16, 16, 21, wide=False)
    for groups in ([0, 20, 10, 40], [1, 40], [0, 39]):
        run(ns, [140] * 20, tails, n, hq, 2, 64, BF16, 16, 21, groups=groups, flags=ns.FLAG_BAD_SEQ, wide=False)


def test_groups_of_eight_bits_that_are_not_as_they_should_be(ns):
    for B in (3, 60):  # (clusters, the line)
        cache = ns.KvPages.new(1, 4 * B, 2, 16, 64, B, 4, scaled=True)
        seqs, count = i32(list(range(B))), i32([50] * B)
        cache.extend(seqs, count)
        x = torch.randn(50 * B, 2, 64, device="cuda").to(BF16)
        cache.write(0, seqs, i32(list(range(0, 50 * B + 1, 50))), x, x)
        for n in (1, 4, 40):
            q = torch.randn(B, n, 8, 64, device="cuda").to(BF16)
            want, _ = cache.attend(0, q, seqs)
            out, _ = cache.attend(0, q, seqs, groups=i32([0, 1, B]))
            assert ns.ops_error() == 0 and (torch.equal(out, want) or 16 < 4 * n <= 128)
            out, _ = cache.attend(0, q, seqs, groups=i32([0, 2, 1, B]))
            assert ns.ops_error(clear=True) == ns.FLAG_BAD_SEQ and (torch.equal(out, want) or 16 < 4 * n <= 128)
