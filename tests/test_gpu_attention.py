"""attend_prompt and attend_paged against softmax attention in 64 bits."""

import random

import pytest
import torch

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


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(dtype)


# ---------------------------------------------------------------------------
# Whole prompts
# ---------------------------------------------------------------------------
def run_prompt(ns, lens, hq, hkv, d, dtype, seed, layout="packed", std=1.0, poison=None, scale=None, max_len=None):
    g = gen(seed)
    T = sum(lens)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    q, k, v = normal(g, (T, hq, d), dtype, std), normal(g, (T, hkv, d), dtype, std), normal(g, (T, hkv, d), dtype)
    if poison is not None:
        poison(q, k, v, cu)
    if layout == "packed":
        dq, dk, dv = q.cuda(), k.cuda(), v.cuda()
    elif layout == "fused":  # slices of one projection's rows
        row = torch.cat([q, k, v], 1).cuda()
        dq, dk, dv = row[:, :hq], row[:, hq:hq + hkv], row[:, hq + hkv:]
    else:  # heads outermost
        dq, dk, dv = (t.transpose(0, 1).contiguous().cuda().transpose(0, 1) for t in (q, k, v))
    scale = d ** -0.5 if scale is None else scale
    out, lse = ns.attend_prompt(dq, dk, dv, torch.tensor(cu, dtype=torch.int32).cuda(),
                                max(lens) if max_len is None else max_len, scale=scale)
    out, lse = out.cpu(), lse.cpu()
    for a, b in zip(cu[:-1], cu[1:]):
        sees = torch.ones(b - a, b - a, dtype=torch.bool).tril()
        for h in range(hq):
            kh = h // (hq // hkv)
            o, z, to, tz = attend_rows(q[a:b, h], k[a:b, kh], v[a:b, kh], sees, scale)
            check(out[a:b, h], o, to, f"out of {a}:{b} head {h}")
            check(lse[a:b, h], z, tz, f"lse of {a}:{b} head {h}")
    assert ns.ops_error() == 0


EDGES = [0, 1, 2, 0, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257, 0]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_lengths(ns, dtype, d):
    run_prompt(ns, EDGES, 4, 2, d, dtype, 1)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (7, 1), (14, 2), (8, 8), (16, 1), (12, 4), (32, 1), (33, 1), (20, 1)])
def test_prompt_heads(ns, hq, hkv):
    run_prompt(ns, [70, 1, 130], hq, hkv, 128, BF16, 2)
    run_prompt(ns, [70, 1, 130], hq, hkv, 64, F16, 3)


@pytest.mark.parametrize("layout", ["fused", "heads"])
def test_prompt_strides(ns, layout):
    run_prompt(ns, [33, 129, 300], 6, 2, 128, BF16, 4, layout)
    run_prompt(ns, [33, 129, 300], 6, 2, 64, F16, 5, layout)


@pytest.mark.parametrize("n", [511, 513, 1000, 1537])
def test_prompt_longer(ns, n):
    run_prompt(ns, [n, 3], 3, 1, 128, BF16, n)
    run_prompt(ns, [n, 3], 2, 1, 64, F16, n)


def test_prompt_peaked_scores(ns):
    """Scores of a few hundred: one key has nearly all the probability."""
    run_prompt(ns, [300, 90], 2, 1, 128, BF16, 6, std=6.0)
    run_prompt(ns, [300, 90], 2, 1, 128, F16, 7, std=6.0)


def test_prompt_rising_and_falling_scores(ns):
    """The running maximum grows with every key, or was largest at the first."""
    def ramp(sign):
        def f(q, k, v, cu):
            for a, b in zip(cu[:-1], cu[1:]):
                q[a:b] = 1.0
                k[a:b] = (sign * torch.arange(b - a) / 16.0)[:, None, None].to(k.dtype)
        return f
    run_prompt(ns, [700], 2, 1, 128, BF16, 8, poison=ramp(1.0))
    run_prompt(ns, [700], 2, 1, 128, BF16, 9, poison=ramp(-1.0))


def test_prompt_lowest_values(ns):
    """Scores near the type's lowest value for some keys (a mask by addition ends there)."""
    def low(q, k, v, cu):
        q[:, :, 1:] = 0
        q[:, :, 0] = 1.0
        k[:, :, 0] = torch.where(torch.arange(k.shape[0])[:, None] % 3 == 1, torch.finfo(k.dtype).min, 0.5).to(k.dtype)
    run_prompt(ns, [200, 70], 2, 1, 64, BF16, 10, poison=low)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), float("-inf")])
def test_prompt_wild_values_reach_only_rows_that_see_them(ns, d, what):
    """Values that are not finite: rows before them, and other sequences, do not see them."""
    def wild(q, k, v, cu):
        v[cu[1] + 70, 0, 5] = what
        v[cu[2] - 1, 0, d - 1] = what
        v[cu[3], 0, 0] = what
    # the reference says NaN for every row that sees one; an infinity alone gives infinities there
    g = gen(11)
    lens, hq = [40, 150, 64, 200], 2
    cu = [0, 40, 190, 254, 454]
    q, k, v = normal(g, (454, hq, d), BF16), normal(g, (454, 1, d), BF16), normal(g, (454, 1, d), BF16)
    wild(q, k, v, cu)
    out, lse = ns.attend_prompt(q.cuda(), k.cuda(), v.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(), max(lens))
    out = out.cpu()
    for a, b in zip(cu[:-1], cu[1:]):
        sees = torch.ones(b - a, b - a, dtype=torch.bool).tril()
        for h in range(hq):
            o, z, to, tz = attend_rows(q[a:b, h], k[a:b, 0], v[a:b, 0], sees, d ** -0.5)
            bad = torch.isnan(o)
            assert not torch.isfinite(out[a:b, h][bad]).any()
            check(out[a:b, h].double().masked_fill(bad, 0), o.masked_fill(bad, 0), to, "rows that see none")


def test_prompt_wild_keys_of_other_rows(ns):
    """Keys that are not finite: rows before them, and other sequences, are as without them."""
    g = gen(12)
    cu = [0, 100, 230]
    q, k, v = normal(g, (230, 2, 128), BF16), normal(g, (230, 1, 128), BF16), normal(g, (230, 1, 128), BF16)
    bounds = torch.tensor(cu, dtype=torch.int32).cuda()
    clean, _ = ns.attend_prompt(q.cuda(), k.cuda(), v.cuda(), bounds, 130)
    k[90:100], k[200:230] = float("nan"), float("inf")
    out, _ = ns.attend_prompt(q.cuda(), k.cuda(), v.cuda(), bounds, 130)
    assert torch.equal(out[:90], clean[:90]) and torch.equal(out[100:200], clean[100:200])
    assert torch.isnan(out[95]).all()


def test_prompt_bound_on_lengths(ns):
    """max_len only bounds: a larger one changes nothing; tokens past a smaller one are left and flagged."""
    g = gen(13)
    q, k, v = normal(g, (300, 2, 64), BF16).cuda(), normal(g, (300, 2, 64), BF16).cuda(), normal(g, (300, 2, 64), BF16).cuda()
    cu = torch.tensor([0, 100, 300], dtype=torch.int32).cuda()
    a, la = ns.attend_prompt(q, k, v, cu, 200)
    b, lb = ns.attend_prompt(q, k, v, cu, 5000)
    assert torch.equal(a, b) and torch.equal(la, lb) and ns.ops_error() == 0
    ns.attend_prompt(q, k, v, cu, 150)
    assert ns.ops_error(clear=True) == ns.FLAG_BAD_SEQ


def test_prompt_offsets_past_32_bits(ns):
    """Token strides that put the last rows past 2^32 elements."""
    T, step = 520, 1 << 23
    g = gen(14)
    vals = [normal(g, (T, 1, 64), BF16) for _ in range(3)]
    buf = torch.empty(T * step, dtype=BF16, device="cuda")
    views = []
    for i, t in enumerate(vals):
        w = buf.as_strided((T, 1, 64), (step, 64, 1), i * 64)
        w.copy_(t)
        views.append(w)
    cu = torch.tensor([0, T], dtype=torch.int32).cuda()
    out, lse = ns.attend_prompt(*views, cu, T)
    want, wl = ns.attend_prompt(*(t.cuda() for t in vals), cu, T)
    assert torch.equal(out, want) and torch.equal(lse, wl)


def test_prompt_other_stream_and_outputs(ns):
    g = gen(15)
    q, k, v = (normal(g, (100, 2, 128), F16).cuda() for _ in range(3))
    cu = torch.tensor([0, 60, 100], dtype=torch.int32).cuda()
    want, wl = ns.attend_prompt(q, k, v, cu, 60)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = torch.empty_like(want), torch.empty_like(wl)
    r = ns.attend_prompt(q, k, v, cu, 60, out=out, lse=lse, stream=s)
    s.synchronize()
    assert r[0] is out and torch.equal(out, want) and torch.equal(lse, wl)


def test_prompt_repeats_bit_for_bit(ns):
    g = gen(16)
    q, k, v = normal(g, (900, 8, 128), BF16).cuda(), normal(g, (900, 2, 128), BF16).cuda(), normal(g, (900, 2, 128), BF16).cuda()
    cu = torch.tensor([0, 650, 900], dtype=torch.int32).cuda()
    a, la = ns.attend_prompt(q, k, v, cu, 650)
    for _ in range(5):
        b, lb = ns.attend_prompt(q, k, v, cu, 650)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_prompt_refusals(ns):
    q = torch.zeros(10, 4, 64, dtype=BF16, device="cuda")
    k = torch.zeros(10, 2, 64, dtype=BF16, device="cuda")
    cu = torch.tensor([0, 10], dtype=torch.int32, device="cuda")
    bad = [
        lambda: ns.attend_prompt(q.float(), k.float(), k.float(), cu, 10),
        lambda: ns.attend_prompt(q, k.half(), k, cu, 10),
        lambda: ns.attend_prompt(q, k[:, :, :32], k[:, :, :32], cu, 10),
        lambda: ns.attend_prompt(q[:, :3], k, k, cu, 10),
        lambda: ns.attend_prompt(q, k, k, cu.long(), 10),
        lambda: ns.attend_prompt(q, k, k, cu.cpu(), 10),
        lambda: ns.attend_prompt(q.cpu(), k, k, cu, 10),
        lambda: ns.attend_prompt(q, k, k, cu, 10, out=torch.empty(10, 4, 64, device="cuda")),
        lambda: ns.attend_prompt(q.transpose(1, 2), k, k, cu, 10),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    worse = [
        lambda: ns.attend_prompt(q, k, k, cu, -1),
        lambda: ns.attend_prompt(q, k, k, cu, 10, scale=0.0),
        lambda: ns.attend_prompt(q, k, k, cu, 10, scale=float("nan")),
        lambda: ns.attend_prompt(torch.zeros(10, 4, 32, dtype=BF16, device="cuda"),
                                 *[torch.zeros(10, 2, 32, dtype=BF16, device="cuda")] * 2, cu, 10),
        # rows that begin off a 16-byte boundary
        lambda: ns.attend_prompt(torch.zeros(10, 4, 65, dtype=BF16, device="cuda")[:, :, 1:], k, k, cu, 10),
        lambda: ns.attend_prompt(q, torch.zeros(10, 2, 68, dtype=BF16, device="cuda")[:, :, :64], k, cu, 10),
    ]
    for f in worse:
        with pytest.raises(ns.NanoSpecError):
            f()
    assert ns.attend_prompt(q[:0], k[:0], k[:0], cu[:1], 0)[0].shape == (0, 4, 64)
    # bounds that leave the tokens are skipped and flagged
    ns.attend_prompt(q, k, k, torch.tensor([0, 11], dtype=torch.int32, device="cuda"), 10)
    assert ns.ops_error(clear=True) == ns.FLAG_BAD_SEQ


# ---------------------------------------------------------------------------
# New tokens over a paged cache
# ---------------------------------------------------------------------------
def make_cache(g, rng, lens, hkv, P, d, dtype, layout="heads", spare=3):
    """A pool whose unused rows hold NaN, the sequences' keys and values, and their table."""
    held = [-(-n // P) for n in lens]
    pages = sum(held) + spare
    order = list(range(pages))
    rng.shuffle(order)
    table = torch.full((len(lens), max(held + [1]) + 2), -1, dtype=torch.int32)
    kp = torch.full((pages, hkv, P, d), float("nan"), dtype=dtype)
    vp = torch.full((pages, hkv, P, d), float("nan"), dtype=dtype)
    keys, vals, at = [], [], 0
    for b, n in enumerate(lens):
        k, v = normal(g, (n, hkv, d), dtype), normal(g, (n, hkv, d), dtype)
        keys.append(k)
        vals.append(v)
        for slot in range(held[b]):
            page = order[at]
            at += 1
            table[b, slot] = page
            m = min(P, n - slot * P)
            kp[page, :, :m] = k[slot * P:slot * P + m].transpose(0, 1)
            vp[page, :, :m] = v[slot * P:slot * P + m].transpose(0, 1)
    if layout == "tokens":  # [pages, page, heads, dim] in memory
        dk, dv = (t.transpose(1, 2).contiguous().cuda().transpose(1, 2) for t in (kp, vp))
    elif layout == "joint":  # keys and values of a page next to each other
        both = torch.stack([kp, vp], 1).cuda()
        dk, dv = both[:, 0], both[:, 1]
    else:
        dk, dv = kp.cuda(), vp.cuda()
    return dk, dv, table, keys, vals


def tree_masks(rng, B, n):
    rows = []
    for _ in range(B):
        bits = []
        for i in range(n):
            parent = rng.randrange(-1, i) if i else -1
            bits.append((1 << i) | (bits[parent] if parent >= 0 else 0))
        rows.append(bits)
    return rows


def signed(rows):
    return torch.tensor([[b - (1 << 64) if b >> 63 else b for b in r] for r in rows], dtype=torch.int64)


def run_paged(ns, lens, n, hq, hkv, d, P, dtype, seed, layout="heads", masks=None, max_len=0, order=None):
    g, rng = gen(seed), random.Random(seed)
    dk, dv, table, keys, vals = make_cache(g, rng, lens, hkv, P, d, dtype, layout)
    order = list(range(len(lens))) if order is None else order
    B = len(order)
    q = normal(g, (B, n, hq, d), dtype)
    if masks == "tree":
        masks = tree_masks(rng, B, n)
    out, lse = ns.attend_paged(q.cuda(), dk, dv, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                               torch.tensor(order, dtype=torch.int32).cuda(),
                               mask=None if masks is None else signed(masks).cuda(), max_len=max_len)
    out, lse = out.cpu(), lse.cpu()
    grp = hq // hkv
    for b, s in enumerate(order):
        N = lens[s]
        sees = torch.zeros(n, N, dtype=torch.bool)
        for i in range(n):
            word = (1 << (i + 1)) - 1 if masks is None else masks[b][i]
            for p in range(N):
                j = p - (N - n)
                sees[i, p] = j < 0 or bool(word >> j & 1)
        for h in range(hq):
            o, z, to, tz = attend_rows(q[b, :, h], keys[s][:, h // grp], vals[s][:, h // grp], sees, d ** -0.5)
            check(out[b, :, h], o, to, f"out of sequence {s} head {h}")
            check(lse[b, :, h], z, tz, f"lse of sequence {s} head {h}")
    assert ns.ops_error() == 0


RAGGED = [1, 2, 7, 8, 9, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 300]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("P", [8, 16, 64, 256])
def test_paged_one_token(ns, dtype, d, P):
    run_paged(ns, RAGGED, 1, 8, 2, d, P, dtype, P + d)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (7, 1), (28, 4), (8, 8), (16, 1), (17, 1), (32, 1), (64, 1)])
def test_paged_heads(ns, hq, hkv):
    run_paged(ns, [5, 200, 1], 1, hq, hkv, 128, 16, BF16, hq)
    run_paged(ns, [5, 200, 1], 1, hq, hkv, 64, 32, F16, hq)


@pytest.mark.parametrize("n", [2, 3, 5, 16, 17, 33, 63, 64])
def test_paged_chain_of_new_tokens(ns, n):
    run_paged(ns, [n, n + 1, n + 63, n + 64, 200 + n], n, 4, 1, 128, 16, BF16, n)
    run_paged(ns, [n, n + 130], n, 2, 2, 64, 8, F16, n)


@pytest.mark.parametrize("n", [1, 4, 10, 60, 64])
def test_paged_draft_tree(ns, n):
    run_paged(ns, [n, n + 1, n + 100, n + 517], n, 8, 2, 128, 16, BF16, n, masks="tree")
    run_paged(ns, [n, n + 77], n, 7, 1, 64, 64, F16, n, masks="tree")


@pytest.mark.parametrize("layout", ["tokens", "joint"])
def test_paged_cache_layouts(ns, layout):
    run_paged(ns, [100, 1, 333], 1, 8, 2, 128, 16, BF16, 21, layout)
    run_paged(ns, [100, 33, 333], 20, 8, 2, 64, 32, F16, 22, layout, masks="tree")


@pytest.mark.parametrize("hq,hkv", [(3, 1), (7, 1), (20, 1), (33, 1), (64, 2), (4, 4)])
@pytest.mark.parametrize("n", [6, 37, 64])
def test_paged_many_rows(ns, hq, hkv, n):
    """Heads that fill their row tiles unevenly, and pages of every kind of size against a tile."""
    run_paged(ns, [n, n + 128, n + 300], n, hq, hkv, 64, 256, BF16, n + hq, masks="tree")
    run_paged(ns, [n + 127, n + 1], n, hq, hkv, 128, 128, F16, n + hq)
    run_paged(ns, [n + 255, 0, n - 1], n, hq, hkv, 128, 8, BF16, n + hq)


def test_paged_queries_off_16_byte_boundaries(ns):
    """Queries that begin off a 16-byte boundary, and with odd strides of pairs, give what aligned ones give."""
    g, rng = gen(40), random.Random(40)
    lens, n = [300, 64, 41], 40
    dk, dv, table, _, _ = make_cache(g, rng, lens, 2, 16, 64, BF16)
    q = normal(g, (3, n, 8, 64), BF16).cuda()
    masks = signed(tree_masks(rng, 3, n)).cuda()
    rest = (dk, dv, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
            torch.tensor([0, 1, 2], dtype=torch.int32).cuda())
    want, wl = ns.attend_paged(q, *rest, mask=masks)
    wide = torch.zeros((3, n, 8, 70), dtype=BF16, device="cuda")[..., 2:66]
    wide.copy_(q)
    out, lse = ns.attend_paged(wide, *rest, mask=masks)
    # both are within their bounds of the exact result: twice the roundings of p and o apart at most
    assert (out.float() - want.float()).abs().max() <= 4 * 2.0 ** -8 * want.float().abs().max()
    assert (lse - wl).abs().max() < 1e-3
    few, fl = ns.attend_paged(wide[:, :2], *rest)
    want, wl = ns.attend_paged(q[:, :2], *rest)
    assert torch.equal(few, want) and torch.equal(fl, wl) and ns.ops_error() == 0


def test_paged_empty_sequences_and_rows(ns):
    """Lengths of zero, fewer positions than new tokens, and masks that leave nothing."""
    run_paged(ns, [0, 40, 0, 1], 1, 8, 2, 128, 16, BF16, 23)
    run_paged(ns, [0, 2, 5, 80], 5, 8, 2, 128, 16, BF16, 24)
    nothing = [[0, 1, 0, 7, 0]] * 3
    run_paged(ns, [5, 4, 90], 5, 4, 1, 64, 8, F16, 25, masks=nothing)
    run_paged(ns, [1, 30], 1, 4, 1, 64, 8, F16, 26, masks=[[0], [0]])


def test_paged_sequences_in_any_order(ns):
    run_paged(ns, [30, 500, 7, 64, 129], 1, 8, 2, 128, 16, BF16, 27, order=[3, 0, 4])


@pytest.mark.parametrize("max_len", [1, 100, 1 << 20])
def test_paged_bound_only_sizes_the_launch(ns, max_len):
    run_paged(ns, [700, 3, 64], 1, 8, 2, 128, 16, BF16, 28, max_len=max_len)
    run_paged(ns, [700, 30, 64], 9, 8, 2, 128, 16, BF16, 29, max_len=max_len, masks="tree")


@pytest.mark.parametrize("lens", [[5000], [9001, 1], [3333, 2, 4000, 64]])
def test_paged_split_and_joined(ns, lens):
    """Few rows and long caches: every item is shared by many CTAs."""
    run_paged(ns, lens, 1, 4, 1, 128, 16, BF16, 30)
    run_paged(ns, [x + 20 for x in lens], 20, 4, 1, 64, 64, F16, 31, masks="tree")


def test_paged_many_short_sequences(ns):
    rng = random.Random(32)
    run_paged(ns, [rng.randrange(0, 40) for _ in range(700)], 1, 2, 1, 64, 8, BF16, 32)


def test_paged_wild_values_of_hidden_nodes(ns):
    """A tree node whose values are not finite reaches only the nodes that see it."""
    for n, lens in ((10, [10, 150]), (40, [41, 200])):
        g, rng = gen(33), random.Random(33)
        dk, dv, table, keys, vals = make_cache(g, rng, lens, 1, 16, 128, BF16)
        masks = tree_masks(rng, 2, n)
        q = normal(g, (2, n, 4, 128), BF16)
        for b, N in enumerate(lens):
            pos = N - n + n // 2
            vals[b][pos, 0, 3] = float("nan")
            vals[b][N - 1, 0, 64] = float("inf")
            dv[table[b, pos // 16], 0, pos % 16, 3] = float("nan")
            dv[table[b, (N - 1) // 16], 0, (N - 1) % 16, 64] = float("inf")
        out, _ = ns.attend_paged(q.cuda(), dk, dv, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                                 torch.tensor([0, 1], dtype=torch.int32).cuda(), mask=signed(masks).cuda())
        out = out.cpu()
        for b, N in enumerate(lens):
            sees = torch.tensor([[p < N - n or bool(masks[b][i] >> (p - N + n) & 1) for p in range(N)] for i in range(n)])
            for h in range(4):
                o, _, to, _ = attend_rows(q[b, :, h], keys[b][:, 0], vals[b][:, 0], sees, 128 ** -0.5)
                bad = torch.isnan(o)
                assert bad.any() and not bad.all()
                assert not torch.isfinite(out[b, :, h][bad]).any()
                check(out[b, :, h].double().masked_fill(bad, 0), o.masked_fill(bad, 0), to, "nodes that see none")


def test_paged_offsets_past_32_bits(ns):
    """Pages whose elements lie past 2^32."""
    hkv, P, d = 8, 64, 128
    pages = (1 << 32) // (hkv * P * d) + 9
    pool = torch.empty((pages, hkv, P, d), dtype=BF16, device="cuda")
    g = gen(34)
    lens = [200, 130]
    small = normal(g, (8, hkv, P, d), BF16).cuda()
    pool[pages - 8:] = small
    table = torch.tensor([[0, 3, 5, 1], [7, 2, 6, -1]], dtype=torch.int32)
    q = normal(g, (2, 1, 32, d), BF16).cuda()
    le, se = torch.tensor(lens, dtype=torch.int32).cuda(), torch.tensor([0, 1], dtype=torch.int32).cuda()
    want, wl = ns.attend_paged(q, small, small, table.cuda(), le, se)
    far = torch.where(table >= 0, table + (pages - 8), table).cuda()
    out, lse = ns.attend_paged(q, pool, pool, far, le, se)
    assert torch.equal(out, want) and torch.equal(lse, wl) and ns.ops_error() == 0


def test_paged_bad_ids_are_skipped_and_flagged(ns):
    g, rng = gen(35), random.Random(35)
    dk, dv, table, keys, vals = make_cache(g, rng, [100, 60], 2, 16, 64, BF16)
    dk.nan_to_num_(), dv.nan_to_num_()
    q = normal(g, (2, 1, 4, 64), BF16).cuda()
    le, se = torch.tensor([100, 60], dtype=torch.int32).cuda(), torch.tensor([0, 1], dtype=torch.int32).cuda()
    want, _ = ns.attend_paged(q, dk, dv, table.cuda(), le, se)
    t = table.clone()
    t[0, 2] = 1 << 20
    out, _ = ns.attend_paged(q, dk, dv, t.cuda(), le, se)
    assert ns.ops_error(clear=True) == 0x1 and torch.equal(out[1], want[1])
    out, lse = ns.attend_paged(q, dk, dv, table.cuda(), le, torch.tensor([7, 1], dtype=torch.int32).cuda())
    assert ns.ops_error(clear=True) == ns.FLAG_BAD_SEQ and torch.equal(out[1], want[1])
    assert (out[0] == 0).all() and torch.isinf(lse[0]).all()
    out, _ = ns.attend_paged(q, dk, dv, table.cuda(), torch.tensor([-5, 60], dtype=torch.int32).cuda(), se)
    assert ns.ops_error(clear=True) == ns.FLAG_BAD_SEQ and torch.equal(out[1], want[1]) and (out[0] == 0).all()


def test_paged_workspace_stream_and_repeats(ns):
    g, rng = gen(36), random.Random(36)
    lens = [3000, 40]
    dk, dv, table, _, _ = make_cache(g, rng, lens, 2, 16, 128, BF16)
    q = normal(g, (2, 1, 8, 128), BF16).cuda()
    args = (q, dk, dv, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
            torch.tensor([0, 1], dtype=torch.int32).cuda())
    want, wl = ns.attend_paged(*args)
    need = ns.load_library().ns_attend_paged_workspace(2, 1, 8, 2, 128)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        out, lse = ns.attend_paged(*args, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl)
    with pytest.raises(ns.NanoSpecError):
        ns.attend_paged(*args, workspace=ws[:need - 1])


def test_paged_in_a_graph(ns):
    """Captured once, replayed with other lengths."""
    g, rng = gen(37), random.Random(37)
    lens = [900, 300]
    dk, dv, table, keys, vals = make_cache(g, rng, lens, 2, 16, 128, BF16)
    q = normal(g, (2, 1, 8, 128), BF16).cuda()
    table, le = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    se = torch.tensor([0, 1], dtype=torch.int32).cuda()
    ns.attend_paged(q, dk, dv, table, le, se)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = ns.attend_paged(q, dk, dv, table, le, se)
    for new in ([900, 300], [17, 1], [640, 299]):
        le.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        want, wl = ns.attend_paged(q, dk, dv, table, le, se)
        assert torch.equal(out, want) and torch.equal(lse, wl)


def test_paged_refusals(ns):
    q = torch.zeros(2, 1, 4, 64, dtype=BF16, device="cuda")
    k = torch.zeros(6, 2, 16, 64, dtype=BF16, device="cuda")
    i32 = {"dtype": torch.int32, "device": "cuda"}
    t, le, se = torch.zeros(3, 2, **i32), torch.zeros(3, **i32), torch.zeros(2, **i32)
    bad = [
        lambda: ns.attend_paged(q.float(), k, k, t, le, se),
        lambda: ns.attend_paged(q, k.half(), k.half(), t, le, se),
        lambda: ns.attend_paged(q, k, k[:, :1], t, le, se),
        lambda: ns.attend_paged(q[:, :, :3], k, k, t, le, se),
        lambda: ns.attend_paged(q, k, k, t, le[:2], se),
        lambda: ns.attend_paged(q, k, k, t, le, se[:1]),
        lambda: ns.attend_paged(q, k, k, t.long(), le, se),
        lambda: ns.attend_paged(q, k, k, t, le, se, mask=torch.zeros(2, 2, dtype=torch.int64, device="cuda")),
        lambda: ns.attend_paged(q.expand(2, 65, 4, 64), k, k, t, le, se),
        lambda: ns.attend_paged(q.cpu(), k, k, t, le, se),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: ns.attend_paged(q, k[:, :, :12], k[:, :, :12], t, le, se),
              lambda: ns.attend_paged(q, k, k, t, le, se, scale=-1.0),
              lambda: ns.attend_paged(q, k, k, t, le, se, max_len=-1),
              lambda: ns.attend_paged(q[..., :32], k[..., :32], k[..., :32], t, le, se)):
        with pytest.raises(ns.NanoSpecError):
            f()
    assert ns.ops_error() == 0


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d,kinds", [(64, ((2, 1), (4, 2), (16, 2))), (128, ((2, 1), (3, 3), (20, 2)))])
def test_paged_few_rows_by_number_of_sequences(ns, dtype, d, kinds):
    """Up to 16 rows: calls of a few items (each split by a cluster, of 16 or of 8) and of many (one line of tiles)."""
    for seqs, hkv in kinds:
        lens = [(1, 700, 2049, 64, 0, 129, 3)[(i * 5 + seqs) % 7] + 13 * (i // 7) for i in range(seqs)]
        run_paged(ns, lens, 1, 4 * hkv, hkv, d, 16, dtype, 40 + seqs)
        run_paged(ns, [x + 5 for x in lens], 5, 3 * hkv, hkv, d, 64, dtype, 41 + seqs, masks="tree")


def test_paged_cluster_repeats_and_lengths_past_its_bound(ns):
    """A call of one sequence around the longest that its CTAs take as a cluster, with the bound on the lengths low."""
    for n in (8191, 8192, 8193, 16384, 16385):
        run_paged(ns, [n], 1, 16, 8, 64, 64, F16, n)
    run_paged(ns, [20000], 1, 8, 2, 64, 64, F16, 50, max_len=1000)


def test_prompt_strides_of_single_and_repeated_heads(ns):
    g = gen(60)
    q, k, v = normal(g, (70, 4, 64), BF16).cuda(), normal(g, (70, 1, 64), BF16).cuda(), normal(g, (70, 1, 64), BF16).cuda()
    cu = torch.tensor([0, 70], dtype=torch.int32).cuda()
    want, wl = ns.attend_prompt(q, k, v, cu, 70)
    one = [torch.as_strided(t, (70, 1, 64), (64, 0, 1)) for t in (k, v)]  # an axis of one may have any stride
    got, gl = ns.attend_prompt(q, *one, cu, 70)
    assert torch.equal(got, want) and torch.equal(gl, wl)
    with pytest.raises(ns.NanoSpecError):  # two heads that are one in memory
        ns.attend_prompt(q, k.expand(70, 2, 64), v.expand(70, 2, 64), cu, 70)
    a, _ = ns.attend_prompt(q[:1], k[:1], v[:1], cu[:1].repeat(2) + torch.tensor([0, 1], device="cuda", dtype=torch.int32), 1)
    assert torch.equal(a, v[:1].expand(1, 4, 64))


@pytest.mark.parametrize("d,P,dtype", [(128, 16, BF16), (64, 64, F16)])
def test_paged_several_long_items_to_a_cta(ns, d, P, dtype):
    """More rows than 16 and far more tiles than SMs: a CTA has whole items and parts of several tiles in a row.
    (What pages hold behind a sequence's end is NaN.)"""
    lens = [150 + 47 * i for i in range(20)]
    run_paged(ns, lens, 24, 16, 16, d, P, dtype, 61, masks="tree")
    run_paged(ns, lens[::-1], 60, 32, 8, d, P, dtype, 62, masks="tree")


def test_paged_wild_values_of_hidden_nodes_of_long_items(ns):
    """Nodes whose values are not finite, behind contexts of several tiles, several items to a CTA."""
    n, lens, hkv = 24, [200 + 61 * i for i in range(16)], 16
    g, rng = gen(63), random.Random(63)
    dk, dv, table, keys, vals = make_cache(g, rng, lens, hkv, 16, 128, BF16)
    masks = tree_masks(rng, len(lens), n)
    q = normal(g, (len(lens), n, hkv, 128), BF16)
    for b, N in enumerate(lens):
        for pos, col, what in ((N - n // 2, 3, float("nan")), (N - 1, 64, float("-inf"))):
            vals[b][pos, :, col] = what
            dv[table[b, pos // 16], :, pos % 16, col] = what
    out, _ = ns.attend_paged(q.cuda(), dk, dv, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                             torch.arange(len(lens), dtype=torch.int32).cuda(), mask=signed(masks).cuda())
    out = out.cpu()
    for b, N in enumerate(lens):
        sees = torch.tensor([[p < N - n or bool(masks[b][i] >> (p - N + n) & 1) for p in range(N)] for i in range(n)])
        for h in range(hkv):
            o, _, to, _ = attend_rows(q[b, :, h], keys[b][:, h], vals[b][:, h], sees, 128 ** -0.5)
            bad = torch.isnan(o)
            assert not torch.isfinite(out[b, :, h][bad]).any()
            check(out[b, :, h].double().masked_fill(bad, 0), o.masked_fill(bad, 0), to, "nodes that see none")


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_wild_values_late_in_long_sequences(ns, d):
    """Values that are not finite many tiles into a sequence: the rows before them do not see them."""
    g = gen(64)
    lens, hq, hkv = [900, 1100, 400], 32, 4
    cu = [0, 900, 2000, 2400]
    q, k, v = normal(g, (2400, hq, d), BF16), normal(g, (2400, hkv, d), BF16), normal(g, (2400, hkv, d), BF16)
    for pos, col, what in ((850, 5, float("nan")), (899, 0, float("inf")), (900 + 700, 9, float("-inf")), (900 + 1030, 5, float("nan")),
                           (2000 + 390, d - 1, float("nan"))):
        v[pos, :, col] = what
    out, _ = ns.attend_prompt(q.cuda(), k.cuda(), v.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(), max(lens))
    out = out.cpu()
    for a, b in zip(cu[:-1], cu[1:]):
        sees = torch.ones(b - a, b - a, dtype=torch.bool).tril()
        for h in range(hq):
            kh = h // (hq // hkv)
            o, _, to, _ = attend_rows(q[a:b, h], k[a:b, kh], v[a:b, kh], sees, d ** -0.5)
            bad = torch.isnan(o)
            assert not torch.isfinite(out[a:b, h][bad]).any()
            check(out[a:b, h].double().masked_fill(bad, 0), o.masked_fill(bad, 0), to, "rows that see none")


@pytest.mark.parametrize("group", [40, 65, 100, 128, 129])
def test_paged_large_groups(ns, group):
    """Query heads that share a key-value head: up to 128 of them are rows of one tile."""
    run_paged(ns, [30, 400, 0, 129], 1, group, 1, 64, 16, BF16, group)
    run_paged(ns, [33, 500], 7, 2 * group, 2, 128, 32, F16, group, masks="tree")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("hq,hkv,d", [(48, 8, 64), (36, 4, 128), (40, 40, 64), (64, 2, 128)])
def test_prompt_many_items(ns, hq, hkv, d, dtype):
    """Calls whose items are two row tiles each (those of few heads and sequences are one, with its keys split)."""
    run_prompt(ns, EDGES, hq, hkv, d, dtype, 70)


@pytest.mark.parametrize("hq", [2, 64])
def test_prompt_scores_that_rise_by_key_tile(ns, hq):
    """Each tile of 128 keys far above or below the one before, whether or not the tiles are split over two halves."""
    g = gen(71)
    n, d = 700, 64
    q, k, v = normal(g, (n, hq, d), BF16), normal(g, (n, 1, d), BF16), normal(g, (n, 1, d), BF16)
    step = torch.tensor([(0, 60, -40, 80, 10, 90)[i // 128] for i in range(n)], dtype=torch.float32)
    q[:, :, 0] = 8.0
    k[:, 0, 0] = step.to(BF16)
    out, lse = ns.attend_prompt(q.cuda(), k.cuda(), v.cuda(), torch.tensor([0, n], dtype=torch.int32).cuda(), n)
    sees = torch.ones(n, n, dtype=torch.bool).tril()
    for h in range(hq):
        o, z, to, tz = attend_rows(q[:, h], k[:, 0], v[:, 0], sees, d ** -0.5)
        check(out[:, h], o, to, f"out of head {h}")
        check(lse[:, h], z, tz, f"lse of head {h}")


@pytest.mark.parametrize("lens,hq,hkv,d", [([2900], 4, 4, 128), ([1500, 130, 700], 4, 1, 64), ([129, 128, 127, 1], 8, 4, 64)])
def test_prompt_few_long_items(ns, lens, hq, hkv, d):
    """Keys split over the two halves of a CTA: even and odd numbers of tiles, several items to a CTA."""
    run_prompt(ns, lens, hq, hkv, d, BF16, 72)


def run_missing_pages(ns, lens, n, hq, hkv, d, P, dtype, seed, share=0.3, masks=None, unaligned=False, all_of=()):
    """Some page ids out of range: no row sees their positions, and everything else is as it is."""
    g, rng = gen(seed), random.Random(seed)
    dk, dv, table, keys, vals = make_cache(g, rng, lens, hkv, P, d, dtype)
    B = len(lens)
    there = []
    for b, N in enumerate(lens):
        gone = [rng.random() < share or b in all_of for _ in range(-(-N // P))]
        for slot, x in enumerate(gone):
            if x:
                table[b, slot] = rng.choice([-1, -(1 << 31), dk.shape[0], (1 << 31) - 1])
        there.append(torch.tensor([not gone[p // P] for p in range(N)], dtype=torch.bool))
    q = normal(g, (B, n, hq, d), dtype)
    if masks == "tree":
        masks = tree_masks(rng, B, n)
    dq = q.cuda()
    if unaligned:
        dq = torch.zeros((B, n, hq, d + 2), dtype=dtype, device="cuda")[..., 2:]
        dq.copy_(q)
    i32 = {"dtype": torch.int32, "device": "cuda"}
    out, lse = ns.attend_paged(dq, dk, dv, table.cuda(), torch.tensor(lens, **i32), torch.arange(B, **i32),
                               mask=None if masks is None else signed(masks).cuda())
    out, lse = out.cpu(), lse.cpu()
    assert ns.ops_error(clear=True) == (0x1 if not all(t.all() for t in there) else 0)
    for b, N in enumerate(lens):
        sees = torch.zeros(n, N, dtype=torch.bool)
        for i in range(n):
            word = (1 << (i + 1)) - 1 if masks is None else masks[b][i]
            for p in range(N):
                sees[i, p] = p < N - n or bool(word >> (p - N + n) & 1)
        sees &= there[b]
        for h in range(hq):
            kh = h // (hq // hkv)
            o, z, to, tz = attend_rows(q[b, :, h], keys[b][:, kh], vals[b][:, kh], sees, d ** -0.5)
            check(out[b, :, h], o, to, f"out of sequence {b} head {h}")
            check(lse[b, :, h], z, tz, f"lse of sequence {b} head {h}")


@pytest.mark.parametrize("P", [8, 16, 64, 128, 256])
@pytest.mark.parametrize("d,dtype", [(64, F16), (128, BF16)])
def test_paged_missing_pages_are_seen_by_no_row(ns, P, d, dtype):
    few = [700, 1, 130]                                  # clusters
    many = [(300, 40, 777, 64, 129, 8)[i % 6] + i for i in range(40)]  # one line of tiles
    run_missing_pages(ns, few, 1, 4, 2, d, P, dtype, 80 + P)
    run_missing_pages(ns, [5000], 1, 8, 1, d, P, dtype, 81 + P)
    run_missing_pages(ns, many, 1, 4, 4, d, P, dtype, 82 + P)
    run_missing_pages(ns, [x + 5 for x in few], 5, 3, 1, d, P, dtype, 83 + P, masks="tree")
    run_missing_pages(ns, [x + 40 for x in few], 40, 4, 2, d, P, dtype, 84 + P, masks="tree")
    run_missing_pages(ns, [x + 33 for x in few], 33, 4, 2, d, P, dtype, 85 + P, unaligned=True)


def test_paged_sequences_of_missing_pages_only(ns):
    for n, hq, seed in ((1, 4, 90), (20, 8, 91)):
        run_missing_pages(ns, [300, 41, 500], n, hq, 2, 64, 16, BF16, seed, share=0.0, all_of=(0, 2))
        run_missing_pages(ns, [300, 41, 500], n, hq, 2, 128, 16, F16, seed, share=1.0)


def test_paged_missing_pages_of_several_long_items_to_a_cta(ns):
    lens = [150 + 47 * i for i in range(20)]
    run_missing_pages(ns, lens, 24, 16, 16, 64, 16, BF16, 92, share=0.1, masks="tree")
    run_missing_pages(ns, lens, 60, 16, 4, 128, 64, F16, 93, share=0.4, masks="tree")


def test_prompt_tokens_without_sequences_are_refused(ns):
    """A call that could compute nothing of its outputs."""
    q = torch.zeros(10, 4, 64, dtype=BF16, device="cuda")
    k = torch.zeros(10, 2, 64, dtype=BF16, device="cuda")
    cu = torch.tensor([0, 10], dtype=torch.int32, device="cuda")
    for args in ((cu, 0), (cu[1:], 10)):
        with pytest.raises(ValueError):
            ns.attend_prompt(q, k, k, *args)
    assert ns.attend_prompt(q[:0], k[:0], k[:0], cu[:1], 0)[0].shape == (0, 4, 64)
    assert ns.attend_prompt(q[:0], k[:0], k[:0], torch.zeros_like(cu), 0)[1].shape == (0, 4)
    assert ns.ops_error() == 0


@pytest.mark.parametrize("n", [1, 40])
def test_paged_strides_of_axes_of_one(ns, n):
    """An axis of one may have any stride: the call is the same, bit for bit, as with dense ones."""
    g, rng = gen(95), random.Random(95)
    P, d = 64, 64
    dk, dv, table, _, _ = make_cache(g, rng, [60], 1, P, d, BF16, spare=0)
    i32 = {"dtype": torch.int32, "device": "cuda"}
    rest = (table.cuda(), torch.tensor([60], **i32), torch.tensor([0], **i32))
    q = normal(g, (1, n, 8, d), BF16).cuda()
    want, wl = ns.attend_paged(q, dk, dv, *rest)
    for s in (0, 3, 12, 8 * d * n + 1):
        qs = torch.as_strided(q, q.shape, (s, 8 * d, d, 1))
        ks, vs = (torch.as_strided(t, t.shape, (s, s, d, 1)) for t in (dk, dv))
        for args in ((qs, dk, dv), (q, ks, vs), (qs, ks, vs)):
            out, lse = ns.attend_paged(*args, *rest)
            assert torch.equal(out, want) and torch.equal(lse, wl)
    one, wl = ns.attend_paged(q[:, :, :1].contiguous(), dk, dv, *rest)
    head = torch.as_strided(q, (1, n, 1, d), (1, 8 * d, 1, 1))
    out, lse = ns.attend_paged(head, dk, dv, *rest)
    assert torch.equal(out, one) and torch.equal(lse, wl) and ns.ops_error() == 0


@pytest.mark.parametrize("seqs", [300, 448, 1500, 4096])
@pytest.mark.parametrize("d,dtype", [(64, F16), (128, BF16)])
def test_paged_many_sequences(ns, seqs, d, dtype):
    """Up to the most sequences of a call, by few and by many rows: every CTA finds its share among all of them."""
    g, rng = gen(seqs), random.Random(seqs)
    P, hkv, pages = 8, 1, 64
    lens = [rng.choice([0, 1, 7, 8, 9, 30, 64]) + (200 if i % 97 == 5 else 0) for i in range(seqs)]
    k, v = normal(g, (pages, hkv, P, d), dtype), normal(g, (pages, hkv, P, d), dtype)
    table = torch.tensor([[rng.randrange(pages) for _ in range(33)] for _ in range(seqs)], dtype=torch.int32)
    i32 = {"dtype": torch.int32, "device": "cuda"}
    rest = (k.cuda(), v.cuda(), table.cuda(), torch.tensor(lens, **i32), torch.arange(seqs, **i32))
    some = [0, 1, 5, 102, seqs // 2, seqs - 2, seqs - 1] + rng.sample(range(seqs), 20)
    for n, hq, off in ((1, 2, 0), (5, 4, 0), (5, 4, 2)):  # (queries off a 16-byte boundary: another kernel)
        q = normal(g, (seqs, n, hq, d), dtype)
        dq = torch.zeros((seqs, n, hq, d + off), dtype=dtype, device="cuda")[..., off:]
        dq.copy_(q)
        out, lse = ns.attend_paged(dq, *rest)
        out, lse = out.cpu(), lse.cpu()
        for b in some:
            N = lens[b]
            rows = [(int(table[b, p // P]), p % P) for p in range(N)]
            kk, vv = (torch.stack([t[x, 0, y] for x, y in rows]) if rows else t[0, 0, :0] for t in (k, v))
            sees = torch.tensor([[p <= N - n + i for p in range(N)] for i in range(n)], dtype=torch.bool).view(n, N)
            for h in range(hq):
                o, z, to, tz = attend_rows(q[b, :, h], kk, vv, sees, d ** -0.5)
                check(out[b, :, h], o, to, f"out of sequence {b} head {h}")
                check(lse[b, :, h], z, tz, f"lse of sequence {b} head {h}")
    assert ns.ops_error() == 0


@pytest.mark.parametrize("d,most", [(64, 16), (128, 12)])
def test_paged_around_the_longest_that_clusters_take(ns, d, most):
    """One sequence of few heads (large CTAs) and of many (small ones), at the most tiles that a CTA of theirs takes."""
    for heads, keys in ((2, 128), (16, 64)):
        for n in (most * 16 * keys - 1, most * 16 * keys, most * 16 * keys + 1):
            run_paged(ns, [n], 1, heads, heads, d, 64, BF16, n)
