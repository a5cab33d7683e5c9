"""Attention over values that are not finite: which rows see them, and whether as +inf, -inf or NaN, exactly."""

import math
import random

import pytest
import torch

from serving_ref import attend_rows, check, with_wild_values
from test_gpu_attention import gen, make_cache, normal, signed, tree_masks

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module")
def ns():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import speculative_decoding_draft_stream_gb300 as p
    from speculative_decoding_draft_stream_gb300 import build

    build.build()
    p.ops_error(clear=True)
    return p


def expect(out, lse, q, k, v, sees, scale, what):
    """One head's rows against the reference with its values made finite, and then with those that are not."""
    o, z, to, tz = attend_rows(q, k, torch.nan_to_num(v.float(), 0.0, 0.0, 0.0).to(v.dtype), sees, scale)
    check(out, with_wild_values(o, v.float(), sees), to, "out of " + what)
    check(lse, z, tz, "lse of " + what)


# (place as a share of the sequence, column, value): one sign, both signs in either order, NaN before and after
WILD = [(0.10, 0, INF), (0.55, 0, INF), (0.30, 1, -INF), (0.60, 1, -INF), (0.20, 2, INF), (0.70, 2, -INF), (0.25, 3, -INF),
        (0.65, 3, INF), (0.40, 4, NAN), (0.50, 5, INF), (0.80, 5, NAN), (0.05, 6, -INF), (0.999, 7, INF), (0.998, 8, -INF),
        (0.999, 9, NAN), (0.97, 10, INF), (0.999, 10, -INF)]


def spoil(v, wild=WILD):
    """v [n, heads, d]: head h has the columns moved by 11 h, so that heads differ."""
    n, heads, d = v.shape
    for share, col, what in wild:
        for h in range(heads):
            v[min(n - 1, int(share * n)), h, (col + 11 * h) % d] = what


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("lens,hq,hkv,d", [
    ([40, 150, 64, 200], 2, 1, 128), ([40, 150, 64, 200], 2, 2, 64),     # an item's keys split over two halves
    ([900, 333], 4, 1, 128), ([700, 129], 2, 1, 64),
    ([300, 1000, 77, 555], 32, 4, 64), ([300, 800, 77, 555], 28, 4, 128),  # heads of a group in a tile
    ([700, 600], 40, 40, 64),                                           # two tiles of one head
])
def test_prompt(ns, lens, hq, hkv, d, dtype):
    g = gen(len(lens) + hq + d)
    T = sum(lens)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    q, k, v = normal(g, (T, hq, d), dtype), normal(g, (T, hkv, d), dtype), normal(g, (T, hkv, d), dtype)
    for a, b in zip(cu[:-1], cu[1:]):
        spoil(v[a:b])
    out, lse = ns.attend_prompt(q.cuda(), k.cuda(), v.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(), max(lens))
    out, lse = out.cpu(), lse.cpu()
    for a, b in zip(cu[:-1], cu[1:]):
        sees = torch.ones(b - a, b - a, dtype=torch.bool).tril()
        for h in range(hq):
            kh = h // (hq // hkv)
            expect(out[a:b, h], lse[a:b, h], q[a:b, h], k[a:b, kh], v[a:b, kh], sees, d ** -0.5, f"{a}:{b} head {h}")
    assert ns.ops_error() == 0


def run_paged(ns, lens, n, hq, hkv, d, P, dtype, seed, tree=True, unaligned=False):
    g, rng = gen(seed), random.Random(seed)
    dk, dv, table, keys, vals = make_cache(g, rng, lens, hkv, P, d, dtype)
    for b, N in enumerate(lens):
        # the context of every row, on columns that the nodes do not touch, and then the nodes
        if N > n:
            spoil(vals[b][:N - n], [(0.3, 40, INF), (0.9, 41, -INF), (0.1, 42, INF), (0.8, 42, -INF), (0.5, 43, NAN),
                                    (0.95, 5, INF), (0.5, 1, -INF)])
        spoil(vals[b][max(0, N - n):])
        for slot in range(-(-N // P)):
            part = vals[b][slot * P:(slot + 1) * P]
            dv[table[b, slot], :, :len(part)] = part.transpose(0, 1).cuda()
    B = len(lens)
    masks = tree_masks(rng, B, n) if tree else None
    q = normal(g, (B, n, hq, d), dtype)
    dq = q.cuda()
    if unaligned:
        dq = torch.zeros((B, n, hq, d + 2), dtype=dtype, device="cuda")[..., 2:]
        dq.copy_(q)
    i32 = {"dtype": torch.int32, "device": "cuda"}
    out, lse = ns.attend_paged(dq, dk, dv, table.cuda(), torch.tensor(lens, **i32), torch.arange(B, **i32),
                               mask=signed(masks).cuda() if tree else None)
    out, lse = out.cpu(), lse.cpu()
    for b, N in enumerate(lens):
        sees = torch.zeros(n, N, dtype=torch.bool)
        for i in range(n):
            word = masks[b][i] if tree else (1 << (i + 1)) - 1
            for p in range(N):
                sees[i, p] = p < N - n or bool(word >> (p - N + n) & 1)
        for h in range(hq):
            kh = h // (hq // hkv)
            expect(out[b, :, h], lse[b, :, h], q[b, :, h], keys[b][:, kh], vals[b][:, kh], sees, d ** -0.5,
                   f"sequence {b} head {h}")
    assert ns.ops_error() == 0


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("d,dtype", [(64, F16), (128, BF16), (64, BF16), (128, F16)])
def test_paged(ns, d, dtype, tree):
    few = [300, 17, 140]
    run_paged(ns, [x + 4 for x in few], 4, 3, 1, d, 16, dtype, 1, tree)         # clusters
    run_paged(ns, [20 + 13 * i for i in range(40)], 4, 8, 4, d, 16, dtype, 2, tree)  # one line of tiles
    run_paged(ns, [3000], 4, 4, 1, d, 64, dtype, 3, tree)
    run_paged(ns, [x + 30 for x in few], 30, 4, 2, d, 16, dtype, 4, tree)       # tcgen05, parts joined
    run_paged(ns, [150 + 47 * i for i in range(16)], 24, 16, 16, d, 16, dtype, 5, tree)  # whole items
    run_paged(ns, [x + 60 for x in few], 60, 4, 2, d, 16, dtype, 6, tree, unaligned=True)  # 64 rows a CTA
    run_paged(ns, few, 1, 4, 2, d, 16, dtype, 7, False)
