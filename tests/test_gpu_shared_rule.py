"""attend_shared where its groups have nothing to share: it is attend_paged, to the bit."""

import pytest
import torch

from test_gpu_shared import BF16, F16, i32, ns  # noqa: F401

pytestmark = pytest.mark.gpu


def cache_of(ns, lens, d, scaled, wide, dtype, seed):  # noqa: F811
    """A cache of a sequence for each length; wide: a table for 2^20 positions, by which a call of few rows shares."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    per = -(-max(lens) // 16)
    c = ns.KvPages.new(1, per * len(lens) + 3, 2, 16, d, len(lens), (1 << 16) if wide else per, dtype=dtype,
                       scaled=scaled)
    seqs = i32(list(range(len(lens))))
    c.extend(seqs, i32(lens))
    T = sum(lens)
    cu = i32([sum(lens[:i]) for i in range(len(lens) + 1)])
    k, v = (torch.randn(T, 2, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    c.write(0, seqs, cu, k, v)
    return c, seqs, g


def both(ns, c, seqs, g, n, hq, d, dtype, groups, **kw):  # noqa: F811
    q = torch.randn(len(seqs), n, hq, d, generator=g, device="cuda").to(dtype)
    want = c.attend(0, q, seqs, **kw)
    got = c.attend(0, q, seqs, groups=i32(groups), **kw)
    assert ns.ops_error() == 0
    return all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("n,hq", [(1, 8), (1, 14), (8, 8), (32, 8)])
def test_groups_of_one(ns, dtype, scaled, n, hq):  # noqa: F811
    for d, lens in ((128, [900, 2000, 333, 40, 1500]), (64, [3000])):
        c, seqs, g = cache_of(ns, lens, d, scaled, True, dtype, n + hq)
        assert both(ns, c, seqs, g, n, hq, d, dtype, list(range(len(lens) + 1)))


@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("n", [8, 32])
def test_contexts_of_less_than_a_tile(ns, scaled, n):  # noqa: F811
    """By max_len no member has 128 positions of context."""
    c, seqs, g = cache_of(ns, [n + 127] * 90 + [n + 3] * 10, 128, scaled, False, BF16, n)
    c.table.copy_(c.table[:1].expand_as(c.table))  # (all of them begin with the same pages)
    assert both(ns, c, seqs, g, n, 8, 128, BF16, [0, 100], max_len=n + 127)


@pytest.mark.parametrize("flaw", [[1, 2, 3], [0, 2, 2], [0, 3, 3, 2], [0, -1, 1, 3]])
def test_groups_that_are_not_as_they_should_be_are_flagged(ns, flaw):  # noqa: F811
    c, seqs, g = cache_of(ns, [400, 300, 200], 64, False, True, BF16, 1)
    for n in (1, 8):
        q = torch.randn(3, n, 8, 64, generator=g, device="cuda").to(BF16)
        want, _ = c.attend(0, q, seqs)
        out, _ = c.attend(0, q, seqs, groups=i32(flaw))
        assert ns.ops_error(clear=True) == ns.FLAG_BAD_SEQ
        assert (out.float() - want.float()).norm() <= 0.01 * want.float().norm()


@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("n,hq,B,length,max_len", [(1, 8, 8, 900, 19200), (8, 8, 24, 900, 908), (32, 8, 40, 700, 700),
                                                   (5, 16, 24, 901, 1000)])
def test_few_keys(ns, scaled, n, hq, B, length, max_len):  # noqa: F811
    """Sequences that share nearly all, up to 192 MB of keys and values by max_len."""
    if scaled and n == 1:
        max_len *= 2
    c, seqs, g = cache_of(ns, [length] * B, 128, scaled, True, BF16, n)
    c.table.copy_(c.table[:1].expand_as(c.table))
    assert B * max_len * 2 * 128 * (2 if scaled and n == 1 else 4) <= 192 << 20
    assert both(ns, c, seqs, g, n, hq, 128, BF16, [0, B], max_len=max_len)
