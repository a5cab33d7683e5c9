"""Pages more than 2^32 bytes into a cache, of 16 and of 8 bits: every call gives the bits that it gives for the same
rows in a small cache."""

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


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


@pytest.mark.parametrize("scaled", [False, True])
def test_far_pages(ns, scaled):
    heads, page, d, own = 4, 16, 128, [40, 37, 9]  # pages of three sequences, the first 30 shared by two of them
    ids = list(range(own[0])) + list(range(own[0], own[0] + 7)) + list(range(own[0] + 7, own[0] + 16))
    first = [ids[:40], ids[:30] + ids[40:47], ids[47:56]]
    lens = [639, 590, 130]
    pages = 2 ** 32 // (heads * page * d * (1 if scaled else 2)) + 4096
    caches = []
    for n, shift in ((64, 0), (pages, pages - 64)):
        c = ns.KvPages.new(1, n, heads, page, d, 3, 64, scaled=scaled)
        for s in range(3):
            c.table[s, :len(first[s])] = i32(first[s]) + shift
        c.lengths.copy_(i32(lens))
        c.refs[shift:] = 1
        caches.append(c)
    assert caches[1].k[0, -64].data_ptr() - caches[1].k.data_ptr() > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = [torch.randn(sum(lens), heads, d, generator=g, device="cuda").to(BF16) for _ in range(2)]
    cu = [0, lens[0], lens[0] + lens[1], sum(lens)]
    seqs = i32([0, 1, 2])
    got = []
    for c in caches:
        # (the second's beginning is the first's, which holds it: the same rows twice are the same bytes)
        rows[0][cu[1]:cu[1] + 480], rows[1][cu[1]:cu[1] + 480] = rows[0][:480], rows[1][:480]
        c.write(0, seqs, i32(cu), *rows)
        out = list(c.read(0, seqs, i32(cu), sum(lens)))
        gq = torch.Generator(device="cuda").manual_seed(2)
        for n in (1, 2, 4, 20):  # (4 rows, 8, 16, 80)
            q = torch.randn(3, n, 16, d + 2, generator=gq, device="cuda").to(BF16)
            dense = q[..., :d].contiguous()
            out += c.attend(0, dense, seqs)
            out += c.attend(0, q[..., :d], seqs)  # (beyond 16 rows, queries that TMA cannot fetch)
            out += c.attend(0, dense, seqs, groups=i32([0, 2, 3]))
        c.compact(i32([2]), i32([0]), i32([[1, 5, 128]]), i32([3]))
        out += c.read(0, i32([2]), i32([0, 3]), 3)
        c.copy(i32([c.k.shape[1] - 64]), i32([c.k.shape[1] - 1]))
        out.append(c.k[0, -1].view(torch.uint8).clone())
        if scaled:
            out.append(c.v_exp[0, -1].clone())
        assert ns.ops_error() == 0
        got.append(out)
    assert len(got[0]) == len(got[1])
    for i, (a, b) in enumerate(zip(*got)):
        assert torch.equal(a, b), f"result {i}"
    assert torch.equal(got[0][0][:480], got[0][0][cu[1]:cu[1] + 480])
    if not scaled:
        assert torch.equal(got[0][0], rows[0]) and torch.equal(got[0][1], rows[1])
