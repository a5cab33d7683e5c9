"""KvPages against its rules, written out one step at a time: tables, lengths
and reference counts equal, every row of every page equal bit for bit."""

import random

import numpy as np
import pytest
import torch

from serving_ref import Pages

pytestmark = pytest.mark.gpu


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


class Both:
    """The cache on the GPU and its rules, step by step on the same data."""

    def __init__(self, ns, layers, pages, heads, page, dim, seqs, slots, dtype=torch.int16, layout="plain", seed=0):
        g = torch.Generator()
        g.manual_seed(seed)
        shape = (layers, pages, heads, page, dim)
        k, v = (torch.randint(-100, 100, shape, generator=g).to(dtype) for _ in range(2))
        if layout == "tokens":
            dk, dv = (t.transpose(2, 3).contiguous().cuda().transpose(2, 3) for t in (k, v))
        elif layout == "pages":  # pages outermost
            dk, dv = (t.transpose(0, 1).contiguous().cuda().transpose(0, 1) for t in (k, v))
        else:
            dk, dv = k.cuda(), v.cuda()
        self.c = ns.KvPages(dk, dv, torch.full((seqs, slots), -1, dtype=torch.int32, device="cuda"), i32([0] * seqs),
                            i32([0] * pages))
        self.r = Pages(k.numpy(), v.numpy(), [[-1] * slots for _ in range(seqs)], [0] * seqs, [0] * pages)
        self.ns, self.g = ns, g
        self.shape = shape

    def same(self, flags=0):
        assert self.ns.ops_error(clear=True) == flags
        assert self.c.table.tolist() == self.r.table
        assert self.c.lengths.tolist() == self.r.lengths
        assert self.c.refs.tolist() == self.r.refs
        assert np.array_equal(self.c.k.cpu().numpy(), self.r.k) and np.array_equal(self.c.v.cpu().numpy(), self.r.v)

    def extend(self, seqs, new):
        self.c.extend(i32(seqs), i32(new))
        return self.r.extend(seqs, new)

    def truncate(self, seqs, new):
        self.c.truncate(i32(seqs), i32(new))
        self.r.truncate(seqs, new)

    def fork(self, src, dst):
        self.c.fork(i32(src), i32(dst))
        self.r.fork(src, dst)

    def write(self, layer, seqs, counts):
        cu = [0]
        for n in counts:
            cu.append(cu[-1] + n)
        shape = (cu[-1], self.shape[2], self.shape[4])
        k, v = (torch.randint(-100, 100, shape, generator=self.g).to(self.c.k.dtype) for _ in range(2))
        self.c.write(layer, i32(seqs), i32(cu), k.cuda(), v.cuda())
        self.r.write(layer, seqs, cu, k.numpy(), v.numpy())

    def compact(self, seqs, base, keep):
        m = max([len(x) for x in keep] + [1])
        rows = [list(x) + [-7] * (m - len(x)) for x in keep]
        self.c.compact(i32(seqs), i32(base), i32(rows), i32([len(x) for x in keep]))
        self.r.compact(seqs, base, keep)


@pytest.mark.parametrize("layout", ["plain", "tokens", "pages"])
@pytest.mark.parametrize("page,dim,heads", [(8, 64, 2), (16, 128, 1), (5, 8, 3), (64, 24, 2), (1, 16, 1)])
def test_random_steps(ns, layout, page, dim, heads):
    rng = random.Random(page * 100 + dim)
    b = Both(ns, 3, 150, heads, page, dim, 9, 40, layout=layout, seed=page)
    cap = 40 * page
    for step in range(40):
        what = rng.choice(["extend", "extend", "truncate", "fork", "write", "compact"])
        seqs = rng.sample(range(9), rng.randrange(1, 9))
        if what == "extend":
            new = [min(rng.choice([0, 1, 2, page, 3 * page + 1]), cap - b.r.lengths[s]) for s in seqs]
            full = b.extend(seqs, new)
            b.same(0 if full else ns.FLAG_NO_PAGES)
            if full and rng.random() < 0.7:
                b.write(rng.randrange(3), seqs, new)
        elif what == "truncate":
            b.truncate(seqs, [rng.randrange(0, b.r.lengths[s] + 3) for s in seqs])
        elif what == "fork":
            empty = [s for s in range(9) if b.r.lengths[s] == 0]
            live = [s for s in range(9) if b.r.lengths[s] > 0]
            if empty and live:
                b.fork([rng.choice(live) for _ in empty], empty)
        elif what == "write":
            # rows of private pages only: the last page, where nobody else holds it
            own = [s for s in seqs if b.r.lengths[s] and b.r.refs[b.r.table[s][b.r.held(s) - 1]] == 1]
            if own:
                b.write(rng.randrange(3), own, [1 + (b.r.lengths[s] - 1) % page for s in own])
        else:
            own = [s for s in seqs if all(b.r.refs[p] == 1 for p in b.r.table[s] if p >= 0)]
            base = [rng.randrange(0, b.r.lengths[s] + 1) for s in own]
            keep = []
            for s, a in zip(own, base):
                left = b.r.lengths[s] - a
                keep.append(sorted(rng.sample(range(left), rng.randrange(0, left + 1))))
            if own:
                b.compact(own, base, keep)
        b.same()


@pytest.mark.parametrize("dtype", [torch.float32, torch.int8, torch.float16])
def test_row_types(ns, dtype):
    b = Both(ns, 2, 30, 2, 8, 32, 4, 8, dtype=dtype)
    b.extend([0, 1], [19, 33])
    b.write(1, [0, 1], [19, 33])
    b.fork([0, 1], [2, 3])
    b.extend([2, 0], [1, 1])
    b.compact([1 - 1], [17], [[1, 2]])
    b.same()


def test_wide_rows_and_long_lists(ns):
    """Rows wider than 512 bytes, and more sequences than one block scans at once."""
    b = Both(ns, 1, 60, 1, 4, 600, 3, 16)
    b.extend([0, 1], [50, 30])
    b.write(0, [0, 1], [50, 30])
    b.compact([0, 1], [1, 0], [[3, 4, 8, 30, 48], list(range(1, 30, 3))])
    b.same()
    n = 2500
    c = Both(ns, 1, n * 2 + 40, 1, 8, 8, n + 5, 3)
    rng = random.Random(3)
    ids = rng.sample(range(n), n)
    c.extend(ids, [rng.randrange(0, 17) for _ in range(n)])
    c.same()
    c.fork(ids[:5], list(range(n, n + 5)))
    c.extend(ids[:5] + list(range(n, n + 5)), [1] * 10)
    c.same()
    c.truncate(ids, [0] * n)
    c.same()


def test_compaction_of_long_chunks(ns):
    b = Both(ns, 2, 300, 2, 16, 64, 2, 150)
    b.extend([0, 1], [2100, 1200])
    b.write(0, [0, 1], [2100, 1200])
    b.write(1, [1, 0], [1200, 2100])
    b.compact([1, 0], [7, 100], [list(range(0, 1193, 2)), [x for x in range(2000) if x % 7]])
    b.same()
    b.compact([0], [0], [[]])
    b.same()


def test_free_with_no_lengths(ns):
    b = Both(ns, 1, 20, 1, 8, 8, 3, 6)
    b.extend([0, 1, 2], [20, 8, 1])
    b.c.truncate(i32([2, 0]))
    b.r.truncate([2, 0], [0, 0])
    b.same()


def test_copy_pages(ns):
    b = Both(ns, 3, 20, 2, 8, 24, 3, 6, layout="pages")
    b.c.copy(i32([3, 3, 7]), i32([9, 2, 19]))
    b.r.copy([3, 3, 7], [9, 2, 19])
    b.same()
    b.c.copy(i32([3, 20, -1]), i32([-1, 4, 5]))
    b.same(0x1)


def test_too_few_pages_changes_nothing(ns):
    b = Both(ns, 2, 6, 1, 8, 8, 4, 8)
    b.extend([0], [20])
    b.same()
    assert not b.extend([1, 0], [24, 10])
    b.same(ns.FLAG_NO_PAGES)
    b.extend([1, 0], [16, 4])
    b.same()
    b.fork([0], [2])
    assert b.extend([2], [0])
    b.same()


def test_both_holders_of_a_page_extend_at_once(ns):
    b = Both(ns, 2, 20, 1, 8, 8, 4, 8)
    b.extend([0], [13])
    b.fork([0, 0], [1, 2])
    b.extend([2, 0, 1], [1, 4, 0])
    b.same()


def test_invalid_sequences_are_skipped_and_flagged(ns):
    b = Both(ns, 1, 40, 1, 8, 8, 4, 5)
    b.extend([0, 1], [20, 9])
    b.same()
    # repeated, out of range, negative, past the table row: the valid entries still happen
    b.c.extend(i32([0, 0, 9, -1, 2, 3]), i32([1, 5, 1, 1, -1, 41]))
    b.r.extend([0], [1])
    b.same(ns.FLAG_BAD_SEQ)
    b.c.truncate(i32([1, 1, 4, 0]), i32([3, 2, 0, -1]))
    b.r.truncate([1], [3])
    b.same(ns.FLAG_BAD_SEQ)
    # busy, repeated and self destinations, a destination that is a source too
    b.c.fork(i32([0, 0, 0, 2, 0, 7]), i32([1, 3, 3, 2, 0, 2]))
    b.r.fork([0], [3])
    b.same(ns.FLAG_BAD_SEQ)
    b.c.fork(i32([0, 2]), i32([2, 1]))
    b.same(ns.FLAG_BAD_SEQ)


def test_compact_skips_bad_entries_and_shared_pages(ns):
    b = Both(ns, 1, 40, 1, 8, 8, 4, 5)
    b.extend([0, 1], [20, 20])
    b.write(0, [0, 1], [20, 20])
    k0, v0 = b.r.k.copy(), b.r.v.copy()
    b.fork([0], [2])
    # not increasing (entry 1), past the end (entry 3): their rows stay; then truncated to 4
    b.c.compact(i32([1]), i32([0]), i32([[5, 5, 6, 20]]), i32([4]))
    p = b.r.table[1][0]
    for t, frm in ((0, 5), (2, 6)):
        b.r.k[0, p, :, t], b.r.v[0, p, :, t] = k0[0, p, :, frm], v0[0, p, :, frm]
    b.r.truncate([1], [4])
    b.same(ns.FLAG_BAD_SEQ)
    # rows of pages that sequence 2 holds too stay as they are
    b.c.compact(i32([0]), i32([0]), i32([[3, 9]]), i32([2]))
    b.r.truncate([0], [2])
    b.same(ns.FLAG_SHARED_PAGE)
    # more kept than the list holds: skipped whole
    b.c.compact(i32([2]), i32([0]), i32([[3, 9]]), i32([3]))
    b.same(ns.FLAG_BAD_SEQ)


def test_write_skips_shared_pages_and_other_tokens(ns):
    b = Both(ns, 2, 20, 1, 8, 8, 4, 5)
    b.extend([0], [12])
    b.fork([0], [1])
    b.write(1, [1], [12])  # every page is shared: nothing is written
    b.same(ns.FLAG_SHARED_PAGE)
    k = torch.ones(9, 1, 8, dtype=torch.int16, device="cuda")
    b.c.write(0, i32([2]), i32([0, 9]), k, k)  # more tokens than the sequence holds
    b.same(ns.FLAG_BAD_SEQ)


def test_offsets_past_32_bits(ns):
    """Pages whose bytes lie past 2^32."""
    pages, heads, page, dim = (1 << 32) // (8 * 64 * 128 * 2) + 12, 8, 64, 128
    k = torch.empty((1, pages, heads, page, dim), dtype=torch.int16, device="cuda")
    refs = torch.ones(pages, dtype=torch.int32, device="cuda")
    refs[pages - 8:] = 0
    c = ns.KvPages(k, k.clone(), torch.full((2, 4), -1, dtype=torch.int32, device="cuda"), i32([0, 0]), refs)
    c.extend(i32([0]), i32([130]))
    assert c.table[0].tolist() == [pages - 8, pages - 7, pages - 6, -1]
    kn = torch.arange(130 * heads * dim, device="cuda").to(torch.int16).view(130, heads, dim)
    c.write(0, i32([0]), i32([0, 130]), kn, kn + 1)
    c.fork(i32([0]), i32([1]))
    c.extend(i32([1]), i32([1]))
    assert c.table[1].tolist() == [pages - 8, pages - 7, pages - 5, -1]
    assert torch.equal(c.k[0, pages - 5, :, :2], kn[128:].transpose(0, 1))
    c.truncate(i32([0]))
    c.compact(i32([1]), i32([0]), i32([[5, 129]]), i32([2]))
    assert torch.equal(c.k[0, pages - 8, :, :2], kn[[5, 129]].transpose(0, 1))
    assert torch.equal(c.v[0, pages - 8, :, :2], (kn + 1)[[5, 129]].transpose(0, 1))
    assert ns.ops_error() == 0


def test_refusals(ns):
    k = torch.zeros(2, 4, 1, 8, 8, dtype=torch.int16, device="cuda")
    t, le, re = torch.zeros(3, 2, dtype=torch.int32, device="cuda"), i32([0] * 3), i32([0] * 4)
    for args in ((k, k[:1], t, le, re), (k, k.half(), t, le, re), (k, k, t.long(), le, re), (k, k, t, le[:2], re),
                 (k, k, t, le, re[:3]), (k.cpu(), k.cpu(), t, le, re), (k.transpose(3, 4), k.transpose(3, 4), t, le, re)):
        with pytest.raises(ValueError):
            ns.KvPages(*args)
    c = ns.KvPages(k, k.clone(), t, le, re)
    for f in (lambda: c.extend(i32([0, 1]), i32([1])), lambda: c.fork(i32([0]), i32([1, 2])),
              lambda: c.truncate(i32([0]).long()), lambda: c.compact(i32([0]), i32([0]), i32([1]), i32([1])),
              lambda: c.write(0, i32([0]), i32([0]), k[0, 0], k[0, 0]),
              lambda: c.write(0, i32([0]), i32([0, 1]), k[0, 0, 0, :1, None], k[0, 0])):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: c.write(2, i32([0]), i32([0, 8]), k[0, 0].transpose(0, 1), k[0, 0].transpose(0, 1)),
              lambda: c.extend(i32([0]), i32([1]), workspace=torch.zeros(16, dtype=torch.uint8, device="cuda")),
              # rows of 12 bytes
              lambda: ns.KvPages(k[..., :6], k[..., :6], t, le, re).truncate(i32([0])),
              # rows that begin off a 16-byte boundary
              lambda: ns.KvPages(torch.zeros(2, 4, 1, 8, 9, dtype=torch.int16, device="cuda")[..., 1:], k, t, le,
                                 re).truncate(i32([0]))):
        with pytest.raises(ns.NanoSpecError):
            f()
    c.truncate(i32([]))
    c.extend(i32([]), i32([]))
    assert ns.ops_error() == 0


@pytest.mark.parametrize("n", [1023, 1024, 1025, 2100])
def test_many_sequences_and_pages_in_one_extend(ns, n):
    """Around the number of sequences, and of given pages, whose bookkeeping one CTA keeps in shared memory."""
    b = Both(ns, 1, 4 * n + 40, 1, 2, 8, 2 * n, 4)
    rng = random.Random(n)
    first = list(range(n))
    rng.shuffle(first)
    b.extend(first, [rng.choice([0, 1, 2, 3, 3]) for _ in first])
    b.same()
    b.fork(list(range(n)), list(range(n, 2 * n)))
    some = rng.sample(range(2 * n), n)
    b.extend(some, [rng.choice([0, 1, 1, 2, 4]) for _ in some])  # copies of shared last pages among them
    b.same()
    again = some[: n // 2]
    b.c.extend(i32(again + again[:3]), i32([1] * (len(again) + 3)))  # the last three are repeated, and skipped
    b.r.extend(again, [1] * len(again))
    b.same(ns.FLAG_BAD_SEQ)


def test_many_pages_for_one_sequence(ns):
    for want in (2047, 2048, 2049, 9000):
        b = Both(ns, 1, 9100, 1, 1, 8, 2, 9050)
        b.extend([1, 0], [37, want - 37])
        b.same()


def test_a_cache_of_another_device_is_refused(ns):
    """Each call looks at the current device, not only the one that made the cache.  A second device is stood in for by
    a cache whose record says so; every argument is refused before it is used."""
    import ctypes

    from test_serving_abi import Pages as Record

    class Cache(ctypes.Structure):
        _fields_ = [("c", Record), ("type", ctypes.c_int8), ("device_type", ctypes.c_int8), ("device", ctypes.c_int8)]

    make = ctypes.pythonapi.PyCapsule_New
    make.restype, make.argtypes = ctypes.py_object, [ctypes.c_void_p] * 3
    name = ctypes.create_string_buffer(b"ns_kv_pages")
    record = Cache(Record(layers=1, pages=4, heads=1, page_size=8, row_bytes=16, max_seqs=2, table_ld=2), 2, 1, 1)
    c = ns.KvPages.new(1, 4, 1, 8, 8, 2, 2)
    c._c = make(ctypes.addressof(record), ctypes.addressof(name), None)
    one, row = i32([0]), torch.zeros(1, 1, 8, dtype=torch.int16, device="cuda")
    for f in (lambda: c.truncate(one), lambda: c.fork(one, one), lambda: c.extend(one, one),
              lambda: c.write(0, one, i32([0, 1]), row, row), lambda: c.compact(one, one, i32([[0]]), one),
              lambda: c.copy(one, one)):
        with pytest.raises(ValueError, match="current CUDA device"):
            f()
    assert ns.ops_error() == 0


def test_write_skips_repeated_sequences(ns):
    """The rows of the first entry of a sequence are written, those of later ones are not."""
    b = Both(ns, 1, 40, 2, 8, 8, 6, 5)
    b.extend([0, 1, 2], [20, 9, 3])
    k, v = (torch.randint(-100, 100, (37, 2, 8), generator=b.g).to(torch.int16) for _ in range(2))
    # 20 tokens of sequence 0, 9 of 1, then 3 of 0 again, 2 of 1 again, 3 of 2
    b.c.write(0, i32([0, 1, 0, 1, 2]), i32([0, 20, 29, 32, 34, 37]), k.cuda(), v.cuda())
    b.r.write(0, [0, 1], [0, 20, 29], k.numpy(), v.numpy())
    b.r.write(0, [2], [0, 3], k.numpy()[34:], v.numpy()[34:])
    b.same(ns.FLAG_BAD_SEQ)


def test_write_of_many_sequences_with_repeated_ones(ns):
    n = 2100
    b = Both(ns, 1, n + 10, 1, 4, 8, n, 2)
    ids = list(range(n))
    random.Random(4).shuffle(ids)
    b.extend(ids, [1 + i % 3 for i in range(n)])
    b.same()
    b.write(0, ids, [1 + i % 3 for i in range(n)])
    b.same()
    seqs = ids[:1500] + ids[7:9] + ids[1500:] + ids[-1:]
    k, v = (torch.randint(-100, 100, (len(seqs), 1, 8), generator=b.g).to(torch.int16) for _ in range(2))
    b.c.write(0, i32(seqs), i32(list(range(len(seqs) + 1))), k.cuda(), v.cuda())
    first = [i for i, s in enumerate(seqs) if s not in seqs[:i]]
    b.r.write(0, [seqs[i] for i in first], list(range(len(first) + 1)), k.numpy()[first], v.numpy()[first])
    b.same(ns.FLAG_BAD_SEQ)


def test_a_caches_tensors_stay(ns):
    """Another tensor in place of one of them would leave the cache working on memory that is given away."""
    c = ns.KvPages.new(1, 4, 1, 8, 8, 2, 2)
    for name in ("k", "v", "table", "lengths", "refs"):
        before = getattr(c, name)
        with pytest.raises(AttributeError):
            setattr(c, name, torch.zeros_like(before))
        assert getattr(c, name) is before
    c.extend(i32([1]), i32([9]))
    assert c.lengths.tolist() == [0, 9] and c.refs.tolist() == [1, 1, 0, 0] and ns.ops_error() == 0
