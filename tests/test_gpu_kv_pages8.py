"""KvPages of 8 bits: codes and exponents are the rule's, bit for bit, wherever rows go."""

import random

import numpy as np
import pytest
import torch

from serving8_ref import E4M3, quantise, values
from serving_ref import Pages

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


def bits(x):
    """The codes of exact values."""
    return x.float().to(E4M3).view(torch.uint8)


def one_page_each(ns, tokens, heads, D, page=16, layers=1):
    c = ns.KvPages.new(layers, -(-tokens // page) + 1, heads, page, D, 1, -(-tokens // page), scaled=True)
    for t in (c.k, c.v):
        t.view(torch.uint8).fill_(0x7f)  # what was there before
    c.extend(i32([0]), i32([tokens]))
    return c


def laid_out(c, name, tokens):
    """(codes, exponents) of sequence 0's positions in layer 0: [tokens, heads, D], [tokens, heads]."""
    pages = c.table[0, :-(-tokens // c.k.shape[3])].long()
    codes = getattr(c, name).view(torch.uint8)[0][pages].transpose(1, 2).flatten(0, 1)[:tokens]
    exps = getattr(c, name + "_exp")[0][pages].transpose(1, 2).flatten(0, 1)[:tokens]
    return codes.cpu(), exps.cpu()


def rows_of_every_size(dt, D, heads, seed):
    """Rows from 2^-50 to the type's largest (as far as it goes), ties and subnormal codes among them."""
    g = torch.Generator().manual_seed(seed)
    rows = []
    for e in range(-50, 60):
        x = torch.randn(heads, D, generator=g).double() * 2.0 ** e
        x[:, ::3] *= 2.0 ** torch.randint(-14, 1, (heads, len(range(0, D, 3))), generator=g).double()
        rows.append(x)
    x = torch.zeros(heads, D).double()
    rows.append(x)
    x = x.clone()
    x[:, 0] = 448.0
    x[:, 1:9] = torch.tensor([0.5 * 2.0 ** -9, 1.5 * 2.0 ** -9, 2.5 * 2.0 ** -9, 17.0, 18.0, 19.0, 21.0, -23.0])
    rows += [x, x * 1.0078125, x * 2.0 ** -3, -x]
    x = torch.stack(rows)
    x = x.clamp(-torch.finfo(dt).max, torch.finfo(dt).max).to(dt)
    x[-2, 0, 5] = torch.finfo(dt).max
    x[-1, heads - 1, 7] = torch.finfo(dt).smallest_normal / 2
    return x


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("D,heads", [(128, 1), (128, 8), (64, 3), (64, 9), (128, 17)])
def test_write_rounds_as_the_rule_says_and_read_gives_it_back(ns, dt, D, heads):
    k, v = rows_of_every_size(dt, D, heads, 1), rows_of_every_size(dt, D, heads, 2)
    n = len(k)
    k[3, 0, 2], k[4, heads - 1, D - 1], v[5, 0, 0] = float("inf"), float("nan"), -float("inf")
    c = one_page_each(ns, n, heads, D)
    cu = i32([0, n])
    c.write(0, i32([0]), cu, k.cuda(), v.cuda())
    for name, x in (("k", k), ("v", v)):
        codes, exps = quantise(x)
        got, got_exps = laid_out(c, name, n)
        assert torch.equal(got_exps, exps)
        assert torch.equal(got.view(E4M3).double(), codes), name
    for dtype in (BF16, F16, None):
        back = c.read(0, i32([0]), cu, n, dtype=dtype)
        for x, got in zip((k, v), back):
            want = values(*quantise(x)).to(dtype or BF16)
            assert got.dtype == want.dtype and torch.equal(got.cpu().nan_to_num(nan=7e4 if got.dtype == BF16 else 9),
                                                           want.nan_to_num(nan=7e4 if got.dtype == BF16 else 9))
            assert torch.equal(got.cpu().isnan(), want.isnan())
    assert ns.ops_error() == 0


def test_no_value_of_16_bits_is_rounded_otherwise(ns):
    """Every bf16 and fp16 value, in rows that they share with a larger one."""
    for dt in (BF16, F16):
        x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dt)
        x = x[torch.isfinite(x)]
        x = x[x.double().abs().argsort(stable=True)]
        x = x[: len(x) // 64 * 64].view(-1, 1, 64)
        c = one_page_each(ns, len(x), 1, 64)
        c.write(0, i32([0]), i32([0, len(x)]), x.cuda(), x.flip(0).cuda())
        codes, exps = quantise(x)
        got, got_exps = laid_out(c, "k", len(x))
        assert torch.equal(got_exps, exps) and torch.equal(got.view(E4M3).double(), codes)
        got, got_exps = laid_out(c, "v", len(x))
        assert torch.equal(got_exps, exps.flip(0)) and torch.equal(got.view(E4M3).double(), codes.flip(0))


class Both:
    """The cache on the GPU and its rules; a rule's row is the codes and, behind them, the exponent."""

    def __init__(self, ns, layers, pages, heads, page, dim, seqs, slots, layout, seed):
        self.g = torch.Generator().manual_seed(seed)
        shape = (layers, pages, heads, page, dim)
        rows = [torch.randint(0, 126, shape, generator=self.g, dtype=torch.uint8) for _ in range(2)]
        exps = [torch.randint(100, 150, shape[:4], generator=self.g, dtype=torch.uint8) for _ in range(2)]
        if layout == "tokens":
            d = [t.transpose(2, 3).contiguous().cuda().transpose(2, 3).view(E4M3) for t in rows]
            x = [t.cuda() for t in exps]
        else:  # pages outermost
            d = [t.transpose(0, 1).contiguous().cuda().transpose(0, 1).view(E4M3) for t in rows]
            x = [t.transpose(0, 1).contiguous().cuda().transpose(0, 1) for t in exps]
        self.c = ns.KvPages(d[0], d[1], torch.full((seqs, slots), -1, dtype=torch.int32, device="cuda"),
                            i32([0] * seqs), i32([0] * pages), x[0], x[1])
        both = [torch.cat((a, b[..., None]), -1).numpy() for a, b in zip(rows, exps)]
        self.r = Pages(both[0], both[1], [[-1] * slots for _ in range(seqs)], [0] * seqs, [0] * pages)
        self.ns, self.heads, self.dim = ns, heads, dim

    def same(self, flags=0):
        assert self.ns.ops_error(clear=True) == flags
        c, r = self.c, self.r
        assert c.table.tolist() == r.table and c.lengths.tolist() == r.lengths and c.refs.tolist() == r.refs
        for t, x, want in ((c.k, c.k_exp, r.k), (c.v, c.v_exp, r.v)):
            assert np.array_equal(t.view(torch.uint8).cpu().numpy(), want[..., :-1])
            assert np.array_equal(x.cpu().numpy(), want[..., -1])

    def write(self, layer, seqs, counts):
        cu = [0]
        for n in counts:
            cu.append(cu[-1] + n)
        new = [torch.randn(cu[-1], self.heads, self.dim, generator=self.g).to(BF16) for _ in range(2)]
        self.c.write(layer, i32(seqs), i32(cu), new[0].cuda(), new[1].cuda())
        q = [quantise(x) for x in new]
        self.r.write(layer, seqs, cu, *[torch.cat((bits(a), b[..., None]), -1).numpy() for a, b in q])


@pytest.mark.parametrize("layout", ["tokens", "pages"])
@pytest.mark.parametrize("page,dim,heads", [(8, 64, 2), (16, 128, 1), (24, 64, 3), (64, 128, 2)])
def test_rows_take_their_exponents_along(ns, layout, page, dim, heads):
    rng = random.Random(page + dim)
    b = Both(ns, 3, 120, heads, page, dim, 8, 30, layout, page)
    cap = 30 * page
    for step in range(30):
        what = rng.choice(["extend", "extend", "truncate", "fork", "compact", "compact", "copy"])
        seqs = rng.sample(range(8), rng.randrange(1, 8))
        if what == "extend":
            new = [min(rng.choice([0, 1, 2, page, 3 * page + 1]), cap - b.r.lengths[s]) for s in seqs]
            b.c.extend(i32(seqs), i32(new))
            full = b.r.extend(seqs, new)
            b.same(0 if full else ns.FLAG_NO_PAGES)
            if full:
                b.write(rng.randrange(3), seqs, new)
        elif what == "truncate":
            new = [rng.randrange(0, b.r.lengths[s] + 3) for s in seqs]
            b.c.truncate(i32(seqs), i32(new))
            b.r.truncate(seqs, new)
        elif what == "fork":
            empty = [s for s in range(8) if b.r.lengths[s] == 0]
            live = [s for s in range(8) if b.r.lengths[s] > 0]
            if empty and live:
                src = [rng.choice(live) for _ in empty]
                b.c.fork(i32(src), i32(empty))
                b.r.fork(src, empty)
        elif what == "compact":
            own = [s for s in seqs if all(b.r.refs[p] == 1 for p in b.r.table[s][:b.r.held(s)])]
            if own:
                base = [rng.randrange(0, b.r.lengths[s] + 1) for s in own]
                keep = [sorted(rng.sample(range(b.r.lengths[s] - a), rng.randrange(0, b.r.lengths[s] - a + 1)))
                        for s, a in zip(own, base)]
                m = max([len(x) for x in keep] + [1])
                b.c.compact(i32(own), i32(base), i32([x + [0] * (m - len(x)) for x in keep]),
                            i32([len(x) for x in keep]))
                b.r.compact(own, base, keep)
        else:
            pages = rng.sample(range(120), 6)
            b.c.copy(i32(pages[:3]), i32(pages[3:]))
            b.r.copy(pages[:3], pages[3:])
        b.same()


def test_long_compaction_in_place(ns):
    """Hundreds of kept rows of one sequence, from right behind where they go to far."""
    b = Both(ns, 2, 90, 2, 16, 64, 1, 80, "tokens", 3)
    b.c.extend(i32([0]), i32([1200]))
    b.r.extend([0], [1200])
    b.write(1, [0], [1200])
    keep = sorted(random.Random(1).sample(range(1100), 700))
    b.c.compact(i32([0]), i32([37]), i32([keep]), i32([700]))
    b.r.compact([0], [37], [keep])
    b.same()


@pytest.mark.parametrize("scaled", [False, True])
def test_read_of_ragged_sequences(ns, scaled):
    g = torch.Generator().manual_seed(5)
    lens, took = [37, 1, 160, 64], [5, 1, 160, 0]
    c = ns.KvPages.new(2, 40, 3, 16, 64, 5, 12, scaled=scaled)
    c.extend(i32([0, 1, 2, 3]), i32(lens))
    k, v = (torch.randn(sum(lens), 3, 64, generator=g).to(BF16) for _ in range(2))
    full = [0]
    for n in lens:
        full.append(full[-1] + n)
    c.write(1, i32([0, 1, 2, 3]), i32(full), k.cuda(), v.cuda())
    order = [2, 0, 3, 1, 2]  # one twice
    cu = [0]
    for s in order:
        cu.append(cu[-1] + took[s])
    T = cu[-1]
    wide = torch.zeros(T + 2, 7, 64, dtype=BF16, device="cuda")
    out = wide[:, 1:4]
    got = c.read(1, i32(order), i32(cu), T + 2, k_out=out)
    assert got[0] is out and (wide[T:] == 0).all() and (wide[:, 4:] == 0).all()
    for got, x in zip(got, (k, v)):
        x = values(*quantise(x)).to(BF16) if scaled else x
        want = torch.cat([x[full[s + 1] - took[s]:full[s + 1]] for s in order])
        assert torch.equal(got[:T].cpu(), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = c.read(1, i32(order), i32(cu), T, stream=s)
    s.synchronize()
    assert torch.equal(again[0], out[:T])
    assert ns.ops_error() == 0
    mark = torch.full((3, 3, 64), 5.0, dtype=BF16, device="cuda")
    c.read(0, i32([7, 1]), i32([0, 1, 3]), 3, k_out=mark, v_out=mark.clone())  # no such sequence; one with the second alone
    assert (mark[:2] == 5).all() and ns.ops_error(clear=True) == ns.FLAG_BAD_SEQ


@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("short", [3, 200])
def test_many_tokens(ns, scaled, short):
    """Calls of which a warp takes several tokens: long sequences and many of a few, one a second time, one that does not
    exist, one whose page another holds, and tokens behind the last."""
    g = torch.Generator().manual_seed(short)
    lens = [5001] + [1 + i % 7 for i in range(short)] + [3100, 1, 17]
    B = len(lens)
    c = ns.KvPages.new(1, 700 + B, 2, 16, 64, B + 3, 400, scaled=scaled)
    c.extend(i32(list(range(B))), i32(lens))
    c.fork(i32([B - 1]), i32([B]))
    for t in (c.k, c.v):
        t.view(torch.uint8 if scaled else BF16).zero_()
    order = list(range(B)) + [0, B + 7]  # a sequence again, one that is not there
    took = lens + [40, 9]
    cu = [0]
    for n in took:
        cu.append(cu[-1] + n)
    T = cu[-1] + 30
    assert T >= 8192
    k, v = (torch.randn(T, 2, 64, generator=g).to(BF16) for _ in range(2))
    c.write(0, i32(order), i32(cu), k.cuda(), v.cuda())
    assert ns.ops_error(clear=True) == ns.FLAG_BAD_SEQ | ns.FLAG_SHARED_PAGE
    mark = torch.full((2, T, 2, 64), 7.0, dtype=BF16, device="cuda")
    got = c.read(0, i32(order), i32(cu), T, k_out=mark[0], v_out=mark[1])
    assert ns.ops_error(clear=True) == ns.FLAG_BAD_SEQ
    for x, out in zip((k, v), got):
        want = values(*quantise(x)).to(BF16) if scaled else x
        want = want.clone()
        want[cu[B - 1]:cu[B]] = 0  # (another holds its page: as it was)
        want[cu[B]:cu[B + 1]] = want[4961:5001]  # the first one's rows, not the second's
        want[cu[B + 1]:] = 7  # nothing there
        if scaled:
            fresh = cu[B - 1], cu[B]
            want[fresh[0]:fresh[1]] = out[fresh[0]:fresh[1]].cpu()  # (no exponents yet)
        assert torch.equal(out.cpu(), want)


def test_invalid_writes_are_skipped(ns):
    c = ns.KvPages.new(1, 8, 2, 8, 64, 4, 4, scaled=True)
    c.k.view(torch.uint8).zero_(), c.v.view(torch.uint8).zero_()
    c.extend(i32([0, 1]), i32([10, 3]))
    c.fork(i32([0]), i32([2]))
    was = [t.view(torch.uint8).clone() for t in (c.k, c.v, c.k_exp, c.v_exp)]
    x = torch.ones(4, 2, 64, dtype=BF16, device="cuda")
    # a page that two hold, no such sequence, more rows than the sequence has
    for seqs, cu, flag in (([0], [0, 1], ns.FLAG_SHARED_PAGE), ([9], [0, 1], ns.FLAG_BAD_SEQ),
                           ([1], [0, 4], ns.FLAG_BAD_SEQ)):
        c.write(0, i32(seqs), i32(cu), x[:1], x[:1])
        assert ns.ops_error(clear=True) == flag
        assert all(torch.equal(a, b.view(torch.uint8)) for a, b in zip(was, (c.k, c.v, c.k_exp, c.v_exp)))
    c.write(0, i32([1, 1]), i32([0, 1, 2]), x[:2], 2 * x[:2])  # a sequence twice: the first counts
    assert ns.ops_error(clear=True) == ns.FLAG_BAD_SEQ
    page = int(c.table[1, 0])
    assert int(c.k_exp[0, page, 0, 2]) == 127 - 8 and int(c.v_exp[0, page, 0, 2]) == 127 - 7


def test_replayed_from_a_graph(ns):
    g = torch.Generator(device="cuda").manual_seed(6)
    c = ns.KvPages.new(1, 20, 4, 16, 128, 2, 8, scaled=True)
    seqs, cu, n = i32([0, 1]), i32([0, 20, 60]), 60
    c.extend(seqs, i32([20, 40]))
    k, v = (torch.randn(n, 4, 128, generator=g, device="cuda").to(BF16) for _ in range(2))
    out = [torch.empty_like(k) for _ in range(2)]
    c.write(0, seqs, cu, k, v), c.read(0, seqs, cu, n, k_out=out[0], v_out=out[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.write(0, seqs, cu, k, v)
        c.read(0, seqs, cu, n, k_out=out[0], v_out=out[1])
    k.mul_(3), v.mul_(-2)
    graph.replay()
    torch.cuda.synchronize()
    for got, x in zip(out, (k, v)):
        assert torch.equal(got.cpu(), values(*quantise(x.cpu())).to(BF16))


def test_refusals(ns):
    new = lambda **kw: ns.KvPages.new(**dict(dict(layers=1, pages=4, kv_heads=2, page_size=16, dim=64, max_seqs=2,
                                                  max_pages=2, scaled=True), **kw))
    c = new()
    x = torch.zeros(1, 2, 64, dtype=BF16, device="cuda")
    t = [c.table, c.lengths, c.refs]
    bad = [
        lambda: new(dim=32),
        lambda: new(page_size=12),
        lambda: ns.KvPages(c.k, c.v, *t, c.k_exp),
        lambda: ns.KvPages(c.k, c.v, *t, c.k_exp[:, :3], c.v_exp),
        lambda: ns.KvPages(c.k, c.v, *t, c.k_exp.int(), c.v_exp),
        lambda: ns.KvPages(c.k, c.v, *t, c.k_exp.cpu(), c.v_exp),
        lambda: ns.KvPages(c.k.to(BF16), c.v.to(BF16), *t, c.k_exp, c.v_exp),
        lambda: c.write(0, i32([0]), i32([0, 1]), x.float(), x.float()),
        lambda: c.write(0, i32([0]), i32([0, 1]), x.to(E4M3), x.to(E4M3)),
        lambda: c.write(0, i32([0]), i32([0, 1]), x, x.half()),
        lambda: c.write(0, i32([0]), i32([0, 1]), x[..., :32], x[..., :32]),
        lambda: c.read(0, i32([0]), i32([0, 1]), 1, dtype=torch.float32),
        lambda: c.read(0, i32([0]), i32([0, 1]), -1),
        lambda: c.read(0, i32([0]), i32([0, 1]), 1, k_out=x.half()),
        lambda: c.read(0, i32([0]), i32([0, 1]), 2, k_out=x),
        lambda: c.read(0, i32([0]), i32([0, 1]), 1, k_out=x[:, :1].expand(1, 2, 64)),
        lambda: c.read(0, i32([0]), i32([0]), 1),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            f()
            pytest.fail(f"call {i} was not refused")
    with pytest.raises(ns.NanoSpecError):
        c.write(1, i32([0]), i32([0, 1]), x, x)
    with pytest.raises(ns.NanoSpecError):
        c.read(-1, i32([0]), i32([0, 1]), 1)
    plain = new(scaled=False, dtype=E4M3)  # rows of bytes, moved as they are
    assert plain.k_exp is None
    plain.extend(i32([0]), i32([1]))
    plain.write(0, i32([0]), i32([0, 1]), x.to(E4M3), x.to(E4M3))
    with pytest.raises(ValueError):
        plain.read(0, i32([0]), i32([0, 1]), 1, dtype=BF16)
    assert ns.ops_error() == 0
