"""Plain references of the serving operators, in 64 bits on the CPU, and the
tolerances of their tests.

Tolerances.  With u the unit roundoff of the 16-bit type (a significand of p
bits, rounded to nearest, is off by 2^-p: p = 8 in bf16, 11 in fp16), an attention output
o = sum p v is rounded once at the end (u |o|) and its probabilities once
before the product (u sum p |v|).  A score is an fp32 sum of D products, each
exact: its error is at most (D + 8) 2^-24 times sum |q k| scale, and moves p
by that factor; sums of n probabilities in fp32 add at most n 2^-24, and the
exponential 2^-21.  So with e = (D + 8) 2^-24 M + n 2^-24 + 2^-20, where M is
the largest sum |q k| scale of the row,
   |lse error| <= e,   |o error| <= (u + 2 e) sum p |v| + u |o|.
(fp16 outputs below its smallest normal number add half of 2^-24.)
"""

import math

import torch

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def attend_rows(q, k, v, sees, scale):
    """q [m, D], k and v [n, D], sees bool [m, n] -> (o, lse, bound on |o| error, bound on |lse| error)."""
    dt, (n, d) = q.dtype, k.shape
    q, k, v = q.double(), k.double(), v.double()
    z = (q @ k.T) * scale
    z = torch.where(sees, z, torch.full_like(z, -math.inf))
    lse = torch.logsumexp(z, -1) if n else torch.full((q.shape[0],), -math.inf, dtype=torch.float64)
    p = torch.exp(z - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None])
    p = torch.where(sees, p, torch.zeros_like(p))
    # a hidden value is no part of the sum, whatever it holds
    wild = ~torch.isfinite(v)
    o = p @ torch.where(wild, torch.zeros_like(v), v)
    a = p @ torch.where(wild, torch.zeros_like(v), v).abs()
    if wild.any():
        o = torch.where((sees.double() @ wild.double()) > 0, torch.full_like(o, math.nan), o)
    big = ((q.abs() @ k.abs().T) * sees).amax(-1) * scale if n else torch.zeros(q.shape[0], dtype=torch.float64)
    e = (d + 8) * 2.0 ** -24 * big + n * 2.0 ** -24 + 2.0 ** -20
    u = UNIT[dt]
    tol = (u + 2 * e)[:, None] * a + u * torch.nan_to_num(o).abs() + (2.0 ** -25 if dt == torch.float16 else 0.0)
    return o, lse, tol, e


def check(got, want, tol, what):
    """|got - want| <= tol, NaN and infinities where they are wanted."""
    got = got.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    fine = torch.isfinite(want)
    assert torch.isfinite(got[fine]).all(), f"{what}: not finite"
    over = ((got - want).abs() - tol)[fine]
    assert over.numel() == 0 or over.max() <= 0, f"{what}: off by {over.max():.3g} more than its bound"


class Pages:
    """The cache's rules, one step at a time, over nested lists (k and v: numpy arrays of rows)."""

    def __init__(self, k, v, table, lengths, refs):
        self.k, self.v = k.copy(), v.copy()
        self.table, self.lengths, self.refs = [list(r) for r in table], list(lengths), list(refs)
        self.P = k.shape[3]

    def held(self, s):
        return -(-self.lengths[s] // self.P)

    def truncate(self, seqs, new):
        for s, n in zip(seqs, new):
            if n >= self.lengths[s]:
                continue
            for slot in range(-(-n // self.P), self.held(s)):
                self.refs[self.table[s][slot]] -= 1
                self.table[s][slot] = -1
            self.lengths[s] = n

    def fork(self, src, dst):
        for a, b in zip(src, dst):
            assert self.lengths[b] == 0
            for slot in range(self.held(a)):
                p = self.table[a][slot]
                self.table[b][slot] = p
                self.refs[p] += 1
            self.lengths[b] = self.lengths[a]

    def extend(self, seqs, new):
        free = [p for p, r in enumerate(self.refs) if r == 0]
        was = list(self.refs)
        gives = []
        for s, n in zip(seqs, new):
            first, want = self.held(s), -(-(self.lengths[s] + n) // self.P)
            copied = n > 0 and self.lengths[s] % self.P != 0 and was[self.table[s][first - 1]] > 1
            gives.append((s, n, first - int(copied), want, copied))
        if sum(w - f for _, _, f, w, _ in gives) > len(free):
            return False
        for s, n, first, want, copied in gives:
            for slot in range(first, want):
                p = free.pop(0)
                if copied and slot == first:
                    old = self.table[s][slot]
                    self.k[:, p], self.v[:, p] = self.k[:, old], self.v[:, old]
                    self.refs[old] -= 1
                self.table[s][slot] = p
                self.refs[p] += 1
            self.lengths[s] += n
        return True

    def row(self, s, pos):
        return self.table[s][pos // self.P], pos % self.P

    def write(self, layer, seqs, cu, k_new, v_new):
        for i, s in enumerate(seqs):
            for t in range(cu[i], cu[i + 1]):
                p, r = self.row(s, self.lengths[s] - (cu[i + 1] - t))
                if self.refs[p] == 1:
                    self.k[layer, p, :, r], self.v[layer, p, :, r] = k_new[t], v_new[t]

    def compact(self, seqs, base, keep):
        for s, b, ks in zip(seqs, base, keep):
            for t, frm in enumerate(ks):
                (p0, r0), (p1, r1) = self.row(s, b + frm), self.row(s, b + t)
                self.k[:, p1, :, r1], self.v[:, p1, :, r1] = self.k[:, p0, :, r0], self.v[:, p0, :, r0]
        self.truncate(seqs, [b + len(ks) for b, ks in zip(base, keep)])

    def copy(self, src, dst):
        for a, b in zip(src, dst):
            self.k[:, b], self.v[:, b] = self.k[:, a], self.v[:, a]


def with_wild_values(o, v, sees):
    """o [m, d] of finite values, as it is where some of v [n, d] are not: a row that sees a NaN, or infinities of both
    signs, in a column has NaN there; infinities of one sign, that infinity (every probability is above 0)."""
    s = sees.double()
    nan, pos, neg = ((s @ w.double()) > 0 for w in (torch.isnan(v), v == math.inf, v == -math.inf))
    o = torch.where(pos, torch.full_like(o, math.inf), torch.where(neg, torch.full_like(o, -math.inf), o))
    return torch.where(nan | (pos & neg), torch.full_like(o, math.nan), o)
