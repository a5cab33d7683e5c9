"""More serving operators around the draft head, as they are measured.

Four kinds of call, each from the smallest to the largest:

* ``rotate``  norms of queries and keys for each head and the position
              rotation, in one pass;
* ``store``   new keys and values quantised into an 8-bit paged cache, and
              read back from it;
* ``decode``  attention of a sequence's new tokens over that cache;
* ``shared``  attention of sequences that share a long prefix, over a cache
              of 16 bits.

``run`` computes them in elementary torch operations (``own`` false) or
through the package's entry points (``own`` true).
"""

from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E4M3 = torch.float8_e4m3fn
LARGEST = 448.0  # of e4m3
DEV = "cuda"


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # One decoded token of one user, norms and rotation of the whole head: latency.
        {"name": "rotate_one_bf16", "op": "rotate", "dtype": "bf16", "q_heads": 32, "kv_heads": 8, "dim": 128,
         "rotary": 128, "tokens": 1, "furthest": 4097, "norm": True, "neighbours": False},
        # The 60-node trees of 16 sequences far into long contexts, half of each head rotated, no norm.
        {"name": "rotate_tree_f16", "op": "rotate", "dtype": "f16", "q_heads": 28, "kv_heads": 4, "dim": 128,
         "rotary": 64, "tokens": 960, "furthest": 1000000, "norm": False, "neighbours": True},
        # A long document's prefill.
        {"name": "rotate_prompt_bf16", "op": "rotate", "dtype": "bf16", "q_heads": 32, "kv_heads": 8, "dim": 128,
         "rotary": 128, "tokens": 16381, "furthest": 16381, "norm": True, "neighbours": False},
        # One decode step: the 60-node trees of 16 sequences into the cache.
        {"name": "store_tree_bf16", "op": "store", "dtype": "bf16", "kv_heads": 8, "dim": 128, "page": 16, "seqs": 16,
         "new": 60, "shortest": 512, "longest": 4096, "mix": 1},
        # Long chunks of eight prompts.
        {"name": "store_prompt_f16", "op": "store", "dtype": "f16", "kv_heads": 4, "dim": 128, "page": 64, "seqs": 8,
         "new": 4001, "shortest": 1, "longest": 900, "mix": 2},
        # One user, one new token, a context of a few thousand tokens: latency.
        {"name": "decode_one_bf16", "op": "decode", "dtype": "bf16", "q_heads": 32, "kv_heads": 8, "dim": 128,
         "page": 16, "seqs": 1, "new": 1, "tree": False, "shortest": 4097, "longest": 4097, "mix": 1},
        # A full batch of one-token steps over contexts of very different lengths.
        {"name": "decode_batch_f16", "op": "decode", "dtype": "f16", "q_heads": 28, "kv_heads": 4, "dim": 128,
         "page": 64, "seqs": 48, "new": 1, "tree": False, "shortest": 200, "longest": 40000, "mix": 7},
        # Verification of 60-node draft trees for 16 sequences with 512 to 4096 tokens of context.
        {"name": "decode_tree_bf16", "op": "decode", "dtype": "bf16", "q_heads": 32, "kv_heads": 8, "dim": 128,
         "page": 16, "seqs": 16, "new": 60, "tree": True, "shortest": 512, "longest": 4096, "mix": 2},
        # Eight continuations of one prompt, a token each: latency.
        {"name": "shared_one_bf16", "op": "shared", "dtype": "bf16", "q_heads": 32, "kv_heads": 8, "dim": 128,
         "page": 16, "groups": 1, "members": 8, "new": 1, "tree": False, "shortest": 2101, "longest": 2101,
         "most_own": 150, "mix": 1},
        # Four long prompts with 16 continuations each, a token each.
        {"name": "shared_batch_f16", "op": "shared", "dtype": "f16", "q_heads": 28, "kv_heads": 4, "dim": 128,
         "page": 64, "groups": 4, "members": 16, "new": 1, "tree": False, "shortest": 3001, "longest": 16000,
         "most_own": 600, "mix": 2},
        # Verification of 60-node draft trees for 16 continuations of one prompt.
        {"name": "shared_tree_bf16", "op": "shared", "dtype": "bf16", "q_heads": 32, "kv_heads": 8, "dim": 128,
         "page": 16, "groups": 1, "members": 16, "new": 60, "tree": True, "shortest": 6007, "longest": 6007,
         "most_own": 400, "mix": 3},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = [(32, 8), (28, 4), (12, 4), (8, 8), (16, 2), (24, 8), (16, 1)]


def draw(rng):
    op = rng.choice(["rotate", "store", "decode", "shared"])
    mix = rng.randrange(1 << 20)
    hq, hkv = rng.choice(HEADS)
    dim = rng.choice([64, 128, 128])
    case = {"op": op, "dtype": rng.choice(["bf16", "f16"]), "q_heads": hq, "kv_heads": hkv, "dim": dim}
    if op == "rotate":
        return case | {"rotary": rng.choice([dim, dim, dim // 2, 32]), "tokens": _log_int(rng, 1, 16381),
                       "furthest": _log_int(rng, 1, 1000000), "norm": rng.random() < 0.6,
                       "neighbours": rng.random() < 0.4, "mix": mix}
    if op == "store":
        seqs = _log_int(rng, 1, 64)
        return {"op": op, "dtype": case["dtype"], "kv_heads": rng.choice([1, 2, 4, 8]), "dim": dim,
                "page": rng.choice([8, 16, 32, 64, 128]), "seqs": seqs, "new": _log_int(rng, 1, 30000 // seqs),
                "shortest": 1, "longest": _log_int(rng, 1, 4000), "mix": mix}
    new = rng.choice([1, 1, 1, rng.randrange(2, 65)])
    case |= {"page": rng.choice([8, 16, 32, 64, 128]), "new": new, "tree": new > 1 and rng.random() < 0.7, "mix": mix}
    if op == "decode":
        longest = _log_int(rng, 1 if new == 1 else 64, 100000 if new == 1 else 8000)
        return case | {"seqs": max(1, min(_log_int(rng, 1, 128), 250000 // longest)),
                       "shortest": _log_int(rng, 1, longest), "longest": longest}
    longest = _log_int(rng, 1, 16000 if new == 1 else 6000)
    seqs = max(1, min(_log_int(rng, 1, 64), (250000 if new == 1 else 100000) // longest))
    groups = min(seqs, _log_int(rng, 1, 6))
    return case | {"groups": groups, "members": max(1, seqs // groups), "shortest": _log_int(rng, 1, longest),
                   "longest": longest, "most_own": _log_int(rng, 1, 1000)}


def _lengths(case, n):
    """n lengths, spread over the logarithm of their range; the last is the longest."""
    r = random.Random(case["mix"])
    return [_log_int(r, case["shortest"], case["longest"]) for _ in range(n - 1)] + [case["longest"]]


def _own_lengths(case):
    """What each member of each group holds behind its prompt."""
    r = random.Random(case["mix"] + 1)
    return [[_log_int(r, 1, case["most_own"]) for _ in range(case["members"])] for _ in range(case["groups"])]


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, dtype, std=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype).mul_(std)


def _rows(g, shape, dtype):
    """Rows of keys or values: each of a size of its own, a few columns larger than the others."""
    x = torch.randn(shape, generator=g, device=DEV, dtype=dtype)
    x *= torch.randn(shape[:-1], generator=g, device=DEV).mul_(0.5).exp_()[..., None].to(dtype)
    x[..., 3::29] *= 6.0
    return x


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _ancestors(n, rng):
    """Bits of every node's ancestors and itself in a random tree whose parents come before their children."""
    bits = []
    for i in range(n):
        parent = rng.randrange(-1, i) if i else -1
        bits.append((1 << i) | (bits[parent] if parent >= 0 else 0))
    return [b - (1 << 64) if b >= 1 << 63 else b for b in bits]


def _table(held, pages, rng, first=()):
    """A table with `held` pages for each sequence, in random order; first[b]: pages that sequence b begins with."""
    order = list(range(pages))
    rng.shuffle(order)
    table = torch.full((len(held), max(held)), -1, dtype=torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32)
    taken = {}
    at = 0
    for b, n in enumerate(held):
        mine = []
        if first:
            who, shared = first[b]
            if who not in taken:
                taken[who] = order[at:at + shared]
                at += shared
            mine = taken[who][:shared]
        mine = mine + order[at:at + n - len(mine)]
        at += n - (first[b][1] if first else 0)
        table[b, :n] = torch.tensor(mine, dtype=torch.int32)
        refs[mine] += 1
    return table.to(DEV), refs.to(DEV)


def prepare(case, seed):
    g = _gen(seed)
    rng = random.Random(int(seed) * 2 + 1)
    op = case["op"]
    dt = DTYPES[case["dtype"]]
    hkv, d = case["kv_heads"], case["dim"]
    if op == "rotate":
        T, hq, R = case["tokens"], case["q_heads"], case["rotary"]
        # a fused projection's output: queries, keys and values are slices of one row
        qkv = _normal(g, (T, hq + 2 * hkv, d), dt)
        last = case["furthest"]
        pos = torch.arange(max(0, last - T), max(0, last - T) + T, device=DEV, dtype=torch.int32)
        inv = 500000.0 ** (-torch.arange(0, R, 2, device=DEV, dtype=torch.float64) / R)
        w = None
        if case["norm"]:
            w = [1.0 + 0.2 * torch.randn(d, generator=g, device=DEV) for _ in range(2)]
            w = [x.to(dt) for x in w]
        return {"op": op, "q": qkv[:, :hq], "k": qkv[:, hq:hq + hkv], "pos": pos, "inv_freq": inv,
                "q_weight": w[0] if w else None, "k_weight": w[1] if w else None, "eps": 1e-6 if w else None,
                "neighbours": case["neighbours"]}
    new, P = case["new"], case["page"]
    if op == "store":
        B = case["seqs"]
        lens = [n + new for n in _lengths(case, B)]
        held = [-(-n // P) for n in lens]
        pages = sum(held) + 5
        table, refs = _table(held, pages, rng)
        codes = [torch.zeros((1, pages, hkv, P, d), dtype=torch.uint8, device=DEV).view(E4M3) for _ in range(2)]
        exps = [torch.full((1, pages, hkv, P), 127, dtype=torch.uint8, device=DEV) for _ in range(2)]
        return {"op": op, "k": codes[0], "v": codes[1], "k_exp": exps[0], "v_exp": exps[1], "table": table,
                "lengths": _i32(lens), "refs": refs, "seqs": _i32(list(range(B))),
                "cu": _i32([new * i for i in range(B + 1)]), "tokens": new * B,
                "k_new": _rows(g, (B * new, hkv, d), dt), "v_new": _rows(g, (B * new, hkv, d), dt)}
    hq = case["q_heads"]
    if op == "decode":
        B = case["seqs"]
        lens = [n + new for n in _lengths(case, B)]
        held = [-(-n // P) for n in lens]
        table, _ = _table(held, sum(held) + 7, rng)
        pages = sum(held) + 7
        k, k_exp = _quantise(_rows(g, (pages, hkv, P, d), dt))
        v, v_exp = _quantise(_rows(g, (pages, hkv, P, d), dt))
        s = {"k": k, "v": v, "k_exp": k_exp, "v_exp": v_exp}
    else:
        B = case["groups"] * case["members"]
        prompts = _lengths(case, case["groups"])
        lens, held, first = [], [], []
        for i, (prompt, tails) in enumerate(zip(prompts, _own_lengths(case))):
            for tail in tails:
                lens.append(prompt + tail + new)
                held.append(-(-lens[-1] // P))
                first.append((i, prompt // P))
        pages = sum(held) - sum((case["members"] - 1) * (p // P) for p in prompts) + 7
        table, _ = _table(held, pages, rng, first)
        s = {"k": _normal(g, (pages, hkv, P, d), dt), "v": _normal(g, (pages, hkv, P, d), dt),
             "groups": _i32([case["members"] * i for i in range(case["groups"] + 1)])}
    mask = None
    if case["tree"]:
        mask = torch.tensor([_ancestors(new, rng) for _ in range(B)], dtype=torch.int64, device=DEV)
    return s | {"op": op, "q": _normal(g, (B, new, hq, d), dt), "table": table, "lengths": _i32(lens),
                "seqs": _i32(list(range(B))), "mask": mask, "scale": d ** -0.5, "max_len": max(lens)}


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    if own:
        return _run_own(state)
    return {"rotate": _rotate, "store": _store, "decode": _attend, "shared": _attend}[state["op"]](state)


def _run_own(s):
    import speculative_decoding_draft_stream_gb300 as ns

    op = s["op"]
    if op == "rotate":
        q, k = ns.norm_rotate(s["q"], s["k"], s["pos"], s["inv_freq"], q_weight=s["q_weight"],
                              k_weight=s["k_weight"], eps=s["eps"], neighbours=s["neighbours"])
        return {"q": q, "k": k}
    if op == "store":
        cache = ns.KvPages(s["k"], s["v"], s["table"], s["lengths"], s["refs"], s["k_exp"], s["v_exp"])
        cache.write(0, s["seqs"], s["cu"], s["k_new"], s["v_new"])
        k, v = cache.read(0, s["seqs"], s["cu"], s["tokens"], dtype=s["k_new"].dtype)
        return {"k": k, "v": v, "k_exp": s["k_exp"], "v_exp": s["v_exp"]}
    if op == "decode":
        out, lse = ns.attend_paged(s["q"], s["k"], s["v"], s["table"], s["lengths"], s["seqs"], mask=s["mask"],
                                   scale=s["scale"], max_len=s["max_len"], k_exp=s["k_exp"], v_exp=s["v_exp"])
        return {"out": out, "lse": lse}
    out, lse = ns.attend_shared(s["q"], s["k"], s["v"], s["table"], s["lengths"], s["seqs"], s["groups"],
                                mask=s["mask"], scale=s["scale"], max_len=s["max_len"])
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _rotate_heads(x, weight, s, cos, sin):
    y = x.float()
    if s["eps"] is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"]) * weight.float()
    R = 2 * s["inv_freq"].numel()
    if s["neighbours"]:
        a, b = y[..., 0:R:2], y[..., 1:R:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = y[..., :R // 2], y[..., R // 2:R]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, y[..., R:]), -1).to(x.dtype)


def _rotate(s):
    angle = s["pos"].double()[:, None, None] * s["inv_freq"]  # in 64 bits: far positions
    cos, sin = angle.cos().float(), angle.sin().float()
    return {"q": _rotate_heads(s["q"], s["q_weight"], s, cos, sin),
            "k": _rotate_heads(s["k"], s["k_weight"], s, cos, sin)}


def _pow2(e):
    """2^e for whole e from -126 to 127, exactly (torch's own powers on a GPU are rounded)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantise(x):
    """Codes (e4m3) and the exponents' bytes of rows: the smallest power of two by which the row fits, within 2^+-40; a
    row that is not finite has 255."""
    x = x.float()
    most = x.abs().amax(-1)
    fine = torch.isfinite(most)
    m, e = torch.frexp(torch.where(fine, most, 0.0))
    e = torch.where(most == 0, -40, (e - 9 + (m > LARGEST / 512).int()).clamp(-40, 40))
    codes = (torch.where(fine[..., None], x, 0.0) * _pow2(-e)[..., None]).clamp(-LARGEST, LARGEST).to(E4M3)
    return codes, torch.where(fine, e + 127, 255).to(torch.uint8)


def _values(codes, exps):
    """What codes and exponents stand for, in 32 bits."""
    scale = torch.where(exps == 255, math.nan, _pow2(torch.where(exps == 255, 0, exps.int() - 127)))
    return codes.float() * scale[..., None]


def _store(s):
    P, seqs, cu, table = s["k"].shape[3], s["seqs"].long(), s["cu"].long(), s["table"]
    tok = torch.arange(s["tokens"], device=table.device)
    i = torch.searchsorted(cu, tok, right=True) - 1
    at = s["lengths"][seqs][i].long() - (cu[1:] - cu[:-1])[i] + tok - cu[i]
    page, row = table[seqs[i], at // P].long(), at % P
    back = []
    for codes, exps, rows in ((s["k"], s["k_exp"], s["k_new"]), (s["v"], s["v_exp"], s["v_new"])):
        c, e = _quantise(rows)
        codes.view(torch.uint8)[0][page, :, row] = c.view(torch.uint8)
        exps[0][page, :, row] = e
        c = codes.view(torch.uint8)[0][page, :, row].view(E4M3)
        back.append(_values(c, exps[0][page, :, row]).to(rows.dtype))
    return {"k": back[0], "v": back[1], "k_exp": s["k_exp"], "v_exp": s["v_exp"]}


def _softmax_parts(scores):
    """In place: exp(scores - row maximum), the row's sum and its log-sum-exp; a row of -inf gives zeros and -inf."""
    m = scores.amax(-1, keepdim=True)
    m0 = m.clamp_min(torch.finfo(scores.dtype).min)
    scores.sub_(m0).exp_()
    total = scores.sum(-1, keepdim=True)
    return scores, total, (m0 + total.log()).squeeze(-1)


def _gather(s, name, page, row, inside):
    rows = s[name].view(torch.uint8)[page, :, row].view(E4M3) if s["op"] == "decode" else s[name][page, :, row]
    x = _values(rows, s[name + "_exp"][page, :, row]) if s["op"] == "decode" else rows.float()
    return x * inside[..., None, None]


def _attend(s):
    q = s["q"]
    B, n, hq, d = q.shape
    hkv, P, N = s["k"].shape[1], s["k"].shape[2], s["max_len"]
    grp = hq // hkv
    table, lens = s["table"][s["seqs"].long()].long(), s["lengths"][s["seqs"].long()].long()
    pos = torch.arange(N, device=q.device)
    page = table[:, pos // P].clamp_min(0)
    inside = pos < lens[:, None]
    kp = _gather(s, "k", page, pos % P, inside)
    qp = q.float().view(B, n, hkv, grp, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, n * grp, d)
    scores = (qp @ kp.permute(0, 2, 3, 1)).mul_(s["scale"]).view(B, hkv, n, grp, N)
    del kp
    node = pos - (lens[:, None] - n)  # a position's node, negative in the context
    rows = torch.arange(n, device=q.device)
    if s["mask"] is None:
        sees = node[:, None, :] <= rows[:, None]
    else:
        sees = (node[:, None, :] < 0) | ((s["mask"][:, :, None] >> node[:, None, :].clamp(0, 63)) & 1).bool()
    sees = sees & inside[:, None, :]
    scores.masked_fill_(~sees[:, None, :, None, :], -math.inf)
    e, total, lse = _softmax_parts(scores)
    vp = _gather(s, "v", page, pos % P, inside)
    out = (e.view(B, hkv, n * grp, N) @ vp.permute(0, 2, 1, 3)).view(B, hkv, n, grp, d)
    out = torch.where(total > 0, out / total, 0.0)
    return {"out": out.permute(0, 2, 1, 3, 4).reshape(B, n, hq, d).to(q.dtype),
            "lse": lse.permute(0, 2, 1, 3).reshape(B, n, hq)}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op, hkv, d = case["op"], case["kv_heads"], case["dim"]
    if op == "rotate":
        n = case["tokens"] * (case["q_heads"] + hkv)
        return {"bytes": 4 * n * d + 4 * case["tokens"] + 4 * case["rotary"],
                "flops": n * (3 * case["rotary"] + (4 * d if case["norm"] else 0))}
    if op == "store":  # 16 bits to 8 and an exponent, and back
        rows = 2 * case["seqs"] * case["new"] * hkv
        return {"bytes": rows * 2 * (3 * d + 1), "flops": rows * d * 4}
    n, hq = case["new"], case["q_heads"]
    if op == "decode":
        lens = [x + n for x in _lengths(case, case["seqs"])]
        return {"bytes": sum(lens) * hkv * (d + 1) * 2 + len(lens) * n * hq * (4 * d + 4),
                "flops": 4 * sum(lens) * n * hq * d}
    prompts, tails = _lengths(case, case["groups"]), _own_lengths(case)
    seqs = case["groups"] * case["members"]
    once = sum(prompts) + sum(x + n for t in tails for x in t)  # (the prompts' last pages are not shared: a few rows)
    every = sum(p + x + n for p, t in zip(prompts, tails) for x in t)
    return {"bytes": once * hkv * d * 4 + seqs * n * hq * (4 * d + 4), "flops": 4 * every * n * hq * d}


# ---------------------------------------------------------------------------
# From the definition, in 64 bits
# ---------------------------------------------------------------------------
def _attend64(q, k, v, sees, scale):
    """q [m, d], k and v [n, d], sees [m, n]: the output and log-sum-exp of every row."""
    z = torch.where(sees, (q.double() @ k.T) * scale, -math.inf)
    lse = torch.logsumexp(z, -1)
    p = torch.exp(z - torch.where(torch.isinf(lse), 0.0, lse)[:, None])
    return p @ v, lse


def _rotated64(x, weight, s, turn):
    """x as complex numbers, multiplied by turn = exp(i angle)."""
    y = x.double()
    if s["eps"] is not None:
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / y.shape[-1] + s["eps"]) * weight.double()
    h = s["inv_freq"].numel()
    if s["neighbours"]:
        z = torch.view_as_complex(y[..., :2 * h].unflatten(-1, (h, 2)).contiguous()) * turn
        return torch.cat((torch.view_as_real(z).flatten(-2), y[..., 2 * h:]), -1)
    z = torch.complex(y[..., :h], y[..., h:2 * h]) * turn
    return torch.cat((z.real, z.imag, y[..., 2 * h:]), -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotate":
        angle = s["pos"].double()[:, None, None] * s["inv_freq"].double()
        turn = torch.polar(torch.ones_like(angle), angle)
        return {"q": _rotated64(s["q"], s["q_weight"], s, turn), "k": _rotated64(s["k"], s["k_weight"], s, turn)}
    if case["op"] == "store":
        back = []
        for x in (s["k_new"].double(), s["v_new"].double()):
            # steps of e4m3 scaled by 2^e: 2^-3 of a value's power of two, 2^-9 at the least
            top = x.abs().amax(-1, keepdim=True)
            e = torch.frexp(top / (LARGEST / 512)).exponent - 9
            e = (e - (top <= LARGEST * _pow2(e - 1).double()).int()).clamp(-40, 40)
            size = torch.frexp(x * _pow2(-e).double()).exponent.clamp_min(-5) - 1
            step = _pow2(size - 3 + e).double()
            back.append(torch.round(x / step) * step)
        return {"k": back[0], "v": back[1], "k_exp": None, "v_exp": None}
    q, P = s["q"], s["k"].shape[2]
    B, n, hq, d = q.shape
    hkv = s["k"].shape[1]
    grp = hq // hkv
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(q.shape[:3], dtype=torch.float64, device=DEV)

    def rows(name, pages, h, N):
        x = s[name].view(torch.uint8).view(s[name].dtype)[pages, h].double()
        if case["op"] == "decode":
            x = x * _pow2(s[name + "_exp"][pages, h].int() - 127)[..., None].double()
        return x.reshape(-1, d)[:N]

    for b in range(B):
        N = int(s["lengths"][b])
        pages = s["table"][b, :-(-N // P)].long()
        sees = torch.ones((n, N), dtype=torch.bool, device=DEV)
        for i in range(n):
            word = (1 << (i + 1)) - 1 if s["mask"] is None else int(s["mask"][b, i])
            sees[i, N - n:] = torch.tensor([bool(word >> j & 1) for j in range(n)], device=DEV)
        for h in range(hkv):
            o, z = _attend64(q[b, :, h * grp:(h + 1) * grp].reshape(n * grp, d), rows("k", pages, h, N),
                             rows("v", pages, h, N), sees.repeat_interleave(grp, 0), s["scale"])
            out[b, :, h * grp:(h + 1) * grp] = o.view(n, grp, d)
            lse[b, :, h * grp:(h + 1) * grp] = z.view(n, grp)
    return {"out": out, "lse": lse}
