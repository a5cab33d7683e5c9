"""The serving operators around the draft head, as they are measured.

Four operators, each with cases from the smallest call to the largest:

* ``prompt``   attention over whole packed prompts (causal, grouped heads);
* ``decode``   attention of a sequence's new tokens (one, or the nodes of a
               draft tree) over a paged key-value cache;
* ``pages``    the cache's bookkeeping and data movement in one decode step:
               truncate, fork, extend (with copies of shared last pages),
               write, compact;
* ``logprobs`` log probabilities of given tokens, with the entropy and the
               top alternatives.

``run`` computes them in elementary torch operations (``own`` false) or
through the package's entry points (``own`` true).
"""

from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
DEV = "cuda"


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # Four short prompts of a small draft model arriving together (one of them a single token): latency.
        {"name": "prompt_short_f16", "op": "prompt", "dtype": "f16", "q_heads": 12, "kv_heads": 4, "dim": 64,
         "seqs": 4, "shortest": 1, "longest": 200, "mix": 3},
        # A prefill batch of ragged prompts, 28 query heads on 4 key-value heads (groups of seven).
        {"name": "prompt_batch_bf16", "op": "prompt", "dtype": "bf16", "q_heads": 28, "kv_heads": 4, "dim": 128,
         "seqs": 16, "shortest": 130, "longest": 2047, "mix": 5},
        # One long document, odd length, the Llama-3-8B head layout.
        {"name": "prompt_long_bf16", "op": "prompt", "dtype": "bf16", "q_heads": 32, "kv_heads": 8, "dim": 128,
         "seqs": 1, "shortest": 16381, "longest": 16381, "mix": 1},
        # One user, one new token, a context of a few thousand tokens: latency.
        {"name": "decode_one_bf16", "op": "decode", "dtype": "bf16", "q_heads": 32, "kv_heads": 8, "dim": 128,
         "page": 16, "seqs": 1, "new": 1, "tree": False, "shortest": 4097, "longest": 4097, "mix": 1},
        # A full batch of one-token steps over contexts of very different lengths.
        {"name": "decode_batch_f16", "op": "decode", "dtype": "f16", "q_heads": 28, "kv_heads": 4, "dim": 128,
         "page": 64, "seqs": 48, "new": 1, "tree": False, "shortest": 200, "longest": 40000, "mix": 7},
        # Verification of 60-node draft trees for 16 sequences with 512 to 4096 tokens of context.
        {"name": "decode_tree_bf16", "op": "decode", "dtype": "bf16", "q_heads": 32, "kv_heads": 8, "dim": 128,
         "page": 16, "seqs": 16, "new": 60, "tree": True, "shortest": 512, "longest": 4096, "mix": 2},
        # After a verification: 16 sequences take back the last step, append 60 nodes, keep the accepted path.
        {"name": "pages_accept_bf16", "op": "pages", "dtype": "bf16", "layers": 16, "kv_heads": 8, "dim": 128,
         "page": 16, "seqs": 16, "children": 0, "new": 60, "keep": 5, "shortest": 512, "longest": 1500, "mix": 4},
        # Branching: every sequence forked four ways, each child extended by a few tokens (its last page copied).
        {"name": "pages_branch_bf16", "op": "pages", "dtype": "bf16", "layers": 16, "kv_heads": 8, "dim": 128,
         "page": 16, "seqs": 16, "children": 4, "new": 5, "keep": 0, "shortest": 300, "longest": 1400, "mix": 6},
        # Eviction: long chunks are appended and every second position of them is dropped again.
        {"name": "pages_evict_f16", "op": "pages", "dtype": "f16", "layers": 12, "kv_heads": 4, "dim": 128,
         "page": 64, "seqs": 8, "children": 0, "new": 4001, "keep": 2000, "shortest": 100, "longest": 900, "mix": 8},
        # One decoded token: its log probability and ten alternatives.
        {"name": "logprobs_one_f32", "op": "logprobs", "dtype": "f32", "rows": 1, "vocab": 128256, "ids": 1, "k": 10,
         "temperature": 1.0},
        # The nodes of a draft tree: each node's children under the verifier's distribution.
        {"name": "logprobs_tree_f32", "op": "logprobs", "dtype": "f32", "rows": 60, "vocab": 151936, "ids": 10,
         "k": 10, "temperature": 0.7},
        # Scoring a prompt: every position's next token, with five alternatives.
        {"name": "logprobs_prompt_bf16", "op": "logprobs", "dtype": "bf16", "rows": 2048, "vocab": 152064, "ids": 1,
         "k": 5, "temperature": 1.0},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = [(32, 8), (28, 4), (12, 4), (8, 8), (16, 2), (24, 8), (16, 1)]


def draw(rng):
    op = rng.choice(["prompt", "decode", "pages", "logprobs"])
    mix = rng.randrange(1 << 20)
    if op == "prompt":
        hq, hkv = rng.choice(HEADS)
        longest = _log_int(rng, 1, 16381)
        seqs = max(1, min(_log_int(rng, 1, 64), int(8.0e9 / (hq * longest * longest))))
        return {"op": op, "dtype": rng.choice(["bf16", "f16"]), "q_heads": hq, "kv_heads": hkv,
                "dim": rng.choice([64, 128, 128]), "seqs": seqs, "shortest": _log_int(rng, 1, longest),
                "longest": longest, "mix": mix}
    if op == "decode":
        hq, hkv = rng.choice(HEADS)
        new = rng.choice([1, 1, 1, rng.randrange(2, 65)])
        longest = _log_int(rng, 1 if new == 1 else 64, 100000 if new == 1 else 8000)
        seqs = max(1, min(_log_int(rng, 1, 128), 250000 // longest))
        return {"op": op, "dtype": rng.choice(["bf16", "f16"]), "q_heads": hq, "kv_heads": hkv,
                "dim": rng.choice([64, 128, 128]), "page": rng.choice([8, 16, 32, 64, 128]), "seqs": seqs, "new": new,
                "tree": new > 1 and rng.random() < 0.7, "shortest": _log_int(rng, 1, longest), "longest": longest,
                "mix": mix}
    if op == "pages":
        seqs = _log_int(rng, 1, 32)
        page = rng.choice([8, 16, 32, 64])
        longest = _log_int(rng, 1, 1500)
        children = rng.choice([0, 0, rng.randrange(1, 6)])
        new = _log_int(rng, 1, 100 if children else max(1, 30000 // seqs // 4))
        keep = 0 if children else rng.randrange(0, new + 1)
        return {"op": op, "dtype": rng.choice(["bf16", "f16"]), "layers": rng.randrange(1, 17),
                "kv_heads": rng.choice([1, 2, 4, 8]), "dim": rng.choice([64, 128]), "page": page, "seqs": seqs,
                "children": children, "new": new, "keep": keep, "shortest": _log_int(rng, 1, longest),
                "longest": longest, "mix": mix}
    vocab = rng.choice([128256, 152064, 151936, rng.randrange(1000, 160000)])
    return {"op": op, "dtype": rng.choice(["f32", "bf16", "f16"]), "rows": _log_int(rng, 1, 1024), "vocab": vocab,
            "ids": rng.randrange(1, 17), "k": rng.randrange(0, 33), "temperature": rng.choice([1.0, 0.7, 1.3])}


def _lengths(case):
    """The sequences' lengths, spread over the logarithm of their range; the last has the longest."""
    r = random.Random(case["mix"])
    return [_log_int(r, case["shortest"], case["longest"]) for _ in range(case["seqs"] - 1)] + [case["longest"]]


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, dtype, std=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype).mul_(std)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _ancestors(n, rng):
    """Bits of every node's ancestors and itself in a random tree whose parents come before their children."""
    bits = []
    for i in range(n):
        parent = rng.randrange(-1, i) if i else -1
        b = (1 << i) | (bits[parent] if parent >= 0 else 0)
        bits.append(b)
    return [b - (1 << 64) if b >= 1 << 63 else b for b in bits]


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    dt = DTYPES[case["dtype"]]
    if op == "prompt":
        lens = _lengths(case)
        T, hq, hkv, d = sum(lens), case["q_heads"], case["kv_heads"], case["dim"]
        # a fused projection's output: queries, keys and values are slices of one row
        qkv = _normal(g, (T, (hq + 2 * hkv), d), dt)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        return {"op": op, "q": q, "k": k, "v": v, "cu": _i32(cu), "max_len": max(lens), "scale": d ** -0.5}
    if op == "decode":
        lens = [n + case["new"] for n in _lengths(case)]
        B, n, hq, hkv, d, P = case["seqs"], case["new"], case["q_heads"], case["kv_heads"], case["dim"], case["page"]
        held = [-(-x // P) for x in lens]
        pages = sum(held) + 7
        k = _normal(g, (pages, hkv, P, d), dt)
        v = _normal(g, (pages, hkv, P, d), dt)
        rng = random.Random(int(seed) * 2 + 1)
        order = list(range(pages))
        rng.shuffle(order)
        table = torch.full((B, max(held)), -1, dtype=torch.int32)
        at = 0
        for b in range(B):
            table[b, :held[b]] = torch.tensor(order[at:at + held[b]], dtype=torch.int32)
            at += held[b]
        mask = None
        if case["tree"]:
            mask = torch.tensor([_ancestors(n, rng) for _ in range(B)], dtype=torch.int64, device=DEV)
        return {"op": op, "q": _normal(g, (B, n, hq, d), dt), "k": k, "v": v, "table": table.to(DEV),
                "lengths": _i32(lens), "seqs": _i32(list(range(B))), "mask": mask, "scale": d ** -0.5,
                "max_len": max(lens)}
    if op == "pages":
        lens = _lengths(case)
        B, P, ch, new = case["seqs"], case["page"], case["children"], case["new"]
        rng = random.Random(int(seed) * 2 + 1)
        held = [-(-x // P) for x in lens]
        grown = [-(-(x + new) // P) for x in lens]
        slots = B * (1 + ch)
        # pages held, pages that a step adds, and some that others hold
        extra = sum(g_ - h + 1 for g_, h in zip(grown, held)) * max(1, ch)
        pages = sum(held) + extra + 16
        L, hkv, d = case["layers"], case["kv_heads"], case["dim"]
        k = _normal(g, (L, pages, hkv, P, d), dt)
        v = _normal(g, (L, pages, hkv, P, d), dt)
        order = list(range(pages))
        rng.shuffle(order)
        table = torch.full((slots, max(grown) + 1), -1, dtype=torch.int32)
        refs = torch.zeros(pages, dtype=torch.int32)
        at = 0
        for b in range(B):
            mine = order[at:at + held[b]]
            at += held[b]
            table[b, :held[b]] = torch.tensor(mine, dtype=torch.int32)
            refs[mine] = 1
        refs[order[at:at + 16]] = 1
        if ch:
            src = [b for b in range(B) for _ in range(ch)]
            seqs = list(range(B, slots))
        else:
            src, seqs = [], list(range(B))
        n = len(seqs)
        ctx = [0] * n if ch else lens
        keep = [sorted(rng.sample(range(new), case["keep"])) for _ in range(n)] if case["keep"] else None
        cu = [new * i for i in range(n + 1)]
        return {"op": op, "k": k, "v": v, "table": table.to(DEV), "lengths": _i32(lens + [0] * (slots - B)),
                "refs": refs.to(DEV), "seqs": _i32(seqs), "src": _i32(src) if ch else None, "ctx": _i32(ctx),
                "new": _i32([new] * n), "cu": _i32(cu), "keep": _i32(keep) if keep else None,
                "n_keep": _i32([case["keep"]] * n), "layer": L - 1,
                "k_new": _normal(g, (n * new, hkv, d), dt), "v_new": _normal(g, (n * new, hkv, d), dt)}
    rows, V = case["rows"], case["vocab"]
    # a language model's logits: a bulk, and a few tokens far above it
    logits = _normal(g, (rows, V), torch.float32, 2.0)
    peaks = torch.randint(0, V, (rows, 20), generator=g, device=DEV)
    logits.scatter_add_(1, peaks, _normal(g, (rows, 20), torch.float32, 3.0) + 6.0)
    ids = torch.randint(0, V, (rows, case["ids"]), generator=g, device=DEV, dtype=torch.int32)
    ids[:, 0] = peaks[:, 0].to(torch.int32)
    return {"op": op, "logits": logits.to(dt), "ids": ids, "k": case["k"], "temperature": case["temperature"]}


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    if own:
        return _run_own(state)
    return {"prompt": _prompt, "decode": _decode, "pages": _pages, "logprobs": _logprobs}[state["op"]](state)


def _run_own(s):
    import speculative_decoding_draft_stream_gb300 as ns

    op = s["op"]
    if op == "prompt":
        out, lse = ns.attend_prompt(s["q"], s["k"], s["v"], s["cu"], s["max_len"], scale=s["scale"])
        return {"out": out, "lse": lse}
    if op == "decode":
        out, lse = ns.attend_paged(s["q"], s["k"], s["v"], s["table"], s["lengths"], s["seqs"], mask=s["mask"],
                                   scale=s["scale"], max_len=s["max_len"])
        return {"out": out, "lse": lse}
    if op == "pages":
        cache = ns.KvPages(s["k"], s["v"], s["table"], s["lengths"], s["refs"])
        cache.truncate(s["seqs"], s["ctx"])
        if s["src"] is not None:
            cache.fork(s["src"], s["seqs"])
        cache.extend(s["seqs"], s["new"])
        cache.write(s["layer"], s["seqs"], s["cu"], s["k_new"], s["v_new"])
        if s["keep"] is not None:
            cache.compact(s["seqs"], s["ctx"], s["keep"], s["n_keep"])
        return {"k": s["k"], "v": s["v"], "table": s["table"], "lengths": s["lengths"], "refs": s["refs"]}
    r = ns.token_logprobs(s["logits"], s["ids"], s["k"], temperature=s["temperature"])
    return {"logprobs": r.logprobs, "entropy": r.entropy, "lse": r.lse, "top_ids": r.top_ids,
            "top_logprobs": r.top_logprobs}


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _softmax_parts(scores):
    """In place: exp(scores - row maximum), the row's sum and its log-sum-exp; a row of -inf gives zeros and -inf."""
    m = scores.amax(-1, keepdim=True)
    m0 = m.clamp_min(torch.finfo(scores.dtype).min)
    scores.sub_(m0).exp_()
    total = scores.sum(-1, keepdim=True)
    return scores, total, (m0 + total.log()).squeeze(-1)


def _prompt(s):
    q, k, v, cu = s["q"], s["k"], s["v"], s["cu"].long()
    T, hq, d = q.shape
    hkv, N = k.shape[1], s["max_len"]
    B, grp = cu.numel() - 1, hq // hkv
    pos = torch.arange(N, device=q.device)
    at = (cu[:-1, None] + pos).clamp_max(T - 1)
    inside = pos < (cu[1:] - cu[:-1])[:, None]
    qp = q[at].float().view(B, N, hkv, grp, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, grp * N, d)
    kp = (k[at].float() * inside[..., None, None]).permute(0, 2, 3, 1)
    vp = (v[at].float() * inside[..., None, None]).permute(0, 2, 1, 3)
    scores = (qp @ kp).mul_(s["scale"]).view(B, hkv, grp, N, N)
    scores.masked_fill_(pos[None, :] > pos[:, None], -math.inf)
    e, total, lse = _softmax_parts(scores)
    out = (e.view(B, hkv, grp * N, N) @ vp).view(B, hkv, grp, N, d) / total
    seq = torch.searchsorted(cu, torch.arange(T, device=q.device), right=True) - 1
    local = torch.arange(T, device=q.device) - cu[seq]
    return {"out": out.permute(0, 3, 1, 2, 4)[seq, local].reshape(T, hq, d).to(q.dtype),
            "lse": lse.permute(0, 3, 1, 2)[seq, local].reshape(T, hq)}


def _decode(s):
    q, k, v = s["q"], s["k"], s["v"]
    B, n, hq, d = q.shape
    hkv, P, N = k.shape[1], k.shape[2], s["max_len"]
    grp = hq // hkv
    table, lens = s["table"][s["seqs"].long()].long(), s["lengths"][s["seqs"].long()].long()
    pos = torch.arange(N, device=q.device)
    page = table[:, pos // P].clamp_min(0)
    inside = pos < lens[:, None]
    kp = k[page, :, pos % P].float() * inside[..., None, None]
    vp = v[page, :, pos % P].float() * inside[..., None, None]
    qp = q.float().view(B, n, hkv, grp, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, n * grp, d)
    scores = (qp @ kp.permute(0, 2, 3, 1)).mul_(s["scale"]).view(B, hkv, n, grp, N)
    node = pos - (lens[:, None] - n)  # a position's node, negative in the context
    rows = torch.arange(n, device=q.device)
    if s["mask"] is None:
        sees = node[:, None, :] <= rows[:, None]
    else:
        sees = (node[:, None, :] < 0) | ((s["mask"][:, :, None] >> node[:, None, :].clamp(0, 63)) & 1).bool()
    sees = sees & inside[:, None, :]
    scores.masked_fill_(~sees[:, None, :, None, :], -math.inf)
    e, total, lse = _softmax_parts(scores)
    out = (e.view(B, hkv, n * grp, N) @ vp.permute(0, 2, 1, 3)).view(B, hkv, n, grp, d)
    out = torch.where(total > 0, out / total, 0.0)
    return {"out": out.permute(0, 2, 1, 3, 4).reshape(B, n, hq, d).to(q.dtype),
            "lse": lse.permute(0, 2, 1, 3).reshape(B, n, hq)}


def _pages(s):
    k, v, table, lengths, refs = s["k"], s["v"], s["table"], s["lengths"], s["refs"]
    P, seqs, new = k.shape[3], s["seqs"].long(), s["new"].long()
    slot = torch.arange(table.shape[1], device=table.device)
    # truncate: pages past the new length lose one holder each
    _plain_truncate(table, lengths, refs, seqs, s["ctx"].long(), slot, P)
    if s["src"] is not None:  # fork: the children hold their parents' pages
        src = s["src"].long()
        rows = table[src]
        table[seqs], lengths[seqs] = rows, lengths[src]
        refs.index_add_(0, rows.clamp_min(0).flatten().long(), (rows >= 0).flatten().to(torch.int32))
    # extend: new pages lowest first, and a copy of a shared last page
    old = lengths[seqs].long()
    held, want = (old + P - 1) // P, (old + new + P - 1) // P
    last = table[seqs, (held - 1).clamp_min(0)].long()
    shared = (old % P != 0) & (new > 0) & (refs[last.clamp_min(0)] > 1)
    first = held - shared.long()
    count = want - first
    start = count.cumsum(0) - count
    free = torch.nonzero(refs == 0).flatten()
    gets = (slot >= first[:, None]) & (slot < want[:, None])
    rank = (start[:, None] + slot - first[:, None]).clamp(0, free.numel() - 1)
    table[seqs] = torch.where(gets, free[rank].to(torch.int32), table[seqs])
    refs.index_add_(0, free[rank].flatten(), gets.flatten().to(torch.int32))
    refs.index_add_(0, last.clamp_min(0), -shared.to(torch.int32))
    lengths[seqs] = (old + new).to(torch.int32)
    copies = torch.nonzero(shared).flatten()
    dst = table[seqs[copies], first[copies]].long()
    k[:, dst] = k[:, last[copies]]
    v[:, dst] = v[:, last[copies]]
    # write the new rows of one layer
    tok = torch.arange(s["k_new"].shape[0], device=table.device)
    cu = s["cu"].long()
    i = torch.searchsorted(cu, tok, right=True) - 1
    at = lengths[seqs][i].long() - (cu[1:] - cu[:-1])[i] + tok - cu[i]
    page = table[seqs[i], at // P].long()
    k[s["layer"]][page, :, at % P] = s["k_new"]
    v[s["layer"]][page, :, at % P] = s["v_new"]
    if s["keep"] is not None:  # compact: kept rows move down in every layer, surplus pages go
        base = s["ctx"].long()[:, None]
        to = base + torch.arange(s["keep"].shape[1], device=table.device)
        frm = base + s["keep"].long()
        rows = table[seqs].long()
        p1, p0 = rows.gather(1, to // P), rows.gather(1, frm // P)
        k[:, p1, :, to % P] = k[:, p0, :, frm % P]
        v[:, p1, :, to % P] = v[:, p0, :, frm % P]
        _plain_truncate(table, lengths, refs, seqs, s["ctx"].long() + s["n_keep"].long(), slot, P)
    return {"k": k, "v": v, "table": table, "lengths": lengths, "refs": refs}


def _plain_truncate(table, lengths, refs, seqs, upto, slot, P):
    rows = table[seqs]
    drop = (slot >= ((upto + P - 1) // P)[:, None]) & (rows >= 0)
    refs.index_add_(0, rows.clamp_min(0).flatten().long(), -drop.flatten().to(torch.int32))
    table[seqs] = torch.where(drop, -1, rows)
    lengths[seqs] = torch.minimum(lengths[seqs], upto.to(torch.int32))


def _logprobs(s):
    x = s["logits"].float()
    V, k = x.shape[1], s["k"]
    z = x / s["temperature"]
    m = z.amax(-1, keepdim=True)
    d = z - m
    e = d.exp()
    total = e.sum(-1, keepdim=True)
    log_total = total.log()
    lp = d.gather(1, s["ids"].long()) - log_total
    entropy = log_total.squeeze(1) - (e * d).sum(-1) / total.squeeze(1)
    # order by value, then by the lower id: an ordered integer of the value above the id
    bits = (x + 0.0).view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    key = key * (1 << 32) + (V - 1 - torch.arange(V, device=x.device))
    top = key.topk(k, dim=-1).values
    ids = V - 1 - (top & 0xFFFFFFFF)
    return {"logprobs": lp, "entropy": entropy, "lse": (m + log_total).squeeze(1), "top_ids": ids.to(torch.int32),
            "top_logprobs": d.gather(1, ids) - log_total}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    size = 4 if case["dtype"] == "f32" else 2
    if op == "prompt":
        lens, hq, hkv, d = _lengths(case), case["q_heads"], case["kv_heads"], case["dim"]
        pairs = sum(n * (n + 1) // 2 for n in lens)
        return {"bytes": sum(lens) * (d * size * 2 * (hq + hkv) + 4 * hq), "flops": 4 * pairs * hq * d}
    if op == "decode":
        n, hq, hkv, d = case["new"], case["q_heads"], case["kv_heads"], case["dim"]
        lens = [x + n for x in _lengths(case)]
        return {"bytes": sum(lens) * hkv * d * size * 2 + len(lens) * n * hq * (2 * d * size + 4),
                "flops": 4 * sum(lens) * n * hq * d}
    if op == "pages":
        lens, P, ch, new = _lengths(case), case["page"], case["children"], case["new"]
        row = case["kv_heads"] * case["dim"] * size * 2  # one token of one layer, keys and values
        n = len(lens) * max(1, ch)
        moved = n * new * row * 2  # the new rows of one layer, read and written
        if ch:
            moved += sum(ch for x in lens if x % P) * P * row * case["layers"] * 2
        moved += n * case["keep"] * row * case["layers"] * 2
        return {"bytes": moved + 4 * sum(-(-(x + new) // P) for x in lens) * max(1, ch), "flops": 0}
    return {"bytes": case["rows"] * (case["vocab"] * size + 8 * (case["ids"] + case["k"] + 1)),
            "flops": 4 * case["rows"] * case["vocab"]}


# ---------------------------------------------------------------------------
# From the definition, in 64 bits
# ---------------------------------------------------------------------------
def _attend64(q, k, v, sees, scale):
    """q [m, d], k and v [n, d], sees [m, n]: the output and log-sum-exp of every row."""
    z = torch.where(sees, (q.double() @ k.double().T) * scale, -math.inf)
    lse = torch.logsumexp(z, -1)
    p = torch.exp(z - torch.where(torch.isinf(lse), 0.0, lse)[:, None])
    return p @ v.double(), lse


def exact(case, seed):
    if case["op"] == "pages":
        return None  # whole numbers, and values that are moved but not computed
    s = prepare(case, seed)
    if case["op"] == "prompt":
        q, k, v, cu = s["q"], s["k"], s["v"], s["cu"].tolist()
        hq, grp = q.shape[1], q.shape[1] // k.shape[1]
        out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
        lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=DEV)
        for a, b in zip(cu[:-1], cu[1:]):
            for r0 in range(a, b, 4096):  # rows by blocks: a block sees nothing past its own end
                r1 = min(b, r0 + 4096)
                sees = torch.arange(a, r1, device=DEV) <= torch.arange(r0, r1, device=DEV)[:, None]
                for h in range(hq):
                    out[r0:r1, h], lse[r0:r1, h] = _attend64(q[r0:r1, h], k[a:r1, h // grp], v[a:r1, h // grp], sees,
                                                            s["scale"])
        return {"out": out, "lse": lse}
    if case["op"] == "decode":
        q, P = s["q"], s["k"].shape[2]
        B, n, hq, d = q.shape
        hkv = s["k"].shape[1]
        grp = hq // hkv
        out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
        lse = torch.zeros(q.shape[:3], dtype=torch.float64, device=DEV)
        for b in range(B):
            N = int(s["lengths"][b])
            pages = s["table"][b, :-(-N // P)].long()
            keys = s["k"][pages].transpose(1, 2).reshape(-1, hkv, d)[:N]
            vals = s["v"][pages].transpose(1, 2).reshape(-1, hkv, d)[:N]
            sees = torch.ones((n, N), dtype=torch.bool, device=DEV)
            for i in range(n):
                word = (1 << (i + 1)) - 1 if s["mask"] is None else int(s["mask"][b, i])
                sees[i, N - n:] = torch.tensor([bool(word >> j & 1) for j in range(n)], device=DEV)
            for h in range(hkv):
                o, z = _attend64(q[b, :, h * grp:(h + 1) * grp].reshape(n * grp, d), keys[:, h], vals[:, h],
                                 sees.repeat_interleave(grp, 0), s["scale"])
                out[b, :, h * grp:(h + 1) * grp] = o.view(n, grp, d)
                lse[b, :, h * grp:(h + 1) * grp] = z.view(n, grp)
        return {"out": out, "lse": lse}
    parts = []
    for r0 in range(0, case["rows"], 128):
        z = s["logits"][r0:r0 + 128].double() / s["temperature"]
        lp = torch.log_softmax(z, -1)
        by_value = torch.sort(s["logits"][r0:r0 + 128].float() + 0.0, dim=-1, descending=True, stable=True).indices
        ids = by_value[:, :case["k"]]
        parts.append((lp.gather(1, s["ids"][r0:r0 + 128].long()), -(lp.exp() * lp).sum(-1), torch.logsumexp(z, -1),
                      ids.to(torch.int32), lp.gather(1, ids)))
    names = ("logprobs", "entropy", "lse", "top_ids", "top_logprobs")
    return {name: torch.cat([p[i] for p in parts]) for i, name in enumerate(names)}
