"""Speculative decoding with the draft head and the serving operators, end to end.

A small randomly initialised transformer (no checkpoint is needed) answers
prompts with several continuations each:

1. prefill: ``attend_prompt`` over all prompts, their keys and values into a
   ``KvPages`` cache; ``token_logprobs`` scores the prompts and gives each
   continuation its first token; ``KvPages.fork`` shares a prompt's pages
   among its continuations;
2. draft: ``Handle.step`` proposes tokens from the dynamic vocabulary, two
   levels deep, a tree under the token that is already chosen;
3. verify: the tree's nodes are appended to the cache (``extend``, ``write``),
   ``KvPages.attend`` lets each node see the context and its ancestors, and
   ``token_logprobs`` names the verifier's choice after each node;
4. accept: the path of nodes that the verifier agrees with is kept
   (``compact``), the rest is dropped, and the stream of candidates grows.

    python -m speculative_decoding_draft_stream_gb300.speculate
"""

from __future__ import annotations

import argparse
from typing import List, NamedTuple, Optional, Tuple

import torch

from .nanospec import Handle
from .serving import KvPages, attend_prompt, ops_error, token_logprobs


class Verifier:
    """Attention layers with a residual stream, learned positions and an output head, in bf16."""

    def __init__(self, V=512, H=256, layers=2, q_heads=4, kv_heads=2, dim=64, positions=1024, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)

        def weight(rows, cols, size):
            return (torch.randn(rows, cols, generator=g) * size).to(torch.bfloat16).to(device)

        self.V, self.H, self.layers, self.q_heads, self.kv_heads, self.dim = V, H, layers, q_heads, kv_heads, dim
        self.emb, self.pos = weight(V, H, 1.0), weight(positions, H, 0.1)
        self.head = weight(V, H, H ** -0.5)
        width = (q_heads + 2 * kv_heads) * dim
        self.qkv = [weight(width, H, 1.5 * H ** -0.5) for _ in range(layers)]
        self.out = [weight(H, q_heads * dim, 0.5 * (q_heads * dim) ** -0.5) for _ in range(layers)]

    @staticmethod
    def norm(x):
        return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-5)).to(torch.bfloat16)

    def forward(self, ids, positions, attend):
        """Final hidden states [T, H] and logits fp32 [T, V]; attend(layer, q, k, v) gives [T, q_heads, dim]."""
        x = self.emb[ids.long()] + self.pos[positions.long()]
        for layer in range(self.layers):
            y = (self.norm(x) @ self.qkv[layer].T).view(len(ids), -1, self.dim)
            q, k, v = y.split([self.q_heads, self.kv_heads, self.kv_heads], 1)
            x = x + attend(layer, q, k, v).reshape(len(ids), -1) @ self.out[layer].T
        h = self.norm(x)
        return h, (h @ self.head.T).float()


class Answer(NamedTuple):
    tokens: List[int]         # the continuation
    logprobs: List[float]     # of its tokens, under the verifier
    accepted: List[int]       # draft tokens accepted by each step


def generate(model: Verifier, prompts: List[List[int]], samples: int = 2, tokens: int = 32, width: int = 4,
             width2: int = 2, page_size: int = 16, window: int = 1024) -> Tuple[List[Answer], List[Optional[float]]]:
    """`samples` continuations of each prompt, at least `tokens` long, and the prompts' mean log probabilities (None
    for a prompt of one token, which has none to be scored).

    A step's tree: the chosen token, `width` proposals for the next one, `width2` for the one after each."""
    dev = model.head.device
    i32 = {"dtype": torch.int32, "device": dev}
    n_prompts, B = len(prompts), len(prompts) * samples
    n = 1 + width + width * width2  # nodes of a tree, parents before children
    longest = max(map(len, prompts)) + 3 * tokens + n  # a step takes up to three of them
    if longest > len(model.pos):
        raise ValueError(f"{longest} positions wanted, the model has {len(model.pos)}")
    per_seq = -(-longest // page_size)
    pages = KvPages.new(model.layers, per_seq * (B + n_prompts), model.kv_heads, page_size, model.dim, B + n_prompts,
                        per_seq, device=dev)

    # Prefill: sequences 0 .. n_prompts - 1 of the cache hold the prompts.
    ids = torch.tensor(sum(prompts, []), **i32)
    lens = torch.tensor([len(p) for p in prompts], **i32)
    cu = torch.cat([torch.zeros(1, **i32), lens.cumsum(0).int()])
    at = torch.cat([torch.arange(len(p), **i32) for p in prompts])
    own = torch.arange(n_prompts, **i32)
    pages.extend(own, lens)

    def prefill(layer, q, k, v):
        pages.write(layer, own, cu, k, v)
        return attend_prompt(q, k, v, cu, max(map(len, prompts)))[0]

    hidden, logits = model.forward(ids, at, prefill)
    following = torch.cat([ids[1:], ids[:1]])
    following[cu[1:].long() - 1] = -1  # the last token of a prompt has none
    scored = token_logprobs(logits, following[:, None], k=samples)
    prompt_scores = [float(scored.logprobs[a:b - 1, 0].mean()) if b - a > 1 else None
                     for a, b in zip(cu.tolist(), cu.tolist()[1:])]

    # Continuations: sequence n_prompts + i shares the pages of prompt i / samples.
    seqs = torch.arange(n_prompts, n_prompts + B, **i32)
    for s in range(samples):
        pages.fork(own, seqs[s::samples].contiguous())
    last = (cu[1:].long() - 1).repeat_interleave(samples)
    which = torch.arange(samples, device=dev).repeat(n_prompts)
    chosen = scored.top_ids[last, which].tolist()
    first_logprobs = scored.top_logprobs[last, which].tolist()
    answers = [Answer([t], [p], []) for t, p in zip(chosen, first_logprobs)]
    tip = hidden[last]  # the hidden state that each chosen token was read from
    length = [len(prompts[i // samples]) for i in range(B)]

    parent = [-1] + [0] * width + [1 + i // width2 for i in range(width * width2)]
    depth = [0] + [1] * width + [2] * (width * width2)
    bits = []
    for i in range(n):
        bits.append((bits[parent[i]] if i else 0) | 1 << i)
    mask = torch.tensor([bits] * B, dtype=torch.int64, device=dev)
    depths = torch.tensor(depth, **i32)
    tree_cu = torch.arange(0, (B + 1) * n, n, **i32)
    grow = torch.full((B,), n, **i32)

    with Handle(model.V, model.H, window, max_tree=n, max_k=max(width, width2), batch=B,
                max_prompt=max(map(len, prompts))) as heads:
        for b in range(B):
            a, z = cu[b // samples], cu[b // samples + 1]
            heads.stream_init(b, ids[a:z].contiguous(), logits[a:z].contiguous())
        # what the last verification saw: no tree yet, and the prompt's last row
        trees = [None] * B
        verified, rows = [logits[i:i + 1].contiguous() for i in last.tolist()], [0] * B
        while min(len(x.tokens) for x in answers) < tokens:
            # Draft: proposals after the chosen token, then after each of them.
            nodes = torch.empty(B, n, **i32)
            nodes[:, 0] = torch.tensor(chosen, **i32)
            state = model.norm(0.3 * tip.float() + model.emb[nodes[:, 0].long()].float())
            for b in range(B):
                one, _ = heads.step(b, trees[b], verified[b], rows[b], model.head, state[b:b + 1].contiguous(), width)
                nodes[b, 1:1 + width] = one[0]
                two_in = model.norm(0.3 * state[b].float() + model.emb[one[0].clamp(min=0).long()].float())
                two, _ = heads.sub_lm_head_logits_topk(b, two_in.contiguous(), width2)
                nodes[b, 1 + width:] = two.reshape(-1)
            nodes.clamp_(min=0)

            # Verify: all trees at once, behind their contexts.
            pages.extend(seqs, grow)
            base = torch.tensor(length, **i32)

            def verify(layer, q, k, v):
                pages.write(layer, seqs, tree_cu, k, v)
                o, _ = pages.attend(layer, q.unflatten(0, (B, n)), seqs, mask=mask, max_len=max(length) + n)
                return o.flatten(0, 1)

            hidden, logits = model.forward(nodes.reshape(-1), (base[:, None] + depths).reshape(-1), verify)
            best = token_logprobs(logits, k=1)
            pick, how = best.top_ids.view(B, n).tolist(), best.top_logprobs.view(B, n).tolist()
            drafted = nodes.tolist()

            # Accept: from the root down, the child that holds the verifier's choice.
            keep = torch.zeros(B, 3, **i32)
            path_len = []
            for b in range(B):
                path = [0]
                while True:
                    want = pick[b][path[-1]]
                    step = [i for i in range(n) if parent[i] == path[-1] and drafted[b][i] == want]
                    answers[b].tokens.append(want)
                    answers[b].logprobs.append(how[b][path[-1]])
                    if not step:
                        break
                    path.append(step[0])
                answers[b].accepted.append(len(path) - 1)
                chosen[b], rows[b] = answers[b].tokens[-1], path[-1]
                keep[b, :len(path)] = torch.tensor(path, **i32)
                path_len.append(len(path))
                trees[b], verified[b] = nodes[b].contiguous(), logits[b * n:(b + 1) * n]
                length[b] += len(path)
            tip = hidden.view(B, n, -1)[torch.arange(B, device=dev), torch.tensor(rows, device=dev)]
            pages.compact(seqs, base, keep, torch.tensor(path_len, **i32))
        flags = heads.get_error()
    flags |= ops_error()
    if flags:
        raise RuntimeError(f"device flags {flags:#x}")
    return answers, prompt_scores


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--samples", type=int, default=2)
    ap.add_argument("--tokens", type=int, default=32)
    args = ap.parse_args()
    g = torch.Generator().manual_seed(1)
    model = Verifier()
    prompts = [torch.randint(model.V, (n,), generator=g).tolist() for n in (5, 64, 131)]
    answers, scores = generate(model, prompts, args.samples, args.tokens)
    for i, a in enumerate(answers):
        score = scores[i // args.samples]
        said = "one token" if score is None else f"mean log probability {score:.2f}"
        print(f"prompt {i // args.samples} ({said}), answer {i % args.samples}: "
              f"{len(a.tokens)} tokens in {len(a.accepted)} steps, mean log probability "
              f"{sum(a.logprobs) / len(a.logprobs):.2f}: {a.tokens[:12]} ...")


if __name__ == "__main__":
    main()
