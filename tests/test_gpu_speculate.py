"""The speculative decoding example: its answers are what the model says one token at a time."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def plain(model, text):
    """Logits of every position of one text: the model in fp32 with plain attention (weights as they are)."""
    dev = model.head.device
    n, g = len(text), model.q_heads // model.kv_heads

    def norm(x):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5)

    ids = torch.tensor(text, device=dev)
    x = model.emb[ids].double() + model.pos[:n].double()
    sees = torch.ones(n, n, dtype=torch.bool, device=dev).tril()
    for layer in range(model.layers):
        y = (norm(x) @ model.qkv[layer].double().T).view(n, -1, model.dim)
        q, k, v = y.split([model.q_heads, model.kv_heads, model.kv_heads], 1)
        k, v = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
        s = torch.einsum("ihd,jhd->hij", q, k) * model.dim ** -0.5
        o = torch.einsum("hij,jhd->ihd", s.masked_fill(~sees, float("-inf")).softmax(-1), v)
        x = x + o.reshape(n, -1) @ model.out[layer].double().T
    return norm(x) @ model.head.double().T


@pytest.mark.parametrize("samples,page", [(1, 16), (3, 8)])
def test_answers_are_the_verifiers_choices(samples, page):
    from speculative_decoding_draft_stream_gb300.speculate import Verifier, generate

    g = torch.Generator().manual_seed(7)
    model = Verifier()
    prompts = [torch.randint(model.V, (n,), generator=g).tolist() for n in (1 if samples == 1 else 2, 33, 100)]
    if samples == 1:
        prompts = prompts[1:]
    answers, scores = generate(model, prompts, samples, tokens=24, page_size=page)
    # Logits are sums of 256 products of bf16 hidden states near 1 and weights near 1/16: about N(0, 1).  Each of the
    # half dozen roundings of the residual path moves them by a few of bf16's 2^-8 of that; 0.15 is 40 of them.
    tol = 0.15
    assert max(max(a.accepted) for a in answers) == 2  # whole paths of a tree are kept, and nothing of one
    assert min(min(a.accepted) for a in answers) == 0
    for i, a in enumerate(answers):
        prompt = prompts[i // samples]
        assert len(a.tokens) >= 24 and len(a.tokens) == 1 + sum(a.accepted) + len(a.accepted)
        z = plain(model, prompt + a.tokens)
        logp = z.log_softmax(-1)
        at = torch.arange(len(prompt) - 1, len(prompt) - 1 + len(a.tokens), device=z.device)
        ids = torch.tensor(a.tokens, device=z.device)
        mine = z[at].gather(1, ids[:, None])[:, 0]
        best = z[at].max(1).values
        assert bool((best[1:] - mine[1:] <= 2 * tol).all())  # greedy, within the two logits' errors
        order = z[at[0]].topk(samples).values
        assert abs(float(mine[0] - order[i % samples])) <= 2 * tol  # the i-th best first token
        got = torch.tensor(a.logprobs, device=z.device, dtype=torch.float64)
        want = logp[at].gather(1, ids[:, None])[:, 0]
        assert bool(((got - want).abs() <= 2 * tol).all())
    for p, s in zip(prompts, scores):
        lp = plain(model, p).log_softmax(-1)
        want = lp[torch.arange(len(p) - 1), torch.tensor(p[1:])].mean()
        assert abs(float(want) - s) <= 2 * tol
    if samples > 1:  # continuations of one prompt begin differently
        for j in range(0, len(answers), samples):
            assert len({answers[j + s].tokens[0] for s in range(samples)}) == samples


@pytest.mark.parametrize("samples", [1, 2])
def test_a_prompt_of_one_token(samples):
    """It is continued like any other; there is nothing in it to score."""
    from speculative_decoding_draft_stream_gb300.speculate import Verifier, generate

    model = Verifier()
    prompts = [[17], [3, 400, 5], [501]]
    answers, scores = generate(model, prompts, samples, tokens=12)
    assert scores[0] is None and scores[2] is None and scores[1] < 0
    tol = 0.15  # (as above)
    for i, a in enumerate(answers):
        prompt = prompts[i // samples]
        z = plain(model, prompt + a.tokens)
        at = torch.arange(len(prompt) - 1, len(prompt) - 1 + len(a.tokens), device=z.device)
        mine = z[at].gather(1, torch.tensor(a.tokens, device=z.device)[:, None])[:, 0]
        assert len(a.tokens) >= 12 and bool((z[at].max(1).values[1:] - mine[1:] <= 2 * tol).all())
        order = z[at[0]].topk(samples).values
        assert abs(float(mine[0] - order[i % samples])) <= 2 * tol
        want = z.log_softmax(-1)[at].gather(1, torch.tensor(a.tokens, device=z.device)[:, None])[:, 0]
        assert bool(((torch.tensor(a.logprobs, device=z.device, dtype=torch.float64) - want).abs() <= 2 * tol).all())


def test_the_command_answers(capsys, monkeypatch):
    from speculative_decoding_draft_stream_gb300 import speculate

    monkeypatch.setattr("sys.argv", ["speculate", "--samples", "1", "--tokens", "6"])
    speculate.main()
    assert capsys.readouterr().out.count("mean log probability") == 6
