"""The example with rotated heads, a cache of 8 bits and shared prompts: its answers are what the model says one token at
a time, over the keys and values that the cache holds."""

import pytest
import torch

from serving8_ref import quantise, values

pytestmark = pytest.mark.gpu


def plain(model, text, prompt, scaled):
    """Logits of every position of one text in 64 bits (weights as they are); with scaled, the positions behind the prompt
    see keys and values as 8 bits hold them."""
    dev = model.head.device
    n, g, h = len(text), model.q_heads // model.kv_heads, model.dim // 2

    def norm(x):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5)

    def rotate(x, weight):
        x = norm(x) * weight.double()
        t = torch.arange(n, device=dev).double()[:, None, None] * model.inv_freq
        a, b = x[..., :h], x[..., h:]
        return torch.cat((a * t.cos() - b * t.sin(), b * t.cos() + a * t.sin()), -1)

    def held(x):
        return values(*quantise(x.to(torch.bfloat16).cpu())).to(dev)

    ids = torch.tensor(text, device=dev)
    x = model.emb[ids].double() + model.pos[:n].double()
    sees = torch.ones(n, n, dtype=torch.bool, device=dev).tril()
    for layer in range(model.layers):
        y = (norm(x) @ model.qkv[layer].double().T).view(n, -1, model.dim)
        q, k, v = y.split([model.q_heads, model.kv_heads, model.kv_heads], 1)
        if model.inv_freq is not None:
            q, k = rotate(q, model.norms[layer][0]), rotate(k, model.norms[layer][1])
        o = []
        for kk, vv in ((k, v), (held(k), held(v)) if scaled else (k, v)):
            s = torch.einsum("ihd,jhd->hij", q, kk.repeat_interleave(g, 1)) * model.dim ** -0.5
            o.append(torch.einsum("hij,jhd->ihd", s.masked_fill(~sees, float("-inf")).softmax(-1),
                                  vv.repeat_interleave(g, 1)))
        o = torch.cat((o[0][:prompt], o[1][prompt:]))
        x = x + o.reshape(n, -1) @ model.out[layer].double().T
    return norm(x) @ model.head.double().T


@pytest.mark.parametrize("rotary,scaled,shared,samples", [
    (True, False, False, 1), (False, True, False, 1), (False, False, True, 3), (True, True, True, 3),
])
def test_answers_are_the_verifiers_choices(rotary, scaled, shared, samples):
    from speculative_decoding_draft_stream_gb300.speculate import Verifier, generate

    g = torch.Generator().manual_seed(9)
    model = Verifier(rotary=rotary)
    prompts = [torch.randint(model.V, (n,), generator=g).tolist() for n in (33, 300)]
    answers, scores = generate(model, prompts, samples, tokens=16, scaled=scaled, shared=shared)
    # As in test_gpu_speculate: logits near N(0, 1), each rounding off by a few of bf16's 2^-8 of that.  A key or value
    # that rounds to another code than here, from another last bit of bf16, is off by a sixteenth in one column of one
    # position.
    tol = 0.15
    assert max(max(a.accepted) for a in answers) == 2
    for i, a in enumerate(answers):
        prompt = prompts[i // samples]
        assert len(a.tokens) >= 16 and len(a.tokens) == 1 + sum(a.accepted) + len(a.accepted)
        z = plain(model, prompt + a.tokens, len(prompt), scaled)
        at = torch.arange(len(prompt) - 1, len(prompt) - 1 + len(a.tokens), device=z.device)
        ids = torch.tensor(a.tokens, device=z.device)
        mine = z[at].gather(1, ids[:, None])[:, 0]
        assert bool((z[at].max(1).values[1:] - mine[1:] <= 2 * tol).all())  # greedy, within the two logits' errors
        got = torch.tensor(a.logprobs, device=z.device, dtype=torch.float64)
        assert bool(((got - z.log_softmax(-1)[at].gather(1, ids[:, None])[:, 0]).abs() <= 2 * tol).all())
    for p, s in zip(prompts, scores):
        lp = plain(model, p, len(p), False).log_softmax(-1)
        assert abs(float(lp[torch.arange(len(p) - 1), torch.tensor(p[1:])].mean()) - s) <= 2 * tol


def test_the_command_answers(capsys, monkeypatch):
    from speculative_decoding_draft_stream_gb300 import speculate

    monkeypatch.setattr("sys.argv", ["speculate", "--samples", "2", "--tokens", "6", "--rotary", "--scaled", "--shared"])
    speculate.main()
    assert capsys.readouterr().out.count("mean log probability") == 12
