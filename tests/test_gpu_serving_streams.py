"""The serving operators on a stream of the caller's choice: what they allocate belongs to that stream."""

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


def calls(ns):
    """Each call that allocates: a function of the stream, which gives its results, and their sizes in bytes."""
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(BF16)

    i32 = {"dtype": torch.int32, "device": "cuda"}
    q, k, v = normal(300, 8, 64), normal(300, 2, 64), normal(300, 2, 64)
    cu = torch.tensor([0, 100, 300], **i32)
    pool_k, pool_v = normal(64, 2, 16, 64), normal(64, 2, 16, 64)
    table = torch.arange(64, **i32).view(2, 32)
    lengths, seqs = torch.tensor([500, 333], **i32), torch.tensor([0, 1], **i32)
    few, many = normal(2, 1, 8, 64), normal(2, 40, 8, 64)
    logits = normal(40, 5000).float()
    ids = torch.randint(0, 5000, (40, 3), generator=g, **i32)
    big_k, big_v = normal(1, 3000, 1, 8, 8), normal(1, 3000, 1, 8, 8)
    grow = torch.tensor([8 * 1400, 8 * 1300], **i32)

    caches = [ns.KvPages(big_k, big_v, torch.full((2, 1500), -1, **i32), torch.zeros(2, **i32), torch.zeros(3000, **i32))
              for _ in range(4)]

    def extended(stream):
        c = caches.pop()
        c.extend(seqs, grow, stream=stream)
        return c.table, c.lengths, c.refs

    need = ns.load_library().ns_attend_paged_workspace
    return {
        "prompt": (lambda s: ns.attend_prompt(q, k, v, cu, 200, stream=s), [300 * 8 * 64 * 2, 300 * 8 * 4]),
        "one token": (lambda s: ns.attend_paged(few, pool_k, pool_v, table, lengths, seqs, stream=s),
                      [2 * 8 * 64 * 2, 2 * 8 * 4, need(2, 1, 8, 2, 64)]),
        "many rows": (lambda s: ns.attend_paged(many, pool_k, pool_v, table, lengths, seqs, stream=s),
                      [2 * 40 * 8 * 64 * 2, 2 * 40 * 8 * 4, need(2, 40, 8, 2, 64)]),
        "log probabilities": (lambda s: ns.token_logprobs(logits, ids, 5, stream=s), [40 * 3 * 4, 40 * 4, 40 * 5 * 4]),
        "extend": (extended, [4 * (4 + 6 * 2 + 3000)]),
    }


@pytest.mark.parametrize("what", ["prompt", "one token", "many rows", "log probabilities", "extend"])
def test_memory_that_the_current_stream_still_uses_is_not_taken(ns, what):
    """Blocks freed on the current stream while work that reads them is still queued there, then a call on another
    stream that nothing orders behind that work: its outputs and workspace must not be those blocks."""
    call, sizes = calls(ns)[what]
    s = torch.cuda.Stream()
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    for _ in range(3):
        held = [torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
        torch.cuda._sleep(100_000_000)  # some 50 ms
        seen = [t.clone() for t in held]  # queued behind the sleep
        del held
        got = call(s)
        torch.cuda.synchronize()
        assert all(bool((t == 0x7f).all()) for t in seen), "memory was written that queued work still had to read"
        assert all(torch.equal(x, y) for x, y in zip(want, got))
    assert ns.ops_error() == 0


def test_results_of_another_stream_outlive_their_tensors(ns):
    """Results that the caller's stream still reads when their tensors are gone are not written over by the next call
    on the other stream."""
    call, _ = calls(ns)["prompt"]
    want = call(None)[0].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = call(s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(100_000_000)
    kept = out.clone()  # queued behind the sleep
    del out, lse
    with torch.cuda.stream(s):
        over = [torch.full((300, 8, 64), 7.0, dtype=BF16, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(kept, want) and len(over) == 4


def test_given_outputs_and_workspace_are_used_as_they_are(ns):
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k, v = (torch.randn(100, 4, 64, generator=g, device="cuda").to(BF16) for _ in range(3))
    cu = torch.tensor([0, 100], dtype=torch.int32, device="cuda")
    want, wl = ns.attend_prompt(q, k, v, cu, 100)
    out, lse = torch.empty_like(want), torch.empty_like(wl)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (s, s.cuda_stream):  # a torch stream, or its handle
        out.zero_()
        s.wait_stream(torch.cuda.current_stream())
        a, b = ns.attend_prompt(q, k, v, cu, 100, out=out, lse=lse, stream=stream)
        s.synchronize()
        assert a is out and b is lse and torch.equal(out, want) and torch.equal(lse, wl)
    assert isinstance(ns.token_logprobs(torch.zeros(2, 9, device="cuda"), stream=s), ns.TokenLogprobs)
