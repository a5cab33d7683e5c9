"""The serving operators have no gradients: calls that would have to record one are refused."""

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
    """Each call as a function of its floating tensors, and those."""
    i32 = {"dtype": torch.int32, "device": "cuda"}

    def f16(*shape):
        return torch.zeros(shape, dtype=BF16, device="cuda")

    cu, one = torch.tensor([0, 10], **i32), torch.tensor([0], **i32)
    table, lengths = torch.tensor([[0, 1]], **i32), torch.tensor([12], **i32)

    def write(k, v, k_new, v_new):
        c = ns.KvPages(k, v, table.clone(), lengths.clone(), torch.ones(4, **i32))
        c.write(0, one, cu, k_new, v_new)

    return {
        "prompt": (lambda q, k, v: ns.attend_prompt(q, k, v, cu, 10), [f16(10, 4, 64), f16(10, 2, 64), f16(10, 2, 64)]),
        "prompt out": (lambda o, z: ns.attend_prompt(f16(10, 4, 64), f16(10, 2, 64), f16(10, 2, 64), cu, 10, out=o, lse=z),
                       [f16(10, 4, 64), torch.zeros(10, 4, device="cuda")]),
        "paged": (lambda q, k, v: ns.attend_paged(q, k, v, table, lengths, one),
                  [f16(1, 1, 4, 64), f16(4, 2, 16, 64), f16(4, 2, 16, 64)]),
        "write": (write, [f16(1, 4, 2, 16, 64), f16(1, 4, 2, 16, 64), f16(10, 2, 64), f16(10, 2, 64)]),
        "log probabilities": (lambda x: ns.token_logprobs(x, None, 2), [torch.zeros(3, 50, device="cuda")]),
    }


@pytest.mark.parametrize("what", ["prompt", "prompt out", "paged", "write", "log probabilities"])
def test_tensors_that_require_gradients_are_refused(ns, what):
    call, tensors = calls(ns)[what]
    call(*tensors)
    for t in tensors:
        t.requires_grad_(True)
        with pytest.raises(ValueError, match="gradient"):
            call(*tensors)
        with torch.no_grad():
            call(*tensors)
        with torch.inference_mode():
            call(*tensors)
        call(*[x.detach() for x in tensors])
        t.requires_grad_(False)
    assert ns.ops_error() == 0
