"""norm_rotate has no gradient: whichever of its floating tensors requires one, the call is refused."""

import pytest
import torch

from test_gpu_rotate import BF16, freqs, ns  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", ["q", "k", "inv_freq", "q_weight", "k_weight", "q_out", "k_out"])
def test_tensors_that_require_gradients_are_refused(ns, which):  # noqa: F811
    def heads(n):
        return torch.ones(4, n, 64, dtype=BF16, device="cuda")

    a = {"q": heads(4), "k": heads(2), "inv_freq": freqs(64), "q_weight": torch.ones(64, dtype=BF16, device="cuda"),
         "k_weight": torch.ones(64, dtype=BF16, device="cuda"), "q_out": heads(4), "k_out": heads(2)}
    pos = torch.arange(4, dtype=torch.int32, device="cuda")

    def call(**kw):
        x = dict(a, **kw)
        return ns.norm_rotate(x.pop("q"), x.pop("k"), pos, x.pop("inv_freq"), eps=1e-6, **x)

    want = [t.clone() for t in call()]
    t = a[which].requires_grad_(True)
    with pytest.raises(ValueError, match=f"{which} requires a gradient"):
        call()
    with torch.no_grad():
        got = call()
    for x, y in ((got, want), (call(**{which: t.detach()}), want)):
        assert all(torch.equal(p, q) for p, q in zip(x, y))
    assert ns.ops_error() == 0
