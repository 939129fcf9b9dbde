"""Gradients of the operators that autograd records (create_graph=True): the
bytes of the ordinary ones, and an error where they are differentiated."""
import pytest
import torch

from context_attention_long_b200 import autograd, build

from test_gpu_cross import lens_of, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()


@pytest.mark.parametrize("op", ["cross", "norm"])
def test_recorded_gradients(op):
    q, k, v = normal(2, 33, 4, 64, seed=1), normal(2, 33, 2, 64, seed=2), normal(2, 33, 2, 64, seed=3)
    w = torch.linspace(0.5, 1.5, 64, device="cuda")
    g = normal(2, 33, 4, 64, seed=4)
    leaves = [t.requires_grad_() for t in ((q, k, v) if op == "cross" else (q, w))]

    def out():
        return autograd.cross_attention(q, k, v, lens_of([33, 8])) if op == "cross" else autograd.qk_norm_rope(q, None, w)[0]
    want = torch.autograd.grad(out(), leaves, g)
    y = out()
    got = torch.autograd.grad(y, leaves, g, create_graph=True)
    for a, b in zip(got, want):
        assert torch.equal(a, b) and a.requires_grad and not b.requires_grad
    with pytest.raises(RuntimeError, match="not offered"):
        (y.float().sum() + got[0].float().square().sum()).backward()
