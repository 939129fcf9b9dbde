"""The gradient of cross attention in the 2-norm, at few states above all,
against the float64 definition.

Tolerances, for independent normal draws.  A gradient carries two independent
roundings to bf16: of dS (P for dV), the product's operand, and of the result.
A rounding is evenly spread up to half a step, 2^-8 of the value's power of two:
2^-8 / sqrt(3) of that in the mean square, and the values spread over the powers
of two (mean square of value over power 2.2, at least 1.5 taken): 0.47 * 2^-8 of
the norm each, 0.67 * 2^-8 both.  Above 32 states Delta takes the saved output,
which adds the roundings of P and its own on a value of 1 / sqrt(n) of dP, at
most 0.67 / sqrt(33) * 2^-8; up to 32 it does not.  Float32 arithmetic is off by
2^-18 (1 + reach) of P (|dP| + |Delta|) at most, reach being some 10 and dS a
third of that or more: 2^-13.  Together below 0.75 * 2^-8; with fewer than 1000
rows the mean squares scatter: 2^-8.  With one state dQ and dK are zero, and
float32 errors are all they hold: 2^-15 (1 + reach) of the magnitudes added.
"""
import numpy as np
import pytest
import torch

from context_attention_long_b200 import api, autograd, build
from oracle import cross

from gpu_util import f64_of
from test_gpu_cross import check_forward, lens_of, normal
from test_gpu_cross_backward import check_backward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()


def check_norms(q, k, v, dout, lens, grads):
    """Per batch element: none may hide behind another's gradient."""
    arrays = [f64_of(t) for t in (q, k, v, dout)]
    for b in range(q.shape[0]):
        one = [a[b:b + 1] for a in arrays]
        n = None if lens is None else [lens[b]]
        refs = cross.cross_attention_backward(*one, n)
        reach = cross.cross_attention(*one[:3], n)[3].max()
        for name, got, ref, size in zip(("dq", "dk", "dv"), grads, refs, refs[3]):
            err, norm = np.linalg.norm(f64_of(got)[b:b + 1] - ref), np.linalg.norm(ref)
            if norm < 1e-9 * np.linalg.norm(size):
                assert err <= 2.0 ** -15 * (reach + 1) * np.linalg.norm(size), (b, name)
            else:
                part = 0.75 if q.shape[1] * q.shape[2] >= 1000 else 1.0
                assert err <= part * 2.0 ** -8 * norm, (b, name, err / norm)


CASES = [  # B, Sq, H, Hk, D, Skv, lens
    (1, 300, 4, 4, 128, 1, None),
    (1, 300, 4, 4, 64, 2, None),
    (1, 300, 4, 4, 128, 3, None),
    (1, 2001, 24, 24, 128, 5, None),
    (1, 301, 4, 2, 64, 8, None),
    (2, 177, 6, 2, 128, 12, None),
    (1, 300, 4, 4, 128, 32, None),                           # the last that counts as few
    (1, 300, 4, 4, 64, 33, None),                            # the first that does not
    (8, 260, 4, 2, 128, 40, [1, 2, 3, 12, 16, 17, 32, 33]),  # side by side
    (6, 77, 6, 1, 64, 300, [300, 2, 0, 31, 129, 3]),
    (3, 1, 28, 4, 128, 90, [5, 90, 1]),                      # a group of seven
    (2, 45, 28, 4, 64, 150, [150, 7]),
    (1, 130, 14, 2, 128, 257, None),
    (40, 3, 4, 2, 64, 50, [(7 * b) % 51 for b in range(40)]),   # passes over rows of several elements
    (2, 700, 5, 5, 128, 513, [513, 100]),
]


@pytest.mark.parametrize("B,Sq,H,Hk,D,Skv,lens", CASES)
def test_gradients_in_the_norm(B, Sq, H, Hk, D, Skv, lens):
    q, dout = normal(B, Sq, H, D, seed=1), normal(B, Sq, H, D, seed=4)
    k, v = normal(B, Skv, Hk, D, seed=2), normal(B, Skv, Hk, D, seed=3)
    out, lse = api.cpattn_cross_attention(q, k, v, lens_of(lens))
    check_forward(q, k, v, lens, out, lse)
    grads = api.cpattn_cross_attention_backward(q, k, v, out, lse, dout, lens_of(lens))
    check_norms(q, k, v, dout, lens, grads)
    check_backward(q, k, v, dout, lens, grads)
    again = api.cpattn_cross_attention_backward(q, k, v, out, lse, dout, lens_of(lens))
    for a, b in zip(grads, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -3e38])
@pytest.mark.parametrize("lens", [[5, 0, 31], [5, 200, 32]])
def test_padding_and_views(junk, lens):
    """K and V inside one projection's output with anything behind few states,
    q head-major."""
    B, Sq, H, Hk, D, Skv = 3, 150, 6, 2, 64, 200
    kv = normal(B, Skv, 2, Hk, D, seed=5)
    q = normal(B, H, Sq, D, seed=6).transpose(1, 2)
    dout = normal(B, Sq, H, D, seed=7)
    clean = kv.clone()
    for b, n in enumerate(lens):
        kv[b, n:], clean[b, n:] = junk, 0
    leaves = [t.detach().requires_grad_() for t in (q, kv[:, :, 0], kv[:, :, 1])]
    grads = torch.autograd.grad(autograd.cross_attention(*leaves, lens_of(lens)), leaves, dout)
    check_norms(q, clean[:, :, 0], clean[:, :, 1], dout, lens, grads)
    check_backward(q, clean[:, :, 0], clean[:, :, 1], dout, lens, grads)


def test_lengths_at_replay():
    """One captured backward whose elements have few states in one replay and
    many in the next, and the other way round."""
    B, Sq, H, Hk, D, Skv = 3, 90, 4, 2, 128, 100
    q, dout = normal(B, Sq, H, D, seed=1), normal(B, Sq, H, D, seed=4)
    k, v = normal(B, Skv, Hk, D, seed=2), normal(B, Skv, Hk, D, seed=3)
    lens = lens_of([100, 3, 40])
    stream = torch.cuda.Stream()

    def step():
        out, lse = api.cpattn_cross_attention(q, k, v, lens)
        return api.cpattn_cross_attention_backward(q, k, v, out, lse, dout, lens)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        grads = step()
    for n in ([100, 3, 40], [2, 77, 32], [33, 1, 0]):
        lens.copy_(lens_of(n))
        graph.replay()
        torch.cuda.synchronize()
        check_norms(q, k, v, dout, n, grads)
        check_backward(q, k, v, dout, n, grads)
