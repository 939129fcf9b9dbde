"""The operators' autograd functions without a GPU: the two bindings are
replaced by torch code, so that what autograd does around them can be seen."""
import pytest
import torch

from context_attention_long_b200 import api, autograd


def _norm(q, k, qw, kw, *_):
    def f(x, w):
        y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
        return y if w is None else y * w
    return f(q, qw), None if k is None else f(k, kw)


def _cross(q, k, v):
    s = torch.einsum("bqhd,bkhd->bhqk", q, k) * q.shape[-1] ** -0.5
    return torch.einsum("bhqk,bkhd->bqhd", s.softmax(-1), v)


def _grads(f, inputs, upstream):
    """First-order gradients of f at the inputs that are there, detached as a
    kernel's are."""
    with torch.enable_grad():
        leaves = [None if t is None else t.detach().requires_grad_() for t in inputs]
        outs = [o for o in f(*leaves) if o is not None]
        there = [t for t in leaves if t is not None]
        got = iter(torch.autograd.grad(outs, there, [g for g in upstream if g is not None], allow_unused=True))
    return tuple(None if t is None else next(got) for t in leaves)


@pytest.fixture(autouse=True)
def _torch_bindings(monkeypatch):
    def norm(q, k, qw, kw, cos, sin, positions, eps, interleaved, pos0):
        with torch.no_grad():
            return _norm(q, k, qw, kw)

    def norm_backward(q, k, gq, gk, qw, kw, cos, sin, positions, eps, interleaved, pos0, want_weights):
        return _grads(_norm, (q, k, qw, kw), (gq, gk))

    def cross(q, k, v, kv_lens):
        with torch.no_grad():
            return _cross(q, k, v), torch.zeros(())

    def cross_backward(q, k, v, out, lse, dout, kv_lens):
        return _grads(lambda *t: (_cross(*t),), (q, k, v), (dout,))
    monkeypatch.setattr(api, "cpattn_qk_norm_rope", norm)
    monkeypatch.setattr(api, "cpattn_qk_norm_rope_backward", norm_backward)
    monkeypatch.setattr(api, "cpattn_cross_attention", cross)
    monkeypatch.setattr(api, "cpattn_cross_attention_backward", cross_backward)


def _leaf(*shape):
    return torch.randn(shape, dtype=torch.float64).requires_grad_()


def _cases():
    q, k, v, w = _leaf(1, 5, 2, 64), _leaf(1, 7, 2, 64), _leaf(1, 7, 2, 64), _leaf(64)
    t = _leaf(1, 5, 2, 64)
    return {
        "cross": ([q, k, v], lambda: autograd.cross_attention(q, k, v), lambda: _cross(q, k, v)),
        "norm": ([q, t, w], lambda: sum(autograd.qk_norm_rope(q, t, w, w)), lambda: sum(_norm(q, t, w, w))),
        "norm of one": ([q], lambda: autograd.qk_norm_rope(q)[0], lambda: _norm(q, None, None, None)[0]),
    }


@pytest.mark.parametrize("name", ["cross", "norm", "norm of one"])
@pytest.mark.parametrize("of", [torch.sum, lambda t: t.pow(3).sum()])   # an upstream gradient without a graph, and with
def test_gradients_of_gradients_raise(name, of):
    leaves, f, plain = _cases()[name]
    want = torch.autograd.grad(of(plain()), leaves)
    loss = of(f())
    grads = torch.autograd.grad(loss, leaves, create_graph=True)
    for a, b in zip(grads, want):              # the first order is there, recorded or not
        torch.testing.assert_close(a.detach(), b, rtol=1e-9, atol=1e-9)
        assert a.requires_grad
    with pytest.raises(RuntimeError, match="not offered"):
        (loss + sum(g.square().sum() for g in grads)).backward()


@pytest.mark.parametrize("name", ["cross", "norm", "norm of one"])
def test_recorded_gradients_may_go_unused(name):
    """A step with create_graph=True that differentiates through other parts
    only, and an ordinary one."""
    leaves, f, plain = _cases()[name]
    other = _leaf(3)
    loss = f().sum() + other.pow(3).sum()
    grads = torch.autograd.grad(loss, [other] + leaves, create_graph=True)
    grads[0].square().sum().backward()
    torch.testing.assert_close(other.grad, 36 * other.detach() ** 3)
    ordinary = torch.autograd.grad(f().sum(), leaves)
    assert not any(g.requires_grad for g in ordinary)


@pytest.mark.parametrize("name", ["cross", "norm", "norm of one"])
def test_recorded_gradients_may_be_changed_in_place(name):
    """As clipping does."""
    leaves, f, plain = _cases()[name]
    want = torch.autograd.grad(plain().sum(), leaves)
    f().sum().backward(create_graph=True)
    with torch.no_grad():
        for t in leaves:
            t.grad.mul_(0.5)
    for t, w in zip(leaves, want):
        torch.testing.assert_close(t.grad.detach(), 0.5 * w, rtol=1e-9, atol=1e-9)
    grads = torch.autograd.grad(f().sum(), leaves, create_graph=True)
    for g, w in zip(grads, want):
        torch.testing.assert_close(g.mul_(2).detach(), 2 * w, rtol=1e-9, atol=1e-9)
    with pytest.raises(RuntimeError, match="not offered"):
        sum(g.sum() for g in grads).backward()
