"""torch.autograd functions over this library's attention kernels, for
training with context-parallel attention (the Ulysses Sequence Parallelism
article, sections 1 and 7: long-context training, causal masking by position).

Each function's forward is one of the library's forward entry points and its
backward the matching backward entry point (the derivative of the forward's
definition: dQ, dK and dV from the forward's output, its log-sum-exp and the
upstream gradient).  Like api.py, this module only marshals arguments: both
passes run in the library's kernels, and nothing here computes.

A backward pass can be captured in a CUDA graph after an eager one on the
capture's stream.  Drop eager results of the same leaves first: autograd keeps
one accumulation node a leaf while a graph that leads to it lives, bound to the
stream it was made on, and a capture may not wait for another stream.
"""
from __future__ import annotations

import torch

from . import api


class RingAttentionFunction(torch.autograd.Function):
    """Attention of (B, S, H, D) bf16 Q, K, V whose sequence is cut into
    `ring_degree` shards (the fused ring kernel; `chunk_lens` for uneven
    shards), causal or not.  The gradient does not depend on the sharding:
    it is the attention backward over the full tensors."""

    @staticmethod
    def forward(ctx, q, k, v, ring_degree, causal, chunk_lens):
        fn = api.cpattn_causal_ring_attention if causal else api.cpattn_ring_attention
        out, lse = fn(q, k, v, ring_degree, chunk_lens)
        ctx.save_for_backward(q, k, v, out, lse)
        ctx.causal = bool(causal)
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, out, lse = ctx.saved_tensors
        dq, dk, dv = api.cpattn_attention_backward(q, k, v, out, lse, dout.contiguous(), ctx.causal)
        return dq, dk, dv, None, None, None


class UlyssesAttentionFunction(torch.autograd.Function):
    """The Ulysses flow on sequence-sharded rank buffers (flat bf16: the
    `degree` ranks' (B, S_r, H, D) buffers concatenated), even or uneven
    `seq_splits` / `head_splits`, causal or not.  The backward runs the
    Ulysses flow's backward on the same layout."""

    @staticmethod
    def forward(ctx, q, k, v, B, S, H, D, degree, seq_splits, head_splits, causal):
        fn = api.cpattn_causal_ulysses_attention if causal else api.cpattn_ulysses_attention
        out, lse = fn(q, k, v, B, S, H, D, degree, seq_splits, head_splits)
        ctx.save_for_backward(q, k, v, out, lse)
        ctx.args = (B, S, H, D, degree, seq_splits, head_splits, bool(causal))
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, out, lse = ctx.saved_tensors
        B, S, H, D, degree, seq_splits, head_splits, causal = ctx.args
        dq, dk, dv = api.cpattn_ulysses_attention_backward(q, k, v, out, lse, dout.contiguous(), B, S, H, D,
                                                           degree, seq_splits, head_splits, causal)
        return (dq, dk, dv) + (None,) * 8


def _readable(t):
    """A gradient as autograd hands it over (any strides, perhaps expanded) in
    a form that the kernels read: unit stride in a head, 16-byte pieces."""
    ok = t.stride(-1) == 1 and t.data_ptr() % 16 == 0 and all(s % 8 == 0 for s in t.stride()[:3])
    return t if ok else t.clone(memory_format=torch.contiguous_format)   # contiguous() keeps an unaligned address


class _FirstOrderOnly(torch.autograd.Function):
    """Passes a backward's gradients, the first n of `tensors`, on as functions
    of all of them whose own gradient raises."""

    @staticmethod
    def forward(ctx, name, n, *tensors):
        ctx.name = name
        return tuple(t.detach() for t in tensors[:n])   # not the inputs themselves: views may not be changed in place

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError(f"{ctx.name}: gradients of its gradients are not offered")


def _first_order_only(name, grads, *inputs):
    """The gradients that a backward returns.  Where autograd records it
    (create_graph=True) they would be constants to a loss of them, which would
    lose that part of its gradient without a word; so they are made functions of
    all that the backward read, and differentiating them raises."""
    if not torch.is_grad_enabled():
        return grads
    there = [g for g in grads if g is not None]
    passed = iter(_FirstOrderOnly.apply(name, len(there), *there, *(t for t in inputs if t is not None)))
    return tuple(None if g is None else next(passed) for g in grads)


class QKNormRopeFunction(torch.autograd.Function):
    """Per-head RMS norm of Q and K with the position rotation.  The backward
    needs only the forward's inputs."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved, pos0):
        q_out, k_out = api.cpattn_qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved, pos0)
        ctx.save_for_backward(q, k, q_weight, k_weight, cos, sin, positions)
        ctx.args = (eps, interleaved, pos0)
        return q_out, k_out

    @staticmethod
    def backward(ctx, dq_out, dk_out):
        q, k, q_weight, k_weight, cos, sin, positions = ctx.saved_tensors
        eps, interleaved, pos0 = ctx.args
        dq, dk, dqw, dkw = api.cpattn_qk_norm_rope_backward(
            q, k, _readable(dq_out), None if k is None else _readable(dk_out), q_weight, k_weight, cos, sin,
            positions, eps, interleaved, pos0, want_weights=any(ctx.needs_input_grad[2:4]))
        return _first_order_only("qk_norm_rope", (dq, dk, dqw, dkw), dq_out, dk_out, q, k, q_weight, k_weight) + \
            (None,) * 6


def qk_norm_rope(q, k=None, q_weight=None, k_weight=None, cos=None, sin=None, positions=None, eps=1e-6,
                 interleaved=True, pos0=0):
    """Differentiable per-head RMS norm of q (B, S, H, D) and k (B, S, Hk, D)
    with the position rotation (api.cpattn_qk_norm_rope); returns (q, k).
    Gradients go to q, k and the weights, not to the tables; first-order only:
    differentiating them (create_graph=True) raises."""
    return QKNormRopeFunction.apply(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved, pos0)


class CrossAttentionFunction(torch.autograd.Function):
    """Attention of q to an encoder's states k, v of another length."""

    @staticmethod
    def forward(ctx, q, k, v, kv_lens):
        out, lse = api.cpattn_cross_attention(q, k, v, kv_lens)
        ctx.save_for_backward(q, k, v, out, lse, kv_lens)
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, out, lse, kv_lens = ctx.saved_tensors
        dout = dout.contiguous()
        dq, dk, dv = api.cpattn_cross_attention_backward(q, k, v, out, lse,
                                                         dout if dout.data_ptr() % 16 == 0 else dout.clone(), kv_lens)
        return _first_order_only("cross_attention", (dq, dk, dv), dout, q, k, v) + (None,)


def cross_attention(q, k, v, kv_lens=None):
    """Differentiable cross attention of q (B, Sq, H, D) to k, v
    (B, Skv, Hk, D) (api.cpattn_cross_attention); returns out (B, Sq, H, D).
    First-order gradients only: differentiating them (create_graph=True) raises."""
    return CrossAttentionFunction.apply(q, k, v, kv_lens)


def ring_attention(q, k, v, ring_degree=1, causal=False, chunk_lens=None):
    """Differentiable fused ring attention; returns out (B, S, H, D) bf16."""
    return RingAttentionFunction.apply(q, k, v, ring_degree, causal, chunk_lens)


def ulysses_attention(q, k, v, B, S, H, D, degree, seq_splits=None, head_splits=None, causal=False):
    """Differentiable Ulysses attention on rank buffers; returns out in the
    same rank-buffer layout."""
    return UlyssesAttentionFunction.apply(q, k, v, B, S, H, D, degree, seq_splits, head_splits, causal)
