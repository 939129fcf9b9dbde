"""Thin PyTorch binding of the C ABI (include/cpattn.h), same function names.

Argument marshalling only: shapes and pointers are read from torch tensors,
outputs are allocated with torch when not given, and every step of the hot path
runs in libcpattn.so's CUDA kernels on the current (or given) CUDA stream.
There is no CPU path: calling without a CUDA device or without the built
library raises.

Layouts: Q/K/V/out are bf16 (B, S, H, D) contiguous; LSE is float32 (B, H, S),
natural log.  See include/cpattn.h for the exact semantics of each call.
"""
from __future__ import annotations

import ctypes

import torch

from . import _native

__all__ = [
    "CpattnError", "cpattn_ring_attention", "cpattn_causal_ring_attention", "cpattn_ring_step",
    "cpattn_causal_ring_step", "cpattn_lse_merge", "cpattn_kv_gather_attention", "cpattn_ulysses_permute",
    "cpattn_ulysses_permute_qkv", "cpattn_ulysses_unpermute", "cpattn_ulysses_qkv_projection",
    "cpattn_ulysses_output_projection", "cpattn_head_sharded_attention",
    "cpattn_causal_head_sharded_attention", "cpattn_ulysses_workspace_bytes",
    "cpattn_unified_workspace_bytes", "cpattn_ulysses_attention", "cpattn_causal_ulysses_attention",
    "cpattn_unified_attention", "cpattn_causal_unified_attention",
    "cpattn_attention_backward_workspace_bytes", "cpattn_attention_backward_ds_bytes", "cpattn_attention_backward",
    "backward_workspace_bytes", "BACKWARD_DS_BUDGET",
    "cpattn_ulysses_attention_backward_workspace_bytes", "cpattn_ulysses_attention_backward",
    "cpattn_qk_norm_rope", "cpattn_qk_norm_rope_backward", "cpattn_qk_norm_rope_backward_workspace_bytes",
    "cpattn_cross_attention", "cpattn_cross_attention_backward", "cpattn_cross_attention_backward_ds_bytes",
    "cpattn_cross_attention_backward_workspace_bytes", "cross_backward_workspace_bytes",
    "cpattn_ulysses_attention_noalloc", "cpattn_ring_chunk_attention", "cpattn_gathered_kv_attention",
    "cpattn_rank_buffer_attention", "cpattn_front_loaded_splits", "cpattn_exchange_bytes",
    "cpattn_plan_exchange", "cpattn_device_status", "cpattn_debug_wait_timeout", "NOALLOC_SCRATCH_BYTES",
    "status_string",
]


CPATTN_ERR_CUDA = 6


class CpattnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where}: {status_string(status)} ({status})"
        if status == CPATTN_ERR_CUDA:
            msg += " -- " + _native.load().cpattn_last_cuda_error_string().decode()
        super().__init__(msg)


def status_string(status: int) -> str:
    return _native.load().cpattn_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != 0:
        raise CpattnError(status, where)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    """Device address of a tensor the library may read or write.  The kernels
    launch on the current CUDA device and index the memory densely, so a host
    tensor, a tensor on another device or a non-contiguous view is refused
    here, before the library sees the pointer."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("tensor arguments must be CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("tensor arguments must be contiguous")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"tensor on {t.device}, but the current device is cuda:{torch.cuda.current_device()}")
    return ctypes.c_void_p(t.data_ptr())


def _need(t, numel, dtype, name):
    """A tensor argument must hold at least `numel` elements of `dtype`: the
    library indexes the memory behind the pointer by the sizes it is given."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() < numel:
        raise ValueError(f"{name} holds {t.numel()} elements, {numel} needed")


def _bshd(q: torch.Tensor, name="q"):
    if q.dim() != 4:
        raise ValueError(f"{name} must be (B, S, H, D)")
    if not q.is_cuda or q.dtype != torch.bfloat16 or not q.is_contiguous():
        raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor")
    B, S, H, D = q.shape
    return B, S, H, D


def _ring(entry, q, k, v, ring_degree, chunk_lens, out, lse, want_lse, stream):
    B, S, H, D = _bshd(q)
    out = torch.empty_like(q) if out is None else out
    if lse is None and want_lse:
        lse = torch.empty((B, H, S), dtype=torch.float32, device=q.device)
    for t, name in ((k, "k"), (v, "v"), (out, "out")):
        _need(t, q.numel(), torch.bfloat16, name)
    _need(lse, B * H * S, torch.float32, "lse")
    _check(getattr(_native.load(), entry)(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, S, D,
                                          int(ring_degree), _native.int_array(chunk_lens), _stream(stream)), entry)
    return out, lse


def cpattn_ring_attention(q, k, v, ring_degree, chunk_lens=None, out=None, lse=None, want_lse=True, stream=None):
    """Fused ring attention; returns (out bf16 (B,S,H,D), lse float32 (B,H,S) or None)."""
    return _ring("cpattn_ring_attention", q, k, v, ring_degree, chunk_lens, out, lse, want_lse, stream)


def cpattn_causal_ring_attention(q, k, v, ring_degree, chunk_lens=None, out=None, lse=None, want_lse=True,
                                 stream=None):
    """Fused causal ring attention (key j visible to query i iff j <= i); returns (out, lse)."""
    return _ring("cpattn_causal_ring_attention", q, k, v, ring_degree, chunk_lens, out, lse, want_lse, stream)


def _ring_step(entry, q, k, v, ring_degree, step, chunk_lens, part_out, part_lse, stream):
    B, S, H, D = _bshd(q)
    if part_out is None:
        part_out = torch.empty((B, S, H, D), dtype=torch.float32, device=q.device)
    if part_lse is None:
        part_lse = torch.empty((B, H, S), dtype=torch.float32, device=q.device)
    _need(k, q.numel(), torch.bfloat16, "k")
    _need(v, q.numel(), torch.bfloat16, "v")
    _need(part_out, q.numel(), torch.float32, "part_out")
    _need(part_lse, B * H * S, torch.float32, "part_lse")
    _check(getattr(_native.load(), entry)(_ptr(q), _ptr(k), _ptr(v), _ptr(part_out), _ptr(part_lse), B, H, S, D,
                                          int(ring_degree), _native.int_array(chunk_lens), int(step),
                                          _stream(stream)), entry)
    return part_out, part_lse


def cpattn_ring_step(q, k, v, ring_degree, step, chunk_lens=None, part_out=None, part_lse=None, stream=None):
    """One ring step for every rank; returns float32 (partial out (B,S,H,D), partial lse (B,H,S))."""
    return _ring_step("cpattn_ring_step", q, k, v, ring_degree, step, chunk_lens, part_out, part_lse, stream)


def cpattn_causal_ring_step(q, k, v, ring_degree, step, chunk_lens=None, part_out=None, part_lse=None,
                            stream=None):
    """One causal ring step for every rank (a chunk after the rank's shard gives out 0, lse -inf)."""
    return _ring_step("cpattn_causal_ring_step", q, k, v, ring_degree, step, chunk_lens, part_out, part_lse, stream)


def cpattn_lse_merge(part_out, part_lse, out_f32=None, out_bf16=None, lse_out=None, want_f32=False,
                     want_bf16=True, stream=None):
    """Merge P float32 partials: part_out (P,B,S,H,D), part_lse (P,B,H,S).
    Returns (out_f32 or None, out_bf16 or None, lse_out)."""
    P, B, S, H, D = part_out.shape
    dev = part_out.device
    if out_f32 is None and want_f32:
        out_f32 = torch.empty((B, S, H, D), dtype=torch.float32, device=dev)
    if out_bf16 is None and want_bf16:
        out_bf16 = torch.empty((B, S, H, D), dtype=torch.bfloat16, device=dev)
    if lse_out is None:
        lse_out = torch.empty((B, H, S), dtype=torch.float32, device=dev)
    n = B * S * H * D
    _need(part_out, P * n, torch.float32, "part_out")
    _need(part_lse, P * B * H * S, torch.float32, "part_lse")
    _need(out_f32, n, torch.float32, "out_f32")
    _need(out_bf16, n, torch.bfloat16, "out_bf16")
    _need(lse_out, B * H * S, torch.float32, "lse_out")
    _check(_native.load().cpattn_lse_merge(_ptr(part_out), _ptr(part_lse), P, B, H, S, D, _ptr(out_f32),
                                           _ptr(out_bf16), _ptr(lse_out), _stream(stream)), "cpattn_lse_merge")
    return out_f32, out_bf16, lse_out


def cpattn_kv_gather_attention(q, k, v, degree, q_lens=None, out=None, lse=None, want_lse=True, stream=None):
    """kv_gather attention; returns (out, lse)."""
    B, S, H, D = _bshd(q)
    out = torch.empty_like(q) if out is None else out
    if lse is None and want_lse:
        lse = torch.empty((B, H, S), dtype=torch.float32, device=q.device)
    for t, name in ((k, "k"), (v, "v"), (out, "out")):
        _need(t, q.numel(), torch.bfloat16, name)
    _need(lse, B * H * S, torch.float32, "lse")
    _check(_native.load().cpattn_kv_gather_attention(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, S, D,
                                                     int(degree), _native.int_array(q_lens), _stream(stream)),
           "cpattn_kv_gather_attention")
    return out, lse


def _flat_numel(B, S, H, D):
    return B * S * H * D


def cpattn_ulysses_permute(x, B, S, H, D, degree, seq_splits=None, head_splits=None, y=None, stream=None):
    """Sequence-sharded rank buffers (flat, any 1/2/4/8-byte dtype) -> head-sharded rank buffers."""
    if y is None:
        y = torch.empty_like(x)
    _need(x, _flat_numel(B, S, H, D), None, "x")
    _need(y, _flat_numel(B, S, H, D), x.dtype, "y")
    _check(_native.load().cpattn_ulysses_permute(_ptr(x), _ptr(y), B, S, H, D, x.element_size(), int(degree),
                                                 _native.int_array(seq_splits), _native.int_array(head_splits),
                                                 _stream(stream)), "cpattn_ulysses_permute")
    return y


def cpattn_ulysses_permute_qkv(q, k, v, B, S, H, D, degree, seq_splits=None, head_splits=None, yq=None, yk=None,
                               yv=None, stream=None):
    """The Q, K and V permutes of the first all-to-all in one launch; returns (yq, yk, yv)."""
    yq = torch.empty_like(q) if yq is None else yq
    yk = torch.empty_like(k) if yk is None else yk
    yv = torch.empty_like(v) if yv is None else yv
    for t, name in ((q, "q"), (k, "k"), (v, "v"), (yq, "yq"), (yk, "yk"), (yv, "yv")):
        _need(t, _flat_numel(B, S, H, D), q.dtype, name)
    _check(_native.load().cpattn_ulysses_permute_qkv(_ptr(q), _ptr(k), _ptr(v), _ptr(yq), _ptr(yk), _ptr(yv), B, S,
                                                     H, D, q.element_size(), int(degree),
                                                     _native.int_array(seq_splits), _native.int_array(head_splits),
                                                     _stream(stream)), "cpattn_ulysses_permute_qkv")
    return yq, yk, yv


def cpattn_ulysses_unpermute(y, B, S, H, D, degree, seq_splits=None, head_splits=None, x=None, stream=None):
    """Head-sharded rank buffers -> sequence-sharded rank buffers (inverse permute)."""
    if x is None:
        x = torch.empty_like(y)
    _need(y, _flat_numel(B, S, H, D), None, "y")
    _need(x, _flat_numel(B, S, H, D), y.dtype, "x")
    _check(_native.load().cpattn_ulysses_unpermute(_ptr(y), _ptr(x), B, S, H, D, y.element_size(), int(degree),
                                                   _native.int_array(seq_splits), _native.int_array(head_splits),
                                                   _stream(stream)), "cpattn_ulysses_unpermute")
    return x


def cpattn_ulysses_qkv_projection(x, w_qkv, B, S, H, D, Dm, degree, seq_splits=None, head_splits=None, yq=None,
                                  yk=None, yv=None, stream=None):
    """Q, K, V projections of the sequence-side activations x (rank buffers
    (B, S_r, Dm) concatenated, bf16) by w_qkv (3*H*D, Dm), stored straight into
    the head-sharded layout; returns flat (yq, yk, yv) of B*S*H*D bf16 each."""
    n = _flat_numel(B, S, H, D)
    yq, yk, yv = (torch.empty(n, dtype=torch.bfloat16, device=x.device) if t is None else t for t in (yq, yk, yv))
    _need(x, B * S * Dm, torch.bfloat16, "x")
    _need(w_qkv, 3 * H * D * Dm, torch.bfloat16, "w_qkv")
    for t, name in ((yq, "yq"), (yk, "yk"), (yv, "yv")):
        _need(t, n, torch.bfloat16, name)
    _check(_native.load().cpattn_ulysses_qkv_projection(_ptr(x), _ptr(w_qkv), _ptr(yq), _ptr(yk), _ptr(yv), B, S, H,
                                                        D, Dm, int(degree), _native.int_array(seq_splits),
                                                        _native.int_array(head_splits), _stream(stream)),
           "cpattn_ulysses_qkv_projection")
    return yq, yk, yv


def cpattn_ulysses_output_projection(yo, w_o, B, S, H, D, Dm, degree, seq_splits=None, head_splits=None, out=None,
                                     stream=None):
    """Output projection by w_o (Dm, H*D) of the head-sharded attention output yo,
    read in place; returns the sequence-side result (rank buffers (B, S_r, Dm)
    concatenated), flat bf16 of B*S*Dm."""
    out = torch.empty(B * S * Dm, dtype=torch.bfloat16, device=yo.device) if out is None else out
    _need(yo, _flat_numel(B, S, H, D), torch.bfloat16, "yo")
    _need(w_o, Dm * H * D, torch.bfloat16, "w_o")
    _need(out, B * S * Dm, torch.bfloat16, "out")
    _check(_native.load().cpattn_ulysses_output_projection(_ptr(yo), _ptr(w_o), _ptr(out), B, S, H, D, Dm,
                                                           int(degree), _native.int_array(seq_splits),
                                                           _native.int_array(head_splits), _stream(stream)),
           "cpattn_ulysses_output_projection")
    return out


def _head_sharded(entry, yq, yk, yv, B, S, H, D, degree, head_splits, yo, lse, want_lse, stream):
    yo = torch.empty_like(yq) if yo is None else yo
    if lse is None and want_lse:
        lse = torch.empty((B, H, S), dtype=torch.float32, device=yq.device)
    for t, name in ((yq, "yq"), (yk, "yk"), (yv, "yv"), (yo, "yo")):
        _need(t, _flat_numel(B, S, H, D), torch.bfloat16, name)
    _need(lse, B * H * S, torch.float32, "lse")
    _check(getattr(_native.load(), entry)(_ptr(yq), _ptr(yk), _ptr(yv), _ptr(yo), _ptr(lse), B, H, S, D,
                                          int(degree), _native.int_array(head_splits), _stream(stream)), entry)
    return yo, lse


def cpattn_head_sharded_attention(yq, yk, yv, B, S, H, D, degree, head_splits=None, yo=None, lse=None,
                                  want_lse=True, stream=None):
    """Local attention on head-sharded rank buffers; returns (yo, lse (B,H,S))."""
    return _head_sharded("cpattn_head_sharded_attention", yq, yk, yv, B, S, H, D, degree, head_splits, yo, lse,
                         want_lse, stream)


def cpattn_causal_head_sharded_attention(yq, yk, yv, B, S, H, D, degree, head_splits=None, yo=None, lse=None,
                                         want_lse=True, stream=None):
    """Causal local attention on head-sharded rank buffers; returns (yo, lse (B,H,S))."""
    return _head_sharded("cpattn_causal_head_sharded_attention", yq, yk, yv, B, S, H, D, degree, head_splits, yo,
                         lse, want_lse, stream)


def cpattn_ulysses_workspace_bytes(B, H, S, D) -> int:
    return int(_native.load().cpattn_ulysses_workspace_bytes(B, H, S, D))


def cpattn_unified_workspace_bytes(B, H, S, D) -> int:
    return int(_native.load().cpattn_unified_workspace_bytes(B, H, S, D))


def _workspace(nbytes, device, workspace):
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return workspace


def _ulysses(entry, q, k, v, B, S, H, D, degree, seq_splits, head_splits, out, lse, want_lse, workspace, stream):
    out = torch.empty_like(q) if out is None else out
    if lse is None and want_lse:
        lse = torch.empty((B, H, S), dtype=torch.float32, device=q.device)
    nbytes = cpattn_ulysses_workspace_bytes(B, H, S, D)
    workspace = _workspace(nbytes, q.device, workspace)
    for t, name in ((q, "q"), (k, "k"), (v, "v"), (out, "out")):
        _need(t, _flat_numel(B, S, H, D), torch.bfloat16, name)
    _need(lse, B * H * S, torch.float32, "lse")
    _check(getattr(_native.load(), entry)(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, S, D,
                                          int(degree), _native.int_array(seq_splits),
                                          _native.int_array(head_splits), _ptr(workspace),
                                          workspace.numel() * workspace.element_size(), _stream(stream)), entry)
    return out, lse


def cpattn_ulysses_attention(q, k, v, B, S, H, D, degree, seq_splits=None, head_splits=None, out=None, lse=None,
                             want_lse=True, workspace=None, stream=None):
    """Ulysses attention on sequence-sharded rank buffers (flat bf16); returns (out, lse)."""
    return _ulysses("cpattn_ulysses_attention", q, k, v, B, S, H, D, degree, seq_splits, head_splits, out, lse,
                    want_lse, workspace, stream)


def cpattn_causal_ulysses_attention(q, k, v, B, S, H, D, degree, seq_splits=None, head_splits=None, out=None,
                                    lse=None, want_lse=True, workspace=None, stream=None):
    """Causal Ulysses attention on sequence-sharded rank buffers (flat bf16); returns (out, lse)."""
    return _ulysses("cpattn_causal_ulysses_attention", q, k, v, B, S, H, D, degree, seq_splits, head_splits, out,
                    lse, want_lse, workspace, stream)


def _unified(entry, q, k, v, ring_degree, ulysses_degree, ring_lens, head_splits, out, lse, want_lse, workspace,
             stream):
    B, S, H, D = _bshd(q)
    out = torch.empty_like(q) if out is None else out
    if lse is None and want_lse:
        lse = torch.empty((B, H, S), dtype=torch.float32, device=q.device)
    nbytes = cpattn_unified_workspace_bytes(B, H, S, D)
    workspace = _workspace(nbytes, q.device, workspace)
    for t, name in ((k, "k"), (v, "v"), (out, "out")):
        _need(t, q.numel(), torch.bfloat16, name)
    _need(lse, B * H * S, torch.float32, "lse")
    _check(getattr(_native.load(), entry)(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, S, D,
                                          int(ring_degree), int(ulysses_degree), _native.int_array(ring_lens),
                                          _native.int_array(head_splits), _ptr(workspace),
                                          workspace.numel() * workspace.element_size(), _stream(stream)), entry)
    return out, lse


def cpattn_unified_attention(q, k, v, ring_degree, ulysses_degree, ring_lens=None, head_splits=None, out=None,
                             lse=None, want_lse=True, workspace=None, stream=None):
    """Unified ring x Ulysses attention on full (B,S,H,D) tensors; returns (out, lse)."""
    return _unified("cpattn_unified_attention", q, k, v, ring_degree, ulysses_degree, ring_lens, head_splits, out,
                    lse, want_lse, workspace, stream)


def cpattn_causal_unified_attention(q, k, v, ring_degree, ulysses_degree, ring_lens=None, head_splits=None,
                                    out=None, lse=None, want_lse=True, workspace=None, stream=None):
    """Causal unified ring x Ulysses attention on full (B,S,H,D) tensors; returns (out, lse)."""
    return _unified("cpattn_causal_unified_attention", q, k, v, ring_degree, ulysses_degree, ring_lens,
                    head_splits, out, lse, want_lse, workspace, stream)


def cpattn_attention_backward_workspace_bytes(B, H, S) -> int:
    return int(_native.load().cpattn_attention_backward_workspace_bytes(B, H, S))


def cpattn_attention_backward_ds_bytes(B, S, causal) -> int:
    return int(_native.load().cpattn_attention_backward_ds_bytes(B, S, 1 if causal else 0))


# Default cap on the dS scratch the backward bindings add to a workspace they
# allocate: the library groups the heads so that their dS tiles fit it, and
# when one head's tiles exceed it the dQ kernel runs instead.
BACKWARD_DS_BUDGET = 8 << 30


def _ds_scratch_bytes(B, H, S, causal, ds_budget):
    """Whole heads of dS scratch within the budget, plus the 256 bytes the
    library may skip to align it (0: no scratch)."""
    per = cpattn_attention_backward_ds_bytes(B, S, causal)
    budget = BACKWARD_DS_BUDGET if ds_budget is None else int(ds_budget)
    heads = min(H, budget // per) if per > 0 else 0
    return 256 + heads * per if heads > 0 else 0


def backward_workspace_bytes(B, H, S, causal=False, ds_budget=None, ulysses_D=None) -> int:
    """Bytes of the workspace the backward bindings allocate: the minimum of
    cpattn_attention_backward (or, given ulysses_D, of the Ulysses backward
    flow) plus whole heads of dS scratch within ds_budget.  A workspace sized
    for causal=False also serves the causal backward."""
    base = (cpattn_attention_backward_workspace_bytes(B, H, S) if ulysses_D is None else
            cpattn_ulysses_attention_backward_workspace_bytes(B, H, S, ulysses_D))
    return base + _ds_scratch_bytes(B, H, S, causal, ds_budget)


def _allocation_budget(device, ds_budget):
    """The dS budget for a workspace the binding allocates itself: the given
    one, or by default BACKWARD_DS_BUDGET capped at half the device's free
    memory (a smaller scratch only means more head groups)."""
    if ds_budget is not None:
        return int(ds_budget)
    free, _ = torch.cuda.mem_get_info(device)
    return min(BACKWARD_DS_BUDGET, free // 2)


def cpattn_attention_backward(q, k, v, out, lse, dout, causal=False, dq=None, dk=None, dv=None, workspace=None,
                              stream=None, ds_budget=None):
    """Gradient of attention over full (B,S,H,D) bf16 tensors given the
    forward's output and LSE; returns (dq, dk, dv) in bf16.  An allocated
    workspace holds up to ds_budget bytes of dS scratch (default
    BACKWARD_DS_BUDGET, capped at half the device's free memory); 0 selects
    the dQ kernel that recomputes S and dP."""
    B, S, H, D = _bshd(q)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if workspace is None:
        workspace = _workspace(backward_workspace_bytes(B, H, S, causal, _allocation_budget(q.device, ds_budget)),
                               q.device, None)
    for t, name in ((k, "k"), (v, "v"), (out, "out"), (dout, "dout"), (dq, "dq"), (dk, "dk"), (dv, "dv")):
        _need(t, q.numel(), torch.bfloat16, name)
    _need(lse, B * H * S, torch.float32, "lse")
    if lse is None:
        raise ValueError("lse is required")
    _check(_native.load().cpattn_attention_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout),
                                                    _ptr(dq), _ptr(dk), _ptr(dv), B, H, S, D, 1 if causal else 0,
                                                    _ptr(workspace), workspace.numel() * workspace.element_size(),
                                                    _stream(stream)), "cpattn_attention_backward")
    return dq, dk, dv


def cpattn_ulysses_attention_backward_workspace_bytes(B, H, S, D) -> int:
    return int(_native.load().cpattn_ulysses_attention_backward_workspace_bytes(B, H, S, D))


def cpattn_ulysses_attention_backward(q, k, v, out, lse, dout, B, S, H, D, degree, seq_splits=None,
                                      head_splits=None, causal=False, dq=None, dk=None, dv=None, workspace=None,
                                      stream=None, ds_budget=None):
    """Backward of the Ulysses flow on sequence-sharded rank buffers (flat
    bf16); returns (dq, dk, dv) in the same layout.  ds_budget as
    cpattn_attention_backward."""
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if workspace is None:
        workspace = _workspace(backward_workspace_bytes(B, H, S, causal, _allocation_budget(q.device, ds_budget),
                                                        ulysses_D=D), q.device, None)
    for t, name in ((q, "q"), (k, "k"), (v, "v"), (out, "out"), (dout, "dout"), (dq, "dq"), (dk, "dk"), (dv, "dv")):
        _need(t, _flat_numel(B, S, H, D), torch.bfloat16, name)
    _need(lse, B * H * S, torch.float32, "lse")
    if lse is None:
        raise ValueError("lse is required")
    _check(_native.load().cpattn_ulysses_attention_backward(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), B, H, S, D,
        int(degree), _native.int_array(seq_splits), _native.int_array(head_splits), 1 if causal else 0,
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)),
        "cpattn_ulysses_attention_backward")
    return dq, dk, dv


def _view(t, name, device, shape=None):
    """(address, strides) of a (B, S, H, D) bf16 view on `device` whose heads'
    elements are consecutive; strides None for a contiguous one."""
    if not isinstance(t, torch.Tensor) or t.dim() != 4 or t.dtype is not torch.bfloat16 or not t.is_cuda:
        raise ValueError(f"{name} must be a 4-D bf16 CUDA tensor (B, S, H, D)")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{device}")
    if t.is_contiguous():
        return t.data_ptr(), None
    st = t.stride()
    if st[3] != 1:
        raise ValueError(f"{name}: the elements of a head must be consecutive (stride 1)")
    return t.data_ptr(), _native.strides_array(st[:3])


def _plain(t, name, device, dtype, shape=None):
    """Address of a contiguous tensor of `dtype` on `device`, or None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{device}")
    return t.data_ptr()


def _raw_stream(stream, device):
    """cudaStream_t of the given or the device's current stream, as a number."""
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream


def _new(like, shape, dtype, stream, returned=True):
    """A tensor that a binding allocates for a call on `stream` (None: the
    current one): a block of that stream's pool.  The allocator hands a block
    out again while the work that last used it may still be queued on the
    pool's own stream, so a block of the current stream's pool could be written
    by both streams at once.  `returned`: the caller will use it on the current
    stream, and its block may not be handed out before that work either."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    current = torch.cuda.current_stream()
    if stream == current:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        t = like.new_empty(shape, dtype=dtype)
    if returned:
        t.record_stream(current)
    return t


def _norm_rope_args(q, k, q_weight, k_weight, cos, sin, positions, device):
    """The checked arguments that the norm's forward and backward share:
    (q, k, weights and tables as addresses, sizes)."""
    qp, qs = _view(q, "q", device)
    B, S, H, D = q.shape
    kp, ks, Hk = None, None, 0
    if k is not None:
        Hk = k.shape[2] if k.dim() == 4 else 0
        kp, ks = _view(k, "k", device, (B, S, Hk, D))
    w = q_weight if q_weight is not None else k_weight
    f32 = w is not None and w.dtype is torch.float32
    dtype = torch.float32 if f32 else torch.bfloat16
    wq = _plain(q_weight, "q_weight", device, dtype, (D,))
    wk = _plain(k_weight, "k_weight", device, dtype, (D,))
    rot = n_pos = 0
    cp = sp = pp = None
    if cos is not None or sin is not None:
        cp = _plain(cos, "cos", device, torch.float32)
        if cp is None or cos.dim() != 2:
            raise ValueError("cos and sin must be two (n_pos, rotary_dim / 2) tables")
        sp = _plain(sin, "sin", device, torch.float32, cos.shape)
        if sp is None:
            raise ValueError("cos and sin must be two (n_pos, rotary_dim / 2) tables")
        n_pos, rot = cos.shape[0], 2 * cos.shape[1]
        pp = _plain(positions, "positions", device, torch.int32, (B, S))
    elif positions is not None:
        raise ValueError("positions need cos and sin tables")
    return qp, qs, kp, ks, wq, wk, int(f32), cp, sp, pp, (B, S, H, Hk, D, rot, n_pos)


def cpattn_qk_norm_rope(q, k=None, q_weight=None, k_weight=None, cos=None, sin=None, positions=None, eps=1e-6,
                        interleaved=True, pos0=0, q_out=None, k_out=None, stream=None):
    """RMS norm of q (B, S, H, D) and k (B, S, Hk, D) for each head, times the
    weights (D,) (both float32 or both bf16), with the position rotation by
    cos / sin (n_pos, rotary_dim / 2) float32 in the same pass.  Views whose
    heads' elements are consecutive are taken as they are.  `positions` (B, S)
    int32 picks each token's table row (default pos0 + s); `interleaved` pairs
    elements (2i, 2i + 1), else (i, i + rotary_dim / 2).  q_out / k_out may be
    q / k.  Returns (q_out, k_out)."""
    device = torch.cuda.current_device()
    qp, qs, kp, ks, wq, wk, f32, cp, sp, pp, sizes = _norm_rope_args(q, k, q_weight, k_weight, cos, sin, positions,
                                                                     device)
    if q_out is None:
        q_out = _new(q, q.shape, q.dtype, stream)
    if k_out is None and k is not None:
        k_out = _new(k, k.shape, k.dtype, stream)
    qop, qos = _view(q_out, "q_out", device, q.shape)
    kop, kos = (None, None) if k is None else _view(k_out, "k_out", device, k.shape)
    _check(_native.load().cpattn_qk_norm_rope(qp, qs, kp, ks, wq, wk, f32, cp, sp, pp, qop, qos, kop, kos, *sizes,
                                              pos0, interleaved, eps, _raw_stream(stream, device)),
           "cpattn_qk_norm_rope")
    return q_out, k_out


def cpattn_qk_norm_rope_backward_workspace_bytes(D) -> int:
    return int(_native.load().cpattn_qk_norm_rope_backward_workspace_bytes(D))


def cpattn_qk_norm_rope_backward(q, k, dq_out, dk_out, q_weight=None, k_weight=None, cos=None, sin=None,
                                 positions=None, eps=1e-6, interleaved=True, pos0=0, dq=None, dk=None,
                                 want_weights=True, workspace=None, stream=None):
    """Gradient of cpattn_qk_norm_rope from its inputs and the gradients of its
    outputs; returns (dq, dk, dq_weight, dk_weight), the last two in the
    weights' type (None where there is no weight, or want_weights is False).
    dq / dk may be dq_out / dk_out."""
    device = torch.cuda.current_device()
    qp, qs, kp, ks, wq, wk, f32, cp, sp, pp, sizes = _norm_rope_args(q, k, q_weight, k_weight, cos, sin, positions,
                                                                     device)
    D = q.shape[3]
    gqp, gqs = _view(dq_out, "dq_out", device, q.shape)
    gkp, gks = (None, None) if k is None else _view(dk_out, "dk_out", device, k.shape)
    dq = _new(q, q.shape, q.dtype, stream) if dq is None else dq
    dk = _new(q, k.shape, k.dtype, stream) if dk is None and k is not None else dk
    dqw = _new(q, (D,), q_weight.dtype, stream) if want_weights and q_weight is not None else None
    dkw = _new(q, (D,), k_weight.dtype, stream) if want_weights and k_weight is not None and k is not None else None
    if workspace is None and (dqw is not None or dkw is not None):
        workspace = _new(q, (cpattn_qk_norm_rope_backward_workspace_bytes(D),), torch.uint8, stream, returned=False)
    dqp, dqs = _view(dq, "dq", device, q.shape)
    dkp, dks = (None, None) if k is None else _view(dk, "dk", device, k.shape)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_native.load().cpattn_qk_norm_rope_backward(
        qp, qs, kp, ks, gqp, gqs, gkp, gks, wq, wk, f32, cp, sp, pp, dqp, dqs, dkp, dks,
        None if dqw is None else dqw.data_ptr(), None if dkw is None else dkw.data_ptr(), *sizes, pos0, interleaved,
        eps, _ptr(workspace), nbytes, _raw_stream(stream, device)), "cpattn_qk_norm_rope_backward")
    return dq, dk, dqw, dkw


def _cross_args(q, k, v, kv_lens, device):
    """The checked q, k, v and lengths of a cross-attention call, and its sizes."""
    qp, qs = _view(q, "q", device)
    B, Sq, H, D = q.shape
    kp, ks = _view(k, "k", device)
    Skv, Hk = k.shape[1], k.shape[2]
    if k.shape[0] != B or k.shape[3] != D:
        raise ValueError(f"k must be (B, Skv, Hk, D) with q's B and D, got {tuple(k.shape)}")
    vp, vs = _view(v, "v", device, k.shape)
    lp = _plain(kv_lens, "kv_lens", device, torch.int32, (B,))
    return qp, qs, kp, ks, vp, vs, lp, (B, H, Hk, Sq, Skv, D)


def cpattn_cross_attention(q, k, v, kv_lens=None, out=None, lse=None, want_lse=True, stream=None):
    """Attention of q (B, Sq, H, D) to an encoder's states k, v (B, Skv, Hk, D)
    of another length, H a multiple of Hk; kv_lens (B,) int32 on the GPU: each
    batch element's valid states (default all).  Views whose heads' elements
    are consecutive are taken as they are.  Returns (out, lse (B, H, Sq))."""
    device = torch.cuda.current_device()
    qp, qs, kp, ks, vp, vs, lp, sizes = _cross_args(q, k, v, kv_lens, device)
    B, H, _, Sq, _, _ = sizes
    if out is None:
        out = _new(q, q.shape, q.dtype, stream)
    if lse is None and want_lse:
        lse = _new(q, (B, H, Sq), torch.float32, stream)
    op = _plain(out, "out", device, torch.bfloat16, q.shape)
    _check(_native.load().cpattn_cross_attention(qp, qs, kp, ks, vp, vs, op,
                                                 _plain(lse, "lse", device, torch.float32, (B, H, Sq)), lp, *sizes,
                                                 _raw_stream(stream, device)), "cpattn_cross_attention")
    return out, lse


def cpattn_cross_attention_backward_ds_bytes(H, Hk, Sq, Skv) -> int:
    return int(_native.load().cpattn_cross_attention_backward_ds_bytes(H, Hk, Sq, Skv))


def cpattn_cross_attention_backward_workspace_bytes(B, H, Hk, Sq, Skv, D) -> int:
    return int(_native.load().cpattn_cross_attention_backward_workspace_bytes(B, H, Hk, Sq, Skv, D))


# dS that the least workspace of the cross-attention backward holds: a pair's, or
# this much of it (kCrossLeastDs of the library).
_CROSS_DS_LEAST = 256 << 20


def cross_backward_workspace_bytes(B, H, Hk, Sq, Skv, D, ds_budget=None) -> int:
    """Bytes of the workspace the cross-attention backward's binding
    allocates: dS of as many (batch element, key head) pairs as fit ds_budget
    (default BACKWARD_DS_BUDGET); of a part of one pair where it does not fit,
    but at least of a pair or 256 MB; and the rest."""
    pair = cpattn_cross_attention_backward_ds_bytes(H, Hk, Sq, Skv)
    budget = BACKWARD_DS_BUDGET if ds_budget is None else int(ds_budget)
    least = min(pair, _CROSS_DS_LEAST)
    ds = min(B * Hk, budget // pair) * pair if 0 < pair <= budget else max(budget, least)
    return cpattn_cross_attention_backward_workspace_bytes(B, H, Hk, Sq, Skv, D) + max(0, ds - least)


# Scratch up to here is allocated whatever the device's free memory.
_CROSS_DS_UNASKED = 256 << 20


def _cross_allocation_budget(device, every, ds_budget):
    """The dS budget for a workspace the cross-attention backward's binding
    allocates itself (`every`: dS of all pairs): the given one, or by default
    BACKWARD_DS_BUDGET, of which no more is newly taken from the device than
    half its free memory.  Memory that torch holds and does not use, such as the
    last step's scratch, is taken already; and the device is asked only for more
    than that, since the question can stall for milliseconds where other
    processes use the driver (training steps of 1.6 ms took 2 to 4 so, asked
    every time)."""
    if ds_budget is not None:
        return int(ds_budget)
    want = min(every, BACKWARD_DS_BUDGET)
    if want > _CROSS_DS_UNASKED:
        held = torch.cuda.memory_stats_as_nested_dict(device)
        idle = held["reserved_bytes"]["all"]["current"] - held["allocated_bytes"]["all"]["current"]
        if want > idle:
            free, _ = torch.cuda.mem_get_info(device)
            want = min(want, max(_CROSS_DS_UNASKED, idle, free // 2))
    return want


def cpattn_cross_attention_backward(q, k, v, out, lse, dout, kv_lens=None, dq=None, dk=None, dv=None, workspace=None,
                                    stream=None, ds_budget=None):
    """Gradient of cpattn_cross_attention from the forward's output and LSE;
    returns (dq, dk, dv), contiguous bf16.  An allocated workspace holds up to
    ds_budget bytes of dS scratch (default BACKWARD_DS_BUDGET, capped at half the
    device's free memory where it is more than 256 MB; halved where memory does
    not allow it), and at least 256 MB or one (batch element, key head) pair's;
    a pair that does not fit is done in ranges of its queries."""
    device = torch.cuda.current_device()
    qp, qs, kp, ks, vp, vs, lp, sizes = _cross_args(q, k, v, kv_lens, device)
    B, H, Hk, Sq, Skv, D = sizes
    dq = _new(q, q.shape, q.dtype, stream) if dq is None else dq
    dk = _new(q, k.shape, k.dtype, stream) if dk is None else dk
    dv = _new(q, v.shape, v.dtype, stream) if dv is None else dv
    if lse is None:
        raise ValueError("lse is required")
    ptrs = [_plain(t, name, device, torch.bfloat16, shape)
            for t, name, shape in ((out, "out", q.shape), (dout, "dout", q.shape), (dq, "dq", q.shape),
                                   (dk, "dk", k.shape), (dv, "dv", k.shape))]
    sp = _plain(lse, "lse", device, torch.float32, (B, H, Sq))
    if workspace is None:
        budget = _cross_allocation_budget(device, B * Hk * cpattn_cross_attention_backward_ds_bytes(H, Hk, Sq, Skv),
                                          ds_budget)
        least = cross_backward_workspace_bytes(B, H, Hk, Sq, Skv, D, 0)
        while workspace is None:
            nbytes = cross_backward_workspace_bytes(B, H, Hk, Sq, Skv, D, budget)
            try:
                workspace = _new(q, (nbytes,), torch.uint8, stream, returned=False)
            except torch.OutOfMemoryError:     # fewer pairs at once
                if nbytes == least:
                    raise
                budget //= 2
    _check(_native.load().cpattn_cross_attention_backward(
        qp, qs, kp, ks, vp, vs, ptrs[0], sp, ptrs[1], lp, *ptrs[2:], *sizes, _ptr(workspace),
        workspace.numel() * workspace.element_size(), _raw_stream(stream, device)), "cpattn_cross_attention_backward")
    return dq, dk, dv


# Size of the library-held scratch of cpattn_ulysses_attention_noalloc
# (CPATTN_NOALLOC_SCRATCH_BYTES in cpattn.h).
NOALLOC_SCRATCH_BYTES = 64 << 20


def cpattn_ulysses_attention_noalloc(q, k, v, B, S, H, D, degree, seq_splits=None, head_splits=None, out=None,
                                     lse=None, want_lse=True, stream=None):
    """Ulysses attention for callers that cannot allocate device memory when
    they call: the scratch lives in a fixed 64 MiB array inside the library
    (see cpattn.h).  `out` and `lse` should be passed in by such callers; when
    omitted they are allocated here with torch for convenience.  Concurrent
    calls on different streams race on the shared scratch."""
    out = torch.empty_like(q) if out is None else out
    if lse is None and want_lse:
        lse = torch.empty((B, H, S), dtype=torch.float32, device=q.device)
    for t, name in ((q, "q"), (k, "k"), (v, "v"), (out, "out")):
        _need(t, _flat_numel(B, S, H, D), torch.bfloat16, name)
    _need(lse, B * H * S, torch.float32, "lse")
    _check(_native.load().cpattn_ulysses_attention_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, S,
                                                           D, int(degree), _native.int_array(seq_splits),
                                                           _native.int_array(head_splits), _stream(stream)),
           "cpattn_ulysses_attention_noalloc")
    return out, lse


def cpattn_ring_chunk_attention(q, k, v, Skv, out, lse, prev_out=None, q_pos0=0, kv_pos0=0, causal=False,
                                kv_batch_rows=None, stream=None):
    """One ring step of one rank over separate buffers, merged into its running
    result.  q (B, Sq, H, D) bf16; k, v (B, kv_batch_rows, H, D) bf16 whose
    first Skv rows per batch element are the chunk; out float32 (an
    intermediate state) or bf16 (the final output), (B, Sq, H, D); lse
    (B, H, Sq) float32, holding prev_out's LSE on entry when prev_out (float32,
    may be `out` itself) is given.  Returns (out, lse)."""
    B, Sq, H, D = _bshd(q)
    rows = k.shape[1] if kv_batch_rows is None else int(kv_batch_rows)
    for t, name in ((k, "k"), (v, "v")):
        _need(t, B * rows * H * D, torch.bfloat16, name)
    if out.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("out must be float32 or bf16")
    _need(out, B * Sq * H * D, out.dtype, "out")
    _need(lse, B * H * Sq, torch.float32, "lse")
    _need(prev_out, B * Sq * H * D, torch.float32, "prev_out")
    _check(_native.load().cpattn_ring_chunk_attention(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                                                      _ptr(prev_out), B, H, Sq, int(Skv), rows, D, int(q_pos0),
                                                      int(kv_pos0), int(bool(causal)),
                                                      int(out.dtype == torch.float32), _stream(stream)),
           "cpattn_ring_chunk_attention")
    return out, lse


def cpattn_gathered_kv_attention(q, k, v, degree, rank, kv_lens=None, out=None, lse=None, want_lse=True,
                                 causal=False, stream=None):
    """Attention of one rank's query shard q (B, kv_lens[rank], H, D) against
    `degree` gathered K/V chunks, k and v (degree, B, kv_batch_rows, H, D)
    bf16, chunk c holding kv_lens[c] valid rows.  Returns (out, lse)."""
    B, Sq, H, D = _bshd(q)
    if k.dim() != 5 or k.shape[0] != degree or k.shape[1] != B:
        raise ValueError("k and v must be (degree, B, kv_batch_rows, H, D)")
    rows = k.shape[2]
    for t, name in ((k, "k"), (v, "v")):
        _need(t, degree * B * rows * H * D, torch.bfloat16, name)
    out = torch.empty_like(q) if out is None else out
    if lse is None and want_lse:
        lse = torch.empty((B, H, Sq), dtype=torch.float32, device=q.device)
    _need(out, B * Sq * H * D, torch.bfloat16, "out")
    _need(lse, B * H * Sq, torch.float32, "lse")
    _check(_native.load().cpattn_gathered_kv_attention(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, D,
                                                       int(degree), _native.int_array(kv_lens), rows, int(rank),
                                                       int(bool(causal)), _stream(stream)),
           "cpattn_gathered_kv_attention")
    return out, lse


def cpattn_rank_buffer_attention(q, k, v, B, S, H, D, degree, seq_splits=None, out=None, lse=None, want_lse=True,
                                 causal=False, stream=None):
    """Attention over a sequence held as rank buffers (B, S_u, H, D)
    concatenated (flat bf16), the layout an all-to-all delivers; every query
    attends all S keys.  Returns (out in the same layout, lse (B, H, S))."""
    out = torch.empty_like(q) if out is None else out
    if lse is None and want_lse:
        lse = torch.empty((B, H, S), dtype=torch.float32, device=q.device)
    for t, name in ((q, "q"), (k, "k"), (v, "v"), (out, "out")):
        _need(t, _flat_numel(B, S, H, D), torch.bfloat16, name)
    _need(lse, B * H * S, torch.float32, "lse")
    _check(_native.load().cpattn_rank_buffer_attention(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, S, D,
                                                       int(degree), _native.int_array(seq_splits),
                                                       int(bool(causal)), _stream(stream)),
           "cpattn_rank_buffer_attention")
    return out, lse


def cpattn_front_loaded_splits(total, parts):
    arr = (ctypes.c_int * max(1, int(parts)))()
    _check(_native.load().cpattn_front_loaded_splits(int(total), int(parts), arr), "cpattn_front_loaded_splits")
    return [int(arr[i]) for i in range(int(parts))]


EXCHANGE_MODES = {"ring": 0, "ulysses": 1, "kv_gather": 2}


def cpattn_exchange_bytes(mode, B, H, S, D, degree, seq_splits=None, head_splits=None, elem_bytes=2):
    """Per-rank (send, recv) bytes of one attention call under an exchange
    ('ring', 'ulysses' or 'kv_gather'); host arithmetic only."""
    send = (ctypes.c_ulonglong * int(degree))()
    recv = (ctypes.c_ulonglong * int(degree))()
    _check(_native.load().cpattn_exchange_bytes(EXCHANGE_MODES[mode], B, H, S, D, elem_bytes, int(degree),
                                                _native.int_array(seq_splits), _native.int_array(head_splits),
                                                send, recv), "cpattn_exchange_bytes")
    return [int(x) for x in send], [int(x) for x in recv]


class _ExchangeEnv(ctypes.Structure):
    _fields_ = [("link_gbs", ctypes.c_double), ("attn_tflops", ctypes.c_double), ("hbm_gbs", ctypes.c_double),
                ("causal", ctypes.c_int)]


class _ExchangePlan(ctypes.Structure):
    _fields_ = [("seconds", ctypes.c_double * 3), ("recv_bytes", ctypes.c_ulonglong * 3),
                ("resident_bytes", ctypes.c_ulonglong * 3), ("flops", ctypes.c_double * 3), ("best", ctypes.c_int)]


def cpattn_plan_exchange(B, H, S, D, degree, link_gbs, attn_tflops, hbm_gbs, causal=False, seq_splits=None,
                         head_splits=None, elem_bytes=2):
    """Exchange-selection model for one attention call over `degree` ranks.
    Returns {"best": mode name, mode name: {"seconds" (None if infeasible),
    "recv_bytes", "resident_bytes", "flops"}}; host arithmetic only."""
    env = _ExchangeEnv(float(link_gbs), float(attn_tflops), float(hbm_gbs), 1 if causal else 0)
    plan = _ExchangePlan()
    _check(_native.load().cpattn_plan_exchange(B, H, S, D, elem_bytes, int(degree), _native.int_array(seq_splits),
                                               _native.int_array(head_splits), ctypes.byref(env),
                                               ctypes.byref(plan)), "cpattn_plan_exchange")
    names = {v: k for k, v in EXCHANGE_MODES.items()}
    out = {"best": names[plan.best]}
    for m, name in names.items():
        out[name] = {"seconds": None if plan.seconds[m] < 0 else float(plan.seconds[m]),
                     "recv_bytes": int(plan.recv_bytes[m]), "resident_bytes": int(plan.resident_bytes[m]),
                     "flops": float(plan.flops[m])}
    return out


def cpattn_device_status(stream=None):
    """Synchronise the stream and read-and-clear the device status word.
    Returns (status, code)."""
    code = ctypes.c_uint(0)
    st = _native.load().cpattn_device_status(_stream(stream), ctypes.byref(code))
    return int(st), int(code.value)


def cpattn_debug_wait_timeout(timeout_us, stream=None):
    _check(_native.load().cpattn_debug_wait_timeout(int(timeout_us), _stream(stream)), "cpattn_debug_wait_timeout")
