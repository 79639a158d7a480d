"""Exact IO-aware softmax attention for GB300 (sm_103a).

O = softmax(scale · Q Kᵀ) V computed tile by tile with an online softmax
("LLM Systems 22: Flash Attention", section 3.1; "08 · FlashAttention",
section 二); the backward recomputes P from the saved log-sum-exp
("LLM Systems 22", section 3.2).  Tensors are bf16 [B, N, H, d] (packed
variable-length batches: [T, H, d] with cu_seqlens); d is 64 or 128.

The compute runs in the hand-written kernels of libfa_gb300.so behind the C
ABI in include/fa.h; PyTorch only provides device memory and streams.  This
module allocates outputs and workspace and calls the binding.
"""
from __future__ import annotations

import contextlib
from typing import NamedTuple

import torch

from . import _binding
from ._binding import (  # noqa: F401  (C-ABI names)
    FaError,
    fa_decode_workspace_bytes,
    fa_fwd_decode,
    fa_bwd,
    fa_bwd_grouped,
    fa_bwd_grouped_workspace_bytes,
    fa_bwd_varlen,
    fa_bwd_varlen_workspace_bytes,
    fa_bwd_workspace_bytes,
    fa_cache8_store,
    fa_cta_order,
    fa_decode_cache8_workspace_bytes,
    fa_fwd,
    fa_fwd_decode_cache8,
    fa_fwd_grouped,
    fa_fwd_varlen,
    fa_get_device_error,
    fa_selftest_wait_timeout,
    fa_set_kernel_events,
)

__all__ = [
    "attention_forward", "attention_backward", "attention_forward_varlen", "attention_backward_varlen",
    "flash_attention", "FaError", "fa_fwd", "fa_bwd", "fa_fwd_varlen", "fa_bwd_varlen",
    "fa_bwd_workspace_bytes", "fa_bwd_varlen_workspace_bytes", "fa_get_device_error", "load_library",
    "attention_decode", "fa_fwd_decode", "fa_decode_workspace_bytes",
    "attention_forward_grouped", "attention_backward_grouped", "flash_attention_grouped", "fa_fwd_grouped",
    "fa_bwd_grouped", "fa_bwd_grouped_workspace_bytes", "Cache8", "cache8_alloc", "cache8_store",
    "attention_decode_cache8", "fa_cache8_store", "fa_fwd_decode_cache8", "fa_decode_cache8_workspace_bytes",
]


def load_library():
    """Load libfa_gb300.so; raises RuntimeError if it has not been built."""
    return _binding.lib()


def attention_forward(q, k, v, causal: bool = False, scale=None, stream=None):
    """Returns (o [B,N,H,d] bf16, lse [B,H,N] fp32)."""
    B, N, H, d = q.shape
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), device=q.device, dtype=torch.float32)
    fa_fwd(q, k, v, o, lse, causal, scale, stream)
    return o, lse


def attention_decode(q, k, v, causal: bool = False, scale=None, stream=None, workspace=None):
    """Decode: q [B,Nq,H,d] (Nq <= 8 newest tokens) against the cache k, v
    [B,Nk,H,d].  Returns (o [B,Nq,H,d] bf16, lse [B,H,Nq] fp32).  causal: the
    new tokens are the cache's last Nq positions (query i sees keys
    j <= Nk - Nq + i)."""
    B, Nq, H, d = q.shape
    Nk = k.shape[1]
    o = torch.empty_like(q)
    lse = torch.empty((B, H, Nq), device=q.device, dtype=torch.float32)
    if workspace is None:
        workspace = torch.empty(max(fa_decode_workspace_bytes(B, H, Nq, Nk, d), 16), device=q.device,
                                dtype=torch.uint8)
    fa_fwd_decode(q, k, v, o, lse, workspace, causal, scale, stream)
    return o, lse


def attention_backward(q, k, v, o, dout, lse, causal: bool = False, scale=None, stream=None, workspace=None):
    """Returns (dq, dk, dv), each [B,N,H,d] bf16."""
    B, N, H, d = q.shape
    if workspace is None:
        workspace = torch.empty(fa_bwd_workspace_bytes(B, H, N, d), device=q.device, dtype=torch.uint8)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, workspace, causal, scale, stream)
    return dq, dk, dv


def attention_forward_varlen(q, k, v, cu_seqlens, max_seqlen: int, causal: bool = False, scale=None, stream=None):
    """Packed batch: q/k/v [T,H,d]; returns (o [T,H,d], lse [nseq,H,max_seqlen])."""
    T, H, d = q.shape
    o = torch.empty_like(q)
    lse = torch.empty((cu_seqlens.numel() - 1, H, max_seqlen), device=q.device, dtype=torch.float32)
    fa_fwd_varlen(q, k, v, o, lse, cu_seqlens, max_seqlen, causal, scale, stream)
    return o, lse


def attention_backward_varlen(q, k, v, o, dout, lse, cu_seqlens, max_seqlen: int, causal: bool = False,
                              scale=None, stream=None, workspace=None):
    T, H, d = q.shape
    nseq = cu_seqlens.numel() - 1
    if workspace is None:
        workspace = torch.empty(fa_bwd_varlen_workspace_bytes(T, nseq, max_seqlen, H, d), device=q.device,
                                dtype=torch.uint8)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    fa_bwd_varlen(q, k, v, o, dout, lse, dq, dk, dv, workspace, cu_seqlens, max_seqlen, causal, scale, stream)
    return dq, dk, dv


class _FlashAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, causal, scale):
        o, lse = attention_forward(q, k, v, causal, scale)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.causal, ctx.scale = causal, scale
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, o, lse = ctx.saved_tensors
        dq, dk, dv = attention_backward(q, k, v, o, do.contiguous(), lse, ctx.causal, ctx.scale)
        return dq, dk, dv, None, None


def flash_attention(q, k, v, causal: bool = False, scale=None):
    """Autograd-aware attention over bf16 [B,N,H,d] CUDA tensors."""
    return _FlashAttention.apply(q, k, v, causal, scale)


# ---------------------------------------------------------------------------
# Grouped heads over packed batches: H query heads share Hk key/value heads.
# ---------------------------------------------------------------------------
# Each call first goes to its compiled counterpart, which returns None where
# something is not in order, or where PyTorch's operations are being recorded; the
# Python path then runs or says what is wrong.
_tracing = torch._C._get_tracing_state
_dispatch_mode, _PROXY = torch._C._get_dispatch_mode, torch._C._TorchDispatchModeKey.PROXY


def _refuse_trace(name: str, recordable: bool = False) -> None:
    """A recorder of PyTorch's operations (torch.jit.trace; torch.fx's make_fx)
    would take down the outputs' allocation and not the kernel: refused, but for
    a call that torch.jit.trace can record as a Python function."""
    if _dispatch_mode(_PROXY) is not None or _tracing() is not None and not recordable:
        raise RuntimeError(f"{name} cannot be recorded by torch.jit.trace or make_fx (torch.jit.trace can record "
                           "flash_attention_grouped)")


def _on_stream(stream, t):
    """What a call on a stream of its own allocates belongs to that stream, so
    that its memory is not handed to another one while the kernels still use
    it.  Refuses a stream of another device than the tensor's."""
    if stream is None:
        return contextlib.nullcontext()
    _binding._stream_of(stream, t.get_device())
    return torch.cuda.stream(stream)


def attention_forward_grouped(q, k, v, cu_seqlens, max_seqlen: int, causal: bool = False, scale=None, stream=None):
    """Packed batch with grouped heads: q [T,H,d], k and v [T,Hk,d] (H a
    multiple of Hk; slices of one wider projection are taken as they are).
    Returns (o [T,H,d] bf16, lse [H,T] fp32); rows behind the last sequence
    get o = 0, lse = -inf."""
    if stream is None:
        out = _binding.native().forward_grouped(q, k, v, cu_seqlens, max_seqlen, causal, scale)
        if out is not None:
            return out
    _refuse_trace("attention_forward_grouped")
    with _on_stream(stream, q):
        return _forward_grouped(_binding._grouped(q, k, v, cu_seqlens), q, k, v, cu_seqlens, max_seqlen, causal, scale)


def _forward_grouped(checked, q, k, v, cu_seqlens, max_seqlen, causal, scale):
    T, H, d = q.shape
    o = torch.empty((T, H, d), device=q.device, dtype=torch.bfloat16)
    lse = torch.empty((H, T), device=q.device, dtype=torch.float32)
    _binding._launch_fwd_grouped(checked, q, k, v, o, lse, cu_seqlens, max_seqlen, causal, scale, None, True)
    return o, lse


def attention_backward_grouped(q, k, v, o, dout, lse, cu_seqlens, max_seqlen: int, causal: bool = False, scale=None,
                               stream=None, workspace=None):
    """Returns (dq [T,H,d], dk, dv [T,Hk,d]), zero in rows behind the last
    sequence.  dk and dv are summed over the query heads that share them."""
    if stream is None and workspace is None:
        out = _binding.native().backward_grouped(q, k, v, cu_seqlens, max_seqlen, causal, scale, o, dout, lse)
        if out is not None:
            return out
    _refuse_trace("attention_backward_grouped")
    with _on_stream(stream, q):
        return _backward_grouped(_binding._grouped(q, k, v, cu_seqlens), q, k, v, o, dout, lse, cu_seqlens, max_seqlen,
                                 causal, scale, workspace)


def _backward_grouped(checked, q, k, v, o, dout, lse, cu_seqlens, max_seqlen, causal, scale, workspace):
    dev, T, H, Hk, d, nseq = checked[:6]
    device = q.device
    if workspace is None:
        n = fa_bwd_grouped_workspace_bytes(nseq, max_seqlen, T, H, Hk, d, causal)
        workspace = torch.empty(n, device=device, dtype=torch.uint8)
    else:
        n = _binding._nbytes(workspace, dev)
    dq = torch.empty((T, H, d), device=device, dtype=torch.bfloat16)
    dk = torch.empty((T, Hk, d), device=device, dtype=torch.bfloat16)
    dv = torch.empty((T, Hk, d), device=device, dtype=torch.bfloat16)
    _binding._launch_bwd_grouped(checked, q, k, v, o, dout, lse, dq, dk, dv, workspace, n, cu_seqlens, max_seqlen, causal,
                                 scale, None, True)
    return dq, dk, dv


class _FlashAttentionGrouped(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, max_seqlen, causal, scale):
        checked = _binding._grouped(q, k, v, cu_seqlens)
        o, lse = _forward_grouped(checked, q, k, v, cu_seqlens, max_seqlen, causal, scale)
        ctx.save_for_backward(q, k, v, o, lse, cu_seqlens)
        ctx.args = max_seqlen, causal, scale
        return o

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, do):
        q, k, v, o, lse, cu_seqlens = ctx.saved_tensors
        max_seqlen, causal, scale = ctx.args
        checked = _binding._grouped(q, k, v, cu_seqlens)  # saved tensors may come back with other strides
        dq, dk, dv = _backward_grouped(checked, q, k, v, o, do.contiguous(), lse, cu_seqlens, max_seqlen, causal, scale, None)
        return dq, dk, dv, None, None, None, None


def flash_attention_grouped(q, k, v, cu_seqlens, max_seqlen: int, causal: bool = False, scale=None):
    """Autograd-aware attention with grouped heads over a packed batch:
    q [T,H,d], k and v [T,Hk,d], cu_seqlens int32 [nseq+1] on the device,
    max_seqlen the longest sequence.  Returns o [T,H,d], zeros in rows behind
    the last sequence.  Differentiable once.  To capture a training step into
    a CUDA graph, run it outside first and let go of that run's graph (its
    outputs and losses): PyTorch cannot capture a backward pass into leaves
    that a graph recorded outside still holds.  torch.jit.trace records it as
    one operation (make_fx is refused; the calls that are not autograd functions
    refuse both)."""
    o = _binding.native().flash_attention_grouped(q, k, v, cu_seqlens, max_seqlen, causal, scale)
    if o is not None:
        return o
    _refuse_trace("flash_attention_grouped", recordable=True)
    return _FlashAttentionGrouped.apply(q, k, v, cu_seqlens, max_seqlen, causal, scale)


# ---------------------------------------------------------------------------
# Paged key/value cache in 8 bits.
# ---------------------------------------------------------------------------
class Cache8(NamedTuple):
    """Pools of e4m3 pages [num_blocks, Hk, block, d] and their scales fp32
    [num_blocks, Hk] (powers of two; the value of a code is code · scale)."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


def cache8_alloc(num_blocks: int, Hk: int, block: int, d: int, device="cuda") -> Cache8:
    """An empty cache of num_blocks pages of `block` tokens (16, 32, 64 or 128)."""
    pages = [torch.zeros((num_blocks, Hk, block, d), device=device, dtype=torch.uint8).view(torch.float8_e4m3fn)
             for _ in range(2)]
    return Cache8(*pages, *(torch.ones((num_blocks, Hk), device=device) for _ in range(2)))


def cache8_store(k, v, cache: Cache8, block_table, cu_seqlens, start, max_new: int, stream=None) -> None:
    """Appends new tokens to the cache: rows cu_seqlens[b] .. cu_seqlens[b+1]-1
    of k, v [T,Hk,d] become tokens start[b], start[b]+1, ... of sequence b,
    in the pages block_table [B,cols] names (int32, as cu_seqlens [B+1] and
    start [B]); max_new is the largest number of new tokens of a sequence."""
    if stream is None and _binding.native().cache8_store(k, v, cache, block_table, cu_seqlens, start, max_new):
        return
    _refuse_trace("cache8_store")
    fa_cache8_store(k, v, cache, block_table, cu_seqlens, start, max_new, stream)


def attention_decode_cache8(q, cache: Cache8, block_table, seqlens, max_seqlen: int, causal: bool = False, scale=None,
                            stream=None, workspace=None):
    """Decode over the 8-bit paged cache: q [B,Nq,H,d] (Nq <= 8 newest tokens),
    seqlens int32 [B] cached tokens (the new ones among them; 0 for an empty
    slot), max_seqlen at least every length.  Returns (o [B,Nq,H,d] bf16, lse
    [B,H,Nq] fp32).  causal as in attention_decode."""
    if stream is None and workspace is None:
        out = _binding.native().decode_cache8(q, cache, block_table, seqlens, max_seqlen, causal, scale)
        if out is not None:
            return out
    _refuse_trace("attention_decode_cache8")
    checked = _binding._decode_cache8(q, cache, block_table, seqlens)
    dev, B, Nq, H, d, _, Hk = checked[:7]
    with _on_stream(stream, q):
        o = torch.empty_like(q)
        lse = torch.empty((B, H, Nq), device=q.device, dtype=torch.float32)
        if workspace is None:
            n = fa_decode_cache8_workspace_bytes(B, Nq, H, Hk, max_seqlen, d)
            workspace = torch.empty(n, device=q.device, dtype=torch.uint8)
        _binding._launch_decode_cache8(checked, q, cache, block_table, seqlens, o, lse, workspace,
                                       _binding._nbytes(workspace, dev), max_seqlen, causal, scale, None)
    return o, lse
