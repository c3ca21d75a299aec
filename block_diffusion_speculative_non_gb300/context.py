"""Binding of the operators on a context store: attention over a shared prefix, collected attention weight, eviction.
Sizes and layouts are those of include/fpd.h.

The operators are short calls (a few microseconds on the GPU), so the checks here are one comparison chain per tensor and
the current stream is asked for once.
"""
from __future__ import annotations

import ctypes

import torch

from . import SharedContext, _check, _ptr, _stream, lib

_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _arg(t, dtype, n, what, dev=None):
    """Device address of a tensor that must be contiguous, of `dtype`, on the current device `dev` and hold at least n
    elements; an int address or None is passed on."""
    if t is None or t.__class__ is int:
        return t
    if t.dtype is dtype and t.numel() >= n and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    if t.dtype is not dtype:
        raise ValueError(f"{what} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous (row-major)")
    if t.numel() < n:
        raise ValueError(f"{what} holds {t.numel()} elements, the call needs {n}")
    raise ValueError(f"{what} is on {t.device}, the current device is cuda:{dev}")


def _here(stream):
    """(current device, address of the stream)"""
    dev = torch.cuda.current_device()
    return dev, torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def fpd_shared_attention_workspace_bytes(batch, block_len, n_q_heads, n_kv_heads, head_dim, prefix_cap, t_cap) -> int:
    return int(lib().fpd_shared_attention_workspace_bytes(batch, block_len, n_q_heads, n_kv_heads, head_dim, prefix_cap,
                                                          t_cap))


def fpd_shared_attention(batch, block_len, n_q_heads, n_kv_heads, head_dim, layer, q, k_blk, v_blk, prefix_store,
                         prefix_cap, prefix_len, kv_store, t_cap, ctx_len, out, lse, workspace, workspace_bytes,
                         stream=None):
    """Attention of a batch over [shared prefix ; own context ; block] of one layer; out and lse are written."""
    n, pos = batch * block_len * n_q_heads, 2 * n_kv_heads * head_dim
    blk = batch * n_kv_heads * block_len * head_dim
    dev, st = _here(stream)
    _check(lib().fpd_shared_attention(
        batch, block_len, n_q_heads, n_kv_heads, head_dim, layer, _arg(q, _BF16, n * head_dim, "q", dev),
        _arg(k_blk, _BF16, blk, "k_blk", dev), _arg(v_blk, _BF16, blk, "v_blk", dev),
        _arg(prefix_store, _BF16, (layer + 1) * prefix_cap * pos, "prefix_store", dev), prefix_cap,
        _arg(prefix_len, _I32, 1, "prefix_len", dev),
        _arg(kv_store, _BF16, (layer + 1) * batch * t_cap * pos, "kv_store", dev), t_cap,
        _arg(ctx_len, _I32, batch, "ctx_len", dev), _arg(out, _BF16, n * head_dim, "out", dev),
        _arg(lse, _F32, n, "lse", dev), _arg(workspace, _U8, workspace_bytes, "workspace", dev), workspace_bytes, st),
           "fpd_shared_attention")


def fpd_context_weights(batch, block_len, n_q_heads, n_kv_heads, head_dim, layer, q, lse, kv_store, t_cap, ctx_len,
                        weights, accumulate=False, stream=None):
    """weights[layer] (+)= the attention weight every context position collects from the rows of q."""
    n, at = batch * block_len * n_q_heads, (layer + 1) * batch * n_kv_heads * t_cap
    dev, st = _here(stream)
    _check(lib().fpd_context_weights(
        batch, block_len, n_q_heads, n_kv_heads, head_dim, layer, _arg(q, _BF16, n * head_dim, "q", dev),
        _arg(lse, _F32, n, "lse", dev), _arg(kv_store, _BF16, at * 2 * head_dim, "kv_store", dev), t_cap,
        _arg(ctx_len, _I32, batch, "ctx_len", dev), _arg(weights, _F32, at, "weights", dev), 1 if accumulate else 0, st),
           "fpd_context_weights")


def fpd_evict_workspace_bytes(n_layers, batch, n_kv_heads, budget) -> int:
    return int(lib().fpd_evict_workspace_bytes(n_layers, batch, n_kv_heads, budget))


def fpd_evict_context(n_layers, batch, n_kv_heads, head_dim, budget, recent, kv_store, t_cap, weights, ctx_len, out_store,
                      out_cap, out_weights, out_len, pos_offset, kept, workspace, workspace_bytes, stream=None):
    """Keeps the last `recent` positions and those with the largest weights, `budget` in all, of every request."""
    heads = n_layers * batch * n_kv_heads
    dev, st = _here(stream)
    _check(lib().fpd_evict_context(
        n_layers, batch, n_kv_heads, head_dim, budget, recent,
        _arg(kv_store, _BF16, heads * 2 * t_cap * head_dim, "kv_store", dev), t_cap,
        _arg(weights, _F32, heads * t_cap, "weights", dev), _arg(ctx_len, _I32, batch, "ctx_len", dev),
        _arg(out_store, _BF16, heads * 2 * out_cap * head_dim, "out_store", dev), out_cap,
        _arg(out_weights, _F32, heads * out_cap, "out_weights", dev), _arg(out_len, _I32, batch, "out_len", dev),
        _arg(pos_offset, _I32, batch, "pos_offset", dev), _arg(kept, _I32, heads * budget, "kept", dev),
        _arg(workspace, _U8, workspace_bytes, "workspace", dev), workspace_bytes, st), "fpd_evict_context")


def fpd_prepare_context_at(model, batch, total_rows, row_off, row_cnt, pos_start, pos_offset, feats, kv_store, t_cap,
                           workspace, workspace_bytes, stream=None):
    arr = (ctypes.c_void_p * len(feats))(*[_ptr(f) for f in feats])
    _check(lib().fpd_prepare_context_at(model, batch, total_rows, _ptr(row_off), _ptr(row_cnt), _ptr(pos_start),
                                        _ptr(pos_offset), arr, _ptr(kv_store), t_cap, _ptr(workspace), workspace_bytes,
                                        _stream(stream)), "fpd_prepare_context_at")


def fpd_shared_workspace_bytes(model, batch, max_block_len, prefix_cap, t_cap) -> int:
    return int(lib().fpd_shared_workspace_bytes(model, batch, max_block_len, prefix_cap, t_cap))


def shared_context(prefix_store=None, prefix_cap=0, prefix_len=None, kv_store=None, t_cap=0, ctx_len=None, pos_offset=None,
                   weights=None, prefix_weights=None, accumulate=False) -> SharedContext:
    """Build an fpd_shared_context; it keeps its tensors alive."""
    c = SharedContext(_ptr(prefix_store), prefix_cap, _ptr(prefix_len), _ptr(kv_store), t_cap, _ptr(ctx_len),
                      _ptr(pos_offset), _ptr(weights), _ptr(prefix_weights), int(bool(accumulate)))
    c._keep = (prefix_store, prefix_len, kv_store, ctx_len, pos_offset, weights, prefix_weights)
    return c


def fpd_draft_block_shared(model, batch, block_len, ctx: SharedContext, anchor, mask_id, hidden_out, layer_hidden,
                           workspace, workspace_bytes, stream=None):
    _check(lib().fpd_draft_block_shared(model, batch, block_len, ctypes.byref(ctx), _ptr(anchor), int(mask_id),
                                        _ptr(hidden_out), _ptr(layer_hidden), _ptr(workspace), workspace_bytes,
                                        _stream(stream)), "fpd_draft_block_shared")
