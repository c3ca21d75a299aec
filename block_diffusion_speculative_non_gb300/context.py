"""Binding of the operators on a context store: attention over a shared prefix, collected attention weight, eviction.
Sizes and layouts are those of include/fpd.h.

The operators are short calls (a few microseconds on the GPU), so their arguments are checked and handed over by the
compiled module `_calls` (csrc/py_calls.cpp); the rest goes through ctypes.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import SharedContext, _check, _stream, lib

_module = None


def _compiled():
    """The compiled calls, bound to the loaded library (raises when they have not been built for this PyTorch)."""
    global _module
    if _module is None:
        here = os.path.dirname(os.path.abspath(__file__))
        if not os.path.exists(os.path.join(here, "_calls.so")):
            raise RuntimeError(f"_calls.so not built in {here}; run __graft_entry__.build()")
        from . import _calls as m
        if m.torch_version != torch.__version__:
            raise RuntimeError(f"_calls.so was built for PyTorch {m.torch_version}, this is {torch.__version__}; "
                               "run __graft_entry__.build()")
        m.bind(*(ctypes.cast(getattr(lib(), f), ctypes.c_void_p).value
                 for f in ("fpd_shared_attention", "fpd_context_weights", "fpd_evict_context")))
        _module = m
    return _module


def _arg(t, dtype, n, what, dev=-1):
    """Device address of a tensor that must be contiguous, of `dtype`, on the current device `dev` and hold at least n
    elements; an int address or None is passed on."""
    return _compiled().arg(t, dtype, n, what, dev)


def _here(stream):
    """(address of the stream, current device)"""
    dev = torch._C._cuda_getDevice()
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream), dev


def fpd_shared_attention_workspace_bytes(batch, block_len, n_q_heads, n_kv_heads, head_dim, prefix_cap, t_cap) -> int:
    return int(lib().fpd_shared_attention_workspace_bytes(batch, block_len, n_q_heads, n_kv_heads, head_dim, prefix_cap,
                                                          t_cap))


def fpd_shared_attention(batch, block_len, n_q_heads, n_kv_heads, head_dim, layer, q, k_blk, v_blk, prefix_store,
                         prefix_cap, prefix_len, kv_store, t_cap, ctx_len, out, lse, workspace, workspace_bytes,
                         stream=None):
    """Attention of a batch over [shared prefix ; own context ; block] of one layer; out and lse are written."""
    _check(_compiled().shared_attention(batch, block_len, n_q_heads, n_kv_heads, head_dim, layer, q, k_blk, v_blk,
                                        prefix_store, prefix_cap, prefix_len, kv_store, t_cap, ctx_len, out, lse,
                                        workspace, workspace_bytes, *_here(stream)), "fpd_shared_attention")


def fpd_context_weights(batch, block_len, n_q_heads, n_kv_heads, head_dim, layer, q, lse, kv_store, t_cap, ctx_len,
                        weights, accumulate=False, stream=None):
    """weights[layer] (+)= the attention weight every context position collects from the rows of q."""
    _check(_compiled().context_weights(batch, block_len, n_q_heads, n_kv_heads, head_dim, layer, q, lse, kv_store, t_cap,
                                       ctx_len, weights, 1 if accumulate else 0, *_here(stream)), "fpd_context_weights")


def fpd_evict_workspace_bytes(n_layers, batch, n_kv_heads, budget) -> int:
    return int(lib().fpd_evict_workspace_bytes(n_layers, batch, n_kv_heads, budget))


def fpd_evict_context(n_layers, batch, n_kv_heads, head_dim, budget, recent, kv_store, t_cap, weights, ctx_len, out_store,
                      out_cap, out_weights, out_len, pos_offset, kept, workspace, workspace_bytes, stream=None):
    """Keeps the last `recent` positions and those with the largest weights, `budget` in all, of every request."""
    _check(_compiled().evict_context(n_layers, batch, n_kv_heads, head_dim, budget, recent, kv_store, t_cap, weights, ctx_len,
                                     out_store, out_cap, out_weights, out_len, pos_offset, kept, workspace,
                                     workspace_bytes, *_here(stream)), "fpd_evict_context")


def _on_device(t, dtype, n, what):
    """_arg on the current device."""
    if t is None or isinstance(t, int):
        return t
    return _arg(t, dtype, n, what, torch._C._cuda_getDevice() if getattr(t, "is_cuda", False) else 0)


def fpd_prepare_context_at(model, batch, total_rows, row_off, row_cnt, pos_start, pos_offset, feats, kv_store, t_cap,
                           workspace, workspace_bytes, stream=None):
    bf, i32 = torch.bfloat16, torch.int32
    arr = (ctypes.c_void_p * len(feats))(*[_on_device(f, bf, total_rows, "feats") for f in feats])
    _check(lib().fpd_prepare_context_at(model, batch, total_rows, _on_device(row_off, i32, batch + 1, "row_off"),
                                        _on_device(row_cnt, i32, batch, "row_cnt"), _on_device(pos_start, i32, batch, "pos_start"),
                                        _on_device(pos_offset, i32, batch, "pos_offset"), arr,
                                        _on_device(kv_store, bf, batch * t_cap, "kv_store"), t_cap,
                                        _on_device(workspace, torch.uint8, workspace_bytes, "workspace"), workspace_bytes,
                                        _stream(stream)), "fpd_prepare_context_at")


def fpd_shared_workspace_bytes(model, batch, max_block_len, prefix_cap, t_cap) -> int:
    return int(lib().fpd_shared_workspace_bytes(model, batch, max_block_len, prefix_cap, t_cap))


def shared_context(prefix_store=None, prefix_cap=0, prefix_len=None, kv_store=None, t_cap=0, ctx_len=None, pos_offset=None,
                   weights=None, prefix_weights=None, accumulate=False) -> SharedContext:
    """Build an fpd_shared_context; it keeps its tensors alive."""
    bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    c = SharedContext(_on_device(prefix_store, bf, prefix_cap, "prefix_store"), prefix_cap, _on_device(prefix_len, i32, 1, "prefix_len"),
                      _on_device(kv_store, bf, t_cap, "kv_store"), t_cap, _on_device(ctx_len, i32, 1, "ctx_len"),
                      _on_device(pos_offset, i32, 1, "pos_offset"), _on_device(weights, f32, t_cap, "weights"),
                      _on_device(prefix_weights, f32, prefix_cap, "prefix_weights"), int(bool(accumulate)))
    c._keep = (prefix_store, prefix_len, kv_store, ctx_len, pos_offset, weights, prefix_weights)
    c._per_request = ((ctx_len, "ctx_len"), (pos_offset, "pos_offset"))
    return c


def fpd_draft_block_shared(model, batch, block_len, ctx: SharedContext, anchor, mask_id, hidden_out, layer_hidden,
                           workspace, workspace_bytes, stream=None):
    for t, what in getattr(ctx, "_per_request", ()):   # its builder did not know the batch
        if isinstance(t, torch.Tensor) and t.numel() < batch:
            raise ValueError(f"{what} holds {t.numel()} elements, the call needs {batch}")
    rows = batch * block_len
    _check(lib().fpd_draft_block_shared(model, batch, block_len, ctypes.byref(ctx), _on_device(anchor, torch.int32, batch, "anchor"),
                                        int(mask_id), _on_device(hidden_out, torch.bfloat16, rows, "hidden_out"),
                                        _on_device(layer_hidden, torch.bfloat16, rows, "layer_hidden"),
                                        _on_device(workspace, torch.uint8, workspace_bytes, "workspace"), workspace_bytes,
                                        _stream(stream)), "fpd_draft_block_shared")
