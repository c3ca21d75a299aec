"""Binding of the paged context cache (append, read, attention with a window and sinks, pages in bf16 or 4 bits) and of the
sampled verification.  Sizes and layouts are those of include/fpd.h.

Like the operators on a context store these are short calls: the compiled module `_calls` checks their arguments.
"""
from __future__ import annotations

import ctypes

import torch

from . import FPD_PAGE_BF16, FPD_PAGE_INT4, PagedStore, _check, lib
from .context import _compiled, _here

_bound = False


def _paged():
    """The compiled calls, with the paged entry points of the loaded library."""
    global _bound
    m = _compiled()
    if not _bound:
        m.bind_paged(*(ctypes.cast(getattr(lib(), f), ctypes.c_void_p).value
                       for f in ("fpd_paged_append", "fpd_paged_read", "fpd_paged_attention", "fpd_verify_sampled")))
        _bound = True
    return m


def fpd_page_bytes(format, page_size, n_kv_heads, head_dim) -> int:
    return int(lib().fpd_page_bytes(format, page_size, n_kv_heads, head_dim))


def paged_store(pages, format, n_layers, n_pages, page_size, n_kv_heads, head_dim, table, table_width=None) -> PagedStore:
    """Build an fpd_paged_store; it keeps its tensors alive.  pages: a device tensor of n_layers * n_pages * fpd_page_bytes bytes
    (bf16 for FPD_PAGE_BF16, uint8 for FPD_PAGE_INT4) or an address; table: int32 [batch, table_width], or an address with
    table_width."""
    one = fpd_page_bytes(format, page_size, n_kv_heads, head_dim)
    if one == 0 or n_layers < 1 or n_pages < 1:
        raise ValueError(f"pages of format {format}, {page_size} positions, {n_kv_heads} heads of {head_dim}, {n_layers} layers of "
                         f"{n_pages}")
    rows = dev = None
    if isinstance(table, torch.Tensor):
        if table.dim() != 2 or (table_width is not None and table_width != table.shape[1]):
            raise ValueError(f"table must be [batch, {table_width or 'table_width'}], got {tuple(table.shape)}")
        rows, table_width, dev = int(table.shape[0]), int(table.shape[1]), table.get_device() if table.is_cuda else -1
    elif table_width is None:
        raise ValueError("a table given by its address needs table_width")
    typ, n = (torch.bfloat16, one // 2) if format == FPD_PAGE_BF16 else (torch.uint8, one)
    p = _compiled().arg(pages, typ, n_layers * n_pages * n, "pages", pages.get_device() if getattr(pages, "is_cuda", False) else 0)
    t = _compiled().arg(table, torch.int32, 0, "table", dev if dev is not None and dev >= 0 else 0)
    s = PagedStore(p, t, format, n_layers, n_pages, page_size, n_kv_heads, head_dim, table_width)
    if isinstance(pages, torch.Tensor):
        if dev is not None and pages.get_device() != dev:
            raise ValueError(f"pages are on {pages.device}, the table on {table.device}")
        dev = pages.get_device()
    s._keep, s._rows, s._dev = (pages, table), rows, dev
    return s


def _store(store: PagedStore, batch, dev) -> int:
    """The struct's address, after what its builder could not know."""
    if not isinstance(store, PagedStore):
        raise TypeError(f"store must be a PagedStore, got {type(store).__name__}")
    rows, at = getattr(store, "_rows", None), getattr(store, "_dev", None)
    if rows is not None and rows < batch:
        raise ValueError(f"the table has {rows} requests, the call needs {batch}")
    if at is not None and at != dev:
        raise ValueError(f"the pages are on cuda:{at}, the current device is cuda:{dev}")
    return ctypes.addressof(store)


def fpd_paged_append(batch, total_rows, store, layer, k, k_ld, v, v_ld, row_off, row_cnt, pos_start, pos_offset, rope, max_pos,
                     stream=None):
    """Writes rows of keys, rotated for their positions, and values into the pages of their requests."""
    st, dev = _here(stream)
    _check(_paged().paged_append(batch, total_rows, _store(store, batch, dev), layer, k, k_ld, v, v_ld, row_off, row_cnt, pos_start,
                                 pos_offset, rope, max_pos, st, dev), "fpd_paged_append")


def fpd_paged_read(batch, total_rows, store, layer, row_off, row_cnt, pos_start, k, v, stream=None):
    """k and v [total_rows, kv heads, h] = the stored rows that an append with the same offsets wrote."""
    st, dev = _here(stream)
    _check(_paged().paged_read(batch, total_rows, _store(store, batch, dev), layer, row_off, row_cnt, pos_start, k, v, st, dev),
           "fpd_paged_read")


def fpd_paged_attention_workspace_bytes(batch, block_len, n_q_heads, store) -> int:
    return int(lib().fpd_paged_attention_workspace_bytes(batch, block_len, n_q_heads, ctypes.byref(store)))


def fpd_paged_attention(batch, block_len, n_q_heads, store, layer, q, k_blk, v_blk, ctx_len, window, sinks, causal, out, lse,
                        workspace, workspace_bytes, stream=None):
    """Attention of blocks over their requests' pages and the blocks' own keys; out and lse are written."""
    st, dev = _here(stream)
    _check(_paged().paged_attention(batch, block_len, n_q_heads, _store(store, batch, dev), layer, q, k_blk, v_blk, ctx_len, window,
                                    sinks, 1 if causal else 0, out, lse, workspace, workspace_bytes, st, dev), "fpd_paged_attention")


def fpd_verify_sampled(batch, block_len, vocab, draft, target, draft_probs, uniform, accept_len, committed, valid_out, stream=None):
    """Keeps drafted ids by given random numbers, so that the committed ids are samples of the target."""
    st, dev = _here(stream)
    _check(_paged().verify_sampled(batch, block_len, vocab, draft, target, draft_probs, uniform, accept_len, committed, valid_out, st,
                                   dev), "fpd_verify_sampled")


def rope_table(max_pos, head_dim, theta, device="cuda") -> torch.Tensor:
    """[max_pos, head_dim / 2, 2] fp32: (cos, sin) of pos theta^(-2i / head_dim), taken in 64 bits."""
    i = torch.arange(0, head_dim, 2, dtype=torch.float64, device=device)
    angle = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * float(theta) ** (i / -head_dim)
    return torch.stack([angle.cos(), angle.sin()], -1).float()
