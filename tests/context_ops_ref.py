"""The operators on a context store written out from their definitions, in 64 bits (torch, any device) and plain Python.
Test infrastructure only."""
import math

import numpy as np
import torch


def attention(q, prefix, prefix_len, store, ctx_len, k_blk, v_blk, batch, block, nkv):
    """q [batch * block, nq, h]; prefix [K|V][nkv][cap][h] or None; store [batch][K|V][nkv][cap][h] or None; lists of
    lengths.  Returns out [batch * block, nq, h], lse [batch * block, nq] and the largest |v| of every row."""
    nq, h = q.shape[1:]
    grp = nq // nkv
    out = torch.zeros(batch, block, nq, h, dtype=torch.float64, device=q.device)
    lse = torch.full((batch, block, nq), -math.inf, dtype=torch.float64, device=q.device)
    vmax = torch.zeros(batch, block, nq, dtype=torch.float64, device=q.device)
    qd = q.double().view(batch, block, nq, h)
    for b in range(batch):
        for g in range(nkv):
            k, v = [], []
            if prefix is not None:
                k.append(prefix[0, g, :prefix_len])
                v.append(prefix[1, g, :prefix_len])
            if store is not None:
                k.append(store[b, 0, g, :ctx_len[b]])
                v.append(store[b, 1, g, :ctx_len[b]])
            if k_blk is not None:
                k.append(k_blk[b, g])
                v.append(v_blk[b, g])
            if not k or sum(x.shape[0] for x in k) == 0:
                continue
            k, v = torch.cat(k).double(), torch.cat(v).double()
            for i in range(g * grp, (g + 1) * grp):
                s = qd[b, :, i] @ k.T / math.sqrt(h)
                lse[b, :, i] = torch.logsumexp(s, 1)
                out[b, :, i] = torch.exp(s - lse[b, :, i, None]) @ v
                vmax[b, :, i] = v.abs().max()
    n = batch * block
    return out.reshape(n, nq, h), lse.reshape(n, nq), vmax.reshape(n, nq)


def context_weights(q, lse, store, ctx_len, batch, block, nkv):
    """[batch][nkv][cap] with NaN from each length on; store [batch][K|V][nkv][cap][h]."""
    nq, h = q.shape[1:]
    grp, cap = nq // nkv, store.shape[3]
    w = torch.full((batch, nkv, cap), math.nan, dtype=torch.float64, device=q.device)
    qd, ld = q.double().view(batch, block, nq, h), lse.double().view(batch, block, nq)
    for b in range(batch):
        for g in range(nkv):
            n = ctx_len[b]
            k = store[b, 0, g, :n].double()
            total = torch.zeros(n, dtype=torch.float64, device=q.device)
            for i in range(g * grp, (g + 1) * grp):
                live = ld[b, :, i] != -math.inf
                s = qd[b, live, i] @ k.T / math.sqrt(h)
                total += torch.exp(s - ld[b, live, i, None]).sum(0)
            w[b, g, :n] = total
    return w


def kept_positions(weights, length, budget, recent):
    """The kept positions of one head, ascending (weights: 1-D sequence)."""
    if length <= budget:
        return list(range(length))
    old = length - recent
    key = [(-math.inf if math.isnan(float(w)) else float(w), not math.isnan(float(w))) for w in weights[:old]]
    order = sorted(range(old), key=lambda t: (-key[t][0], not key[t][1], t))   # -inf ranks before NaN
    return sorted(order[:budget - recent]) + list(range(old, length))


def evict(store, weights, ctx_len, budget, recent, out_store, out_cap):
    """numpy arrays: store [layers][batch][2][nkv][cap][h], weights [layers][batch][nkv][cap].  Returns the new store (rows
    past the new lengths as in out_store), weights, lengths and kept positions."""
    layers, batch, _, nkv = store.shape[:4]
    out, ow = out_store.copy(), np.zeros((layers, batch, nkv, out_cap), np.float32)
    kept = np.full((layers, batch, nkv, budget), -1, np.int32)
    for l in range(layers):
        for b in range(batch):
            for g in range(nkv):
                keep = kept_positions(weights[l, b, g], ctx_len[b], budget, recent)
                m = len(keep)
                kept[l, b, g, :m] = keep
                ow[l, b, g, :m] = weights[l, b, g, keep]
                out[l, b, :, g, :m] = store[l, b, :, g, keep].transpose(1, 0, 2) if m else out[l, b, :, g, :0]
    return out, ow, np.minimum(np.asarray(ctx_len), budget).astype(np.int32), kept
