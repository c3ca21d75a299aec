"""The paged context cache and the sampled verification written out from their definitions, in 64 bits.  Test infrastructure
only."""
import math
from fractions import Fraction

import numpy as np
import torch

SCALES = [(8 + m) * 2.0 ** (e - 18) if e else m * 2.0 ** -17 for e in range(32) for m in range(8)]
TOP = SCALES.index(2.0 ** 13)


def quantise(x):
    """x [..., h] float64 -> codes [..., h] in -7..7, scale bytes [..., h / 16]."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    big = np.where(np.isnan(g), 0, np.abs(g)).max(-1)
    byte = np.minimum(np.searchsorted(7 * np.array(SCALES[:TOP + 1]), big), TOP)
    s = np.array(SCALES)[byte][..., None]
    with np.errstate(all="ignore"):
        n = np.where(s > 0, g / np.where(s > 0, s, 1), 0.0)
    n = np.where(np.isnan(g) | (s == 0), 0, np.clip(np.rint(n), -7, 7))
    return n.reshape(x.shape).astype(np.int64), byte.astype(np.uint8)


def pack(codes, byte):
    """Code bytes [..., h / 2] (dim 2 i in the lower half) and scale bytes."""
    c = (codes + 8).reshape(*codes.shape[:-1], codes.shape[-1] // 2, 2)
    return (c[..., 0] + 16 * c[..., 1]).astype(np.uint8), byte


def stands_for(codes, byte):
    s = np.array(SCALES)[byte]
    return (codes.reshape(*codes.shape[:-1], codes.shape[-1] // 16, 16) * s[..., None]).reshape(codes.shape)


def rotate(k, cs):
    """k [..., h] float64, cs [..., h / 2, 2] (cos, sin): rotate-half, rounded to fp32 and to bf16 (float64 values)."""
    lo, hi = np.split(k, 2, -1)
    c, s = cs[..., 0], cs[..., 1]
    r = np.concatenate([lo * c - hi * s, hi * c + lo * s], -1)
    return torch.from_numpy(r).float().to(torch.bfloat16).double().numpy()


def visible(L, n, window, sinks, causal):
    """[L, n] bool: row j stands at position n - L + j."""
    row, t = np.arange(n - L, n)[:, None], np.arange(n)[None]
    ok = np.ones((L, n), bool)
    if window:
        ok &= (t < sinks) | (row - t < window)
    if causal:
        ok &= t <= row
    return ok


def attention(q, keys, values, L, window, sinks, causal):
    """q [batch * L, nq, h]; keys, values: for every request [nkv, n_b, h] float64 tensors.  Returns out, lse [batch * L, nq] and
    the largest |v| that a row sees."""
    nq, h = q.shape[1:]
    B = len(keys)
    qd = q.double().view(B, L, nq, h)
    out = torch.zeros(B, L, nq, h, dtype=torch.float64, device=q.device)
    lse = torch.full((B, L, nq), -math.inf, dtype=torch.float64, device=q.device)
    vmax = torch.zeros(B, L, nq, dtype=torch.float64, device=q.device)
    for b in range(B):
        nkv, n = keys[b].shape[:2]
        if n == 0:
            continue
        ok = torch.from_numpy(visible(L, n, window, sinks, causal)).to(q.device)
        for i in range(nq):
            g = i // (nq // nkv)
            s = (qd[b, :, i] @ keys[b][g].T / math.sqrt(h)).masked_fill(~ok, -math.inf)
            lse[b, :, i] = torch.logsumexp(s, 1)
            live = lse[b, :, i] > -math.inf
            out[b, live, i] = torch.exp(s[live] - lse[b, live, i, None]) @ values[b][g]
            vmax[b, :, i] = values[b][g].abs().max()
    n = B * L
    return out.reshape(n, nq, h), lse.reshape(n, nq), vmax.reshape(n, nq)


def verify_sampled(draft, target, probs, uniform):
    """Exact rational arithmetic, one request: (accept, committed, valid); arrays [L-1], [L, V], [L-1, V] or None, [L]."""
    L, V = target.shape

    def w(x):
        return Fraction(float(x)) if x > 0 else Fraction(0)

    n = 0
    while n < L - 1:
        d = int(draft[n])
        if not 0 <= d < V:
            break
        q = w(probs[n, d]) if probs is not None else Fraction(1)
        if not Fraction(float(uniform[n])) * q < w(target[n, d]):
            break
        n += 1
    own = [w(x) for x in target[n]]
    r = own
    if n < L - 1:
        if probs is not None:
            r = [max(a - w(b), Fraction(0)) for a, b in zip(own, probs[n])]
        else:
            r = [Fraction(0) if i == draft[n] else a for i, a in enumerate(own)]
        if sum(r) == 0:
            r = own
    total, run, token = sum(r), Fraction(0), -1
    x = Fraction(float(uniform[L - 1])) * total
    if total > 0:
        for i, a in enumerate(r):
            run += a
            if run > x:
                token = i
                break
    committed = [int(v) for v in draft[:n]] + [token] + [-1] * (L - 1 - n)
    return n + 1, committed, int(n == L - 1)
