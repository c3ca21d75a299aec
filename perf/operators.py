"""Work and timing cases of the operators on a context store: attention of a batch over a prefix that its requests
share (fpd_shared_attention), the attention weight that each stored position has collected (fpd_context_weights), and
the eviction of the positions with the least of it (fpd_evict_context).

A case is a dict of plain values; its "op" names the operator.  Stores are laid out as include/fpd.h says:
[layer][request][K|V][kv head][position][head dim] bf16.  Queries and keys have unit root mean square, as after the
per-head RMSNorm and the rotation; values are N(0, 1).
"""
import math

import numpy as np
import torch

own = False

LAYERS = 2      # layers in the stores of the attention and weight cases; the calls read the last one


def listed():
    return [
        # single-token decoding of four requests on the small test shape: launch latency
        dict(name="shared_decode_small", op="attention", batch=4, block=1, nq=8, nkv=2, h=64, prefix=512, slack=0, own_cap=64,
             blk=True),
        # eight text blocks of 16 positions behind one 2048-position scene, each with a ragged context of its own
        dict(name="shared_text_b8", op="attention", batch=8, block=16, nq=32, nkv=8, h=128, prefix=2048, slack=0, own_cap=256,
             blk=True),
        # odd sizes: 5 query heads to a kv head, a prefix that ends inside a tile and before its store does, no block keys
        dict(name="shared_odd", op="attention", batch=3, block=7, nq=20, nkv=4, h=128, prefix=4999, slack=5, own_cap=131,
             blk=False),
        # single-token decoding of 16 requests behind a very long prefix: the read of the prefix
        dict(name="shared_decode_long", op="attention", batch=16, block=1, nq=32, nkv=8, h=128, prefix=65536, slack=0,
             own_cap=512, blk=True),
        # four trajectories of 385 positions drafted for one scene
        dict(name="shared_primitive_b4", op="attention", batch=4, block=385, nq=32, nkv=8, h=128, prefix=4096, slack=0,
             own_cap=128, blk=True),
        # 64 text blocks behind a 16384-position prefix: the tensor cores
        dict(name="shared_text_b64", op="attention", batch=64, block=16, nq=32, nkv=8, h=128, prefix=16384, slack=0,
             own_cap=512, blk=True),
        # one block of 16 positions on the small test shape: launch latency
        dict(name="weights_small", op="weights", batch=1, block=16, nq=8, nkv=2, h=64, cap=144, longest=128),
        # ragged contexts of eight text blocks
        dict(name="weights_text_b8", op="weights", batch=8, block=16, nq=32, nkv=8, h=128, cap=2048, longest=2048),
        # a shared prefix, read by all rows of 64 text blocks
        dict(name="weights_prefix", op="weights", batch=1, block=1024, nq=32, nkv=8, h=128, cap=16384, longest=16384),
        # half of a 128-position context goes, small test shape: launch latency
        dict(name="evict_small", op="evict", layers=5, batch=1, nkv=2, h=64, cap=144, longest=128, budget=64, recent=16),
        # the batch-1 text context: 2048 positions to 1024
        dict(name="evict_text", op="evict", layers=5, batch=1, nkv=8, h=128, cap=2304, longest=2048, budget=1024,
             recent=256),
        # eight ragged long contexts to at most 4096 positions each
        dict(name="evict_batch", op="evict", layers=5, batch=8, nkv=8, h=128, cap=16384, longest=16384, budget=4096,
             recent=512),
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "weights", "evict"])
    h, nkv = rng.choice([64, 128, 128]), rng.choice([1, 2, 4, 8])
    if op == "evict":
        layers, batch, cap = rng.randint(1, 5), _spread(rng, 1, 8), _spread(rng, 8, 16384)
        longest = rng.randint(max(1, cap // 2), cap)
        budget = rng.randint(max(1, longest // 8), max(1, longest))
        return dict(op=op, layers=layers, batch=batch, nkv=nkv, h=h, cap=cap, longest=longest, budget=budget,
                    recent=rng.randint(0, budget))
    nq = nkv * rng.choice([1, 2, 3, 4, 4, 5, 8])
    batch, block = _spread(rng, 1, 64), _spread(rng, 1, 385)
    while batch * block > 1540:
        batch = max(1, batch // 2)
    if op == "weights":
        cap = _spread(rng, 8, 16384)
        while nq * batch * block * cap > 32 * 1024 * 16384 // 2 or batch * cap > 65536:
            cap = max(8, cap // 2)
        return dict(op=op, batch=batch, block=block, nq=nq, nkv=nkv, h=h, cap=cap, longest=rng.randint(max(1, cap // 2), cap))
    prefix, own_cap = _spread(rng, 1, 65536), rng.choice([0, 1, 2, 3]) and _spread(rng, 1, 1024)
    while nq * batch * block * prefix > 32 * 1024 * 16384 // 2:
        prefix = max(1, prefix // 2)
    while nq * batch * block * (own_cap + block) > 32 * 1540 * 1024:
        own_cap //= 2
        if own_cap == 0:
            break
    return dict(op=op, batch=batch, block=block, nq=nq, nkv=nkv, h=h, prefix=prefix, slack=rng.choice([0, 0, 1, 77]),
                own_cap=own_cap, blk=rng.random() < 0.75)


def _lens(batch, longest):
    """Ragged lengths of the requests: the first is the longest, some are empty."""
    return [longest * ((7 * b + 10) % 11) // 10 for b in range(batch)]


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def prepare(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev).manual_seed(seed * 9176 + 11)
    bf = torch.bfloat16

    def normal(*shape):
        return torch.randn(*shape, device=dev, generator=gen).to(bf)

    def unit(*shape):   # rows of unit root mean square
        x = torch.randn(*shape, device=dev, generator=gen)
        return (x * x.square().mean(-1, keepdim=True).rsqrt()).to(bf)

    def store(layers, batch, nkv, cap, h):
        s = torch.empty(layers, batch, 2, nkv, cap, h, device=dev, dtype=bf)
        for i in range(layers):
            s[i, :, 0] = unit(batch, nkv, cap, h)
            s[i, :, 1] = normal(batch, nkv, cap, h)
        return s

    def ints(v):
        return torch.tensor(v, device=dev, dtype=torch.int32)

    B, nkv, h = case["batch"], case["nkv"], case["h"]
    if case["op"] == "evict":
        shape = (case["layers"], B, nkv, case["cap"])
        # collected weights: a few positions hold most of it, some hold none
        w = torch.rand(*shape, device=dev, generator=gen).clamp_min(1e-6).log().neg().pow(3)
        w = torch.where(torch.rand(*shape, device=dev, generator=gen) < 0.05, torch.zeros_like(w), w)
        lens = _lens(B, case["longest"])
        w = torch.where(torch.arange(case["cap"], device=dev) < ints(lens)[:, None, None], w, torch.zeros_like(w))
        cap_out = case["budget"]
        return dict(case=case, store=store(case["layers"], B, nkv, case["cap"], h), weights=w, lens=ints(lens),
                    out_store=torch.zeros(case["layers"], B, 2, nkv, cap_out, h, device=dev, dtype=bf),
                    out_weights=torch.zeros(case["layers"], B, nkv, cap_out, device=dev), out_len=ints([0] * B),
                    kept=torch.full((case["layers"], B, nkv, cap_out), -1, device=dev, dtype=torch.int32))
    rows = B * case["block"]
    q = unit(rows, case["nq"], h)
    if case["op"] == "weights":
        s = store(LAYERS, B, nkv, case["cap"], h)
        lens = ints(_lens(B, case["longest"]))
        # the softmax's own denominators, over the context and a block of as many keys as the block has positions
        kb = unit(B, nkv, case["block"], h)
        keys = torch.cat([s[-1, :, 0], kb], 2).float()
        qs = _grouped(q, B, case["block"], nkv).float()
        lse = torch.empty(B, nkv, qs.shape[2], device=dev)
        ok = torch.cat([_before(lens, case["cap"]), torch.ones(B, case["block"], device=dev, dtype=torch.bool)], 1)
        for b in range(B):
            sc = torch.where(ok[b][None, None], qs[b] @ keys[b].transpose(1, 2) / math.sqrt(h), -math.inf)
            lse[b] = torch.logsumexp(sc, -1)
        lse = lse.view(B, nkv, case["block"], -1).permute(0, 2, 1, 3).reshape(rows, case["nq"]).contiguous()
        return dict(case=case, q=q, lse=lse, store=s, lens=lens,
                    weights=torch.zeros(LAYERS, B, nkv, case["cap"], device=dev))
    T, P = case["own_cap"], case["prefix"]
    return dict(case=case, q=q, k_blk=unit(B, nkv, case["block"], h) if case["blk"] else None,
                v_blk=normal(B, nkv, case["block"], h) if case["blk"] else None,
                prefix=store(LAYERS, 1, nkv, P + case["slack"], h), prefix_len=ints([P]),
                store=store(LAYERS, B, nkv, T, h) if T else None, lens=ints(_lens(B, T)) if T else None,
                out=torch.zeros(rows, case["nq"], h, device=dev, dtype=bf), lse=torch.zeros(rows, case["nq"], device=dev))


def _grouped(x, batch, block, nkv):
    """[batch * block, heads, ...] -> [batch, kv heads, block * group, ...]"""
    x = x.view(batch, block, nkv, x.shape[1] // nkv, *x.shape[2:])
    return x.transpose(1, 2).reshape(batch, nkv, block * x.shape[3], *x.shape[4:])


def _before(lens, n):
    return torch.arange(n, device=lens.device) < lens[:, None]


def _plain_attention(s):
    c = s["case"]
    B, L, nkv, h = c["batch"], c["block"], c["nkv"], c["h"]
    q = _grouped(s["q"], B, L, nkv).float() / math.sqrt(h)
    R = q.shape[2]
    # prefix: all requests' rows of a kv head against the same keys
    flat = q.transpose(0, 1).reshape(nkv, B * R, h)
    kp, vp = s["prefix"][-1, 0].float()
    sp = flat @ kp.transpose(1, 2)
    sp.masked_fill_(~_before(s["prefix_len"], kp.shape[1])[0], -math.inf)
    # the request's own keys: its context and its block
    k = [t for t in (s["store"][-1, :, 0] if c["own_cap"] else None, s["k_blk"]) if t is not None]
    v = [t for t in (s["store"][-1, :, 1] if c["own_cap"] else None, s["v_blk"]) if t is not None]
    top = sp.amax(-1).view(nkv, B, R).transpose(0, 1)
    if k:
        k, v = torch.cat(k, 2).float(), torch.cat(v, 2).float()
        so = q @ k.transpose(2, 3)
        if c["own_cap"]:
            so[..., :c["own_cap"]].masked_fill_(~_before(s["lens"], c["own_cap"])[:, None, None], -math.inf)
        top = torch.maximum(top, so.amax(-1))
    sp = torch.exp(sp - top.transpose(0, 1).reshape(nkv, B * R, 1))
    den = sp.sum(-1).view(nkv, B, R).transpose(0, 1)
    num = (sp @ vp).view(nkv, B, R, h).transpose(0, 1)
    if torch.is_tensor(k):
        so = torch.exp(so - top[..., None])
        den = den + so.sum(-1)
        num = num + so @ v
    out = (num / den[..., None]).view(B, nkv, L, -1, h).transpose(1, 2).reshape(B * L, c["nq"], h)
    lse = (top + torch.log(den)).view(B, nkv, L, -1).transpose(1, 2).reshape(B * L, c["nq"])
    return [out.to(torch.bfloat16), lse]


def _plain_weights(s):
    c = s["case"]
    q = _grouped(s["q"], c["batch"], c["block"], c["nkv"]).float() / math.sqrt(c["h"])
    lse = _grouped(s["lse"], c["batch"], c["block"], c["nkv"])
    k = s["store"][-1, :, 0].float()
    w = torch.exp(q @ k.transpose(2, 3) - lse[..., None]).sum(2)
    out = s["weights"].clone()
    out[-1] = torch.where(_before(s["lens"], c["cap"])[:, None], w, out[-1])
    return [out]


def _plain_evict(s):
    c = s["case"]
    lens, w = s["lens"], s["weights"]
    at = torch.arange(c["cap"], device=w.device)
    n = lens[:, None, None]
    rank = torch.where(at >= n - c["recent"], math.inf, w)   # the most recent positions stay whatever their weight
    rank = torch.where(at < n, rank, -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :c["budget"]]
    new_len = torch.clamp(lens, max=c["budget"])
    held = torch.arange(c["budget"], device=w.device) < new_len[:, None, None]
    order = torch.sort(torch.where(held, order, c["cap"]), dim=-1).values   # back into the order of the positions
    src = torch.where(held, order, 0)
    kept = torch.where(held, order, -1).to(torch.int32)
    rows = torch.gather(s["store"], 4, src[:, :, None, :, :, None].expand(-1, -1, 2, -1, -1, c["h"]))
    out = torch.where(held[None, :, None, :, :, None], rows, s["out_store"])
    weights = torch.where(held, torch.gather(w, -1, src), torch.zeros((), device=w.device))
    return [out, weights, new_len, kept]


def _workspace(state, lib_bytes):
    """The caller's scratch memory, kept with the state as a serving loop keeps it."""
    if "workspace" not in state:
        state["workspace"] = torch.empty(max(16, lib_bytes()), dtype=torch.uint8, device=state["weights" if "weights" in state else "q"].device)
    return state["workspace"]


def _own_attention(s):
    import block_diffusion_speculative_non_gb300 as fpd
    c = s["case"]
    shape = (c["batch"], c["block"], c["nq"], c["nkv"], c["h"])
    cap = c["prefix"] + c["slack"]
    ws = _workspace(s, lambda: fpd.fpd_shared_attention_workspace_bytes(*shape, cap, c["own_cap"]))
    fpd.fpd_shared_attention(*shape, LAYERS - 1, s["q"], s["k_blk"], s["v_blk"], s["prefix"], cap, s["prefix_len"],
                             s["store"], c["own_cap"], s["lens"], s["out"], s["lse"], ws, ws.numel())
    return [s["out"], s["lse"]]


def _own_weights(s):
    import block_diffusion_speculative_non_gb300 as fpd
    c = s["case"]
    fpd.fpd_context_weights(c["batch"], c["block"], c["nq"], c["nkv"], c["h"], LAYERS - 1, s["q"], s["lse"], s["store"],
                            c["cap"], s["lens"], s["weights"], False)
    return [s["weights"]]


def _own_evict(s):
    import block_diffusion_speculative_non_gb300 as fpd
    c = s["case"]
    ws = _workspace(s, lambda: fpd.fpd_evict_workspace_bytes(c["layers"], c["batch"], c["nkv"], c["budget"]))
    fpd.fpd_evict_context(c["layers"], c["batch"], c["nkv"], c["h"], c["budget"], c["recent"], s["store"], c["cap"],
                          s["weights"], s["lens"], s["out_store"], c["budget"], s["out_weights"], s["out_len"], None,
                          s["kept"], ws, ws.numel())
    return [s["out_store"], s["out_weights"], s["out_len"], s["kept"]]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"attention": _own_attention, "weights": _own_weights, "evict": _own_evict}[op](state)
    return {"attention": _plain_attention, "weights": _plain_weights, "evict": _plain_evict}[op](state)


def exact(case, seed):
    """The same outputs from the definitions in 64 bits, one request and kv head at a time."""
    s = prepare(case, seed)
    B, nkv, h = case["batch"], case["nkv"], case["h"]
    if case["op"] == "evict":
        w, lens = s["weights"].cpu().numpy().astype(np.float64), s["lens"].cpu().tolist()
        kept = np.full((case["layers"], B, nkv, case["budget"]), -1, np.int32)
        out, out_w = s["out_store"].clone(), np.zeros(kept.shape)
        for b, n in enumerate(lens):
            m = min(n, case["budget"])
            for i in range(case["layers"]):
                for g in range(nkv):
                    old = max(0, n - case["recent"])
                    best = sorted(np.lexsort((np.arange(old), -w[i, b, g, :old]))[:max(0, m - (n - old))].tolist())
                    keep = (best + list(range(old, n)))[-m:] if m else []
                    kept[i, b, g, :m] = keep
                    out_w[i, b, g, :m] = w[i, b, g, keep]
                    if m:
                        out[i, b, :, g, :m] = s["store"][i, b, :, g, torch.tensor(keep, device=out.device)]
        return [out.double(), torch.from_numpy(out_w), np.minimum(np.array(lens, np.int32), np.int32(case["budget"])), kept]
    L, grp = case["block"], case["nq"] // nkv
    q = s["q"].double().view(B, L, nkv, grp, h)
    if case["op"] == "weights":
        out, lse = s["weights"].double(), s["lse"].double().view(B, L, nkv, grp)
        for b, n in enumerate(s["lens"].cpu().tolist()):
            for g in range(nkv):
                sc = torch.einsum("lih,th->lit", q[b, :, g], s["store"][-1, b, 0, g, :n].double()) * h ** -0.5
                out[-1, b, g, :n] = (sc - lse[b, :, g, :, None]).exp_().sum((0, 1))
        return [out]
    out = torch.empty(B, L, nkv, grp, h, dtype=torch.float64, device=q.device)
    lse = torch.empty(B, L, nkv, grp, dtype=torch.float64, device=q.device)
    lens = s["lens"].cpu().tolist() if case["own_cap"] else [0] * B
    for g in range(nkv):
        shared = [s["prefix"][-1, 0, x, g, :case["prefix"]].double() for x in (0, 1)]
        for b in range(B):
            kv = []
            for x, blk in ((0, s["k_blk"]), (1, s["v_blk"])):
                parts = [shared[x]]
                if lens[b]:
                    parts.append(s["store"][-1, b, x, g, :lens[b]].double())
                if blk is not None:
                    parts.append(blk[b, g].double())
                kv.append(torch.cat(parts))
            sc = torch.einsum("lih,th->lit", q[b, :, g], kv[0]) * h ** -0.5
            lse[b, :, g] = torch.logsumexp(sc, -1)
            out[b, :, g] = torch.einsum("lit,th->lih", torch.softmax(sc, -1), kv[1])
    return [out.reshape(B * L, case["nq"], h), lse.reshape(B * L, case["nq"])]


def work(case):
    B, nkv, h = case["batch"], case["nkv"], case["h"]
    if case["op"] == "evict":
        lens = _lens(B, case["longest"])
        left = sum(min(n, case["budget"]) for n in lens)
        heads = case["layers"] * nkv
        # weights of all positions; kept rows of K and V and their weights in and out; the kept positions
        return {"bytes": heads * (4 * sum(lens) + left * (2 * 2 * 2 * h + 4) + 2 * 4 * case["budget"] * B), "flops": 0}
    rows = B * case["block"] * case["nq"]
    per_request = case["block"] * case["nq"]
    if case["op"] == "weights":
        keys = sum(_lens(B, case["longest"]))
        return {"bytes": rows * (2 * h + 4) + nkv * keys * (2 * h + 4), "flops": 2 * per_request * keys * h}
    own_keys = sum(_lens(B, case["own_cap"])) + (B * case["block"] if case["blk"] else 0)
    return {"bytes": rows * (2 * 2 * h + 4) + nkv * (case["prefix"] + own_keys) * 2 * 2 * h,
            "flops": 4 * h * (rows * case["prefix"] + per_request * own_keys)}
