"""Work and timing cases of the operators on a paged context cache (append with the rotation, attention over the pages with
a window and sinks, pages held in 4 bits) and of the sampled verification of a drafted block.

A case is a dict of plain values; its "op" names the operator.  Layouts are those of include/fpd.h: the pages of a layer are
[page][K|V][kv head] slabs of `page` positions; a slab is [position][head dim] bf16 ("bf16"), or [position][head dim / 2] bytes
of 4-bit codes followed by [position][head dim / 16] scale bytes ("int4").  A code n + 8 and its group's scale s stand for n s,
-7 <= n <= 7; the scale byte holds 5 exponent and 3 mantissa bits, the upper bits of an fp16 number without its sign.
Keys have unit root mean square, as after the per-head RMSNorm; values are N(0, 1).
"""
import math

import numpy as np
import torch

own = False

LAYERS = 2        # layers in the page pools; the calls use the last one
THETA = 1e6
TOP_SCALE = 224   # the largest scale byte in use, 2^13


def listed():
    return [
        # a decode step appends one position to each of four requests, small test shape: launch latency
        dict(name="append_step_small", op="append", form="bf16", batch=4, nkv=2, h=64, page=16, rows=1, ctx=500, even=True),
        # a speculative step of eight requests keeps up to 16 positions of each block, 4-bit pages
        dict(name="append_text_int4", op="append", form="int4", batch=8, nkv=8, h=128, page=64, rows=16, ctx=2048, even=False),
        # eight ragged prompts enter the cache
        dict(name="append_prompts", op="append", form="bf16", batch=8, nkv=8, h=128, page=64, rows=8192, ctx=0, even=False),
        # single-token decoding of four requests on the small test shape: launch latency
        dict(name="paged_step_small", op="attention", form="bf16", batch=4, block=1, nq=8, nkv=2, h=64, page=16, ctx=512,
             blk=True, window=0, sinks=0, causal=False),
        # eight text blocks of 16 positions over ragged contexts
        dict(name="paged_text_b8", op="attention", form="bf16", batch=8, block=16, nq=32, nkv=8, h=128, page=64, ctx=2048,
             blk=True, window=0, sinks=0, causal=False),
        # single-token decoding of 16 requests with long contexts: the read of the keys
        dict(name="paged_step_long", op="attention", form="bf16", batch=16, block=1, nq=32, nkv=8, h=128, page=64, ctx=32768,
             blk=True, window=0, sinks=0, causal=False),
        # four trajectories of 385 positions that look back at 1024 positions and the first 64
        dict(name="window_primitive_b4", op="attention", form="bf16", batch=4, block=385, nq=32, nkv=8, h=128, page=128, ctx=4096,
             blk=True, window=1024, sinks=64, causal=False),
        # odd sizes: 5 query heads to a kv head, a window that starts inside a page, causal, the block's keys already appended
        dict(name="window_odd", op="attention", form="bf16", batch=3, block=7, nq=20, nkv=4, h=128, page=16, ctx=4999,
             blk=False, window=333, sinks=5, causal=True),
        # single-token decoding of 16 requests with very long contexts in 4 bits: the read of the keys
        dict(name="int4_step_long", op="attention", form="int4", batch=16, block=1, nq=32, nkv=8, h=128, page=64, ctx=65536,
             blk=True, window=0, sinks=0, causal=False),
        # 64 text blocks over contexts in 4 bits: the products
        dict(name="int4_text_b64", op="attention", form="int4", batch=64, block=16, nq=32, nkv=8, h=128, page=64, ctx=4096,
             blk=True, window=0, sinks=0, causal=False),
        # one block of the small test shape whose drafter took its best ids: launch latency
        dict(name="verify_small", op="verify", batch=1, block=16, vocab=4096, probs=False),
        # 64 sampled text blocks over the full vocabulary
        dict(name="verify_text_b64", op="verify", batch=64, block=16, vocab=151936, probs=True),
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "attention", "verify"])
    if op == "verify":
        batch, block, vocab = _spread(rng, 1, 64), rng.randint(2, 32), _spread(rng, 2, 151936)
        while batch * block * vocab > 64 * 16 * 151936:
            batch = max(1, batch // 2)
        return dict(op=op, batch=batch, block=block, vocab=vocab, probs=rng.random() < 0.6)
    form, h, nkv, page = rng.choice(["bf16", "int4"]), rng.choice([64, 128, 128]), rng.choice([1, 2, 4, 8]), rng.choice([16, 32, 64, 128])
    batch = _spread(rng, 1, 64)
    if op == "append":
        rows = _spread(rng, 1, 8192)
        while batch * rows > 32768:
            batch = max(1, batch // 2)
        return dict(op=op, form=form, batch=batch, nkv=nkv, h=h, page=page, rows=rows, ctx=rng.choice([0, _spread(rng, 1, 8192)]),
                    even=rng.random() < 0.5)
    nq, block, ctx = nkv * rng.choice([1, 2, 3, 4, 4, 5, 8]), _spread(rng, 1, 385), _spread(rng, 1, 65536)
    while batch * block > 1540 or batch * ctx > 1 << 20:
        batch = max(1, batch // 2)
        if batch == 1:
            break
    while nq * batch * block * ctx > 32 * 1540 * 4096:
        ctx = max(1, ctx // 2)
    window = rng.choice([0, 0, _spread(rng, 1, 4096)])
    return dict(op=op, form=form, batch=batch, block=block, nq=nq, nkv=nkv, h=h, page=page, ctx=ctx, blk=rng.random() < 0.75,
                window=window, sinks=rng.choice([0, 1, 4, 100]) if window else 0, causal=rng.random() < 0.4)


def _lens(batch, longest):
    """Ragged lengths of the requests: the first is the longest, some are empty."""
    return [longest * ((7 * b + 10) % 11) // 10 for b in range(batch)]


def _sizes(case):
    """(context lengths, appended rows, pages of a request's table) of a case on pages."""
    B = case["batch"]
    lens = _lens(B, case["ctx"])
    rows = [0] * B
    if case["op"] == "append":
        rows = [case["rows"]] * B if case["even"] else _lens(B, case["rows"])
    return lens, rows, max(1, -(-max(n + r for n, r in zip(lens, rows)) // case["page"]))


def _page_elems(case):
    """Elements of a page: bf16 numbers, or bytes."""
    h, n = case["h"], 2 * case["nkv"] * case["page"]
    return n * h if case["form"] == "bf16" else n * (h // 2 + h // 16)


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def prepare(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev).manual_seed(seed * 7919 + 23)
    bf = torch.bfloat16

    def ints(v):
        return torch.tensor(v, device=dev, dtype=torch.int32)

    def unit(*shape):   # rows of unit root mean square
        x = torch.randn(*shape, device=dev, generator=gen)
        return (x * x.square().mean(-1, keepdim=True).rsqrt()).to(bf)

    B = case["batch"]
    if case["op"] == "verify":
        L, V = case["block"], case["vocab"]
        # the target's logits and the drafter's, which are near them; the drafted ids come from the drafter's probabilities
        t = torch.randn(B, L, V, device=dev, generator=gen).mul_(2.5)
        d = torch.randn(B, L - 1, V, device=dev, generator=gen).mul_(0.7).add_(t[:, :-1])
        t = torch.softmax(t, -1)
        if case["probs"]:
            d = torch.softmax(d, -1)
            at = torch.rand(B, L - 1, 1, device=dev, generator=gen).double()
            c = torch.cumsum(d.double(), -1)
            draft = torch.searchsorted(c, at * c[..., -1:], right=True)[..., 0].clamp_max(V - 1).to(torch.int32)
        else:
            draft, d = d.argmax(-1).to(torch.int32), None
        return dict(case=case, draft=draft, target=t, probs=d, uniform=torch.rand(B, L, device=dev, generator=gen),
                    accept=ints([0] * B), committed=torch.zeros(B, L, device=dev, dtype=torch.int32), valid=ints([0] * B))
    nkv, h, page = case["nkv"], case["h"], case["page"]
    lens, rows, width = _sizes(case)
    n_pages = B * width + 3
    table = torch.randperm(n_pages, device=dev, generator=gen)[:B * width].view(B, width).to(torch.int32)
    if case["form"] == "bf16":
        pool = torch.empty(LAYERS, n_pages, 2, nkv, page, h, device=dev, dtype=bf)
        for i in range(LAYERS):
            pool[i, :, 0] = unit(n_pages, nkv, page, h)
            pool[i, :, 1] = torch.randn(n_pages, nkv, page, h, device=dev, generator=gen).to(bf)
    else:
        # codes over their whole range, scales around those of unit values
        pool = torch.empty(LAYERS, n_pages, 2, nkv, page * (h // 2 + h // 16), device=dev, dtype=torch.uint8)
        for i in range(LAYERS):
            x = torch.randn(n_pages, 2, nkv, page * h // 2, 2, device=dev, generator=gen).mul_(3.3).round_().clamp_(-7, 7).add_(8)
            pool[i, ..., :page * h // 2] = (x[..., 0] + 16 * x[..., 1]).to(torch.uint8)
            pool[i, ..., page * h // 2:] = torch.randint(100, 109, (n_pages, 2, nkv, page * h // 16), device=dev, generator=gen,
                                                         dtype=torch.uint8)
    s = dict(case=case, pool=pool, table=table, lens=ints(lens))
    if case["op"] == "append":
        n, nq = sum(rows), 4 * nkv
        off = [0]
        for r in rows:
            off.append(off[-1] + r)
        # keys and values lie in the rows of a fused projection's output
        qkv = unit(max(1, n), nq + 2 * nkv, h).view(max(1, n), -1)
        qkv[:, (nq + nkv) * h:] = torch.randn(max(1, n), nkv * h, device=dev, generator=gen).to(bf)
        top = max(a + b for a, b in zip(lens, rows)) + 64
        angle = torch.arange(top, device=dev, dtype=torch.float64)[:, None] * THETA ** (
            torch.arange(0, h, 2, device=dev, dtype=torch.float64) / -h)
        s.update(total=n, qkv=qkv, off=ints(off), rope=torch.stack([angle.cos(), angle.sin()], -1).float(),
                 pos_offset=ints([(37 * b) % 64 for b in range(B)]),
                 k_back=torch.zeros(max(1, n), nkv, h, device=dev, dtype=bf),
                 v_back=torch.zeros(max(1, n), nkv, h, device=dev, dtype=bf))
        return s
    L, nq = case["block"], case["nq"]
    s.update(q=unit(B * L, nq, h), k_blk=unit(B, nkv, L, h) if case["blk"] else None,
             v_blk=torch.randn(B, nkv, L, h, device=dev, generator=gen).to(bf) if case["blk"] else None,
             out=torch.zeros(B * L, nq, h, device=dev, dtype=bf), lse=torch.zeros(B * L, nq, device=dev))
    return s


# ---- plain forms --------------------------------------------------------------------------------------------------------

def _scales(dev):
    """The values of the scale bytes in use, in order."""
    return (torch.arange(TOP_SCALE + 1, device=dev, dtype=torch.int16) << 7).view(torch.float16).float()


def _plain_slots(s):
    """Request, page, place in the page and position in the sequence of every appended row."""
    c, off, lens = s["case"], s["off"].long(), s["lens"].long()
    r = torch.arange(s["total"], device=off.device)
    b = torch.searchsorted(off, r, right=True) - 1
    slot = lens[b] + r - off[b]
    return s["table"].long()[b, slot // c["page"]], slot % c["page"], slot + s["pos_offset"].long()[b]


def _plain_append(s):
    c, n = s["case"], s["total"]
    nkv, h, page = c["nkv"], c["h"], c["page"]
    at, place, pos = _plain_slots(s)
    k, v = s["qkv"][:n, 4 * nkv * h:].view(n, 2, nkv, h).unbind(1)
    cos, sin = (t[:, None] for t in s["rope"].double()[pos].unbind(-1))
    lo, hi = k.double().chunk(2, -1)
    # in 64 bits: a 4-bit code goes by the rounded key, which may lie next to a border
    k = torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1).to(torch.bfloat16)
    x = torch.stack([k, v], 1)
    if c["form"] == "bf16":
        s["pool"][-1, at, :, :, place] = x
        return [s["pool"]]
    g = x.float().view(n, 2, nkv, h // 16, 16)
    values = _scales(x.device)
    byte = torch.searchsorted(7 * values, g.abs().amax(-1)).clamp_max(TOP_SCALE)   # the smallest s with 7 s >= the largest
    scale = values[byte][..., None]
    codes = torch.where(scale > 0, torch.round(g / scale), torch.zeros((), device=x.device)).clamp(-7, 7)
    pair = (codes + 8).to(torch.uint8).view(n, 2, nkv, h // 2, 2)
    body = s["pool"][-1, ..., :page * h // 2].view(-1, 2, nkv, page, h // 2)
    body[at, :, :, place] = pair[..., 0] + 16 * pair[..., 1]
    s["pool"][-1, ..., page * h // 2:].view(-1, 2, nkv, page, h // 16)[at, :, :, place] = byte.to(torch.uint8)
    back = (codes * scale).view(n, 2, nkv, h).to(torch.bfloat16)
    s["k_back"][:n], s["v_back"][:n] = back[:, 0], back[:, 1]
    return [s["k_back"], s["v_back"]]


def _plain_context(s):
    """Keys and values of the requests' table, [batch, 2, kv heads, positions, h] fp32."""
    c = s["case"]
    B, nkv, h, page = c["batch"], c["nkv"], c["h"], c["page"]
    x = s["pool"][-1][s["table"].long()]
    if c["form"] == "int4":
        body = x[..., :page * h // 2]
        codes = torch.stack([body & 15, body >> 4], -1).float().sub_(8).view(*x.shape[:-1], page, h // 16, 16)
        scale = (x[..., page * h // 2:].to(torch.int16) << 7).view(torch.float16).float().view(*x.shape[:-1], page, h // 16, 1)
        x = codes.mul_(scale).view(*x.shape[:-1], page, h)
    return x.permute(0, 2, 3, 1, 4, 5).reshape(B, 2, nkv, -1, h).float()


def _visible(s, n_slots):
    """[batch, L, slots + block keys]: which keys a row sees."""
    c, dev = s["case"], s["lens"].device
    L, lens = c["block"], s["lens"].long()[:, None]
    pos = torch.arange(n_slots, device=dev)[None].expand(c["batch"], -1)
    there = pos < lens
    if c["blk"]:
        pos = torch.cat([pos, lens + torch.arange(L, device=dev)], 1)
        there = torch.cat([there, torch.ones(c["batch"], L, device=dev, dtype=torch.bool)], 1)
    row = (lens + (0 if c["blk"] else -L) + torch.arange(L, device=dev))[:, :, None]
    ok, pos = there[:, None].expand(-1, L, -1), pos[:, None]
    if c["window"]:
        ok = ok & ((pos < c["sinks"]) | (row - pos < c["window"]))
    return ok & (pos <= row) if c["causal"] else ok


def _plain_attention(s):
    c = s["case"]
    B, L, nq, nkv, h = c["batch"], c["block"], c["nq"], c["nkv"], c["h"]
    x = _plain_context(s)
    ok = _visible(s, x.shape[3])
    if c["blk"]:
        x = torch.cat([x, torch.stack([s["k_blk"], s["v_blk"]], 1).float()], 3)
    q = s["q"].float().view(B, L, nkv, -1, h).permute(0, 2, 3, 1, 4).reshape(B, nkv, -1, h) / math.sqrt(h)
    sc = (q @ x[:, 0].transpose(2, 3)).view(B, nkv, nq // nkv, L, -1)
    sc.masked_fill_(~ok[:, None, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros((), device=top.device), top)
    sc = sc.sub_(top).exp_()
    den = sc.sum(-1, keepdim=True)
    out = (sc.view(B, nkv, -1, sc.shape[-1]) @ x[:, 1]).view(B, nkv, -1, L, h)
    out = torch.where(den > 0, out / den, torch.zeros((), device=den.device))
    lse = (top + den.log())[..., 0]
    return [out.permute(0, 3, 1, 2, 4).reshape(B * L, nq, h).to(torch.bfloat16), lse.permute(0, 3, 1, 2).reshape(B * L, nq)]


def _plain_verify(s):
    c = s["case"]
    B, L = c["batch"], c["block"]
    d = s["draft"].long()[..., None]
    p = torch.gather(s["target"][:, :-1], 2, d)[..., 0].double()
    q = torch.gather(s["probs"], 2, d)[..., 0].double() if c["probs"] else 1.0
    ok = s["uniform"][:, :-1].double() * q < p
    n = torch.cumprod(ok.long(), 1).sum(1)
    each = torch.arange(B, device=n.device)
    # the last token comes from what the target has left over the drafter at the first refusal, or from its last row
    r = s["target"][each, n].double()
    last = torch.clamp_max(n, L - 2)
    if c["probs"]:
        left = (r - s["probs"][each, last].double()).clamp_min(0)
    else:
        left = r.clone()
        left[each, d[each, last, 0]] = 0
    r = torch.where((n < L - 1)[:, None] & (left.sum(1) > 0)[:, None], left, r)
    sums = torch.cumsum(r, 1)
    token = torch.searchsorted(sums, s["uniform"][:, -1:].double() * sums[:, -1:], right=True)[:, 0]
    at = torch.arange(L, device=n.device)[None]
    drafted = torch.cat([d[..., 0], token[:, None]], 1)
    committed = torch.where(at < n[:, None], drafted, torch.where(at == n[:, None], token[:, None], -1)).to(torch.int32)
    return [(n + 1).to(torch.int32), committed, (n == L - 1).to(torch.int32)]


# ---- the framework's calls ----------------------------------------------------------------------------------------------

def _store(s):
    """The handle of the pages, kept with the state as a serving loop keeps it."""
    import block_diffusion_speculative_non_gb300 as fpd
    if "store" not in s:
        c = s["case"]
        form = fpd.FPD_PAGE_INT4 if c["form"] == "int4" else fpd.FPD_PAGE_BF16
        s["store"] = fpd.paged_store(s["pool"], form, LAYERS, s["pool"].shape[1], c["page"], c["nkv"], c["h"], s["table"])
    return s["store"]


def _own_append(s):
    import block_diffusion_speculative_non_gb300 as fpd
    c, n, store = s["case"], s["total"], _store(s)
    nkv, h, ld = c["nkv"], c["h"], s["qkv"].shape[1]
    k, v = s["qkv"][:, 4 * nkv * h:5 * nkv * h], s["qkv"][:, 5 * nkv * h:]
    fpd.fpd_paged_append(c["batch"], n, store, LAYERS - 1, k, ld, v, ld, s["off"], None, s["lens"], s["pos_offset"], s["rope"],
                         s["rope"].shape[0])
    if c["form"] == "bf16":
        return [s["pool"]]
    fpd.fpd_paged_read(c["batch"], n, store, LAYERS - 1, s["off"], None, s["lens"], s["k_back"], s["v_back"])
    return [s["k_back"], s["v_back"]]


def _own_attention(s):
    import block_diffusion_speculative_non_gb300 as fpd
    c, store = s["case"], _store(s)
    if "workspace" not in s:
        need = fpd.fpd_paged_attention_workspace_bytes(c["batch"], c["block"], c["nq"], store)
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device=s["q"].device)
    ws = s["workspace"]
    fpd.fpd_paged_attention(c["batch"], c["block"], c["nq"], store, LAYERS - 1, s["q"], s["k_blk"], s["v_blk"], s["lens"],
                            c["window"], c["sinks"], c["causal"], s["out"], s["lse"], ws, ws.numel())
    return [s["out"], s["lse"]]


def _own_verify(s):
    import block_diffusion_speculative_non_gb300 as fpd
    c = s["case"]
    fpd.fpd_verify_sampled(c["batch"], c["block"], c["vocab"], s["draft"], s["target"], s["probs"], s["uniform"], s["accept"],
                           s["committed"], s["valid"])
    return [s["accept"], s["committed"], s["valid"]]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "attention": _own_attention, "verify": _own_verify}[op](state)
    return {"append": _plain_append, "attention": _plain_attention, "verify": _plain_verify}[op](state)


# ---- the definitions in 64 bits -----------------------------------------------------------------------------------------

def _exact_scale(big):
    """Scale of a group whose largest magnitude is `big`: the smallest of 8..15 times 2^e (e >= -17; less than 8 at the
    smallest e) that is at least a seventh of it, at most 2^13."""
    big = np.asarray(big, np.float64) / 7
    e = np.maximum(np.floor(np.log2(np.maximum(big, 2.0 ** -60))) - 3, -17)
    return np.minimum(np.ceil(big / 2.0 ** e) * 2.0 ** e, 8192.0)


def _exact_append(s):
    c, n = s["case"], s["total"]
    nkv, h, page = c["nkv"], c["h"], c["page"]
    kv = s["qkv"][:n, 4 * nkv * h:].float().cpu().numpy().astype(np.float64).reshape(n, 2, nkv, h)
    lens, rows, _ = _sizes(c)
    slot = np.concatenate([np.arange(a, a + r) for a, r in zip(lens, rows)]) if n else np.zeros(0, int)
    req = np.repeat(np.arange(c["batch"]), rows)
    table, first = s["table"].cpu().numpy(), s["pos_offset"].cpu().numpy()
    turn = s["rope"].cpu().numpy().astype(np.float64)[slot + first[req]]
    z = (kv[:, 0, :, :h // 2] + 1j * kv[:, 0, :, h // 2:]) * (turn[:, None, :, 0] + 1j * turn[:, None, :, 1])
    key = torch.from_numpy(np.concatenate([z.real, z.imag], -1)).to(torch.bfloat16).double().numpy()
    both = np.stack([key, kv[:, 1]])
    if c["form"] == "bf16":
        pool = s["pool"].double()
        where = torch.from_numpy(table[req, slot // page]).long().to(pool.device), torch.from_numpy(slot % page).to(pool.device)
        for i in range(2):
            pool[-1, :, i].permute(0, 2, 1, 3)[where] = torch.from_numpy(both[i]).to(pool.device)
        return [pool]
    g = both.reshape(2, n, nkv, h // 16, 16)
    scale = _exact_scale(np.abs(g).max(-1))[..., None]
    back = (np.clip(np.rint(g / np.where(scale > 0, scale, 1)), -7, 7) * scale).reshape(2, n, nkv, h)
    if not n:
        back = np.zeros((2, 1, nkv, h))
    return [torch.from_numpy(back[0]), torch.from_numpy(back[1])]


def _exact_attention(s):
    c = s["case"]
    B, L, nq, nkv, h, page = c["batch"], c["block"], c["nq"], c["nkv"], c["h"], c["page"]
    dev = s["q"].device
    q = s["q"].double().view(B, L, nkv, nq // nkv, h)
    out = torch.zeros(q.shape, dtype=torch.float64, device=dev)
    lse = torch.full(q.shape[:-1], -math.inf, dtype=torch.float64, device=dev)
    for b, n in enumerate(_lens(B, c["ctx"])):
        ids = s["table"][b, :-(-n // page)].long()
        for g in range(nkv):
            slab = s["pool"][-1, ids, :, g]
            kv = []
            for i in range(2):
                x = slab[:, i]
                if c["form"] == "int4":
                    half = page * h // 2
                    byte = x[:, :half].to(torch.int32)
                    code = torch.stack([byte % 16, byte // 16], -1).reshape(-1, h // 16, 16) - 8
                    bits = x[:, half:].to(torch.int32).reshape(-1, h // 16, 1)
                    e, m = bits // 8, bits % 8
                    x = code * torch.where(e > 0, (8 + m) * 2.0 ** (e - 18).double(), m * 2.0 ** -17)
                x = x.reshape(-1, h).double()[:n]
                kv.append(torch.cat([x, s["k_blk" if i == 0 else "v_blk"][b, g].double()]) if c["blk"] else x)
            total = kv[0].shape[0]
            if total == 0:
                continue
            key, row = torch.arange(total, device=dev)[None], torch.arange(total - L, total, device=dev)[:, None]
            hide = torch.zeros(L, total, dtype=torch.bool, device=dev)
            if c["window"]:
                hide |= (key >= c["sinks"]) & (key <= row - c["window"])
            if c["causal"]:
                hide |= key > row
            sc = torch.einsum("lih,th->lit", q[b, :, g], kv[0]) * h ** -0.5
            sc.masked_fill_(hide[:, None], -math.inf)
            lse[b, :, g] = torch.logsumexp(sc, -1)
            out[b, :, g] = torch.einsum("lit,th->lih", torch.nan_to_num(torch.softmax(sc, -1)), kv[1])
    return [out.reshape(B * L, nq, h), lse.reshape(B * L, nq)]


def _exact_verify(s):
    c = s["case"]
    B, L = c["batch"], c["block"]
    draft, u = s["draft"].cpu().numpy(), s["uniform"].cpu().numpy().astype(np.float64)
    accept, committed = np.zeros(B, np.int32), np.full((B, L), -1, np.int32)
    for b in range(B):
        n = 0
        while n < L - 1:
            q = float(s["probs"][b, n, draft[b, n]]) if c["probs"] else 1.0
            if not u[b, n] * q < float(s["target"][b, n, draft[b, n]]):
                break
            n += 1
        w = s["target"][b, n].cpu().numpy().astype(np.float64)
        if n < L - 1:
            less = w.copy()
            if c["probs"]:
                less = np.maximum(0, less - s["probs"][b, n].cpu().numpy())
            else:
                less[draft[b, n]] = 0
            w = less if less.any() else w
        up = np.cumsum(w)
        committed[b, :n], committed[b, n], accept[b] = draft[b, :n], int(np.argmax(up > u[b, -1] * up[-1])), n + 1
    return [accept, committed, (accept == L).astype(np.int32)]


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "verify": _exact_verify}[case["op"]](s)


# ---- work ---------------------------------------------------------------------------------------------------------------

def work(case):
    B = case["batch"]
    if case["op"] == "verify":
        # one row of each request, of the target and the drafter, and the drafted ids' entries
        return {"bytes": B * (case["vocab"] * (8 if case["probs"] else 4) + case["block"] * 20), "flops": 0}
    nkv, h = case["nkv"], case["h"]
    held = 2 * h if case["form"] == "bf16" else h // 2 + h // 16   # bytes of a stored row
    lens, rows, _ = _sizes(case)
    if case["op"] == "append":
        # keys and values in and into the pages, the angles of their positions; 4-bit pages: also what they stand for
        turns = max(rows) * h * 4
        return {"bytes": sum(rows) * 2 * nkv * (2 * h + held + (2 * h if case["form"] == "int4" else 0)) + turns, "flops": 0}
    L, grp = case["block"], case["nq"] // nkv
    lb = L if case["blk"] else 0
    seen, pairs = 0, 0
    for n in lens:
        row = np.arange(n + lb - L, n + lb)
        end = np.minimum(row + 1, n + lb) if case["causal"] else np.full(L, n + lb)
        end = np.maximum(end, 0)
        start = np.maximum(row - case["window"] + 1, 0) if case["window"] else np.zeros(L, int)
        first = np.minimum(np.minimum(case["sinks"], start), end) if case["window"] else np.zeros(L, int)
        pairs += int((np.maximum(end - start, 0) + first).sum())
        lo, hi = int(start.min()), int(end.max())   # the rows' ranges follow one another
        keys = max(0, hi - lo) + int(first.max())
        seen += keys * held - min(lb, keys) * (held - 2 * h)   # block keys come as bf16
    return {"bytes": B * L * case["nq"] * (4 * h + 4) + 2 * nkv * seen, "flops": 4 * h * grp * nkv * pairs}
