"""GPU: the paged context cache and the sampled verification against their definitions in 64 bits (tests/paged_ref.py).

Attention tolerances.  A score is an fp32 sum of h <= 128 products of unit-RMS rows (4-bit keys: what stands for such rows): their
absolute sum over sqrt(h) stays below 16 here, and each of the at most 16 accumulation steps is off by at most 2^-23 of it, so a score
is off by less than 16 * 16 * 2^-23 = 2^-15 (and is scaled in fp32: below 2^-17).  A weight of a bf16 page is then off by 2^-15
relative, 2^-17 more as two bf16 terms and 2^-22 from ex2: below 2^-14, in the numerator against max |v| and again in the
denominator.  A weight of a 4-bit page enters the second product as one fp16 number, half a step 2^-11, against max |v| once (the
denominator is summed in fp32).  out: (2 * 2^-14 + 2^-11 for 4 bits) max |v| plus the bf16 rounding, 2^-8 |out|.  lse: 2^-14.
`scale` > 1 multiplies q and with it every score error.  Appended keys and values, their codes and scales, and everything that
sampled verification returns are exact."""
import math

import numpy as np
import pytest
import torch

import paged_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


@pytest.fixture(scope="module")
def pkg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_diffusion_speculative_non_gb300 as p
    p.lib()
    return p


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def unit(gen, *shape):
    x = torch.randn(*shape, device=DEV, generator=gen)
    return x * x.square().mean(-1, keepdim=True).rsqrt()


class Pool:
    """A pool of pages with a random table.  What no length covers is stale: NaN in bf16 pages, any byte in 4-bit ones; table entries
    behind the last page of a request are not page ids."""

    def __init__(self, pkg, form, lens, nkv, h, page, seed=0, layers=2, extra=0, spare=2):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        self.pkg, self.form, self.nkv, self.h, self.page, self.layers, self.lens = pkg, form, nkv, h, page, layers, list(lens)
        B = len(lens)
        need = [-(-(n + extra) // page) for n in lens]
        self.width, self.n_pages = max(1, max(need)), sum(need) + spare
        perm = torch.randperm(self.n_pages, generator=gen, device=DEV).tolist()
        table = np.full((B, self.width), -77, np.int32)
        table[:, 1::2] = 1 << 29
        for b, n in enumerate(need):
            table[b, :n], perm = perm[:n], perm[n:]
        self.table = torch.from_numpy(table).to(DEV)
        self.int4 = form == "int4"
        self.slab = page * (h // 2 + h // 16) if self.int4 else page * h
        shape = (layers, self.n_pages, 2, nkv, self.slab)
        if self.int4:
            self.pages = torch.randint(0, 256, shape, device=DEV, generator=gen, dtype=torch.uint8)
        else:
            self.pages = torch.full(shape, math.nan, dtype=BF, device=DEV)
        self.keys, self.values = [], []   # what the last layer holds, [nkv, n, h] float64
        for b, n in enumerate(lens):
            k, v = unit(gen, nkv, n, h).to(BF).double(), torch.randn(nkv, n, h, device=DEV, generator=gen).to(BF).double()
            k, v = self.put(b, 0, k, v)
            self.keys.append(k)
            self.values.append(v)
        self.ctx_len = i32(lens)

    def put(self, b, at, k, v, layer=-1):
        """Writes rows [nkv, n, h] to slots at.. of request b, by the definition; returns what they stand for."""
        n, h, page = k.shape[1], self.h, self.page
        table = self.table[b].cpu().numpy()
        out = []
        for i, x in enumerate((k, v)):
            if self.int4:
                codes, byte = ref.quantise(x.cpu().numpy())
                cb, sb = ref.pack(codes, byte)
                out.append(torch.from_numpy(ref.stands_for(codes, byte)).to(DEV))
                cb, sb = torch.from_numpy(cb).to(DEV), torch.from_numpy(sb).to(DEV)
            else:
                out.append(x)
            for t0 in range(at - at % page, at + n, page):
                lo, hi = max(t0, at), min(t0 + page, at + n)
                if lo >= hi:
                    continue
                slab = self.pages[layer, int(table[t0 // page]), i]
                if self.int4:
                    slab[:, :page * h // 2].view(self.nkv, page, h // 2)[:, lo - t0:hi - t0] = cb[:, lo - at:hi - at]
                    slab[:, page * h // 2:].view(self.nkv, page, h // 16)[:, lo - t0:hi - t0] = sb[:, lo - at:hi - at]
                else:
                    slab.view(self.nkv, page, h)[:, lo - t0:hi - t0] = x[:, lo - at:hi - at].to(BF)
        return out

    def store(self, **kw):
        a = dict(pages=self.pages, format=int(self.int4), n_layers=self.layers, n_pages=self.n_pages, page_size=self.page,
                 n_kv_heads=self.nkv, head_dim=self.h, table=self.table)
        a.update(kw)
        return self.pkg.paged_store(**a)


class Problem:
    def __init__(self, pkg, form, lens, L, nq, nkv, h, page, blk=True, window=0, sinks=0, causal=False, seed=0, scale=1.0):
        self.pkg, self.pool, self.B, self.L, self.nq = pkg, Pool(pkg, form, lens, nkv, h, page, seed), len(lens), L, nq
        gen = torch.Generator(device=DEV).manual_seed(seed + 1000)
        self.mask, self.scale = (window, sinks, causal), scale
        self.q = (scale * unit(gen, self.B * L, nq, h)).to(BF)
        self.kb = unit(gen, self.B, nkv, L, h).to(BF) if blk else None
        self.vb = torch.randn(self.B, nkv, L, h, device=DEV, generator=gen).to(BF) if blk else None
        self.out = torch.full((self.B * L, nq, h), math.nan, dtype=BF, device=DEV)
        self.lse = torch.full((self.B * L, nq), math.nan, device=DEV)
        self.st = self.pool.store()

    def workspace(self):
        n = self.pkg.fpd_paged_attention_workspace_bytes(self.B, self.L, self.nq, self.st)
        assert n > 0
        return torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)   # fp32 NaN everywhere

    def run(self, ws=None, lse=True, stream=None):
        ws = self.workspace() if ws is None else ws
        self.pkg.fpd_paged_attention(self.B, self.L, self.nq, self.st, self.pool.layers - 1, self.q, self.kb, self.vb, self.pool.ctx_len,
                                     *self.mask, self.out, self.lse if lse else None, ws, ws.numel(), stream)
        return self.out, self.lse

    def want(self):
        k, v = self.pool.keys, self.pool.values
        if self.kb is not None:
            k = [torch.cat([a, self.kb[b].double()], 1) for b, a in enumerate(k)]
            v = [torch.cat([a, self.vb[b].double()], 1) for b, a in enumerate(v)]
        return ref.attention(self.q, k, v, self.L, *self.mask)

    def check(self, out, lse):
        want, wlse, vmax = self.want()
        tol = (2 * 2.0 ** -14 * self.scale + (2.0 ** -11 if self.pool.int4 else 0)) * vmax[..., None] + 2.0 ** -8 * want.abs()
        off = (out.double() - want).abs()
        assert not out.isnan().any() and bool((off <= tol).all()), float((off / tol.clamp_min(1e-30)).max())
        live = wlse > -math.inf
        assert torch.equal(lse == -math.inf, ~live) and not lse.isnan().any()
        assert bool(((lse.double() - wlse).abs()[live] <= 2.0 ** -14 * self.scale).all())
        assert (out[~live] == 0).all()
        return want


CASES = {
    "one_token": dict(lens=[1], L=1, nq=4, nkv=1, h=64, page=16),
    "tokens_ragged": dict(lens=[0, 1, 15, 16, 17, 63, 64, 65, 500], L=1, nq=8, nkv=2, h=64, page=16),
    "tokens_128": dict(lens=[700, 0, 33, 128], L=1, nq=32, nkv=8, h=128, page=32),
    "long_token": dict(lens=[9001], L=1, nq=8, nkv=2, h=128, page=64),
    "text": dict(lens=[300, 0, 129, 1, 2048], L=16, nq=32, nkv=8, h=128, page=64),
    "text_64": dict(lens=[130, 77], L=16, nq=16, nkv=4, h=64, page=128),
    "group_5": dict(lens=[200, 91, 12], L=7, nq=20, nkv=4, h=128, page=16),
    "group_1": dict(lens=[66, 0, 1000], L=3, nq=2, nkv=2, h=64, page=32),
    "group_3_rows_33": dict(lens=[310], L=11, nq=6, nkv=2, h=128, page=128),
    "group_16": dict(lens=[130, 64], L=2, nq=16, nkv=1, h=128, page=16),
    "group_128": dict(lens=[400, 3], L=3, nq=128, nkv=1, h=64, page=64),
    "primitive": dict(lens=[600, 37], L=385, nq=16, nkv=4, h=128, page=128),
    "primitive_64": dict(lens=[600, 37, 0], L=129, nq=8, nkv=2, h=64, page=16),
    "many_texts": dict(lens=[(61 * i) % 600 for i in range(45)], L=16, nq=32, nkv=8, h=128, page=64),
    "many_rows_24": dict(lens=[(61 * i) % 400 for i in range(60)], L=6, nq=16, nkv=4, h=64, page=32),
    "many_rows_96": dict(lens=[(47 * i) % 500 for i in range(40)], L=12, nq=32, nkv=4, h=128, page=16),
    "many_rows_160": dict(lens=[(83 * i) % 700 for i in range(30)], L=40, nq=16, nkv=4, h=64, page=128),
    "long_text": dict(lens=[7013], L=16, nq=4, nkv=1, h=128, page=64),
    "long_ragged": dict(lens=[8190, 0, 65], L=3, nq=4, nkv=1, h=64, page=16),
    "many": dict(lens=[(37 * i) % 90 for i in range(200)], L=2, nq=4, nkv=2, h=64, page=16),
}
MASKS = {"all": {}, "causal": dict(causal=True), "window": dict(window=50), "window_sinks": dict(window=33, sinks=5),
         "sinks_causal": dict(window=100, sinks=70, causal=True), "own": dict(window=1, causal=True),
         "appended": dict(blk=False), "appended_causal": dict(blk=False, causal=True),
         "appended_window": dict(blk=False, window=40, sinks=1, causal=True), "wide": dict(window=2 ** 31 - 1, sinks=2 ** 31 - 1)}


@pytest.mark.parametrize("form", ["bf16", "int4"])
@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("name", CASES)
def test_attention(pkg, name, mask, form):
    p = Problem(pkg, form, **CASES[name], **MASKS[mask], seed=len(name))
    p.check(*p.run())
    assert pkg.fpd_device_status() == 0


@pytest.mark.parametrize("form", ["bf16", "int4"])
@pytest.mark.parametrize("scale", [20.0, 400.0])
@pytest.mark.parametrize("name", ["tokens_128", "text", "group_5", "primitive"])
def test_large_scores(pkg, name, scale, form):
    p = Problem(pkg, form, **CASES[name], window=90, sinks=3, scale=scale)
    p.check(*p.run())


@pytest.mark.parametrize("form", ["bf16", "int4"])
def test_rows_without_a_key(pkg, form):
    """No key at all; and rows before position 0, which a causal block without block keys has where the context is shorter."""
    p = Problem(pkg, form, lens=[0, 0, 0], L=5, nq=8, nkv=2, h=64, page=16, blk=False)
    out, lse = p.run()
    assert (out == 0).all() and (lse == -math.inf).all()
    p = Problem(pkg, form, lens=[3, 0, 20], L=9, nq=8, nkv=2, h=128, page=16, blk=False, causal=True, window=4)
    out, lse = p.run()
    p.check(out, lse)
    assert (lse.view(3, 9, 8)[0, :6] == -math.inf).all() and (lse.view(3, 9, 8)[0, 6:] > -math.inf).all()


@pytest.mark.parametrize("name", ["tokens_128", "text", "primitive"])
def test_what_is_not_finite_reaches_rows_that_see_it_and_no_other_request(pkg, name):
    p = Problem(pkg, "bf16", **CASES[name], window=64, sinks=2)
    b, n = 0, CASES[name]["lens"][0]
    clean = [t.clone() for t in p.run()]
    spoilt = p.pool.pages.clone()
    k, v = p.pool.keys[b].clone(), p.pool.values[b].clone()
    k[0, 1], v[0, 1] = math.nan, math.inf          # a sink: every row of the request in kv head 0 sees it
    p.pool.put(b, 0, k, v)
    out, lse = p.run()
    L, grp = p.L, p.nq // p.pool.nkv
    hit = torch.zeros(p.B * L, p.nq, dtype=torch.bool, device=DEV)
    hit.view(p.B, L, p.nq)[b, :, :grp] = True
    assert out[hit].isnan().all() and lse[hit].isnan().all()
    assert torch.equal(out[~hit], clean[0][~hit]) and torch.equal(lse[~hit], clean[1][~hit])
    p.pool.pages.copy_(spoilt)
    k, v = p.pool.keys[b].clone(), p.pool.values[b].clone()
    k[:, n // 2], v[:, n // 2] = math.inf, math.nan   # where no row's window reaches
    assert n // 2 < n - 64 and n // 2 >= 2
    p.pool.put(b, 0, k, v)
    out, lse = p.run()
    assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])


@pytest.mark.parametrize("form", ["bf16", "int4"])
@pytest.mark.parametrize("mask", ["window_sinks", "sinks_causal", "causal", "appended_window"])
@pytest.mark.parametrize("name", ["tokens_128", "text", "group_5", "primitive_64", "group_16", "long_text", "long_ragged"])
def test_values_that_are_not_finite_stay_where_they_are_seen(pkg, name, mask, form):
    """Infinite and NaN values behind a window's start and later in a causal block: rows that do not see them are as they were, rows
    that do have no number in those dims."""
    p = Problem(pkg, form, **CASES[name], **MASKS[mask])
    window, sinks, causal = p.mask
    nkv, h, L, grp = p.pool.nkv, p.pool.h, p.L, p.nq // p.pool.nkv
    clean, wlse, vmax = p.want()
    sees = torch.zeros(p.B, L, p.nq, h, dtype=torch.bool, device=DEV)
    for b, n in enumerate(p.pool.lens):
        total = n + (L if p.kb is not None else 0)
        if total == 0:
            continue
        vis = torch.from_numpy(ref.visible(L, total, window, sinks, causal)).to(DEV)
        for t in {total - 1, total - L // 2 - 1, total - L - window + 1, total - L - window + L // 2, n // 3} & set(range(total)):
            value, dims = (math.nan, slice(0, h)) if t % 2 else (-math.inf, slice(3, h // 2))
            if t < n:
                if form == "int4":
                    continue   # a stored 4-bit value is finite
                v = p.pool.values[b][:1, t:t + 1].clone()
                v[..., dims] = value
                page = int(p.pool.table[b, t // p.pool.page])
                p.pool.pages[-1, page, 1].view(nkv, p.pool.page, h)[0, t % p.pool.page] = v[0, 0].to(BF)
            else:
                p.vb[b, 0, t - n, dims] = value
            sees[b, :, :grp, dims] |= vis[:, t, None, None]
    out, lse = p.run()
    sees = sees.view(p.B * L, p.nq, h)
    assert not out[sees].isfinite().any()
    tol = (2 * 2.0 ** -14 + (2.0 ** -11 if form == "int4" else 0)) * vmax[..., None] + 2.0 ** -8 * clean.abs()
    assert bool(((out.double() - clean).abs() <= tol)[~sees].all())
    live = wlse > -math.inf
    assert bool(((lse.double() - wlse).abs()[live] <= 2.0 ** -14).all()) and pkg.fpd_device_status() == 0


def test_scores_of_minus_infinity(pkg):
    """Infinite keys that give every visible key of a row the score -inf: weight 0, not NaN, beside keys that count."""
    p = Problem(pkg, "bf16", lens=[40, 70], L=2, nq=4, nkv=2, h=64, page=16, blk=False)
    p.q.abs_()
    k = p.pool.keys[0].clone()
    k[:] = -math.inf
    p.pool.put(0, 0, k, p.pool.values[0])
    out, lse = p.run()
    assert (out[:2] == 0).all() and (lse[:2] == -math.inf).all() and not out.isnan().any()
    k = p.pool.keys[1].clone()
    k[:, ::2] = -math.inf
    p.pool.keys[1], keep = k[:, 1::2], p.pool.put(1, 0, k, p.pool.values[1])
    p.pool.values[1] = p.pool.values[1][:, 1::2]
    want, wlse, _ = ref.attention(p.q, p.pool.keys, p.pool.values, 2, 0, 0, False)
    out, lse = p.run()
    assert (out[2:].double() - want[2:]).abs().max() < 0.03 and (lse[2:].double() - wlse[2:]).abs().max() < 2.0 ** -14


@pytest.mark.parametrize("form", ["bf16", "int4"])
@pytest.mark.parametrize("name", ["tokens_ragged", "text", "primitive", "long_token"])
def test_repeats_are_bit_identical_and_lse_is_optional(pkg, name, form):
    p = Problem(pkg, form, **CASES[name])
    out, lse = (t.clone() for t in p.run())
    for k in range(3):
        p.out.fill_(7)
        p.lse.fill_(7)
        o, _ = p.run(lse=k < 2)
        assert torch.equal(o, out) and (k == 2 or torch.equal(p.lse, lse))
    assert (p.lse == 7).all()


@pytest.mark.parametrize("form", ["bf16", "int4"])
@pytest.mark.parametrize("name", ["tokens_ragged", "text", "primitive_64"])
def test_captured_call_follows_lengths_and_table(pkg, name, form):
    p = Problem(pkg, form, **CASES[name], window=70, sinks=3)
    ws = p.workspace()
    p.run(ws)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            p.run(ws)
    torch.cuda.current_stream().wait_stream(s)
    rng = np.random.default_rng(1)
    for k in range(3):
        lens = [int(rng.integers(0, n + 1)) for n in CASES[name]["lens"]]
        p.pool.ctx_len.copy_(i32(lens))
        if k == 2:   # the same pages in other places
            to = torch.randperm(p.pool.n_pages, device=DEV)
            moved = torch.empty_like(p.pool.pages)
            moved[:, to] = p.pool.pages
            p.pool.pages.copy_(moved)
            held = (p.pool.table >= 0) & (p.pool.table < p.pool.n_pages)
            p.pool.table[held] = to[p.pool.table[held].long()].int()
        ws.fill_(0xFF)
        p.out.fill_(math.nan)
        g.replay()
        keep = p.pool.keys, p.pool.values
        p.pool.keys, p.pool.values = [x[:, :n] for x, n in zip(keep[0], lens)], [x[:, :n] for x, n in zip(keep[1], lens)]
        p.check(p.out, p.lse)
        p.pool.keys, p.pool.values = keep


def test_workspace_at_any_16_byte_offset(pkg):
    p = Problem(pkg, "bf16", **CASES["text"])
    out, lse = (t.clone() for t in p.run())
    n = p.workspace().numel()
    for off in (16, 48, 240):
        buf = torch.full((n + 512,), 0xFF, dtype=torch.uint8, device=DEV)
        p.out.fill_(7)
        p.run(buf[off:off + n])
        assert torch.equal(p.out, out) and (buf[:off] == 0xFF).all() and (buf[off + n:] == 0xFF).all()
    with pytest.raises(pkg.FpdError, match="workspace"):
        p.run(buf[:n - 256])


@pytest.mark.parametrize("form", ["bf16", "int4"])
def test_two_graphs_share_a_workspace(pkg, form):
    ps = [Problem(pkg, form, **CASES[name], causal=True) for name in ("many_texts", "primitive", "tokens_128")]
    want = [tuple(t.clone() for t in p.run()) for p in ps]
    ws = torch.full((max(p.workspace().numel() for p in ps),), 0xFF, dtype=torch.uint8, device=DEV)
    graphs, s = [], torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for p in ps:
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=s):
                p.run(ws)
    torch.cuda.current_stream().wait_stream(s)
    for turn in ((0, 1, 2), (2, 0, 1), (1, 0, 0, 2)):
        for p in ps:
            p.out.fill_(math.nan)
        for i in turn:
            graphs[i].replay()
        for p, (out, lse) in zip(ps, want):
            assert torch.equal(p.out, out) and torch.equal(p.lse, lse)


def test_more_key_tiles_than_31_bits_are_refused(pkg):
    B, nkv, h = 64, 8, 64
    pages = torch.zeros(pkg.fpd_page_bytes(pkg.FPD_PAGE_BF16, 16, nkv, h) // 2, dtype=BF, device=DEV)
    table = i32([[0]] * B)   # never read: the sizes are refused before a launch
    st = pkg.paged_store(pages, pkg.FPD_PAGE_BF16, 1, 1, 16, nkv, h, table.data_ptr(), table_width=2 ** 30 // 16)
    assert pkg.fpd_paged_attention_workspace_bytes(B, 1, nkv, st) == 0
    q = torch.zeros(B, nkv, h, dtype=BF, device=DEV)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    with pytest.raises(pkg.FpdError, match="31 bits"):
        pkg.fpd_paged_attention(B, 1, nkv, st, 0, q, None, None, i32([0] * B), 0, 0, False, torch.empty_like(q), None, ws, ws.numel())


@pytest.mark.parametrize("form", ["bf16", "int4"])
def test_two_streams_two_workspaces(pkg, form):
    ps = [Problem(pkg, form, **CASES[n], seed=i) for i, n in enumerate(("text", "primitive"))]
    want = [[t.clone() for t in p.run()] for p in ps]
    streams, ws = [torch.cuda.Stream() for _ in ps], [p.workspace() for p in ps]
    torch.cuda.synchronize()
    for _ in range(5):
        for p, s, w in zip(ps, streams, ws):
            p.out.fill_(7)
            s.wait_stream(torch.cuda.current_stream())
            p.run(w, stream=s)
    torch.cuda.synchronize()
    for p, (o, l) in zip(ps, want):
        assert torch.equal(p.out, o) and torch.equal(p.lse, l)


@pytest.mark.parametrize("form", ["bf16", "int4"])
def test_pages_past_32_bit_offsets(pkg, form):
    """Pages whose bytes lie past 2^32 and 2^33 of a layer, and a second layer behind them."""
    nkv, h, page = 8, 128, 128
    one = pkg.fpd_page_bytes(int(form == "int4"), page, nkv, h)
    n_pages = (1 << 33) // one + 5
    pages = torch.empty(2 * n_pages * one, dtype=torch.uint8, device=DEV)
    small = Problem(pkg, form, lens=[300, 129, 0], L=3, nq=32, nkv=nkv, h=h, page=page)
    out, lse = (t.clone() for t in small.run())
    raw = small.pool.pages[-1].view(torch.uint8).reshape(small.pool.n_pages, one) if form == "bf16" else small.pool.pages[-1].reshape(-1, one)
    far = [n_pages - 1 - i * 2 for i in range(small.pool.n_pages)]
    layer = pages.view(2, n_pages, one)[1]
    for i, f in enumerate(far):
        layer[f] = raw[i]
    held = (small.pool.table >= 0) & (small.pool.table < small.pool.n_pages)
    small.pool.table[held] = i32(far)[small.pool.table[held].long()]
    small.st = small.pool.store(pages=pages.view(BF) if form == "bf16" else pages, n_pages=n_pages)
    small.out.fill_(7)
    small.run()
    assert torch.equal(small.out, out) and torch.equal(small.lse, lse)
    k, v = torch.zeros(429, nkv, h, dtype=BF, device=DEV), torch.zeros(429, nkv, h, dtype=BF, device=DEV)
    pkg.fpd_paged_read(3, 429, small.st, 1, i32([0, 300, 429, 429]), None, None, k, v)
    for b, (x, y) in enumerate(((0, 300), (300, 429))):
        assert torch.equal(k[x:y].double(), small.pool.keys[b].transpose(0, 1)) and torch.equal(v[x:y].double(), small.pool.values[b].transpose(0, 1))


def test_lengths_and_pages_outside_are_recorded(pkg):
    p = Problem(pkg, "bf16", lens=[64, 64], L=2, nq=8, nkv=2, h=64, page=32)
    out, lse = (t.clone() for t in p.run())
    p.pool.ctx_len.copy_(i32([-5, 1000]))
    p.run()
    assert pkg.fpd_device_status() == 5
    assert torch.equal(p.out[2:], out[2:])
    p.pool.ctx_len.copy_(i32([64, 64]))
    p.pool.table[0, 1] = p.pool.n_pages
    p.run()
    assert pkg.fpd_device_status() == 8
    assert torch.equal(p.out[2:], out[2:]) and not p.out.isnan().any()
    k = torch.full((128, 2, 64), 7, dtype=BF, device=DEV)
    pkg.fpd_paged_read(2, 128, p.st, 1, i32([0, 64, 128]), None, None, k, k.clone())
    assert pkg.fpd_device_status() == 8 and (k[32:64] == 7).all() and not (k[64:] == 7).all()


# ---- append and read -----------------------------------------------------------------------------------------------------

APPENDS = {
    "steps": dict(lens=[0, 5, 16, 499], rows=[1, 1, 1, 1], nkv=2, h=64, page=16),
    "ragged": dict(lens=[0, 3, 64, 100, 7], rows=[40, 0, 16, 129, 1], nkv=8, h=128, page=64),
    "prompt": dict(lens=[0], rows=[700], nkv=1, h=128, page=128),
    "heads_3": dict(lens=[31, 0], rows=[33, 95], nkv=3, h=64, page=32),
    "heads_40": dict(lens=[2, 9], rows=[5, 6], nkv=40, h=128, page=16),
    "nothing": dict(lens=[4, 4], rows=[0, 0], nkv=2, h=64, page=16),
}


def append_want(pool, lens, rows, k, v, off, table, offset, counts=None):
    """What an append leaves in the last layer: writes into the pool by the definition."""
    for b, n in enumerate(rows):
        n = n if counts is None else min(n, counts[b])
        if n == 0:
            continue
        kk, vv = k[off[b]:off[b] + n].double().cpu().numpy(), v[off[b]:off[b] + n].double()
        if table is not None:
            pos = np.arange(lens[b], lens[b] + n) + offset[b]
            kk = ref.rotate(kk, table.cpu().numpy().astype(np.float64)[pos][:, None])
        pool.put(b, lens[b], torch.from_numpy(kk).to(DEV).transpose(0, 1), vv.transpose(0, 1))


@pytest.mark.parametrize("form", ["bf16", "int4"])
@pytest.mark.parametrize("turn", [True, False])
@pytest.mark.parametrize("name", APPENDS)
def test_append_and_read(pkg, name, turn, form):
    c = APPENDS[name]
    lens, rows, nkv, h = c["lens"], c["rows"], c["nkv"], c["h"]
    pool = Pool(pkg, form, lens, nkv, h, c["page"], extra=max(rows))
    gen = torch.Generator(device=DEV).manual_seed(9)
    total, off = sum(rows), np.concatenate([[0], np.cumsum(rows)]).tolist()
    wide = torch.randn(total + 3, (2 * nkv + 3) * h, device=DEV, generator=gen).to(BF)   # rows of a fused projection
    k, v = wide[:, h:(nkv + 1) * h], wide[:, (nkv + 2) * h:(2 * nkv + 2) * h]
    offset = [11 * b for b in range(len(lens))]
    rope = pkg.rope_table(max(lens) + max(rows) + 11 * len(lens), h, 1e6)
    before = pool.pages.clone()
    pkg.fpd_paged_append(len(lens), total, pool.store(), 1, k, wide.shape[1], v, wide.shape[1], i32(off), None, pool.ctx_len,
                         i32(offset) if turn else None, rope if turn else None, rope.shape[0] if turn else 0)
    got = pool.pages.clone()
    pool.pages.copy_(before)
    heads = [x[:total].reshape(total, nkv, h) for x in (k, v)]
    append_want(pool, lens, rows, *heads, off, rope if turn else None, offset)
    assert torch.equal(got.view(torch.uint8), pool.pages.view(torch.uint8))   # every byte, stale ones and other layers too
    pool.pages.copy_(got)
    kb, vb = torch.full((total + 1, nkv, h), 9, dtype=BF, device=DEV), torch.full((total + 1, nkv, h), 9, dtype=BF, device=DEV)
    pkg.fpd_paged_read(len(lens), total, pool.store(), 1, i32(off), None, pool.ctx_len, kb, vb)
    want = heads[1].double()
    if form == "int4":
        want = torch.from_numpy(ref.stands_for(*ref.quantise(want.cpu().numpy()))).to(DEV)
    assert torch.equal(vb[:total].double(), want) and (kb[total:] == 9).all() and (vb[total:] == 9).all()
    if not turn and form == "bf16":
        assert torch.equal(kb[:total], heads[0])
    assert pkg.fpd_device_status() == 0


@pytest.mark.parametrize("form", ["bf16", "int4"])
def test_append_counts_and_rows_that_do_not_fit(pkg, form):
    lens, rows, nkv, h = [10, 0, 3], [20, 9, 30], 2, 64
    pool = Pool(pkg, form, lens, nkv, h, 16, extra=30)
    gen = torch.Generator(device=DEV).manual_seed(2)
    off = [0, 20, 29, 59]
    k, v = (torch.randn(64, nkv, h, device=DEV, generator=gen).to(BF) for _ in range(2))
    rope = pkg.rope_table(26, h, 1e6)
    before = pool.pages.clone()
    # fewer rows than their room; positions from 26 on have no angle; rows past row_off[batch] (launched for 64) are not written
    counts = [20, 0, 5]
    pkg.fpd_paged_append(3, 64, pool.store(), 1, k, nkv * h, v, nkv * h, i32(off), i32(counts), pool.ctx_len, None, rope, 26)
    assert pkg.fpd_device_status() == 6
    got = pool.pages.clone()
    pool.pages.copy_(before)
    append_want(pool, lens, rows, k, v, off, rope, [0, 0, 0], [16, 0, 5])
    assert torch.equal(got.view(torch.uint8), pool.pages.view(torch.uint8))
    # slots before the table, behind it, and on a page that is none
    for start, code in (([-40, pool.width * 16, pool.width * 16 - 1], 6), ([0, 0, 0], 0)):
        pool.pages.copy_(before)
        if code == 0:
            pool.table[0, 0], code = pool.n_pages, 8
        pkg.fpd_paged_append(3, 59, pool.store(), 1, k, nkv * h, v, nkv * h, i32(off), i32([1, 1, 1] if code == 6 else [1, 0, 0]),
                             i32(start), None, None, 0)
        assert pkg.fpd_device_status() in (code, 8)


def test_four_bit_codes_at_the_edges(pkg):
    """Ties, zeros, the smallest and largest scales, subnormal and non-finite numbers, all bf16 numbers as a group's largest."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(BF)
    rng = np.random.default_rng(4)
    rows = []
    big = bits[~bits.isnan()].double().numpy()
    mix = np.clip(rng.integers(-15, 16, (len(big), 15)) / 14.0, -1, 1) * np.where(np.isinf(big), 1e38, np.abs(big))[:, None]   # ties and steps
    rows.append(np.concatenate([big[:, None], mix], 1))
    odd = rng.choice([0.0, -0.0, 1.0, -3.5, math.inf, -math.inf, math.nan, 1e-30, 57344.0, 65536.0, 2.0 ** -17], (4096, 16))
    rows.append(odd)
    x = np.concatenate(rows)
    x = x[:len(x) // 4 * 4].reshape(-1, 1, 64)
    k = torch.from_numpy(x).to(torch.float32).to(BF).to(DEV)
    n = k.shape[0]
    pool = Pool(pkg, "int4", [0], 1, 64, 128, extra=n)
    pkg.fpd_paged_append(1, n, pool.store(), 1, k, 64, k, 64, i32([0, n]), None, None, None, None, 0)
    got = pool.pages.clone()
    pool.put(0, 0, k.double().transpose(0, 1), k.double().transpose(0, 1))
    assert torch.equal(got, pool.pages)
    kb, vb = torch.empty_like(k), torch.empty_like(k)
    pkg.fpd_paged_read(1, n, pool.store(), 1, i32([0, n]), None, None, kb, vb)
    want = ref.stands_for(*ref.quantise(k.double().cpu().numpy()))
    assert torch.equal(kb.double().cpu(), torch.from_numpy(want)) and torch.equal(kb, vb)


def test_captured_append_follows_counts_and_positions(pkg):
    pool = Pool(pkg, "int4", [0, 0], 2, 64, 16, extra=64)
    k, v = (torch.randn(16, 2, 64, device=DEV).to(BF) for _ in range(2))
    off, cnt, start, rope, st = i32([0, 8, 16]), i32([0, 0]), i32([0, 0]), pkg.rope_table(64, 64, 1e6), pool.store()

    def call():
        pkg.fpd_paged_append(2, 16, st, 1, k, 128, v, 128, off, cnt, start, None, rope, 64)
    call()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            call()
    at = [0, 0]
    for c in ([3, 8], [0, 1], [8, 5]):
        before = pool.pages.clone()
        cnt.copy_(i32(c))
        start.copy_(i32(at))
        g.replay()
        got = pool.pages.clone()
        pool.pages.copy_(before)
        append_want(pool, at, [8, 8], k, v, [0, 8], rope, [0, 0], c)
        assert torch.equal(got, pool.pages)
        at = [a + b for a, b in zip(at, c)]


# ---- sampled verification ------------------------------------------------------------------------------------------------

def verify(pkg, draft, target, probs, uniform, valid=True):
    B, L, V = target.shape
    acc, com, val = i32([-9] * B), torch.full((B, L), -9, dtype=torch.int32, device=DEV), i32([-9] * B)
    dev = [None if t is None else torch.as_tensor(t).to(DEV) for t in (draft, target, probs, uniform)]
    pkg.fpd_verify_sampled(B, L, V, dev[0].int(), dev[1], dev[2], dev[3], acc, com, val if valid else None)
    return acc.tolist(), com.tolist(), val.tolist()


def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("B,L,V", [(1, 2, 1), (3, 2, 2), (40, 5, 7), (64, 16, 33), (9, 40, 1000), (5, 3, 4096), (2, 700, 5), (3, 4, 16385),
                                   (2, 3, 16400), (3, 6, 20001), (2, 4, 50000)])
def test_verify_sampled(pkg, B, L, V, probs):
    rng = np.random.default_rng(B * 1000 + V)
    t = rng.normal(size=(B, L, V)) * 2
    p, q = softmax(t), softmax(t[:, :-1] + 0.4 * rng.normal(size=(B, L - 1, V)))
    draft = np.stack([[rng.choice(V, p=q[b, i].astype(np.float64) / q[b, i].astype(np.float64).sum()) if probs else q[b, i].argmax()
                       for i in range(L - 1)] for b in range(B)]).astype(np.int32)
    u = rng.random((B, L)).astype(np.float32)
    u[0, -1] = 0
    u[-1, -1] = np.nextafter(np.float32(1), np.float32(0))
    if B > 2:
        u[1, 0] = 0
    acc, com, val = verify(pkg, draft, p, q if probs else None, u)
    for b in range(B):
        assert (acc[b], com[b], val[b]) == ref.verify_sampled(draft[b], p[b], q[b] if probs else None, u[b]), b
    assert verify(pkg, draft, p, q if probs else None, u, valid=False)[:2] == (acc, com)
    assert pkg.fpd_device_status() == 0


@pytest.mark.parametrize("V", [6, 16388])
def test_verify_sampled_at_the_edges(pkg, V):
    """Rows without probability, without anything left over the drafter, with negative and NaN entries, weights that do not sum to 1,
    very small ones, ids outside the vocabulary."""
    L, rows = 3, []

    def row(p0, p1, p2, q0, q1, draft, u):
        rows.append([np.zeros((3, V), np.float32), np.zeros((2, V), np.float32), draft, u])
        for i, w in enumerate((p0, p1, p2)):
            for k, x in w.items():
                rows[-1][0][i, k] = x
        for i, w in enumerate((q0, q1)):
            for k, x in w.items():
                rows[-1][1][i, k] = x

    e, nan = V - 1, math.nan
    one = {0: 0.5, e: 0.5}
    row(one, one, one, one, one, [0, e], [0.99, 0.99, 0.5])            # all kept
    row({e: 1.0}, one, one, {0: 1.0}, one, [0, 0], [0.0, 0.5, 0.7])    # p(d) = 0 is never kept
    row({0: 0.3, 2: 0.3}, one, one, {0: 0.9, 2: 0.9}, one, [0, 0], [0.9, 0.5, 0.6])   # nothing left: the target's own row
    row({}, one, one, one, one, [0, 0], [0.5, 0.5, 0.5])               # no probability at all
    row({0: -1.0, 1: nan, 3: 0.25}, one, one, {0: 0.5, 1: nan, 3: -2.0}, one, [1, 0], [0.1, 0.5, 0.9])
    row({0: 40.0, 3: 24.0}, one, one, {0: 8.0, 3: 30.0}, one, [3, 0], [0.9, 0.5, 0.3])   # weights
    row({0: 1e-38, 1: 3e-39, e: 1e-44}, one, one, {0: 1e-39}, one, [2, 0], [0.5, 0.5, 0.95])
    row(one, one, one, one, one, [-1, 0], [0.0, 0.0, 0.2])             # ids outside the vocabulary
    row(one, one, one, one, one, [0, V], [0.0, 0.0, 0.8])
    row({0: 1.0}, {0: 1.0, 1: 2.0 ** -60}, one, {0: 1.0}, {0: 1.0}, [0, 0], [0.5, 1.0, 0.5])   # u = 1 refuses equals; 2^-60 is left
    p, q, draft, u = (np.stack([np.asarray(r[i]) for r in rows]) for i in range(4))
    u = u.astype(np.float32)
    for probs in (q, None):
        acc, com, val = verify(pkg, draft.astype(np.int32), p, probs, u)
        for b in range(len(rows)):
            assert (acc[b], com[b], val[b]) == ref.verify_sampled(draft[b], p[b], None if probs is None else q[b], u[b]), (b, probs is None)
        assert pkg.fpd_device_status() in (1, 3)


def test_verify_sampled_follows_the_targets_distribution(pkg):
    """Over a grid of both random numbers and the drafter's own draws, the first committed id comes as often as the target says."""
    p, q, N = np.array([0.5, 0.25, 0.125, 0.125], np.float32), np.array([0.125, 0.5, 0.25, 0.125], np.float32), 64
    g = (np.arange(N) + 0.5) / N
    u = np.stack(np.meshgrid(g, g, indexing="ij"), -1).reshape(-1, 2).astype(np.float32)
    B, seen = len(u), np.zeros(4)
    t, d = np.broadcast_to(p, (B, 2, 4)).copy(), np.broadcast_to(q, (B, 1, 4)).copy()
    for k in range(4):
        _, com, _ = verify(pkg, np.full((B, 1), k, np.int32), t, d, u)
        seen += q[k] * np.bincount(np.array(com)[:, 0], minlength=4) / B
    assert np.abs(seen - p).max() <= 1 / N


def test_verify_sampled_full_vocabulary(pkg):
    """The full vocabulary against the running sums in 64 bits, in which a row's draw is never nearer than 2^-40 to a border here."""
    B, L, V = 8, 4, 151936
    gen = torch.Generator(device=DEV).manual_seed(5)
    t = torch.randn(B, L, V, device=DEV, generator=gen) * 2
    p, q = torch.softmax(t, -1), torch.softmax(t[:, :-1] + 0.5 * torch.randn(B, L - 1, V, device=DEV, generator=gen), -1)
    draft, u = q.argmax(-1).int(), torch.rand(B, L, device=DEV, generator=gen)
    for probs in (q, None):
        acc, com, _ = verify(pkg, draft, p, probs, u)
        for b in range(B):
            n = acc[b] - 1
            r = p[b, n].double()
            if n < L - 1:
                if probs is not None:
                    r = (r - q[b, n].double()).clamp_min(0)
                else:
                    r[draft[b, n].long()] = 0
            c = torch.cumsum(r, 0)
            x = float(u[b, -1].double() * c[-1])
            assert float((c - x).abs().min()) > 2.0 ** -40
            assert com[b][n] == int((c > x).int().argmax())


# ---- together ------------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("form", ["bf16", "int4"])
def test_blocks_drafted_verified_and_appended(pkg, form):
    """Three speculative steps over pages: a block attends to its request's pages, is verified by given random numbers, and the kept
    positions' keys and values join the pages at the device's counts.  Each step's attention agrees with fpd_shared_attention over
    a contiguous store of what the pages hold."""
    B, L, nq, nkv, h, page, V, cap = 3, 6, 8, 2, 64, 16, 50, 128
    gen = torch.Generator(device=DEV).manual_seed(1)
    pool = Pool(pkg, form, [20, 0, 47], nkv, h, page, extra=3 * L)
    st, lens, rope = pool.store(), pool.ctx_len, pkg.rope_table(cap, h, 1e6)
    ws = torch.empty(pkg.fpd_paged_attention_workspace_bytes(B, L, nq, st), dtype=torch.uint8, device=DEV)
    off, anchor, start = i32([0, L, 2 * L, 3 * L]), i32([0] * B), i32([0] * B)
    acc, com, val = i32([0] * B), torch.zeros(B, L, dtype=torch.int32, device=DEV), i32([0] * B)
    host = lens.tolist()
    for step in range(3):
        q, kr = unit(gen, B * L, nq, h).to(BF), unit(gen, B * L, nkv, h).to(BF)
        v = torch.randn(B * L, nkv, h, device=DEV, generator=gen).to(BF)
        kb, vb = (x.view(B, L, nkv, h).transpose(1, 2).contiguous() for x in (kr, v))
        out, lse = torch.zeros(B * L, nq, h, dtype=BF, device=DEV), torch.zeros(B * L, nq, device=DEV)
        pkg.fpd_paged_attention(B, L, nq, st, 1, q, kb, vb, lens, 0, 0, False, out, lse, ws, ws.numel())
        # the same from a contiguous store
        rows = np.concatenate([[0], np.cumsum(host)]).tolist()
        k_all, v_all = (torch.zeros(max(1, rows[-1]), nkv, h, dtype=BF, device=DEV) for _ in range(2))
        pkg.fpd_paged_read(B, rows[-1], st, 1, i32(rows), None, None, k_all, v_all)
        flat = torch.zeros(1, B, 2, nkv, cap, h, dtype=BF, device=DEV)
        for b, n in enumerate(host):
            flat[0, b, 0, :, :n], flat[0, b, 1, :, :n] = (x[rows[b]:rows[b + 1]].transpose(0, 1) for x in (k_all, v_all))
        out2, lse2 = torch.zeros_like(out), torch.zeros_like(lse)
        w2 = torch.empty(pkg.fpd_shared_attention_workspace_bytes(B, L, nq, nkv, h, 0, cap), dtype=torch.uint8, device=DEV)
        pkg.fpd_shared_attention(B, L, nq, nkv, h, 0, q, kb, vb, None, 0, None, flat, cap, lens, out2, lse2, w2, w2.numel())
        vmax = max(float(v_all.abs().max()), float(v.abs().max()))
        tol = (4 * 2.0 ** -14 + (2.0 ** -11 if form == "int4" else 0)) * vmax + 2.0 ** -7 * out2.double().abs()
        assert bool(((out.double() - out2.double()).abs() <= tol).all()) and float((lse - lse2).abs().max()) < 2.0 ** -13
        t = softmax(torch.randn(B, L, V, generator=torch.Generator().manual_seed(step)).numpy() * 2)
        draft = torch.from_numpy(t[:, :-1].argmax(-1).astype(np.int32)).to(DEV)
        u = torch.rand(B, L, device=DEV, generator=gen)
        pkg.fpd_verify_sampled(B, L, V, draft, torch.from_numpy(t).to(DEV), None, u, acc, com, val)
        want = [ref.verify_sampled(draft[b].tolist(), t[b], None, u[b].tolist()) for b in range(B)]
        assert acc.tolist() == [w[0] for w in want] and com.tolist() == [w[1] for w in want]
        pkg.fpd_sd_advance(B, L, pool.width * page, acc, com, lens, start, anchor)
        assert start.tolist() == host
        before = pool.pages.clone()
        pkg.fpd_paged_append(B, B * L, st, 1, kr, nkv * h, v, nkv * h, off, acc, start, None, rope, cap)
        got = pool.pages.clone()
        pool.pages.copy_(before)
        append_want(pool, host, [L] * B, kr, v, [0, L, 2 * L], rope, [0] * B, acc.tolist())
        assert torch.equal(got.view(torch.uint8), pool.pages.view(torch.uint8))
        host = [a + n for a, n in zip(host, acc.tolist())]
        assert lens.tolist() == host
    assert pkg.fpd_device_status() == 0
