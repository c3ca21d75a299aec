"""GPU: the operators on a context store (fpd_shared_attention, fpd_context_weights, fpd_evict_context) against their
definitions in 64 bits (tests/context_ops_ref.py).

Tolerances.  A score is an fp32 sum of h <= 128 products of unit-RMS rows: the products' absolute sum over sqrt(h) stays
below 0.64 sqrt(128) = 7.3 on average (below 16 here), and every one of the at most 16 accumulation steps of 8 or 16
products is off by at most 2^-23 of it, so a score is off by less than 16 * 16 * 2^-23 = 2^-15 (and is scaled in fp32, 2^-24
of |s log2 e| < 64: below 2^-17).  A softmax weight is then off by 2^-15 relative, by 2^-17 more from entering the second
product as two bf16 terms, and by 2^-22 from ex2: below 2^-14 in all, in the numerator against max |v| and again in the
denominator.  out: 2 * 2^-14 max |v| plus the bf16 rounding, 2^-8 |out|.  lse: the relative error of a sum of weights, 2^-14
absolute.  weights: sums of positive terms, 2^-14 relative.  `scale` > 1 multiplies q and with it every score error."""
import math

import numpy as np
import pytest
import torch

import context_ops_ref as ref

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


def make_store(gen, layers, batch, nkv, cap, h, lens, stale=math.nan):
    """Keys and values; positions from each length on hold `stale`."""
    s = torch.empty(layers, batch, 2, nkv, cap, h, dtype=BF, device=DEV)
    s[:, :, 0] = unit(gen, layers, batch, nkv, cap, h).to(BF)
    s[:, :, 1] = torch.randn(layers, batch, nkv, cap, h, device=DEV, generator=gen).to(BF)
    for b, n in enumerate(lens):
        s[:, b, :, :, n:] = stale
    return s


class Problem:
    def __init__(self, B, L, nq, nkv, h, P, p_cap, lens, t_cap, blk, seed=0, scale=1.0, stale=math.nan, layers=2):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        self.shape, self.layer = (B, L, nq, nkv, h), layers - 1
        self.P, self.p_cap, self.lens, self.t_cap, self.scale = P, p_cap, lens, t_cap, scale
        self.q = (scale * unit(gen, B * L, nq, h)).to(BF)
        self.kb = unit(gen, B, nkv, L, h).to(BF) if blk else None
        self.vb = torch.randn(B, nkv, L, h, device=DEV, generator=gen).to(BF) if blk else None
        self.prefix = make_store(gen, layers, 1, nkv, p_cap, h, [P], stale) if p_cap else None
        self.store = make_store(gen, layers, B, nkv, t_cap, h, lens, stale) if t_cap else None
        self.p_len = i32([P]) if p_cap else None
        self.c_len = i32(lens) if t_cap else None
        self.out = torch.full((B * L, nq, h), math.nan, dtype=BF, device=DEV)
        self.lse = torch.full((B * L, nq), math.nan, device=DEV)

    def workspace(self, pkg):
        n = pkg.fpd_shared_attention_workspace_bytes(*self.shape, self.p_cap, self.t_cap)
        assert n > 0 or (not self.p_cap and not self.t_cap)
        return torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device=DEV)   # fp32 NaN everywhere

    def run(self, pkg, ws=None, lse=True, stream=None):
        ws = self.workspace(pkg) if ws is None else ws
        pkg.fpd_shared_attention(*self.shape, self.layer, self.q, self.kb, self.vb, self.prefix, self.p_cap, self.p_len,
                                 self.store, self.t_cap, self.c_len, self.out, self.lse if lse else None, ws, ws.numel(),
                                 stream)
        return self.out, self.lse

    def want(self):
        B, L, nq, nkv, h = self.shape
        return ref.attention(self.q, None if self.prefix is None else self.prefix[self.layer, 0], self.P,
                             None if self.store is None else self.store[self.layer], self.lens, self.kb, self.vb, B, L, nkv)

    def check(self, want=None, lse=True):
        out, l, vmax = self.want() if want is None else want
        err = (self.out.double() - out).abs() - 2.0 ** -8 * out.abs() - 2 * 2.0 ** -14 * self.scale * vmax[..., None]
        assert not (err > 0).any() and torch.isfinite(self.out.float()).all(), f"out off by {err.max().item():.2e} over its bound"
        if lse:
            none = l == -math.inf
            assert torch.equal(self.lse == -math.inf, none)
            d = (self.lse.double() - l)[~none].abs()
            assert d.numel() == 0 or d.max().item() <= 2.0 ** -14 * self.scale, d.max().item()


ATTN = {
    # B, L, nq, nkv, h, prefix, prefix cap, own lengths, own cap, block keys
    "one_token_one_key": (1, 1, 1, 1, 64, 1, 1, [0], 0, False),
    "one_token_block_only": (1, 1, 4, 2, 128, 0, 0, [0], 0, True),
    "decode_small": (4, 1, 8, 2, 64, 512, 512, [64, 38, 0, 9], 64, True),
    "decode_h128": (5, 1, 32, 8, 128, 777, 800, [3, 0, 64, 65, 1], 80, True),
    "text_block": (3, 16, 32, 8, 128, 2048, 2048, [256, 0, 131], 256, True),
    "group_5": (3, 7, 20, 4, 128, 1999, 2003, [131, 1, 0], 131, False),
    "group_3_h64": (2, 9, 6, 2, 64, 130, 130, [63, 64], 70, True),
    "group_1": (2, 33, 4, 4, 128, 127, 127, [128, 129], 129, True),
    "one_kv_head": (2, 16, 8, 1, 128, 4097, 4100, [5, 6], 8, True),
    "prefix_only": (4, 16, 32, 8, 128, 1000, 1000, [0] * 4, 0, False),
    "no_prefix": (4, 16, 8, 2, 128, 0, 0, [1, 127, 128, 300], 300, True),
    "empty_prefix": (2, 5, 8, 2, 128, 0, 40, [7, 0], 9, True),
    "tile_edges": (3, 8, 8, 2, 128, 64, 65, [63, 64, 65], 65, False),
    "tile_edges_128": (3, 40, 8, 2, 128, 128, 129, [127, 128, 129], 130, True),
    "long_block": (2, 385, 8, 2, 128, 300, 300, [77, 0], 128, True),
    "long_block_h64": (2, 200, 8, 2, 64, 1000, 1024, [0, 513], 600, True),
    "long_block_h64_tc": (2, 300, 8, 2, 64, 2500, 2511, [0, 513], 600, True),
    "many_rows": (24, 16, 8, 1, 128, 700, 704, [i * 5 for i in range(24)], 120, True),
    "wide_group": (9, 1, 128, 2, 128, 3000, 3000, [i for i in range(9)], 9, True),
    "long_prefix": (2, 1, 8, 2, 128, 70001, 70016, [500, 2], 512, True),
    # sizes on each side of the rules between the kernels: own parts on mma.sync beside the prefix on tcgen05, runs that span
    # units, one call without a prefix on tcgen05, heads per kv head that no 128 rows hold
    "many_text_blocks": (40, 16, 32, 8, 128, 1000, 1001, [(37 * i) % 65 for i in range(40)], 64, True),
    "many_text_blocks_h64": (40, 16, 16, 8, 64, 2100, 2100, [(37 * i) % 65 for i in range(40)], 64, False),
    "spanning_runs": (4, 385, 32, 8, 128, 1500, 1600, [128, 0, 5, 77], 128, True),
    "no_prefix_tc": (12, 40, 16, 4, 128, 0, 0, [(91 * i) % 700 for i in range(12)], 700, True),
    "prefix_only_tc": (16, 16, 20, 4, 128, 3001, 3001, [0] * 16, 0, False),
    "group_130": (3, 2, 130, 1, 128, 900, 900, [70, 0, 9], 70, True),
    "group_7_h64": (30, 16, 14, 2, 64, 1700, 1700, [i for i in range(30)], 31, True),
    "block_of_5000": (1, 5000, 2, 1, 128, 100, 100, [50], 64, True),
    "block_of_2900_h64": (2, 2900, 3, 3, 64, 0, 0, [50, 0], 64, True),
    "last_lane_only": (9, 15, 16, 4, 128, 2500, 2500, [i * 30 for i in range(9)], 256, True),
    # own units of which some CTAs take several before all take turns, or all of them; few rows of many requests on mma.sync
    "own_first_then_turns": (60, 4, 16, 8, 128, 500, 500, [(113 * i) % 901 for i in range(60)], 900, True),
    "own_apart": (20, 1, 32, 8, 128, 9000, 9000, [(113 * i) % 701 for i in range(20)], 700, False),
    "own_apart_h64": (40, 2, 16, 8, 64, 2999, 3000, [(113 * i) % 601 for i in range(40)], 600, True),
    "many_decodes": (150, 1, 16, 8, 128, 1500, 1500, [(7 * i) % 51 for i in range(150)], 50, True),
    "many_decodes_h64": (150, 1, 16, 8, 64, 1500, 1501, [(7 * i) % 51 for i in range(150)], 50, False),
}


@pytest.mark.parametrize("name", list(ATTN))
def test_shared_attention(pkg, name):
    p = Problem(*ATTN[name], seed=len(name))
    p.run(pkg)
    torch.cuda.synchronize()
    p.check()
    assert pkg.fpd_device_status() == 0


@pytest.mark.parametrize("h", [64, 128])
@pytest.mark.parametrize("L", [1, 48])
def test_rows_without_a_key(pkg, h, L):
    """Lengths of zero everywhere and no block keys: output 0 and lse -inf, beside requests that have keys."""
    p = Problem(3, L, 8, 2, h, 0, 16, [0, 5, 0], 16, False, seed=3)
    p.run(pkg)
    p.check()
    assert (p.out.view(3, L, 8, h)[0] == 0).all() and (p.lse.view(3, L, 8)[2] == -math.inf).all()
    q = Problem(2, L, 8, 2, h, 0, 0, [0, 0], 0, False, seed=3)   # neither store nor block
    q.run(pkg)
    assert (q.out == 0).all() and (q.lse == -math.inf).all()


@pytest.mark.parametrize("scale", [8.0, 40.0])
@pytest.mark.parametrize("name", ["decode_h128", "text_block", "many_rows", "long_block_h64", "long_block_h64_tc"])
def test_large_scores(pkg, name, scale):
    """Scores up to hundreds: one key takes nearly all of a row, the running maximum jumps."""
    p = Problem(*ATTN[name], seed=5, scale=scale)
    p.run(pkg)
    p.check()


@pytest.mark.parametrize("name", ["decode_h128", "text_block", "many_rows"])
def test_scores_of_minus_infinity(pkg, name):
    """Keys so large that q . k overflows to -inf get weight 0; a row that has other keys is not disturbed."""
    p = Problem(*ATTN[name], seed=6)
    B, L, nq, nkv, h = p.shape
    p.q[..., 0] = 1.0
    p.prefix[p.layer, 0, 0, :, : p.P // 2, 0] = -3.0e38
    p.prefix[p.layer, 0, 0, :, : p.P // 2, 1:] = 0
    p.q *= 8   # 8 * -3e38 overflows fp32; the other keys' first dimension stays of unit size
    p.scale = 8.0
    p.run(pkg)
    p.check()


@pytest.mark.parametrize("name", ["decode_h128", "text_block", "many_rows"])
def test_nan_reaches_its_own_rows_only(pkg, name):
    p = Problem(*ATTN[name], seed=7)
    p.run(pkg)
    clean = p.out.clone(), p.lse.clone()
    p.q[1] = math.nan
    p.run(pkg)
    assert p.out[1].isnan().all() and p.lse[1].isnan().all()
    keep = [r for r in range(p.q.shape[0]) if r != 1]
    assert torch.equal(p.out[keep], clean[0][keep]) and torch.equal(p.lse[keep], clean[1][keep])


@pytest.mark.parametrize("name", ["decode_small", "text_block", "group_5", "tile_edges_128", "long_block", "many_rows",
                                  "own_first_then_turns", "own_apart_h64", "many_decodes"])
def test_every_key_counts_once(pkg, name):
    """Keys of 0 make every weight equal; value t is 1 in dimension t % h, so output dimension d counts keys."""
    p = Problem(*ATTN[name], seed=8, stale=0.0)
    B, L, nq, nkv, h = p.shape
    one = lambda n: (torch.arange(n, device=DEV)[:, None] % h == torch.arange(h, device=DEV)).to(BF)
    for s, n in ((p.prefix, p.p_cap), (p.store, p.t_cap)):
        if s is not None:
            s[:, :, 0], s[:, :, 1] = 0, one(n)
    if p.kb is not None:
        p.kb.zero_()
        p.vb[:] = one(L)
    p.run(pkg)
    for b in range(B):
        cnt = one(p.P).double().sum(0) + one(p.lens[b]).double().sum(0) + (one(L).double().sum(0) if p.kb is not None else 0)
        total = cnt.sum()
        got = p.out.view(B, L, nq, h)[b].double()
        assert ((got - cnt / total).abs() <= 2.0 ** -8 * cnt / total + 2.0 ** -20).all(), b
        assert (p.lse.view(B, L, nq)[b].double() - math.log(total)).abs().max() < 2.0 ** -20


def test_repeats_are_bit_identical_and_lse_is_optional(pkg):
    for name in ("decode_h128", "long_block", "many_rows"):
        p = Problem(*ATTN[name], seed=9)
        p.run(pkg)
        a, l = p.out.clone(), p.lse.clone()
        p.out.fill_(math.nan)
        p.lse.fill_(math.nan)
        p.run(pkg, lse=False)
        assert torch.equal(p.out, a) and p.lse.isnan().all()
        p.run(pkg)
        assert torch.equal(p.lse, l)


@pytest.mark.parametrize("name", ["decode_h128", "text_block", "many_rows", "own_first_then_turns", "own_apart"])
def test_captured_call_follows_lengths_on_the_device(pkg, name):
    """One graph, replayed after the lengths on the device have changed; captured on a stream of its own."""
    p = Problem(*ATTN[name], seed=10, stale=0.5)
    ws = p.workspace(pkg)
    p.run(pkg, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.run(pkg, ws)
    for new in (p.P // 3, 0, p.P):
        p.P = new
        p.p_len.fill_(new)
        p.lens = [n // 2 for n in p.lens]
        p.c_len.copy_(i32(p.lens))
        ws.fill_(0xFF)
        p.out.fill_(math.nan)
        g.replay()
        torch.cuda.synchronize()
        p.check()


@pytest.mark.parametrize("name", ["prefix_only_tc", "no_prefix_tc"])
def test_nothing_to_attend_to_on_large_calls(pkg, name):
    """The same sizes with every length 0: no keys but the block's, or none at all."""
    p = Problem(*ATTN[name], seed=14)
    p.run(pkg)
    p.P, p.lens = 0, [0] * p.shape[0]
    for t in (p.p_len, p.c_len):
        if t is not None:
            t.zero_()
    p.run(pkg)
    p.check()
    assert pkg.fpd_device_status() == 0


def test_workspace_at_any_16_byte_offset(pkg):
    for name in ("text_block", "many_text_blocks"):
        p = Problem(*ATTN[name], seed=15)
        n = pkg.fpd_shared_attention_workspace_bytes(*p.shape, p.p_cap, p.t_cap)
        raw = torch.full((n + 512,), 0xFF, dtype=torch.uint8, device=DEV)
        for off in (16, 48, 112):
            p.out.fill_(math.nan)
            pkg.fpd_shared_attention(*p.shape, p.layer, p.q, p.kb, p.vb, p.prefix, p.p_cap, p.p_len, p.store, p.t_cap,
                                     p.c_len, p.out, p.lse, raw.data_ptr() + off, n)
            p.check()
        assert (raw[n + 112:] == 0xFF).all()


def test_stores_past_32_bit_offsets(pkg):
    """The layer, request and positions in use start past 2^32 elements; everything below them is another layer."""
    B, L, nq, nkv, h, cap = 2, 16, 8, 2, 128, 5_000_000
    need = 2 * B * 2 * nkv * cap * h * 2
    if torch.cuda.mem_get_info()[0] < need + (4 << 30):
        pytest.skip("needs %d GB" % (need >> 30))
    gen = torch.Generator(device=DEV).manual_seed(5)
    store = torch.empty(2, B, 2, nkv, cap, h, dtype=BF, device=DEV)
    lens = [1500, 1333]
    for b, n in enumerate(lens):
        store[1, b, 0, :, :n] = unit(gen, nkv, n, h).to(BF)
        store[1, b, 1, :, :n] = torch.randn(nkv, n, h, device=DEV, generator=gen).to(BF)
    q = unit(gen, B * L, nq, h).to(BF)
    small = store[1, :, :, :, :1600].contiguous()
    want, lse_want, vmax = ref.attention(q, None, 0, small, lens, None, None, B, L, nkv)
    out, lse = torch.empty(B * L, nq, h, dtype=BF, device=DEV), torch.empty(B * L, nq, device=DEV)
    # as the requests' own store, and request by request as a prefix (the store of one request, layer 2 + b of its kind)
    ws = torch.empty(max(pkg.fpd_shared_attention_workspace_bytes(B, L, nq, nkv, h, 0, cap),
                         pkg.fpd_shared_attention_workspace_bytes(1, L, nq, nkv, h, cap, 0)), dtype=torch.uint8, device=DEV)
    pkg.fpd_shared_attention(B, L, nq, nkv, h, 1, q, None, None, None, 0, None, store, cap, i32(lens), out, lse, ws, ws.numel())
    bound = 2.0 ** -8 * want.abs() + 2 * 2.0 ** -14 * vmax[..., None]
    assert ((out.double() - want).abs() <= bound).all() and (lse.double() - lse_want).abs().max() < 2.0 ** -14
    for b in range(B):
        o, l = torch.empty(L, nq, h, dtype=BF, device=DEV), torch.empty(L, nq, device=DEV)
        pkg.fpd_shared_attention(1, L, nq, nkv, h, 2 + b, q[b * L:(b + 1) * L].contiguous(), None, None, store, cap, i32(lens[b:b + 1]),
                                 None, 0, None, o, l, ws, ws.numel())
        sl = slice(b * L, (b + 1) * L)
        assert ((o.double() - want[sl]).abs() <= bound[sl]).all()
    w = torch.full((2, B, nkv, cap), -1.0, device=DEV)
    pkg.fpd_context_weights(B, L, nq, nkv, h, 1, q, lse, store, cap, i32(lens), w, False)
    ww = ref.context_weights(q, lse, small, lens, B, L, nkv)
    assert weights_close(w[1, :, :, :1600], ww) and (w[0] == -1).all() and (w[1, :, :, 1600:] == -1).all()
    w.clamp_min_(0)
    budget = 700
    ews = torch.empty(pkg.fpd_evict_workspace_bytes(2, B, nkv, budget), dtype=torch.uint8, device=DEV)
    n_d = i32(lens)
    store[0, :, :, :, :1600] = 0
    before = store[:, :, :, :, :1600].contiguous()
    wb = w[..., :1600].cpu().numpy()
    pkg.fpd_evict_context(2, B, nkv, h, budget, 100, store, cap, w, n_d, store, cap, w, n_d, None, None, ews, ews.numel())
    bn = before.view(torch.int16).cpu().numpy()
    o, ow, n, _ = ref.evict(bn, wb, lens, budget, 100, bn, 1600)
    assert np.array_equal(store[:, :, :, :, :1600].contiguous().view(torch.int16).cpu().numpy(), o)
    assert np.array_equal(w[..., :1600].cpu().numpy(), ow) and n_d.tolist() == [budget] * B
    assert pkg.fpd_device_status() == 0


def test_two_streams_two_workspaces(pkg):
    a, b = Problem(*ATTN["text_block"], seed=11), Problem(*ATTN["long_block"], seed=12)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    w1, w2 = a.workspace(pkg), b.workspace(pkg)
    torch.cuda.synchronize()
    for _ in range(3):
        a.run(pkg, w1, stream=s1)
        b.run(pkg, w2, stream=s2)
    torch.cuda.synchronize()
    a.check()
    b.check()


def test_lengths_outside_the_store_are_clamped_and_recorded(pkg):
    p = Problem(2, 4, 8, 2, 128, 64, 64, [10, 10], 10, True, seed=13)
    p.p_len.fill_(65)
    p.c_len.fill_(11)
    p.run(pkg)
    p.check()   # as with the capacities
    assert pkg.fpd_device_status() == 5
    p.p_len.fill_(-1)
    p.run(pkg)
    p.P = 0
    p.check()
    assert pkg.fpd_device_status() == 5


# ---- collected weights --------------------------------------------------------------------------------------------

WEIGHTS = {
    # B, L, nq, nkv, h, lengths, cap
    "one": (1, 1, 1, 1, 64, [1], 1),
    "small": (1, 16, 8, 2, 64, [128], 144),
    "ragged": (4, 16, 32, 8, 128, [700, 0, 65, 64], 701),
    "group_5": (2, 7, 20, 4, 128, [129, 127], 200),
    "group_3_h64": (3, 31, 6, 2, 64, [33, 1, 200], 300),
    "many_rows": (1, 700, 8, 2, 128, [1000], 1003),
    "many_rows_h64": (2, 300, 4, 1, 64, [513, 100], 513),
    "few_keys_many_rows": (1, 1024, 32, 2, 128, [17], 40),
    "single_token": (8, 1, 32, 8, 128, [2000, 1, 5, 64, 1999, 0, 3, 128], 2048),
    "wide_group": (2, 1, 128, 1, 128, [3000, 65], 3000),
    # tcgen05: 5 and 3 heads per kv head leave rows of a tile unused, 128 fill it with one position; more requests than a
    # warp counts at a time, some empty; few rows over long contexts
    "group_5_tc": (3, 60, 20, 4, 128, [129, 0, 127], 200),
    "group_3_h64_tc": (2, 100, 6, 2, 64, [257, 300], 300),
    "wide_group_tc": (2, 3, 128, 1, 128, [700, 65], 700),
    "many_requests_tc": (40, 40, 16, 4, 128, [(97 * i) % 300 if i % 7 else 0 for i in range(40)], 300),
    "few_rows_tc": (13, 4, 32, 8, 128, [1100 - 90 * i for i in range(13)], 1111),
    "few_rows_h64_tc": (26, 1, 16, 8, 64, [(211 * i) % 600 for i in range(26)], 600),
    "few_rows_long_h64_tc": (6, 1, 32, 8, 64, [9000, 1, 0, 4097, 513, 8192], 9000),
    "group_130": (2, 2, 130, 1, 128, [100, 65], 130),
    "nothing_tc": (2, 80, 8, 2, 128, [0, 0], 300),
}


def weight_problem(name, seed=0, scale=1.0):
    B, L, nq, nkv, h, lens, cap = WEIGHTS[name]
    p = Problem(B, L, nq, nkv, h, 0, 0, lens, cap, True, seed=seed, scale=scale)
    _, lse, _ = p.want()
    p.lse = lse.float()
    return p


def run_weights(pkg, p, w, accumulate=False):
    pkg.fpd_context_weights(*p.shape, p.layer, p.q, p.lse, p.store, p.t_cap, p.c_len, w, accumulate)


def weights_close(got, want, scale=1.0):
    rel = (got.double() - want).abs() / want.clamp_min(2.0 ** -100)
    return rel[~want.isnan()].numel() == 0 or rel[~want.isnan()].max().item() <= 2.0 ** -14 * scale


@pytest.mark.parametrize("name", list(WEIGHTS))
def test_context_weights(pkg, name):
    p = weight_problem(name, seed=len(name))
    B, L, nq, nkv, h = p.shape
    w = torch.full((2, B, nkv, p.t_cap), -7.0, device=DEV)
    run_weights(pkg, p, w)
    want = ref.context_weights(p.q, p.lse, p.store[p.layer], p.lens, B, L, nkv)
    assert (w[0] == -7).all() and torch.equal(w[1] == -7, want.isnan())   # another layer, and behind each length
    assert weights_close(w[1], want)
    first = w[1].clone()
    run_weights(pkg, p, w)
    assert torch.equal(w[1], first)   # written again, bit for bit
    run_weights(pkg, p, w, accumulate=True)
    assert torch.equal(w[1], torch.where(want.isnan(), first, first + first))
    assert pkg.fpd_device_status() == 0


@pytest.mark.parametrize("name", ["ragged", "many_rows"])
def test_weights_of_large_scores_and_of_rows_without_keys(pkg, name):
    p = weight_problem(name, seed=4, scale=20.0)
    B, L, nq, nkv, h = p.shape
    p.lse[0] = -math.inf        # a row that saw no key hands out nothing
    w = torch.zeros(2, B, nkv, p.t_cap, device=DEV)
    run_weights(pkg, p, w)
    assert weights_close(w[1], ref.context_weights(p.q, p.lse, p.store[p.layer], p.lens, B, L, nkv), 20.0)


@pytest.mark.parametrize("name", ["ragged", "many_requests_tc"])
def test_a_nan_query_spoils_its_own_request_only(pkg, name):
    p = weight_problem(name, seed=8)
    B, L, nq, nkv, h = p.shape
    w = torch.zeros(2, B, nkv, p.t_cap, device=DEV)
    run_weights(pkg, p, w)
    clean = w.clone()
    p.q[L + 1] = math.nan       # request 1
    run_weights(pkg, p, w)
    keep = [b for b in range(B) if b != 1]
    assert torch.equal(w[:, keep], clean[:, keep]) and w[1, 1, :, :p.lens[1]].isnan().all()


@pytest.mark.parametrize("name", ["small", "ragged", "group_5", "group_3_h64", "many_rows", "many_rows_h64", "group_5_tc", "group_3_h64_tc",
                                  "wide_group_tc", "few_rows_tc"])
def test_rows_without_a_key_give_nothing_whatever_they_hold(pkg, name):
    """A row with lse -inf is left out even where its query holds NaN or infinities (a padded position of a batch).  A key whose
    scores overflow to -inf has weight 0."""
    p = weight_problem(name, seed=17)
    B, L, nq, nkv, h = p.shape
    gen = torch.Generator(device=DEV).manual_seed(18)
    out = torch.rand(B * L, nq, device=DEV, generator=gen) < 0.3
    p.lse[out] = -math.inf
    p.q[out] = 0
    w = torch.zeros(2, B, nkv, p.t_cap, device=DEV)
    run_weights(pkg, p, w)
    clean = w.clone()
    assert weights_close(w[1], ref.context_weights(p.q, p.lse, p.store[p.layer], p.lens, B, L, nkv))
    for bad in (math.nan, math.inf, -math.inf):
        p.q[out] = bad
        run_weights(pkg, p, w)
        assert torch.equal(w, clean), bad
    p.q[out] = math.nan
    p.q[..., 0][~out] = 8
    p.store[p.layer, :, 0, :, :1, 0] = -3.0e38
    run_weights(pkg, p, w)
    assert (w[1, [b for b in range(B) if p.lens[b]], :, 0] == 0).all()
    assert weights_close(w[1], ref.context_weights(p.q, p.lse, p.store[p.layer], p.lens, B, L, nkv))


@pytest.mark.parametrize("name", ["small", "group_5", "many_rows", "group_3_h64_tc"])
def test_only_minus_infinity_means_no_key(pkg, name):
    """The lowest finite lse is a number: exp(s - lse) overflows to inf.  An lse of inf gives 0, NaN gives NaN."""
    B, _, _, nkv, _ = WEIGHTS[name][:5]
    for value, want in ((torch.finfo(torch.float32).min, math.inf), (math.inf, None), (math.nan, math.nan)):
        q = weight_problem(name, seed=19)
        q.lse[0, 0] = value                        # kv head 0 of request 0
        w, clean = torch.zeros(2, B, nkv, q.t_cap, device=DEV), torch.zeros(2, B, nkv, q.t_cap, device=DEV)
        run_weights(pkg, q, w)
        q.lse[0, 0] = -math.inf                    # the same without the row
        run_weights(pkg, q, clean)
        got, rest = w[1, 0, 0, :q.lens[0]], clean[1, 0, 0, :q.lens[0]]
        if want is None:
            assert torch.equal(got, rest)
        else:
            assert torch.equal(got, torch.full_like(got, want)) or (math.isnan(want) and got.isnan().all())
        w[1, 0, 0], clean[1, 0, 0] = 0, 0
        assert torch.equal(w, clean)


def test_rows_hand_out_one_in_all(pkg):
    """Without block keys, the weights of a request's positions and its share of the prefix's add up to its rows."""
    p = Problem(3, 16, 32, 8, 128, 500, 512, [100, 0, 33], 128, False, seed=21)
    B, L, nq, nkv, h = p.shape
    p.run(pkg)
    w, pw = torch.zeros(2, B, nkv, 128, device=DEV), torch.zeros(2, 1, nkv, 512, device=DEV)
    run_weights(pkg, p, w)
    pkg.fpd_context_weights(1, B * L, nq, nkv, h, p.layer, p.q, p.lse, p.prefix, 512, p.p_len, pw, False)
    total = w[1].double().sum() + pw[1].double().sum()
    assert abs(total.item() - B * L * nq) < 2.0 ** -14 * B * L * nq


# ---- eviction -----------------------------------------------------------------------------------------------------

EVICT = {
    # layers, B, nkv, h, cap, lengths, budget, recent, out cap
    "one": (1, 1, 1, 64, 4, [2], 1, 0, 1),
    "small": (5, 1, 2, 64, 144, [128], 64, 16, 64),
    "ragged": (2, 5, 2, 128, 300, [300, 0, 100, 99, 101], 100, 7, 128),
    "all_recent": (1, 2, 2, 128, 200, [200, 150], 60, 60, 60),
    "no_recent": (2, 2, 1, 64, 257, [257, 256], 255, 0, 300),
    "long": (1, 1, 2, 64, 16384, [16384], 4096, 512, 4096),
    "unstaged": (1, 2, 1, 64, 40000, [39999, 16385], 9000, 100, 9001),
    "unstaged_most": (1, 1, 1, 64, 33000, [32769], 32768, 1, 33000),
    "keep_one": (2, 3, 2, 128, 1000, [1000, 1, 513], 1, 1, 1),
}


def evict_problem(name, seed=0):
    layers, B, nkv, h, cap, lens, budget, recent, out_cap = EVICT[name]
    rng = np.random.default_rng(seed)
    store = torch.from_numpy(rng.integers(-2**15, 2**15, size=(layers, B, 2, nkv, cap, h), dtype=np.int16))
    w = rng.exponential(size=(layers, B, nkv, cap)).astype(np.float32) ** 3
    w[rng.random(w.shape) < 0.2] = 0.0
    w[rng.random(w.shape) < 0.2] = np.float32(0.25)   # ties around and off the border
    special = rng.random(w.shape)
    w[special < 0.02] = np.nan
    w[(special > 0.02) & (special < 0.03)] = np.inf
    w[(special > 0.03) & (special < 0.04)] = -np.inf
    w[(special > 0.04) & (special < 0.06)] = -0.0
    w[(special > 0.06) & (special < 0.08)] = -1.5
    return store, w


def same_floats(a, b):
    return np.array_equal(np.asarray(a), np.asarray(b), equal_nan=True)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("name", list(EVICT))
def test_evict_context(pkg, name, in_place):
    layers, B, nkv, h, cap, lens, budget, recent, out_cap = EVICT[name]
    if in_place:
        out_cap = cap
    store, w = evict_problem(name, seed=len(name))
    s_d, w_d, n_d = store.to(DEV).view(BF), torch.from_numpy(w).to(DEV), i32(lens)
    if in_place:
        o_d, ow_d, on_d = s_d, w_d, n_d
        out0 = store.numpy().copy()
    else:
        o_d = torch.full((layers, B, 2, nkv, out_cap, h), 7, dtype=torch.int16, device=DEV).view(BF)
        ow_d, on_d = torch.full((layers, B, nkv, out_cap), -3.0, device=DEV), i32([-1] * B)
        out0 = np.full((layers, B, 2, nkv, out_cap, h), 7, np.int16)
    off = i32([10 * b for b in range(B)])
    kept = torch.full((layers, B, nkv, budget), -9, dtype=torch.int32, device=DEV)
    ws = torch.full((pkg.fpd_evict_workspace_bytes(layers, B, nkv, budget),), 0xFF, dtype=torch.uint8, device=DEV)
    pkg.fpd_evict_context(layers, B, nkv, h, budget, recent, s_d, cap, w_d, n_d, o_d, out_cap, ow_d, on_d, off, kept, ws,
                          ws.numel())
    torch.cuda.synchronize()
    assert pkg.fpd_device_status() == 0
    out, ow, n, k = ref.evict(store.numpy(), w, lens, budget, recent, out0, out_cap)
    assert np.array_equal(kept.cpu().numpy(), k)
    assert np.array_equal(on_d.cpu().numpy(), n)
    assert off.tolist() == [10 * b + lens[b] - int(n[b]) for b in range(B)]
    assert same_floats(ow_d.cpu().numpy(), ow)
    assert np.array_equal(o_d.view(torch.int16).cpu().numpy(), out)
    if not in_place:
        assert n_d.tolist() == lens and same_floats(w_d.cpu().numpy(), w)


def test_evict_without_kept_and_offsets_twice(pkg):
    """Optional outputs left out; a second eviction of the same store in place goes on from the first."""
    layers, B, nkv, h, cap, lens = 2, 2, 2, 128, 400, [400, 333]
    store, w = evict_problem("ragged", 1)[0], None
    rng = np.random.default_rng(2)
    store = torch.from_numpy(rng.integers(-2**15, 2**15, size=(layers, B, 2, nkv, cap, h), dtype=np.int16))
    w = rng.exponential(size=(layers, B, nkv, cap)).astype(np.float32)
    s_d, w_d, n_d = store.to(DEV).view(BF), torch.from_numpy(w).to(DEV), i32(lens)
    out, ow, n = store.numpy(), w, lens
    for budget, recent in ((200, 20), (50, 0)):
        ws = torch.empty(pkg.fpd_evict_workspace_bytes(layers, B, nkv, budget), dtype=torch.uint8, device=DEV)
        pkg.fpd_evict_context(layers, B, nkv, h, budget, recent, s_d, cap, w_d, n_d, s_d, cap, w_d, n_d, None, None, ws,
                              ws.numel())
        out, ow, n, _ = ref.evict(out, ow, list(n), budget, recent, out, cap)
        assert np.array_equal(s_d.view(torch.int16).cpu().numpy(), out)
        assert np.array_equal(w_d.cpu().numpy(), ow) and n_d.tolist() == list(n)


def test_attend_collect_evict_attend(pkg):
    """The operators as they are used together: attend, collect the weights, evict, attend to what is left."""
    p = Problem(4, 16, 32, 8, 128, 600, 640, [300, 150, 0, 299], 320, True, seed=31, layers=1)
    B, L, nq, nkv, h = p.shape
    p.run(pkg)
    w, pw = torch.zeros(1, B, nkv, 320, device=DEV), torch.zeros(1, 1, nkv, 640, device=DEV)
    run_weights(pkg, p, w)
    pkg.fpd_context_weights(1, B * L, nq, nkv, h, 0, p.q, p.lse, p.prefix, 640, p.p_len, pw, False)
    for store, weights, lens, b, cap, budget, recent in ((p.store, w, p.c_len, B, 320, 128, 32), (p.prefix, pw, p.p_len, 1, 640, 256, 0)):
        before, wb, nb = store.clone(), weights.cpu().numpy(), lens.tolist()
        ws = torch.empty(pkg.fpd_evict_workspace_bytes(1, b, nkv, budget), dtype=torch.uint8, device=DEV)
        pkg.fpd_evict_context(1, b, nkv, h, budget, recent, store, cap, weights, lens, store, cap, weights, lens, None, None,
                              ws, ws.numel())
        want = ref.evict(before.view(torch.int16).cpu().numpy(), wb, nb, budget, recent, before.view(torch.int16).cpu().numpy(), cap)
        assert np.array_equal(store.view(torch.int16).cpu().numpy(), want[0]) and lens.tolist() == want[2].tolist()
    p.P, p.lens = p.p_len.item(), p.c_len.tolist()
    p.run(pkg)
    p.check()
    assert pkg.fpd_device_status() == 0
