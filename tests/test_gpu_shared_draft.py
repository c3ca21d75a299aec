"""GPU: the block pass of a batch behind a shared prefix (SharedDraft, fpd_prepare_context_at, fpd_draft_block_shared), with
and without eviction, on the three execution paths.

A request behind a prefix must draft what it drafts with its whole context in a store of its own: the oracle runs on such
stores, put together from what the GPU prepared (each stage on the GPU's own inputs).  After an eviction slots and rotary
positions differ, which the oracle's store cannot say; there the fp32 restatement of the drafter (tests/fp32_restatement.py)
runs on the GPU's store with its rotation shifted.  Tolerance: 2e-2 of a row's largest value, as everywhere (bf16 storage
points of five layers)."""
import dataclasses

import numpy as np
import pytest
import torch

import fp32_restatement
import synth
from _util import assert_rows_close, bits_of, dev_i32

pytestmark = pytest.mark.gpu
DEV = "cuda"
TINY = synth.TINY
# two layers with the full-size heads, one of whose GEMM shapes takes every path of the context preparation
WIDE = dataclasses.replace(TINY, n_layers=2, n_q_heads=8, n_kv_heads=2, head_dim=128, vocab=1024)


@pytest.fixture(scope="module")
def pkg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_diffusion_speculative_non_gb300 as p
    return p


@pytest.fixture(scope="module")
def orc():
    import oracle
    oracle.build()
    return oracle


def build(pkg, shape, B, L, t_cap, p_cap, seed, collect=True, max_pos=None, fp8=False):
    w = synth.make_weights(shape, seed)
    dr = pkg.Drafter(shape, w, B, L, t_cap, device=DEV, max_pos=max_pos or p_cap + t_cap + L, fp8=fp8)
    return w, dr, dr.shared(B, L, t_cap, p_cap, collect=collect)


def rows_of(feats, lo, hi):
    return [f[lo:hi] for f in feats]


def fill(sd, shape, P, lens, seed):
    """Prefix of P rows in two appends, own contexts of `lens`; returns the host features."""
    pf = synth.make_features(shape, max(P, 1), seed)
    cut = P // 3
    for lo, hi in ((0, cut), (cut, P)):
        if hi > lo:
            sd.prepare_prefix(rows_of(pf, lo, hi))
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    of = synth.make_features(shape, max(int(off[-1]), 1), seed + 1)
    if off[-1]:
        sd.append(off, rows_of(of, 0, int(off[-1])))
    return pf, of, off


def combined(sd, P, b, n):
    """[layers][1][K|V][heads][P + n][h]: the prefix and request b's own context as one store, as the GPU holds them."""
    parts = [sd.prefix_kv[:, :, :, :, :P]] if sd.prefix_kv is not None else []
    if sd.kv is not None:
        parts.append(sd.kv[:, b:b + 1, :, :, :n])
    return bits_of(torch.cat(parts, 4).contiguous())


CASES = {
    # shape, batch, block, prefix, own lengths: positions in all
    "few_token": (TINY, 2, 8, 100, [30, 0]),           # 16: the weight-streaming path
    "few_token_one": (TINY, 1, 2, 65, [1]),
    "weight_tile": (TINY, 3, 16, 70, [0, 70, 9]),      # 48
    "token_tile": (TINY, 20, 16, 33, [(7 * b) % 30 for b in range(20)]),   # 320
    "wide_few_token": (WIDE, 1, 16, 200, [90]),
    "wide_weight_tile": (WIDE, 8, 16, 130, [20 * b for b in range(8)]),
    "wide_token_tile": (WIDE, 3, 150, 300, [100, 0, 65]),
}


@pytest.mark.parametrize("name", list(CASES))
def test_prefix_and_own_contexts_draft_as_one_store(pkg, orc, name):
    shape, B, L, P, lens = CASES[name]
    t_cap = max(max(lens), 1) + 3
    w, dr, sd = build(pkg, shape, B, L, t_cap, P + 5, seed=len(name))
    om = orc.Model(shape, w)
    pf, of, off = fill(sd, shape, P, lens, 50)
    assert sd.prefix_len.item() == P and sd.ctx_len.tolist() == list(lens) and sd.pos_offset.tolist() == [P] * B
    # the stores: slot i of an own context is position P + i
    anchor = np.arange(5, 5 + B).astype(np.int32)
    lh = torch.empty(shape.n_layers, B * L, shape.d_model, dtype=torch.bfloat16, device=DEV)
    hid = sd.draft_block(dev_i32(anchor), shape.vocab - 1, layer_hidden=lh)
    torch.cuda.synchronize()
    assert pkg.fpd_device_status() == 0
    for b in range(0, B, max(1, B // 3)):
        n = lens[b]
        feats = [np.concatenate([p[:P], o[off[b]:off[b + 1]]]) for p, o in zip(pf, of)]
        kv_ref = orc.prepare_context(om, np.array([0, P + n], np.int32), feats, P + n)
        kv = combined(sd, P, b, n)
        for l in range(shape.n_layers):
            for x in range(2):
                assert_rows_close(kv[l, 0, x].reshape(-1, shape.head_dim), kv_ref[l, 0, x].reshape(-1, shape.head_dim), f"store {l} {x}")
        o_hid, o_lh = orc.draft_block(om, kv, P + n, np.array([P + n], np.int32), anchor[b:b + 1], shape.vocab - 1, L,
                                      want_layers=True)
        sl = slice(b * L, (b + 1) * L)
        for l in range(shape.n_layers):
            assert_rows_close(bits_of(lh[l, sl]), o_lh[l], f"request {b} layer {l}")
        assert_rows_close(bits_of(hid[sl]), o_hid, f"request {b} hidden")


@pytest.mark.parametrize("which", ["prefix_only", "own_only", "nothing"])
def test_stores_may_be_left_out(pkg, orc, which):
    """No own store, no prefix, or neither (the block alone); the rotary offset then counts from the prefix or from 0."""
    B, L, P, lens = 3, 8, 40, [20, 0, 7]
    w = synth.make_weights(TINY, 5)
    dr = pkg.Drafter(TINY, w, B, L, 64, device=DEV, max_pos=200)
    sd = dr.shared(B, L, 0 if which != "own_only" else 32, 0 if which != "prefix_only" else P)
    if which == "prefix_only":
        sd.prepare_prefix(synth.make_features(TINY, P, 3))
    elif which == "own_only":
        off = np.concatenate([[0], np.cumsum(lens)])
        sd.append(off, synth.make_features(TINY, int(off[-1]), 4))
    om, anchor = orc.Model(TINY, w), np.array([1, 2, 3], np.int32)
    hid = sd.draft_block(dev_i32(anchor), TINY.vocab - 1)
    # pos_offset left out means the prefix's length
    sd.context.pos_offset = None
    assert torch.equal(sd.draft_block(dev_i32(anchor), TINY.vocab - 1), hid)
    for b in range(B):
        T = {"prefix_only": P, "own_only": lens[b], "nothing": 0}[which]
        kv = combined(sd, P if which == "prefix_only" else 0, b, T if which == "own_only" else 0) if which != "nothing" else \
            np.zeros((TINY.n_layers, 1, 2, TINY.n_kv_heads, 1, TINY.head_dim), np.uint16)
        kv = kv if kv.shape[4] else np.zeros((TINY.n_layers, 1, 2, TINY.n_kv_heads, 1, TINY.head_dim), np.uint16)
        o = orc.draft_block(om, kv, max(T, 1), np.array([T], np.int32), anchor[b:b + 1], TINY.vocab - 1, L)
        assert_rows_close(bits_of(hid[b * L:(b + 1) * L]), o, f"request {b}")
    assert pkg.fpd_device_status() == 0


def test_shared_pass_with_8_bit_weights_runs_the_same_gemms(pkg):
    """With 8-bit weights the few-token pass over a prefix stays as near to the plain pass over one store as two attention
    kernels of the same rounding are: one layer, a few bf16 steps through the 8-bit rounding (4 x 2e-2, as tests/test_gpu_fp8)."""
    shape = dataclasses.replace(TINY, n_layers=1)
    w, dr, sd = build(pkg, shape, 1, 16, 64, 64, seed=9, fp8=True)
    feats = synth.make_features(shape, 90, 6)
    sd.prepare_prefix(rows_of(feats, 0, 60))
    sd.append([0, 30], rows_of(feats, 60, 90))
    one = pkg.Drafter(shape, w, 1, 16, 96, device=DEV, fp8=True)
    one.prepare_context(1, [0, 90], feats)
    a = sd.draft_block(dev_i32([7]), shape.vocab - 1)
    b = one.draft_block(1, 16, dev_i32([90]), dev_i32([7]), shape.vocab - 1)
    assert_rows_close(bits_of(a), bits_of(b), "8-bit", tol=8e-2)


def collected(sd, hid_shape, weights_before=None):
    return sd.weights.clone(), sd.prefix_weights.clone()


@pytest.mark.parametrize("shape,B,L", [(TINY, 1, 8), (TINY, 2, 16), (WIDE, 3, 100)])
def test_evicted_contexts_draft_at_their_positions(pkg, monkeypatch, shape, B, L):
    P, lens = 80, [60 - 13 * b for b in range(B)]
    w, dr, sd = build(pkg, shape, B, L, 64, 96, seed=11)
    fill(sd, shape, P, lens, 70)
    anchor = dev_i32(np.arange(3, 3 + B))
    before = sd.kv.clone(), sd.prefix_kv.clone()
    sd.draft_block(anchor, shape.vocab - 1)
    # every row hands out 1 in all, some of it to the block
    got = sd.weights.double().sum((2, 3)).sum(1) + sd.prefix_weights.double().sum((2, 3))[:, 0]
    rows = B * L * shape.n_q_heads
    assert (got > 0.2 * rows).all() and (got < rows).all()
    first = sd.weights.clone()
    sd.draft_block(anchor, shape.vocab - 1)
    assert torch.equal(sd.weights, first + first)       # the same pass again adds the same weights
    kept = torch.empty(shape.n_layers, B, shape.n_kv_heads, 24, dtype=torch.int32, device=DEV)
    wv = sd.weights.clone()
    sd.evict(24, 8, kept)
    sd.evict_prefix(40, 4)
    new = [min(n, 24) for n in lens]
    assert sd.ctx_len.tolist() == new and sd.prefix_len.item() == 40
    assert sd.pos_offset.tolist() == [P + n - m for n, m in zip(lens, new)] and sd.prefix_offset.item() == P - 40
    for l in range(shape.n_layers):
        for b in range(B):
            for g in range(shape.n_kv_heads):
                k = kept[l, b, g, :new[b]].long()
                assert torch.equal(sd.kv[l, b, :, g, :new[b]], before[0][l, b, :, g, k])
                assert torch.equal(sd.weights[l, b, g, :new[b]], wv[l, b, g, k])
                if lens[b] > 24:   # none of the dropped weighs more than the lightest of those kept for their weight
                    left = torch.ones(lens[b], dtype=torch.bool, device=DEV)
                    left[k] = False
                    assert wv[l, b, g, :lens[b]][left].max() <= wv[l, b, g, k[:16]].min()
    hid = sd.draft_block(anchor, shape.vocab - 1)
    torch.cuda.synchronize()
    assert pkg.fpd_device_status() == 0
    wf, rope = fp32_restatement.weights_f32(w), fp32_restatement._rope
    for b in range(B):
        T = 40 + new[b]
        shift = P + lens[b] - T     # rotary position of the block less the number of context positions
        monkeypatch.setattr(fp32_restatement, "_rope", lambda x, pos, theta, h: rope(x, pos + shift, theta, h))
        want = fp32_restatement.draft_block(shape, wf, combined(sd, 40, b, new[b]), T, 3 + b, shape.vocab - 1, L)
        monkeypatch.undo()
        assert_rows_close(bits_of(hid[b * L:(b + 1) * L]), synth.f32_to_bf16_bits(want), f"request {b}")


def test_append_goes_on_behind_an_eviction(pkg, orc):
    """Rows appended after an eviction sit in the next free slots, rotated for where the sequence is."""
    w, dr, sd = build(pkg, TINY, 2, 8, 48, 32, seed=12)
    pf, of, off = fill(sd, TINY, 32, [40, 30], 90)
    sd.draft_block(dev_i32([1, 2]), TINY.vocab - 1)
    sd.evict(20, 20)
    assert sd.ctx_len.tolist() == [20, 20] and sd.pos_offset.tolist() == [52, 42]
    new = synth.make_features(TINY, 9, 91)
    sd.append([0, 5, 9], new)
    om = orc.Model(TINY, w)
    for b, (lo, hi, start) in enumerate(((0, 5, 72), (5, 9, 62))):
        want = orc.prepare_context(om, np.array([0, hi - lo], np.int32), rows_of(new, lo, hi), 80, pos_start=[start])
        got = bits_of(sd.kv[:, b, :, :, 20:20 + hi - lo].contiguous())
        assert_rows_close(got.reshape(-1, TINY.head_dim), want[:, 0, :, :, start:start + hi - lo].reshape(-1, TINY.head_dim), f"append {b}")
    assert sd.ctx_len.tolist() == [25, 24] and pkg.fpd_device_status() == 0


@pytest.mark.parametrize("shape", [TINY, WIDE])
def test_positions_past_the_rotary_table_are_recorded(pkg, shape):
    w, dr, sd = build(pkg, shape, 1, 8, 100, 8, seed=13, max_pos=110)
    feats = synth.make_features(shape, 100, 92)
    sd.pos_offset.fill_(105)
    sd.kv.fill_(3.0)
    for rows in (20, 100):      # below and above the rows that take the one-GEMM path
        sd.ctx_len.zero_()
        sd.append([0, rows], rows_of(feats, 0, rows))
        assert pkg.fpd_device_status() == 6
        assert (sd.kv[:, :, :, :, 5:] == 3).all() and not (sd.kv[:, :, :, :, :5] == 3).all()
    sd.ctx_len.fill_(5)
    sd.draft_block(dev_i32([1]), 5)
    torch.cuda.synchronize()
    assert pkg.fpd_device_status() == 5     # block positions clamped to the table
    sd.pos_offset.fill_(-7)
    sd.draft_block(dev_i32([1]), 5)
    torch.cuda.synchronize()
    assert pkg.fpd_device_status() == 5


def test_refusals_with_a_model(pkg):
    w, dr, sd = build(pkg, TINY, 1, 8, 16, 16, seed=14)
    an, hid = dev_i32([1]), torch.empty(8, TINY.d_model, dtype=torch.bfloat16, device=DEV)

    def call(ctx, ws=None):
        n = sd.workspace.numel() if ws is None else ws
        pkg.fpd_draft_block_shared(dr.handle, 1, 8, ctx, an, 5, hid, None, sd.workspace, n)

    for bad, status in ((pkg.shared_context(sd.prefix_kv, 16), 1), (pkg.shared_context(prefix_cap=16, prefix_len=sd.prefix_len), 1),
                        (pkg.shared_context(kv_store=sd.kv, t_cap=16), 1), (pkg.shared_context(weights=sd.weights), 1),
                        (pkg.shared_context(sd.prefix_kv, 16, sd.prefix_len, weights=sd.weights), 1),
                        (pkg.shared_context(t_cap=-1), 2)):
        with pytest.raises(pkg.FpdError) as e:
            call(bad)
        assert e.value.status == status
    with pytest.raises(pkg.FpdError) as e:
        call(sd.context, ws=64)
    assert e.value.status == 3
    with pytest.raises(ValueError):
        dr.shared(1, 8, 16).evict(8, 0)     # nothing was collected
    with pytest.raises(ValueError, match="the call needs"):
        pkg.fpd_evict_context(TINY.n_layers, 2, TINY.n_kv_heads, TINY.head_dim, 8, 0, sd.kv, 16, sd.weights, sd.ctx_len, sd.kv, 16,
                              sd.weights, sd.ctx_len, None, None, sd.workspace, sd.workspace.numel())


def spec_steps(pkg, dr, sd, st, feats, steps, budget):
    """Text speculative steps behind the prefix: draft, argmax, verify against a fixed target, advance, append, evict."""
    out = []
    for k in range(steps):
        hid = sd.draft_block(st.anchor, dr.shape.vocab - 1, hidden_out=st.hidden)
        dr.constrain_argmax(st.batch, st.block_len, hid, tokens_out=st.tokens)
        st.target[:, :-1].copy_(st.tokens)
        st.target[:, 3 + k:].fill_(11)      # the target goes its own way there
        pkg.fpd_verify(0, st.batch, st.block_len, st.tokens, st.target, None, None, -1, st.accept, st.committed, st.valid)
        pkg.fpd_sd_advance(st.batch, st.block_len, sd.t_cap, st.accept, st.committed, sd.ctx_len, st.pos_start, st.anchor)
        sd.append_rows(st.batch * st.block_len, st.row_off, st.accept, st.pos_start, feats[k])
        sd.evict(budget, budget // 2)
        out.append((st.hidden.clone(), st.accept.clone(), sd.ctx_len.clone(), sd.pos_offset.clone()))
    return out


def test_speculative_steps_behind_a_prefix_in_a_graph(pkg):
    """Draft, verify, advance, append and evict, three steps: eager and as one captured graph, bit for bit."""
    B, L, P, lens, budget = 2, 8, 40, [22, 17], 24
    w, dr, sd = build(pkg, TINY, B, L, 40, 48, seed=15)
    feats = [[torch.from_numpy(f.view(np.int16)).to(DEV).view(torch.bfloat16) for f in synth.make_features(TINY, B * L, 200 + k)]
             for k in range(3)]

    def start():
        for t in (sd.kv, sd.prefix_kv, sd.weights, sd.prefix_weights, sd.ctx_len, sd.prefix_len, sd.pos_offset, sd.prefix_offset):
            t.zero_()
        fill(sd, TINY, P, lens, 95)
        st.anchor.copy_(dev_i32([4, 9]))

    st = dr.spec_state(B, L, lens, [4, 9])
    start()
    eager = spec_steps(pkg, dr, sd, st, feats, 3, budget)
    kv, wts = sd.kv.clone(), sd.weights.clone()
    torch.cuda.synchronize()
    assert pkg.fpd_device_status() == 0
    total = [n + int(sum(e[1][b].item() for e in eager)) for b, n in enumerate(lens)]
    assert (sd.pos_offset + sd.ctx_len).tolist() == [P + t for t in total]      # no position is lost count of
    assert sd.ctx_len.max().item() <= budget
    start()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = spec_steps(pkg, dr, sd, st, feats, 3, budget)
    start()
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(eager, captured):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
    assert torch.equal(sd.kv, kv) and torch.equal(sd.weights, wts) and pkg.fpd_device_status() == 0


def test_rows_without_a_slot_or_a_position_are_not_counted(pkg):
    """Rows past the rotary table or the store are recorded and left out of the lengths: what is drafted is what the rows
    that are there give."""
    P, n = 30, 12
    w, dr, sd = build(pkg, TINY, 1, 8, 40, 30, seed=16, max_pos=50)
    pf, of = synth.make_features(TINY, P + 5, 96), synth.make_features(TINY, 40, 97)
    sd.prepare_prefix(rows_of(pf, 0, 25))
    sd.prepare_prefix(rows_of(pf, 25, P + 5))            # 5 rows past prefix_cap
    assert pkg.fpd_device_status() == 6
    assert sd.prefix_len.item() == P and sd.pos_offset.tolist() == [P]
    sd.append([0, n], rows_of(of, 0, n))
    assert pkg.fpd_device_status() == 0 and sd.ctx_len.tolist() == [n]
    hid = sd.draft_block(dev_i32([3]), 5)                # positions 42..49: the last that fit
    torch.cuda.synchronize()
    assert pkg.fpd_device_status() == 0
    sd.ctx_len.zero_()
    sd.append([0, 40], of)                               # 20 of 40 rows have a position
    assert pkg.fpd_device_status() == 6 and sd.ctx_len.tolist() == [20]
    w2, dr2, alone = build(pkg, TINY, 1, 8, 40, 30, seed=16, max_pos=50)
    alone.prepare_prefix(rows_of(pf, 0, 25))
    alone.prepare_prefix(rows_of(pf, 25, P))
    alone.append([0, n], rows_of(of, 0, n))
    assert torch.equal(alone.draft_block(dev_i32([3]), 5), hid) and pkg.fpd_device_status() == 0


def test_appends_refuse_what_they_cannot_hold(pkg):
    w, dr, sd = build(pkg, TINY, 2, 8, 16, 16, seed=17)
    f = synth.make_features(TINY, 20, 98)
    for off, feats, what in (([0, 17, 20], f, "more rows"), ([0, 20], f, "row_off"), ([1, 5, 9], f, "row_off"), ([0, 9, 5], f, "row_off"),
                             ([0, 5, 9], rows_of(f, 0, 8), "the call needs"), ([0, 5, 9], f[:-1], "feature tensors")):
        with pytest.raises(ValueError, match=what):
            sd.append(off, feats)
    with pytest.raises(ValueError, match="the call needs"):
        sd.prepare_prefix([f[0]] + rows_of(f[1:], 0, 8))
    with pytest.raises(pkg.FpdError):
        sd.prepare_prefix(f)                             # 20 rows, 16 slots
    assert sd.ctx_len.tolist() == [0, 0] and sd.prefix_len.item() == 0 and sd.pos_offset.tolist() == [0, 0]


def test_draft_calls_refuse_tensors_of_another_type_or_size(pkg):
    w, dr, sd = build(pkg, TINY, 2, 8, 16, 16, seed=18)
    for bad in (torch.tensor([1, 2], device=DEV), torch.tensor([1, 2], dtype=torch.int32), dev_i32([1])):
        with pytest.raises(ValueError, match="anchor"):
            sd.draft_block(bad, 5)
    h = torch.empty(16, TINY.d_model, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="hidden_out"):
        sd.draft_block(dev_i32([1, 2]), 5, hidden_out=h[1:])
    with pytest.raises(ValueError, match="layer_hidden"):
        sd.draft_block(dev_i32([1, 2]), 5, hidden_out=h, layer_hidden=h)
    one = pkg.shared_context(sd.prefix_kv, 16, sd.prefix_len, sd.kv, 16, sd.ctx_len[:1], sd.pos_offset)
    with pytest.raises(ValueError, match="ctx_len holds 1 elements"):
        pkg.fpd_draft_block_shared(dr.handle, 2, 8, one, dev_i32([1, 2]), 5, h, None, sd.workspace, sd.workspace.numel())


def test_workspace_of_sizes_that_the_block_pass_refuses_is_zero(pkg):
    w, dr, sd = build(pkg, TINY, 2, 8, 16, 16, seed=19)
    size = lambda *a: pkg.fpd_shared_workspace_bytes(dr.handle, *a)
    big = (1 << 26) // TINY.n_q_heads // 8
    assert size(2, 8, 16, 16) > 0 and size(1, 2, 1 << 30, 1 << 30) > 0
    for bad in ((big + 1, 8, 16, 16), (1 << 30, 8, 16, 16), (9, 1 << 20, 16, 16), (2, 8, (1 << 30) + 1, 16), (2, 8, 16, (1 << 30) + 1), (2, 1, 16, 16)):
        assert size(*bad) == 0, bad


def test_two_objects_on_two_streams(pkg):
    """Objects share the drafter's weights alone: passes and evictions of both at once give what each gives by itself."""
    w, dr, a = build(pkg, TINY, 3, 16, 64, 48, seed=20)
    b = dr.shared(2, 8, 40, 48, collect=True)
    anchor = dev_i32([4, 9, 2])

    def steps(sd, n):
        out = []
        for _ in range(3):
            out.append(sd.draft_block(anchor[:n], 5))
            sd.evict(16, 4)
            sd.evict_prefix(20, 0)
        return out + [sd.kv.clone(), sd.weights.clone(), sd.prefix_weights.clone()]

    def reset(sd, P, lens, seed):
        for t in (sd.kv, sd.prefix_kv, sd.weights, sd.prefix_weights, sd.ctx_len, sd.prefix_len, sd.pos_offset, sd.prefix_offset):
            t.zero_()
        fill(sd, TINY, P, lens, seed)

    sets = ((a, 3, 40, [50, 0, 33], 60), (b, 2, 45, [7, 40], 70))
    want = []
    for sd, n, P, lens, seed in sets:
        reset(sd, P, lens, seed)
        want.append(steps(sd, n))
    for sd, n, P, lens, seed in sets:
        reset(sd, P, lens, seed)
    torch.cuda.synchronize()
    got = []
    for sd, n, *_ in sets:
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got.append(steps(sd, n))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for g, v in zip(got, want) for x, y in zip(g, v)) and pkg.fpd_device_status() == 0
