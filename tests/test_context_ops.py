"""CPU: what the operators on a context store refuse before they touch the device, their workspace sizes, and the
reference's own selection rule."""
import ctypes

import numpy as np
import pytest

import context_ops_ref as ref


@pytest.fixture(scope="module")
def fpd():
    import __graft_entry__ as g
    g._compile_all()
    import block_diffusion_speculative_non_gb300 as pkg
    return pkg


A = 1 << 20   # an address that is never dereferenced


def attn(fpd, **kw):
    a = dict(batch=2, block=4, nq=8, nkv=2, h=64, layer=0, q=A, kb=A, vb=A, pre=A, p_cap=16, p_len=A, kv=A, t_cap=8, c_len=A,
             out=A, lse=A, ws=A, n=1 << 30)
    a.update(kw)
    return fpd.lib().fpd_shared_attention(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), 2), (dict(block=0), 2), (dict(h=96), 4), (dict(nq=7), 2), (dict(nkv=0), 2), (dict(nq=1, nkv=2), 2),
    (dict(layer=-1), 2), (dict(p_cap=-1), 2), (dict(t_cap=-1), 2), (dict(p_cap=(1 << 30) + 1), 2),
    (dict(batch=1 << 20, block=1 << 12), 2), (dict(batch=1 << 14, block=1 << 10, nq=8), 2),
    (dict(q=None), 1), (dict(out=None), 1), (dict(ws=None), 1), (dict(vb=None), 1), (dict(kb=None), 1),
    (dict(pre=None), 1), (dict(p_len=None), 1), (dict(p_cap=0), 1), (dict(p_cap=0, pre=None), 1),
    (dict(kv=None), 1), (dict(c_len=None), 1), (dict(t_cap=0), 1),
    (dict(q=A + 8), 1), (dict(out=A + 2), 1), (dict(kv=A + 4), 1), (dict(ws=A + 8), 1), (dict(kb=A + 2), 1),
])
def test_shared_attention_refuses(fpd, kw, status):
    assert attn(fpd, **kw) == status, fpd.fpd_last_error()
    assert fpd.fpd_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), 2), (dict(h=32), 4), (dict(nq=3), 2), (dict(t_cap=0), 2), (dict(layer=-2), 2), (dict(q=None), 1),
    (dict(lse=None), 1), (dict(kv=None), 1), (dict(c_len=None), 1), (dict(w=None), 1), (dict(q=A + 2), 1), (dict(w=A + 4), 1),
    (dict(batch=1 << 10, block=1, t_cap=1 << 30), 2),
])
def test_context_weights_refuses(fpd, kw, status):
    a = dict(batch=2, block=4, nq=8, nkv=2, h=64, layer=0, q=A, lse=A, kv=A, t_cap=8, c_len=A, w=A, acc=0)
    a.update(kw)
    assert fpd.lib().fpd_context_weights(*a.values(), None) == status, fpd.fpd_last_error()


FAR = 1 << 40


@pytest.mark.parametrize("kw,status", [
    (dict(layers=0), 2), (dict(batch=0), 2), (dict(nkv=0), 2), (dict(h=80), 4), (dict(budget=0), 2), (dict(recent=-1), 2),
    (dict(recent=9), 2), (dict(budget=17, recent=0), 2), (dict(t_cap=0), 2), (dict(out_cap=0), 2),
    (dict(kv=None), 1), (dict(w=None), 1), (dict(c_len=None), 1), (dict(out=None), 1), (dict(ow=None), 1),
    (dict(on=None), 1), (dict(ws=None), 1), (dict(kv=A + 8), 1), (dict(kept=A + 4), 1),
    (dict(n=16), 3), (dict(n=300, kept=A), 3),
    (dict(out=A), 1),                                   # store in place, weights not
    (dict(ow=A * 2), 1),                                # weights in place, store not
    (dict(out=A, ow=A * 2), 1),                         # in place with another capacity
    (dict(out=A + 4096), 1), (dict(ow=A * 2 + 16), 1),   # overlapping, not in place
])
def test_evict_refuses(fpd, kw, status):
    a = dict(layers=2, batch=2, nkv=2, h=64, budget=8, recent=2, kv=A, t_cap=32, w=A * 2, c_len=A * 3, out=FAR, out_cap=16,
             ow=2 * FAR, on=A * 3, off=None, kept=None, ws=3 * FAR, n=1 << 20)
    a.update(kw)
    assert fpd.lib().fpd_evict_context(*a.values(), None) == status, fpd.fpd_last_error()


def test_model_calls_refuse(fpd):
    l = fpd.lib()
    feats = (ctypes.c_void_p * 1)(A)
    assert l.fpd_prepare_context_at(None, 1, 1, A, None, None, A, feats, A, 8, A, 1, None) == 1
    assert l.fpd_prepare_context_at(None, 1, 1, A, None, None, None, feats, A, 8, A, 1, None) == 1
    assert l.fpd_draft_block_shared(None, 1, 16, ctypes.byref(fpd.shared_context()), A, 0, A, None, A, 1, None) == 1
    assert l.fpd_draft_block_shared(None, 1, 16, None, A, 0, A, None, A, 1, None) == 1
    assert l.fpd_shared_workspace_bytes(None, 1, 16, 8, 8) == 0


def test_workspace_sizes_of_refused_calls_are_zero(fpd):
    assert fpd.fpd_shared_attention_workspace_bytes(0, 1, 8, 2, 64, 8, 8) == 0
    assert fpd.fpd_shared_attention_workspace_bytes(1, 1, 8, 2, 65, 8, 8) == 0
    assert fpd.fpd_shared_attention_workspace_bytes(1, 1, 8, 2, 64, -1, 8) == 0
    assert fpd.fpd_evict_workspace_bytes(0, 1, 2, 8) == 0
    assert fpd.fpd_evict_workspace_bytes(5, 3, 8, 100) >= 5 * 3 * 8 * 100 * 4 + 12


def test_binding_checks_tensors(fpd):
    """Type, layout and size of a tensor are checked before its address is used."""
    import torch
    with pytest.raises(ValueError, match="must be torch.bfloat16"):
        fpd._arg(torch.zeros(4), torch.bfloat16, 4, "q")
    with pytest.raises(ValueError, match="contiguous"):
        fpd._arg(torch.zeros(4, 4)[:, :2], torch.float32, 4, "lse")
    with pytest.raises(ValueError, match="the call needs 5"):
        fpd._arg(torch.zeros(4), torch.float32, 5, "lse")
    with pytest.raises(ValueError, match="current device"):
        fpd._arg(torch.zeros(4), torch.float32, 4, "lse", 0)
    assert fpd._arg(None, torch.int32, 4, "ctx_len") is None and fpd._arg(64, torch.int32, 4, "ctx_len") == 64


def test_compiled_calls_refuse_what_is_no_argument(fpd):
    """Counts, integers and objects of the compiled calls: a Python error, and nothing reaches the library."""
    import torch
    calls = fpd.context._compiled()
    att = [1, 1, 8, 2, 64, 0] + [64] * 4 + [8, 64, 64, 8, 64, 64, 64, 64, 1, None, 0]
    with pytest.raises(TypeError, match="20 arguments, the call takes 21"):
        calls.shared_attention(*att[:-1])
    with pytest.raises(OverflowError):
        calls.shared_attention(2 ** 40, *att[1:])
    with pytest.raises(OverflowError):
        calls.shared_attention(*att[:18], -1, *att[19:])                       # a negative workspace size
    with pytest.raises(TypeError):
        calls.shared_attention(1.5, *att[1:])
    with pytest.raises(TypeError, match="prefix_store must be a tensor"):
        calls.shared_attention(*att[:9], [1.0], *att[10:])
    with pytest.raises(ValueError, match="lse must be torch.float32, got torch.int32"):
        calls.shared_attention(*att[:16], torch.zeros(8, dtype=torch.int32), *att[17:])
    with pytest.raises(ValueError, match="current device"):
        calls.context_weights(1, 1, 8, 2, 64, 0, torch.zeros(512, dtype=torch.bfloat16), 64, 64, 8, 64, 64, 0, None, 0)
    with pytest.raises(ValueError, match="kv_store holds 4 elements, the call needs 9223372036854775807"):
        big = 2 ** 31 - 1                                                      # sizes whose product passes 64 bits
        calls.evict_context(big, big, big, 128, 8, 0, torch.zeros(4, dtype=torch.bfloat16), big, *[64] * 3, 8, *[64] * 6, None, 0)
    assert calls.shared_attention(0, *att[1:]) != 0                            # the library's own refusal
    assert calls.evict_context(0, 1, 2, 64, 8, 0, 64, 8, 64, 64, 64, 8, 64, 64, None, None, 64, 8, None, 0) != 0


def test_model_calls_check_tensors(fpd):
    """A tensor on the host, of another type or too small is refused before the library sees its address."""
    import torch
    i32, bf = torch.zeros(4, dtype=torch.int32), torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="anchor is on cpu"):
        fpd.fpd_draft_block_shared(64, 2, 8, fpd.shared_context(), i32, 0, 64, None, 64, 64)
    with pytest.raises(ValueError, match="anchor must be torch.int32, got torch.int64"):
        fpd.fpd_draft_block_shared(64, 2, 8, fpd.shared_context(), i32.long(), 0, 64, None, 64, 64)
    with pytest.raises(ValueError, match="hidden_out holds 4 elements, the call needs 16"):
        fpd.fpd_draft_block_shared(64, 2, 8, fpd.shared_context(), 64, 0, bf[:4], None, 64, 64)
    with pytest.raises(ValueError, match="ctx_len is on cpu"):
        fpd.shared_context(kv_store=64, t_cap=8, ctx_len=i32)
    with pytest.raises(ValueError, match="weights must be torch.float32"):
        fpd.shared_context(weights=bf)
    with pytest.raises(ValueError, match="row_off holds 4 elements, the call needs 5"):
        fpd.fpd_prepare_context_at(64, 4, 4, i32, None, None, 64, [64], 64, 8, 64, 64)
    with pytest.raises(ValueError, match="pos_offset must be torch.int32"):
        fpd.fpd_prepare_context_at(64, 4, 4, 64, None, None, i32.long(), [64], 64, 8, 64, 64)


def test_shared_draft_refuses_more_positions_than_the_drafter_has(fpd):
    """A Drafter that was not told max_pos has its own t_cap + max_block_len rotary positions: no room behind a long prefix."""
    import types
    dr = types.SimpleNamespace(max_pos=528, max_pos_given=False)
    with pytest.raises(ValueError, match="max_pos"):
        fpd.SharedDraft(dr, 8, 16, 512, 4096)
    with pytest.raises(ValueError, match="max_pos"):
        fpd.SharedDraft(dr, 8, 17, 512)
    with pytest.raises(AttributeError):      # past the check
        fpd.SharedDraft(dr, 8, 16, 500, 12)


def test_compiling_the_library_compiles_the_python_calls(fpd, monkeypatch, tmp_path):
    """What this file's fixture builds is enough for the compiled calls, and they are made again when their source is newer."""
    import os

    import __graft_entry__ as g
    made = tmp_path / "_calls.so"
    made.write_bytes(b"")
    os.utime(made, (1, 1))
    monkeypatch.setattr(g, "PKG", str(tmp_path))
    g._compile_all()
    assert made.stat().st_size > 0


def test_selection_rule_of_the_reference():
    nan, inf = float("nan"), float("inf")
    assert ref.kept_positions([5, 1, 3, 2], 4, 4, 0) == [0, 1, 2, 3]
    assert ref.kept_positions([5, 1, 3, 2], 4, 2, 0) == [0, 2]
    assert ref.kept_positions([5, 1, 3, 2], 4, 2, 1) == [0, 3]
    assert ref.kept_positions([1, 1, 1, 1], 4, 2, 0) == [0, 1]          # ties: the lower position
    assert ref.kept_positions([nan, -inf, 0.0, -0.0, inf], 5, 3, 0) == [2, 3, 4]
    assert ref.kept_positions([nan, -inf, nan], 3, 2, 0) == [0, 1]      # NaN below -inf
    assert ref.kept_positions([9, 9, 9], 3, 2, 2) == [1, 2]
    out, w, n, kept = ref.evict(np.arange(8, dtype=np.int16).reshape(1, 1, 2, 1, 4, 1), np.array([[[[3, 1, 2, 0]]]], np.float32),
                                [4], 2, 0, np.zeros((1, 1, 2, 1, 2, 1), np.int16), 2)
    assert out.reshape(2, 2).tolist() == [[0, 2], [4, 6]] and w.tolist() == [[[[3, 2]]]] and n.tolist() == [2]
    assert kept.tolist() == [[[[0, 2]]]]


# ---- how the shared attention cuts its work -------------------------------------------------------------------------

def plan(fpd, batch, L, nq, nkv, h, p_cap, t_cap, blk=True, sms=152):
    lib = fpd.lib()
    lib.fpd_test_shared_plan.argtypes = [ctypes.c_int] * 9 + [ctypes.POINTER(ctypes.c_int32)]
    out = (ctypes.c_int32 * 12)()
    assert lib.fpd_test_shared_plan(batch, L, L if blk else 0, nq, nkv, h, p_cap, t_cap, sms, out) == 0
    return dict(zip(("pre_tc", "own_tc", "pre_tiles", "pre_splits", "own_tiles", "own_splits", "pre_runs", "pre_pieces",
                     "own_cost", "grid", "own_ctas", "own_alone"), list(out)))


def walk(pl, batch, L, nq, nkv, P, sms=152):
    """The runs of every CTA of the tcgen05 kernel, as it takes them: (cta, unit, first tile, last tile, slots it writes)."""
    grp = nq // nkv
    rpt = 128 // grp * grp
    units = pl["pre_tiles"] * nkv if pl["pre_tc"] else 0
    own_n = pl["own_tiles"] * nkv * batch * (pl["own_splits"] // 2) if pl["own_tc"] else 0
    tiles = -(-P // 128)
    total, grid = units * tiles, pl["grid"]
    G = min(pl["pre_runs"], max(total, 1))
    W = 0
    if pl["own_cost"] and total >= 16 * G and G == grid:
        even, first = own_n // G, G - own_n % G
        W = min(pl["own_cost"], total // (2 * G * (even + 1) - own_n))
        shortest = (total + W * own_n) // G - 1 - W * (even + 1)
        if -(-tiles // shortest) + 1 > pl["pre_pieces"]:
            W = 0

    def start(i):
        return i * (total + W * own_n) // G - W * (even * i + max(0, i - first)) if W else i * total // G

    def run_of(t):
        return max(c for c in range(G) if start(c) <= t) if W else ((t + 1) * G - 1) // total

    own, alone = [], pl["own_ctas"] * pl["own_alone"]
    for c in range(grid):
        i = grid - 1 - c
        i += alone if i >= pl["own_ctas"] else 0
        while i < own_n:
            own.append(i)
            i += pl["own_ctas"] if i < alone else grid
    assert sorted(own) == list(range(own_n))        # every own run once
    runs = []
    for c in range(grid):
        if total == 0:
            runs += [(c, u, 0, 0, list(range(pl["pre_splits"]))) for u in range(c, units, grid)]
        x, end = (start(c), start(c + 1)) if c < G else (0, 0)
        while x < end:
            u = x // tiles
            e = min(end, (u + 1) * tiles)
            keys = batch * L * grp - u % pl["pre_tiles"] * 2 * rpt <= rpt
            piece = c - run_of(u * tiles)
            slots = [2 * piece, 2 * piece + 1] if keys else [piece]
            if e == (u + 1) * tiles:
                slots += range(slots[-1] + 1, pl["pre_splits"])
            runs.append((c, u, x - u * tiles, e - u * tiles, slots))
            x = e
    return runs, units, tiles


SHAPES = [(1, 16, 32, 8, 128), (8, 16, 32, 8, 128), (64, 16, 32, 8, 128), (4, 385, 32, 8, 128), (16, 1, 32, 8, 128), (3, 7, 20, 4, 128),
          (2, 200, 8, 1, 64), (30, 33, 14, 2, 64), (9, 15, 16, 4, 128), (200, 16, 8, 8, 128), (5, 61, 128, 1, 128), (1, 1, 130, 1, 64)]


@pytest.mark.parametrize("B,L,nq,nkv,h", SHAPES)
def test_shared_plan_covers_every_tile_and_slot_once(fpd, B, L, nq, nkv, h):
    """For the planned capacities and every shorter prefix: each key tile of each unit falls in one run, and each partial
    slot of a unit is written by exactly one run (or marked empty by its last)."""
    for sms in (152, 148, 20):
        for p_cap in (1, 100, 1000, 4096, 16384, 65536, 200001):
            for t_cap in (0, 64, 1000):
                pl = plan(fpd, B, L, nq, nkv, h, p_cap, t_cap, sms=sms)
                assert pl["pre_splits"] >= 1 and pl["own_splits"] >= 1
                if not pl["pre_tc"]:
                    assert pl["pre_splits"] <= 128
                    continue
                assert 1 <= pl["pre_runs"] <= pl["grid"] <= sms
                for P in sorted({0, 1, 129, p_cap // 7, p_cap // 2, p_cap - 1, p_cap}):
                    if P > p_cap or P < 0:
                        continue
                    runs, units, tiles = walk(pl, B, L, nq, nkv, P, sms)
                    seen, slots = {u: [] for u in range(units)}, {u: [] for u in range(units)}
                    for c, u, lo, hi, sl in runs:
                        seen[u] += range(lo, hi)
                        slots[u] += sl
                    for u in range(units):
                        assert seen[u] == list(range(tiles)), (pl, P, u)
                        assert sorted(slots[u]) == list(range(pl["pre_splits"])), (pl, P, u, slots[u])


def check_cover(fpd, B, L, nq, nkv, h, p_cap, t_cap, sms):
    pl = plan(fpd, B, L, nq, nkv, h, p_cap, t_cap, sms=sms)
    assert pl["pre_splits"] >= 1 and pl["own_splits"] >= 1, pl
    if not pl["pre_tc"]:
        return
    assert 1 <= pl["pre_runs"] <= pl["grid"] <= sms, pl
    for P in sorted({0, 1, min(129, p_cap), p_cap // 2, p_cap}):
        runs, units, tiles = walk(pl, B, L, nq, nkv, P, sms)
        seen, slots = {u: [] for u in range(units)}, {u: [] for u in range(units)}
        for c, u, lo, hi, sl in runs:
            seen[u] += range(lo, hi)
            slots[u] += sl
        for u in range(units):
            assert seen[u] == list(range(tiles)) and sorted(slots[u]) == list(range(pl["pre_splits"])), (pl, P, u)


@pytest.mark.parametrize("sms", [1, 2, 3, 7])
def test_shared_plan_covers_on_few_sms(fpd, sms):
    check_cover(fpd, 1, 2, 128, 2, 128, 18305, 1000, sms)
    for B, L, nq, nkv, h in SHAPES[:8]:
        for p_cap in (100, 4096, 20000):
            for t_cap in (0, 1000):
                check_cover(fpd, B, L, nq, nkv, h, p_cap, t_cap, sms)


def test_shared_plan_rules(fpd):
    """The calls whose choice the comments beside the rules quote."""
    assert not plan(fpd, 1, 16, 32, 8, 128, 512, 0)["pre_tc"]                      # small: mma.sync
    p = plan(fpd, 8, 16, 32, 8, 128, 2048, 256)
    assert p["pre_tc"] and p["own_tc"] and p["pre_runs"] == 64                     # four runs per unit of 256 rows
    p = plan(fpd, 64, 16, 32, 8, 128, 16384, 512)
    assert p["pre_tc"] and not p["own_tc"] and p["pre_runs"] == 152                # own parts of 64 rows on mma.sync
    assert plan(fpd, 64, 16, 32, 8, 128, 1024, 2048)["own_tc"]
    p = plan(fpd, 4, 385, 32, 8, 128, 4096, 128)
    assert p["pre_tc"] and p["own_tc"] and p["own_cost"] > 0                       # shorter prefix runs beside own runs
    p = plan(fpd, 16, 1, 32, 8, 128, 65536, 512)
    assert p["pre_tc"] and p["own_tc"] and p["pre_runs"] + p["own_ctas"] == 152      # own runs beside the prefix's read
    assert p["own_ctas"] * p["own_alone"] >= 16 * 8
    p = plan(fpd, 64, 4, 32, 8, 128, 512, 1024)
    assert p["own_alone"] > 0 and p["own_ctas"] * p["own_alone"] < 64 * 8          # some of them, then all CTAs in turn
    assert not plan(fpd, 200, 1, 32, 8, 128, 2500, 60)["own_tc"]                   # many short own parts on mma.sync
    assert plan(fpd, 200, 1, 32, 8, 128, 2500, 1024)["own_tc"]
    p = plan(fpd, 2, 2, 130, 1, 128, 20000, 0)
    assert not p["pre_tc"] and not p["own_tc"]                                     # 130 heads do not fit 128 rows


# ---- how the collected weights' key tiles are dealt -----------------------------------------------------------------

def shares(fpd, lens, nkv, ctas, walked=None, max_units=100000):
    lib, I = fpd.lib(), ctypes.c_int
    P = ctypes.POINTER(ctypes.c_int32)
    lib.fpd_test_weight_shares.argtypes = [I, I, P, P, I, I, I, P, P]
    a, b = ((ctypes.c_int32 * len(lens))(*v) for v in (lens, walked or lens))
    out, n = (ctypes.c_int32 * (4 * max_units))(), ctypes.c_int32()
    got = []
    for c in range(ctas):
        assert lib.fpd_test_weight_shares(len(lens), nkv, a, b, c, ctas, max_units, out, ctypes.byref(n)) == 0
        got.append([tuple(out[4 * i:4 * i + 4]) for i in range(n.value)])
    return got


@pytest.mark.parametrize("lens", [[1], [0, 0], [128, 129, 0, 1], [2000, 1, 5, 64, 1999, 0, 3, 128], [0] * 40 + [300] + [0] * 50,
                                  [(97 * i) % 700 for i in range(75)]])
def test_weight_shares_cover_every_key_tile_once(fpd, lens):
    for nkv in (1, 8):
        for ctas in (1, 2, 7, 152):
            got = shares(fpd, lens, nkv, ctas)
            tiles = [(b, g, t) for b, n in enumerate(lens) for g in range(nkv) for t in range(-(-n // 128))]
            seen = [(b, g, k // 128 + i) for c in got for b, g, k, nk in c for i in range(nk)]
            assert seen == tiles
            per = [sum(u[3] for u in c) for c in got]
            assert max(per) - min(per) <= 1


def test_weight_shares_end_under_lengths_that_change(fpd):
    """Shorter or longer lengths after the count: a walk that ends, within the requests and kv heads."""
    rng = np.random.default_rng(3)
    for k in range(60):
        n = int(rng.integers(1, 70))
        lens = rng.integers(0, 2000, n).tolist()
        walked = [0] * n if k % 3 == 0 else rng.integers(0, 2000, n).tolist()
        for c in shares(fpd, lens, 2, 9, walked):
            assert all(0 <= b < n and 0 <= g < 2 and k0 < walked[b] and nk in (1, 2) for b, g, k0, nk in c)
