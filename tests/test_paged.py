"""CPU: what the paged context cache and the sampled verification refuse before they touch the device, how the attention's key
tiles are shared out, and the references' own rules."""
import ctypes

import numpy as np
import pytest

import paged_ref as ref


@pytest.fixture(scope="module")
def fpd():
    import __graft_entry__ as g
    g._compile_all()
    import block_diffusion_speculative_non_gb300 as pkg
    return pkg


A = 1 << 20   # an address that is never dereferenced


def store(fpd, **kw):
    a = dict(pages=A, table=A, format=0, n_layers=2, n_pages=9, page_size=16, n_kv_heads=2, head_dim=64, table_width=4)
    a.update(kw)
    return fpd.PagedStore(*a.values())


STORES = [(dict(format=2), 1), (dict(format=-1), 1), (dict(head_dim=96), 4), (dict(page_size=8), 4), (dict(page_size=48), 4),
          (dict(page_size=256), 4), (dict(n_kv_heads=0), 2), (dict(n_layers=0), 2), (dict(n_pages=0), 2), (dict(table_width=0), 2),
          (dict(table_width=(1 << 30) // 16 + 1), 2), (dict(pages=None), 1), (dict(table=None), 1), (dict(pages=A + 8), 1),
          (dict(table=A + 2), 1)]


def append(fpd, st=None, **kw):
    a = dict(batch=2, rows=4, store=ctypes.byref(st or store(fpd)), layer=1, k=A, k_ld=128, v=A, v_ld=128, off=A, cnt=None, start=None,
             offset=None, rope=A, max_pos=64)
    a.update(kw)
    return fpd.lib().fpd_paged_append(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), 2), (dict(rows=-1), 2), (dict(rows=(1 << 26) + 1), 2), (dict(layer=2), 2), (dict(layer=-1), 2), (dict(store=None), 1),
    (dict(k=None), 1), (dict(v=None), 1), (dict(off=None), 1), (dict(k_ld=120), 2), (dict(v_ld=132), 2), (dict(max_pos=0), 2),
    (dict(k=A + 8), 1), (dict(v=A + 2), 1), (dict(rope=A + 8), 1)])
def test_append_refuses(fpd, kw, status):
    assert append(fpd, **kw) == status, fpd.fpd_last_error()
    assert fpd.fpd_last_error()


@pytest.mark.parametrize("kw,status", STORES)
def test_store_is_checked_by_every_call(fpd, kw, status):
    st = store(fpd, **kw)
    p = ctypes.byref(st)
    assert append(fpd, st) == status
    assert fpd.lib().fpd_paged_read(1, 1, p, 0, A, None, None, A, A, None) == status
    assert attention(fpd, st) == status
    if "pages" not in kw and "table" not in kw:
        assert fpd.lib().fpd_paged_attention_workspace_bytes(1, 1, 2, p) == 0


def test_read_refuses(fpd):
    p, call = ctypes.byref(store(fpd)), fpd.lib().fpd_paged_read
    assert call(0, 1, p, 0, A, None, None, A, A, None) == 2 and call(1, -1, p, 0, A, None, None, A, A, None) == 2
    assert call(1, 1, p, 0, None, None, None, A, A, None) == 1 and call(1, 1, p, 0, A, None, None, None, A, None) == 1
    assert call(1, 1, p, 0, A, None, None, A, A + 8, None) == 1 and call(1, 1, p, 2, A, None, None, A, A, None) == 2


def attention(fpd, st=None, **kw):
    a = dict(batch=2, block=4, nq=8, store=ctypes.byref(st or store(fpd)), layer=0, q=A, kb=A, vb=A, lens=A, window=0, sinks=0, causal=0,
             out=A, lse=A, ws=A, n=1 << 30)
    a.update(kw)
    return fpd.lib().fpd_paged_attention(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), 2), (dict(block=0), 2), (dict(nq=7), 2), (dict(nq=1), 2), (dict(nq=258), 4), (dict(layer=5), 2), (dict(window=-1), 2),
    (dict(sinks=-1), 2), (dict(batch=1 << 20, block=1 << 12), 2), (dict(batch=1 << 14, block=1 << 10), 2), (dict(q=None), 1),
    (dict(kb=None), 1), (dict(vb=None), 1), (dict(lens=None), 1), (dict(out=None), 1), (dict(ws=None), 1), (dict(q=A + 8), 1),
    (dict(out=A + 4), 1), (dict(ws=A + 8), 1), (dict(vb=A + 2), 1), (dict(store=None), 1)])
def test_attention_refuses(fpd, kw, status):
    assert attention(fpd, **kw) == status, fpd.fpd_last_error()
    assert fpd.fpd_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), 2), (dict(block=1), 2), (dict(vocab=0), 2), (dict(vocab=(1 << 26) + 1), 2), (dict(batch=1 << 20, block=1 << 11), 2),
    (dict(draft=None), 1), (dict(target=None), 1), (dict(u=None), 1), (dict(accept=None), 1), (dict(committed=None), 1),
    (dict(target=A + 4), 1), (dict(probs=A + 8), 1)])
def test_verify_sampled_refuses(fpd, kw, status):
    a = dict(batch=2, block=4, vocab=10, draft=A, target=A, probs=None, u=A, accept=A, committed=A, valid=None)
    a.update(kw)
    assert fpd.lib().fpd_verify_sampled(*a.values(), None) == status, fpd.fpd_last_error()
    assert fpd.fpd_last_error()


def test_page_bytes(fpd):
    assert fpd.fpd_page_bytes(fpd.FPD_PAGE_BF16, 64, 8, 128) == 2 * 8 * 64 * 256
    assert fpd.fpd_page_bytes(fpd.FPD_PAGE_INT4, 64, 8, 128) == 2 * 8 * 64 * 72
    assert fpd.fpd_page_bytes(fpd.FPD_PAGE_INT4, 16, 1, 64) == 2 * 16 * 36
    assert fpd.fpd_page_bytes(0, 17, 8, 128) == 0 and fpd.fpd_page_bytes(0, 16, 8, 80) == 0 and fpd.fpd_page_bytes(7, 16, 8, 64) == 0


def test_binding_checks_tensors(fpd):
    """Type, place, layout and size of a tensor are checked before the library sees its address."""
    import torch
    bf, i32 = torch.zeros(4096, dtype=torch.bfloat16), torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError, match="pages of format"):
        fpd.paged_store(64, 0, 1, 4, 17, 2, 64, 64, 4)
    with pytest.raises(ValueError, match="current device"):
        fpd.paged_store(bf, 0, 1, 1, 16, 1, 64, 64, 4)
    with pytest.raises(ValueError, match="pages must be torch.uint8"):
        fpd.paged_store(bf, 1, 1, 1, 16, 1, 64, 64, 4)
    with pytest.raises(ValueError, match="table must be"):
        fpd.paged_store(64, 0, 1, 1, 16, 1, 64, i32)
    with pytest.raises(ValueError, match="needs table_width"):
        fpd.paged_store(64, 0, 1, 1, 16, 1, 64, 64)
    import types
    calls = fpd.paged._paged()
    kept = fpd.PagedStore(64, 64, 0, 1, 4, 16, 2, 64, 4)
    st = ctypes.addressof(kept)
    att = [1, 2, 4, st, 0, 64, None, None, 64, 0, 0, 0, 64, None, 64, 1, None, 0]
    with pytest.raises(TypeError, match="17 arguments, the call takes 18"):
        calls.paged_attention(*att[:-1])
    with pytest.raises(ValueError, match="q holds 4096 elements, the call needs 8192"):
        calls.paged_attention(16, *att[1:5], bf, *att[6:])
    with pytest.raises(ValueError, match="ctx_len must be torch.int32"):
        calls.paged_attention(*att[:8], i32.long(), *att[9:])
    with pytest.raises(OverflowError):
        calls.paged_attention(*att[:9], 1 << 40, *att[10:])
    app = [1, 2, st, 0, 64, 128, 64, 128, 64, None, None, None, None, 0, None, 0]
    wide = bf.view(8, 512)
    with pytest.raises(ValueError, match="k must have 2 rows of at least 128 elements, 384 elements apart"):
        calls.paged_append(*app[:4], wide[:, :128], 384, *app[6:])
    with pytest.raises(ValueError, match="k must have 20 rows"):
        calls.paged_append(1, 20, *app[2:4], wide[:, :128], 512, *app[6:])
    with pytest.raises(ValueError, match="k must have 2 rows of at least 128"):
        calls.paged_append(*app[:4], wide[:, :64], 512, *app[6:])
    with pytest.raises(ValueError, match="the rows of k must be contiguous"):
        calls.paged_append(*app[:4], wide[:, ::2], 512, *app[6:])
    with pytest.raises(ValueError, match="k is on cpu"):
        calls.paged_append(*app[:4], wide[:, 128:256], 512, *app[6:])
    with pytest.raises(ValueError, match="k holds 4096 elements, the call needs 8192"):
        calls.paged_read(1, 64, st, 0, 64, None, None, bf, 64, None, 0)
    with pytest.raises(ValueError, match="target holds 4 elements, the call needs 20"):
        calls.verify_sampled(1, 2, 10, 64, torch.zeros(4), None, 64, 64, 64, None, None, 0)
    s = fpd.PagedStore(64, 64, 0, 1, 4, 16, 2, 64, 4)
    s._rows, s._dev = 2, 0
    with pytest.raises(ValueError, match="the table has 2 requests, the call needs 3"):
        fpd.paged._store(s, 3, 0)
    with pytest.raises(ValueError, match="the pages are on cuda:0, the current device is cuda:1"):
        fpd.paged._store(s, 1, 1)
    with pytest.raises(TypeError, match="must be a PagedStore"):
        fpd.paged._store(types.SimpleNamespace(), 1, 0)
    assert calls.paged_attention(0, *att[1:]) != 0 and calls.verify_sampled(0, 2, 10, *[64] * 7, None, 0) != 0


# ---- how the key tiles are shared out ------------------------------------------------------------------------------------

def walk(fpd, lens, L, lb, grp, nkv, rows, window, sinks, causal, kt, cost, runs, walked=None, most=4000):
    f, P, I = fpd.lib().fpd_test_paged_walk, ctypes.POINTER(ctypes.c_int32), ctypes.c_int
    f.argtypes = [I] * 11 + [P, P, I, I, I, P, P]
    a, b = ((ctypes.c_int32 * len(lens))(*v) for v in (lens, walked or lens))
    out, n = (ctypes.c_int32 * (7 * most))(), ctypes.c_int32()
    got = []
    for c in range(runs):
        assert f(len(lens), L, lb, grp, nkv, rows, window, sinks, causal, kt, cost, a, b, runs, c, most, out, ctypes.byref(n)) == 0
        got.append([tuple(out[7 * i:7 * i + 7]) for i in range(n.value)])
    return got


def tiles(fpd, T, rt, L, lb, grp, rows, window, sinks, causal, kt, most=4000):
    f, P, I = fpd.lib().fpd_test_paged_tiles, ctypes.POINTER(ctypes.c_int32), ctypes.c_int
    f.argtypes = [I] * 11 + [P, P]
    out, n = (ctypes.c_int32 * (5 * most))(), ctypes.c_int32()
    assert f(L, lb, grp, rows, window, sinks, causal, kt, T, rt, most, out, ctypes.byref(n)) == 0
    return [tuple(out[5 * i:5 * i + 5]) for i in range(n.value)]


SHAPES = [dict(L=1, grp=4, rows=16), dict(L=7, grp=5, rows=64), dict(L=16, grp=4, rows=64), dict(L=100, grp=3, rows=64),
          dict(L=385, grp=4, rows=256), dict(L=33, grp=1, rows=16), dict(L=3, grp=128, rows=64)]
MASKS = [(0, 0, 0), (0, 0, 1), (1, 0, 0), (9, 3, 1), (70, 64, 0), (300, 130, 1), (2 ** 30, 5, 0), (64, 2 ** 30, 1), (128, 1, 1)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("blk", [0, 1])
def test_a_units_tiles_hold_what_its_rows_see(fpd, shape, blk):
    L, grp, rows = shape["L"], shape["grp"], shape["rows"]
    for window, sinks, causal in MASKS:
        for T in (0, 1, 63, 64, 65, 200, 1000):
            n = T + (L if blk else 0)
            see = ref.visible(L, n, window, sinks, causal) if n else np.zeros((L, 0), bool)
            for kt in (64, 128):
                for rt in range(-(-L * grp // rows)):
                    j0, j1 = rt * rows // grp, (min(L * grp, (rt + 1) * rows) - 1) // grp
                    held = np.zeros(n, int)
                    got = tiles(fpd, T, rt, L, L if blk else 0, grp, rows, window, sinks, causal, kt)
                    for ctx, k0, valid, pos, full in got:
                        assert 1 <= valid <= kt and k0 % kt == 0 and pos == (k0 if ctx else T + k0)
                        assert k0 + valid <= (T if ctx else L)
                        held[pos:pos + valid] += 1
                        if full:
                            assert valid == kt and see[j0:j1 + 1, pos:pos + kt].all()
                    assert held.max(initial=0) <= 1
                    assert (held[see[j0:j1 + 1].any(0)] == 1).all()
                    # no tile without a key that some row sees, but for keys between the rows' own ranges
                    if not window:
                        for ctx, k0, valid, pos, full in got:
                            assert see[j0:j1 + 1, pos:pos + valid].any()


@pytest.mark.parametrize("cost", [0, 3])
@pytest.mark.parametrize("lens", [[0], [1], [130, 0, 64, 1000], [5] * 300, [(97 * i) % 700 for i in range(75)]])
def test_walks_cover_every_tile_once(fpd, lens, cost):
    for L, lb, grp, rows, nkv, (window, sinks, causal), kt in [
            (1, 1, 4, 16, 2, (0, 0, 0), 64), (16, 16, 4, 64, 8, (0, 0, 0), 128), (30, 0, 5, 64, 1, (100, 70, 1), 64),
            (30, 30, 5, 64, 3, (0, 0, 1), 64)]:
        for runs in (1, 7, 304):
            got = walk(fpd, lens, L, lb, grp, nkv, rows, window, sinks, causal, kt, cost, runs)
            flat = [(p, c) for c, parts in enumerate(got) for p in parts]
            want = [(b, g, rt, max(1, len(tiles(fpd, T, rt, L, lb, grp, rows, window, sinks, causal, kt))))
                    for b, T in enumerate(lens) for g in range(nkv) for rt in range(-(-L * grp // rows))]
            at, i = 0, 0
            for (b, g, rt, t0, t1, n, last), c in flat:   # in order, each unit's parts one behind the other
                assert (b, g, rt, n) == want[i] and t0 == at and t0 < t1 <= n
                at = t1
                if t1 == n:
                    assert last == c
                    at, i = 0, i + 1
                elif t0 == 0:
                    ends = [e for (p, e) in flat if p[:3] == (b, g, rt) and p[4] == n]
                    assert ends == [last]
            assert i == len(want) and at == 0
            # a run's tiles and the ends of its units, within the even share
            share = -(-sum(w[3] + cost for w in want) // min(runs, sum(w[3] + cost for w in want)))
            assert max(sum(p[4] - p[3] for p in parts) + cost * sum(p[4] == p[5] for p in parts[:-1]) for parts in got) <= share


def test_walks_stay_in_bounds_under_lengths_that_change(fpd):
    rng = np.random.default_rng(5)
    for k in range(40):
        n = int(rng.integers(1, 200))
        lens = rng.integers(0, 2000, n).tolist()
        other = [0] * n if k % 3 == 0 else rng.integers(0, 2000, n).tolist()
        for window, sinks, causal in ((0, 0, 0), (50, 3, 1)):
            for c, parts in enumerate(walk(fpd, lens, 20, 20, 5, 2, 64, window, sinks, causal, 64, k % 4, 9, other)):
                for b, g, rt, t0, t1, m, last in parts:
                    assert 0 <= b < n and 0 <= g < 2 and 0 <= rt < 2 and 0 <= t0 < t1 <= m and c <= last < 9


# ---- the references ------------------------------------------------------------------------------------------------------

def test_quantiser_of_the_reference():
    x = np.zeros((1, 32))
    x[0, :3] = [7, -7, 3.5]
    x[0, 16:19] = [np.inf, np.nan, 1.0]
    n, b = ref.quantise(x)
    assert n[0, :4].tolist() == [7, -7, 4, 0] and ref.SCALES[b[0, 0]] == 1.0          # 3.5 is a tie: to the even 4
    assert n[0, 16:19].tolist() == [7, 0, 0] and ref.SCALES[b[0, 1]] == 2.0 ** 13
    code, _ = ref.pack(n, b)
    assert code[0, 0] == (7 + 8) + 16 * (8 - 7)
    rng = np.random.default_rng(0)
    x = rng.normal(size=(50, 64)) * 10.0 ** rng.integers(-3, 4, (50, 1))
    n, b = ref.quantise(x)
    s = np.repeat(np.array(ref.SCALES)[b], 16, -1)
    assert (np.abs(x - ref.stands_for(n, b)) <= s / 2).all() and np.abs(n).max() <= 7
    assert (7 * np.array(ref.SCALES)[b - 1] < np.abs(x.reshape(50, 4, 16)).max(-1)).all()   # no smaller scale would do


def test_sampled_verification_of_the_reference_gives_the_targets_distribution():
    """Over a grid of the two random numbers the first committed id comes as often as the target says."""
    p, q, N = np.array([0.5, 0.25, 0.125, 0.125], np.float32), np.array([0.125, 0.5, 0.25, 0.125], np.float32), 64
    seen = np.zeros(4)
    for d in range(4):
        for i in range(N):
            for j in range(N):
                _, c, _ = ref.verify_sampled([d], np.stack([p, p]), q[None], [(i + 0.5) / N, (j + 0.5) / N])
                seen[c[0]] += q[d]
    assert np.abs(seen / N ** 2 - p).max() <= 1 / N
