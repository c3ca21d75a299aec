// k_attention_shared_tc.cu — the shared-prefix attention on the 5th-generation tensor cores.  The formulas and the partials
// are those of k_attention_shared.cu.
//
// A CTA works on two "lanes", each a 128-row S / P / O set in tensor memory with a softmax warpgroup of its own, so
// that one lane's softmax runs while the tensor core works for the other.  Warps:
//   0, 2   TMA producers of K and Q, and of V: tiles of 128 keys (64-dim boxes, 128-byte swizzle), two K and three V deep;
//   1      MMA issuer: S = Q K^T, then O += (P_hi + P_lo) V with P read from tensor memory; a lane's next S is issued right
//          behind its product, so that it waits for its own softmax alone;
//   3..6   softmax of lane 0, 7..10 of lane 1: one thread per query row, the 128 scores of a tile in registers (one read of
//          tensor memory per tile), p = 2^(s log2e/sqrt(h) - m) written back over S as two bf16 terms; O is rescaled only
//          when the maximum rises by more than 2^8 (p stays below 2^8: O / l is exact either way).
//
// A lane's rows are whole positions, the kv head's heads of each (128 rows, or less when the heads do not divide it): one
// box of a [position][head][h] map of q.  A unit is a pair of such row tiles of a part's rows in one kv head: the lanes hold
// one tile each and share every K/V tile.  Where a unit has the rows of one lane only (few blocks, the own part of a text
// block, the last rows of a long one), both lanes hold the same rows and take the even and the odd key tiles: such a unit is
// a read of the keys, and two key streams keep the copies in flight.  The prefix's (unit, key tile) space is cut into one
// contiguous run of tiles per CTA, so that all SMs finish together whatever the number of rows; a run that spans units
// leaves a partial in each.  The own part's units follow, dealt out from the other end: the CTAs without a run of the prefix
// take as many of them first as fit beside such a run, then all CTAs take turns (64 tokens behind 4096 positions with
// contexts to 1024: 60 us, 89 when all took turns from the start); where every CTA has a run, the prefix's runs are shorter
// by what a CTA has of them.
//
// What bounds it: with many rows the tensor core, 48 products of 64 cycles per pair of tiles and key tile, 72 % of the
// cycles busy at 64 blocks of 16 positions behind 16384 keys (237 us, 1.16 PFLOP/s of the formula's 4 h, 1.74 of products;
// the clock falls to 1.6-1.9 GHz under the power limit); with few rows the read of the keys, 6.7 TB/s while it lasts at 16
// tokens behind 65536 positions (59 us in all, 42 the floor: the start and the merge do not overlap it).  An own unit costs
// about 5 us besides 1.1 us per tile: its first S waits for its Q and K, and its partial goes out before the next one's product.
#include <cstring>

#include "attn_tc_prims.cuh"
#include "fpd_context.cuh"

namespace fpd {

namespace {
using namespace attn_tc;

constexpr int QR = 128, KT = 128;      // most rows of a lane, keys of a tile
constexpr int kThreads = 11 * 32;
constexpr int KST = 2, VST = 3;        // K and V ring slots: a K tile is free once S is, a V tile only behind the softmax
constexpr int kTmemCols = 512;         // S/P of lane t at 128 t, O of lane t at 256 + 128 t
constexpr uint32_t kTmemO = 256;
constexpr float kRescaleLog2 = 8.f;
constexpr int ATOM_BYTES = KT * 64 * 2;   // 128 rows x 64 dims

// shared memory: Q[2] | K[KST] | V[VST] | barriers
template <int HD>
struct Lay {
  static constexpr int TILE = KT * HD * 2, ATOMS = HD / 64;
  static constexpr int Q = 0, K = 2 * TILE, V = K + KST * TILE, BAR = V + VST * TILE;
};
// barriers: q_full, q_empty [lane], k_full, k_empty, v_full, v_empty [slot], s_full, p_full, pv_done [lane], end
enum {
  B_Q = 0,
  B_QE = B_Q + 2,
  B_KF = B_QE + 2,
  B_KE = B_KF + KST,
  B_VF = B_KE + KST,
  B_VE = B_VF + VST,
  B_SF = B_VE + VST,
  B_PF = B_SF + 2,
  B_PV = B_PF + 2,
  B_END = B_PV + 2,
  B_N = B_END + 1
};
template <int HD>
constexpr size_t smem_bytes() {
  return 1024 + (size_t)Lay<HD>::BAR + 8 * B_N + 16;
}
static_assert(smem_bytes<128>() <= 232448, "tile set exceeds the shared memory of one CTA");
static_assert(2 * QR * (128 * 4 + 16) <= (KST + VST) * Lay<128>::TILE && 2 * QR * (64 * 4 + 16) <= (KST + VST) * Lay<64>::TILE,
              "the staged partials must fit in the K and V slots");

// Division by a number known on the host (Granlund and Montgomery's multiply, add and shift; exact for 32-bit operands).
struct FastDiv {
  uint32_t d, m, s1, s2;
  void set(uint32_t n) {
    d = n;
    uint32_t l = 0;
    while ((1ull << l) < n) l++;
    m = (uint32_t)(((1ull << 32) * ((1ull << l) - n)) / n + 1);
    s1 = l > 0 ? 1 : 0;
    s2 = l > 0 ? l - 1 : 0;
  }
  __device__ __forceinline__ int div(int x) const {
    const uint32_t t = __umulhi(m, (uint32_t)x);
    return (int)((t + (((uint32_t)x - t) >> s1)) >> s2);
  }
};

struct TcArgs {
  CUtensorMap tm_q;                               // q as [rows][nq][h], boxes of npt positions x grp heads
  CUtensorMap tm_pre, tm_own, tm_kblk, tm_vblk;   // [rows][h] views of the prefix, the own store, the block keys and values
  SharedAttn a;
  int grp, npt, rpt;                     // heads per kv head, positions and rows of a lane
  int pre_tiles, pre_units, pre_slots;   // row pairs per kv head, units, partial slots of a prefix row (0 units: not here)
  int pre_runs;                          // CTAs that share the prefix's tiles
  int pre_pieces;                        // most runs of a unit
  int own_ctas, own_alone;               // CTAs, from the last, that take own units up to own_alone by themselves
  int own_cost;                          // an own run in key tiles of the prefix, or 0: even runs
  int own_tiles, own_units, own_splits;  // the same for the own part, with the key splits of a unit
  int own_slot0;                         // first partial slot of the own part
  FastDiv by_grp, by_pre_tiles, by_own_tiles, by_own_units, by_nkv;
};

// One run of key tiles of one unit.
struct Seg {
  bool prefix, keys;           // keys: one lane's rows, the lanes take even and odd tiles
  int g, row0, nrows, n0;      // rows row0 .. of the part's nrows; the part's first row in [rows]
  int slot, pad_end;           // partial slot (of lane 0); slots up to pad_end that this run does not fill are marked empty
  int T, kb, ke, n_ctx, n_tiles;
  int krow, vrow, brow;        // first row of the stores' keys and values and of the block's in the tensor maps

  __device__ void range(int kb_, int ke_) {
    kb = kb_;
    ke = ke_;
    const int ce = min(ke, T), bb = max(kb, T);
    n_ctx = ce > kb ? (ce - kb + KT - 1) / KT : 0;
    n_tiles = n_ctx + (ke > bb ? (ke - bb + KT - 1) / KT : 0);
  }
  __device__ void tile(int i, int& first, int& valid, bool& ctx) const {
    ctx = i < n_ctx;
    first = ctx ? kb + i * KT : max(kb, T) + (i - n_ctx) * KT;
    valid = min(KT, (ctx ? min(ke, T) : ke) - first);
  }
  __device__ int lane_tiles(int t) const { return keys ? (n_tiles - t + 1) / 2 : n_tiles; }
  __device__ int lane_row0(int t, int rpt) const { return row0 + (keys ? 0 : t * rpt); }
};

// The runs of this CTA, in order.
struct Walk {
  const TcArgs& p;
  int P, P_tiles, G, c, own_i, W, own_even, own_first;   // own runs: own_even each, one more from CTA own_first on
  long long x, x_end, total;
  int empty_u;      // an empty prefix still marks its partial slots
  __device__ Walk(const TcArgs& p_) : p(p_) {
    c = blockIdx.x;
    P = p.pre_units ? clamp_ctx(p.a.prefix_len[0], p.a.p_cap) : 0;
    P_tiles = (P + KT - 1) / KT;
    total = (long long)p.pre_units * P_tiles;
    G = (int)min((long long)p.pre_runs, max(total, 1ll));
    W = 0;
    if (p.own_cost && total >= 16ll * G && G == (int)gridDim.x) {
      const int own_n = p.own_units * p.own_splits;
      own_even = own_n / G;
      own_first = G - own_n % G;
      // no run shorter than half of the average, and no more runs in a unit than there are partial slots
      W = (int)min((long long)p.own_cost, total / (2ll * G * (own_even + 1) - own_n));
      const int shortest = (int)((total + (long long)W * own_n) / G) - 1 - W * (own_even + 1);
      if ((P_tiles + shortest - 1) / shortest + 1 > p.pre_pieces) W = 0;
    }
    x = c < G ? run_start(c) : 0;
    x_end = c < G ? run_start(c + 1) : 0;
    empty_u = total == 0 ? c : p.pre_units;
    own_i = (int)gridDim.x - 1 - c;
    if (own_i >= p.own_ctas) own_i += p.own_alone;
  }
  // run c starts at tile c total / G, or, with own runs that count as W tiles each, where the runs before it end; the run
  // that holds tile t is the last one that starts at or before it
  // (64-bit divisions cost a few hundred cycles: only where 32 bits do not hold the products)
  __device__ long long run_start(int i) const {
    if (W) {
      const long long own_n = p.own_units * p.own_splits;
      return i * (total + W * own_n) / G - (long long)W * (own_even * i + max(0, i - own_first));
    }
    return total < (1 << 20) ? (uint32_t)i * (uint32_t)total / (uint32_t)G : i * total / G;
  }
  __device__ int run_of(long long t) const {
    if (W) {
      int lo = 0, hi = G;   // run_start(lo) <= t < run_start(hi)
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (run_start(mid) <= t) lo = mid; else hi = mid;
      }
      return lo;
    }
    return total < (1 << 20) ? (int)((((uint32_t)t + 1) * (uint32_t)G - 1) / (uint32_t)total) : (int)(((t + 1) * G - 1) / total);
  }
  __device__ void rows(Seg& s, int qp, int nrows) const {
    s.row0 = qp * 2 * p.rpt;
    s.nrows = nrows;
    s.keys = nrows - s.row0 <= p.rpt;
  }
  __device__ void prefix_unit(Seg& s, int u) const {
    s.prefix = true;
    s.g = p.by_pre_tiles.div(u);
    rows(s, u - s.g * p.pre_tiles, p.a.rows * p.grp);
    s.n0 = 0;
    s.T = P;
    s.krow = s.g * p.a.p_cap;
    s.vrow = (p.a.nkv + s.g) * p.a.p_cap;
    s.brow = 0;
  }
  __device__ bool more() const { return empty_u < p.pre_units || x < x_end || own_i < p.own_units * p.own_splits; }
  __device__ bool next(Seg& s) {
    if (empty_u < p.pre_units) {
      prefix_unit(s, empty_u);
      s.range(0, 0);
      s.slot = 0;
      s.pad_end = p.pre_slots;
      empty_u += gridDim.x;
      return true;
    }
    if (x < x_end) {
      const int u = total < (1 << 20) ? (int)((uint32_t)x / (uint32_t)P_tiles) : (int)(x / P_tiles);
      const long long u0 = (long long)u * P_tiles, e = min(x_end, u0 + P_tiles);
      prefix_unit(s, u);
      s.range((int)(x - u0) * KT, (int)min((long long)P, (e - u0) * KT));
      const int piece = c - run_of(u0);   // runs since the one that holds the unit's first tile
      s.slot = s.keys ? 2 * piece : piece;
      s.pad_end = e == u0 + P_tiles ? p.pre_slots : 0;
      x = e;
      return true;
    }
    if (own_i < p.own_units * p.own_splits) {
      const int split = p.by_own_units.div(own_i), u = own_i - split * p.own_units;
      const int bg = p.by_own_tiles.div(u), b = p.by_nkv.div(bg);
      s.prefix = false;
      s.g = bg - b * p.a.nkv;
      rows(s, u - bg * p.own_tiles, p.a.L * p.grp);
      s.n0 = b * p.a.L;
      s.T = p.a.ck ? clamp_ctx(p.a.ctx_len[b], p.a.t_cap) : 0;
      s.krow = ((b * 2 + 0) * p.a.nkv + s.g) * p.a.t_cap;
      s.vrow = ((b * 2 + 1) * p.a.nkv + s.g) * p.a.t_cap;
      s.brow = (b * p.a.nkv + s.g) * p.a.lb;
      const int n = s.T + p.a.lb, nt = (n + KT - 1) / KT;
      if (p.own_splits == 1) s.range(0, n);
      else s.range((int)((long long)split * nt / p.own_splits) * KT, (int)min((long long)n, (split + 1ll) * nt / p.own_splits * KT));
      s.slot = p.own_slot0 + 2 * split;
      s.pad_end = s.slot + 2;
      own_i += own_i < p.own_alone ? p.own_ctas : (int)gridDim.x;
      return true;
    }
    return false;
  }
};

// (a, b) >= 0 -> two packed bf16 pairs, a = hi_a + lo_a to 2^-16: hi keeps the upper half of the word (no rounding, so the
// rest is exact in fp32), lo is the rest rounded.  Fewer steps per pair than rounding hi to nearest.
__device__ __forceinline__ void split_trunc(float a, float b, uint32_t& hi, uint32_t& lo) {
  const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
  hi = __byte_perm(ua, ub, 0x7632);
  const uint64_t rest = add2(pack2(a, b), pack2(-__uint_as_float(ua & 0xFFFF0000u), -__uint_as_float(ub & 0xFFFF0000u)));
  float ra, rb;
  unpack2(rest, ra, rb);
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(rb), "f"(ra));
}
__device__ __forceinline__ void st8(float* dst, const float* v) {   // 32-byte aligned
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]),
               "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1) shared_tc_kernel(const __grid_constant__ TcArgs p) {
  using S = Lay<HD>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + B_N);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t bar0 = tc::smem_u32(bars);
  auto bar = [&](int i) { return bar0 + 8 * i; };
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // warp: known uniform

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; t++) {
      tc::mbar_init(bar(B_Q + t), 1);
      tc::mbar_init(bar(B_QE + t), 1);
      tc::mbar_init(bar(B_SF + t), 1);
      tc::mbar_init(bar(B_PF + t), 4);
      tc::mbar_init(bar(B_PV + t), 1);
    }
    for (int s = 0; s < KST; s++) {
      tc::mbar_init(bar(B_KF + s), 1);
      tc::mbar_init(bar(B_KE + s), 1);
    }
    for (int s = 0; s < VST; s++) {
      tc::mbar_init(bar(B_VF + s), 1);
      tc::mbar_init(bar(B_VE + s), 1);
    }
    tc::mbar_init(bar(B_END), 1);
    *abort_flag = 0;
    tc::fence_barrier_init();
    tc::tma_prefetch(&p.tm_q);
    if (p.pre_units) tc::tma_prefetch(&p.tm_pre);
    if (p.own_units && p.a.ck) tc::tma_prefetch(&p.tm_own);
    if (p.own_units && p.a.lb) {
      tc::tma_prefetch(&p.tm_kblk);
      tc::tma_prefetch(&p.tm_vblk);
    }
  }
  if (warp == 1) {
    tc::tmem_alloc(tc::smem_u32(tmem_slot), kTmemCols);
    tc::tmem_relinquish();
  }
  __syncwarp();   // a CTA barrier counts a whole warp: single-lane roles reconverge before every one
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  pdl_wait();
  pdl_trigger();

  Walk walk(p);
  Seg sg;

  if (warp == 0 || warp == 2) {
    // ---------------- TMA producers: K and Q (warp 0), V (warp 2) ----------------
    // one each: a K slot is free much earlier than a V slot, and its copy must not queue behind a V that waits
    if (lane == 0) {
      const bool is_v = warp == 2;
      const int ST = is_v ? VST : KST, full = is_v ? B_VF : B_KF, empty = is_v ? B_VE : B_KE;
      const uint32_t ring = tc::smem_u32(smem + (is_v ? S::V : S::K));
      const CUtensorMap* blk = is_v ? &p.tm_vblk : &p.tm_kblk;
      int n = 0, nq[2] = {0, 0};   // tiles and Q loads since the start: ring slot and phase
      while (!*abort_flag && walk.next(sg)) {
        const CUtensorMap* ctx_map = sg.prefix ? &p.tm_pre : &p.tm_own;
        const int row0 = is_v ? sg.vrow : sg.krow;
        for (int i = 0; i < sg.n_tiles && !*abort_flag; i++) {
          const int s = n % ST;
          int first, valid;
          bool ctx;
          sg.tile(i, first, valid, ctx);
          if (n >= ST && !wait_bar(bar(empty + s), ((n / ST) & 1) ^ 1)) { *abort_flag = 1; break; }
          tc::mbar_arrive_expect_tx(bar(full + s), S::TILE);
          const int row = ctx ? row0 + first : sg.brow + first - sg.T;
          for (int h = 0; h < S::ATOMS; h++)
            tc::tma_load_2d(ring + s * S::TILE + h * ATOM_BYTES, ctx ? ctx_map : blk, h * 64, row, bar(full + s));
          n++;
          if (is_v || i > 0) continue;
          // Q behind the first K tile, whose slot is free one S before Q's (with the last S of the run before)
          for (int t = 0; t < 2; t++) {
            if (sg.lane_tiles(t) == 0) continue;
            if (nq[t] > 0 && !wait_bar(bar(B_QE + t), (nq[t] & 1) ^ 1)) { *abort_flag = 1; break; }
            tc::mbar_arrive_expect_tx(bar(B_Q + t), p.rpt * HD * 2);
            for (int h = 0; h < S::ATOMS; h++)
              tc::tma_load_3d(tc::smem_u32(smem + S::Q) + t * S::TILE + h * ATOM_BYTES, &p.tm_q, h * 64, sg.g * p.grp,
                              sg.n0 + p.by_grp.div(sg.lane_row0(t, p.rpt)), bar(B_Q + t));
            nq[t]++;
          }
        }
      }
      if (*abort_flag) {   // a wait ran out: let the copies in flight land before the CTA's memory goes
        for (int i = max(0, n - ST); i < n; i++) tc::mbar_wait(bar(full + i % ST), (i / ST) & 1);
        for (int t = 0; t < 2; t++)
          if (nq[t] > 0) tc::mbar_wait(bar(B_Q + t), (nq[t] & 1) ^ 1);
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    {
      const uint32_t on = elect_one();
      constexpr uint32_t id_s = idesc_bf16(QR, KT, 0);   // Q x K, both K-major in shared memory
      constexpr uint32_t id_o = idesc_bf16(QR, HD, 1);   // P (tensor memory) x V (MN-major in shared memory)
      const uint64_t dq = tc::sw128_kmajor_desc(tc::smem_u32(smem + S::Q)), dk = tc::sw128_kmajor_desc(tc::smem_u32(smem + S::K));
      const uint64_t dv = sw128_mn_desc(tc::smem_u32(smem + S::V), ATOM_BYTES);
      int n0 = 0, nq[2] = {0, 0}, nl[2] = {0, 0};        // ring tiles, Q loads, lane tiles so far
      auto fail = [&]() { *abort_flag = 1; return false; };
      auto wait_k = [&](int n) { return wait_bar(bar(B_KF + n % KST), (n / KST) & 1) || fail(); };
      auto wait_v = [&](int n) { return wait_bar(bar(B_VF + n % VST), (n / VST) & 1) || fail(); };
      auto issue_s = [&](int t, int slot) {   // S_t = Q_t K^T, K from the slot
        const uint64_t da = dq + t * (S::TILE >> 4), db = dk + slot * (S::TILE >> 4);
#pragma unroll
        for (int kk = 0; kk < HD / 16; kk++) {
          const uint64_t step = ((kk >> 2) * ATOM_BYTES + (kk & 3) * 32) >> 4;   // stays inside the address field
          umma_ss_if(on, tmem + t * KT, da + step, db + step, id_s, kk > 0 ? 1u : 0u);
        }
        commit_if(on, bar(B_SF + t));
      };
      auto pv = [&](int t, int slot, uint32_t accumulate) {   // O_t (+)= (P_hi + P_lo)_t V
        if (!wait_bar(bar(B_PF + t), nl[t] & 1)) return fail();
        nl[t]++;
        tc::tc_fence_after();
        const uint64_t dvs = dv + slot * (S::TILE >> 4);
        const uint32_t pt = tmem + t * KT;
#pragma unroll
        for (int kk = 0; kk < KT / 16; kk++) {
          // keys 16 kk .. 16 kk + 15: chunk kk / 2, half kk % 2 -> hi at 32 c + 8 h, lo at 32 c + 16 + 8 h
          const uint32_t col = 32 * (kk >> 1) + 8 * (kk & 1);
          const uint64_t db = dvs + (kk * 16 * 128 >> 4);
          umma_ts_if(on, tmem + kTmemO + t * 128, pt + col, db, id_o, kk > 0 ? 1u : accumulate);
          umma_ts_if(on, tmem + kTmemO + t * 128, pt + col + 16, db, id_o, 1u);
        }
        commit_if(on, bar(B_PV + t));
        return true;
      };
      auto uni = [&](int v) { return __shfl_sync(0xffffffffu, v, 0); };
      bool ok = true;
      while (ok && !*abort_flag && walk.next(sg)) {
        const int nt = sg.n_tiles;
        if (nt == 0) continue;
        for (int t = 0; t < 2 && ok; t++) {
          if (sg.lane_tiles(t) == 0) continue;
          ok = wait_bar(bar(B_Q + t), nq[t] & 1) || fail();
          nq[t]++;
        }
        tc::tc_fence_after();
        // Between a lane's P and its product stands nothing but the wait for P: a pair's other waits are done while the tensor
        // core still has work.
        if (!sg.keys) {
          // a lane's next S follows its own product, so no lane waits for the other's softmax
          if (ok && (ok = wait_k(n0))) {
            tc::tc_fence_after();
            const int k0 = uni(n0 % KST);
            issue_s(0, k0);
            issue_s(1, k0);
            commit_if(on, bar(B_KE + k0));
          }
          if (nt == 1) {
            commit_if(on, bar(B_QE + 0));
            commit_if(on, bar(B_QE + 1));
          }
          if (ok) ok = wait_v(n0);
          for (int i = 0; i < nt && ok && !*abort_flag; i++) {
            const int n = n0 + i, vs = uni(n % VST), ks = uni((n + 1) % KST), acc = uni(i > 0);
            const bool more = i + 1 < nt;
            if (!(ok = pv(0, vs, acc))) break;
            if (more) {   // these copies started a whole tile ago
              if (!(ok = wait_k(n + 1) && wait_v(n + 1))) break;
              tc::tc_fence_after();
              issue_s(0, ks);
              if (i + 2 == nt) commit_if(on, bar(B_QE + 0));
            }
            if (!(ok = pv(1, vs, acc))) break;
            commit_if(on, bar(B_VE + vs));
            if (more) {
              issue_s(1, ks);
              commit_if(on, bar(B_KE + ks));
              if (i + 2 == nt) commit_if(on, bar(B_QE + 1));
            }
          }
        } else {
          for (int i = 0; i < min(2, nt) && ok; i++) {
            if (!(ok = wait_k(n0 + i))) break;
            tc::tc_fence_after();
            const int ks = uni((n0 + i) % KST);
            issue_s(i, ks);
            commit_if(on, bar(B_KE + ks));
            if (i + 2 >= nt) commit_if(on, bar(B_QE + i));
          }
          for (int i = 0; i < nt && ok && !*abort_flag; i++) {
            const int n = n0 + i, t = i & 1, vs = uni(n % VST), ks = uni((n + 2) % KST), acc = uni(i > 1);
            if (!(ok = wait_v(n) && pv(t, vs, acc))) break;
            commit_if(on, bar(B_VE + vs));
            if (i + 2 < nt) {
              if (!(ok = wait_k(n + 2))) break;
              tc::tc_fence_after();
              issue_s(t, ks);
              commit_if(on, bar(B_KE + ks));
              if (i + 4 >= nt) commit_if(on, bar(B_QE + t));   // the lane's last S
            }
          }
        }
        n0 += nt;
      }
      // everything issued is done before tensor memory is freed (at once, unless a wait ran out)
      commit_if(on, bar(B_END));
      tc::mbar_wait(bar(B_END), 0);
    }
  } else {
    // ---------------- softmax of lane t: thread = query row = TMEM lane ----------------
    const int t = (warp - 3) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const float sl2 = rsqrtf((float)HD) * 1.4426950408889634f;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t st = tmem + lane_off + t * KT, ot = tmem + lane_off + kTmemO + t * 128;
    // row r of the lane: index of its output row, or -1
    auto out_row = [&](const Seg& s) -> long long {
      const int qi = s.lane_row0(t, p.rpt) + r;
      const int pos = p.by_grp.div(qi);
      return r < p.rpt && qi < s.nrows ? (long long)(s.n0 + pos) * p.a.nq + s.g * p.grp + qi - pos * p.grp : -1;
    };
    int cnt = 0, other = 0, base = 0;   // tiles of this lane and of the other so far: phases of S, P and PV; of both: V slots
    while (!*abort_flag && walk.next(sg)) {
      const bool warp_rows = quarter * 32 < p.rpt && sg.lane_row0(t, p.rpt) + quarter * 32 < sg.nrows;   // else padding
      const int i0 = sg.keys ? t : 0, step = sg.keys ? 2 : 1;
      float m_ref = -INFINITY, l = 0.f;
      bool first_tile = true;
      for (int i = i0; i < sg.n_tiles && !*abort_flag; i += step, cnt++) {
        int first, valid;
        bool ctx;
        sg.tile(i, first, valid, ctx);
        if (!wait_bar(bar(B_SF + t), cnt & 1)) *abort_flag = 1;
        tc::tc_fence_after();
        if (warp_rows) {
          float sv[KT];
#pragma unroll
          for (int c = 0; c < KT; c += 32) tmem_ld32_nowait(st + c, sv + c);
#pragma unroll
          for (int c = 0; c < KT; c += 32) wait_ld32(sv + c);
          if (valid < KT) {   // a partial tile (warp-uniform)
#pragma unroll
            for (int e = 0; e < KT; e++)
              if (e >= valid) sv[e] = -INFINITY;
          }
          float mq[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
          for (int e = 4; e + 7 < KT; e += 8)
#pragma unroll
            for (int u = 0; u < 4; u++) mq[u] = max3(mq[u], sv[e + u], sv[e + 4 + u]);
#pragma unroll
          for (int u = 0; u < 4; u++) mq[u] = fmaxf(mq[u], sv[KT - 4 + u]);
          const float mx = max3(fmaxf(mq[0], mq[1]), mq[2], mq[3]) * sl2;
          const bool need = mx > m_ref + kRescaleLog2;
          if (__any_sync(0xffffffffu, need)) {   // tcgen05.ld/st are warp-wide: every lane takes part
            const float m_new = need ? mx : m_ref;
            const float cf = (m_ref == -INFINITY) ? 0.f : ex2(m_ref - m_new);
            if (!first_tile) {
              // O may only be rescaled once every product into it has finished
              if (!wait_bar(bar(B_PV + t), (cnt - 1) & 1)) *abort_flag = 1;
              tc::tc_fence_after();
#pragma unroll 1
              for (int c0 = 0; c0 < HD; c0 += 16) {
                float o[16];
                tc::tmem_ld16(ot + c0, o);
#pragma unroll
                for (int e = 0; e < 16; e++) o[e] *= cf;
                tmem_st16(ot + c0, o);
              }
            }
            l *= cf;
            m_ref = m_new;
          }
          const float nm = m_ref == -INFINITY ? 0.f : -m_ref;   // every score so far -inf: weight 0, not NaN
          const uint64_t sl22 = pack2(sl2, sl2), nm2 = pack2(nm, nm);
          uint64_t lq[2] = {0ull, 0ull};
#pragma unroll
          for (int c0 = 0; c0 < KT; c0 += 16) {
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              float x0, x1;
              unpack2(fma2(pack2(sv[c0 + e], sv[c0 + e + 1]), sl22, nm2), x0, x1);
              const float p0 = ex2(x0), p1 = ex2(x1);
              lq[(e >> 1) & 1] = add2(lq[(e >> 1) & 1], pack2(p0, p1));
              split_trunc(p0, p1, hi[e / 2], lo[e / 2]);
            }
            const uint32_t pt = st + (c0 & ~31) + (c0 & 16) / 2;   // 32 keys: 16 columns of hi, 16 of lo
            tmem_st8(pt, hi);
            tmem_st8(pt + 16, lo);
          }
          float la, lb;
          unpack2(add2(lq[0], lq[1]), la, lb);
          l += la + lb;
          tmem_wait_st();
        }
        first_tile = false;
        if (valid < KT && (sg.keys || t == 0)) {
          // V rows past the last key -> 0 before the product: 0 x a stale non-finite value would be NaN.  A pair's lane 1 comes
          // after lane 0's product.  Row k: 128 bytes at k * 128 in each 64-dim atom (the swizzle permutes within a row).
          const int n = base + i, s = n % VST;
          if (!wait_bar(bar(B_VF + s), (n / VST) & 1)) *abort_flag = 1;
          uint8_t* tile = smem + S::V + s * S::TILE;
          for (int c = r; c < (KT - valid) * 8 * S::ATOMS; c += QR) {
            const int k = valid + c / (8 * S::ATOMS), h = (c >> 3) & (S::ATOMS - 1), q = c & 7;
            *reinterpret_cast<uint4*>(tile + h * ATOM_BYTES + k * 128 + q * 16) = make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(B_PF + t));
      }
      other += sg.lane_tiles(1 - t);
      base += sg.n_tiles;
      if (!first_tile && !wait_bar(bar(B_PV + t), (cnt - 1) & 1)) *abort_flag = 1;
      // behind the last run the K and V slots are free once the other lane's products are done too: rows go through them
      // (16 bytes of padding each, so that a warp's writes spread over the banks) and out as one bulk copy per row.
      // Written directly, 32 rows at a time, a CTA's partials took 4 us instead of 2.
      const bool staged = !walk.more();
      if (staged && other > 0 && !wait_bar(bar(B_PV + 1 - t), (other - 1) & 1)) *abort_flag = 1;
      tc::tc_fence_after();
      if (warp_rows) {
        const long long orow = out_row(sg);
        const size_t n_out = (size_t)p.a.rows * p.a.nq;
        const int slot = sg.slot + (sg.keys ? t : 0);
        if (!first_tile) {
          float* dst = p.a.o_part + ((size_t)slot * n_out + (orow < 0 ? 0 : orow)) * HD;
          uint8_t* row = smem + S::K + (t * QR + r) * (HD * 4 + 16);
#pragma unroll
          for (int c0 = 0; c0 < HD; c0 += 64) {
            float o[64];
            tmem_ld32_nowait(ot + c0, o);
            tmem_ld32_nowait(ot + c0 + 32, o + 32);
            wait_ld32(o);
            wait_ld32(o + 32);
            if (staged) {
#pragma unroll
              for (int e = 0; e < 64; e += 4)
                *reinterpret_cast<float4*>(row + (c0 + e) * 4) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            } else if (orow >= 0) {
#pragma unroll
              for (int e = 0; e < 64; e += 8) st8(dst + c0 + e, o + e);
            }
          }
          if (staged && orow >= 0 && !*abort_flag) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(tc::smem_u32(row)),
                         "r"(HD * 4)
                         : "memory");
            asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group 0;" ::: "memory");
          }
        }
        if (orow >= 0) {
          p.a.ml[(size_t)slot * n_out + orow] = make_float2(m_ref, l);
          if (!sg.keys || t == 1)
            for (int s = slot + 1; s < sg.pad_end; s++) p.a.ml[(size_t)s * n_out + orow] = make_float2(-INFINITY, 0.f);
        }
      }
      tc::tc_fence_before();   // O has been read: the next run's first product follows this lane's next P
    }
  }

  __syncwarp();
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

cudaError_t shared_attn_tc_init_attributes() {
  cudaError_t e = cudaFuncSetAttribute(shared_tc_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes<128>());
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(shared_tc_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes<64>());
  return e;
}

// The parts of the call that the plan gives to the tensor cores.
cudaError_t launch_shared_tc(const SharedAttn& a, const SharedPlan& pl, cudaStream_t st) {
  TcArgs p;
  memset(&p, 0, sizeof(p));
  p.a = a;
  p.grp = a.nq / a.nkv;
  p.npt = QR / p.grp;
  p.rpt = p.npt * p.grp;
  p.own_slot0 = pl.pre_splits;
  p.by_grp.set(p.grp);
  p.by_nkv.set(a.nkv);
  if (pl.pre_tc) {
    p.pre_tiles = pl.pre_tiles;
    p.pre_units = pl.pre_tiles * a.nkv;
    p.pre_slots = pl.pre_splits;
    p.pre_runs = pl.pre_runs;
    p.pre_pieces = pl.pre_pieces;
    p.own_cost = pl.own_cost;
    p.by_pre_tiles.set(p.pre_tiles);
  }
  if (pl.own_tc) {
    p.own_tiles = pl.own_tiles;
    p.own_units = pl.own_tiles * a.nkv * a.batch;
    p.own_splits = pl.own_splits / 2;
    p.own_ctas = pl.own_ctas;
    p.own_alone = pl.own_ctas * pl.own_alone;
    p.by_own_tiles.set(p.own_tiles);
    p.by_own_units.set(p.own_units);
  }
  const uint64_t str[1] = {(uint64_t)a.h * 2};
  const uint32_t box[2] = {64u, (uint32_t)KT};
  auto map = [&](CUtensorMap* tm, const bf16* base, uint64_t rows) {
    const uint64_t dims[2] = {(uint64_t)a.h, rows};
    return make_tmap_nd(tm, base, 2, dims, str, box);
  };
  const uint64_t qd[3] = {(uint64_t)a.h, (uint64_t)a.nq, (uint64_t)a.rows}, qs[2] = {(uint64_t)a.h * 2, (uint64_t)a.h * 2 * a.nq};
  const uint32_t qb[3] = {64u, (uint32_t)p.grp, (uint32_t)p.npt};
  cudaError_t e = make_tmap_nd(&p.tm_q, a.q, 3, qd, qs, qb);
  if (p.pre_units && e == cudaSuccess) e = map(&p.tm_pre, a.pk, (uint64_t)2 * a.nkv * a.p_cap);
  if (p.own_units && a.ck && e == cudaSuccess) e = map(&p.tm_own, a.ck, (uint64_t)a.batch * 2 * a.nkv * a.t_cap);
  if (p.own_units && a.lb) {
    if (e == cudaSuccess) e = map(&p.tm_kblk, a.kblk, (uint64_t)a.batch * a.nkv * a.lb);
    if (e == cudaSuccess) e = map(&p.tm_vblk, a.vblk, (uint64_t)a.batch * a.nkv * a.lb);
  }
  if (e != cudaSuccess) return e;
  return a.h == 128 ? launch_k(shared_tc_kernel<128>, pl.tc_grid, kThreads, smem_bytes<128>(), st, p)
                    : launch_k(shared_tc_kernel<64>, pl.tc_grid, kThreads, smem_bytes<64>(), st, p);
}

}  // namespace fpd
