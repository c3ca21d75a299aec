// k_paged_tc.cu — attention over pages for many rows, on the 5th-generation tensor cores.  Formulas and cut of the work as in
// k_paged_attention.cu and paged_sched.cuh, with tiles of 128 keys.
//
// A CTA works on two "lanes", each a 128-row S / P / O set in tensor memory with a softmax warpgroup of its own (one thread per
// query row), so that one lane's softmax runs while the tensor core works for the other.  A lane's rows are whole positions, the kv
// head's heads of each.  Where a unit has more rows than a lane, it has the rows of two, which share every K/V tile; where a request
// has at most a lane's (a text block), each lane walks a run of its own, with its own tiles, warps and barriers: one's way out of a
// unit and into the next is hidden behind the other's tiles.
//
// bf16 pages: TMA, one box per page and 64 dims (a coordinate past the pool, which reads zeros, for a page that is none); P enters as
// two bf16 terms.
// 4-bit pages: warps decode tiles into the swizzled layout, K as bf16 and V as fp16 (7 bits either way, exact).  The pairs that decode
// together are dims i and i + 4 of 8, so Q is stored in that order too, and O comes out in it.  P enters as one fp16 term, p 2^7 (p
// stays below 2^8; weights down to 2^-31 count); the block's own keys are bf16 and take the bf16 products.
//
// Bound by a lane's chain, S -> softmax -> P -> product -> next S: 2.1 to 2.8 us a tile of 128 keys, 1.2 to 1.5 of them softmax (its
// instructions, at one to two softmax warps a scheduler), and for 4-bit pages by the decoding beside it (0.7 us of a team's four warps for
// K or V of a tile).  8 texts of 16 positions, contexts to 2048: 27 us; 64 texts over 4-bit pages to 4096: 121 us (0.28 PFLOP/s of the
// formula); 4 trajectories of 385 positions with a window of 1024: 74 us (0.43).
#include <cstring>

#include "attn_tc_prims.cuh"
#include "paged_decode.cuh"
#include "paged_masks.cuh"
#include "paged_sched.cuh"

namespace fpd {

namespace {
using namespace attn_tc;

constexpr int QR = 128, KT = kPagedTcTile;
constexpr int KST = 2;
template <bool INT4>
constexpr int kVst = INT4 ? 2 : 3;     // V slots; 4-bit pages leave one to the codes
constexpr int kRawSlots = 3;           // most slots of a ring of codes and scales, each a tile's K or V
constexpr int kTmemCols = 512;         // S/P of lane t at 128 t, O of lane t at 256 + 128 t
constexpr uint32_t kTmemO = 256;
constexpr float kRescaleLog2 = 8.f;
constexpr int ATOM_BYTES = KT * 64 * 2;

struct TcArgs {
  CUtensorMap tm_q, tm_pages, tm_kblk, tm_vblk;
  PagedAttn a;
  PagedShape s;
  int runs, npt, rpt, solo;   // positions and rows of a lane; whether the lanes have runs of their own
};

// A part of a unit as this kernel walks it.  One warp walks a run, a few parts ahead, and leaves what it finds in shared memory: walks
// of their own took every warp some 40 registers, spilled at each unit.
constexpr int kSegs = 4;
struct Seg {
  PagedUnit u;                              // u.b < 0: the run is over
  int whole, first;                         // first: the unit starts here
  int t0, n_tiles, row0, last_run;
  __device__ PagedTile tile(int i) const { return tile_at(u, KT, t0 + i); }
};

template <int HD, bool INT4>
struct Lay {
  static constexpr int TILE = KT * HD * 2, ATOMS = HD / 64, VST = kVst<INT4>;
  static constexpr int RAW_BYTES = KT * (HD / 2 + HD / 16);
  // 4 bits, lanes on their own: the codes begin behind the rows of Q that are there
  static constexpr int Q = 0, RAW = 2 * TILE, K = (RAW + (INT4 ? kRawSlots * RAW_BYTES : 0) + 1023) / 1024 * 1024;
  static constexpr int V = K + KST * TILE, SEG = V + VST * TILE, BAR = SEG + 2 * kSegs * (int)sizeof(Seg);
};
enum {
  B_Q = 0,
  B_QE = B_Q + 2,
  B_KF = B_QE + 2,
  B_KE = B_KF + KST,
  B_VF = B_KE + KST,
  B_VE = B_VF + 3,
  B_SF = B_VE + 3,
  B_PF = B_SF + 2,
  B_PV = B_PF + 2,
  B_END = B_PV + 2,
  B_RF = B_END + 2,    // codes: full, empty [ring][slot]
  B_RE = B_RF + 2 * kRawSlots,
  B_GF = B_RE + 2 * kRawSlots,   // parts of units: full, empty [run][slot]
  B_GE = B_GF + 2 * kSegs,
  B_N = B_GE + 2 * kSegs
};
template <int HD, bool INT4>
constexpr size_t smem_bytes() {
  return 1024 + (size_t)Lay<HD, INT4>::BAR + 8 * B_N + 16;
}
static_assert(smem_bytes<128, false>() <= 232448 && smem_bytes<128, true>() <= 232448, "tile set exceeds the shared memory of one CTA");

// Warp 1 issues the products, of both lanes or of lane 0, and warp 3 those of lane 1 on its own.  bf16: warps 0 and 2 copy, K with Q
// and V, or all of a lane; softmax from 4 on.  4 bits: warp 0 copies codes (and warp 2 those of lane 1 on its own), the others below 8
// decode, and softmax takes the scores in two halves (128 registers a thread).
template <bool INT4>
struct Roles {
  static constexpr int THREADS = INT4 ? 512 : 384, SOFTMAX = INT4 ? 8 : 4;
};

__device__ __forceinline__ void split_trunc(float a, float b, uint32_t& hi, uint32_t& lo) {   // a, b >= 0: hi + lo to 2^-16
  const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
  hi = __byte_perm(ua, ub, 0x7632);
  const uint64_t rest = add2(pack2(a, b), pack2(-__uint_as_float(ua & 0xFFFF0000u), -__uint_as_float(ub & 0xFFFF0000u)));
  float ra, rb;
  unpack2(rest, ra, rb);
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(rb), "f"(ra));
}
__device__ __forceinline__ void st8(void* dst, const uint32_t (&v)[8]) {   // 32-byte aligned
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]),
               "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
constexpr uint32_t idesc_f16(int M, int N, int b_mn) {   // fp16 A and B, fp32 accumulator
  return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }   // bits 0 .. n - 1

template <int HD, bool INT4>
__global__ void __launch_bounds__(Roles<INT4>::THREADS, 1) paged_tc_kernel(const __grid_constant__ TcArgs p) {
  using S = Lay<HD, INT4>;
  constexpr int VST = S::VST;
  using Ro = Roles<INT4>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + B_N);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t bar0 = tc::smem_u32(bars);
  auto bar = [&](int i) { return bar0 + 8 * i; };
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const PagedAttn& a = p.a;
  const PagedShape& sh = p.s;
  const int grp = sh.grp, nrows = a.L * grp;
  // 4 bits: quarters of the lanes that no unit's rows reach (a text block's 64) decode instead (64 texts, when the lanes
  // still shared a unit: 177 us without them, 168 with)
  const int live = INT4 ? (min(nrows, p.rpt) + 31) / 32 : 4;
  const bool solo = p.solo;
  const int quarter = warp & 3;
  const bool helps = INT4 && warp >= Ro::SOFTMAX && quarter >= live;
  const int own = solo ? 4 : 2;                                            // decoding warps from here to 7 beside the helpers
  const int NW = (8 - own + 2 * (4 - live)) / (solo ? 2 : 1);              // decoding warps of a team: of a lane, or all
  const int decodes = helps ? 8 - own + (warp >= Ro::SOFTMAX + 4 ? 4 - live : 0) + quarter - live : warp - own, team = solo ? decodes / NW : 0;
  // arrivals that fill a tile, and Q: from every warp of the team, or from the one that issues the copies; and that read a part
  const int fill = INT4 ? NW : 1, fill_q = INT4 ? live : 1, readers = 1 + (INT4 ? NW : solo ? 0 : 1) + (solo ? 1 : 2) * live;

  if (tid == 0) {
    for (int t = 0; t < 2; t++) {
      tc::mbar_init(bar(B_Q + t), fill_q);
      tc::mbar_init(bar(B_QE + t), 1);
      tc::mbar_init(bar(B_SF + t), 1);
      tc::mbar_init(bar(B_PF + t), live);
      tc::mbar_init(bar(B_PV + t), 1);
    }
    for (int s = 0; s < KST; s++) {
      tc::mbar_init(bar(B_KF + s), fill);
      tc::mbar_init(bar(B_KE + s), 1);
    }
    for (int s = 0; s < VST; s++) {
      tc::mbar_init(bar(B_VF + s), fill);
      tc::mbar_init(bar(B_VE + s), 1);
    }
    for (int s = 0; s < 2 * kRawSlots; s++) {
      tc::mbar_init(bar(B_RF + s), 1);
      tc::mbar_init(bar(B_RE + s), NW);
    }
    for (int s = 0; s < 2 * kSegs; s++) {
      tc::mbar_init(bar(B_GF + s), 1);
      tc::mbar_init(bar(B_GE + s), readers);
    }
    for (int t = 0; t < 2; t++) tc::mbar_init(bar(B_END + t), 1);
    *abort_flag = 0;
    tc::fence_barrier_init();
    if (!INT4) {
      tc::tma_prefetch(&p.tm_q);
      tc::tma_prefetch(&p.tm_pages);
      if (a.lb) {
        tc::tma_prefetch(&p.tm_kblk);
        tc::tma_prefetch(&p.tm_vblk);
      }
    }
  }
  if (warp == 1) {
    tc::tmem_alloc(tc::smem_u32(tmem_slot), kTmemCols);
    tc::tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();
  const DeviceLens lens{a.ctx_len, a.pg.cap()};
  const bool walks = warp == 0 || (solo && warp == 2);
  PagedWalk<DeviceLens> walk =
      walks ? make_walk(sh, lens, a.batch, p.runs, solo ? 2 * blockIdx.x + warp / 2 : blockIdx.x) : PagedWalk<DeviceLens>(sh, lens, a.batch, 1, 1, 1);
  __syncwarp();   // a CTA barrier counts a whole warp: single-lane roles reconverge before every one
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  // the run of the warp: lane 1's on its own, or else the CTA's
  const bool softmaxes = warp >= Ro::SOFTMAX && !helps;
  const int ln = !solo ? 0 : softmaxes ? (warp - Ro::SOFTMAX) >> 2 : warp < 4 ? warp >> 1 : team;
  Seg* const segs = reinterpret_cast<Seg*>(smem + S::SEG) + ln * kSegs;
  const int b_gf = B_GF + ln * kSegs, b_ge = B_GE + ln * kSegs;
  const Seg* sg = segs;
  int n_seg = 0;
  auto walk_next = [&]() {
    const int s = n_seg % kSegs;
    Seg w;
    int t1;
    if (walk.next(w.u, w.t0, t1, w.last_run)) {
      w.whole = w.t0 == 0 && t1 == w.u.len();
      w.first = w.t0 == 0;
      w.n_tiles = max(0, min(t1, w.u.tiles()) - w.t0);   // an empty unit has none
      w.row0 = w.u.rt * sh.rows;
    } else {
      w.u.b = -1;
    }
    if (n_seg >= kSegs && !wait_bar(bar(b_ge + s), ((n_seg / kSegs) & 1) ^ 1)) *abort_flag = 1;
    __syncwarp();
    if (lane == 0) {
      segs[s] = w;
      tc::mbar_arrive(bar(b_gf + s));
    }
    __syncwarp();
    sg = segs + s;
    n_seg++;
    return w.u.b >= 0;
  };
  auto next = [&]() {   // the others: done with the part before
    __syncwarp();
    if (n_seg > 0 && lane == 0) tc::mbar_arrive(bar(b_ge + (n_seg - 1) % kSegs));
    if (!wait_bar(bar(b_gf + n_seg % kSegs), (n_seg / kSegs) & 1)) *abort_flag = 1;
    sg = segs + n_seg % kSegs;
    n_seg++;
    return !*abort_flag && sg->u.b >= 0;
  };

  // 4 bits: Q of a lane on its own takes the rows that there are, and the codes' rings what that leaves
  const int q_atom = INT4 && solo ? live * 32 * 128 : ATOM_BYTES, q_bytes = S::ATOMS * q_atom;
  auto q_at = [&](int l) { return tc::smem_u32(smem + S::Q) + l * q_bytes; };
  const int raw_slots = solo && live == 3 ? 2 : kRawSlots;
  const uint32_t raws = tc::smem_u32(smem) + (solo ? 2 * q_bytes + ln * raw_slots * S::RAW_BYTES : S::RAW);
  const int b_rf = B_RF + ln * kRawSlots, b_re = B_RE + ln * kRawSlots;

  auto drain = [&](int first, int copies, int slots) {   // the copies into a ring that may still be in flight
    for (int i = max(0, copies - slots); i < copies; i++) tc::mbar_wait(bar(first + i % slots), (i / slots) & 1);
  };

  if (!INT4 && (warp == 0 || warp == 2)) {
    // ---------------- TMA producers: K and Q (warp 0) and V (warp 2), or all of a lane; lane i copies a tile's page i ----------------
    const int bp = min(KT, a.pg.page);   // rows of a box
    int n = 0, copied[2] = {0, 0}, nq[2] = {0, 0};   // tiles; copies of K and V; loads of Q
    auto page_for = [&](int i) {   // of this lane's part of tile i
      if (i >= sg->n_tiles) return 0;
      const PagedTile t = sg->tile(i);
      return t.ctx && lane * bp < t.valid ? page_of(a.pg, sg->u.b, t.k0 + lane * bp) : 0;
    };
    bool ok = true;
    while (ok && !*abort_flag && (walks ? walk_next() : next())) {
      int id = page_for(0);
      for (int i = 0; i < sg->n_tiles && ok; i++, n++) {
        const PagedTile t = sg->tile(i);
        const int id_now = id;
        id = page_for(i + 1);
        for (int is_v = !solo && warp == 2; is_v < (!solo && warp == 0 ? 1 : 2); is_v++) {
          const int ST = is_v ? VST : KST, round = solo ? n : n / ST, s = solo ? ln : n - round * ST, full = (is_v ? B_VF : B_KF) + s;
          if (round > 0) ok = wait_bar(bar((is_v ? B_VE : B_KE) + s), (round & 1) ^ 1);
          ok = __all_sync(0xffffffffu, ok && !*abort_flag);
          if (!ok) break;
          const bool mine = t.ctx ? lane * bp < t.valid : lane == 0;
          const int boxes = __popc(__ballot_sync(0xffffffffu, mine));
          if (lane == 0) tc::mbar_arrive_expect_tx(bar(full), t.ctx ? boxes * bp * HD * 2 : S::TILE);
          __syncwarp();
          if (mine) {
            for (int h = 0; h < S::ATOMS; h++) {
              const uint32_t dst = tc::smem_u32(smem + (is_v ? S::V : S::K)) + s * S::TILE + h * ATOM_BYTES;
              if (t.ctx)
                tc::tma_load_3d(dst + lane * bp * 128, &p.tm_pages, h * 64,
                                ((is_v ? a.pg.nkv : 0) + sg->u.g) * a.pg.page + ((t.k0 + lane * bp) & (a.pg.page - 1)),
                                id_now < 0 ? a.pg.n_pages : id_now, bar(full));
              else
                tc::tma_load_2d(dst, is_v ? &p.tm_vblk : &p.tm_kblk, h * 64, (sg->u.b * a.pg.nkv + sg->u.g) * a.lb + t.k0, bar(full));
            }
          }
          copied[is_v]++;
          if (is_v || i > 0) continue;
          // Q behind the first K tile, whose slot is free one S before Q's (with the last S of the part before)
          for (int l = ln; l < (solo ? ln + 1 : 2) && ok; l++) {
            if (nq[l] > 0) ok = wait_bar(bar(B_QE + l), (nq[l] & 1) ^ 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 0) {
              tc::mbar_arrive_expect_tx(bar(B_Q + l), p.rpt * HD * 2);
              for (int h = 0; h < S::ATOMS; h++)
                tc::tma_load_3d(tc::smem_u32(smem + S::Q) + l * S::TILE + h * ATOM_BYTES, &p.tm_q, h * 64, sg->u.g * grp,
                                sg->u.b * a.L + (sg->row0 + (solo ? 0 : l * p.rpt)) / grp, bar(B_Q + l));
            }
            nq[l]++;
          }
          if (!ok) break;
        }
      }
    }
    if (!ok) *abort_flag = 1;
    if (*abort_flag) {   // a wait ran out: let the copies in flight land before the CTA's memory goes
      drain(B_KF + ln, copied[0], solo ? 1 : KST);
      drain(B_VF + ln, copied[1], solo ? 1 : VST);
      for (int l = 0; l < 2; l++) drain(B_Q + l, nq[l], 1);
    }
  } else if (INT4 && walks) {
    // ---------------- codes of the context tiles, K and V in turn, by bulk copies: lanes 2 i + part copy from page i ----------------
    const int kp = min(KT, a.pg.page), part = lane & 1, pi = lane >> 1;   // part: codes, scales
    const uint32_t w = part ? HD / 16 : HD / 2;
    int h = 0;   // halves of tiles so far
    bool ok = true;
    auto page_for = [&](int i) {
      if (i >= sg->n_tiles || pi >= KT / 16) return 0;
      const PagedTile t = sg->tile(i);
      return t.ctx && pi * kp < t.valid ? page_of(a.pg, sg->u.b, t.k0 + pi * kp) : 0;
    };
    while (ok && !*abort_flag && walk_next()) {
      int id = page_for(0);
#pragma unroll 1
      for (int i = 0; i < sg->n_tiles && ok; i++) {
        const PagedTile t = sg->tile(i);
        if (!t.ctx) break;
        const int id_now = id, in = t.k0 & (a.pg.page - 1);
        id = page_for(i + 1);
        const int rows = pi < KT / 16 ? min(kp, ceil_div(t.valid, 16) * 16 - pi * kp) : 0;   // whole groups of 16 positions
        const uint32_t bytes = rows > 0 && id_now >= 0 ? rows * w : 0, total = __reduce_add_sync(0xffffffffu, bytes);
        const uint32_t at = (part ? KT * (HD / 2) : 0) + pi * kp * w;
#pragma unroll 1
        for (int v = 0; v < 2; v++, h++) {
          const int round = h / raw_slots, s = h - round * raw_slots, full = b_rf + s;
          if (round > 0) ok = wait_bar(bar(b_re + s), (round & 1) ^ 1);
          ok = __all_sync(0xffffffffu, ok && !*abort_flag);
          if (!ok) break;
          if (rows > 0 && id_now < 0) {   // a page that is none: zeros
            for (uint32_t j = 0; j < rows * w; j += 16)
              asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(raws + s * S::RAW_BYTES + at + j), "r"(0) : "memory");
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive_expect_tx(bar(full), total);
          __syncwarp();
          if (bytes)
            tc::bulk_load(raws + s * S::RAW_BYTES + at, slab_of(a.pg, id_now, v, sg->u.g) + (part ? a.pg.page * (HD / 2) : 0) + in * w, bytes,
                          bar(full));
        }
      }
    }
    if (!ok) *abort_flag = 1;
    if (*abort_flag) drain(b_rf, h, raw_slots);
  } else if (INT4 && ((warp < Ro::SOFTMAX && warp >= own) || helps)) {
    // ---------------- decoding warps ----------------
    // A tile's K or V is HD / 8 items, each 32 rows by 32 dims of every row; a team's warps take turns at them, a thread a row.  One
    // copy of the code for all: unrolled, a third of the stalls were for instructions.
    const int wd = solo ? decodes - team * NW : decodes;
    if (helps && lane == 0) a.spoilt[blockIdx.x * 8 + warp - Ro::SOFTMAX] = 0;
    const uint32_t ks = tc::smem_u32(smem + S::K), vs = tc::smem_u32(smem + S::V);
    int n = 0, nh = 0, nq = 0;   // tiles, halves of context tiles and Q loads so far
    // chunk of 8 dims ch of row r in a tile of 64-dim atoms
    auto put = [&](uint32_t row, int ch, uint4 v, int atom = ATOM_BYTES) {
      asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"((row ^ ((ch & 7) << 4)) + (ch >> 3) * atom), "r"(v.x), "r"(v.y),
                   "r"(v.z), "r"(v.w)
                   : "memory");
    };
    auto row_at = [&](uint32_t tile, int r) { return tile + r * 128 + ((r & 7) << 4); };   // its chunk 0; chunk c at c ^ (r & 7)
    // 32 bf16 rows from row r0 of a tile on, in the order of the decoded ones; from(r): a row's address, null for zeros.  A warp's load
    // has whole rows.
    auto put_bf16 = [&](uint32_t tile, int r0, int atom, auto from) {
      constexpr int PER = HD / 8, RPL = 32 / PER;   // chunks of a row, rows of a load
      const int ch = lane % PER, r_in = lane / PER;
#pragma unroll 1
      for (int i0 = 0; i0 < 32 / RPL; i0 += 8) {
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; i++) {
          const bf16* row = from(r0 + (i0 + i) * RPL + r_in);
          v[i] = row ? __ldg(reinterpret_cast<const uint4*>(row) + ch) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 8; i++)
          put(row_at(tile, r0 + (i0 + i) * RPL + r_in), ch, make_uint4(__byte_perm(v[i].x, v[i].z, 0x5410), __byte_perm(v[i].x, v[i].z, 0x7632),
                                                                       __byte_perm(v[i].y, v[i].w, 0x5410), __byte_perm(v[i].y, v[i].w, 0x7632)), atom);
      }
    };
    // 32 dims of row r of the codes in a slot (past `valid`: zeros) into row r of a tile: the j-th of the row's HD / 32 chunks of 16
    // bytes, counted from one that differs between rows, so that neither a load nor a store of 8 rows has a bank twice
    auto put_codes = [&](uint32_t tile, uint32_t raw, int r, int j, bool valid, bool is_v) {
      constexpr int CH = HD / 32;
      const int ch = (j + (HD == 128 ? r >> 1 : r >> 2)) & (CH - 1);
      uint32_t c[4], two_scales;
      asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3]) : "r"(raw + r * (HD / 2) + ch * 16));
      asm volatile("{\n .reg .u16 x;\n ld.shared.u16 x, [%1];\n cvt.u32.u16 %0, x;\n}" : "=r"(two_scales) : "r"(raw + KT * (HD / 2) + r * (HD / 16) + ch * 2));
      if (!valid) two_scales = 0;   // what is stale stands for nothing
      const uint32_t half = (row_at(tile, r) ^ ((ch & 1) << 6)) + (ch >> 1) * ATOM_BYTES;   // chunks 4 ch ..
      uint32_t x[4][4];
      if (is_v) {
        const Scale2 s0((two_scales & 0xFF) * 0x00800080u), s1((two_scales >> 8) * 0x00800080u);
        decode4(c[0], s0, x[0]);
        decode4(c[1], s0, x[1]);
        decode4(c[2], s1, x[2]);
        decode4(c[3], s1, x[3]);
      } else {
        const Scale2Bf s0(two_scales & 0xFF), s1(two_scales >> 8);
        decode4_bf16(c[0], s0, x[0]);
        decode4_bf16(c[1], s0, x[1]);
        decode4_bf16(c[2], s1, x[2]);
        decode4_bf16(c[3], s1, x[3]);
      }
#pragma unroll
      for (int i = 0; i < 4; i++) put(half, i, make_uint4(x[i][0], x[i][1], x[i][2], x[i][3]));
    };
    auto done = [&](int b) {   // this warp's rows are written, for the tensor core to read
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar(b));
    };
    bool ok = true;
    auto wait = [&](int b, uint32_t parity) {
      ok = __all_sync(0xffffffffu, wait_bar(bar(b), parity));
      return ok;
    };
    while (ok && !*abort_flag && next()) {
      const size_t blk = ((size_t)sg->u.b * a.pg.nkv + sg->u.g) * a.lb;
      if (sg->n_tiles > 0) {   // Q beside the first K tile: an item for 32 rows, from the second warp on
        const int lanes = solo ? 1 : 2;
        for (int i = 0; i < lanes * live && ok; i++) {
          const int l = i < live ? ln : 1, k = i < live ? i : i - live;
          if ((i + 1) % NW != wd) continue;
          if (nq > 0 && !wait(B_QE + l, (nq & 1) ^ 1)) break;
          const int q0 = sg->row0 + (solo ? 0 : l * p.rpt);
          put_bf16(q_at(l), k * 32, q_atom, [&](int r) -> const bf16* {
            const int qi = q0 + r, j = sh.by_grp.div(qi);
            return r < p.rpt && qi < nrows ? a.q + ((size_t)(sg->u.b * a.L + j) * a.nq + sg->u.g * grp + qi - j * grp) * HD : nullptr;
          });
          done(B_Q + l);
        }
        nq++;
      }
      // Whether or not it has an item, a warp waits for all slots and codes of its team, and its arrival fills and frees them: a wait
      // on a parity must begin neither two phases early nor two late.
#pragma unroll 1
      for (int i = 0, nt = sg->n_tiles; i < nt && ok && !*abort_flag; i++, n++) {
        const PagedTile t = sg->tile(i);
#pragma unroll 1
        for (int is_v = 0; is_v < 2 && ok; is_v++) {
          const int slots = is_v ? VST : KST, round = solo ? n : n / slots, s = solo ? ln : n - round * slots;
          if (round > 0 && !wait((is_v ? B_VE : B_KE) + s, (round & 1) ^ 1)) break;
          const uint32_t tile = (is_v ? vs : ks) + s * S::TILE;
          if (t.ctx) {
            const int turn = nh / raw_slots, slot = nh - turn * raw_slots;
            if (!wait(b_rf + slot, turn & 1)) break;
            nh++;
#pragma unroll 1
            for (int item = wd; item < HD / 8; item += NW) {
              const int r = 32 * (item & 3) + lane;
              put_codes(tile, raws + slot * S::RAW_BYTES, r, item >> 2, r < t.valid, is_v);
            }
            done((is_v ? B_VF : B_KF) + s);
            if (lane == 0) tc::mbar_arrive(bar(b_re + slot));
          } else {
            const bf16* first = (is_v ? a.vblk : a.kblk) + (blk + t.k0) * HD;
#pragma unroll 1
            for (int k = wd; k < 4; k += NW) put_bf16(tile, 32 * k, ATOM_BYTES, [&](int r) { return r < t.valid ? first + (size_t)r * HD : nullptr; });
            done((is_v ? B_VF : B_KF) + s);
          }
        }
      }
    }
    if (!ok) *abort_flag = 1;
  } else if (warp == 1 || (solo && warp == 3)) {
    // ---------------- MMA issuer ----------------
    const uint32_t on = elect_one();
    constexpr uint32_t id_s = idesc_bf16(QR, KT, 0);   // Q x K, both K-major in shared memory
    constexpr uint32_t id_o = idesc_bf16(QR, HD, 1);   // P (tensor memory) x V (MN-major in shared memory)
    constexpr uint32_t id_h = idesc_f16(QR, HD, 1);
    const uint64_t dk = tc::sw128_kmajor_desc(tc::smem_u32(smem + S::K)), dv = sw128_mn_desc(tc::smem_u32(smem + S::V), ATOM_BYTES);
    int n0 = 0, nq = 0, nl[2] = {0, 0};        // ring tiles, Q loads, lane tiles so far
    auto uni = [&](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    auto fail = [&]() { *abort_flag = 1; return false; };
    auto wait_k = [&](int n) { return (solo ? wait_bar(bar(B_KF + ln), n & 1) : wait_bar(bar(B_KF + n % KST), (n / KST) & 1)) || fail(); };
    auto wait_v = [&](int n) { return (solo ? wait_bar(bar(B_VF + ln), n & 1) : wait_bar(bar(B_VF + n % VST), (n / VST) & 1)) || fail(); };
    auto issue_s = [&](int t, int slot) {   // S_t = Q_t K^T, K from the slot
      const uint64_t da = tc::sw128_kmajor_desc(q_at(t)), db = dk + slot * (S::TILE >> 4);
#pragma unroll
      for (int kk = 0; kk < HD / 16; kk++) {
        const uint32_t in = (kk & 3) * 32;   // sums stay inside the address field
        umma_ss_if(on, tmem + t * KT, da + (((kk >> 2) * q_atom + in) >> 4), db + (((kk >> 2) * ATOM_BYTES + in) >> 4), id_s, kk > 0 ? 1u : 0u);
      }
      commit_if(on, bar(B_SF + t));
    };
    auto pv = [&](int t, int slot, uint32_t accumulate, bool half) {   // O_t (+)= P_t V
      if (!wait_bar(bar(B_PF + t), nl[t] & 1)) return fail();
      nl[t]++;
      tc::tc_fence_after();
      const uint64_t dvs = dv + slot * (S::TILE >> 4);
      const uint32_t pt = tmem + t * KT;
      if (INT4 && half) {   // one fp16 term: keys 16 kk .. in columns 8 kk ..
#pragma unroll
        for (int kk = 0; kk < KT / 16; kk++)
          umma_ts_if(on, tmem + kTmemO + t * 128, pt + 8 * kk, dvs + (kk * 16 * 128 >> 4), id_h, kk > 0 ? 1u : accumulate);
      } else {
#pragma unroll
        for (int kk = 0; kk < KT / 16; kk++) {
          // keys 16 kk .. 16 kk + 15: chunk kk / 2, half kk % 2 -> hi at 32 c + 8 h, lo at 32 c + 16 + 8 h
          const uint32_t col = 32 * (kk >> 1) + 8 * (kk & 1);
          const uint64_t db = dvs + (kk * 16 * 128 >> 4);
          umma_ts_if(on, tmem + kTmemO + t * 128, pt + col, db, id_o, kk > 0 ? 1u : accumulate);
          umma_ts_if(on, tmem + kTmemO + t * 128, pt + col + 16, db, id_o, 1u);
        }
      }
      commit_if(on, bar(B_PV + t));
      return true;
    };
    bool ok = true;
    while (ok && !*abort_flag && next()) {
      const int nt = sg->n_tiles;
      if (nt == 0) continue;
      for (int l = ln; l < (solo ? ln + 1 : 2) && ok; l++) ok = wait_bar(bar(B_Q + l), nq & 1) || fail();
      nq++;
      tc::tc_fence_after();
      const int nc = sg->u.ns + sg->u.nm - sg->t0;   // tiles of the pages; the block's follow
      // Between a lane's P and its product stands nothing but the wait for P: a pair's other waits are done while the tensor
      // core still has work.
      if (!solo) {
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
          const bool more = i + 1 < nt, half = i < nc;
          if (!(ok = pv(0, vs, acc, half))) break;
          if (more) {   // these copies started a whole tile ago
            if (!(ok = wait_k(n + 1) && wait_v(n + 1))) break;
            tc::tc_fence_after();
            issue_s(0, ks);
            if (i + 2 == nt) commit_if(on, bar(B_QE + 0));
          }
          if (!(ok = pv(1, vs, acc, half))) break;
          commit_if(on, bar(B_VE + vs));
          if (more) {
            issue_s(1, ks);
            commit_if(on, bar(B_KE + ks));
            if (i + 2 == nt) commit_if(on, bar(B_QE + 1));
          }
        }
      } else {
        for (int i = 0; i <= nt && ok && !*abort_flag; i++) {   // S of tile i behind the product of tile i - 1
          if (i > 0) {
            const int vs = uni(ln), acc = uni(i > 1);
            if (!(ok = wait_v(n0 + i - 1) && pv(ln, vs, acc, i - 1 < nc))) break;
            commit_if(on, bar(B_VE + ln));
          }
          if (i == nt) break;
          if (!(ok = wait_k(n0 + i))) break;
          tc::tc_fence_after();
          issue_s(ln, uni(ln));
          commit_if(on, bar(B_KE + ln));
          if (i + 1 == nt) commit_if(on, bar(B_QE + ln));
        }
      }
      n0 += nt;
    }
    // everything issued is done before tensor memory is freed (at once, unless a wait ran out)
    commit_if(on, bar(B_END + ln));
    tc::mbar_wait(bar(B_END + ln), 0);
  } else if (softmaxes) {
    // ---------------- softmax of lane t: thread = query row = TMEM lane ----------------
    const int t = (warp - Ro::SOFTMAX) >> 2, r = quarter * 32 + lane;
    const float sl2 = rsqrtf((float)HD) * 1.4426950408889634f;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t st = tmem + lane_off + t * KT, o_mine = tmem + lane_off + kTmemO + t * 128;
    const int run = solo ? 2 * blockIdx.x + t : blockIdx.x;
    const bool speaks = quarter == 0 && (solo || t == 0) && lane == 0;
    if (speaks) a.desc[run] = make_int4(-1, 0, 0, 0);
    unsigned spoilt_units = 0;   // parts of the run, from 31 on together, that came out whole and with something that is no number
    int n_units = 0;
    int cnt = 0;   // tiles so far: phases of S, P and PV
    while (!*abort_flag && next()) {
      const int lrow0 = sg->row0 + (solo ? 0 : t * p.rpt);
      const bool warp_rows = quarter * 32 < p.rpt && lrow0 + quarter * 32 < nrows;   // else padding
      const int row_pos = sg->u.n - a.L + sh.by_grp.div(lrow0 + r);
      float m_ref = -INFINITY, l = 0.f;
      bool first_tile = true;
      for (int i = 0; i < sg->n_tiles && !*abort_flag; i++, cnt++) {
        const PagedTile tl = sg->tile(i);
        const bool half = INT4 && tl.ctx;   // P as one fp16 term
        if (!wait_bar(bar(B_SF + t), cnt & 1)) *abort_flag = 1;
        tc::tc_fence_after();
        if (warp_rows) {
          constexpr int W = KT / 2;   // scores held at a time (all 128: spills, 90 against 78 us for windows at four trajectories)
          float sv[W];
          uint32_t see[KT / 32];   // keys before `hi` that lie before `lo_end` or from `start` on, as bits
          const bool full = tile_full(sh, sg->u, tl);
          if (!full) {
            const int hi = sh.causal ? min(tl.valid, row_pos - tl.pos + 1) : tl.valid;
            const int lo_end = sh.window ? sh.sinks - tl.pos : KT, start = sh.window ? row_pos - sh.window + 1 - tl.pos : 0;
#pragma unroll
            for (int w = 0; w < KT / 32; w++) see[w] = below(hi - 32 * w) & (below(lo_end - 32 * w) | ~below(start - 32 * w));
          }
          auto load = [&](int k0) {
#pragma unroll
            for (int c = 0; c < W; c += 32) tmem_ld32_nowait(st + k0 + c, sv + c);
#pragma unroll
            for (int c = 0; c < W; c += 32) wait_ld32(sv + c);
            if (!full) {
#pragma unroll
              for (int w = 0; w < W / 32; w++) {
                const uint32_t bits = W == KT || k0 == 0 ? see[w] : see[KT / 32 - W / 32 + w];
#pragma unroll
                for (int e = 0; e < 32; e++) sv[32 * w + e] = (bits >> e) & 1 ? sv[32 * w + e] : -INFINITY;
              }
            }
          };
          uint64_t lq[2] = {0ull, 0ull};
#pragma unroll 1
          for (int k0 = 0; k0 < (tl.valid > W ? KT : W); k0 += W) {
            load(k0);
            float mq[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
            for (int e = 4; e + 7 < W; e += 8)
#pragma unroll
              for (int u = 0; u < 4; u++) mq[u] = max3(mq[u], sv[e + u], sv[e + 4 + u]);
#pragma unroll
            for (int u = 0; u < 4; u++) mq[u] = fmaxf(mq[u], sv[W - 4 + u]);
            const float mx = max3(fmaxf(mq[0], mq[1]), mq[2], mq[3]) * sl2;
            const bool need = mx > m_ref + kRescaleLog2;
            if (__any_sync(0xffffffffu, need)) {   // tcgen05.ld/st are warp-wide: every lane takes part
              // by a power of two where there is something to bring along: exact, for the weights of the first half too
              const float m_new = !need ? m_ref : m_ref == -INFINITY ? mx : m_ref + ceilf(mx - m_ref);
              const float cf = (m_ref == -INFINITY) ? 0.f : ex2(m_ref - m_new);
              if (!first_tile) {
                // O may only be rescaled once every product into it has finished
                if (!wait_bar(bar(B_PV + t), (cnt - 1) & 1)) *abort_flag = 1;
                tc::tc_fence_after();
#pragma unroll 1
                for (int c0 = 0; c0 < HD; c0 += 16) {
                  float o[16];
                  tc::tmem_ld16(o_mine + c0, o);
#pragma unroll
                  for (int e = 0; e < 16; e++) o[e] *= cf;
                  tmem_st16(o_mine + c0, o);
                }
              }
              if (k0 > 0) {   // weights already written: pairs of fp16, or of bf16
                float la, lb;
                unpack2(lq[0], la, lb);
                lq[0] = pack2(la * cf, lb * cf);
                unpack2(lq[1], la, lb);
                lq[1] = pack2(la * cf, lb * cf);
                uint32_t by = pack_f16(cf, cf);   // rounded, the power of two itself
                if (!half) asm("cvt.rn.bf16x2.f32 %0, %1, %1;" : "=r"(by) : "f"(cf));
#pragma unroll 1
                for (int c0 = 0; c0 < (half ? k0 / 2 : k0); c0 += 16) {
                  float w[16];
                  tmem_wait_st();
                  tc::tmem_ld16(st + c0, w);
                  uint32_t v[16];
#pragma unroll
                  for (int e = 0; e < 16; e++) {
                    const uint32_t x = __float_as_uint(w[e]);
                    v[e] = half ? hmul2(x, by) : mul_bf16x2(x, by);
                  }
                  tmem_st16(st + c0, v);
                }
              }
              l *= cf;
              m_ref = m_new;
            }
            // every score so far -inf: weight 0, not NaN.  fp16 weights are p 2^7, and V has 2^-7
            const float nm = m_ref == -INFINITY ? 0.f : (half ? 7.f : 0.f) - m_ref;
            const uint64_t sl22 = pack2(sl2, sl2), nm2 = pack2(nm, nm);
            if (half) {
#pragma unroll
              for (int c0 = 0; c0 < W; c0 += 16) {
                uint32_t hi[8];
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                  float x0, x1;
                  unpack2(fma2(pack2(sv[c0 + e], sv[c0 + e + 1]), sl22, nm2), x0, x1);
                  const float p0 = ex2(x0), p1 = ex2(x1);
                  lq[(e >> 1) & 1] = add2(lq[(e >> 1) & 1], pack2(p0, p1));
                  hi[e / 2] = pack_f16(p0, p1);
                }
                tmem_st8(st + (k0 + c0) / 2, hi);
              }
            } else {
#pragma unroll
              for (int c0 = 0; c0 < W; c0 += 16) {
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                  float x0, x1;
                  unpack2(fma2(pack2(sv[c0 + e], sv[c0 + e + 1]), sl22, nm2), x0, x1);
                  const float p0 = ex2(x0), p1 = ex2(x1);
                  lq[(e >> 1) & 1] = add2(lq[(e >> 1) & 1], pack2(p0, p1));
                  split_trunc(p0, p1, hi[e / 2], lo[e / 2]);
                }
                const uint32_t pt = st + k0 + (c0 & ~31) + (c0 & 16) / 2;   // 32 keys: 16 columns of hi, 16 of lo
                tmem_st8(pt, hi);
                tmem_st8(pt + 16, lo);
              }
            }
          }
          if (tl.valid <= W) {   // no key in the second half
            const uint32_t zero[16] = {};
            const int from = half ? W / 2 : W;
#pragma unroll
            for (int c = 0; c < W; c += 16)
              if (c < from) tmem_st16(st + from + c, zero);
          }
          float la, lb;
          unpack2(add2(lq[0], lq[1]), la, lb);
          l += half ? (la + lb) * 0.0078125f : la + lb;
          tmem_wait_st();
        }
        first_tile = false;
        int h_lo, h_hi;
        hidden_from_all(sh, sg->u, tl, h_lo, h_hi);
        if (!INT4 && (tl.valid < KT || h_hi > h_lo) && (solo || t == 0)) {
          // V rows past the last key, and those that no row sees -> 0 before the product: 0 x a value that is not finite would be
          // NaN.  A pair's lane 1 comes after lane 0's product.  Row k: 128 bytes at k * 128 in each 64-dim atom (the swizzle
          // permutes within a row).
          const int round = solo ? cnt : cnt / VST, s = solo ? t : cnt - round * VST;
          if (!wait_bar(bar(B_VF + s), round & 1)) *abort_flag = 1;
          uint8_t* tile = smem + S::V + s * S::TILE;
          const int rows = KT - tl.valid + h_hi - h_lo;
          for (int c = r; c < rows * 8 * S::ATOMS; c += QR) {
            const int z = c / (8 * S::ATOMS), k = z < h_hi - h_lo ? h_lo + z : tl.valid + z - (h_hi - h_lo);
            const int h = (c >> 3) & (S::ATOMS - 1), q = c & 7;
            *reinterpret_cast<uint4*>(tile + h * ATOM_BYTES + k * 128 + q * 16) = make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(B_PF + t));
      }
      if (!first_tile && !wait_bar(bar(B_PV + t), (cnt - 1) & 1)) *abort_flag = 1;
      tc::tc_fence_after();
      if (warp_rows) {
        const bool has = r < p.rpt && lrow0 + r < nrows, none = l == 0.f;
        const int qi = lrow0 + r;
        const int j = sh.by_grp.div(qi);
        const size_t orow = has ? (size_t)(sg->u.b * a.L + j) * a.nq + sg->u.g * grp + qi - j * grp : 0;
        const size_t prow = (size_t)(2 * run + sg->first) * sh.rows + (solo ? r : t * p.rpt + r);
        const float by = sg->whole ? (none ? 0.f : 1.f / l) : 1.f;
        bool spoilt = false;
        // 16 dims at a time, in a loop that stays short: unrolled, its code took longer to fetch than to run
#pragma unroll 1
        for (int c0 = 0; c0 < HD; c0 += 16) {
          float o[16];
          if (sg->n_tiles > 0) {
            tmem_ld16_nowait(o_mine + c0, o);
            wait_ld16(o);
          }
#pragma unroll
          for (int e = 0; e < 16; e++) {
            o[e] = none ? 0.f : o[e] * by;
            spoilt |= !(fabsf(o[e]) < INFINITY);
          }
          if (!has) continue;
          // dim e of 8 in its place: 4-bit pages leave the dims in the order 0 4 1 5 2 6 3 7
          auto dim = [&](int e) { return INT4 ? o[(e & ~7) + ((e & 3) << 1) + ((e >> 2) & 1)] : o[e]; };
          if (sg->whole) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; i++) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(dim(2 * i + 1)), "f"(dim(2 * i)));
            st8(a.out + orow * HD + c0, w);
          } else {
#pragma unroll
            for (int h = 0; h < 16; h += 8) {
              uint32_t w[8];
#pragma unroll
              for (int i = 0; i < 8; i++) w[i] = __float_as_uint(dim(h + i));
              st8(a.o_part + prow * HD + c0 + h, w);
            }
          }
        }
        if (sg->whole && has && spoilt) spoilt_units |= 1u << min(n_units, 31);
        if (has) {
          if (!sg->whole) a.ml[prow] = make_float2(m_ref, l);
          else if (a.lse) a.lse[orow] = none ? -INFINITY : (m_ref + log2f(l)) * 0.69314718055994531f;
        }
      }
      if (speaks && sg->first && !sg->whole) a.desc[run] = make_int4(sg->u.b, sg->u.g, sg->u.rt, sg->last_run);   // left to others
      tc::tc_fence_before();   // O has been read: the next run's first product follows this lane's next P
      n_units++;
    }
    spoilt_units = __reduce_or_sync(0xffffffffu, spoilt_units);
    if (lane == 0) a.spoilt[blockIdx.x * 8 + warp - Ro::SOFTMAX] = spoilt_units;
  }

  __syncwarp();
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

template <int HD, bool INT4>
cudaError_t attribute() {
  return cudaFuncSetAttribute(paged_tc_kernel<HD, INT4>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes<HD, INT4>());
}

}  // namespace

cudaError_t paged_tc_init_attributes() {
  cudaError_t e = attribute<128, false>();
  if (e == cudaSuccess) e = attribute<128, true>();
  if (e == cudaSuccess) e = attribute<64, false>();
  if (e == cudaSuccess) e = attribute<64, true>();
  return e;
}

cudaError_t launch_paged_tc(const PagedAttn& a, const PagedShape& s, const PagedPlan& pl, cudaStream_t st) {
  TcArgs p;
  memset(&p, 0, sizeof(p));
  p.a = a;
  p.s = s;
  p.runs = pl.runs;
  p.solo = pl.solo;
  p.npt = pl.rows / (pl.solo ? 1 : 2) / s.grp;
  p.rpt = p.npt * s.grp;
  const uint64_t h = a.pg.h;
  if (a.pg.format == FPD_PAGE_BF16) {
    const uint64_t qd[3] = {h, (uint64_t)a.nq, (uint64_t)a.batch * a.L}, qs[2] = {h * 2, h * 2 * a.nq};
    const uint32_t qb[3] = {64u, (uint32_t)s.grp, (uint32_t)p.npt};
    cudaError_t e = make_tmap_nd(&p.tm_q, a.q, 3, qd, qs, qb);
    const uint64_t dims[3] = {h, (uint64_t)2 * a.pg.nkv * a.pg.page, (uint64_t)a.pg.n_pages}, strides[2] = {h * 2, a.pg.page_bytes};
    const uint32_t box[3] = {64u, (uint32_t)std::min(KT, a.pg.page), 1u};
    if (e == cudaSuccess) e = make_tmap_nd(&p.tm_pages, a.pg.base, 3, dims, strides, box);
    if (a.lb) {
      const uint64_t bd[2] = {h, (uint64_t)a.batch * a.pg.nkv * a.lb}, bs[1] = {h * 2};
      const uint32_t bb[2] = {64u, (uint32_t)KT};
      if (e == cudaSuccess) e = make_tmap_nd(&p.tm_kblk, a.kblk, 2, bd, bs, bb);
      if (e == cudaSuccess) e = make_tmap_nd(&p.tm_vblk, a.vblk, 2, bd, bs, bb);
    }
    if (e != cudaSuccess) return e;
    return h == 128 ? launch_k(paged_tc_kernel<128, false>, pl.grid, Roles<false>::THREADS, smem_bytes<128, false>(), st, p)
                    : launch_k(paged_tc_kernel<64, false>, pl.grid, Roles<false>::THREADS, smem_bytes<64, false>(), st, p);
  }
  return h == 128 ? launch_k(paged_tc_kernel<128, true>, pl.grid, Roles<true>::THREADS, smem_bytes<128, true>(), st, p)
                  : launch_k(paged_tc_kernel<64, true>, pl.grid, Roles<true>::THREADS, smem_bytes<64, true>(), st, p);
}

}  // namespace fpd
