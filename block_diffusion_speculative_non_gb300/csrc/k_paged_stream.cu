// k_paged_stream.cu — attention over pages for few rows (single tokens, short blocks): at most 16 rows of a request share a kv
// head, so a call is a read of the keys.  Formulas and cut of the work as in k_paged_attention.cu and paged_sched.cuh.
//
// A warp has a run of its own and a ring of its own in shared memory, filled by bulk copies that one or a few of its lanes issue:
// no barrier between warps, and 130 KB and more of copies in flight per SM.  The keys are the 16 rows of the products and the
// queries their columns, S^T = K Q^T and O^T = V^T P^T on mma.sync m16n8k16, so that up to 8 query rows cost one product (with the
// queries as rows half of the products and registers of a single token's 4 heads would be padding, and the 4-bit form would be
// bound by products).  P^T goes from the accumulator's layout to the second product's by movmatrix.
//
// bf16 pages: tiles of 16 keys through TMA (64-dim boxes, 128-byte swizzle), read by ldmatrix; P as two bf16 terms.
// 4-bit pages: a product's operands are made in registers from the codes as they lie in the page.  A thread takes what it
// can use whole: of K, for two keys, the 32 (h = 64: 16) consecutive dims 32 c..; of V, for four keys, the 16 (8) dims 16 g..
// (c = lane % 4, g = lane / 4; the order of dims and keys inside a product is free).  Code n + 8 in bits 6..9 (2..5) of an fp16
// number of exponent 4 (8) reads 16 + n + 8 (256 + n + 8), and one fused multiply-add with s' = s 2^-7 takes it to n s'
// exactly (7 bits; 264 s' stays in range): 10 instructions for 8 dims.  Keys then need fp16 queries: each row is scaled by a power of
// two to a largest magnitude in [1, 2), so only elements below 2^-14 of it lose bits, 2^-25 of it at most.  P enters as fp16, half a
// step 2^-11, scaled by 2^14, so that weights keep it down to 2^-28 of the largest.  Block keys are bf16 and take the bf16
// products, their operands straight from global memory.
#include <cstring>

#include "attn_body.cuh"
#include "attn_tc_prims.cuh"
#include "paged_decode.cuh"
#include "paged_masks.cuh"
#include "paged_sched.cuh"

namespace fpd {

namespace {
using attn::ex2_approx;

constexpr int KT = kPagedTile;
constexpr uint32_t kSmemMax = 232448;

struct Args {
  CUtensorMap tm_pages, tm_kblk, tm_vblk;   // bf16: pages as [page][K|V, kv head, position][h], block keys and values as rows
  PagedAttn a;
  PagedShape s;
  int runs;
  bool per_cta;   // a CTA has a unit, its warps share the unit's tiles and put it together; no runs, no partials
};

__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Query rows of a warp: NT columns tiles of 8.  State of the softmax for rows 8 j + 2 c + e; O^T of dims by rows.
template <int H, int NT>
struct State {
  float o[H / 16][NT][4];
  float m[NT][2], l[NT][2];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < H / 16; i++)
#pragma unroll
      for (int j = 0; j < NT; j++) o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.f;
#pragma unroll
    for (int j = 0; j < NT; j++) {
      m[j][0] = m[j][1] = -INFINITY;
      l[j][0] = l[j][1] = 0.f;
    }
  }
};

// One step of the softmax over 16 M keys: s[mt][j][2 half + e], key half of m-tile mt, row 8 j + 2 c + e -> p 2^BIAS; O and l are
// brought to the new maximum.  sc: log2(e) / sqrt(h) and what the scores lack, per row.
template <int H, int NT, int M, int BIAS>
__device__ __forceinline__ void softmax_step(State<H, NT>& st, float (&s)[M][NT][4], const float (&sc)[NT][2]) {
  float mn[NT][2];
  bool up = false;
#pragma unroll
  for (int j = 0; j < NT; j++)
#pragma unroll
    for (int e = 0; e < 2; e++) {
      float mx = fmaxf(s[0][j][e], s[0][j][2 + e]);
#pragma unroll
      for (int i = 1; i < M; i++) mx = fmaxf(mx, fmaxf(s[i][j][e], s[i][j][2 + e]));
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      mn[j][e] = fmaxf(st.m[j][e], mx * sc[j][e]);
      up |= mn[j][e] > st.m[j][e];
    }
  if (__any_sync(0xffffffffu, up)) {
#pragma unroll
    for (int j = 0; j < NT; j++)
#pragma unroll
      for (int e = 0; e < 2; e++) {
        const float c = st.m[j][e] == -INFINITY ? 0.f : ex2_approx(st.m[j][e] - mn[j][e]);
        st.m[j][e] = mn[j][e];
        st.l[j][e] *= c;
#pragma unroll
        for (int i = 0; i < H / 16; i++) {
          st.o[i][j][e] *= c;
          st.o[i][j][2 + e] *= c;
        }
      }
  }
#pragma unroll
  for (int j = 0; j < NT; j++)
#pragma unroll
    for (int e = 0; e < 2; e++) {
      const float base = st.m[j][e] == -INFINITY ? 0.f : (float)BIAS - st.m[j][e];   // no key so far: weights 0, not NaN
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < M; i++)
#pragma unroll
        for (int h = 0; h < 4; h += 2) {
          s[i][j][h + e] = ex2_approx(fmaf(s[i][j][h + e], sc[j][e], base));
          sum += s[i][j][h + e];
        }
      st.l[j][e] += sum;
    }
}

template <int H, int NT, bool INT4>
struct Ring {
  static constexpr int HALF = INT4 ? KT * (H / 2 + H / 16) : 16 * H * 2;   // bytes of a slot's K or V: 64 or 16 keys
  static constexpr int SLOT = 2 * HALF;
  static constexpr int WARPS = INT4 && NT == 1 ? 12 : 8, SLOTS = INT4 && NT == 1 ? 2 : 3;
  static constexpr int BARS = WARPS * SLOTS * SLOT;
  static constexpr size_t BYTES = 1024 + BARS + WARPS * SLOTS * 8;
};

template <int H, int NT, bool INT4>
__global__ void __launch_bounds__(Ring<H, NT, INT4>::WARPS * 32, 1) paged_stream_kernel(const __grid_constant__ Args p) {
  using Rg = Ring<H, NT, INT4>;
  constexpr int R = 8 * NT, ST = Rg::SLOTS, MT = H / 16;
  constexpr int BIAS = INT4 ? 14 : 0;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int g = lane >> 2, c = lane & 3;
  uint8_t* ring = smem + warp * ST * Rg::SLOT;
  const uint32_t ring_s = tc::smem_u32(ring);
  const uint32_t bars = tc::smem_u32(smem + Rg::BARS) + warp * ST * 8;
  const PagedAttn& a = p.a;
  const PagedShape& sh = p.s;
  const int nrows = a.L * sh.grp;
  if (lane == 0) {
    for (int i = 0; i < ST; i++) tc::mbar_init(bars + 8 * i, 1);
    tc::fence_barrier_init();
  }
  __syncwarp();
  if (!INT4 && tid == 0) {
    tc::tma_prefetch(&p.tm_pages);
    if (a.lb) {
      tc::tma_prefetch(&p.tm_kblk);
      tc::tma_prefetch(&p.tm_vblk);
    }
  }
  pdl_wait();
  pdl_trigger();
  const DeviceLens lens{a.ctx_len, a.pg.cap()};
  const int run = blockIdx.x + warp * gridDim.x;
  if (!p.per_cta && run >= p.runs) return;
  PagedWalk<DeviceLens> walk = p.per_cta ? PagedWalk<DeviceLens>(sh, lens, a.batch, 1, 1, 1) : make_walk(sh, lens, a.batch, p.runs, run);
  const float sl2 = rsqrtf((float)H) * 1.4426950408889634f;
  if (!p.per_cta && lane == 0) a.desc[run] = make_int4(-1, 0, 0, 0);
  int cnt = 0;      // slots filled and emptied so far: place in the ring and phase
  bool ok = true;
  unsigned spoilt_units = 0;   // parts of the run, from 31 on together, that came out whole and with something that is no number
  int n_units = 0;

  PagedUnit u;
  int t0, t1, last_run;
  bool more;
  if (p.per_cta) {
    const int bg = blockIdx.x / sh.tiles;
    u.b = bg / sh.nkv;
    u.g = bg - u.b * sh.nkv;
    unit_tiles(sh, lens(u.b), blockIdx.x - bg * sh.tiles, u);
    t0 = warp * u.tiles() / Rg::WARPS;
    t1 = (warp + 1) * u.tiles() / Rg::WARPS;
    more = true;
  } else {
    more = walk.next(u, t0, t1, last_run);
  }
  for (; ok && more; more = !p.per_cta && walk.next(u, t0, t1, last_run)) {
    const int nt = min(t1, u.tiles());
    State<H, NT> st;
    st.clear();
    // ---- queries: row 8 j + g of the tile in the lanes 4 g + c ----
    const bf16* qrow[NT];
    float sc[NT][2];
    uint32_t qf[MT][NT][2];
    auto load_q = [&]() {   // behind the first copies' requests
#pragma unroll
      for (int j = 0; j < NT; j++) {
        const int qi = u.rt * R + 8 * j + g;
        qrow[j] = qi < nrows ? a.q + ((size_t)(u.b * a.L + qi / sh.grp) * a.nq + u.g * sh.grp + qi % sh.grp) * H : nullptr;
      }
      if constexpr (!INT4) {
#pragma unroll
        for (int j = 0; j < NT; j++) {
          sc[j][0] = sc[j][1] = sl2;
#pragma unroll
          for (int k = 0; k < MT; k++)
#pragma unroll
            for (int e = 0; e < 2; e++) qf[k][j][e] = qrow[j] ? __ldg(reinterpret_cast<const uint32_t*>(qrow[j] + 16 * k + 8 * e + 2 * c)) : 0u;
        }
      } else {
#pragma unroll
        for (int j = 0; j < NT; j++) {
          // dims H / 4 c ..: 8 of them per word of codes; product 2 w + e takes dims (2 e, 2 e + 4) and (2 e + 1, 2 e + 5) of word w
          float x[H / 4], big = 0.f;
#pragma unroll
          for (int w = 0; w < H / 32; w++) {
            const uint4 v = qrow[j] ? __ldg(reinterpret_cast<const uint4*>(qrow[j] + H / 4 * c + 8 * w)) : make_uint4(0, 0, 0, 0);
            const uint32_t r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; i++) {
              x[8 * w + 2 * i] = __uint_as_float(r[i] << 16);
              x[8 * w + 2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
            }
          }
#pragma unroll
          for (int i = 0; i < H / 4; i++) big = fmaxf(big, fabsf(x[i]));
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
          const int ex = min(max((int)(__float_as_uint(big) >> 23) - 127, -100), 100);   // the scale and its inverse stay normal
          const float down = __uint_as_float((uint32_t)(127 - ex) << 23), back = __uint_as_float((uint32_t)(127 + ex) << 23) * 128.f;
#pragma unroll
          for (int w = 0; w < H / 32; w++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
              qf[2 * w + e][j][0] = pack_f16(x[8 * w + 2 * e] * down, x[8 * w + 2 * e + 4] * down);
              qf[2 * w + e][j][1] = pack_f16(x[8 * w + 2 * e + 1] * down, x[8 * w + 2 * e + 5] * down);
            }
          sc[j][0] = sl2 * __shfl_sync(0xffffffffu, back, 8 * c);       // row 2 c is lane group 2 c
          sc[j][1] = sl2 * __shfl_sync(0xffffffffu, back, 8 * c + 4);
        }
      }
    };
    int pos_row[NT][2];
#pragma unroll
    for (int j = 0; j < NT; j++)
#pragma unroll
      for (int e = 0; e < 2; e++) pos_row[j][e] = u.n - a.L + (u.rt * R + 8 * j + 2 * c + e) / sh.grp;
    auto see = [&](int pos, int row) { return row_sees(sh, row, pos); };

    if constexpr (!INT4) {
      // ---- bf16: slots of 16 keys; a tile is up to four of them ----
      constexpr int SUB = KT / 16;
      const int steps = (nt - t0) * SUB;   // those past a tile's keys are passed over
      auto keys_of = [&](int i, PagedTile& t) {
        t = tile_at(u, KT, t0 + i / SUB);
        const int k = (i % SUB) * 16;
        t.k0 += k;
        t.pos += k;
        t.valid = min(16, t.valid - k);
        return t.valid > 0;
      };
      // the page of a step's keys is looked up one step ahead of its copies
      auto page_for = [&](int i) {
        PagedTile t;
        if (i >= steps || !keys_of(i, t) || !t.ctx) return 0;
        return page_of(a.pg, u.b, t.k0);
      };
      int filled = cnt, at_step = 0, next_id = page_for(0);
      auto fill = [&]() {   // the next step that has keys
        PagedTile t;
        while (at_step < steps) {
          const bool has = keys_of(at_step, t);
          const int id = next_id;
          next_id = page_for(at_step + 1);
          at_step++;
          if (!has) continue;
          if (lane == 0) {
            const uint32_t s = filled % ST, bar = bars + 8 * s, dst = ring_s + s * Rg::SLOT;
            tc::mbar_arrive_expect_tx(bar, Rg::SLOT);
            const int in = t.k0 & (a.pg.page - 1);
            for (int h = 0; h < H / 64; h++) {
              if (t.ctx) {   // a page that is none: a coordinate past the pool, which reads zeros
                const int z = id < 0 ? a.pg.n_pages : id;
                tc::tma_load_3d(dst + h * 2048, &p.tm_pages, h * 64, u.g * a.pg.page + in, z, bar);
                tc::tma_load_3d(dst + Rg::HALF + h * 2048, &p.tm_pages, h * 64, (a.pg.nkv + u.g) * a.pg.page + in, z, bar);
              } else {
                const int row = (u.b * a.pg.nkv + u.g) * a.lb + t.k0;
                tc::tma_load_2d(dst + h * 2048, &p.tm_kblk, h * 64, row, bar);
                tc::tma_load_2d(dst + Rg::HALF + h * 2048, &p.tm_vblk, h * 64, row, bar);
              }
            }
          }
          filled++;
          return;
        }
      };
      for (int i = 0; i < ST; i++) fill();
      load_q();
      for (int i = 0; i < steps && ok; i++) {
        PagedTile t;
        if (!keys_of(i, t)) continue;
        const uint32_t s = cnt % ST, ks = ring_s + s * Rg::SLOT, vs = ks + Rg::HALF;
        ok = attn_tc::wait_bar(bars + 8 * s, (cnt / ST) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        int h_lo, h_hi;
        hidden_from_all(sh, u, t, h_lo, h_hi);
        if (t.valid < 16 || h_hi > h_lo) {
          // V rows past the last key, and those that no row sees -> 0: 0 x a value that is not finite would be NaN
          for (int q = lane; q < (16 - t.valid + h_hi - h_lo) * (H / 8); q += 32) {
            const int z = q / (H / 8), r = z < h_hi - h_lo ? h_lo + z : t.valid + z - (h_hi - h_lo), ch = q % (H / 8);
            asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(vs + (ch >> 3) * 2048 + r * 128 + (ch & 7) * 16), "r"(0) : "memory");
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
        float sv[1][NT][4];
#pragma unroll
        for (int j = 0; j < NT; j++) sv[0][j][0] = sv[0][j][1] = sv[0][j][2] = sv[0][j][3] = 0.f;
        // chunk of 8 dims ch of row r: box ch / 8, swizzled 16-byte place
        auto at = [&](uint32_t base, int r, int ch) { return base + (ch >> 3) * 2048 + r * 128 + (((ch & 7) ^ (r & 7)) << 4); };
#pragma unroll
        for (int k = 0; k < MT; k++) {
          uint32_t f[4];   // (keys lo, dims lo), (keys hi, dims lo), (keys lo, dims hi), (keys hi, dims hi)
          attn::ldsm_x4(at(ks, (lane & 7) + ((lane >> 3) & 1) * 8, 2 * k + (lane >> 4)), f[0], f[1], f[2], f[3]);
#pragma unroll
          for (int j = 0; j < NT; j++) attn::mma_bf16(sv[0][j], f[0], f[1], f[2], f[3], qf[k][j][0], qf[k][j][1]);
        }
        const int k_last = t.pos + 15;
        const bool full = t.valid == 16 && (!sh.window || k_last < sh.sinks || u.p1 - t.pos < sh.window) && (!sh.causal || k_last <= u.p0);
        if (!full) {
#pragma unroll
          for (int j = 0; j < NT; j++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
              const int k = g + (e >> 1) * 8;
              if (k >= t.valid || !see(t.pos + k, pos_row[j][e & 1])) sv[0][j][e] = -INFINITY;
            }
        }
        softmax_step<H, NT, 1, BIAS>(st, sv, sc);
        uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
        for (int j = 0; j < NT; j++)
#pragma unroll
          for (int e = 0; e < 2; e++) {
            split_bf16x2(sv[0][j][2 * e], sv[0][j][2 * e + 1], hi[j][e], lo[j][e]);
            hi[j][e] = transpose8(hi[j][e]);
            lo[j][e] = transpose8(lo[j][e]);
          }
#pragma unroll
        for (int i2 = 0; i2 < MT; i2++) {
          uint32_t f[4];   // transposed: (dims lo, keys lo), (dims hi, keys lo), (dims lo, keys hi), (dims hi, keys hi)
          attn::ldsm_x4_t(at(vs, (lane & 7) + (lane >> 4) * 8, 2 * i2 + ((lane >> 3) & 1)), f[0], f[1], f[2], f[3]);
#pragma unroll
          for (int j = 0; j < NT; j++) {
            attn::mma_bf16(st.o[i2][j], f[0], f[1], f[2], f[3], hi[j][0], hi[j][1]);
            attn::mma_bf16(st.o[i2][j], f[0], f[1], f[2], f[3], lo[j][0], lo[j][1]);
          }
        }
        cnt++;
        __syncwarp();
        fill();
      }
      if (!ok)   // a wait ran out: let the copies in flight land before the CTA's memory goes
        for (int i = cnt; i < filled; i++) tc::mbar_wait(bars + 8 * (i % ST), (i / ST) & 1);
    } else {
      // ---- 4 bits: slots of 64 keys ----
      const int nc = min(nt, u.ns + u.nm);   // context tiles; the block's follow
      const int kp = min(KT, a.pg.page), part = lane & 3, pi = lane >> 2;   // lanes 4 i + part copy from page i of a tile
      auto page_for = [&](int i) {
        if (i >= nc || lane >= 16) return 0;
        const PagedTile t = tile_at(u, KT, i);
        return pi * kp < t.valid ? page_of(a.pg, u.b, t.k0 + pi * kp) : 0;
      };
      int filled = cnt, next_i = t0, next_id = page_for(t0);
      auto fill = [&]() {
        if (next_i >= nc) return;
        const PagedTile t = tile_at(u, KT, next_i);
        const int id = next_id;
        next_id = page_for(++next_i);
        const uint32_t s = filled % ST, bar = bars + 8 * s;
        const int rows = lane < 16 ? min(kp, ceil_div(t.valid, 16) * 16 - pi * kp) : 0;   // whole groups of 16 positions
        const int in = t.k0 & (a.pg.page - 1), w = part & 1 ? H / 16 : H / 2;             // scales or codes
        const uint32_t dst = ring_s + s * Rg::SLOT + (part >> 1) * Rg::HALF + (part & 1 ? KT * (H / 2) : 0) + pi * kp * w;
        uint32_t bytes = rows > 0 ? rows * w : 0;
        if (bytes && id < 0) {   // a page that is none: zeros
          for (uint32_t i = 0; i < bytes; i += 16) asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(dst + i), "r"(0) : "memory");
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          bytes = 0;
        }
        const uint32_t total = __reduce_add_sync(0xffffffffu, bytes);
        if (lane == 0) tc::mbar_arrive_expect_tx(bar, total);
        __syncwarp();
        if (bytes) {
          const uint8_t* src = slab_of(a.pg, id, part >> 1, u.g) + (part & 1 ? a.pg.page * (H / 2) : 0) + in * w;
          tc::bulk_load(dst, src, bytes, bar);
        }
        filled++;
      };
      for (int i = 0; i < ST; i++) fill();
      load_q();
      const int kk = (g >> 1) + 4 * (g & 1);   // row g of a product is key kk of its 16, row g + 8 key kk + 8
      for (int i = t0; i < nc && ok; i++) {
        const PagedTile t = tile_at(u, KT, i);
        const uint32_t s = cnt % ST;
        ok = attn_tc::wait_bar(bars + 8 * s, (cnt / ST) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint8_t* kc = ring + s * Rg::SLOT;
        const uint8_t *ksc = kc + KT * (H / 2), *vc = kc + Rg::HALF, *vsc = vc + KT * (H / 2);
        float sv[4][NT][4];
#pragma unroll
        for (int mt = 0; mt < 4; mt++) {
#pragma unroll
          for (int j = 0; j < NT; j++) sv[mt][j][0] = sv[mt][j][1] = sv[mt][j][2] = sv[mt][j][3] = 0.f;
          const int k0 = 16 * mt + kk, k1 = k0 + 8;
          uint32_t w0[H / 32], w1[H / 32], raw0, raw1;
          if constexpr (H == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(kc + k0 * 64 + 16 * c), y = *reinterpret_cast<const uint4*>(kc + k1 * 64 + 16 * c);
            w0[0] = x.x, w0[1] = x.y, w0[2] = x.z, w0[3] = x.w;
            w1[0] = y.x, w1[1] = y.y, w1[2] = y.z, w1[3] = y.w;
            raw0 = *reinterpret_cast<const unsigned short*>(ksc + k0 * 8 + 2 * c);
            raw1 = *reinterpret_cast<const unsigned short*>(ksc + k1 * 8 + 2 * c);
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(kc + k0 * 32 + 8 * c), y = *reinterpret_cast<const uint2*>(kc + k1 * 32 + 8 * c);
            w0[0] = x.x, w0[1] = x.y, w1[0] = y.x, w1[1] = y.y;
            raw0 = ksc[k0 * 4 + c];
            raw1 = ksc[k1 * 4 + c];
          }
#pragma unroll
          for (int q = 0; q < H / 32; q += 2) {   // two words have one scale
            const Scale2 s0(((raw0 >> (4 * q)) & 0xFF) * 0x00800080u), s1(((raw1 >> (4 * q)) & 0xFF) * 0x00800080u);
#pragma unroll
            for (int v = 0; v < 2; v++) {
              uint32_t x[4], y[4];
              decode4(w0[q + v], s0, x);
              decode4(w1[q + v], s1, y);
#pragma unroll
              for (int e = 0; e < 2; e++) {
                const uint32_t f[4] = {x[2 * e], y[2 * e], x[2 * e + 1], y[2 * e + 1]};
#pragma unroll
                for (int j = 0; j < NT; j++) mma_f16(sv[mt][j], f, qf[2 * (q + v) + e][j][0], qf[2 * (q + v) + e][j][1]);
              }
            }
          }
        }
        if (!tile_full(sh, u, t)) {
#pragma unroll
          for (int mt = 0; mt < 4; mt++)
#pragma unroll
            for (int j = 0; j < NT; j++)
#pragma unroll
              for (int e = 0; e < 4; e++) {
                const int k = 16 * mt + kk + (e >> 1) * 8;
                if (k >= t.valid || !see(t.pos + k, pos_row[j][e & 1])) sv[mt][j][e] = -INFINITY;
              }
        }
        softmax_step<H, NT, 4, BIAS>(st, sv, sc);
#pragma unroll
        for (int mt = 0; mt < 4; mt++) {
          uint32_t pf[NT][2];
#pragma unroll
          for (int j = 0; j < NT; j++) {
            pf[j][0] = transpose8(pack_f16(sv[mt][j][0], sv[mt][j][1]));
            pf[j][1] = transpose8(pack_f16(sv[mt][j][2], sv[mt][j][3]));
          }
          if (16 * mt >= t.valid) break;   // what lies behind is stale
          uint32_t f[2][H / 8];            // keys (c, c + 4) and (c + 8, c + 12), dims H / 8 g ..
#pragma unroll
          for (int hp = 0; hp < 2; hp++) {
            const int ka = 16 * mt + 8 * hp + c, kb = ka + 4;
            uint32_t ra, rb, wa[H / 64], wb[H / 64];
            if constexpr (H == 128) {
              const uint2 x = *reinterpret_cast<const uint2*>(vc + ka * 64 + 8 * g), y = *reinterpret_cast<const uint2*>(vc + kb * 64 + 8 * g);
              wa[0] = x.x, wa[1] = x.y, wb[0] = y.x, wb[1] = y.y;
              ra = vsc[ka * 8 + g];
              rb = vsc[kb * 8 + g];
            } else {
              wa[0] = *reinterpret_cast<const uint32_t*>(vc + ka * 32 + 4 * g);
              wb[0] = *reinterpret_cast<const uint32_t*>(vc + kb * 32 + 4 * g);
              ra = vsc[ka * 4 + (g >> 1)];
              rb = vsc[kb * 4 + (g >> 1)];
            }
            if (ka >= t.valid) ra = 0;   // stale scales may be no numbers
            if (kb >= t.valid) rb = 0;
            const Scale2 sp((ra << 7) | (rb << 23));
#pragma unroll
            for (int v = 0; v < H / 64; v++) {
              uint32_t x[4], y[4];
              decode4(__byte_perm(wa[v], wb[v], 0x5410), sp, x);
              decode4(__byte_perm(wa[v], wb[v], 0x7632), sp, y);
#pragma unroll
              for (int e = 0; e < 4; e++) {
                f[hp][8 * v + e] = x[e];
                f[hp][8 * v + 4 + e] = y[e];
              }
            }
          }
#pragma unroll
          for (int i2 = 0; i2 < MT; i2++) {
            const uint32_t fr[4] = {f[0][2 * i2], f[0][2 * i2 + 1], f[1][2 * i2], f[1][2 * i2 + 1]};
#pragma unroll
            for (int j = 0; j < NT; j++) mma_f16(st.o[i2][j], fr, pf[j][0], pf[j][1]);
          }
        }
        cnt++;
        __syncwarp();
        fill();
      }
      if (!ok)
        for (int i = cnt; i < filled; i++) tc::mbar_wait(bars + 8 * (i % ST), (i / ST) & 1);
      // ---- block keys: bf16, 16 at a time, from global memory ----
      for (int i = max(t0, nc); i < nt && ok; i++) {
        const PagedTile t = tile_at(u, KT, i);
        const size_t base = (((size_t)u.b * a.pg.nkv + u.g) * a.lb + t.k0) * H;
        for (int k0 = 0; k0 < t.valid; k0 += 16) {
          float sv[1][NT][4], plain[NT][2];
#pragma unroll
          for (int j = 0; j < NT; j++) {
            sv[0][j][0] = sv[0][j][1] = sv[0][j][2] = sv[0][j][3] = 0.f;
            plain[j][0] = plain[j][1] = sl2;
          }
          auto key = [&](const bf16* from, int k) { return k0 + k < t.valid ? from + base + (size_t)(k0 + k) * H : nullptr; };
          const bf16 *ka = key(a.kblk, g), *kb = key(a.kblk, g + 8);
          auto ld = [](const bf16* q, int d) { return q ? __ldg(reinterpret_cast<const uint32_t*>(q + d)) : 0u; };
#pragma unroll
          for (int k = 0; k < MT; k++) {
            const int d = 16 * k + 2 * c;
            const uint32_t f0 = ld(ka, d), f1 = ld(kb, d), f2 = ld(ka, d + 8), f3 = ld(kb, d + 8);
#pragma unroll
            for (int j = 0; j < NT; j++) attn::mma_bf16(sv[0][j], f0, f1, f2, f3, ld(qrow[j], d), ld(qrow[j], d + 8));
          }
#pragma unroll
          for (int j = 0; j < NT; j++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
              const int k = k0 + g + (e >> 1) * 8;
              if (k >= t.valid || !see(t.pos + k, pos_row[j][e & 1])) sv[0][j][e] = -INFINITY;
            }
          softmax_step<H, NT, 1, BIAS>(st, sv, plain);
          uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
          for (int j = 0; j < NT; j++)
#pragma unroll
            for (int e = 0; e < 2; e++) {   // O carries the values' 2^-7 too
              split_bf16x2(sv[0][j][2 * e] * 0.0078125f, sv[0][j][2 * e + 1] * 0.0078125f, hi[j][e], lo[j][e]);
              hi[j][e] = transpose8(hi[j][e]);
              lo[j][e] = transpose8(lo[j][e]);
            }
          uint32_t v[4][H / 16];   // keys 2 c, 2 c + 1, 2 c + 8, 2 c + 9, dims H / 8 g ..
#pragma unroll
          for (int q = 0; q < 4; q++) {
            const bf16* from = key(a.vblk, 2 * c + (q & 1) + 8 * (q >> 1));
#pragma unroll
            for (int w = 0; w < H / 64; w++) {
              const uint4 x = from ? __ldg(reinterpret_cast<const uint4*>(from + H / 8 * g + 8 * w)) : make_uint4(0, 0, 0, 0);
              v[q][4 * w] = x.x, v[q][4 * w + 1] = x.y, v[q][4 * w + 2] = x.z, v[q][4 * w + 3] = x.w;
            }
          }
#pragma unroll
          for (int i2 = 0; i2 < MT; i2++) {
            const uint32_t f0 = __byte_perm(v[0][i2], v[1][i2], 0x5410), f1 = __byte_perm(v[0][i2], v[1][i2], 0x7632);
            const uint32_t f2 = __byte_perm(v[2][i2], v[3][i2], 0x5410), f3 = __byte_perm(v[2][i2], v[3][i2], 0x7632);
#pragma unroll
            for (int j = 0; j < NT; j++) {
              attn::mma_bf16(st.o[i2][j], f0, f1, f2, f3, hi[j][0], hi[j][1]);
              attn::mma_bf16(st.o[i2][j], f0, f1, f2, f3, lo[j][0], lo[j][1]);
            }
          }
        }
      }
    }

    // ---- the rows' sums, and out ----
    const bool whole = !p.per_cta && t0 == 0 && t1 == u.len();
    const int slot = 2 * run + (t0 == 0 ? 1 : 0);
    bool spoilt = false;
#pragma unroll
    for (int j = 0; j < NT; j++)
#pragma unroll
      for (int e = 0; e < 2; e++) {
        float l = st.l[j][e];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        const int r = 8 * j + 2 * c + e, qi = u.rt * R + r;
        if (qi >= nrows) continue;
        const float ul = INT4 ? l * 6.103515625e-05f : l;   // 2^-14
        const bool none = l == 0.f;
        const float by = whole ? (none ? 0.f : (INT4 ? 128.f : 1.f) / l) : (INT4 ? 0.0078125f : 1.f);
        const size_t row = whole ? (size_t)(u.b * a.L + qi / sh.grp) * a.nq + u.g * sh.grp + qi % sh.grp : (size_t)slot * R + r;
        float x[H / 8];   // 4 bits: dims H / 8 g ..; bf16: dims 16 i + g and 16 i + g + 8
#pragma unroll
        for (int i = 0; i < MT; i++) {
          x[2 * i] = none ? 0.f : st.o[i][j][e] * by;
          x[2 * i + 1] = none ? 0.f : st.o[i][j][2 + e] * by;
          spoilt |= !(fabsf(x[2 * i]) < INFINITY && fabsf(x[2 * i + 1]) < INFINITY);
        }
        if (whole) {
          bf16* dst = a.out + row * H;
          if constexpr (INT4) {
#pragma unroll
            for (int i = 0; i < H / 8; i += 2)
              *reinterpret_cast<__nv_bfloat162*>(dst + H / 8 * g + i) = __floats2bfloat162_rn(x[i], x[i + 1]);
          } else {
#pragma unroll
            for (int i = 0; i < H / 8; i++) dst[16 * (i >> 1) + g + 8 * (i & 1)] = __float2bfloat16_rn(x[i]);
          }
          if (a.lse && g == 0) a.lse[row] = none ? -INFINITY : (st.m[j][e] + log2f(ul)) * 0.69314718055994531f;
        } else {
          float* dst = p.per_cta ? reinterpret_cast<float*>(ring) + r * H : a.o_part + row * H;
          if constexpr (INT4) {
#pragma unroll
            for (int i = 0; i < H / 8; i += 4) *reinterpret_cast<float4*>(dst + H / 8 * g + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
          } else {
#pragma unroll
            for (int i = 0; i < H / 8; i++) dst[16 * (i >> 1) + g + 8 * (i & 1)] = x[i];
          }
          if (g == 0) (p.per_cta ? reinterpret_cast<float2*>(ring + R * H * 4)[r] : a.ml[row]) = make_float2(st.m[j][e], ul);
        }
      }
    if (whole && __any_sync(0xffffffffu, spoilt)) spoilt_units |= 1u << min(n_units, 31);
    n_units++;
    if (!p.per_cta && lane == 0 && t0 == 0 && t1 < u.len()) a.desc[run] = make_int4(u.b, u.g, u.rt, last_run);   // left to others
  }
  if (!p.per_cta) {
    if (lane == 0) a.spoilt[run] = spoilt_units;
    return;
  }
  __syncthreads();   // the warps' shares, each in its own ring
  for (int i = tid; i < min(R, nrows - u.rt * R) * (H / 4); i += Rg::WARPS * 32) {
    const int r = i / (H / 4), d = 4 * (i % (H / 4)), qi = u.rt * R + r;
    float2 v[Rg::WARPS];
    float mx = -INFINITY, den = 0.f;
#pragma unroll
    for (int w = 0; w < Rg::WARPS; w++) {
      v[w] = reinterpret_cast<const float2*>(smem + w * ST * Rg::SLOT + R * H * 4)[r];
      if (v[w].y != 0.f) mx = fmaxf(mx, v[w].x);
    }
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < Rg::WARPS; w++) {
      const float by = v[w].y == 0.f ? 0.f : ex2_approx(v[w].x - mx);
      if (by == 0.f) continue;
      den += v[w].y * by;
      const float4 o = *reinterpret_cast<const float4*>(smem + w * ST * Rg::SLOT + (r * H + d) * 4);
      sum.x += o.x * by, sum.y += o.y * by, sum.z += o.z * by, sum.w += o.w * by;
    }
    const bool none = den == 0.f;
    const float by = none ? 0.f : 1.f / den;
    const size_t row = (size_t)(u.b * a.L + sh.by_grp.div(qi)) * a.nq + u.g * sh.grp + qi - sh.by_grp.div(qi) * sh.grp;
    uint2 w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(none ? 0.f : sum.y * by), "f"(none ? 0.f : sum.x * by));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(none ? 0.f : sum.w * by), "f"(none ? 0.f : sum.z * by));
    *reinterpret_cast<uint2*>(a.out + row * H + d) = w;
    if (a.lse && d == 0) a.lse[row] = none ? -INFINITY : (mx + log2f(den)) * 0.69314718055994531f;
  }
}

template <int H, int NT, bool INT4>
cudaError_t attribute() {
  using Rg = Ring<H, NT, INT4>;
  static_assert(Rg::BYTES <= kSmemMax, "rings exceed the shared memory of one CTA");
  return cudaFuncSetAttribute(paged_stream_kernel<H, NT, INT4>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Rg::BYTES);
}
template <int H, bool INT4>
cudaError_t attributes() {
  cudaError_t e = attribute<H, 1, INT4>();
  return e != cudaSuccess ? e : attribute<H, 2, INT4>();
}

template <int H, bool INT4>
cudaError_t launch(const Args& p, int num_sms, cudaStream_t st) {
  const int grid = p.per_cta ? p.a.batch * p.s.nkv * p.s.tiles : std::min(p.runs, num_sms);
  if (p.s.rows == 8) return launch_k(paged_stream_kernel<H, 1, INT4>, grid, Ring<H, 1, INT4>::WARPS * 32, Ring<H, 1, INT4>::BYTES, st, p);
  return launch_k(paged_stream_kernel<H, 2, INT4>, grid, Ring<H, 2, INT4>::WARPS * 32, Ring<H, 2, INT4>::BYTES, st, p);
}

}  // namespace

int paged_stream_warps(int rows, int format) {
  return rows == 8 && format == FPD_PAGE_INT4 ? Ring<128, 1, true>::WARPS : Ring<128, 1, false>::WARPS;
}

cudaError_t paged_stream_init_attributes() {
  cudaError_t e = attributes<128, false>();
  if (e == cudaSuccess) e = attributes<128, true>();
  if (e == cudaSuccess) e = attributes<64, false>();
  if (e == cudaSuccess) e = attributes<64, true>();
  return e;
}

cudaError_t launch_paged_stream(const PagedAttn& a, const PagedShape& s, const PagedPlan& pl, bool per_cta, cudaStream_t st) {
  Args p;
  memset(&p, 0, sizeof(p));
  p.a = a;
  p.s = s;
  p.runs = pl.runs;
  p.per_cta = per_cta;
  const uint64_t h = a.pg.h;
  cudaError_t e = cudaSuccess;
  if (a.pg.format == FPD_PAGE_BF16) {
    const uint64_t dims[3] = {h, (uint64_t)2 * a.pg.nkv * a.pg.page, (uint64_t)a.pg.n_pages}, strides[2] = {h * 2, a.pg.page_bytes};
    const uint32_t box[3] = {64u, 16u, 1u};
    e = make_tmap_nd(&p.tm_pages, a.pg.base, 3, dims, strides, box);
    if (a.lb) {
      const uint64_t bd[2] = {h, (uint64_t)a.batch * a.pg.nkv * a.lb}, bs[1] = {h * 2};
      if (e == cudaSuccess) e = make_tmap_nd(&p.tm_kblk, a.kblk, 2, bd, bs, box);
      if (e == cudaSuccess) e = make_tmap_nd(&p.tm_vblk, a.vblk, 2, bd, bs, box);
    }
    if (e != cudaSuccess) return e;
    return h == 128 ? launch<128, false>(p, pl.grid, st) : launch<64, false>(p, pl.grid, st);
  }
  return h == 128 ? launch<128, true>(p, pl.grid, st) : launch<64, true>(p, pl.grid, st);
}

}  // namespace fpd
