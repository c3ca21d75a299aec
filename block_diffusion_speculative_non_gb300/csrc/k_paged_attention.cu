// k_paged_attention.cu — attention of blocks over paged contexts: the choice between its two kernels, and the merge of partials.
//   out_r = sum_t exp(s_rt - lse_r) v_t,   s_rt = q_r . k_t / sqrt(h),   lse_r = log sum_t exp(s_rt),   t over what row r sees
//
// k_paged_stream.cu takes calls in which at most 16 rows of a request share a kv head, k_paged_tc.cu the others; paged_sched.cuh cuts
// the work of both.
#include <cmath>

#include "attn_body.cuh"
#include "paged_repair.cuh"
#include "paged_sched.cuh"

namespace fpd {

namespace {
using namespace attn;

struct Args {
  PagedAttn a;
  PagedShape s;
  int runs, spoilt_words;   // words of `spoilt` of a run
};

constexpr int kMergeWarps = 4, kMergeWays = 8;

// A row of a unit summed over the keys it sees, by one warp (paged_repair.cuh).
template <int H>
__device__ __forceinline__ void store_repaired(const Args& p, const PagedUnit& u, int qi, float m) {
  const PagedAttn& a = p.a;
  float acc[H / 32], den;
  repair_row<H>(a, p.s, u, qi, m, acc, den);
  const int j = p.s.by_grp.div(qi), grp = p.s.grp, lane = threadIdx.x & 31;
  bf16* dst = a.out + ((size_t)(u.b * a.L + j) * a.nq + u.g * grp + qi - j * grp) * H;
#pragma unroll
  for (int e = 0; e < H / 32; e++) dst[lane + 32 * e] = __float2bfloat16_rn(den == 0.f ? 0.f : acc[e] / den);
}
// The units among the parts `bad` of run c that it finished by itself: rows that hold something that is no number once more.
template <int H>
__device__ __noinline__ void repair_run(const Args& p, int c, unsigned bad) {
  const PagedAttn& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, grp = p.s.grp;
  PagedWalk<DeviceLens> walk = make_walk(p.s, DeviceLens{a.ctx_len, a.pg.cap()}, a.batch, p.runs, c);
  PagedUnit u;
  int t0, t1, last;
  for (int n = 0; walk.next(u, t0, t1, last); n++) {
    if (t0 != 0 || t1 != u.len() || !(bad >> min(n, 31) & 1)) continue;
    for (int qi = u.rt * p.s.rows + warp; qi < min(a.L * grp, (u.rt + 1) * p.s.rows); qi += blockDim.x >> 5) {
      const int j = p.s.by_grp.div(qi);
      const bf16* row = a.out + ((size_t)(u.b * a.L + j) * a.nq + u.g * grp + qi - j * grp) * H;
      bool spoilt = false;
      for (int d = lane; d < H; d += 32) spoilt |= !(fabsf(__bfloat162float(row[d])) < INFINITY);
      if (__any_sync(0xffffffffu, spoilt)) store_repaired<H>(p, u, qi, NAN);
    }
  }
}

// The units that runs share: CTA (c, y) puts together rows of the unit that run c starts and leaves unfinished, from slots
// 2 c + 1, 2 (c + 1), .. in that order; a warp has RPW rows.  The partials are requested with their weights, not behind them.
// WAYS > 1, few units cut into many parts: CTA (u, y) has row y of unit u, whose first run it looks for, and its warps share the
// partials (one context of 39520 positions, 82 rows, 304 parts: 24 us in all, 87 with a
// warp for two rows; one token of a context of 65536 in 8 kv heads, 152 parts each: 55 and 70, in 4 bits 33 and 56).
template <int H, int RPW, int WAYS = 1>
__global__ void __launch_bounds__((WAYS > 1 ? WAYS : kMergeWarps) * 32) paged_merge_kernel(const __grid_constant__ Args p) {
  static_assert(WAYS == 1 || RPW == 1, "a CTA shares one row");
  constexpr int DPL = H / 32, U = 8 / RPW;
  pdl_wait();
  pdl_trigger();
  const PagedAttn& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, R = p.s.rows, grp = p.s.grp;
  const bool masks = p.s.window || p.s.causal;
  if (masks && blockIdx.y == 0) {   // units that a run finished by itself and that came out with something that is no number
    for (int run = blockIdx.x; run < p.runs; run += gridDim.x) {
      unsigned bad = 0;
      for (int i = 0; i < p.spoilt_words; i++) bad |= a.spoilt[run * p.spoilt_words + i];
      if (bad) repair_run<H>(p, run, bad);
    }
  }
  int c = blockIdx.x;
  if constexpr (WAYS > 1) {
    __shared__ int first;
    if (threadIdx.x == 0) first = -1;
    __syncthreads();
    const int rt = blockIdx.x % p.s.tiles, bg = blockIdx.x / p.s.tiles, g = bg % p.s.nkv, b = bg / p.s.nkv;
    for (int run = threadIdx.x; run < p.runs; run += WAYS * 32) {
      const int4 d = a.desc[run];
      if (d.x == b && d.y == g && d.z == rt) first = run;
    }
    __syncthreads();
    c = first;
    if (c < 0) return;   // a run has finished it
  }
  const int4 d = a.desc[c];
  const int r0 = WAYS > 1 ? blockIdx.y : (blockIdx.y * kMergeWarps + warp) * RPW, rows = min(R, a.L * grp - d.z * R);
  if (d.x < 0 || r0 >= rows) return;
  const int pieces = d.w - c + 1;
  auto slot = [&](int i, int r) { return (size_t)(i == 0 ? 2 * c + 1 : 2 * (c + i)) * R + min(r, rows - 1); };
  float mx[RPW], den[RPW], num[RPW][DPL];
#pragma unroll
  for (int q = 0; q < RPW; q++) {
    mx[q] = -INFINITY;
    den[q] = 0.f;
#pragma unroll
    for (int e = 0; e < DPL; e++) num[q][e] = 0.f;
  }
  for (int i0 = WAYS > 1 ? warp * U : 0; i0 < pieces; i0 += WAYS * U) {   // the softmax of the partials, U at a time
    float t[RPW][U][DPL];
    float2 v[RPW][U];
#pragma unroll
    for (int q = 0; q < RPW; q++)
#pragma unroll
      for (int u = 0; u < U; u++) {
        const size_t at = slot(min(i0 + u, pieces - 1), r0 + q);
        v[q][u] = __ldcg(a.ml + at);
        const float* op = a.o_part + at * H + lane * DPL;
        if constexpr (DPL == 4) {
          const float4 f = __ldcg(reinterpret_cast<const float4*>(op));
          t[q][u][0] = f.x, t[q][u][1] = f.y, t[q][u][2] = f.z, t[q][u][3] = f.w;
        } else {
          const float2 f = __ldcg(reinterpret_cast<const float2*>(op));
          t[q][u][0] = f.x, t[q][u][1] = f.y;
        }
      }
#pragma unroll
    for (int q = 0; q < RPW; q++) {
      float m = mx[q];
#pragma unroll
      for (int u = 0; u < U; u++) {
        if (i0 + u >= pieces) v[q][u].y = 0.f;   // l = 0: no weight, whatever the rest holds
        if (v[q][u].y != 0.f) m = fmaxf(m, v[q][u].x);
      }
      const float back = den[q] == 0.f ? 0.f : ex2_approx(mx[q] - m);
      mx[q] = m;
      den[q] *= back;
#pragma unroll
      for (int e = 0; e < DPL; e++) num[q][e] = back == 0.f ? 0.f : num[q][e] * back;
#pragma unroll
      for (int u = 0; u < U; u++) {
        const float w = v[q][u].y == 0.f ? 0.f : ex2_approx(v[q][u].x - m);
        den[q] += v[q][u].y == 0.f ? 0.f : v[q][u].y * w;
#pragma unroll
        for (int e = 0; e < DPL; e++) num[q][e] += w != 0.f ? t[q][u][e] * w : 0.f;
      }
    }
  }
  if constexpr (WAYS > 1) {   // the warps' sums, in their order
    __shared__ float2 stat[WAYS];
    __shared__ float part[WAYS][H];
    if (lane == 0) stat[warp] = make_float2(mx[0], den[0]);
#pragma unroll
    for (int e = 0; e < DPL; e++) part[warp][lane * DPL + e] = num[0][e];
    __syncthreads();
    if (warp > 0) return;
    float m = -INFINITY;
    for (int w = 0; w < WAYS; w++)
      if (stat[w].y != 0.f) m = fmaxf(m, stat[w].x);
    den[0] = 0.f;
#pragma unroll
    for (int e = 0; e < DPL; e++) num[0][e] = 0.f;
    for (int w = 0; w < WAYS; w++) {
      const float by = stat[w].y == 0.f ? 0.f : ex2_approx(stat[w].x - m);
      den[0] += stat[w].y == 0.f ? 0.f : stat[w].y * by;
#pragma unroll
      for (int e = 0; e < DPL; e++) num[0][e] += by != 0.f ? part[w][lane * DPL + e] * by : 0.f;
    }
    mx[0] = m;
  }
#pragma unroll
  for (int q = 0; q < RPW; q++) {
    if (r0 + q >= rows) break;
    const int qi = d.z * R + r0 + q, j = p.s.by_grp.div(qi);
    const bool none = den[q] == 0.f;
    float by = 1.f / den[q];
    bool spoilt = false;
#pragma unroll
    for (int e = 0; e < DPL; e++) spoilt |= !none && !(fabsf(num[q][e] * by) < INFINITY);
    const size_t row = (size_t)(d.x * a.L + j) * a.nq + d.y * grp + qi - j * grp;
    if (masks && fabsf(den[q]) < INFINITY && __any_sync(0xffffffffu, spoilt)) {
      PagedUnit u;
      unit_tiles(p.s, clamp_ctx(a.ctx_len[d.x], a.pg.cap()), d.z, u);
      u.b = d.x;
      u.g = d.y;
      store_repaired<H>(p, u, qi, mx[q]);
    } else {
      bf16* dst = a.out + row * H + lane * DPL;
#pragma unroll
      for (int e = 0; e < DPL; e += 2)
        *reinterpret_cast<__nv_bfloat162*>(dst + e) = __floats2bfloat162_rn(none ? 0.f : num[q][e] * by, none ? 0.f : num[q][e + 1] * by);
    }
    if (a.lse && lane == 0) a.lse[row] = none ? -INFINITY : (mx[q] + log2f(den[q])) * 0.69314718055994531f;
  }
}

// parts of a unit from which on a CTA merges one row (blocks of 16, 38 parts a unit: 41.5 us against 48.7; 19 parts: 31.3 against 30.7; 10:
// 36.9 against 28.8)
constexpr int kManyParts = 24;
constexpr int kUnitCost = 3;   // what a unit costs besides its tiles, in tiles (0, 2 and 3: 103, 97 and 95 us at four trajectories with a window)

// The most tiles that a unit can have.
long long most_tiles(const Args& p) {
  const PagedShape& s = p.s;
  const int kt = s.kt();
  long long n = ceil_div(p.a.pg.cap(), kt);
  if (s.window) n = std::min(n, ((long long)s.window + s.L) / kt + 2 + ceil_div(std::min(s.sinks, 1 << 29), kt));
  return n + ceil_div(s.lb, kt);
}

// Few short units: a CTA each, whose warps have at most two tiles, does without partials and the merge's launch.  (Rows of one position
// see the same keys, so nothing needs a repair.)  4 tokens, 8 kv heads, us in runs and so: contexts to 512 16.4 and 11.1, to 1024 (three
// tiles a warp) 13.4 and 15.9; 4 bits, to 1024 11.9 and 10.0, to 2048 (three tiles) 13.8 and 14.8.
bool unit_per_cta(const Args& p, const PagedPlan& pl) {
  const PagedShape& s = p.s;
  if (s.L > 1 && (s.window || s.causal)) return false;
  const long long units = (long long)p.a.batch * s.nkv * s.tiles;
  return units <= pl.sms && most_tiles(p) <= 2 * paged_stream_warps(s.rows, p.a.pg.format);
}

template <int H>
cudaError_t launch(const Args& p, const PagedPlan& pl, cudaStream_t st) {
  const bool alone = pl.kernel == kPagedStream && unit_per_cta(p, pl);
  const cudaError_t e = pl.kernel == kPagedStream ? launch_paged_stream(p.a, p.s, pl, alone, st) : launch_paged_tc(p.a, p.s, pl, st);
  if (e != cudaSuccess || alone) return e;
  const int rows = std::min(pl.rows, p.a.L * p.s.grp);
  const long long units = (long long)p.a.batch * p.s.nkv * p.s.tiles;
  if (pl.runs > kManyParts * units && most_tiles(p) > kManyParts)
    return launch_k(paged_merge_kernel<H, 1, kMergeWays>, dim3((unsigned)units, rows), kMergeWays * 32, 0, st, p);
  auto merge = [&](auto kernel, int rpw) { return launch_k(kernel, dim3(pl.runs, ceil_div(rows, rpw * kMergeWarps)), kMergeWarps * 32, 0, st, p); };
  if (pl.kernel == kPagedStream) return merge(paged_merge_kernel<H, 1>, 1);
  // two partials a unit, mostly: more rows a warp (windows at four trajectories 78 -> 74 us, 3 blocks of few units 16.6 -> 17.3)
  return pl.runs <= 2 * units ? merge(paged_merge_kernel<H, 4>, 4) : merge(paged_merge_kernel<H, 2>, 2);
}

}  // namespace

PagedPlan paged_attn_plan(int batch, int L, int nq, int nkv, int format, int t_cap, int num_sms) {
  PagedPlan pl{};
  pl.sms = num_sms;
  const int grp = nq / nkv, n = L * grp;
  // 16 rows, us by the stream kernel and by tcgen05: one context of 65536 73 and 70 (4 bits 55 and 63), 8 to 2048 28 and 24 (22 and 23),
  // 64 to 4096 109 and 121 (76 and 114), 16 to 16384 109 and 116 (69 and 105)
  pl.kernel = n <= 16 ? kPagedStream : kPagedTc;
  // tcgen05: units of one lane's rows (4 bits: 96, so that warps are left to decode for either lane), or as few of two lanes as there can
  // be, of even sizes.  128 rows of 64 requests: 137 us as one lane each, 164 as two (96 rows, 4 bits: 144 and 201); 1540 rows of 4 requests:
  // 154 us in units of one lane, each with its own copies of K and V, 119 in units of two (with a window 85 and 78).
  const int npt = 128 / grp, tiles = ceil_div(L, 2 * npt);
  pl.solo = pl.kernel == kPagedTc && L <= npt && n <= (format == FPD_PAGE_INT4 ? 96 : 128);
  pl.rows = n <= 8 ? 8 : n <= 16 ? 16 : pl.solo ? n : 2 * grp * ceil_div(L, 2 * tiles);
  pl.tiles = ceil_div(n, pl.rows);
  // no more runs than there can be tiles
  const long long most = (long long)batch * nkv * pl.tiles * (ceil_div(t_cap, kPagedTile) + ceil_div(L, kPagedTile));
  pl.too_large = most + 2ll * batch * nkv * pl.tiles * (1 + kUnitCost) > INT32_MAX;
  if (pl.kernel == kPagedStream) {
    pl.runs = (int)std::min<long long>(most, (long long)num_sms * paged_stream_warps(pl.rows, format));
    pl.grid = std::min(num_sms, pl.runs);
  } else {
    const int lanes = pl.solo ? 2 : 1;   // runs of a CTA
    pl.grid = (int)std::min<long long>(num_sms, (most + lanes - 1) / lanes);
    pl.runs = pl.grid * lanes;
  }
  return pl;
}

cudaError_t paged_attn_init_attributes() {
  const cudaError_t e = paged_stream_init_attributes();
  return e != cudaSuccess ? e : paged_tc_init_attributes();
}

cudaError_t launch_paged_attention(const PagedAttn& a, const PagedPlan& pl, cudaStream_t st) {
  Args p;
  p.a = a;
  // positions stay below 2^30 + 2^26: a longer window hides nothing; nor does causal from the only, last position
  constexpr int kFar = 1200000000;
  p.s = paged_shape(a.L, a.lb, a.nq / a.pg.nkv, a.pg.nkv, pl.rows, a.window > kFar ? 0 : a.window, std::min(a.sinks, kFar), a.causal && a.L > 1,
                    pl.kernel == kPagedTc ? kPagedTcTile : kPagedTile, kUnitCost);
  p.runs = pl.runs;
  p.spoilt_words = pl.kernel == kPagedStream ? 1 : pl.solo ? 4 : 8;
  return a.pg.h == 128 ? launch<128>(p, pl, st) : launch<64>(p, pl, st);
}

}  // namespace fpd
