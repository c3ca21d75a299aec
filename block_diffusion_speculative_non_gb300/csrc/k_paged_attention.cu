// k_paged_attention.cu — attention of blocks over paged contexts, on mma.sync, and the merge of partials:
//   out_r = sum_t exp(s_rt - lse_r) v_t,   s_rt = q_r . k_t / sqrt(h),   lse_r = log sum_t exp(s_rt),   t over what row r sees
//
// The work is cut as paged_sched.cuh says.  A CTA of four warps walks its run in tiles of 64 keys, copied ahead into shared
// memory; WM warps have 16 rows each and the other factor of the four shares a tile's keys, so that few rows (single tokens)
// keep all warps at work.  A warp's softmax statistics and O stay in registers.
#include <cmath>

#include "attn_body.cuh"
#include "paged_sched.cuh"

namespace fpd {

namespace {
using namespace attn;

constexpr int kThreads = NWARP * 32;

struct Args {
  PagedAttn a;
  PagedShape s;
  int runs;
};

// One warp's 16 rows over NK keys of a tile (rows key0.. of the swizzled K and V tiles); p_lo, p_hi: positions of rows
// lane / 4 and lane / 4 + 8; first: position of the first key.
template <int H, int NK>
__device__ __forceinline__ void tile_math(uint32_t ks, uint32_t vs, const uint32_t (&qf)[H / 16][4], float (&o)[H / 8][4], float (&m)[2],
                                          float (&l)[2], bool full, const PagedShape& sh, int first, int valid, int p_lo, int p_hi,
                                          int lane, float sl2) {
  constexpr int NKS = H / 16, NOT = H / 8;
  float s[NK / 8][4];
#pragma unroll
  for (int n = 0; n < NK / 8; n++) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
  for (int kp = 0; kp < NK / 16; kp++)
#pragma unroll
    for (int kk = 0; kk < NKS; kk++) {
      const int key = kp * 16 + (lane & 7) + ((lane >> 4) << 3), c = kk * 2 + ((lane >> 3) & 1);
      uint32_t b0, b1, b2, b3;
      ldsm_x4(swz<H>(ks, key, c), b0, b1, b2, b3);
      mma_bf16(s[2 * kp], qf[kk][0], qf[kk][1], qf[kk][2], qf[kk][3], b0, b1);
      mma_bf16(s[2 * kp + 1], qf[kk][0], qf[kk][1], qf[kk][2], qf[kk][3], b2, b3);
    }
  if (!full) {
#pragma unroll
    for (int n = 0; n < NK / 8; n++)
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const int k = n * 8 + (lane & 3) * 2 + (e & 1), pos = first + k, row = e < 2 ? p_lo : p_hi;
        const bool see = k < valid && (!sh.window || pos < sh.sinks || row - pos < sh.window) && (!sh.causal || pos <= row);
        if (!see) s[n][e] = -INFINITY;
      }
  }
  float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
  for (int n = 0; n < NK / 8; n++) {
    mx0 = fmaxf(mx0, fmaxf(s[n][0], s[n][1]));
    mx1 = fmaxf(mx1, fmaxf(s[n][2], s[n][3]));
  }
  mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
  mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
  mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
  mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
  const float mn0 = fmaxf(m[0], mx0 * sl2), mn1 = fmaxf(m[1], mx1 * sl2);
  const float c0 = m[0] == -INFINITY ? 0.f : ex2_approx(m[0] - mn0), c1 = m[1] == -INFINITY ? 0.f : ex2_approx(m[1] - mn1);
  m[0] = mn0;
  m[1] = mn1;
  const float n0 = mn0 == -INFINITY ? 0.f : -mn0, n1 = mn1 == -INFINITY ? 0.f : -mn1;   // no key so far: weights 0, not NaN
  float ps0 = 0.f, ps1 = 0.f;
#pragma unroll
  for (int n = 0; n < NK / 8; n++) {
    s[n][0] = ex2_approx(fmaf(s[n][0], sl2, n0));
    s[n][1] = ex2_approx(fmaf(s[n][1], sl2, n0));
    s[n][2] = ex2_approx(fmaf(s[n][2], sl2, n1));
    s[n][3] = ex2_approx(fmaf(s[n][3], sl2, n1));
    ps0 += s[n][0] + s[n][1];
    ps1 += s[n][2] + s[n][3];
  }
  l[0] = l[0] * c0 + ps0;
  l[1] = l[1] * c1 + ps1;
#pragma unroll
  for (int n = 0; n < NOT; n++) {
    o[n][0] *= c0;
    o[n][1] *= c0;
    o[n][2] *= c1;
    o[n][3] *= c1;
  }
#pragma unroll
  for (int kk = 0; kk < NK / 16; kk++) {
    uint32_t h0, h1, h2, h3, l0_, l1_, l2_, l3_;
    split_bf16x2(s[2 * kk][0], s[2 * kk][1], h0, l0_);
    split_bf16x2(s[2 * kk][2], s[2 * kk][3], h1, l1_);
    split_bf16x2(s[2 * kk + 1][0], s[2 * kk + 1][1], h2, l2_);
    split_bf16x2(s[2 * kk + 1][2], s[2 * kk + 1][3], h3, l3_);
#pragma unroll
    for (int np = 0; np < NOT / 2; np++) {
      const int key = kk * 16 + (lane & 7) + (((lane >> 3) & 1) << 3), c = np * 2 + (lane >> 4);
      uint32_t b0, b1, b2, b3;
      ldsm_x4_t(swz<H>(vs, key, c), b0, b1, b2, b3);
      mma_bf16(o[2 * np], h0, h1, h2, h3, b0, b1);
      mma_bf16(o[2 * np + 1], h0, h1, h2, h3, b2, b3);
      mma_bf16(o[2 * np], l0_, l1_, l2_, l3_, b0, b1);
      mma_bf16(o[2 * np + 1], l0_, l1_, l2_, l3_, b2, b3);
    }
  }
}

// Shared memory: Q of 16 WM rows, two K and V tiles.  The keys' shares of O meet in the K and V tiles.
template <int H, int WM>
struct Mem {
  bf16 q[WM * 16 * H];
  bf16 kv[2][2][KT * H];
};

template <int H, int WM, bool INT4>
__global__ void __launch_bounds__(kThreads) paged_mma_kernel(const __grid_constant__ Args p) {
  constexpr int WK = NWARP / WM, NK = KT / WK, R = WM * 16, CH = H / 8, NKS = H / 16, NOT = H / 8;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  Mem<H, WM>& sm = *reinterpret_cast<Mem<H, WM>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wm = warp % WM, wk = warp / WM;
  const PagedAttn& a = p.a;
  const PagedShape& sh = p.s;
  const int nrows = a.L * sh.grp, cap = a.pg.cap();
  pdl_wait();
  pdl_trigger();
  PagedWalk<DeviceLens> walk = make_walk(sh, DeviceLens{a.ctx_len, cap}, a.batch, p.runs, blockIdx.x);
  const float sl2 = rsqrtf((float)H) * 1.4426950408889634f;
  const uint32_t q_s = smem_addr(sm.q);
  int4 left = make_int4(-1, 0, 0, 0);   // the unit that this run leaves unfinished

  PagedUnit u;
  int t0, t1, last_run;
  while (walk.next(u, t0, t1, last_run)) {
    for (int idx = tid; idx < R * CH; idx += kThreads) {
      const int r = idx / CH, c = idx % CH, qi = u.rt * R + r;
      const bool ok = qi < nrows;
      const bf16* src = a.q;
      if (ok) src = a.q + ((size_t)(u.b * a.L + qi / sh.grp) * a.nq + u.g * sh.grp + qi % sh.grp) * H + c * 8;
      cp_async16(swz<H>(q_s, r, c), src, ok);
    }
    cp_async_commit();
    auto load = [&](int buf, int i) {
      const PagedTile t = tile_at(u, KT, i);
      const uint32_t ks = smem_addr(sm.kv[buf][0]), vs = smem_addr(sm.kv[buf][1]);
      if (!t.ctx) {
        const size_t base = (((size_t)u.b * a.pg.nkv + u.g) * a.lb + t.k0) * H;
        for (int idx = tid; idx < KT * CH; idx += kThreads) {
          const int r = idx / CH, c = idx % CH;
          const bool ok = r < t.valid;
          const size_t at = ok ? base + (size_t)r * H + c * 8 : 0;
          cp_async16(swz<H>(ks, r, c), a.kblk + at, ok);
          cp_async16(swz<H>(vs, r, c), a.vblk + at, ok);
        }
      } else {
        for (int idx = tid; idx < KT * CH; idx += kThreads) {
          const int r = idx / CH, c = idx % CH;
          bool ok = r < t.valid;
          int id = -1;
          if (ok) id = page_of(a.pg, u.b, t.k0 + r);
          ok = id >= 0;
          const int in = (t.k0 + r) & (a.pg.page - 1);
          const uint8_t* k = ok ? slab_of(a.pg, id, 0, u.g) : a.pg.base;
          const uint8_t* v = ok ? slab_of(a.pg, id, 1, u.g) : a.pg.base;
          if (!INT4) {
            const size_t at = ok ? ((size_t)in * H + c * 8) * 2 : 0;
            cp_async16(swz<H>(ks, r, c), k + at, ok);
            cp_async16(swz<H>(vs, r, c), v + at, ok);
          } else {
            auto deq = [&](const uint8_t* slab, uint32_t dst) {
              uint32_t w[4] = {0, 0, 0, 0};
              if (ok) {
                const uint32_t code = *reinterpret_cast<const uint32_t*>(slab + in * (H / 2) + c * 4);
                const float s = scale_value(slab[a.pg.page * (H / 2) + in * (H / 16) + c / 2]);
#pragma unroll
                for (int e = 0; e < 4; e++)
                  asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                      : "=r"(w[e])
                      : "f"(((int)((code >> (8 * e + 4)) & 15) - 8) * s), "f"(((int)((code >> (8 * e)) & 15) - 8) * s));
              }
              asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
            };
            deq(k, swz<H>(ks, r, c));
            deq(v, swz<H>(vs, r, c));
          }
        }
      }
      cp_async_commit();
    };
    const int nt = min(t1, u.tiles());   // an empty unit has no tile
    if (t0 < nt) load(0, t0);

    float o[NOT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < NOT; n++) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    uint32_t qf[NKS][4];
    if (t0 < nt) cp_async_wait<1>(); else cp_async_wait<0>();
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < NKS; kk++)
      ldsm_x4(swz<H>(q_s, wm * 16 + (lane & 15), kk * 2 + (lane >> 4)), qf[kk][0], qf[kk][1], qf[kk][2], qf[kk][3]);
    const int r_lo = u.rt * R + wm * 16 + (lane >> 2);
    const int p_lo = u.n - a.L + r_lo / sh.grp, p_hi = u.n - a.L + (r_lo + 8) / sh.grp;
    for (int i = t0; i < nt; i++) {
      const int buf = (i - t0) & 1;
      if (i + 1 < nt) {
        load(buf ^ 1, i + 1);
        cp_async_wait<1>();
      } else {
        cp_async_wait<0>();
      }
      __syncthreads();
      const PagedTile t = tile_at(u, KT, i);
      const bool full = tile_full(sh, u, t);
      const int k0 = wk * NK;
      if (k0 < t.valid)
        tile_math<H, NK>(smem_addr(sm.kv[buf][0]) + k0 * H * 2, smem_addr(sm.kv[buf][1]) + k0 * H * 2, qf, o, m, l, full, sh,
                         t.pos + k0, t.valid - k0, p_lo, p_hi, lane, sl2);
      __syncthreads();
    }
#pragma unroll
    for (int e = 0; e < 2; e++) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
    }
    if (WK > 1) {   // the keys' shares, in the order of their warps
      __syncthreads();   // a unit without a tile: Q may still be read
      float* share = reinterpret_cast<float*>(sm.kv);   // [WK][R][H]
      float2* stat = reinterpret_cast<float2*>(sm.q);   // [WK][R]
#pragma unroll
      for (int half = 0; half < 2; half++) {
        const int r = wm * 16 + (lane >> 2) + half * 8;
        float* dst = share + ((size_t)wk * R + r) * H + (lane & 3) * 2;
#pragma unroll
        for (int n = 0; n < NOT; n++) *reinterpret_cast<float2*>(dst + n * 8) = make_float2(o[n][half * 2], o[n][half * 2 + 1]);
        if ((lane & 3) == 0) stat[wk * R + r] = make_float2(m[half], l[half]);
      }
      __syncthreads();
      if (wk == 0) {
#pragma unroll
        for (int half = 0; half < 2; half++) {
          const int r = wm * 16 + (lane >> 2) + half * 8;
          float mx = -INFINITY, den = 0.f, wgt[WK];
#pragma unroll
          for (int w = 0; w < WK; w++) mx = fmaxf(mx, stat[w * R + r].x);
#pragma unroll
          for (int w = 0; w < WK; w++) {
            const float2 v = stat[w * R + r];
            wgt[w] = v.x == -INFINITY ? (v.y == v.y ? 0.f : 1.f) : ex2_approx(v.x - mx);   // a NaN sum counts
            den += v.y * wgt[w];
          }
          m[half] = mx;
          l[half] = den;
#pragma unroll
          for (int n = 0; n < NOT; n++) {
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int w = 0; w < WK; w++) {
              const float2 v = *reinterpret_cast<const float2*>(share + ((size_t)w * R + r) * H + (lane & 3) * 2 + n * 8);
              if (wgt[w] != 0.f) {
                sum.x += v.x * wgt[w];
                sum.y += v.y * wgt[w];
              }
            }
            o[n][half * 2] = sum.x;
            o[n][half * 2 + 1] = sum.y;
          }
        }
      }
    }
    const bool whole = t0 == 0 && t1 == u.len();
    const int slot = 2 * blockIdx.x + (t0 == 0 ? 1 : 0);
    if (wk == 0) {
#pragma unroll
      for (int half = 0; half < 2; half++) {
        const int r = wm * 16 + (lane >> 2) + half * 8, qi = u.rt * R + r;
        if (qi >= nrows) continue;
        if (whole) {
          const size_t row = (size_t)(u.b * a.L + qi / sh.grp) * a.nq + u.g * sh.grp + qi % sh.grp;
          const bool none = l[half] == 0.f;
          const float inv = none ? 0.f : 1.f / l[half];
          bf16* dst = a.out + row * H + (lane & 3) * 2;
#pragma unroll
          for (int n = 0; n < NOT; n++)
            *reinterpret_cast<__nv_bfloat162*>(dst + n * 8) =
                none ? __floats2bfloat162_rn(0.f, 0.f) : __floats2bfloat162_rn(o[n][half * 2] * inv, o[n][half * 2 + 1] * inv);
          if (a.lse && (lane & 3) == 0) a.lse[row] = none ? -INFINITY : (m[half] + log2f(l[half])) * 0.69314718055994531f;
        } else {
          const size_t row = (size_t)slot * R + r;
          float* dst = a.o_part + row * H + (lane & 3) * 2;
#pragma unroll
          for (int n = 0; n < NOT; n++) *reinterpret_cast<float2*>(dst + n * 8) = make_float2(o[n][half * 2], o[n][half * 2 + 1]);
          if ((lane & 3) == 0) a.ml[row] = make_float2(m[half], l[half]);
        }
      }
    }
    if (t0 == 0 && t1 < u.len()) left = make_int4(u.b, u.g, u.rt, last_run);
    __syncthreads();   // Q and the tiles are refilled for the next unit
  }
  if (tid == 0) a.desc[blockIdx.x] = left;
}

// The units that runs share: CTA (c, y) puts together rows of the unit that run c starts and leaves unfinished, from slots
// 2 c + 1, 2 (c + 1), .. in that order; a warp has RPW rows.  The partials are requested with their weights, not behind them.
constexpr int kMergeWarps = 4;
template <int H, int RPW>
__global__ void __launch_bounds__(kMergeWarps * 32) paged_merge_kernel(const __grid_constant__ Args p) {
  constexpr int DPL = H / 32, U = 8 / RPW;
  pdl_wait();
  pdl_trigger();
  const PagedAttn& a = p.a;
  const int c = blockIdx.x, lane = threadIdx.x & 31, R = p.s.rows, grp = p.s.grp;
  const int4 d = a.desc[c];
  const int r0 = (blockIdx.y * kMergeWarps + (threadIdx.x >> 5)) * RPW, rows = min(R, a.L * grp - d.z * R);
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
  for (int i0 = 0; i0 < pieces; i0 += U) {   // the softmax of the partials, U at a time
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
#pragma unroll
  for (int q = 0; q < RPW; q++) {
    if (r0 + q >= rows) break;
    const int qi = d.z * R + r0 + q, j = p.s.by_grp.div(qi);
    const bool none = den[q] == 0.f;
    const float by = 1.f / den[q];
    const size_t row = (size_t)(d.x * a.L + j) * a.nq + d.y * grp + qi - j * grp;
    bf16* dst = a.out + row * H + lane * DPL;
#pragma unroll
    for (int e = 0; e < DPL; e += 2)
      *reinterpret_cast<__nv_bfloat162*>(dst + e) = __floats2bfloat162_rn(none ? 0.f : num[q][e] * by, none ? 0.f : num[q][e + 1] * by);
    if (a.lse && lane == 0) a.lse[row] = none ? -INFINITY : (mx[q] + log2f(den[q])) * 0.69314718055994531f;
  }
}

template <int H, bool INT4>
auto mma_kernel(int rows) {
  return rows == 32 ? paged_mma_kernel<H, 2, INT4> : paged_mma_kernel<H, 4, INT4>;
}
template <int H>
size_t mma_smem(int rows) {
  return rows == 32 ? sizeof(Mem<H, 2>) : sizeof(Mem<H, 4>);
}

template <int H>
cudaError_t attributes() {
  for (int rows : {32, 64}) {
    cudaError_t e = cudaFuncSetAttribute(mma_kernel<H, false>(rows), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)mma_smem<H>(rows));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(mma_kernel<H, true>(rows), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)mma_smem<H>(rows));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int H>
cudaError_t launch(const Args& p, const PagedPlan& pl, cudaStream_t st) {
  cudaError_t e;
  if (pl.kernel == kPagedStream) {
    e = launch_paged_stream(p.a, p.s, pl, st);
  } else if (pl.kernel == kPagedTc) {
    e = launch_paged_tc(p.a, p.s, pl, st);
  } else {
    auto k = p.a.pg.format == FPD_PAGE_INT4 ? mma_kernel<H, true>(pl.rows) : mma_kernel<H, false>(pl.rows);
    e = launch_k(k, pl.runs, kThreads, mma_smem<H>(pl.rows), st, p);
  }
  if (e != cudaSuccess) return e;
  const int rows = std::min(pl.rows, p.a.L * p.s.grp);
  if (pl.kernel == kPagedStream) return launch_k(paged_merge_kernel<H, 1>, dim3(pl.runs, ceil_div(rows, kMergeWarps)), kMergeWarps * 32, 0, st, p);
  return launch_k(paged_merge_kernel<H, 2>, dim3(pl.runs, ceil_div(rows, 2 * kMergeWarps)), kMergeWarps * 32, 0, st, p);
}

}  // namespace

PagedPlan paged_attn_plan(int batch, int L, int nq, int nkv, int h, int format, int t_cap, int num_sms) {
  PagedPlan pl{};
  const int n = L * (nq / nkv);
  const int grp = nq / nkv;
  pl.kernel = n <= 16 ? kPagedStream : kPagedTc;
  pl.rows = n <= 8 ? 8 : n <= 16 ? 16 : 2 * (128 / grp * grp);
  pl.tiles = ceil_div(n, pl.rows);
  // no more runs than there can be tiles
  const long long most = (long long)batch * nkv * pl.tiles * (ceil_div(t_cap, kPagedTile) + ceil_div(L, kPagedTile));
  pl.runs = (int)std::min<long long>(most, (long long)num_sms * (pl.kernel == kPagedStream ? paged_stream_warps() : pl.kernel == kPagedTc ? 1 : 2));
  pl.grid = pl.kernel == kPagedStream ? std::min(num_sms, pl.runs) : pl.runs;
  return pl;
}

cudaError_t paged_attn_init_attributes() {
  cudaError_t e = attributes<128>();
  if (e == cudaSuccess) e = attributes<64>();
  if (e == cudaSuccess) e = paged_stream_init_attributes();
  return e != cudaSuccess ? e : paged_tc_init_attributes();
}

cudaError_t launch_paged_attention(const PagedAttn& a, const PagedPlan& pl, cudaStream_t st) {
  Args p;
  p.a = a;
  // positions stay below 2^30 + 2^26: a longer window hides nothing
  constexpr int kFar = 1200000000;
  p.s = paged_shape(a.L, a.lb, a.nq / a.pg.nkv, a.pg.nkv, pl.rows, a.window > kFar ? 0 : a.window, std::min(a.sinks, kFar), a.causal, KT);
  p.runs = pl.runs;
  return a.pg.h == 128 ? launch<128>(p, pl, st) : launch<64>(p, pl, st);
}

}  // namespace fpd
