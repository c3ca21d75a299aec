// k_context_weights.cu — the attention weight that each stored context position collects from a block's queries:
//   weights[b][g][t] (+)= sum over the rows r of request b in kv head g of exp(q_r . k_t / sqrt(h) - lse_r)
// with lse_r the attention's own log-sum-exp, so that every row hands out a total weight of 1 over all its keys.
//
// The sum runs over the query rows of one key, so keys take the product's row side: a warp holds 16 keys as A
// fragments for the whole kernel and streams the query rows past them; the exponentials of a key stay in the quad of
// lanes that owns it, and no intermediate leaves the registers.  One CTA owns its keys: no atomics, a fixed order.
//
// Bounds: 2 h flops and one 2^x per row and key, 2 h bytes per key.  This small form is latency (16 rows over 128 keys:
// 2.6 us); with many rows it is held back by the legacy matrix path and by reading the queries once per 64 keys (4096 rows
// over 16384 keys 855 us against 129 on tcgen05).
#include <algorithm>
#include <cfloat>

#include "attn_body.cuh"
#include "fpd_context.cuh"

namespace fpd {

namespace {
using namespace attn;

template <int H>
struct WeightSmem {
  bf16 k[KT * H];
  bf16 q[2][QT * H];
  float l2[2][QT];   // lse log2(e) of the rows; -inf (rows that hold no key and past the last row): weight 0, whatever their score
};

template <int H>
__global__ void __launch_bounds__(NWARP * 32) weights_mma_kernel(const __grid_constant__ CtxWeights a, int key_tiles) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ __align__(128) unsigned char smem_raw[];
  constexpr int CH = H / 8, NKS = H / 16;
  WeightSmem<H>& sm = *reinterpret_cast<WeightSmem<H>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bg = blockIdx.x / key_tiles, k0 = (int)(blockIdx.x % key_tiles) * KT;
  const int b = bg / a.nkv, g = bg % a.nkv, grp = a.nq / a.nkv, nrows = a.L * grp;
  const int T = clamp_ctx(a.ctx_len[b], a.t_cap);
  if (k0 >= T) return;
  const float log2e = 1.4426950408889634f, sl2 = rsqrtf((float)H) * log2e;
  const bf16* kc = a.ck + ((size_t)b * 2 * a.nkv + g) * a.t_cap * H;
  for (int idx = tid; idx < KT * CH; idx += NWARP * 32) {
    const int r = idx / CH, c = idx % CH;
    const bool ok = k0 + r < T;
    cp_async16(swz<H>(smem_addr(sm.k), r, c), ok ? kc + (size_t)(k0 + r) * H + c * 8 : kc, ok);
  }
  auto load_q = [&](int buf, int r0) {
    for (int idx = tid; idx < QT * CH; idx += NWARP * 32) {
      const int r = idx / CH, c = idx % CH, qi = r0 + r;
      const bool ok = qi < nrows;
      const bf16* src = a.q;
      if (ok) src = a.q + (((size_t)b * a.L + qi / grp) * a.nq + g * grp + qi % grp) * H + c * 8;
      cp_async16(swz<H>(smem_addr(sm.q[buf]), r, c), src, ok);
    }
    if (tid < QT) {
      const int qi = r0 + tid;
      float v = -INFINITY;
      if (qi < nrows) {
        const float lse = a.lse[((size_t)b * a.L + qi / grp) * a.nq + g * grp + qi % grp];
        v = lse * log2e;
        if (v == -INFINITY && lse != v) v = -FLT_MAX;   // a finite lse that overflows here is a row that has keys
      }
      sm.l2[buf][tid] = v;
    }
    cp_async_commit();
  };
  load_q(0, 0);
  const int nt = ceil_div(nrows, QT);
  uint32_t kf[NKS][4];
  float w0 = 0.f, w1 = 0.f;   // keys warp * 16 + lane / 4 and + 8: this lane's columns
  for (int it = 0; it < nt; it++) {
    const int buf = it & 1;
    if (it + 1 < nt) {
      load_q(buf ^ 1, (it + 1) * QT);
      cp_async_wait<1>();
    } else {
      cp_async_wait<0>();
    }
    __syncthreads();
    if (it == 0) {
      const int r = warp * 16 + (lane & 15);
#pragma unroll
      for (int kk = 0; kk < NKS; kk++)
        ldsm_x4(swz<H>(smem_addr(sm.k), r, kk * 2 + (lane >> 4)), kf[kk][0], kf[kk][1], kf[kk][2], kf[kk][3]);
    }
    float t0 = 0.f, t1 = 0.f;   // this tile's share first: the long sum has one term per tile
#pragma unroll
    for (int np = 0; np < QT / 16; np++) {
      float s[2][4] = {};
#pragma unroll
      for (int kk = 0; kk < NKS; kk++) {
        const int row = np * 16 + (lane & 7) + ((lane >> 4) << 3), c = kk * 2 + ((lane >> 3) & 1);
        uint32_t b0, b1, b2, b3;
        ldsm_x4(swz<H>(smem_addr(sm.q[buf]), row, c), b0, b1, b2, b3);
        mma_bf16(s[0], kf[kk][0], kf[kk][1], kf[kk][2], kf[kk][3], b0, b1);
        mma_bf16(s[1], kf[kk][0], kf[kk][1], kf[kk][2], kf[kk][3], b2, b3);
      }
#pragma unroll
      for (int e = 0; e < 2; e++) {
        const float2 l = *reinterpret_cast<const float2*>(&sm.l2[buf][np * 16 + e * 8 + (lane & 3) * 2]);
        const bool x = l.x != -INFINITY, y = l.y != -INFINITY;
        t0 += (x ? ex2_approx(fmaf(s[e][0], sl2, -l.x)) : 0.f) + (y ? ex2_approx(fmaf(s[e][1], sl2, -l.y)) : 0.f);
        t1 += (x ? ex2_approx(fmaf(s[e][2], sl2, -l.x)) : 0.f) + (y ? ex2_approx(fmaf(s[e][3], sl2, -l.y)) : 0.f);
      }
    }
    w0 += t0;
    w1 += t1;
    __syncthreads();
  }
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    w0 += __shfl_xor_sync(0xffffffffu, w0, o);
    w1 += __shfl_xor_sync(0xffffffffu, w1, o);
  }
  if ((lane & 3) == 0) {
    float* dst = a.weights + ((size_t)b * a.nkv + g) * a.t_cap;
    const int t = k0 + warp * 16 + (lane >> 2);
    if (t < T) dst[t] = a.accumulate ? dst[t] + w0 : w0;
    if (t + 8 < T) dst[t + 8] = a.accumulate ? dst[t + 8] + w1 : w1;
  }
}

}  // namespace

cudaError_t ctx_weights_init_attributes() {
  cudaError_t e = cudaFuncSetAttribute(weights_mma_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)sizeof(WeightSmem<128>));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(weights_mma_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(WeightSmem<64>));
  if (e == cudaSuccess) e = ctx_weights_tc_init_attributes();
  return e;
}

cudaError_t launch_ctx_weights(const CtxWeights& a, int num_sms, cudaStream_t st) {
  // The kernel whose time (us, fitted to 276 calls) is the smaller: on average 0.5 % from the better one over 476.  mma.sync: a
  // CTA's row tiles in turn, and the SM's share of all tiles.  tcgen05: tensor memory to set up, the query tiles in turn, the
  // SM's share of the key tiles, and a step from one head's keys to the next.  (16 positions, 8 kv heads: 8192 keys 8.2 on
  // tcgen05 against 12.5, 2048 keys 5.4 on mma.sync against 6.3; 64 requests of 512 keys at h = 64 13.9 on mma.sync against
  // 18.4.)
  const int grp = a.nq / a.nkv, rt = ceil_div(a.L * grp, QT);
  if (ctx_weights_tc_supported(a)) {
    const bool wide = a.h == 128;
    const int nqt = ceil_div(a.L, std::min(128 / grp, a.L));
    const double heads = (double)a.batch * a.nkv / num_sms;
    const double mma_us = 2 + (wide ? 1.7 : 1.15) * rt + heads * ceil_div(a.t_cap, KT) * (0.12 + (wide ? 0.5 : 0.25) * rt);
    const double tc_us = 5 + 0.8 * nqt + heads * (ceil_div(a.t_cap, 128) * ((wide ? 0.28 : 0.15) + 0.27 * nqt) + 2.1);
    if (tc_us < mma_us) return launch_ctx_weights_tc(a, num_sms, st);
  }
  const int key_tiles = ceil_div(a.t_cap, KT);
  const int grid = a.batch * a.nkv * key_tiles;
  return a.h == 128 ? launch_k(weights_mma_kernel<128>, grid, NWARP * 32, sizeof(WeightSmem<128>), st, a, key_tiles)
                    : launch_k(weights_mma_kernel<64>, grid, NWARP * 32, sizeof(WeightSmem<64>), st, a, key_tiles);
}

}  // namespace fpd
