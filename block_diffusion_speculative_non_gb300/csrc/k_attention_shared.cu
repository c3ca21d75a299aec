// k_attention_shared.cu — attention of a batch of blocks whose requests share a long context prefix:
//   out_r = sum_t exp(s_rt - lse_r) v_t,   s_rt = q_r . k_t / sqrt(h),   lse_r = log sum_t exp(s_rt)
// with t over [prefix ; the request's own context ; its block].
//
// The prefix is one request's K/V, so the query rows of ALL requests that use a kv head form the rows of one product:
// each prefix key is read once per kv head and row tile instead of once per request.  The own context and the block
// are the ordinary attention of one request.  Both parts leave unnormalised partials (o, m, l) per split of their keys;
// the softmax of a row is put together from them in split order (deterministic, no atomics).
//
// This file has the small form (mma.sync), the merge and the choice between the forms; k_attention_shared_tc.cu the large one.
// Bounds: per row and key 4 h flops (6 h with the weights as two bf16 terms), per key 4 h bytes once for up to 256 rows.  So
// few rows are a read of the keys, many rows tensor work, and small calls neither: launches and latency (4 tokens behind 512
// positions: 5.9 us on the GPU, half of it the merge).
#include <cmath>

#include "attn_body.cuh"
#include "fpd_context.cuh"

namespace fpd {

namespace {
using namespace attn;

// ---- work units -------------------------------------------------------------------------------------------------
// Unit u of the prefix part: (split, kv head, row tile), row tiles fastest, so that the CTAs which read the same keys
// run next to one another.  Own part: (split, request, kv head, row tile).
struct Unit {
  int b, g, qt, split;     // split: index among all partials of a row
  int n0, nrows;           // first row of the part in [rows], rows (position, head) of the part and kv head
  int T, n_keys;           // keys from the store, all keys
  int k_begin, k_end;
  const bf16 *kc, *vc, *kb, *vb;
};

// Cuts n_keys into `splits` runs of whole tiles as evenly as the tile count allows.
__device__ __forceinline__ void split_range(int n_keys, int splits, int s, int tile, int& k0, int& k1) {
  const long long nt = (n_keys + tile - 1) / tile;
  k0 = (int)(s * nt / splits) * tile;
  k1 = min(n_keys, (int)((s + 1) * nt / splits) * tile);
}

template <int H>
__device__ __forceinline__ Unit decode_unit(const SharedAttn& a, const SharedPlan& pl, bool prefix, int u, int tile) {
  Unit w;
  if (prefix) {
    w.qt = u % pl.pre_tiles;
    u /= pl.pre_tiles;
    w.g = u % a.nkv;
    const int s = u / a.nkv;
    w.b = 0;
    w.split = s;
    w.n0 = 0;
    w.nrows = a.rows * (a.nq / a.nkv);
    w.T = w.n_keys = clamp_ctx(a.prefix_len[0], a.p_cap);
    w.kc = a.pk + (size_t)w.g * a.p_cap * H;
    w.vc = a.pv + (size_t)w.g * a.p_cap * H;
    w.kb = w.vb = nullptr;
    split_range(w.n_keys, pl.pre_splits, s, tile, w.k_begin, w.k_end);
  } else {
    w.qt = u % pl.own_tiles;
    u /= pl.own_tiles;
    w.g = u % a.nkv;
    u /= a.nkv;
    w.b = u % a.batch;
    const int s = u / a.batch;
    w.split = pl.pre_splits + s;
    w.n0 = w.b * a.L;
    w.nrows = a.L * (a.nq / a.nkv);
    w.T = a.ck ? clamp_ctx(a.ctx_len[w.b], a.t_cap) : 0;
    w.n_keys = w.T + a.lb;
    const size_t off = ((size_t)w.b * 2 * a.nkv + w.g) * a.t_cap * H;
    w.kc = a.ck + off;
    w.vc = a.cv + off;
    const size_t boff = ((size_t)w.b * a.nkv + w.g) * a.lb * H;
    w.kb = a.kblk + boff;
    w.vb = a.vblk + boff;
    split_range(w.n_keys, pl.own_splits, s, tile, w.k_begin, w.k_end);
  }
  return w;
}

// One 64-row tile over one split on mma.sync (the tile math of attn_body.cuh).  Two CTAs of 80 KB per SM, two K/V buffers.
// Bound by the legacy matrix path: 64 blocks of 16 positions behind 16384 keys took 1240 us here, 0.22 PFLOP/s of the
// formula, and take 310 us on tcgen05; it stays for what is too small to notice.
template <int H>
__global__ void __launch_bounds__(NWARP * 32) shared_mma_kernel(const __grid_constant__ SharedAttn a, const __grid_constant__ SharedPlan pl,
                                                                int pre_units) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ __align__(128) unsigned char smem_raw[];
  constexpr int CH = H / 8, NKS = H / 16, NOT = H / 8;
  Smem<H>& sm = *reinterpret_cast<Smem<H>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool prefix = (int)blockIdx.x < pre_units;
  const Unit w = decode_unit<H>(a, pl, prefix, prefix ? blockIdx.x : blockIdx.x - pre_units, KT);
  const int grp = a.nq / a.nkv;
  const float sl2 = rsqrtf((float)H) * 1.4426950408889634f;

  const uint32_t q_s = smem_addr(sm.q);
  for (int idx = tid; idx < QT * CH; idx += NWARP * 32) {
    const int r = idx / CH, c = idx % CH, qi = w.qt * QT + r;
    const bool ok = qi < w.nrows;
    const bf16* src = a.q;
    if (ok) src = a.q + ((size_t)(w.n0 + qi / grp) * a.nq + w.g * grp + qi % grp) * H + c * 8;
    cp_async16(swz<H>(q_s, r, c), src, ok);
  }
  cp_async_commit();
  auto load_kv = [&](int buf, int k0) {
    const uint32_t ks = smem_addr(sm.k[buf]), vs = smem_addr(sm.v[buf]);
    for (int idx = tid; idx < KT * CH; idx += NWARP * 32) {
      const int r = idx / CH, c = idx % CH, t = k0 + r;
      const bool ok = t < w.k_end;
      const bf16 *ksrc = a.q, *vsrc = a.q;   // any mapped address: zero bytes are read when !ok
      if (ok) {
        ksrc = t < w.T ? w.kc + (size_t)t * H + c * 8 : w.kb + (size_t)(t - w.T) * H + c * 8;
        vsrc = t < w.T ? w.vc + (size_t)t * H + c * 8 : w.vb + (size_t)(t - w.T) * H + c * 8;
      }
      cp_async16(swz<H>(ks, r, c), ksrc, ok);
      cp_async16(swz<H>(vs, r, c), vsrc, ok);
    }
    cp_async_commit();
  };
  const int n_tiles = w.k_end > w.k_begin ? (w.k_end - w.k_begin + KT - 1) / KT : 0;
  if (n_tiles > 0) load_kv(0, w.k_begin);

  float o[NOT][4];
#pragma unroll
  for (int n = 0; n < NOT; n++) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
  uint32_t qf[NKS][4];
  if (n_tiles > 0)
    cp_async_wait<1>();
  else
    cp_async_wait<0>();
  __syncthreads();
  {
    const int r = warp * 16 + (lane & 15);
#pragma unroll
    for (int kk = 0; kk < NKS; kk++) ldsm_x4(swz<H>(q_s, r, kk * 2 + (lane >> 4)), qf[kk][0], qf[kk][1], qf[kk][2], qf[kk][3]);
  }
  for (int it = 0; it < n_tiles; it++) {
    const int buf = it & 1, k0 = w.k_begin + it * KT;
    if (it + 1 < n_tiles) {
      load_kv(buf ^ 1, k0 + KT);
      cp_async_wait<1>();
    } else {
      cp_async_wait<0>();
    }
    __syncthreads();
    attn_tile_math<H, KT, true>(smem_addr(sm.k[buf]), smem_addr(sm.v[buf]), qf, o, m0, m1, l0, l1, k0, w.k_end, lane, sl2);
    __syncthreads();
  }
  l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
  l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
#pragma unroll
  for (int half = 0; half < 2; half++) {
    const int qi = w.qt * QT + warp * 16 + (lane >> 2) + half * 8;
    if (qi >= w.nrows) continue;
    const size_t orow = (size_t)(w.n0 + qi / grp) * a.nq + w.g * grp + qi % grp;
    const size_t prow = (size_t)w.split * a.rows * a.nq + orow;
    const float m = half ? m1 : m0, l = half ? l1 : l0;
    if (n_tiles > 0) {
      float* dst = a.o_part + prow * H + (lane & 3) * 2;
#pragma unroll
      for (int n = 0; n < NOT; n++) *reinterpret_cast<float2*>(dst + n * 8) = make_float2(o[n][half * 2], o[n][half * 2 + 1]);
    }
    if ((lane & 3) == 0) a.ml[prow] = make_float2(m, l);
  }
}

// The softmax of one (row, head) from its partials: M = max m_s over the partials that hold a key (l_s != 0; a NaN sum
// counts, so that it reaches the output), den = sum l_s 2^(m_s - M), out = sum o_s 2^(m_s - M) / den,
// lse = (M + log2 den) ln 2.  W warps share an output and take every W-th partial, eight at a time, so that the reads of
// many partials do not queue behind one another; the warps' sums are added in warp order, so repeats
// of a call are bit-identical (other sizes, capacities or SM counts may cut the keys, and with them the sums, elsewhere).
template <int H, int W>
__global__ void __launch_bounds__(256) shared_merge_kernel(bf16* __restrict__ out, float* __restrict__ lse,
                                                           const float* __restrict__ o_part, const float2* __restrict__ ml,
                                                           int nsplit, int n_out) {
  pdl_wait();
  pdl_trigger();
  constexpr int DPL = H / 32;
  __shared__ float part[8][H];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w = warp % W;
  const int r = blockIdx.x * (8 / W) + warp / W;
  const bool ok = r < n_out;
  float mx = -INFINITY;
  for (int s0 = 0; ok && s0 < nsplit; s0 += 32) {
    const float2 v = s0 + lane < nsplit ? __ldcg(ml + (size_t)(s0 + lane) * n_out + r) : make_float2(-INFINITY, 0.f);
    mx = fmaxf(mx, warp_max(v.y == 0.f ? -INFINITY : v.x));
  }
  float den = 0.f, num[DPL];
#pragma unroll
  for (int e = 0; e < DPL; e++) num[e] = 0.f;
  for (int s0 = 0; ok && s0 < nsplit; s0 += 32) {
    const float2 v = s0 + lane < nsplit ? __ldcg(ml + (size_t)(s0 + lane) * n_out + r) : make_float2(-INFINITY, 0.f);
    const float wl = v.y == 0.f ? 0.f : exp2f(v.x - mx);   // lane s: weight of partial s0 + s
    den += warp_sum(v.y == 0.f ? 0.f : v.y * wl);
    const float* op = o_part + ((size_t)s0 * n_out + r) * H + lane * DPL;
    for (int u0 = w; u0 < min(32, nsplit - s0); u0 += 8 * W) {
      float t[8][DPL], wgt[8];
#pragma unroll
      for (int u = 0; u < 8; u++) {
        const int s = u0 + u * W;
        wgt[u] = __shfl_sync(0xffffffffu, wl, s & 31);
        if (s >= 32 || s0 + s >= nsplit) wgt[u] = 0.f;
#pragma unroll
        for (int e = 0; e < DPL; e++) t[u][e] = 0.f;
        if (wgt[u] != 0.f) {
          if constexpr (DPL == 4) {
            const float4 f = __ldcg(reinterpret_cast<const float4*>(op + (size_t)s * n_out * H));
            t[u][0] = f.x;
            t[u][1] = f.y;
            t[u][2] = f.z;
            t[u][3] = f.w;
          } else {
            const float2 f = __ldcg(reinterpret_cast<const float2*>(op + (size_t)s * n_out * H));
            t[u][0] = f.x;
            t[u][1] = f.y;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < 8; u++)
#pragma unroll
        for (int e = 0; e < DPL; e++) num[e] += wgt[u] != 0.f ? t[u][e] * wgt[u] : 0.f;
    }
  }
  if (W > 1) {
#pragma unroll
    for (int e = 0; e < DPL; e++) part[warp][lane * DPL + e] = num[e];
    __syncthreads();
    if (w != 0) return;
#pragma unroll
    for (int k = 1; k < W; k++)
#pragma unroll
      for (int e = 0; e < DPL; e++) num[e] += part[warp + k][lane * DPL + e];
  }
  if (!ok) return;
  const bool none = den == 0.f;   // no key at all (or every score -inf): output 0, lse -inf
  bf16* dst = out + (size_t)r * H + lane * DPL;
#pragma unroll
  for (int e = 0; e < DPL; e += 2)
    *reinterpret_cast<__nv_bfloat162*>(dst + e) =
        __floats2bfloat162_rn(none ? 0.f : num[e] / den, none ? 0.f : num[e + 1] / den);
  if (lse && lane == 0) lse[r] = none ? -INFINITY : (mx + log2f(den)) * 0.69314718055994531f;
}

// The same for up to 8 partials and many outputs: a warp puts together four consecutive ones, lane 8 i + s holding (m, l) of
// output i's partial s, so that one round trip brings the weights of four outputs and each of the next two the partials of
// two (one output per warp, three dependent round trips each, read the partials of 49280 outputs at 2 TB/s: 41 us).
template <int H>
__global__ void __launch_bounds__(256) shared_merge4_kernel(bf16* __restrict__ out, float* __restrict__ lse,
                                                            const float* __restrict__ o_part, const float2* __restrict__ ml,
                                                            int nsplit, int n_out) {
  pdl_wait();
  pdl_trigger();
  constexpr int DPL = H / 32;
  const int lane = threadIdx.x & 31, r0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * 4;
  if (r0 >= n_out) return;
  const int mine = r0 + (lane >> 3), s = lane & 7;
  const float2 v = s < nsplit && mine < n_out ? __ldcg(ml + (size_t)s * n_out + mine) : make_float2(-INFINITY, 0.f);
  float mx = v.y == 0.f ? -INFINITY : v.x;
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float wl = v.y == 0.f ? 0.f : exp2f(v.x - mx);
  float den = v.y == 0.f ? 0.f : v.y * wl;
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
  if (lse && s == 0 && mine < n_out) lse[mine] = den == 0.f ? -INFINITY : (mx + log2f(den)) * 0.69314718055994531f;
#pragma unroll 1
  for (int i0 = 0; i0 < 4; i0 += 2) {
    float t[2][8][DPL], wgt[2][8];
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
      for (int u = 0; u < 8; u++) {
        wgt[i][u] = __shfl_sync(0xffffffffu, wl, (i0 + i) * 8 + u);   // 0 past the last partial and the last output
#pragma unroll
        for (int e = 0; e < DPL; e++) t[i][u][e] = 0.f;
        if (wgt[i][u] != 0.f) {
          const float* op = o_part + ((size_t)u * n_out + r0 + i0 + i) * H + lane * DPL;
          if constexpr (DPL == 4) {
            const float4 f = __ldcg(reinterpret_cast<const float4*>(op));
            t[i][u][0] = f.x;
            t[i][u][1] = f.y;
            t[i][u][2] = f.z;
            t[i][u][3] = f.w;
          } else {
            const float2 f = __ldcg(reinterpret_cast<const float2*>(op));
            t[i][u][0] = f.x;
            t[i][u][1] = f.y;
          }
        }
      }
#pragma unroll
    for (int i = 0; i < 2; i++) {
      float num[DPL];
#pragma unroll
      for (int e = 0; e < DPL; e++) num[e] = 0.f;
#pragma unroll
      for (int u = 0; u < 8; u++)
#pragma unroll
        for (int e = 0; e < DPL; e++) num[e] += wgt[i][u] != 0.f ? t[i][u][e] * wgt[i][u] : 0.f;
      const float d = __shfl_sync(0xffffffffu, den, (i0 + i) * 8);
      if (r0 + i0 + i >= n_out) continue;
      const bool none = d == 0.f;
      bf16* dst = out + (size_t)(r0 + i0 + i) * H + lane * DPL;
#pragma unroll
      for (int e = 0; e < DPL; e += 2)
        *reinterpret_cast<__nv_bfloat162*>(dst + e) =
            __floats2bfloat162_rn(none ? 0.f : num[e] / d, none ? 0.f : num[e + 1] / d);
    }
  }
}

template <int H>
cudaError_t launch_merge(const SharedAttn& a, int nsplit, cudaStream_t st) {
  const int n_out = a.rows * a.nq;
  auto go = [&](auto* k, int per_cta) {
    return launch_k(k, ceil_div(n_out, per_cta), 256, 0, st, a.out, a.lse, (const float*)a.o_part, (const float2*)a.ml, nsplit, n_out);
  };
  // many outputs fill the GPU with one warp for one or four of them; up to 8 partials are one round of loads for a warp
  if (nsplit <= 8 && n_out >= 8192) return go(shared_merge4_kernel<H>, 32);
  if (nsplit <= 8 || n_out >= 65536) return go(shared_merge_kernel<H, 1>, 8);
  if (nsplit <= 16) return go(shared_merge_kernel<H, 2>, 4);
  return nsplit <= 32 ? go(shared_merge_kernel<H, 4>, 2) : go(shared_merge_kernel<H, 8>, 1);
}

__global__ void rope_base_kernel(int32_t* base, const int32_t* ctx_len, const int32_t* prefix_len, const int32_t* pos_offset,
                                 int batch, int t_cap, int p_cap) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= batch) return;
  const int off = pos_offset ? pos_offset[b] : (prefix_len ? clamp_ctx(prefix_len[0], p_cap) : 0);
  const int cl = ctx_len ? clamp_ctx(ctx_len[b], t_cap) : 0;
  base[b] = (off < 0 || off > INT32_MAX - cl) ? -1 : off + cl;
}

}  // namespace

// Split count of a part on the 64-row kernel, `base` row tiles times heads and kt key tiles each, for `slots` resident CTAs:
// the time is close to waves * (tiles per CTA + c), c what a CTA pays besides its tiles (Q, the partial out, its share
// of the merge); the smallest cost wins, ties to fewer splits.
static int mma_splits(long base, int kt, int slots) {
  double best = 0;
  int best_s = 1;
  for (int s = 1; s <= std::min(kt, 128); s = s < 16 ? s + 1 : s + s / 16) {
    const long units = base * s;
    const double cost = (units <= slots ? 1.0 : (double)units / slots) * (ceil_div(kt, s) + 2);
    if (s == 1 || cost < best) {
      best = cost;
      best_s = s;
    }
  }
  return best_s;
}

// Splits of both parts where the whole call is on the 64-row kernel, chosen together (units and kt as above; kt 0: no such
// part).  In key tiles, a split pays 3 besides its own; the call takes its longest split or 0.6 of the work over the resident
// CTAs, and 0.1 and one per 10^6 outputs for every partial that the merge reads.  Over 65 calls 4 % from the best of their
// combinations, 10 % with each part by itself (16 x 8 positions at h = 64 over 1500 and 300 keys 11.8 against 14.9 us).
struct MmaSplits {
  int pre = 0, own = 0;
  MmaSplits(long pre_units, int pre_kt, long own_units, int own_kt, double outputs, int slots) {
    struct Cut {
      int n;
      double tiles, work;
    } cut[2][16];
    int cuts[2] = {0, 0};
    auto list = [&](int part, long units, int kt) {
      if (!kt) {
        cut[part][cuts[part]++] = {0, 0, 0};
        return;
      }
      for (int s : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64, 96, 128, kt}) {
        if (s > std::min(kt, 128) || (cuts[part] && cut[part][cuts[part] - 1].n == s)) continue;
        const double t = ceil_div(kt, s) + 3;
        cut[part][cuts[part]++] = {s, t, (double)units * s * t};
      }
    };
    list(0, pre_units, pre_kt);
    list(1, own_units, own_kt);
    const double per_partial = 0.1 + 1e-6 * outputs;
    double best = 0;
    for (int i = 0; i < cuts[0]; i++)
      for (int j = 0; j < cuts[1]; j++) {
        const Cut &p = cut[0][i], &o = cut[1][j];
        const double t = std::max(std::max(p.tiles, o.tiles), 0.6 * (p.work + o.work) / slots) + (p.n + o.n) * per_partial;
        if ((i || j) && t >= best) continue;
        best = t;
        pre = p.n;
        own = o.n;
      }
  }
};

// How the tcgen05 kernel's CTAs share the prefix's key tiles (kt of each of `units` units) beside the own part's runs (segs of
// own_kt key tiles).  Either even runs, which may span units, or s runs per unit.  A run costs about kSeg us besides its
// tiles (Q, the first copies, the partial out); a partial is written and read once.  With many rows (pair) the time is the
// longest run's or, with the own part's runs, the average over the SMs.  A prefix under few rows is a read of its keys that
// does not need every SM: the CTAs without a run of the prefix take own runs meanwhile.
struct PrefixRuns {
  double us = 0;
  int runs = 0;      // CTAs that share the prefix
  int alone = 0;     // own runs that each of the others takes before all take turns
  double kSeg = 5.0, kOwn, kTile;
  PrefixRuns(bool pair, int h, long units, int kt, long segs, int own_kt, double part_us, double mem_us, int num_sms) {
    kOwn = h == 128 ? 1.1 : 1.0;
    kTile = pair ? (h == 128 ? 2.2 : 1.7) : kOwn;
    const double own_run = kSeg + 0.6 * kOwn * own_kt;   // contexts at 0.6 of what they may hold
    const long total = units * kt;
    auto with_own = [&](long r, double pre, long& first) {
      const long left = num_sms - r;
      double best = 0;
      for (long k = 0; k == 0 || (left > 0 && (k - 1) * own_run < pre && (k - 1) * left < segs); k++) {
        const long turns = segs > k * left ? ceil_div(segs - k * left, (long)num_sms) : 0;
        const double t = std::max(pre + turns * own_run, (k + turns) * own_run);
        if (k == 0 || t < best) {
          best = t;
          first = k;
        }
      }
      return best;
    };
    auto consider = [&](long r, double tiles, int n, double pieces) {
      const double pre = n * kSeg + std::max(kTile * tiles, mem_us);
      double t = pre;
      long first = 0;
      if (segs > num_sms - r || !pair) t = with_own(r, pre, first);
      if (segs && pair) t = std::max(pre, (r * pre + segs * (kSeg + kOwn * own_kt)) / num_sms);
      t += pieces * part_us;
      if (!runs || t < us) {
        us = t;
        runs = (int)r;
        alone = (int)first;
      }
    };
    for (long s = 1; s <= kt && (s == 1 || units * s <= num_sms); s++)
      if (units * s <= num_sms) consider(units * s, ceil_div(kt, (int)s), 1, s);
    for (int r = segs && !pair ? std::max(1, num_sms / 2) : num_sms;; r = std::min(r + 4, num_sms)) {
      if (total >= r) consider(r, (double)total / r, 2, (double)r / units + 1);
      if (r == num_sms) break;
    }
  }
};

SharedPlan shared_attn_plan(int batch, int L, int lb, int nq, int nkv, int h, int p_cap, int t_cap, int num_sms) {
  SharedPlan pl{};
  const int grp = nq / nkv, pre_rows = batch * L * grp, own_rows = L * grp, own_keys = t_cap + lb;
  // tcgen05 needs whole positions in 128 rows and tensor maps whose rows are 32-bit coordinates
  const int lane_rows = grp <= 128 ? 128 / grp * grp : 0;
  const bool own_tma = lane_rows && (long long)batch * 2 * nkv * t_cap < INT32_MAX && (long long)batch * nkv * lb < INT32_MAX;
  const bool pre_tma = lane_rows && (long long)2 * nkv * p_cap < INT32_MAX;
  // Up to 3.5 64 x 64 tiles of h = 128 per SM, or 13 of h = 64, the whole call goes to mma.sync, which has no tensor memory,
  // descriptors or rings to set up: 16 rows over 512 + 16 keys 8.6 against 11.4 us, 4 x 16 rows at h = 64 over 64 + 16 keys 5.9
  // against 9.4, 16 x 4 rows at h = 64 over 400 and 600 keys 13.1 against 15.6; above it tcgen05 wins (4 x 64 rows over 400 and 600
  // keys 17.9 against 23.6, 512 rows over 2048 24.5 against 43).  Over 554 calls 0.5 % from the better kernel on average.
  const long long tiles64 = (long long)nkv * ceil_div(pre_rows, QT) * ceil_div(p_cap, KT) +
                            (long long)nkv * batch * ceil_div(own_rows, QT) * ceil_div(own_keys, KT);
  const bool small = 2 * tiles64 <= (h == 128 ? 7ll : 26ll) * num_sms;
  pl.pre_tc = p_cap && pre_tma && !small;
  pl.own_tc = own_keys && own_tma && !small;
  pl.pre_tiles = p_cap ? ceil_div(pre_rows, pl.pre_tc ? 2 * lane_rows : QT) : 0;
  const long pre_units = (long)pl.pre_tiles * nkv;
  const int pre_kt = ceil_div(p_cap, 128), own_kt = ceil_div(t_cap, 128) + ceil_div(lb, 128);
  const bool pair = pre_rows > lane_rows;
  // us per partial of every row: written and read at 3 TB/s, and the merge's own step
  const double part_us = (double)batch * L * nq * h * 8 / 3e6 + (pair ? 0.2 : 0.4);
  auto prefix_runs = [&](long segs) {
    const double mem_us = pair ? 0.0 : 4.0 * h * nkv * p_cap / 6.7e6;
    return PrefixRuns(pair, h, pre_units, pre_kt, segs, own_kt, part_us, mem_us, num_sms);
  };
  if (pl.own_tc && own_rows <= QT) {
    // Own parts of at most one 64-row tile: a run each on tcgen05 beside the prefix's, with two partials, or a kernel of
    // mma.sync tiles before it (4 us, and 0.9 us a tile of 64 keys less 1 per unit and SM; h = 64: 0.7).  200 tokens behind 2048
    // positions: 62 against 106 us with contexts up to 60, 178 against 167 up to 1024; 64 of 4 positions behind 8192 80 against 89
    // up to 384; 64 of 16 171 against 190 up to 128, 238 against 214 up to 1500; 24 of 16 behind 1024 34 against 35 without
    // contexts, 57 against 41 up to 768.  Over 348 such calls the choice is on average 0.7 % from the better one.  Without a prefix
    // more than 32 rows of more than one unit per SM: 64 blocks of 16 with contexts up to 384 50 against 62 us, up to 1500 105
    // against 100.
    const double own_runs = (double)nkv * batch / num_sms, tiles = ceil_div(own_keys, KT);
    const int splits = mma_splits((long)nkv * batch, (int)tiles, 2 * num_sms);
    if (pl.pre_tc)
      pl.own_tc = prefix_runs(0).us + splits * part_us + 4 + own_runs * ((h == 128 ? 0.9 : 0.7) * tiles - 1) >=
                  prefix_runs((long)nkv * batch).us + 2 * part_us;
    else if (!p_cap)
      pl.own_tc = !(own_rows > 32 && own_runs > 1 && 0.9 * tiles < 7 + 0.9 * own_kt);
  }
  pl.own_tiles = own_keys ? ceil_div(own_rows, pl.own_tc ? 2 * lane_rows : QT) : 0;
  const long own_units = (long)pl.own_tiles * nkv * batch;
  if (pl.own_tiles && !pl.own_tc) pl.own_splits = mma_splits(own_units, ceil_div(own_keys, KT), 2 * num_sms);
  if (pl.pre_tiles && !pl.pre_tc) {
    const MmaSplits m(pre_units, ceil_div(p_cap, KT), own_units, pl.own_tc ? 0 : ceil_div(own_keys, KT), (double)batch * L * nq * h,
                      2 * num_sms);
    pl.pre_splits = m.pre;
    pl.own_splits = m.own;
  }
  if (pl.own_tc) {
    pl.own_splits = 2;
    if (!pl.pre_tc) pl.own_splits *= (int)std::max(1l, std::min<long>(own_kt / 2, num_sms / own_units));
  }
  const long own_segs = pl.own_tc ? own_units * (pl.own_splits / 2) : 0;
  if (pl.pre_tc) {
    const PrefixRuns pr = prefix_runs(own_segs);
    pl.pre_runs = pr.runs;
    pl.own_alone = pr.alone;
    const long total = pre_units * pre_kt;
    // a unit's tiles span at most ceil(runs / units) + 1 of the even runs (one less when the runs divide evenly), and no
    // more runs than it has tiles; a unit with one lane's rows leaves two partials per run
    pl.pre_pieces = (int)ceil_div(pl.pre_runs, (int)pre_units) + (pl.pre_runs % pre_units ? 1 : 0);
    if (own_segs && pl.pre_runs == num_sms && total >= 16l * num_sms) {
      // own runs are counted at about 0.6 of the tiles they may have; the kernel gives that up where shorter contexts would
      // leave more pieces than this
      const long even = own_segs / num_sms;
      const long w = std::min<long>((long)((pr.kSeg + 0.6 * pr.kOwn * own_kt) / pr.kTile + 0.5), total / (2l * num_sms * (even + 1) - own_segs));
      pl.own_cost = (int)w;
      const long shortest = (total + w * own_segs) / num_sms - 1 - w * (even + 1);
      pl.pre_pieces = std::max(pl.pre_pieces, (int)((pre_kt + shortest - 1) / shortest) + 1);
    }
    pl.pre_splits = pl.pre_pieces = std::min(pre_kt, pl.pre_pieces);
    if ((pre_rows - 1) % (2 * lane_rows) < lane_rows) pl.pre_splits *= 2;
  }
  if (pl.pre_tc || pl.own_tc) pl.tc_grid = (int)std::min<long>(num_sms, pl.pre_runs + own_segs);
  pl.own_ctas = pl.tc_grid - pl.pre_runs;
  return pl;
}

cudaError_t shared_attn_init_attributes() {
  cudaError_t e = cudaFuncSetAttribute(shared_mma_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)sizeof(Smem<128>));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(shared_mma_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem<64>));
  if (e == cudaSuccess) e = shared_attn_tc_init_attributes();
  return e;
}

cudaError_t launch_shared_attention(const SharedAttn& a, const SharedPlan& pl, cudaStream_t st) {
  const int pre_units = pl.pre_tc ? 0 : pl.pre_tiles * a.nkv * pl.pre_splits;
  const int units = pre_units + (pl.own_tc ? 0 : pl.own_tiles * a.nkv * a.batch * pl.own_splits);
  cudaError_t e = cudaSuccess;
  if (units > 0)
    e = a.h == 128 ? launch_k(shared_mma_kernel<128>, units, NWARP * 32, sizeof(Smem<128>), st, a, pl, pre_units)
                   : launch_k(shared_mma_kernel<64>, units, NWARP * 32, sizeof(Smem<64>), st, a, pl, pre_units);
  if (e == cudaSuccess && pl.tc_grid) e = launch_shared_tc(a, pl, st);
  if (e != cudaSuccess) return e;
  return a.h == 128 ? launch_merge<128>(a, pl.splits(), st) : launch_merge<64>(a, pl.splits(), st);
}

cudaError_t launch_rope_base(int32_t* base, const int32_t* ctx_len, const int32_t* prefix_len, const int32_t* pos_offset,
                             int batch, int t_cap, int p_cap, cudaStream_t st) {
  return launch_k(rope_base_kernel, ceil_div(batch, 128), 128, 0, st, base, ctx_len, prefix_len, pos_offset, batch, t_cap,
                  p_cap);
}

}  // namespace fpd
