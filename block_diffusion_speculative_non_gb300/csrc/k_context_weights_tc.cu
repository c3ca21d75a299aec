// k_context_weights_tc.cu — collected attention weight (k_context_weights.cu has the formula) on the 5th-generation tensor
// cores, for many query rows.
//
// Keys are the product's rows here as well: S^T = K Q^T with 128 keys in the 128 lanes of tensor memory and the query rows
// in its columns, so the sum over rows is a sum along one thread's registers.  A CTA takes units of 128 keys and runs all
// query rows of their request and kv head past them, 128 rows at a time, even tiles on one lane and odd ones on the other;
// each lane has two S buffers, so the next product runs while a tile is summed.  Per score: one product, one fma, one
// 2^x, one add: the special-function unit (32 a cycle) and the tensor core (128 x 128 x h in 512 cycles at h = 128) are
// about level.  Warps:
//   0      TMA producer of K (three units deep), 3: of Q (three tiles deep; a 4-d map of [request][position][head][h] whose
//          box is the kv head's heads, rows past the request's block come back as 0);
//   1      MMA issuer;
//   2      -lse log2(e) of a tile's rows into shared memory (-inf for rows without a key and past the last row: weight 0);
//   4..7   lane 0, 8..11 lane 1: a thread is a key.  Lane 1 hands its sum to lane 0, which writes: a fixed order.
#include <cstring>

#include "attn_tc_prims.cuh"
#include "fpd_context.cuh"

namespace fpd {

namespace {
using namespace attn_tc;

constexpr int KT = 128, QT = 128;
constexpr int kThreads = 12 * 32;
constexpr int RST = 3, LST = 8;          // K and Q ring slots, lse slots
constexpr int ATOM_BYTES = 128 * 64 * 2;
enum {
  B_KF = 0,
  B_KE = B_KF + RST,
  B_QF = B_KE + RST,
  B_QE = B_QF + RST,
  B_SF = B_QE + RST,     // [lane][buffer]
  B_SE = B_SF + 4,
  B_LF = B_SE + 4,
  B_LE = B_LF + LST,
  B_CF = B_LE + LST,     // lane 1's sums of a unit, [unit parity]
  B_CE = B_CF + 2,
  B_END = B_CE + 2,
  B_N = B_END + 1
};
template <int HD>
struct Lay {
  static constexpr int TILE = 128 * HD * 2, ATOMS = HD / 64;
  static constexpr int K = 0, Q = RST * TILE, L2 = Q + RST * TILE, COMB = L2 + LST * QT * 4, BAR = COMB + 2 * KT * 4;
  static constexpr size_t BYTES = 1024 + (size_t)BAR + 8 * B_N + 16;
  static_assert(BYTES <= 232448, "tile set exceeds the shared memory of one CTA");
};

struct WtArgs {
  CUtensorMap tm_k, tm_q;
  CtxWeights a;
  int grp, npt, rpt, nqt;   // heads per kv head, positions and rows of a query tile, tiles of a request
  int key_tiles, units;     // by capacity: units = batch * nkv * key_tiles
};

template <int HD>
__global__ void __launch_bounds__(kThreads, 1) weights_tc_kernel(const __grid_constant__ WtArgs p) {
  using S = Lay<HD>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* l2s = reinterpret_cast<float*>(smem + S::L2);
  float* comb = reinterpret_cast<float*>(smem + S::COMB);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + B_N);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t bar0 = tc::smem_u32(bars);
  auto bar = [&](int i) { return bar0 + 8 * i; };
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < RST; s++) {
      tc::mbar_init(bar(B_KF + s), 1);
      tc::mbar_init(bar(B_KE + s), 1);
      tc::mbar_init(bar(B_QF + s), 1);
      tc::mbar_init(bar(B_QE + s), 1);
    }
    for (int s = 0; s < 4; s++) {
      tc::mbar_init(bar(B_SF + s), 1);
      tc::mbar_init(bar(B_SE + s), 4);
    }
    for (int s = 0; s < LST; s++) {
      tc::mbar_init(bar(B_LF + s), 1);
      tc::mbar_init(bar(B_LE + s), 4);
    }
    for (int s = 0; s < 2; s++) {
      tc::mbar_init(bar(B_CF + s), 4);
      tc::mbar_init(bar(B_CE + s), 4);
    }
    tc::mbar_init(bar(B_END), 1);
    *abort_flag = 0;
    tc::fence_barrier_init();
  }
  // a query tile of fewer than 128 rows (heads per kv head that do not divide it) leaves the slots' last rows as they are now
  for (int i = threadIdx.x; i < RST * S::TILE / 16; i += kThreads)
    *reinterpret_cast<uint4*>(smem + S::Q + i * 16) = make_uint4(0, 0, 0, 0);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  if (warp == 1) {
    tc::tmem_alloc(tc::smem_u32(tmem_slot), 512);
    tc::tmem_relinquish();
  }
  __syncwarp();
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  pdl_wait();
  pdl_trigger();

  // this CTA's units that hold a key
  int u = (int)blockIdx.x - (int)gridDim.x, b = 0, g = 0, k0 = 0, T = 0;
  auto next = [&]() {
    for (u += gridDim.x; u < p.units; u += gridDim.x) {
      const int bg = u / p.key_tiles;
      b = bg / p.a.nkv;
      g = bg % p.a.nkv;
      k0 = (u % p.key_tiles) * KT;
      T = clamp_ctx(p.a.ctx_len[b], p.a.t_cap);
      if (k0 < T) return true;
    }
    return false;
  };
  const int nrows = p.a.L * p.grp;

  if (warp == 0 || warp == 3) {
    if (lane == 0) {
      const bool is_q = warp == 3;
      const int full = is_q ? B_QF : B_KF, empty = is_q ? B_QE : B_KE;
      const uint32_t ring = tc::smem_u32(smem + (is_q ? S::Q : S::K));
      int n = 0;
      while (!*abort_flag && next()) {
        for (int q = 0; q < (is_q ? p.nqt : 1) && !*abort_flag; q++) {
          const int s = n % RST;
          if (n >= RST && !wait_bar(bar(empty + s), ((n / RST) & 1) ^ 1)) { *abort_flag = 1; break; }
          tc::mbar_arrive_expect_tx(bar(full + s), is_q ? p.rpt * HD * 2 : S::TILE);
          for (int h = 0; h < S::ATOMS; h++) {
            const uint32_t dst = ring + s * S::TILE + h * ATOM_BYTES;
            if (is_q) tc::tma_load_4d(dst, &p.tm_q, h * 64, g * p.grp, q * p.npt, b, bar(full + s));
            else tc::tma_load_2d(dst, &p.tm_k, h * 64, (b * 2 * p.a.nkv + g) * p.a.t_cap + k0, bar(full + s));
          }
          n++;
        }
      }
      if (*abort_flag)   // a wait ran out: let the copies in flight land before the CTA's memory goes
        for (int i = max(0, n - RST); i < n; i++) tc::mbar_wait(bar(full + i % RST), (i / RST) & 1);
    }
  } else if (warp == 1) {
    const uint32_t on = elect_one();
    const uint64_t dk = tc::sw128_kmajor_desc(tc::smem_u32(smem + S::K)), dq = tc::sw128_kmajor_desc(tc::smem_u32(smem + S::Q));
    int nk = 0, nq = 0, nl[2] = {0, 0};
    auto uni = [&](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    bool ok = true;
    while (ok && !*abort_flag && next()) {
      if (!(ok = wait_bar(bar(B_KF + nk % RST), (nk / RST) & 1))) break;
      const int ks = uni(nk % RST);
      for (int q = 0; q < p.nqt && !*abort_flag; q++, nq++) {
        const int t = q & 1, buf = uni(nl[t] & 1), qs = uni(nq % RST);
        if (!(ok = wait_bar(bar(B_QF + qs), (nq / RST) & 1))) break;
        if (nl[t] >= 2 && !(ok = wait_bar(bar(B_SE + 2 * t + buf), ((nl[t] >> 1) & 1) ^ 1))) break;
        tc::tc_fence_after();
        const uint32_t id = idesc_bf16(KT, 32 * ceil_div(uni(min(p.rpt, nrows - q * p.rpt)), 32), 0);
        const uint64_t da = dk + ks * (S::TILE >> 4), db = dq + qs * (S::TILE >> 4);
        const uint32_t d = tmem + uni(t) * 256 + buf * 128;
#pragma unroll
        for (int kk = 0; kk < HD / 16; kk++) {
          const uint64_t step = ((kk >> 2) * ATOM_BYTES + (kk & 3) * 32) >> 4;
          umma_ss_if(on, d, da + step, db + step, id, kk > 0 ? 1u : 0u);
        }
        commit_if(on, bar(B_SF + 2 * t + buf));
        commit_if(on, bar(B_QE + qs));
        nl[t]++;
      }
      commit_if(on, bar(B_KE + ks));
      nk++;
    }
    if (!ok) *abort_flag = 1;
    // everything issued is done before tensor memory is freed (at once, unless a wait ran out)
    commit_if(on, bar(B_END));
    tc::mbar_wait(bar(B_END), 0);
  } else if (warp == 2) {
    // four tiles' values are read together, so that a read's latency is paid once per group
    int off[4], pos[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int r = i * 32 + lane;
      pos[i] = r < p.rpt ? r / p.grp : INT32_MAX / 2;
      off[i] = r / p.grp * p.a.nq + r % p.grp;
    }
    int n = 0;
    while (!*abort_flag && next()) {
      const float* src = p.a.lse + (size_t)b * p.a.L * p.a.nq + g * p.grp;
      for (int q0 = 0; q0 < p.nqt && !*abort_flag; q0 += 4) {
        float v[4][4];
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const int n0 = (q0 + j) * p.npt;
            v[j][i] = q0 + j < p.nqt && n0 + pos[i] < p.a.L ? src[(size_t)n0 * p.a.nq + off[i]] : -INFINITY;
          }
#pragma unroll
        for (int j = 0; j < 4; j++) {
          if (q0 + j >= p.nqt) break;
          const int s = n % LST;
          if (n >= LST && !wait_bar(bar(B_LE + s), ((n / LST) & 1) ^ 1)) *abort_flag = 1;
#pragma unroll
          for (int i = 0; i < 4; i++)
            l2s[s * QT + i * 32 + lane] = v[j][i] == -INFINITY ? -INFINITY : -v[j][i] * 1.4426950408889634f;
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(bar(B_LF + s));
          n++;
        }
      }
    }
  } else {
    const int t = (warp - 4) >> 2, quarter = warp & 3, key = quarter * 32 + lane;
    const float sl2 = rsqrtf((float)HD) * 1.4426950408889634f;
    const uint64_t sl22 = pack2(sl2, sl2);
    const uint32_t st = tmem + ((uint32_t)(quarter * 32) << 16) + t * 256;
    int n0 = 0, cnt = 0, nu = 0;
    while (!*abort_flag && next()) {
      float w = 0.f;
      for (int q = t; q < p.nqt && !*abort_flag; q += 2, cnt++) {
        const int buf = cnt & 1, s = (n0 + q) % LST, nv = min(p.rpt, nrows - q * p.rpt);
        if (!wait_bar(bar(B_SF + 2 * t + buf), (cnt >> 1) & 1)) *abort_flag = 1;
        tc::tc_fence_after();
        float sv[QT];
#pragma unroll
        for (int c = 0; c < QT; c += 32)
          if (c < nv) tmem_ld32_nowait(st + buf * 128 + c, sv + c);
#pragma unroll
        for (int c = 0; c < QT; c += 32)
          if (c < nv) wait_ld32(sv + c);
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(B_SE + 2 * t + buf));
        if (!wait_bar(bar(B_LF + s), ((n0 + q) / LST) & 1)) *abort_flag = 1;
        uint64_t acc[2] = {0ull, 0ull};   // this tile's share first: the long sum has one term per tile
#pragma unroll
        for (int c = 0; c < QT; c += 32) {
          if (c >= nv) continue;
#pragma unroll
          for (int e = c; e < c + 32; e += 4) {
            const ulonglong2 nl = *reinterpret_cast<const ulonglong2*>(l2s + s * QT + e);
            float x0, x1, x2, x3;
            unpack2(fma2(pack2(sv[e], sv[e + 1]), sl22, nl.x), x0, x1);
            unpack2(fma2(pack2(sv[e + 2], sv[e + 3]), sl22, nl.y), x2, x3);
            acc[0] = add2(acc[0], pack2(ex2(x0), ex2(x1)));
            acc[1] = add2(acc[1], pack2(ex2(x2), ex2(x3)));
          }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(B_LE + s));
        float a0, a1;
        unpack2(add2(acc[0], acc[1]), a0, a1);
        w += a0 + a1;
      }
      n0 += p.nqt;
      // lane 1's sums to lane 0, warp by warp
      const int cs = nu & 1;
      float* slot = comb + cs * KT + key;
      if (t == 1) {
        if (nu >= 2 && !wait_bar(bar(B_CE + cs), ((nu >> 1) & 1) ^ 1)) *abort_flag = 1;
        *slot = w;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(B_CF + cs));
      } else {
        if (!wait_bar(bar(B_CF + cs), (nu >> 1) & 1)) *abort_flag = 1;
        w += *slot;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(B_CE + cs));
        if (k0 + key < T && !*abort_flag) {
          float* dst = p.a.weights + ((size_t)b * p.a.nkv + g) * p.a.t_cap + k0 + key;
          *dst = p.a.accumulate ? *dst + w : w;
        }
      }
      nu++;
    }
  }

  __syncwarp();
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

}  // namespace

cudaError_t ctx_weights_tc_init_attributes() {
  cudaError_t e = cudaFuncSetAttribute(weights_tc_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Lay<128>::BYTES);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(weights_tc_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Lay<64>::BYTES);
  return e;
}

// A query tile is whole positions of the kv head's heads; tensor-map rows are 32-bit coordinates.
bool ctx_weights_tc_supported(const CtxWeights& a) {
  return a.nq / a.nkv <= QT && (long long)a.batch * 2 * a.nkv * a.t_cap < INT32_MAX;
}

cudaError_t launch_ctx_weights_tc(const CtxWeights& a, int num_sms, cudaStream_t st) {
  WtArgs p;
  memset(&p, 0, sizeof(p));
  p.a = a;
  p.grp = a.nq / a.nkv;
  p.npt = std::min(QT / p.grp, a.L);
  p.rpt = p.npt * p.grp;
  p.nqt = ceil_div(a.L, p.npt);
  p.key_tiles = ceil_div(a.t_cap, KT);
  p.units = a.batch * a.nkv * p.key_tiles;
  const uint64_t row = (uint64_t)a.h * 2;
  const uint64_t kd[2] = {(uint64_t)a.h, (uint64_t)a.batch * 2 * a.nkv * a.t_cap}, ks[1] = {row};
  const uint32_t kb[2] = {64u, (uint32_t)KT};
  cudaError_t e = make_tmap_nd(&p.tm_k, a.ck, 2, kd, ks, kb);
  const uint64_t qd[4] = {(uint64_t)a.h, (uint64_t)a.nq, (uint64_t)a.L, (uint64_t)a.batch};
  const uint64_t qs[3] = {row, row * a.nq, row * a.nq * a.L};
  const uint32_t qb[4] = {64u, (uint32_t)p.grp, (uint32_t)p.npt, 1u};
  if (e == cudaSuccess) e = make_tmap_nd(&p.tm_q, a.q, 4, qd, qs, qb);
  if (e != cudaSuccess) return e;
  const int grid = std::min(p.units, num_sms);
  return a.h == 128 ? launch_k(weights_tc_kernel<128>, grid, kThreads, Lay<128>::BYTES, st, p)
                    : launch_k(weights_tc_kernel<64>, grid, kThreads, Lay<64>::BYTES, st, p);
}

}  // namespace fpd
