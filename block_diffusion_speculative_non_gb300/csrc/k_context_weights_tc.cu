// k_context_weights_tc.cu — collected attention weight (k_context_weights.cu has the formula) on the 5th-generation tensor
// cores, for many query rows.
//
// Keys are the product's rows here as well: S^T = K Q^T with 128 keys in the 128 lanes of tensor memory and the query rows
// in its columns, so the sum over rows is a sum along one thread's registers.  A CTA takes an even share of all the key
// tiles that hold a key, two at a time where they belong to the same request and kv head: every query tile of 128 rows that
// passes is multiplied with both, and a thread sums both keys of its tensor-memory lane, so that a query tile's copy and a
// row's lse serve two keys (with one key tile per CTA the copies were 7.4 TB/s of L2 reads; with one key per thread the
// shared-memory reads of lse, which compete with the product's operands, cost 20 %).  S is double buffered: the next
// product runs while a tile is summed.  Per score: one product, one fma, one 2^x, one add.  Warps:
//   0      TMA producer of K (three tiles deep), 3: of Q (three tiles deep; a 4-d map of [request][position][head][h] whose
//          box is the kv head's heads, rows past the request's block come back as 0);
//   1      MMA issuer; it zeroes the query rows that warp 2 names before the tile's first product;
//   2      -lse log2(e) of a tile's rows into shared memory (-inf for rows without a key and past the last row: weight 0), and
//          which rows have no key: what such a row holds must not count, and NaN would pass through the -inf;
//   4..19  sums: warp = [32 of the tile's columns][32 of the keys].  The four parts of a key's sum are added in a fixed order.
//
// Measured: 4096 rows per kv head over 16384 keys, 8 kv heads: 129 us, 1.07 PFLOP/s (the floor is 72).  The sums bound it
// (issue slots 57 % busy, special-function unit 54 %); the products alone take 93.
#include <cstring>

#include "attn_tc_prims.cuh"
#include "fpd_context.cuh"
#include "weights_share.cuh"

namespace fpd {

namespace {
using namespace attn_tc;

constexpr int KT = kShareTile, QT = 128;
constexpr int kConsumers = 16;           // warps that sum
constexpr int kThreads = (4 + kConsumers) * 32;
constexpr int RST = 3, LST = 8;          // K and Q ring slots, lse slots
constexpr int ATOM_BYTES = 128 * 64 * 2;
enum {
  B_KF = 0,
  B_KE = B_KF + RST,
  B_QF = B_KE + RST,
  B_QE = B_QF + RST,
  B_SF = B_QE + RST,     // [buffer]
  B_SE = B_SF + 2,
  B_LF = B_SE + 2,
  B_LE = B_LF + LST,
  B_CF = B_LE + LST,     // sums of a unit to be put together, [unit parity]
  B_CE = B_CF + 2,
  B_END = B_CE + 2,
  B_N = B_END + 1
};
template <int HD>
struct Lay {
  static constexpr int TILE = 128 * HD * 2, ATOMS = HD / 64;
  static constexpr int K = 0, Q = RST * TILE, L2 = Q + RST * TILE, DEAD = L2 + LST * QT * 4, COMB = DEAD + LST * 4 * 4, BAR = COMB + 2 * 2 * 3 * KT * 4;
  static constexpr size_t BYTES = 1024 + (size_t)BAR + 8 * B_N + 16;
  static_assert(BYTES <= 232448, "tile set exceeds the shared memory of one CTA");
};

struct WtArgs {
  CUtensorMap tm_k, tm_q;
  CtxWeights a;
  int grp, npt, rpt, nqt;   // heads per kv head, positions and rows of a query tile, tiles of a request
};

struct CtxLen {
  const int32_t* ctx_len;
  int t_cap;
  __host__ __device__ int operator()(int b) const {
#ifdef __CUDA_ARCH__
    return clamp_ctx(ctx_len[b], t_cap);
#else
    return 0;   // device lengths
#endif
  }
};

// Zeroes the rows of a query tile whose bits are set, for the products that follow; by a whole warp.
template <int HD>
__device__ __noinline__ void zero_rows(uint8_t* tile, uint4 rows) {
  const int lane = threadIdx.x & 31, atom = lane >> 3, chunk = lane & 7;   // a row: 128 bytes in each 64-dim atom
  for (int r = 0; r < QT; r++) {
    const uint32_t word = r < 32 ? rows.x : r < 64 ? rows.y : r < 96 ? rows.z : rows.w;
    if (((word >> (r & 31)) & 1) && atom < HD / 64)
      *reinterpret_cast<uint4*>(tile + atom * ATOM_BYTES + r * 128 + chunk * 16) = make_uint4(0, 0, 0, 0);
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1) weights_tc_kernel(const __grid_constant__ WtArgs p) {
  using S = Lay<HD>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* l2s = reinterpret_cast<float*>(smem + S::L2);
  uint32_t* dead = reinterpret_cast<uint32_t*>(smem + S::DEAD);
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
    for (int s = 0; s < LST; s++) {
      tc::mbar_init(bar(B_LF + s), 1);
      tc::mbar_init(bar(B_LE + s), kConsumers);
    }
    for (int s = 0; s < 2; s++) {
      tc::mbar_init(bar(B_SF + s), 1);
      tc::mbar_init(bar(B_SE + s), kConsumers);
      tc::mbar_init(bar(B_CF + s), kConsumers);
      tc::mbar_init(bar(B_CE + s), kConsumers);
    }
    tc::mbar_init(bar(B_END), 1);
    *abort_flag = 0;
    tc::fence_barrier_init();
    tc::tma_prefetch(&p.tm_k);
    tc::tma_prefetch(&p.tm_q);
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

  Share<CtxLen> sh(CtxLen{p.a.ctx_len, p.a.t_cap}, p.a.batch, p.a.nkv, blockIdx.x, gridDim.x);
  const int nrows = p.a.L * p.grp;

  if (warp == 0 || warp == 3) {
    if (lane == 0) {
      const bool is_q = warp == 3;
      const int full = is_q ? B_QF : B_KF, empty = is_q ? B_QE : B_KE;
      const uint32_t ring = tc::smem_u32(smem + (is_q ? S::Q : S::K));
      int n = 0;
      while (!*abort_flag && sh.next()) {
        for (int q = 0; q < (is_q ? p.nqt : sh.nk) && !*abort_flag; q++) {
          const int s = n % RST;
          if (n >= RST && !wait_bar(bar(empty + s), ((n / RST) & 1) ^ 1)) { *abort_flag = 1; break; }
          tc::mbar_arrive_expect_tx(bar(full + s), is_q ? p.rpt * HD * 2 : S::TILE);
          for (int h = 0; h < S::ATOMS; h++) {
            const uint32_t dst = ring + s * S::TILE + h * ATOM_BYTES;
            if (is_q) tc::tma_load_4d(dst, &p.tm_q, h * 64, sh.g * p.grp, q * p.npt, sh.b, bar(full + s));
            else tc::tma_load_2d(dst, &p.tm_k, h * 64, (sh.b * 2 * p.a.nkv + sh.g) * p.a.t_cap + sh.k0 + q * KT, bar(full + s));
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
    int nk = 0, nq = 0;
    auto uni = [&](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    bool ok = true;
    while (ok && !*abort_flag && sh.next()) {
      const int nt = uni(sh.nk), k0s = uni(nk % RST), k1s = uni((nk + 1) % RST);
      ok = wait_bar(bar(B_KF + k0s), (nk / RST) & 1) && (nt < 2 || wait_bar(bar(B_KF + k1s), ((nk + 1) / RST) & 1));
      for (int q = 0; q < p.nqt && ok && !*abort_flag; q++, nq++) {
        const int qs = uni(nq % RST), buf = uni(nq & 1);
        // whole 32-column chunks: the sums read no column that the product has not written
        const uint32_t id = idesc_bf16(KT, 32 * ceil_div(uni(min(p.rpt, nrows - q * p.rpt)), 32), 0);
        if (!(ok = wait_bar(bar(B_QF + qs), (nq / RST) & 1) && wait_bar(bar(B_LF + nq % LST), (nq / LST) & 1))) break;
        const uint4 none = *reinterpret_cast<const uint4*>(dead + nq % LST * 4);
        if (none.x | none.y | none.z | none.w) zero_rows<HD>(smem + S::Q + qs * S::TILE, none);
        if (nq >= 2 && !(ok = wait_bar(bar(B_SE + buf), ((nq >> 1) & 1) ^ 1))) break;
        tc::tc_fence_after();
        const uint64_t db = dq + qs * (S::TILE >> 4);
#pragma unroll
        for (int t = 0; t < 2; t++) {
          if (t < nt) {
            const uint64_t da = dk + (t ? k1s : k0s) * (S::TILE >> 4);
#pragma unroll
            for (int kk = 0; kk < HD / 16; kk++) {
              const uint64_t step = ((kk >> 2) * ATOM_BYTES + (kk & 3) * 32) >> 4;
              umma_ss_if(on, tmem + t * 256 + buf * 128, da + step, db + step, id, kk > 0 ? 1u : 0u);
            }
          }
        }
        commit_if(on, bar(B_SF + buf));
        commit_if(on, bar(B_QE + qs));
      }
      commit_if(on, bar(B_KE + k0s));
      if (nt == 2) commit_if(on, bar(B_KE + k1s));
      nk += nt;
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
    while (!*abort_flag && sh.next()) {
      const float* src = p.a.lse + (size_t)sh.b * p.a.L * p.a.nq + sh.g * p.grp;
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
          for (int i = 0; i < 4; i++) {
            const bool none = v[j][i] == -INFINITY;
            l2s[s * QT + i * 32 + lane] = none ? -INFINITY : -v[j][i] * 1.4426950408889634f;
            const uint32_t rows = __ballot_sync(0xffffffffu, none && (q0 + j) * p.npt + pos[i] < p.a.L);
            if (lane == 0) dead[s * 4 + i] = rows;
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(bar(B_LF + s));
          n++;
        }
      }
    }
  } else {
    const int slice = (warp - 4) >> 2, quarter = warp & 3, key = quarter * 32 + lane;
    const float sl2 = rsqrtf((float)HD) * 1.4426950408889634f;
    const uint64_t sl22 = pack2(sl2, sl2);
    const uint32_t st = tmem + ((uint32_t)(quarter * 32) << 16) + slice * 32;
    int n = 0, nu = 0;   // query tiles and units so far
    while (!*abort_flag && sh.next()) {
      float w[2] = {0.f, 0.f};   // this lane's key of each tile
      for (int q = 0; q < p.nqt && !*abort_flag; q++, n++) {
        const int s = n % LST, buf = n & 1;
        const bool live = slice * 32 < min(p.rpt, nrows - q * p.rpt);
        if (!wait_bar(bar(B_LF + s), (n / LST) & 1)) *abort_flag = 1;
        if (!wait_bar(bar(B_SF + buf), (n >> 1) & 1)) *abort_flag = 1;
        tc::tc_fence_after();
        // this tile's share first: the long sum has one term per tile.  16 columns at a time: 32 of both keys would not
        // fit the 96 registers of 20 warps (the spills doubled the time)
        uint64_t a0[2] = {0ull, 0ull}, a1[2] = {0ull, 0ull};
#pragma unroll
        for (int c = 0; c < 32; c += 16) {
          float s0[16], s1[16];
          if (live) {
            tmem_ld16_nowait(st + buf * 128 + c, s0);
            tmem_ld16_nowait(st + 256 + buf * 128 + c, s1);   // of a single tile: whatever is there, not used
            wait_ld16(s0);
            wait_ld16(s1);
          }
          if (c == 16) {
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(bar(B_SE + buf));
          }
          if (!live) continue;
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const ulonglong2 nl = *reinterpret_cast<const ulonglong2*>(l2s + s * QT + slice * 32 + c + e);
            float x0, x1, x2, x3;
            unpack2(fma2(pack2(s0[e], s0[e + 1]), sl22, nl.x), x0, x1);
            unpack2(fma2(pack2(s0[e + 2], s0[e + 3]), sl22, nl.y), x2, x3);
            a0[0] = add2(a0[0], pack2(ex2(x0), ex2(x1)));
            a0[1] = add2(a0[1], pack2(ex2(x2), ex2(x3)));
            unpack2(fma2(pack2(s1[e], s1[e + 1]), sl22, nl.x), x0, x1);
            unpack2(fma2(pack2(s1[e + 2], s1[e + 3]), sl22, nl.y), x2, x3);
            a1[0] = add2(a1[0], pack2(ex2(x0), ex2(x1)));
            a1[1] = add2(a1[1], pack2(ex2(x2), ex2(x3)));
          }
        }
        float u, v;
        unpack2(add2(a0[0], a0[1]), u, v);
        w[0] += u + v;
        unpack2(add2(a1[0], a1[1]), u, v);
        w[1] += u + v;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(B_LE + s));
      }
      // the four column slices of a key's sum: the first one's warp adds and writes
      const int cs = nu & 1;
      float* slot = comb + cs * 6 * KT + key;
      if (nu >= 2 && !wait_bar(bar(B_CE + cs), ((nu >> 1) & 1) ^ 1)) *abort_flag = 1;
      if (slice > 0) {
        slot[(slice - 1) * 2 * KT] = w[0];
        slot[((slice - 1) * 2 + 1) * KT] = w[1];
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar(B_CF + cs));
      if (slice == 0) {
        if (!wait_bar(bar(B_CF + cs), (nu >> 1) & 1)) *abort_flag = 1;
        float* dst = p.a.weights + ((size_t)sh.b * p.a.nkv + sh.g) * p.a.t_cap + sh.k0 + key;
        for (int t = 0; t < sh.nk; t++, dst += KT) {
          const float sum = ((w[t] + slot[t * KT]) + slot[(2 + t) * KT]) + slot[(4 + t) * KT];
          if (sh.k0 + t * KT + key < sh.T && !*abort_flag) *dst = p.a.accumulate ? *dst + sum : sum;
        }
        __syncwarp();
      }
      if (lane == 0) tc::mbar_arrive(bar(B_CE + cs));
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
  const uint64_t row = (uint64_t)a.h * 2;
  const uint64_t kd[2] = {(uint64_t)a.h, (uint64_t)a.batch * 2 * a.nkv * a.t_cap}, ks[1] = {row};
  const uint32_t kb[2] = {64u, (uint32_t)KT};
  cudaError_t e = make_tmap_nd(&p.tm_k, a.ck, 2, kd, ks, kb);
  const uint64_t qd[4] = {(uint64_t)a.h, (uint64_t)a.nq, (uint64_t)a.L, (uint64_t)a.batch};
  const uint64_t qs[3] = {row, row * a.nq, row * a.nq * a.L};
  const uint32_t qb[4] = {64u, (uint32_t)p.grp, (uint32_t)p.npt, 1u};
  if (e == cudaSuccess) e = make_tmap_nd(&p.tm_q, a.q, 4, qd, qs, qb);
  if (e != cudaSuccess) return e;
  const int grid = (int)std::min<long long>((long long)a.batch * a.nkv * ceil_div(a.t_cap, KT), num_sms);
  return a.h == 128 ? launch_k(weights_tc_kernel<128>, grid, kThreads, Lay<128>::BYTES, st, p)
                    : launch_k(weights_tc_kernel<64>, grid, kThreads, Lay<64>::BYTES, st, p);
}

}  // namespace fpd
