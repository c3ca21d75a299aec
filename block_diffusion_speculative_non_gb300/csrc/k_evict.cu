// k_evict.cu — eviction from a context store by collected attention weight: of the T positions of a (layer, request,
// kv head) keep the last `recent` ones and, of the others, the `budget - recent` with the largest weight (ties: the
// lower position), in the order of their positions.
//
// Two kernels.  evict_select_kernel: one CTA per (layer, request, kv head) finds the smallest kept weight and turns it into
// the list of kept positions with one ordered scan; it also moves the weights.  The weight is found by radix selection on
// an order-preserving integer key (11 + 11 + 10 bits, shared-memory histograms); up to 256 positions are ranked directly
// instead, four threads a position.
// evict_copy_kernel / evict_inplace_kernel: the kept K and V rows.  The result is a function of the inputs alone (integer
// counts, fixed order).
//
// Bound by HBM: every kept row once in and once out, every weight once in.  8 ragged contexts of up to 16384 positions in
// five layers to 4096: 208 us where 182 is the floor, the copy at 5.9 TB/s and 20 to 30 us of selection before it (issue
// slots: about ten instructions per weight and pass, five passes); 2048 positions to 1024: 19 us, half of it the selection's
// chain of barriers.
#include "fpd_context.cuh"

namespace fpd {

namespace {

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kStage = 16 * kSelThreads;           // weights held in shared memory at a time: 16 rows of 32 per warp
constexpr int kBins = 2048;
constexpr int kRank = 256;

struct SelSmem {
  float stage[kStage];
  uint32_t hist[kBins];
  uint64_t warp_sum[kSelWarps];
  uint32_t bin, below;
};

// Larger weight, larger key; -0 counts as 0, and NaN below everything.
__device__ __forceinline__ uint32_t weight_key(float v) {
  if (v != v) return 0u;
  const uint32_t u = __float_as_uint(v == 0.f ? 0.f : v);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive sum over the CTA's threads, and the total.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* warp_sum, uint64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  __syncthreads();   // warp_sum may still be read from the previous scan
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    uint64_t w = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t t = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += t;
    }
    warp_sum[lane] = w;
  }
  __syncthreads();
  total = warp_sum[31];
  return inc - v + (warp ? warp_sum[warp - 1] : 0);
}

// 32 registers a thread, so that two CTAs share an SM: this kernel is a chain of short steps between barriers.  Loops are
// left rolled: a small context makes one short pass through the code, and unrolled loops made that pass slower.
__global__ void __launch_bounds__(kSelThreads, 2) evict_select_kernel(const __grid_constant__ Evict e) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ __align__(16) unsigned char smem_raw[];
  SelSmem& sm = *reinterpret_cast<SelSmem*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, head = blockIdx.x, b = (head / e.nkv) % e.batch;
  const float* w = e.weights + (size_t)head * e.t_cap;
  for (int i = tid; i < kBins; i += kSelThreads) sm.hist[i] = 0;
  const int T = clamp_ctx(e.ctx_len[b], e.t_cap), m = min(T, e.budget);
  if (tid == 0 && head < e.batch * e.nkv && head % e.nkv == 0) e.old_len[b] = T;   // layer 0, kv head 0 of each request
  const int old = T > e.budget ? T - e.recent : 0;   // positions that compete; below the budget all stay
  const int need = T > e.budget ? e.budget - e.recent : 0;
  const bool staged = T <= kStage, ranked = T <= kRank;
  __syncthreads();
  if (staged) {   // the weights, and the histogram of their keys' upper bits on the way
#pragma unroll 4
    for (int p = tid; p < T; p += kSelThreads) {
      const float v = w[p];
      sm.stage[p] = v;
      if (p < old) {
        if (ranked) sm.hist[p] = weight_key(v);   // up to 256 keys, 0 behind them
        else atomicAdd(&sm.hist[weight_key(v) >> 21], 1u);
      }
    }
    __syncthreads();
  }
  // ---- the need-th largest key: `thr`, of which the first `ties` positions stay ----
  uint32_t thr = 0xFFFFFFFFu;
  int ties = 0;
  if (need > 0 && ranked) {
    const int p = tid >> 2, part = tid & 3;
    if (warp * 8 < old) {
      const uint32_t k = sm.hist[p];
      int greater = 0, before = 0;
      for (int q = part * 4; q < old; q += 16) {
        const uint4 o = *reinterpret_cast<const uint4*>(sm.hist + q);
        greater += (o.x > k) + (o.y > k) + (o.z > k) + (o.w > k);
        before += (o.x == k && q < p) + (o.y == k && q + 1 < p) + (o.z == k && q + 2 < p) + (o.w == k && q + 3 < p);
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        greater += __shfl_xor_sync(0xffffffffu, greater, o);
        before += __shfl_xor_sync(0xffffffffu, before, o);
      }
      if (part == 0 && p < old && greater + before == need - 1) {   // exactly one position has this rank
        sm.bin = k;
        sm.below = need - greater;
      }
    }
    __syncthreads();
    thr = sm.bin;
    ties = (int)sm.below;
  } else if (need > 0) {
    uint32_t prefix = 0;
    int rest = need;
#pragma unroll 1
    for (int pass = 0; pass < 3; pass++) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
      if (pass > 0 || !staged)
        for (int p = tid; p < old; p += kSelThreads) {
          const uint32_t k = weight_key(staged ? sm.stage[p] : w[p]);
          if (pass == 0 || (k >> (shift + bits)) == prefix) atomicAdd(&sm.hist[(k >> shift) & ((1u << bits) - 1)], 1u);
        }
      __syncthreads();
      // thread t owns bins kBins - 1 - 2 t and the one below: sums run from the largest key down
      const int hi = kBins - 1 - 2 * tid;
      const uint32_t c1 = sm.hist[hi], c0 = sm.hist[hi - 1];
      sm.hist[hi] = sm.hist[hi - 1] = 0;   // for the next pass
      uint64_t total;
      const uint32_t above = (uint32_t)block_scan(c1 + c0, sm.warp_sum, total);
      if (above < (uint32_t)rest && above + c1 + c0 >= (uint32_t)rest) {
        const bool first = above + c1 >= (uint32_t)rest;
        sm.bin = first ? hi : hi - 1;
        sm.below = first ? above : above + c1;
      }
      __syncthreads();
      prefix = (prefix << bits) | sm.bin;
      rest -= (int)sm.below;
    }
    thr = prefix;
    ties = rest;
  }
  // ---- ordered list of the kept positions, the weights moved along ----
  // A warp takes up to 16 rows of 32 consecutive positions; lane i keeps row i's masks of the positions that stay outright
  // and of those equal to thr, whose turn the counts before them decide.
  float* ow = e.out_weights + (size_t)head * e.out_cap;
  int32_t* kept = e.kept + (size_t)head * e.budget;
  uint64_t base = 0;   // kept outright so far | equal to thr so far << 32
#pragma unroll 1
  for (int c0 = 0; c0 < T; c0 += kStage) {
    const int n = min(kStage, T - c0);
    if (!staged) {
      __syncthreads();
#pragma unroll 4
      for (int p = tid; p < n; p += kSelThreads) sm.stage[p] = w[c0 + p];
      __syncthreads();
    }
    const int rows = (n + kSelThreads - 1) / kSelThreads, r0 = warp * rows * 32;
    uint32_t my_sure = 0, my_tie = 0;
    for (int i = 0; i < rows && r0 + i * 32 < n; i++) {
      const int at = r0 + i * 32 + lane, p = c0 + at;
      const uint32_t k = at < n ? weight_key(sm.stage[at]) : 0u;
      const uint32_t sure = __ballot_sync(0xffffffffu, at < n && (p >= old || k > thr));
      const uint32_t tie = __ballot_sync(0xffffffffu, at < n && p < old && k == thr && need > 0);
      if (lane == i) {
        my_sure = sure;
        my_tie = tie;
      }
    }
    uint64_t total;
    const uint64_t before =
        base + block_scan((uint64_t)__popc(my_sure) | ((uint64_t)__popc(my_tie) << 32), sm.warp_sum, total);
    // in place, slot i of this chunk is at or before its position: every weight it can overwrite has been staged
    for (int i = 0; i < rows && r0 + i * 32 < n; i++) {
      const uint32_t sure = __shfl_sync(0xffffffffu, my_sure, i), tie = __shfl_sync(0xffffffffu, my_tie, i);
      const uint64_t bf = __shfl_sync(0xffffffffu, before, i);
      const uint32_t lt = (1u << lane) - 1;
      const int at_tie = (int)(bf >> 32) + __popc(tie & lt);
      if (((sure >> lane) & 1) || (((tie >> lane) & 1) && at_tie < ties)) {
        const int slot = (int)(uint32_t)bf + __popc(sure & lt) + min(at_tie, ties);
        kept[slot] = c0 + r0 + i * 32 + lane;
        ow[slot] = sm.stage[r0 + i * 32 + lane];
      }
    }
    base += total;
  }
  for (int i = m + tid; i < e.budget; i += kSelThreads) kept[i] = -1;
  __syncthreads();
  for (int i = m + tid; i < e.out_cap; i += kSelThreads) ow[i] = 0.f;
}

constexpr int kMoveThreads = 256, kMoveRows = 64;

// Into another store: 64 kept rows of one (layer, request, K|V, kv head) per CTA, 16 bytes per thread and load.
template <int CH>   // 16-byte chunks per row
__global__ void __launch_bounds__(kMoveThreads) evict_copy_kernel(const __grid_constant__ Evict e, int chunks) {
  pdl_wait();
  pdl_trigger();
  constexpr int PER = kMoveRows * CH / kMoveThreads;
  const int hk = blockIdx.x / chunks, i0 = (int)(blockIdx.x % chunks) * kMoveRows;   // [layer][request][K|V][kv head]
  const int g = hk % e.nkv, lb = hk / e.nkv / 2, b = lb % e.batch;
  const int T = e.old_len[b], m = min(T, e.budget);
  if (blockIdx.x == 0)
    for (int r = threadIdx.x; r < e.batch; r += kMoveThreads) {
      const int t = e.old_len[r], n = min(t, e.budget);
      e.out_len[r] = n;
      if (e.pos_offset) e.pos_offset[r] += t - n;
    }
  const int32_t* kept = e.kept + ((size_t)lb * e.nkv + g) * e.budget;
  const uint4* src = reinterpret_cast<const uint4*>(e.store) + (size_t)hk * e.t_cap * CH;
  uint4* dst = reinterpret_cast<uint4*>(e.out_store) + (size_t)hk * e.out_cap * CH;
  uint4 v[PER];
#pragma unroll
  for (int u = 0; u < PER; u++) {
    const int idx = threadIdx.x + u * kMoveThreads, i = i0 + idx / CH;
    if (i < m) v[u] = src[(size_t)kept[i] * CH + idx % CH];
  }
#pragma unroll
  for (int u = 0; u < PER; u++) {
    const int idx = threadIdx.x + u * kMoveThreads, i = i0 + idx / CH;
    if (i < m) dst[(size_t)i * CH + idx % CH] = v[u];
  }
}

// In place: slot i takes a row from position kept[i] >= i.  One CTA walks all slots of a 64-byte column slab of one
// (layer, request, K|V, kv head) in ascending steps: it holds a step's rows in registers before it writes them, and a
// later step reads only positions behind every slot written so far.
constexpr int kSlabChunks = 4, kInThreads = 512, kInPer = 4;
template <int CH>
__global__ void __launch_bounds__(kInThreads) evict_inplace_kernel(const __grid_constant__ Evict e) {
  pdl_wait();
  pdl_trigger();
  constexpr int SLABS = CH / kSlabChunks, ROWS = kInThreads / kSlabChunks;
  const int hk = blockIdx.x / SLABS, slab = blockIdx.x % SLABS;
  const int g = hk % e.nkv, lb = hk / e.nkv / 2, b = lb % e.batch;
  const int T = e.old_len[b], m = min(T, e.budget);
  if (blockIdx.x == 0)
    for (int r = threadIdx.x; r < e.batch; r += kInThreads) {
      const int t = e.old_len[r], n = min(t, e.budget);
      e.out_len[r] = n;
      if (e.pos_offset) e.pos_offset[r] += t - n;
    }
  if (T <= e.budget) return;   // nothing moves
  const int32_t* kept = e.kept + ((size_t)lb * e.nkv + g) * e.budget;
  uint4* row = reinterpret_cast<uint4*>(e.out_store) + (size_t)hk * e.t_cap * CH + slab * kSlabChunks + threadIdx.x % kSlabChunks;
  for (int i0 = 0; i0 < m; i0 += ROWS * kInPer) {
    uint4 v[kInPer];
#pragma unroll
    for (int u = 0; u < kInPer; u++) {
      const int i = i0 + u * ROWS + threadIdx.x / kSlabChunks;
      if (i < m) v[u] = row[(size_t)kept[i] * CH];
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kInPer; u++) {
      const int i = i0 + u * ROWS + threadIdx.x / kSlabChunks;
      if (i < m) row[(size_t)i * CH] = v[u];
    }
  }
}

}  // namespace

cudaError_t evict_init_attributes() {
  return cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(SelSmem));
}

cudaError_t launch_evict(const Evict& e, cudaStream_t st) {
  const int heads = e.layers * e.batch * e.nkv;
  cudaError_t err = launch_k(evict_select_kernel, heads, kSelThreads, sizeof(SelSmem), st, e);
  if (err != cudaSuccess) return err;
  if (e.in_place)
    return e.h == 128 ? launch_k(evict_inplace_kernel<16>, heads * 2 * (16 / kSlabChunks), kInThreads, 0, st, e)
                      : launch_k(evict_inplace_kernel<8>, heads * 2 * (8 / kSlabChunks), kInThreads, 0, st, e);
  const int chunks = ceil_div(e.budget, kMoveRows);
  return e.h == 128 ? launch_k(evict_copy_kernel<16>, heads * 2 * chunks, kMoveThreads, 0, st, e, chunks)
                    : launch_k(evict_copy_kernel<8>, heads * 2 * chunks, kMoveThreads, 0, st, e, chunks);
}

}  // namespace fpd
