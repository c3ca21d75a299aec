// k_verify_sampled.cu — verification of a drafted block by given random numbers:
//   keep d_{i+1} while u_i q_i(d_{i+1}) < p_i(d_{i+1});  the last id from r = max(p_n - q_n, 0), or from p_{L-1}, by its running sum
//
// Only one row of each request is summed, whichever the refusal picks: bound by reading it (and the drafter's).  A cluster of CTAs
// shares a row; each warp finds the refusal for itself and sums a contiguous range of ids; the range that holds the draw is found
// from the warps' sums, through the cluster's shared memory, and its CTA goes over that range alone a second time.
//
// The running sum's order must not decide an id, so sums are pairs of fp32 numbers, about 2^-46 apart from the exact ones: p - q
// with its rounding error, Knuth's two-sum throughout.  (In fp64, at 2 additions per clock and SM, the 64 rows of 151936 ids below took 86 us,
// 75 more than their read.)
#include "fpd_paged.cuh"

namespace fpd {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kCluster = 8;

__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float2 peer_pair(const float2* p, uint32_t rank) {
  uint32_t at;
  float2 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at));
  return v;
}

__device__ __forceinline__ float weight(float v) { return v > 0.f ? v : 0.f; }   // negative and NaN: 0

// A sum as x + y, |y| at most half a step of x.
__device__ __forceinline__ float2 two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fadd_rn(s, -a);
  return make_float2(s, __fadd_rn(__fadd_rn(a, -__fadd_rn(s, -t)), __fadd_rn(b, -t)));
}
__device__ __forceinline__ float2 add(float2 a, float2 b) {
  const float2 s = two_sum(a.x, b.x);
  const float e = __fadd_rn(s.y, __fadd_rn(a.y, b.y)), h = __fadd_rn(s.x, e);
  return make_float2(h, __fadd_rn(e, -__fadd_rn(h, -s.x)));
}
__device__ __forceinline__ bool above(float2 a, float2 b) { return a.x > b.x || (a.x == b.x && a.y > b.y); }
__device__ __forceinline__ float2 shfl(float2 v, int lane) {
  return make_float2(__shfl_sync(0xffffffffu, v.x, lane), __shfl_sync(0xffffffffu, v.y, lane));
}
__device__ __forceinline__ float2 warp_total(float2 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = add(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
  return v;
}
__device__ __forceinline__ float2 warp_running(float2 v, int lane) {   // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float2 t = make_float2(__shfl_up_sync(0xffffffffu, v.x, o), __shfl_up_sync(0xffffffffu, v.y, o));
    if (lane >= o) v = add(t, v);
  }
  return v;
}

// What the last id is drawn from: id's weight is max(p - q, 0), q null: p, 0 for id `gone`.  As a pair, exactly.
struct Row {
  const float *p, *q;
  int gone;
  __device__ __forceinline__ float2 of(float p_, float q_, int id) const {
    if (id == gone) return make_float2(0.f, 0.f);
    const float2 d = two_sum(weight(p_), -weight(q_));
    return d.x > 0.f ? d : make_float2(0.f, 0.f);
  }
  __device__ __forceinline__ float2 at(int id) const { return of(p[id], q ? q[id] : 0.f, id); }
};

// One warp's sum over [begin, end); VEC: begin is a multiple of 4 and the rows are 16-byte aligned.
template <bool VEC>
__device__ __forceinline__ float2 range_sum(const Row& r, int begin, int end, int lane) {
  float s = 0.f, lo = 0.f;
  auto one = [&](float p, float q, int id) {
    const float2 w = r.of(p, q, id), t = two_sum(s, w.x);
    s = t.x;
    lo = __fadd_rn(lo, __fadd_rn(t.y, w.y));
  };
  if (VEC) {
    constexpr int U = 4;
    for (int i0 = begin + 4 * lane; i0 < end; i0 += 128 * U) {
      float4 p[U], q[U];
#pragma unroll
      for (int u = 0; u < U; u++) {
        const int i = i0 + 128 * u;
        p[u] = q[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < end) {   // ranges end at multiples of 4, or with the row, which is one too
          p[u] = __ldcs(reinterpret_cast<const float4*>(r.p + i));
          if (r.q) q[u] = __ldcs(reinterpret_cast<const float4*>(r.q + i));
        }
      }
#pragma unroll
      for (int u = 0; u < U; u++) {
        const int i = i0 + 128 * u;
        one(p[u].x, q[u].x, i);
        one(p[u].y, q[u].y, i + 1);
        one(p[u].z, q[u].z, i + 2);
        one(p[u].w, q[u].w, i + 3);
      }
    }
  } else {
    constexpr int U = 8;
    for (int i0 = begin + lane; i0 < end; i0 += 32 * U) {
      float p[U], q[U];
#pragma unroll
      for (int u = 0; u < U; u++) {
        const int i = i0 + 32 * u;
        p[u] = q[u] = 0.f;
        if (i < end) {
          p[u] = __ldcs(r.p + i);
          if (r.q) q[u] = __ldcs(r.q + i);
        }
      }
#pragma unroll
      for (int u = 0; u < U; u++) one(p[u], q[u], i0 + 32 * u);
    }
  }
  return warp_total(two_sum(s, lo));
}

// Among the lanes' sums (0 past n), which follow one another from `start` on: the first whose running sum exceeds x, or, where rounding
// leaves none, the last that is not 0; `start` becomes the sum before it.  -1: all are 0.
__device__ __forceinline__ int pick(float2 mine, float2 x, float2& start, int lane, float2* total) {
  const float2 run = add(start, warp_running(mine, lane));
  const unsigned held = __ballot_sync(0xffffffffu, mine.x > 0.f), over = __ballot_sync(0xffffffffu, mine.x > 0.f && above(run, x)) & held;
  if (total) *total = shfl(run, 31);
  const int at = over ? __ffs(over) - 1 : 31 - __clz(held);
  if (at > 0) start = shfl(run, at - 1);
  return at;
}

template <bool VEC>
__global__ void __launch_bounds__(kThreads, 4) verify_sampled_kernel(const __grid_constant__ VerifySampled a, int ctas, int range) {
  pdl_wait();
  pdl_trigger();
  __shared__ float2 cta_sum, part[kWarps], part2[kWarps];
  __shared__ int found, last_held;
  const int b = blockIdx.x / ctas, rank = ctas > 1 ? (int)cta_rank() : 0;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, L = a.L, V = a.vocab;
  const int32_t* draft = a.draft + (size_t)b * (L - 1);
  const float* u = a.uniform + (size_t)b * L;
  const float u_last = u[L - 1];
  if (tid == 0) {
    found = INT32_MAX;
    last_held = -1;
  }
  int n = L - 1;   // the first refusal, found by every warp for itself
  for (int i0 = 0; i0 < L - 1; i0 += 32) {
    const int i = i0 + lane;
    bool refuse = false;
    if (i < L - 1) {
      const int d = draft[i];
      if (d >= 0 && d < V) {
        const float p = weight(a.target[((size_t)b * L + i) * V + d]);
        const float q = a.probs ? weight(a.probs[((size_t)b * (L - 1) + i) * V + d]) : 1.f;
        refuse = !((double)u[i] * q < (double)p);   // 48 bits: exact
      } else {
        record_check(kCheckBadToken);
        refuse = true;
      }
    }
    const unsigned m = __ballot_sync(0xffffffffu, refuse);
    if (m) {
      n = i0 + __ffs(m) - 1;
      break;
    }
  }
  Row row;
  row.p = a.target + ((size_t)b * L + n) * V;
  row.q = n < L - 1 && a.probs ? a.probs + ((size_t)b * (L - 1) + n) * V : nullptr;
  row.gone = n < L - 1 && !a.probs ? draft[n] : -1;
  const int w0 = (rank * kWarps + warp) * range, begin = min(V, w0), end = min(V, w0 + range);
  for (int pass = 0; pass < 2; pass++) {
    const float2 mine = range_sum<VEC>(row, begin, end, lane);
    if (lane == 0) part[warp] = mine;
    __syncthreads();
    const float2 warps = lane < kWarps ? part[lane] : make_float2(0.f, 0.f);
    float2 start = make_float2(0.f, 0.f), total = warp_total(warps);
    int at = 0;
    float2 x;
    if (ctas > 1) {
      if (tid == 0) cta_sum = total;
      cluster_barrier();
      const float2 all = lane < kCluster ? peer_pair(&cta_sum, lane) : make_float2(0.f, 0.f);
      total = warp_total(all);
      x = two_sum(__fmul_rn(u_last, total.x), fmaf(u_last, total.x, -__fmul_rn(u_last, total.x)) + u_last * total.y);
      at = pick(all, x, start, lane, nullptr);
      cluster_barrier();   // nobody's sum changes or goes while others read it
    } else {
      x = two_sum(__fmul_rn(u_last, total.x), fmaf(u_last, total.x, -__fmul_rn(u_last, total.x)) + u_last * total.y);
    }
    if (total.x > 0.f) {
      if (rank != at) return;
      const int w = pick(warps, x, start, lane, nullptr);
      // the picked range once more, a few consecutive ids per thread
      const int r0 = min(V, (rank * kWarps + w) * range), r1 = min(V, r0 + range), per = ceil_div(r1 - r0, kThreads);
      const int i0 = min(r1, r0 + tid * per), i1 = min(r1, i0 + per);
      float2 own = make_float2(0.f, 0.f);
      int last = -1;
#pragma unroll 4
      for (int i = i0; i < i1; i++) {
        const float2 v = row.at(i);
        if (v.x > 0.f) last = i;
        own = add(own, v);
      }
      const float2 run = warp_running(own, lane);
      if (lane == 31) part2[warp] = run;
      if (last >= 0) atomicMax(&last_held, last);
      __syncthreads();
      float2 s = start;
      for (int k = 0; k < warp; k++) s = add(s, part2[k]);
      const float2 before = shfl(run, lane > 0 ? lane - 1 : 0);
      if (lane > 0) s = add(s, before);
      if (own.x > 0.f && above(add(s, own), x)) {   // not every such thread holds the draw: the lowest id wins
        for (int i = i0; i < i1; i++) {
          const float2 v = row.at(i);
          s = add(s, v);
          if (v.x > 0.f && above(s, x)) {
            atomicMin(&found, i);
            break;
          }
        }
      }
      __syncthreads();
      const int token = found != INT32_MAX ? found : last_held;
      int32_t* out = a.committed + (size_t)b * L;
      for (int i = tid; i < L; i += kThreads) out[i] = i < n ? draft[i] : (i == n ? token : -1);
      if (tid == 0) {
        a.accept[b] = n + 1;
        if (a.valid) a.valid[b] = n == L - 1;
      }
      return;
    }
    if (pass == 1 || (!row.q && row.gone < 0)) break;
    row.q = nullptr;   // nothing left over the drafter: the target's own row
    row.gone = -1;
    __syncthreads();
  }
  if (rank == 0) {   // a row without any probability
    int32_t* out = a.committed + (size_t)b * L;
    for (int i = tid; i < L; i += kThreads) out[i] = i < n ? draft[i] : -1;
    if (tid == 0) {
      record_check(kCheckNoLegalId);
      a.accept[b] = n + 1;
      if (a.valid) a.valid[b] = n == L - 1;
    }
  }
}

}  // namespace

cudaError_t launch_verify_sampled(const VerifySampled& a, cudaStream_t st) {
  // one CTA sums a short row in the time that a cluster takes to meet (8192 ids, 1 and 64 rows: 6.5 and 7.8 us, in a cluster 6.2 and 9.9;
  // 16384 ids: 8.8 and 11.3, 6.4 and 10.0; 151936 ids: 71 and 85, 13 and 24)
  const int ctas = a.vocab > 8192 ? kCluster : 1;
  const int range = ceil_div(ceil_div(a.vocab, ctas * kWarps), 4) * 4;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.batch * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  count_launch();
  return cudaLaunchKernelEx(&cfg, a.vocab % 4 == 0 ? verify_sampled_kernel<true> : verify_sampled_kernel<false>, a, ctas, range);
}

}  // namespace fpd
