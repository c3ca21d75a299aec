// k_verify_sampled.cu — verification of a drafted block by given random numbers:
//   keep d_{i+1} while u_i q_i(d_{i+1}) < p_i(d_{i+1});  the last id from r = max(p_n - q_n, 0), or from p_{L-1}, by its running sum
//
// Only one row of each request is summed, whichever the refusal picks: bound by reading it (and the drafter's).  A cluster of CTAs
// shares a row; each warp sums a contiguous range of ids, the range that holds the draw is found from the warps' sums through the
// cluster's shared memory, and its CTA goes over that range alone a second time.
//
// The running sum's order must not decide an id, so sums are kept to about 2^-44: p - q with its rounding error, a lane's sum as
// two fp32 numbers, the lanes' sums in fp64 (fp64 throughout would take longer than the read: the rate is 2 additions per clock
// and SM).
#include "fpd_paged.cuh"

namespace fpd {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32, kCluster = 8;

__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ double peer_double(const double* p, uint32_t rank) {
  uint32_t at;
  double v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(at));
  return v;
}

__device__ __forceinline__ float weight(float v) { return v > 0.f ? v : 0.f; }   // negative and NaN: 0

// a lane's sum: s + lo
struct Sum {
  float s = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x, float x_lo) {
    const float t = __fadd_rn(s, x), b = __fadd_rn(t, -s);
    lo = __fadd_rn(lo, __fadd_rn(__fadd_rn(__fadd_rn(s, -__fadd_rn(t, -b)), __fadd_rn(x, -b)), x_lo));
    s = t;
  }
  // max(p - q, 0), exactly: the difference and what its rounding lost
  __device__ __forceinline__ void add_diff(float p, float q) {
    const float d = __fadd_rn(p, -q);
    if (!(d > 0.f)) return;
    const float b = __fadd_rn(d, -p);
    add(d, __fadd_rn(__fadd_rn(p, -__fadd_rn(d, -b)), __fadd_rn(-q, -b)));
  }
};

// What the last id is drawn from: ids [0, vocab) with weight max(p - q, 0), q null: p, without id `gone`.
struct Row {
  const float *p, *q;
  int gone;
  __device__ __forceinline__ double at(int id) const {
    if (id == gone) return 0.0;
    const double w = (double)weight(p[id]);
    return q ? fmax(w - (double)weight(q[id]), 0.0) : w;
  }
};

__device__ __forceinline__ double warp_sum_d(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ double warp_scan_d(double v, int lane) {   // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  return v;
}

// One warp's sum over [begin, end); VEC: begin is a multiple of 4 and the rows are 16-byte aligned.
template <bool VEC>
__device__ __forceinline__ double range_sum(const Row& r, int begin, int end, int lane) {
  Sum a;
  auto one = [&](float p, float q, int id) {
    if (id == r.gone) return;
    if (r.q) a.add_diff(weight(p), weight(q)); else a.add(weight(p), 0.f);
  };
  if (VEC) {
    constexpr int U = 4;
    for (int i0 = begin + 4 * lane; i0 < end; i0 += 128 * U) {
      float4 p[U], q[U];
#pragma unroll
      for (int u = 0; u < U; u++) {
        const int i = i0 + 128 * u;
        p[u] = q[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i + 3 < end) {   // ranges end at multiples of 4 but for the row's end, which is one too
          p[u] = __ldg(reinterpret_cast<const float4*>(r.p + i));
          if (r.q) q[u] = __ldg(reinterpret_cast<const float4*>(r.q + i));
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
          p[u] = __ldg(r.p + i);
          if (r.q) q[u] = __ldg(r.q + i);
        }
      }
#pragma unroll
      for (int u = 0; u < U; u++) one(p[u], q[u], i0 + 32 * u);
    }
  }
  return warp_sum_d((double)a.s + (double)a.lo);
}

template <bool VEC>
__global__ void __launch_bounds__(kThreads) verify_sampled_kernel(const __grid_constant__ VerifySampled a, int ctas, int range) {
  pdl_wait();
  pdl_trigger();
  __shared__ int refused;
  __shared__ double cta_total, warp_part[kWarps], scan[kWarps];
  __shared__ int found, last_held;
  const int b = blockIdx.x / ctas, rank = ctas > 1 ? (int)cta_rank() : 0;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, L = a.L, V = a.vocab;
  const int32_t* draft = a.draft + (size_t)b * (L - 1);
  const float* u = a.uniform + (size_t)b * L;
  if (tid == 0) refused = L - 1;
  __syncthreads();
  for (int i = tid; i < L - 1; i += kThreads) {
    const int d = draft[i];
    bool keep = false;
    if (d >= 0 && d < V) {
      const double p = weight(a.target[((size_t)b * L + i) * V + d]);
      const double q = a.probs ? (double)weight(a.probs[((size_t)b * (L - 1) + i) * V + d]) : 1.0;
      keep = (double)u[i] * q < p;
    } else {
      record_check(kCheckBadToken);
    }
    if (!keep) atomicMin(&refused, i);   // the smallest: no order in it
  }
  __syncthreads();
  const int n = refused;
  Row row;
  row.p = a.target + ((size_t)b * L + n) * V;
  row.q = n < L - 1 && a.probs ? a.probs + ((size_t)b * (L - 1) + n) * V : nullptr;
  row.gone = n < L - 1 && !a.probs ? draft[n] : -1;
  const int w0 = (rank * kWarps + warp) * range, begin = min(V, w0), end = min(V, w0 + range);
  const bool whole = row.q == nullptr && row.gone < 0;
  for (int pass = 0; pass < 2; pass++) {
    const double mine = range_sum<VEC>(row, begin, end, lane);
    if (lane == 0) warp_part[warp] = mine;
    __syncthreads();
    if (tid == 0) {
      double t = 0;
      for (int w = 0; w < kWarps; w++) t += warp_part[w];
      cta_total = t;
    }
    if (ctas > 1) cluster_barrier(); else __syncthreads();
    // the CTA that holds the draw is the first whose running sum exceeds it; where rounding leaves none, the last with a sum
    double part[kCluster], total = 0;
#pragma unroll
    for (int c = 0; c < kCluster; c++) {
      part[c] = c >= ctas ? 0.0 : ctas > 1 ? peer_double(&cta_total, c) : cta_total;
      total += part[c];
    }
    const double x = (double)u[L - 1] * total;
    double run = 0, before = 0, held_before = 0;
    int at = -1, held = -1;
#pragma unroll
    for (int c = 0; c < kCluster; c++) {
      if (part[c] > 0) {
        held = c;
        held_before = run;
        if (at < 0 && run + part[c] > x) {
          at = c;
          before = run;
        }
      }
      run += part[c];
    }
    if (at < 0) {
      at = held;
      before = held_before;
    }
    if (ctas > 1) cluster_barrier();   // nobody's total changes or goes while others read it
    if (total > 0) {
      if (rank != at) return;
      run = before;
      held = -1;
      int pick = -1;
      double start = before, held_start = before;
      for (int w = 0; w < kWarps && pick < 0; w++) {
        if (warp_part[w] > 0) {
          held = w;
          held_start = run;
          if (run + warp_part[w] > x) {
            pick = w;
            start = run;
          }
        }
        run += warp_part[w];
      }
      if (pick < 0) {
        pick = held;
        start = held_start;
      }
      // the picked range once more, a run of ids per thread
      const int r0 = min(V, (rank * kWarps + pick) * range), r1 = min(V, r0 + range), per = ceil_div(r1 - r0, kThreads);
      const int i0 = min(r1, r0 + tid * per), i1 = min(r1, i0 + per);
      double mine2 = 0;
      int last = -1;
      for (int i = i0; i < i1; i++) {
        const double w = row.at(i);
        if (w > 0) last = i;
        mine2 += w;
      }
      const double inc = warp_scan_d(mine2, lane);
      if (lane == 31) scan[warp] = inc;
      if (tid == 0) {
        found = INT32_MAX;
        last_held = -1;
      }
      __syncthreads();
      double s = start + (inc - mine2);
      for (int w = 0; w < warp; w++) s += scan[w];
      if (last >= 0) atomicMax(&last_held, last);
      if (mine2 > 0 && s + mine2 > x) {   // not every such thread holds the draw: the lowest id wins
        for (int i = i0; i < i1; i++) {
          const double w = row.at(i);
          s += w;
          if (w > 0 && s > x) {
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
    if (whole || pass == 1) break;
    row.q = nullptr;   // nothing left over the drafter: the target's own row
    row.gone = -1;
  }
  if (rank == 0) {
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

cudaError_t verify_sampled_init_attributes() { return cudaSuccess; }

cudaError_t launch_verify_sampled(const VerifySampled& a, cudaStream_t st) {
  // one CTA sums a short row in the time that a cluster takes to meet
  const int ctas = a.vocab > 16384 ? kCluster : 1;
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
