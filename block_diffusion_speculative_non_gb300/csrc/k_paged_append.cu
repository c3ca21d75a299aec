// k_paged_append.cu — rows into the pages of a context cache, the keys rotated on the way, and back out of them.
//
//   key of row r at position pos:  k'_i = k_i cos_i - k_{i + h/2} sin_i,  k'_{i + h/2} = k_{i + h/2} cos_i + k_i sin_i,  i < h/2
//
// A thread has 16 dims of a row, 8 of each half, so that a rotation stays inside it, in one or more kv heads of K and V; two
// neighbours have a 4-bit group.  The first loads go out before the row's request, slot and page are known.  Bound by the copy: 4 h bytes in and 2 h (or
// 9 h / 16) bytes out per row and kv head, K or V.
#include "fpd_paged.cuh"

namespace fpd {

namespace {

constexpr int kThreads = 256;

// Where row r goes; false for a row that is skipped.
struct Place {
  int id, in_page;   // page and place in it
  long long pos;     // rotary position
};
__device__ __forceinline__ bool place_of(const PagedRows& a, int r, bool check_pos, Place& w) {
  int lo = 0, hi = a.batch;   // request b with row_off[b] <= r < row_off[b + 1]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.row_off[mid] <= r) lo = mid; else hi = mid;
  }
  const int i = r - a.row_off[lo];
  if (i < 0 || r >= a.row_off[a.batch] || (a.row_cnt && i >= a.row_cnt[lo])) return false;
  const long long slot = (long long)(a.pos_start ? a.pos_start[lo] : 0) + i;
  w.pos = slot + (a.pos_offset ? a.pos_offset[lo] : 0);
  if (slot < 0 || slot >= a.pg.cap() || (check_pos && (w.pos < 0 || w.pos >= a.max_pos))) {
    record_check(kCheckBadPosition);
    return false;
  }
  w.id = page_of(a.pg, lo, (int)slot);
  w.in_page = (int)slot & (a.pg.page - 1);
  return w.id >= 0;
}

// RN(x1 c + x2 s) to fp32 but for 2^-20 of the cases that lie next to a tie: the products' and the sum's rounding errors are
// carried along.  A 4-bit code goes by the result's bf16 rounding, and a key next to a border of it must not depend on the
// order of two roundings.
__device__ __forceinline__ float dot2(float x1, float c, float x2, float s) {
  const float p = __fmul_rn(x1, c), q = __fmul_rn(x2, s);
  const float pe = fmaf(x1, c, -p), qe = fmaf(x2, s, -q);
  const float d = __fadd_rn(p, q), b = __fadd_rn(d, -p);
  const float e = __fadd_rn(__fadd_rn(p, -__fadd_rn(d, -b)), __fadd_rn(q, -b));
  const float r = __fadd_rn(d, __fadd_rn(e, __fadd_rn(pe, qe)));
  return fabsf(d) < INFINITY ? r : d;
}

__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; i++) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Codes of 8 dims, whose group's other 8 the neighbouring thread has.
__device__ __forceinline__ uint32_t quant8(const float (&x)[8], int& byte) {
  float big = 0.f;
#pragma unroll
  for (int i = 0; i < 8; i++) big = fmaxf(big, fabsf(x[i]));   // a NaN does not count
  big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
  byte = scale_byte(big);
  const float s = scale_value(byte), inv = s > 0.f ? 1.f / s : 0.f;
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) w |= code_of(x[i], s, inv) << (4 * i);
  return w;
}

// Thread: 16 dims (e) of row r, in slabs (K, then V heads) s0 .. of the row, four at a time.
template <int H, bool INT4>
__global__ void __launch_bounds__(kThreads, INT4 ? 2 : 3) append_kernel(const __grid_constant__ PagedRows a, int per) {
  pdl_wait();
  pdl_trigger();
  constexpr int E = H / 16, U = 4;   // threads of a row, slabs in flight
  const int nkv = a.pg.nkv, e = threadIdx.x % E, r = blockIdx.x * (kThreads / E) + threadIdx.x / E;
  const int s0 = blockIdx.y * per, s1 = min(2 * nkv, s0 + per);
  const bool here = r < a.total_rows;
  uint4 u[U][2];
  auto load = [&](int s) {
#pragma unroll
    for (int i = 0; i < U; i++) {
      const int g = s + i < nkv ? s + i : s + i - nkv;
      u[i][0] = u[i][1] = make_uint4(0, 0, 0, 0);
      if (here && s + i < s1) {
        const bf16* src = (s + i >= nkv ? a.v + (size_t)r * a.v_ld : a.k + (size_t)r * a.k_ld) + (size_t)g * H + 8 * e;
        u[i][0] = __ldcs(reinterpret_cast<const uint4*>(src));
        u[i][1] = __ldcs(reinterpret_cast<const uint4*>(src + H / 2));
      }
    }
  };
  load(s0);
  Place w;
  const bool ok = here && place_of(a, r, a.rope != nullptr, w);
  const bool turn = ok && a.rope && s0 < nkv;
  float4 cs[4];   // (cos, sin) of dims 8 e ..
  if (turn) {
    const float4* at = reinterpret_cast<const float4*>(a.rope + (size_t)w.pos * (H / 2) + 8 * e);
#pragma unroll
    for (int i = 0; i < 4; i++) cs[i] = __ldg(at + i);
  }
  uint8_t* page = ok ? slab_of(a.pg, w.id, 0, 0) : nullptr;   // the slabs of a page follow one another
  for (int s = s0; s < s1; s += U) {
#pragma unroll
    for (int i = 0; i < U; i++) {
      if (s + i >= s1) break;   // the same for all threads
      uint4 u0 = u[i][0], u1 = u[i][1];
      float x0[8], x1[8];
      if (turn && s + i < nkv) {
        unpack8(u0, x0);
        unpack8(u1, x1);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float4 t = cs[j / 2];
          const float a0 = x0[j], b0 = x1[j], a1 = x0[j + 1], b1 = x1[j + 1];
          x0[j] = dot2(a0, t.x, b0, -t.y);
          x1[j] = dot2(b0, t.x, a0, t.y);
          x0[j + 1] = dot2(a1, t.z, b1, -t.w);
          x1[j + 1] = dot2(b1, t.z, a1, t.w);
        }
        u0 = pack8(x0);
        u1 = pack8(x1);
      }
      uint8_t* slab = page + (size_t)(s + i) * a.pg.slab_bytes;
      if (!INT4) {
        if (ok) {
          bf16* dst = reinterpret_cast<bf16*>(slab) + (size_t)w.in_page * H + 8 * e;
          *reinterpret_cast<uint4*>(dst) = u0;
          *reinterpret_cast<uint4*>(dst + H / 2) = u1;
        }
      } else {
        unpack8(u0, x0);   // as rounded to bf16
        unpack8(u1, x1);
        int c0, c1;
        const uint32_t w0 = quant8(x0, c0), w1 = quant8(x1, c1);   // every thread: neighbours exchange their maxima
        if (ok) {
          uint8_t* code = slab + w.in_page * (H / 2) + 4 * e;
          *reinterpret_cast<uint32_t*>(code) = w0;
          *reinterpret_cast<uint32_t*>(code + H / 4) = w1;
          if ((e & 1) == 0) {
            uint8_t* sc = slab + a.pg.page * (H / 2) + w.in_page * (H / 16) + e / 2;
            sc[0] = (uint8_t)c0;
            sc[H / 32] = (uint8_t)c1;
          }
        }
      }
    }
    if (s + U < s1) load(s + U);
  }
}

template <int H, bool INT4>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ PagedRows a, int row_threads, int rows_per_cta) {
  pdl_wait();
  pdl_trigger();
  constexpr int E = H / 16;
  const int nkv = a.pg.nkv;
  const int rr = threadIdx.x / row_threads, in_row = threadIdx.x - rr * row_threads;
  const int r = blockIdx.x * rows_per_cta + rr;
  const int item = blockIdx.y * row_threads + in_row;
  const int slab = item / E, e = item % E;   // here e is a group of 16 consecutive dims
  Place w;
  if (rr >= rows_per_cta || r >= a.total_rows || slab >= 2 * nkv || !place_of(a, r, false, w)) return;
  const bool is_v = slab >= nkv;
  const int g = is_v ? slab - nkv : slab;
  const uint8_t* p = slab_of(a.pg, w.id, is_v, g);
  bf16* dst = (is_v ? a.v_out : a.k_out) + ((size_t)r * nkv + g) * H + 16 * e;
  if (!INT4) {
    const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const bf16*>(p) + (size_t)w.in_page * H + 16 * e);
    const uint4 v0 = src[0], v1 = src[1];
    reinterpret_cast<uint4*>(dst)[0] = v0;
    reinterpret_cast<uint4*>(dst)[1] = v1;
  } else {
    const uint2 c = *reinterpret_cast<const uint2*>(p + w.in_page * (H / 2) + 8 * e);
    const float s = scale_value(p[a.pg.page * (H / 2) + w.in_page * (H / 16) + e]);
    float x0[8], x1[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
      x0[i] = (float)((int)((c.x >> (4 * i)) & 15) - 8) * s;
      x1[i] = (float)((int)((c.y >> (4 * i)) & 15) - 8) * s;
    }
    reinterpret_cast<uint4*>(dst)[0] = pack8(x0);
    reinterpret_cast<uint4*>(dst)[1] = pack8(x1);
  }
}

template <class K>
cudaError_t launch_rows(K kernel, const PagedRows& a, cudaStream_t st) {
  // a row's threads, cut into CTAs along y where one does not hold them
  const int all = 2 * a.pg.nkv * (a.pg.h / 16), row_threads = std::min(all, kThreads), rows = kThreads / row_threads;
  const dim3 grid((a.total_rows + rows - 1) / rows, ceil_div(all, row_threads));
  return launch_k(kernel, grid, kThreads, 0, st, a, row_threads, rows);
}

}  // namespace

cudaError_t launch_paged_append(const PagedRows& a, cudaStream_t st) {
  const bool q = a.pg.format == FPD_PAGE_INT4;
  // few rows: a thread for each slab; many: a thread keeps its angles for a row's slabs, as long as the GPU stays full (1024 threads on
  // each of its 152 SMs; eight prompts, 36864 rows: 66.8 us with a thread for each slab, 53 so, 85 % of the copy rate)
  const int slabs = 2 * a.pg.nkv, e = a.pg.h / 16;
  const int per = (int)std::min<long long>(slabs, std::max<long long>(1, (long long)a.total_rows * e * slabs / (152 * 1024)));
  const dim3 grid(ceil_div(a.total_rows, kThreads / e), ceil_div(slabs, per));
  auto go = [&](auto k) { return launch_k(k, grid, kThreads, 0, st, a, per); };
  if (a.pg.h == 128) return go(q ? append_kernel<128, true> : append_kernel<128, false>);
  return go(q ? append_kernel<64, true> : append_kernel<64, false>);
}

cudaError_t launch_paged_read(const PagedRows& a, cudaStream_t st) {
  const bool q = a.pg.format == FPD_PAGE_INT4;
  if (a.pg.h == 128) return launch_rows(q ? read_kernel<128, true> : read_kernel<128, false>, a, st);
  return launch_rows(q ? read_kernel<64, true> : read_kernel<64, false>, a, st);
}

}  // namespace fpd
