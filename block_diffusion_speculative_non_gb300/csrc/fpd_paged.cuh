// fpd_paged.cuh — the paged context cache inside libfpd: layout of the pages, the 4-bit form, launch interfaces.  The public
// calls are in include/fpd.h.
#pragma once

#include <cuda_fp16.h>

#include "fpd_context.cuh"

namespace fpd {

// One layer of a page pool.  A page is [K|V][kv head] slabs of `page` positions; a slab is [position][h] bf16, or
// [position][h / 2] code bytes followed by [position][h / 16] scale bytes.
struct Pages {
  uint8_t* base;           // page 0 of the layer
  const int32_t* table;    // device [batch][width]
  size_t page_bytes;
  uint32_t slab_bytes;
  int format, n_pages, page, page_shift, width, nkv, h;
  __host__ __device__ int cap() const { return width << page_shift; }
};

// Bytes of a stored row of one kv head, codes and scales together.
__host__ __device__ constexpr int row_bytes(int format, int h) { return format == FPD_PAGE_INT4 ? h / 2 + h / 16 : 2 * h; }

// Page of slot t of request b; an id outside the pool is recorded and -1.
__device__ __forceinline__ int page_of(const Pages& p, int b, int t) {
  const int id = p.table[(size_t)b * p.width + (t >> p.page_shift)];
  if ((unsigned)id < (unsigned)p.n_pages) return id;
  record_check(kCheckBadPage);
  return -1;
}
__device__ __forceinline__ uint8_t* slab_of(const Pages& p, int id, int is_v, int g) {
  return p.base + (size_t)id * p.page_bytes + (size_t)(is_v * p.nkv + g) * p.slab_bytes;
}

// ---- the 4-bit form: 16 consecutive dims share a scale s, x stands as n s with -7 <= n <= 7, held as n + 8 -----------------
// The scale byte is the upper bits of an fp16 number without its sign: 5 exponent and 3 mantissa bits, (8 + m) 2^(e - 18) or
// m 2^-17, up to 2^13.  So n s has at most 7 significant bits and lies in fp16's range: it is exact in bf16 and in fp16.
constexpr int kTopScale = 28 << 3;
__device__ __forceinline__ float scale_value(int byte) { return __half2float(__ushort_as_half((unsigned short)(byte << 7))); }
// The smallest scale with 7 s >= big (big >= 0, finite or infinite; the top one where there is none).
__device__ __forceinline__ int scale_byte(float big) {
  // start from a seventh, cut to the scale's bits (an fp16 number towards zero, without its lower 7 bits): exact or one below
  const float want = fminf(big * (1.f / 7.f), 8192.f);
  int b = (__half_as_ushort(__float2half_rz(want)) >> 7) & 0xFF;
  if (b > 0) b--;                                   // the product may have been rounded up past a border
  while (b < kTopScale && 7.f * scale_value(b) < big) b++;   // 7 s has 7 bits: exact.  At most three steps
  return b;
}
// Code of x: n = x / s rounded to nearest, ties to even, within -7..7; inv = 1 / s.  A quotient of 8 by 4 bits that is not a
// tie is at least 2^-9 away from one, and a tie has 5 bits, which the corrected quotient keeps.
__device__ __forceinline__ uint32_t code_of(float x, float s, float inv) {
  if (!(fabsf(x) < INFINITY)) return x != x || s == 0.f ? 8 : (x > 0.f ? 15 : 1);
  float q = x * inv;
  q = fmaf(fmaf(-q, s, x), inv, q);
  return (uint32_t)(8 + (int)rintf(fminf(fmaxf(q, -7.f), 7.f)));
}

// ---- append and read -----------------------------------------------------------------------------------------------------
struct PagedRows {
  Pages pg;
  const bf16 *k, *v;       // append: rows k_ld and v_ld elements apart
  bf16 *k_out, *v_out;     // read: [total_rows][nkv][h]
  int k_ld, v_ld;
  const int32_t *row_off, *row_cnt, *pos_start, *pos_offset;
  const float2* rope;      // [max_pos][h / 2] (cos, sin) or null
  int batch, total_rows, max_pos;
};
cudaError_t launch_paged_append(const PagedRows& a, cudaStream_t st);
cudaError_t launch_paged_read(const PagedRows& a, cudaStream_t st);

// ---- attention -------------------------------------------------------------------------------------------------------------
struct PagedAttn {
  Pages pg;
  const bf16* q;                // [batch * L][nq][h]
  const bf16 *kblk, *vblk;      // [batch][nkv][L][h] or null
  const int32_t* ctx_len;       // device [batch]
  bf16* out;
  float* lse;                   // or null
  float* o_part;                // [2 runs][rows of a tile][h]
  float2* ml;                   // [2 runs][rows of a tile]: running maximum (base 2) and sum
  int4* desc;                   // [runs]: request, kv head, row tile and last run of the unit that a run leaves unfinished
  uint32_t* spoilt;             // [runs][words]: which of a run's parts came out with something that is no number
  int batch, L, lb, nq, window, sinks, causal;   // lb: block keys, L or 0
};
enum PagedKernel { kPagedStream, kPagedTc };
struct PagedPlan {
  PagedKernel kernel;
  int rows, tiles;     // rows of a row tile, row tiles of a request and kv head
  bool solo;           // k_paged_tc.cu: row tiles of one lane
  bool too_large;      // more key tiles than 31 bits hold
  int sms, grid, runs; // SMs, CTAs, and the runs that share the key tiles (of CTAs, or of their warps)
};
PagedPlan paged_attn_plan(int batch, int L, int nq, int nkv, int format, int t_cap, int num_sms);
cudaError_t paged_attn_init_attributes();
cudaError_t launch_paged_attention(const PagedAttn& a, const PagedPlan& pl, cudaStream_t st);

// ---- sampled verification ----------------------------------------------------------------------------------------------------
struct VerifySampled {
  const int32_t* draft;
  const float *target, *probs, *uniform;   // probs null: the drafted ids were certain
  int32_t *accept, *committed, *valid;
  int batch, L, vocab;
};
cudaError_t launch_verify_sampled(const VerifySampled& a, cudaStream_t st);

}  // namespace fpd
