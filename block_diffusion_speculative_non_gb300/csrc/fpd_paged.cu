// fpd_paged.cu — the C ABI of the paged context cache and of the sampled verification: host-side validation, workspace carving
// and launches.  Stated in include/fpd.h.
#include <cstdarg>
#include <cstdio>
#include <mutex>

#include "fpd_paged.cuh"
#include "fpd_scope.cuh"

using namespace fpd;

namespace {

fpd_status refuse(fpd_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return set_last_error(s, buf);
}
fpd_status cuda_error(cudaError_t e, const char* where) { return refuse(FPD_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e)); }
bool aligned(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// SMs of the current device, the kernels' attributes set on the first call.
cudaError_t device_ready(int* sms) {
  static std::mutex mu;
  static int count[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (!count[dev]) {
    int n = 0;
    e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = paged_attn_init_attributes();
    if (e != cudaSuccess) return e;
    count[dev] = n;
  }
  *sms = count[dev];
  return cudaSuccess;
}

fpd_status check_page(int format, int page, int nkv, int h) {
  if (format != FPD_PAGE_BF16 && format != FPD_PAGE_INT4) return refuse(FPD_ERR_INVALID_ARG, "page format %d", format);
  if (h != 64 && h != 128) return refuse(FPD_ERR_UNSUPPORTED, "head_dim %d (64 or 128)", h);
  if (page != 16 && page != 32 && page != 64 && page != 128) return refuse(FPD_ERR_UNSUPPORTED, "page_size %d (16, 32, 64 or 128)", page);
  if (nkv < 1 || nkv > 1 << 12) return refuse(FPD_ERR_SHAPE, "n_kv_heads %d", nkv);
  return FPD_OK;
}
size_t slab_bytes(int format, int page, int h) { return (size_t)page * row_bytes(format, h); }

// Sizes alone: what a workspace query needs.
fpd_status check_store_sizes(const fpd_paged_store* s) {
  if (!s) return refuse(FPD_ERR_INVALID_ARG, "null store");
  fpd_status e = check_page(s->format, s->page_size, s->n_kv_heads, s->head_dim);
  if (e) return e;
  if (s->n_layers < 1 || s->n_pages < 1 || s->table_width < 1 || s->table_width > kMaxStoreCap / s->page_size)
    return refuse(FPD_ERR_SHAPE, "n_layers %d, n_pages %d, table_width %d", s->n_layers, s->n_pages, s->table_width);
  return FPD_OK;
}
fpd_status check_store(const fpd_paged_store* s, int layer, Pages* out) {
  fpd_status e = check_store_sizes(s);
  if (e) return e;
  if (layer < 0 || layer >= s->n_layers) return refuse(FPD_ERR_SHAPE, "layer %d of %d", layer, s->n_layers);
  if (!s->pages || !s->table) return refuse(FPD_ERR_INVALID_ARG, "null pages or table");
  if (!aligned(s->pages) || ((uintptr_t)s->table & 3)) return refuse(FPD_ERR_INVALID_ARG, "pages are not 16-byte or the table not 4-byte aligned");
  Pages p{};
  p.slab_bytes = (uint32_t)slab_bytes(s->format, s->page_size, s->head_dim);
  p.page_bytes = (size_t)2 * s->n_kv_heads * p.slab_bytes;
  p.base = (uint8_t*)s->pages + (size_t)layer * s->n_pages * p.page_bytes;
  p.table = s->table;
  p.format = s->format;
  p.n_pages = s->n_pages;
  p.page = s->page_size;
  for (p.page_shift = 4; 1 << p.page_shift < p.page;) p.page_shift++;
  p.width = s->table_width;
  p.nkv = s->n_kv_heads;
  p.h = s->head_dim;
  *out = p;
  return FPD_OK;
}

fpd_status check_rows(int batch, int total_rows, const int32_t* row_off) {
  if (batch < 1 || total_rows < 0 || total_rows > kMaxAttnRows) return refuse(FPD_ERR_SHAPE, "batch %d, total_rows %d", batch, total_rows);
  if (!row_off) return refuse(FPD_ERR_INVALID_ARG, "null row_off");
  return FPD_OK;
}

fpd_status check_queries(int batch, int block_len, int nq, int nkv) {
  if (batch < 1 || block_len < 1) return refuse(FPD_ERR_SHAPE, "batch %d, block_len %d", batch, block_len);
  if (nq < nkv || nq % nkv) return refuse(FPD_ERR_SHAPE, "n_q_heads %d must be a multiple of n_kv_heads %d", nq, nkv);
  if (nq / nkv > 128) return refuse(FPD_ERR_UNSUPPORTED, "%d query heads per kv head (at most 128)", nq / nkv);
  if ((long long)batch * block_len > kMaxAttnRows || (long long)batch * block_len * nq > kMaxAttnRows)
    return refuse(FPD_ERR_SHAPE, "batch * block_len * n_q_heads exceeds %lld", kMaxAttnRows);
  return FPD_OK;
}

struct AttnWs {
  PagedPlan plan;
  float* o_part;
  float2* ml;
  int4* desc;
  uint32_t* spoilt;
  size_t bytes;
};
AttnWs carve(void* base, int batch, int L, int nq, const fpd_paged_store* s, int sms) {
  AttnWs w{};
  w.plan = paged_attn_plan(batch, L, nq, s->n_kv_heads, s->format, s->table_width * s->page_size, sms);
  const size_t n = (size_t)2 * w.plan.runs * w.plan.rows;
  const size_t lead = align_up((uintptr_t)base, 256) - (uintptr_t)base;   // the workspace itself is 16-byte aligned
  const size_t ml_at = align_up(n * s->head_dim * sizeof(float), 256), desc_at = ml_at + align_up(n * sizeof(float2), 256);
  w.o_part = (float*)((char*)base + lead);
  w.ml = (float2*)((char*)base + lead + ml_at);
  w.desc = (int4*)((char*)base + lead + desc_at);
  const size_t spoilt_at = desc_at + align_up((size_t)w.plan.runs * sizeof(int4), 256);
  w.spoilt = (uint32_t*)((char*)base + lead + spoilt_at);
  w.bytes = 256 + spoilt_at + (size_t)w.plan.runs * 8 * sizeof(uint32_t);
  return w;
}

}  // namespace

extern "C" {

size_t fpd_page_bytes(int format, int page_size, int n_kv_heads, int head_dim) {
  if (check_page(format, page_size, n_kv_heads, head_dim)) return 0;
  return 2 * (size_t)n_kv_heads * slab_bytes(format, page_size, head_dim);
}

fpd_status fpd_paged_append(int batch, int total_rows, const fpd_paged_store* store, int layer, const void* k, int k_ld,
                            const void* v, int v_ld, const int32_t* row_off, const int32_t* row_cnt, const int32_t* pos_start,
                            const int32_t* pos_offset, const float* rope, int max_pos, void* stream) {
  ApiScope scope("fpd_paged_append", stream);
  PagedRows a{};
  fpd_status s = check_store(store, layer, &a.pg);
  if (s || (s = check_rows(batch, total_rows, row_off))) return s;
  if (!k || !v) return refuse(FPD_ERR_INVALID_ARG, "null k or v");
  const int row = store->n_kv_heads * store->head_dim;
  if (k_ld < row || v_ld < row || k_ld % 8 || v_ld % 8)
    return refuse(FPD_ERR_SHAPE, "k_ld %d and v_ld %d must be multiples of 8 and at least %d", k_ld, v_ld, row);
  if (rope && max_pos < 1) return refuse(FPD_ERR_SHAPE, "max_pos %d", max_pos);
  if (!aligned(k) || !aligned(v) || !aligned(rope)) return refuse(FPD_ERR_INVALID_ARG, "a device pointer is not 16-byte aligned");
  if (total_rows == 0) return scope.done(FPD_OK);
  a.k = (const bf16*)k;
  a.v = (const bf16*)v;
  a.k_ld = k_ld;
  a.v_ld = v_ld;
  a.row_off = row_off;
  a.row_cnt = row_cnt;
  a.pos_start = pos_start;
  a.pos_offset = pos_offset;
  a.rope = (const float2*)rope;
  a.batch = batch;
  a.total_rows = total_rows;
  a.max_pos = max_pos;
  const cudaError_t e = launch_paged_append(a, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_error(e, "fpd_paged_append");
  return scope.done(FPD_OK);
}

fpd_status fpd_paged_read(int batch, int total_rows, const fpd_paged_store* store, int layer, const int32_t* row_off,
                          const int32_t* row_cnt, const int32_t* pos_start, void* k, void* v, void* stream) {
  ApiScope scope("fpd_paged_read", stream);
  PagedRows a{};
  fpd_status s = check_store(store, layer, &a.pg);
  if (s || (s = check_rows(batch, total_rows, row_off))) return s;
  if (!k || !v) return refuse(FPD_ERR_INVALID_ARG, "null k or v");
  if (!aligned(k) || !aligned(v)) return refuse(FPD_ERR_INVALID_ARG, "a device pointer is not 16-byte aligned");
  if (total_rows == 0) return scope.done(FPD_OK);
  a.k_out = (bf16*)k;
  a.v_out = (bf16*)v;
  a.row_off = row_off;
  a.row_cnt = row_cnt;
  a.pos_start = pos_start;
  a.batch = batch;
  a.total_rows = total_rows;
  const cudaError_t e = launch_paged_read(a, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_error(e, "fpd_paged_read");
  return scope.done(FPD_OK);
}

size_t fpd_paged_attention_workspace_bytes(int batch, int block_len, int n_q_heads, const fpd_paged_store* store) {
  if (check_store_sizes(store) || check_queries(batch, block_len, n_q_heads, store->n_kv_heads)) return 0;
  int sms = 0;
  if (device_ready(&sms) != cudaSuccess) return 0;
  const AttnWs w = carve(nullptr, batch, block_len, n_q_heads, store, sms);
  return w.plan.too_large ? 0 : w.bytes;
}

fpd_status fpd_paged_attention(int batch, int block_len, int n_q_heads, const fpd_paged_store* store, int layer, const void* q,
                               const void* k_blk, const void* v_blk, const int32_t* ctx_len, int window, int sinks, int causal,
                               void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  ApiScope scope("fpd_paged_attention", stream);
  PagedAttn a{};
  fpd_status s = check_store(store, layer, &a.pg);
  if (s || (s = check_queries(batch, block_len, n_q_heads, store->n_kv_heads))) return s;
  if (window < 0 || sinks < 0) return refuse(FPD_ERR_SHAPE, "window %d, sinks %d", window, sinks);
  if (!q || !ctx_len || !out || !workspace) return refuse(FPD_ERR_INVALID_ARG, "null pointer argument");
  if (!k_blk != !v_blk) return refuse(FPD_ERR_INVALID_ARG, "k_blk and v_blk go together");
  const void* al[] = {q, k_blk, v_blk, out, workspace};
  for (const void* p : al)
    if (!aligned(p)) return refuse(FPD_ERR_INVALID_ARG, "a device pointer is not 16-byte aligned");
  int sms = 0;
  cudaError_t e = device_ready(&sms);
  if (e != cudaSuccess) return cuda_error(e, "device query");
  const AttnWs w = carve(workspace, batch, block_len, n_q_heads, store, sms);
  if (w.plan.too_large) return refuse(FPD_ERR_SHAPE, "batch %d of %d pages: more key tiles than 31 bits hold", batch, store->table_width);
  if (w.bytes > workspace_bytes) return refuse(FPD_ERR_CAPACITY, "workspace %zu < %zu bytes", workspace_bytes, w.bytes);
  a.q = (const bf16*)q;
  a.kblk = (const bf16*)k_blk;
  a.vblk = (const bf16*)v_blk;
  a.ctx_len = ctx_len;
  a.out = (bf16*)out;
  a.lse = lse;
  a.o_part = w.o_part;
  a.ml = w.ml;
  a.desc = w.desc;
  a.spoilt = w.spoilt;
  a.batch = batch;
  a.L = block_len;
  a.lb = k_blk ? block_len : 0;
  a.nq = n_q_heads;
  a.window = window;
  a.sinks = window ? sinks : 0;
  a.causal = causal != 0;
  e = launch_paged_attention(a, w.plan, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_error(e, "fpd_paged_attention");
  return scope.done(FPD_OK);
}

fpd_status fpd_verify_sampled(int batch, int block_len, int vocab, const int32_t* draft, const float* target,
                              const float* draft_probs, const float* uniform, int32_t* accept_len, int32_t* committed,
                              int32_t* valid_out, void* stream) {
  ApiScope scope("fpd_verify_sampled", stream);
  if (batch < 1 || block_len < 2 || vocab < 1) return refuse(FPD_ERR_SHAPE, "batch %d, block_len %d, vocab %d", batch, block_len, vocab);
  if (batch > 1 << 26 || vocab > 1 << 26 || (long long)batch * block_len > 1ll << 30)
    return refuse(FPD_ERR_SHAPE, "batch %d, block_len %d, vocab %d", batch, block_len, vocab);
  if (!draft || !target || !uniform || !accept_len || !committed) return refuse(FPD_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(target) || !aligned(draft_probs)) return refuse(FPD_ERR_INVALID_ARG, "a device pointer is not 16-byte aligned");
  VerifySampled a{draft, target, draft_probs, uniform, accept_len, committed, valid_out, batch, block_len, vocab};
  const cudaError_t e = launch_verify_sampled(a, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_error(e, "fpd_verify_sampled");
  return scope.done(FPD_OK);
}

}  // extern "C"
