// fpd_context.cu — the C ABI of the operators on a context store (attention over a shared prefix, collected attention
// weight, eviction): host-side validation, workspace carving and launches.  Stated in include/fpd.h.
#include <algorithm>
#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <mutex>

#include "fpd_context.cuh"
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

// SMs of the current device, its kernel attributes set on the first call.
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
    if (e == cudaSuccess) e = shared_attn_init_attributes();
    if (e == cudaSuccess) e = ctx_weights_init_attributes();
    if (e == cudaSuccess) e = evict_init_attributes();
    if (e != cudaSuccess) return e;
    count[dev] = n;
  }
  *sms = count[dev];
  return cudaSuccess;
}

fpd_status check_heads(int batch, int block_len, int nq, int nkv, int h) {
  if (batch < 1 || block_len < 1) return refuse(FPD_ERR_SHAPE, "batch %d, block_len %d", batch, block_len);
  if (h != 64 && h != 128) return refuse(FPD_ERR_UNSUPPORTED, "head_dim %d (64 or 128)", h);
  if (nkv < 1 || nq < nkv || nq % nkv) return refuse(FPD_ERR_SHAPE, "n_q_heads %d must be a multiple of n_kv_heads %d", nq, nkv);
  if ((long long)batch * block_len > kMaxAttnRows || (long long)batch * block_len * nq > kMaxAttnRows)
    return refuse(FPD_ERR_SHAPE, "batch * block_len * n_q_heads exceeds %lld", kMaxAttnRows);
  return FPD_OK;
}

struct AttnWs {
  SharedPlan plan;
  float* o_part;
  float2* ml;
  size_t bytes;
};
// lb is planned as block_len whether or not a call passes block keys: one workspace size serves both.
AttnWs carve(void* base, int batch, int L, int nq, int nkv, int h, int p_cap, int t_cap, int sms) {
  AttnWs w{};
  w.plan = shared_attn_plan(batch, L, L, nq, nkv, h, p_cap, t_cap, sms);
  const size_t n = (size_t)batch * L * nq * w.plan.splits();
  const size_t lead = align_up((uintptr_t)base, 256) - (uintptr_t)base;   // the workspace itself is 16-byte aligned
  const size_t ml_at = align_up(n * h * sizeof(float), 256);
  w.o_part = (float*)((char*)base + lead);
  w.ml = (float2*)((char*)base + lead + ml_at);
  w.bytes = 256 + ml_at + n * sizeof(float2);
  return w;
}

}  // namespace

namespace fpd {
cudaError_t context_ops_init() {
  int sms;
  return device_ready(&sms);
}
}  // namespace fpd

extern "C" {

size_t fpd_shared_attention_workspace_bytes(int batch, int block_len, int n_q_heads, int n_kv_heads, int head_dim,
                                            int prefix_cap, int t_cap) {
  if (check_heads(batch, block_len, n_q_heads, n_kv_heads, head_dim)) return 0;
  if (prefix_cap < 0 || t_cap < 0 || prefix_cap > kMaxStoreCap || t_cap > kMaxStoreCap) return 0;
  int sms = 0;
  if (device_ready(&sms) != cudaSuccess) return 0;
  return carve(nullptr, batch, block_len, n_q_heads, n_kv_heads, head_dim, prefix_cap, t_cap, sms).bytes;
}

fpd_status fpd_shared_attention(int batch, int block_len, int n_q_heads, int n_kv_heads, int head_dim, int layer,
                                const void* q, const void* k_blk, const void* v_blk, const void* prefix_store,
                                int prefix_cap, const int32_t* prefix_len, const void* kv_store, int t_cap,
                                const int32_t* ctx_len, void* out, float* lse, void* workspace, size_t workspace_bytes,
                                void* stream) {
  ApiScope scope("fpd_shared_attention", stream);
  fpd_status s = check_heads(batch, block_len, n_q_heads, n_kv_heads, head_dim);
  if (s) return s;
  if (layer < 0 || prefix_cap < 0 || t_cap < 0 || prefix_cap > kMaxStoreCap || t_cap > kMaxStoreCap)
    return refuse(FPD_ERR_SHAPE, "layer %d, prefix_cap %d, t_cap %d", layer, prefix_cap, t_cap);
  if (!q || !out || !workspace) return refuse(FPD_ERR_INVALID_ARG, "null pointer argument");
  if (!k_blk != !v_blk) return refuse(FPD_ERR_INVALID_ARG, "k_blk and v_blk go together");
  if ((prefix_cap > 0) != (prefix_store && prefix_len) || (!prefix_cap && (prefix_store || prefix_len)))
    return refuse(FPD_ERR_INVALID_ARG, "prefix_cap %d needs prefix_store and prefix_len, 0 neither", prefix_cap);
  if ((t_cap > 0) != (kv_store && ctx_len) || (!t_cap && (kv_store || ctx_len)))
    return refuse(FPD_ERR_INVALID_ARG, "t_cap %d needs kv_store and ctx_len, 0 neither", t_cap);
  const void* al[] = {q, k_blk, v_blk, prefix_store, kv_store, out, workspace};
  for (const void* p : al)
    if (!aligned(p)) return refuse(FPD_ERR_INVALID_ARG, "a device pointer is not 16-byte aligned");
  int sms = 0;
  cudaError_t e = device_ready(&sms);
  if (e != cudaSuccess) return cuda_error(e, "device query");
  const AttnWs w = carve(workspace, batch, block_len, n_q_heads, n_kv_heads, head_dim, prefix_cap, t_cap, sms);
  if (w.bytes > workspace_bytes) return refuse(FPD_ERR_CAPACITY, "workspace %zu < %zu bytes", workspace_bytes, w.bytes);
  SharedAttn a{};
  const size_t pre_half = (size_t)n_kv_heads * prefix_cap * head_dim, own_half = (size_t)n_kv_heads * t_cap * head_dim;
  a.q = (const bf16*)q;
  if (prefix_cap) {
    a.pk = (const bf16*)prefix_store + (size_t)layer * 2 * pre_half;
    a.pv = a.pk + pre_half;
  }
  if (t_cap) {
    a.ck = (const bf16*)kv_store + (size_t)layer * batch * 2 * own_half;
    a.cv = a.ck + own_half;
  }
  a.kblk = (const bf16*)k_blk;
  a.vblk = (const bf16*)v_blk;
  a.prefix_len = prefix_len;
  a.ctx_len = ctx_len;
  a.out = (bf16*)out;
  a.lse = lse;
  a.o_part = w.o_part;
  a.ml = w.ml;
  a.batch = batch;
  a.L = block_len;
  a.lb = k_blk ? block_len : 0;
  a.nq = n_q_heads;
  a.nkv = n_kv_heads;
  a.h = head_dim;
  a.p_cap = prefix_cap;
  a.t_cap = t_cap;
  a.rows = batch * block_len;
  e = launch_shared_attention(a, w.plan, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_error(e, "fpd_shared_attention");
  return scope.done(FPD_OK);
}

fpd_status fpd_context_weights(int batch, int block_len, int n_q_heads, int n_kv_heads, int head_dim, int layer,
                               const void* q, const float* lse, const void* kv_store, int t_cap, const int32_t* ctx_len,
                               float* weights, int accumulate, void* stream) {
  ApiScope scope("fpd_context_weights", stream);
  fpd_status s = check_heads(batch, block_len, n_q_heads, n_kv_heads, head_dim);
  if (s) return s;
  if (layer < 0 || t_cap < 1 || t_cap > kMaxStoreCap) return refuse(FPD_ERR_SHAPE, "layer %d, t_cap %d", layer, t_cap);
  if ((long long)batch * n_kv_heads * ceil_div(t_cap, 64) > INT32_MAX)
    return refuse(FPD_ERR_SHAPE, "batch * n_kv_heads * t_cap %lld is too large", (long long)batch * n_kv_heads * t_cap);
  if (!q || !lse || !kv_store || !ctx_len || !weights) return refuse(FPD_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(q) || !aligned(lse) || !aligned(kv_store) || !aligned(weights))
    return refuse(FPD_ERR_INVALID_ARG, "a device pointer is not 16-byte aligned");
  int sms = 0;
  cudaError_t e = device_ready(&sms);
  if (e != cudaSuccess) return cuda_error(e, "device query");
  CtxWeights a{};
  a.q = (const bf16*)q;
  a.lse = lse;
  a.ck = (const bf16*)kv_store + (size_t)layer * batch * 2 * n_kv_heads * t_cap * head_dim;
  a.ctx_len = ctx_len;
  a.weights = weights + (size_t)layer * batch * n_kv_heads * t_cap;
  a.batch = batch;
  a.L = block_len;
  a.nq = n_q_heads;
  a.nkv = n_kv_heads;
  a.h = head_dim;
  a.t_cap = t_cap;
  a.accumulate = accumulate != 0;
  e = launch_ctx_weights(a, sms, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_error(e, "fpd_context_weights");
  return scope.done(FPD_OK);
}

size_t fpd_evict_workspace_bytes(int n_layers, int batch, int n_kv_heads, int budget) {
  if (n_layers < 1 || batch < 1 || n_kv_heads < 1 || budget < 1) return 0;
  return align_up((size_t)batch * sizeof(int32_t), 256) + (size_t)n_layers * batch * n_kv_heads * budget * sizeof(int32_t);
}

fpd_status fpd_evict_context(int n_layers, int batch, int n_kv_heads, int head_dim, int budget, int recent, const void* kv_store,
                             int t_cap, const float* weights, const int32_t* ctx_len, void* out_store, int out_cap,
                             float* out_weights, int32_t* out_len, int32_t* pos_offset, int32_t* kept, void* workspace,
                             size_t workspace_bytes, void* stream) {
  ApiScope scope("fpd_evict_context", stream);
  if (n_layers < 1 || batch < 1 || n_kv_heads < 1 || t_cap < 1 || out_cap < 1 || t_cap > kMaxStoreCap || out_cap > kMaxStoreCap)
    return refuse(FPD_ERR_SHAPE, "n_layers %d, batch %d, n_kv_heads %d, t_cap %d, out_cap %d", n_layers, batch, n_kv_heads,
                  t_cap, out_cap);
  if (head_dim != 64 && head_dim != 128) return refuse(FPD_ERR_UNSUPPORTED, "head_dim %d (64 or 128)", head_dim);
  if (recent < 0 || budget < 1 || recent > budget || budget > out_cap)
    return refuse(FPD_ERR_SHAPE, "0 <= recent %d <= budget %d <= out_cap %d does not hold", recent, budget, out_cap);
  const long long heads = (long long)n_layers * batch * n_kv_heads;
  if (heads * 2 * std::max(8, ceil_div(budget, 64)) > INT32_MAX) return refuse(FPD_ERR_SHAPE, "%lld heads times budget %d is too large", heads, budget);
  if (!kv_store || !weights || !ctx_len || !out_store || !out_weights || !out_len || !workspace)
    return refuse(FPD_ERR_INVALID_ARG, "null pointer argument");
  const void* al[] = {kv_store, weights, out_store, out_weights, kept, workspace};
  for (const void* p : al)
    if (!aligned(p)) return refuse(FPD_ERR_INVALID_ARG, "a device pointer is not 16-byte aligned");
  const size_t need = fpd_evict_workspace_bytes(n_layers, batch, n_kv_heads, budget);
  if (need > workspace_bytes) return refuse(FPD_ERR_CAPACITY, "workspace %zu < %zu bytes", workspace_bytes, need);
  // in place means both the store and its weights, at the same capacity; any other overlap would be read after it is written
  const size_t src_bytes = (size_t)heads * 2 * t_cap * head_dim * sizeof(bf16), dst_bytes = (size_t)heads * 2 * out_cap * head_dim * sizeof(bf16);
  const size_t sw_bytes = (size_t)heads * t_cap * sizeof(float), dw_bytes = (size_t)heads * out_cap * sizeof(float);
  auto overlap = [](const void* a, size_t na, const void* b, size_t nb) {
    return (uintptr_t)a < (uintptr_t)b + nb && (uintptr_t)b < (uintptr_t)a + na;
  };
  const bool in_place = kv_store == out_store;
  if (in_place != (weights == out_weights) || (in_place && t_cap != out_cap))
    return refuse(FPD_ERR_INVALID_ARG, "in place, out_store, out_weights and out_cap are kv_store, weights and t_cap");
  if (!in_place && (overlap(kv_store, src_bytes, out_store, dst_bytes) || overlap(weights, sw_bytes, out_weights, dw_bytes)))
    return refuse(FPD_ERR_INVALID_ARG, "the new store or its weights overlap the old ones");
  int sms = 0;
  cudaError_t e = device_ready(&sms);
  if (e != cudaSuccess) return cuda_error(e, "device query");
  Evict v{};
  v.store = (const bf16*)kv_store;
  v.out_store = (bf16*)out_store;
  v.weights = weights;
  v.out_weights = out_weights;
  v.ctx_len = ctx_len;
  v.out_len = out_len;
  v.pos_offset = pos_offset;
  v.old_len = (int32_t*)workspace;
  v.kept = kept ? kept : (int32_t*)((char*)workspace + align_up((size_t)batch * sizeof(int32_t), 256));
  v.layers = n_layers;
  v.batch = batch;
  v.nkv = n_kv_heads;
  v.h = head_dim;
  v.t_cap = t_cap;
  v.out_cap = out_cap;
  v.budget = budget;
  v.recent = recent;
  v.in_place = in_place;
  e = launch_evict(v, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_error(e, "fpd_evict_context");
  return scope.done(FPD_OK);
}

}  // extern "C"
