// fpd_context.cuh — launch interfaces of the operators on a context store: attention over a shared prefix, collected
// attention weight, eviction (internal to libfpd; the public calls are in include/fpd.h).
#pragma once

#include "fpd_kernels.cuh"

namespace fpd {

constexpr int kMaxStoreCap = 1 << 30;             // positions of a store: key indices and tile ends stay below 2^31
constexpr long long kMaxAttnRows = 1ll << 26;     // batch * block_len * n_q_heads of one attention call
cudaError_t context_ops_init();                   // kernel attributes, once per device

// Attention of a batch over [shared prefix ; own context ; block].  Every pointer may belong to one layer's slice.
struct SharedAttn {
  const bf16* q;                        // [rows][nq][h]
  const bf16 *pk, *pv;                  // prefix K and V [nkv][p_cap][h], or null
  const bf16 *ck, *cv;                  // own context K and V of request 0 ([nkv][t_cap][h]; requests 2 nkv t_cap h apart), or null
  const bf16 *kblk, *vblk;              // [batch][nkv][L][h], or null
  const int32_t *prefix_len, *ctx_len;  // device [1], [batch]
  bf16* out;                            // [rows][nq][h]
  float* lse;                           // [rows][nq] or null
  float* o_part;                        // [splits][rows][nq][h], 32-byte aligned
  float2* ml;                           // [splits][rows][nq]: running maximum (base 2) and sum
  int batch, L, lb, nq, nkv, h, p_cap, t_cap, rows;   // lb: keys of the block, L or 0; rows = batch * L
};

// How the work of a call is cut.  The prefix part has the rows of all requests per kv head, the own part one request's;
// each goes to tcgen05 (units of 256 rows, k_attention_shared_tc.cu) or to mma.sync (tiles of 64 rows).
struct SharedPlan {
  bool pre_tc, own_tc;
  int pre_tiles, pre_splits;            // row units of a kv head (0: no such part), partials of a row
  int own_tiles, own_splits;            // the same per request
  int pre_runs, pre_pieces;             // CTAs that share the prefix's tiles, most of them in one unit
  int own_cost;                         // an own run in the prefix's key tiles, 0: not counted when the prefix is shared out
  int tc_grid;                          // CTAs of the tcgen05 kernel
  int own_ctas, own_alone;              // of them, from the last, without a run of the prefix; own runs that each takes first
  int splits() const { return pre_splits + own_splits; }
};
SharedPlan shared_attn_plan(int batch, int L, int lb, int nq, int nkv, int h, int p_cap, int t_cap, int num_sms);
cudaError_t shared_attn_init_attributes();
cudaError_t shared_attn_tc_init_attributes();
cudaError_t launch_shared_tc(const SharedAttn& a, const SharedPlan& pl, cudaStream_t st);
cudaError_t launch_shared_attention(const SharedAttn& a, const SharedPlan& pl, cudaStream_t st);

// weights[b][g][t] (+)= sum over the request's rows of kv head g of exp(q . k_t / sqrt(h) - lse)
struct CtxWeights {
  const bf16* q;            // [batch * L][nq][h]
  const float* lse;         // [batch * L][nq]
  const bf16* ck;           // K of request 0, [nkv][t_cap][h]; requests 2 nkv t_cap h apart
  const int32_t* ctx_len;   // device [batch]
  float* weights;           // [batch][nkv][t_cap]
  int batch, L, nq, nkv, h, t_cap, accumulate;
};
cudaError_t ctx_weights_init_attributes();
bool ctx_weights_tc_supported(const CtxWeights& a);
cudaError_t ctx_weights_tc_init_attributes();
cudaError_t launch_ctx_weights_tc(const CtxWeights& a, int num_sms, cudaStream_t st);
cudaError_t launch_ctx_weights(const CtxWeights& a, int num_sms, cudaStream_t st);

struct Evict {
  const bf16* store;
  bf16* out_store;
  const float* weights;
  float* out_weights;
  const int32_t* ctx_len;
  int32_t *out_len, *pos_offset, *kept, *old_len;   // pos_offset null or [batch]; old_len scratch [batch]
  int layers, batch, nkv, h, t_cap, out_cap, budget, recent;
  bool in_place;                                    // out_store is store
};
cudaError_t evict_init_attributes();
cudaError_t launch_evict(const Evict& e, cudaStream_t st);

// base[b] = ctx_len[b] (clamped to [0, t_cap]; 0 without one) + pos_offset[b]: the rotary position of a block's first
// slot.  Without pos_offset the prefix's length stands in for it.
cudaError_t launch_rope_base(int32_t* base, const int32_t* ctx_len, const int32_t* prefix_len, const int32_t* pos_offset,
                             int batch, int t_cap, int p_cap, cudaStream_t st);

}  // namespace fpd
