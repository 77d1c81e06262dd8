// Internal declarations of what lies between a layer's ternary products: cache,
// attention, residual join.
#pragma once

#include "bitnet_internal.h"

namespace bitnet {

// Largest grid of workgroups of t threads: the runtime counts threads in 32 bits.
constexpr int64_t max_grid(int threads) { return ((int64_t)1 << 32) / threads - 1; }

// Paged 8-bit cache of one layer's keys and values (bitnet_kv_cache, validated).
struct KvCache {
  int8_t* k;                 // [pages][kv_heads][page][head_dim]
  int8_t* v;                 // [pages][kv_heads][head_dim][page]
  float* k_scale;            // [pages][kv_heads]
  float* v_scale;
  int pages, kv_heads, page, head_dim;
};
// Ragged batch (bitnet_kv_batch, validated).
struct KvBatch {
  const int32_t* table;      // [seqs][width] page ids
  const int32_t* q_start;    // [seqs + 1]
  const int32_t* kv_len;     // [seqs]
  int seqs, width, tokens, max_new, max_len;
};

// What one sequence of a batch adds: rows [s0, s0 + n) at positions first ..
// first + n - 1 (negative ones have no place in the cache); it then holds len
// tokens.  The numbers lie in device memory, where the host cannot check them:
// they are clamped to the batch, so that no kernel leaves its buffers.
struct SeqSpan {
  int s0, n, first, len;
};
__device__ __forceinline__ SeqSpan seq_span(const KvBatch& b, int seq) {
  const int t0 = b.q_start[seq], t1 = b.q_start[seq + 1], ln = b.kv_len[seq];
  SeqSpan r;
  r.s0 = min(max(t0, 0), b.tokens);
  r.n = min(max(t1, r.s0), b.tokens) - r.s0;
  r.len = min(max(ln, 0), b.max_len);
  r.first = r.len - r.n;
  return r;
}

// New rows of the cache and the queries that are rotated beside them.
struct KvRows {
  const void *k, *v, *q;     // q: nullptr for none
  void* q_out;               // [tokens][q_heads][head_dim]
  int64_t k_stride, v_stride, q_stride;   // elements between tokens
  int q_heads;
  const float *cos, *sin;    // [positions][rot / 2]
  int rot;                   // rotated dims (0: none)
  int neighbours;            // pairs (2i, 2i + 1) instead of (i, i + rot / 2)
};
// Workgroups of the launch.
int64_t kv_append_grid(const KvCache& c, const KvBatch& b, bool queries);
hipError_t launch_kv_append(const KvCache& c, const KvBatch& b, const KvRows& r, bool bf16,
                            hipStream_t s);

// Attention of the batch's query rows over the cache.
struct AttnArgs {
  const void* q;             // [tokens][q_heads][head_dim], q_stride elements between tokens
  void* out;                 // [tokens][q_heads][head_dim]
  float* lse;                // [tokens][q_heads] or nullptr
  int64_t q_stride;
  int q_heads, window;       // window 0: every earlier token
  float scale;
};
size_t attention_workspace_bytes(const KvCache& c, const KvBatch& b, int q_heads);
// Whether the launches' grids are within the runtime's limits.
bool attention_fits(const KvCache& c, const KvBatch& b, int q_heads);
hipError_t launch_attention(const KvCache& c, const KvBatch& b, const AttnArgs& a, bool q_bf16,
                            bool out_bf16, void* workspace, hipStream_t s);
// Residual join (bitnet_residual, validated).
struct ResidualArgs {
  const void *y, *h, *gate;
  void *h_out, *u;
  const float *post, *pre;
  int8_t* xq;
  float* xs;
  int64_t K, gate_stride;
  float scale, eps;
};
hipError_t launch_residual(const ResidualArgs& a, bool y_bf16, bool h_bf16, bool u_bf16, int64_t M,
                           hipStream_t s);

}  // namespace bitnet
