// Shared by the attention kernels: what a workgroup works on, and how a launch
// splits the keys of a sequence over workgroups.
#pragma once

#include "layer_internal.h"

namespace bitnet {

constexpr int kAttnStep = 64;   // keys of one step
// Weights e^(s - m) dv below 2^-kReach of their row's largest may count as 0 in the output: a
// row's sums (the softmax sum divides by dv, 2^-40 or more) then stay in fp32's range whatever
// step's reference they are taken over, and 2^24 such weights are less than half of fp32's last
// bit of the row's.
constexpr float kReach = 48.0f;

// Columns [c0, c0 + nc) of a sequence's (row, query head of the group) pairs, rows
// outermost, and the 64-key steps that those rows see.
struct AttnTile {
  SeqSpan sp;
  int c0, nc;              // nc <= 0: nothing
  int step0, steps;
};
__device__ __forceinline__ AttnTile attn_tile(const KvBatch& b, int seq, int tile, int cols,
                                              int group, int window) {
  AttnTile t;
  t.sp = seq_span(b, seq);
  t.c0 = tile * cols;
  t.nc = min(min(t.sp.n, b.max_new) * group - t.c0, cols);
  const int p0 = t.sp.first + t.c0 / group;                       // first and last row's positions
  const int p1 = t.sp.first + (t.c0 + max(t.nc, 1) - 1) / group;
  const int lo = window > 0 ? max(p0 - window + 1, 0) : 0;
  t.step0 = lo / kAttnStep;
  t.steps = p1 < lo ? 0 : p1 / kAttnStep + 1 - t.step0;
  return t;
}

// Dims d0 .. d0 + W - 1 of a query row that begins at element `base`; zeros past
// the head's D (a multiple of 16, as d0 + W at most passes it as a whole).  Rows are
// aligned to their elements only.
template <bool BF16, int W>
__device__ __forceinline__ void load_dims(const void* q, int64_t base, int d0, int D, float x[W]) {
  const bool in = d0 < D;
  const int64_t at = base + (in ? d0 : 0);
  if (BF16) {
    uint16_t w[W];
    __builtin_memcpy(w, reinterpret_cast<const uint16_t*>(q) + at, sizeof(w));
#pragma unroll
    for (int j = 0; j < W; ++j) x[j] = in ? bf16_bits_to_float(w[j]) : 0.0f;
  } else {
    float w[W];
    __builtin_memcpy(w, reinterpret_cast<const float*>(q) + at, sizeof(w));
#pragma unroll
    for (int j = 0; j < W; ++j) x[j] = in ? w[j] : 0.0f;
  }
}

// Steps of each part when a tile's steps are split over at most `splits` workgroups:
// equal parts of at least `least`, so that a short sequence uses few of them.  A tile
// of one part is written by its workgroup, the others by the join kernel.
__device__ __forceinline__ int attn_part(int steps, int splits, int least) {
  return max((steps + splits - 1) / splits, least);
}

// What both kernels' launches share.
struct AttnPlan {
  int group, page_shift;
  int cols, tiles;          // columns a workgroup, tiles of a sequence
  int splits, least;
  int part_cols;            // columns of a tile's partial sums
  int waves;                // of a workgroup
};
// A part of a tile in the workspace: part_cols columns of head_dim + 4 floats: the
// maximum m (log2), the sum of 2^(x - m) / dv, two unused, and the sums over 2^(x - m) vc.
hipError_t launch_attn_join(const KvCache& c, const KvBatch& b, const AttnArgs& a,
                            const AttnPlan& p, bool out_bf16, const float* part,
                            hipStream_t s);

inline AttnPlan attn_plan(const KvCache& c, const KvBatch& b, int q_heads, int cols,
                          int workgroups, int least) {
  AttnPlan p{};
  p.group = q_heads / c.kv_heads;
  p.page_shift = 4;
  while ((1 << p.page_shift) < c.page) ++p.page_shift;
  const int64_t all = (int64_t)b.max_new * p.group;
  p.cols = cols;
  p.tiles = (int)((all + cols - 1) / cols);
  p.part_cols = (int)(all < cols ? all : cols);
  p.least = least;
  const int64_t units = (int64_t)b.seqs * c.kv_heads * p.tiles;
  const int64_t steps = ((int64_t)b.max_len + kAttnStep - 1) / kAttnStep;
  const int64_t want = (workgroups + units - 1) / units;
  const int64_t most = (steps + least - 1) / least;
  const int64_t s = want < most ? want : most;
  p.splits = s < 1 ? 1 : (int)s;
  return p;
}
inline size_t attn_workspace(const KvCache& c, const KvBatch& b, const AttnPlan& p) {
  if (p.splits == 1) return 0;
  return (size_t)b.seqs * c.kv_heads * p.tiles * p.splits * p.part_cols * (c.head_dim + 4) *
         sizeof(float);
}

// Few rows (attn_decode.hip), many rows (attn_prompt.hip).
AttnPlan attn_decode_plan(const KvCache& c, const KvBatch& b, int q_heads);
hipError_t launch_attn_decode(const KvCache& c, const KvBatch& b, const AttnArgs& a,
                              const AttnPlan& p, bool q_bf16, bool out_bf16, void* workspace,
                              hipStream_t s);
AttnPlan attn_prompt_plan(const KvCache& c, const KvBatch& b, int q_heads);
hipError_t launch_attn_prompt(const KvCache& c, const KvBatch& b, const AttnArgs& a,
                              const AttnPlan& p, bool q_bf16, bool out_bf16, void* workspace,
                              hipStream_t s);

}  // namespace bitnet
