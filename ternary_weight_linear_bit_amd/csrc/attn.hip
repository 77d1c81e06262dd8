// Attention over the paged 8-bit cache: which kernel a call takes, and the join of
// the parts that either of them leaves.
#include "attn_internal.h"

namespace bitnet {
namespace {

constexpr int kThreads = 256;

// Joins the parts of a tile's columns: the softmax formula over their maxima and sums.
// A workgroup takes join_cols() columns, `ways` threads for each 4 dims of a column,
// which take every ways-th part and are joined in LDS, so that the order of the sums is
// fixed.
template <bool OB>
__global__ __launch_bounds__(kThreads) void attn_join_kernel(const KvCache c, const KvBatch b,
                                                             const AttnArgs a,
                                                             const AttnPlan plan, int ways, int cols,
                                                             const float* __restrict__ part) {
  __shared__ float4 sy[kThreads];
  __shared__ float2 sml[kThreads];
  const int chunks = (plan.part_cols + cols - 1) / cols;
  const int u = blockIdx.x / chunks, first = (blockIdx.x - u * chunks) * cols;
  const int ct = u % plan.tiles;
  const int head = u / plan.tiles % c.kv_heads;
  const int seq = u / plan.tiles / c.kv_heads;
  const AttnTile tile = attn_tile(b, seq, ct, plan.cols, plan.group, a.window);
  if (first >= tile.nc) return;
  const int each = attn_part(tile.steps, plan.splits, plan.least);
  if (tile.steps <= each) return;   // written by its only part
  const int used = (tile.steps + each - 1) / each;
  const int D = c.head_dim, d4 = D / 4;
  const int at_once = kThreads / (d4 * ways);   // columns
  const int t = threadIdx.x % (d4 * ways), mine = threadIdx.x / (d4 * ways);
  const int way = t / d4, d = (t - way * d4) * 4;
  const int64_t stride = (int64_t)plan.part_cols * (D + 4);
  const int end = min(first + cols, tile.nc);
  for (int c0 = first; c0 < end; c0 += at_once) {
    const int col = c0 + mine;
    const bool on = mine < at_once && col < end;
    const float* p = part + (int64_t)u * plan.splits * stride + (int64_t)col * (D + 4);
    float top = -INFINITY, l = 0.0f;
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [&](float2 ml, float4 z) {   // y, l at the maximum `top`
      const float f = ml.x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ml.x - top);
      l = __builtin_fmaf(ml.y, f, l);
      y.x = __builtin_fmaf(z.x, f, y.x);
      y.y = __builtin_fmaf(z.y, f, y.y);
      y.z = __builtin_fmaf(z.z, f, y.z);
      y.w = __builtin_fmaf(z.w, f, y.w);
    };
    if (on) {
      for (int s = way; s < used; s += ways) top = fmaxf(top, p[s * stride]);
      for (int s = way; s < used; s += ways)
        add(*reinterpret_cast<const float2*>(p + s * stride),
            *reinterpret_cast<const float4*>(p + s * stride + 4 + d));
    }
    if (ways > 1) {
      __syncthreads();   // the columns before are joined
      sy[threadIdx.x] = y;
      sml[threadIdx.x] = make_float2(top, l);
      __syncthreads();
      if (way == 0 && on) {
        for (int i = 1; i < ways; ++i) top = fmaxf(top, sml[threadIdx.x + i * d4].x);
        l = 0.0f;
        y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int i = 0; i < ways; ++i) add(sml[threadIdx.x + i * d4], sy[threadIdx.x + i * d4]);
      }
    }
    if (way > 0 || !on) continue;
    const float r = l > 0.0f ? 1.0f / l : 0.0f;
    const int oc = tile.c0 + col, row = oc / plan.group;
    const int64_t at =
        (tile.sp.s0 + row) * (int64_t)a.q_heads + head * plan.group + (oc - row * plan.group);
    if (OB)
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + at * D + d) =
          make_uint2(bf16x2_rne(y.x * r, y.y * r), bf16x2_rne(y.z * r, y.w * r));
    else
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + at * D + d) =
          make_float4(y.x * r, y.y * r, y.z * r, y.w * r);
    if (d == 0 && a.lse)
      a.lse[at] = l > 0.0f ? 0.69314718055994530942f * (top + __builtin_amdgcn_logf(l)) : -INFINITY;
  }
}

// Threads for 4 dims of a column: as many as there are parts, up to a workgroup's.
int join_ways(const KvCache& c, const AttnPlan& p) {
  int ways = 1;
  while (ways < p.splits && 2 * ways * (c.head_dim / 4) <= kThreads) ways *= 2;
  return ways;
}
// Columns of a workgroup: those that its threads take at once, but 16 of the prompt
// kernel's tiles (a column each: 84480 workgroups, 90 us for six parts of prompts).
int join_cols(const KvCache& c, const AttnPlan& p, int ways) {
  const int at_once = kThreads / (c.head_dim / 4 * ways);
  return p.cols > 16 && at_once < 16 ? 16 : at_once;
}

// Whether a call takes the prompt kernel.  cols: rows x query heads of a kv head.  Its
// workgroups of 128 columns have to fill half of the chip (us, decode and prompt kernel, 32
// heads on 8, bf16: one prompt of 256 tokens 11.2 and 15.8, of 512 26.9 and 21.8, of 1024
// 61 and 50; 256 rows behind 3840 tokens 62 and 64, 512 behind 3584 109 and 70).  From 48
// columns on it is also taken where the cache passes the L2s, since the decode kernel reads
// it for every 16 columns (12 rows a sequence, 8 sequences of 8192 tokens: 85 and 69, 16 of
// them: 135 and 92; 8 of 4096: 51 and 53; 64 rows of one of 32768: 113 and 106, 32 rows of
// one of 65536: 121 and 139; 4 rows of 16 of 8192: 50 and 75).
bool many_rows(const KvCache& c, const KvBatch& b, int q_heads) {
  const int64_t pairs = (int64_t)b.seqs * c.kv_heads;
  const int64_t cols = (int64_t)b.max_new * (q_heads / c.kv_heads);
  return pairs * cols >= 128 * 128 ||
         (cols >= 48 && pairs * b.max_len >= (int64_t)(64 << 20) / (2 * c.head_dim));
}

}  // namespace

hipError_t launch_attn_join(const KvCache& c, const KvBatch& b, const AttnArgs& a,
                            const AttnPlan& p, bool out_bf16, const float* part,
                            hipStream_t s) {
  int ways = join_ways(c, p), cols = join_cols(c, p, ways);
  const int64_t grid = (int64_t)b.seqs * c.kv_heads * p.tiles * ((p.part_cols + cols - 1) / cols);
  void* args[] = {(void*)&c, (void*)&b, (void*)&a, (void*)&p, (void*)&ways, (void*)&cols,
                  (void*)&part};
  return hipLaunchKernel(out_bf16 ? (const void*)attn_join_kernel<true>
                                  : (const void*)attn_join_kernel<false>,
                         dim3((unsigned)grid), dim3(kThreads), args, 0, s);
}

size_t attention_workspace_bytes(const KvCache& c, const KvBatch& b, int q_heads) {
  return attn_workspace(c, b, many_rows(c, b, q_heads) ? attn_prompt_plan(c, b, q_heads)
                                                       : attn_decode_plan(c, b, q_heads));
}

bool attention_fits(const KvCache& c, const KvBatch& b, int q_heads) {
  const AttnPlan p = many_rows(c, b, q_heads) ? attn_prompt_plan(c, b, q_heads)
                                              : attn_decode_plan(c, b, q_heads);
  const int64_t tiles = (int64_t)b.seqs * c.kv_heads * p.tiles;
  return tiles * p.splits <= max_grid(512) && (p.splits == 1 || tiles * p.part_cols <= max_grid(kThreads));
}

hipError_t launch_attention(const KvCache& c, const KvBatch& b, const AttnArgs& a, bool q_bf16,
                            bool out_bf16, void* workspace, hipStream_t s) {
  if (many_rows(c, b, a.q_heads))
    return launch_attn_prompt(c, b, a, attn_prompt_plan(c, b, a.q_heads), q_bf16, out_bf16, workspace, s);
  return launch_attn_decode(c, b, a, attn_decode_plan(c, b, a.q_heads), q_bf16, out_bf16, workspace, s);
}

}  // namespace bitnet
