// Attention over the paged 8-bit cache: which kernel a call takes, and the join of
// the parts that either of them leaves.
#include "attn_internal.h"

namespace bitnet {
namespace {

constexpr int kThreads = 256;

// Joins the parts of one column: the softmax formula over their maxima and sums.  A
// workgroup a column; thread (d, k) takes dims 4 d .. and parts k, k + parts at once, ..,
// and the threads of equal d are joined in LDS, so that the order of the sums is fixed.
template <bool OB>
__global__ __launch_bounds__(kThreads) void attn_join_kernel(const KvCache c, const KvBatch b,
                                                             const AttnArgs a,
                                                             const AttnPlan plan, float unit,
                                                             const float* __restrict__ part) {
  __shared__ float4 sy[kThreads];
  __shared__ float2 sml[kThreads];
  const int u = blockIdx.x / plan.part_cols, col = blockIdx.x % plan.part_cols;
  const int ct = u % plan.tiles;
  const int head = u / plan.tiles % c.kv_heads;
  const int seq = u / plan.tiles / c.kv_heads;
  const AttnTile tile = attn_tile(b, seq, ct, plan.cols, plan.group, a.window);
  if (col >= tile.nc) return;
  const int each = attn_part(tile.steps, plan.splits, plan.least);
  if (tile.steps <= each) return;   // written by its only part
  const int used = (tile.steps + each - 1) / each;
  const int D = c.head_dim, d4 = D / 4, groups = kThreads / d4;
  const int k = threadIdx.x / d4, d = (threadIdx.x - k * d4) * 4;
  const int64_t stride = (int64_t)plan.part_cols * (D + 4);
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
  if (k < groups) {
    for (int s = k; s < used; s += groups) top = fmaxf(top, p[s * stride]);
    for (int s = k; s < used; s += groups)
      add(*reinterpret_cast<const float2*>(p + s * stride),
          *reinterpret_cast<const float4*>(p + s * stride + 4 + d));
    sy[threadIdx.x] = y;
    sml[threadIdx.x] = make_float2(top, l);
  }
  __syncthreads();
  if (k > 0) return;
  const int n = groups < used ? groups : used;
  for (int i = 1; i < n; ++i) top = fmaxf(top, sml[i * d4 + threadIdx.x].x);
  l = 0.0f;
  y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int i = 0; i < n; ++i) add(sml[i * d4 + threadIdx.x], sy[i * d4 + threadIdx.x]);
  const float r = l > 0.0f ? 1.0f / (l * unit) : 0.0f;
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

// Columns (rows x query heads of a kv head) from which the prompt kernel is taken.  32
// sequences of 1000 tokens, 8 kv heads: 32 columns 25.6 us with the decode kernel, 31.1
// with this one; 48 columns 36.6 and 32.0; 64 columns 43.8 and 31.9.  Few sequences and
// heads do not fill the chip with its workgroups: one of 4096 tokens takes 15.8 and 23.5
// us with 64 columns, 26.0 and 30.3 with 256.
bool many_rows(const KvCache& c, const KvBatch& b, int q_heads) {
  const int64_t cols = (int64_t)b.max_new * (q_heads / c.kv_heads);
  return cols >= ((int64_t)b.seqs * c.kv_heads >= 32 ? 48 : 512);
}

}  // namespace

hipError_t launch_attn_join(const KvCache& c, const KvBatch& b, const AttnArgs& a,
                            const AttnPlan& p, float unit, bool out_bf16, const float* part,
                            hipStream_t s) {
  const int64_t grid = (int64_t)b.seqs * c.kv_heads * p.tiles * p.part_cols;
  void* args[] = {(void*)&c, (void*)&b, (void*)&a, (void*)&p, (void*)&unit, (void*)&part};
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
