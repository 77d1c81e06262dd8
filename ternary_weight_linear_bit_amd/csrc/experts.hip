// Ternary products whose rows are grouped by expert, with bias, activation, gating and residual
// behind the product; a dense product is the case of one expert with every row.
//
//   v = RN32(RN32(acc * RN32(gamma_e * d)) + b),  a = act(v) or RN32(act(v) * u),
//   y = RN(RN32(a + residual)),  u as v of the second matrix.
//
// Weights lie in the prefill layout (blocks of 32 rows x 128 k, 1024 bytes, in the lanes' order).
#include "experts_internal.h"

namespace bitnet {
namespace {

typedef int v16i __attribute__((ext_vector_type(16)));

// ---------------------------------------------------------------------------
// few rows an expert: the weights stream once from memory
// ---------------------------------------------------------------------------
//
// A workgroup takes 32 output rows of one expert (of both its matrices) and up to 32 slots; its W
// waves share the k steps, and their integer sums meet in LDS (order does not matter to them).
// Lane (r, h) of the 32 x 32 x 32 product holds row r: weights as the layout's 16 bytes a lane,
// the slots' rows straight from memory (a few KiB that all workgroups share; lanes without a slot
// read the first slot's, and nothing of theirs is kept).
constexpr int kFewRows = 32;

template <int W, bool GATED>
__global__ __launch_bounds__(64 * W) void experts_few_kernel(const ExpertArgs a, int nblocks) {
  constexpr int NM = GATED ? 2 : 1;
  __shared__ int sum[NM][kFewRows][33];
  __shared__ int row_of[kFewRows];
  __shared__ float d_of[kFewRows];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, h = lane >> 5;
  const int nb = (int)blockIdx.x % nblocks;
  const ExpertTile t = expert_tile<kFewRows>(a, (int)blockIdx.x / nblocks);
  if (t.rows <= 0) return;
  const int steps = (a.K + 127) / 128;
  const size_t at = ((size_t)t.expert * nblocks + nb) * steps * 1024;
  const uint4* wp[2] = {reinterpret_cast<const uint4*>(a.w + at) + lane,
                        reinterpret_cast<const uint4*>((GATED ? a.up : a.w) + at) + lane};
  for (int i = tid; i < NM * kFewRows * 33; i += 64 * W) (&sum[0][0][0])[i] = 0;
  const int mine = r < t.rows ? input_row(a, t.slot0 + r) : -1;
  if (wave == 0 && h == 0) {
    row_of[r] = mine;
    d_of[r] = mine < 0 ? 0.0f : a.xs[mine];
  }
  const int8_t* x = a.xq + (size_t)max(mine, 0) * a.K;
  v16i acc[NM];
#pragma unroll
  for (int m = 0; m < NM; ++m) acc[m] = (v16i){};
  for (int s = wave; s < steps; s += W) {
    const int k = 128 * s + 64 * h;
    const int8_t* xk = x + (k < a.K ? k : 0);      // past K the weights are 0
    v4i xv[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) xv[j] = *reinterpret_cast<const v4i*>(xk + 16 * j);
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      const uint4 w = wp[m][(size_t)s * 64];
      const uint32_t wd[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[m] = __builtin_amdgcn_mfma_i32_32x32x32_i8(xv[j], weights_64(wd[j]), acc[m], 0, 0, 0);
    }
  }
  __syncthreads();
  // lane l holds output row l % 32 and slots 8 (v / 4) + 4 (l / 32) + v % 4
#pragma unroll
  for (int m = 0; m < NM; ++m)
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int sl = 8 * (v >> 2) + 4 * h + (v & 3);
      if (sl < t.rows) atomicAdd(&sum[m][sl][r], acc[m][v]);
    }
  __syncthreads();
  const int n = 32 * nb + (tid & 31);
  if (n >= a.N) return;
  const size_t en = (size_t)t.expert * a.N + n;
  const float g0 = a.w_scale[t.expert], b0 = a.bias ? a.bias[en] : 0.0f;
  const float g1 = GATED ? a.up_scale[t.expert] : 0.0f, b1 = GATED && a.up_bias ? a.up_bias[en] : 0.0f;
  for (int sl = tid >> 5; sl < t.rows; sl += 2 * W) {
    if (row_of[sl] < 0) continue;
    const float d = d_of[sl];
    float v = acc_64(sum[0][sl][tid & 31]) * (g0 * d);
    if (a.bias) v = v + b0;
    v = activate(v, a.act);
    if (GATED) {
      float u = acc_64(sum[NM - 1][sl][tid & 31]) * (g1 * d);
      if (a.up_bias) u = u + b1;
      v = v * u;
    }
    const size_t o = (size_t)(t.slot0 + sl) * a.N + n;
    store_output(a, o, v);
  }
}

int64_t few_grid(const ExpertArgs& a) {
  return many_tiles(a, kFewRows) * ((a.N + 31) / 32);
}

}  // namespace

bool experts_fit(const ExpertArgs& a) { return few_grid(a) <= max_grid(512); }

hipError_t launch_experts(const ExpertArgs& a, hipStream_t s) {
  // tiles of each shape, if the slots were spread evenly over the experts
  const int64_t used = a.experts < a.slots ? a.experts : a.slots, each = (a.slots + used - 1) / used;
  auto tiles = [&](int rows, int cols) {
    return used * ((each + rows - 1) / rows) * ((a.N + cols - 1) / cols);
  };
  const int wide = a.up ? 128 : 256;
  if (each > 8 && tiles(kFewRows, 32) > 512) {
    if (each >= 192 && tiles(128, wide) >= 256) return launch_experts_many(a, 128, s);
    return launch_experts_many(a, tiles(64, wide) >= 256 ? 64 : 32, s);
  }
  const int nblocks = (a.N + 31) / 32;
  const dim3 grid((unsigned)few_grid(a));
  if (a.up)
    hipLaunchKernelGGL((experts_few_kernel<8, true>), grid, dim3(512), 0, s, a, nblocks);
  else
    hipLaunchKernelGGL((experts_few_kernel<8, false>), grid, dim3(512), 0, s, a, nblocks);
  return hipGetLastError();
}

}  // namespace bitnet
