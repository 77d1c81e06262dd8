// Ternary products whose rows are grouped by expert, with bias, activation, gating and residual
// behind the product; a dense product is the case of one expert with every row.
//
//   v = RN32(RN32(acc * RN32(gamma_e * d)) + b),  a = act(v) or RN32(act(v) * u),
//   y = RN(RN32(a + residual)),  u as v of the second matrix.
//
// Weights lie in the prefill layout (blocks of 32 rows x 128 k, 1024 bytes, in the lanes' order).
#include "experts_internal.h"

#include <math.h>

namespace bitnet {
namespace {

typedef int v16i __attribute__((ext_vector_type(16)));

// ---------------------------------------------------------------------------
// few rows an expert: the weights stream once from memory
// ---------------------------------------------------------------------------
//
// A workgroup takes up to 32 slots of one expert and 32 output rows (of both its matrices); its 8
// waves share the k steps, S of them in flight a wave, and their integer sums meet in LDS (order
// does not matter to them).  Lane (r, h) of the 32 x 32 x 32 product holds row r: weights as the
// layout's 16 bytes a lane, the slots' rows straight from memory (a few KiB that all workgroups
// share; lanes without a slot read another's, and nothing of theirs is kept).  Past the end of K, and
// in steps past the last, x is read outside its buffer, which gives zeros.
// Bound by latency (the offsets, the pair and the row are loads behind each other; the weights need
// the first alone and are under way meanwhile): one token through gate and up of two 2560 -> 6912
// experts, 17.7 MB, 6.3-7.6 us replayed from a graph; 2560 -> 2560 3.8-4.4.  A load of x touches as many lines as
// there are rows, so that from about 16 rows on the staged kernel is faster where it fills the chip
// (4096 -> 14336 at 32 rows: 11.9 us here, 9.5 there; at 8 rows 7.5 and 8.4).  Two steps in flight
// against one: 14336 -> 4096, one row, two experts 9.2 and 10.6 us; K = 2560 8.2 and 7.6.
constexpr int kFewRows = 32, kFewWaves = 8;

template <int S, bool GATED>
__global__ __launch_bounds__(64 * kFewWaves) void experts_few_kernel(const ExpertArgs a, int nblocks) {
  constexpr int NM = GATED ? 2 : 1, W = kFewWaves;
  __shared__ int sum[NM][kFewRows][33];
  __shared__ int row_of[kFewRows];
  __shared__ float d_of[kFewRows];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, h = lane >> 5;
  const int nb = (int)blockIdx.x % nblocks;
  const int tile = (int)blockIdx.x / nblocks;
  const ExpertSpan t = expert_span<kFewRows>(a, tile);
  if (t.n == 0) return;
  const int slot0 = t.slot0 + (tile - t.tile0) * kFewRows, rows = min(t.slot0 + t.n - slot0, kFewRows);
  const int K = a.K, steps = (K + 127) / 128;
  const uint32_t bytes = (uint32_t)steps * 1024u;
  const size_t at = ((size_t)t.expert * nblocks + nb) * bytes;
  __amdgpu_buffer_rsrc_t wr[NM];
  wr[0] = make_uniform_rsrc(a.w + at, bytes);
  if (GATED) wr[NM - 1] = make_uniform_rsrc(a.up + at, bytes);
  uint4 wv[S][NM];
  v4i xv[S][4];
  auto wload = [&](int i, int s) {
#pragma unroll
    for (int m = 0; m < NM; ++m) wv[i][m] = bload16_nt(wr[m], (uint32_t)s * 1024u + 16u * (uint32_t)lane);
  };
#pragma unroll
  for (int i = 0; i < S; ++i) wload(i, wave + i * W);     // these need the expert alone
  const bool gather = a.pair != nullptr;
  const int mine = r < rows ? input_row(a, slot0 + r) : -1;
  const auto xr = gather ? make_uniform_rsrc(a.xq, (uint32_t)((int64_t)a.rows * K))
                         : make_uniform_rsrc(a.xq + (size_t)slot0 * K, (uint32_t)(rows * K));
  const uint32_t xo = (uint32_t)(gather ? max(mine, 0) : min(r, rows - 1)) * (uint32_t)K + 64u * (uint32_t)h;
  auto xload = [&](int i, int s) {
    const uint32_t o = 128 * s + 64 * h < K ? xo + 128u * (uint32_t)s : kOob;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      xv[i][j] = __builtin_amdgcn_raw_buffer_load_b128(xr, (int)(o + 16u * (uint32_t)j), 0, 0);
  };
#pragma unroll
  for (int i = 0; i < S; ++i) xload(i, wave + i * W);
  for (int i = tid; i < NM * kFewRows * 33; i += 64 * W) (&sum[0][0][0])[i] = 0;
  if (wave == 0 && h == 0) {
    row_of[r] = mine;
    d_of[r] = mine < 0 ? 0.0f : a.xs[mine];
  }
  v16i acc[NM];
#pragma unroll
  for (int m = 0; m < NM; ++m) acc[m] = (v16i){};
  for (int s = wave; s < steps; s += S * W) {
#pragma unroll
    for (int i = 0; i < S; ++i) {
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        const uint32_t wd[4] = {wv[i][m].x, wv[i][m].y, wv[i][m].z, wv[i][m].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[m] = __builtin_amdgcn_mfma_i32_32x32x32_i8(xv[i][j], weights_64(wd[j]), acc[m], 0, 0, 0);
      }
      wload(i, s + (i + S) * W);
      xload(i, s + (i + S) * W);
    }
  }
  __syncthreads();
  // lane l holds output row l % 32 and slots 8 (v / 4) + 4 (l / 32) + v % 4
#pragma unroll
  for (int m = 0; m < NM; ++m)
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int sl = 8 * (v >> 2) + 4 * h + (v & 3);
      if (sl < rows) atomicAdd(&sum[m][sl][r], acc[m][v]);
    }
  __syncthreads();
  const int c = tid & 31, n = 32 * nb + c;
  if (n >= a.N) return;
  const size_t en = (size_t)t.expert * a.N + n;
  const float g0 = a.w_scale[t.expert], b0 = a.bias ? a.bias[en] : 0.0f;
  const float g1 = GATED ? a.up_scale[t.expert] : 0.0f, b1 = GATED && a.up_bias ? a.up_bias[en] : 0.0f;
  for (int sl = tid >> 5; sl < rows; sl += 2 * W) {
    if (row_of[sl] < 0) continue;
    const float d = d_of[sl];
    float v = acc_64(sum[0][sl][c]) * (g0 * d);
    if (a.bias) v = v + b0;
    v = activate(v, a.act);
    if (GATED) {
      float u = acc_64(sum[NM - 1][sl][c]) * (g1 * d);
      if (a.up_bias) u = u + b1;
      v = v * u;
    }
    store_output(a, (size_t)(slot0 + sl) * a.N + n, v);
  }
}

int64_t few_grid(const ExpertArgs& a) { return many_tiles(a, kFewRows) * ((a.N + 31) / 32); }

template <int S>
hipError_t launch_few(const ExpertArgs& a, hipStream_t s) {
  const int nblocks = (a.N + 31) / 32;
  const dim3 grid((unsigned)few_grid(a)), block(64 * kFewWaves);
  if (a.up)
    hipLaunchKernelGGL((experts_few_kernel<S, true>), grid, block, 0, s, a, nblocks);
  else
    hipLaunchKernelGGL((experts_few_kernel<S, false>), grid, block, 0, s, a, nblocks);
  return hipGetLastError();
}

}  // namespace

// Of the kernels that take large calls the one with 32 x 8 blocks has most threads (rounded up to the
// XCDs).
bool experts_fit(const ExpertArgs& a) {
  const int64_t blocks = ((int64_t)a.N + 31) / 32, weights = a.up ? 2 * blocks : blocks;
  return many_tiles(a, 32) * ((weights + 7) / 8) + 8 <= max_grid(256);
}

hipError_t launch_experts(const ExpertArgs& a, hipStream_t s) {
  // The kernel is chosen for slots spread evenly over the experts; how they are spread is known
  // on the device alone.  An expert's last tile is half full on average.
  const int64_t used = a.experts < a.slots ? a.experts : a.slots;
  const double each = (double)a.slots / (double)used;
  auto tiles = [&](int rows) {
    if (!a.offset) return (double)((a.slots + rows - 1) / rows);
    const double t = each / rows + 0.5;
    return (double)used * (t < 1.0 ? 1.0 : t);
  };
  const int blocks = (a.N + 31) / 32, weights = a.up ? 2 * blocks : blocks, steps = (a.K + 127) / 128;
  auto groups = [&](int rows, int wide) { return tiles(rows) * ((weights + wide - 1) / wide); };
  // Few rows: one block of weights a workgroup, while that gives at most a workgroup a compute
  // unit (two with up to 8 rows, and one only with few or short rows, whose loads are its cost):
  // 2560 -> 2560 at 96 rows, 240 workgroups, 6.1 us against 7.9 of the next choice; at 128, 320 of them,
  // 8.7 against 8.0.
  const double few = tiles(kFewRows) * blocks;
  if ((few <= 256 && (each <= 16 || steps <= 64)) || (few <= 512 && each <= 8))
    return steps > 32 ? launch_few<2>(a, s) : launch_few<1>(a, s);
  // 32 slots, and the k steps shared by eight or four groups of waves while the workgroups do
  // not fill the compute units otherwise
  if (groups(32, 2) <= 256) return launch_experts_many(a, kMany32x2, s);
  if (groups(32, 4) <= 256) return launch_experts_many(a, kMany32x4, s);
  // 32 x 8, 64 x 8, 96 x 8 or 64 x 16 blocks: the least time, with what a step and what lies beside
  // the steps of a workgroup takes alone on its compute unit, and among `held` of them (us, fitted to
  // measured calls: over 116 of them the choice is 0.8% above the least in the geometric mean, 24% at worst,
  // 512 tokens through gate and up of two of eight 2560 -> 6912 experts, 41.4 us for 33.5).  A last round's workgroups count as those that run alone while rounds are few.
  struct Shape {
    ManyTile tile;
    int rows, wide, held;
    double alone, among, beside;
  };
  const Shape shapes[] = {{kMany32x8, 32, 8, 4, 0.30, 0.23, 0.9},
                          {kMany64x8, 64, 8, 4, 0.58, 0.35, 2.0},
                          {kMany96x8, 96, 8, 3, 0.85, 0.50, 3.0},
                          {kMany64x16, 64, 16, 2, 0.68, 0.57, 6.3}};
  ManyTile best = kMany32x8;
  double least = 0;
  for (const Shape& p : shapes) {
    const double r = groups(p.rows, p.wide) / 256, each_round = p.among * steps + p.beside;
    auto some = [&](double n) {
      return n <= 0 ? 0 : n <= 1 ? p.alone * steps + p.beside : each_round * ceil(n);
    };
    const double time = r <= p.held ? some(r)
                        : r <= 2 * p.held ? each_round * p.held + some(r - p.held)
                                          : each_round * (r + 0.4);
    if (least == 0 || time < least) {
      least = time;
      best = p.tile;
    }
  }
  return launch_experts_many(a, best, s);
}

}  // namespace bitnet
