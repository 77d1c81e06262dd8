// Internal declarations of a feed-forward of ternary experts: routing, products grouped by
// expert, and the combination of their outputs.
#pragma once

#include "layer_internal.h"

namespace bitnet {

constexpr int kMaxExperts = 1024;   // counters of a workgroup's pairs by expert lie in LDS
constexpr int kMaxTopk = 32;        // a lane a choice
constexpr int64_t kMaxRouted = (int64_t)1 << 24;   // pairs that are planned: a workgroup's counts are held in 16 bits

// Which rows belong to which expert (bitnet_routing, validated).
struct Routing {
  int32_t* expert;     // [tokens][topk]
  float* weight;       // [tokens][topk]
  int32_t* offset;     // [experts + 1]
  int32_t* pair;       // [pairs]
  int32_t* slot;       // [pairs]
  int tokens, topk, experts, pairs;
};
enum RouteScore { kSoftmax = 0, kChosen = 1, kSigmoid = 2 };
size_t route_workspace_bytes(int64_t tokens, int topk, int experts);
// logits nullptr: r.expert is given and only the plan is made.
hipError_t launch_route(const Routing& r, const void* logits, bool bf16, int64_t stride, int score,
                        float scale, void* workspace, hipStream_t s);

// A ternary product with what follows it.  Slots are rows of y; with `offset` they belong to
// experts, without it all to matrix 0.
enum Act { kActNone = 0, kActRelu2 = 1, kActSilu = 2, kActGelu = 3 };
struct ExpertArgs {
  const int32_t* offset;     // [experts + 1] first slot of each expert, or nullptr: one matrix
  const int32_t* pair;       // [slots] input row times `topk`, or nullptr: a slot is its input row
  const uint8_t *w, *up;     // [experts] matrices in the prefill layout; up: nullptr for none
  const float *w_scale, *up_scale;     // [experts]
  const float *bias, *up_bias;         // [experts][N] or nullptr
  const int8_t* xq;          // [rows][K]
  const float* xs;           // [rows]
  const void* residual;      // [slots][N] like y, or nullptr
  void* y;                   // [slots][N]
  int slots, rows, experts, topk, N, K, act, y_bf16;
};
// Most tiles of `rows` slots that `slots` slots of `experts` experts make.
inline int64_t expert_tiles(int64_t slots, int64_t experts, int rows) {
  return slots / rows + (slots < experts ? slots : experts);
}
inline int64_t many_tiles(const ExpertArgs& a, int rows) {
  return a.offset ? expert_tiles(a.slots, a.experts, rows) : ((int64_t)a.slots + rows - 1) / rows;
}
bool experts_fit(const ExpertArgs& a);
// Tiles of the kernel for many rows (experts_many.hip): slots x blocks of 32 weight rows; in the first
// two eight and four groups of waves share the k steps.
enum ManyTile { kMany32x2, kMany32x4, kMany32x8, kMany64x8, kMany96x8, kMany64x16 };
hipError_t launch_experts_many(const ExpertArgs& a, ManyTile tile, hipStream_t s);
hipError_t launch_experts(const ExpertArgs& a, hipStream_t s);

// out[m] = residual[m] + sum_j weight[m][j] y[slot[m][j]].
constexpr int64_t kCombineCols = (int64_t)1 << 23;   // most of a row
hipError_t launch_combine(const Routing& r, const void* y, bool y_bf16, int64_t K,
                          const void* residual, void* out, bool out_bf16, hipStream_t s);

// The expert that tile t belongs to, where each expert's slots are cut into tiles of ROWS: its first
// slot, its slots (0: there is no such tile) and its first tile.  The offsets lie in device memory,
// where the host cannot check them: they are clamped to the batch.  A wave reads 64 experts' offsets
// at once.
struct ExpertSpan {
  int expert, slot0, n, tile0;
};
__device__ __forceinline__ int wave_scan(int v) {   // inclusive; within rows of 16 lanes, then across
#define BITNET_SCAN(ctrl, rows) v += __builtin_amdgcn_update_dpp(0, v, ctrl, rows, 0xf, false)
  BITNET_SCAN(0x111, 0xf);
  BITNET_SCAN(0x112, 0xf);
  BITNET_SCAN(0x114, 0xf);
  BITNET_SCAN(0x118, 0xf);
  BITNET_SCAN(0x142, 0xa);
  BITNET_SCAN(0x143, 0xc);
#undef BITNET_SCAN
  return v;
}
template <int ROWS>
__device__ __forceinline__ ExpertSpan expert_span(const ExpertArgs& a, int t) {
  if (!a.offset) return {0, 0, t * (int64_t)ROWS < a.slots ? a.slots : 0, 0};
  const int lane = threadIdx.x & 63;
  for (int e0 = 0, base = 0; e0 < a.experts; e0 += 64) {
    const int e = e0 + lane;
    int lo = 0, n = 0;
    if (e < a.experts) {
      lo = min(max(a.offset[e], 0), a.slots);
      n = min(max(a.offset[e + 1], lo), a.slots) - lo;
    }
    const int tiles = (n + ROWS - 1) / ROWS;
    const int upto = base + wave_scan(tiles);
    const uint64_t past = __ballot(upto > t);
    if (past) {
      const int l = __ffsll((unsigned long long)past) - 1;
      return {e0 + l, __builtin_amdgcn_readlane(lo, l), __builtin_amdgcn_readlane(n, l),
              __builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(tiles, l)};
    }
    base = __builtin_amdgcn_readlane(upto, 63);
  }
  return {0, 0, 0, 0};
}
// Tiles of all experts.  Offsets that make experts' slots overlap give more than a plan has, up to experts times
// slots / ROWS, beyond 31 bits: no more are counted than the grid was made for.  (Each lane's sum is below 2^30,
// the wave's taken without sign.)
template <int ROWS>
__device__ __forceinline__ int count_tiles(const ExpertArgs& a) {
  if (!a.offset) return (a.slots + ROWS - 1) / ROWS;
  const int lane = threadIdx.x & 63, most = a.slots / ROWS + min(a.slots, a.experts);
  int n = 0;
  for (int e = lane; e < a.experts; e += 64) {
    const int lo = min(max(a.offset[e], 0), a.slots);
    n += (min(max(a.offset[e + 1], lo), a.slots) - lo + ROWS - 1) / ROWS;
  }
  return (int)min((uint32_t)wave_sum(min(n, most)), (uint32_t)most);
}
// Input row of a slot; -1 where the device's numbers name none.
__device__ __forceinline__ int input_row(const ExpertArgs& a, int slot) {
  if (!a.pair) return slot < a.rows ? slot : -1;
  const int p = a.pair[slot];
  if (p < 0) return -1;
  const int row = (int)((uint32_t)p / (uint32_t)a.topk);
  return row < a.rows ? row : -1;
}

// 16 weights of the prefill layout (codes q + 1) as the int8 operand -64 q, in natural k order: the
// code XOR 1 is -q in two bits, and a field moved to a byte's two top bits is 64 times that, so
// that a shift and a mask make four weights and no sum of x has to be taken off the products.
// The products' sums are -64 acc: at most 64 * 128 * K <= 2^30.
__device__ __forceinline__ v4i weights_64(uint32_t w) {
  constexpr uint32_t top = 0xc0c0c0c0u, one = 0x40404040u;
  v4i a;
  a.x = (int)__builtin_amdgcn_bitop3_b32(w << 6, top, one, 0x6a);   // (w & top) ^ one
  a.y = (int)__builtin_amdgcn_bitop3_b32(w << 4, top, one, 0x6a);
  a.z = (int)__builtin_amdgcn_bitop3_b32(w << 2, top, one, 0x6a);
  a.w = (int)__builtin_amdgcn_bitop3_b32(w, top, one, 0x6a);
  return a;
}
// acc from that sum (exact: 24 bits times 2^6; a sum of 0 is +0).
__device__ __forceinline__ float acc_64(int sum) { return fmaf((float)sum, -0x1p-6f, 0.0f); }

// e^x for x <= 0, the rounding of x log2 e made up for (it is x 2^-24 otherwise).  x log2 e is finite: an
// infinite one has no rounding to make up for and would leave NaN, so callers bound x.
__device__ __forceinline__ float exp_neg(float x) {
  const float t = x * 0x1.715476p+0f;                       // log2 e, rounded
  const float lo = fmaf(x, 0x1.4ae0cp-26f, fmaf(x, 0x1.715476p+0f, -t));
  const float p = __builtin_amdgcn_exp2f(t);
  return fmaf(p, lo * 0x1.62e43p-1f, p);
}
__device__ __forceinline__ float relu2(float v) {
  const float a = __builtin_elementwise_maximum(v, 0.0f);      // (NaN stays)
  return a * a;
}
// v / (1 + e^-v), by e^-|v|, for |v| <= kSiluNear or NaN
constexpr float kSiluNear = 87.0f;     // e^-87 is a normal number
__device__ __forceinline__ float silu_near(float v) {
  const float e = exp_neg(-fabsf(v));
  return (v < 0.0f ? v * e : v) * __builtin_amdgcn_rcpf(1.0f + e);
}
// Of any v.  The exponential gives 0 for what is below 2^-126, 88 times which is not: past kSiluNear a factor e^-32
// stays apart (1 + e^-|v| is 1 with and without it).  Beyond 200 e^-|v| is 0.
__device__ __forceinline__ float silu(float v) {
  const float a = fminf(fabsf(v), 200.0f);
  const bool far = a > kSiluNear;
  const float e = exp_neg(far ? 32.0f - a : -a);
  return (v < 0.0f ? v * e * (far ? 0x1.c8465p-47f : 1.0f) : v) * __builtin_amdgcn_rcpf(1.0f + e);
}
// v times the normal distribution's integral up to v
__device__ __forceinline__ float gelu(float v) {
  // integral up to -a = e^(-a^2 / 2) t Q(t), t = 1 / (1 + 0.28 a): a fit of the least largest error
  // over a in [0, 6], 9.3e-9, by weighted least squares (Lawson's method)
  const float a = fabsf(v);
  const float t = __builtin_amdgcn_rcpf(fmaf(a, 0.28f, 1.0f));
  float q = -0x1.b163fcp-4f;
  q = fmaf(q, t, 0x1.8f3b24p-2f);
  q = fmaf(q, t, -0x1.e55cd8p-3f);
  q = fmaf(q, t, 0x1.135d3p-2f);
  q = fmaf(q, t, 0x1.147778p-4f);
  q = fmaf(q, t, 0x1.dd44e4p-4f);
  q = q * t * __builtin_amdgcn_exp2f(a * a * -0x1.715476p-1f);
  return v * (v < 0.0f ? q : 1.0f - q);
}
__device__ __forceinline__ float activate(float v, int act) {
  return act == kActRelu2 ? relu2(v) : act == kActSilu ? silu(v) : act == kActGelu ? gelu(v) : v;
}
// The same of M values.  Where no lane of the wave has a value past kSiluNear, SiLU goes without what those take
// (4096 tokens through gate and up of 2560 -> 6912: 257 us, 265 with it); the bits are the same.
template <int M>
__device__ __forceinline__ void activate(float (&v)[M], int act) {
  if (act == kActRelu2) {
#pragma unroll
    for (int i = 0; i < M; ++i) v[i] = relu2(v[i]);
  } else if (act == kActGelu) {
#pragma unroll
    for (int i = 0; i < M; ++i) v[i] = gelu(v[i]);
  } else if (act == kActSilu) {
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < M; ++i) most = fmaxf(most, fabsf(v[i]));
    if (__any(most > kSiluNear)) {
#pragma unroll
      for (int i = 0; i < M; ++i) v[i] = silu(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < M; ++i) v[i] = silu_near(v[i]);
    }
  }
}

// y[o] = RN(a + residual[o])
__device__ __forceinline__ void store_output(const ExpertArgs& a, size_t o, float v) {
  if (a.y_bf16) {
    if (a.residual) v = v + bf16_bits_to_float(static_cast<const uint16_t*>(a.residual)[o]);
    static_cast<uint16_t*>(a.y)[o] = float_to_bf16_rne(v);
  } else {
    if (a.residual) v = v + static_cast<const float*>(a.residual)[o];
    static_cast<float*>(a.y)[o] = v;
  }
}

}  // namespace bitnet
