// Routing of tokens to experts: each token's largest logits, and the pairs (token, choice)
// sorted by expert; and the combination of the experts' outputs.
#include "experts_internal.h"

namespace bitnet {
namespace {

// ---------------------------------------------------------------------------
// choice: a wave a token
// ---------------------------------------------------------------------------

// Order-preserving key of a logit: 0 for -inf and NaN, which are never chosen; -0 counts as 0.
__device__ __forceinline__ uint32_t logit_key(float x) {
  if (!(x > -INFINITY)) return 0u;
  const uint32_t b = __float_as_uint(x == 0.0f ? 0.0f : x);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
  return v;
}
__device__ __forceinline__ float wave_fsum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}
// x - m, 0 where they are the same (infinities too)
__device__ __forceinline__ float below(float x, float m) { return x == m ? 0.0f : x - m; }

struct RouteArgs {
  Routing r;
  const void* logits;
  int64_t stride;
  int score;
  float scale;
};

// Token m's choices, by one wave; lane l holds experts V l .. V l + V - 1, so that the first lane
// with the largest key has the lowest index.  Lane j < topk returns choice j.
template <int V, bool BF16>
__device__ __forceinline__ int choose(const RouteArgs& a, int m) {
  const int lane = threadIdx.x & 63;
  const Routing& r = a.r;
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane * V + i;
    key[i] = 0u;
    if (e < r.experts) {
      const int64_t at = (int64_t)m * a.stride + e;
      key[i] = logit_key(BF16 ? bf16_bits_to_float(static_cast<const uint16_t*>(a.logits)[at])
                              : static_cast<const float*>(a.logits)[at]);
    }
  }
  uint32_t all[V];
#pragma unroll
  for (int i = 0; i < V; ++i) all[i] = key[i];
  int mine = -1;
  uint32_t mine_key = 0u, top = 0u;
  for (int j = 0; j < r.topk; ++j) {
    uint32_t best = key[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < V; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
      }
    const uint32_t most = wave_umax(best);
    if (j == 0) top = most;
    if (most == 0u) break;
    const int l = __ffsll((unsigned long long)__ballot(best == most)) - 1;
    const int i = __builtin_amdgcn_readlane(at, l);
    if (lane == j) {
      mine = l * V + i;
      mine_key = most;
    }
    if (lane == l) {
#pragma unroll
      for (int q = 0; q < V; ++q)
        if (q == i) key[q] = 0u;
    }
  }
  float w = 0.0f;
  if (top != 0u) {
    if (a.score == kSigmoid) {
      const float z = key_logit(mine_key);
      w = mine < 0 ? 0.0f : 1.0f / (1.0f + expf(-z));
    } else {
      const float big = key_logit(top);
      const float own = mine < 0 ? 0.0f : expf(below(key_logit(mine_key), big));
      float total = own;
      if (a.score == kSoftmax) {
        total = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (all[i]) total += expf(below(key_logit(all[i]), big));
      }
      w = own / wave_fsum(total);
    }
  }
  if (lane < r.topk) {
    r.expert[(int64_t)m * r.topk + lane] = mine;
    r.weight[(int64_t)m * r.topk + lane] = w * a.scale;
  }
  return mine;
}

// ---------------------------------------------------------------------------
// plan: a stable counting sort of the pairs by expert
// ---------------------------------------------------------------------------

constexpr int kPairs = 512;      // pairs of a workgroup
constexpr int kWaves = kPairs / 64;

// Lanes of the wave with the same expert (-1: none) as this one.
__device__ __forceinline__ uint64_t same_expert(int e, int bits) {
  uint64_t m = __ballot(e >= 0);
  if (e < 0) m = 0;
  for (int b = 0; b < bits; ++b) {
    const uint64_t on = __ballot((e >> b) & 1);
    m &= ((e >> b) & 1) ? on : ~on;
  }
  return m;
}

// Counts the workgroup's pairs (one a thread, in order) by expert: count[wave][e] becomes the number
// of the expert's pairs in earlier waves, total[e] of all; returns the pair's rank in its wave.
__device__ __forceinline__ int count_pairs(int e, int experts, int* count, int* total) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int i = tid; i < kWaves * experts; i += kPairs) count[i] = 0;
  __syncthreads();
  int bits = 0;
  while ((1 << bits) < experts) ++bits;
  const uint64_t m = same_expert(e, bits);
  const int rank = __popcll(m & ((1ull << lane) - 1));
  if (e >= 0 && rank == 0) count[wave * experts + e] = __popcll(m);
  __syncthreads();
  for (int x = tid; x < experts; x += kPairs) {
    int n = 0;
    for (int w = 0; w < kWaves; ++w) {
      const int c = count[w * experts + x];
      count[w * experts + x] = n;
      n += c;
    }
    total[x] = n;
  }
  __syncthreads();
  return rank;
}

__device__ __forceinline__ int pair_expert(const Routing& r, int p) {
  if (p >= r.pairs) return -1;
  const int e = r.expert[p];
  return e >= 0 && e < r.experts ? e : -1;
}

template <int V, bool BF16>
__global__ __launch_bounds__(256) void route_choose_kernel(const RouteArgs a) {
  const int m = (int)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (m < a.r.tokens) choose<V, BF16>(a, m);
}

__global__ __launch_bounds__(kPairs) void route_count_kernel(const Routing r, int* hist) {
  extern __shared__ int lds[];
  int* total = lds + kWaves * r.experts;
  count_pairs(pair_expert(r, (int)blockIdx.x * kPairs + threadIdx.x), r.experts, lds, total);
  for (int x = threadIdx.x; x < r.experts; x += kPairs)
    hist[(int64_t)blockIdx.x * r.experts + x] = total[x];
}

__global__ __launch_bounds__(kPairs) void route_place_kernel(const Routing r, const int* hist,
                                                            int blocks) {
  extern __shared__ int lds[];
  int* total = lds + kWaves * r.experts;
  int* first = total + r.experts;          // first slot of the expert's pairs of this workgroup
  int* sums = first + r.experts;           // [kWaves]
  const int tid = threadIdx.x, E = r.experts, b = (int)blockIdx.x;
  const int p = b * kPairs + tid;
  const int e = pair_expert(r, p);
  const int rank = count_pairs(e, E, lds, total);
  // pairs of each expert in all workgroups, and in earlier ones; then the experts' first slots
  int base = 0;
  for (int x0 = 0; x0 < E; x0 += kPairs) {
    const int x = x0 + tid;
    int all = 0, before = 0;
    if (x < E)
      for (int q = 0; q < blocks; ++q) {
        const int c = hist[(int64_t)q * E + x];
        all += c;
        if (q < b) before += c;
      }
    const int upto = wave_scan(all);
    if ((tid & 63) == 63) sums[tid >> 6] = upto;
    __syncthreads();
    int add = base;
    for (int w = 0; w < (tid >> 6); ++w) add += sums[w];
    if (x < E) first[x] = add + upto - all + before;
    if (b == 0 && x < E) {
      if (x == 0) r.offset[0] = 0;
      r.offset[x + 1] = add + upto;
    }
    for (int w = 0; w < kWaves; ++w) base += sums[w];
    __syncthreads();
  }
  if (p < r.pairs) {
    int slot = -1;
    if (e >= 0) {
      slot = first[e] + lds[(tid >> 6) * E + e] + rank;
      r.pair[slot] = p;
    }
    r.slot[p] = slot;
    if (p >= base) r.pair[p] = -1;         // slots behind the last pair
  }
}

// ---------------------------------------------------------------------------
// combination
// ---------------------------------------------------------------------------

template <bool YB, bool OB>
__global__ __launch_bounds__(256) void combine_kernel(const Routing r, const void* y, int64_t K,
                                                      const void* residual, void* out) {
  const int64_t total = (int64_t)r.tokens * K;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / K, k = i - m * K;
    float v = 0.0f;
    if (residual)
      v = OB ? bf16_bits_to_float(static_cast<const uint16_t*>(residual)[i])
             : static_cast<const float*>(residual)[i];
    for (int j = 0; j < r.topk; ++j) {
      const int s = r.slot[m * r.topk + j];
      if (s < 0 || s >= r.pairs) continue;
      const int64_t o = (int64_t)s * K + k;
      const float x = YB ? bf16_bits_to_float(static_cast<const uint16_t*>(y)[o])
                         : static_cast<const float*>(y)[o];
      v = v + r.weight[m * r.topk + j] * x;
    }
    if (OB)
      static_cast<uint16_t*>(out)[i] = float_to_bf16_rne(v);
    else
      static_cast<float*>(out)[i] = v;
  }
}

int route_blocks(int64_t pairs) { return (int)((pairs + kPairs - 1) / kPairs); }

}  // namespace

size_t route_workspace_bytes(int64_t tokens, int topk, int experts) {
  return (size_t)route_blocks(tokens * topk) * experts * sizeof(int);
}

hipError_t launch_route(const Routing& r, const void* logits, bool bf16, int64_t stride, int score,
                        float scale, void* workspace, hipStream_t s) {
  if (logits && r.tokens > 0) {
    const RouteArgs a{r, logits, stride, score, scale};
    const dim3 grid((unsigned)((r.tokens + 3) / 4));
#define BITNET_CHOOSE(V)                                                                      \
  if (bf16)                                                                                   \
    hipLaunchKernelGGL((route_choose_kernel<V, true>), grid, dim3(256), 0, s, a);             \
  else                                                                                        \
    hipLaunchKernelGGL((route_choose_kernel<V, false>), grid, dim3(256), 0, s, a)
    if (r.experts <= 64) {
      BITNET_CHOOSE(1);
    } else if (r.experts <= 256) {
      BITNET_CHOOSE(4);
    } else {
      BITNET_CHOOSE(16);
    }
#undef BITNET_CHOOSE
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int blocks = route_blocks(r.pairs);    // (0 without tokens: the offsets are written)
  int* hist = static_cast<int*>(workspace);
  if (blocks > 0) {
    hipLaunchKernelGGL(route_count_kernel, dim3(blocks), dim3(kPairs),
                       (kWaves + 1) * r.experts * sizeof(int), s, r, hist);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(route_place_kernel, dim3(blocks > 0 ? blocks : 1), dim3(kPairs),
                     ((kWaves + 2) * r.experts + kWaves) * sizeof(int), s, r, hist, blocks);
  return hipGetLastError();
}

hipError_t launch_combine(const Routing& r, const void* y, bool y_bf16, int64_t K,
                          const void* residual, void* out, bool out_bf16, hipStream_t s) {
  int64_t blocks = ((int64_t)r.tokens * K + 255) / 256;
  if (blocks > 65536) blocks = 65536;
  const dim3 grid((unsigned)blocks);
  if (y_bf16 && out_bf16)
    hipLaunchKernelGGL((combine_kernel<true, true>), grid, dim3(256), 0, s, r, y, K, residual, out);
  else if (y_bf16)
    hipLaunchKernelGGL((combine_kernel<true, false>), grid, dim3(256), 0, s, r, y, K, residual, out);
  else if (out_bf16)
    hipLaunchKernelGGL((combine_kernel<false, true>), grid, dim3(256), 0, s, r, y, K, residual, out);
  else
    hipLaunchKernelGGL((combine_kernel<false, false>), grid, dim3(256), 0, s, r, y, K, residual, out);
  return hipGetLastError();
}

}  // namespace bitnet
