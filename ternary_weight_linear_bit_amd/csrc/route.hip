// Routing of tokens to experts: each token's largest logits, and the pairs (token, choice)
// sorted by expert; and the combination of the experts' outputs.
#include "experts_internal.h"

namespace bitnet {
namespace {

// ---------------------------------------------------------------------------
// choice: 16, 32 or 64 lanes a token
// ---------------------------------------------------------------------------
//
// A logit and its expert's number are held as one double in [1, 2), the logit's order-preserving key
// in the upper and 1023 - e in the lower of 42 mantissa bits, so that a maximum takes one
// instruction and equal logits go to the lowest number; 0 stands for one that is never chosen.  A
// lane sorts its V candidates (a comparison is a min and a max), then the token's topk largest are
// taken from the heads of its lanes' lists.  Bound by vector instructions: 16384 tokens over 256
// experts, 16.8 MB, 12 us, of which they take 61% with four waves a SIMD, the rest waits for loads and the exchange of
// ranks (a wave a token with shuffled maxima took about 50).

// 0 for -inf and NaN; -0 counts as 0.
__device__ __forceinline__ double candidate(float x, int e) {
  if (!(x > -INFINITY)) return 0.0;
  uint32_t b = __float_as_uint(x + 0.0f);
  b ^= (uint32_t)((int)b >> 31) | 0x80000000u;
  const uint64_t u = (0x3ffull << 52) | ((uint64_t)b << 10) | (uint64_t)(1023 - e);
  return __longlong_as_double((long long)u);
}
__device__ __forceinline__ int candidate_expert(double c) {
  return c == 0.0 ? -1 : 1023 - (int)((uint64_t)__double_as_longlong(c) & 1023u);
}
__device__ __forceinline__ float candidate_logit(double c) {
  const uint32_t b = (uint32_t)((uint64_t)__double_as_longlong(c) >> 10);
  return __uint_as_float(b ^ ((b & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}

// Maximum (doubles) and sum (floats) over L lanes.
#define BITNET_ROW(v, ctrl) __builtin_amdgcn_update_dpp(0, (v), (ctrl), 0xf, 0xf, true)
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = (uint32_t)BITNET_ROW((int)(uint32_t)u, CTRL);
  const uint32_t hi = (uint32_t)BITNET_ROW((int)(uint32_t)(u >> 32), CTRL);
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(BITNET_ROW(__float_as_int(v), CTRL));
}
#undef BITNET_ROW
struct Larger {
  __device__ double operator()(double a, double b) const { return __builtin_fmax(a, b); }
  __device__ float operator()(float a, float b) const { return a + b; }    // floats are summed
};
template <int L, typename T>
__device__ __forceinline__ T over_lanes(T v) {
  const Larger f;
  v = f(v, dpp<0xb1>(v));      // lane ^ 1
  v = f(v, dpp<0x4e>(v));      // lane ^ 2
  v = f(v, dpp<0x141>(v));     // half-row mirror
  v = f(v, dpp<0x140>(v));     // row mirror
  if (L >= 32) v = f(v, __shfl_xor(v, 16, 64));
  if (L == 64) v = f(v, __shfl_xor(v, 32, 64));
  return v;
}

// Batcher's merge exchange of V values, largest first.
template <int V>
__device__ __forceinline__ void sort_down(double (&c)[V]) {
#pragma unroll
  for (int p = 1; p < V; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < V; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < V && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const double a = c[i + j], b = c[i + j + k];
            c[i + j] = __builtin_fmax(a, b);
            c[i + j + k] = __builtin_fmin(a, b);
          }
}

struct RouteArgs {
  Routing r;
  const void* logits;
  int64_t stride;
  int score;
  float scale;
};

// e^(x - m) for x <= m; 1 where they are the same (infinities too)
__device__ __forceinline__ float power(float x, float m) {
  return x == m ? 1.0f : exp_neg(fmaxf(x - m, -200.0f));
}

// Token m's choices by L lanes; lane l of them holds experts V l .. V l + V - 1.  Lane j < topk
// (<= L) of the token writes choice j and returns its expert.
template <int L, int V, bool BF16>
__device__ __forceinline__ int choose(const RouteArgs& a, int m) {
  const Routing& r = a.r;
  const int l = threadIdx.x & (L - 1);
  const int64_t at = (int64_t)m * a.stride + l * V;
  const int n = r.experts - l * V;
  float x[V];
  constexpr int W = 16 / (BF16 ? 2 : 4);       // elements of 16 bytes
  if (V >= W && n >= V && ((reinterpret_cast<uintptr_t>(a.logits) + (size_t)at * (16 / W)) & 15) == 0) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(a.logits) + at * (16 / W));
#pragma unroll
    for (int i = 0; i < V / W; ++i) {
      const uint4 u = q[i];
      const uint32_t d[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (BF16) {
          x[(W * i + 2 * e) % V] = __uint_as_float(d[e] << 16);
          x[(W * i + 2 * e + 1) % V] = __uint_as_float(d[e] & 0xffff0000u);
        } else {
          x[(W * i + e) % V] = __uint_as_float(d[e]);
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      x[i] = i >= n ? -INFINITY
             : BF16 ? bf16_bits_to_float(static_cast<const uint16_t*>(a.logits)[at + i])
                    : static_cast<const float*>(a.logits)[at + i];
  }
  double c[V];
#pragma unroll
  for (int i = 0; i < V; ++i) c[i] = candidate(x[i], l * V + i);
  sort_down(c);
  double mine = 0.0, first = 0.0;
  for (int j = 0; j < r.topk; ++j) {
    const double most = over_lanes<L>(c[0]);
    if (j == 0) first = most;
    if (l == j) mine = most;
    if (c[0] == most) {         // its next one; of more than 8 no more than the first 8 are taken
#pragma unroll
      for (int i = 0; i < V - 1; ++i)
        if (i < 8 || r.topk > 8) c[i] = c[i + 1];
      if (V <= 8 || r.topk > 8) c[V - 1] = 0.0;
    }
  }
  const int e = candidate_expert(mine);
  const float z = candidate_logit(mine), top = candidate_logit(first);
  float w = 0.0f, total = 1.0f;
  if (a.score == kSigmoid) {
    // 1 / (1 + e^-z), by e^-|z|
    const float p = exp_neg(fmaxf(-fabsf(z), -200.0f));
    w = (z < 0.0f ? p : 1.0f) / (1.0f + p);
  } else {
    w = power(z, top);
    float part = e < 0 ? 0.0f : w;
    if (a.score == kSoftmax) {
      part = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (x[i] > -INFINITY) part += power(x[i], top);
    }
    total = over_lanes<L>(part);
  }
  if (l < r.topk) {
    r.expert[(int64_t)m * r.topk + l] = e;
    r.weight[(int64_t)m * r.topk + l] = e < 0 ? 0.0f : w / total * a.scale;
  }
  return e;
}

// ---------------------------------------------------------------------------
// plan: a stable counting sort of the pairs by expert
// ---------------------------------------------------------------------------
//
// A workgroup takes some tokens, in rounds of at most 1024 pairs: it chooses their experts, ranks each
// pair among the workgroup's pairs of its expert and leaves the counts.  One workgroup's counts are the plan;
// of several, a second launch adds those of earlier workgroups (7 us for 256 of them over 256
// experts; a workgroup reads 128 KiB of counts).  64 tokens over 64 experts: one launch, 6.0 us.

constexpr int kPairs = 1024;     // threads, and most pairs of a round
constexpr int kWaves = kPairs / 64;

// Tokens of a workgroup: 64 (what its lanes choose for at once, up to 256 experts), and more, in
// rounds of up to 1024 pairs, where there would be more than 512 workgroups: each of them reads the
// counts of all in the second launch.
constexpr int tokens_of(int64_t tokens, int topk) {
  const int64_t round = kPairs / topk, each = (tokens + 511) / 512, least = round < 64 ? round : 64;
  if (each <= round) return (int)(each > least ? each : least);
  return (int)((each + round - 1) / round * round);
}
// A workgroup's pairs, 33759 at most, are counted in 16 bits (they grow with the tokens).
constexpr int most_pairs_of_a_workgroup() {
  int most = 0;
  for (int topk = 1; topk <= kMaxTopk; ++topk) {
    const int pairs = tokens_of(kMaxRouted / topk, topk) * topk;
    most = pairs > most ? pairs : most;
  }
  return most;
}
static_assert(most_pairs_of_a_workgroup() <= 65535, "counts of 16 bits");

// Lanes of the wave with the same expert as this one; none for -1.
__device__ __forceinline__ uint64_t same_expert(int e, int experts) {
  uint64_t m = __ballot(e >= 0);
  if (e < 0) m = 0;
  for (int b = 0; (1 << b) < experts; ++b) {
    const uint64_t on = __ballot((e >> b) & 1);
    m &= ((e >> b) & 1) ? on : ~on;
  }
  return m;
}

// First slot of each expert from its pairs all(x) and those in earlier workgroups before(x): first[x] =
// before(x) + the pairs of smaller experts.  Returns the number of all pairs.  sums: [kWaves].
template <typename All, typename Before>
__device__ __forceinline__ int first_slots(const Routing& r, All all, Before before, int* first, int* sums,
                                           bool writes) {
  const int tid = threadIdx.x;
  int base = 0;
  for (int x0 = 0; x0 < r.experts; x0 += kPairs) {
    const int x = x0 + tid, n = x < r.experts ? all(x) : 0;
    const int upto = wave_scan(n);
    if ((tid & 63) == 63) sums[tid >> 6] = upto;
    __syncthreads();
    int add = base;
    for (int w = 0; w < kWaves; ++w) {
      if (w < (tid >> 6)) add += sums[w];
      base += sums[w];
    }
    if (x < r.experts) {
      first[x] = add + upto - n + before(x);
      if (writes) {
        if (x == 0) r.offset[0] = 0;
        r.offset[x + 1] = add + upto;
      }
    }
    __syncthreads();
  }
  return base;
}

__device__ __forceinline__ void place(const Routing& r, int p, int e, int rank, const int* first, int used) {
  int slot = -1;
  if (e >= 0) {
    slot = first[e] + rank;
    r.pair[slot] = p;
  }
  r.slot[p] = slot;
  if (p >= used) r.pair[p] = -1;         // places behind the last slot
}

// L = 0: the experts are given.  ONE: one workgroup has all pairs; otherwise slot[] holds each
// pair's rank in its workgroup, and hist [workgroups][experts rounded up to 8] its counts.
template <int L, int V, bool BF16, bool ONE>
__global__ __launch_bounds__(kPairs) void route_kernel(const RouteArgs a, int tokens, uint16_t* hist) {
  extern __shared__ int lds[];
  const Routing& r = a.r;
  const int E = r.experts, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int* count = lds;                      // [kWaves][E]: the expert's pairs in the wave, then in earlier ones
  int* total = count + kWaves * E;       // [E]
  int* first = total + E;                // [E]
  int* sums = first + E;                 // [kWaves]
  int* chosen = sums + kWaves;           // [kPairs]
  const int m1 = (int)min(((int64_t)blockIdx.x + 1) * tokens, (int64_t)r.tokens), round = kPairs / r.topk;
  int m0 = (int)blockIdx.x * tokens;
  for (int x = tid; x < E; x += kPairs) total[x] = 0;
  do {
    const int here = min(m1 - m0, round), pairs = here * r.topk, p = m0 * r.topk + tid;
    for (int i = tid; i < kWaves * E; i += kPairs) count[i] = 0;
    int e = -1;
    if constexpr (L == 0) {
      if (tid < pairs) e = r.expert[p];
      if (e >= E) e = -1;
    } else {
      for (int m = tid / L; m < here; m += kPairs / L) {
        const int c = choose<L, V, BF16>(a, m0 + m);
        if ((tid & (L - 1)) < r.topk) chosen[m * r.topk + (tid & (L - 1))] = c;
      }
    }
    __syncthreads();
    if (L != 0 && tid < pairs) e = chosen[tid];
    const uint64_t same = same_expert(e, E);
    int rank = __popcll(same & ((1ull << lane) - 1));
    if (e >= 0 && rank == 0) count[wave * E + e] = __popcll(same);
    __syncthreads();
    for (int x = tid; x < E; x += kPairs) {
      int n = total[x];                  // those of the tokens before
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const int c = count[w * E + x];
        count[w * E + x] = n;
        n += c;
      }
      total[x] = n;
    }
    __syncthreads();
    if (e >= 0) rank += count[wave * E + e];
    if constexpr (ONE) {
      const int used = first_slots(r, [&](int x) { return total[x]; }, [](int) { return 0; }, first, sums, true);
      if (tid < pairs) place(r, p, e, rank, first, used);
      return;
    }
    if (tid < pairs) r.slot[p] = rank;
    m0 += round;
    __syncthreads();
  } while (m0 < m1);
  for (int x = tid; x < E; x += kPairs) hist[(size_t)blockIdx.x * ((E + 7) & ~7) + x] = (uint16_t)total[x];
}

__global__ __launch_bounds__(kPairs) void route_place_kernel(const Routing r, int tokens,
                                                            const uint16_t* hist, int blocks) {
  extern __shared__ int lds[];
  const int E = r.experts, E8 = (E + 7) & ~7, tid = threadIdx.x, b = (int)blockIdx.x;
  int *all = lds, *before = all + E8, *first = before + E8, *sums = first + E;
  for (int i = tid; i < 2 * E8; i += kPairs) lds[i] = 0;
  const int p1 = (int)min(((int64_t)b + 1) * tokens, (int64_t)r.tokens) * r.topk;
  int p = b * tokens * r.topk + tid, e = -1, rank = 0;
  auto load = [&]() {
    if (p < p1) {
      e = r.expert[p];
      if (e >= E) e = -1;
      rank = r.slot[p];
    }
  };
  load();
  __syncthreads();
  // a thread adds 8 experts' counts of every (groups)th workgroup, 8 loads in flight
  const int per = E8 / 8, groups = min(kPairs / per, 64), g = tid / per, x8 = tid - g * per;
  if (g < groups) {
    int na[8] = {}, nb[8] = {};
    for (int q0 = g; q0 < blocks; q0 += 8 * groups) {
      uint4 u[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int q = q0 + j * groups;
        u[j] = make_uint4(0u, 0u, 0u, 0u);
        if (q < blocks) u[j] = *reinterpret_cast<const uint4*>(hist + (size_t)q * E8 + 8 * x8);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t d[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = (int)((d[i >> 1] >> (16 * (i & 1))) & 0xffffu);
          na[i] += c;
          nb[i] += q0 + j * groups < b ? c : 0;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (8 * x8 + i < E) {      // (counts behind the last expert were not written)
        atomicAdd(&all[i * per + x8], na[i]);       // neighbouring lanes in neighbouring banks
        atomicAdd(&before[i * per + x8], nb[i]);
      }
  }
  __syncthreads();
  const int used = first_slots(r, [&](int x) { return all[(x & 7) * per + (x >> 3)]; },
                               [&](int x) { return before[(x & 7) * per + (x >> 3)]; }, first, sums, b == 0);
  while (p < p1) {
    place(r, p, e, rank, first, used);
    p += kPairs;
    load();
  }
}

// ---------------------------------------------------------------------------
// combination
// ---------------------------------------------------------------------------

// A workgroup takes a token's columns, W = 8 of them (or 1, unaligned) a thread, and the rows of four
// choices at once, so that their loads overlap; which rows they are is the same for all threads.
// Bound by memory: 4093 tokens of six bf16 rows of 2560, fp32 out, 197 MB in 42 us (4.7 TB/s).
template <bool BF16, int W>
__device__ __forceinline__ void load_cols(const void* p, int64_t at, float (&v)[W]) {
  if constexpr (W == 1) {
    v[0] = BF16 ? bf16_bits_to_float(static_cast<const uint16_t*>(p)[at]) : static_cast<const float*>(p)[at];
  } else if constexpr (BF16) {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
    const uint32_t d[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(d[i] << 16);
      v[2 * i + 1] = __uint_as_float(d[i] & 0xffff0000u);
    }
  } else {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 u = q[i];
      v[4 * i] = u.x;
      v[4 * i + 1] = u.y;
      v[4 * i + 2] = u.z;
      v[4 * i + 3] = u.w;
    }
  }
}

template <bool YB, bool OB, int W>
__global__ __launch_bounds__(256) void combine_kernel(const Routing r, const void* y, int64_t K,
                                                      const void* residual, void* out) {
  const int64_t k = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * W;
  if (k >= K) return;
  for (int64_t m = blockIdx.x; m < r.tokens; m += gridDim.x) {
    float v[W] = {};
    if (residual) load_cols<OB, W>(residual, m * K + k, v);
    const int32_t* slot = r.slot + m * r.topk;
    const float* weight = r.weight + m * r.topk;
    for (int j0 = 0; j0 < r.topk; j0 += 4) {
      float x[4][W], w[4];
      bool on[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        on[j] = false;
        if (j0 + j < r.topk) {
          const int s = slot[j0 + j];
          on[j] = s >= 0 && s < r.pairs;
          w[j] = weight[j0 + j];
          if (on[j]) load_cols<YB, W>(y, (int64_t)s * K + k, x[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (on[j]) {
#pragma unroll
          for (int i = 0; i < W; ++i) v[i] = v[i] + w[j] * x[j][i];
        }
    }
    if constexpr (W == 1) {
      if (OB)
        static_cast<uint16_t*>(out)[m * K + k] = float_to_bf16_rne(v[0]);
      else
        static_cast<float*>(out)[m * K + k] = v[0];
    } else if constexpr (OB) {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + m * K + k) =
          make_uint4(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]), bf16x2_rne(v[4], v[5]), bf16x2_rne(v[6], v[7]));
    } else {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + m * K + k);
      o[0] = make_float4(v[0], v[1], v[2], v[3]);
      o[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
}

int route_blocks(int64_t tokens, int topk) {
  const int t = tokens_of(tokens, topk);
  return (int)((tokens + t - 1) / t);
}

template <int L, int V, bool BF16>
void launch_first(const RouteArgs& a, int blocks, uint16_t* hist, hipStream_t s) {
  const size_t lds = ((kWaves + 2) * a.r.experts + kWaves + kPairs) * sizeof(int);
  const int tokens = tokens_of(a.r.tokens, a.r.topk);
  if (blocks <= 1)
    hipLaunchKernelGGL((route_kernel<L, V, BF16, true>), dim3(1), dim3(kPairs), lds, s, a, tokens, hist);
  else
    hipLaunchKernelGGL((route_kernel<L, V, BF16, false>), dim3(blocks), dim3(kPairs), lds, s, a, tokens, hist);
}

template <bool BF16>
void launch_choice(const RouteArgs& a, int blocks, uint16_t* hist, hipStream_t s) {
  const int E = a.r.experts;
  if (a.r.topk <= 16 && E <= 64)
    launch_first<16, 4, BF16>(a, blocks, hist, s);
  else if (a.r.topk <= 16 && E <= 256)
    launch_first<16, 16, BF16>(a, blocks, hist, s);
  else if (E <= 512)
    launch_first<32, 16, BF16>(a, blocks, hist, s);
  else
    launch_first<64, 16, BF16>(a, blocks, hist, s);
}

}  // namespace

size_t route_workspace_bytes(int64_t tokens, int topk, int experts) {
  const int blocks = route_blocks(tokens, topk);
  return blocks <= 1 ? 0 : (size_t)blocks * ((experts + 7) & ~7) * sizeof(uint16_t);
}

hipError_t launch_route(const Routing& r, const void* logits, bool bf16, int64_t stride, int score,
                        float scale, void* workspace, hipStream_t s) {
  const int blocks = route_blocks(r.tokens, r.topk);     // (0 without tokens: the offsets are written)
  uint16_t* hist = static_cast<uint16_t*>(workspace);
  const RouteArgs a{r, logits, stride, score, scale};
  if (!logits)
    launch_first<0, 1, false>(a, blocks, hist, s);
  else if (bf16)
    launch_choice<true>(a, blocks, hist, s);
  else
    launch_choice<false>(a, blocks, hist, s);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || blocks <= 1) return e;
  const int E8 = (r.experts + 7) & ~7;
  hipLaunchKernelGGL(route_place_kernel, dim3(blocks), dim3(kPairs), (2 * E8 + r.experts + kWaves) * sizeof(int), s,
                     r, tokens_of(r.tokens, r.topk), hist, blocks);
  return hipGetLastError();
}

namespace {
template <int W>
hipError_t launch_combine_w(const Routing& r, const void* y, bool y_bf16, int64_t K, const void* residual,
                            void* out, bool out_bf16, hipStream_t s) {
  const int64_t cols = (K + W - 1) / W;
  const int threads = cols >= 256 ? 256 : (int)((cols + 63) / 64) * 64;
  const int64_t parts = (cols + threads - 1) / threads;
  // Columns lie in the grid's second dimension, at most 2^15 parts of them.  What the runtime counts leaves at least
  // 511 workgroups in the first; where tokens are more, one takes several of them.
  static_assert(kCombineCols / 256 <= 65535, "the grid's second dimension");
  const int64_t across = max_grid(256) / parts;
  const dim3 grid((unsigned)(r.tokens < across ? r.tokens : across), (unsigned)parts), block(threads);
#define BITNET_COMBINE(YB, OB) \
  hipLaunchKernelGGL((combine_kernel<YB, OB, W>), grid, block, 0, s, r, y, K, residual, out)
  if (y_bf16 && out_bf16)
    BITNET_COMBINE(true, true);
  else if (y_bf16)
    BITNET_COMBINE(true, false);
  else if (out_bf16)
    BITNET_COMBINE(false, true);
  else
    BITNET_COMBINE(false, false);
#undef BITNET_COMBINE
  return hipGetLastError();
}
}  // namespace

hipError_t launch_combine(const Routing& r, const void* y, bool y_bf16, int64_t K,
                          const void* residual, void* out, bool out_bf16, hipStream_t s) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(y) | reinterpret_cast<uintptr_t>(residual) |
                       reinterpret_cast<uintptr_t>(out);
  return K % 8 == 0 && (at & 15) == 0 ? launch_combine_w<8>(r, y, y_bf16, K, residual, out, out_bf16, s)
                                      : launch_combine_w<1>(r, y, y_bf16, K, residual, out, out_bf16, s);
}

}  // namespace bitnet
