// A block's output joins the residual stream, and the next block's input leaves
// normalised and quantised, in one pass per token.
//
//   z  = y, or RN32(RN32(y r1) post) with a norm behind the block
//   t  = RN32(z scale), z first multiplied by the gate if there is one
//   h' = RN(RN32(h + t)) in the stream's type, written to h_out
//   u  = h', or RN32(RN32(h' r2) pre) with a norm before the next block
//   codes and scale of u as the activation quantiser forms them.
// r = RN32(1 / sqrt(RN32(ms + eps))) with ms the exactly rounded mean of squares
// (the same functions as the activation prologue's norm), so every result is
// independent of the order of the sums.
//
// Bound by memory: y and h are read once, h' and the codes written once (4093 x 4096,
// bf16 block, fp32 stream, both norms: 41-43 us, 4.3-4.5 TB/s; one token of 2560: 3.7 us
// in a graph, the chain of two sums and a maximum).  One
// workgroup per token; each thread keeps its first H groups of 8 values in
// registers from the first sum to the last store.  Rows beyond that read h' again
// (never h, which h_out may replace).  The K % 8 last values of a row go one to a
// thread.  Groups are loaded and stored whole at any alignment (the hardware takes
// 16-byte accesses at element alignment): rows of odd lengths have no other path.
#include "layer_internal.h"

#include <type_traits>

namespace bitnet {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// W consecutive elements (8 or 1), aligned to the element.
template <bool BF16, int W>
__device__ __forceinline__ void rs_load(const void* x, int64_t i, float v[W]) {
  if constexpr (W == 1) {
    v[0] = BF16 ? bf16_bits_to_float(reinterpret_cast<const uint16_t*>(x)[i])
                : reinterpret_cast<const float*>(x)[i];
  } else if constexpr (BF16) {
    u32x4 d;
    __builtin_memcpy(&d, reinterpret_cast<const uint16_t*>(x) + i, 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(d[j] << 16);
      v[2 * j + 1] = __uint_as_float(d[j] & 0xffff0000u);
    }
  } else {
    u32x4 d[2];
    __builtin_memcpy(&d[0], reinterpret_cast<const float*>(x) + i, 16);
    __builtin_memcpy(&d[1], reinterpret_cast<const float*>(x) + i + 4, 16);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(d[j / 4][j % 4]);
  }
}
// Rounds v to the type, stores it, and leaves the stored values in v.
template <bool BF16, int W>
__device__ __forceinline__ void rs_store(void* x, int64_t i, float v[W]) {
  if constexpr (W == 1) {
    if (BF16) {
      const uint16_t r = float_to_bf16_rne(v[0]);
      reinterpret_cast<uint16_t*>(x)[i] = r;
      v[0] = bf16_bits_to_float(r);
    } else {
      reinterpret_cast<float*>(x)[i] = v[0];
    }
  } else if constexpr (BF16) {
    u32x4 d;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      d[j] = bf16x2_rne(v[2 * j], v[2 * j + 1]);
      v[2 * j] = __uint_as_float(d[j] << 16);
      v[2 * j + 1] = __uint_as_float(d[j] & 0xffff0000u);
    }
    __builtin_memcpy(reinterpret_cast<uint16_t*>(x) + i, &d, 16);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32x4 d = {__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]),
                       __float_as_uint(v[4 * h + 2]), __float_as_uint(v[4 * h + 3])};
      __builtin_memcpy(reinterpret_cast<float*>(x) + i + 4 * h, &d, 16);
    }
  }
}

// YB / HB: bf16 y (and gate), bf16 stream.  NT threads, H groups of 8 held by each.
template <bool YB, bool HB, int NT, int H>
__global__ __launch_bounds__(NT) void residual_kernel(const ResidualArgs p, int u_bf16) {
  constexpr int NW = NT / 64;
  __shared__ float wmax[NW];
  __shared__ double wss[NW];
  __shared__ unsigned long long limbs[kSqLimbs];
  __shared__ uint32_t sqwork[kSqWork];
  __shared__ float sh_ms;
  using Eight = std::integral_constant<int, 8>;
  using One = std::integral_constant<int, 1>;
  const int64_t m = blockIdx.x, K = p.K, at = m * K;
  const int64_t n = K / 8;   // groups of the row
  const int tid = threadIdx.x;
  const int64_t last = n * 8 + tid;   // the thread's value behind them
  const bool one = last < K;

  // r of the values that each(f) visits; every thread calls it
  auto norm_factor = [&](double ss, auto each) -> float {
    ss = wave_sum_f64(ss);
    __syncthreads();   // wss may still be read from the norm before
    if ((tid & 63) == 0) wss[tid >> 6] = ss;
    __syncthreads();
    ss = 0.0;
#pragma unroll
    for (int i = 0; i < NW; ++i) ss += wss[i];
    float ms;
    if (!mean_sq_fast(ss, K, ms)) {   // near a rounding boundary (the same for all threads)
      if (tid < kSqLimbs) limbs[tid] = 0ull;
      __syncthreads();
      each([&](float v) { sq_limbs_add(limbs, v); });
      __syncthreads();
      if (tid == 0) sh_ms = sq_limbs_mean(limbs, K, sqwork);
      __syncthreads();
      ms = sh_ms;
    }
    return rms_factor_of_mean(ms, p.eps);
  };

  float y[H][8], v[H][8], y1[1], v1[1];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const int64_t g = tid + (int64_t)h * NT;
    if (g < n) {
      rs_load<YB, 8>(p.y, at + g * 8, y[h]);
      rs_load<HB, 8>(p.h, at + g * 8, v[h]);
    }
  }
  if (one) {
    rs_load<YB, 1>(p.y, at + last, y1);
    rs_load<HB, 1>(p.h, at + last, v1);
  }
  float r1 = 1.0f;
  if (p.post) {
    double ss = 0.0;
    auto each_y = [&](auto f) {
#pragma unroll
      for (int h = 0; h < H; ++h)
        if (tid + (int64_t)h * NT < n)
#pragma unroll
          for (int j = 0; j < 8; ++j) f(y[h][j]);
      for (int64_t g = tid + (int64_t)H * NT; g < n; g += NT) {
        float a[8];
        rs_load<YB, 8>(p.y, at + g * 8, a);
#pragma unroll
        for (int j = 0; j < 8; ++j) f(a[j]);
      }
      if (one) f(y1[0]);
    };
    each_y([&](float a) { ss += (double)a * (double)a; });
    r1 = norm_factor(ss, each_y);
  }

  // h' of the W values from element k on, from their y and h; the stored values stay in x
  auto join = [&](auto w8, int64_t k, const float* yy, float* x) {
    constexpr int W = decltype(w8)::value;
    float w[W], gt[W];
    if (p.post) rs_load<false, W>(p.post, k, w);
    if (p.gate) rs_load<YB, W>(p.gate, m * p.gate_stride + k, gt);
#pragma unroll
    for (int j = 0; j < W; ++j) {
      float z = yy[j];
      if (p.post) z = norm_value(z, r1, w[j]);
      if (p.gate) z = __fmul_rn(z, gt[j]);
      x[j] = __fadd_rn(x[j], __fmul_rn(z, p.scale));
    }
    rs_store<HB, W>(p.h_out, at + k, x);
  };
  double ss = 0.0;
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const int64_t g = tid + (int64_t)h * NT;
    if (g < n) {
      join(Eight{}, g * 8, y[h], v[h]);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += (double)v[h][j] * (double)v[h][j];
    }
  }
  for (int64_t g = tid + (int64_t)H * NT; g < n; g += NT) {
    float a[8], x[8];
    rs_load<YB, 8>(p.y, at + g * 8, a);
    rs_load<HB, 8>(p.h, at + g * 8, x);
    join(Eight{}, g * 8, a, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss += (double)x[j] * (double)x[j];
  }
  if (one) {
    join(One{}, last, y1, v1);
    ss += (double)v1[0] * (double)v1[0];
  }
  if (!p.u && !p.xq) return;

  float r2 = 1.0f;
  if (p.pre)
    r2 = norm_factor(ss, [&](auto f) {   // h' from registers, then from the thread's own stores
#pragma unroll
      for (int h = 0; h < H; ++h)
        if (tid + (int64_t)h * NT < n)
#pragma unroll
          for (int j = 0; j < 8; ++j) f(v[h][j]);
      for (int64_t g = tid + (int64_t)H * NT; g < n; g += NT) {
        float x[8];
        rs_load<HB, 8>(p.h_out, at + g * 8, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) f(x[j]);
      }
      if (one) f(v1[0]);
    });
  // u of W values of h'; returns their largest magnitude
  auto normed = [&](auto w8, int64_t k, float* x) -> float {
    constexpr int W = decltype(w8)::value;
    float w[W], a = 0.0f;
    if (p.pre) rs_load<false, W>(p.pre, k, w);
#pragma unroll
    for (int j = 0; j < W; ++j) {
      if (p.pre) x[j] = norm_value(x[j], r2, w[j]);
      a = fmaxf(a, fabsf(x[j]));
    }
    return a;
  };
  // u of the held values replaces h'
  float a = 0.0f;
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const int64_t g = tid + (int64_t)h * NT;
    if (g < n) a = fmaxf(a, normed(Eight{}, g * 8, v[h]));
  }
  for (int64_t g = tid + (int64_t)H * NT; g < n; g += NT) {
    float x[8];
    rs_load<HB, 8>(p.h_out, at + g * 8, x);
    a = fmaxf(a, normed(Eight{}, g * 8, x));
  }
  if (one) a = fmaxf(a, normed(One{}, last, v1));
  float s = 0.0f;
  if (p.xq) {
    a = wave_max(a);
    if ((tid & 63) == 0) wmax[tid >> 6] = a;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NW; ++i) a = fmaxf(a, wmax[i]);
    const float astar = fmaxf(a, kEps);
    s = kQb / astar;
    if (tid == 0) p.xs[m] = astar / kQb;
  }
  auto finish = [&](auto w8, int64_t k, float* u) {
    constexpr int W = decltype(w8)::value;
    if (p.xq) {
      if constexpr (W == 1) {
        p.xq[at + k] = (int8_t)(uint8_t)rne_bits(u[0], s);
      } else {
        const u32x2 q = {quant4(u, s), quant4(u + 4, s)};
        __builtin_memcpy(p.xq + at + k, &q, 8);
      }
    }
    if (p.u) {
      if (u_bf16)
        rs_store<true, W>(p.u, at + k, u);
      else
        rs_store<false, W>(p.u, at + k, u);
    }
  };
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const int64_t g = tid + (int64_t)h * NT;
    if (g < n) finish(Eight{}, g * 8, v[h]);
  }
  for (int64_t g = tid + (int64_t)H * NT; g < n; g += NT) {
    float x[8];
    rs_load<HB, 8>(p.h_out, at + g * 8, x);
    normed(Eight{}, g * 8, x);
    finish(Eight{}, g * 8, x);
  }
  if (one) finish(One{}, last, v1);
}

// Threads of a workgroup.  Rows of up to 4096 fit one or two groups a thread; one each
// for few tokens, whose time is the chain of the sums (2560 wide: 4.1 -> 3.8 us), and
// small workgroups for small rows (4096 x 640: 15.2 -> 10.3 us).  Longer rows take more
// threads (2048 x 8192, fp32 stream: 57.6 -> 48.6 us; one token of 14336: 9.9 -> 6.1),
// but sixteen waves leave a compute unit one workgroup, so that many tokens rather read
// part of h' again (2048 x 10240, bf16: 59.6 with 1024 threads, 47.6 with 512).
template <bool YB, bool HB>
const void* residual_pick(int64_t K, int64_t M, int* threads) {
  if (K <= 1024) {
    *threads = 128;
    return (const void*)residual_kernel<YB, HB, 128, 1>;
  }
  if (K <= 4096 && M > 64) {
    *threads = 256;
    return (const void*)residual_kernel<YB, HB, 256, 2>;
  }
  if (K <= 4096) {
    *threads = 512;
    return (const void*)residual_kernel<YB, HB, 512, 1>;
  }
  if (K <= 8192 || M > 256) {
    *threads = 512;
    return (const void*)residual_kernel<YB, HB, 512, 2>;
  }
  *threads = 1024;
  return (const void*)residual_kernel<YB, HB, 1024, 2>;
}

}  // namespace

hipError_t launch_residual(const ResidualArgs& a, bool y_bf16, bool h_bf16, bool u_bf16, int64_t M,
                           hipStream_t s) {
  int threads;
  const void* kern = y_bf16 ? (h_bf16 ? residual_pick<true, true>(a.K, M, &threads)
                                      : residual_pick<true, false>(a.K, M, &threads))
                            : (h_bf16 ? residual_pick<false, true>(a.K, M, &threads)
                                      : residual_pick<false, false>(a.K, M, &threads));
  const int ub = u_bf16 ? 1 : 0;
  void* args[] = {(void*)&a, (void*)&ub};
  return hipLaunchKernel(kern, dim3((unsigned)M), dim3((unsigned)threads), args, 0, s);
}

}  // namespace bitnet
