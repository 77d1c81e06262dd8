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
// Bound by memory: y and h are read once, h' and the codes written once.  One
// workgroup per token; each thread keeps its first H groups of 8 values in
// registers from the first sum to the last store.  Rows beyond that read h' again
// (never h, which h_out may replace).
#include "bitnet_internal.h"

namespace bitnet {
namespace {

template <bool BF16>
__device__ __forceinline__ float rs_load1(const void* x, int64_t i) {
  if (BF16) return bf16_bits_to_float(reinterpret_cast<const uint16_t*>(x)[i]);
  return reinterpret_cast<const float*>(x)[i];
}
template <bool BF16>
__device__ __forceinline__ void rs_store1(void* x, int64_t i, float v) {
  if (BF16)
    reinterpret_cast<uint16_t*>(x)[i] = float_to_bf16_rne(v);
  else
    reinterpret_cast<float*>(x)[i] = v;
}

// W consecutive elements (8 from a 16-byte aligned address, or 1).
template <bool BF16, int W>
__device__ __forceinline__ void rs_load(const void* x, int64_t i, float v[W]) {
  if (W == 1) {
    v[0] = rs_load1<BF16>(x, i);
  } else if (BF16) {
    const uint4 a = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(x) + i);
    const uint32_t d[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < W / 2; ++j) {
      v[2 * j] = __uint_as_float(d[j] << 16);
      v[2 * j + 1] = __uint_as_float(d[j] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int h = 0; h < W / 4; ++h) {
      const float4 a = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(x) + i)[h];
      v[4 * h] = a.x;
      v[4 * h + 1] = a.y;
      v[4 * h + 2] = a.z;
      v[4 * h + 3] = a.w;
    }
  }
}
// Rounds v to the type, stores it, and leaves the stored values in v.
template <bool BF16, int W>
__device__ __forceinline__ void rs_store(void* x, int64_t i, float v[W]) {
  if (W == 1) {
    rs_store1<BF16>(x, i, v[0]);
    if (BF16) v[0] = bf16_bits_to_float(float_to_bf16_rne(v[0]));
  } else if (BF16) {
    uint32_t w[W / 2 + 1];
#pragma unroll
    for (int j = 0; j < W / 2; ++j) {
      w[j] = bf16x2_rne(v[2 * j], v[2 * j + 1]);
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(x) + i) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(x) + i);
#pragma unroll
    for (int h = 0; h < W / 4; ++h)
      p[h] = make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
  }
}

// YB / HB: bf16 y (and gate), bf16 stream.  W: elements a group (8 or 1).  NT
// threads, H groups held by each.
template <bool YB, bool HB, int W, int NT, int H>
__global__ __launch_bounds__(NT) void residual_kernel(const ResidualArgs p, int u_bf16) {
  constexpr int NW = NT / 64;
  __shared__ float wmax[NW];
  __shared__ double wss[NW];
  __shared__ unsigned long long limbs[kSqLimbs];
  __shared__ uint32_t sqwork[kSqWork];
  __shared__ float sh_ms;
  const int64_t m = blockIdx.x, K = p.K, at = m * K;
  const int64_t n = K / W;   // groups of the row (K is a multiple of W)
  const int tid = threadIdx.x;

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

  float y[H][W], v[H][W];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const int64_t g = tid + (int64_t)h * NT;
    if (g < n) {
      rs_load<YB, W>(p.y, at + g * W, y[h]);
      rs_load<HB, W>(p.h, at + g * W, v[h]);
    }
  }
  float r1 = 1.0f;
  if (p.post) {
    double ss = 0.0;
    auto each_y = [&](auto f) {
#pragma unroll
      for (int h = 0; h < H; ++h)
        if (tid + (int64_t)h * NT < n)
#pragma unroll
          for (int j = 0; j < W; ++j) f(y[h][j]);
      for (int64_t g = tid + (int64_t)H * NT; g < n; g += NT) {
        float a[W];
        rs_load<YB, W>(p.y, at + g * W, a);
#pragma unroll
        for (int j = 0; j < W; ++j) f(a[j]);
      }
    };
    each_y([&](float a) { ss += (double)a * (double)a; });
    r1 = norm_factor(ss, each_y);
  }

  // h' of group g from its y and h, stored; the stored values stay in x
  auto join = [&](int64_t g, const float* yy, float* x) {
    float w[W], gt[W];
    if (p.post) rs_load<false, W>(p.post, g * W, w);
    if (p.gate) rs_load<YB, W>(p.gate, m * p.gate_stride + g * W, gt);
#pragma unroll
    for (int j = 0; j < W; ++j) {
      float z = yy[j];
      if (p.post) z = norm_value(z, r1, w[j]);
      if (p.gate) z = __fmul_rn(z, gt[j]);
      x[j] = __fadd_rn(x[j], __fmul_rn(z, p.scale));
    }
    rs_store<HB, W>(p.h_out, at + g * W, x);
  };
  double ss = 0.0;
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const int64_t g = tid + (int64_t)h * NT;
    if (g < n) {
      join(g, y[h], v[h]);
#pragma unroll
      for (int j = 0; j < W; ++j) ss += (double)v[h][j] * (double)v[h][j];
    }
  }
  for (int64_t g = tid + (int64_t)H * NT; g < n; g += NT) {
    float a[W], x[W];
    rs_load<YB, W>(p.y, at + g * W, a);
    rs_load<HB, W>(p.h, at + g * W, x);
    join(g, a, x);
#pragma unroll
    for (int j = 0; j < W; ++j) ss += (double)x[j] * (double)x[j];
  }
  if (!p.u && !p.xq) return;

  // visits the thread's groups of h' (from registers, then from h_out: its own stores)
  auto each_group = [&](auto f) {
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int64_t g = tid + (int64_t)h * NT;
      if (g < n) f(g, v[h]);
    }
    for (int64_t g = tid + (int64_t)H * NT; g < n; g += NT) {
      float x[W];
      rs_load<HB, W>(p.h_out, at + g * W, x);
      f(g, x);
    }
  };
  float r2 = 1.0f;
  if (p.pre)
    r2 = norm_factor(ss, [&](auto f) {
      each_group([&](int64_t, const float* x) {
#pragma unroll
        for (int j = 0; j < W; ++j) f(x[j]);
      });
    });
  auto normed = [&](int64_t g, const float* x, float* u) {
    float w[W];
    if (p.pre) rs_load<false, W>(p.pre, g * W, w);
#pragma unroll
    for (int j = 0; j < W; ++j) u[j] = p.pre ? norm_value(x[j], r2, w[j]) : x[j];
  };
  // u of the held groups replaces h' in v
  float a = 0.0f;
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const int64_t g = tid + (int64_t)h * NT;
    if (g < n) {
      normed(g, v[h], v[h]);
#pragma unroll
      for (int j = 0; j < W; ++j) a = fmaxf(a, fabsf(v[h][j]));
    }
  }
  for (int64_t g = tid + (int64_t)H * NT; g < n; g += NT) {
    float x[W];
    rs_load<HB, W>(p.h_out, at + g * W, x);
    normed(g, x, x);
#pragma unroll
    for (int j = 0; j < W; ++j) a = fmaxf(a, fabsf(x[j]));
  }
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
  auto finish = [&](int64_t g, float* u) {
    if (p.xq) {
      if (W == 1) {
        const float q = rintf(__fmul_rn(u[0], s));
        p.xq[at + g] = (int8_t)(int)fminf(fmaxf(q, -128.0f), 127.0f);
      } else {
        *reinterpret_cast<uint2*>(p.xq + at + g * W) =
            make_uint2(quant4(u, s), quant4(u + 4 % W, s));
      }
    }
    if (p.u) {
      if (u_bf16)
        rs_store<true, W>(p.u, at + g * W, u);
      else
        rs_store<false, W>(p.u, at + g * W, u);
    }
  };
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const int64_t g = tid + (int64_t)h * NT;
    if (g < n) finish(g, v[h]);
  }
  for (int64_t g = tid + (int64_t)H * NT; g < n; g += NT) {
    float x[W];
    rs_load<HB, W>(p.h_out, at + g * W, x);
    normed(g, x, x);
    finish(g, x);
  }
}

// Threads of a workgroup.  Rows of up to 4096 fit one or two groups a thread; one each
// for few tokens, whose time is the chain of the sums (2560 wide: 4.1 -> 3.8 us), and
// small workgroups for small rows (4096 x 640: 15.2 -> 10.3 us).  Longer rows take more
// threads (2048 x 8192, fp32 stream: 57.6 -> 48.6 us; one token of 14336: 9.9 -> 6.1),
// but sixteen waves leave a compute unit one workgroup, so that many tokens rather read
// part of h' again (2048 x 10240, bf16: 59.6 with 1024 threads, 47.6 with 512).
template <bool YB, bool HB>
const void* residual_pick(bool vec, int64_t K, int64_t M, int* threads) {
  if (!vec) {
    *threads = 256;
    return (const void*)residual_kernel<YB, HB, 1, 256, 8>;
  }
  if (K <= 1024) {
    *threads = 128;
    return (const void*)residual_kernel<YB, HB, 8, 128, 1>;
  }
  if (K <= 4096 && M > 64) {
    *threads = 256;
    return (const void*)residual_kernel<YB, HB, 8, 256, 2>;
  }
  if (K <= 4096) {
    *threads = 512;
    return (const void*)residual_kernel<YB, HB, 8, 512, 1>;
  }
  if (K <= 8192 || M > 256) {
    *threads = 512;
    return (const void*)residual_kernel<YB, HB, 8, 512, 2>;
  }
  *threads = 1024;
  return (const void*)residual_kernel<YB, HB, 8, 1024, 2>;
}

}  // namespace

hipError_t launch_residual(const ResidualArgs& a, bool y_bf16, bool h_bf16, bool u_bf16, int64_t M,
                           hipStream_t s) {
  const auto al = [](const void* p, uintptr_t b) { return ((uintptr_t)p & (b - 1)) == 0; };
  const bool vec = a.K % 8 == 0 && al(a.y, 16) && al(a.h, 16) && al(a.gate, 16) && al(a.h_out, 16) &&
                   al(a.u, 16) && al(a.post, 16) && al(a.pre, 16) && al(a.xq, 8) &&
                   a.gate_stride % 8 == 0;
  int threads;
  const void* kern = y_bf16 ? (h_bf16 ? residual_pick<true, true>(vec, a.K, M, &threads)
                                      : residual_pick<true, false>(vec, a.K, M, &threads))
                            : (h_bf16 ? residual_pick<false, true>(vec, a.K, M, &threads)
                                      : residual_pick<false, false>(vec, a.K, M, &threads));
  const int ub = u_bf16 ? 1 : 0;
  void* args[] = {(void*)&a, (void*)&ub};
  return hipLaunchKernel(kern, dim3((unsigned)M), dim3((unsigned)threads), args, 0, s);
}

}  // namespace bitnet
