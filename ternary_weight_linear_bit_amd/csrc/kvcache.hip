// Appending keys and values to the paged 8-bit cache, with the rotation of the
// queries and keys by their positions.
//
// One page of one head holds P tokens as int8 codes and one scale d:
//   x ~ code * d.  For the rows x that a call adds to a page (keys after their
//   rotation), need = RN32(max(max|x|, RN32(1e-5)) / 127); a page that the call
//   begins takes d' = need, a page with earlier tokens d' = max(d, need) and, if
//   that is larger, its earlier codes c become rne(RN32(c * RN32(d / d'))).  New
//   codes are clip(rne(RN32(x * RN32(1 / d'))), -127, 127).
// Rotation of a pair (a, b) by an angle with cosine c and sine s from the caller's
// tables: (RN32(RN32(a c) - RN32(b s)), RN32(RN32(b c) + RN32(a s))).
//
// Keys lie [P][D] and values [D][P] in their page: both are then the 16
// consecutive bytes that a lane of the attention kernel's matrix products takes
// (along the head's dims for q.k, along the tokens for p.v), so that kernel moves
// codes from memory to the matrix cores without a transposition.
//
// One workgroup per (sequence, touched page, kv head, keys or values), so that the
// page's new maximum, its scale and its earlier codes have one owner; further
// workgroups of the same launch rotate the queries.
#include "bitnet_internal.h"

namespace bitnet {
namespace {

constexpr int kKvThreads = 256;

template <bool BF16>
__device__ __forceinline__ float kv_load1(const void* x, int64_t i) {
  if (BF16) return bf16_bits_to_float(reinterpret_cast<const uint16_t*>(x)[i]);
  return reinterpret_cast<const float*>(x)[i];
}

// 8 consecutive elements from index i; VEC: the address is 16-byte aligned.
template <bool BF16, bool VEC>
__device__ __forceinline__ void kv_load8(const void* x, int64_t i, float v[8]) {
  if (!VEC) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = kv_load1<BF16>(x, i + j);
  } else if (BF16) {
    const uint4 a = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(x) + i);
    const uint32_t d[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(d[j] << 16);
      v[2 * j + 1] = __uint_as_float(d[j] & 0xffff0000u);
    }
  } else {
    const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(x) + i);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 a = p[h];
      v[4 * h] = a.x;
      v[4 * h + 1] = a.y;
      v[4 * h + 2] = a.z;
      v[4 * h + 3] = a.w;
    }
  }
}

// Dims d0 .. d0 + 7 of one head's row at `x`, rotated: cs / sn are the position's
// rows of the tables (rot / 2 entries).  Dims from rot on pass through.
template <bool BF16, bool VEC>
__device__ __forceinline__ void rotated8(const void* x, int64_t base, int d0, int rot,
                                         bool neighbours, const float* cs, const float* sn,
                                         float v[8]) {
  kv_load8<BF16, VEC>(x, base + d0, v);
  if (d0 >= rot) return;
  const int half = rot >> 1;
  if (neighbours) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      if (d0 + j < rot) {
        const float c = cs[(d0 + j) >> 1], s = sn[(d0 + j) >> 1];
        const float a = v[j], b = v[j + 1];
        v[j] = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
        v[j + 1] = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
      }
    }
    return;
  }
  float w[8];
  if (VEC && (half & 7) == 0) {   // the 8 partners are one group too
    kv_load8<BF16, true>(x, base + (d0 < half ? d0 + half : d0 - half), w);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int d = d0 + j;
      w[j] = d < rot ? kv_load1<BF16>(x, base + (d < half ? d + half : d - half)) : 0.0f;
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int d = d0 + j;
    if (d < half) {
      v[j] = __fsub_rn(__fmul_rn(v[j], cs[d]), __fmul_rn(w[j], sn[d]));
    } else if (d < rot) {
      v[j] = __fadd_rn(__fmul_rn(v[j], cs[d - half]), __fmul_rn(w[j], sn[d - half]));
    }
  }
}

__device__ __forceinline__ int kv_code(float x, float inv) {
  return (int)fminf(fmaxf(rintf(__fmul_rn(x, inv)), -127.0f), 127.0f);
}

// The codes in the bytes of w selected by `mask` (0xff per byte), at a larger scale.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, uint32_t mask, float f) {
  uint32_t o = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const float c = (float)(int8_t)(w >> (8 * b));
    o |= ((uint32_t)(int)rintf(__fmul_rn(c, f)) & 0xffu) << (8 * b);
  }
  return (w & ~mask) | (o & mask);
}

// 0xff in each byte b of a dword at slot s with s + b < lim.
__device__ __forceinline__ uint32_t below_mask(int s, int lim) {
  const int n = lim - s;
  return n >= 4 ? 0xffffffffu : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
}

template <bool BF16, bool VEC>
__global__ __launch_bounds__(kKvThreads) void kv_append_kernel(const KvCache c, const KvBatch b,
                                                               const KvRows r, int pages_per_seq,
                                                               int page_units, int q_blocks) {
  extern __shared__ uint4 tile4[];   // values: the page's codes [D][P]
  __shared__ float wmax[kKvThreads / 64];
  const int tid = threadIdx.x;
  int unit = blockIdx.x;
  const int D = c.head_dim, P = c.page, G = D / 8;

  if (unit >= page_units) {   // rotate queries: kKvQRows rows of one sequence
    unit -= page_units;
    const int seq = unit / q_blocks;
    const SeqSpan sp = seq_span(b, seq);
    const int i0 = (unit - seq * q_blocks) * kKvQRows;
    const int i1 = min(min(i0 + kKvQRows, sp.n), b.max_new);
    const int per_row = r.q_heads * G;
    for (int i = i0; i < i1; ++i) {
      const int64_t t = sp.s0 + i;
      const int pos = sp.first + i;
      const float* cs = r.cos + (int64_t)max(pos, 0) * (r.rot >> 1);
      const float* sn = r.sin + (int64_t)max(pos, 0) * (r.rot >> 1);
      const int rot = pos < 0 ? 0 : r.rot;   // a row without a place is copied
      // a pass covers whole heads and reads all of its values before it writes
      // any, which makes q_out == q safe
      for (int g0 = 0; g0 < per_row; g0 += kKvThreads / G * G) {
        const int g = g0 + tid;
        const bool on = tid < kKvThreads / G * G && g < per_row;
        float v[8];
        const int d0 = on ? g % G * 8 : 0;
        const int64_t head = on ? g / G : 0;
        if (on) rotated8<BF16, VEC>(r.q, t * r.q_stride + head * D, d0, rot, r.neighbours, cs, sn, v);
        __syncthreads();
        if (!on) continue;
        const int64_t o = t * ((int64_t)r.q_heads * D) + head * D + d0;
        if (BF16) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = bf16x2_rne(v[2 * j], v[2 * j + 1]);
          *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(r.q_out) + o) =
              make_uint4(w[0], w[1], w[2], w[3]);
        } else {
          float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(r.q_out) + o);
          p[0] = make_float4(v[0], v[1], v[2], v[3]);
          p[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
      }
    }
    return;
  }

  const bool vals = unit & 1;
  unit >>= 1;
  const int head = unit % c.kv_heads;
  unit /= c.kv_heads;
  const int seq = unit / pages_per_seq;
  const SeqSpan sp = seq_span(b, seq);
  // the page's positions that this call adds: slots [lo, hi)
  const int at0 = max(sp.first, 0);
  const int end = min(sp.len, sp.first + b.max_new);   // max_new bounds every sequence's rows
  const int pg = at0 / P + (unit - seq * pages_per_seq);
  const int lo = max(at0 - pg * P, 0), hi = min(end - pg * P, P);
  if (lo >= hi) return;
  const int pid = b.table[(int64_t)seq * b.width + pg];
  if (pid < 0 || pid >= c.pages) return;

  const int64_t t0 = sp.s0 + (pg * P + lo - sp.first);
  const void* src = vals ? r.v : r.k;
  const int64_t stride = vals ? r.v_stride : r.k_stride;
  const int rot = vals ? 0 : r.rot;
  const int items = (hi - lo) * G;
  auto load = [&](int it, float v[8]) {
    const int slot = it / G, d0 = (it - slot * G) * 8;
    const int64_t pos = (int64_t)pg * P + lo + slot;
    const int half = rot >> 1;
    rotated8<BF16, VEC>(src, (t0 + slot) * stride + (int64_t)head * D, d0, rot, r.neighbours,
                        r.cos + pos * half, r.sin + pos * half, v);
  };

  float* scale = (vals ? c.v_scale : c.k_scale) + (int64_t)pid * c.kv_heads + head;
  const float d_old = lo > 0 ? *scale : 0.0f;
  float a = 0.0f;
  for (int it = tid; it < items; it += kKvThreads) {
    float v[8];
    load(it, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) a = fmaxf(a, fabsf(v[j]));
  }
  a = wave_max(a);
  if ((tid & 63) == 0) wmax[tid >> 6] = a;
  __syncthreads();   // also: every thread has the old scale
#pragma unroll
  for (int i = 0; i < kKvThreads / 64; ++i) a = fmaxf(a, wmax[i]);
  const float need = fmaxf(a, kEps) / kQb;
  const float d = fmaxf(need, d_old);
  const bool grown = lo > 0 && d > d_old;
  const float f = d_old / d, inv = 1.0f / d;
  if (tid == 0) *scale = d;

  const int64_t page_at = ((int64_t)pid * c.kv_heads + head) * P * D;
  if (!vals) {
    int8_t* dst = c.k + page_at;
    if (grown) {
      for (int i = tid; i < lo * D / 16; i += kKvThreads) {
        uint4* p = reinterpret_cast<uint4*>(dst) + i;
        const uint4 w = *p;
        *p = make_uint4(rescale4(w.x, ~0u, f), rescale4(w.y, ~0u, f), rescale4(w.z, ~0u, f),
                        rescale4(w.w, ~0u, f));
      }
    }
    for (int it = tid; it < items; it += kKvThreads) {
      float v[8];
      load(it, v);
      uint32_t w[2] = {0u, 0u};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        w[j >> 2] |= ((uint32_t)kv_code(v[j], inv) & 0xffu) << (8 * (j & 3));
      *reinterpret_cast<uint2*>(dst + (int64_t)lo * D + (int64_t)it * 8) = make_uint2(w[0], w[1]);
    }
    return;
  }

  // values: the 16-byte groups of slots that hold new (or, with a larger scale,
  // earlier) tokens pass through LDS, where the new codes take their bytes
  int8_t* dst = c.v + page_at;
  uint8_t* tile = reinterpret_cast<uint8_t*>(tile4);
  const int c0 = grown ? 0 : lo / 16, c1 = (hi + 15) / 16, nc = c1 - c0;
  for (int i = tid; i < D * nc; i += kKvThreads) {
    const int row = i / nc, s = (c0 + i - row * nc) * 16;
    if (s >= lo && s + 16 <= hi) continue;   // new tokens only
    uint4 w = *reinterpret_cast<const uint4*>(dst + row * P + s);
    if (grown) {
      w.x = rescale4(w.x, below_mask(s, lo), f);
      w.y = rescale4(w.y, below_mask(s + 4, lo), f);
      w.z = rescale4(w.z, below_mask(s + 8, lo), f);
      w.w = rescale4(w.w, below_mask(s + 12, lo), f);
    }
    *reinterpret_cast<uint4*>(tile + row * P + s) = w;
  }
  __syncthreads();
  for (int it = tid; it < items; it += kKvThreads) {
    float v[8];
    load(it, v);
    const int slot = it / G, d0 = (it - slot * G) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) tile[(d0 + j) * P + lo + slot] = (uint8_t)kv_code(v[j], inv);
  }
  __syncthreads();
  for (int i = tid; i < D * nc; i += kKvThreads) {
    const int row = i / nc, s = (c0 + i - row * nc) * 16;
    *reinterpret_cast<uint4*>(dst + row * P + s) = *reinterpret_cast<const uint4*>(tile + row * P + s);
  }
}

}  // namespace

hipError_t launch_kv_append(const KvCache& c, const KvBatch& b, const KvRows& r, bool bf16,
                            hipStream_t s) {
  const int pages_per_seq = (b.max_new + c.page - 2) / c.page + 1;
  const int64_t page_units = (int64_t)b.seqs * pages_per_seq * c.kv_heads * 2;
  const int q_blocks = r.q ? (b.max_new + kKvQRows - 1) / kKvQRows : 0;
  const int64_t grid = page_units + (int64_t)b.seqs * q_blocks;
  if (grid > 2147483647) return hipErrorInvalidValue;
  const auto a16 = [](const void* p, int64_t stride, size_t es) {
    return p == nullptr || (((uintptr_t)p & 15u) == 0 && (stride * es) % 16 == 0);
  };
  const size_t es = bf16 ? 2 : 4;
  const bool vec = a16(r.k, r.k_stride, es) && a16(r.v, r.v_stride, es) && a16(r.q, r.q_stride, es);
  const int pu = (int)page_units;
  const void* kern = bf16 ? (vec ? (const void*)kv_append_kernel<true, true>
                                 : (const void*)kv_append_kernel<true, false>)
                          : (vec ? (const void*)kv_append_kernel<false, true>
                                 : (const void*)kv_append_kernel<false, false>);
  void* args[] = {(void*)&c, (void*)&b, (void*)&r, (void*)&pages_per_seq, (void*)&pu,
                  (void*)&q_blocks};
  return hipLaunchKernel(kern, dim3((unsigned)grid), dim3(kKvThreads), args,
                         (size_t)c.page * c.head_dim, s);
}

}  // namespace bitnet
