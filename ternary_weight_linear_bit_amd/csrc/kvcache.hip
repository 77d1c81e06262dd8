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
// workgroups of the same launch rotate the queries.  A thread's item is a pair of
// groups of W dims that rotate into each other (so that queries can be rotated in
// place); it stays in registers from the maximum to the codes.
//
// Prompts are bound by memory (4096 bf16 tokens of 20 + 5 + 5 heads: 13.4 us, 4.5 TB/s;
// 1374 fp32 tokens of 64 + 64 + 64 heads in seven sequences: 54.6 us, 3.7 TB/s), single
// tokens by the chain of dependent loads (row numbers and length; page id, row, angles;
// scale and earlier codes; 3.7 us in a graph): each link's loads are issued together.
#include "layer_internal.h"

namespace bitnet {
namespace {

constexpr int kKvThreads = 256;

template <int W>
using vec = float __attribute__((ext_vector_type(W)));

// W consecutive elements from element i, aligned to the element (the hardware takes
// 16-byte loads at any element's alignment).
template <bool BF16, int W>
__device__ __forceinline__ vec<W> kv_load(const void* x, int64_t i) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  vec<W> v;
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
    u32x4 a, b;
    __builtin_memcpy(&a, reinterpret_cast<const float*>(x) + i, 16);
    __builtin_memcpy(&b, reinterpret_cast<const float*>(x) + i + 4, 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = __uint_as_float(a[j]);
      v[j + 4] = __uint_as_float(b[j]);
    }
  }
  return v;
}

// A pair of groups of W dims: dims a .. a + W - 1 and b .. b + W - 1.  Of a rotated
// head's D / (2 W) pairs the first rot / (2 W) hold, in the order of halves, dims that
// turn into each other; the others, and all in the order of neighbours, lie side by side.
template <int W>
struct Pair {
  vec<W> x, y;
  int a, b;
};
template <int W>
__device__ __forceinline__ void place(Pair<W>& p, int j, int rot, bool neighbours) {
  const int half = rot >> 1;
  const bool apart = !neighbours && j * W < half;
  p.a = apart ? j * W : neighbours ? 2 * W * j : rot + 2 * (j * W - half);
  p.b = apart ? p.a + half : p.a + W;
}
// The angles that turn a pair: W entries of the position's table rows, from the one
// of dim a on.  (W = 8 takes rot % 16 == 0, so a pair is rotated as a whole or not.)
template <int W>
struct Angles {
  vec<W> c, s;
};
template <int W>
__device__ __forceinline__ bool turned(const Pair<W>& p, int rot, bool neighbours) {
  return p.a < (neighbours ? rot : rot >> 1);
}
template <int W>
__device__ __forceinline__ void load_angles(Angles<W>& g, const Pair<W>& p, const float* cs,
                                            const float* sn, int rot, bool neighbours) {
  if (turned(p, rot, neighbours)) {
    const int at = neighbours ? p.a >> 1 : p.a;
    g.c = kv_load<false, W>(cs, at);
    g.s = kv_load<false, W>(sn, at);
  }
}
__device__ __forceinline__ float turn_a(float a, float b, float c, float s) {
  return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
}
__device__ __forceinline__ float turn_b(float a, float b, float c, float s) {
  return __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}
template <int W>
__device__ __forceinline__ void rotate(Pair<W>& p, const Angles<W>& g, int rot, bool neighbours) {
  if (!turned(p, rot, neighbours)) return;
  const vec<W> x = p.x, y = p.y;
  if (!neighbours || W == 1) {
#pragma unroll
    for (int j = 0; j < W; ++j) {
      p.x[j] = turn_a(x[j], y[j], g.c[j], g.s[j]);
      p.y[j] = turn_b(x[j], y[j], g.c[j], g.s[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j + 1 < W; j += 2) {
      const int k = (W + j) / 2;
      p.x[j] = turn_a(x[j], x[j + 1], g.c[j / 2], g.s[j / 2]);
      p.x[j + 1] = turn_b(x[j], x[j + 1], g.c[j / 2], g.s[j / 2]);
      p.y[j] = turn_a(y[j], y[j + 1], g.c[k], g.s[k]);
      p.y[j + 1] = turn_b(y[j], y[j + 1], g.c[k], g.s[k]);
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

// W codes of one group to consecutive bytes.
template <int W>
__device__ __forceinline__ void store_codes(int8_t* at, vec<W> x, float inv) {
  if constexpr (W == 1) {
    *at = (int8_t)kv_code(x[0], inv);
  } else {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int j = 0; j < W; ++j) w[j >> 2] |= ((uint32_t)kv_code(x[j], inv) & 0xffu) << (8 * (j & 3));
    *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
  }
}

template <bool BF16, int W>
__device__ __forceinline__ void store_row(void* out, int64_t i, vec<W> v) {
  if (BF16) {
    uint16_t* p = reinterpret_cast<uint16_t*>(out) + i;
    if constexpr (W == 1) {
      *p = float_to_bf16_rne(v[0]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < W / 2; ++j) w[j] = bf16x2_rne(v[2 * j], v[2 * j + 1]);
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
    float* p = reinterpret_cast<float*>(out) + i;
    if constexpr (W == 1) {
      *p = v[0];
    } else {
#pragma unroll
      for (int h = 0; h < W / 4; ++h)
        reinterpret_cast<float4*>(p)[h] = make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
    }
  }
}

// W: dims a group (8, or 1 where the rotated dims are no whole pairs of groups).  H: pairs that a thread keeps; a page with more reads its rows again.
template <bool BF16, int W, int H>
__global__ __launch_bounds__(kKvThreads) void kv_append_kernel(const KvCache c, const KvBatch b,
                                                               const KvRows r, int pages_per_seq,
                                                               int page_units) {
  extern __shared__ uint4 tile4[];   // values: the page's codes [D][P]
  __shared__ float wmax[kKvThreads / 64];
  const int tid = threadIdx.x;
  int unit = blockIdx.x;
  const int D = c.head_dim, P = c.page, J = D / (2 * W);   // J: pairs of a head

  if (unit >= page_units) {   // rotate one row of a sequence's queries
    unit -= page_units;
    const int seq = unit / b.max_new, i = unit - seq * b.max_new;
    const SeqSpan sp = seq_span(b, seq);
    if (i >= sp.n) return;
    const int64_t t = sp.s0 + i;
    const int pos = sp.first + i;
    const int rot = pos < 0 ? 0 : r.rot;   // a row without a place is copied
    const bool neighbours = pos < 0 || r.neighbours;
    const int64_t at = (int64_t)max(pos, 0) * (r.rot >> 1);
    for (int it = tid; it < r.q_heads * J; it += kKvThreads) {
      const int head = it / J;
      Pair<W> p;
      Angles<W> g;
      place(p, it - head * J, rot, neighbours);
      const int64_t base = t * r.q_stride + (int64_t)head * D;
      p.x = kv_load<BF16, W>(r.q, base + p.a);
      p.y = kv_load<BF16, W>(r.q, base + p.b);
      load_angles(g, p, r.cos + at, r.sin + at, rot, neighbours);
      rotate(p, g, rot, neighbours);
      const int64_t o = (t * r.q_heads + head) * D;
      store_row<BF16, W>(r.q_out, o + p.a, p.x);
      store_row<BF16, W>(r.q_out, o + p.b, p.y);
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

  const int items = (hi - lo) * J;   // pairs of the new rows
  const int64_t t0 = sp.s0 + (pg * P + lo - sp.first);
  const void* src = vals ? r.v : r.k;
  const int64_t stride = vals ? r.v_stride : r.k_stride;
  const int rot = vals ? 0 : r.rot;
  const bool neighbours = vals || r.neighbours;
  auto load = [&](int it, Pair<W>& p, Angles<W>& g) {
    const int slot = it / J;
    place(p, it - slot * J, rot, neighbours);
    const int64_t base = (t0 + slot) * stride + (int64_t)head * D;
    p.x = kv_load<BF16, W>(src, base + p.a);
    p.y = kv_load<BF16, W>(src, base + p.b);
    const int64_t at = ((int64_t)pg * P + lo + slot) * (rot >> 1);
    load_angles(g, p, r.cos + at, r.sin + at, rot, neighbours);
  };
  Pair<W> p[H];
  {
    Angles<W> g[H];
#pragma unroll
    for (int h = 0; h < H; ++h)
      if (tid + h * kKvThreads < items) load(tid + h * kKvThreads, p[h], g[h]);
    if (pid < 0 || pid >= c.pages) return;
#pragma unroll
    for (int h = 0; h < H; ++h)
      if (tid + h * kKvThreads < items) rotate(p[h], g[h], rot, neighbours);
  }
  float* scale = (vals ? c.v_scale : c.k_scale) + (int64_t)pid * c.kv_heads + head;
  const float d_old = lo > 0 ? *scale : 0.0f;
  const int64_t page_at = ((int64_t)pid * c.kv_heads + head) * P * D;
  int8_t* vdst = c.v + page_at;
  uint8_t* tile = reinterpret_cast<uint8_t*>(tile4);
  const int c0 = lo / 16, c1 = (hi + 15) / 16;
  if (vals) {   // 16-byte groups of slots that hold other tokens too: first and last
    for (int i = tid; i < 2 * D; i += kKvThreads) {
      const int row = i >> 1, s = (i & 1 ? c1 - 1 : c0) * 16;
      if ((i & 1) && c1 - 1 == c0) continue;
      if (s < lo || s + 16 > hi)
        *reinterpret_cast<uint4*>(tile + row * P + s) = *reinterpret_cast<const uint4*>(vdst + row * P + s);
    }
  }
  float a = 0.0f;
#pragma unroll
  for (int h = 0; h < H; ++h)
    if (tid + h * kKvThreads < items)
#pragma unroll
      for (int j = 0; j < W; ++j) a = fmaxf(a, fmaxf(fabsf(p[h].x[j]), fabsf(p[h].y[j])));
  for (int it = tid + H * kKvThreads; it < items; it += kKvThreads) {
    Pair<W> q;
    Angles<W> g;
    load(it, q, g);
    rotate(q, g, rot, neighbours);
#pragma unroll
    for (int j = 0; j < W; ++j) a = fmaxf(a, fmaxf(fabsf(q.x[j]), fabsf(q.y[j])));
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

  auto each = [&](auto put) {
#pragma unroll
    for (int h = 0; h < H; ++h)
      if (tid + h * kKvThreads < items) put(tid + h * kKvThreads, p[h]);
    for (int it = tid + H * kKvThreads; it < items; it += kKvThreads) {
      Pair<W> q;
      Angles<W> g;
      load(it, q, g);
      rotate(q, g, rot, neighbours);
      put(it, q);
    }
  };
  if (!vals) {
    int8_t* dst = c.k + page_at;
    if (grown) {
      for (int i = tid; i < lo * D / 16; i += kKvThreads) {
        uint4* w4 = reinterpret_cast<uint4*>(dst) + i;
        const uint4 w = *w4;
        *w4 = make_uint4(rescale4(w.x, ~0u, f), rescale4(w.y, ~0u, f), rescale4(w.z, ~0u, f),
                         rescale4(w.w, ~0u, f));
      }
    }
    each([&](int it, const Pair<W>& q) {
      int8_t* at = dst + (lo + it / J) * D;
      store_codes<W>(at + q.a, q.x, inv);
      store_codes<W>(at + q.b, q.y, inv);
    });
    return;
  }

  if (grown) {   // earlier codes at the larger scale, whole 16-byte groups
    const int groups = (lo + 15) / 16;
    for (int i = tid; i < D * groups; i += kKvThreads) {
      const int row = i / groups, s = (i - row * groups) * 16;
      uint4 w = *reinterpret_cast<const uint4*>(vdst + row * P + s);
      w.x = rescale4(w.x, below_mask(s, lo), f);
      w.y = rescale4(w.y, below_mask(s + 4, lo), f);
      w.z = rescale4(w.z, below_mask(s + 8, lo), f);
      w.w = rescale4(w.w, below_mask(s + 12, lo), f);
      *reinterpret_cast<uint4*>(tile + row * P + s) = w;
    }
    __syncthreads();
  }
  each([&](int it, const Pair<W>& q) {
    uint8_t* at = tile + lo + it / J;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      at[(q.a + j) * P] = (uint8_t)kv_code(q.x[j], inv);
      at[(q.b + j) * P] = (uint8_t)kv_code(q.y[j], inv);
    }
  });
  __syncthreads();
  const int s0 = grown ? 0 : c0, nc = c1 - s0;
  for (int i = tid; i < D * nc; i += kKvThreads) {
    const int row = i / nc, s = (s0 + i - row * nc) * 16;
    *reinterpret_cast<uint4*>(vdst + row * P + s) = *reinterpret_cast<const uint4*>(tile + row * P + s);
  }
}

template <int W, int H>
const void* append_pick(bool bf16) {
  return bf16 ? (const void*)kv_append_kernel<true, W, H> : (const void*)kv_append_kernel<false, W, H>;
}

}  // namespace

namespace {
int pages_touched(const KvCache& c, const KvBatch& b) { return (b.max_new + c.page - 2) / c.page + 1; }
int64_t page_workgroups(const KvCache& c, const KvBatch& b) {
  return (int64_t)b.seqs * pages_touched(c, b) * c.kv_heads * 2;
}
}  // namespace

// A row of queries a workgroup (four rows a thread's loop, in the first version of this kernel:
// 77 instead of 57 us for 1374 fp32 tokens of 64 + 64 + 64 heads).
int64_t kv_append_grid(const KvCache& c, const KvBatch& b, bool queries) {
  return page_workgroups(c, b) + (queries ? (int64_t)b.seqs * b.max_new : 0);
}

hipError_t launch_kv_append(const KvCache& c, const KvBatch& b, const KvRows& r, bool bf16,
                            hipStream_t s) {
  const int pages_per_seq = pages_touched(c, b);
  const int64_t grid = kv_append_grid(c, b, r.q != nullptr);
  const bool groups = r.rot % 16 == 0;   // whole pairs of groups rotate
  const int pu = (int)page_workgroups(c, b);
  const int rows = b.max_new < c.page ? b.max_new : c.page;   // of one page
  const bool few = rows * (c.head_dim / 16) <= kKvThreads;
  const void* kern = !groups ? append_pick<1, 4>(bf16) : few ? append_pick<8, 1>(bf16) : append_pick<8, 2>(bf16);
  void* args[] = {(void*)&c, (void*)&b, (void*)&r, (void*)&pages_per_seq, (void*)&pu};
  return hipLaunchKernel(kern, dim3((unsigned)grid), dim3(kKvThreads), args,
                         (size_t)c.page * c.head_dim, s);
}

}  // namespace bitnet
