// Attention over the paged 8-bit cache for many query rows: prompts, and parts of
// prompts behind cached tokens.  Definition, and the kernel for few rows:
// attn_decode.hip.
//
// Bound by the vector and matrix instructions together: 8192 tokens of 32 heads on 8, 128
// dims, bf16, take 590-628 us, box to box (875-932 TFLOP/s; a library product of bf16 matrices
// reaches 1208 on this card), with vector instructions in 56% of the cycles and matrix ones
// in 40%.
// Random data draw the clock down: zeros run 17% faster.  Staging a step deeper behind half
// the barriers, raised wave priority around the products, issue-order hints, values read a
// group ahead and the two key tiles' products in turn all measured within 2%.
//
// A workgroup takes 128 columns (256 with eight waves), (row, query head of the group)
// pairs, 32 a wave; the waves share each step of 64 keys in LDS.  The codes are turned into
// fp16 on their way there, exactly (a code's byte becomes the low mantissa bits of 1024 +
// code + 128, one permute and half a packed subtraction a value), once for all columns: the
// int8 products of the decode kernel would need two digits of the weights, 6 more vector
// instructions a pair, at the same matrix rate.
//   * Queries: scaled by a power of two to a largest value in [2^10, 2^11), then fp16
//     (bf16 queries fit exactly); fp32 queries take two fp16 terms (22 bits).
//   * Weights p = 2^(x - m + 7), x = log2 e s + log2 dv (the page's scale joins the
//     exponent), rounded to fp16 (within 2^-11 of each, finer than bf16's 2^-8); for fp32 in
//     and out p = 2^(x - m + 14) in two terms (2^-22).  m follows the largest x of the steps
//     when that lies more than 2^8 apart, so that the accumulators are seldom rescaled and a
//     row whose large weight is met early keeps the small ones that come after it; p stays
//     below 2^15.  Weights that are too small for fp16 beside the largest of their own step
//     are seen by the least of the rounded ones; where the row's sums are so small that it
//     matters, what rounding left of them is added in a second round of the step's products
//     (Weights, below).  With m as the running maximum alone such rows lost what is below
//     2^-32 of the largest weight, and 8192 tokens took 2-4% less.
//   * Sums over keys and the softmax sum are fp32 (the latter of the unrounded p, over
//     each page's dv: of the rounded ones, two a dot instruction, lse lost 2^-12).
// Products: S[key][column] = K Q^T in 32 x 32 tiles, where row r of a tile reads key
// 16 (r / 16) + 8 (r / 4 % 2) + 4 (r / 8 % 2) + r % 4: a lane's 16 results are then keys
// 8 h .. 8 h + 7 and 16 + 8 h .. of its column (h = lane / 32), the operands of
// O[dim][column] = V^T P^T as they stand, so the weights never leave their lane.
// Two LDS buffers, one barrier a step; the next step's codes are loaded while this one's
// are used.
#include "attn_internal.h"

#include <type_traits>

namespace bitnet {
namespace {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int kStep = kAttnStep;

// Byte offset of 16-byte group `at` of a row in LDS (of a key's dims, of a dim's keys).
// A 16-byte access takes 16 lanes at a time, lanes 0-3, 12-15, 20-23, 24-27 and 4-7, 8-11,
// 16-19, 28-31 of each half wave, whose groups have to differ modulo 256 bytes: the
// permutations give each row of such a set another place (conflict cycles at 8192 tokens:
// 33.8 -> 8.6 million of 119 -> 93 million LDS cycles).
template <int DP>
__device__ __forceinline__ int k_group(int key, int at) {
  const int f = DP == 64 ? key >> 1 : key ^ ((key >> 1) & 4);   // two rows of 64 dims fill 256 bytes
  return key * DP * 2 + (((at ^ (at >> 3)) ^ f) & (DP / 8 - 1)) * 16;
}
__device__ __forceinline__ int v_group(int dim, int at) {
  const int f = ((dim >> 1) & 3) | ((dim >> 2) & 4);
  return dim * kStep * 2 + ((at ^ f) & 7) * 16;
}

// Weights of PT fp16 terms: p = 2^(x - m + kLift), at most 2^15, which keep 11 PT bits from
// kHeld on.  m is set anew where a step's largest x lies more than kSlack above or kSink
// below it.
template <int PT>
struct Weights {
  static constexpr float kLift = PT == 1 ? 7.0f : 14.0f, kSlack = 15.0f - kLift, kSink = 8.0f;
  static constexpr float kHeld = PT == 1 ? 0x1p-14f : 0x1p-3f;
  static constexpr float kUp = PT == 1 ? 0x1p29f : 0x1p33f;   // the second round's, over those
};
// A smaller weight lacks at most 2^-25, and a sum over a step's 64 keys, codes up to 127, at
// most 2^-12: less than 2^-24 of the row's largest sum where that is kSums or more.
constexpr float kSums = 0x1p12f;

// Four codes as fp16 pairs.
__device__ __forceinline__ void codes_to_h4(uint32_t w, uint32_t out[2]) {
  const uint32_t u = w ^ 0x80808080u;   // code + 128
  const v2h off = {(_Float16)1152.0f, (_Float16)1152.0f};
  const v2h a = __builtin_bit_cast(v2h, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)) - off;
  const v2h b = __builtin_bit_cast(v2h, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)) - off;
  out[0] = __builtin_bit_cast(uint32_t, a);
  out[1] = __builtin_bit_cast(uint32_t, b);
}

__device__ __forceinline__ uint32_t h2_of(float a, float b) {
  const f32x2_t f = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, v2h));
}
__device__ __forceinline__ void h2_rest(uint32_t h, float& a, float& b) {
  const v2h v = __builtin_bit_cast(v2h, h);
  a -= (float)v[0];
  b -= (float)v[1];
}

__device__ __forceinline__ float halves_max(float v) {
  const uint32_t u = __float_as_uint(v);
  auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __builtin_fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float halves_sum(float v) {
  const uint32_t u = __float_as_uint(v);
  auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}
__device__ __forceinline__ float lane_of(float v, int lane) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}

// A positive finite float, by its bits (this file is compiled without NaN semantics).
__device__ __forceinline__ bool is_scale(float v) {
  return __float_as_uint(v) - 1u < 0x7f7fffffu;
}

// NW: waves (32 columns each).  QT / PT: fp16 terms of a query and of a weight.
template <int DP, int NW, int QT, int PT, bool QB, bool OB>
__global__ __launch_bounds__(64 * NW, DP == 64 ? 3 : DP == 128 ? 2 : 1) void attn_prompt_kernel(
    const KvCache c, const KvBatch b, const AttnArgs a, const AttnPlan plan,
    float* __restrict__ part) {
  constexpr int kThreads = 64 * NW, kCols = 32 * NW;
  constexpr int KC = DP / 16, DT = DP / 32, NL = DP / (16 * NW);   // NL: 16-code loads of K (and V) a thread
  constexpr int kKBytes = kStep * DP * 2, kBuf = 2 * kKBytes;
  extern __shared__ uint4 lds4[];
  uint8_t* lds = reinterpret_cast<uint8_t*>(lds4);
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, col = lane & 31, h = lane >> 5;

  // kv heads run fastest (a head's workgroups then meet in few XCDs' L2), the last
  // rows, which see most keys, start first
  int unit = blockIdx.x;
  const int head = unit % c.kv_heads;
  unit /= c.kv_heads;
  const int split = unit % plan.splits;
  unit /= plan.splits;
  const int seq = unit % b.seqs;
  const int ct = plan.tiles - 1 - unit / b.seqs;
  const int group = plan.group;
  const AttnTile tile = attn_tile(b, seq, ct, kCols, group, a.window);
  if (tile.nc <= 0) return;
  const int each = attn_part(tile.steps, plan.splits, plan.least);
  const int s_lo = split * each, s_hi = min(s_lo + each, tile.steps);
  if (split > 0 && s_lo >= s_hi) return;
  const bool alone = tile.steps <= each;

  const int D = c.head_dim, P = c.page;
  const bool live = wave * 32 + col < tile.nc;
  const int cc = tile.c0 + min(wave * 32 + col, tile.nc - 1);
  const int row = cc / group;
  const int64_t t_row = tile.sp.s0 + row;
  const int q_head = head * group + (cc - row * group);
  const int pos = tile.sp.first + row;
  const int from = a.window > 0 ? max(pos - a.window + 1, 0) : 0;   // visible: from .. pos
  // positions of the wave's first and last columns (its mask-free steps)
  const int pos_lo = __builtin_amdgcn_readlane(pos, 0), pos_hi = __builtin_amdgcn_readlane(pos, 31);
  const int from_hi = __builtin_amdgcn_readlane(from, 31), from_lo = __builtin_amdgcn_readlane(from, 0);

  // queries: dims 16 kc + 8 h .. + 7 of the lane's column
  v8h q[QT][KC];
  float qscale;
  {
    const int64_t base = t_row * a.q_stride + (int64_t)q_head * D;
    auto load8 = [&](int d0, float x[8]) { load_dims<QB, 8>(a.q, base, d0, D, x); };
    float amax = 0.0f;
#pragma unroll
    for (int kc = 0; kc < KC; ++kc) {
      float x[8];
      load8(16 * kc + 8 * h, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(x[j]));
    }
    amax = halves_max(amax);
    // 2^10 over the power of two at or below amax (a row below 2^-107 keeps fewer bits)
    const int e = max((int)(__float_as_uint(amax) >> 23), 20);
    float up = __uint_as_float((uint32_t)(264 - e) << 23);
    qscale = __uint_as_float((uint32_t)(e - 10) << 23) * fabsf(a.scale) * 1.44269504088896340736f;
    if (a.scale < 0.0f) up = -up;   // scales of the products are then never negative
#pragma unroll
    for (int kc = 0; kc < KC; ++kc) {
      float x[8];
      load8(16 * kc + 8 * h, x);
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= up;
#pragma unroll
      for (int n = 0; n < QT; ++n) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          w[j] = h2_of(x[2 * j], x[2 * j + 1]);
          if (n + 1 < QT) h2_rest(w[j], x[2 * j], x[2 * j + 1]);
        }
        const uint4 u = make_uint4(w[0], w[1], w[2], w[3]);
        q[n][kc] = __builtin_bit_cast(v8h, u);
      }
    }
  }

  // Pages of a step's four groups of 16 keys: group lane % 4 in each lane.  An id
  // outside the cache reads page 0; its keys are not seen.
  const int last = max(tile.sp.len - 1, 0);
  const int32_t* table = b.table + (int64_t)seq * b.width;
  auto page_of = [&](int step) -> int {
    return table[min(step * kStep + (lane & 3) * 16, last) >> plan.page_shift];
  };
  auto clamped = [&](int pid) -> uint32_t { return (uint32_t)pid < (uint32_t)c.pages ? pid : 0; };

  // Codes of a step: thread t stages 16 dims of the keys key_of(n), and 16 keys (group
  // t % 4) of dims dim_of(n).  A wave's keys of one n lie in one group.
  const int kc_of = tid % (DP / 16), vq = tid & 3;
  auto key_of = [&](int n) -> int { return (tid + n * kThreads) / (DP / 16); };
  auto dim_of = [&](int n) -> int { return (tid + n * kThreads) >> 2; };
  auto group_of = [&](int n) -> int { return (wave * 64 + n * kThreads) / (DP / 16) / 16; };
  const uint32_t page_bytes = (uint32_t)c.kv_heads * P * D;   // below 2^31
  const int8_t *k_head = c.k + (int64_t)head * P * D, *v_head = c.v + (int64_t)head * P * D;
  // offsets in a page, for its first 64 slots (a page of 128 adds those of the step)
  uint32_t koff[NL], voff[NL];
#pragma unroll
  for (int n = 0; n < NL; ++n) {
    // dims past the head read dim 0: their queries are 0
    koff[n] = (key_of(n) & (P - 1)) * D + (kc_of * 16 < D ? kc_of * 16 : 0);
    voff[n] = min(dim_of(n), D - 1) * P + ((vq * 16) & (P - 1));
  }
  uint4 kr[NL], vr[NL];
  auto load = [&](int step, int pid) {
    const int at = (step * kStep) & (P - 1);
    const uint32_t page = clamped(pid);
#pragma unroll
    for (int n = 0; n < NL; ++n) {
      const uint32_t pk = __builtin_amdgcn_readlane(page, group_of(n));
      kr[n] = *reinterpret_cast<const uint4*>(k_head + ((uint64_t)pk * page_bytes + at * D) + koff[n]);
    }
    const int8_t* vp = v_head + ((uint64_t)page * page_bytes + at);
#pragma unroll
    for (int n = 0; n < NL; ++n) vr[n] = *reinterpret_cast<const uint4*>(vp + voff[n]);
  };
  auto stage = [&](uint8_t* buf) {
#pragma unroll
    for (int n = 0; n < NL; ++n) {
      const uint32_t kw[4] = {kr[n].x, kr[n].y, kr[n].z, kr[n].w};
      const uint32_t vw[4] = {vr[n].x, vr[n].y, vr[n].z, vr[n].w};
      uint32_t x[8], y[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        codes_to_h4(kw[j], x + 2 * j);
        codes_to_h4(vw[j], y + 2 * j);
      }
      const int key = key_of(n), dim = dim_of(n);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        *reinterpret_cast<uint4*>(buf + k_group<DP>(key, 2 * kc_of + j)) =
            make_uint4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
        *reinterpret_cast<uint4*>(buf + kKBytes + v_group(dim, 2 * vq + j)) =
            make_uint4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
      }
    }
  };

  // scales of a step's groups: loaded a step ahead, looked at when they are used
  int g0, g1, g2;   // pages of this step, the next, the one after
  float dk, dv;
  auto scales = [&](int pid) {
    const uint64_t at = (uint64_t)clamped(pid) * (uint32_t)c.kv_heads + head;
    dk = c.k_scale[at];
    dv = c.v_scale[at];
  };

  const int first = tile.step0 + s_lo, end = tile.step0 + s_hi;
  using Wt = Weights<PT>;
  float m = -INFINITY, l = 0.0f;   // l, o: over 2^(m - kLift)
  float most = -INFINITY;          // the largest x so far
  v16f o[DT];
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
#pragma unroll
    for (int j = 0; j < 16; ++j) o[dt][j] = 0.0f;

  // row of a 32-key tile that the lane's operand reads
  const int krow = 16 * (col >> 4) + 8 * ((col >> 2) & 1) + 4 * ((col >> 3) & 1) + (col & 3);

  // logits of a step's 32-key tile kt, over qscale and their keys' scales.  slow: with few
  // values in flight (off the loop's common path, whose registers count)
  auto logits = [&](const uint8_t* buf, int kt, v16f& t, bool slow = false) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 16; ++j) t[j] = 0.0f;
    const int key = kt * 32 + krow;
#pragma unroll
    for (int kc = 0; kc < KC; ++kc) {
      const v8h kk = *reinterpret_cast<const v8h*>(buf + k_group<DP>(key, 2 * kc + h));
#pragma unroll
      for (int n = 0; n < QT; ++n)
        t = __builtin_amdgcn_mfma_f32_32x32x16_f16(kk, q[n][kc], t, 0, 0, 0);
      if (slow) __builtin_amdgcn_sched_barrier(0);
    }
  };
  // fp16 terms of weights; see(w): pairs of the first ones
  auto terms = [&](float p[8], v8h pf[PT], auto see) __attribute__((always_inline)) {
#pragma unroll
    for (int n = 0; n < PT; ++n) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = h2_of(p[2 * j], p[2 * j + 1]);
        if (n == 0) see(w[j]);
        if (n + 1 < PT) h2_rest(w[j], p[2 * j], p[2 * j + 1]);
      }
      const uint4 u = make_uint4(w[0], w[1], w[2], w[3]);
      pf[n] = __builtin_bit_cast(v8h, u);
    }
  };
  // the terms of a step's group g join the sums
  auto join = [&](const uint8_t* buf, int g, const v8h pf[PT], bool slow = false) __attribute__((always_inline)) {
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) {
      const int dim = 32 * dt + col;
      const v8h vv = *reinterpret_cast<const v8h*>(buf + kKBytes + v_group(dim, 2 * g + h));
#pragma unroll
      for (int n = 0; n < PT; ++n)
        o[dt] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vv, pf[n], o[dt], 0, 0, 0);
      if (slow) __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto times = [&](float f) __attribute__((always_inline)) {
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int j = 0; j < 16; ++j) o[dt][j] *= f;
  };

  // One step from buffer B.  Loads run ahead without a test for the end: past it they
  // read the sequence's last page again.
  auto body = [&](auto B, int step) {   // B: 0 or 1, a constant where the loop is unrolled
    const uint8_t* buf = lds + B * kBuf;
    // no page: scale -1; a scale that no visible key can have (another page's memory): 1
    const float dk_now = (uint32_t)g0 < (uint32_t)c.pages ? dk : -1.0f;
    const float dv_now = is_scale(dv) ? dv : 1.0f;
    scales(g1);
    g0 = g1;
    g1 = g2;
    const int key0 = step * kStep;
    // some column of the wave sees some key of this step
    const bool any = key0 <= pos_hi && key0 + kStep - 1 >= from_lo;
    v16f s[2];
    logits(buf, 0, s[0]);
    logits(buf, 1, s[1]);
    stage(lds + (1 - B) * kBuf);
    g2 = page_of(step + 3);   // before the codes: the next step waits for it, not for them
    load(step + 2, g1);
    if (any) {
      const float lv = __builtin_amdgcn_logf(dv_now), rdv = __builtin_amdgcn_rcpf(dv_now);
      float ck[4], lg[4], rg[4];
      bool there[4], hole = false;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float k = lane_of(dk_now, g);
        there[g] = (int)__float_as_uint(k) >= 0;   // by its sign bit
        hole = hole || !there[g];
        ck[g] = fmaxf(qscale * k, 1e-38f);   // above 0: unseen keys' -inf stays -inf
        lg[g] = lane_of(lv, g);
        rg[g] = lane_of(rdv, g);
      }
      // group g holds s[g / 2][8 (g % 2) + j], j = 0 .. 7: key 16 g + 8 h + j
      const bool whole = !hole && key0 + kStep - 1 <= pos_lo && key0 >= from_hi;
      if (!whole) {
        const int hi = pos - key0 - 8 * h, lo = from - key0 - 8 * h;
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float x = s[g >> 1][8 * (g & 1) + j];
            s[g >> 1][8 * (g & 1) + j] =
                (there[g] & (16 * g + j <= hi) & (16 * g + j >= lo)) ? x : -INFINITY;
          }
      }
      float mx = -INFINITY;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float t = s[g >> 1][8 * (g & 1)];
#pragma unroll
        for (int j = 1; j < 8; ++j) t = __builtin_fmaxf(t, s[g >> 1][8 * (g & 1) + j]);
        mx = __builtin_fmaxf(mx, __builtin_fmaf(t, ck[g], lg[g]));
      }
      mx = halves_max(mx);
      most = __builtin_fmaxf(most, mx);
      const float to = mx == -INFINITY ? m : __builtin_fmaxf(mx, most - kReach);
      if (__builtin_amdgcn_ballot_w64((to > m + Wt::kSlack) | (to < m - Wt::kSink))) {
        const float alpha = to == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - to);
        m = to;
        l *= alpha;
        times(alpha);
      }
      const float ref = m == -INFINITY ? 0.0f : m - Wt::kLift;
      v2h least = {(_Float16)65504.0f, (_Float16)65504.0f};   // of the weights
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float p[8], sum = 0.0f;
        const float off = lg[g] - ref;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          p[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[g >> 1][8 * (g & 1) + j], ck[g], off));
          sum += p[j];
        }
        l = __builtin_fmaf(sum, rg[g], l);
        v8h pf[PT];
        terms(p, pf, [&](uint32_t w) {
          least = __builtin_elementwise_minimum(least, __builtin_bit_cast(v2h, w));
        });
        join(buf, g, pf);
      }
      // Weights below kHeld (or unseen, where the step is not whole): whether it matters what
      // they lack
      bool small = !whole | (least[0] < (_Float16)Wt::kHeld) | (least[1] < (_Float16)Wt::kHeld);
      if (__builtin_expect(__builtin_amdgcn_ballot_w64(small) != 0, 0)) {
        float large = 0.0f;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
#pragma unroll
          for (int j = 0; j < 16; ++j) large = __builtin_fmaxf(large, __builtin_fabsf(o[dt][j]));
        small = (halves_max(large) < kSums) & (l > 0.0f);
      }
      // The second round: what is lacking, over a reference kUp lower.  It is held to 11 PT
      // bits or 2^-25 / kUp, as weights down to 2^-kReach of the row's largest (2^(kLift - 48)
      // and more) need.  (The tiles in a loop, so that registers spill inside it if they have
      // to; for bf16 heads of 128 dims they suffice unrolled.)
      if (__builtin_expect(__builtin_amdgcn_ballot_w64(small) != 0, 0)) {
        times(Wt::kUp);
#pragma unroll(QT == 1 && DP == 128 ? 2 : 1)
        for (int kt = 0; kt < 2; ++kt) {
          const int hi = pos - key0 - 8 * h - 32 * kt, lo = from - key0 - 8 * h - 32 * kt;
          v16f t;
          logits(buf, kt, t, true);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const float k = lane_of(dk_now, 2 * kt + g), c1 = fmaxf(qscale * k, 1e-38f);
            const float c0 = lane_of(lv, 2 * kt + g) - ref;
            const bool on = (int)__float_as_uint(k) >= 0;
            float p[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(t[8 * g + j], c1, c0));
              p[j] = (on & (16 * g + j <= hi) & (16 * g + j >= lo) & (x < Wt::kHeld)) ? x : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int n = 0; n < PT; ++n) h2_rest(h2_of(p[2 * j], p[2 * j + 1]), p[2 * j], p[2 * j + 1]);
#pragma unroll
            for (int j = 0; j < 8; ++j) p[j] *= Wt::kUp;
            v8h pf[PT];
            terms(p, pf, [](uint32_t) {});
            join(buf, 2 * kt + g, pf, true);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
        times(1.0f / Wt::kUp);
      }
    }
    lds_barrier();
  };

  if (first < end) {
    g0 = page_of(first);
    g1 = page_of(first + 1);
    g2 = page_of(first + 2);
    load(first, g0);
    scales(g0);
    stage(lds);
    load(first + 1, g1);
    lds_barrier();
    if (wave * 32 >= tile.nc) {   // no columns: the wave only stages (a sequence of few rows)
      for (int step = first; step < end; ++step) {
        g1 = g2;
        stage(lds + (1 - ((step - first) & 1)) * kBuf);
        g2 = page_of(step + 3);
        load(step + 2, g1);
        lds_barrier();
      }
    } else if constexpr (DP <= 128 && QT == 1) {   // the buffers' offsets in the instructions
      for (int step = first;;) {
        body(std::integral_constant<int, 0>{}, step);
        if (++step >= end) break;
        body(std::integral_constant<int, 1>{}, step);
        if (++step >= end) break;
      }
    } else {   // (the registers do not suffice for that)
      for (int step = first; step < end; ++step) body((step - first) & 1, step);
    }
  }

  l = halves_sum(l);
  if (!live) return;
  // sums over 2^top, near the largest weight
  const float top = most - Wt::kLift, back = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - most);
  l *= back;
  if (!alone) {
    float* p = part + (((int64_t)(seq * c.kv_heads + head) * plan.tiles + ct) * plan.splits + split) *
                          plan.part_cols * (D + 4) +
               (int64_t)(wave * 32 + col) * (D + 4);
    if (h == 0) *reinterpret_cast<float2*>(p) = make_float2(top, l);
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int d = 32 * dt + 8 * w + 4 * h;
        if (d < D)
          *reinterpret_cast<float4*>(p + 4 + d) =
              make_float4(o[dt][4 * w] * back, o[dt][4 * w + 1] * back, o[dt][4 * w + 2] * back,
                          o[dt][4 * w + 3] * back);
      }
    return;
  }
  const float r = l > 0.0f ? back / l : 0.0f;
  const int64_t at = (t_row * a.q_heads + q_head) * D;
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int d = 32 * dt + 8 * w + 4 * h;
      if (d >= D) continue;
      const float y0 = o[dt][4 * w] * r, y1 = o[dt][4 * w + 1] * r, y2 = o[dt][4 * w + 2] * r,
                  y3 = o[dt][4 * w + 3] * r;
      if (OB)
        *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + at + d) =
            make_uint2(bf16x2_rne(y0, y1), bf16x2_rne(y2, y3));
      else
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + at + d) = make_float4(y0, y1, y2, y3);
    }
  if (h == 0 && a.lse)
    a.lse[t_row * a.q_heads + q_head] =
        l > 0.0f ? 0.69314718055994530942f * (top + __builtin_amdgcn_logf(l)) : -INFINITY;
}

template <int DP>
const void* pick_prompt(bool qb, bool ob) {
  return qb ? (ob ? (const void*)attn_prompt_kernel<DP, 4, 1, 1, true, true>
                  : (const void*)attn_prompt_kernel<DP, 4, 1, 1, true, false>)
            : (ob ? (const void*)attn_prompt_kernel<DP, 4, 2, 1, false, true>
                  : (const void*)attn_prompt_kernel<DP, 4, 2, 2, false, false>);
}

constexpr int kTileCols = 128, kWideCols = 256;

int64_t tiles_of(const KvCache& c, const KvBatch& b, int q_heads, int cols) {
  const int64_t all = (int64_t)b.max_new * (q_heads / c.kv_heads);
  return (int64_t)b.seqs * c.kv_heads * ((all + cols - 1) / cols);
}

}  // namespace

AttnPlan attn_prompt_plan(const KvCache& c, const KvBatch& b, int q_heads) {
  return attn_plan(c, b, q_heads, kTileCols, 512, 8);
}

hipError_t launch_attn_prompt(const KvCache& c, const KvBatch& b, const AttnArgs& a,
                              const AttnPlan& plan, bool q_bf16, bool out_bf16, void* workspace,
                              hipStream_t s) {
  AttnPlan p = plan;
  float* part = static_cast<float*>(workspace);
  const int dp = c.head_dim <= 64 ? 64 : c.head_dim <= 128 ? 128 : 256;
  // Eight waves share a step's conversion between 256 columns: bf16 queries of 65 to 128
  // dims with a workgroup for every compute unit (8192 tokens of 32 heads: 627 -> 599 us).
  // Fewer take four waves, whose workgroups are twice as many (and split the keys).
  const bool wide = dp == 128 && q_bf16 && tiles_of(c, b, a.q_heads, kWideCols) >= 256;
  if (wide) {
    p = attn_plan(c, b, a.q_heads, kWideCols, 1, 8);
    p.splits = 1;
  }
  const int64_t grid = (int64_t)b.seqs * c.kv_heads * p.tiles * p.splits;
  const void* kern = wide ? (out_bf16 ? (const void*)attn_prompt_kernel<128, 8, 1, 1, true, true>
                                      : (const void*)attn_prompt_kernel<128, 8, 1, 1, true, false>)
                     : dp == 64 ? pick_prompt<64>(q_bf16, out_bf16)
                     : dp == 128 ? pick_prompt<128>(q_bf16, out_bf16) : pick_prompt<256>(q_bf16, out_bf16);
  const size_t lds = (size_t)2 * 2 * kStep * dp * 2;   // two buffers of K and V in fp16
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  void* args[] = {(void*)&c, (void*)&b, (void*)&a, (void*)&p, (void*)&part};
  const hipError_t e = hipLaunchKernel(kern, dim3((unsigned)grid), dim3(p.cols * 2), args, lds, s);
  if (e != hipSuccess || p.splits == 1) return e;
  return launch_attn_join(c, b, a, p, out_bf16, part, s);
}

}  // namespace bitnet
