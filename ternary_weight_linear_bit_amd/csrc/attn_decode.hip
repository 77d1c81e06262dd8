// Attention over the paged 8-bit cache for few query rows: single tokens, drafted
// tokens (long ones: attn_prompt.hip).
//
// Query row i of a sequence with n new rows and len cached tokens has position
// pos = len - n + i and sees the keys j with max(0, pos - window + 1) <= j <= pos
// (window 0: from 0).  With codes kc, vc and the page's scales dk, dv:
//   s_j = scale dk (q . kc_j),  out = sum_j e^(s_j - m) dv vc_j / sum_j e^(s_j - m),
//   lse = m + ln sum_j e^(s_j - m).
// A row without keys gives zeros and lse = -inf; a page id outside the cache holds
// no keys.
//
// Bound by memory: every visible code is read once (64 sequences of 1 .. 8191 tokens, 32
// heads on 8, 128 dims: 137 us, 4.3 TB/s; four of 65536, fp32: 108 us, 4.8 TB/s; a large
// copy reaches 4.75).  Small calls are bound by one step's latency and two launches (one
// sequence of 2049 tokens: 11.8 us).  Non-temporal loads were 7-10% slower.  The codes go from
// memory to the int8 matrix cores as they are, with no conversion and no LDS: it is the other
// operand that is turned into 8-bit digits, a query row (once) and the weights of a step (16 a
// lane), each digit with its own product; the int32 sums are exact.
//   * Queries x with |x| <= X: v = rne(x V / X), V = 127 * 256^2, in three signed base-256
//     digits (2^-24 of their row's largest value; with two the logits of bf16 queries were
//     2^-16 off, and lse, an fp32 output, with them).
//   * Weights: 2^14 of them is the power of two above the step's largest, and a pass takes two
//     digits of what the passes before left, 15 more bits each, until every weight of the
//     wave's step is within 2^-11 of itself (2^-22 with fp32 in and out) or below 2^-48 of the
//     row's largest.  Two passes are common (three in fp32).  A fixed point against the row's
//     largest weight, in one pass, ran 64 sequences in 131 us, and 256 rows behind 3840 tokens
//     (16 columns a workgroup, bound by vector instructions) in 53 instead of 62, and lost what
//     is 2^-16 of it: of a row whose first key has 95% of the weight, and no value, a third of
//     the output.
// Converting the codes to 16-bit floats instead would take 320 vector instructions
// a lane and step of 64 keys, the digits of a pass take about 50.
//
// The page's scale dv joins the exponent: x_j = log2 e s_j + log2 dv, weights
// 2^(x_j - max x), so that the weights' fixed-point range fits the largest product
// whatever the pages' scales are; the softmax sum takes each weight over its dv.
//
// A wave takes 64 keys a step.  Products: S[key][row] = K Q^T from 16-key tiles,
// where row r of tile t reads key 16 (r / 4) + 4 t + r % 4, so that the lane with
// row column c and quarter g (lanes 16 g ..) ends up with the 16 consecutive keys
// 16 g .. 16 g + 15: exactly the operand of O[dim][row] = V^T P^T, whose other side
// is 16 consecutive bytes of the cache's value rows.  Weights never leave their lane.
// Columns are (row, query head of the group) pairs, 16 a workgroup.  The NW waves of a
// workgroup take every NW-th step and are joined in LDS; the keys of a sequence are
// split over workgroups (attn_part) and joined by a second kernel.
#include "attn_internal.h"

#include <type_traits>

namespace bitnet {
namespace {

constexpr int kWaves = 4, kManyWaves = 8, kStep = kAttnStep, kCols = 16;
constexpr int kQd = 3;                 // digits of a query
constexpr float kQTop = 8323072.0f;    // 127 * 256^2: a query row's largest value
constexpr float kLift = 14.0f;         // weights of a step: at most 2^14, two digits
constexpr float kPass = 0x1p-15f;      // unit of a pass over that of the pass before
constexpr float kRound = kRneMagic + 128.0f;

// Byte K of four dwords, a first.
template <int K>
__device__ __forceinline__ uint32_t bytes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  constexpr uint32_t sel = 0x0c0c0000u | ((4u + K) << 8) | K;
  const uint32_t lo = __builtin_amdgcn_perm(b, a, sel);
  const uint32_t hi = __builtin_amdgcn_perm(d, c, sel);
  return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
}

// Three digits (most significant first) of four values x >= -1, <= 1 times kQTop.  With
// u = v + 0x8080 byte j of u is digit j, its top bit flipped for all but the highest.
__device__ __forceinline__ void query_digits(const float x[4], uint32_t out[kQd]) {
  uint32_t u[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) u[j] = (uint32_t)((int)rintf(__fmul_rn(x[j], kQTop)) + 0x8080);
  out[2] = bytes4<0>(u[0], u[1], u[2], u[3]) ^ 0x80808080u;
  out[1] = bytes4<1>(u[0], u[1], u[2], u[3]) ^ 0x80808080u;
  out[0] = bytes4<2>(u[0], u[1], u[2], u[3]);
}
// Two digits of four values |y| <= 2^14 `unit` in units: adding kRound units rounds to
// nearest even and leaves the integer, and 0x80, in the float's low bits (see rne_bits).
__device__ __forceinline__ void weight_digits(const float y[4], float unit, uint32_t out[2]) {
  uint32_t u[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) u[j] = __float_as_uint(__fadd_rn(y[j], kRound * unit));
  out[1] = bytes4<0>(u[0], u[1], u[2], u[3]) ^ 0x80808080u;
  out[0] = bytes4<1>(u[0], u[1], u[2], u[3]);
}
// What that rounding leaves of a value, at most half a unit: both differences are exact.
__device__ __forceinline__ float weight_rest(float y, float unit) {
  return __fsub_rn(y, __fsub_rn(__fadd_rn(y, kRound * unit), kRound * unit));
}
// 2^n of a whole n <= 126, exactly; 0 far below.  (A larger n only meets sums of 0.)
__device__ __forceinline__ float power_of_2(float n) {
  return __builtin_amdgcn_ldexpf(1.0f, (int)fminf(fmaxf(n, -200.0f), 126.0f));
}

// The number that a product's int32 digit sums stand for.
__device__ __forceinline__ float joined(const int d[kQd]) {
  const float t = (float)(d[0] * 256 + d[1]);   // |digit sum| < 2^22: exact in int32
  return __builtin_fmaf(t, 256.0f, (float)d[2]);
}

// max / sum over the four 16-lane rows of the wave (lanes with equal lane % 16)
__device__ __forceinline__ float rows_max(float v) {
  const uint32_t u = __float_as_uint(v);
  auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const float w = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(w), __float_as_uint(w), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float rows_sum(float v) {
  const uint32_t u = __float_as_uint(v);
  auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const float w = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(w), __float_as_uint(w), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// NW: waves.  B: bits that each weight keeps.
template <int DP, int NW, int B, bool QB, bool OB>
__global__ __launch_bounds__(64 * NW, DP <= 128 ? 2 : 1) void attn_decode_kernel(
    const KvCache c, const KvBatch b, const AttnArgs a, const AttnPlan plan,
    float* __restrict__ part) {
  constexpr int kThreads = 64 * NW;
  constexpr int KC = DP / 64, DT = DP / 16, HT = DT < 32 / NW ? DT : 32 / NW;   // 16 HT dims joined at a time
  __shared__ float sm[NW][kCols], sl[NW][kCols];
  __shared__ float so[NW][kCols][16 * HT + 4];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, col = lane & 15, g = lane >> 4;
  int unit = blockIdx.x;
  const int split = unit % plan.splits;
  unit /= plan.splits;
  const int ct = unit % plan.tiles;
  const int head = unit / plan.tiles % c.kv_heads;
  const int seq = unit / plan.tiles / c.kv_heads;
  const int group = plan.group;
  const AttnTile tile = attn_tile(b, seq, ct, kCols, group, a.window);
  if (tile.nc <= 0) return;
  const int each = attn_part(tile.steps, plan.splits, plan.least);
  const int s_lo = split * each, s_hi = min(s_lo + each, tile.steps);
  if (split > 0 && s_lo >= s_hi) return;
  const bool alone = tile.steps <= each;   // the only part of this tile

  const int D = c.head_dim, P = c.page;
  const int cc = tile.c0 + min(col, tile.nc - 1);
  const int row = cc / group;
  const int64_t t_row = tile.sp.s0 + row;
  const int q_head = head * group + (cc - row * group);
  const int pos = tile.sp.first + row;
  const int from = a.window > 0 ? max(pos - a.window + 1, 0) : 0;   // visible: from .. pos

  // queries: digits of dims 64 kc + 16 g .. + 15 of the lane's column
  v4i qd[kQd][KC];
  float qscale;
  {
    float q[KC][16];
    float amax = 0.0f;
    const int64_t base = t_row * a.q_stride + (int64_t)q_head * D;
#pragma unroll
    for (int kc = 0; kc < KC; ++kc) {
      const int d0 = kc * 64 + g * 16;
      load_dims<QB, 16>(a.q, base, d0, D, q[kc]);
#pragma unroll
      for (int j = 0; j < 16; ++j) amax = fmaxf(amax, fabsf(q[kc][j]));
    }
    amax = rows_max(amax);
    const float up = amax < 0x1p-64f ? 0x1p64f : 1.0f;   // keeps 1 / amax finite
    const float inv = amax > 0.0f ? 1.0f / (amax * up) : 0.0f;
    qscale = amax / kQTop * a.scale * 1.44269504088896340736f;
#pragma unroll
    for (int kc = 0; kc < KC; ++kc)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = __fmul_rn(__fmul_rn(q[kc][4 * w + j], up), inv);
        uint32_t d[kQd];
        query_digits(x, d);
#pragma unroll
        for (int n = 0; n < kQd; ++n) qd[n][kc][w] = (int)d[n];
      }
  }

  // page ids of the groups of 16 keys that the lane reads: keys of group col / 4,
  // values of group g
  const int last = max(tile.sp.len - 1, 0);
  const int32_t* table = b.table + (int64_t)seq * b.width;
  auto page_of = [&](int step, int quarter) -> int {
    const int j = min(step * kStep + quarter * 16, last);
    return table[j >> plan.page_shift];
  };
  int64_t koff[KC];   // clamped: dims past the head read dim 0 (their query digits are 0)
#pragma unroll
  for (int kc = 0; kc < KC; ++kc) koff[kc] = kc * 64 + g * 16 < D ? kc * 64 + g * 16 : 0;
  v4i kr[4][KC], vr[DT];
  auto load_k = [&](int step, int pid) {
    const int64_t p = (uint32_t)pid < (uint32_t)c.pages ? pid : 0;
    const int slot = (step * kStep + (col >> 2) * 16) & (P - 1);
    const int8_t* at = c.k + ((p * c.kv_heads + head) * P + slot + (col & 3)) * D;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int kc = 0; kc < KC; ++kc)
        kr[t][kc] = *reinterpret_cast<const v4i*>(at + 4 * t * D + koff[kc]);
  };
  auto load_v = [&](int step, int pid) {
    const int64_t p = (uint32_t)pid < (uint32_t)c.pages ? pid : 0;
    const int slot = (step * kStep + g * 16) & (P - 1);
    const int8_t* at = c.v + (p * c.kv_heads + head) * P * D + slot;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
      vr[dt] = *reinterpret_cast<const v4i*>(at + min(16 * dt + col, D - 1) * P);
  };

  // m: the largest x so far.  l, o: over 2^r, a whole number.
  float m = -INFINITY, r = 0.0f, l = 0.0f;
  float o[DT][4];
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[dt][i] = 0.0f;

  const int s_begin = tile.step0 + s_lo + wave, s_end = tile.step0 + s_hi;
  // pages of this step, of the next and of the one after: an id is loaded ahead of the
  // codes of the step before its own, so that no wait for it waits for them
  int pid_v = 0, pid_k1 = 0, pid_v1 = 0, pid_k2 = 0, pid_v2 = 0;
  float dk = 0.0f, dv = 1.0f;
  auto scales = [&](int pid) {
    const int64_t at = (int64_t)((uint32_t)pid < (uint32_t)c.pages ? pid : 0) * c.kv_heads + head;
    dk = c.k_scale[at];
    dv = c.v_scale[at];
  };
  if (s_begin < s_end) {
    const int pk = page_of(s_begin, col >> 2);
    pid_v = page_of(s_begin, g);
    pid_k1 = page_of(s_begin + NW, col >> 2);
    pid_v1 = page_of(s_begin + NW, g);
    load_k(s_begin, pk);
    scales(pid_v);
    load_v(s_begin, pid_v);
  }
  for (int step = s_begin; step < s_end; step += NW) {
    const bool more = step + NW < s_end;
    float x[4][4];   // the products first, as numbers
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      v4i s[kQd];
#pragma unroll
      for (int n = 0; n < kQd; ++n) {
        s[n] = (v4i){0, 0, 0, 0};
#pragma unroll
        for (int kc = 0; kc < KC; ++kc)
          s[n] = __builtin_amdgcn_mfma_i32_16x16x64_i8(kr[t][kc], qd[n][kc], s[n], 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        int d[kQd];
#pragma unroll
        for (int n = 0; n < kQd; ++n) d[n] = s[n][i];
        x[t][i] = joined(d);
      }
    }
    pid_k2 = page_of(step + 2 * NW, col >> 2);
    pid_v2 = page_of(step + 2 * NW, g);
    if (more) load_k(step + NW, pid_k1);

    // x = log2 e s + log2 dv of the lane's 16 keys; -inf where the row sees none
    const int j0 = step * kStep + g * 16;
    const bool there = (uint32_t)pid_v < (uint32_t)c.pages;
    const float rdv = there && j0 <= pos && j0 + 15 >= from ? 1.0f / dv : 0.0f;
    const float ck = qscale * dk, lv = __builtin_amdgcn_logf(dv);   // log2
    const int hi = there ? pos - j0 : -1, lo = from - j0;   // visible: lo <= key <= hi
    float mx = -INFINITY;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float y = __builtin_fmaf(x[t][i], ck, lv);
        x[t][i] = 4 * t + i <= hi && 4 * t + i >= lo ? y : -INFINITY;
        mx = fmaxf(mx, x[t][i]);
      }
    mx = rows_max(mx);
    m = fmaxf(m, mx);
    const float rest = ceilf(m) - (kReach + 1.0f);   // weights below 2^rest may be lost
    const float to = mx == -INFINITY ? r : fmaxf(ceilf(mx), rest) - kLift;
    const float alpha = power_of_2(r - to), floor = fmaxf(power_of_2(rest - to), 0x1p-126f);
    r = to;
    float sum = 0.0f;
    uint32_t low = 0x7f800000u;   // the least weight from `floor` on, less that: by its bits,
                                 // as those of negative numbers are larger
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = __builtin_amdgcn_exp2f(x[t][i] - r);
        x[t][i] = p;
        sum += p;
        low = min(low, __float_as_uint(p - floor));
      }
    l = __builtin_fmaf(l, alpha, sum * rdv);
    if (more) scales(pid_v1);

    // Two digits of every weight; then, as long as some weight of the wave is not held to
    // B bits (it is off by at most half of `unit`), two digits of what they left.
    float unit = 1.0f;
    auto pass = [&](auto first) {
      v4i pd[2];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        uint32_t d[2];
        if (!first.value)
#pragma unroll
          for (int i = 0; i < 4; ++i) x[t][i] = weight_rest(x[t][i], unit * (1.0f / kPass));
        weight_digits(x[t], unit, d);
        pd[0][t] = (int)d[0];
        pd[1][t] = (int)d[1];
      }
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) {
        v4i y[2];
#pragma unroll
        for (int n = 0; n < 2; ++n)
          y[n] = __builtin_amdgcn_mfma_i32_16x16x64_i8(vr[dt], pd[n], (v4i){0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float s = (float)(y[0][i] * 256 + y[1][i]);   // |digit sum| < 2^21: exact in int32
          o[dt][i] = first.value ? __builtin_fmaf(o[dt][i], alpha, s) : __builtin_fmaf(s, unit, o[dt][i]);
        }
      }
    };
    pass(std::true_type{});
    const float least = __uint_as_float(low) + floor;   // at least 2^-35 of the reference
    while (__builtin_amdgcn_ballot_w64(least < unit * (1 << (B - 1)))) {
      unit *= kPass;
      pass(std::false_type{});
    }
    if (more) {
      load_v(step + NW, pid_v1);
      pid_v = pid_v1;
      pid_k1 = pid_k2;
      pid_v1 = pid_v2;
    }
  }

  // join the waves: each scales its sums to the common maximum
  m = ceilf(m);
  const float back = m == -INFINITY ? 0.0f : power_of_2(r - m);   // to sums over 2^m
  l = rows_sum(l) * back;
  if (g == 0) {
    sm[wave][col] = m;
    sl[wave][col] = l;
  }
  __syncthreads();
  float top = sm[0][col], total = 0.0f;
#pragma unroll
  for (int w = 1; w < NW; ++w) top = fmaxf(top, sm[w][col]);
#pragma unroll
  for (int w = 0; w < NW; ++w)
    total += sm[w][col] == -INFINITY ? 0.0f : sl[w][col] * __builtin_amdgcn_exp2f(sm[w][col] - top);
  const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - top) * back;
  const int64_t pu = (int64_t)blockIdx.x * plan.part_cols;
#pragma unroll
  for (int h0 = 0; h0 < DT; h0 += HT) {
    if (h0 > 0) __syncthreads();
    if (col < tile.nc)
#pragma unroll
      for (int dt = 0; dt < HT; ++dt)
        *reinterpret_cast<float4*>(&so[wave][col][16 * dt + 4 * g]) =
            make_float4(o[h0 + dt][0] * f, o[h0 + dt][1] * f, o[h0 + dt][2] * f, o[h0 + dt][3] * f);
    __syncthreads();
    // 4 dims a thread
    const int nd = min(16 * HT, D - 16 * h0);
    for (int e = tid; e < tile.nc * (nd / 4); e += kThreads) {
      const int ec = e / (nd / 4), d = (e - ec * (nd / 4)) * 4;
      float4 y = *reinterpret_cast<const float4*>(&so[0][ec][d]);
#pragma unroll
      for (int w = 1; w < NW; ++w) {
        const float4 z = *reinterpret_cast<const float4*>(&so[w][ec][d]);
        y.x += z.x;
        y.y += z.y;
        y.z += z.z;
        y.w += z.w;
      }
      if (alone) {
        float et = sm[0][ec], el = 0.0f;
#pragma unroll
        for (int w = 1; w < NW; ++w) et = fmaxf(et, sm[w][ec]);
#pragma unroll
        for (int w = 0; w < NW; ++w)
          el += sm[w][ec] == -INFINITY ? 0.0f : sl[w][ec] * __builtin_amdgcn_exp2f(sm[w][ec] - et);
        const float rl = el > 0.0f ? 1.0f / el : 0.0f;
        const int oc = tile.c0 + ec, orow = oc / group;
        const int64_t at = ((tile.sp.s0 + orow) * a.q_heads + head * group + (oc - orow * group)) * D +
                           16 * h0 + d;
        if (OB)
          *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + at) =
              make_uint2(bf16x2_rne(y.x * rl, y.y * rl), bf16x2_rne(y.z * rl, y.w * rl));
        else
          *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + at) =
              make_float4(y.x * rl, y.y * rl, y.z * rl, y.w * rl);
      } else {
        *reinterpret_cast<float4*>(part + (pu + ec) * (D + 4) + 4 + 16 * h0 + d) = y;
      }
    }
  }
  if (wave == 0 && g == 0 && col < tile.nc) {
    if (!alone)
      *reinterpret_cast<float2*>(part + (pu + col) * (D + 4)) = make_float2(top, total);
    else if (a.lse)
      a.lse[t_row * a.q_heads + q_head] =
          total > 0.0f ? 0.69314718055994530942f * (top + __builtin_amdgcn_logf(total)) : -INFINITY;
  }
}

template <int DP, int NW>
const void* pick_decode(bool qb, bool ob) {
  return qb ? (ob ? (const void*)attn_decode_kernel<DP, NW, 11, true, true>
                  : (const void*)attn_decode_kernel<DP, NW, 11, true, false>)
            : (ob ? (const void*)attn_decode_kernel<DP, NW, 11, false, true>
                  : (const void*)attn_decode_kernel<DP, NW, 22, false, false>);
}
template <int NW>
const void* pick_decode(int dim, bool qb, bool ob) {
  if constexpr (NW == kWaves)
    if (dim > 128) return pick_decode<256, NW>(qb, ob);
  return dim <= 64 ? pick_decode<64, NW>(qb, ob) : pick_decode<128, NW>(qb, ob);
}

constexpr int64_t kOneLaunch = kManyWaves;   // steps up to which no keys are split

}  // namespace

// Two workgroups per compute unit; no part is shorter than one step a wave.  (Four
// times as many: 64 sequences of uneven lengths up to 8129 tokens 120 -> 112 us, but 63 of
// 4096 103 -> 112 and four of 65536 112 -> 122: a part's start and end cost about as much as
// four steps.)  Up to eight steps, eight waves a workgroup take them at one step a wave in
// one launch (300 tokens of 20 heads, in a graph, 10.5 -> 9.8 us with the join; 1000 tokens at
// two steps a wave 10.8 -> 14.3).
AttnPlan attn_decode_plan(const KvCache& c, const KvBatch& b, int q_heads) {
  AttnPlan p = attn_plan(c, b, q_heads, kCols, 512, kWaves);
  p.waves = kWaves;
  if (p.splits > 1 && b.max_len <= kOneLaunch * kStep && c.head_dim <= 128) {
    p.splits = 1;
    p.waves = kManyWaves;
  }
  return p;
}

hipError_t launch_attn_decode(const KvCache& c, const KvBatch& b, const AttnArgs& a,
                              const AttnPlan& p, bool q_bf16, bool out_bf16, void* workspace,
                              hipStream_t s) {
  const int64_t grid = (int64_t)b.seqs * c.kv_heads * p.tiles * p.splits;
  float* part = static_cast<float*>(workspace);
  const void* kern = p.waves == kManyWaves ? pick_decode<kManyWaves>(c.head_dim, q_bf16, out_bf16)
                                           : pick_decode<kWaves>(c.head_dim, q_bf16, out_bf16);
  void* args[] = {(void*)&c, (void*)&b, (void*)&a, (void*)&p, (void*)&part};
  const hipError_t e = hipLaunchKernel(kern, dim3((unsigned)grid), dim3(64 * p.waves), args, 0, s);
  if (e != hipSuccess || p.splits == 1) return e;
  return launch_attn_join(c, b, a, p, out_bf16, part, s);
}

}  // namespace bitnet
