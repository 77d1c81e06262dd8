// Experts' products with many rows: int8 contraction on the matrix cores.
//
// A workgroup takes BM slots of one expert and 64 WN rows of weights (of gate and up 32 WN each, so
// that a lane holds both values of an output and the activation needs no memory); 2 WN waves,
// each with (BM / 2) slots x 64 rows as 32 x 32 blocks of int32 sums.  K advances in steps of 128:
//  * the slots' rows, gathered, are staged in LDS (two buffers, a barrier a step), step s + 1
//    between the matrix instructions of step s;
//  * each wave loads its weights straight from memory, 1 KiB a load, and expands them with a
//    shift and a mask per four weights to -64 q (weights_64), so that neither operand needs sums
//    or shuffles;
//  * loads run two steps ahead.
#include "experts_internal.h"

namespace bitnet {
namespace {

typedef int v16i __attribute__((ext_vector_type(16)));

constexpr int kXcds = 8;
constexpr int kStep = 128;      // k of a step

// Byte of 16-byte group g of staged row t.  A 16-byte access takes 16 lanes at a time, lanes 0-3,
// 12-15, 20-23, 24-27 and 4-7, 8-11, 16-19, 28-31 of each half wave, whose groups have to differ
// modulo 256 bytes (two rows): XORed with the row's number over two they do, both where a
// matrix instruction reads 32 rows and where 8 lanes write a row.
__device__ __forceinline__ int group_at(int t, int g) { return t * kStep + 16 * (g ^ ((t >> 1) & 7)); }

template <int BM, int WN, int DX, int OCC, bool GATED>
__global__ __launch_bounds__(128 * WN, OCC) void experts_many_kernel(const ExpertArgs a, int ntiles) {
  constexpr int T = 128 * WN;              // threads
  constexpr int COLS = GATED ? 32 : 64;    // outputs of a wave
  constexpr int TB = BM / 64;              // 32-slot blocks of a wave
  constexpr int XG = BM * 8 / T;           // 16-byte groups a thread stages
  constexpr int OUT = 16 * COLS;           // floats of the unit that leaves through LDS
  constexpr int BUF = BM * kStep > 4 * WN * OUT ? BM * kStep : 4 * WN * OUT;   // half of the units too
  static_assert(XG >= 1 && BM <= T, "shapes");
  __shared__ __attribute__((aligned(16))) uint8_t xs[2][BUF];
  __shared__ float d_of[BM];
  __shared__ int row_of[BM];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wt = wave / WN, wr = wave % WN;
  const int r = lane & 31, h = lane >> 5;
  const int K = a.K, steps = (K + kStep - 1) / kStep, nblocks = (a.N + 31) / 32;
  // workgroup b runs on XCD b % 8: each XCD takes a contiguous run of tiles, those of one
  // expert's slots beside each other, so that they share its L2
  const int tiles = ntiles * count_tiles<BM>(a);
  const int per_xcd = (tiles + kXcds - 1) / kXcds;
  const int t = (int)(blockIdx.x % kXcds) * per_xcd + (int)(blockIdx.x / kXcds);
  if ((int)(blockIdx.x / kXcds) >= per_xcd || t >= tiles) return;
  const int mt = t / ntiles, nt = t - mt * ntiles;
  const ExpertTile et = expert_tile<BM>(a, mt);
  if (et.rows <= 0) return;

  if (tid < BM) {
    const int row = tid < et.rows ? input_row(a, et.slot0 + tid) : -1;
    row_of[tid] = row;
    d_of[tid] = row < 0 ? 0.0f : a.xs[row];
  }
  // rows without a slot read the tile's first row or row 0; nothing of theirs is kept
  const bool gather = a.pair != nullptr;
  const auto xr = gather
      ? make_uniform_rsrc(a.xq, (uint32_t)min((int64_t)a.rows * K, (int64_t)0xffffffffu))
      : make_uniform_rsrc(a.xq + (size_t)et.slot0 * K, (uint32_t)(et.rows * K));
  uint32_t xo[XG];
#pragma unroll
  for (int i = 0; i < XG; ++i) {
    const int sl = (tid >> 3) + T / 8 * i;
    int row = 0;
    if (sl < et.rows) row = gather ? max(input_row(a, et.slot0 + sl), 0) : sl;
    xo[i] = (uint32_t)row * (uint32_t)K + 16u * (uint32_t)(tid & 7);
  }
  // this wave's two blocks of 32 weight rows: neighbours, or the same of gate and up
  const int rb = nt * ((GATED ? 32 : 64) * WN / 32) + (GATED ? wr : 2 * wr);
  const uint32_t blk = (uint32_t)steps * 1024u;
  const size_t expert_at = (size_t)et.expert * nblocks * blk;
  const int nb = max(0, min(GATED ? 1 : 2, nblocks - rb));
  const auto wr0 = make_uniform_rsrc(a.w + expert_at + (size_t)rb * blk, (uint32_t)nb * blk);
  const auto wr1 = GATED ? make_uniform_rsrc(a.up + expert_at + (size_t)rb * blk, (uint32_t)nb * blk) : wr0;

  // (steps past the end read what lies there, or zeros past the buffers; nothing uses them)
  auto xload = [&](uint4 (&v)[XG], int s) {
#pragma unroll
    for (int i = 0; i < XG; ++i) v[i] = bload16(xr, xo[i] + (uint32_t)s * kStep);
  };
  auto wload = [&](uint4 (&v)[2], int s) {
    const uint32_t o = (uint32_t)s * 1024u + 16u * (uint32_t)lane;
    v[0] = bload16(wr0, o);
    v[1] = bload16(wr1, GATED ? o : o + blk);
  };
  auto stage = [&](const uint4& v, int i, uint8_t* buf) {
    *reinterpret_cast<uint4*>(buf + group_at((tid >> 3) + T / 8 * i, tid & 7)) = v;
  };
  auto aread = [&](const uint8_t* buf, int i, int j) -> v4i {
    return *reinterpret_cast<const v4i*>(buf + group_at(wt * (BM / 2) + 32 * i + r, 4 * h + j));
  };

  v16i acc[TB][2];
#pragma unroll
  for (int i = 0; i < TB; ++i)
#pragma unroll
    for (int b = 0; b < 2; ++b) acc[i][b] = (v16i){};

  auto body = [&](uint4 (&xv)[XG], uint4 (&wv)[2], int s) {
    const uint8_t* cur = xs[s & 1];
    uint8_t* nxt = xs[(s + 1) & 1];
    const uint32_t wd[2][4] = {{wv[0].x, wv[0].y, wv[0].z, wv[0].w}, {wv[1].x, wv[1].y, wv[1].z, wv[1].w}};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v4i x[TB], w[2];
#pragma unroll
      for (int i = 0; i < TB; ++i) x[i] = aread(cur, i, j);
#pragma unroll
      for (int b = 0; b < 2; ++b) w[b] = weights_64(wd[b][j]);
#pragma unroll
      for (int i = 0; i < XG; ++i)
        if (j == i * 4 / XG) stage(xv[i], i, nxt);
      if (j == 3) {
        // every use of xv and wv is above: the loads reuse their registers
        asm volatile("" : "+v"(w[0]), "+v"(w[1])::"memory");
        xload(xv, s + 1 + DX);
        wload(wv, s + 2);
      }
#pragma unroll
      for (int i = 0; i < TB; ++i)
#pragma unroll
        for (int b = 0; b < 2; ++b)
          acc[i][b] = __builtin_amdgcn_mfma_i32_32x32x32_i8(x[i], w[b], acc[i][b], 0, 0, 0);
    }
    lds_barrier();     // step s + 1 is staged; nobody reads xs[s & 1] any more
  };

  uint4 x0[XG], xv[DX][XG], wv[2][2];
  xload(x0, 0);
#pragma unroll
  for (int d = 0; d < 2; ++d) {
    asm volatile("" ::: "memory");
    if (d < DX) xload(xv[d], d + 1);
    wload(wv[d], d);
  }
#pragma unroll
  for (int i = 0; i < XG; ++i) stage(x0[i], i, xs[0]);
  lds_barrier();
  int s = 0;
  for (; s + 1 < steps; s += 2) {
    body(xv[0], wv[0], s);
    body(xv[DX - 1], wv[1], s + 1);
  }
  if (s < steps) body(xv[0], wv[0], s);

  // 16 slots at a time through LDS (free behind the last barrier), so that rows leave in 16 bytes
  // a lane.  Lane l holds weight row l % 32 and slots 8 (v / 4) + 4 (l / 32) + v % 4.
  float* unit = reinterpret_cast<float*>(&xs[0][0]) + wave * OUT;
  const int n0 = rb * 32;
  float gamma[2], bias[2];
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const float* sc = GATED && b ? a.up_scale : a.w_scale;
    const float* bs = GATED && b ? a.up_bias : a.bias;
    const int n = n0 + r + (GATED ? 0 : 32 * b);
    gamma[b] = sc[et.expert];
    bias[b] = bs && n < a.N ? bs[(size_t)et.expert * a.N + n] : 0.0f;
  }
  const bool has0 = a.bias != nullptr, has1 = GATED ? a.up_bias != nullptr : has0;
  const int es = a.y_bf16 ? 2 : 4;
  const bool wide = ((reinterpret_cast<uintptr_t>(a.y) | reinterpret_cast<uintptr_t>(a.residual) |
                      ((size_t)a.N * es)) & 15u) == 0;
#pragma unroll
  for (int i = 0; i < TB; ++i)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float v0[8], v1[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = d_of[wt * (BM / 2) + 32 * i + 16 * q + 8 * (e >> 2) + 4 * h + (e & 3)];
        v0[e] = acc_64(acc[i][0][8 * q + e]) * (gamma[0] * d);
        v1[e] = acc_64(acc[i][1][8 * q + e]) * (gamma[1] * d);
        if (has0) v0[e] = v0[e] + bias[0];
        if (has1) v1[e] = v1[e] + bias[1];
      }
      if (a.act != kActNone) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v0[e] = activate(v0[e], a.act);
          if (!GATED) v1[e] = activate(v1[e], a.act);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int sl = 8 * (e >> 2) + 4 * h + (e & 3);
        if constexpr (GATED) {
          unit[(sl ^ h) * 32 + r] = v0[e] * v1[e];
        } else {
          unit[sl * 64 + (r ^ (32 * h))] = v0[e];
          unit[sl * 64 + ((32 + r) ^ (32 * h))] = v1[e];
        }
      }
      // a lane takes 8 columns of a slot
#pragma unroll
      for (int p = 0; p < OUT / 512; ++p) {
        const int sl = (lane + 64 * p) / (COLS / 8), c = 8 * (lane % (COLS / 8));
        const int odd = (sl >> 2) & 1;
        const float* from = GATED ? unit + (sl ^ odd) * 32 + c : unit + sl * 64 + (c ^ (32 * odd));
        const float4 lo = *reinterpret_cast<const float4*>(from);
        const float4 hi = *reinterpret_cast<const float4*>(from + 4);
        float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        const int ml = wt * (BM / 2) + 32 * i + 16 * q + sl, n = n0 + c;
        if (row_of[ml] < 0 || n >= a.N) continue;
        const size_t o = (size_t)(et.slot0 + ml) * a.N + n;
        if (wide && n + 8 <= a.N) {
          typedef uint32_t u4 __attribute__((ext_vector_type(4)));
          if (a.y_bf16) {
            if (a.residual) {
              const uint4 z = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.residual) + o);
              const uint32_t zw[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                v[2 * e] = v[2 * e] + __uint_as_float(zw[e] << 16);
                v[2 * e + 1] = v[2 * e + 1] + __uint_as_float(zw[e] & 0xffff0000u);
              }
            }
            const u4 w = {bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]), bf16x2_rne(v[4], v[5]),
                          bf16x2_rne(v[6], v[7])};
            __builtin_nontemporal_store(w, reinterpret_cast<u4*>(static_cast<uint16_t*>(a.y) + o));
          } else {
            if (a.residual) {
              const float4* z = reinterpret_cast<const float4*>(static_cast<const float*>(a.residual) + o);
              const float4 z0 = z[0], z1 = z[1];
              const float zw[8] = {z0.x, z0.y, z0.z, z0.w, z1.x, z1.y, z1.z, z1.w};
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = v[e] + zw[e];
            }
            u4* y = reinterpret_cast<u4*>(static_cast<float*>(a.y) + o);
#pragma unroll
            for (int p2 = 0; p2 < 2; ++p2) {
              const u4 w = {__float_as_uint(v[4 * p2]), __float_as_uint(v[4 * p2 + 1]),
                            __float_as_uint(v[4 * p2 + 2]), __float_as_uint(v[4 * p2 + 3])};
              __builtin_nontemporal_store(w, y + p2);
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (n + e < a.N) store_output(a, o + e, v[e]);
        }
      }
    }
}

template <int BM, int WN, int DX, int OCC>
hipError_t launch_many(const ExpertArgs& a, hipStream_t s) {
  const int bn = a.up ? 32 * WN : 64 * WN;
  const int ntiles = (a.N + bn - 1) / bn;
  const int64_t grid = (many_tiles(a, BM) * ntiles + kXcds - 1) / kXcds * kXcds;
  if (a.up)
    hipLaunchKernelGGL((experts_many_kernel<BM, WN, DX, OCC, true>), dim3((unsigned)grid), dim3(128 * WN), 0, s, a, ntiles);
  else
    hipLaunchKernelGGL((experts_many_kernel<BM, WN, DX, OCC, false>), dim3((unsigned)grid), dim3(128 * WN), 0, s, a, ntiles);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_experts_many(const ExpertArgs& a, int bm, hipStream_t s) {
  switch (bm) {
    case 128: return launch_many<128, 4, 1, 4>(a, s);
    case 64: return launch_many<64, 4, 2, 4>(a, s);
    default: return launch_many<64, 2, 2, 2>(a, s);
  }
}

}  // namespace bitnet
