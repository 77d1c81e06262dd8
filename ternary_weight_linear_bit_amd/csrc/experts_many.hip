// Experts' products with many rows: int8 contraction on the matrix cores.
//
// A workgroup takes BM slots of one expert and 64 WN rows of weights (of gate and up 32 WN each, so
// that a lane holds both values of an output and the activation needs no memory), in 32 x 32 blocks
// of int32 sums.  K advances in steps of 128:
//  * the slots' rows, gathered, are staged in LDS (two buffers, a barrier a step), step s + 1
//    between the matrix instructions of step s;
//  * each wave loads its weights straight from memory, 1 KiB a load, and expands them with a
//    shift and a mask per four weights to -64 q (weights_64), so that neither operand needs sums
//    or shuffles;
//  * weights are loaded two steps ahead, x one or two ahead of its staging (more would cost a wave a
//    SIMD with 64 slots).
//
// Bound by the matrix cores at the clock that power allows: 8192 x 14336 x 8192 dense in 641-676 us
// (2.8-3.0 POPS; matrix instructions alone reach 4.2 on such operands), 4096 tokens through gate and up
// of two of eight 2560 -> 6912 experts in 229-237 us (2.5 POPS), where the tiles' beginnings and ends
// count.  Weights expanded to -64 q take 4 vector instructions a matrix instruction with 64 slots
// and 2.7 with 96.  Few rows an expert are bound by memory: 64 tokens over 64 experts of 2560 -> 1152, 94
// MB of weights, 21 us (4.4 TB/s).
#include "experts_internal.h"

namespace bitnet {
namespace {

typedef int v16i __attribute__((ext_vector_type(16)));

constexpr int kXcds = 8;
constexpr int kStep = 128;      // k of a step
constexpr int kChunk = 1 << 21; // bytes of x that a chunk of tiles reads

// Byte of 16-byte group g of staged row t.  A 16-byte access takes 16 lanes at a time, lanes 0-3,
// 12-15, 20-23, 24-27 and 4-7, 8-11, 16-19, 28-31 of each half wave, whose groups have to differ
// modulo 256 bytes (two rows): XORed with the row's number over two they do, both where a
// matrix instruction reads 32 rows and where 8 lanes write a row.
__device__ __forceinline__ int group_at(int t, int g) { return t * kStep + 16 * (g ^ ((t >> 1) & 7)); }

// WN waves of TB 32-slot blocks x 64 weight rows; KS groups of them share the k steps.  DX: steps that
// x is loaded ahead of its staging.
template <int TB, int WN, int KS, int DX, bool GATED>
__global__ __launch_bounds__(64 * WN * KS, TB == 3 ? 3 : 4) void experts_many_kernel(const ExpertArgs a, int ntiles) {
  constexpr int BM = 32 * TB;              // slots of a workgroup
  constexpr int T = 64 * WN;               // threads of a group
  constexpr int COLS = GATED ? 32 : 64;    // outputs of a wave
  constexpr int XG = BM * 8 / T;           // 16-byte groups a thread stages
  constexpr int OUT = 16 * COLS;           // floats of the unit that leaves through LDS
  constexpr int STAGED = 2 * KS * BM * kStep, UNITS = WN * OUT * 4;
  // half of the groups' sums at a time (a quarter, and so on) meet those of the others
  constexpr int SUMS = KS / 2 * WN * TB * 2 * 16 * 64 * 4;
  constexpr int BYTES = STAGED > UNITS ? (STAGED > SUMS ? STAGED : SUMS) : (UNITS > SUMS ? UNITS : SUMS);
  static_assert(XG >= 1 && (KS & (KS - 1)) == 0, "shapes");
  __shared__ __attribute__((aligned(16))) uint8_t lds[BYTES];
  __shared__ float scale_of[GATED ? 2 : 1][BM];      // gamma d of each matrix
  __shared__ int row_of[BM];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kg = wave / WN, wr = wave % WN, gt = tid % T;
  const int r = lane & 31, h = lane >> 5;
  const int K = a.K, steps = (K + kStep - 1) / kStep, nblocks = (a.N + 31) / 32;
  // Workgroup b runs on XCD b % 8: each XCD takes a contiguous run of tiles.  An expert's tiles go by
  // chunks of slot tiles whose rows stay in its L2, and in a chunk slot tiles first, so that each
  // block of weights is read by them one after another.
  const int tiles = ntiles * count_tiles<BM>(a);
  const int per_xcd = (tiles + kXcds - 1) / kXcds;
  const int t = (int)(blockIdx.x % kXcds) * per_xcd + (int)(blockIdx.x / kXcds);
  if ((int)(blockIdx.x / kXcds) >= per_xcd || t >= tiles) return;
  const ExpertSpan et = expert_span<BM>(a, t / ntiles);
  if (et.n == 0) return;
  const int mtiles = (et.n + BM - 1) / BM, most = max(1, min(8, kChunk / (BM * K)));
  const int u = t - et.tile0 * ntiles, chunk = u / (most * ntiles), v = u - chunk * most * ntiles;
  const int across = min(most, mtiles - chunk * most), nt = v / across;
  const int slot0 = et.slot0 + (chunk * most + v - nt * across) * BM, rows = min(et.slot0 + et.n - slot0, BM);

  for (int i = tid; i < BM; i += T * KS) {
    const int row = i < rows ? input_row(a, slot0 + i) : -1;
    const float d = row < 0 ? 0.0f : a.xs[row];
    row_of[i] = row;
    scale_of[0][i] = a.w_scale[et.expert] * d;
    if (GATED) scale_of[GATED ? 1 : 0][i] = a.up_scale[et.expert] * d;
  }
  // rows without a slot read the tile's first row or row 0; nothing of theirs is kept
  const bool gather = a.pair != nullptr;
  const auto xr = gather
      ? make_uniform_rsrc(a.xq, (uint32_t)((int64_t)a.rows * K))       // (at most 2^31)
      : make_uniform_rsrc(a.xq + (size_t)slot0 * K, (uint32_t)(rows * K));
  uint32_t xo[XG];
#pragma unroll
  for (int i = 0; i < XG; ++i) {
    const int sl = (gt >> 3) + T / 8 * i;
    int row = 0;
    if (sl < rows) row = gather ? max(input_row(a, slot0 + sl), 0) : sl;
    xo[i] = (uint32_t)row * (uint32_t)K + 16u * (uint32_t)(gt & 7);
  }
  // this wave's two blocks of 32 weight rows: neighbours, or the same of gate and up
  const int rb = nt * ((GATED ? 32 : 64) * WN / 32) + (GATED ? wr : 2 * wr);
  const uint32_t blk = (uint32_t)steps * 1024u;
  const size_t expert_at = (size_t)et.expert * nblocks * blk;
  const int nb = max(0, min(GATED ? 1 : 2, nblocks - rb));
  const auto wr0 = make_uniform_rsrc(a.w + expert_at + (size_t)rb * blk, (uint32_t)nb * blk);
  const auto wr1 = GATED ? make_uniform_rsrc(a.up + expert_at + (size_t)rb * blk, (uint32_t)nb * blk) : wr0;

  // (steps past the end read what lies there, or zeros past the buffers; nothing uses them)
  auto xload = [&](uint4 (&v)[XG], int it) {
#pragma unroll
    for (int i = 0; i < XG; ++i) v[i] = bload16(xr, xo[i] + (uint32_t)(it * KS + kg) * kStep);
  };
  auto wload = [&](uint4 (&v)[2], int it) {
    const uint32_t o = (uint32_t)(it * KS + kg) * 1024u + 16u * (uint32_t)lane;
    v[0] = bload16(wr0, o);
    v[1] = bload16(wr1, GATED ? o : o + blk);
  };
  auto stage = [&](const uint4& v, int i, uint8_t* buf) {
    *reinterpret_cast<uint4*>(buf + group_at((gt >> 3) + T / 8 * i, gt & 7)) = v;
  };
  auto aread = [&](const uint8_t* buf, int i, int j) -> v4i {
    return *reinterpret_cast<const v4i*>(buf + group_at(32 * i + r, 4 * h + j));
  };

  v16i acc[TB][2];
#pragma unroll
  for (int i = 0; i < TB; ++i)
#pragma unroll
    for (int b = 0; b < 2; ++b) acc[i][b] = (v16i){};

  // Iteration it of this group: step it KS + kg, staged in buffer it & 1.
  auto buffer = [&](int it) { return lds + ((it & 1) * KS + kg) * (BM * kStep); };
  auto body = [&](uint4 (&xv)[XG], uint4 (&wv)[2], int it) {
    const uint8_t* cur = buffer(it);
    uint8_t* nxt = buffer(it + 1);
    const uint32_t wd[2][4] = {{wv[0].x, wv[0].y, wv[0].z, wv[0].w}, {wv[1].x, wv[1].y, wv[1].z, wv[1].w}};
    const bool on = KS == 1 || it * KS + kg < steps;
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
        xload(xv, it + 1 + DX);
        wload(wv, it + 2);
      }
      if (on) {
#pragma unroll
        for (int i = 0; i < TB; ++i)
#pragma unroll
          for (int b = 0; b < 2; ++b)
            acc[i][b] = __builtin_amdgcn_mfma_i32_32x32x32_i8(x[i], w[b], acc[i][b], 0, 0, 0);
      }
    }
    lds_barrier();     // iteration it + 1 is staged; nobody reads this one's buffer any more
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
  for (int i = 0; i < XG; ++i) stage(x0[i], i, buffer(0));
  lds_barrier();
  const int its = (steps + KS - 1) / KS;
  int it = 0;
  for (; it + 1 < its; it += 2) {
    body(xv[0], wv[0], it);
    body(xv[DX - 1], wv[1], it + 1);
  }
  if (it < its) body(xv[0], wv[0], it);

  // the groups' sums: the upper half's go to the lower half, until group 0 has all
  if constexpr (KS > 1) {
    int* sums = reinterpret_cast<int*>(lds) + lane;
    constexpr int R = TB * 2 * 16;
#pragma unroll
    for (int half = KS / 2; half >= 1; half /= 2) {
      if (kg >= half && kg < 2 * half) {
        int* to = sums + (wave - half * WN) * (R * 64);
#pragma unroll
        for (int q = 0; q < R; ++q) to[q * 64] = acc[q / 32][q / 16 % 2][q % 16];
      }
      __syncthreads();
      if (kg < half) {
        const int* from = sums + wave * (R * 64);
#pragma unroll
        for (int q = 0; q < R; ++q) acc[q / 32][q / 16 % 2][q % 16] += from[q * 64];
      }
      __syncthreads();
    }
    if (kg > 0) return;
  }

  // 16 slots at a time through LDS (free behind the last barrier), so that rows leave in 16 bytes
  // a lane.  Lane l holds weight row l % 32 and slots 8 (v / 4) + 4 (l / 32) + v % 4.
  float* unit = reinterpret_cast<float*>(lds) + wave * OUT;
  const int n0 = rb * 32;
  float bias[2];
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const float* bs = GATED && b ? a.up_bias : a.bias;
    const int n = n0 + r + (GATED ? 0 : 32 * b);
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
        const int sl = 32 * i + 16 * q + 8 * (e >> 2) + 4 * h + (e & 3);
        v0[e] = acc_64(acc[i][0][8 * q + e]) * scale_of[0][sl];
        v1[e] = acc_64(acc[i][1][8 * q + e]) * scale_of[GATED ? 1 : 0][sl];
        if (has0) v0[e] = v0[e] + bias[0];
        if (has1) v1[e] = v1[e] + bias[1];
      }
      if (a.act != kActNone) {
        activate(v0, a.act);
        if (!GATED) activate(v1, a.act);
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
        const int ml = 32 * i + 16 * q + sl, n = n0 + c;
        if (row_of[ml] < 0 || n >= a.N) continue;
        const size_t o = (size_t)(slot0 + ml) * a.N + n;
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

template <int TB, int WN, int KS, int DX>
hipError_t launch_many(const ExpertArgs& a, hipStream_t s) {
  const int bn = a.up ? 32 * WN : 64 * WN;
  const int ntiles = (int)(((int64_t)a.N + bn - 1) / bn);     // (N is up to 2^31 - 32)
  const dim3 grid((unsigned)((many_tiles(a, 32 * TB) * ntiles + kXcds - 1) / kXcds * kXcds)), block(64 * WN * KS);
  if (a.up)
    hipLaunchKernelGGL((experts_many_kernel<TB, WN, KS, DX, true>), grid, block, 0, s, a, ntiles);
  else
    hipLaunchKernelGGL((experts_many_kernel<TB, WN, KS, DX, false>), grid, block, 0, s, a, ntiles);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_experts_many(const ExpertArgs& a, ManyTile tile, hipStream_t s) {
  switch (tile) {
    case kMany32x2: return launch_many<1, 1, 8, 1>(a, s);
    case kMany32x4: return launch_many<1, 2, 4, 2>(a, s);
    case kMany32x8: return launch_many<1, 4, 1, 2>(a, s);
    case kMany64x8: return launch_many<2, 4, 1, 1>(a, s);
    case kMany96x8: return launch_many<3, 4, 1, 1>(a, s);
    case kMany64x16: return launch_many<2, 8, 1, 1>(a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace bitnet
