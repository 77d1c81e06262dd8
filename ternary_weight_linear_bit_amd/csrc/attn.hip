// Attention over the paged 8-bit cache.
//
// Query row i of a sequence with n new rows and len cached tokens has position
// pos = len - n + i and sees the keys j with max(0, pos - window + 1) <= j <= pos
// (window 0: from 0).  With codes kc, vc and the page's scales dk, dv:
//   s_j = scale * dk * (q . kc_j),  m = max s_j,
//   out = sum_j exp(s_j - m) dv vc_j / sum_j exp(s_j - m),  lse = m + ln sum.
// A row without keys gives zeros and lse = -inf.  A page id outside the cache
// holds no keys.
#include "bitnet_internal.h"

namespace bitnet {
namespace {

constexpr int kAttnThreads = 256;

// One workgroup per query row and head; 256 keys at a time.
template <bool QB, bool OB>
__global__ __launch_bounds__(kAttnThreads) void attn_row_kernel(const KvCache c, const KvBatch b,
                                                                const AttnArgs a) {
  __shared__ float qs[256], ps[kAttnThreads], red[4];
  __shared__ int64_t at[kAttnThreads];
  const int tid = threadIdx.x, head = blockIdx.y;
  const int D = c.head_dim, P = c.page;
  const int kvh = head / (a.q_heads / c.kv_heads);
  const SeqSpan sp = seq_span(b, blockIdx.z);
  const int i = blockIdx.x;
  if (i >= sp.n) return;
  const int64_t t = sp.s0 + i;
  const int pos = sp.first + i;
  for (int d = tid; d < D; d += kAttnThreads) {
    const int64_t o = t * a.q_stride + (int64_t)head * D + d;
    qs[d] = QB ? bf16_bits_to_float(reinterpret_cast<const uint16_t*>(a.q)[o])
               : reinterpret_cast<const float*>(a.q)[o];
  }
  __syncthreads();
  float m = -INFINITY, l = 0.0f, o = 0.0f;
  const int j0 = a.window > 0 ? max(0, pos - a.window + 1) : 0;
  for (int base = j0; base <= pos; base += kAttnThreads) {
    const int j = base + tid;
    float s = -INFINITY, dv = 0.0f;
    int64_t va = 0;
    if (j <= pos) {
      const int pid = b.table[(int64_t)blockIdx.z * b.width + j / P];
      if (pid >= 0 && pid < c.pages) {
        const int64_t ph = (int64_t)pid * c.kv_heads + kvh;
        const int8_t* kr = c.k + (ph * P + j % P) * D;
        float dot = 0.0f;
        for (int d = 0; d < D; ++d) dot += qs[d] * (float)kr[d];
        s = dot * c.k_scale[ph] * a.scale;
        dv = c.v_scale[ph];
        va = ph * P * D + j % P;
      }
    }
    float mt = s;
    for (int x = 32; x > 0; x >>= 1) mt = fmaxf(mt, __shfl_xor(mt, x, 64));
    __syncthreads();
    if ((tid & 63) == 0) red[tid >> 6] = mt;
    __syncthreads();
    mt = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float mn = fmaxf(m, mt);
    const float f = m == -INFINITY ? 0.0f : expf(m - mn);
    const float p = s == -INFINITY ? 0.0f : expf(s - mn);
    m = mn;
    float lt = p;
    for (int x = 32; x > 0; x >>= 1) lt += __shfl_xor(lt, x, 64);
    __syncthreads();
    if ((tid & 63) == 0) red[tid >> 6] = lt;
    ps[tid] = p * dv;
    at[tid] = va;
    __syncthreads();
    l = l * f + (red[0] + red[1] + red[2] + red[3]);
    if (tid < D) {
      o *= f;
      for (int x = 0; x < kAttnThreads; ++x)
        if (ps[x] != 0.0f) o += ps[x] * (float)c.v[at[x] + (int64_t)tid * P];
    }
  }
  if (tid < D) {
    const float y = l > 0.0f ? o / l : 0.0f;
    const int64_t w = (t * a.q_heads + head) * D + tid;
    if (OB)
      reinterpret_cast<uint16_t*>(a.out)[w] = float_to_bf16_rne(y);
    else
      reinterpret_cast<float*>(a.out)[w] = y;
  }
  if (tid == 0 && a.lse) a.lse[t * a.q_heads + head] = l > 0.0f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t attention_workspace_bytes(const KvCache&, const KvBatch&, int) { return 0; }

hipError_t launch_attention(const KvCache& c, const KvBatch& b, const AttnArgs& a, bool q_bf16,
                            bool out_bf16, void*, hipStream_t s) {
  const void* kern = q_bf16 ? (out_bf16 ? (const void*)attn_row_kernel<true, true>
                                        : (const void*)attn_row_kernel<true, false>)
                            : (out_bf16 ? (const void*)attn_row_kernel<false, true>
                                        : (const void*)attn_row_kernel<false, false>);
  void* args[] = {(void*)&c, (void*)&b, (void*)&a};
  return hipLaunchKernel(kern, dim3((unsigned)b.max_new, (unsigned)a.q_heads, (unsigned)b.seqs),
                         dim3(kAttnThreads), args, 0, s);
}

}  // namespace bitnet
