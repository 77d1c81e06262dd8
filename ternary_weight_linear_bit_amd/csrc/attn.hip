// Attention over the paged 8-bit cache: which kernel a call takes.
#include "bitnet_internal.h"

namespace bitnet {

size_t attention_workspace_bytes(const KvCache& c, const KvBatch& b, int q_heads) {
  return attn_decode_workspace(c, b, q_heads);
}

hipError_t launch_attention(const KvCache& c, const KvBatch& b, const AttnArgs& a, bool q_bf16,
                            bool out_bf16, void* workspace, hipStream_t s) {
  return launch_attn_decode(c, b, a, q_bf16, out_bf16, workspace, s);
}

}  // namespace bitnet
