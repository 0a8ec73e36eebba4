// Paged attention over a bf16 cache, and the choice of the cache type's kernels.
#include "attention_kernels.h"

namespace rax {

template hipError_t launch_attention_of<uint16_t>(const AttentionArgs&, hipStream_t, const KTimer&);
extern template hipError_t launch_attention_of<uint8_t>(const AttentionArgs&, hipStream_t, const KTimer&);
extern template hipError_t launch_attention_of<float>(const AttentionArgs&, hipStream_t, const KTimer&);

hipError_t launch_paged_attention(const AttentionArgs& a, hipStream_t stream, const KTimer& tm) {
  if (a.dtype == LORA_F32) return launch_attention_of<float>(a, stream, tm);
  if (a.c.dtype == LORA_FP8E4M3) return launch_attention_of<uint8_t>(a, stream, tm);
  return launch_attention_of<uint16_t>(a, stream, tm);
}

}  // namespace rax
