// Paged attention over an fp32 cache.
#include "attention_kernels.h"

namespace rax {
template hipError_t launch_attention_of<float>(const AttentionArgs&, hipStream_t, const KTimer&);
}
