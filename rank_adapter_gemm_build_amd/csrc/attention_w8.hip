// Paged attention over an e4m3 cache.
#include "attention_kernels.h"

namespace rax {
template hipError_t launch_attention_of<uint8_t>(const AttentionArgs&, hipStream_t, const KTimer&);
}
