// Shared attention over an e4m3 cache.
#include "shared_kernels.h"

namespace rax {
template hipError_t launch_shared_of<uint8_t>(const SharedArgs&, hipStream_t, const KTimer&);
}
