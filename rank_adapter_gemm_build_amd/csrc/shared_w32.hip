// Shared attention over an fp32 cache.
#include "shared_kernels.h"

namespace rax {
template hipError_t launch_shared_of<float>(const SharedArgs&, hipStream_t, const KTimer&);
}
