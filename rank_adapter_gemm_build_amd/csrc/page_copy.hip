// Page copy: the keys and values of the first tokens of page src[i] to page dst[i], in all layers.
//
// What bounds it: memory, each cell read and written once.  A workgroup takes one page of keys or
// of values of one layer, or where those are few and large every gridDim.z-th slab of one, 16 bytes a lane and load, in the order in which the cells lie (heads
// inside tokens or tokens inside heads), with the loads of kCopyBatch chunks on the way together.  Measured: 448 pages of
// 16 tokens in 32 layers 170 us (5.6 TB/s read and written), 200 of 64 in e4m3 in 8 layers 73 (5.8), 3 in 32 layers 4.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "beam.h"
#include "device_util.h"

namespace rax {

constexpr int kCopyThreads = 256, kCopyBatch = 4, kCopySlab = kCopyBatch * kCopyThreads;   // slab: 16 KiB

__global__ __launch_bounds__(kCopyThreads) void page_copy_kernel(PageCopyArgs a, int cell_bytes) {
  const int pair = blockIdx.x, which = blockIdx.y;   // which: layer and k or v
  const int src = page_or_none(a.src[pair], a.c.num_pages), dst = page_or_none(a.dst[pair], a.c.num_pages);
  if (src < 0 || dst < 0 || src == dst) return;
  const int page_size = 1 << a.c.page_shift, n = a.tokens ? clamp_int(a.tokens[pair], 0, page_size) : page_size;
  char* const base = reinterpret_cast<char*>(a.cells[which]);
  const char* const from = base + (long long)src * a.c.page_stride * cell_bytes;
  char* const to = base + (long long)dst * a.c.page_stride * cell_bytes;
  const int chunks = a.c.dim * cell_bytes / 16, items = n * a.c.heads * chunks;   // at most 2^10 2^10 2^6
  const long long token = a.c.token_stride * cell_bytes, head = a.c.head_stride * cell_bytes;
  for (int i0 = blockIdx.z * kCopySlab + threadIdx.x; i0 < items; i0 += gridDim.z * kCopySlab) {
    uint4 v[kCopyBatch];
    long long at[kCopyBatch];
#pragma unroll
    for (int k = 0; k < kCopyBatch; ++k) {
      const int i = i0 + k * kCopyThreads;
      if (i >= items) continue;
      const int row = fast_quot(i, a.per_row), chunk = i - row * chunks;
      int t, h;
      if (a.head_major) {
        h = (int)((unsigned)row / (unsigned)n);
        t = row - h * n;
      } else {
        t = fast_quot(row, a.per_inner);
        h = row - t * a.c.heads;
      }
      at[k] = t * token + h * head + chunk * 16;
      v[k] = ld16(from + at[k]);
    }
#pragma unroll
    for (int k = 0; k < kCopyBatch; ++k)
      if (i0 + k * kCopyThreads < items) st16(to + at[k], v[k]);
  }
}

hipError_t launch_page_copy(const PageCopyArgs& a, hipStream_t stream, const KTimer& tm) {
  const int cell = a.c.dtype == LORA_F32 ? 4 : a.c.dtype == LORA_BF16 ? 2 : 1;
  // eight workgroups for each of 256 compute units, if the pages have slabs for them (4 pages of 16 MiB, keys and values, in 2
  // layers: 1014 us with a workgroup a page, 110 with 128)
  const int slabs = ((a.c.dim * cell / 16 * a.c.heads << a.c.page_shift) + kCopySlab - 1) / kCopySlab;   // of a page: at most 2^16
  const int parts = (int)std::min<long long>(slabs, std::max(1LL, 2048 / ((long long)a.pairs * 2 * a.layers)));
  RAX_LAUNCH(tm, page_copy_kernel, dim3(a.pairs, 2 * a.layers, parts), dim3(kCopyThreads), 0u, stream, a, cell);
  return hipGetLastError();
}

}  // namespace rax
