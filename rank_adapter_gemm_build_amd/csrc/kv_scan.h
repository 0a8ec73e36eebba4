// Prefix sum of the paged-cache kernels: capped, so that no word of device memory makes it wrap.
#pragma once

#include "device_util.h"
#include "kv_index.h"

namespace rax {

// inclusive, with all lanes active: wave_inclusive_scan's lane moves with the capped sum
template <int CTRL, int ROWS> __device__ __forceinline__ int sat_step(int x) {
  return sat_add(x, __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ int wave_sat_scan(int x) {
  x = sat_step<0x111, 0xf>(x);   // row_shr:1
  x = sat_step<0x112, 0xf>(x);   // row_shr:2
  x = sat_step<0x114, 0xf>(x);   // row_shr:4
  x = sat_step<0x118, 0xf>(x);   // row_shr:8
  x = sat_step<0x142, 0xa>(x);   // row_bcast:15, rows 1 and 3
  return sat_step<0x143, 0xc>(x);   // row_bcast:31, rows 2 and 3
}

}  // namespace rax
