// Rotary append: the rotary turn of a step's q and k heads, and its keys and values into
// the paged cache.
//
// Pair i of a head at position p turns by the angle p f_i: (a, b) -> amplitude * (a cos -
// b sin, a sin + b cos).  f_i is kept in turns a position in 64 bits, so the angle's whole
// turns drop out exactly (p f_i - round(p f_i)) and the remaining fraction, at most half a
// turn, is good to 2^-26 of a turn in fp32 at any 31-bit position.
#include <hip/hip_runtime.h>

#include "device_util.h"
#include "kv.h"

namespace rax {

constexpr int kRotaryThreads = 256;

__device__ __forceinline__ float load_act(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ float load_act(const float* p) { return *p; }
__device__ __forceinline__ void store_act(uint16_t* p, float v) { *p = (uint16_t)f32_to_bf16(v); }
__device__ __forceinline__ void store_act(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_cell(uint16_t* p, float v, float) { store_act(p, v); }
__device__ __forceinline__ void store_cell(float* p, float v, float) { *p = v; }
__device__ __forceinline__ void store_cell(uint8_t* p, float v, float scale) {
  *p = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(fp8_clamp(v / scale), 0.f, 0, false);
}

// T: activations, C: cache.  One workgroup a token.
template <typename T, typename C>
__global__ __launch_bounds__(kRotaryThreads) void rotary_append_kernel(RotaryArgs a) {
  __shared__ float cs[LORA_MAX_HEAD_DIM / 2], sn[LORA_MAX_HEAD_DIM / 2];
  const int t = blockIdx.x, tid = threadIdx.x, D = a.c.dim, half = a.rot / 2;
  const double p = a.positions[t];
  for (int i = tid; i < half; i += kRotaryThreads) {
    double x = p * a.turns[i];
    x -= rint(x);
    if constexpr (sizeof(T) == 4) {
      double s, c;
      sincospi(2.0 * x, &s, &c);
      cs[i] = (float)c * a.amplitude;
      sn[i] = (float)s * a.amplitude;
    } else {
      float s, c;
      sincospif(2.0f * (float)x, &s, &c);
      cs[i] = c * a.amplitude;
      sn[i] = s * a.amplitude;
    }
  }
  __syncthreads();
  const int slot = a.slots[t], page = slot >> a.c.page_shift, off = slot & ((1 << a.c.page_shift) - 1);
  const bool stored = slot >= 0 && page < a.c.num_pages;
  const long long row = stored ? page * a.c.page_stride + off * a.c.token_stride : 0;
  const T* in = reinterpret_cast<const T*>(a.qkv) + (size_t)t * a.ldqkv;
  T* q = reinterpret_cast<T*>(a.q_out) + (size_t)t * a.ldq;
  C *kc = reinterpret_cast<C*>(a.c.k) + row, *vc = reinterpret_cast<C*>(a.c.v) + row;
  const int turned = a.q_heads + a.c.heads, per = D - half;   // items of a head: pairs, then single values
  for (int e = tid; e < turned * per; e += kRotaryThreads) {
    const int h = e / per, i = e - h * per;
    int d0, d1 = -1;
    float x, y = 0.f;
    if (i < half) {
      d0 = a.interleaved ? 2 * i : i;
      d1 = a.interleaved ? 2 * i + 1 : i + half;
      const float u = load_act(in + h * D + d0), w = load_act(in + h * D + d1);
      x = u * cs[i] - w * sn[i];
      y = u * sn[i] + w * cs[i];
    } else {
      d0 = i + half;
      x = load_act(in + h * D + d0);
    }
    if (h < a.q_heads) {
      store_act(q + h * D + d0, x);
      if (d1 >= 0) store_act(q + h * D + d1, y);
    } else if (stored) {
      C* k = kc + (h - a.q_heads) * a.c.head_stride;
      store_cell(k + d0, x, a.c.k_scale);
      if (d1 >= 0) store_cell(k + d1, y, a.c.k_scale);
    }
  }
  if (stored)
    for (int e = tid; e < a.c.heads * D; e += kRotaryThreads) {
      const int h = e / D, d = e - h * D;
      store_cell(vc + h * a.c.head_stride + d, load_act(in + turned * D + e), a.c.v_scale);
    }
}

hipError_t launch_rotary_append(const RotaryArgs& a, hipStream_t stream, const KTimer& tm) {
  const dim3 grid(a.num_tokens), block(kRotaryThreads);
  if (a.dtype == LORA_F32)
    RAX_LAUNCH(tm, (rotary_append_kernel<float, float>), grid, block, 0u, stream, a);
  else if (a.c.dtype == LORA_FP8E4M3)
    RAX_LAUNCH(tm, (rotary_append_kernel<uint16_t, uint8_t>), grid, block, 0u, stream, a);
  else
    RAX_LAUNCH(tm, (rotary_append_kernel<uint16_t, uint16_t>), grid, block, 0u, stream, a);
  return hipGetLastError();
}

}  // namespace rax
