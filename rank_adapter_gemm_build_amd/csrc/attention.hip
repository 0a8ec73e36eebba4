// Paged attention: out = softmax(scale q K^T) V over the cached keys a token sees, in one
// pass over the keys with a running maximum m and sum l: for a batch of scores s_j,
//   m' = max(m, max_j s_j),  l' = l e^(m - m') + sum_j e^(s_j - m'),
//   o' = o e^(m - m') + sum_j e^(s_j - m') v_j,   out = o / l.
#include <hip/hip_runtime.h>

#include <cmath>

#include "device_util.h"
#include "kv.h"

namespace rax {

__device__ __forceinline__ float cell_f32(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ float cell_f32(float v) { return v; }
__device__ __forceinline__ float cell_f32(uint8_t v) { return __builtin_amdgcn_cvt_f32_fp8((int)v, 0); }

// One wave per (new token, query head); 64 keys at a time, one per lane for the scores,
// then the lanes own the head's values (4 each at most).
template <typename T, typename C>
__global__ __launch_bounds__(64) void paged_attention_kernel(AttentionArgs a) {
  const int t = blockIdx.x, h = blockIdx.y, lane = threadIdx.x, D = a.c.dim;
  const int ps = a.c.page_shift, max_len = a.max_pages << ps;
  int r = -1;
  SeqRows s{};
  for (int b = 0; b < a.num_seqs && r < 0; b += 64) {
    const int i = b + lane;
    SeqRows x{};
    if (i < a.num_seqs) x = seq_rows(a.query_start[i], a.query_start[i + 1], a.seq_lens[i], a.num_tokens, max_len);
    const unsigned long long m = __ballot(i < a.num_seqs && x.n > 0 && t >= x.start && t < x.start + x.n);
    if (m) {
      const int src = __ffsll((long long)m) - 1;
      r = b + src;
      s.start = __shfl(x.start, src);
      s.n = __shfl(x.n, src);
      s.len = __shfl(x.len, src);
    }
  }
  if (r < 0) return;
  const KeyRange keys = token_keys(t - s.start, s.n, s.len, a.window);
  const int kh = h / (a.q_heads / a.c.heads);
  const T* q = reinterpret_cast<const T*>(a.q) + (size_t)t * a.ldq + (size_t)h * D;
  const C* K = reinterpret_cast<const C*>(a.c.k) + kh * a.c.head_stride;
  const C* V = reinterpret_cast<const C*>(a.c.v) + kh * a.c.head_stride;
  const int32_t* table = a.table + (size_t)r * a.ld_table;
  const bool f8 = sizeof(C) == 1;
  const float ks = f8 ? a.c.k_scale : 1.f, vs = f8 ? a.c.v_scale : 1.f;
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j0 = keys.lo; j0 < keys.hi; j0 += 64) {
    const int j = j0 + lane;
    int page = -1;
    if (j < keys.hi) page = page_or_none(table[j >> ps], a.c.num_pages);
    const long long at = (long long)page * a.c.page_stride + (j & ((1 << ps) - 1)) * a.c.token_stride;
    float sc = -INFINITY;
    if (page >= 0) {
      float dot = 0.f;
      for (int d = 0; d < D; ++d) dot = fmaf(cell_f32(q[d]), cell_f32(K[at + d]), dot);
      sc = dot * ks * a.scale;
    }
    float mx = sc;
    for (int d = 32; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
    const float mn = fmaxf(m, mx);
    if (mn == -INFINITY) continue;
    const float alpha = __expf(m - mn);
    const float p = page >= 0 ? __expf(sc - mn) : 0.f;
    m = mn;
    l = l * alpha + p;
    for (int i = 0; i < 4; ++i) o[i] *= alpha;
    unsigned long long there = __ballot(page >= 0);
    while (there) {
      const int src = __ffsll((long long)there) - 1;
      there &= there - 1;
      const float pj = __shfl(p, src);
      const long long aj = __shfl(at, src);
      for (int i = 0; i < 4; ++i)
        if (lane + 64 * i < D) o[i] = fmaf(pj, cell_f32(V[aj + lane + 64 * i]), o[i]);
    }
  }
  for (int d = 32; d >= 1; d >>= 1) l += __shfl_xor(l, d);
  T* out = reinterpret_cast<T*>(a.out) + (size_t)t * a.ldo + (size_t)h * D;
  const float inv = m == -INFINITY ? 0.f : vs / l;
  for (int i = 0; i < 4; ++i)
    if (lane + 64 * i < D) {
      if constexpr (sizeof(T) == 4) out[lane + 64 * i] = o[i] * inv;
      else out[lane + 64 * i] = (uint16_t)f32_to_bf16(o[i] * inv);
    }
  if (a.lse && lane == 0) a.lse[(size_t)t * a.q_heads + h] = m == -INFINITY ? -INFINITY : m + logf(l);
}

hipError_t launch_paged_attention(const AttentionArgs& a, hipStream_t stream, const KTimer& tm) {
  const dim3 grid(a.num_tokens, a.q_heads), block(64);
  if (a.dtype == LORA_F32)
    RAX_LAUNCH(tm, (paged_attention_kernel<float, float>), grid, block, 0u, stream, a);
  else if (a.c.dtype == LORA_FP8E4M3)
    RAX_LAUNCH(tm, (paged_attention_kernel<uint16_t, uint8_t>), grid, block, 0u, stream, a);
  else
    RAX_LAUNCH(tm, (paged_attention_kernel<uint16_t, uint16_t>), grid, block, 0u, stream, a);
  return hipGetLastError();
}

}  // namespace rax
