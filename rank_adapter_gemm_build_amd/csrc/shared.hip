// Shared attention over a bf16 cache, the choice of the cache type's kernels, and the merge of a row's two results.
#include "shared_kernels.h"

#include <algorithm>

namespace rax {

template hipError_t launch_shared_of<uint16_t>(const SharedArgs&, hipStream_t, const KTimer&);
extern template hipError_t launch_shared_of<uint8_t>(const SharedArgs&, hipStream_t, const KTimer&);
extern template hipError_t launch_shared_of<float>(const SharedArgs&, hipStream_t, const KTimer&);

hipError_t launch_shared_attention(const SharedArgs& s, hipStream_t stream, const KTimer& tm) {
  if (s.a.dtype == LORA_F32) return launch_shared_of<float>(s, stream, tm);
  if (s.a.c.dtype == LORA_FP8E4M3) return launch_shared_of<uint8_t>(s, stream, tm);
  return launch_shared_of<uint16_t>(s, stream, tm);
}

// The rows of a sequence that shares: a workgroup takes every gridDim.y-th of its tokens, 4 dims a thread and step.
template <typename T> __global__ __launch_bounds__(256) void shared_merge_kernel(SharedArgs s, FastDiv per_head) {
  const AttentionArgs& a = s.a;
  const int r = blockIdx.x, D = a.c.dim, chunks = D / 4;
  if (s.from[r] == 0) return;
  const SeqRows x = seq_rows(a.query_start[r], a.query_start[r + 1], a.seq_lens[r], a.num_tokens, a.max_pages << a.c.page_shift);
  const float2 *ml1 = reinterpret_cast<const float2*>(s.common_line.state_ml), *ml2 = reinterpret_cast<const float2*>(s.own_line.state_ml);
  for (int i = blockIdx.y; i < x.n; i += gridDim.y)
    for (int e = threadIdx.x; e < a.q_heads * chunks; e += 256) {
      const int h = fast_quot(e, per_head), d = (e - h * chunks) * 4;
      const size_t row = (size_t)(x.start + i) * a.q_heads + h;
      const float2 u = ml1[row], v = ml2[row];
      const f32x4_t p = *reinterpret_cast<const f32x4_t*>(s.common_line.state_o + row * D + d);
      const f32x4_t q = *reinterpret_cast<const f32x4_t*>(s.own_line.state_o + row * D + d);
      const float m = fmaxf(u.x, v.x), f1 = __builtin_amdgcn_exp2f(u.x - finite_top(m)), f2 = __builtin_amdgcn_exp2f(v.x - finite_top(m));
      const float l = u.y * f1 + v.y * f2;
      write4(reinterpret_cast<T*>(a.out) + (size_t)(x.start + i) * a.ldo + (size_t)h * D + d,
             (p * f1 + q * f2) * (l == 0.f ? 0.f : over_sum(a.c.v_scale, l)));
      if (a.lse && d == 0) a.lse[row] = log_sum(m, l);
    }
}

hipError_t launch_shared_merge(const SharedArgs& s, hipStream_t stream, const KTimer& tm) {
  const dim3 grid(s.a.num_seqs, std::min(64, std::max(1, (s.a.num_tokens + s.a.num_seqs - 1) / s.a.num_seqs)));
  const FastDiv per_head = fast_div(s.a.c.dim / 4);
  if (s.a.dtype == LORA_F32) RAX_LAUNCH(tm, shared_merge_kernel<float>, grid, dim3(256), 0u, stream, s, per_head);
  else RAX_LAUNCH(tm, shared_merge_kernel<uint16_t>, grid, dim3(256), 0u, stream, s, per_head);
  return hipGetLastError();
}

}  // namespace rax
