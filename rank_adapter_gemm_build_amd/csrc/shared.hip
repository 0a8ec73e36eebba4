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

// A workgroup takes every gridDim.y-th token of a sequence, and 256 / S chunks of 4 dims of its heads; S threads have every
// S-th kJoin of the parts of a chunk and join theirs in LDS.
template <typename T, int S> __global__ __launch_bounds__(256) void shared_merge_kernel(SharedArgs s, FastDiv per_head) {
  constexpr int kChunks = 256 / S;
  __shared__ float4 o_s[S > 1 ? S : 1][S > 1 ? kChunks : 1];
  __shared__ float2 ml_s[S > 1 ? S : 1][S > 1 ? kChunks : 1];
  const AttentionArgs& a = s.a;
  const LinePlan plan = *s.plan;
  const SeqPlan q = s.seqs[blockIdx.x];
  if (plan.own_work == 0) return;
  const int D = a.c.dim, chunks = D / 4, group = a.group_size, e = (int)(blockIdx.z * kChunks + threadIdx.x % kChunks), slice = threadIdx.x / kChunks;
  const int h = fast_quot(e, per_head), d = (e - h * chunks) * 4, kh = fast_quot(h, a.group), hg = h - kh * group;
  const bool there = h < a.q_heads;
  const SeqRows x = seq_rows(a.query_start[blockIdx.x], a.query_start[blockIdx.x + 1], a.seq_lens[blockIdx.x], a.num_tokens,
                             a.max_pages << a.c.page_shift);
  const GroupPlan g = s.groups[q.group];
  float m, l;
  f32x4_t o;
  const auto add = [&](const float2* y, const f32x4_t* v, int n) {   // n results, in order
    float top = m;
    for (int k = 0; k < n; ++k) top = fmaxf(top, y[k].x);
    const float keep = __builtin_amdgcn_exp2f(m - finite_top(top));
    l *= keep;
    o *= keep;
    for (int k = 0; k < n; ++k) {
      const float f = __builtin_amdgcn_exp2f(y[k].x - finite_top(top));
      l += y[k].y * f;
      o += v[k] * f;
    }
    m = top;
  };
  // a row of a unit whose first step is `at`: its state, or its parts, kJoin at a time
  const auto add_unit = [&](const LineShape& line, int at, int steps, int work, int workers, int lrow, size_t row) {
    const int first = share_owner(work, workers, at), parts = share_owner(work, workers, at + steps - 1) - first + 1;
    if (parts == 1) {
      if (slice > 0) return;
      const float2 y = reinterpret_cast<const float2*>(line.state_ml)[row];
      const f32x4_t v = *reinterpret_cast<const f32x4_t*>(line.state_o + row * D + d);
      add(&y, &v, 1);
      return;
    }
    const auto part_o = cells_at(reinterpret_cast<const char*>(line.part_o), true);   // below 2^31 bytes
    const auto part_ml = cells_at(reinterpret_cast<const char*>(line.part_ml), true);
    for (int k0 = slice * kJoin; k0 < parts; k0 += S * kJoin) {
      float2 y[kJoin];
      f32x4_t v[kJoin];
#pragma unroll
      for (int k = 0; k < kJoin; ++k) {
        const uint32_t p = ((uint32_t)part_slot(first, k0 + k) << line.rows_log2) + (uint32_t)lrow;
        y[k] = __builtin_bit_cast(float2, load_words<2, 0>(part_ml, k0 + k < parts ? p * 8 : kNowhere, 0));
        v[k] = __builtin_bit_cast(f32x4_t, load_words<4, 0>(part_o, k0 + k < parts ? (p * D + d) * 4 : kNowhere, 0));
        if (k0 + k >= parts) y[k].x = -INFINITY;
      }
      add(y, v, kJoin);
    }
  };
  const int own_steps = own_span(x, q.from, s.own_line.step_log2).steps, own_blocks = row_blocks(x.n, group, s.own_line.rows_log2);
  const int common_blocks = row_blocks(g.n, group, s.common_line.rows_log2);
  for (int i = blockIdx.y; i < x.n; i += gridDim.y) {
    const size_t row = (size_t)(x.start + i) * a.q_heads + h;
    m = -INFINITY;
    l = 0.f;
    o = f32x4_t{0.f, 0.f, 0.f, 0.f};
    const int own_row = i * group + hg, own_at = q.at + (kh * own_blocks + (own_row >> s.own_line.rows_log2)) * own_steps;
    // else written by the first launch
    const bool mine = there && !(q.from == 0 && share_owner(plan.own_work, plan.own_workers, own_at) ==
                                                    share_owner(plan.own_work, plan.own_workers, own_at + own_steps - 1));
    const int r = (x.start + i - g.start) * group + hg;   // of the group's rows, unless sequences overlap
    if (mine && q.from > 0 && r >= 0 && r < g.n * group) {
      add_unit(s.common_line, g.at + (kh * common_blocks + (r >> s.common_line.rows_log2)) * g.steps, g.steps, plan.common_work,
               plan.common_workers, r & ((1 << s.common_line.rows_log2) - 1), row);
    }
    if (mine) add_unit(s.own_line, own_at, own_steps, plan.own_work, plan.own_workers, own_row & ((1 << s.own_line.rows_log2) - 1), row);
    if constexpr (S > 1) {
      const int c = threadIdx.x % kChunks;
      if (slice > 0) {
        o_s[slice][c] = make_float4(o[0], o[1], o[2], o[3]);
        ml_s[slice][c] = make_float2(m, l);
      }
      __syncthreads();
      if (slice == 0) {
        float2 y[S - 1];
        f32x4_t v[S - 1];
#pragma unroll
        for (int k = 1; k < S; ++k) {
          y[k - 1] = ml_s[k][c];
          v[k - 1] = f32x4_t{o_s[k][c].x, o_s[k][c].y, o_s[k][c].z, o_s[k][c].w};
        }
        add(y, v, S - 1);
      }
      __syncthreads();
    }
    if (!mine || slice > 0) continue;
    write4(reinterpret_cast<T*>(a.out) + (size_t)(x.start + i) * a.ldo + (size_t)h * D + d, o * (l == 0.f ? 0.f : over_sum(a.c.v_scale, l)));
    if (a.lse && d == 0) a.lse[row] = log_sum(m, l);
  }
}

constexpr long long kMergeSplit = 1 << 14;   // most chunks of such rows

hipError_t launch_shared_merge(const SharedArgs& s, hipStream_t stream, const KTimer& tm) {
  const int tokens = (s.a.num_tokens + s.a.num_seqs - 1) / s.a.num_seqs;
  const FastDiv per_head = fast_div(s.a.c.dim / 4);
  const int chunks = s.a.q_heads * s.a.c.dim / 4;
  // Few rows: their parts may be many, and the chip has room (32 heads of 128: one sequence of 131071 tokens 38 us with a
  // thread a chunk, 8 with eight; 16 rows over 8000 common tokens 9.5 and 6.4; 64 rows with few parts 5.5 and 10)
  const bool split = (long long)s.a.num_tokens * chunks <= kMergeSplit;
  const dim3 grid(s.a.num_seqs, std::min(64, std::max(1, tokens)), split ? (chunks + 31) / 32 : (chunks + 255) / 256);
  const auto launch = [&](auto kernel) { RAX_LAUNCH(tm, kernel, grid, dim3(256), 0u, stream, s, per_head); };
  if (s.a.dtype == LORA_F32) split ? launch(shared_merge_kernel<float, 8>) : launch(shared_merge_kernel<float, 1>);
  else split ? launch(shared_merge_kernel<uint16_t, 8>) : launch(shared_merge_kernel<uint16_t, 1>);
  return hipGetLastError();
}

}  // namespace rax
