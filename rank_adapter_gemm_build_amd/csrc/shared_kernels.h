// Shared attention: sequences of a group have their first tokens in common pages, and those are read once
// for all of them.  With the common keys' (m1, l1, o1) of a row and its own keys' (m2, l2, o2), maxima, sums of
// 2^(s - m) and sums of weighted values as in the paged attention,
//   m = max(m1, m2), f_i = 2^(m_i - m), out = (f1 o1 + f2 o2) / (f1 l1 + f2 l2), lse = (m + log2(f1 l1 + f2 l2)) ln 2.
//
// Two lines of steps as in the paged attention, in one launch: one of the groups, whose "sequence" has the rows of all
// its members and the common keys, all of which every row sees; one of the sequences with the keys from there on.  A launch
// after it joins what the rows have in the workspace: parts of units that several shares had, and the results of the two
// lines.  (The parts are large, and a tree in the first launch, as the paged attention has it, would add them in few
// workgroups: 64 rows a head over 8000 common tokens 77 us, of them 45 in the tree.)  A whole unit of a sequence that
// shares nothing writes its output at once.
//
// Where both lines are long each workgroup has a share of both, half of them in the other order, so that on a compute unit
// the products of one go with the loads of the other.  Own keys are often few: each wave takes shares of the own line by
// itself, with no join in the workgroup (192 sequences of 150 own keys 52 -> 30 us).
//
// What bounds it: reading the keys and values once; with many rows the common line's products.  Measured (32 query and 8 kv
// heads of 128, both launches): 4 sequences with 704 common tokens 17 us; 24 groups of 8 with 1000 to 6000 in e4m3 80 (bytes
// 39); 64 sequences with 8000 69 to 72 (26); 256 with 32000 390 to 399 (206).  With wide blocks and heads of 128 registers spill in
// e4m3 (17 to 19) and, where sequences have many rows, in bf16 (30).
#pragma once

#include "attention_kernels.h"
#include "shared.h"
#include "wide_kernels.h"

namespace rax {

struct OwnLine {
  static constexpr bool kState = true, kTree = false;
  const SharedArgs& s;
  const int* from_s;
  __device__ __forceinline__ int from(int r) const { return uniform(from_s[r]); }
  __device__ __forceinline__ int count() const { return s.a.num_seqs; }
  __device__ __forceinline__ SeqRows rows(int r, int max_len) const {
    const const_words_t lens = const_words(s.a.seq_lens), starts = const_words(s.a.query_start);
    return seq_rows(starts[r], starts[r + 1], lens[r], s.a.num_tokens, max_len);
  }
  __device__ __forceinline__ SeqSpan span(int r, const SeqRows& x, int step_log2) const { return own_span(x, from(r), step_log2); }
  __device__ __forceinline__ KeyRange keys(int r, int i, const SeqRows& x) const { return own_keys(i, x, from(r)); }
  __device__ __forceinline__ int table_row(int r) const { return r; }
  __device__ __forceinline__ bool state(int r) const { return from(r) > 0; }
  __device__ __forceinline__ float* state_o() const { return s.own_line.state_o; }
  __device__ __forceinline__ float* state_ml() const { return s.own_line.state_ml; }
  __device__ __forceinline__ float* part_o() const { return s.own_line.part_o; }
  __device__ __forceinline__ float* part_ml() const { return s.own_line.part_ml; }
};

struct CommonLine {
  static constexpr bool kState = true, kTree = false;
  const SharedArgs& s;
  const int *group_s, *common_s, *lead_s;   // first sequence, common tokens, first member that takes part
  const int* even_s;                        // steps that count as one, where units are cut evenly
  __device__ __forceinline__ int count() const { return s.num_groups; }
  __device__ __forceinline__ SeqRows rows(int g, int max_len) const {
    const const_words_t starts = const_words(s.a.query_start);
    return seq_rows(starts[uniform(group_s[g])], starts[uniform(group_s[g + 1])], uniform(common_s[g]), s.a.num_tokens, max_len);
  }
  __device__ __forceinline__ int merged(int g) const { return even_s ? uniform(even_s[g]) : 1; }
  __device__ __forceinline__ SeqSpan span(int g, const SeqRows& x, int step_log2) const {
    SeqSpan y = common_span(x, step_log2);
    if (even_s) y.steps = (int)(((unsigned)y.steps + (unsigned)merged(g) - 1u) / (unsigned)merged(g));
    return y;
  }
  __device__ __forceinline__ KeyRange keys(int, int, const SeqRows& x) const { return KeyRange{0, x.len}; }
  __device__ __forceinline__ int table_row(int g) const { return uniform(lead_s[g]); }
  __device__ __forceinline__ bool state(int) const { return true; }
  __device__ __forceinline__ float* state_o() const { return s.common_line.state_o; }
  __device__ __forceinline__ float* state_ml() const { return s.common_line.state_ml; }
  __device__ __forceinline__ float* part_o() const { return s.common_line.part_o; }
  __device__ __forceinline__ float* part_ml() const { return s.common_line.part_ml; }
};

// Steps before this thread's run of `mine`, and the whole line's, from the scans of all waves
struct LineSums {
  int before, work;
};
__device__ __forceinline__ LineSums line_sums(int scan, int mine, const int* waves, int stride, int w) {
  LineSums x{scan - mine, 0};
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    if (v < w) x.before += waves[v * stride];
    x.work = sat_add(x.work, waves[v * stride]);
  }
  x.work = uniform(x.work);
  return x;
}

// SRT, SRW: row tiles and row waves of the own line, SRW = 0: one wave a share; PRT, PRW: of the common line, PRW = 4: wide
// blocks; ONCE: the own line's cells pass the caches as a stream
template <typename C, int DB, int RT, int RW> constexpr int line_lds() {   // 16-byte units
  if constexpr (RW == 4) return wide_lds<DB>() / 16;
  else if constexpr (RW == 0) return 0;
  else return join_lds<C, DB, RT, 4, RW>();
}
template <typename C, int DB, int SRT, int SRW, int PRT, int PRW, bool ONCE>
__global__ __launch_bounds__(256, DB > 128 ? 1 : 2) void shared_attention_kernel(SharedArgs s) {
  constexpr int kThreads = 256, kOwnRows = SRW == 0 ? 4 : 4 + SRT / 2 + SRW / 2, kCommonRows = PRW == 4 ? kWideRowsLog2 : 4 + PRT / 2 + PRW / 2;
  constexpr int kOwnLds = line_lds<C, DB, SRT, SRW>(), kCommonLds = line_lds<C, DB, PRT, PRW>(), kJoinUnits = kOwnLds > kCommonLds ? kOwnLds : kCommonLds;
  extern __shared__ float4 lds[];
  __shared__ int part_s[4][2];
  __shared__ int units_s[kEvenGroups], steps_s[kEvenGroups], even_s[kEvenGroups];   // wide units: of each group, their steps, steps that count as one
  const AttentionArgs& a = s.a;
  const int n = a.num_seqs, groups = s.num_groups, max_len = a.max_pages << a.c.page_shift, group = a.group_size;
  const int tid = threadIdx.x, lane = lane_id(), w = uniform(tid >> 6);
  int *own_sums = reinterpret_cast<int*>(lds + kJoinUnits), *from_s = own_sums + n, *common_sums = from_s + n,
      *lead_s = common_sums + groups, *common_s = lead_s + groups, *group_s = common_s + groups;   // group_s: one longer

  // ---- groups, then the sequences' own line, then the common one
  constexpr int kOwnWaves = SRW == 0 ? 4 : 1;   // shares of the own line that a workgroup has
  for (int g = tid; groups > 0 && g <= groups; g += kThreads) {
    group_s[g] = clamp_int(s.group_start[g], 0, n);
    if (g < groups) {
      common_s[g] = clamp_int(s.common[g], 0, max_len);
      lead_s[g] = n;
    }
  }
  lds_barrier();
  const int per = (n + kThreads - 1) / kThreads, r0 = min(n, tid * per), r1 = min(n, r0 + per);
  int own = 0;
  for (int i = r0; i < r1; ++i) {
    const SeqRows x = seq_rows(a.query_start[i], a.query_start[i + 1], a.seq_lens[i], a.num_tokens, max_len);
    const int g = group_of(group_s, groups, i), from = g >= 0 ? own_from(x, common_s[g], max_len) : 0;
    const long long all = (long long)(a.c.heads * row_blocks(x.n, group, kOwnRows)) * own_span(x, from, s.own_line.step_log2).steps;
    from_s[i] = from;
    if (from > 0) (void)__hip_atomic_fetch_min(lead_s + g, i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    own_sums[i] = own;
    own = sat_add(own, all < kPlanCap ? (int)all : kPlanCap);
  }
  lds_barrier();
  const int gper = (groups + kThreads - 1) / kThreads, g0 = min(groups, tid * gper), g1 = min(groups, g0 + gper);
  int common = 0;
  for (int g = g0; g < g1; ++g) {
    if (lead_s[g] >= n) lead_s[g] = common_s[g] = 0;   // no sequence takes part (read by others before the last barrier only)
    const SeqRows x = seq_rows(a.query_start[group_s[g]], a.query_start[group_s[g + 1]], common_s[g], a.num_tokens, max_len);
    const int units = a.c.heads * row_blocks(x.n, group, kCommonRows), steps = common_span(x, s.common_line.step_log2).steps;
    const long long all = (long long)units * steps;
    if (PRW == 4 && g < kEvenGroups) {
      units_s[g] = units;
      steps_s[g] = steps;
    }
    common_sums[g] = common;
    common = sat_add(common, all < kPlanCap ? (int)all : kPlanCap);
  }
  const int own_scan = wave_sat_scan(own), common_scan = wave_sat_scan(common);
  if (lane == 63) {
    part_s[w][0] = own_scan;
    part_s[w][1] = common_scan;
  }
  lds_barrier();
  const LineSums o = line_sums(own_scan, own, &part_s[0][0], 2, w);
  LineSums c = line_sums(common_scan, common, &part_s[0][1], 2, w);
  // no work, or more than the host counted with: sequences that overlap (the sums are capped)
  const bool fits = o.work < kPlanCap && c.work < kPlanCap;
  const int grid = (int)gridDim.x, block = (int)blockIdx.x;
  LineSplit split = split_lines(c.work, s.common_line.min_steps, o.work, kOwnWaves * s.own_line.min_steps, grid);
  const int own_workers = min(kOwnWaves * split.own, (o.work + s.own_line.min_steps - 1) / s.own_line.min_steps);
  for (int i = r0; i < r1; ++i) own_sums[i] += o.before;
  // Wide units of one head, whose workgroups should read the same keys at the same time, are cut in even parts where that
  // costs at most an eighth more for the largest share: the least of 64 sizes with which there are workgroups for all parts.
  bool even = false;
  if (PRW == 4 && groups <= kEvenGroups && fits && c.work > 0) {
    const int most = even_most(c.work, split.common, lane);
    long long shares = 0;
    for (int g = 0; g < groups; ++g) shares += (long long)units_s[g] * even_parts(steps_s[g], most).parts;
    const uint64_t good = __builtin_amdgcn_ballot_w64(shares <= split.common);
    even = good != 0;
    if (even) {
      const int size = even_most(c.work, split.common, __builtin_ctzll(good));
      c = LineSums{0, 0};
      for (int g = 0; g < groups; ++g) {
        const EvenParts y = even_parts(steps_s[g], size);
        if (g < g0) c.before += units_s[g] * y.parts;
        if (g == tid) even_s[g] = y.steps;
        if (g >= g0 && g < g1) common_sums[g] = 0;
        c.work += units_s[g] * y.parts;
      }
      c.work = split.common = uniform(c.work);
    }
  }
  for (int g = g0; g < g1; ++g) common_sums[g] += c.before;
  if (block == 0) {   // for the merge
    if (tid == 0) *s.plan = fits ? LinePlan{c.work, split.common, o.work, own_workers} : LinePlan{0, 0, 0, 0};
    for (int i = r0; i < r1; ++i) s.seqs[i] = SeqPlan{from_s[i], own_sums[i], from_s[i] > 0 ? group_of(group_s, groups, i) : 0, 0};
    for (int g = g0; g < g1; ++g) {
      const SeqRows x = seq_rows(a.query_start[group_s[g]], a.query_start[group_s[g + 1]], common_s[g], a.num_tokens, max_len);
      const int steps = common_span(x, s.common_line.step_log2).steps;
      s.groups[g] = GroupPlan{common_sums[g], even ? (int)(((unsigned)steps + (unsigned)even_s[g] - 1u) / (unsigned)even_s[g]) : steps, x.start, x.n};
    }
  }
  if (!fits || o.work == 0) return;
  const int bc = split.common > 0 ? share_of_block(block, split.common) : split.common;
  const int bo = block >= split.own_at ? share_of_block(block - split.own_at, split.own) : split.own;
  if (bc >= split.common && bo >= split.own) return;
  lds_barrier();
  const OwnLine own_line{s, from_s};
  const CommonLine common_line{s, group_s, common_s, lead_s, even ? even_s : nullptr};
  const bool own_first = 2 * block >= grid;
#pragma unroll 1
  for (int turn = 0; turn < 2; ++turn) {
    if ((turn == 0) == own_first) {
      if constexpr (SRW == 0) {
        if (bo < split.own && 4 * bo + w < own_workers)
          attend_shares<C, DB, SRT, 1, 1, ONCE>(a, own_line, lds, own_sums, 4 * bo + w, o.work, own_workers, s.own_line.step_log2);
        lds_barrier();   // the waves are together again
      } else {
        if (bo < split.own) attend_shares<C, DB, SRT, 4, SRW, ONCE>(a, own_line, lds, own_sums, bo, o.work, split.own, s.own_line.step_log2);
      }
    } else {
      if constexpr (PRW == 4) {
        // Those that begin later take precedence on their compute unit over those that have been at it since the start: both
        // end at about the same time (256 sequences with 32000 common tokens 421 -> 402 us).
        if (own_first) __builtin_amdgcn_s_setprio(1);
        if (bc < split.common) attend_wide<C, DB>(a, common_line, lds, common_sums, bc, c.work, split.common, s.common_line.step_log2);
      } else {
        if (bc < split.common) attend_shares<C, DB, PRT, 4, PRW, false>(a, common_line, lds, common_sums, bc, c.work, split.common, s.common_line.step_log2);
      }
    }
  }
}

template <typename C, int DB, int SRT, int SRW, int PRT, int PRW, bool ONCE>
static void launch_shared_shape(const SharedArgs& s, hipStream_t stream, const KTimer& tm) {
  constexpr int own = line_lds<C, DB, SRT, SRW>(), common = line_lds<C, DB, PRT, PRW>();
  RAX_LAUNCH(tm, (shared_attention_kernel<C, DB, SRT, SRW, PRT, PRW, ONCE>), dim3(s.a.workers), dim3(256),
             (uint32_t)(16 * (own > common ? own : common) + sizeof(int) * (2 * s.a.num_seqs + 4 * s.num_groups + 1)), stream, s);
}
template <typename C, int DB> static void launch_shared_lines(const SharedArgs& s, hipStream_t stream, const KTimer& tm) {
  const bool once = s.a.read_once != 0;
  if constexpr (sizeof(C) < 4 && DB <= 128) {
    if (s.common_line.row_waves == 4) {
      if (s.own_line.row_tiles == 2) launch_shared_shape<C, DB, 2, 2, 1, 4, false>(s, stream, tm);
      else if (once) launch_shared_shape<C, DB, 1, 0, 1, 4, true>(s, stream, tm);
      else launch_shared_shape<C, DB, 1, 0, 1, 4, false>(s, stream, tm);
      return;
    }
  }
  if constexpr (DB > 128) {
    if (s.own_line.row_waves == 2) launch_shared_shape<C, DB, 1, 2, 1, 2, false>(s, stream, tm);
    else if (once) launch_shared_shape<C, DB, 1, 0, 1, 2, true>(s, stream, tm);
    else launch_shared_shape<C, DB, 1, 0, 1, 2, false>(s, stream, tm);
  }
  if constexpr (sizeof(C) == 4 && DB <= 128) {
    if (s.common_line.row_waves == 2 && s.own_line.row_tiles == 1) {
      if (once) launch_shared_shape<C, DB, 1, 0, 2, 2, true>(s, stream, tm);
      else launch_shared_shape<C, DB, 1, 0, 2, 2, false>(s, stream, tm);
      return;
    }
  }
  if constexpr (DB <= 128) {
    if (s.own_line.row_tiles == 2) launch_shared_shape<C, DB, 2, 2, 2, 2, false>(s, stream, tm);
    else if (once) launch_shared_shape<C, DB, 1, 0, 2, 1, true>(s, stream, tm);
    else launch_shared_shape<C, DB, 1, 0, 2, 1, false>(s, stream, tm);
  }
}
template <typename C> hipError_t launch_shared_of(const SharedArgs& s, hipStream_t stream, const KTimer& tm) {
  if (s.a.c.dim <= 64) launch_shared_lines<C, 64>(s, stream, tm);
  else if (s.a.c.dim <= 128) launch_shared_lines<C, 128>(s, stream, tm);
  else launch_shared_lines<C, 256>(s, stream, tm);
  return hipGetLastError();
}

}  // namespace rax
