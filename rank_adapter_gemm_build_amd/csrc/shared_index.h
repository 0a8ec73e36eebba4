// Index arithmetic of the shared attention, for the kernels and the host (and run on the host by the CPU
// tests).  Every function takes what comes from device memory as it is and returns a range in bounds.
#pragma once

#include "kv_index.h"

namespace rax {

// The group of sequence i, or -1: the last g in [0, groups) with start[g] <= i, if i < start[g + 1].  start
// holds values in [0, num_seqs].
RAX_HD int group_of(const int* start, int groups, int i) {
  int lo = -1, hi = groups;   // start[lo] <= i < start[hi], were they rising
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= i) lo = mid; else hi = mid;
  }
  return lo >= 0 && i < start[lo + 1] ? lo : -1;
}

// The first key of a sequence's own line: the number of common tokens where it takes part (its new tokens
// come after them all), else 0.
RAX_HD int own_from(const SeqRows& s, int common, int max_len) {
  const int c = clamp_int(common, 0, max_len);
  return s.n > 0 && s.len - s.n >= c ? c : 0;
}
// what seq_span and token_keys are for a sequence's keys from `from` on (no window)
RAX_HD SeqSpan own_span(const SeqRows& s, int from, int step_log2) {
  SeqSpan x{0u, 0};
  if (s.n <= 0) return x;
  x.base = (unsigned)from & ~15u;
  const unsigned hi = (unsigned)token_keys(s.n - 1, s.n, s.len, 0).hi, span = hi > x.base ? hi - x.base : 0u;
  x.steps = (int)((span + ((1u << step_log2) - 1u)) >> step_log2);
  if (x.steps < 1) x.steps = 1;
  return x;
}
RAX_HD KeyRange own_keys(int i, const SeqRows& s, int from) {
  KeyRange k = token_keys(i, s.n, s.len, 0);
  k.lo = from;
  return k;
}
// the common tokens of a group, for all of its rows; none if no sequence takes part
RAX_HD SeqSpan common_span(const SeqRows& s, int step_log2) {
  SeqSpan x{0u, 0};
  if (s.n > 0 && s.len > 0) x.steps = (int)(((unsigned)s.len + ((1u << step_log2) - 1u)) >> step_log2);
  return x;
}

// The units of a group cut in even parts of at most `most` steps: their number, and the steps of a part.
struct EvenParts {
  int parts, steps;
};
RAX_HD EvenParts even_parts(int steps, int most) {
  EvenParts x{0, 1};
  if (steps > 0) {
    x.parts = (int)(((unsigned)steps + (unsigned)most - 1u) / (unsigned)most);
    x.steps = (int)(((unsigned)steps + (unsigned)x.parts - 1u) / (unsigned)x.parts);
    x.parts = (int)(((unsigned)steps + (unsigned)x.steps - 1u) / (unsigned)x.steps);   // none is empty
  }
  return x;
}
// The i-th size tried for them, from the least possible one to an eighth more.
RAX_HD int even_most(int work, int workers, int i) {
  const int least = (int)(((unsigned)work + (unsigned)workers - 1u) / (unsigned)workers);
  return least + (int)(((long long)least * i) >> 9);
}

// Workgroups of the two lines in a launch of `grid` (a multiple of the dies), and the first of the own line's.  Where both
// fit side by side each has its own workgroups; where one needs less than half of the grid it gets what it needs
// and the other the rest; else every workgroup has a share of both.  common_min, own_min: least steps of a workgroup; a short
// common line has up to kFewShares workgroups all the same: the chip has room for them, and the merge joins what they cut (160
// rows a kv head over 200 / 3000 common tokens, bf16, 28 / 31 us at the least steps, 15 / 20 so; 112 rows over 20 in fp32 heads of
// 256 46 and 19).
constexpr int kFewShares = 256;
struct LineSplit {
  int common, own, own_at;
};

RAX_HD LineSplit split_lines(int common_work, int common_min, int own_work, int own_min, int grid) {
  LineSplit s;
  const int few = common_work < kFewShares ? common_work : kFewShares, least = (int)(((long long)common_work + common_min - 1) / common_min);
  const int c = least > few ? least : few, o = (int)(((long long)own_work + own_min - 1) / own_min);
  s.common = c < grid ? c : grid;
  s.own = o < grid ? o : grid;
  s.own_at = 0;
  if (whole_dies(s.common) + whole_dies(s.own) <= grid || 2 * whole_dies(s.common) < grid) {
    s.own_at = whole_dies(s.common);
    if (s.own > grid - s.own_at) s.own = grid - s.own_at;
  } else if (2 * whole_dies(s.own) < grid) {
    s.own_at = grid - whole_dies(s.own);
    s.common = s.own_at;
  }
  return s;
}

}  // namespace rax
