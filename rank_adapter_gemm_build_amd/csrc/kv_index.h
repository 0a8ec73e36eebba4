// Index arithmetic of the paged cache, shared by the kernels and the host (and run on the
// host by the CPU tests): what a request needs of the ring of free pages, where a key
// lies, which keys a block of query rows sees.  Every function takes what comes from
// device memory (lengths, page ids) as it is and returns a range that stays in bounds.
#pragma once

#include <stdint.h>

#if defined(__HIPCC__)
#define RAX_HD __host__ __device__ __forceinline__
#else
#define RAX_HD inline
#endif

namespace rax {

constexpr int kPlanCap = 1 << 30;   // sums of the page plan saturate here

// a + b for 0 <= a, b <= kPlanCap, capped (an associative sum, so a scan may use it)
RAX_HD int sat_add(int a, int b) { return a < kPlanCap - b ? a + b : kPlanCap; }

struct RequestNeed {
  int n;        // tokens in the batch
  int have;     // pages of the past tokens
  int need;     // pages to draw
  int back;     // pages to give back
  int invalid;  // 1: lengths out of range
  int live;     // 1: gets its tokens into the cache if its pages are granted
};

// max_pages << page_shift fits 31 bits
RAX_HD RequestNeed request_need(int past, int fresh, int page_shift, int max_pages) {
  RequestNeed q{0, 0, 0, 0, 0, 0};
  if (past < 0 || fresh < -1) {
    q.invalid = 1;
    return q;
  }
  const int n = fresh > 0 ? fresh : 0;
  const long long end = (long long)past + n, cap = (long long)max_pages << page_shift;
  q.n = n < kPlanCap ? n : kPlanCap;
  if (end > cap) {
    q.invalid = 1;
    return q;
  }
  const int up = (1 << page_shift) - 1;
  q.have = (int)(((long long)past + up) >> page_shift);
  if (fresh < 0) {
    q.back = q.have;
    return q;
  }
  q.need = (int)((end + up) >> page_shift) - q.have;
  q.live = 1;
  return q;
}

// place `offset` after `head` in a ring of n (0 <= head < n, 0 <= offset <= n)
RAX_HD int ring_at(int head, int offset, int n) {
  const long long p = (long long)head + offset;
  return (int)(p >= n ? p - n : p);
}
RAX_HD int ring_head(int head, int n) {
  const int h = head % n;
  return h < 0 ? h + n : h;
}

// the page of key tile `key` in a block table row, or -1
RAX_HD int page_or_none(int page, int num_pages) { return page >= 0 && page < num_pages ? page : -1; }

// ------------------------------------------------------------------ attention
RAX_HD int clamp_int(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// The new tokens of one sequence: first row of q, number of rows, cached length.
struct SeqRows {
  int start, n, len;
};
RAX_HD SeqRows seq_rows(int s0, int s1, int len, int num_tokens, int max_len) {
  SeqRows s;
  s.start = clamp_int(s0, 0, num_tokens);
  const int e = clamp_int(s1, 0, num_tokens);
  s.n = e > s.start ? e - s.start : 0;
  s.len = clamp_int(len, 0, max_len);
  return s;
}

struct KeyRange {
  int lo, hi;
};
// keys that the new token i of n sees (empty: hi <= lo)
RAX_HD KeyRange token_keys(int i, int n, int len, int window) {
  const int pos = len - n + i;              // > -2^31: n <= num_tokens, i < n
  KeyRange k;
  k.hi = pos + 1 > 0 ? pos + 1 : 0;
  k.lo = window > 0 && pos >= window ? pos - window + 1 : 0;
  return k;
}

// What a sequence is to the attention's workgroups: its keys (those any of its new tokens
// sees), from `base`, a multiple of 16, in `steps` runs of step_keys; at least one step
// where there are new tokens, so that rows which see nothing are written too.
struct SeqSpan {
  unsigned base;
  int steps;
};
RAX_HD SeqSpan seq_span(const SeqRows& s, int window, int step_log2) {
  SeqSpan x{0u, 0};
  if (s.n <= 0) return x;
  const KeyRange first = token_keys(0, s.n, s.len, window), last = token_keys(s.n - 1, s.n, s.len, window);
  x.base = (unsigned)first.lo & ~15u;
  const unsigned hi = (unsigned)last.hi, span = hi > x.base ? hi - x.base : 0u;
  x.steps = (int)((span + ((1u << step_log2) - 1u)) >> step_log2);
  if (x.steps < 1) x.steps = 1;
  return x;
}
// Units of a sequence: kv heads times blocks of 2^rows_log2 rows.
RAX_HD int row_blocks(int n, int group, int rows_log2) {
  return (int)(((unsigned)n * (unsigned)group + ((1u << rows_log2) - 1u)) >> rows_log2);   // n * group <= 2^30
}
// The least step_log2 >= least with which the line of all units' steps is below kPlanCap for
// sequences of up to max_len keys that share num_tokens tokens; -1 if there is none up to 30.
RAX_HD int line_step_log2(int least, int num_seqs, int num_tokens, int max_len, int heads, int group, int rows_log2) {
  const double units = ((double)row_blocks(num_tokens, group, rows_log2) + num_seqs) * heads;
  int s = least;
  while (s <= 30 && units * ((double)(max_len >> s) + 2.0) >= kPlanCap) ++s;
  return s <= 30 ? s : -1;
}

// Workgroups of the attention on a device of `cus` compute units: two each, as fit in registers and
// LDS, half of them above 128 dims.  Both numbers are multiples of the dies, over which neighbouring
// workgroups are dealt in turn: share_of_block needs that to reach every share.
constexpr int kDies = 8;
inline int attention_workers(int cus) {
  const int w = 2 * cus / (2 * kDies) * (2 * kDies);
  return w < 2 * kDies ? 2 * kDies : (w > 512 ? 512 : w);
}
RAX_HD int whole_dies(int n) { return (n + kDies - 1) / kDies * kDies; }
// The share of workgroup `block`, or `workers` if it has none: neighbouring shares on one die (the
// row blocks of a head read its keys from one L2), and as many on each.
RAX_HD int share_of_block(int block, int workers) {
  const int per = (workers + kDies - 1) / kDies, place = block / kDies;
  const int b = place < per ? block % kDies * per + place : workers;
  return b < workers ? b : workers;
}
// Contiguous equal shares of `work` steps: worker b of g takes [share_start(b), share_start(b + 1)).
RAX_HD int share_start(int work, int g, int b) {
  const unsigned q = (unsigned)work / (unsigned)g, rem = (unsigned)work - q * (unsigned)g;
  return (int)(q * (unsigned)b + ((unsigned)b < rem ? (unsigned)b : rem));
}
// the worker whose share holds step x (0 <= x < work)
RAX_HD int share_owner(int work, int g, int x) {
  const unsigned q = (unsigned)work / (unsigned)g, rem = (unsigned)work - q * (unsigned)g, wide = rem * (q + 1u);
  return (int)((unsigned)x < wide ? (unsigned)x / (q + 1u) : rem + ((unsigned)x - wide) / q);
}

// Workspace slot of part p of a unit that begins in workgroup `first`: a workgroup's
// second slot is the unit's that begins in it, its first the one's that began before.
RAX_HD int part_slot(int first, int p) { return p == 0 ? 2 * first + 1 : 2 * (first + p); }

// Division by a fixed d in [1, 2^16] of numbers below 2^31: with s = floor(log2 d), n / d =
// (n ceil(2^(32 + s) / d)) >> (32 + s), as the multiplier's excess, below d < 2^(s + 1),
// times n stays below 2^(32 + s); a power of two is the shift alone (mul 0).
struct FastDiv {
  unsigned mul;
  int shift;
};
inline FastDiv fast_div(int d) {
  FastDiv f{0u, 0};
  while ((2 << f.shift) <= d) ++f.shift;
  if (d != 1 << f.shift) f.mul = (unsigned)(((1ULL << (32 + f.shift)) + (unsigned)d - 1u) / (unsigned)d);
  return f;
}
RAX_HD int fast_quot(int n, FastDiv f) {
  const unsigned x = f.mul ? (unsigned)(((unsigned long long)(unsigned)n * f.mul) >> 32) : (unsigned)n;
  return (int)(x >> f.shift);
}

}  // namespace rax
