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

}  // namespace rax
