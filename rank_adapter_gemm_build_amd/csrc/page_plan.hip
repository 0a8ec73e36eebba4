// Page plan of one step: positions, slots, block table entries and the ring of free pages
// from the request lengths.
//
// With n_r, need_r and back_r of request r (kv_index.h) and exclusive prefix sums over the
// requests, token t of request r lies at position past_r + t - start_r; the e-th page
// drawn is ring[head + e] and belongs to the request with first_r <= e < first_r +
// need_r; the e-th page given back goes to ring[head + free + e].  So after one scan of
// three sums over at most 4096 requests every output element is found on its own by a
// binary search in the prefix sums (in LDS).
//
// What bounds it: latency, a chain of two loads, the scan, a search and two more loads
// (a few us); only steps of some 100,000 prompt tokens write enough to count.  So every
// workgroup does the whole scan by itself and takes its part of the elements, several
// loads at a time, and the last one to finish writes the cursor, which the others read.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "device_util.h"
#include "kv.h"
#include "kv_scan.h"

namespace rax {

constexpr int kPlanThreads = 512, kPlanWaves = kPlanThreads / 64, kPlanPer = LORA_MAX_SEQS / kPlanThreads;
constexpr int kPlanBatch = 4;   // elements of a thread whose loads are on the way together

// last r in [0, n) with start[r] <= x (start[0] = 0)
__device__ __forceinline__ int last_at_most(const int* start, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ __launch_bounds__(kPlanThreads) void page_plan_kernel(PagePlanArgs a) {
  // exclusive sums of tokens, pages drawn and pages given back; past length (its
  // complement where the tokens get no slots)
  extern __shared__ int lds[];
  __shared__ int part[3][kPlanWaves], taken_s, invalid_s, refused_s;
  const int R = a.num_seqs, T = a.num_tokens, N = a.num_pages, tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  int *tok = lds, *drawn = tok + R + 1, *given = drawn + R + 1, *before = given + R + 1;
  const int per = (R + kPlanThreads - 1) / kPlanThreads;   // each thread a run of consecutive requests
  const int r0 = min(R, tid * per), count = min(R, r0 + per) - r0;
  int past[kPlanPer], fresh[kPlanPer];
#pragma unroll
  for (int i = 0; i < kPlanPer; ++i) {
    past[i] = fresh[i] = 0;
    if (i < count) {
      past[i] = a.past[r0 + i];
      fresh[i] = a.fresh[r0 + i];
    }
  }
  const int head = ring_head(a.cursor[0], N), free_pages = clamp_int(a.cursor[1], 0, N);
  const bool first_wg = blockIdx.x == 0;
  if (tid == 0) taken_s = invalid_s = refused_s = 0;

  int sn = 0, sp = 0, sb = 0, invalid = 0;
#pragma unroll
  for (int i = 0; i < kPlanPer; ++i)
    if (i < count) {
      const RequestNeed q = request_need(past[i], fresh[i], a.page_shift, a.max_pages);
      sn = sat_add(sn, q.n);
      sp = sat_add(sp, q.need);
      sb = sat_add(sb, q.back);
      invalid += q.invalid;
    }
  int in = wave_sat_scan(sn), ip = wave_sat_scan(sp), ib = wave_sat_scan(sb);
  if (lane == 63) {
    part[0][w] = in;
    part[1][w] = ip;
    part[2][w] = ib;
  }
  __syncthreads();
  // exclusive prefixes of this thread's run: the lane before's, then the waves before
  in = __shfl_up(in, 1);
  ip = __shfl_up(ip, 1);
  ib = __shfl_up(ib, 1);
  if (lane == 0) in = ip = ib = 0;
  int total = 0;
#pragma unroll
  for (int v = 0; v < kPlanWaves; ++v) {
    if (v < w) {
      in = sat_add(in, part[0][v]);
      ip = sat_add(ip, part[1][v]);
      ib = sat_add(ib, part[2][v]);
    }
    total = sat_add(total, part[0][v]);
  }
  int taken = 0, refused = 0;
#pragma unroll
  for (int i = 0; i < kPlanPer; ++i)
    if (i < count) {
      const int r = r0 + i;
      const RequestNeed q = request_need(past[i], fresh[i], a.page_shift, a.max_pages);
      const int start = min(in, T);
      tok[r] = start;
      drawn[r] = ip;
      given[r] = ib;
      in = sat_add(in, q.n);
      ip = sat_add(ip, q.need);
      ib = sat_add(ib, q.back);
      const bool granted = q.live && (q.need == 0 || ip <= free_pages);
      before[r] = granted ? past[i] : ~past[i];
      if (granted && q.need > 0) taken = ip;
      if (q.live && !granted) ++refused;
      if (first_wg) {
        a.query_start[r] = start;
        a.seq_lens[r] = granted ? past[i] + q.n : 0;
      }
    }
  if (count > 0 && r0 + count == R) {
    tok[R] = min(in, T);
    drawn[R] = ip;
    given[R] = ib;
  }
  if (R == 0 && tid == 0) tok[0] = drawn[0] = given[0] = 0;
  if (taken) atomicMax(&taken_s, taken);
  if (refused) atomicAdd(&refused_s, refused);
  if (!first_wg) invalid = 0;                 // lengths are counted once
  __syncthreads();
  taken = taken_s;
  const int tokens = tok[R], back = min(given[R], N - free_pages);   // a ring of N places holds no more
  if (first_wg && tid == 0) {
    a.query_start[R] = tokens;
    invalid += total - tokens + (given[R] - back);
  }

  const int step = gridDim.x * kPlanThreads, g = blockIdx.x * kPlanThreads + tid, up = (1 << a.page_shift) - 1;
  // elements: the batch's tokens, the pages drawn, the pages given back
  const int drawn_at = T, given_at = T + taken, all = given_at + back;
  for (int e0 = g; e0 < all; e0 += kPlanBatch * step) {
    int row[kPlanBatch], at[kPlanBatch], page[kPlanBatch];
    bool was[kPlanBatch];   // the page id comes from a row's existing part
#pragma unroll
    for (int k = 0; k < kPlanBatch; ++k) {
      const int e = e0 + k * step;
      row[k] = at[k] = 0;
      page[k] = -1;
      was[k] = false;
      if (e >= all) continue;
      const bool token = e < drawn_at, draw = !token && e < given_at;
      const int x = token ? e : draw ? e - drawn_at : e - given_at;
      if (token && x >= tokens) continue;   // padding: position 0, no slot
      const int* sums = token ? tok : draw ? drawn : given;
      const int r = last_at_most(sums, R, x), i = x - sums[r], p = before[r];
      const int had = p < 0 ? ~p : p, have = (int)(((unsigned)had + (unsigned)up) >> a.page_shift);
      const int32_t *entry = a.table + (size_t)r * a.ld_table, *src = nullptr;
      row[k] = r;
      if (token) {
        at[k] = (int)((unsigned)had + (unsigned)i);   // wraps only past the table's capacity
        const int c = at[k] >> a.page_shift;
        was[k] = p >= 0 && c < have;
        if (p >= 0) src = c < have ? entry + c : a.ring + ring_at(head, drawn[r] + c - have, N);
      } else if (draw) {   // x < taken: r is granted, its past a length
        at[k] = have + i;
        src = a.ring + ring_at(head, x, N);
      } else {
        at[k] = ring_at(head, free_pages + x, N);
        src = entry + i;
      }
      if (src) page[k] = *src;
    }
#pragma unroll
    for (int k = 0; k < kPlanBatch; ++k) {
      const int e = e0 + k * step, id = page_or_none(page[k], N);
      if (e >= all) continue;
      if (e < drawn_at) {
        invalid += was[k] && id < 0;
        a.positions[e] = at[k];
        a.slots[e] = id >= 0 ? (id << a.page_shift) + (at[k] & up) : -1;
      } else {
        invalid += id < 0;
        if (e < given_at) a.table[(size_t)row[k] * a.ld_table + at[k]] = id;
        else a.ring[at[k]] = id;
      }
    }
  }

  if (invalid) atomicAdd(&invalid_s, invalid);
  __syncthreads();
  if (tid != 0) return;
  int bad = invalid_s;
  if (gridDim.x > 1) {   // the last workgroup writes what the others still had to read (cursor_out may be cursor)
    if (bad) {
      __hip_atomic_fetch_add(&a.cursor[3], bad, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the count has arrived before this workgroup says so
    }
    if (__hip_atomic_fetch_add(&a.cursor[2], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != (int)gridDim.x - 1) return;
    bad = __hip_atomic_exchange(&a.cursor[3], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    a.cursor[2] = 0;
  }
  a.cursor_out[0] = ring_at(head, taken, N);
  a.cursor_out[1] = free_pages - taken + back;
  a.meta[0] = total;
  a.meta[1] = taken;
  a.meta[2] = back;
  a.meta[3] = refused_s;
  a.meta[4] = bad;
  a.meta[5] = free_pages - taken + back;
  a.meta[6] = a.meta[7] = 0;
}

hipError_t launch_page_plan(const PagePlanArgs& a, hipStream_t stream, const KTimer& tm) {
  const size_t lds = (4 * (size_t)a.num_seqs + 3) * sizeof(int);
  // two tokens a thread; of ended requests, whose pages are not known here, 64 a workgroup
  const int wgs = std::min(256, std::max({1, (a.num_tokens + 2 * kPlanThreads - 1) / (2 * kPlanThreads), (a.num_seqs + 63) / 64}));
  RAX_LAUNCH(tm, page_plan_kernel, dim3(wgs), dim3(kPlanThreads), (uint32_t)lds, stream, a);
  return hipGetLastError();
}

}  // namespace rax
