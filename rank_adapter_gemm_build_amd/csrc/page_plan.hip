// Page plan of one step: positions, slots, block table entries and the ring of free pages
// from the request lengths.
//
// With n_r, need_r and back_r of request r (kv_index.h) and exclusive prefix sums over the
// requests, token t of request r lies at position past_r + t - start_r; the e-th page
// drawn is ring[head + e] and belongs to the request with first_r <= e < first_r +
// need_r; the e-th page given back goes to ring[head + free + e].  So after one scan of
// three sums over at most 4096 requests every output element is found on its own by a
// binary search in the prefix sums (in LDS).
#include <hip/hip_runtime.h>

#include "device_util.h"
#include "kv.h"

namespace rax {

constexpr int kPlanThreads = 256;

__device__ __forceinline__ int wave_sat_scan(int x) {   // inclusive
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(x, d);
    if (lane_id() >= d) x = sat_add(x, y);
  }
  return x;
}

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
  extern __shared__ int lds[];
  __shared__ int part[3][kPlanThreads / 64], taken_s, invalid_s, refused_s;
  const int R = a.num_seqs, T = a.num_tokens, N = a.num_pages, tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  int *tok = lds, *drawn = tok + R + 1, *given = drawn + R + 1;
  const int head = ring_head(a.cursor[0], N), free_pages = clamp_int(a.cursor[1], 0, N);
  const bool first_wg = blockIdx.x == 0;
  if (tid == 0) taken_s = invalid_s = refused_s = 0;

  // each thread a run of consecutive requests
  const int per = (R + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(R, tid * per), r1 = min(R, r0 + per);
  int sn = 0, sp = 0, sb = 0, invalid = 0;
  for (int r = r0; r < r1; ++r) {
    const RequestNeed q = request_need(a.past[r], a.fresh[r], a.page_shift, a.max_pages);
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
  for (int v = 0; v < kPlanThreads / 64; ++v) {
    if (v < w) {
      in = sat_add(in, part[0][v]);
      ip = sat_add(ip, part[1][v]);
      ib = sat_add(ib, part[2][v]);
    }
    total = sat_add(total, part[0][v]);
  }
  int taken = 0;
  int refused = 0;
  for (int r = r0; r < r1; ++r) {
    const int past = a.past[r];
    const RequestNeed q = request_need(past, a.fresh[r], a.page_shift, a.max_pages);
    tok[r] = min(in, T);
    drawn[r] = ip;
    given[r] = ib;
    in = sat_add(in, q.n);
    ip = sat_add(ip, q.need);
    ib = sat_add(ib, q.back);
    const bool granted = q.live && (q.need == 0 || ip <= free_pages);
    if (granted && q.need > 0) taken = ip;
    if (q.live && !granted) ++refused;
    if (first_wg) {
      a.query_start[r] = tok[r];
      a.seq_lens[r] = granted ? past + q.n : 0;
    }
  }
  if (r1 == R && r0 < r1) {
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
  const int back = min(given[R], N - free_pages);   // a ring of N places holds no more
  if (first_wg && tid == 0) {
    a.query_start[R] = tok[R];
    invalid += total - tok[R] + (given[R] - back);
  }

  const int step = gridDim.x * kPlanThreads, g = blockIdx.x * kPlanThreads + tid;
  for (int t = g; t < T; t += step) {
    int pos = 0, slot = -1;
    if (t < tok[R]) {
      const int r = last_at_most(tok, R, t);
      const int past = a.past[r];
      const RequestNeed q = request_need(past, a.fresh[r], a.page_shift, a.max_pages);
      pos = (int)((unsigned)past + (unsigned)(t - tok[r]));   // wraps only past the table's capacity
      if (q.live && (q.need == 0 || sat_add(drawn[r], q.need) <= free_pages)) {
        const int at = pos >> a.page_shift;
        int page;
        if (at < q.have) {
          page = page_or_none(a.table[(size_t)r * a.ld_table + at], N);
          invalid += page < 0;
        } else {
          page = page_or_none(a.ring[ring_at(head, drawn[r] + at - q.have, N)], N);
        }
        if (page >= 0) slot = (page << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
      }
    }
    a.positions[t] = pos;
    a.slots[t] = slot;
  }
  for (int e = g; e < taken; e += step) {
    const int r = last_at_most(drawn, R, e);
    const RequestNeed q = request_need(a.past[r], a.fresh[r], a.page_shift, a.max_pages);
    const int page = page_or_none(a.ring[ring_at(head, e, N)], N);
    invalid += page < 0;
    a.table[(size_t)r * a.ld_table + q.have + e - drawn[r]] = page;
  }
  for (int e = g; e < back; e += step) {
    const int r = last_at_most(given, R, e);
    const int page = page_or_none(a.table[(size_t)r * a.ld_table + e - given[r]], N);
    invalid += page < 0;
    a.ring[ring_at(head, free_pages + e, N)] = page;
  }

  // the last workgroup writes what the others still had to read (cursor_out may be cursor)
  if (invalid) atomicAdd(&invalid_s, invalid);
  __syncthreads();
  if (tid == 0) {
    if (invalid_s) atomicAdd(&a.cursor[3], invalid_s);
    __threadfence();
    if (atomicAdd(&a.cursor[2], 1) == (int)gridDim.x - 1) {
      __threadfence();
      const int bad = atomicExch(&a.cursor[3], 0);
      a.cursor[2] = 0;
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
  }
}

hipError_t launch_page_plan(const PagePlanArgs& a, hipStream_t stream, const KTimer& tm) {
  const size_t lds = 3 * (size_t)(a.num_seqs + 1) * sizeof(int);
  RAX_LAUNCH(tm, page_plan_kernel, dim3(1), dim3(kPlanThreads), (uint32_t)lds, stream, a);
  return hipGetLastError();
}

}  // namespace rax
