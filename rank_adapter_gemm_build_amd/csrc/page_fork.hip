// Page fork: block table rows that follow their parents, in place, with the pages that rows share
// counted, those that need a page of their own drawn and those that nothing holds given back.
//
// Row i continues old row parents[i].  With k_r granted children of old row r, a full page of r
// changes its number of holders by k_r - 1; a partly filled page stays with the first child, and
// every other child draws a page: the n-th of them ring[head + n].  A page whose last holder goes
// gets a bit in `freed`; at the end the bits, in order of the page ids, follow the ring's free pages.
// So the result does not depend on the order of the atomics.
//
// What bounds it: latency, a chain of loads (parents and lengths, table, counts), a scan and
// the hand-over to the workgroup that finishes last.  Table columns are independent of each
// other, so a workgroup takes a strip of kForkColumns of all rows, a lane a row: the old entries go to
// LDS, where the new rows find them after a barrier, which makes the call work in place.  Beams lie
// side by side and hold mostly the same pages: the changes of a run of lanes with one page are
// summed first, and for pages that all beams of a request hold come to nothing, which leaves few atomics.
// Every workgroup scans the rows by itself.  The one that finishes last writes what the others
// had to read: lengths, ring, cursor.  Up to 256 rows a workgroup has 256 threads and each one row, else 1024 and four: 257 to 1024
// rows pay for three passes, sums over lanes among them, that find no row.  Measured, pages of 16: 4 rows of 777 tokens 6.5 us,
// 1024 of up to 8191 17.4, 4096 of 8191 75, 64 of 2^20 131 (64 strips a workgroup, one after the other).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "beam.h"
#include "device_util.h"
#include "fork_index.h"
#include "kv_scan.h"

namespace rax {

namespace {

__device__ __forceinline__ int atomic_add_agent(int* p, int v) {
  return __hip_atomic_fetch_add(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Exclusive sum over the workgroup's threads, and the total (capped).  part: LDS, not in use before the barrier in here.
template <int WAVES> __device__ __forceinline__ int block_scan(int x, int* part, int tid, int& total) {
  const int lane = tid & 63, w = tid >> 6, in = wave_sat_scan(x);
  if (lane == 63) part[w] = in;
  __syncthreads();
  int before = __shfl_up(in, 1);
  if (lane == 0) before = 0;
  total = 0;
#pragma unroll
  for (int v = 0; v < WAVES; ++v) {
    if (v < w) before = sat_add(before, part[v]);
    total = sat_add(total, part[v]);
  }
  return before;
}

// The sum of `change` over a run of neighbouring lanes with one page, in the run's last lane; 0 in the others.  All lanes active.
__device__ __forceinline__ int run_sum(int page, int change, int lane) {
  const int sum = wave_inclusive_scan(change), before = __shfl_up(page, 1), after = __shfl_down(page, 1);
  const unsigned long long heads = __ballot(lane == 0 || before != page);
  const int head = 63 - __clzll(heads & (~0ull >> (63 - lane)));
  const int skip = __shfl(sum, max(head - 1, 0));
  return lane == 63 || after != page ? sum - (head > 0 ? skip : 0) : 0;
}

}  // namespace

// T: threads; PER: rows of a thread
template <int T, int PER> __global__ __launch_bounds__(T) void page_fork_kernel(PageForkArgs a) {
  constexpr int C = kForkColumns, W = T / 64;
  // of an old row: its entries in the strip, its length, its first child, its number of granted children
  extern __shared__ int4 strip_s[];
  __shared__ int part_s[2][W], invalid_s, last_s;
  const int R = a.rows, N = a.num_pages, ps = a.page_shift, tid = threadIdx.x, lane = tid & 63;
  int *len_s = reinterpret_cast<int*>(strip_s + R), *first_s = len_s + R, *kids_s = first_s + R;
  const bool first_wg = blockIdx.x == 0;

  // ---- rows, a run of consecutive ones for each thread
  const int per = (R + T - 1) / T, r0 = min(R, tid * per), count = min(R, r0 + per) - r0;
  int parent[PER], len[PER], invalid = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    parent[i] = -1;
    len[i] = 0;
    if (i < count) {
      parent[i] = a.parents[r0 + i];
      len[i] = a.lens[r0 + i];
    }
  }
  const int head = ring_head(a.cursor[0], N), free_pages = clamp_int(a.cursor[1], 0, N);
  if (tid == 0) invalid_s = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (i < count) {
      first_s[r0 + i] = R;
      kids_s[r0 + i] = 0;
    }
  int longest = 0;   // pages of the longest row
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (i >= count) continue;
    const int p = parent_or_none(parent[i], R);
    const RowPages own = row_pages(len[i], ps, a.max_pages);
    if (first_wg) invalid += own.invalid + (p != parent[i] && parent[i] != -1);
    parent[i] = p;
    len[i] = own.invalid ? 0 : len[i];
    len_s[r0 + i] = len[i];
    longest = max(longest, own.all());
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (parent[i] >= 0) atomicMin(&first_s[parent[i]], r0 + i);
  __syncthreads();
  int need = 0, draw[PER], size[PER];   // place among the drawn pages (-1: draws none); length of the new row
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    size[i] = parent[i] >= 0 ? len_s[parent[i]] : 0;
    draw[i] = parent[i] >= 0 && first_s[parent[i]] != r0 + i && (size[i] & ((1 << ps) - 1)) > 0 ? 0 : -1;
    need += draw[i] == 0;
  }
  for (int d = 32; d > 0; d >>= 1) longest = max(longest, __shfl_xor(longest, d));
  if (lane == 0) part_s[1][tid >> 6] = longest;
  int needs, place = block_scan<W>(need, part_s[0], tid, needs);
#pragma unroll
  for (int v = 0; v < W; ++v) longest = max(longest, part_s[1][v]);
  const int taken = min(needs, free_pages);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (draw[i] == 0) {
      draw[i] = place < free_pages ? place : -1;
      if (place >= free_pages) {
        parent[i] = -1;
        size[i] = 0;
      }
      ++place;
    }
    if (parent[i] >= 0) atomicAdd(&kids_s[parent[i]], 1);
    if (first_wg && i < count && draw[i] < 0) {
      a.copy_src[r0 + i] = a.copy_dst[r0 + i] = -1;
      a.copy_tokens[r0 + i] = 0;
    }
  }
  __syncthreads();

  // ---- strips of columns
  const int strips = (longest + C - 1) / C;
  const bool whole = a.ld_table % 4 == 0 && (reinterpret_cast<uintptr_t>(a.table) & 15u) == 0;   // 16 bytes of a row at a time
  for (int b = blockIdx.x; b < (strips + kDies - 1) / kDies * kDies; b += gridDim.x) {
    const int strip = strip_of_block(b, strips), c0 = strip * C;
    if (strip >= strips) continue;
    int old[PER][C];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int used = row_pages(len[i], ps, a.max_pages).all() - c0;   // entries of this row in the strip
      const int32_t* src = a.table + (size_t)(r0 + i) * a.ld_table + c0;
#pragma unroll
      for (int k = 0; k < C; ++k) old[i][k] = -1;
      if (i >= count || used <= 0) continue;
      if (whole && c0 + C <= a.max_pages) {
        const int4 v = *reinterpret_cast<const int4*>(src);
        old[i][0] = v.x;
        old[i][1] = used > 1 ? v.y : -1;
        old[i][2] = used > 2 ? v.z : -1;
        old[i][3] = used > 3 ? v.w : -1;
      } else {
#pragma unroll
        for (int k = 0; k < C; ++k)
          if (k < used) old[i][k] = src[k];
      }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (i >= count) continue;
      const int used = row_pages(len[i], ps, a.max_pages).all() - c0;
#pragma unroll
      for (int k = 0; k < C; ++k) {
        old[i][k] = page_or_none(old[i][k], N);
        invalid += k < used && old[i][k] < 0;
      }
      strip_s[r0 + i] = make_int4(old[i][0], old[i][1], old[i][2], old[i][3]);
    }
    __syncthreads();   // every entry of the strip has been read
    // new rows
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const RowPages pages = row_pages(size[i], ps, a.max_pages);
      const int used = pages.all() - c0;
      if (i >= count || used <= 0) continue;
      const int4 v = strip_s[parent[i]];
      int id[C] = {v.x, v.y, v.z, v.w};
      if (draw[i] >= 0 && pages.full >= c0 && pages.full < c0 + C) {   // its last page lies here, and is its own
        const int fresh = page_or_none(a.ring[ring_at(head, draw[i], N)], N);
        int src = -1;
#pragma unroll
        for (int k = 0; k < C; ++k)
          if (c0 + k == pages.full) {
            src = id[k];
            id[k] = fresh;
          }
        const bool both = fresh >= 0 && src >= 0;
        invalid += fresh < 0;
        a.copy_src[r0 + i] = both ? src : -1;
        a.copy_dst[r0 + i] = both ? fresh : -1;
        a.copy_tokens[r0 + i] = both ? pages.part : 0;
      }
      int32_t* dst = a.table + (size_t)(r0 + i) * a.ld_table + c0;
      if (whole && used >= C) *reinterpret_cast<int4*>(dst) = make_int4(id[0], id[1], id[2], id[3]);
      else {
#pragma unroll
        for (int k = 0; k < C; ++k)
          if (k < used) dst[k] = id[k];
      }
    }
    // holders of the old rows' pages.  Lane by lane the rows lie PER apart, so runs are those of every PER-th row.
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const RowPages own = row_pages(len[i], ps, a.max_pages);
      const int kids = i < count ? kids_s[r0 + i] : 1;
      int change[C], before[C];
#pragma unroll
      for (int k = 0; k < C; ++k) change[k] = run_sum(old[i][k], old[i][k] >= 0 ? holders_change(own, c0 + k, kids) : 0, lane);
#pragma unroll
      for (int k = 0; k < C; ++k) {
        before[k] = -1;
        if (change[k] != 0 && old[i][k] >= 0) before[k] = atomic_add_agent(&a.shares[old[i][k]], change[k]);
      }
#pragma unroll
      for (int k = 0; k < C; ++k)
        if (before[k] >= 0 && before[k] + change[k] < 0)
          __hip_atomic_fetch_or(&a.freed[old[i][k] >> 5], 1u << (old[i][k] & 31), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();   // the strip's entries in LDS are done with
  }
  if (invalid) atomicAdd(&invalid_s, invalid);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // this wave's atomics have arrived
  __syncthreads();
  if (tid == 0) {
    if (invalid_s) {
      atomic_add_agent(&a.cursor[3], invalid_s);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
    last_s = atomic_add_agent(&a.cursor[2], 1) == (int)gridDim.x - 1;
  }
  __syncthreads();
  if (!last_s) return;

  // ---- the last workgroup: lengths, freed pages to the ring's end in order of their ids
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (i < count) a.lens[r0 + i] = size[i];
  const int words = (N + 31) / 32, run = (words + T - 1) / T;
  const int w0 = min(words, tid * run), w1 = min(words, w0 + run);
  int mine = 0, back;
  for (int i = w0; i < w1; ++i) mine += __popc(__hip_atomic_load(&a.freed[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
  int at = block_scan<W>(mine, part_s[0], tid, back);
  const int kept = min(back, N - free_pages);   // a ring of N places holds no more
  if (mine > 0)
    for (int i = w0; i < w1; ++i) {
      uint32_t bits = __hip_atomic_load(&a.freed[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (bits == 0) continue;
      __hip_atomic_store(&a.freed[i], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      for (; bits; bits &= bits - 1) {
        const int page = 32 * i + __ffs(bits) - 1;
        __hip_atomic_store(&a.shares[page], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (at < kept) a.ring[ring_at(head, free_pages + at, N)] = page;
        ++at;
      }
    }
  if (tid != 0) return;
  const int bad = __hip_atomic_exchange(&a.cursor[3], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  a.cursor[2] = 0;
  a.cursor[0] = ring_at(head, taken, N);
  a.cursor[1] = free_pages - taken + kept;
  a.meta[0] = taken;
  a.meta[1] = kept;
  a.meta[2] = needs - taken;
  a.meta[3] = bad + (back - kept);
  a.meta[4] = free_pages - taken + kept;
  a.meta[5] = a.meta[6] = a.meta[7] = 0;
}

hipError_t launch_page_fork(const PageForkArgs& a, hipStream_t stream, const KTimer& tm) {
  const int strips = (a.max_pages + kForkColumns - 1) / kForkColumns, wgs = std::min(256, whole_dies(strips));
  const uint32_t lds = (uint32_t)(7 * sizeof(int) * a.rows);
  if (a.rows <= 256) RAX_LAUNCH(tm, (page_fork_kernel<256, 1>), dim3(wgs), dim3(256), lds, stream, a);
  else RAX_LAUNCH(tm, (page_fork_kernel<1024, LORA_MAX_SEQS / 1024>), dim3(wgs), dim3(1024), lds, stream, a);
  return hipGetLastError();
}

}  // namespace rax
