// Page fork: block table rows that follow their parents, in place, with the pages that rows share
// counted, those that need a page of their own drawn and those that nothing holds given back.
//
// Row i continues old row parents[i].  With k_r granted children of old row r, a full page of r
// changes its number of holders by k_r - 1; a partly filled page stays with the first child, and
// every other child draws a page: the n-th of them ring[head + n].  A page whose last holder goes
// gets a bit in `freed`; at the end the bits, in order of the page ids, follow the ring's free pages.
// So the result does not depend on the order of the atomics.
//
// What bounds it: latency, a chain of loads (parents and lengths, table, counts), two scans and
// the hand-over to the workgroup that finishes last.  Table columns are independent of each
// other, so a workgroup takes a strip of columns of all rows: it reads the entries of its new rows
// into registers, and writes them after a barrier, which makes the call work in place.  Every
// workgroup scans the rows by itself.  The workgroup that finishes last writes what the others
// had to read: lengths, ring, cursor.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "beam.h"
#include "device_util.h"
#include "fork_index.h"
#include "kv_scan.h"

namespace rax {

namespace {

constexpr int kForkWaves = kForkThreads / 64, kForkRows = LORA_MAX_SEQS / kForkThreads;   // rows of a thread

__device__ __forceinline__ int atomic_add_agent(int* p, int v) {
  return __hip_atomic_fetch_add(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// exclusive sum over the workgroup's threads, and the total (capped)
__device__ __forceinline__ int block_scan(int x, int* part, int tid, int& total) {
  const int lane = tid & 63, w = tid >> 6, in = wave_sat_scan(x);
  if (lane == 63) part[w] = in;
  __syncthreads();
  int before = __shfl_up(in, 1);
  if (lane == 0) before = 0;
  total = 0;
#pragma unroll
  for (int v = 0; v < kForkWaves; ++v) {
    if (v < w) before = sat_add(before, part[v]);
    total = sat_add(total, part[v]);
  }
  __syncthreads();
  return before;
}

}  // namespace

__global__ __launch_bounds__(kForkThreads) void page_fork_kernel(PageForkArgs a) {
  // of an old row: its length, its first child, its number of granted children; of a new
  // one: its parent (-1 if it has none or is refused) and its place among the drawn pages (-1: draws none)
  extern __shared__ int lds[];
  __shared__ int part_s[kForkWaves], refused_s, invalid_s, last_s;
  const int R = a.rows, N = a.num_pages, ps = a.page_shift, tid = threadIdx.x;
  int *len_s = lds, *first_s = len_s + R, *kids_s = first_s + R, *parent_s = kids_s + R, *draw_s = parent_s + R;
  const int head = ring_head(a.cursor[0], N), free_pages = clamp_int(a.cursor[1], 0, N);
  const bool first_wg = blockIdx.x == 0;
  if (tid == 0) refused_s = invalid_s = 0;

  // ---- rows, a run of consecutive ones for each thread
  const int per = (R + kForkThreads - 1) / kForkThreads, r0 = min(R, tid * per), count = min(R, r0 + per) - r0;
  int parent[kForkRows], invalid = 0;
#pragma unroll
  for (int i = 0; i < kForkRows; ++i) {
    parent[i] = -1;
    if (i >= count) continue;
    const int p = a.parents[r0 + i], len = a.lens[r0 + i];
    parent[i] = parent_or_none(p, R);
    const RowPages own = row_pages(len, ps, a.max_pages);
    if (first_wg) invalid += own.invalid + (p != parent[i] && p != -1);
    len_s[r0 + i] = own.invalid ? 0 : len;
    first_s[r0 + i] = R;
    kids_s[r0 + i] = 0;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kForkRows; ++i)
    if (parent[i] >= 0) atomicMin(&first_s[parent[i]], r0 + i);
  __syncthreads();
  int need = 0;
  bool draws[kForkRows];
#pragma unroll
  for (int i = 0; i < kForkRows; ++i) {
    draws[i] = parent[i] >= 0 && first_s[parent[i]] != r0 + i && (len_s[parent[i]] & ((1 << ps) - 1)) > 0;
    need += draws[i];
  }
  int needs, refused = 0;
  int place = block_scan(need, part_s, tid, needs);
  const int taken = min(needs, free_pages);
#pragma unroll
  for (int i = 0; i < kForkRows; ++i) {
    if (i >= count) continue;
    int draw = -1;
    if (draws[i]) {
      if (place < free_pages) draw = place;
      else {
        parent[i] = -1;
        ++refused;
      }
      ++place;
    }
    if (parent[i] >= 0) atomicAdd(&kids_s[parent[i]], 1);
    parent_s[r0 + i] = parent[i];
    draw_s[r0 + i] = draw;
    if (first_wg && draw < 0) {
      a.copy_src[r0 + i] = a.copy_dst[r0 + i] = -1;
      a.copy_tokens[r0 + i] = 0;
    }
  }
  if (first_wg && refused) atomicAdd(&refused_s, refused);
  __syncthreads();

  // ---- strips of columns
  const int C = a.columns, shift = 31 - __clz(C), strips = (a.max_pages + C - 1) / C;
  for (int strip = blockIdx.x; strip < strips; strip += gridDim.x) {
    const int c0 = strip * C;
    int id[kForkPer], old[kForkPer];   // entry of the new row, of the old one (-1: none)
    bool write[kForkPer], holds[kForkPer];
#pragma unroll
    for (int k = 0; k < kForkPer; ++k) {
      const int e = k * kForkThreads + tid, i = e >> shift, c = c0 + (e & (C - 1));
      write[k] = holds[k] = false;
      id[k] = old[k] = -1;
      if (i >= R || c >= a.max_pages) continue;
      const int p = parent_s[i];
      write[k] = p >= 0 && c < row_pages(len_s[p], ps, a.max_pages).all();
      holds[k] = c < row_pages(len_s[i], ps, a.max_pages).all();
      if (write[k]) id[k] = a.table[(size_t)p * a.ld_table + c];
      if (holds[k]) old[k] = a.table[(size_t)i * a.ld_table + c];
    }
#pragma unroll
    for (int k = 0; k < kForkPer; ++k) {   // holders of the old rows' pages
      const int e = k * kForkThreads + tid, i = e >> shift, c = c0 + (e & (C - 1));
      if (!holds[k]) continue;
      const int page = page_or_none(old[k], N), change = holders_change(row_pages(len_s[i], ps, a.max_pages), c, kids_s[i]);
      invalid += page < 0;
      old[k] = -1;   // from here on a page that nothing holds any more
      if (page < 0 || change == 0) continue;
      const int before = atomic_add_agent(&a.shares[page], change);
      if (before >= 0 && before + change < 0) old[k] = page;
    }
#pragma unroll
    for (int k = 0; k < kForkPer; ++k) {
      const int e = k * kForkThreads + tid, i = e >> shift, c = c0 + (e & (C - 1));
      if (holds[k] && old[k] >= 0)
        __hip_atomic_fetch_or(&a.freed[old[k] >> 5], 1u << (old[k] & 31), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (!write[k]) continue;
      id[k] = page_or_none(id[k], N);
      const RowPages pages = row_pages(len_s[parent_s[i]], ps, a.max_pages);
      if (c != pages.full || draw_s[i] < 0) continue;
      const int fresh = page_or_none(a.ring[ring_at(head, draw_s[i], N)], N);   // the new row's own last page
      invalid += fresh < 0;
      const bool both = fresh >= 0 && id[k] >= 0;
      a.copy_src[i] = both ? id[k] : -1;
      a.copy_dst[i] = both ? fresh : -1;
      a.copy_tokens[i] = both ? pages.part : 0;
      id[k] = fresh;
    }
    __syncthreads();   // every entry of the strip has been read
#pragma unroll
    for (int k = 0; k < kForkPer; ++k) {
      const int e = k * kForkThreads + tid, i = e >> shift, c = c0 + (e & (C - 1));
      if (write[k]) a.table[(size_t)i * a.ld_table + c] = id[k];
    }
  }
  if (invalid) atomicAdd(&invalid_s, invalid);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // this wave's atomics have arrived
  __syncthreads();
  if (tid == 0) {
    if (invalid_s) atomic_add_agent(&a.cursor[3], invalid_s);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    last_s = atomic_add_agent(&a.cursor[2], 1) == (int)gridDim.x - 1;
  }
  __syncthreads();
  if (!last_s) return;

  // ---- the last workgroup: lengths, freed pages to the ring's end in order of their ids
  for (int i = tid; i < R; i += kForkThreads) a.lens[i] = parent_s[i] >= 0 ? len_s[parent_s[i]] : 0;
  const int words = (N + 31) / 32, run = (words + kForkThreads - 1) / kForkThreads;
  const int w0 = min(words, tid * run), w1 = min(words, w0 + run);
  int mine = 0, back;
  for (int i = w0; i < w1; ++i) mine += __popc(__hip_atomic_load(&a.freed[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
  int at = block_scan(mine, part_s, tid, back);
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

hipError_t launch_page_fork(const PageForkArgs& given, hipStream_t stream, const KTimer& tm) {
  PageForkArgs a = given;
  a.columns = fork_columns(a.rows);
  const int strips = (a.max_pages + a.columns - 1) / a.columns, wgs = std::min(512, strips);
  RAX_LAUNCH(tm, page_fork_kernel, dim3(wgs), dim3(kForkThreads), (uint32_t)(5 * sizeof(int) * a.rows), stream, a);
  return hipGetLastError();
}

}  // namespace rax
