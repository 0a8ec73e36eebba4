// Beam selection: of a request's beams b and tokens v the `best` candidates with the largest
// w_b s(b, v), s(b, v) = score_b + x[b][v] - ln sum_u exp x[b][u], in one pass over the logits.
//
// Within a row the order of the candidates is that of the logits, so a row's best are found and
// its log sum is formed side by side while the row streams by, and only the joining of rows needs
// the sums.  A workgroup has a share of one row.  Of each request the last workgroup to finish
// joins: it forms the rows' log sums and picks among the shares' lists.
//
// Sum.  Each lane keeps a maximum and the sum of exponentials relative to it; a lane's largest
// term is then exactly 1, and lanes, waves and shares are joined in 64 bits, so the few terms
// that make up a peaked distribution's sum carry no rounding of an exponential.  Scores are
// formed in 64 bits: candidates of two beams may lie next to each other.
// Equal terms after a larger one all round the same way, in every lane, so a lane's fp32 sum goes to 64 bits every
// kBeamRun tiles.  In units of 2^-24 of the sum a run then has at most 32 from additions of loads and 7 from those within one,
// about 3 for each move of its maximum, and a term d below the maximum 2.2 d + 2, of up to 65536 a lane 20 on average.
// They cannot all be at their most (32 needs one large term, the others none), so the 2^-18 of the contract, 64 units,
// hold for every vocabulary and number of rows.  (Without the runs: 2^-16 at 256 tiles a wave.)
//
// Lists.  A candidate is one 64-bit word that sorts as (row, value, token) do: complement of the
// row, value as an ordered integer, complement of the token.  A wave appends to its list in LDS
// what is not below its `floor`: at first the best-th largest of its lanes' maxima, then the
// best-th entry of the list itself whenever that is cut back to `best` (each entry's place is the
// number of larger ones).  After the first tile hits are rare, and a tile costs little more
// than its exponentials.
//
// What bounds it: reading the logits; next to that the exponential, 4 of some 12 vector
// cycles a value; then the join, 8 to 10 us of one workgroup a request.  Measured: 64 requests of 8 beams over
// 128000 tokens in bf16 38 us (3.4 TB/s; reading alone 22), 24 of 6 over 50001 in fp32 with 12 candidates
// 21, 1 of 4 over 32000 10.
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cmath>

#include "beam.h"
#include "device_util.h"

namespace rax {

namespace {

typedef unsigned long long u64;
constexpr int kBeamThreads = 64 * kBeamWaves;
constexpr int kListCap = 2 * LORA_MAX_BEAMS + 64 * 8;   // a list before it is cut back, and one load of every lane
constexpr float kLog2e = 1.44269504088896341f;
constexpr int kBeamRun = 8;   // tiles whose terms a lane adds in fp32

struct Entry {   // a candidate of the join
  double rank;
  u64 key;
};
// A weight of infinity (above 0 as all are) times a score of 0 is taken as 0: every rank is a number, and within a row the
// ranks keep the order of the scores.
__device__ __forceinline__ double rank_of(double score, float weight) { return score == 0.0 ? 0.0 : score * (double)weight; }

__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) { return __uint_as_float(u ^ (~(uint32_t)((int)u >> 31) | 0x80000000u)); }
// never 0: a value in a list is at least -FLT_MAX
__device__ __forceinline__ u64 key_of(int row, float v, int token) {
  return (u64)(63 - row) << 56 | (u64)ordered(v + 0.f) << 24 | (0xffffffu - (uint32_t)token);   // -0 as 0
}
__device__ __forceinline__ float key_value(u64 key) { return unordered((uint32_t)(key >> 24)); }
__device__ __forceinline__ int key_token(u64 key) { return (int)(0xffffffu - (uint32_t)(key & 0xffffffu)); }
__device__ __forceinline__ int key_row(u64 key) { return 63 - (int)(key >> 56); }

__device__ __forceinline__ u64 get_word(const u64* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ void put_word(u64* p, u64 v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// Maximum, and sum in 64 bits, over the wave by lane moves (row_shr 1, 2, 4, 8, row_bcast 15 and 31), in every lane
template <int CTRL, int ROWS> __device__ __forceinline__ float max_step(float v) {
  return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(-INFINITY), __float_as_int(v), CTRL, ROWS, 0xf, false)));
}
__device__ __forceinline__ float wave_max(float v) {
  v = max_step<0x118, 0xf>(max_step<0x114, 0xf>(max_step<0x112, 0xf>(max_step<0x111, 0xf>(v))));
  v = max_step<0x143, 0xc>(max_step<0x142, 0xa>(v));
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
template <int CTRL, int ROWS> __device__ __forceinline__ double sum_step(double v) {
  const u64 u = (u64)__double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xf, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xf, false);
  return v + __longlong_as_double((long long)((u64)hi << 32 | lo));
}
__device__ __forceinline__ double wave_sum64(double v) {
  v = sum_step<0x118, 0xf>(sum_step<0x114, 0xf>(sum_step<0x112, 0xf>(sum_step<0x111, 0xf>(v))));
  v = sum_step<0x143, 0xc>(sum_step<0x142, 0xa>(v));
  const u64 u = (u64)__double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, 63), hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 63);
  return __longlong_as_double((long long)((u64)hi << 32 | lo));
}
// sum of the lanes' l at maxima m, relative to the largest maximum
__device__ __forceinline__ double joined_sum(float m, double l, float& top) {
  top = wave_max(m);
  return wave_sum64(m == top ? l : l * exp((double)m - (double)top));   // m = -inf: 0
}

// the n-th largest of the lanes' keys, 0 if n is above 64
__device__ __forceinline__ uint32_t nth_of_lanes(uint32_t key, int n) {
  uint32_t at = 0;
#pragma unroll
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t test = at | 1u << bit;
    if (__popcll(__ballot(key >= test)) >= n) at = test;
  }
  return at;
}

template <typename T> struct Chunk;   // 16 bytes of logits
template <> struct Chunk<uint16_t> {
  static constexpr int kN = 8;
  static constexpr uint32_t kNone = 0xff80ff80u;
  __device__ __forceinline__ static float at(const uint4& c, int e) {
    const uint32_t w = (&c.x)[e / 2];
    return e & 1 ? bf16_hi(w) : bf16_lo(w);
  }
};
template <> struct Chunk<float> {
  static constexpr int kN = 4;
  static constexpr uint32_t kNone = 0xff800000u;
  __device__ __forceinline__ static float at(const uint4& c, int e) { return __uint_as_float((&c.x)[e]); }
};

// Numbers of list[0..n) that are above `mine`, kAhead at a time (the loads of a step are on the way together);
// list[n..) up to the next multiple of kAhead holds zeros.
constexpr int kAhead = 8;
__device__ __forceinline__ int above(const u64* list, int n, u64 mine) {
  int place = 0;
  for (int j = 0; j < n; j += kAhead) {
    ulonglong2 two[kAhead / 2];
#pragma unroll
    for (int k = 0; k < kAhead / 2; ++k) two[k] = *reinterpret_cast<const ulonglong2*>(list + j + 2 * k);
#pragma unroll
    for (int k = 0; k < kAhead / 2; ++k) place += (two[k].x > mine) + (two[k].y > mine);
  }
  return place;
}

// Cut a wave's list of n entries back to its `best` largest, in order, with zeros behind them; returns their number.  Every
// entry is counted against all: of a long list first those whose value is below the best-th largest go (250 entries: 3 us
// without).
__device__ __forceinline__ int cut_list(u64* list, u64* sorted, int n, int best, int lane) {
  if (n > 2 * LORA_MAX_BEAMS) {
    constexpr int kHold = kListCap / 64;
    uint32_t value[kHold], floor_ = 0;
#pragma unroll
    for (int k = 0; k < kHold; ++k) value[k] = k * 64 + lane < n ? (uint32_t)(list[k * 64 + lane] >> 24) : 0u;
#pragma unroll 1
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t test = floor_ | 1u << bit;
      int count = 0;
#pragma unroll
      for (int k = 0; k < kHold; ++k) count += __popcll(__ballot(value[k] >= test));
      if (count >= best) floor_ = test;
    }
    int left = 0;
#pragma unroll
    for (int k = 0; k < kHold; ++k) {   // places that have been read are written
      const u64 mask = __ballot(value[k] >= floor_);
      const u64 e = list[k * 64 + lane];
      wave_lds_sync();
      if (value[k] >= floor_) list[left + __popcll(mask & ((1ull << lane) - 1ull))] = e;
      left += __popcll(mask);
    }
    n = left;
  }
  if (lane < kAhead) list[n + lane] = 0;
  wave_lds_sync();
  for (int i = lane; i < n; i += 64) {
    const u64 mine = list[i];
    const int place = above(list, n, mine);
    if (place < best) sorted[place] = mine;
  }
  wave_lds_sync();
  n = min(n, best);
  if (lane < n) list[lane] = sorted[lane];
  if (lane < kAhead) list[n + lane] = 0;
  wave_lds_sync();
  return n;
}

// the want-th largest of the workgroup's values, N a thread, or 0; sums: LDS
template <int N> __device__ __forceinline__ uint32_t nth_of_group(const uint32_t (&values)[N], int want, uint32_t (&sums)[2][kBeamWaves], int lane, int w) {
  uint32_t at = 0;
#pragma unroll 1
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t test = at | 1u << bit;
    int count = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) count += __popcll(__ballot(values[k] >= test));
    if (lane == 0) sums[bit & 1][w] = (uint32_t)count;
    __syncthreads();
    if ((int)(sums[bit & 1][0] + sums[bit & 1][1] + sums[bit & 1][2] + sums[bit & 1][3]) >= want) at = test;
  }
  return at;
}

}  // namespace

template <typename T>
__global__ __launch_bounds__(kBeamThreads) void beam_select_kernel(BeamArgs a) {
  using C = Chunk<T>;
  constexpr int N = C::kN, U = kBeamLoads;
  __shared__ __attribute__((aligned(16))) u64 lists[kBeamWaves][kListCap + kAhead + LORA_MAX_BEAMS];
  __shared__ double lse_s[LORA_MAX_BEAMS];
  __shared__ int counts[kBeamWaves], last_s, count_s;
  const int tid = threadIdx.x, lane = lane_id(), w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int row = blockIdx.x / a.segs, seg = blockIdx.x - row * a.segs, request = row / a.beams, beam = row - request * a.beams;
  const int best = a.best;

  // ---- this workgroup's share of the row.  Loads are of aligned 16 bytes; a row that begins
  // inside one has its first and last values fetched singly.
  const T* const x = reinterpret_cast<const T*>(a.logits) + (size_t)row * a.ld;
  const int shift = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
  const uint4* const chunks = reinterpret_cast<const uint4*>(x - shift);
  const auto load = [&](int tile, uint4 (&c)[U]) {
    const int first_ = tile * U * 64 * N - shift;   // token of the tile's first value
    if (first_ >= 0 && first_ + U * 64 * N <= a.vocab) {
#pragma unroll
      for (int u = 0; u < U; ++u) c[u] = chunks[(tile * U + u) * 64 + lane];
      return;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int first = first_ + (u * 64 + lane) * N;
      c[u] = make_uint4(C::kNone, C::kNone, C::kNone, C::kNone);
      if (first >= 0 && first + N <= a.vocab) {
        c[u] = chunks[(tile * U + u) * 64 + lane];
      } else if (first > -N && first < a.vocab) {
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (first + e >= 0 && first + e < a.vocab) {
            if constexpr (sizeof(T) == 4) (&c[u].x)[e] = __float_as_uint(x[first + e]);
            else {
              uint32_t& word = (&c[u].x)[e / 2];
              word = e & 1 ? (word & 0xffffu) | (uint32_t)x[first + e] << 16 : (word & 0xffff0000u) | x[first + e];
            }
          }
      }
    }
  };
  const int tile_n = 64 * U * N, tiles = (a.vocab + shift + tile_n - 1) / tile_n, stride = a.segs * kBeamWaves;
  const int tile0 = seg * kBeamWaves + w;   // this wave among the row's
  int tile = tile0;
  uint4 cur[U];
  // the request's beams, one a lane (over: 0 read, 1 ended, 2 without a candidate)
  float lane_score = -INFINITY, lane_weight = 1.f;
  int over = 2;
  if (lane < a.beams) {
    const int r = request * a.beams + lane;
    lane_score = a.scores[r];
    if (a.weights) lane_weight = a.weights[r];
    over = a.ended ? a.ended[r] : 0;
  }
  load(tile, cur);
  over = !(lane_score > -INFINITY) || !(lane_weight > 0.f) ? 2 : over != 0;
  const bool live = __builtin_amdgcn_readlane(over, beam) == 0;   // else the row is not read
  if (live) {
    u64 *list = lists[w], *sorted = list + kListCap + kAhead;
    float m = -INFINITY, l = 0.f, floor_ = -FLT_MAX, sum_m = -INFINITY;
    double sum_l = 0.0;   // of the runs before, relative to sum_m
    const auto end_run = [&] {
      if (__any(sum_l != 0.0 && m != sum_m)) sum_l *= m == sum_m ? 1.0 : exp((double)sum_m - (double)m);
      sum_l += (double)l;
      sum_m = m;
      l = 0.f;
    };
    int n = 0, run = 0;
    for (bool first = true; tile < tiles; tile += stride, first = false) {
      if (run++ == kBeamRun) {
        end_run();
        run = 1;
      }
      float top[U], all = -INFINITY;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        top[u] = -INFINITY;
#pragma unroll
        for (int e = 0; e < N; ++e) top[u] = fmaxf(top[u], C::at(cur[u], e));
        all = fmaxf(all, top[u]);
      }
      const float mn = fmaxf(m, all), base = mn == -INFINITY ? 0.f : mn;
      l *= __builtin_amdgcn_exp2f((m - base) * kLog2e);
      m = mn;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float part = 0.f;
#pragma unroll
        for (int e = 0; e < N; ++e) part += __builtin_amdgcn_exp2f((C::at(cur[u], e) - base) * kLog2e);
        l += part;
      }
      if (first) floor_ = fmaxf(floor_, unordered(nth_of_lanes(ordered(all), best)));
      if (__any(all >= floor_)) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (!__any(top[u] >= floor_)) continue;
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const float v = C::at(cur[u], e);
            const bool hit = v >= floor_;
            const u64 mask = __ballot(hit);
            if (mask == 0) continue;
            if (hit) list[n + __popcll(mask & ((1ull << lane) - 1ull))] = key_of(beam, v, ((tile * U + u) * 64 + lane) * N + e - shift);
            n += __popcll(mask);
          }
          if (n > max(LORA_MAX_BEAMS, 2 * best)) {   // room for another load; tokens to come are higher, so equal values no longer enter
            n = cut_list(list, sorted, n, best, lane);
            if (n == best) floor_ = unordered(ordered(key_value(list[best - 1])) + 1u);
          }
        }
      }
      if (tile + stride < tiles) load(tile + stride, cur);   // no tile ahead: other waves' arithmetic hides the load (38 us, 39 with one)
    }
    n = cut_list(list, sorted, n, best, lane);
    // the wave's sum
    float top;
    end_run();
    const double sum = joined_sum(m, sum_l, top);
    if (lane == 0) {
      counts[w] = n;
      put_word(a.sums + 2 * ((size_t)row * stride + tile0), (u64)__float_as_uint(top));
      put_word(a.sums + 2 * ((size_t)row * stride + tile0) + 1, (u64)__double_as_longlong(sum));
    }
    __syncthreads();
    // the workgroup's list
    u64* out = a.keys + ((size_t)row * a.segs + seg) * best;
    int total = 0;
#pragma unroll
    for (int v = 0; v < kBeamWaves; ++v) total += counts[v];
    if (lane < n) {
      const u64 mine = list[lane];
      int place = lane;
#pragma unroll
      for (int v = 1; v < kBeamWaves; ++v) place += above(lists[(w + v) % kBeamWaves], counts[(w + v) % kBeamWaves], mine);
      if (place < best) put_word(out + place, mine);
    }
    if (tid >= total && tid < best) put_word(out + tid, 0);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // every store of this wave has arrived
  }
  __syncthreads();
  if (tid == 0) {
    last_s = __hip_atomic_fetch_add(&a.arrived[request], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == a.beams * a.segs - 1;
    if (last_s) __hip_atomic_store(&a.arrived[request], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (!last_s) return;

  // ---- the request's join
  __shared__ float score_s[LORA_MAX_BEAMS], weight_s[LORA_MAX_BEAMS];
  __shared__ int over_s[LORA_MAX_BEAMS];   // 0: read, 1: ended, 2: gives no candidate
  __shared__ uint32_t floors_s[2][kBeamWaves];
  constexpr int kFetch = 4, kEntries = LORA_MAX_BEAMS * (2 + kFetch * kBeamWaves);   // ended beams, those kept, new ones
  constexpr int kLists = (kBeamMaxLists + kBeamThreads - 1) / kBeamThreads;
  static_assert(sizeof(Entry) * (kEntries + kAhead + LORA_MAX_BEAMS) <= sizeof(lists), "the lists' LDS holds the join's");
  Entry *entries = reinterpret_cast<Entry*>(&lists[0][0]), *sorted = entries + kEntries + kAhead;
  const int row0 = request * a.beams, lists_n = a.beams * a.segs, n = lists_n * best;
  // (2048 of 64 lists: 50 us in rounds of all, 60 list by list; 65536 of 1024: 6200 and 100)
  const bool many = n > 2 * kFetch * kBeamThreads;
  const u64* const keys = a.keys + (size_t)row0 * a.segs * best;   // of a row that was not read: what an earlier call left, and not taken
  u64 key[kFetch];   // the first of all candidates, unless they are many
  const auto fetch = [&](int i) -> u64 { return !many && i < n ? get_word(keys + i) : 0; };
#pragma unroll
  for (int k = 0; k < kFetch; ++k) key[k] = fetch(k * kBeamThreads + tid);
  // the rows' log sums, kRows of a wave's at a time
  constexpr int kRows = 4;
  const int parts = a.segs * kBeamWaves;
  for (int j0 = w; j0 < a.beams; j0 += kRows * kBeamWaves) {
    float m[kRows];
    double l[kRows];
    const auto part = [&](int j, int i, float& pm, double& pl) {
      const u64* p = a.sums + 2 * ((size_t)(row0 + j) * parts + i);
      pm = i < parts ? __uint_as_float((uint32_t)get_word(p)) : -INFINITY;
      pl = i < parts ? __longlong_as_double((long long)get_word(p + 1)) : 0.0;
    };
#pragma unroll
    for (int k = 0; k < kRows; ++k)
      if (j0 + k * kBeamWaves < a.beams) part(j0 + k * kBeamWaves, lane, m[k], l[k]);
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int j = j0 + k * kBeamWaves;
      if (j >= a.beams || __builtin_amdgcn_readlane(over, j) != 0) continue;
      for (int i = 64 + lane; i - lane < parts; i += 64) {
        float pm;
        double pl;
        part(j, i, pm, pl);
        const float nm = fmaxf(m[k], pm);
        l[k] = (m[k] == nm ? l[k] : l[k] * exp((double)m[k] - (double)nm)) + (pm == nm ? pl : pl * exp((double)pm - (double)nm));
        m[k] = nm;
      }
      float top;
      const double sum = joined_sum(m[k], l[k], top);
      if (lane == 0) lse_s[j] = (double)top + log(sum);   // no finite logit, or one that is NaN or +inf: not a number, no candidate
    }
  }
  if (w == 0) {
    if (lane < a.beams) {
      score_s[lane] = lane_score;
      weight_s[lane] = lane_weight;
      over_s[lane] = over;
    }
    // ended beams
    const u64 mask = __ballot(over == 1);
    if (over == 1) entries[__popcll(mask & ((1ull << lane) - 1ull))] = Entry{rank_of((double)lane_score, lane_weight), key_of(lane, 0.f, a.end_token)};
    if (lane == 0) count_s = __popcll(mask);
  }
  __syncthreads();
  const auto candidate = [&](u64 k) {
    const int j = key_row(k);
    return over_s[j] == 1 ? (double)score_s[j] : (double)score_s[j] + ((double)key_value(k) - lse_s[j]);
  };
  // a candidate, and its rank rounded down as an ordered integer; 0: none
  const auto ranked = [&](u64 k, int beam_, Entry& e) -> uint32_t {
    e = Entry{-INFINITY, k};
    if (k == 0 || over_s[beam_] != 0) return 0;
    const double s = candidate(k);
    e.rank = rank_of(s, weight_s[key_row(k)]);
    return s > -INFINITY ? ordered(__double2float_rd(e.rank)) : 0;
  };
  const auto take = [&](const Entry& e, bool pass) {
    const u64 mask = __ballot(pass);
    if (mask == 0) return;
    int at = 0;
    if (lane == 0) at = atomicAdd(&count_s, __popcll(mask));
    at = __shfl(at, 0) + __popcll(mask & ((1ull << lane) - 1ull));
    if (pass) entries[at] = e;
  };
  // the list cut back to its `best`, in order; returns their number.  As in cut_list, a long one first to those that can be
  // among them (1000 entries: 50 us without)
  const auto cut = [&]() -> int {
    __syncthreads();
    int c = count_s;
    if (c > 2 * LORA_MAX_BEAMS) {
      constexpr int kHold = (kEntries + kBeamThreads - 1) / kBeamThreads;
      uint32_t down[kHold];
#pragma unroll
      for (int k = 0; k < kHold; ++k) down[k] = k * kBeamThreads + tid < c ? ordered(__double2float_rd(entries[k * kBeamThreads + tid].rank)) : 0u;
      const uint32_t floor_ = nth_of_group(down, best, floors_s, lane, w);
      if (tid == 0) count_s = 0;
#pragma unroll 1
      for (int i0 = 0; i0 < c; i0 += kBeamThreads) {   // places that have been read are written
        const Entry e = entries[i0 + tid];
        __syncthreads();
        take(e, i0 + tid < c && ordered(__double2float_rd(e.rank)) >= floor_);
      }
      __syncthreads();
      c = count_s;
    }
    if (tid < kAhead) entries[c + tid] = Entry{-INFINITY, 0};   // below every other
    __syncthreads();
    for (int i = tid; i < c; i += kBeamThreads) {
      const Entry own = entries[i];
      int place = 0;
      for (int j = 0; j < c; j += kAhead) {
        Entry o[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) o[k] = entries[j + k];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) place += o[k].rank > own.rank || (o[k].rank == own.rank && o[k].key > own.key);
      }
      if (place < best) sorted[place] = own;
    }
    __syncthreads();
    const int kept = min(c, best);
    if (tid < kept) entries[tid] = sorted[tid];
    if (tid == 0) count_s = kept;
    __syncthreads();
    return kept;
  };
  if (!many) {
    // A round of kFetch a thread: those of the best-th largest of a wave's lanes' own best and above come on the list, at most
    // kFetch for each of `best` lanes a wave.
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += kFetch * kBeamThreads) {
      if (i0 > 0) (void)cut();
      Entry e[kFetch];
      uint32_t down[kFetch], mine = 0;
#pragma unroll
      for (int k = 0; k < kFetch; ++k) {
        const int i = i0 + k * kBeamThreads + tid;
        down[k] = ranked(key[k], min(i / (a.segs * best), a.beams - 1), e[k]);
        mine = max(mine, down[k]);
        key[k] = fetch(i + kFetch * kBeamThreads);
      }
      const uint32_t least = nth_of_lanes(mine, best);
      if (lane == 0) floors_s[0][w] = least;
      __syncthreads();
      const uint32_t floor_ = max(max(max(floors_s[0][0], floors_s[0][1]), max(floors_s[0][2], floors_s[0][3])), 1u);
#pragma unroll
      for (int k = 0; k < kFetch; ++k) take(e[k], down[k] >= floor_);
    }
  } else {
    // Many lists, each in order: kFetch of each at a time (and thread: where the lists are fewer several have one), and of a
    // list no more once one is below the floor: at first the value
    // that lists_best lists reach with their q-th, so that there are `best` candidates above it, then the last of the list
    // whenever that is cut back.
    const int q = (best + lists_n - 1) / lists_n, lists_best = (best + q - 1) / q;
    Entry e, last{};
    uint32_t at[kLists], floor_ = 0;
    const auto list_beam = [&](int i) { return min(i / a.segs, a.beams - 1); };
#pragma unroll
    for (int j = 0; j < kLists; ++j) {
      const int i = j * kBeamThreads + tid;
      at[j] = ranked(i < lists_n ? get_word(keys + (size_t)i * best + (q - 1)) : 0, list_beam(i), e);
    }
    floor_ = max(nth_of_group(at, lists_best, floors_s, lane, w), 1u);
    bool full = false;
    unsigned open = ~0u;   // lists of this thread that go on, as bits
    int side = 0;          // threads of a list, as a power of two
    while (lists_n << (side + 1) <= kBeamThreads) ++side;
    for (int e0 = 0; e0 < best && __syncthreads_or(open != 0); e0 += kFetch << side) {
#pragma unroll 1
      for (int i0 = 0, bit = 0; i0 < kLists * kBeamThreads; i0 += kBeamThreads, ++bit) {
        const int i = (i0 + tid) >> side, at_list = e0 + (tid & ((1 << side) - 1)) * kFetch;
        if (i >= lists_n) open &= ~(1u << bit);
        if (i0 >= lists_n << side) continue;
        u64 next[kFetch];
#pragma unroll
        for (int k = 0; k < kFetch; ++k) {
          next[k] = 0;
          if ((open >> bit & 1) && at_list + k < best) next[k] = get_word(keys + (size_t)i * best + at_list + k);
        }
        __syncthreads();
        const int c = count_s;
        __syncthreads();
        if (c + kFetch * kBeamThreads > kEntries && cut() == best) {
          full = true;
          last = entries[best - 1];
          floor_ = max(floor_, ordered(__double2float_rd(last.rank)));
        }
        uint32_t down = 0;
#pragma unroll
        for (int k = 0; k < kFetch; ++k) {
          down = ranked(next[k], list_beam(i), e);
          take(e, down >= floor_ && (!full || e.rank > last.rank || (e.rank == last.rank && e.key > last.key)));
        }
        if (down < floor_) open &= ~(1u << bit);
      }
      open &= (1u << kLists) - 1u;
    }
  }
  (void)cut();
  const int found = count_s;
  if (tid < best) {
    const int out = request * best + tid;
    int parent = -1, token = -1, done = 0;
    float s = -INFINITY;
    if (tid < found) {
      const u64 key = entries[tid].key;
      const int j = key_row(key);
      parent = row0 + j;
      token = key_token(key);
      done = over_s[j] == 1 || token == a.end_token;
      s = (float)candidate(key);
    }
    a.parents[out] = parent;
    a.tokens[out] = token;
    a.scores_out[out] = s;
    if (a.ended_out) a.ended_out[out] = done;
  }
}

hipError_t launch_beam_select(const BeamArgs& a, hipStream_t stream, const KTimer& tm) {
  const dim3 grid((unsigned)(a.requests * a.beams * a.segs)), block(kBeamThreads);
  if (a.dtype == LORA_F32) RAX_LAUNCH(tm, beam_select_kernel<float>, grid, block, 0u, stream, a);
  else RAX_LAUNCH(tm, beam_select_kernel<uint16_t>, grid, block, 0u, stream, a);
  return hipGetLastError();
}

}  // namespace rax
