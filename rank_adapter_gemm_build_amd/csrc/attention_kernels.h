// Paged attention: out = softmax(scale q K^T) V over the cached keys a token sees, in one
// pass over the keys with a running maximum m and sum l (base 2, s = scale log2(e) q.k):
//   m' = max(m, max_j s_j),  l' = l 2^(m - m') + sum_j 2^(s_j - m'),
//   o' = o 2^(m - m') + sum_j 2^(s_j - m') v_j,   out = o / l,  lse = (m + log2 l) ln 2.
//
// What bounds it: reading the keys and values (2 * len * kv heads * dim elements a
// sequence); the work on each is done by the matrix cores in a small part of that time.
//
// Rows.  The new tokens of a sequence times the query heads of one kv head share its keys:
// row x = token * group + head.  A wave holds RT tiles of 16 rows; of a workgroup's W waves
// RW have rows side by side, the others split the keys (KW = W / RW).  A workgroup of one wave
// (many short sequences) needs no join and no LDS.
//
// Tiles.  Both products keep the rows in the matrix cores' column (lane % 16), so maxima,
// sums and the correction of o stay in the lane they are used in, and nothing passes
// through LDS between the products:
//   S^T = K Q^T: lane (c, g = lane / 16) gets row c's scores of keys 4 g + 0..3 of each
//   group of 16 keys; these are exactly its operand values of O^T = V^T P^T when the second product's
//   contraction index 8 g + i stands for key 4 g + i of the first (i < 4) or second group.
//   K is the operand as it lies in memory (a lane loads 16 bytes of one key; whole_keys). V needs
//   several keys of one dim in a register: a lane loads EC consecutive dims of each of its
//   keys and the pairs are put together by one byte permutation each.  MFMA e of a block
//   then computes the dims {m EC + e}, so a lane ends with EC consecutive dims of its row.
//   Weights enter the 16-bit product as two bf16 parts (2^-16 relative, not 2^-8): the
//   second product is far from binding.  e4m3 cells are widened to bf16, which is exact.
//   fp32 caches use the fp32 matrix cores, 4 keys (or dims) at a time, with no permutation.
// A tile's keys are loaded again as soon as its first product has read them, its values
// after the second, so every wave keeps 8 to 16 KB on the way, and a part's first tile is
// loaded before the part before it is joined and written.
//
// Split.  The steps (KW tiles) of all sequences, kv heads and row blocks form one
// line, cut into equal contiguous shares, one a workgroup, whatever the lengths.  What a
// workgroup has of a unit (sequence, head, row block) that others share goes to the
// workspace as (m, l, o); the parts join in a tree, the last one to arrive at a node adding
// them in order of the keys, so the result does not depend on which that is.
//
// Measured: 256 sequences of 2000 to 4000 tokens, 32 query and 8 kv heads of 128, bf16:
// 482 to 498 us, 6.3 to 6.5 TB/s (a plain streaming read reaches 6.15, a copy 5.3); one of
// 131071 88 us, 6.1 TB/s; one of 777 11 us, latency: 2 us launch, 1 the line, 1 the part, 2.5 page
// ids and first tile, 4.5 join.
#pragma once

#include <hip/hip_runtime.h>

#include <cmath>
#include <type_traits>

#include "device_util.h"
#include "kv.h"
#include "kv_scan.h"

namespace rax {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kJoin = 8;        // parts of a unit that one workgroup adds

// Read-only words at a wave-uniform index through the scalar cache (written by earlier
// launches only).
typedef const __attribute__((address_space(4))) int32_t* const_words_t;
__device__ __forceinline__ const_words_t const_words(const int32_t* p) { return (const_words_t)(uintptr_t)p; }
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
// The value as if it were new here.  What follows from it is then computed where it is used;
// otherwise the compiler computes everything that the parts' loop does not change ahead of
// the loop and keeps it in spilled registers, over 100 instructions before the first load.
__device__ __forceinline__ int here(int v) {
  asm volatile("" : "+s"(v));
  return v;
}
__device__ __forceinline__ int here_lane(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Cells are read through buffer descriptors, whose base is a group of keys at one kv head:
// the lane's part of an address is one register, kept for all tiles, and a lane whose
// offset is kNowhere, or a group whose descriptor is empty (a page outside the cache, a
// tile past the last), reads zeros without a memory access or a branch.
constexpr uint32_t kNowhere = 0x80000000u;
constexpr int kStreaming = 2;   // buffer access bit nt
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ __amdgpu_buffer_rsrc_t cells_at(const char* base, bool ok) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, ok ? 0x7fffffff : 0, 0x00027000);
}
template <int N> struct Words {
  uint32_t w[N];
};
template <int N, int AUX = 0> __device__ __forceinline__ Words<N> load_words(__amdgpu_buffer_rsrc_t r, uint32_t ofs, uint32_t sofs) {
  Words<N> x;
  if constexpr (N == 4) {
    const u32x4_t v = __builtin_amdgcn_raw_buffer_load_b128(r, ofs, sofs, AUX);
    x.w[0] = v[0]; x.w[1] = v[1]; x.w[2] = v[2]; x.w[3] = v[3];
  } else if constexpr (N == 2) {
    const u32x2_t v = __builtin_amdgcn_raw_buffer_load_b64(r, ofs, sofs, AUX);
    x.w[0] = v[0]; x.w[1] = v[1];
  } else {
    x.w[0] = __builtin_amdgcn_raw_buffer_load_b32(r, ofs, sofs, AUX);
  }
  return x;
}

// A pair of loads covers 128 bytes of each of 16 keys.  Each load takes whole lines, of 8 keys
// (streamed lines that two loads touch cost more: 64 sequences to 8192, e4m3 rows of 128
// bytes, 118 -> 108 us, bf16 to 4096 106.5 -> 102.3; rows that follow each other in memory
// within 2 % either way; heads of 80, whose rows are not whole lines, 93 -> 94; 256-byte pieces of 4 keys no better): lane c16 of `a` holds key c16 % 8, of `b` 8 + c16 % 8, bytes 64 (c16 / 8)
// on.  The matrix cores' operands have key c16 in lane c16, the first 64 bytes in one and the
// others in the next, so the lanes of a row of 16 exchange with those 8 away.
__device__ __forceinline__ void whole_keys(uint4& a, uint4& b) {
  const auto step = [](uint32_t& u, uint32_t& v) {
    const int x = (int)u, y = (int)v;
    u = (uint32_t)__builtin_amdgcn_update_dpp(x, y, 0x128, 0xf, 0xc, false);   // row_ror:8 into lanes 8..15
    v = (uint32_t)__builtin_amdgcn_update_dpp(y, x, 0x128, 0xf, 0x3, false);   // into lanes 0..7
  };
  step(a.x, b.x);
  step(a.y, b.y);
  step(a.z, b.z);
  step(a.w, b.w);
}

// What workgroups hand to each other inside a launch goes past the caches that the XCDs do
// not share (agent scope, bit sc1), access by access; a fence of that scope would write back
// and drop the whole L2 instead, which took some 10 us each time.
constexpr int kAgentScope = 16;
__device__ __forceinline__ void put_shared(__amdgpu_buffer_rsrc_t r, uint32_t ofs, f32x4_t v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), r, ofs, 0, kAgentScope);
}
__device__ __forceinline__ f32x4_t get_shared(__amdgpu_buffer_rsrc_t r, uint32_t ofs) {
  return __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, ofs, 0, kAgentScope));
}
__device__ __forceinline__ void put_shared2(__amdgpu_buffer_rsrc_t r, uint32_t ofs, float x, float y) {
  __builtin_amdgcn_raw_buffer_store_b64(u32x2_t{__float_as_uint(x), __float_as_uint(y)}, r, ofs, 0, kAgentScope);
}
__device__ __forceinline__ float2 get_shared2(__amdgpu_buffer_rsrc_t r, uint32_t ofs) {
  const u32x2_t v = __builtin_amdgcn_raw_buffer_load_b64(r, ofs, 0, kAgentScope);
  return make_float2(__uint_as_float(v[0]), __uint_as_float(v[1]));
}
// Barrier for what lies in LDS: __syncthreads would also wait for the wave's loads and
// stores of global memory, 2 to 3 us each time.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}
// every store of this wave has arrived
__device__ __forceinline__ void stores_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// maximum and sum over the four lanes that share lane % 16
__device__ __forceinline__ float max_over_groups(float v) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum_over_groups(float v) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// C: cache type, DB: head_dim rounded up to 64, 128 or 256
template <typename C, int DB> struct AttnTile {
  static constexpr bool kF32 = sizeof(C) == 4, kF8 = sizeof(C) == 1;
  static constexpr int kGroups = kF32 ? 1 : 2;   // groups of 16 keys in a tile
  static constexpr int kKeys = 16 * kGroups;
  static constexpr int kKLoads = DB * (int)sizeof(C) / 64;     // 16-byte loads a lane makes for a group's keys
  static constexpr int kKElems = 16 / (int)sizeof(C);          // dims of such a load
  static constexpr int kQFrags = DB * (kF32 ? 4 : 2) / 64;     // 16-byte registers of a row tile
  static constexpr int kEC = kF32 || DB == 64 ? 4 : 8;         // consecutive dims of V in a lane
  static constexpr int kVB = DB / (16 * kEC);                  // blocks of 16 kEC dims
  static constexpr int kVW = kEC * (int)sizeof(C) / 4;         // words of kEC cells
  static constexpr int kPitch = 16 * kEC + 4;                  // floats of a row in the join buffer
};

// workspace slot of part p of a unit that begins in workgroup `first`: a workgroup's
// second slot is the unit's that begins in it, its first the one's that began before
__device__ __forceinline__ int part_slot(int first, int p) { return p == 0 ? 2 * first + 1 : 2 * (first + p); }

// a word of cells with those that are not finite cleared (e4m3 has no infinities)
template <typename C> __device__ __forceinline__ uint32_t without_odd(uint32_t v) {
  if constexpr (sizeof(C) == 4) return (v & 0x7f800000u) == 0x7f800000u ? 0u : v;
  else if constexpr (sizeof(C) == 2)
    return ((v & 0x7f80u) == 0x7f80u ? 0u : v & 0xffffu) | ((v & 0x7f800000u) == 0x7f800000u ? 0u : v & 0xffff0000u);
  else return v & ~((((((v & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u)) >> 7) * 0xffu);
}
// cell e of some words
template <typename C, int N> __device__ __forceinline__ float cell_value(const Words<N>& x, int e) {
  if constexpr (sizeof(C) == 4) return __uint_as_float(x.w[e]);
  else if constexpr (sizeof(C) == 2) return __uint_as_float(e & 1 ? x.w[e / 2] & 0xffff0000u : x.w[e / 2] << 16);
  else {
    const uint32_t byte = (x.w[e / 4] >> (8 * (e % 4))) & 0xffu;
    return (byte & 0x7fu) == 0x7fu ? __uint_as_float(0x7fc00000u) : 0.f;   // only its being NaN matters
  }
}

// finished dims of a row, and its log sum of weights (sum l at maximum m)
// (the conversion instruction rounds to nearest even and keeps NaN, as f32_to_bf16 does in
// some ten: that took 1 us at a part's end)
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const bf16x2_t v = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ void write4(uint16_t* p, f32x4_t y) {
  *reinterpret_cast<uint2*>(p) = make_uint2(bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3]));
}
__device__ __forceinline__ void write4(float* p, f32x4_t y) { *reinterpret_cast<f32x4_t*>(p) = y; }
__device__ __forceinline__ void write8(uint16_t* p, f32x4_t y, f32x4_t z) {
  st16(p, make_uint4(bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3]), bf16_pair(z[0], z[1]), bf16_pair(z[2], z[3])));
}
// l is 0 (nothing seen, or scores of minus infinity only), NaN (a NaN score; the maximum
// passes over it) or at least 1 / 2: the maximum's own weight is 1, and a part's join keeps that
__device__ __forceinline__ float log_sum(float m, float l) {
  return l == 0.f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.693147180559945309f;
}
// The maximum that weights are taken relative to. A part without a finite score has the maximum
// minus infinity and by that the weight 0 in a join; its sums, 0 or NaN, are added like all others.
__device__ __forceinline__ float finite_top(float m) { return m == -INFINITY ? 0.f : m; }
// scale / l, good to 2^-22
__device__ __forceinline__ float over_sum(float scale, float l) { return scale * __builtin_amdgcn_rcpf(l); }

// last r in [0, n) with sums[r] <= x (sums[0] = 0)
__device__ __forceinline__ int last_sum_at_most(const int* sums, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// A share's part of a unit.
struct Part {
  int start;              // of the sequence's tokens
  int row0, rows, kh;     // rows and kv head
  int s0, s1, steps, at;  // steps [s0, s1) of the unit's, and its place on the line
};

// RT: row tiles of a wave; W: waves; RW: those that have rows side by side; ONCE: every line of
// the cache is read by one workgroup only, and passes the caches as a stream
template <typename C, int DB, int RT, int W, int RW, bool ONCE>
__global__ __launch_bounds__(64 * W, DB > 128 ? 1 : 2) void paged_attention_kernel(AttentionArgs a) {
  using S = AttnTile<C, DB>;
  using T = std::conditional_t<S::kF32, float, uint16_t>;
  constexpr int G = S::kGroups, NK = S::kKLoads, NP = NK > 1 ? NK / 2 : 1, NQ = S::kQFrags, EC = S::kEC, VB = S::kVB, VW = S::kVW;
  extern __shared__ float4 lds[];
  using JoinRows = float[16][S::kPitch];
  __shared__ int part_s[W][3], last_s;

  constexpr int kAux = ONCE ? kStreaming : 0;
  constexpr int kThreads = 64 * W, KW = W / RW;   // KW: waves that split the keys
  constexpr int kRowsLog2 = 4 + RT / 2 + RW / 2, kRows = 1 << kRowsLog2, kKeysLog2 = S::kF32 ? 4 : 5;
  const int tid = threadIdx.x, lane = lane_id(), w = W == 1 ? 0 : uniform(tid >> 6), rw = w % RW, kw = w / RW;
  JoinRows* buf = reinterpret_cast<JoinRows*>(lds);                                  // [W]
  float2* stats = reinterpret_cast<float2*>(buf + (KW > 1 ? W : 0));                 // [W][RT][16]: maxima and sums
  int* sums = reinterpret_cast<int*>(stats + (KW > 1 ? W * RT * 16 : kRows));        // [2][num_seqs]: steps before each
  const int c16 = lane & 15, g4 = lane >> 4;
  const int D = a.c.dim, ps = a.c.page_shift, max_len = a.max_pages << ps, group = a.group_size;
  const const_words_t lens = const_words(a.seq_lens), starts = const_words(a.query_start);

  // ---- the line: steps before each sequence, and its shares
  const int per = (a.num_seqs + kThreads - 1) / kThreads;
  const int r0 = min(a.num_seqs, tid * per), r1 = min(a.num_seqs, r0 + per);
  constexpr int kWholeLog2 = W == 1 ? 5 : 2;
  // Two lines: in steps, and in steps 2^kWholeLog2 times as long, of which every unit has one
  // if no sequence is longer.  The second is taken if that holds and the units fill a quarter
  // of the workgroups and no more than all: 64 sequences of 100 to 500 tokens, 8 heads, 24.9 us
  // uncut, 29.2 cut; with 8 sequences 13.4, 11.9; with one 12.6, 11.3.  One-wave workgroups:
  // 256 sequences of 100 to 500 tokens 71.0 us uncut, 79.7 cut.
  int mine = 0, mine_whole = 0;
  bool long_one = false;
  int* whole_sums = sums + a.num_seqs;
  for (int i = r0; i < r1; ++i) {
    const SeqRows s = seq_rows(a.query_start[i], a.query_start[i + 1], a.seq_lens[i], a.num_tokens, max_len);
    const int units = a.c.heads * row_blocks(s.n, group, kRowsLog2), steps = seq_span(s, a.window, a.step_log2).steps;
    sums[i] = mine;
    whole_sums[i] = mine_whole;
    const long long all = (long long)units * steps;
    mine = sat_add(mine, all < kPlanCap ? (int)all : kPlanCap);
    mine_whole = sat_add(mine_whole, units);
    long_one |= steps > (1 << kWholeLog2);
  }
  const int scan = wave_sat_scan(mine), scan_whole = wave_sat_scan(mine_whole);
  long_one = __any(long_one);
  if (lane == 63) {
    part_s[w][0] = scan;
    part_s[w][1] = scan_whole;
    part_s[w][2] = long_one;
  }
  lds_barrier();
  int work_ = 0, units = 0, before = scan - mine, units_before = scan_whole - mine_whole;
#pragma unroll
  for (int v = 0; v < W; ++v) {
    if (v < w) {
      before += part_s[v][0];
      units_before += part_s[v][1];
    }
    work_ = sat_add(work_, part_s[v][0]);
    units = sat_add(units, part_s[v][1]);
    long_one |= part_s[v][2] != 0;
  }
  const bool by_unit = uniform(!long_one && a.step_log2 + kWholeLog2 < 31 && units <= (int)gridDim.x && units >= (int)gridDim.x / 4) != 0;
  work_ = uniform(by_unit ? units : work_);
  // no work, or more than the host counted with: sequences that overlap (the sums are capped)
  if (work_ == 0 || work_ >= kPlanCap) return;
  for (int i = r0; i < r1; ++i) sums[i] = by_unit ? whole_sums[i] + units_before : sums[i] + before;
  const int step_log2 = a.step_log2 + (by_unit ? kWholeLog2 : 0), tiles_log2 = step_log2 - kKeysLog2;   // tiles of a step
  const int workers_ = by_unit ? work_ : min((work_ + a.min_steps - 1) / a.min_steps, (int)gridDim.x);
  static_assert(kDies == kXcds, "shares are dealt over the XCDs");
  const int b_ = share_of_block((int)blockIdx.x, workers_);
  if (b_ >= workers_) return;
  lds_barrier();

  const uint32_t tok_b = (uint32_t)a.c.token_stride * (uint32_t)sizeof(C);   // below 2^27
  const float qs = a.scale * a.c.k_scale * 1.44269504088896341f;
  uint32_t kofs[NP], vofs[VB];   // lane's place in a group of keys, of values
#pragma unroll
  for (int f = 0; f < NP; ++f) {
    const uint32_t at = (NK > 1 ? 128u * f + 64u * (c16 >> 3) : 0u) + 16u * g4;   // in the key's row
    kofs[f] = at < (uint32_t)D * (uint32_t)sizeof(C) ? (uint32_t)(NK > 1 ? c16 & 7 : c16) * tok_b + at : kNowhere;
  }
#pragma unroll
  for (int vb = 0; vb < VB; ++vb) {
    const int d = (vb * 16 + c16) * EC;
    vofs[vb] = d < D ? (uint32_t)(4 * g4) * tok_b + d * (uint32_t)sizeof(C) : kNowhere;
  }
  const auto part_o = cells_at(reinterpret_cast<const char*>(a.part_o), true);   // below 2^31 bytes
  const auto part_ml = cells_at(reinterpret_cast<const char*>(a.part_ml), true);

  uint4 q[RT][NQ], K[G][NK];
  Words<VW> V[VB][4 * G];
  int lo[RT], hi[RT];                   // keys that row c16 of each row tile sees
  float m[RT], l[RT];
  f32x4_t o[RT][VB * EC];

  // ---- output of a part, or its place in the workspace
  auto out_row = [&](const Part& p, int lrow) {   // element of out, element of lse
    const int row = p.row0 + lrow, i = fast_quot(row, a.group), h = p.kh * group + row - i * group;
    struct At {
      T* out;
      size_t lse;
    };
    return At{reinterpret_cast<T*>(a.out) + (size_t)(p.start + i) * a.ldo + (size_t)h * D, (size_t)(p.start + i) * a.q_heads + h};
  };
  auto join = [&](const Part& p) {
    const int D = here(a.c.dim), b = here(b_), work = here(work_), workers = here(workers_);
    const int tid = here_lane((int)threadIdx.x), c16 = tid & 15, g4 = (tid >> 4) & 3;
    const bool whole = p.s0 == 0 && p.s1 == p.steps;
    const int first = whole ? b : share_owner(work, workers, p.at);
    auto part_row = [&](int k, int lrow) { return (uint32_t)part_slot(first, k) * (uint32_t)kRows + (uint32_t)lrow; };
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      l[rt] = sum_over_groups(l[rt]);
      if (KW > 1 && g4 == 0) stats[(w * RT + rt) * 16 + c16] = make_float2(m[rt], l[rt]);
    }
    if constexpr (KW > 1) lds_barrier();
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int lrow = (rw * RT + rt) * 16 + c16;
      float top = m[rt], sum = l[rt], f = 1.f;
      if constexpr (KW > 1) {
        float2 y[KW];
#pragma unroll
        for (int j = 0; j < KW; ++j) {
          y[j] = stats[((rw + j * RW) * RT + rt) * 16 + c16];
          top = fmaxf(top, y[j].x);
        }
        sum = 0.f;
#pragma unroll
        for (int j = 0; j < KW; ++j) sum += y[j].y * __builtin_amdgcn_exp2f(y[j].x - finite_top(top));
        f = __builtin_amdgcn_exp2f(m[rt] - finite_top(top));
      }
      if (whole) f = sum == 0.f ? 0.f : f * over_sum(a.c.v_scale, sum);
      if (kw == 0 && g4 == 0 && lrow < p.rows) {
        if (!whole) put_shared2(part_ml, part_row(b - first, lrow) * 8, top, sum);
        else if (a.lse) a.lse[out_row(p, lrow).lse] = log_sum(top, sum);
      }
      if constexpr (KW == 1) {   // this wave alone has the row: EC consecutive dims at a time
        if (lrow < p.rows) {
          T* out = out_row(p, lrow).out;
          const uint32_t at = part_row(b - first, lrow) * D;
#pragma unroll
          for (int vb = 0; vb < VB; ++vb)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int d = (vb * 16 + 4 * g4 + k) * EC;
              if (d >= D) continue;
              f32x4_t y[EC / 4];
#pragma unroll
              for (int e = 0; e < EC; ++e) y[e / 4][e % 4] = o[rt][vb * EC + e][k] * f;
              if (!whole) {
#pragma unroll
                for (int e = 0; e < EC / 4; ++e) put_shared(part_o, (at + d + 4 * e) * 4, y[e]);
              } else if constexpr (EC == 8) {
                write8(out + d, y[0], y[1]);
              } else {
                write4(out + d, y[0]);
              }
            }
        }
      } else {
        constexpr int kTileRows = 16 * RT * (RW - 1) + 16;   // local rows of this row tile lie below
#pragma unroll
        for (int vb = 0; vb < VB; ++vb) {
          if (rt + vb > 0) lds_barrier();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float* d = &buf[w][c16][(4 * g4 + k) * EC];
#pragma unroll
            for (int e = 0; e < EC; e += 4)
              *reinterpret_cast<f32x4_t*>(d + e) = f32x4_t{o[rt][vb * EC + e][k] * f, o[rt][vb * EC + e + 1][k] * f,
                                                          o[rt][vb * EC + e + 2][k] * f, o[rt][vb * EC + e + 3][k] * f};
          }
          lds_barrier();
          constexpr int kChunks = 4 * EC;   // of 4 dims
          const int n = min(p.rows - rt * 16, kTileRows);
          for (int it = tid; it < n * kChunks; it += kThreads) {
            const int d4 = it % kChunks, y = it / kChunks, rv = y / (16 * RT), row16 = y - rv * 16 * RT;   // y: local row - 16 rt
            const int d = vb * 16 * EC + d4 * 4, row = rt * 16 + y;
            if (row16 >= 16 || d >= D) continue;
            f32x4_t v[KW], acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < KW; ++j) v[j] = *reinterpret_cast<const f32x4_t*>(&buf[rv + j * RW][row16][d4 * 4]);
#pragma unroll
            for (int j = 0; j < KW; ++j) acc += v[j];
            if (whole) write4(out_row(p, row).out + d, acc);
            else put_shared(part_o, (part_row(b - first, row) * D + d) * 4, acc);
          }
        }
      }
    }
    if (!whole) {
      // Parts join in a tree, kJoin at a time: of the workgroups of a node the last to arrive
      // adds their parts, in order, and goes on to the next level with the sum.
      const int parts = share_owner(work, workers, p.at + p.steps - 1) - first + 1;
      float2* row_sums = KW > 1 ? reinterpret_cast<float2*>(lds) : stats;   // of the node
      int k0 = b - first;
      for (int level = 0, stride = 1; stride < parts; ++level, stride *= kJoin) {
        k0 -= k0 % (stride * kJoin);
        const int n = min(kJoin, (parts - k0 + stride - 1) / stride);
        const bool root = stride * kJoin >= parts;
        if (n == 1) continue;
        stores_done();
        lds_barrier();
        if (tid == 0) {
          int* arrived = a.arrived + level * a.counters + first + k0;
          last_s = __hip_atomic_fetch_add(arrived, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == n - 1;
          if (last_s) __hip_atomic_store(arrived, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        lds_barrier();
        if (!last_s) break;
        for (int it = tid; it < p.rows * (DB / 4); it += kThreads) {
          const int lrow = it / (DB / 4), d = it % (DB / 4) * 4;
          if (d >= D) continue;
          f32x4_t v[kJoin];
          float2 x[kJoin];
#pragma unroll
          for (int k = 0; k < kJoin; ++k) {
            const uint32_t at = part_row(k0 + k * stride, lrow);
            x[k] = get_shared2(part_ml, k < n ? at * 8 : kNowhere);
            v[k] = get_shared(part_o, k < n ? (at * D + d) * 4 : kNowhere);
          }
          float mm = -INFINITY, ll = 0.f;
          f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < kJoin; ++k)
            if (k < n) mm = fmaxf(mm, x[k].x);
#pragma unroll
          for (int k = 0; k < kJoin; ++k)
            if (k < n) {
              const float f = __builtin_amdgcn_exp2f(x[k].x - finite_top(mm));
              ll += x[k].y * f;
              acc += v[k] * f;
            }
          if (root) {
            const auto y = out_row(p, lrow);
            write4(y.out + d, acc * (ll == 0.f ? 0.f : over_sum(a.c.v_scale, ll)));
            if (a.lse && d == 0) a.lse[y.lse] = log_sum(mm, ll);
          } else {
            const uint32_t at = part_row(k0, lrow);
            put_shared(part_o, (at * D + d) * 4, acc);
            // the row's other threads still read its sums: they are written after the loop
            if (d == 0) row_sums[lrow] = make_float2(mm, ll);
          }
        }
        lds_barrier();
        if (!root)
          for (int lrow = tid; lrow < p.rows; lrow += kThreads)
            put_shared2(part_ml, part_row(k0, lrow) * 8, row_sums[lrow].x, row_sums[lrow].y);
      }
    }
    lds_barrier();
  };

  // ---- the parts of the share; a part's first tile is on its way while the one before is
  // joined and written
  int x = share_start(work_, workers_, b_);
  const int x1 = share_start(work_, workers_, b_ + 1);
  int r = uniform(last_sum_at_most(sums, a.num_seqs, x));
  Part prev{};
  bool joining = false;
  for (;;) {
    const bool more = x < x1;
    const int D = here(a.c.dim), ps = here(a.c.page_shift), max_len = a.max_pages << ps;
    const uint32_t tok_b = (uint32_t)here((int)(a.c.token_stride * (long long)sizeof(C)));
    Part p{};
    unsigned base = 0, any_lo = 0, any_hi = 0, all_lo = 0, all_hi = 0, t = 0, t_end = 0;
    const_words_t table = const_words(a.table);
    const char *kbase = reinterpret_cast<const char*>(a.c.k), *vbase = reinterpret_cast<const char*>(a.c.v);

    struct Place {
      long long at[G];   // byte offset of each group
      bool ok[G];        // its page lies in the cache
    };
    auto page_of = [&](unsigned tile, int (&page)[G]) {   // raw ids; beyond the keys: none
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const unsigned key = base + tile * S::kKeys + 16 * i;
        page[i] = -1;
        if (tile < t_end && key < any_hi) page[i] = table[key >> ps];
      }
    };
    auto place_of = [&](unsigned tile, const int (&page)[G]) {
      Place y;
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const unsigned key = base + tile * S::kKeys + 16 * i;
        const int id = page_or_none(page[i], a.c.num_pages);
        y.ok[i] = id >= 0;
        y.at[i] = ((long long)(id >= 0 ? id : 0) * a.c.page_stride +
                   (long long)(key & ((1u << ps) - 1u)) * a.c.token_stride) * (long long)sizeof(C);
      }
      return y;
    };
    auto load_k = [&](const Place& y) {
#pragma unroll
      for (int i = 0; i < G; ++i)
#pragma unroll
        for (int f = 0; f < NK; ++f)
          K[i][f] = __builtin_bit_cast(uint4, load_words<4, kAux>(cells_at(kbase + y.at[i], y.ok[i]), kofs[NK > 1 ? f / 2 : f], f % 2 * 8 * tok_b));
    };
    auto load_v = [&](const Place& y) {
#pragma unroll
      for (int i = 0; i < 4 * G; ++i)
#pragma unroll
        for (int vb = 0; vb < VB; ++vb)
          V[vb][i] = load_words<VW, kAux>(cells_at(vbase + y.at[i / 4], y.ok[i / 4]), vofs[vb], (uint32_t)(i % 4) * tok_b);
    };
    int page[G];
    Place cur{}, nxt{};

    if (more) {
      SeqRows s = seq_rows(starts[r], starts[r + 1], lens[r], a.num_tokens, max_len);
      SeqSpan span = seq_span(s, a.window, step_log2);
      int blocks = row_blocks(s.n, group, kRowsLog2), seq_at = uniform(sums[r]);
      while (x >= seq_at + a.c.heads * blocks * span.steps) {   // the next sequence with new tokens
        ++r;
        s = seq_rows(starts[r], starts[r + 1], lens[r], a.num_tokens, max_len);
        span = seq_span(s, a.window, step_log2);
        blocks = row_blocks(s.n, group, kRowsLog2);
        seq_at = uniform(sums[r]);
      }
      const int unit = (int)((unsigned)(x - seq_at) / (unsigned)span.steps);
      p.start = s.start;
      p.at = seq_at + unit * span.steps;
      p.steps = span.steps;
      p.s0 = x - p.at;
      p.s1 = min(span.steps, x1 - p.at);
      p.kh = blocks == 1 ? unit : (int)((unsigned)unit / (unsigned)blocks);
      p.row0 = (unit - p.kh * blocks) * kRows;
      p.rows = min(kRows, s.n * group - p.row0);
      base = span.base;

      // rows of this wave, and its tiles: those of the part that any (all) of its rows see
      const int wrow0 = p.row0 + rw * 16 * RT, wrows = min(16 * RT, p.row0 + p.rows - wrow0);
      if (wrows > 0) {
        const KeyRange k0 = token_keys(fast_quot(wrow0, a.group), s.n, s.len, a.window);
        const KeyRange k1 = token_keys(fast_quot(wrow0 + wrows - 1, a.group), s.n, s.len, a.window);
        any_lo = k0.lo;
        any_hi = k1.hi;
        all_lo = k1.lo;
        all_hi = k0.hi;
      }
      const unsigned tile_end = (unsigned)p.s1 << tiles_log2;
      t = ((unsigned)p.s0 << tiles_log2) + kw;
      t_end = t;
      if (any_hi > any_lo) {
        t_end = min(tile_end, (any_hi - base + S::kKeys - 1) / S::kKeys);
        const unsigned first = any_lo > base ? (any_lo - base) / S::kKeys : 0u;
        if (first > t) t += (first - t + KW - 1) / KW * KW;
      }
      t = (unsigned)uniform((int)t);
      t_end = (unsigned)uniform((int)t_end);
      table = const_words(a.table + (size_t)r * a.ld_table);
      kbase += (long long)p.kh * a.c.head_stride * (long long)sizeof(C);
      vbase += (long long)p.kh * a.c.head_stride * (long long)sizeof(C);

      page_of(t, page);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const int row = wrow0 + rt * 16 + c16;
        const bool there = rt * 16 + c16 < wrows;
        const int i = there ? fast_quot(row, a.group) : 0, h = there ? p.kh * group + row - i * group : 0;
        const KeyRange k = token_keys(i, s.n, s.len, a.window);
        lo[rt] = there ? k.lo : 0;
        hi[rt] = there ? k.hi : 0;
        const T* src = reinterpret_cast<const T*>(a.q) + (size_t)(s.start + i) * a.ldq + (size_t)h * D;
#pragma unroll
        for (int f = 0; f < NQ; ++f) {
          int d;
          if constexpr (S::kF8) d = (f / 2) * 64 + g4 * 16 + (f & 1) * 8;
          else if constexpr (S::kF32) d = f * 16 + g4 * 4;
          else d = f * 32 + g4 * 8;
          q[rt][f] = keep_if(ld16(src + (d < D ? d : 0)), there && d < D);
        }
      }
      cur = place_of(t, page);
      load_k(cur);
      load_v(cur);
      page_of(t + KW, page);
    }
    if (joining) join(prev);
    if (!more) break;

#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      m[rt] = -INFINITY;
      l[rt] = 0.f;
#pragma unroll
      for (int j = 0; j < VB * EC; ++j) o[rt][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    bool odd = false;   // a value that is not finite was left out of the products
    const unsigned t_first = t;
    for (; t < t_end; t += KW) {
      const unsigned key0 = base + t * S::kKeys;
      nxt = place_of(t + KW, page);
      page_of(t + 2 * KW, page);
      if constexpr (NK > 1) {
#pragma unroll
        for (int i = 0; i < G; ++i)
#pragma unroll
          for (int f = 0; f < NK; f += 2) whole_keys(K[i][f], K[i][f + 1]);
      }
      // scores
      f32x4_t sc[RT][G];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int i = 0; i < G; ++i) {
          f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int f = 0; f < NK; ++f) {
            if constexpr (S::kF32) {
              acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(K[i][f].x), __uint_as_float(q[rt][f].x), acc, 0, 0, 0);
              acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(K[i][f].y), __uint_as_float(q[rt][f].y), acc, 0, 0, 0);
              acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(K[i][f].z), __uint_as_float(q[rt][f].z), acc, 0, 0, 0);
              acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(K[i][f].w), __uint_as_float(q[rt][f].w), acc, 0, 0, 0);
            } else if constexpr (S::kF8) {
              const uint4 k0 = fp8x8_to_bf16x8(make_uint2(K[i][f].x, K[i][f].y)), k1 = fp8x8_to_bf16x8(make_uint2(K[i][f].z, K[i][f].w));
              acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, k0), __builtin_bit_cast(bf16x8_t, q[rt][2 * f]), acc, 0, 0, 0);
              acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, k1), __builtin_bit_cast(bf16x8_t, q[rt][2 * f + 1]), acc, 0, 0, 0);
            } else {
              acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, K[i][f]), __builtin_bit_cast(bf16x8_t, q[rt][f]), acc, 0, 0, 0);
            }
          }
          sc[rt][i] = acc;
        }
      sched_fence();
      load_k(nxt);
      sched_fence();

      // weights: 2^(s - m)
      const bool partly = key0 < all_lo || key0 + S::kKeys > all_hi;   // some row does not see some key
      bool masked = partly;
#pragma unroll
      for (int i = 0; i < G; ++i) masked |= !cur.ok[i];
      masked = uniform((int)masked) != 0;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
        for (int i = 0; i < G; ++i) sc[rt][i] *= qs;
        if (masked) {
#pragma unroll
          for (int i = 0; i < G; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const unsigned key = key0 + 16 * i + 4 * g4 + k;
              sc[rt][i][k] = cur.ok[i] && key >= (unsigned)lo[rt] && key < (unsigned)hi[rt] ? sc[rt][i][k] : -INFINITY;
            }
        }
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < G; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) mx = fmaxf(mx, sc[rt][i][k]);
        mx = max_over_groups(mx);
        if (__any(mx > m[rt])) {
          const float mn = fmaxf(m[rt], mx), keep = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m[rt] - mn);
          m[rt] = mn;
          l[rt] *= keep;
#pragma unroll
          for (int j = 0; j < VB * EC; ++j) o[rt][j] *= keep;
        }
        const float mz = finite_top(m[rt]);
#pragma unroll
        for (int i = 0; i < G; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            sc[rt][i][k] = __builtin_amdgcn_exp2f(sc[rt][i][k] - mz);
            l[rt] += sc[rt][i][k];
          }
      }
      // Weight 0 times a value that is not finite would be NaN: values that no row sees are
      // cleared, and of those that some rows see and others do not, what is not finite
      // (added to the rows that see it at the part's end).
      if (partly) {
        bool found = false;
#pragma unroll
        for (int i = 0; i < 4 * G; ++i) {
          const unsigned key = key0 + 16 * (i / 4) + 4 * g4 + i % 4;
          const bool any = key >= any_lo && key < any_hi, all = key >= all_lo && key < all_hi;
#pragma unroll
          for (int vb = 0; vb < VB; ++vb)
#pragma unroll
            for (int k = 0; k < VW; ++k) {
              const uint32_t v = any ? V[vb][i].w[k] : 0u, clean = all ? v : without_odd<C>(v);
              found |= clean != v;
              V[vb][i].w[k] = clean;
            }
        }
        odd |= __any(found) != 0;
      }
      // o += weights times values
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        if constexpr (S::kF32) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int vb = 0; vb < VB; ++vb)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                o[rt][vb * 4 + e] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(V[vb][k].w[e]), sc[rt][0][k], o[rt][vb * 4 + e], 0, 0, 0);
        }
      }
      if constexpr (!S::kF32) {
        // the upper 16 bits of a weight, and the rest rounded to bf16; the rest of a weight
        // above 0 stays above 0, so that times an infinity it adds nothing but that infinity
        uint4 ph[RT], pl[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          uint32_t *hw = &ph[rt].x, *lw = &pl[rt].x;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float a0 = sc[rt][k / 2][2 * (k % 2)], a1 = sc[rt][k / 2][2 * (k % 2) + 1];
            const uint32_t u0 = __float_as_uint(a0), u1 = __float_as_uint(a1);
            hw[k] = __builtin_amdgcn_perm(u1, u0, 0x07060302u);
            const float b0 = fmaxf(a0 - __uint_as_float(u0 & 0xffff0000u), a0 > 0.f ? 1e-30f : 0.f);
            const float b1 = fmaxf(a1 - __uint_as_float(u1 & 0xffff0000u), a1 > 0.f ? 1e-30f : 0.f);
            lw[k] = bf16_pair(b0, b1);
          }
        }
#pragma unroll
        for (int vb = 0; vb < VB; ++vb)
#pragma unroll
          for (int e4 = 0; e4 < EC; e4 += 4) {   // 4 dims at a time, of this lane's 8 keys, as bf16 pairs
            uint32_t y[8][2];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if constexpr (S::kF8) {
                const int v = (int)V[vb][i].w[e4 / 4];
                y[i][0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, false));
                y[i][1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, true));
              } else {
                y[i][0] = V[vb][i].w[e4 / 2];
                y[i][1] = V[vb][i].w[e4 / 2 + 1];
              }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t sel = e & 1 ? 0x07060302u : 0x05040100u;
              const uint4 vt = make_uint4(__builtin_amdgcn_perm(y[1][e / 2], y[0][e / 2], sel),
                                          __builtin_amdgcn_perm(y[3][e / 2], y[2][e / 2], sel),
                                          __builtin_amdgcn_perm(y[5][e / 2], y[4][e / 2], sel),
                                          __builtin_amdgcn_perm(y[7][e / 2], y[6][e / 2], sel));
#pragma unroll
              for (int rt = 0; rt < RT; ++rt) {
                f32x4_t& d = o[rt][vb * EC + e4 + e];
                d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, vt), __builtin_bit_cast(bf16x8_t, pl[rt]), d, 0, 0, 0);
                d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, vt), __builtin_bit_cast(bf16x8_t, ph[rt]), d, 0, 0, 0);
              }
            }
          }
      }
      sched_fence();
      load_v(nxt);
      sched_fence();
      cur = nxt;
    }

    if (odd) {   // what was left out: key by key of this wave's tiles that some rows see and others do not
#pragma unroll 1
      for (unsigned tile = t_first; tile < t_end; tile += KW) {
        const unsigned key0 = base + tile * S::kKeys;
        if (key0 >= all_lo && key0 + S::kKeys <= all_hi) continue;
        int ids[G];
        page_of(tile, ids);
        const Place y = place_of(tile, ids);
#pragma unroll
        for (int i = 0; i < G; ++i)
#pragma unroll 1
          for (int j = 0; j < 16; ++j) {
            const unsigned key = key0 + 16 * i + j;
            if (key >= all_lo && key < all_hi) continue;
#pragma unroll
            for (int vb = 0; vb < VB; ++vb)
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int d = (vb * 16 + 4 * g4 + k) * EC;
                const Words<VW> cell = load_words<VW>(cells_at(vbase + y.at[i], y.ok[i]), d < D ? d * (uint32_t)sizeof(C) : kNowhere, j * tok_b);
#pragma unroll
                for (int e = 0; e < EC; ++e) {
                  const float v = cell_value<C>(cell, e);
                  const bool use = fabsf(v) == INFINITY || v != v;
#pragma unroll
                  for (int rt = 0; rt < RT; ++rt)
                    if (use && key >= (unsigned)lo[rt] && key < (unsigned)hi[rt]) o[rt][vb * EC + e][k] += v;
                }
              }
          }
      }
    }
    prev = p;
    joining = true;
    x = p.at + p.s1;
  }
}

template <typename C, int DB, int RT, int W, int RW, bool ONCE>
static void launch_shape(const AttentionArgs& a, hipStream_t stream, const KTimer& tm) {
  const uint32_t join = W > RW ? W * 16 * (AttnTile<C, DB>::kPitch + 2 * RT) : 2 * 16 * RT * RW;
  RAX_LAUNCH(tm, (paged_attention_kernel<C, DB, RT, W, RW, ONCE>), dim3(a.workers), dim3(64 * W),
             (uint32_t)sizeof(float) * (join + 2 * a.num_seqs), stream, a);
}
template <typename C, int DB, bool ONCE>
static void launch_rows(const AttentionArgs& a, hipStream_t stream, const KTimer& tm) {
  if (a.waves == 1) launch_shape<C, DB, 1, 1, 1, ONCE>(a, stream, tm);
  else if (a.row_tiles == 1) launch_shape<C, DB, 1, 4, 1, ONCE>(a, stream, tm);
  else launch_shape<C, DB, 2, 4, 1, ONCE>(a, stream, tm);
}
template <typename C, int DB> static void launch_reads(const AttentionArgs& a, hipStream_t stream, const KTimer& tm) {
  if (a.row_waves == 2) launch_shape<C, DB, 2, 4, 2, false>(a, stream, tm);
  else if (a.read_once) launch_rows<C, DB, true>(a, stream, tm);
  else launch_rows<C, DB, false>(a, stream, tm);
}
template <typename C> hipError_t launch_attention_of(const AttentionArgs& a, hipStream_t stream, const KTimer& tm) {
  if (a.c.dim <= 64) launch_reads<C, 64>(a, stream, tm);
  else if (a.c.dim <= 128) launch_reads<C, 128>(a, stream, tm);
  else launch_reads<C, 256>(a, stream, tm);
  return hipGetLastError();
}

}  // namespace rax
