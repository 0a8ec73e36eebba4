// Paged attention: out = softmax(scale q K^T) V over the cached keys a token sees, in one
// pass over the keys with a running maximum m and sum l (base 2, s = scale log2(e) q.k):
//   m' = max(m, max_j s_j),  l' = l 2^(m - m') + sum_j 2^(s_j - m'),
//   o' = o 2^(m - m') + sum_j 2^(s_j - m') v_j,   out = o / l,  lse = (m + log2 l) ln 2.
//
// What bounds it: reading the keys and values (2 * len * kv heads * dim elements a
// sequence); the work on each is done by the matrix cores in a small part of that time.
//
// Rows.  The new tokens of a sequence times the query heads of one kv head share its keys:
// row x = token * group + head.  A wave holds RT tiles of 16 rows; a workgroup of 4 waves
// has row_waves row groups, the other waves split the keys (key_waves = 4 / row_waves).
//
// Tiles.  Both products keep the rows in the matrix cores' column (lane % 16), so maxima,
// sums and the correction of o stay in the lane they are used in, and nothing passes
// through LDS between the products:
//   S^T = K Q^T: lane (c, g = lane / 16) gets row c's scores of keys 4 g + 0..3 of each
//   group of 16 keys; these are exactly its operand values of O^T = V^T P^T when the second product's
//   contraction index 8 g + i stands for key 4 g + i of the first (i < 4) or second group.
//   K is the operand as it lies in memory (a lane loads 16 bytes of one key).  V needs
//   several keys of one dim in a register: a lane loads EC consecutive dims of each of its
//   keys and the pairs are put together by one byte permutation each.  MFMA e of a block
//   then computes the dims {m EC + e}, so a lane ends with EC consecutive dims of its row.
//   Weights enter the 16-bit product as two bf16 parts (2^-16 relative, not 2^-8): the
//   second product is far from binding.  e4m3 cells are widened to bf16, which is exact.
//   fp32 caches use the fp32 matrix cores, 4 keys (or dims) at a time, with no permutation.
// A tile's keys are loaded again as soon as its first product has read them, its values
// after the second, so every wave keeps 8 to 16 KB on the way.
//
// Split.  The steps (key_waves tiles) of all sequences, kv heads and row blocks form one
// line, cut into equal contiguous shares, one a workgroup, whatever the lengths.  What a
// workgroup has of a unit (sequence, head, row block) that others share goes to the
// workspace as (m, l, o); the last one to arrive adds the parts in order of the keys, so
// the result does not depend on which that is.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "device_util.h"
#include "kv.h"

namespace rax {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kAttnThreads = 256;
constexpr int kAttnWaves = kAttnThreads / 64;

// Read-only words at a wave-uniform index through the scalar cache (written by earlier
// launches only).
typedef const __attribute__((address_space(4))) int32_t* const_words_t;
__device__ __forceinline__ const_words_t const_words(const int32_t* p) { return (const_words_t)(uintptr_t)p; }
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Cells are read through buffer descriptors, whose base is a group of keys at one kv head:
// the lane's part of an address is one register, kept for all tiles, and a lane whose
// offset is kNowhere, or a group whose descriptor is empty (a page outside the cache, a
// tile past the last), reads zeros without a memory access or a branch.
constexpr uint32_t kNowhere = 0x80000000u;
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ __amdgpu_buffer_rsrc_t cells_at(const char* base, bool ok) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, ok ? 0x7fffffff : 0, 0x00027000);
}
template <int N> struct Words {
  uint32_t w[N];
};
template <int N> __device__ __forceinline__ Words<N> load_words(__amdgpu_buffer_rsrc_t r, uint32_t ofs, uint32_t sofs) {
  Words<N> x;
  if constexpr (N == 4) {
    const u32x4_t v = __builtin_amdgcn_raw_buffer_load_b128(r, ofs, sofs, 0);
    x.w[0] = v[0]; x.w[1] = v[1]; x.w[2] = v[2]; x.w[3] = v[3];
  } else if constexpr (N == 2) {
    const u32x2_t v = __builtin_amdgcn_raw_buffer_load_b64(r, ofs, sofs, 0);
    x.w[0] = v[0]; x.w[1] = v[1];
  } else {
    x.w[0] = __builtin_amdgcn_raw_buffer_load_b32(r, ofs, sofs, 0);
  }
  return x;
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
  static constexpr int kGroups = kF32 ? 1 : 2;                 // groups of 16 keys in a tile
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

// four finished dims of a row: weights' sum l at maximum m
template <typename T>
__device__ __forceinline__ void write_row(const AttentionArgs& a, int t, int h, int d, f32x4_t o, float m, float l) {
  const float f = m == -INFINITY ? 0.f : a.c.v_scale / l;
  T* out = reinterpret_cast<T*>(a.out) + (size_t)t * a.ldo + (size_t)h * a.c.dim + d;
  f32x4_t y = {0.f, 0.f, 0.f, 0.f};
  if (m != -INFINITY) y = o * f;
  if constexpr (sizeof(T) == 4) *reinterpret_cast<f32x4_t*>(out) = y;
  else *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
  if (a.lse && d == 0)
    a.lse[(size_t)t * a.q_heads + h] = m == -INFINITY ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
}

template <typename C, int DB, int RT>
__global__ __launch_bounds__(kAttnThreads, DB > 128 ? 1 : 2) void paged_attention_kernel(AttentionArgs a) {
  using S = AttnTile<C, DB>;
  using T = std::conditional_t<S::kF32, float, uint16_t>;
  constexpr int G = S::kGroups, NK = S::kKLoads, NQ = S::kQFrags, EC = S::kEC, VB = S::kVB, VW = S::kVW;
  __shared__ float buf[kAttnWaves][16][S::kPitch];
  __shared__ float ml[kAttnWaves][RT][16][2];
  __shared__ int part_s[kAttnWaves], start_s, seq_s, last_s;
  static_assert(sizeof(buf) >= 8 * kMaxParts * sizeof(float), "the join's weights lie in buf");

  const int tid = threadIdx.x, lane = lane_id(), w = uniform(tid >> 6);
  const int c16 = lane & 15, g4 = lane >> 4;
  const int D = a.c.dim, ps = a.c.page_shift, max_len = a.max_pages << ps, group = a.group_size;
  const int rw_log2 = a.row_waves >> 1, row_waves = a.row_waves, kw_log2 = 2 - rw_log2, key_waves = 1 << kw_log2;   // 1, 2 or 4
  const int rw = w & (row_waves - 1), kw = w >> rw_log2;
  constexpr int kRowsLog2 = RT == 2 ? 5 : 4, kKeysLog2 = S::kF32 ? 4 : 5;
  const int rows_log2 = kRowsLog2 + rw_log2, rows_wg = 1 << rows_log2;
  const int tiles_log2 = a.step_log2 - kKeysLog2;   // tiles of a step
  const const_words_t lens = const_words(a.seq_lens), starts = const_words(a.query_start);

  // ---- this workgroup's share: the line's length, then the sequence that its first step falls in
  auto steps_of = [&](const SeqRows& s) {
    return a.c.heads * row_blocks(s.n, group, rows_log2) * seq_span(s, a.window, a.step_log2).steps;
  };
  const int per = (a.num_seqs + kAttnThreads - 1) / kAttnThreads;
  const int r0 = min(a.num_seqs, tid * per), r1 = min(a.num_seqs, r0 + per);
  int mine = 0;
  for (int r = r0; r < r1; ++r) {
    const SeqRows s = seq_rows(a.query_start[r], a.query_start[r + 1], a.seq_lens[r], a.num_tokens, max_len);
    mine += steps_of(s);
  }
  int scan = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(scan, d);
    if (lane >= d) scan += y;
  }
  if (lane == 63) part_s[w] = scan;
  __syncthreads();
  int work = 0, before = scan - mine;
#pragma unroll
  for (int v = 0; v < kAttnWaves; ++v) {
    if (v < w) before += part_s[v];
    work += part_s[v];
  }
  work = uniform(work);
  if (work == 0) return;
  const int full = (work + a.min_steps - 1) / a.min_steps;
  const int workers = full < (long long)gridDim.x ? (int)full : (int)gridDim.x;
  // neighbouring shares on one XCD: the row blocks of a head read its keys from one L2
  const int b = (int)(blockIdx.x % kXcds) * (int)(gridDim.x / kXcds) + (int)(blockIdx.x / kXcds);
  if (b >= workers) return;
  const int x0 = share_start(work, workers, b), x1 = share_start(work, workers, b + 1);
  if (mine > 0 && x0 >= before && x0 < before + mine) {
    int at = before;
    for (int r = r0; r < r1; ++r) {
      const SeqRows s = seq_rows(a.query_start[r], a.query_start[r + 1], a.seq_lens[r], a.num_tokens, max_len);
      const int n = steps_of(s);
      if (x0 < at + n) {
        seq_s = r;
        start_s = at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  int r = uniform(seq_s);
  int seq_at = uniform(start_s);

  const uint32_t tok_b = (uint32_t)a.c.token_stride * (uint32_t)sizeof(C);   // below 2^27
  const float qs = a.scale * a.c.k_scale * 1.44269504088896341f;
  uint32_t kofs[NK], vofs[VB];   // lane's place in a group of keys, of values
#pragma unroll
  for (int f = 0; f < NK; ++f)
    kofs[f] = f * S::kKElems * 4 + g4 * S::kKElems < D ? (uint32_t)c16 * tok_b + 16u * g4 + 64u * f : kNowhere;
#pragma unroll
  for (int vb = 0; vb < VB; ++vb) {
    const int d = (vb * 16 + c16) * EC;
    vofs[vb] = d < D ? (uint32_t)(4 * g4) * tok_b + d * (uint32_t)sizeof(C) : kNowhere;
  }

  for (int x = x0; x < x1;) {
    const SeqRows s = seq_rows(starts[r], starts[r + 1], lens[r], a.num_tokens, max_len);
    const SeqSpan span = seq_span(s, a.window, a.step_log2);
    const int blocks = row_blocks(s.n, group, rows_log2), seq_work = a.c.heads * blocks * span.steps;
    if (x >= seq_at + seq_work) {
      seq_at += seq_work;
      ++r;
      continue;
    }
    const int unit = (int)((unsigned)(x - seq_at) / (unsigned)span.steps), unit_at = seq_at + unit * span.steps;
    const int s0 = x - unit_at, s1 = min(span.steps, x1 - unit_at);
    const int kh = blocks == 1 ? unit : (int)((unsigned)unit / (unsigned)blocks), row0 = (unit - kh * blocks) * rows_wg;
    const int rows = min(rows_wg, s.n * group - row0);
    x = unit_at + s1;

    // ---- rows of this wave: queries, the keys each sees
    const int wrow0 = row0 + rw * 16 * RT, wrows = min(16 * RT, row0 + rows - wrow0);
    uint4 q[RT][NQ];
    int lo[RT], hi[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int row = wrow0 + rt * 16 + c16;
      const bool there = rt * 16 + c16 < wrows;
      const int i = there ? fast_quot(row, a.group) : 0, h = there ? kh * group + row - i * group : 0;
      const KeyRange k = token_keys(i, s.n, s.len, a.window);
      lo[rt] = there ? k.lo : 0;
      hi[rt] = there ? k.hi : 0;
      const T* p = reinterpret_cast<const T*>(a.q) + (size_t)(s.start + i) * a.ldq + (size_t)h * D;
#pragma unroll
      for (int f = 0; f < NQ; ++f) {
        int d;
        if constexpr (S::kF8) d = (f / 2) * 64 + g4 * 16 + (f & 1) * 8;
        else if constexpr (S::kF32) d = f * 16 + g4 * 4;
        else d = f * 32 + g4 * 8;
        q[rt][f] = keep_if(ld16(p + (d < D ? d : 0)), there && d < D);
      }
    }
    float m[RT], l[RT];
    f32x4_t o[RT][VB * EC];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      m[rt] = -INFINITY;
      l[rt] = 0.f;
#pragma unroll
      for (int j = 0; j < VB * EC; ++j) o[rt][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }

    // ---- tiles of this wave: those of the share that any (all) of its rows see
    unsigned any_lo = 0, any_hi = 0, all_lo = 0, all_hi = 0;
    if (wrows > 0) {
      const KeyRange k0 = token_keys(fast_quot(wrow0, a.group), s.n, s.len, a.window);
      const KeyRange k1 = token_keys(fast_quot(wrow0 + wrows - 1, a.group), s.n, s.len, a.window);
      any_lo = k0.lo;
      any_hi = k1.hi;
      all_lo = k1.lo;
      all_hi = k0.hi;
    }
    const unsigned tile_end = (unsigned)s1 << tiles_log2;
    unsigned t = ((unsigned)s0 << tiles_log2) + kw, t_end = t;
    if (any_hi > any_lo) {
      t_end = min(tile_end, (any_hi - span.base + S::kKeys - 1) / S::kKeys);
      const unsigned first = any_lo > span.base ? (any_lo - span.base) / S::kKeys : 0u;
      if (first > t) t += (first - t + key_waves - 1) >> kw_log2 << kw_log2;
    }
    t = (unsigned)uniform((int)t);
    t_end = (unsigned)uniform((int)t_end);
    const const_words_t table = const_words(a.table + (size_t)r * a.ld_table);
    const char* kbase = reinterpret_cast<const char*>(a.c.k) + (long long)kh * a.c.head_stride * (long long)sizeof(C);
    const char* vbase = reinterpret_cast<const char*>(a.c.v) + (long long)kh * a.c.head_stride * (long long)sizeof(C);

    struct Place {
      long long at[G];   // byte offset of each group
      bool ok[G];        // its page lies in the cache
    };
    auto page_of = [&](unsigned tile, int (&page)[G]) {   // raw ids; beyond the keys: none
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const unsigned key = span.base + tile * S::kKeys + 16 * i;
        page[i] = -1;
        if (tile < t_end && key < any_hi) page[i] = table[key >> ps];
      }
    };
    auto place_of = [&](unsigned tile, const int (&page)[G]) {
      Place p;
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const unsigned key = span.base + tile * S::kKeys + 16 * i;
        const int id = page_or_none(page[i], a.c.num_pages);
        p.ok[i] = id >= 0;
        p.at[i] = ((long long)(id >= 0 ? id : 0) * a.c.page_stride +
                   (long long)(key & ((1u << ps) - 1u)) * a.c.token_stride) * (long long)sizeof(C);
      }
      return p;
    };
    uint4 K[G][NK];
    Words<VW> V[VB][4 * G];
    auto load_k = [&](const Place& p) {
#pragma unroll
      for (int i = 0; i < G; ++i)
#pragma unroll
        for (int f = 0; f < NK; ++f)
          K[i][f] = __builtin_bit_cast(uint4, load_words<4>(cells_at(kbase + p.at[i], p.ok[i]), kofs[f], 0));
    };
    auto load_v = [&](const Place& p) {
#pragma unroll
      for (int i = 0; i < 4 * G; ++i)
#pragma unroll
        for (int vb = 0; vb < VB; ++vb) 
          V[vb][i] = load_words<VW>(cells_at(vbase + p.at[i / 4], p.ok[i / 4]), vofs[vb], (uint32_t)(i % 4) * tok_b);
    };

    int page[G];
    Place cur{}, nxt{};
    if (t < t_end) {
      page_of(t, page);
      cur = place_of(t, page);
      load_k(cur);
      load_v(cur);
      page_of(t + key_waves, page);
    }
    for (; t < t_end; t += key_waves) {
      const unsigned key0 = span.base + t * S::kKeys;
      nxt = place_of(t + key_waves, page);
      page_of(t + 2 * key_waves, page);
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
      bool masked = key0 < all_lo || key0 + S::kKeys > all_hi;
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
        const float mz = m[rt] == -INFINITY ? 0.f : m[rt];
#pragma unroll
        for (int i = 0; i < G; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            sc[rt][i][k] = __builtin_amdgcn_exp2f(sc[rt][i][k] - mz);
            l[rt] += sc[rt][i][k];
          }
      }
      // Weight 0 times a value that is not finite would be NaN: values that no row sees
      // are cleared; where some row sees such a value and others may not, row by row.
      bool rowwise = false;
      if (masked) {
        bool odd = false;
#pragma unroll
        for (int i = 0; i < 4 * G; ++i) {
          const unsigned key = key0 + 16 * (i / 4) + 4 * g4 + i % 4;
          const uint32_t keep = cur.ok[i / 4] && key >= any_lo && key < any_hi ? 0xffffffffu : 0u;
#pragma unroll
          for (int vb = 0; vb < VB; ++vb)
#pragma unroll
            for (int k = 0; k < VW; ++k) {
              const uint32_t v = V[vb][i].w[k] & keep;
              V[vb][i].w[k] = v;
              if constexpr (S::kF32) odd |= (v & 0x7f800000u) == 0x7f800000u;
              else if constexpr (S::kF8) odd |= (((v & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0u;
              else odd |= (v & 0x7f80u) == 0x7f80u || (v & 0x7f800000u) == 0x7f800000u;
            }
        }
        rowwise = __any(odd);
      }
      // o += weights times values.  Row by row (row >= 0): the values that this row does not
      // see cleared, and only its sums kept.
      auto values = [&](auto row_by_row, int row, f32x4_t (&acc)[VB * EC], const f32x4_t (&p)[G], int rt) {
        constexpr bool kRow = decltype(row_by_row)::value;
        uint32_t keep[4 * G];
#pragma unroll
        for (int i = 0; i < 4 * G; ++i) {
          keep[i] = 0xffffffffu;
          if constexpr (kRow) {
            const unsigned key = key0 + 16 * (i / 4) + 4 * g4 + i % 4;
            const unsigned rlo = (unsigned)__builtin_amdgcn_readlane(lo[rt], row), rhi = (unsigned)__builtin_amdgcn_readlane(hi[rt], row);
            keep[i] = key >= rlo && key < rhi ? 0xffffffffu : 0u;
          }
        }
        auto begin = [&](const f32x4_t& d) { return kRow ? f32x4_t{0.f, 0.f, 0.f, 0.f} : d; };
        auto finish = [&](f32x4_t& d, f32x4_t x) {
          if constexpr (!kRow) d = x;
          else if (c16 == row) d += x;
        };
        if constexpr (S::kF32) {
#pragma unroll
          for (int vb = 0; vb < VB; ++vb)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              f32x4_t x = begin(acc[vb * 4 + e]);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                x = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(V[vb][k].w[e] & keep[k]), p[0][k], x, 0, 0, 0);
              finish(acc[vb * 4 + e], x);
            }
        } else {
          // the upper 16 bits of a weight, and the rest rounded to bf16; the rest of a weight
          // above 0 stays above 0, so that times an infinity it adds nothing but that infinity
          uint4 ph, pl;
          uint32_t *hw = &ph.x, *lw = &pl.x;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float a0 = p[k / 2][2 * (k % 2)], a1 = p[k / 2][2 * (k % 2) + 1];
            const uint32_t u0 = __float_as_uint(a0), u1 = __float_as_uint(a1);
            hw[k] = __builtin_amdgcn_perm(u1, u0, 0x07060302u);
            const float b0 = fmaxf(a0 - __uint_as_float(u0 & 0xffff0000u), a0 > 0.f ? 1e-30f : 0.f);
            const float b1 = fmaxf(a1 - __uint_as_float(u1 & 0xffff0000u), a1 > 0.f ? 1e-30f : 0.f);
            const bf16x2_t bb = {(__bf16)b0, (__bf16)b1};
            lw[k] = __builtin_bit_cast(uint32_t, bb);
          }
#pragma unroll
          for (int vb = 0; vb < VB; ++vb) {
            // 4 dims at a time: words wq and wq + 1 of 8 keys as bf16 pairs
#pragma unroll
            for (int e4 = 0; e4 < EC; e4 += 4) {
              uint32_t x[8][2];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                if constexpr (S::kF8) {
                  const int v = (int)(V[vb][i].w[e4 / 4] & keep[i]);
                  x[i][0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, false));
                  x[i][1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, true));
                } else {
                  x[i][0] = V[vb][i].w[e4 / 2] & keep[i];
                  x[i][1] = V[vb][i].w[e4 / 2 + 1] & keep[i];
                }
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t sel = e & 1 ? 0x07060302u : 0x05040100u;
                const uint4 vt = make_uint4(__builtin_amdgcn_perm(x[1][e / 2], x[0][e / 2], sel),
                                            __builtin_amdgcn_perm(x[3][e / 2], x[2][e / 2], sel),
                                            __builtin_amdgcn_perm(x[5][e / 2], x[4][e / 2], sel),
                                            __builtin_amdgcn_perm(x[7][e / 2], x[6][e / 2], sel));
                f32x4_t d = begin(acc[vb * EC + e4 + e]);
                d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, vt), __builtin_bit_cast(bf16x8_t, pl), d, 0, 0, 0);
                d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, vt), __builtin_bit_cast(bf16x8_t, ph), d, 0, 0, 0);
                finish(acc[vb * EC + e4 + e], d);
              }
            }
          }
        }
      };
      if (!rowwise) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) values(std::false_type{}, 0, o[rt], sc[rt], rt);
      } else {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll 1
          for (int row = 0; row < 16; ++row) values(std::true_type{}, row, o[rt], sc[rt], rt);
      }
      sched_fence();
      load_v(nxt);
      sched_fence();
      cur = nxt;
    }

    // ---- join of the workgroup's waves; then the output, or a part for the workspace
    const bool whole = s0 == 0 && s1 == span.steps;
    const int first_wg = whole ? b : share_owner(work, workers, unit_at);
    const int slot = s0 == 0 ? 2 * b + 1 : 2 * b;
    const uint32_t slot_row = (uint32_t)slot * a.part_rows;   // the workspace stays below 2^31 bytes
    const auto part_o = cells_at(reinterpret_cast<const char*>(a.part_o), true);
    const auto part_ml = cells_at(reinterpret_cast<const char*>(a.part_ml), true);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      l[rt] = sum_over_groups(l[rt]);
      if (g4 == 0) {
        ml[w][rt][c16][0] = m[rt];
        ml[w][rt][c16][1] = l[rt];
      }
    }
    __syncthreads();
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      float top = m[rt];
      for (int v = rw; v < kAttnWaves; v += row_waves) top = fmaxf(top, ml[v][rt][c16][0]);
      const float f = m[rt] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m[rt] - top);
#pragma unroll
      for (int vb = 0; vb < VB; ++vb) {
        if (rt + vb > 0) __syncthreads();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float* d = &buf[w][c16][(4 * g4 + k) * EC];
#pragma unroll
          for (int e = 0; e < EC; e += 4)
            *reinterpret_cast<f32x4_t*>(d + e) = f32x4_t{o[rt][vb * EC + e][k] * f, o[rt][vb * EC + e + 1][k] * f,
                                                        o[rt][vb * EC + e + 2][k] * f, o[rt][vb * EC + e + 3][k] * f};
        }
        __syncthreads();
        constexpr int kChunks = 4 * EC;   // of 4 dims
        for (int it = tid; it < row_waves * 16 * kChunks; it += kAttnThreads) {
          const int d4 = it % kChunks, y = it / kChunks, row16 = y % 16, rv = y / 16;
          const int lrow = rv * 16 * RT + rt * 16 + row16, d = vb * 16 * EC + d4 * 4;
          if (lrow >= rows || d >= D) continue;
          float mm = -INFINITY, ll = 0.f;
          f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
          for (int v = rv; v < kAttnWaves; v += row_waves) mm = fmaxf(mm, ml[v][rt][row16][0]);
          for (int v = rv; v < kAttnWaves; v += row_waves) {
            const float mv = ml[v][rt][row16][0];
            if (mv != -INFINITY) ll += ml[v][rt][row16][1] * __builtin_amdgcn_exp2f(mv - mm);
            acc += *reinterpret_cast<const f32x4_t*>(&buf[v][row16][d4 * 4]);
          }
          if (whole) {
            const int row = row0 + lrow, i = fast_quot(row, a.group), h = kh * group + row - i * group;
            write_row<T>(a, s.start + i, h, d, acc, mm, ll);
          } else {
            put_shared(part_o, ((slot_row + lrow) * D + d) * 4, acc);
            if (d == 0) put_shared2(part_ml, (slot_row + lrow) * 8, mm, ll);
          }
        }
      }
    }
    if (!whole) {
      const int last_wg = share_owner(work, workers, unit_at + span.steps - 1), parts = last_wg - first_wg + 1;
      stores_done();
      __syncthreads();
      if (tid == 0) {
        const int n = __hip_atomic_fetch_add(&a.arrived[first_wg], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        last_s = n == parts - 1;
        if (last_s) __hip_atomic_store(&a.arrived[first_wg], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      __syncthreads();
      if (last_s) {
        float* weight = &buf[0][0][0];   // [8][parts]
        for (int y0 = 0; y0 < rows; y0 += 8) {
          {   // 32 threads a row: maximum, sum, weights of the parts
            const int y = tid >> 5, i0 = tid & 31, lrow = y0 + y;
            float mm = -INFINITY, ll = 0.f;
            if (lrow < rows) {
              for (int p = i0; p < parts; p += 32)
                mm = fmaxf(mm, get_shared2(part_ml, ((uint32_t)part_slot(first_wg, p) * a.part_rows + lrow) * 8).x);
            }
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) mm = fmaxf(mm, __shfl_xor(mm, d));
            if (lrow < rows) {
              for (int p = i0; p < parts; p += 32) {
                const float2 x2 = get_shared2(part_ml, ((uint32_t)part_slot(first_wg, p) * a.part_rows + lrow) * 8);
                const float f = x2.x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(x2.x - mm);
                weight[y * kMaxParts + p] = f;
                ll += x2.y * f;
              }
            }
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) ll += __shfl_xor(ll, d);
            if (i0 == 0) {
              ml[0][0][y][0] = mm;
              ml[0][0][y][1] = ll;
            }
          }
          __syncthreads();
          for (int it = tid; it < 8 * DB / 4; it += kAttnThreads) {
            const int y = it / (DB / 4), d = it % (DB / 4) * 4, lrow = y0 + y;
            if (lrow >= rows || d >= D) continue;
            f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
            for (int p0 = 0; p0 < parts; p0 += 8) {
              f32x4_t v[8];
#pragma unroll
              for (int p = 0; p < 8; ++p)
                v[p] = get_shared(part_o, p0 + p < parts ? (((uint32_t)part_slot(first_wg, p0 + p) * a.part_rows + lrow) * D + d) * 4 : kNowhere);
#pragma unroll
              for (int p = 0; p < 8; ++p)
                if (p0 + p < parts) acc += weight[y * kMaxParts + p0 + p] * v[p];
            }
            const int row = row0 + lrow, i = fast_quot(row, a.group), h = kh * group + row - i * group;
            write_row<T>(a, s.start + i, h, d, acc, ml[0][0][y][0], ml[0][0][y][1]);
          }
          __syncthreads();
        }
      }
    }
    __syncthreads();
  }
}

template <typename C, int DB>
static void launch_rows(const AttentionArgs& a, hipStream_t stream, const KTimer& tm) {
  const dim3 grid(a.workers), block(kAttnThreads);
  if (a.row_tiles == 1)
    RAX_LAUNCH(tm, (paged_attention_kernel<C, DB, 1>), grid, block, 0u, stream, a);
  else
    RAX_LAUNCH(tm, (paged_attention_kernel<C, DB, 2>), grid, block, 0u, stream, a);
}
template <typename C> static void launch_dim(const AttentionArgs& a, hipStream_t stream, const KTimer& tm) {
  if (a.c.dim <= 64) launch_rows<C, 64>(a, stream, tm);
  else if (a.c.dim <= 128) launch_rows<C, 128>(a, stream, tm);
  else launch_rows<C, 256>(a, stream, tm);
}

hipError_t launch_paged_attention(const AttentionArgs& a, hipStream_t stream, const KTimer& tm) {
  if (a.dtype == LORA_F32) launch_dim<float>(a, stream, tm);
  else if (a.c.dtype == LORA_FP8E4M3) launch_dim<uint8_t>(a, stream, tm);
  else launch_dim<uint16_t>(a, stream, tm);
  return hipGetLastError();
}

}  // namespace rax
