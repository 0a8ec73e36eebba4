// The shares of a line whose units have many rows, all of which see all keys: the products bound it, not the reading.
//
// A workgroup has kWideRows rows, 32 a wave, and its four waves share tiles of kWideKeys keys and values in LDS, twice: the next tile
// is on its way to one half while the other is used, with one barrier a tile.  As in the paged attention both products
// keep the rows in the matrix cores' column (here lane % 32), so that nothing passes through LDS between them:
//   S^T = K Q^T (32 keys, 16 dims a step): lane (r, h = lane / 32) gets row r's scores of keys 8 (i / 4) + 4 h + i % 4;
//   these are its operand values of O^T = V^T P^T when the second product's contraction index 8 h + j stands for key
//   8 (j / 4) + 4 h + j % 4 of a step's 16.
// K is read as it lies, 16 bytes of a key; V by transposing reads, which give a lane 4 keys of one dim.  Chunk c (16
// bytes) of key r lies at chunk c ^ (r % chunks) of its row for K, c ^ 2 (r % 4) for V: without that the keys of a read
// would all lie in the same banks.
//
// Weights are taken relative to a maximum that is moved only when a score passes it by 2^kSlack, so that most
// tiles leave o as it is; they enter the product in two bf16 parts, as in the paged attention.  16-bit cells
// go from memory to LDS directly; 8-bit ones are widened on the way.
//
// Measured, bf16, 1024 rows a kv head over 32000 keys: 255 us, 0.53 PFLOP/s of the products needed, 0.8 of those done, at
// 1.6 to 1.8 GHz, which this load lets the chip run at.  Of a wave's 4800 cycles a tile 1500 go by before the tile is there (its
// loads are issued late: a wave takes its page's id out of an array by its own number, and the compiler keeps that array in scratch, a
// store and a load before the address is known), 670 in the first product, 1450 in the exponentials, 1130 in the second product; the other wave of the SIMD works meanwhile, so the
// matrix cores are busy half of the time.  With each tile on its way for one and a half others, at two barriers a tile, 297 us.
#pragma once

#include "attention_kernels.h"
#include "shared.h"

namespace rax {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef short i16x4_t __attribute__((ext_vector_type(4)));

constexpr int kWideRows = 1 << kWideRowsLog2, kWideKeys = 1 << kWideKeysLog2;
constexpr float kSlack = 6.f;
constexpr int kSchedProducts = 0x8, kSchedReads = 0x100;   // instruction classes of a schedule: matrix products, LDS reads
// bytes of LDS: two tiles of keys and values
template <int D> constexpr int wide_lds() { return 2 * 2 * kWideKeys * D * 2; }

typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) u32x4_t lds_words;
typedef __attribute__((address_space(3))) i16x4_t lds_four;
__device__ __forceinline__ lds_char* lds_at(void* p) { return (lds_char*)(__attribute__((address_space(3))) void*)p; }

// 16 bytes of each lane from memory to LDS, at `to` on in order of the lanes.  The compiler is not told that LDS changes: it
// would wait for the next tile before every read of this one.  Arrival is waited for by stores_done.  m0, which holds the place in
// LDS and is read when the load is issued, is left as it was: the compiler reserves it, and takes no note of its being changed.
__device__ __forceinline__ void load_to_lds(u32x4_t r, uint32_t ofs, uint32_t sofs, lds_char* to) {
#if defined(__HIP_DEVICE_COMPILE__)
  uint32_t kept;
  asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, %4 offen lds\n\ts_mov_b32 m0, %0"
               : "=&s"(kept) : "s"((uint32_t)(uintptr_t)to), "v"(ofs), "s"(r), "s"(sofs) : "memory");
#endif
}
__device__ __forceinline__ u32x4_t cells_words(const char* base) {
  const uintptr_t u = reinterpret_cast<uintptr_t>(base);
  return u32x4_t{(uint32_t)uniform((int)(uint32_t)u), (uint32_t)uniform((int)((uint32_t)(u >> 32) & 0xffffu)), 0x7fffffffu, 0x00027000u};
}

// The rests of two weights (bf16, none negative), above 0 where the weights' upper parts are, so that times an infinity they add
// nothing but that infinity; the rest of a weight of 0 stays 0.  (As integers bf16 numbers that are not negative keep their order.)
__device__ __forceinline__ uint32_t above_zero(uint32_t rest, uint32_t upper) {
  typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
  const u16x2_t least = {0x0da2, 0x0da2};   // 1e-30
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, rest),
                                                                __builtin_elementwise_min(__builtin_bit_cast(u16x2_t, upper), least)));
}

template <typename C, int D, class Line>
__device__ __forceinline__ void attend_wide(const AttentionArgs& a, const Line line, float4* lds, const int* sums, int b_, int work_, int workers_,
                                            int step_log2) {
  constexpr bool kF8 = sizeof(C) == 1;
  constexpr int CPR = D * 2 / 16;                  // 16-byte chunks of a row in LDS
  constexpr int kTile = kWideKeys * D * 2;         // bytes of a tile of keys
  constexpr int kPieces = kTile / 1024 / 4;        // 1 KiB pieces of a tile that a wave moves
  constexpr int kPieceKeys = 1024 / (D * 2);       // keys of a piece
  constexpr int KS = D / 16, MB = D / 32;          // contraction steps of the first product, blocks of dims of the second
  const int tid = threadIdx.x, lane = lane_id(), w = uniform(tid >> 6), r32 = lane & 31, h = lane >> 5;
  const int ps = a.c.page_shift, max_len = a.max_pages << ps, group = a.group_size;
  const bool flip = a.scale < 0.f;                 // the products of -q: the scale is then positive
  // above 0, so that a score of minus infinity stays one; the least number above 0, times which no other score counts (below 2^-20)
  const float qs = fmaxf(fabsf(a.scale) * a.c.k_scale * 1.44269504088896341f, 1.4e-45f);
  lds_char* const tiles = lds_at(lds);             // [2][K, V]

  // a lane's place in a tile: of its key's chunks; of the key and 4 dims that it supplies to a transposing read
  int kread[KS], vread[MB];
#pragma unroll
  for (int f = 0; f < KS; ++f) kread[f] = r32 * (D * 2) + (((2 * f + h) ^ (r32 % CPR)) * 16);
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
    const int key = 4 * h + (lane % 16) / 4, dim = mb * 32 + (lane & 16) + 4 * (lane % 4);
    vread[mb] = key * (D * 2) + (((dim / 8) ^ (2 * (key % 4))) * 16) + dim % 8 * 2;
  }
  int x = share_start(work_, workers_, b_);
  const int x1 = share_start(work_, workers_, b_ + 1);
  int r = uniform(last_sum_at_most(sums, line.count(), x));
  while (x < x1) {
    // ---- the part
    SeqRows s = line.rows(r, max_len);
    SeqSpan span = line.span(r, s, step_log2);
    int blocks = row_blocks(s.n, group, kWideRowsLog2), seq_at = uniform(sums[r]);
    while (x >= seq_at + a.c.heads * blocks * span.steps) {   // the next sequence with rows and keys
      ++r;
      s = line.rows(r, max_len);
      span = line.span(r, s, step_log2);
      blocks = row_blocks(s.n, group, kWideRowsLog2);
      seq_at = uniform(sums[r]);
    }
    const int unit = (int)((unsigned)(x - seq_at) / (unsigned)span.steps);
    Part p{};
    p.start = s.start;
    p.at = seq_at + unit * span.steps;
    p.steps = span.steps;
    p.s0 = x - p.at;
    p.s1 = min(span.steps, x1 - p.at);
    p.kh = (int)((unsigned)unit / (unsigned)blocks);
    p.row0 = (unit - p.kh * blocks) * kWideRows;
    p.rows = min(kWideRows, s.n * group - p.row0);
    const unsigned keys = (unsigned)s.len;
    const const_words_t table = const_words(a.table + (size_t)line.table_row(r) * a.ld_table);

    // ---- queries: a row that is not there stands for the block's first (no branch: see attend_shares)
    const int lrow = w * 32 + r32;
    const bool there = lrow < p.rows;
    const int row = p.row0 + (there ? lrow : 0), qi = fast_quot(row, a.group), qh = p.kh * group + row - qi * group;
    const size_t out_row = (size_t)(s.start + qi) * a.q_heads + qh;
    uint4 q[KS];
    {
      const uint16_t* src = reinterpret_cast<const uint16_t*>(a.q) + (size_t)(s.start + qi) * a.ldq + (size_t)qh * D;
      const uint32_t sign = flip ? 0x80008000u : 0u;
#pragma unroll
      for (int f = 0; f < KS; ++f) {
        q[f] = ld16(src + f * 16 + h * 8);
        q[f] = make_uint4(q[f].x ^ sign, q[f].y ^ sign, q[f].z ^ sign, q[f].w ^ sign);
      }
    }

    // ---- tiles.  Keys past the last, and of pages outside the cache, are read from the cache's first page
    // and left out afterwards (absent: those groups of 16 keys, as bits)
    const char *kbase = reinterpret_cast<const char*>(a.c.k) + (long long)p.kh * a.c.head_stride * (long long)sizeof(C);
    const char *vbase = reinterpret_cast<const char*>(a.c.v) + (long long)p.kh * a.c.head_stride * (long long)sizeof(C);
    // wave w moves keys 16 w .. 16 w + 15 of a tile, kPieceKeys a piece
    const uint32_t tok_b = (uint32_t)a.c.token_stride * (uint32_t)sizeof(C);   // below 2^27
    const int key_in_piece = lane / CPR, slot = lane % CPR;
    uint32_t kofs[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      kofs[i] = (uint32_t)key_in_piece * tok_b + (uint32_t)((slot ^ ((i * kPieceKeys + key_in_piece) % CPR)) * 8 * (int)sizeof(C));
    const uint32_t vofs = (uint32_t)key_in_piece * tok_b + (uint32_t)((slot ^ (2 * (key_in_piece % 4))) * 8 * (int)sizeof(C));
    Words<2> staged[kF8 ? 2 * kPieces : 1];   // 8-bit cells on the way: 8 of a key a lane
    const auto page_ids = [&](unsigned tile, int (&page)[4]) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const unsigned key = tile * kWideKeys + 16 * g;
        page[g] = -1;
        if (key < keys) page[g] = table[key >> ps];
      }
    };
    const auto absent_of = [&](const int (&page)[4]) {
      int bits = 0;
#pragma unroll
      for (int g = 0; g < 4; ++g) bits |= (page_or_none(page[g], a.c.num_pages) < 0) << g;
      return uniform(bits);
    };
    const auto issue = [&](unsigned tile, const int (&page)[4], int half) {
      const int id = max(page_or_none(w < 2 ? (w == 0 ? page[0] : page[1]) : (w == 2 ? page[2] : page[3]), a.c.num_pages), 0);
      const unsigned key = tile * kWideKeys + 16u * w;
      const long long at = ((long long)id * a.c.page_stride + (long long)(key & ((1u << ps) - 1u)) * a.c.token_stride) * (long long)sizeof(C);
      lds_char* const to = tiles + half * 2 * kTile + w * kPieces * 1024;
      if constexpr (kF8) {
        const auto kr = cells_at(kbase + at, true), vr = cells_at(vbase + at, true);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          staged[2 * i] = load_words<2>(kr, kofs[i], (uint32_t)(i * kPieceKeys) * tok_b);
          staged[2 * i + 1] = load_words<2>(vr, vofs, (uint32_t)(i * kPieceKeys) * tok_b);
        }
      } else {
        const u32x4_t kr = cells_words(kbase + at), vr = cells_words(vbase + at);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          load_to_lds(kr, kofs[i], (uint32_t)(i * kPieceKeys) * tok_b, to + i * 1024);
          load_to_lds(vr, vofs, (uint32_t)(i * kPieceKeys) * tok_b, to + kTile + i * 1024);
        }
      }
    };
    const auto commit = [&](int half) {
      if constexpr (kF8) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          lds_char* const to = tiles + half * 2 * kTile + (w * kPieces + i) * 1024 + lane * 16;
          *(lds_words*)to = __builtin_bit_cast(u32x4_t, fp8x8_to_bf16x8(make_uint2(staged[2 * i].w[0], staged[2 * i].w[1])));
          *(lds_words*)(to + kTile) = __builtin_bit_cast(u32x4_t, fp8x8_to_bf16x8(make_uint2(staged[2 * i + 1].w[0], staged[2 * i + 1].w[1])));
        }
      }
    };

    f32x16_t o[MB];
    float m = -INFINITY, l = 0.f;
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[mb][i] = 0.f;
    const unsigned per_step = (unsigned)line.merged(r) << (step_log2 - kWideKeysLog2);   // tiles
    const unsigned t0 = (unsigned)p.s0 * per_step, t1 = min((unsigned)p.s1 * per_step, (keys + kWideKeys - 1u) / kWideKeys);
    int page[4], page_next[4];
    page_ids(t0, page);
    issue(t0, page, 0);
    commit(0);
    page_ids(t0 + 1, page_next);
    int half = 0;
#pragma unroll 1
    for (unsigned t = t0; t < t1; ++t, half ^= 1) {
      const int absent = absent_of(page);
      const bool masked = absent != 0 || (t + 1) * kWideKeys > keys;
      stores_done();      // this wave's pieces of the tile have arrived
      lds_barrier();      // and the others'; the other half is no longer read
#pragma unroll
      for (int g = 0; g < 4; ++g) page[g] = page_next[g];
      if (t + 1 < t1) {
        issue(t + 1, page, half ^ 1);
        page_ids(t + 2, page_next);
      }
      lds_char *kt = tiles + half * 2 * kTile, *vt = kt + kTile;
      if (masked) {       // values that are left out are cleared: their weight is 0, and they may be anything
        for (int c = tid; c < kTile / 16; c += 256) {
          const int key = c / CPR;
          if ((absent >> (key / 16) & 1) || t * kWideKeys + key >= keys) *(lds_words*)(vt + c * 16) = u32x4_t{0, 0, 0, 0};
        }
        lds_barrier();
      }
      f32x16_t sc[2];
      u32x4_t kf[2][KS];
      sched_fence();
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int f = 0; f < KS; ++f) kf[kb][f] = *(const lds_words*)(kt + kread[f] + kb * 32 * (D * 2));
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
        for (int i = 0; i < 16; ++i) sc[kb][i] = 0.f;
#pragma unroll
        for (int f = 0; f < KS; ++f)
          sc[kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, kf[kb][f]), __builtin_bit_cast(bf16x8_t, q[f]), sc[kb], 0, 0, 0);
      }
      // the second half's reads go between the first half's products
      __builtin_amdgcn_sched_group_barrier(kSchedReads, KS, 0);
#pragma unroll
      for (int f = 0; f < KS; ++f) {
        __builtin_amdgcn_sched_group_barrier(kSchedProducts, 1, 0);
        __builtin_amdgcn_sched_group_barrier(kSchedReads, 1, 0);
      }
      __builtin_amdgcn_sched_group_barrier(kSchedProducts, KS, 0);
      sched_fence();
      if (masked) {
        const int left = (int)(keys - t * kWideKeys), h4 = 4 * here_lane(h);   // keys from the tile's first on
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (h4 >= left - (kb * 32 + 8 * (i / 4) + i % 4) || (absent >> (2 * kb + i / 8) & 1)) sc[kb][i] = -INFINITY;
      }
      float mx = -INFINITY;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, sc[kb][i]);
      {
        const auto y = __builtin_amdgcn_permlane32_swap(__float_as_uint(mx), __float_as_uint(mx), false, false);
        mx = fmaxf(__uint_as_float(y[0]), __uint_as_float(y[1]));
      }
      mx *= qs;
      if (__any(mx > m + kSlack || (m == -INFINITY && mx > m))) {
        const float mn = fmaxf(m, mx), keep = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - mn);
        m = mn;
        l *= keep;
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) o[mb] *= keep;
      }
      const float mz = finite_top(m);
      uint4 ph[2][2], pl[2][2];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int s2 = 0; s2 < 2; ++s2) {
          uint32_t *hw = &ph[kb][s2].x, *lw = &pl[kb][s2].x;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float e[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              e[y] = __builtin_amdgcn_exp2f(fmaf(sc[kb][8 * s2 + 2 * k + y], qs, -mz));
              l += e[y];
            }
            const uint32_t u0 = __float_as_uint(e[0]), u1 = __float_as_uint(e[1]);
            hw[k] = __builtin_amdgcn_perm(u1, u0, 0x07060302u);
            lw[k] = above_zero(bf16_pair(e[0] - __uint_as_float(u0 & 0xffff0000u), e[1] - __uint_as_float(u1 & 0xffff0000u)), hw[k]);
          }
        }
      // o += weights times values, 16 keys at a time; the reads of the next 16 go between the products of these
      sched_fence();
      uint4 vf[4][MB];
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          lds_char* const at = vt + vread[mb] + ks * 16 * (D * 2);
          const uint2 v0 = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_four*)at));
          const uint2 v1 = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_four*)(at + 8 * D * 2)));
          vf[ks][mb] = make_uint4(v0.x, v0.y, v1.x, v1.y);
        }
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          const bf16x8_t v = __builtin_bit_cast(bf16x8_t, vf[ks][mb]);
          o[mb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, __builtin_bit_cast(bf16x8_t, pl[ks / 2][ks % 2]), o[mb], 0, 0, 0);
          o[mb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, __builtin_bit_cast(bf16x8_t, ph[ks / 2][ks % 2]), o[mb], 0, 0, 0);
        }
      __builtin_amdgcn_sched_group_barrier(kSchedReads, 2 * MB, 0);
#pragma unroll
      for (int i = 0; i < 3 * MB; ++i) {
        __builtin_amdgcn_sched_group_barrier(kSchedProducts, 2, 0);
        __builtin_amdgcn_sched_group_barrier(kSchedReads, 2, 0);
      }
      __builtin_amdgcn_sched_group_barrier(kSchedProducts, 2 * MB, 0);
      sched_fence();
      if (t + 1 < t1) commit(half ^ 1);
    }

    // ---- the part's results: the rows' state, or a place in the workspace
    {
      const auto y = __builtin_amdgcn_permlane32_swap(__float_as_uint(l), __float_as_uint(l), false, false);
      l = __uint_as_float(y[0]) + __uint_as_float(y[1]);
    }
    const bool whole = p.s0 == 0 && p.s1 == p.steps;
    const int first = whole ? b_ : share_owner(work_, workers_, p.at);
    const auto part_o = cells_at(reinterpret_cast<const char*>(line.part_o()), true);   // below 2^31 bytes
    const auto part_ml = cells_at(reinterpret_cast<const char*>(line.part_ml()), true);
    float2* const state_ml = reinterpret_cast<float2*>(line.state_ml());
    const uint32_t place = (uint32_t)part_slot(first, b_ - first) * kWideRows + (uint32_t)lrow;
    if (there) {
      if (h == 0) {
        if (whole) state_ml[out_row] = make_float2(m, l);
        else put_shared2(part_ml, place * 8, m, l);
      }
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int d = mb * 32 + 8 * i + 4 * h;
          const f32x4_t y = {o[mb][4 * i], o[mb][4 * i + 1], o[mb][4 * i + 2], o[mb][4 * i + 3]};
          if (whole) write4(line.state_o() + out_row * D + d, y);
          else put_shared(part_o, (place * D + d) * 4, y);
        }
    }
    lds_barrier();
    x = p.at + p.s1;
  }
}

}  // namespace rax
