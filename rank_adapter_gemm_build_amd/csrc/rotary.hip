// Rotary append: the rotary turn of a step's q and k heads, and its keys and values into
// the paged cache.
//
// Pair i of a head at position p turns by the angle p f_i: (a, b) -> amplitude * (a cos -
// b sin, a sin + b cos).  f_i is kept in turns a position as the sum of two doubles, and the whole
// turns drop out inside an fma: the fraction is good to 2^-50 of a turn while p f_i is below 2^50
// turns, then to 2^-26 in fp32 for 16-bit rows. (One double alone: 2^-25 at f = 1 and 31-bit
// positions, and in proportion for faster frequencies; 4425 tokens take 21.2 us either way, 64 4.4.)
//
// What bounds it: reading the rows and writing q and the cells once.  The cosines of a
// token serve all of its heads, so a workgroup takes whole tokens (several of a few short
// heads) and keeps them in LDS; its loads are on their way while they are computed.
// Everything moves in chunks of 16 bytes of a row (V values: 8 bf16 or 4 fp32), two a
// thread and item, so that neighbouring lanes have neighbouring chunks; stores bypass (4425
// rows of 32 + 2 * 8 heads of 128: 28.9 -> 24.2 us; with two neighbouring chunks a lane they
// would cost instead, 32.9 -> 35.4):
//   - pairs (2i, 2i + 1): a chunk holds whole pairs; two chunks half a head apart;
//   - pairs (i, i + half), half a multiple of V: a chunk and the one half away;
//   - any other half: the chunks' partners are not aligned, so the turned heads go through
//     LDS, kRotarySlice bytes of heads at a time, and are picked up value by value.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "device_util.h"
#include "kv.h"

namespace rax {

constexpr int kRotaryThreads = 256, kRotaryTokens = 16, kRotarySlice = 16384;

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// a chunk of a row as values
__device__ __forceinline__ void to_floats(uint4 c, float (&x)[8]) { unpack8(c, x); }
__device__ __forceinline__ void to_floats(uint4 c, float (&x)[4]) {
  x[0] = __uint_as_float(c.x); x[1] = __uint_as_float(c.y); x[2] = __uint_as_float(c.z); x[3] = __uint_as_float(c.w);
}
__device__ __forceinline__ void store_cells(uint16_t* p, const float (&x)[8], float) {
  __builtin_nontemporal_store(u32x4_t{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                      pack_bf16x2(x[6], x[7])}, reinterpret_cast<u32x4_t*>(p));
}
__device__ __forceinline__ void store_cells(float* p, const float (&x)[4], float) {
  __builtin_nontemporal_store(u32x4_t{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                                      __float_as_uint(x[3])}, reinterpret_cast<u32x4_t*>(p));
}
__device__ __forceinline__ void store_cells(uint8_t* p, const float (&x)[8], float scale) {
  int w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(fp8_clamp(x[4 * i] / scale), fp8_clamp(x[4 * i + 1] / scale), 0, false);
    w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(fp8_clamp(x[4 * i + 2] / scale), fp8_clamp(x[4 * i + 3] / scale), w[i], true);
  }
  __builtin_nontemporal_store(u32x2_t{(uint32_t)w[0], (uint32_t)w[1]}, reinterpret_cast<u32x2_t*>(p));
}
__device__ __forceinline__ float one_float(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ float one_float(const float* p) { return *p; }

enum RotaryPairs { kInterleaved, kHalves, kOddHalves };

// T: activations, C: cache
template <typename T, typename C, int PAIRS>
__global__ __launch_bounds__(kRotaryThreads) void rotary_append_kernel(RotaryArgs a) {
  constexpr int V = 16 / (int)sizeof(T);   // values of a chunk
  // a slice of heads (kOddHalves), then cos, sin of [token][pair]: no more than the launch's
  // tokens need, for as many workgroups a compute unit as registers allow
  extern __shared__ uint4 lds[];
  __shared__ int slot_s[kRotaryTokens];
  uint4* slice = lds;
  float2* turn = reinterpret_cast<float2*>(lds + (PAIRS == kOddHalves ? kRotarySlice / 16 : 0));
  const int tid = threadIdx.x, D = a.c.dim, half = a.rot / 2, turned = a.q_heads + a.c.heads;
  const int t0 = blockIdx.x * a.tokens_wg, tokens = min(a.tokens_wg, a.num_tokens - t0);

  auto fill_turns = [&]() {
    for (int e = tid; e < tokens * half; e += kRotaryThreads) {
      const int t = fast_quot(e, a.per_half), i = e - t * half;
      const double p = a.positions[t0 + t], f = a.turns[2 * i];
      const double x = fma(p, f, -rint(p * f)) + p * a.turns[2 * i + 1];
      if constexpr (sizeof(T) == 4) {
        double s, c;
        sincospi(2.0 * x, &s, &c);
        turn[e] = make_float2((float)c * a.amplitude, (float)s * a.amplitude);
      } else {
        float s, c;
        sincospif(2.0f * (float)x, &s, &c);
        turn[e] = make_float2(c * a.amplitude, s * a.amplitude);
      }
    }
    if (tid < tokens) slot_s[tid] = a.slots[t0 + tid];
  };
  auto put = [&](int t, int h, int d, const float (&x)[V]) {
    if (h < a.q_heads) {
      store_cells(reinterpret_cast<T*>(a.q_out) + (size_t)(t0 + t) * a.ldq + h * D + d, x, 1.f);
      return;
    }
    const int slot = slot_s[t], page = slot >> a.c.page_shift;
    if (slot < 0 || page >= a.c.num_pages) return;
    const bool key = h < turned;
    C* p = reinterpret_cast<C*>(key ? a.c.k : a.c.v) + page * a.c.page_stride +
           (slot & ((1 << a.c.page_shift) - 1)) * a.c.token_stride + (h - (key ? a.q_heads : turned)) * a.c.head_stride + d;
    store_cells(p, x, key ? a.c.k_scale : a.c.v_scale);
  };
  const T* rows = reinterpret_cast<const T*>(a.qkv);
  const int per_head = D / (2 * V), heads = turned + a.c.heads;

  // items of two chunks, from head h0 on
  auto direct = [&](int h0, auto before_use) {
    const int per_token = (heads - h0) * per_head, items = tokens * per_token;
    constexpr int U = 2;
    bool first = true;
    for (int e0 = tid; first || e0 < items; e0 += U * kRotaryThreads) {
      uint4 c[U][2];
      int tt[U], hh[U], d0[U], d1[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int e = e0 + u * kRotaryThreads;
        tt[u] = -1;
        if (e < items) {
          tt[u] = tokens == 1 ? 0 : e / per_token;
          const int j = e - tt[u] * per_token, h = fast_quot(j, a.per_head), i = j - h * per_head;
          hh[u] = h0 + h;
          d0[u] = V * i;
          d1[u] = D / 2 + V * i;
          if (PAIRS == kHalves && hh[u] < turned) {
            const int j = i - half / V;   // the first half / V items hold pairs
            d0[u] = j < 0 ? V * i : a.rot + V * j;
            d1[u] = j < 0 ? half + V * i : (D + a.rot) / 2 + V * j;
          }
          const T* p = rows + (size_t)(t0 + tt[u]) * a.ldqkv + hh[u] * D;
          c[u][0] = ld16(p + d0[u]);
          c[u][1] = ld16(p + d1[u]);
        }
      }
      if (first) before_use();
      first = false;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (tt[u] < 0) continue;
        float x[V], y[V];
        to_floats(c[u][0], x);
        to_floats(c[u][1], y);
        if (hh[u] < turned) {
          const float2* cs = turn + tt[u] * half;
          if constexpr (PAIRS == kHalves) {
            if (d0[u] < half)
#pragma unroll
              for (int k = 0; k < V; ++k) {
                const float2 r = cs[d0[u] + k];
                const float v = x[k], w = y[k];
                x[k] = v * r.x - w * r.y;
                y[k] = v * r.y + w * r.x;
              }
          } else if constexpr (PAIRS == kInterleaved) {
#pragma unroll
            for (int k = 0; k < V; k += 2) {
              const int i = (d0[u] + k) / 2, j = (d1[u] + k) / 2;
              if (i < half) {
                const float2 r = cs[i];
                const float v = x[k], w = x[k + 1];
                x[k] = v * r.x - w * r.y;
                x[k + 1] = v * r.y + w * r.x;
              }
              if (j < half) {
                const float2 r = cs[j];
                const float v = y[k], w = y[k + 1];
                y[k] = v * r.x - w * r.y;
                y[k + 1] = v * r.y + w * r.x;
              }
            }
          }
        }
        put(tt[u], hh[u], d0[u], x);
        put(tt[u], hh[u], d1[u], y);
      }
    }
  };
  if constexpr (PAIRS != kOddHalves) {
    direct(0, [&]() {
      fill_turns();
      __syncthreads();
    });
  } else {
    direct(turned, [&]() {
      fill_turns();
      __syncthreads();
    });
    // turned heads: slices of whole heads through LDS
    const T* in = reinterpret_cast<const T*>(slice);
    const int slice_heads = kRotarySlice / (D * (int)sizeof(T)), chunks_head = D / V, all = tokens * turned;
    for (int g0 = 0; g0 < all; g0 += slice_heads) {
      const int n = min(slice_heads, all - g0);
      for (int e = tid; e < n * chunks_head; e += kRotaryThreads) {
        const int g = fast_quot(e, a.per_chunk), t = fast_quot(g0 + g, a.per_turned), h = g0 + g - t * turned;
        slice[e] = ld16(rows + (size_t)(t0 + t) * a.ldqkv + h * D + (e - g * chunks_head) * V);
      }
      __syncthreads();   // the whole slice is read: q_out may be the rows themselves
      for (int e = tid; e < n * chunks_head; e += kRotaryThreads) {
        const int g = fast_quot(e, a.per_chunk), t = fast_quot(g0 + g, a.per_turned), h = g0 + g - t * turned;
        const int d = (e - g * chunks_head) * V;
        const T* head = in + g * D;
        float x[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const int dk = d + k, i = dk < half ? dk : dk - half;
          x[k] = one_float(head + dk);
          if (dk < a.rot) {
            const float2 r = turn[t * half + i];
            const float w = one_float(head + (dk < half ? dk + half : i));
            x[k] = dk < half ? x[k] * r.x - w * r.y : w * r.y + x[k] * r.x;
          }
        }
        put(t, h, d, x);
      }
      __syncthreads();
    }
  }
}

template <int PAIRS>
static void launch_pairs(const RotaryArgs& a, const dim3& grid, hipStream_t stream, const KTimer& tm) {
  const dim3 block(kRotaryThreads);
  const uint32_t lds = (uint32_t)((PAIRS == kOddHalves ? kRotarySlice : 0) + a.tokens_wg * (a.rot / 2) * (int)sizeof(float2));
  if (a.dtype == LORA_F32)
    RAX_LAUNCH(tm, (rotary_append_kernel<float, float, PAIRS>), grid, block, lds, stream, a);
  else if (a.c.dtype == LORA_FP8E4M3)
    RAX_LAUNCH(tm, (rotary_append_kernel<uint16_t, uint8_t, PAIRS>), grid, block, lds, stream, a);
  else
    RAX_LAUNCH(tm, (rotary_append_kernel<uint16_t, uint16_t, PAIRS>), grid, block, lds, stream, a);
}

hipError_t launch_rotary_append(const RotaryArgs& args, hipStream_t stream, const KTimer& tm) {
  RotaryArgs a = args;
  const int values = a.dtype == LORA_F32 ? 4 : 8;   // of a chunk
  const int items = (a.q_heads + 2 * a.c.heads) * (a.c.dim / (2 * values));
  // two items a thread, as long as the chip stays full of workgroups
  a.tokens_wg = std::max(1, std::min({kRotaryTokens, 2 * kRotaryThreads / items, a.num_tokens / 1024}));
  a.per_half = fast_div(a.rot / 2);
  a.per_head = fast_div(a.c.dim / (2 * values));
  a.per_chunk = fast_div(a.c.dim / values);
  a.per_turned = fast_div(a.q_heads + a.c.heads);
  const dim3 grid((a.num_tokens + a.tokens_wg - 1) / a.tokens_wg);
  if (a.interleaved) launch_pairs<kInterleaved>(a, grid, stream, tm);
  else if (a.rot % (2 * values) == 0) launch_pairs<kHalves>(a, grid, stream, tm);
  else launch_pairs<kOddHalves>(a, grid, stream, tm);
  return hipGetLastError();
}

}  // namespace rax
