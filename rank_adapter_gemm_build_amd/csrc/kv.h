// Launchers of the operators between the packed q/k/v projection and the o projection:
// page plan, rotary append, paged attention (device code in the .hip files).
#pragma once

#include <hip/hip_runtime_api.h>

#include "common.h"
#include "kv_index.h"

namespace rax {

struct PagePlanArgs {
  const int32_t *past, *fresh;
  int32_t *ring, *cursor, *cursor_out, *table, *seq_lens, *query_start, *positions, *slots, *meta;
  int num_seqs, num_tokens, page_shift, num_pages, ld_table, max_pages;
};
hipError_t launch_page_plan(const PagePlanArgs& a, hipStream_t stream, const KTimer& tm);

// A layer's cache as the kernels address it (strides in elements)
struct CacheView {
  void *k, *v;
  long long page_stride, token_stride, head_stride;
  int num_pages, page_shift, heads, dim, dtype;
  float k_scale, v_scale;
};

struct RotaryArgs {
  const void* qkv;
  void* q_out;
  const int32_t *positions, *slots;
  const double* turns;   // [rot / 2][2]: turns a position, as a sum of two
  CacheView c;
  int ldqkv, ldq, dtype, q_heads, num_tokens, rot, interleaved;
  float amplitude;
  // set by the launcher: tokens of a workgroup; divisors of the item numbers
  int tokens_wg;
  FastDiv per_half, per_head, per_chunk, per_turned;
};
hipError_t launch_rotary_append(const RotaryArgs& a, hipStream_t stream, const KTimer& tm);

struct AttentionArgs {
  const void* q;
  void* out;
  float* lse;            // may be null
  const int32_t *table, *seq_lens, *query_start;
  CacheView c;
  int ldq, ldo, dtype, q_heads, num_seqs, num_tokens, ld_table, max_pages, window;
  float scale;
  // the launch's shape and workspace
  int waves, row_tiles, row_waves;   // of a workgroup; its rows: 16 * row_tiles * row_waves
  int read_once;                     // no line of the cache is read by two workgroups
  int workers, min_steps;            // workgroups; steps each has at least
  int step_log2;                     // keys of a step
  int group_size;                    // query heads of a kv head
  FastDiv group;
  float *part_o, *part_ml;           // two slots a workgroup: [rows][dim], [rows][2]
  int *arrived, counters;            // [kJoinLevels][counters], zero between launches
};
constexpr int kJoinLevels = 4;       // 8^4 parts of a unit: more than there are workgroups
// Shape of a workgroup by the rows (new tokens times query heads of a kv head) that the mean
// sequence has, and the number of sequences times kv heads.
constexpr int kMaxRows = 64;
struct AttnRows {
  int tiles, waves;   // row tiles of a wave; waves that share the keys, the others split them
  int rows() const { return 16 * tiles * waves; }
};
AttnRows attention_rows(long long rows, long long heads);
// keys that a workgroup's waves take at a time (log2): a tile each, the waves that do not
// share rows side by side
inline int attention_step_log2(const AttentionArgs& a) {
  int s = a.dtype == LORA_F32 ? 4 : 5;
  for (int w = a.waves / a.row_waves; w > 1; w /= 2) ++s;
  return s;
}
hipError_t launch_paged_attention(const AttentionArgs& a, hipStream_t stream, const KTimer& tm);

}  // namespace rax
