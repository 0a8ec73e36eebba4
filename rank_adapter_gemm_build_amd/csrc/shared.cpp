// Host side of the shared attention (include/raxlora.h): argument checks, object lifetime, shape of the
// launches.  Every argument check runs before the first HIP call.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <new>

#include "kv_host.h"
#include "shared.h"

using rax::cache_view;
using rax::check_act;
using rax::check_cache;
using rax::check_device;
using rax::check_head_dim;
using rax::check_rows;
using rax::DeviceGuard;
using rax::fail;
using rax::hip_fail;
using rax::log2_of;
using rax::ok;
using rax::timer_for;

struct lora_shared {
  int device = 0, max_seqs = 0, max_tokens = 0, q_heads = 0, kv_heads = 0, dim = 0;
  int workers = 0;            // workgroups
  // device, of the common line and of the own line
  float *part_o[2] = {}, *part_ml[2] = {}, *state_o[2] = {}, *state_ml[2] = {};
  rax::LinePlan* plan = nullptr;   // device, and for the two below
  rax::SeqPlan* seqs = nullptr;
  rax::GroupPlan* groups = nullptr;
};

namespace {

// Shape of a line with blocks of 2^rows_log2 rows, waves that split the keys of a step or, with one wave a share, none.
rax::LineShape line_shape(const rax::AttentionArgs& a, int row_tiles, int row_waves, int units, int rows_log2) {
  rax::LineShape s{};
  s.row_tiles = row_tiles;
  s.row_waves = row_waves;
  s.rows_log2 = rows_log2;
  int least = a.dtype == LORA_F32 ? 4 : 5;   // keys of a tile
  if (row_waves == 4) least = rax::kWideKeysLog2;
  else if (row_waves > 0)
    for (int w = 4 / row_waves; w > 1; w /= 2) ++least;
  // at least so many keys a workgroup: fewer cost more in the join than they save
  s.min_steps = row_waves == 0 ? 1 : std::max(1, std::max(128, 4 << rows_log2) >> least);
  s.step_log2 = rax::line_step_log2(least, units, a.num_tokens, a.max_pages << a.c.page_shift, a.c.heads, a.group_size, rows_log2);
  return s;
}

}  // namespace

extern "C" {

lora_status lora_shared_create(lora_shared** out, int device, int max_seqs, int max_tokens,
                                         int num_q_heads, int num_kv_heads, int head_dim) {
  if (!out) return fail(LORA_ERR_INVALID_ARG, "out must not be NULL");
  *out = nullptr;
  if (max_seqs < 1 || max_seqs > LORA_MAX_SEQS)
    return fail(LORA_ERR_SHAPE, "max_seqs %d outside [1, %d]", max_seqs, LORA_MAX_SEQS);
  if (max_tokens < 1 || max_tokens > (1 << 24)) return fail(LORA_ERR_SHAPE, "max_tokens %d outside [1, 2^24]", max_tokens);
  if (num_kv_heads < 1 || num_kv_heads > 1024 || num_q_heads < 1 || num_q_heads > 1024 || num_q_heads % num_kv_heads)
    return fail(LORA_ERR_SHAPE, "num_q_heads %d must be a multiple of num_kv_heads %d, both in [1, 1024]", num_q_heads,
                num_kv_heads);
  if ((long long)max_tokens * (num_q_heads / num_kv_heads) > (1LL << 30))
    return fail(LORA_ERR_SHAPE, "max_tokens %d times %d query heads of a kv head is above 2^30", max_tokens,
                num_q_heads / num_kv_heads);
  lora_status st = check_head_dim(head_dim);
  if (st != LORA_OK) return st;
  if ((st = check_device(device)) != LORA_OK) return st;
  DeviceGuard g(device);
  if (g.err != hipSuccess) return hip_fail(g.err, "hipSetDevice");
  int cus = 0;
  hipError_t e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, device);
  if (e != hipSuccess) return hip_fail(e, "hipDeviceGetAttribute");
  lora_shared* a = new (std::nothrow) lora_shared;
  if (!a) return fail(LORA_ERR_OOM, "out of host memory");
  a->device = device;
  a->workers = rax::attention_workers(cus);
  a->max_seqs = max_seqs;
  a->max_tokens = max_tokens;
  a->q_heads = num_q_heads;
  a->kv_heads = num_kv_heads;
  a->dim = head_dim;
  const size_t state = (size_t)max_tokens * num_q_heads * sizeof(float);
  for (int i = 0; i < 2 && e == hipSuccess; ++i) {
    const size_t part = 2 * (size_t)a->workers * (i == 0 ? 1 << rax::kWideRowsLog2 : rax::kMaxRows) * sizeof(float);   // two slots a workgroup
    e = hipMalloc(reinterpret_cast<void**>(&a->part_o[i]), part * head_dim);
    if (e == hipSuccess) e = hipMalloc(reinterpret_cast<void**>(&a->part_ml[i]), part * 2);
    if (e == hipSuccess) e = hipMalloc(reinterpret_cast<void**>(&a->state_o[i]), state * head_dim);
    if (e == hipSuccess) e = hipMalloc(reinterpret_cast<void**>(&a->state_ml[i]), state * 2);
  }
  if (e == hipSuccess) e = hipMalloc(reinterpret_cast<void**>(&a->plan), sizeof(rax::LinePlan));
  if (e == hipSuccess) e = hipMalloc(reinterpret_cast<void**>(&a->seqs), max_seqs * sizeof(rax::SeqPlan));
  if (e == hipSuccess) e = hipMalloc(reinterpret_cast<void**>(&a->groups), max_seqs * sizeof(rax::GroupPlan));
  if (e != hipSuccess) {
    (void)lora_shared_destroy(a);
    return hip_fail(e, "shared attention workspace");
  }
  *out = a;
  return ok();
}

lora_status lora_shared_destroy(lora_shared* attention) {
  if (!attention) return ok();
  DeviceGuard g(attention->device);
  for (int i = 0; i < 2; ++i) {
    if (attention->part_o[i]) (void)hipFree(attention->part_o[i]);
    if (attention->part_ml[i]) (void)hipFree(attention->part_ml[i]);
    if (attention->state_o[i]) (void)hipFree(attention->state_o[i]);
    if (attention->state_ml[i]) (void)hipFree(attention->state_ml[i]);
  }
  if (attention->plan) (void)hipFree(attention->plan);
  if (attention->seqs) (void)hipFree(attention->seqs);
  if (attention->groups) (void)hipFree(attention->groups);
  delete attention;
  return ok();
}

lora_status lora_shared_attention(const lora_shared* attention, const void* q, int ldq, lora_dtype dtype,
                                      const lora_kv_cache* cache, const int32_t* block_table, int ld_table, int max_pages,
                                      const int32_t* seq_lens, const int32_t* query_start, int num_seqs, int num_tokens,
                                      const int32_t* group_start, const int32_t* common_lens, int num_groups, float scale,
                                      void* out, int ldo, float* lse, hipStream_t stream) {
  if (!attention) return fail(LORA_ERR_INVALID_ARG, "attention must not be NULL");
  lora_status st = check_cache(cache);
  if (st != LORA_OK) return st;
  if ((st = check_act(dtype, cache)) != LORA_OK) return st;
  if (cache->num_heads != attention->kv_heads || cache->head_dim != attention->dim)
    return fail(LORA_ERR_SHAPE, "cache has %d heads of %d, the attention object %d of %d", cache->num_heads,
                cache->head_dim, attention->kv_heads, attention->dim);
  if (num_seqs < 0 || num_tokens < 0 || num_groups < 0)
    return fail(LORA_ERR_SHAPE, "num_seqs, num_tokens and num_groups must not be negative");
  if (num_seqs > attention->max_seqs || num_groups > attention->max_seqs)
    return fail(LORA_ERR_CAPACITY, "num_seqs = %d or num_groups = %d exceeds max_seqs = %d", num_seqs, num_groups, attention->max_seqs);
  if (num_tokens > attention->max_tokens)
    return fail(LORA_ERR_CAPACITY, "num_tokens = %d exceeds max_tokens = %d", num_tokens, attention->max_tokens);
  if (max_pages < 1 || (long long)max_pages * cache->page_size > 0x7fffffffLL)
    return fail(LORA_ERR_SHAPE, "max_pages %d outside [1, (2^31 - 1) / page_size]", max_pages);
  if (ld_table < max_pages) return fail(LORA_ERR_SHAPE, "ld_table = %d < max_pages = %d", ld_table, max_pages);
  if (!std::isfinite(scale)) return fail(LORA_ERR_INVALID_ARG, "scale must be finite");
  const long long width = (long long)attention->q_heads * attention->dim;
  if ((st = check_rows("q", q, ldq, width, num_tokens)) != LORA_OK) return st;
  if ((st = check_rows("out", out, ldo, width, num_tokens)) != LORA_OK) return st;
  if (num_seqs > 0 && (!block_table || !seq_lens || !query_start))
    return fail(LORA_ERR_INVALID_ARG, "block_table, seq_lens and query_start must not be NULL");
  if (num_groups > 0 && (!group_start || !common_lens))
    return fail(LORA_ERR_INVALID_ARG, "group_start and common_lens must not be NULL");
  if (num_seqs == 0 || num_tokens == 0) return ok();
  rax::SharedArgs s{};
  rax::AttentionArgs& a = s.a;
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.table = block_table;
  a.seq_lens = seq_lens;
  a.query_start = query_start;
  a.c = cache_view(cache);
  a.ldq = ldq;
  a.ldo = ldo;
  a.dtype = dtype;
  a.q_heads = attention->q_heads;
  a.num_seqs = num_seqs;
  a.num_tokens = num_tokens;
  a.ld_table = ld_table;
  a.max_pages = max_pages;
  a.scale = scale;
  a.waves = 4;
  a.group_size = attention->q_heads / attention->kv_heads;
  a.group = rax::fast_div(a.group_size);
  a.workers = attention->workers / (attention->dim > 128 ? 2 : 1);
  s.group_start = group_start;
  s.common = common_lens;
  s.num_groups = group_start ? num_groups : 0;
  s.plan = attention->plan;
  s.seqs = attention->seqs;
  s.groups = attention->groups;
  // rows a kv head of the mean sequence and the mean group
  const long long seq_rows = ((long long)num_tokens + num_seqs - 1) / num_seqs * a.group_size;
  const long long group_rows = ((long long)num_tokens + std::max(1, num_groups) - 1) / std::max(1, num_groups) * a.group_size;
  const bool many = seq_rows > 16;
  // Above 128 dims a wave has one row tile: with two the registers spill, and a wait for them waits for the stores
  // before (16 heads of 192, 64 rows a kv head over 8000 common tokens, fp32 366 -> 182 us, bf16 88 -> 81; 20 rows over 100
  // common tokens 105 -> 26 and 39 -> 18; where the products count it costs: prompts of 500 tokens in bf16 365 -> 377).
  const bool large = attention->dim > 128;
  // Own keys are few as a rule: with up to 16 rows a wave has its own share and no join in the workgroup.
  s.own_line = !many ? line_shape(a, 1, 0, num_seqs, 4) : large ? line_shape(a, 1, 2, num_seqs, 5) : line_shape(a, 2, 2, num_seqs, 6);
  // Wide blocks for more rows than one of them holds, of 8-bit cells for more than two (heads of 128; blocks of 32 and wide, us:
  // one group over 8000 tokens, 96 rows 35 and 33, 132 rows 37 and 39, 256 rows 57 and 43; over 32000 132 rows 104 and 85, 1024
  // rows 363 and 266; 8 groups over 4000 112 rows 80 and 84, 132 rows 124 and 97, 256 rows 138 and 122; e4m3, 8 groups over 4000: 192
  // rows 102 and 112, 260 rows 138 and 152, 320 rows 153 and 161, 384 rows 176 and 172, 512 rows 218 and 203; one over 8000: 320 rows
  // 51 and 66, 512 rows 66 and 74; over 32000 141 and 126, 180 and 158 for 384 and 512).  Where few tokens are common blocks of 32
  // stay ahead (200 tokens: 256 rows 20 and 26, e4m3 512 rows 30 and 34); the lengths are on the device, so the rule goes by rows.
  // Above kWideGroups groups their tables do not fit into LDS beside the tiles.
  const bool wide = group_rows > (cache->dtype == LORA_FP8E4M3 ? 256 : 128) && dtype == LORA_BF16 &&
                    (attention->dim == 64 || attention->dim == 128) && num_groups <= rax::kWideGroups;
  // Else blocks of 32 whose waves split the keys, of 64 and two such pairs for many rows in fp32, where their products bind
  // (16 groups over 3000 tokens, heads of 128, blocks of 32 and of 64, us: bf16 36 rows 58 and 68, 64 rows 63 and 70, 128 rows 101
  // and 105; fp32 165 and 156, 176 and 158, 304 and 292).  Where sequences have many rows both lines have the same shape.
  s.common_line = wide ? line_shape(a, 1, 4, num_groups, rax::kWideRowsLog2)
                       : large ? line_shape(a, 1, 2, num_groups, 5)
                       : many || (dtype == LORA_F32 && group_rows > 32) ? line_shape(a, 2, 2, num_groups, 6) : line_shape(a, 2, 1, num_groups, 5);
  if (s.own_line.step_log2 < 0 || s.common_line.step_log2 < 0)
    return fail(LORA_ERR_SHAPE, "num_tokens %d times %d query heads is too much for one call", num_tokens, attention->q_heads);
  // own keys that one block of rows reads, in whole 128-byte lines, need no place in the caches
  const long long cell = cache->dtype == LORA_F32 ? 4 : cache->dtype == LORA_FP8E4M3 ? 1 : 2;
  const long long strides = cache->page_stride | cache->token_stride | cache->head_stride | cache->head_dim;
  a.read_once = !many && strides * cell % 128 == 0 &&
                (reinterpret_cast<uintptr_t>(cache->k) | reinterpret_cast<uintptr_t>(cache->v)) % 128 == 0;
  rax::LineShape* const lines[2] = {&s.common_line, &s.own_line};
  for (int i = 0; i < 2; ++i) {
    lines[i]->part_o = attention->part_o[i];
    lines[i]->part_ml = attention->part_ml[i];
    lines[i]->state_o = attention->state_o[i];
    lines[i]->state_ml = attention->state_ml[i];
  }
  DeviceGuard g(attention->device);
  if (g.err != hipSuccess) return hip_fail(g.err, "hipSetDevice");
  hipError_t e = rax::launch_shared_attention(s, stream, timer_for(rax::kKShared));
  if (e != hipSuccess) return hip_fail(e, "shared attention launch");
  e = rax::launch_shared_merge(s, stream, timer_for(rax::kKMerge));
  if (e != hipSuccess) return hip_fail(e, "shared attention merge launch");
  return ok();
}

}  // extern "C"
