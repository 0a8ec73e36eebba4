// Host side of the paged-cache operators of the C ABI (include/raxlora.h): argument
// checks, object lifetimes, dispatch.  As everywhere, every argument check runs before
// the first HIP call.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "host_util.h"
#include "kv.h"

using rax::aligned16;
using rax::check_device;
using rax::DeviceGuard;
using rax::fail;
using rax::hip_fail;
using rax::ok;
using rax::timer_for;

struct lora_rotary {
  int device = 0, rot = 0, interleaved = 0;
  float amplitude = 1.f;
  double* turns = nullptr;   // device, [rot / 2][2]
};

struct lora_attention {
  int device = 0, max_seqs = 0, max_tokens = 0, q_heads = 0, kv_heads = 0, dim = 0;
  int workers = 0;                               // workgroups of 4 waves
  float *part_o = nullptr, *part_ml = nullptr;   // device
  int* arrived = nullptr;                        // device, zero between calls
};

namespace rax {
// Larger blocks read the keys fewer times, but where there are few units each is cut into
// many parts, whose join one workgroup does: the more blocks, the more of those.  Measured
// (sequences of equal numbers of rows) with blocks of 64, 32, 16 rows: 64 rows of 32 x 8 heads 116, 114, 185 us, of 64 x 8 heads
// 174, 213, 330; of 1 x 8 heads 77, 46, 31; 32 rows of 16 x 8 heads (-, 55, 62).  Four row
// waves (128 rows) were slower than two everywhere (128 rows of 128 x 4 heads 205 us, 149).
AttnRows attention_rows(long long rows, long long heads) {
  if (rows > 32 && heads * ((rows + 63) / 64) >= 256) return {2, 2};
  if (rows > 16 && heads * ((rows + 31) / 32) >= 128) return {2, 1};
  return {1, 1};
}
}  // namespace rax

namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;
constexpr double kPerTurn = 0x1.45f306dc9c883p-3, kPerTurnLow = -0x1.6b01ec5417056p-57;   // 1 / (2 pi)

bool page_size_ok(int p) { return p >= 16 && p <= 1024 && (p & (p - 1)) == 0; }
int log2_of(int p) {
  int s = 0;
  while ((1 << s) < p) ++s;
  return s;
}

lora_status check_pages(int page_size, int num_pages) {
  if (!page_size_ok(page_size)) return fail(LORA_ERR_SHAPE, "page_size %d is not a power of two in [16, 1024]", page_size);
  if (num_pages < 1 || (long long)num_pages * page_size > 0x7fffffffLL)
    return fail(LORA_ERR_SHAPE, "num_pages %d outside [1, (2^31 - 1) / page_size]", num_pages);
  return LORA_OK;
}

lora_status check_rot(int rot_dim) {
  if (rot_dim < 2 || rot_dim > LORA_MAX_HEAD_DIM || rot_dim % 2)
    return fail(LORA_ERR_SHAPE, "rot_dim %d is not an even number in [2, %d]", rot_dim, LORA_MAX_HEAD_DIM);
  return LORA_OK;
}

lora_status check_head_dim(int dim) {
  if (dim > LORA_MAX_HEAD_DIM) return fail(LORA_ERR_SHAPE, "head_dim %d above %d", dim, LORA_MAX_HEAD_DIM);
  if (dim < 16 || dim % 16) return fail(LORA_ERR_ALIGN, "head_dim %d is not a positive multiple of 16", dim);
  return LORA_OK;
}

lora_status check_cache(const lora_kv_cache* c) {
  if (!c) return fail(LORA_ERR_INVALID_ARG, "cache must not be NULL");
  if (!c->k || !c->v) return fail(LORA_ERR_INVALID_ARG, "cache->k and cache->v must not be NULL");
  if (c->dtype != LORA_BF16 && c->dtype != LORA_F32 && c->dtype != LORA_FP8E4M3)
    return fail(LORA_ERR_DTYPE, "unknown cache dtype %d", (int)c->dtype);
  if (c->dtype == LORA_FP8E4M3 &&
      !(std::isfinite(c->k_scale) && std::isfinite(c->v_scale) && c->k_scale > 0 && c->v_scale > 0))
    return fail(LORA_ERR_INVALID_ARG, "k_scale and v_scale must be positive and finite");
  lora_status st = check_pages(c->page_size, c->num_pages);
  if (st != LORA_OK) return st;
  if (c->num_heads < 1 || c->num_heads > 1024) return fail(LORA_ERR_SHAPE, "num_heads %d outside [1, 1024]", c->num_heads);
  if ((st = check_head_dim(c->head_dim)) != LORA_OK) return st;
  // strides: no two elements share an address (each stride spans everything that varies faster)
  struct Axis {
    long long stride, n;
  } ax[3] = {{c->page_stride, c->num_pages}, {c->token_stride, c->page_size}, {c->head_stride, c->num_heads}};
  std::sort(ax, ax + 3, [](const Axis& a, const Axis& b) { return a.stride < b.stride; });
  long long span = c->head_dim;
  for (const Axis& x : ax) {
    if (x.n == 1 && x.stride >= 0) continue;
    if (x.stride < span) return fail(LORA_ERR_SHAPE, "cache strides overlap (stride %lld below %lld)", x.stride, span);
    if (x.stride > (1LL << 60) / x.n) return fail(LORA_ERR_SHAPE, "cache stride %lld too large", x.stride);
    span = x.stride * (x.n - 1) + span;
  }
  if (c->token_stride >= (1LL << 25)) return fail(LORA_ERR_SHAPE, "token_stride %lld is not below 2^25", (long long)c->token_stride);
  if (c->page_stride % 16 || c->token_stride % 16 || c->head_stride % 16 || !aligned16(c->k) || !aligned16(c->v))
    return fail(LORA_ERR_ALIGN, "cache strides must be multiples of 16 elements and k, v 16-byte aligned");
  return LORA_OK;
}

lora_status check_act(lora_dtype dtype, const lora_kv_cache* c) {
  if (dtype != LORA_BF16 && dtype != LORA_F32) return fail(LORA_ERR_DTYPE, "activations must be bfloat16 or float32");
  if ((dtype == LORA_F32) != (c->dtype == LORA_F32))
    return fail(LORA_ERR_DTYPE, "float32 activations take a float32 cache, bfloat16 ones a bfloat16 or e4m3 cache");
  return LORA_OK;
}

lora_status check_rows(const char* what, const void* p, int ld, long long width, int rows) {
  if (rows > 0 && !p) return fail(LORA_ERR_INVALID_ARG, "%s is NULL", what);
  if (ld < width) return fail(LORA_ERR_SHAPE, "%s: row stride %d below its width %lld", what, ld, width);
  if (ld % 8 || !aligned16(p)) return fail(LORA_ERR_ALIGN, "%s must be 16-byte aligned with a row stride a multiple of 8", what);
  return LORA_OK;
}

rax::CacheView cache_view(const lora_kv_cache* c) {
  rax::CacheView v{};
  v.k = c->k;
  v.v = c->v;
  v.page_stride = c->page_stride;
  v.token_stride = c->token_stride;
  v.head_stride = c->head_stride;
  v.num_pages = c->num_pages;
  v.page_shift = log2_of(c->page_size);
  v.heads = c->num_heads;
  v.dim = c->head_dim;
  v.dtype = c->dtype;
  const bool f8 = c->dtype == LORA_FP8E4M3;
  v.k_scale = f8 ? c->k_scale : 1.f;
  v.v_scale = f8 ? c->v_scale : 1.f;
  return v;
}

}  // namespace

extern "C" {

lora_status lora_page_plan(int device, const int32_t* past_lens, const int32_t* new_lens, int num_seqs, int num_tokens,
                           int page_size, int num_pages, int32_t* free_pages, int32_t* cursor, int32_t* cursor_out,
                           int32_t* block_table, int ld_table, int max_pages, int32_t* seq_lens, int32_t* query_start,
                           int32_t* positions, int32_t* slots, int32_t* meta, hipStream_t stream) {
  if (!free_pages || !cursor || !cursor_out || !query_start || !meta)
    return fail(LORA_ERR_INVALID_ARG, "free_pages, cursor, cursor_out, query_start and meta must not be NULL");
  if (num_seqs < 0 || num_seqs > LORA_MAX_SEQS)
    return fail(LORA_ERR_SHAPE, "num_seqs %d outside [0, %d]", num_seqs, LORA_MAX_SEQS);
  if (num_tokens < 0 || num_tokens > rax::kPlanCap) return fail(LORA_ERR_SHAPE, "num_tokens %d outside [0, 2^30]", num_tokens);
  if (num_seqs > 0 && (!past_lens || !new_lens || !seq_lens || !block_table))
    return fail(LORA_ERR_INVALID_ARG, "past_lens, new_lens, seq_lens and block_table must not be NULL");
  if (num_tokens > 0 && (!positions || !slots)) return fail(LORA_ERR_INVALID_ARG, "positions and slots must not be NULL");
  lora_status st = check_pages(page_size, num_pages);
  if (st != LORA_OK) return st;
  if (max_pages < 1 || (long long)max_pages * page_size > 0x7fffffffLL)
    return fail(LORA_ERR_SHAPE, "max_pages %d outside [1, (2^31 - 1) / page_size]", max_pages);
  if (ld_table < max_pages) return fail(LORA_ERR_SHAPE, "ld_table = %d < max_pages = %d", ld_table, max_pages);
  DeviceGuard g(device);
  if (g.err != hipSuccess) return hip_fail(g.err, "hipSetDevice");
  rax::PagePlanArgs a{};
  a.past = past_lens;
  a.fresh = new_lens;
  a.ring = free_pages;
  a.cursor = cursor;
  a.cursor_out = cursor_out;
  a.table = block_table;
  a.seq_lens = seq_lens;
  a.query_start = query_start;
  a.positions = positions;
  a.slots = slots;
  a.meta = meta;
  a.num_seqs = num_seqs;
  a.num_tokens = num_tokens;
  a.page_shift = log2_of(page_size);
  a.num_pages = num_pages;
  a.ld_table = ld_table;
  a.max_pages = max_pages;
  const hipError_t e = rax::launch_page_plan(a, stream, timer_for(rax::kKPagePlan));
  if (e != hipSuccess) return hip_fail(e, "page plan launch");
  return ok();
}

lora_status lora_rotary_frequencies(int rot_dim, double base, int scaling, double factor, double original_len, double low,
                                    double high, double* freqs) {
  if (!freqs) return fail(LORA_ERR_INVALID_ARG, "freqs must not be NULL");
  lora_status st = check_rot(rot_dim);
  if (st != LORA_OK) return st;
  if (scaling < LORA_ROPE_PLAIN || scaling > LORA_ROPE_DIM) return fail(LORA_ERR_SHAPE, "unknown scaling %d", scaling);
  if (!std::isfinite(base) || base <= 1) return fail(LORA_ERR_INVALID_ARG, "base must be finite and above 1");
  if (scaling != LORA_ROPE_PLAIN && !(std::isfinite(factor) && factor >= 1))
    return fail(LORA_ERR_INVALID_ARG, "factor must be finite and at least 1");
  const bool blended = scaling == LORA_ROPE_WAVELENGTH || scaling == LORA_ROPE_DIM;
  if (blended && !(std::isfinite(original_len) && original_len > 0 && std::isfinite(high) && low > 0 && low < high))
    return fail(LORA_ERR_INVALID_ARG, "original_len must be positive and 0 < low < high");
  const int half = rot_dim / 2;
  double lo = 0, hi = 0;
  if (scaling == LORA_ROPE_DIM) {
    // the (fractional) pair that makes n turns over original_len
    auto pair_of = [&](double n) { return rot_dim * std::log(original_len / (kTwoPi * n)) / (2.0 * std::log(base)); };
    lo = std::min(std::max(std::floor(pair_of(high)), 0.0), rot_dim - 1.0);
    hi = std::min(std::max(std::ceil(pair_of(low)), 0.0), rot_dim - 1.0);
  }
  for (int i = 0; i < half; ++i) {
    const double f = std::pow(base, -2.0 * i / rot_dim);
    double w = 1.0;   // share of f kept unscaled
    if (scaling == LORA_ROPE_LINEAR) w = 0.0;
    if (scaling == LORA_ROPE_WAVELENGTH) w = (original_len * f / kTwoPi - low) / (high - low);
    if (scaling == LORA_ROPE_DIM) w = 1.0 - (i - lo) / std::max(hi - lo, 0.001);
    w = std::min(std::max(w, 0.0), 1.0);
    freqs[i] = scaling == LORA_ROPE_PLAIN ? f : w * f + (1.0 - w) * f / factor;
  }
  return ok();
}

lora_status lora_rotary_create(lora_rotary** out, int device, int rot_dim, int interleaved, const double* freqs,
                               double amplitude) {
  if (!out || !freqs) return fail(LORA_ERR_INVALID_ARG, "out and freqs must not be NULL");
  *out = nullptr;
  lora_status st = check_rot(rot_dim);
  if (st != LORA_OK) return st;
  if (!std::isfinite((float)amplitude)) return fail(LORA_ERR_INVALID_ARG, "amplitude must be finite");
  double turns[LORA_MAX_HEAD_DIM];
  for (int i = 0; i < rot_dim / 2; ++i) {
    if (!std::isfinite(freqs[i])) return fail(LORA_ERR_INVALID_ARG, "freqs[%d] is not finite", i);
    turns[2 * i] = freqs[i] * kPerTurn;
    turns[2 * i + 1] = std::fma(freqs[i], kPerTurn, -turns[2 * i]) + freqs[i] * kPerTurnLow;
  }
  if ((st = check_device(device)) != LORA_OK) return st;
  DeviceGuard g(device);
  if (g.err != hipSuccess) return hip_fail(g.err, "hipSetDevice");
  lora_rotary* r = new (std::nothrow) lora_rotary;
  if (!r) return fail(LORA_ERR_OOM, "out of host memory");
  r->device = device;
  r->rot = rot_dim;
  r->interleaved = interleaved != 0;
  r->amplitude = (float)amplitude;
  const size_t bytes = sizeof(double) * rot_dim;
  hipError_t e = hipMalloc(reinterpret_cast<void**>(&r->turns), bytes);
  if (e == hipSuccess) e = hipMemcpy(r->turns, turns, bytes, hipMemcpyHostToDevice);
  if (e != hipSuccess) {
    if (r->turns) (void)hipFree(r->turns);
    delete r;
    return hip_fail(e, "rotary frequencies");
  }
  *out = r;
  return ok();
}

lora_status lora_rotary_destroy(lora_rotary* rotary) {
  if (!rotary) return ok();
  DeviceGuard g(rotary->device);
  (void)hipFree(rotary->turns);
  delete rotary;
  return ok();
}

lora_status lora_rotary_append(const lora_rotary* rotary, const void* qkv, int ldqkv, lora_dtype dtype, int num_q_heads,
                               const int32_t* positions, const int32_t* slots, int num_tokens, void* q_out, int ldq,
                               const lora_kv_cache* cache, hipStream_t stream) {
  if (!rotary) return fail(LORA_ERR_INVALID_ARG, "rotary must not be NULL");
  lora_status st = check_cache(cache);
  if (st != LORA_OK) return st;
  if ((st = check_act(dtype, cache)) != LORA_OK) return st;
  if (num_tokens < 0) return fail(LORA_ERR_SHAPE, "num_tokens = %d < 0", num_tokens);
  if (num_q_heads < 1 || num_q_heads > 1024 || num_q_heads % cache->num_heads)
    return fail(LORA_ERR_SHAPE, "num_q_heads %d is not a multiple of the cache's %d heads up to 1024", num_q_heads,
                cache->num_heads);
  if (rotary->rot > cache->head_dim)
    return fail(LORA_ERR_SHAPE, "rot_dim %d above head_dim %d", rotary->rot, cache->head_dim);
  const long long D = cache->head_dim;
  if ((st = check_rows("qkv", qkv, ldqkv, (num_q_heads + 2LL * cache->num_heads) * D, num_tokens)) != LORA_OK) return st;
  if ((st = check_rows("q_out", q_out, ldq, num_q_heads * D, num_tokens)) != LORA_OK) return st;
  if (num_tokens > 0 && (!positions || !slots)) return fail(LORA_ERR_INVALID_ARG, "positions and slots must not be NULL");
  if (num_tokens == 0) return ok();
  DeviceGuard g(rotary->device);
  if (g.err != hipSuccess) return hip_fail(g.err, "hipSetDevice");
  rax::RotaryArgs a{};
  a.qkv = qkv;
  a.q_out = q_out;
  a.positions = positions;
  a.slots = slots;
  a.turns = rotary->turns;
  a.c = cache_view(cache);
  a.ldqkv = ldqkv;
  a.ldq = ldq;
  a.dtype = dtype;
  a.q_heads = num_q_heads;
  a.num_tokens = num_tokens;
  a.rot = rotary->rot;
  a.interleaved = rotary->interleaved;
  a.amplitude = rotary->amplitude;
  const hipError_t e = rax::launch_rotary_append(a, stream, timer_for(rax::kKRotary));
  if (e != hipSuccess) return hip_fail(e, "rotary append launch");
  return ok();
}

lora_status lora_attention_create(lora_attention** out, int device, int max_seqs, int max_tokens, int num_q_heads,
                                  int num_kv_heads, int head_dim) {
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
  lora_attention* a = new (std::nothrow) lora_attention;
  if (!a) return fail(LORA_ERR_OOM, "out of host memory");
  a->device = device;
  a->workers = rax::attention_workers(cus);
  a->max_seqs = max_seqs;
  a->max_tokens = max_tokens;
  a->q_heads = num_q_heads;
  a->kv_heads = num_kv_heads;
  a->dim = head_dim;
  // two slots a workgroup of at most 64 rows, or of 16 rows and one wave, 4 times as many
  const size_t part = 2 * (size_t)a->workers * rax::kMaxRows * sizeof(float);
  const size_t counters = sizeof(int) * rax::kJoinLevels * 4 * a->workers;
  e = hipMalloc(reinterpret_cast<void**>(&a->part_o), part * head_dim);
  if (e == hipSuccess) e = hipMalloc(reinterpret_cast<void**>(&a->part_ml), part * 2);
  if (e == hipSuccess) e = hipMalloc(reinterpret_cast<void**>(&a->arrived), counters);
  if (e == hipSuccess) e = hipMemset(a->arrived, 0, counters);
  if (e == hipSuccess) e = hipDeviceSynchronize();
  if (e != hipSuccess) {
    (void)lora_attention_destroy(a);
    return hip_fail(e, "attention workspace");
  }
  *out = a;
  return ok();
}

lora_status lora_attention_destroy(lora_attention* attention) {
  if (!attention) return ok();
  DeviceGuard g(attention->device);
  if (attention->part_o) (void)hipFree(attention->part_o);
  if (attention->part_ml) (void)hipFree(attention->part_ml);
  if (attention->arrived) (void)hipFree(attention->arrived);
  delete attention;
  return ok();
}

lora_status lora_paged_attention(const lora_attention* attention, const void* q, int ldq, lora_dtype dtype,
                                 const lora_kv_cache* cache, const int32_t* block_table, int ld_table, int max_pages,
                                 const int32_t* seq_lens, const int32_t* query_start, int num_seqs, int num_tokens,
                                 float scale, int window, void* out, int ldo, float* lse, hipStream_t stream) {
  if (!attention) return fail(LORA_ERR_INVALID_ARG, "attention must not be NULL");
  lora_status st = check_cache(cache);
  if (st != LORA_OK) return st;
  if ((st = check_act(dtype, cache)) != LORA_OK) return st;
  if (cache->num_heads != attention->kv_heads || cache->head_dim != attention->dim)
    return fail(LORA_ERR_SHAPE, "cache has %d heads of %d, the attention object %d of %d", cache->num_heads,
                cache->head_dim, attention->kv_heads, attention->dim);
  if (num_seqs < 0 || num_tokens < 0) return fail(LORA_ERR_SHAPE, "num_seqs and num_tokens must not be negative");
  if (num_seqs > attention->max_seqs)
    return fail(LORA_ERR_CAPACITY, "num_seqs = %d exceeds max_seqs = %d", num_seqs, attention->max_seqs);
  if (num_tokens > attention->max_tokens)
    return fail(LORA_ERR_CAPACITY, "num_tokens = %d exceeds max_tokens = %d", num_tokens, attention->max_tokens);
  if (max_pages < 1 || (long long)max_pages * cache->page_size > 0x7fffffffLL)
    return fail(LORA_ERR_SHAPE, "max_pages %d outside [1, (2^31 - 1) / page_size]", max_pages);
  if (ld_table < max_pages) return fail(LORA_ERR_SHAPE, "ld_table = %d < max_pages = %d", ld_table, max_pages);
  if (!std::isfinite(scale)) return fail(LORA_ERR_INVALID_ARG, "scale must be finite");
  if (window < 0) return fail(LORA_ERR_INVALID_ARG, "window = %d < 0", window);
  const long long width = (long long)attention->q_heads * attention->dim;
  if ((st = check_rows("q", q, ldq, width, num_tokens)) != LORA_OK) return st;
  if ((st = check_rows("out", out, ldo, width, num_tokens)) != LORA_OK) return st;
  if (num_seqs > 0 && (!block_table || !seq_lens || !query_start))
    return fail(LORA_ERR_INVALID_ARG, "block_table, seq_lens and query_start must not be NULL");
  if (num_seqs == 0 || num_tokens == 0) return ok();
  DeviceGuard g(attention->device);
  if (g.err != hipSuccess) return hip_fail(g.err, "hipSetDevice");
  rax::AttentionArgs a{};
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
  a.window = window;
  a.scale = scale;
  a.group_size = attention->q_heads / attention->kv_heads;
  a.group = rax::fast_div(a.group_size);
  const long long mean_rows = ((long long)num_tokens + num_seqs - 1) / num_seqs * a.group_size;
  const rax::AttnRows rows = rax::attention_rows(mean_rows, (long long)num_seqs * attention->kv_heads);
  a.row_tiles = rows.tiles;
  a.row_waves = rows.waves;
  // One wave a workgroup where there is a unit for half of the waves and the table's width
  // bounds their keys: 256 sequences of 16 to 128 tokens took 26.2 us against 33.7, of 100 to
  // 500 70.4 against 77.8; of 400 to 990 153.9 against 142.7 with 4 waves.
  a.waves = rows.rows() == 16 && (long long)num_seqs * attention->kv_heads >= 2 * attention->workers &&
            (long long)max_pages * cache->page_size <= 640 ? 1 : 4;
  // two workgroups a compute unit fit in registers, above 128 dims one
  a.workers = attention->workers * (4 / a.waves) / (attention->dim > 128 ? 2 : 1);
  // Keys that one block of rows reads, in whole 128-byte lines, need no place in the caches:
  // 256 sequences of 2000 to 4000 tokens 541 -> 489 us, one of 131071 99.6 -> 88.5; where lines
  // or keys are shared it costs (heads of 80 93 -> 100 us, 64 rows of 32 x 8 heads 119 -> 152).
  const long long cell = cache->dtype == LORA_F32 ? 4 : cache->dtype == LORA_FP8E4M3 ? 1 : 2;
  const long long strides = cache->page_stride | cache->token_stride | cache->head_stride | cache->head_dim;
  a.read_once = rows.waves == 1 && mean_rows <= rows.rows() && strides * cell % 128 == 0 &&
                (reinterpret_cast<uintptr_t>(cache->k) | reinterpret_cast<uintptr_t>(cache->v)) % 128 == 0;
  a.step_log2 = rax::attention_step_log2(a);
  // at least so many keys a workgroup: fewer cost more in the join than they save
  a.min_steps = a.waves == 1 ? 1 : std::max(1, std::max(128, 4 * rows.rows()) >> a.step_log2);
  a.step_log2 = rax::line_step_log2(a.step_log2, num_seqs, num_tokens, max_pages * cache->page_size, attention->kv_heads,
                                    a.group_size, log2_of(rows.rows()));
  if (a.step_log2 < 0)
    return fail(LORA_ERR_SHAPE, "num_tokens %d times %d query heads is too much for one call", num_tokens, attention->q_heads);
  a.part_o = attention->part_o;
  a.part_ml = attention->part_ml;
  a.arrived = attention->arrived;
  a.counters = 4 * attention->workers;
  const hipError_t e = rax::launch_paged_attention(a, stream, timer_for(rax::kKAttention));
  if (e != hipSuccess) return hip_fail(e, "paged attention launch");
  return ok();
}

}  // extern "C"
