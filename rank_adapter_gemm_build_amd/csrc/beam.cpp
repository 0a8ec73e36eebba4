// Host side of the operators of beam search over the paged cache (include/raxlora.h): argument
// checks, object lifetimes, dispatch.  Every argument check runs before the first HIP call.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <new>

#include "beam.h"
#include "kv_host.h"

using rax::cache_view;
using rax::check_cache;
using rax::check_device;
using rax::check_pages;
using rax::DeviceGuard;
using rax::fail;
using rax::hip_fail;
using rax::log2_of;
using rax::ok;
using rax::timer_for;

struct lora_beams {
  int device = 0, max_requests = 0, beams = 0, vocab = 0, candidates = 0;
  unsigned long long* keys = nullptr;   // device
  unsigned long long* sums = nullptr;   // device
  int* arrived = nullptr;               // device, zero between calls
};

namespace rax {
// Workgroups enough for the chip's compute units several times over, and a wave has no more tiles than that leaves.
int beam_segs(long long rows, int vocab, int size) {
  const long long tiles = ((long long)vocab * size + 15 + kBeamTileBytes - 1) / kBeamTileBytes;   // of a row
  const long long per_wave = std::max(1LL, rows * tiles / kBeamMaxWaves);
  return (int)((tiles + per_wave * kBeamWaves - 1) / (per_wave * kBeamWaves));
}
}  // namespace rax

namespace {

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && na > 0 && nb > 0 && x < y + nb && y < x + na;
}

}  // namespace

extern "C" {

lora_status lora_beams_create(lora_beams** out, int device, int max_requests, int beams, int vocab, int candidates) {
  if (!out) return fail(LORA_ERR_INVALID_ARG, "out must not be NULL");
  *out = nullptr;
  if (max_requests < 1 || max_requests > LORA_MAX_SEQS)
    return fail(LORA_ERR_SHAPE, "max_requests %d outside [1, %d]", max_requests, LORA_MAX_SEQS);
  if (beams < 1 || beams > LORA_MAX_BEAMS || candidates < 1 || candidates > LORA_MAX_BEAMS)
    return fail(LORA_ERR_SHAPE, "beams %d and candidates %d must be in [1, %d]", beams, candidates, LORA_MAX_BEAMS);
  if (vocab < 1 || vocab > LORA_MAX_VOCAB) return fail(LORA_ERR_SHAPE, "vocab %d outside [1, 2^24]", vocab);
  lora_status st = check_device(device);
  if (st != LORA_OK) return st;
  DeviceGuard g(device);
  if (g.err != hipSuccess) return hip_fail(g.err, "hipSetDevice");
  lora_beams* b = new (std::nothrow) lora_beams;
  if (!b) return fail(LORA_ERR_OOM, "out of host memory");
  b->device = device;
  b->max_requests = max_requests;
  b->beams = beams;
  b->vocab = vocab;
  b->candidates = candidates;
  size_t shares = 0;   // the most that a call of up to max_requests requests has
  for (long long n = 1; n <= max_requests; ++n)
    for (int size = 2; size <= 4; size += 2)
      shares = std::max(shares, (size_t)(n * beams) * (size_t)rax::beam_segs(n * beams, vocab, size));
  hipError_t e = hipMalloc(reinterpret_cast<void**>(&b->keys), shares * candidates * sizeof(unsigned long long));
  if (e == hipSuccess) e = hipMalloc(reinterpret_cast<void**>(&b->sums), shares * rax::kBeamWaves * 2 * sizeof(unsigned long long));
  if (e == hipSuccess) e = hipMalloc(reinterpret_cast<void**>(&b->arrived), max_requests * sizeof(int));
  if (e == hipSuccess) e = hipMemset(b->arrived, 0, max_requests * sizeof(int));
  if (e == hipSuccess) e = hipDeviceSynchronize();
  if (e != hipSuccess) {
    (void)lora_beams_destroy(b);
    return hip_fail(e, "beam selection workspace");
  }
  *out = b;
  return ok();
}

lora_status lora_beams_destroy(lora_beams* beams) {
  if (!beams) return ok();
  DeviceGuard g(beams->device);
  if (beams->keys) (void)hipFree(beams->keys);
  if (beams->sums) (void)hipFree(beams->sums);
  if (beams->arrived) (void)hipFree(beams->arrived);
  delete beams;
  return ok();
}

lora_status lora_beam_select(const lora_beams* beams, const void* logits, int ldlogits, lora_dtype dtype, const float* scores,
                             const int32_t* ended, int end_token, const float* weights, int num_requests, int32_t* parents,
                             int32_t* tokens, float* scores_out, int32_t* ended_out, hipStream_t stream) {
  if (!beams) return fail(LORA_ERR_INVALID_ARG, "beams must not be NULL");
  if (dtype != LORA_BF16 && dtype != LORA_F32) return fail(LORA_ERR_DTYPE, "logits must be bfloat16 or float32");
  if (num_requests < 0) return fail(LORA_ERR_SHAPE, "num_requests = %d < 0", num_requests);
  if (num_requests > beams->max_requests)
    return fail(LORA_ERR_CAPACITY, "num_requests = %d exceeds max_requests = %d", num_requests, beams->max_requests);
  if (ldlogits < beams->vocab) return fail(LORA_ERR_SHAPE, "ldlogits = %d < vocab = %d", ldlogits, beams->vocab);
  if (end_token < -1 || end_token >= beams->vocab || (ended && end_token < 0))
    return fail(LORA_ERR_INVALID_ARG, "end_token %d outside [%d, %d)", end_token, ended ? 0 : -1, beams->vocab);
  if (num_requests > 0 && (!logits || !scores || !parents || !tokens || !scores_out))
    return fail(LORA_ERR_INVALID_ARG, "logits, scores, parents, tokens and scores_out must not be NULL");
  const int size = dtype == LORA_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % size) return fail(LORA_ERR_ALIGN, "logits must be aligned to their type");
  const size_t in = 4 * (size_t)num_requests * beams->beams, n = 4 * (size_t)num_requests * beams->candidates;
  const bool same = beams->beams == beams->candidates;   // a request's outputs then lie where its own inputs do
  const void* const outs[4] = {parents, tokens, scores_out, ended_out};
  // one request's outputs are written while others' logits are read
  const size_t rows = (size_t)num_requests * beams->beams, read = rows > 0 ? ((rows - 1) * ldlogits + beams->vocab) * size : 0;
  for (int i = 0; i < 4; ++i) {
    if (overlap(outs[i], n, logits, read)) return fail(LORA_ERR_INVALID_ARG, "an output overlaps logits");
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], n, outs[j], n)) return fail(LORA_ERR_INVALID_ARG, "two outputs overlap");
    const void* const ins[3] = {scores, ended, weights};
    for (int j = 0; j < 3; ++j)
      if (overlap(outs[i], n, ins[j], in) && !(same && outs[i] == ins[j] && ((i == 2 && j == 0) || (i == 3 && j == 1))))
        return fail(LORA_ERR_INVALID_ARG, "an output overlaps scores, ended or weights");
  }
  if (num_requests == 0) return ok();
  DeviceGuard g(beams->device);
  if (g.err != hipSuccess) return hip_fail(g.err, "hipSetDevice");
  rax::BeamArgs a{};
  a.logits = logits;
  a.scores = scores;
  a.weights = weights;
  a.ended = ended;
  a.parents = parents;
  a.tokens = tokens;
  a.ended_out = ended_out;
  a.scores_out = scores_out;
  a.ld = ldlogits;
  a.dtype = dtype;
  a.requests = num_requests;
  a.beams = beams->beams;
  a.vocab = beams->vocab;
  a.best = beams->candidates;
  a.end_token = end_token;
  a.segs = rax::beam_segs((long long)num_requests * beams->beams, beams->vocab, size);
  a.keys = beams->keys;
  a.sums = beams->sums;
  a.arrived = beams->arrived;
  const hipError_t e = rax::launch_beam_select(a, stream, timer_for(rax::kKBeam));
  if (e != hipSuccess) return hip_fail(e, "beam selection launch");
  return ok();
}

lora_status lora_page_fork(int device, const int32_t* parents, int num_rows, int32_t* lens, int page_size, int num_pages,
                           int32_t* free_pages, int32_t* cursor, int32_t* shares, int32_t* block_table, int ld_table,
                           int max_pages, int32_t* copy_src, int32_t* copy_dst, int32_t* copy_tokens, int32_t* scratch,
                           int32_t* meta, hipStream_t stream) {
  if (num_rows < 0 || num_rows > LORA_MAX_SEQS)
    return fail(LORA_ERR_SHAPE, "num_rows %d outside [0, %d]", num_rows, LORA_MAX_SEQS);
  if (!free_pages || !cursor || !shares || !scratch || !meta)
    return fail(LORA_ERR_INVALID_ARG, "free_pages, cursor, shares, scratch and meta must not be NULL");
  if (num_rows > 0 && (!parents || !lens || !block_table || !copy_src || !copy_dst || !copy_tokens))
    return fail(LORA_ERR_INVALID_ARG, "parents, lens, block_table, copy_src, copy_dst and copy_tokens must not be NULL");
  lora_status st = check_pages(page_size, num_pages);
  if (st != LORA_OK) return st;
  if (max_pages < 1 || (long long)max_pages * page_size > 0x7fffffffLL)
    return fail(LORA_ERR_SHAPE, "max_pages %d outside [1, (2^31 - 1) / page_size]", max_pages);
  if (ld_table < max_pages) return fail(LORA_ERR_SHAPE, "ld_table = %d < max_pages = %d", ld_table, max_pages);
  // the workgroups of a call read and write these at the same time
  const size_t rows = num_rows, pages = num_pages, table = rows > 0 ? (rows - 1) * ld_table + max_pages : 0;
  const struct {
    const void* at;
    size_t words;
  } vecs[] = {{parents, rows},     {lens, rows},     {copy_src, rows},     {copy_dst, rows},            {copy_tokens, rows}, {free_pages, pages},
              {cursor, 4}, {shares, pages}, {block_table, table}, {scratch, (pages + 31) / 32}, {meta, LORA_FORK_META}};
  for (const auto& x : vecs)
    for (const auto* y = vecs; y != &x; ++y)
      if (overlap(x.at, 4 * x.words, y->at, 4 * y->words)) return fail(LORA_ERR_INVALID_ARG, "two vectors overlap");
  if (num_rows == 0) return ok();
  DeviceGuard g(device);
  if (g.err != hipSuccess) return hip_fail(g.err, "hipSetDevice");
  rax::PageForkArgs a{};
  a.parents = parents;
  a.lens = lens;
  a.ring = free_pages;
  a.cursor = cursor;
  a.shares = shares;
  a.table = block_table;
  a.copy_src = copy_src;
  a.copy_dst = copy_dst;
  a.copy_tokens = copy_tokens;
  a.meta = meta;
  a.freed = reinterpret_cast<uint32_t*>(scratch);
  a.rows = num_rows;
  a.page_shift = log2_of(page_size);
  a.num_pages = num_pages;
  a.ld_table = ld_table;
  a.max_pages = max_pages;
  const hipError_t e = rax::launch_page_fork(a, stream, timer_for(rax::kKFork));
  if (e != hipSuccess) return hip_fail(e, "page fork launch");
  return ok();
}

lora_status lora_page_copy(int device, const lora_kv_cache* layers, int num_layers, const int32_t* src, const int32_t* dst,
                           const int32_t* tokens, int num_pairs, hipStream_t stream) {
  if (!layers) return fail(LORA_ERR_INVALID_ARG, "layers must not be NULL");
  if (num_layers < 1 || num_layers > LORA_MAX_LAYERS)
    return fail(LORA_ERR_SHAPE, "num_layers %d outside [1, %d]", num_layers, LORA_MAX_LAYERS);
  if (num_pairs < 0 || num_pairs > (1 << 20)) return fail(LORA_ERR_SHAPE, "num_pairs %d outside [0, 2^20]", num_pairs);
  rax::PageCopyArgs a{};
  const lora_kv_cache& f = layers[0];
  for (int i = 0; i < num_layers; ++i) {
    const lora_kv_cache& c = layers[i];
    lora_status st = check_cache(&c);
    if (st != LORA_OK) return st;
    if (c.page_stride != f.page_stride || c.token_stride != f.token_stride || c.head_stride != f.head_stride ||
        c.num_pages != f.num_pages || c.page_size != f.page_size || c.num_heads != f.num_heads || c.head_dim != f.head_dim ||
        c.dtype != f.dtype)
      return fail(LORA_ERR_SHAPE, "layer %d differs from layer 0 in its sizes, strides or type", i);
    a.cells[2 * i] = c.k;
    a.cells[2 * i + 1] = c.v;
  }
  if (num_pairs > 0 && (!src || !dst)) return fail(LORA_ERR_INVALID_ARG, "src and dst must not be NULL");
  if (num_pairs == 0) return ok();
  DeviceGuard g(device);
  if (g.err != hipSuccess) return hip_fail(g.err, "hipSetDevice");
  a.src = src;
  a.dst = dst;
  a.tokens = tokens;
  a.c = cache_view(&f);
  a.pairs = num_pairs;
  a.layers = num_layers;
  a.head_major = f.num_heads > 1 && f.head_stride > f.token_stride;
  a.per_row = rax::fast_div(f.head_dim * (f.dtype == LORA_F32 ? 4 : f.dtype == LORA_BF16 ? 2 : 1) / 16);
  a.per_inner = rax::fast_div(f.num_heads);
  const hipError_t e = rax::launch_page_copy(a, stream, timer_for(rax::kKCopy));
  if (e != hipSuccess) return hip_fail(e, "page copy launch");
  return ok();
}

}  // extern "C"
