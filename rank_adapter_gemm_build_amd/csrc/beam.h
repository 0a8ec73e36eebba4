// Launchers of the operators of beam search over the paged cache: beam selection, page fork, page
// copy (device code in the .hip files).
#pragma once

#include <hip/hip_runtime_api.h>

#include "common.h"
#include "kv.h"

namespace rax {

// ------------------------------------------------------------------ beam selection
struct BeamArgs {
  const void* logits;
  const float *scores, *weights;   // weights may be null
  const int32_t* ended;            // may be null
  int32_t *parents, *tokens, *ended_out;   // ended_out may be null
  float* scores_out;
  long long ld;
  int dtype, requests, beams, vocab, best, end_token;
  // the launch's shape and workspace
  int segs;                        // workgroups of a row
  unsigned long long* keys;        // [rows][segs][best]
  unsigned long long* sums;        // [rows][segs * kBeamWaves][2]: maximum (fp32) and sum (fp64) of a wave
  int* arrived;                    // [requests], zero between launches
};
constexpr int kBeamWaves = 4, kBeamLoads = 4;                  // waves of a workgroup; 16-byte loads of a lane and tile
constexpr int kBeamTileBytes = kBeamLoads * 64 * 16;           // of a wave
constexpr int kBeamMaxWaves = 12 * 256;                         // of a launch whose waves have one tile each
// Most lists of a request, rows times workgroups of a row: with p tiles a wave, rows * tiles < (p + 1) kBeamMaxWaves, there are
// at most rows * (tiles / (p kBeamWaves) + 1).
constexpr int kBeamMaxLists = 2 * kBeamMaxWaves / kBeamWaves + LORA_MAX_BEAMS;
int beam_segs(long long rows, int vocab, int size);            // workgroups that share a row of such values
hipError_t launch_beam_select(const BeamArgs& a, hipStream_t stream, const KTimer& tm);

// ------------------------------------------------------------------ page fork
struct PageForkArgs {
  const int32_t* parents;
  int32_t *lens, *ring, *cursor, *shares, *table, *copy_src, *copy_dst, *copy_tokens, *meta;
  uint32_t* freed;                 // [(num_pages + 31) / 32], zero between launches
  int rows, page_shift, num_pages, ld_table, max_pages;
};
hipError_t launch_page_fork(const PageForkArgs& a, hipStream_t stream, const KTimer& tm);

// ------------------------------------------------------------------ page copy
struct PageCopyArgs {
  const int32_t *src, *dst, *tokens;   // tokens may be null: whole pages
  CacheView c;                         // of every layer, but for its pointers
  int pairs, layers;
  int head_major;                      // heads lie further apart than tokens
  FastDiv per_row, per_inner;          // chunks of a head's row; of the inner axis (heads, unless head_major)
  void* cells[2 * LORA_MAX_LAYERS];    // k and v of each layer
};
hipError_t launch_page_copy(const PageCopyArgs& a, hipStream_t stream, const KTimer& tm);

}  // namespace rax
