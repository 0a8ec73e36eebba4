// Launchers of the shared attention (device code in the .hip files).
#pragma once

#include <hip/hip_runtime_api.h>

#include "kv.h"
#include "shared_index.h"

namespace rax {

// A line of steps (the common tokens' or the sequences' own) in a launch.
struct LineShape {
  int row_tiles, row_waves;          // of a workgroup, as AttentionArgs
  int min_steps, step_log2;
  float *part_o, *part_ml;           // as AttentionArgs
  int* arrived;
  float *state_o, *state_ml;         // [num_tokens * q_heads][dim], [..][2]: what the merge takes
};
struct SharedArgs {
  AttentionArgs a;                   // its members of a line are not used
  const int32_t *group_start, *common;
  int num_groups;
  int32_t* from;                     // [num_seqs]: first key of each sequence's own line, 0 where nothing is shared
  LineShape common_line, own_line;
};
hipError_t launch_shared_attention(const SharedArgs& s, hipStream_t stream, const KTimer& tm);
hipError_t launch_shared_merge(const SharedArgs& s, hipStream_t stream, const KTimer& tm);

}  // namespace rax
