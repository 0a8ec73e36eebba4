// Launchers of the shared attention (device code in the .hip files).
#pragma once

#include <hip/hip_runtime_api.h>

#include "kv.h"
#include "shared_index.h"

namespace rax {

constexpr int kWideRowsLog2 = 7, kWideKeysLog2 = 6;   // wide blocks: rows of a workgroup, keys of a tile
constexpr int kWideGroups = 1024;  // most groups of a call that has them
constexpr int kEvenGroups = 16;    // most groups whose wide units are cut in even parts
// A line of steps (the common tokens' or the sequences' own) in a launch.
struct LineShape {
  int row_tiles, row_waves;          // of a workgroup, as AttentionArgs (own_line: row_waves 0 for one wave a share)
  int rows_log2;                     // of a block
  int min_steps, step_log2;          // least steps of a workgroup (or wave); keys of a step
  float *part_o, *part_ml;           // as AttentionArgs: results of units that several share
  float *state_o, *state_ml;         // [num_tokens * q_heads][dim], [..][2]: of whole ones
};
// What the first launch tells the merge: steps and shares of both lines; where a sequence's and a group's steps begin on
// their lines, and what the group has.
struct SeqPlan {
  int from, at, group, unused;       // first key of its own line: above 0 where it shares the keys before
};
struct GroupPlan {
  int at, steps, start, n;           // steps of a unit; first token and tokens
};
struct LinePlan {
  int common_work, common_workers, own_work, own_workers;
};
struct SharedArgs {
  AttentionArgs a;                   // its members of a line are not used
  const int32_t *group_start, *common;
  int num_groups;
  LinePlan* plan;
  SeqPlan* seqs;                     // [num_seqs]
  GroupPlan* groups;                 // [num_groups]
  LineShape common_line, own_line;
};
hipError_t launch_shared_attention(const SharedArgs& s, hipStream_t stream, const KTimer& tm);
hipError_t launch_shared_merge(const SharedArgs& s, hipStream_t stream, const KTimer& tm);

}  // namespace rax
