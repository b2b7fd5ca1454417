// attention_shared.h — arguments, schedule and launcher of attention for a batch over a
// shared quantised prefix and private quantised tails (attention_shared.cu), called by
// the C ABI (api.cpp).
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "rrq_params.h"

namespace rrq {

// The cache is walked in tiles of `tile` tokens.  A unit is a run of tiles that one set
// of query rows attends to: the prefix of kv head g with up to 128 rows (row tile rt),
// or the tail of sequence b at kv head g with its `group` rows.  All units' tiles stand
// in one line (prefix units first, then the tails by sequence and head), cut into
// `grid` ranges of equal cost (a cost per tile, and one per tail for its start and end):
// range c belongs to CTA c, and a unit that crosses ranges leaves one partial state per
// range, merged at the end.
struct SharedArgs {
  const void* q;  // [batch × hq × d] fp16 or bf16
  void* out;      // the same
  int bf16;
  const uint8_t* k_codes[2];  // prefix, tails
  const uint8_t* v_codes[2];
  const float* k_norms[2];
  const float* v_norms[2];
  const int32_t* lens;
  int64_t batch, prefix, cap;
  int hq, hkv, group, d;
  int64_t rows;          // query rows of a kv head: batch × group, row b·group + j
  int row_tiles;         // ⌈rows / 128⌉
  int tile;              // tokens per tile
  int ptiles;            // tiles of the prefix
  int grid;              // ranges
  int pcost, tcost;      // cost of a tile of the prefix, of a tail
  int scost;             // of a tail besides its tiles
  int min_cost;          // of a range
  int units_p;           // prefix units: hkv · row_tiles, or 0 without a prefix
  int parts_p, parts_t;  // most ranges that share a prefix unit, a tail unit
  int k_bits, v_bits;
  uint64_t k_seed, v_seed;
  float kscale;          // scale · log2 e / d (over k_alpha)
  float k_levels[kMaxLevels], v_levels[kMaxLevels];
  // The tensor-core kernel's fp16 levels are rn(alpha · c): a power of two that brings the
  // largest level into [1, 2), times, for the default codebooks, the factor in [1, 2)
  // for which the rounded levels are nearest to the exact ones.
  float k_alpha, v_alpha;
  // workspace
  int* begin;     // [grid] a range's first segment, −1 for a range without tiles
  int* counts;    // [units] parts of every unit: prefix units (g · row_tiles + rt), then tails (b · hkv + g)
  int4* segs;     // two words per segment, those of a range one after the other (SharedSegment)
  float* qrot;    // rotated queries, row (g·rows + r), d values (d = 512), or in their place
  __half* qh;     //   the same as fp16 times a power of two per row,
  __half* ql;     //   what that rounding left,
  float* qexp;    //   and the power of two taken out
  float2* stats;  // (m, l) of part p, kv head g, row r at (p·hkv + g)·rows + r; prefix parts, then tail parts
  float* acc;     // the same rows × d
};

// Fills the schedule's fields from batch, hq, hkv, d, prefix and cap for the current
// device; false for a shape that is not supported (or an invalid one).
bool attention_shared_plan(SharedArgs* a);
// Sets alpha (and divides kscale by it) from the levels; `default_k`, `default_v`: the
// default codebook.
void attention_shared_levels(SharedArgs* a, bool default_k, bool default_v);
// Bytes of the workspace of a planned call; with `base` also sets its pointers.
size_t attention_shared_layout(SharedArgs* a, void* base);
cudaError_t launch_attention_shared(const SharedArgs& a, cudaStream_t stream);
// The partial states on the tensor cores (d ≤ 256), between the two launches of
// launch_attention_shared.  cudaErrorNotSupported where the layout cannot be had.
cudaError_t launch_shared_tc(const SharedArgs& a, cudaStream_t stream);

}  // namespace rrq
