// rope.h -- the handle, argument block and launcher of the rotary positions (host side).
#pragma once

#include "attn.h"

constexpr int kRopeMaxPairs = 128;

struct moe_rope {
  moe_rope_config cfg;
  int device;
  double freq[kRopeMaxPairs];        // radians a position
  uint64_t turns[kRopeMaxPairs];     // the same in turns, times 2^64
};

namespace moe {

// Rows of one array: heads of `units` units of 16 elements, of which the first
// `turned` are rotated and the others copied.
struct RopeSeg {
  const uint16_t *src;
  uint16_t *dst;
  long long src_row, src_head;       // elements
  long long dst_row, dst_head;       // dst_row: of a row, or of a place within a page
  long long dst_page;
  int heads, units, turned;
  int cached;                        // rows go to their slots
  int first;                         // threads of a row before this array's
};

constexpr int kRopeSegs = 4;

struct RopeArgs {
  uint64_t turns[kRopeMaxPairs];
  RopeSeg seg[kRopeSegs];
  const int32_t *positions, *slots;
  float factor;
  int T, segs, per_row, rows_per_block, interleaved, f16, page_shift, num_slots;
};

void rope_args(const moe_rope &rope, int num_rows, const int32_t *positions, RopeArgs *a);
// Adds an array; units that neither turn nor move (in place) are left out.
void rope_add(RopeArgs *a, const RopeSeg &s);
cudaError_t launch_rope(RopeArgs *a, cudaStream_t stream);

}  // namespace moe
