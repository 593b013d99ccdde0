// latent.h -- the handle, argument block and launchers of the latent attention (host side).
#pragma once

#include "attn.h"

constexpr int kLatDim = 512, kLatRope = 64, kLatRow = kLatDim + kLatRope;   // elements of a cached token
constexpr int kLatHead = 128;                                               // of a head's own key part and of its value

struct moe_latent {
  moe_latent_config cfg;
  int device;
  int num_sms;
  int page_shift;
};

namespace moe {

struct LatArgs {
  RowView q, q_rope, out;     // [T][heads][512], [T][heads][64], [T][heads][512]
  const int32_t *cu;          // [B + 1]
  const int32_t *cached;      // [B]
  const int32_t *block_table; // [B][max_pages]
  const uint64_t *tree_mask;  // [T] or null
  const uint16_t *cache;      // [num_pages][page][576]
  float *lse;                 // [T][heads] or null
  int B, T, heads, page_shift, max_pages, num_pages, f16;
  float scale;
  unsigned stall;             // bytes that a copy's barrier expects and that never come (MOE_ATTN_TEST_STALL); else 0
  unsigned long long wait_ns; // limit of a device wait
};

// Byte offsets of the workspace, after the control words.
struct LatWs {
  size_t desc, stat, part, total;
};
LatWs lat_ws(int num_sms);
cudaError_t lat_tree_setup(int f16);     // opt-in shared memory (idempotent)
cudaError_t launch_lat_tree(const LatArgs &a, uint8_t *ws, int num_sms, cudaStream_t stream);

}  // namespace moe
