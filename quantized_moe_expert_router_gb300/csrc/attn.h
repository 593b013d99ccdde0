// attn.h -- the handle, argument blocks and launchers of the attention beside
// the FFN and of its paged cache (host side).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "moe.h"

struct moe_attn {
  moe_attn_config cfg;
  int device;
  int num_sms;
  int page_shift;             // log2 of the page size
};

namespace moe {

// Rows as the kernels see them (strides in elements).
struct RowView {
  uint16_t *p;
  long long row, head;
};

struct KvPlanArgs {
  const int32_t *cached, *fresh, *free_pages, *parents;
  int32_t *block_table, *cu, *slots, *positions, *info;
  uint64_t *tree_mask;
  int B, T, num_free, max_pages, num_pages, page_shift;
};
cudaError_t launch_kv_plan(const KvPlanArgs &a, cudaStream_t stream);

struct KvAppendArgs {
  RowView k, v;
  const int32_t *slots;
  uint16_t *k_cache, *v_cache;
  int T, kv_heads, head_dim, page_shift, num_slots;
};
cudaError_t launch_kv_append(const KvAppendArgs &a, int num_sms, cudaStream_t stream);

struct AttnArgs {
  RowView q, k, v, out;       // k, v: the packed rows of a prompt; unused over a cache
  const int32_t *cu;          // [B + 1]
  const int32_t *cached;      // [B]; null for a prompt
  const int32_t *block_table; // [B][max_pages]; null for a prompt
  const uint64_t *tree_mask;  // [T] or null
  const uint16_t *k_cache, *v_cache;
  float *lse;                 // [T][q_heads] or null
  int B, T, q_heads, kv_heads, group, head_dim, page_shift, max_pages, num_pages, f16;
  float scale;
  unsigned stall;             // bytes that a copy's barrier expects and that never come (MOE_ATTN_TEST_STALL); else 0
  unsigned long long wait_ns; // limit of a device wait
};
// First 256 bytes of the workspace: zero between calls, but for the flags.
constexpr int kAttnCtrlBytes = 256;
constexpr int kAttnCtrlNext = 0, kAttnCtrlDone = 1, kAttnCtrlFlags = 2;   // ints

// Byte offsets of moe_attn_tree's workspace (after the control words): that of
// the calls with many rows per request, and all of it.
struct AttnWideWs {
  size_t desc, stat, part, total;
};
struct AttnTreeWs {             // up to `stat`: zero between calls, but for the flags
  size_t tickets, stat, part, total;
  AttnWideWs wide;
};
// Opt-in shared memory of the tcgen05 kernels (idempotent).
cudaError_t attn_wide_setup(int head_dim, int f16);
AttnWideWs attn_wide_ws(size_t off, int head_dim, int num_sms);
cudaError_t launch_attn_prompt(const AttnArgs &a, int *ctrl, int num_sms, cudaStream_t stream);
cudaError_t launch_attn_wide_tree(const AttnArgs &a, uint8_t *ws, const AttnWideWs &w, int num_sms, cudaStream_t stream);

AttnTreeWs attn_tree_ws(int head_dim, int num_sms);
cudaError_t attn_tree_setup(int head_dim, int f16);
cudaError_t launch_attn_tree(const AttnArgs &a, uint8_t *ws, int num_sms, cudaStream_t stream);

}  // namespace moe
