// attn_api.cu -- the extern "C" entry points of the attention beside the FFN
// (include/moe.h).  Host side only: argument checks, workspace arithmetic and
// launches.
#include <math.h>
#include <string.h>

#include <new>

#include "attn_host.h"

using namespace moe;

namespace {

AttnArgs attn_args(const moe_attn &L, int B, int T) {
  AttnArgs a;
  memset(&a, 0, sizeof(a));
  a.B = B;
  a.T = T;
  a.q_heads = L.cfg.q_heads;
  a.kv_heads = L.cfg.kv_heads;
  a.group = L.cfg.q_heads / L.cfg.kv_heads;
  a.head_dim = L.cfg.head_dim;
  a.page_shift = L.page_shift;
  a.max_pages = L.cfg.max_pages;
  a.num_pages = L.cfg.num_pages;
  a.f16 = L.cfg.dtype == MOE_ATTN_F16;
  a.scale = L.cfg.softmax_scale;
  const bool stall = L.cfg.flags & MOE_ATTN_TEST_STALL;
  a.stall = stall ? 16 : 0;
  a.wait_ns = stall ? 20000000ull : 2000000000ull;
  return a;
}

size_t attn_ws_bytes(const moe_attn &L) { return attn_tree_ws(L.cfg.head_dim, L.num_sms).total; }

}  // namespace

extern "C" {

moe_status moe_attn_create(const moe_attn_config *cfg, int device, moe_attn_t *out) {
  if (!cfg || !out || device < 0) return MOE_ERR_INVALID_ARG;
  if ((cfg->flags & ~MOE_ATTN_TEST_STALL) || !(cfg->softmax_scale > 0.f) || !isfinite(cfg->softmax_scale)) return MOE_ERR_INVALID_ARG;
  if (cfg->dtype != MOE_ATTN_BF16 && cfg->dtype != MOE_ATTN_F16) return MOE_ERR_INVALID_ARG;
  if (cfg->kv_heads < 1 || cfg->q_heads < cfg->kv_heads || cfg->q_heads % cfg->kv_heads ||
      cfg->q_heads / cfg->kv_heads > 128 || cfg->q_heads > 1024)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (cfg->head_dim != 64 && cfg->head_dim != 128) return MOE_ERR_UNSUPPORTED_SHAPE;
  const int shift = page_shift_of(cfg->page_size);
  if (shift < 0 || cfg->num_pages < 1 || cfg->max_pages < 1) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (((long long)cfg->num_pages << shift) >= (1LL << 31) || ((long long)cfg->max_pages << shift) > (1LL << 30))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  DeviceGuard g(device);
  int sms = 0;
  if (!g.ok || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) return MOE_ERR_CUDA;
  const int f16 = cfg->dtype == MOE_ATTN_F16;
  if (attn_wide_setup(cfg->head_dim, f16) != cudaSuccess || attn_tree_setup(cfg->head_dim, f16) != cudaSuccess)
    return MOE_ERR_CUDA;
  moe_attn *a = new (std::nothrow) moe_attn;
  if (!a) return MOE_ERR_OUT_OF_MEMORY;
  a->cfg = *cfg;
  a->device = device;
  a->num_sms = sms;
  a->page_shift = shift;
  *out = a;
  return MOE_OK;
}

moe_status moe_attn_destroy(moe_attn_t attn) {
  delete attn;
  return MOE_OK;
}

moe_status moe_attn_workspace_bytes(moe_attn_t attn, int num_requests, int num_rows, size_t *bytes) {
  if (!attn || !bytes || !counts_ok(num_requests, num_rows)) return MOE_ERR_INVALID_ARG;
  if (num_requests > MOE_ATTN_MAX_REQUESTS || num_rows > MOE_ATTN_MAX_ROWS) return MOE_ERR_UNSUPPORTED_SHAPE;
  *bytes = attn_ws_bytes(*attn);
  return MOE_OK;
}

moe_status moe_attn_get_device_status(moe_attn_t attn, void *ws, cudaStream_t stream, int32_t *flags) {
  if (!attn || !given(ws) || !flags) return MOE_ERR_INVALID_ARG;
  DeviceGuard g(attn->device);
  if (!g.ok) return MOE_ERR_CUDA;
  int32_t got = 0;
  cudaError_t err = cudaMemcpyAsync(&got, static_cast<int *>(ws) + kAttnCtrlFlags, sizeof(got), cudaMemcpyDeviceToHost, stream);
  // the control words and the tickets: what a call has to find at zero
  if (err == cudaSuccess) err = cudaMemsetAsync(ws, 0, attn_tree_ws(attn->cfg.head_dim, attn->num_sms).stat, stream);
  if (err == cudaSuccess) err = cudaStreamSynchronize(stream);
  if (err != cudaSuccess) return MOE_ERR_CUDA;
  *flags = got;
  return MOE_OK;
}

moe_status moe_kv_plan(moe_attn_t attn, int num_requests, int num_rows, const int32_t *cached, const int32_t *fresh,
                       const int32_t *free_pages, int num_free, const int32_t *parents, int32_t *block_table,
                       int32_t *cu, int32_t *slots, int32_t *positions, uint64_t *tree_mask, int32_t *info,
                       cudaStream_t stream) {
  if (!attn || !counts_ok(num_requests, num_rows) || num_free < 0) return MOE_ERR_INVALID_ARG;
  if (num_requests > MOE_ATTN_MAX_REQUESTS || num_rows > MOE_ATTN_MAX_ROWS) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!words(cu) || !words(info)) return MOE_ERR_INVALID_ARG;
  if (num_requests && (!words(cached) || !words(fresh) || !words(block_table))) return MOE_ERR_INVALID_ARG;
  if (num_rows && (!words(slots) || !words(positions))) return MOE_ERR_INVALID_ARG;
  if ((num_free && !words(free_pages)) || (parents && !words(parents))) return MOE_ERR_INVALID_ARG;
  if (tree_mask && (!parents || !aligned8(tree_mask))) return MOE_ERR_INVALID_ARG;
  DeviceGuard g(attn->device);
  if (!g.ok) return MOE_ERR_CUDA;
  KvPlanArgs a;
  a.cached = cached; a.fresh = fresh; a.free_pages = free_pages; a.parents = parents;
  a.block_table = block_table; a.cu = cu; a.slots = slots; a.positions = positions; a.info = info;
  a.tree_mask = tree_mask;
  a.B = num_requests; a.T = num_rows; a.num_free = num_free;
  a.max_pages = attn->cfg.max_pages; a.num_pages = attn->cfg.num_pages; a.page_shift = attn->page_shift;
  return cuda_status(launch_kv_plan(a, stream));
}

moe_status moe_kv_append(moe_attn_t attn, int num_rows, const moe_attn_rows *k, const moe_attn_rows *v,
                         const int32_t *slots, void *k_cache, void *v_cache, cudaStream_t stream) {
  if (!attn || num_rows < 0) return MOE_ERR_INVALID_ARG;
  if (num_rows > MOE_ATTN_MAX_ROWS) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (num_rows == 0) return MOE_OK;
  KvAppendArgs a;
  a.T = num_rows; a.kv_heads = attn->cfg.kv_heads; a.head_dim = attn->cfg.head_dim;
  if (!row_view(k, num_rows, a.kv_heads, a.head_dim, &a.k) || !row_view(v, num_rows, a.kv_heads, a.head_dim, &a.v) ||
      !words(slots) || !given(k_cache) || !given(v_cache))
    return MOE_ERR_INVALID_ARG;
  a.slots = slots;
  a.k_cache = static_cast<uint16_t *>(k_cache);
  a.v_cache = static_cast<uint16_t *>(v_cache);
  a.page_shift = attn->page_shift;
  a.num_slots = attn->cfg.num_pages << attn->page_shift;
  DeviceGuard g(attn->device);
  if (!g.ok) return MOE_ERR_CUDA;
  return cuda_status(launch_kv_append(a, attn->num_sms, stream));
}

moe_status moe_attn_prompt(moe_attn_t attn, int num_requests, int num_rows, const moe_attn_rows *q,
                           const moe_attn_rows *k, const moe_attn_rows *v, const int32_t *cu,
                           const moe_attn_rows *out, float *lse, void *ws, size_t ws_bytes, cudaStream_t stream) {
  if (!attn || !counts_ok(num_requests, num_rows)) return MOE_ERR_INVALID_ARG;
  if (num_requests > MOE_ATTN_MAX_REQUESTS || num_rows > MOE_ATTN_MAX_ROWS) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (num_rows == 0 || num_requests == 0) return MOE_OK;
  AttnArgs a = attn_args(*attn, num_requests, num_rows);
  if (!row_view(q, num_rows, a.q_heads, a.head_dim, &a.q) || !row_view(k, num_rows, a.kv_heads, a.head_dim, &a.k) ||
      !row_view(v, num_rows, a.kv_heads, a.head_dim, &a.v) || !row_view(out, num_rows, a.q_heads, a.head_dim, &a.out) ||
      !words(cu) || !given(ws) || !lse_ok(lse))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < attn_ws_bytes(*attn)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  a.cu = cu;
  a.lse = lse;
  DeviceGuard g(attn->device);
  if (!g.ok) return MOE_ERR_CUDA;
  return cuda_status(launch_attn_prompt(a, nullptr, static_cast<int *>(ws), attn->num_sms, stream));
}

moe_status moe_attn_tree(moe_attn_t attn, int num_requests, int num_rows, const moe_attn_rows *q, const int32_t *cu,
                         const int32_t *cached, const int32_t *block_table, const uint64_t *tree_mask,
                         const void *k_cache, const void *v_cache, const moe_attn_rows *out, float *lse, void *ws,
                         size_t ws_bytes, cudaStream_t stream) {
  if (!attn || !counts_ok(num_requests, num_rows)) return MOE_ERR_INVALID_ARG;
  if (num_requests > MOE_ATTN_MAX_REQUESTS || num_rows > MOE_ATTN_MAX_ROWS) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (num_rows == 0 || num_requests == 0) return MOE_OK;
  AttnArgs a = attn_args(*attn, num_requests, num_rows);
  if (!row_view(q, num_rows, a.q_heads, a.head_dim, &a.q) || !row_view(out, num_rows, a.q_heads, a.head_dim, &a.out) ||
      !words(cu) || !words(cached) || !words(block_table) || !given(k_cache) || !given(v_cache) || !given(ws) ||
      (tree_mask && !aligned8(tree_mask)) || !lse_ok(lse))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < attn_ws_bytes(*attn)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  a.cu = cu;
  a.cached = cached;
  a.block_table = block_table;
  a.tree_mask = tree_mask;
  a.k_cache = static_cast<const uint16_t *>(k_cache);
  a.v_cache = static_cast<const uint16_t *>(v_cache);
  a.lse = lse;
  DeviceGuard g(attn->device);
  if (!g.ok) return MOE_ERR_CUDA;
  return cuda_status(launch_attn_tree(a, static_cast<uint8_t *>(ws), attn->num_sms, stream));
}

}  // extern "C"
