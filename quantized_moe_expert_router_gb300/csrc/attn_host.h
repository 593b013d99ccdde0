// attn_host.h -- argument checks that the entry points of the attention, of the
// rotary positions and of the latent attention share (host side).
#pragma once

#include "attn.h"

namespace moe {

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
inline bool given(const void *p) { return p && aligned16(p); }
// Arrays of words: their own alignment (a free list is advanced by a few pages).
inline bool words(const void *p) { return p && ((uintptr_t)p & 3u) == 0; }
inline bool aligned8(const void *p) { return ((uintptr_t)p & 7u) == 0; }
inline bool lse_ok(const float *p) { return ((uintptr_t)p & 3u) == 0; }

inline moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// Restores the caller's current device on scope exit.
struct DeviceGuard {
  int prev = -1;
  bool ok = false, changed = false;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) return;
    changed = prev != dev;
    ok = !changed || cudaSetDevice(dev) == cudaSuccess;
  }
  ~DeviceGuard() {
    if (ok && changed) cudaSetDevice(prev);
  }
};

// Checks a row view and fills in the strides of axes of length one.
inline bool row_view(const moe_attn_rows *r, int rows, int heads, int head_dim, RowView *v) {
  if (!r || !given(r->data)) return false;
  v->p = static_cast<uint16_t *>(r->data);
  v->head = heads > 1 ? r->head_stride : head_dim;
  v->row = rows > 1 ? r->row_stride : head_dim;
  for (const long long s : {v->row, v->head})
    if (s <= 0 || s % 8 || s > (1LL << 36)) return false;
  return true;
}

inline bool counts_ok(int num_requests, int num_rows) { return num_requests >= 0 && num_rows >= 0; }

// log2 of a page size, or -1.
inline int page_shift_of(int page_size) {
  for (int s = 4; s <= 7; s++)
    if (page_size == 1 << s) return s;
  return -1;
}

}  // namespace moe
