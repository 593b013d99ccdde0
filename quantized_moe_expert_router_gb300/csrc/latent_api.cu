// latent_api.cu -- the extern "C" entry points of the rotary positions and of the latent
// attention (include/moe.h).  Host side only: argument checks, frequencies, workspace
// arithmetic and launches.
#include <math.h>
#include <string.h>

#include <new>

#include "attn_host.h"
#include "latent.h"
#include "rope.h"

using namespace moe;

namespace {

constexpr double kTwoPi = 6.283185307179586476925;

bool positive(double x) { return x > 0.0 && isfinite(x); }

// Radians a position of pair i (the formulas stand in moe.h).
void frequencies(const moe_rope_config &c, double *f) {
  const double n = c.dims, pairs = c.dims / 2;
  const double base = c.scaling == MOE_ROPE_BASE ? c.theta * pow(c.factor, n / (n - 2)) : c.theta;
  double lo = 0, hi = 1;
  if (c.scaling == MOE_ROPE_YARN) {
    auto pair_of = [&](double turns) { return pairs * log(c.original / (turns * kTwoPi)) / log(c.theta); };
    lo = fmax(floor(pair_of(c.high)), 0.0);
    hi = fmin(ceil(pair_of(c.low)), n - 1);
    hi = lo + fmax(hi - lo, 0.001);
  }
  for (int i = 0; i < c.dims / 2; i++) {
    const double w = pow(base, -2.0 * i / n);
    double share = 1;            // of the unscaled frequency
    if (c.scaling == MOE_ROPE_LINEAR) share = 0;
    if (c.scaling == MOE_ROPE_YARN) share = 1 - fmin(fmax((i - lo) / (hi - lo), 0.0), 1.0);
    if (c.scaling == MOE_ROPE_BANDS) share = fmin(fmax((c.original * w / kTwoPi - c.low) / (c.high - c.low), 0.0), 1.0);
    f[i] = share * w + (1 - share) * (w / c.factor);
  }
}

// f radians in turns, times 2^64: f's 53 bits times 64 of 2^66 / (2 pi), rounded once.  A quotient in 64 bits would be off by
// 2^-53 of itself, which a position of 2^31 makes some 90 of the 2^-32 turns that the kernel takes.
uint64_t turns_of(double f) {
  int e;
  const uint64_t bits = (uint64_t)ldexp(frexp(f, &e), 53);   // f = bits 2^(e - 53), e <= 1
  const int shift = 55 - e;
  if (shift > 120) return 0;
  const unsigned __int128 product = (unsigned __int128)bits * 0xA2F9836E4E44152Aull;
  return (uint64_t)((product + ((unsigned __int128)1 << (shift - 1))) >> shift);
}

// A row array: source, destination rows.
RopeSeg seg_rows(const RowView &src, const RowView &dst, int heads, int units, int turned) {
  RopeSeg s;
  memset(&s, 0, sizeof(s));
  s.src = src.p; s.src_row = src.row; s.src_head = src.head;
  s.dst = dst.p; s.dst_row = dst.row; s.dst_head = dst.head;
  s.heads = heads; s.units = units; s.turned = turned;
  return s;
}
// A row array whose rows go to their slots: a place is `row` elements long, a page `page` and a head `head`.
RopeSeg seg_cache(const RowView &src, uint16_t *cache, long long row, long long head, long long page, int heads, int units, int turned) {
  RopeSeg s = seg_rows(src, RowView{cache, row, head}, heads, units, turned);
  s.dst_page = page;
  s.cached = 1;
  return s;
}

LatArgs lat_args(const moe_latent &L, int B, int T) {
  LatArgs a;
  memset(&a, 0, sizeof(a));
  a.B = B;
  a.T = T;
  a.heads = L.cfg.heads;
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

}  // namespace

extern "C" {

moe_status moe_rope_create(const moe_rope_config *cfg, int device, moe_rope_t *out) {
  if (!cfg || !out || device < 0) return MOE_ERR_INVALID_ARG;
  if (cfg->dims < 16 || cfg->dims > 2 * kRopeMaxPairs || cfg->dims % 16) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (cfg->layout != MOE_ROPE_HALF && cfg->layout != MOE_ROPE_INTERLEAVED) return MOE_ERR_INVALID_ARG;
  if (cfg->dtype != MOE_ATTN_BF16 && cfg->dtype != MOE_ATTN_F16) return MOE_ERR_INVALID_ARG;
  if (cfg->scaling < MOE_ROPE_PLAIN || cfg->scaling > MOE_ROPE_BANDS || cfg->flags) return MOE_ERR_INVALID_ARG;
  if (!(cfg->theta > 1.0) || !positive(cfg->theta) || !positive(cfg->attn_factor)) return MOE_ERR_INVALID_ARG;
  if (cfg->scaling != MOE_ROPE_PLAIN && (!(cfg->factor >= 1.0) || !positive(cfg->factor))) return MOE_ERR_INVALID_ARG;
  if (cfg->scaling == MOE_ROPE_YARN || cfg->scaling == MOE_ROPE_BANDS)
    if (cfg->original < 1 || !positive(cfg->low) || !positive(cfg->high) || !(cfg->low < cfg->high)) return MOE_ERR_INVALID_ARG;
  moe_rope *r = new (std::nothrow) moe_rope;
  if (!r) return MOE_ERR_OUT_OF_MEMORY;
  memset(r, 0, sizeof(*r));
  r->cfg = *cfg;
  r->device = device;
  frequencies(*cfg, r->freq);
  // frequencies are at most one radian, so the turns stay below 2^64
  for (int i = 0; i < cfg->dims / 2; i++) r->turns[i] = turns_of(r->freq[i]);
  *out = r;
  return MOE_OK;
}

moe_status moe_rope_destroy(moe_rope_t rope) {
  delete rope;
  return MOE_OK;
}

moe_status moe_rope_frequencies(moe_rope_t rope, double *freq) {
  if (!rope || !freq) return MOE_ERR_INVALID_ARG;
  memcpy(freq, rope->freq, sizeof(double) * (rope->cfg.dims / 2));
  return MOE_OK;
}

moe_status moe_rope_apply(moe_rope_t rope, int num_rows, int head_dim, const int32_t *positions, int q_heads,
                          const moe_attn_rows *q, const moe_attn_rows *q_out, int k_heads, const moe_attn_rows *k,
                          const moe_attn_rows *k_out, cudaStream_t stream) {
  if (!rope || num_rows < 0 || q_heads < 0 || k_heads < 0) return MOE_ERR_INVALID_ARG;
  if (num_rows > MOE_ATTN_MAX_ROWS || q_heads > MOE_ROPE_MAX_HEADS || k_heads > MOE_ROPE_MAX_HEADS || head_dim < rope->cfg.dims ||
      head_dim > MOE_ROPE_MAX_HEAD_DIM || head_dim % 16)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (num_rows == 0 || q_heads + k_heads == 0) return MOE_OK;
  if (!words(positions)) return MOE_ERR_INVALID_ARG;
  RopeArgs a;
  rope_args(*rope, num_rows, positions, &a);
  RowView src, dst;
  for (int z = 0; z < 2; z++) {
    const int heads = z ? k_heads : q_heads;
    if (heads == 0) continue;
    if (!row_view(z ? k : q, num_rows, heads, head_dim, &src) || !row_view(z ? k_out : q_out, num_rows, heads, head_dim, &dst))
      return MOE_ERR_INVALID_ARG;
    rope_add(&a, seg_rows(src, dst, heads, head_dim / 16, rope->cfg.dims / 16));
  }
  DeviceGuard g(rope->device);
  if (!g.ok) return MOE_ERR_CUDA;
  return cuda_status(launch_rope(&a, stream));
}

moe_status moe_rope_append(moe_attn_t attn, moe_rope_t rope, int num_rows, const int32_t *positions, const int32_t *slots,
                           const moe_attn_rows *q, const moe_attn_rows *q_out, const moe_attn_rows *k,
                           const moe_attn_rows *v, void *k_cache, void *v_cache, cudaStream_t stream) {
  if (!attn || !rope || num_rows < 0) return MOE_ERR_INVALID_ARG;
  if (attn->device != rope->device || attn->cfg.dtype != rope->cfg.dtype) return MOE_ERR_INVALID_ARG;
  const int d = attn->cfg.head_dim, kv = attn->cfg.kv_heads;
  if (num_rows > MOE_ATTN_MAX_ROWS || rope->cfg.dims > d) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (num_rows == 0) return MOE_OK;
  RowView vq, vo, vk, vv;
  if (!row_view(q, num_rows, attn->cfg.q_heads, d, &vq) || !row_view(q_out, num_rows, attn->cfg.q_heads, d, &vo) ||
      !row_view(k, num_rows, kv, d, &vk) || !row_view(v, num_rows, kv, d, &vv) || !words(positions) || !words(slots) ||
      !given(k_cache) || !given(v_cache))
    return MOE_ERR_INVALID_ARG;
  RopeArgs a;
  rope_args(*rope, num_rows, positions, &a);
  a.slots = slots;
  a.page_shift = attn->page_shift;
  a.num_slots = attn->cfg.num_pages << attn->page_shift;
  const long long head = (long long)d << attn->page_shift;
  rope_add(&a, seg_rows(vq, vo, attn->cfg.q_heads, d / 16, rope->cfg.dims / 16));
  rope_add(&a, seg_cache(vk, static_cast<uint16_t *>(k_cache), d, head, head * kv, kv, d / 16, rope->cfg.dims / 16));
  rope_add(&a, seg_cache(vv, static_cast<uint16_t *>(v_cache), d, head, head * kv, kv, d / 16, 0));
  DeviceGuard g(attn->device);
  if (!g.ok) return MOE_ERR_CUDA;
  return cuda_status(launch_rope(&a, stream));
}

moe_status moe_latent_create(const moe_latent_config *cfg, int device, moe_latent_t *out) {
  if (!cfg || !out || device < 0) return MOE_ERR_INVALID_ARG;
  if ((cfg->flags & ~MOE_ATTN_TEST_STALL) || !(cfg->softmax_scale >= 1e-30f && cfg->softmax_scale <= 1e30f)) return MOE_ERR_INVALID_ARG;
  if (cfg->dtype != MOE_ATTN_BF16 && cfg->dtype != MOE_ATTN_F16) return MOE_ERR_INVALID_ARG;
  if (cfg->heads < 1 || cfg->heads > MOE_LATENT_MAX_HEADS) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (cfg->latent_dim != kLatDim || cfg->rope_dim != kLatRope || cfg->head_dim != kLatHead) return MOE_ERR_UNSUPPORTED_SHAPE;
  const int shift = page_shift_of(cfg->page_size);
  if (shift < 0 || cfg->num_pages < 1 || cfg->max_pages < 1) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (((long long)cfg->num_pages << shift) >= (1LL << 31) || ((long long)cfg->max_pages << shift) > (1LL << 30))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  DeviceGuard g(device);
  int sms = 0;
  if (!g.ok || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) return MOE_ERR_CUDA;
  const int f16 = cfg->dtype == MOE_ATTN_F16;
  if (lat_tree_setup(f16) != cudaSuccess || attn_wide_latent_setup(f16) != cudaSuccess) return MOE_ERR_CUDA;
  moe_latent *l = new (std::nothrow) moe_latent;
  if (!l) return MOE_ERR_OUT_OF_MEMORY;
  l->cfg = *cfg;
  l->device = device;
  l->num_sms = sms;
  l->page_shift = shift;
  *out = l;
  return MOE_OK;
}

moe_status moe_latent_destroy(moe_latent_t lat) {
  delete lat;
  return MOE_OK;
}

moe_status moe_latent_workspace_bytes(moe_latent_t lat, int num_requests, int num_rows, size_t *bytes) {
  if (!lat || !bytes || !counts_ok(num_requests, num_rows)) return MOE_ERR_INVALID_ARG;
  if (num_requests > MOE_ATTN_MAX_REQUESTS || num_rows > MOE_ATTN_MAX_ROWS) return MOE_ERR_UNSUPPORTED_SHAPE;
  *bytes = lat_ws(lat->num_sms).total;
  return MOE_OK;
}

moe_status moe_latent_get_device_status(moe_latent_t lat, void *ws, cudaStream_t stream, int32_t *flags) {
  if (!lat || !given(ws) || !flags) return MOE_ERR_INVALID_ARG;
  DeviceGuard g(lat->device);
  if (!g.ok) return MOE_ERR_CUDA;
  int32_t got = 0;
  cudaError_t err = cudaMemcpyAsync(&got, static_cast<int *>(ws) + kAttnCtrlFlags, sizeof(got), cudaMemcpyDeviceToHost, stream);
  if (err == cudaSuccess) err = cudaMemsetAsync(ws, 0, kAttnCtrlBytes, stream);   // what a call has to find at zero
  if (err == cudaSuccess) err = cudaStreamSynchronize(stream);
  if (err != cudaSuccess) return MOE_ERR_CUDA;
  *flags = got;
  return MOE_OK;
}

moe_status moe_latent_plan(moe_latent_t lat, int num_requests, int num_rows, const int32_t *cached, const int32_t *fresh,
                           const int32_t *free_pages, int num_free, const int32_t *parents, int32_t *block_table,
                           int32_t *cu, int32_t *slots, int32_t *positions, uint64_t *tree_mask, int32_t *info,
                           cudaStream_t stream) {
  if (!lat) return MOE_ERR_INVALID_ARG;
  // the plan is that of any cache of these pages
  moe_attn pages;
  memset(&pages, 0, sizeof(pages));
  pages.cfg.num_pages = lat->cfg.num_pages;
  pages.cfg.max_pages = lat->cfg.max_pages;
  pages.device = lat->device;
  pages.page_shift = lat->page_shift;
  return moe_kv_plan(&pages, num_requests, num_rows, cached, fresh, free_pages, num_free, parents, block_table, cu, slots,
                     positions, tree_mask, info, stream);
}

moe_status moe_latent_append(moe_latent_t lat, moe_rope_t rope, int num_rows, const int32_t *positions, const int32_t *slots,
                             const moe_attn_rows *c, const moe_attn_rows *k_rope, const moe_attn_rows *q,
                             const moe_attn_rows *q_out, const moe_attn_rows *k_out, void *cache, cudaStream_t stream) {
  if (!lat || !rope || num_rows < 0 || !q != !q_out) return MOE_ERR_INVALID_ARG;
  if (lat->device != rope->device || lat->cfg.dtype != rope->cfg.dtype) return MOE_ERR_INVALID_ARG;
  if (num_rows > MOE_ATTN_MAX_ROWS || rope->cfg.dims > kLatRope) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (num_rows == 0) return MOE_OK;
  RowView vc, vk, vq, vo, vr;
  if (!row_view(c, num_rows, 1, kLatDim, &vc) || !row_view(k_rope, num_rows, 1, kLatRope, &vk) || !words(positions) ||
      !words(slots) || !given(cache))
    return MOE_ERR_INVALID_ARG;
  if (q && (!row_view(q, num_rows, lat->cfg.heads, kLatRope, &vq) || !row_view(q_out, num_rows, lat->cfg.heads, kLatRope, &vo)))
    return MOE_ERR_INVALID_ARG;
  // k_rope is read for the cache by other threads than those that write k_out
  if (k_out && (!row_view(k_out, num_rows, 1, kLatRope, &vr) || vr.p == vk.p)) return MOE_ERR_INVALID_ARG;
  RopeArgs a;
  rope_args(*rope, num_rows, positions, &a);
  a.slots = slots;
  a.page_shift = lat->page_shift;
  a.num_slots = lat->cfg.num_pages << lat->page_shift;
  const long long page = (long long)kLatRow << lat->page_shift;
  uint16_t *at = static_cast<uint16_t *>(cache);
  rope_add(&a, seg_cache(vc, at, kLatRow, 0, page, 1, kLatDim / 16, 0));
  rope_add(&a, seg_cache(vk, at + kLatDim, kLatRow, 0, page, 1, kLatRope / 16, rope->cfg.dims / 16));
  if (q) rope_add(&a, seg_rows(vq, vo, lat->cfg.heads, kLatRope / 16, rope->cfg.dims / 16));
  if (k_out) rope_add(&a, seg_rows(vk, vr, 1, kLatRope / 16, rope->cfg.dims / 16));
  DeviceGuard g(lat->device);
  if (!g.ok) return MOE_ERR_CUDA;
  return cuda_status(launch_rope(&a, stream));
}

moe_status moe_latent_prompt(moe_latent_t lat, int num_requests, int num_rows, const moe_attn_rows *q, const moe_attn_rows *k,
                             const moe_attn_rows *k_rope, const moe_attn_rows *v, const int32_t *cu, const moe_attn_rows *out,
                             float *lse, void *ws, size_t ws_bytes, cudaStream_t stream) {
  if (!lat || !counts_ok(num_requests, num_rows)) return MOE_ERR_INVALID_ARG;
  if (num_requests > MOE_ATTN_MAX_REQUESTS || num_rows > MOE_ATTN_MAX_ROWS) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (num_rows == 0 || num_requests == 0) return MOE_OK;
  const LatArgs l = lat_args(*lat, num_requests, num_rows);
  AttnArgs a;
  memset(&a, 0, sizeof(a));
  RowView r;
  if (!row_view(q, num_rows, l.heads, kLatHead + kLatRope, &a.q) || !row_view(k, num_rows, l.heads, kLatHead, &a.k) ||
      !row_view(k_rope, num_rows, 1, kLatRope, &r) || !row_view(v, num_rows, l.heads, kLatHead, &a.v) ||
      !row_view(out, num_rows, l.heads, kLatHead, &a.out) || !words(cu) || !given(ws) || !lse_ok(lse))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < lat_ws(lat->num_sms).total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  a.B = num_requests;
  a.T = num_rows;
  a.q_heads = a.kv_heads = l.heads;
  a.group = 1;
  a.head_dim = kLatHead;
  a.f16 = l.f16;
  a.scale = l.scale;
  a.stall = l.stall;
  a.wait_ns = l.wait_ns;
  a.cu = cu;
  a.lse = lse;
  DeviceGuard g(lat->device);
  if (!g.ok) return MOE_ERR_CUDA;
  return cuda_status(launch_attn_prompt(a, &r, static_cast<int *>(ws), lat->num_sms, stream));
}

moe_status moe_latent_tree(moe_latent_t lat, int num_requests, int num_rows, const moe_attn_rows *q,
                           const moe_attn_rows *q_rope, const int32_t *cu, const int32_t *cached, const int32_t *block_table,
                           const uint64_t *tree_mask, const void *cache, const moe_attn_rows *out, float *lse, void *ws,
                           size_t ws_bytes, cudaStream_t stream) {
  if (!lat || !counts_ok(num_requests, num_rows)) return MOE_ERR_INVALID_ARG;
  if (num_requests > MOE_ATTN_MAX_REQUESTS || num_rows > MOE_ATTN_MAX_ROWS) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (num_rows == 0 || num_requests == 0) return MOE_OK;
  LatArgs a = lat_args(*lat, num_requests, num_rows);
  if (!row_view(q, num_rows, a.heads, kLatDim, &a.q) || !row_view(q_rope, num_rows, a.heads, kLatRope, &a.q_rope) ||
      !row_view(out, num_rows, a.heads, kLatDim, &a.out) || !words(cu) || !words(cached) || !words(block_table) || !given(cache) ||
      !given(ws) || (tree_mask && !aligned8(tree_mask)) || !lse_ok(lse))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < lat_ws(lat->num_sms).total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  a.cu = cu;
  a.cached = cached;
  a.block_table = block_table;
  a.tree_mask = tree_mask;
  a.cache = static_cast<const uint16_t *>(cache);
  a.lse = lse;
  DeviceGuard g(lat->device);
  if (!g.ok) return MOE_ERR_CUDA;
  return cuda_status(launch_lat_tree(a, static_cast<uint8_t *>(ws), lat->num_sms, stream));
}

}  // extern "C"
