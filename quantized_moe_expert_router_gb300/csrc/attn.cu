// attn.cu -- softmax attention of packed query rows, over the packed rows of a
// prompt or over the paged cache.
//
// One warp per (row, query head).  The lanes hold the head's elements; the
// warp goes through the visible tokens with the running maximum m and sum l
// of the softmax: for a token of score s,
//   m' = max(m, s), l = l e^(m - m') + e^(s - m'), o = o e^(m - m') + e^(s - m') v,
// and the result is o / l, with the log-sum-exp m + ln l.
#include <cuda_bf16.h>
#include <math.h>

#include "attn.h"
#include "gemv_core.cuh"

namespace moe {

__device__ __forceinline__ float attn_to_f32(uint16_t v, int f16) {
  return f16 ? __half2float(__ushort_as_half(v)) : __uint_as_float((uint32_t)v << 16);
}
__device__ __forceinline__ uint16_t attn_from_f32(float v, int f16) {
  return f16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

template <int D>
__global__ void __launch_bounds__(256) attn_rows_kernel(const AttnArgs a) {
  constexpr int N = D / 32;                        // elements of a lane: lane, lane + 32, ...
  const int lane = threadIdx.x & 31;
  const long long w = (blockIdx.x * 256LL + threadIdx.x) >> 5;
  const int t = (int)(w / a.q_heads), h = (int)(w - (long long)t * a.q_heads), hk = h / a.group;
  if (t >= a.T) return;
  int lo = 0, hi = a.B;                            // largest b with cu[b] <= t (empty requests share an offset)
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(a.cu + mid) <= t) lo = mid; else hi = mid - 1;
  }
  if (lo >= a.B || __ldg(a.cu + lo) > t) return;   // a row of no request
  const int b = lo, r0 = __ldg(a.cu + b), i = t - r0, n = min(__ldg(a.cu + b + 1), a.T) - r0;
  const int c = a.cached ? max(__ldg(a.cached + b), 0) : 0;
  const uint64_t word = a.tree_mask ? a.tree_mask[t] : 0;
  long long last = a.tree_mask ? (long long)c + min(n, 64) : (long long)c + i + 1;   // tokens from here on are not visible
  if (a.block_table) last = min(last, (long long)a.max_pages << a.page_shift);

  float q[N], o[N];
#pragma unroll
  for (int e = 0; e < N; e++) {
    q[e] = attn_to_f32(a.q.p[t * a.q.row + h * a.q.head + lane + 32 * e], a.f16) * a.scale;
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < last; j++) {
    if (a.tree_mask && j >= c && !((word >> (j - c)) & 1)) continue;
    const uint16_t *kp, *vp;
    if (a.block_table) {
      const int pg = __ldg(a.block_table + (size_t)b * a.max_pages + (j >> a.page_shift));
      if ((unsigned)pg >= (unsigned)a.num_pages) continue;
      const long long at =
          ((((long long)pg * a.kv_heads + hk) << a.page_shift) + (j & ((1 << a.page_shift) - 1))) * D;
      kp = a.k_cache + at;
      vp = a.v_cache + at;
    } else {
      kp = a.k.p + (long long)(r0 + j) * a.k.row + hk * a.k.head;
      vp = a.v.p + (long long)(r0 + j) * a.v.row + hk * a.v.head;
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < N; e++) s = fmaf(q[e], attn_to_f32(kp[lane + 32 * e], a.f16), s);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(kFull, s, x);
    const float m1 = fmaxf(m, s), f = m1 == -INFINITY ? 0.f : __expf(m - m1), p = m1 == -INFINITY ? 0.f : __expf(s - m1);
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < N; e++) o[e] = fmaf(o[e], f, p * attn_to_f32(vp[lane + 32 * e], a.f16));
    m = m1;
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : NAN);
#pragma unroll
  for (int e = 0; e < N; e++) a.out.p[t * a.out.row + h * a.out.head + lane + 32 * e] = attn_from_f32(o[e] * inv, a.f16);
  if (a.lse && lane == 0) a.lse[(size_t)t * a.q_heads + h] = l == 0.f ? -INFINITY : m + logf(l);
}

cudaError_t launch_attn_rows(const AttnArgs &a, int num_sms, cudaStream_t stream) {
  const long long warps = (long long)a.T * a.q_heads;
  const unsigned grid = (unsigned)((warps + 7) / 8);
  if (a.head_dim == 64) attn_rows_kernel<64><<<grid, 256, 0, stream>>>(a);
  else attn_rows_kernel<128><<<grid, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace moe
