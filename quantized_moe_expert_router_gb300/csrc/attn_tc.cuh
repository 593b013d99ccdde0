// attn_tc.cuh -- tensor-memory, tensor-core and tensor-map pieces of the
// attention kernels (sm_103a).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include "attn.h"
#include "gemv_core.cuh"

namespace moe {

__device__ __forceinline__ void at_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void at_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Wait for this thread's tensor-memory loads into r.  The empty statements make
// the registers depend on the wait: without them the compiler may move their
// first uses, which depend on the load instructions alone, before it.
template <int N>
__device__ __forceinline__ void at_wait_ld(float (&r)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; i++) asm volatile("" : "+f"(r[i])::"memory");
}
__device__ __forceinline__ void at_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of this warp's 32 tensor-memory lanes into r[0..31]; complete
// after at_wait_ld.
__device__ __forceinline__ void at_ld32(uint32_t taddr, float *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
        "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
        "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void at_st16(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void at_st32(uint32_t taddr, const float *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "f"(r[8]), "f"(r[9]),
      "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15]), "f"(r[16]), "f"(r[17]), "f"(r[18]),
      "f"(r[19]), "f"(r[20]), "f"(r[21]), "f"(r[22]), "f"(r[23]), "f"(r[24]), "f"(r[25]), "f"(r[26]), "f"(r[27]),
      "f"(r[28]), "f"(r[29]), "f"(r[30]), "f"(r[31])
      : "memory");
}

// 32 columns of 16 of this warp's tensor-memory lanes as fragments: of columns
// 8 i + 2 (lane & 3), + 1, row lane / 4 in r[4 i], r[4 i + 1] and row lane / 4 + 8
// in r[4 i + 2], r[4 i + 3].
__device__ __forceinline__ void at_ld_frag(uint32_t taddr, float *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(taddr)
      : "memory");
}
// Word i of lane q of a quad <-> word q of lane i.
__device__ __forceinline__ void at_quad_transpose(uint32_t (&w)[4], int q) {
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const uint32_t got = __shfl_xor_sync(kFull, (q & 1) ? w[i] : w[i + 1], 1);
    if (q & 1) w[i] = got; else w[i + 1] = got;
  }
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const uint32_t got = __shfl_xor_sync(kFull, (q & 2) ? w[i] : w[i + 2], 2);
    if (q & 2) w[i] = got; else w[i + 2] = got;
  }
}

// Shared-memory descriptors of tiles of 128-byte rows under the 128-byte
// swizzle (16-byte piece c of row r at piece c ^ (r & 7); 8 rows = 1024 bytes).
//   K-major (rows are M or N, the row's elements are K): 8-row groups 1024
//     bytes apart; a k-step of 16 elements advances the start by 32 bytes.
//   MN-major (rows are K, the row's 64 elements are N): 8-row groups of K 1024
//     bytes apart (stride), the next 64 N elements `lead` bytes on; a k-step of
//     16 rows advances the start by 2048 bytes.
__device__ __forceinline__ uint64_t at_desc(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lead >> 4) & 0x3FFFu) << 16) | ((uint64_t)(1024u >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
// Instruction descriptor: fp32 accumulator, A and B both bf16 or both f16,
// M = 128; `bt`: B is MN-major.
__device__ __forceinline__ constexpr uint32_t at_idesc(bool f16, int n, bool bt) {
  return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | (bt ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
         ((128u >> 4) << 24);
}
__device__ __forceinline__ void at_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void at_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// True in one lane of the warp.
__device__ __forceinline__ bool at_elect() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ void at_commit(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void at_tma_3d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void at_tma_4d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, int c3, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void at_fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ float at_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float at_max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float2 at_add2(float2 a, float2 b) {
  uint64_t ra = *reinterpret_cast<uint64_t *>(&a), rb = *reinterpret_cast<uint64_t *>(&b), rd;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(rd) : "l"(ra), "l"(rb));
  return *reinterpret_cast<float2 *>(&rd);
}
// Two fp32 values to the element type, the first in the low half.
template <bool F16>
__device__ __forceinline__ uint32_t at_pack(float lo, float hi) {
  uint32_t r;
  if constexpr (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Bits 15 and 31 set where the low or high element is infinite or NaN: the
// exponent field is all ones exactly when adding its lowest bit carries.
template <bool F16>
__device__ __forceinline__ uint32_t at_nonfinite(uint32_t w) {
  return F16 ? ((w & 0x7C007C00u) + 0x04000400u) & 0x80008000u : ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}
template <bool F16>
__device__ __forceinline__ float at_value(uint16_t v) {
  if constexpr (F16) return __half2float(__ushort_as_half(v));
  else return __uint_as_float((uint32_t)v << 16);
}

// x / d for 0 <= x, 0 < d.  Up to 2^22 by a reciprocal, whose quotient is off by
// one at most there, put right by the remainder: a fifth of the latency of the
// integer division, which the start of a short call would pay several times in
// a row (and the 64-bit one is a longer routine still).
__device__ __forceinline__ int at_idiv(int x, int d) {
  if ((x | d) >> 22) return x / d;
  int q = (int)(__int2float_rn(x) * __frcp_rn(__int2float_rn(d)));
  const int r = x - q * d;
  q += (r >= d) - (r < 0);
  return q;
}
__device__ __forceinline__ long long at_div(long long x, long long d) {
  return (x | d) >> 31 ? x / d : (long long)at_idiv((int)x, (int)d);
}

// A bounded wait of a whole warp, which goes on or gives up together (what follows are
// instructions of whole warps).
__device__ __forceinline__ bool at_wait(uint64_t *bar, uint32_t parity, const AttnArgs &a, int *ctrl) {
  const bool ok = __all_sync(kFull, mbar_wait_bounded(bar, parity, a.wait_ns));
  if (!ok && (threadIdx.x & 31) == 0) atomicOr(ctrl + kAttnCtrlFlags, MOE_FLAG_TIMEOUT);
  return ok;
}

// The share of a CTA in the line of units (chunks or key tiles) of all items.
// work[b]: units of the requests before b; request b has items(b) items of
// nch(b) units each.  Two ways to cut the line:
//   parts   every item in equal parts of `len` units, a CTA each, when there are
//           CTAs enough for a `len` of at most 31 units above the mean: a CTA then
//           sets up, joins and stores one part only;
//   even    CTA i takes units [total i / ctas, total (i + 1) / ctas), whatever
//           items they belong to: long and short items together, many items.
// bf16, D = 128, us with parts and always even: 1 row tile x 8 heads at 1000 tokens
// 8.2, 11.7; 8 requests of up to 8 rows at up to 4000 16.9, 23.2; 3 at 300 8.6, 21.6; 1
// at 30000 26.7, 28.6; 4 of up to 64 rows at up to 9000 (attn_wide.cu) 27.5, 30.5.
struct AtShare {
  long long x0, x1;            // this CTA's units
  long long per, rem;          // even: units of a CTA, and CTAs with one more
  int ctas;
  int c0, c1;                  // parts (len > 0): the CTAs of the item's first and last part
  int len;
  __device__ __forceinline__ long long start(long long i) const { return i * per + min(i, rem); }
  __device__ __forceinline__ int cta_of(long long x) const {
    const long long big = rem * (per + 1);
    return (int)(x < big ? at_div(x, per + 1) : rem + at_div(x - big, per));
  }
  // CTAs that hold the first and the last unit of an item of this CTA
  __device__ __forceinline__ void ctas_of(long long item0, long long last, int &a, int &b) const {
    if (len) {
      a = c0;
      b = c1;
    } else {
      a = item0 >= x0 ? (int)blockIdx.x : cta_of(item0);
      b = last < x1 ? (int)blockIdx.x : cta_of(last);
    }
  }
  // where CTA a, which holds the item's first unit, keeps its part: a CTA's first part is in its slot 0
  __device__ __forceinline__ int first_slot(int a, long long item0) const { return 2 * a + (!len && start(a) < item0); }
};
// All threads of the CTA (NW warps) call this; `scratch` is NW x 32 ints.
template <int NW, typename Items, typename Nch>
__device__ __forceinline__ AtShare at_share(const long long *work, int B, long long total, int nitems, int min_len,
                                            int (*scratch)[32], Items items, Nch nch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, grid = gridDim.x, me = blockIdx.x;
  AtShare r;
  r.x0 = r.x1 = 0;
  r.c0 = r.c1 = r.len = 0;
  r.ctas = (int)min((total + min_len - 1) / min_len, (long long)grid);
  if (total == 0) return r;
  const long long mean = at_div(total + grid - 1, grid);
  if (nitems <= grid && mean < (1 << 28)) {
    // the smallest len of 32 candidates that does with the CTAs there are
    const int len0 = max(min_len, (int)mean), len = len0 + lane;
    int parts = 0;
    for (int b = warp; b < B; b += NW) parts += items(b) * at_idiv(nch(b) + len - 1, len);
    scratch[warp][lane] = parts;
    __syncthreads();
    parts = 0;
#pragma unroll
    for (int w = 0; w < NW; w++) parts += scratch[w][lane];
    const unsigned fits = __ballot_sync(kFull, parts <= grid);
    if (fits) {
      r.len = len0 + __ffs(fits) - 1;
      int before = 0;
      for (int b0 = 0; b0 < B; b0 += 32) {
        const int b = b0 + lane, n = b < B ? nch(b) : 1, per_item = at_idiv(n + r.len - 1, r.len);
        const int v = b < B ? items(b) * per_item : 0;
        int incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int t = __shfl_up_sync(kFull, incl, o);
          if (lane >= o) incl += t;
        }
        const int at = me - before - (incl - v);   // place among the request's parts
        const unsigned mine = __ballot_sync(kFull, at >= 0 && at < v);
        if (mine) {
          const int src = __ffs(mine) - 1, pi = __shfl_sync(kFull, per_item, src), place = __shfl_sync(kFull, at, src);
          const int nn = __shfl_sync(kFull, n, src), item = at_idiv(place, pi), k = place - item * pi;
          const long long item0 = work[b0 + src] + (long long)item * nn;
          r.x0 = item0 + (long long)k * r.len;
          r.x1 = min(r.x0 + r.len, item0 + nn);
          r.c0 = me - k;
          r.c1 = r.c0 + pi - 1;
          break;
        }
        before += __shfl_sync(kFull, incl, 31);
      }
      return r;
    }
  }
  r.per = at_div(total, r.ctas);
  r.rem = total - r.per * r.ctas;
  if (me < r.ctas) {
    r.x0 = r.start(me);
    r.x1 = r.start(me + 1);
  }
  return r;
}

using AttnMapEncodeFn = PFN_cuTensorMapEncodeTiled_v12000;
inline AttnMapEncodeFn attn_map_encoder() {
  static AttnMapEncodeFn fn = []() -> AttnMapEncodeFn {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<AttnMapEncodeFn>(p);
  }();
  return fn;
}

// A cache [pages][kv_heads][page][D] in boxes of 64 elements x `tokens` tokens
// under the 128-byte swizzle.
inline cudaError_t attn_encode_cache(CUtensorMap *map, const void *base, const AttnArgs &a, int tokens) {
  const AttnMapEncodeFn enc = attn_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t page = 1ull << a.page_shift, row = 2ull * a.head_dim;
  const cuuint64_t dims[4] = {(cuuint64_t)a.head_dim, page, (cuuint64_t)a.kv_heads, (cuuint64_t)a.num_pages};
  const cuuint64_t strides[3] = {row, row * page, row * page * a.kv_heads};
  const cuuint32_t box[4] = {64, (cuuint32_t)tokens, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult e = enc(map, a.f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                         const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return e == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace moe
