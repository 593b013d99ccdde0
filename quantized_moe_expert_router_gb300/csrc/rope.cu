// rope.cu -- rotary positions: rows of heads turned by their positions, in place, to
// another array, or straight into a paged cache (moe_rope_apply, moe_rope_append,
// moe_latent_append).
//
// Pair i of a head, (x, y), becomes s (x cos a - y sin a, x sin a + y cos a) with a = p f_i.
// A product in fp32 would lose the angle of far positions (p = 10^6: an error of 0.06),
// so f_i comes as turns a position in 64-bit fixed point and p f_i is an integer product
// whose whole turns fall off: what is left is exact to p 2^-64 turns, and its upper 32 bits, taken
// as signed, are the angle within [-pi, pi], off by 2^-29 at most.  As an fp32 number of radians it is off by
// 2^-21 (two roundings and that of 2 pi), and there the SFU's sine and cosine are off by at most 2^-21.1
// absolutely: 2^-20 in all, against the 2^-8 or 2^-11 of the result's own rounding; the products are fp32.
#include <string.h>

#include "gemv_core.cuh"
#include "rope.h"

namespace moe {

constexpr int kRopeThreads = 128;

__device__ __forceinline__ float2 rope_unpack(uint32_t w, int f16) {
  if (f16) return __half22float2(*reinterpret_cast<const __half2 *>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t rope_pack(float lo, float hi, int f16) {
  uint32_t r;
  if (f16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A thread has one unit of 16 elements, 8 of the first half of the turned part (or of the copied one) and the 8
// in their place in the second half, which hold 8 pairs in either layout; of HP heads, so
// that the 8 sines and cosines serve HP heads and 2 HP loads of 16 bytes wait together.
// Threads of a row: array by array, units of a head side by side, then heads, a thread's own ones as far apart as the
// threads reach: neighbouring threads touch neighbouring 16 bytes in every instruction.
//
// Bound: HBM.  16384 rows, q of 16 heads and k, v of 8 of 128: 40.6 us, 6.4 TB/s (a plain copy has 6.6 to 6.7); 16384
// latent rows with q of 64 heads, 128 bytes of every 384: 49.4 us, 6.0 TB/s; 8192 rows, q of 24 heads and k of 4, half of
// 128 elements turned: 18.1 us, 6.5 TB/s; one row 2.0 us, a launch.  Eight CTAs of 128 threads an SM (64 registers) keep
// most loads in flight: with 6 and 10 CTAs the latent rows took 54.3 and 64.9 us, with 256 threads 57.3.
template <bool F16, bool INTERLEAVED, int HP>
__global__ void __launch_bounds__(kRopeThreads, 8) rope_kernel(const __grid_constant__ RopeArgs a) {
  pdl_wait();                                      // the kernel before is done: what follows reads its results
  const int i = blockIdx.y * kRopeThreads + threadIdx.x;
  const int r = i / a.per_row, t = blockIdx.x * a.rows_per_block + r;
  if (r >= a.rows_per_block || t >= a.T) return;
  int k = i - r * a.per_row, z = 0;
#pragma unroll
  for (int e = 1; e < kRopeSegs; e++) z += e < a.segs && k >= a.seg[e].first;
  const RopeSeg &s = a.seg[z];
  k -= s.first;
  const int h0 = k / s.units, u = k - h0 * s.units, apart = (s.heads + HP - 1) / HP;   // first head, and from one to the next
  const bool turned = u < s.turned;
  const int pos = __ldg(a.positions + t);
  const int slot = s.cached ? __ldg(a.slots + t) : 0;
  // elements of the unit's two vectors
  const int e0 = turned ? 8 * u : 8 * (s.turned + u), e1 = e0 + 8 * (turned ? s.turned : s.units - s.turned);
  const uint16_t *src = s.src + t * s.src_row + h0 * s.src_head;
  uint4 x[HP], y[HP];
#pragma unroll
  for (int h = 0; h < HP; h++) {
    x[h] = y[h] = make_uint4(0u, 0u, 0u, 0u);
    if (h0 + h * apart >= s.heads) continue;
    x[h] = *reinterpret_cast<const uint4 *>(src + h * apart * s.src_head + e0);
    y[h] = *reinterpret_cast<const uint4 *>(src + h * apart * s.src_head + e1);
  }
  if (pos < 0 || (s.cached && (unsigned)slot >= (unsigned)a.num_slots)) return;
  uint16_t *dst = s.dst + h0 * s.dst_head;
  if (s.cached) dst += (slot >> a.page_shift) * s.dst_page + (slot & ((1 << a.page_shift) - 1)) * s.dst_row;
  else dst += t * s.dst_row;
  if (turned) {
    float cs[8], sn[8];
#pragma unroll
    for (int e = 0; e < 8; e++) {
      const int pair = !INTERLEAVED ? 8 * u + e : 4 * u + (e & 3) + (e & 4 ? 4 * s.turned : 0);
      const int part = (int)(((uint64_t)(uint32_t)pos * a.turns[pair]) >> 32);        // turns times 2^32, signed
      const float angle = (float)part * (6.283185307179586f / 4294967296.f);
      sn[e] = __sinf(angle) * a.factor;
      cs[e] = __cosf(angle) * a.factor;
    }
#pragma unroll
    for (int h = 0; h < HP; h++) {
      uint32_t v[8] = {x[h].x, x[h].y, x[h].z, x[h].w, y[h].x, y[h].y, y[h].z, y[h].w};
      if (INTERLEAVED) {
#pragma unroll
        for (int e = 0; e < 8; e++) {                // a word is a pair
          const float2 p = rope_unpack(v[e], F16);
          v[e] = rope_pack(p.x * cs[e] - p.y * sn[e], p.x * sn[e] + p.y * cs[e], F16);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; e++) {                // words e and e + 4 hold two pairs
          const float2 p = rope_unpack(v[e], F16), q = rope_unpack(v[e + 4], F16);
          v[e] = rope_pack(p.x * cs[2 * e] - q.x * sn[2 * e], p.y * cs[2 * e + 1] - q.y * sn[2 * e + 1], F16);
          v[e + 4] = rope_pack(p.x * sn[2 * e] + q.x * cs[2 * e], p.y * sn[2 * e + 1] + q.y * cs[2 * e + 1], F16);
        }
      }
      x[h] = make_uint4(v[0], v[1], v[2], v[3]);
      y[h] = make_uint4(v[4], v[5], v[6], v[7]);
    }
  }
#pragma unroll
  for (int h = 0; h < HP; h++) {
    if (h0 + h * apart >= s.heads) continue;
    *reinterpret_cast<uint4 *>(dst + h * apart * s.dst_head + e0) = x[h];
    *reinterpret_cast<uint4 *>(dst + h * apart * s.dst_head + e1) = y[h];
  }
}

void rope_args(const moe_rope &rope, int num_rows, const int32_t *positions, RopeArgs *a) {
  memset(a, 0, sizeof(*a));
  memcpy(a->turns, rope.turns, sizeof(a->turns));
  a->T = num_rows;
  a->positions = positions;
  a->factor = rope.cfg.attn_factor;
  a->interleaved = rope.cfg.layout == MOE_ROPE_INTERLEAVED;
  a->f16 = rope.cfg.dtype == MOE_ATTN_F16;
}

void rope_add(RopeArgs *a, const RopeSeg &s) {
  RopeSeg &d = a->seg[a->segs];
  d = s;
  if (!s.cached && s.src == s.dst && s.src_row == s.dst_row && s.src_head == s.dst_head) d.units = s.turned;
  if (d.units > 0 && d.heads > 0) a->segs++;
}

namespace {
typedef void (*RopeKernel)(const RopeArgs);
template <int HP>
RopeKernel rope_pick(const RopeArgs &a) {
  if (a.f16) return a.interleaved ? rope_kernel<true, true, HP> : rope_kernel<true, false, HP>;
  return a.interleaved ? rope_kernel<false, true, HP> : rope_kernel<false, false, HP>;
}
}  // namespace

cudaError_t launch_rope(RopeArgs *a, cudaStream_t stream) {
  if (!a->segs || !a->T) return cudaSuccess;
  long long units = 0;
  for (int z = 0; z < a->segs; z++) units += (long long)a->seg[z].heads * a->seg[z].units;
  // A thread a head until the GPU has some 400 of them an SM, then one for 4 heads, which need a fourth of the sines.  us with one
  // and with 4 heads, 40 heads of 128 and 8 of v: 64 rows 2.6, 2.9; 256 rows 4.1, 3.2; 1024 rows 8.5, 5.2.
  const int hp = units * a->T <= (1 << 16) ? 1 : 4;
  int per_row = 0;
  for (int z = 0; z < a->segs; z++) {
    a->seg[z].first = per_row;
    per_row += (a->seg[z].heads + hp - 1) / hp * a->seg[z].units;
  }
  a->per_row = per_row;
  a->rows_per_block = per_row >= kRopeThreads ? 1 : kRopeThreads / per_row;
  const dim3 grid((unsigned)((a->T + a->rows_per_block - 1) / a->rows_per_block),
                  (unsigned)((a->rows_per_block * per_row + kRopeThreads - 1) / kRopeThreads));
  cudaLaunchConfig_t cfg = {};                     // its launch beside the end of the kernel before
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kRopeThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, hp == 1 ? rope_pick<1>(*a) : rope_pick<4>(*a), *a);
}

}  // namespace moe
