// attn_prompt.cu -- causal attention over whole packed prompts on the
// 5th-generation tensor cores (moe_attn_prompt).
//
// The G query heads of a kv head are rows of one matrix: row r = token * G + g
// of a request, so a key tile serves all of them and short prompts fill the
// 128-row tensor-core tiles.  An item is (request, kv head, 256 rows): two row
// tiles of 128 that share every key/value tile of 128 tokens.  With c =
// softmax_scale * log2(e), per row tile and key tile j:
//   S = Q K_j^T                                   (tcgen05, both from shared memory)
//   m' = max(m, max S);  P = 2^(c (S - m'));  l = l 2^(c (m - m')) + sum P
//   O = O 2^(c (m - m')) + P V_j                  (tcgen05, P from tensor memory)
// and at the end o = O / l, lse = softmax_scale * m + ln l.  The running maximum
// that P is taken against moves only when the true one passes it by 2^8 (in P's
// terms): P then stays below 2^8, which bf16 and f16 hold, l is summed in fp32
// from the unrounded values, and O (in tensor memory) is hardly ever rescaled.
// P is rounded to the element type because the tensor cores multiply equal
// types; O and l stay fp32.
//
// One CTA per SM, 12 warps:
//   warps 0-3, 4-7  softmax of row tile 0 and 1: a thread owns a row, so the
//                   maximum and the sum need no exchange between threads;
//                   also the rare rescaling of O and the epilogue
//   warp 8          key/value tiles by tensor-map copies (128-byte swizzle)
//                   into a ring, in the order K0 K1 V0 K2 V1 ..; takes the items
//   warp 9          MMA issue: S of tile j + 1 is issued with PV of tile j, so
//                   one row tile's softmax runs while the other's MMAs do
//   warps 10-11     Q rows into swizzled shared memory (cp.async, zero for rows
//                   past the end); the scan described below
// Tensor memory: S0, S1 (128 columns each, P over their first 64), O0, O1.
//
// A tile that reaches past the first row's token holds keys that some rows, or
// all, may not see.  Their scores are replaced by -infinity, so P is 0; but 0
// times an infinite or NaN v is NaN, so warps 10-11 scan those tiles' v, zero
// such elements and note their tokens, and the epilogue adds them to the
// rows that do see the token.
//
// Items are taken from a counter, those with most key tiles first: an item's
// length depends on its row tile alone, so with the requests ranked by
// length the k-th longest .. ranges have a closed form (struct Order).
//
// Bound: with G = 8, D = 128 and long prompts the tensor pipe (2 x 512 cycles
// a row tile and key tile); with D = 64 the exponentials.
#include <math.h>

#include "attn_tc.cuh"

namespace moe {

constexpr int kApThreads = 384;
constexpr int kApRows = 256, kApTile = 128;      // rows of an item; rows of a row tile, tokens of a key tile
constexpr int kApRegsSoft = 208, kApRegsRest = 88;
constexpr int kApWTma = 8, kApWMma = 9, kApWHelp = 10;
constexpr int kApMaxB = MOE_ATTN_MAX_REQUESTS;
constexpr float kApSlack = 8.f;                  // log2 of the largest P

template <int D>
struct ApGeom {
  static constexpr int kTileBytes = kApTile * D * 2;
  static constexpr int kSlots = D == 128 ? 4 : 8;
  static constexpr int kSmem = 2 * kTileBytes + kSlots * kTileBytes + 1024;
};

struct ApArgs {
  CUtensorMap kmap, vmap;      // (64, 1, 128) boxes over [rows][kv_heads][D], 128-byte swizzle
  AttnArgs a;
  int *ctrl;                   // workspace control words
  int magic;                   // ceil(2^16 / group)
};

struct ApItem {
  int b, hk, row0;             // request, kv head, first row (of the request's rows)
  int first;                   // the request's first packed row
  int tok0, g0;                // token and group place of row0
  int rows;                    // rows of the item (<= 256)
  int n0, n1;                  // key tiles of the two row tiles
};

struct ApSmem {
  uint64_t kv_full[8], kv_empty[8];
  uint64_t q_full, q_empty, s_full[2], p_full[2], o_done[2], v_clean[3], v_next, sched_full[2], sched_empty[2], drain;
  uint32_t tmem;
  int wsum[2][kApThreads / 32];
  ApItem item[2];
  uint32_t bad[2][2][3][4];    // by item parity, scanning warp and masked tile: tokens with a non-finite v
  // requests by falling length
  uint16_t order[kApMaxB];
  int tiles[kApMaxB];          // 256-row items per kv head of the k-th longest
  int before[kApMaxB + 1];     // items (per kv head) of row tiles in which fewer than k + 1 requests take part
};

// The idx-th item (per kv head) by falling row tile: row tiles [tiles[k], tiles[k - 1])
// have the k longest requests.
__device__ __forceinline__ void ap_item(const ApSmem &s, const ApArgs &p, int idx, ApItem &it) {
  const AttnArgs &a = p.a;
  const int e = idx / a.kv_heads;
  it.hk = idx - e * a.kv_heads;
  int lo = 0, hi = a.B - 1;                        // largest k with before[k] <= e
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.before[mid] <= e) lo = mid; else hi = mid - 1;
  }
  const int k = lo + 1, off = e - s.before[lo];
  const int rt = s.tiles[lo] - 1 - off / k;
  it.b = s.order[off % k];
  it.first = __ldg(a.cu + it.b);
  const int n = min(__ldg(a.cu + it.b + 1), a.T) - it.first;
  it.row0 = rt * kApRows;
  it.rows = (int)min((long long)kApRows, (long long)n * a.group - it.row0);
  it.tok0 = it.row0 / a.group;
  it.g0 = it.row0 - it.tok0 * a.group;
  it.n0 = (it.tok0 + (((it.g0 + min(it.rows, kApTile) - 1) * p.magic) >> 16)) / kApTile + 1;
  it.n1 = it.rows > kApTile ? (it.tok0 + (((it.g0 + it.rows - 1) * p.magic) >> 16)) / kApTile + 1 : 0;
}

// Positions in the ring's order K0 K1 V0 K2 V1 .. V[n-1] of an item of n tiles.
__device__ __forceinline__ int ap_pos_k(int j) { return j ? 2 * j - 1 : 0; }
__device__ __forceinline__ int ap_pos_v(int j, int n) { return j + 1 < n ? 2 * j + 2 : 2 * n - 1; }

template <int D, bool F16>
__global__ void __launch_bounds__(kApThreads, 1) attn_prompt_kernel(const __grid_constant__ ApArgs p) {
  extern __shared__ uint8_t dsm[];
  __shared__ ApSmem s;
  using G = ApGeom<D>;
  constexpr int kSlots = G::kSlots, kTB = G::kTileBytes, kHalves = D / 64;
  const AttnArgs &a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t smem0 = (smem_u32(dsm) + 1023u) & ~1023u;
  const uint32_t q_smem = smem0, ring = smem0 + 2 * kTB;
  uint8_t *const generic0 = dsm + (smem0 - smem_u32(dsm));

  if (tid == 0) {
    for (int i = 0; i < kSlots; i++) {
      mbar_init(&s.kv_full[i], 1);
      mbar_init(&s.kv_empty[i], 1);
    }
    mbar_init(&s.q_full, 64);
    mbar_init(&s.q_empty, 1);
    for (int i = 0; i < 2; i++) {
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.p_full[i], 4);
      mbar_init(&s.o_done[i], 1);
      mbar_init(&s.sched_full[i], 1);
      mbar_init(&s.sched_empty[i], 11);            // 8 softmax warps, MMA warp, 2 helper warps
    }
    for (int i = 0; i < 3; i++) mbar_init(&s.v_clean[i], 2);
    mbar_init(&s.v_next, 1);
    mbar_init(&s.drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kApWMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s.tmem)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // requests by falling number of row tiles (equal ones by index), every CTA alike
  for (int b = tid; b < a.B; b += kApThreads) {
    const int lo = __ldg(a.cu + b), n = max(0, min(__ldg(a.cu + b + 1), a.T) - lo);
    s.before[b] = lo < 0 ? 0 : (int)(((long long)n * a.group + kApRows - 1) / kApRows);
  }
  __syncthreads();
  for (int b = tid; b < a.B; b += kApThreads) {
    const int mine = s.before[b];
    int rank = 0;
    for (int o = 0; o < a.B; o++) rank += s.before[o] > mine || (s.before[o] == mine && o < b);
    s.order[rank] = (uint16_t)b;
    s.tiles[rank] = mine;
  }
  at_fence_before();
  __syncthreads();
  at_fence_after();
  int total = 0;                                   // items per kv head
  for (int k0 = 0; k0 < a.B; k0 += kApThreads) {
    const int k = k0 + tid;
    // row tiles [tiles[k], tiles[k - 1]) hold the k longest requests each
    const int v = k > 0 && k < a.B ? k * (s.tiles[k - 1] - s.tiles[k]) : 0;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += t;
    }
    if (lane == 31) s.wsum[0][warp] = incl;
    __syncthreads();
    int at = total;
#pragma unroll
    for (int w = 0; w < kApThreads / 32; w++) {
      at += w < warp ? s.wsum[0][w] : 0;
      total += s.wsum[0][w];
    }
    if (k < a.B) s.before[k] = at + incl;
    __syncthreads();
  }
  total = (total + a.B * s.tiles[a.B - 1]) * a.kv_heads;   // row tiles that every request has come last
  const uint32_t tb = s.tmem;
  const float c = a.scale * 1.44269504088896340736f;

  if (warp < 8) {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kApRegsSoft));
    const int h = warp >> 2, ri = tid & 255;       // row of the item
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t ts = tb + lanes + 128u * h, to = tb + lanes + 256u + 128u * h;
    uint32_t ns = 0;                               // tiles of this half so far
    bool ok = true;
    for (int i = 0;; i++) {
      if (!mbar_wait_bounded(&s.sched_full[i & 1], (uint32_t)(i >> 1) & 1u)) {
        atomicOr(p.ctrl + kAttnCtrlFlags, MOE_FLAG_TIMEOUT);
        break;
      }
      const ApItem it = s.item[i & 1];
      if (it.b < 0) break;
      const int nt = h ? it.n1 : it.n0;
      const int x = it.g0 + ri, dt = (x * p.magic) >> 16;
      const bool real = ri < it.rows;
      const int lim = it.tok0 + (real ? dt : ((it.g0 + it.rows - 1) * p.magic) >> 16);   // last visible token
      float m = -INFINITY;                         // the maximum that P is taken against
      float2 l2 = make_float2(0.f, 0.f);
      for (int j = 0; j < nt; j++, ns++) {
        if (!mbar_wait_bounded(&s.s_full[h], ns & 1u)) {
          atomicOr(p.ctrl + kAttnCtrlFlags, MOE_FLAG_TIMEOUT);
          ok = false;
          break;
        }
        at_fence_after();
        float v[128];
#pragma unroll
        for (int q = 0; q < 4; q++) at_ld32(ts + 32u * q, v + 32 * q);
        at_wait_ld();
        const int col0 = kApTile * j;
        if (__any_sync(kFull, col0 + kApTile - 1 > lim)) {
          const int vis = lim - col0;
#pragma unroll
          for (int q = 0; q < 128; q++) v[q] = q > vis ? -INFINITY : v[q];
        }
        float mx[4];
#pragma unroll
        for (int q = 0; q < 4; q++) {
          mx[q] = fmaxf(v[32 * q], v[32 * q + 1]);
#pragma unroll
          for (int e = 2; e < 32; e += 2) mx[q] = at_max3(mx[q], v[32 * q + e], v[32 * q + e + 1]);
        }
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        if (j == 0) {
          m = top;
        } else if (__any_sync(kFull, (top - m) * c > kApSlack)) {
          const float m1 = fmaxf(m, top), f = m1 == -INFINITY ? 1.f : at_exp2((m - m1) * c);
          m = m1;
          l2.x *= f;
          l2.y *= f;
          if (!mbar_wait_bounded(&s.o_done[h], (ns - 1u) & 1u)) {
            atomicOr(p.ctrl + kAttnCtrlFlags, MOE_FLAG_TIMEOUT);
            ok = false;
            break;
          }
          at_fence_after();
#pragma unroll 1
          for (int q = 0; q < D / 32; q++) {
            float o[32];
            at_ld32(to + 32u * q, o);
            at_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; e++) o[e] *= f;
            at_st32(to + 32u * q, o);
          }
          at_wait_st();
        }
        const float mc = m == -INFINITY ? 0.f : -m * c;
        const float2 c2 = make_float2(c, c), mc2 = make_float2(mc, mc);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int q = 0; q < 4; q++) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; e++) {
            float2 t = ffma2(make_float2(v[32 * q + 2 * e], v[32 * q + 2 * e + 1]), c2, mc2);
            t.x = at_exp2(t.x);
            t.y = at_exp2(t.y);
            sum[e & 1] = at_add2(sum[e & 1], t);
            pk[e] = at_pack<F16>(t.x, t.y);
          }
          at_st16(ts + 16u * q, pk);
        }
        l2 = at_add2(l2, at_add2(sum[0], sum[1]));
        at_wait_st();
        at_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.p_full[h]);
      }
      if (!ok) break;
      if (nt > 0) {
        // ---------------------------------------------------------- epilogue
        if (!mbar_wait_bounded(&s.o_done[h], (ns - 1u) & 1u)) {
          atomicOr(p.ctrl + kAttnCtrlFlags, MOE_FLAG_TIMEOUT);
          break;
        }
        at_fence_after();
        const float l = l2.x + l2.y;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int t = it.first + it.tok0 + dt, hq = it.hk * a.group + x - dt * a.group;
        const int mt0 = (it.tok0 + 1) / kApTile;   // first masked tile
        uint32_t anybad = 0;
#pragma unroll
        for (int w = 0; w < 12; w++) anybad |= s.bad[i & 1][0][w >> 2][w & 3] | s.bad[i & 1][1][w >> 2][w & 3];
        uint16_t *dst = a.out.p + (long long)t * a.out.row + (long long)hq * a.out.head;
#pragma unroll 1
        for (int q = 0; q < D / 32; q++) {
          float o[32];
          at_ld32(to + 32u * q, o);
          at_wait_ld();
          if (anybad) {
            for (int w = 0; w < 12; w++) {
              uint32_t bits = s.bad[i & 1][0][w >> 2][w & 3] | s.bad[i & 1][1][w >> 2][w & 3];
              for (; bits; bits &= bits - 1) {
                const int tok = (mt0 + (w >> 2)) * kApTile + 32 * (w & 3) + __ffs(bits) - 1;
                if (tok > lim) continue;
                const uint16_t *vp = a.v.p + (long long)(it.first + tok) * a.v.row + (long long)it.hk * a.v.head + 32 * q;
#pragma unroll
                for (int e = 0; e < 32; e++) {
                  const float u = at_value<F16>(__ldg(vp + e));
                  if (!isfinite(u)) o[e] += u;
                }
              }
            }
          }
          if (real) {
#pragma unroll
            for (int e = 0; e < 4; e++) {
              uint4 w;
              w.x = at_pack<F16>(o[8 * e] * inv, o[8 * e + 1] * inv);
              w.y = at_pack<F16>(o[8 * e + 2] * inv, o[8 * e + 3] * inv);
              w.z = at_pack<F16>(o[8 * e + 4] * inv, o[8 * e + 5] * inv);
              w.w = at_pack<F16>(o[8 * e + 6] * inv, o[8 * e + 7] * inv);
              *reinterpret_cast<uint4 *>(dst + 32 * q + 8 * e) = w;
            }
          }
        }
        at_fence_before();
        if (a.lse && real) a.lse[(size_t)t * a.q_heads + hq] = l == 0.f ? -INFINITY : m * a.scale + logf(l);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.sched_empty[i & 1]);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kApRegsRest));
    if (warp == kApWTma) {
      // ---------------------------------------------------------- items and key/value tiles
      if (lane == 0) {
        int pos = 0, idx = blockIdx.x;
        bool ok = true;
        for (int i = 0; ok; i++) {
          if (i >= 2 && !mbar_wait_bounded(&s.sched_empty[i & 1], (uint32_t)((i >> 1) - 1) & 1u)) {
            atomicOr(p.ctrl + kAttnCtrlFlags, MOE_FLAG_TIMEOUT);
            break;
          }
          ApItem it;
          it.b = -1;
          if (idx < total) ap_item(s, p, idx, it);
          s.item[i & 1] = it;
          mbar_arrive(&s.sched_full[i & 1]);
          if (idx >= total) break;
          idx = gridDim.x + atomicAdd(p.ctrl + kAttnCtrlNext, 1);
          const int n = max(it.n0, it.n1);
          for (int q = 0; q < 2 * n; q++, pos++) {
            // K0 K1 V0 K2 V1 .. K[n-1] V[n-2] V[n-1]
            const bool isk = q < 2 * n - 1 && (q == 0 || (q & 1));
            const int j = isk ? (q + 1) >> 1 : (q == 2 * n - 1 ? n - 1 : (q >> 1) - 1);
            const int slot = pos % kSlots;
            if (pos >= kSlots && !mbar_wait_bounded(&s.kv_empty[slot], (uint32_t)(pos / kSlots - 1) & 1u)) {
              atomicOr(p.ctrl + kAttnCtrlFlags, MOE_FLAG_TIMEOUT);
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&s.kv_full[slot], (uint32_t)kTB);
            for (int hf = 0; hf < kHalves; hf++)
              at_tma_3d(ring + slot * kTB + hf * (kApTile * 128), isk ? &p.kmap : &p.vmap, 64 * hf, it.hk,
                        it.first + j * kApTile, &s.kv_full[slot]);
          }
        }
        // copies in flight land before the CTA ends
        for (int q = (pos > kSlots ? pos - kSlots : 0); q < pos; q++)
          mbar_wait_bounded(&s.kv_full[q % kSlots], (uint32_t)(q / kSlots) & 1u);
        // the last CTA to have taken its last item leaves the counters at zero
        __threadfence();
        if (atomicAdd(p.ctrl + kAttnCtrlDone, 1) == (int)gridDim.x - 1) {
          p.ctrl[kAttnCtrlNext] = 0;
          p.ctrl[kAttnCtrlDone] = 0;
        }
      }
      __syncwarp();
    } else if (warp == kApWMma) {
      // ---------------------------------------------------------- MMA issue
      if (lane == 0) {
        constexpr uint32_t id_s = at_idesc(F16, kApTile, false), id_o = at_idesc(F16, D, true);
        int base = 0;
        uint32_t clean[3] = {0, 0, 0};
        uint32_t np[2] = {0, 0};
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
          if (ok && !mbar_wait_bounded(bar, parity)) {
            atomicOr(p.ctrl + kAttnCtrlFlags, MOE_FLAG_TIMEOUT);
            ok = false;
          }
          return ok;
        };
        auto issue_s = [&](int h, int slot) {
#pragma unroll
          for (int k = 0; k < D / 16; k++) {
            const uint32_t off = (uint32_t)((k >> 2) * (kApTile * 128) + (k & 3) * 32);
            at_mma_ss(tb + 128u * h, at_desc(q_smem + h * kTB + off, 16), at_desc(ring + slot * kTB + off, 16), id_s, k > 0);
          }
          at_commit(&s.s_full[h]);
        };
        auto issue_o = [&](int h, int slot, int j) {
#pragma unroll
          for (int k = 0; k < kApTile / 16; k++)
            at_mma_ts(tb + 256u + 128u * h, tb + 128u * h + 8u * k, at_desc(ring + slot * kTB + 2048u * k, kApTile * 128),
                      id_o, (uint32_t)(j > 0 || k > 0));
          at_commit(&s.o_done[h]);
        };
        for (int i = 0; ok; i++) {
          if (!wait(&s.sched_full[i & 1], (uint32_t)(i >> 1) & 1u)) break;
          const ApItem it = s.item[i & 1];
          if (it.b < 0) break;
          const int n = max(it.n0, it.n1), mt0 = (it.tok0 + 1) / kApTile;
          if (!wait(&s.q_full, (uint32_t)i & 1u)) break;
          if (!wait(&s.kv_full[base % kSlots], (uint32_t)(base / kSlots) & 1u)) break;
          at_fence_after();
          issue_s(0, base % kSlots);
          if (it.n1 > 0) issue_s(1, base % kSlots);
          at_commit(&s.kv_empty[base % kSlots]);
          if (n == 1) at_commit(&s.q_empty);
          for (int j = 0; j < n && ok; j++) {
            const int pk = base + ap_pos_k(j + 1), pv = base + ap_pos_v(j, n);
            const bool next = j + 1 < n;
            if (next && !wait(&s.kv_full[pk % kSlots], (uint32_t)(pk / kSlots) & 1u)) break;
            if (!wait(&s.kv_full[pv % kSlots], (uint32_t)(pv / kSlots) & 1u)) break;
            if (j >= mt0) {
              const int z = j - mt0;               // a constant index in each of the three cases
              const uint32_t ph = z == 0 ? clean[0]++ : (z == 1 ? clean[1]++ : clean[2]++);
              if (!wait(&s.v_clean[z], ph & 1u)) break;
            }
            if (!next) mbar_arrive(&s.v_next);     // the next item's scans may signal
#pragma unroll
            for (int h = 0; h < 2; h++) {
              const int nh = h ? it.n1 : it.n0;
              if (j < nh) {
                if (!wait(&s.p_full[h], np[h]++ & 1u)) break;
                at_fence_after();
                issue_o(h, pv % kSlots, j);
                if (j + 1 < nh) issue_s(h, pk % kSlots);
              }
            }
            if (!ok) break;
            at_commit(&s.kv_empty[pv % kSlots]);
            if (next) at_commit(&s.kv_empty[pk % kSlots]);
            if (j + 2 == n) at_commit(&s.q_empty);
          }
          base += 2 * n;
          mbar_arrive(&s.sched_empty[i & 1]);
        }
        // every MMA issued has completed before tensor memory is released
        at_commit(&s.drain);
        mbar_wait_bounded(&s.drain, 0u);
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------- Q rows, and the scan of masked tiles' v
      const int ht = tid - 32 * kApWHelp;
      int base = 0;
      bool ok = true;
      for (int i = 0; ok; i++) {
        if (!mbar_wait_bounded(&s.sched_full[i & 1], (uint32_t)(i >> 1) & 1u)) break;
        const ApItem it = s.item[i & 1];
        if (it.b < 0) break;
        const int n = max(it.n0, it.n1), mt0 = (it.tok0 + 1) / kApTile;
        if (lane < 12) s.bad[i & 1][warp - kApWHelp][lane >> 2][lane & 3] = 0u;
        __syncwarp();
        if (i > 0 && !mbar_wait_bounded(&s.q_empty, (uint32_t)(i - 1) & 1u)) break;
        constexpr int kChunks = D / 8;
        const int ch = ht % kChunks;
        const uint32_t qd = q_smem + (uint32_t)(ch >> 3) * (kApTile * 128);
        for (int r = ht / kChunks; r < kApRows; r += 64 / kChunks) {
          if (r >= kApTile && it.n1 == 0) break;
          const int x = it.g0 + r, dt = (x * p.magic) >> 16;
          const uint16_t *src = a.q.p + (long long)(it.first + it.tok0 + dt) * a.q.row +
                                (long long)(it.hk * a.group + x - dt * a.group) * a.q.head + 8 * ch;
          const int rr = r & (kApTile - 1);
          at_cp16(qd + (r >= kApTile ? kTB : 0) + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4), r < it.rows ? src : a.q.p,
                  r < it.rows);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        at_fence_async();
        mbar_arrive(&s.q_full);
        // the MMA warp has seen this item's predecessor's scans: a barrier is
        // never a phase ahead of its reader
        if (i > 0 && !mbar_wait_bounded(&s.v_next, (uint32_t)(i - 1) & 1u)) break;
        for (int j = mt0; j < n; j++) {
          const int pv = base + ap_pos_v(j, n), slot = pv % kSlots;
          if (!mbar_wait_bounded(&s.kv_full[slot], (uint32_t)(pv / kSlots) & 1u)) {
            ok = false;
            break;
          }
          uint8_t *tile = generic0 + 2 * kTB + slot * kTB;
          const int r0 = max(0, it.tok0 + 1 - j * kApTile);      // earlier tokens are seen by every row
          for (int hf = 0; hf < kHalves; hf++)
            for (int e = r0 * 8 + ht; e < kApTile * 8; e += 64) {
              uint4 *at = reinterpret_cast<uint4 *>(tile + hf * (kApTile * 128)) + e;
              const uint4 w = *at;
              const uint32_t f[4] = {at_nonfinite<F16>(w.x), at_nonfinite<F16>(w.y), at_nonfinite<F16>(w.z), at_nonfinite<F16>(w.w)};
              if (f[0] | f[1] | f[2] | f[3]) {
                uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int z = 0; z < 4; z++) u[z] &= ~(((f[z] >> 15) & 0x00010001u) * 0xFFFFu);
                *at = make_uint4(u[0], u[1], u[2], u[3]);
                atomicOr(&s.bad[i & 1][warp - kApWHelp][j - mt0][(e >> 3) >> 5], 1u << ((e >> 3) & 31));
              }
            }
          at_fence_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.v_clean[j - mt0]);
        }
        base += 2 * n;
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.sched_empty[i & 1]);
      }
    }
  }
  at_fence_before();
  __syncthreads();
  if (warp == kApWMma) {
    at_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tb), "r"(512) : "memory");
  }
}

namespace {
typedef void (*ApKernel)(const ApArgs);
ApKernel ap_kernel(int head_dim, int f16) {
  if (head_dim == 64) return f16 ? attn_prompt_kernel<64, true> : attn_prompt_kernel<64, false>;
  return f16 ? attn_prompt_kernel<128, true> : attn_prompt_kernel<128, false>;
}
int ap_smem(int head_dim) { return head_dim == 64 ? ApGeom<64>::kSmem : ApGeom<128>::kSmem; }
}  // namespace

cudaError_t attn_prompt_setup(int head_dim, int f16) {
  const ApKernel k = ap_kernel(head_dim, f16);
  cudaFuncAttributes at;
  cudaError_t err = cudaFuncGetAttributes(&at, k);
  if (err != cudaSuccess) return err;
  // the register shares of the warpgroups have to fit what the CTA is launched with
  if (at.numRegs * kApThreads < kApRegsSoft * 256 + kApRegsRest * 128) return cudaErrorInvalidConfiguration;
  return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, ap_smem(head_dim));
}

static cudaError_t encode_rows(CUtensorMap *map, const RowView &r, int T, int heads, int head_dim, int f16) {
  const AttnMapEncodeFn enc = attn_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)heads, (cuuint64_t)T};
  const cuuint64_t strides[2] = {(cuuint64_t)r.head * 2, (cuuint64_t)r.row * 2};
  const cuuint32_t box[3] = {64, 1, kApTile};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult e = enc(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, r.p, dims, strides,
                         box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return e == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t launch_attn_prompt(const AttnArgs &a, int *ctrl, int num_sms, cudaStream_t stream) {
  ApArgs p;
  p.a = a;
  p.ctrl = ctrl;
  p.magic = (65536 + a.group - 1) / a.group;
  cudaError_t err = encode_rows(&p.kmap, a.k, a.T, a.kv_heads, a.head_dim, a.f16);
  if (err == cudaSuccess) err = encode_rows(&p.vmap, a.v, a.T, a.kv_heads, a.head_dim, a.f16);
  if (err != cudaSuccess) return err;
  // items at most: every request may end inside a row tile
  const long long items = (((long long)a.T * a.group + kApRows - 1) / kApRows + a.B) * a.kv_heads;
  const int grid = (int)(items < num_sms ? items : num_sms);
  ap_kernel(a.head_dim, a.f16)<<<grid, kApThreads, ap_smem(a.head_dim), stream>>>(p);
  return cudaGetLastError();
}

}  // namespace moe
