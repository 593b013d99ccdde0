// attn_tree.cu -- attention of a few query rows per request over the paged
// cache (moe_attn_tree): single tokens and drafted trees.
//
// The fresh rows' G query heads of a kv head are rows of one matrix (row r =
// fresh row * G + g), so every key and value is read once for all of them.
// An item is (request, kv head, row tile of 16 or 32 rows).  Its context is cut
// into chunks (16 tokens at D = 128, 32 at D = 64: 4 KB of keys, 4 KB of
// values), the chunks of all items stand in one line, and every CTA takes an
// equal range of that line whatever the requests' lengths are.  A warp owns
// every 8th chunk of its CTA's range with its own ring of two stages, filled by
// tensor-map copies (128-byte swizzle, so the fragment loads below do not
// conflict), and keeps running softmax statistics and sums of its own:
//   S = Q K^T, P = 2^(c (S - m)), l += sum P, O += P V,  c = softmax_scale * log2(e)
// with mma.sync m16n8k16 (16 or 32 rows are far too few for a 128-row tcgen05
// tile, and the cache's bytes bound the kernel).  m moves only when a score
// passes it by 2^8 (in P's terms), checked by one vote per chunk; P is rounded to
// the element type for the product, l and O are fp32 sums of the unrounded P
// and the products.  At the end of an item's part the 8 warps join in shared
// memory, in warp order.  A part that is not the whole context goes to the
// workspace, and the CTA that finishes an item's last part (a counter per item)
// joins the parts in the order of the context: no second launch, and no
// dependence on which CTA came last.
//
// Scores of tokens that a row does not see are replaced by -infinity.  Their v
// is multiplied by P = 0, so v past the context is zeroed in shared memory,
// and a drafted row's v that is infinite or NaN is added to the rows that see
// it and then zeroed.
#include <math.h>

#include "attn_tc.cuh"

namespace moe {

constexpr int kAtThreads = 256, kAtWarps = 8;
constexpr int kAtStages = 2;
constexpr int kAtStageBytes = 8192;
constexpr int kAtMinChunks = 8;                  // chunks of a CTA at least: one per warp costs no more time than one
constexpr int kAtExtra = 31;                     // chunks above the mean that are cheaper than a second part in a CTA
constexpr int kAtMaxB = MOE_ATTN_MAX_REQUESTS;
constexpr float kAtSlack = 8.f;
constexpr int kAtMostRows = 32;                  // mean rows of a request and kv head; more go to attn_wide.cu

struct AtArgs {
  CUtensorMap kmap, vmap;      // (64, 16, 1, 1) boxes over [pages][kv_heads][page_size][D]
  AttnArgs a;
  int *ctrl;                   // workspace control words
  int *tickets;                // per CTA that holds an item's first part: parts done; zero between calls
  float *part;                 // [2 * grid][rows][D]
  float2 *stat;                // [2 * grid][rows]  (m, l)
  int magic;                   // ceil(2^16 / group)
};

struct AtSmem {
  uint64_t full[kAtWarps][kAtStages];
  long long work[kAtMaxB + 1]; // chunks of the requests before
  int first[kAtMaxB], n[kAtMaxB], cached[kAtMaxB];   // first packed row, fresh rows, cached tokens
  long long wsum[kAtWarps];
  int wsum2[kAtWarps];
  int cand[kAtWarps][32];
  float2 stat[kAtWarps][32];   // (m, l) by warp and row
  int last;
};

template <int D>
struct AtGeom {
  static constexpr int kTok = 2048 / D;          // tokens of a chunk
  static constexpr int kLd = D + 8;              // row stride of the joining buffer (floats)
  static constexpr int kJoin = kAtWarps * 16 * kLd * 4;
  static constexpr int kSmem = kAtWarps * kAtStages * kAtStageBytes + kJoin + 1024;
};

template <bool F16>
__device__ __forceinline__ void at_mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void at_ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void at_ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// A place in the line of chunks: request, kv head, row tile, chunk; innermost
// last, so that the row tiles of a kv head read the same keys one after another.
struct AtPos {
  int b, hk, rt, chunk;
  int tiles, nch;              // row tiles of the request, chunks of its context
};
template <int TOK, int ROWS>
__device__ __forceinline__ void at_request(const AtSmem &s, const AttnArgs &a, AtPos &p) {
  const int n = s.n[p.b];
  p.tiles = (int)(((long long)n * a.group + ROWS - 1) / ROWS);
  p.nch = (int)((min((long long)s.cached[p.b] + n, (long long)a.max_pages << a.page_shift) + TOK - 1) / TOK);
}
template <int TOK, int ROWS>
__device__ __forceinline__ AtPos at_pos(const AtSmem &s, const AttnArgs &a, long long x) {
  int lo = 0, hi = a.B - 1;                        // largest b with work[b] <= x: requests without rows have no chunks
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.work[mid] <= x) lo = mid; else hi = mid - 1;
  }
  AtPos p;
  p.b = lo;
  at_request<TOK, ROWS>(s, a, p);
  const long long off = x - s.work[lo];
  const int item = (int)at_div(off, p.nch);
  p.chunk = (int)(off - (long long)item * p.nch);
  p.hk = at_idiv(item, p.tiles);
  p.rt = item - p.hk * p.tiles;
  return p;
}
// `step` chunks on (a place that exists).
template <int TOK, int ROWS>
__device__ __forceinline__ void at_advance(const AtSmem &s, const AttnArgs &a, AtPos &p, int step) {
  p.chunk += step;
  while (p.chunk >= p.nch) {
    p.chunk -= p.nch;
    if (++p.rt == p.tiles) {
      p.rt = 0;
      if (++p.hk == a.kv_heads) {
        p.hk = 0;
        do p.b++; while (s.n[p.b] == 0);
        at_request<TOK, ROWS>(s, a, p);
      }
    }
  }
}

// MT: row tiles of 16 rows per item.
template <int D, bool F16, int MT>
__global__ void __launch_bounds__(kAtThreads, 1) attn_tree_kernel(const __grid_constant__ AtArgs p) {
  extern __shared__ uint8_t dsm[];
  __shared__ AtSmem s;
  using G = AtGeom<D>;
  constexpr int kTok = G::kTok, kRows = 16 * MT, kHalves = D / 64, kBlocks = kTok / 16;
  const AttnArgs &a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q4 = lane & 3;
  const uint32_t smem0 = (smem_u32(dsm) + 1023u) & ~1023u;
  const uint32_t ring = smem0 + warp * (kAtStages * kAtStageBytes);
  uint8_t *const gen0 = dsm + (smem0 - smem_u32(dsm));
  uint8_t *const gring = gen0 + warp * (kAtStages * kAtStageBytes);
  float *const join = reinterpret_cast<float *>(gen0 + kAtWarps * kAtStages * kAtStageBytes);

  if (tid < kAtWarps * kAtStages) {
    mbar_init(&s.full[0][0] + tid, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // the line of chunks, every CTA alike
  long long total = 0;
  int nitems = 0;
  for (int b0 = 0; b0 < a.B; b0 += kAtThreads) {
    const int b = b0 + tid;
    long long v = 0;
    int items = 0;
    if (b < a.B) {
      const int lo = __ldg(a.cu + b), hi = __ldg(a.cu + b + 1), cached = max(__ldg(a.cached + b), 0);
      s.first[b] = lo;
      s.n[b] = lo < 0 ? 0 : max(0, min(hi, a.T) - lo);
      s.cached[b] = cached;
      AtPos q;
      q.b = b;
      at_request<kTok, kRows>(s, a, q);
      items = q.tiles * a.kv_heads;
      v = (long long)items * q.nch;
    }
    long long incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += u;
    }
    items = __reduce_add_sync(kFull, items);
    if (lane == 31) {
      s.wsum[warp] = incl;
      s.wsum2[warp] = items;
    }
    __syncthreads();
    long long at = total;
#pragma unroll
    for (int w = 0; w < kAtWarps; w++) {
      at += w < warp ? s.wsum[w] : 0;
      total += s.wsum[w];
      nitems += s.wsum2[w];
    }
    if (b < a.B) s.work[b] = at + incl - v;
    __syncthreads();
  }
  const AtShare share = at_share<kAtWarps>(
      s.work, a.B, total, nitems, kAtMinChunks, kAtExtra, s.cand,
      [&](int b) {
        AtPos q;
        q.b = b;
        at_request<kTok, kRows>(s, a, q);
        return q.tiles * a.kv_heads;
      },
      [&](int b) {
        AtPos q;
        q.b = b;
        at_request<kTok, kRows>(s, a, q);
        return q.nch;
      });
  const long long x0 = share.x0, x1 = share.x1;
  if (x0 >= x1) return;

  const float c = a.scale * 1.44269504088896340736f;
  bool ok = true;                                  // no wait of this warp has run out
  // the warp's chunks: x0 + warp, + 8, ..; `xp` is the next to be copied
  AtPos sp = at_pos<kTok, kRows>(s, a, x0);
  long long xp = x0 + warp;
  AtPos pp = sp;
  if (xp < x1) at_advance<kTok, kRows>(s, a, pp, warp);
  uint32_t kp = 0, kc = 0;                         // chunks copied, consumed
  auto issue = [&]() {
    const int stage = kp % kAtStages;
    if (lane == 0) {
      uint64_t *bar = &s.full[warp][stage];
      const uint32_t dst = ring + stage * kAtStageBytes;
      mbar_arrive_expect_tx(bar, kAtStageBytes);
#pragma unroll
      for (int k = 0; k < kBlocks; k++) {
        const int tok = pp.chunk * kTok + 16 * k, col = tok >> a.page_shift;
        const int id = col < a.max_pages ? __ldg(a.block_table + (size_t)pp.b * a.max_pages + col) : -1;
        const int page = (unsigned)id < (unsigned)a.num_pages ? id : a.num_pages;   // past the end: reads zeros
        const int place = tok & ((1 << a.page_shift) - 1);
#pragma unroll
        for (int hf = 0; hf < kHalves; hf++) {
          at_tma_4d(dst + (k * kHalves + hf) * 2048, &p.kmap, 64 * hf, place, pp.hk, page, bar);
          at_tma_4d(dst + kAtStageBytes / 2 + (k * kHalves + hf) * 2048, &p.vmap, 64 * hf, place, pp.hk, page, bar);
        }
      }
    }
    kp++;
    xp += kAtWarps;
    if (xp < x1) at_advance<kTok, kRows>(s, a, pp, kAtWarps);
  };
  for (int i = 0; i < kAtStages && xp < x1; i++) issue();

  long long xc = x0 + warp, xs = x0;               // the warp's next chunk; start of the part
  int nparts = 0;
  while (xs < x1) {
    // ---------------------------------------------------------------- a part of one item
    const int b = sp.b, nch = sp.nch, hk = sp.hk, row0 = sp.rt * kRows;
    const long long item0 = xs - sp.chunk;         // the item's place in the line
    const long long xe = min(x1, item0 + nch);
    const int first = s.first[b], n = s.n[b], cached = s.cached[b];
    const int ctx = (int)min((long long)cached + n, (long long)a.max_pages << a.page_shift);
    const int rows = (int)min((long long)kRows, (long long)n * a.group - row0);
    const int i0 = at_idiv(row0, a.group), g0 = row0 - i0 * a.group;
    // fresh row and query head of row r of the item
    auto row_of = [&](int r, int &i, int &hq) {
      const int dt = ((g0 + r) * p.magic) >> 16;
      i = i0 + dt;
      hq = hk * a.group + g0 + r - dt * a.group;
    };
    // o, m and l of a row -> the result: elements col .. col + N - 1
    auto emit = [&](int r, int col, float top, float sum, const float *acc) {
      int i, hq;
      row_of(r, i, hq);
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      uint16_t *dst = a.out.p + (long long)(first + i) * a.out.row + (long long)hq * a.out.head + col;
#pragma unroll
      for (int e = 0; e < D / 64; e++)
        *reinterpret_cast<uint2 *>(dst + 4 * e) = make_uint2(at_pack<F16>(acc[4 * e] * inv, acc[4 * e + 1] * inv),
                                                             at_pack<F16>(acc[4 * e + 2] * inv, acc[4 * e + 3] * inv));
      if (a.lse && col == 0)
        a.lse[(size_t)(first + i) * a.q_heads + hq] = sum == 0.f ? -INFINITY : top * a.scale + logf(sum);
    };

    uint32_t qf[MT][D / 16][4];
    uint64_t word[MT][2];                          // tree: the row's word; else bits unused and the row's place in `lim`
    int lim[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; mt++)
#pragma unroll
      for (int z = 0; z < 2; z++) {
        const int r = 16 * mt + g + 8 * z;
        int i, hq;
        row_of(min(r, rows - 1), i, hq);
        const uint16_t *src = a.q.p + (long long)(first + i) * a.q.row + (long long)hq * a.q.head;
        const bool real = r < rows;
#pragma unroll
        for (int k = 0; k < D / 16; k++) {
          qf[mt][k][z] = real ? __ldg(reinterpret_cast<const uint32_t *>(src + 16 * k + 2 * q4)) : 0u;
          qf[mt][k][2 + z] = real ? __ldg(reinterpret_cast<const uint32_t *>(src + 16 * k + 8 + 2 * q4)) : 0u;
        }
        word[mt][z] = a.tree_mask ? a.tree_mask[first + i] : 0;
        lim[mt][z] = i;
      }
    // whether row (mt, z) sees the fresh row f (0 <= f, its token inside the context)
    auto sees = [&](int mt, int z, int f) {
      return a.tree_mask ? f < 64 && ((word[mt][z] >> (f & 63)) & 1) : f <= lim[mt][z];
    };
    float o[MT][D / 8][4], m[MT][2], l[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; mt++) {
#pragma unroll
      for (int d = 0; d < D / 8; d++)
#pragma unroll
        for (int e = 0; e < 4; e++) o[mt][d][e] = 0.f;
      m[mt][0] = m[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.f;
    }

    for (; xc < xe; xc += kAtWarps, kc++) {
      const int stage = kc % kAtStages, tok0 = (int)(xc - item0) * kTok;
      if (ok && !mbar_wait_bounded(&s.full[warp][stage], (kc / kAtStages) & 1u)) {
        atomicOr(p.ctrl + kAttnCtrlFlags, MOE_FLAG_TIMEOUT);
        ok = false;
      }
      if (ok) {
        const uint32_t ks = ring + stage * kAtStageBytes, vs = ks + kAtStageBytes / 2;
        float sc[MT][kTok / 8][4];
#pragma unroll
        for (int mt = 0; mt < MT; mt++)
#pragma unroll
          for (int t = 0; t < kTok / 8; t++)
#pragma unroll
            for (int e = 0; e < 4; e++) sc[mt][t][e] = 0.f;
        {
          const int row = (lane & 7) + 8 * (lane >> 4), kh = (lane >> 3) & 1;
#pragma unroll
          for (int k = 0; k < D / 16; k++)
#pragma unroll
            for (int t = 0; t < kBlocks; t++) {
              uint32_t kf[4];
              at_ldsm4(kf, ks + (t * kHalves + (k >> 2)) * 2048 + row * 128 + (((2 * (k & 3) + kh) ^ (row & 7)) << 4));
#pragma unroll
              for (int mt = 0; mt < MT; mt++) {
                at_mma16<F16>(sc[mt][2 * t], qf[mt][k], kf[0], kf[1]);
                at_mma16<F16>(sc[mt][2 * t + 1], qf[mt][k], kf[2], kf[3]);
              }
            }
        }
        bool whole = tok0 + kTok <= cached;        // every row sees the whole chunk
        bool held[kBlocks];
#pragma unroll
        for (int t = 0; t < kBlocks; t++) {
          const int col = (tok0 + 16 * t) >> a.page_shift;
          const int id = col < a.max_pages ? __ldg(a.block_table + (size_t)b * a.max_pages + col) : -1;
          held[t] = (unsigned)id < (unsigned)a.num_pages;
          whole = whole && held[t];
        }
        if (!whole) {
#pragma unroll
          for (int mt = 0; mt < MT; mt++)
#pragma unroll
            for (int t = 0; t < kTok / 8; t++)
#pragma unroll
              for (int e = 0; e < 4; e++) {
                const int tok = tok0 + 8 * t + 2 * q4 + (e & 1);
                const bool v = held[t >> 1] && tok < ctx && (tok < cached || sees(mt, e >> 1, tok - cached));
                if (!v) sc[mt][t][e] = -INFINITY;
              }
        }
        float top[MT][2];
        bool up = false;
#pragma unroll
        for (int mt = 0; mt < MT; mt++)
#pragma unroll
          for (int z = 0; z < 2; z++) {
            top[mt][z] = fmaxf(sc[mt][0][2 * z], sc[mt][0][2 * z + 1]);
#pragma unroll
            for (int t = 1; t < kTok / 8; t++) top[mt][z] = at_max3(top[mt][z], sc[mt][t][2 * z], sc[mt][t][2 * z + 1]);
            up |= (top[mt][z] - m[mt][z]) * c > kAtSlack;      // -inf - -inf: NaN, not above
          }
        if (__any_sync(kFull, up)) {
#pragma unroll
          for (int mt = 0; mt < MT; mt++)
#pragma unroll
            for (int z = 0; z < 2; z++) {
              float m1 = fmaxf(m[mt][z], top[mt][z]);
              m1 = fmaxf(m1, __shfl_xor_sync(kFull, m1, 1));
              m1 = fmaxf(m1, __shfl_xor_sync(kFull, m1, 2));
              const float f = m1 == -INFINITY ? 1.f : at_exp2((m[mt][z] - m1) * c);
              m[mt][z] = m1;
              l[mt][z] *= f;
#pragma unroll
              for (int d = 0; d < D / 8; d++) {
                o[mt][d][2 * z] *= f;
                o[mt][d][2 * z + 1] *= f;
              }
            }
        }
        uint32_t pf[MT][kBlocks][4];
#pragma unroll
        for (int mt = 0; mt < MT; mt++)
#pragma unroll
          for (int z = 0; z < 2; z++) {
            const float mc = m[mt][z] == -INFINITY ? 0.f : -m[mt][z] * c;
#pragma unroll
            for (int t = 0; t < kTok / 8; t++) {
              const float e0 = at_exp2(fmaf(sc[mt][t][2 * z], c, mc)), e1 = at_exp2(fmaf(sc[mt][t][2 * z + 1], c, mc));
              l[mt][z] += e0 + e1;
              pf[mt][t >> 1][2 * (t & 1) + z] = at_pack<F16>(e0, e1);
            }
          }
        if (!whole) {
          uint8_t *vt = gring + stage * kAtStageBytes + kAtStageBytes / 2;
          uint32_t bad = 0;
          for (int e = lane; e < kTok * D / 8; e += 32) {
            const int tok = tok0 + 16 * (e / (16 * kHalves * 8)) + ((e >> 3) & 15);
            if (tok < cached) continue;
            uint4 *at = reinterpret_cast<uint4 *>(vt) + e;
            if (tok >= ctx) {
              *at = make_uint4(0u, 0u, 0u, 0u);
            } else {
              const uint4 w = *at;
              bad |= at_nonfinite<F16>(w.x) | at_nonfinite<F16>(w.y) | at_nonfinite<F16>(w.z) | at_nonfinite<F16>(w.w);
            }
          }
          __syncwarp();
          if (__any_sync(kFull, bad != 0)) {
            for (int t = max(0, cached - tok0); t < min(kTok, ctx - tok0); t++)
#pragma unroll
              for (int d = 0; d < D / 8; d++) {
                const uint32_t off = ((t >> 4) * kHalves + (d >> 3)) * 2048 + (t & 15) * 128 + (((d & 7) ^ (t & 7)) << 4) + 4 * q4;
                const uint32_t w = *reinterpret_cast<const uint32_t *>(vt + off);
                if (!at_nonfinite<F16>(w)) continue;
                const float u[2] = {at_value<F16>((uint16_t)(w & 0xFFFFu)), at_value<F16>((uint16_t)(w >> 16))};
#pragma unroll
                for (int mt = 0; mt < MT; mt++)
#pragma unroll
                  for (int z = 0; z < 2; z++)
                    if (held[t >> 4] && sees(mt, z, tok0 + t - cached)) {
                      if (!isfinite(u[0])) o[mt][d][2 * z] += u[0];
                      if (!isfinite(u[1])) o[mt][d][2 * z + 1] += u[1];
                    }
              }
            __syncwarp();
            for (int e = lane; e < kTok * D / 8; e += 32) {
              uint32_t *at = reinterpret_cast<uint32_t *>(vt) + 4 * e;
              const int tok = tok0 + 16 * (e / (16 * kHalves * 8)) + ((e >> 3) & 15);
              if (tok < cached) continue;
#pragma unroll
              for (int z = 0; z < 4; z++) at[z] &= ~(((at_nonfinite<F16>(at[z]) >> 15) & 0x00010001u) * 0xFFFFu);
            }
          }
          at_fence_async();                        // before the stage is copied into again
          __syncwarp();
        }
        {
          const int row = (lane & 7) + 8 * ((lane >> 3) & 1), dh = lane >> 4;
#pragma unroll
          for (int t = 0; t < kBlocks; t++)
#pragma unroll
            for (int d = 0; d < D / 16; d++) {
              uint32_t vf[4];
              at_ldsm4t(vf, vs + (t * kHalves + (d >> 2)) * 2048 + row * 128 + (((2 * (d & 3) + dh) ^ (row & 7)) << 4));
#pragma unroll
              for (int mt = 0; mt < MT; mt++) {
                at_mma16<F16>(o[mt][2 * d], pf[mt][t], vf[0], vf[1]);
                at_mma16<F16>(o[mt][2 * d + 1], pf[mt][t], vf[2], vf[3]);
              }
            }
        }
      }
      __syncwarp();                                // the stage is read
      if (ok && xp < x1) issue();
    }

    // ------------------------------------------------------------ join
    // Eight sources of 16 rows at a time, in shared memory: first the warps, in
    // warp order; then, in the CTA that finishes the item's last part, the
    // parts in the order of the context.  One loop for both, so that the second
    // runs instructions that are at hand.
    const bool entire = xs == item0 && xe == item0 + nch;
    const int slot = 2 * blockIdx.x + (nparts > 0);
    nparts++;
#pragma unroll
    for (int mt = 0; mt < MT; mt++)
#pragma unroll
      for (int z = 0; z < 2; z++) {
        float v = l[mt][z];
        v += __shfl_xor_sync(kFull, v, 1);
        v += __shfl_xor_sync(kFull, v, 2);
        if (q4 == 0) s.stat[warp][16 * mt + g + 8 * z] = make_float2(m[mt][z], v);
      }
    int c0 = 0, c1 = 0, slot0 = 0;                 // the CTAs that hold the item's first and last chunk
    bool parts = false;
    for (int mt = 0, k0 = 0;;) {
      constexpr int N = D / 16;                    // 16 threads a row, N elements each
      const int r = tid >> 4, col = (tid & 15) * N, r32 = 16 * mt + r;
      float top = -INFINITY, sum = 0.f, acc[N];
#pragma unroll
      for (int e = 0; e < N; e++) acc[e] = 0.f;
      for (;;) {
        float *mine = join + warp * (16 * G::kLd);
        if (!parts) {
#pragma unroll
          for (int q = 0; q < MT; q++)
            if (q == mt)
#pragma unroll
              for (int e = 0; e < D / 8; e++)
#pragma unroll
                for (int z = 0; z < 2; z++)
                  *reinterpret_cast<float2 *>(mine + (g + 8 * z) * G::kLd + 8 * e + 2 * q4) =
                      make_float2(o[q][e][2 * z], o[q][e][2 * z + 1]);
        } else {
          const int k = k0 + warp;
          const size_t at = (size_t)(k == c0 ? slot0 : 2 * k) * kRows + 16 * mt;
          const int rr = min(16, rows - 16 * mt);
          if (lane < 16) {
            float2 st = make_float2(-INFINITY, 0.f);
            if (k <= c1 && lane < rr) st = __ldcg(p.stat + at + lane);
            s.stat[warp][16 * mt + lane] = st;
          }
          if (k <= c1) {
            constexpr int kPer = 128 / D;          // rows of a warp's load
#pragma unroll 4
            for (int q = lane / (D / 4); q < rr; q += kPer) {
              const int e = 4 * (lane % (D / 4));
              *reinterpret_cast<float4 *>(mine + q * G::kLd + e) =
                  __ldcg(reinterpret_cast<const float4 *>(p.part + (at + q) * D + e));
            }
          }
        }
        __syncthreads();
        if (r32 < rows) {
          float t1 = top;
#pragma unroll
          for (int w = 0; w < kAtWarps; w++) t1 = fmaxf(t1, s.stat[w][r32].x);
          const float f0 = top == -INFINITY ? 1.f : at_exp2((top - t1) * c);
          top = t1;
          sum *= f0;
#pragma unroll
          for (int e = 0; e < N; e++) acc[e] *= f0;
#pragma unroll 2
          for (int w = 0; w < kAtWarps; w++) {
            const float2 st = s.stat[w][r32];
            if (st.y == 0.f) continue;             // a source in which the row sees nothing, or none
            const float f = at_exp2((st.x - top) * c);
            sum = fmaf(st.y, f, sum);
            const float4 *src = reinterpret_cast<const float4 *>(join + w * (16 * G::kLd) + r * G::kLd + col);
#pragma unroll
            for (int e = 0; e < N / 4; e++) {
              const float4 u = src[e];
              acc[4 * e] = fmaf(u.x, f, acc[4 * e]);
              acc[4 * e + 1] = fmaf(u.y, f, acc[4 * e + 1]);
              acc[4 * e + 2] = fmaf(u.z, f, acc[4 * e + 2]);
              acc[4 * e + 3] = fmaf(u.w, f, acc[4 * e + 3]);
            }
          }
        }
        if (!parts || (k0 += kAtWarps) > c1) break;
        __syncthreads();                           // the buffer is read
      }
      if (r32 < rows) {
        if (parts || entire) {
          emit(r32, col, top, sum, acc);
        } else {
          float4 *dst = reinterpret_cast<float4 *>(p.part + ((size_t)slot * kRows + r32) * D + col);
#pragma unroll
          for (int e = 0; e < N / 4; e++) dst[e] = make_float4(acc[4 * e], acc[4 * e + 1], acc[4 * e + 2], acc[4 * e + 3]);
          if ((tid & 15) == 0) p.stat[(size_t)slot * kRows + r32] = make_float2(top, sum);
        }
      }
      __syncthreads();
      if (++mt < MT) {
        k0 = c0;
        continue;
      }
      if (parts || entire) break;
      share.ctas_of(item0, item0 + nch - 1, c0, c1);
      slot0 = share.first_slot(c0, item0);
      if (tid == 0) {
        // release: the CTA's part, ordered before by the barrier; acquire: the others'
        int got;
        asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(got) : "l"(p.tickets + c0) : "memory");
        s.last = got == c1 - c0;
        if (got == c1 - c0) p.tickets[c0] = 0;
      }
      __syncthreads();
      if (!s.last) break;
      parts = true;
      mt = 0;
      k0 = c0;
    }
    xs = xe;
    if (xs < x1) at_advance<kTok, kRows>(s, a, sp, nch - sp.chunk);
  }
  // copies in flight (after a wait ran out) land before the CTA ends
  if (!ok)
    for (uint32_t k = kp > kAtStages ? kp - kAtStages : 0; k < kp; k++)
      mbar_wait_bounded(&s.full[warp][k % kAtStages], (k / kAtStages) & 1u);
}

namespace {
typedef void (*AtKernel)(const AtArgs);
template <int D, bool F16>
AtKernel at_kernel2(int mt) {
  return mt == 1 ? attn_tree_kernel<D, F16, 1> : attn_tree_kernel<D, F16, 2>;
}
AtKernel at_kernel(int head_dim, int f16, int mt) {
  if (head_dim == 64) return f16 ? at_kernel2<64, true>(mt) : at_kernel2<64, false>(mt);
  return f16 ? at_kernel2<128, true>(mt) : at_kernel2<128, false>(mt);
}
int at_smem(int head_dim) { return head_dim == 64 ? AtGeom<64>::kSmem : AtGeom<128>::kSmem; }
}  // namespace

cudaError_t attn_tree_setup(int head_dim, int f16) {
  for (int mt = 1; mt <= 2; mt++) {
    const cudaError_t err = cudaFuncSetAttribute(at_kernel(head_dim, f16, mt), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 at_smem(head_dim));
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

AttnTreeWs attn_tree_ws(int head_dim, int num_sms) {
  AttnTreeWs w;
  size_t off = kAttnCtrlBytes;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = (off + bytes + 255) / 256 * 256;
    return at;
  };
  w.tickets = take(4 * (size_t)num_sms);
  w.stat = take(8 * (size_t)(2 * num_sms) * 32);
  w.part = take(4 * (size_t)(2 * num_sms) * 32 * head_dim);
  w.wide = attn_wide_ws(off, head_dim, num_sms);
  w.total = w.wide.total;
  return w;
}

cudaError_t launch_attn_tree(const AttnArgs &a, uint8_t *ws, int num_sms, cudaStream_t stream) {
  const AttnTreeWs w = attn_tree_ws(a.head_dim, num_sms);
  const long long rows = ((long long)a.T * a.group + a.B - 1) / a.B;   // of a request and kv head, on the average
  if (rows > kAtMostRows) return launch_attn_wide_tree(a, ws, w.wide, num_sms, stream);
  AtArgs p;
  p.a = a;
  p.magic = (65536 + a.group - 1) / a.group;
  cudaError_t err = attn_encode_cache(&p.kmap, a.k_cache, a, 16);
  if (err == cudaSuccess) err = attn_encode_cache(&p.vmap, a.v_cache, a, 16);
  if (err != cudaSuccess) return err;
  p.ctrl = reinterpret_cast<int *>(ws);
  p.tickets = reinterpret_cast<int *>(ws + w.tickets);
  p.stat = reinterpret_cast<float2 *>(ws + w.stat);
  p.part = reinterpret_cast<float *>(ws + w.part);
  const int mt = rows <= 16 ? 1 : 2;
  at_kernel(a.head_dim, a.f16, mt)<<<num_sms, kAtThreads, at_smem(a.head_dim), stream>>>(p);
  return cudaGetLastError();
}

}  // namespace moe
