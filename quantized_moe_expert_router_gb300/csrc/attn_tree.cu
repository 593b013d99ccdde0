// attn_tree.cu -- attention of a few query rows per request over the paged
// cache (moe_attn_tree): single tokens and drafted trees.
//
// The fresh rows' G query heads of a kv head are rows of one matrix (row r =
// fresh row * G + g), so every key and value is read once for 16 of them.  An
// item is (request, kv head, row tile of 16 rows).  Its context is cut into
// chunks (16 tokens at D = 128, 32 at D = 64: 4 KB of keys, 4 KB of values), and
// the chunks of all items stand in one line that the grid shares.  A warp has a
// ring of two stages of its own, filled by tensor-map copies (128-byte swizzle,
// so the fragment loads below do not conflict), and goes from chunk to chunk
// without a barrier, with the running statistics of a softmax:
//   S = Q K^T, P = 2^(c (S - m)), l += sum P, O += P V,  c = softmax_scale * log2(e)
// with mma.sync m16n8k16 (16 rows are far too few for a 128-row tcgen05 tile, and
// the cache's bytes bound the kernel).  m moves only when a score passes it by
// 2^8 (in P's terms), checked by one vote per chunk; P is rounded to the element
// type for the product, l and O are fp32 sums of the unrounded P and the
// products.  Two kernels share this and differ in who joins what:
//   attn_few_kernel   a CTA takes a part of one item (at_share), its warps every
//                     8th chunk of it, and joins their sums in shared memory;
//   attn_many_kernel  (more items than CTAs) a warp takes an equal range of the
//                     line; an item that lies in it is stored from the registers,
//                     and only the first and the last one of a warp are joined,
//                     when all warps are done.
// us in the few and the many kernel, bf16, D = 128, 8 kv heads of 4: 64 requests of
// a row at 500 34.7, 16.4 (512 items); 20 at 500 17.0, 12.5 (160); 18 at 500 10.8,
// 12.7 (144); 8 of up to 8 rows at up to 4000 16.8, 20.5; 1 row at 1000 8.0, 10.7.
// Parts of an item in several CTAs go to the workspace, and the CTA that finishes
// its last part (a counter per item) joins them: no second launch.  All joins
// go in the order of the context, so the result does not depend on timing.
//
// Scores of tokens that a row does not see are replaced by -infinity.  Their v
// is multiplied by P = 0, so v past the context is zeroed in shared memory,
// and a drafted row's v that is infinite or NaN is added to the rows that see
// it and then zeroed.
//
// Bound: long contexts by HBM: 16 requests of a row at up to 100000 tokens, 8 kv
// heads of 8, read 2.8 GB in 405 us, 7.0 TB/s (a plain copy has 6.8).  Short ones by
// the latencies of one call: 1 row at 1000 takes 8.0 us for 4 MB (9.0 among other calls; launch 1.5,
// lengths and shares 2, page numbers and keys 2, a warp's chunk 0.8, the two joins 1.5); 8
// requests of 2 to 8 drafted rows at 500 to 4000 take 17 us for 58 MB, the longest
// with two row tiles that each read the chunks.
#include <math.h>

#include "attn_tc.cuh"

namespace moe {

constexpr int kAtThreads = 256, kAtWarps = 8;
constexpr int kAtStages = 2;
constexpr int kAtStageBytes = 8192;
constexpr int kAtRows = 16;                      // rows of an item
constexpr int kAtMaxB = MOE_ATTN_MAX_REQUESTS;
constexpr float kAtSlack = 8.f;
// Calls that stay here and not on attn_wide.cu, whose tiles of 128 rows read the
// context once for all of them: up to kAtMostRows rows of a request and kv head on
// the average, and more while the contexts, as long as the block table's rows,
// are at most kAtMostChunks chunks a warp with each of the row tiles of 16.  bf16,
// D = 128, 4 kv heads, us here and there (chunks a warp):
//   32 rows, 1 request of 8000: 16.4, 21.5 (3.3);    256 rows, 1 of 500: 12.3, 16.2 (1.9)
//   128 rows, 1 of 4000: 16.4, 18.1 (6.6);           192 rows: 18.6, 18.0 (10);     256 rows: 22.6, 18.0 (13)
//   64 rows, 1 of 30000: 31.7, 28.9 (25);            128 rows: 53.3, 29.4 (49)
// The rule knows the call's sizes only; the lengths are on the device.  A table that is
// wider than the contexts counts as long contexts: 256 rows, 1 of 500, in a table of
// 131072 tokens takes 16.8 there (11.7 here), 8 of them 23.0 (29.5).  A long part of a
// prompt among single tokens goes by the mean: 256 tokens at 4000 among 255 of one at
// 1000, 4 heads of 4, 111 (apart 24 + 87); 1024 at 0 among 63, 8 heads of 1, 91 (23 + 47).
constexpr int kAtMostRows = 32, kAtMostChunks = 10;
constexpr int kAtMinChunks = 8;                  // chunks of a CTA at least, one a warp: 1 row at 1000, us with 4, 8, 16: 8.8, 8.0, 9.0

struct AtArgs {
  CUtensorMap kmap, vmap;      // (64, 16, 1, 1) boxes over [pages][kv_heads][page_size][D]
  AttnArgs a;
  int *ctrl;                   // workspace control words
  int *tickets;                // per CTA that holds an item's first part: parts done; zero between calls
  float *part;                 // [2 * grid][16][D]  parts of the items that a CTA shares with others
  float2 *stat;                // [2 * grid][16]     (m, l)
  int magic;                   // ceil(2^16 / group)
};

// The requests, and where their chunks stand in the line.
struct AtTable {
  long long work[kAtMaxB + 1]; // chunks of the requests before
  int first[kAtMaxB], n[kAtMaxB], cached[kAtMaxB];   // first packed row, fresh rows, cached tokens
  long long wsum[kAtWarps];
  int wsum2[kAtWarps];
};

// A place in the line of chunks: request, kv head, row tile, chunk; innermost
// last, so that the row tiles of a kv head read the same keys one after another.
struct AtPos {
  int b, hk, rt, chunk;
  int tiles, nch;              // row tiles of the request, chunks of its context
};

template <int D>
struct AtGeom {
  static constexpr int kTok = 2048 / D;          // tokens of a chunk
  static constexpr int kLd = D + 8;              // row stride of a part in shared memory (floats)
  static constexpr int kRing = kAtWarps * kAtStages * kAtStageBytes;
  static constexpr int kSmem = kRing + kAtWarps * kAtRows * kLd * 4 + 1024;
  static_assert(kAtRows * kLd * 4 <= kAtStages * kAtStageBytes, "a warp's second part takes the place of its ring");
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
template <int TOK>
__device__ __forceinline__ void at_request(const AtTable &s, const AttnArgs &a, AtPos &p) {
  const int n = s.n[p.b];
  // rows <= 2^20 x 128; the block table's tokens <= 2^30, and `cached` is at most that
  p.tiles = (n * a.group + kAtRows - 1) / kAtRows;
  p.nch = (min(s.cached[p.b] + n, a.max_pages << a.page_shift) + TOK - 1) / TOK;
}
// Fills in the table; every CTA does the same.  All threads; ends with a barrier.
template <int TOK>
__device__ __forceinline__ void at_table(AtTable &s, const AttnArgs &a, long long &total, int &nitems) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  total = 0;
  nitems = 0;
  for (int b0 = 0; b0 < a.B; b0 += kAtThreads) {
    const int b = b0 + tid;
    long long v = 0;
    int items = 0;
    if (b < a.B) {
      const int lo = __ldg(a.cu + b), hi = __ldg(a.cu + b + 1);
      const int cached = min(max(__ldg(a.cached + b), 0), a.max_pages << a.page_shift);   // no sum with rows passes 2^31
      s.first[b] = lo;
      s.n[b] = lo < 0 ? 0 : max(0, min(hi, a.T) - lo);
      s.cached[b] = cached;
      AtPos q;
      q.b = b;
      at_request<TOK>(s, a, q);
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
}
template <int TOK>
__device__ __forceinline__ AtPos at_pos(const AtTable &s, const AttnArgs &a, long long x) {
  int lo = 0, hi = a.B - 1;                        // largest b with work[b] <= x: requests without rows have no chunks
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.work[mid] <= x) lo = mid; else hi = mid - 1;
  }
  AtPos p;
  p.b = lo;
  at_request<TOK>(s, a, p);
  const long long off = x - s.work[lo];
  const int item = (int)at_div(off, p.nch);
  p.chunk = (int)(off - (long long)item * p.nch);
  p.hk = at_idiv(item, p.tiles);
  p.rt = item - p.hk * p.tiles;
  return p;
}
// On to the next items while p.chunk is past the end (to a place that exists).
template <int TOK>
__device__ __forceinline__ void at_settle(const AtTable &s, const AttnArgs &a, AtPos &p) {
  while (p.chunk >= p.nch) {
    p.chunk -= p.nch;
    if (++p.rt == p.tiles) {
      p.rt = 0;
      if (++p.hk == a.kv_heads) {
        p.hk = 0;
        do p.b++; while (s.n[p.b] == 0);
        at_request<TOK>(s, a, p);
      }
    }
  }
}

// The rows of an item.
struct AtItem {
  int first, hk, rows, i0, g0; // first packed row of the request; rows; fresh row and group place of row 0
  __device__ __forceinline__ AtItem(const AtTable &s, const AttnArgs &a, const AtPos &p) {
    const int row0 = p.rt * kAtRows;
    first = s.first[p.b];
    hk = p.hk;
    rows = min(kAtRows, s.n[p.b] * a.group - row0);
    i0 = at_idiv(row0, a.group);
    g0 = row0 - i0 * a.group;
  }
  // fresh row and query head of row r
  __device__ __forceinline__ void row(const AttnArgs &a, int magic, int r, int &i, int &hq) const {
    const int dt = ((g0 + r) * magic) >> 16;
    i = i0 + dt;
    hq = hk * a.group + g0 + r - dt * a.group;
  }
};

// Copies the keys and values of the chunk at p into a stage (one lane).
template <int D>
__device__ __forceinline__ void at_copy(const AtArgs &g, const AtPos &p, uint32_t dst, uint64_t *bar) {
  constexpr int kTok = AtGeom<D>::kTok, kHalves = D / 64;
  const AttnArgs &a = g.a;
  mbar_arrive_expect_tx(bar, kAtStageBytes + a.stall);
#pragma unroll
  for (int k = 0; k < kTok / 16; k++) {
    const int tok = p.chunk * kTok + 16 * k, col = tok >> a.page_shift;
    const int id = col < a.max_pages ? __ldg(a.block_table + (size_t)p.b * a.max_pages + col) : -1;
    const int page = (unsigned)id < (unsigned)a.num_pages ? id : a.num_pages;   // past the end: reads zeros
    const int place = tok & ((1 << a.page_shift) - 1);
#pragma unroll
    for (int hf = 0; hf < kHalves; hf++) {
      at_tma_4d(dst + (k * kHalves + hf) * 2048, &g.kmap, 64 * hf, place, p.hk, page, bar);
      at_tma_4d(dst + kAtStageBytes / 2 + (k * kHalves + hf) * 2048, &g.vmap, 64 * hf, place, p.hk, page, bar);
    }
  }
}

// A warp's work on an item: its rows in fragments, and the sums so far.
template <int D, bool F16>
struct AtSums {
  static constexpr int kTok = AtGeom<D>::kTok, kHalves = D / 64, kBlocks = kTok / 16;
  uint32_t qf[D / 16][4];
  uint64_t word[2];            // the rows' words of the tree mask
  int lim[2];                  // the rows' fresh rows
  int b, cached, ctx;          // request, its cached tokens, and the end of its context
  float o[D / 8][4], m[2], l[2];
  bool far;                    // a row of the lane takes m off its scores before it scales them
  __device__ __forceinline__ void begin(const AtTable &s, const AtArgs &p, const AtItem &it, int request) {
    const AttnArgs &a = p.a;
    const int g = (threadIdx.x & 31) >> 2, q4 = threadIdx.x & 3;
    b = request;
    cached = s.cached[b];
    ctx = min(cached + s.n[b], a.max_pages << a.page_shift);
#pragma unroll
    for (int z = 0; z < 2; z++) {
      const int r = g + 8 * z;
      int i, hq;
      it.row(a, p.magic, min(r, it.rows - 1), i, hq);
      const uint16_t *src = a.q.p + (long long)(it.first + i) * a.q.row + (long long)hq * a.q.head;
      const bool real = r < it.rows;
#pragma unroll
      for (int k = 0; k < D / 16; k++) {
        qf[k][z] = real ? __ldg(reinterpret_cast<const uint32_t *>(src + 16 * k + 2 * q4)) : 0u;
        qf[k][2 + z] = real ? __ldg(reinterpret_cast<const uint32_t *>(src + 16 * k + 8 + 2 * q4)) : 0u;
      }
      word[z] = a.tree_mask ? a.tree_mask[it.first + i] : 0;
      lim[z] = i;
      m[z] = -INFINITY;
      l[z] = 0.f;
    }
    far = false;
#pragma unroll
    for (int d = 0; d < D / 8; d++)
#pragma unroll
      for (int e = 0; e < 4; e++) o[d][e] = 0.f;
  }
  // whether row z of the lane sees the fresh row f (0 <= f, its token inside the context)
  __device__ __forceinline__ bool sees(const AttnArgs &a, int z, int f) const {
    return a.tree_mask ? f < 64 && ((word[z] >> (f & 63)) & 1) : f <= lim[z];
  }
  // whether the page of each 16 tokens of chunk ch is in the cache
  __device__ __forceinline__ void pages(const AttnArgs &a, int ch, bool (&held)[kBlocks]) const {
#pragma unroll
    for (int t = 0; t < kBlocks; t++) {
      const int col = (ch * kTok + 16 * t) >> a.page_shift;
      const int id = col < a.max_pages ? __ldg(a.block_table + (size_t)b * a.max_pages + col) : -1;
      held[t] = (unsigned)id < (unsigned)a.num_pages;
    }
  }
  // Adds the chunk from token tok0 on, which lies in the stage at `ring` (`gring`).
  __device__ __forceinline__ void add(const AttnArgs &a, float c, uint32_t ring, uint8_t *gring, int tok0, const bool (&held)[kBlocks]) {
    const int lane = threadIdx.x & 31, q4 = lane & 3;
    bool whole_seen = tok0 + kTok <= cached;       // every row sees the whole chunk
#pragma unroll
    for (int t = 0; t < kBlocks; t++) whole_seen = whole_seen && held[t];
    const uint32_t ks = ring, vs = ring + kAtStageBytes / 2;
    float sc[kTok / 8][4];
    {
      // two sums a tile, of even and odd steps: four or more chains of products
      float s2[2][kTok / 8][4];
#pragma unroll
      for (int w = 0; w < 2; w++)
#pragma unroll
        for (int t = 0; t < kTok / 8; t++)
#pragma unroll
          for (int e = 0; e < 4; e++) s2[w][t][e] = 0.f;
      const int row = (lane & 7) + 8 * (lane >> 4), kh = (lane >> 3) & 1;
#pragma unroll
      for (int k = 0; k < D / 16; k++)
#pragma unroll
        for (int t = 0; t < kBlocks; t++) {
          uint32_t kf[4];
          at_ldsm4(kf, ks + (t * kHalves + (k >> 2)) * 2048 + row * 128 + (((2 * (k & 3) + kh) ^ (row & 7)) << 4));
          at_mma16<F16>(s2[k & 1][2 * t], qf[k], kf[0], kf[1]);
          at_mma16<F16>(s2[k & 1][2 * t + 1], qf[k], kf[2], kf[3]);
        }
#pragma unroll
      for (int t = 0; t < kTok / 8; t++)
#pragma unroll
        for (int e = 0; e < 4; e++) sc[t][e] = s2[0][t][e] + s2[1][t][e];
    }
    if (!whole_seen) {
#pragma unroll
      for (int t = 0; t < kTok / 8; t++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const int tok = tok0 + 8 * t + 2 * q4 + (e & 1);
          const bool v = held[t >> 1] && tok < ctx && (tok < cached || sees(a, e >> 1, tok - cached));
          if (!v) sc[t][e] = -INFINITY;
        }
    }
    float top[2];
    bool up = false;
#pragma unroll
    for (int z = 0; z < 2; z++) {
      top[z] = fmaxf(sc[0][2 * z], sc[0][2 * z + 1]);
#pragma unroll
      for (int t = 1; t < kTok / 8; t++) top[z] = at_max3(top[z], sc[t][2 * z], sc[t][2 * z + 1]);
      up |= (top[z] - m[z]) * c > kAtSlack;    // -inf - -inf: NaN, not above
    }
    float ref[2] = {m[0], m[1]};                   // what c takes off the scores with them
    if (__any_sync(kFull, up || far)) {
      far = false;
#pragma unroll
      for (int z = 0; z < 2; z++) {
        float m1 = fmaxf(m[z], top[z]);
        m1 = fmaxf(m1, __shfl_xor_sync(kFull, m1, 1));
        m1 = fmaxf(m1, __shfl_xor_sync(kFull, m1, 2));
        const float f = m1 == -INFINITY ? 1.f : at_exp2((m[z] - m1) * c);
        m[z] = m1;
        l[z] *= f;
#pragma unroll
        for (int d = 0; d < D / 8; d++) {
          o[d][2 * z] *= f;
          o[d][2 * z + 1] *= f;
        }
        const bool own = at_far(m1, c);
        const float off = own ? -m1 : 0.f;
        ref[z] = own ? 0.f : m1;
        far |= own;
#pragma unroll
        for (int t = 0; t < kTok / 8; t++) {
          sc[t][2 * z] += off;
          sc[t][2 * z + 1] += off;
        }
      }
    }
    uint32_t pf[kBlocks][4];
#pragma unroll
    for (int z = 0; z < 2; z++) {
      const float mc = ref[z] == -INFINITY ? 0.f : -ref[z] * c;
#pragma unroll
      for (int t = 0; t < kTok / 8; t++) {
        const float e0 = at_exp2(fmaf(sc[t][2 * z], c, mc)), e1 = at_exp2(fmaf(sc[t][2 * z + 1], c, mc));
        l[z] += e0 + e1;
        pf[t >> 1][2 * (t & 1) + z] = at_pack<F16>(e0, e1);
      }
    }
    if (!whole_seen) {
      uint8_t *vt = gring + kAtStageBytes / 2;
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
            for (int z = 0; z < 2; z++)
              if (held[t >> 4] && sees(a, z, tok0 + t - cached)) {
                if (!isfinite(u[0])) o[d][2 * z] += u[0];
                if (!isfinite(u[1])) o[d][2 * z + 1] += u[1];
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
          at_mma16<F16>(o[2 * d], pf[t], vf[0], vf[1]);
          at_mma16<F16>(o[2 * d + 1], pf[t], vf[2], vf[3]);
        }
    }
    __syncwarp();                                  // the stage is read
  }
  // The sums over the quad's columns.
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int z = 0; z < 2; z++) {
      l[z] += __shfl_xor_sync(kFull, l[z], 1);
      l[z] += __shfl_xor_sync(kFull, l[z], 2);
    }
  }
  // O of the warp's rows, and their statistics, in shared memory.
  __device__ __forceinline__ void put(float *dst, float2 *stat) const {
    constexpr int kLd = AtGeom<D>::kLd;
    const int lane = threadIdx.x & 31, g = lane >> 2, q4 = lane & 3;
#pragma unroll
    for (int z = 0; z < 2; z++) {
      if (q4 == 0) stat[g + 8 * z] = make_float2(m[z], l[z]);
#pragma unroll
      for (int d = 0; d < D / 8; d++)
        *reinterpret_cast<float2 *>(dst + (g + 8 * z) * kLd + 8 * d + 2 * q4) = make_float2(o[d][2 * z], o[d][2 * z + 1]);
    }
  }
};

// A row being joined: N of its elements.
template <int N>
struct AtRow {
  float top = kAtLeast, sum = 0.f, acc[N];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int e = 0; e < N; e++) acc[e] = 0.f;
  }
  // K more parts of the row: their statistics and the lane's elements
  template <int K>
  __device__ __forceinline__ void add(const float2 (&st)[K], const float4 (&v)[K][N / 4], float c) {
    float t1 = top;
#pragma unroll
    for (int k = 0; k < K; k++) t1 = fmaxf(t1, st[k].x);
    const float f0 = top == t1 ? 1.f : at_exp2((top - t1) * c);
    top = t1;
    sum *= f0;
#pragma unroll
    for (int e = 0; e < N; e++) acc[e] *= f0;
#pragma unroll
    for (int k = 0; k < K; k++) {
      const bool some = !(st[k].y < 0.f);        // else no part (v may hold anything)
      const float f = some ? at_exp2((st[k].x - t1) * c) : 0.f;
      sum = fmaf(st[k].y, f, sum);
#pragma unroll
      for (int e = 0; e < N / 4; e++) {
        acc[4 * e] = fmaf(some ? v[k][e].x : 0.f, f, acc[4 * e]);
        acc[4 * e + 1] = fmaf(some ? v[k][e].y : 0.f, f, acc[4 * e + 1]);
        acc[4 * e + 2] = fmaf(some ? v[k][e].z : 0.f, f, acc[4 * e + 2]);
        acc[4 * e + 3] = fmaf(some ? v[k][e].w : 0.f, f, acc[4 * e + 3]);
      }
    }
  }
};

// The row to its place: elements N hl .. of a lane's 16.
template <int N, bool F16>
__device__ __forceinline__ void at_emit(const AtArgs &p, const AtItem &it, int r, int hl, const AtRow<N> &row) {
  const AttnArgs &a = p.a;
  int i, hq;
  it.row(a, p.magic, r, i, hq);
  const float inv = row.sum == 0.f ? 0.f : 1.f / row.sum;
  uint16_t *dst = a.out.p + (long long)(it.first + i) * a.out.row + (long long)hq * a.out.head + N * hl;
#pragma unroll
  for (int e = 0; e < N / 4; e++)
    *reinterpret_cast<uint2 *>(dst + 4 * e) = make_uint2(at_pack<F16>(row.acc[4 * e] * inv, row.acc[4 * e + 1] * inv),
                                                         at_pack<F16>(row.acc[4 * e + 2] * inv, row.acc[4 * e + 3] * inv));
  if (a.lse && hl == 0)
    a.lse[(size_t)(it.first + i) * a.q_heads + hq] = row.sum == 0.f ? -INFINITY : row.top * a.scale + logf(row.sum);
}
// A row of a part that goes to the workspace.
template <int D, int N>
__device__ __forceinline__ void at_keep(const AtArgs &p, int slot, int r, int hl, const AtRow<N> &row) {
  const size_t at = (size_t)slot * kAtRows + r;
  float4 *dst = reinterpret_cast<float4 *>(p.part + at * D + N * hl);
#pragma unroll
  for (int k = 0; k < N / 4; k++) dst[k] = make_float4(row.acc[4 * k], row.acc[4 * k + 1], row.acc[4 * k + 2], row.acc[4 * k + 3]);
  if (hl == 0) p.stat[at] = make_float2(row.top, row.sum);
}
// One more part of the item whose first part CTA c0 holds: whether it was the
// last of `parts`.  Release: the CTA's part, ordered before by a barrier; acquire:
// the others'.
__device__ __forceinline__ bool at_ticket(const AtArgs &p, int c0, int parts) {
  int got;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(got) : "l"(p.tickets + c0) : "memory");
  if (got + 1 == parts) p.tickets[c0] = 0;
  return got + 1 == parts;
}
// Row r of an item from its parts in the workspace: CTA c0's in `slot0`, those
// of the CTAs up to c1 in their slot 0.
template <int D, int N>
__device__ __forceinline__ void at_gather(const AtArgs &p, int c0, int c1, int slot0, int r, int hl, float c, AtRow<N> &row) {
  for (int k0 = c0; k0 <= c1; k0 += 8) {           // eight parts at a time, so that their loads wait together
    float2 st[8];
    float4 v[8][N / 4];
#pragma unroll
    for (int q = 0; q < 8; q++) {
      const int k = min(k0 + q, c1);
      const size_t ps = (size_t)(k == c0 ? slot0 : 2 * k) * kAtRows + r;
      st[q] = k0 + q <= c1 ? __ldcg(p.stat + ps) : make_float2(-INFINITY, kAtNoPart);
#pragma unroll
      for (int w = 0; w < N / 4; w++) v[q][w] = __ldcg(reinterpret_cast<const float4 *>(p.part + ps * D + N * hl) + w);
    }
    row.add(st, v, c);
  }
}

// ------------------------------------------------------------------ few items
struct AtFewSmem {
  uint64_t full[kAtWarps][kAtStages];
  AtTable t;
  int cand[kAtWarps][32];
  float2 stat[kAtWarps][kAtRows];                  // (m, l) by warp
  int last;
};

template <int D, bool F16>
__global__ void __launch_bounds__(kAtThreads, 1) attn_few_kernel(const __grid_constant__ AtArgs p) {
  extern __shared__ uint8_t dsm[];
  __shared__ AtFewSmem s;
  using G = AtGeom<D>;
  constexpr int kTok = G::kTok, kLd = G::kLd;
  const AttnArgs &a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t smem0 = (smem_u32(dsm) + 1023u) & ~1023u;
  const uint32_t ring = smem0 + warp * (kAtStages * kAtStageBytes);
  uint8_t *const gen0 = dsm + (smem0 - smem_u32(dsm));
  uint8_t *const gring = gen0 + warp * (kAtStages * kAtStageBytes);
  float *const join = reinterpret_cast<float *>(gen0 + G::kRing);

  if (tid < kAtWarps * kAtStages) {
    mbar_init(&s.full[0][0] + tid, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  long long total;
  int nitems;
  at_table<kTok>(s.t, a, total, nitems);
  auto request = [&](int b) {
    AtPos q;
    q.b = b;
    at_request<kTok>(s.t, a, q);
    return q;
  };
  const AtShare share =
      at_share<kAtWarps>(s.t.work, a.B, total, nitems, kAtMinChunks, s.cand,
                         [&](int b) { return request(b).tiles * a.kv_heads; }, [&](int b) { return request(b).nch; });
  const long long x0 = share.x0, x1 = share.x1;
  if (x0 >= x1) return;

  const float c = a.scale * 1.44269504088896340736f;
  bool ok = true;                                  // no wait of this warp has run out
  // the warp's chunks: x0 + warp, + 8, ..; `xp` is the next to be copied
  AtPos sp = at_pos<kTok>(s.t, a, x0), pp = sp;
  long long xp = x0 + warp;
  pp.chunk += warp;
  if (xp < x1) at_settle<kTok>(s.t, a, pp);
  uint32_t kp = 0, kc = 0;                         // chunks copied, consumed
  auto issue = [&]() {
    const int stage = kp++ % kAtStages;
    if (lane == 0) at_copy<D>(p, pp, ring + stage * kAtStageBytes, &s.full[warp][stage]);
    xp += kAtWarps;
    pp.chunk += kAtWarps;
    if (xp < x1) at_settle<kTok>(s.t, a, pp);
  };
  for (int i = 0; i < kAtStages && xp < x1; i++) issue();

  long long xc = x0 + warp;                        // the warp's next chunk
  int nparts = 0;
  for (long long xs = x0; xs < x1;) {
    // ---------------------------------------------------------------- a part of one item
    const AtItem it(s.t, a, sp);
    const long long item0 = xs - sp.chunk;         // the item's place in the line
    const long long xe = min(x1, item0 + sp.nch);
    AtSums<D, F16> w;
    w.begin(s.t, p, it, sp.b);
    for (; xc < xe; xc += kAtWarps, kc++) {
      const int stage = kc % kAtStages, ch = (int)(xc - item0);
      bool held[AtSums<D, F16>::kBlocks];
      w.pages(a, ch, held);
      if (ok && !mbar_wait_bounded(&s.full[warp][stage], (kc / kAtStages) & 1u, a.wait_ns)) {
        atomicOr(p.ctrl + kAttnCtrlFlags, MOE_FLAG_TIMEOUT);
        ok = false;
      }
      ok = __all_sync(kFull, ok);
      if (!ok) continue;
      w.add(a, c, ring + stage * kAtStageBytes, gring + stage * kAtStageBytes, ch * kTok, held);
      if (xp < x1) issue();
    }
    w.finish();

    // ---------------------------------------------------------------- the warps join, 16 threads a row
    constexpr int N = D / 16;
    const int r = tid >> 4, hl = tid & 15;
    const bool entire = xs == item0 && xe == item0 + sp.nch;
    w.put(join + warp * (kAtRows * kLd), s.stat[warp]);
    __syncthreads();
    if (r < it.rows) {
      AtRow<N> row;
      row.clear();
#pragma unroll 1
      for (int q = 0; q < kAtWarps; q += 4) {
        float2 st[4];
        float4 v[4][N / 4];
#pragma unroll
        for (int e = 0; e < 4; e++) {
          st[e] = s.stat[q + e][r];
          const float4 *src = reinterpret_cast<const float4 *>(join + (q + e) * (kAtRows * kLd) + r * kLd + N * hl);
#pragma unroll
          for (int k = 0; k < N / 4; k++) v[e][k] = src[k];
        }
        row.add(st, v, c);
      }
      if (entire) at_emit<N, F16>(p, it, r, hl, row);
      else at_keep<D>(p, 2 * blockIdx.x + (nparts > 0), r, hl, row);
    }
    nparts++;
    __syncthreads();
    if (!entire) {
      int c0, c1;
      share.ctas_of(item0, item0 + sp.nch - 1, c0, c1);
      if (tid == 0) s.last = at_ticket(p, c0, c1 - c0 + 1);
      __syncthreads();
      if (s.last && r < it.rows) {
        AtRow<N> row;
        row.clear();
        at_gather<D>(p, c0, c1, share.first_slot(c0, item0), r, hl, c, row);
        at_emit<N, F16>(p, it, r, hl, row);
      }
      __syncthreads();
    }
    xs = xe;
    sp.chunk = sp.nch;
    if (xs < x1) at_settle<kTok>(s.t, a, sp);
  }
  // copies in flight (after a wait ran out) land before the CTA ends
  if (!ok)
    for (uint32_t k = kp > kAtStages ? kp - kAtStages : 0; k < kp; k++)
      mbar_wait_bounded(&s.full[warp][k % kAtStages], (k / kAtStages) & 1u, a.wait_ns);
}

// ----------------------------------------------------------------- many items
struct AtSeg {                 // a warp's part of an item
  long long item0;             // the item's place in the line; -1: none
  AtPos at;
};
struct AtManySmem {
  uint64_t full[kAtWarps][kAtStages];
  AtTable t;
  AtSeg seg[kAtWarps][2];
  float2 stat[kAtWarps][2][kAtRows];               // (m, l)
  int last[2];
};
static_assert(kAtThreads == kAtWarps * 2 * kAtRows && kAtRows == 2 * kAtWarps, "one thread a statistic; two rows a warp");

template <int D, bool F16>
__global__ void __launch_bounds__(kAtThreads, 1) attn_many_kernel(const __grid_constant__ AtArgs p) {
  extern __shared__ uint8_t dsm[];
  __shared__ AtManySmem s;
  using G = AtGeom<D>;
  constexpr int kTok = G::kTok, kLd = G::kLd;
  const AttnArgs &a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q4 = lane & 3;
  const uint32_t smem0 = (smem_u32(dsm) + 1023u) & ~1023u;
  const uint32_t ring = smem0 + warp * (kAtStages * kAtStageBytes);
  uint8_t *const gen0 = dsm + (smem0 - smem_u32(dsm));
  uint8_t *const gring = gen0 + warp * (kAtStages * kAtStageBytes);
  // a warp's two parts: beside the rings, and in the place of its ring
  auto part_of = [&](int w, int z) {
    return reinterpret_cast<float *>(z ? gen0 + w * (kAtStages * kAtStageBytes) : gen0 + G::kRing + w * (kAtRows * kLd * 4));
  };

  if (tid < kAtWarps * kAtStages) {
    mbar_init(&s.full[0][0] + tid, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid < 2 * kAtWarps) s.seg[tid >> 1][tid & 1].item0 = -1;
  (&s.stat[0][0][0])[tid] = make_float2(-INFINITY, kAtNoPart);       // until there is a part
  long long total;
  int nitems;
  at_table<kTok>(s.t, a, total, nitems);
  // warp i of `warps` takes chunks start(i) .. start(i + 1): per or per + 1 of them
  const int ctas = (int)min((total + kAtWarps - 1) / kAtWarps, (long long)gridDim.x), warps = ctas * kAtWarps;
  if ((int)blockIdx.x >= ctas) return;
  const long long per = at_div(total, warps), rem = total - per * warps;
  auto start = [&](int i) { return i * per + min((long long)i, rem); };
  auto cta_of = [&](long long x) {
    const long long big = rem * (per + 1);
    return (int)(x < big ? at_div(x, per + 1) : rem + at_div(x - big, per)) / kAtWarps;
  };
  const int me = blockIdx.x * kAtWarps + warp;
  const long long x0 = start(me), x1 = start(me + 1);

  const float c = a.scale * 1.44269504088896340736f;
  bool ok = true;                                  // no wait of this warp has run out
  if (x0 < x1) {
    AtPos sp = at_pos<kTok>(s.t, a, x0), pp = sp;
    long long xp = x0;                             // the next chunk to be copied, at `pp`
    uint32_t kp = 0, kc = 0;                       // chunks copied, consumed
    auto issue = [&]() {
      const int stage = kp % kAtStages;
      if (lane == 0) at_copy<D>(p, pp, ring + stage * kAtStageBytes, &s.full[warp][stage]);
      kp++;
      pp.chunk++;
      if (++xp < x1) at_settle<kTok>(s.t, a, pp);
    };
    for (int i = 0; i < kAtStages && xp < x1; i++) issue();

    for (long long x = x0; x < x1;) {
      // ---------------------------------------------------------------- a part of one item
      const AtItem it(s.t, a, sp);
      const long long item0 = x - sp.chunk;        // the item's place in the line
      const int c1 = (int)min((long long)sp.nch, x1 - item0);                // end of the part, in the item's chunks
      const bool whole = sp.chunk == 0 && c1 == sp.nch;
      AtSums<D, F16> w;
      w.begin(s.t, p, it, sp.b);
      for (int ch = sp.chunk; ch < c1; ch++, kc++) {
        const int stage = kc % kAtStages;
        bool held[AtSums<D, F16>::kBlocks];
        w.pages(a, ch, held);
        if (ok && !mbar_wait_bounded(&s.full[warp][stage], (kc / kAtStages) & 1u, a.wait_ns)) {
          atomicOr(p.ctrl + kAttnCtrlFlags, MOE_FLAG_TIMEOUT);
          ok = false;
        }
        ok = __all_sync(kFull, ok);
        if (!ok) continue;
        w.add(a, c, ring + stage * kAtStageBytes, gring + stage * kAtStageBytes, ch * kTok, held);
        if (xp < x1) issue();
      }
      w.finish();
      if (whole) {
        // a quad holds pairs of a row; a transpose within it gives each lane 16 bytes of 64
#pragma unroll
        for (int z = 0; z < 2; z++) {
          int i, hq;
          it.row(a, p.magic, g + 8 * z, i, hq);
          const bool real = g + 8 * z < it.rows;
          const float inv = w.l[z] == 0.f ? 0.f : 1.f / w.l[z];
          uint16_t *dst = a.out.p + (long long)(it.first + i) * a.out.row + (long long)hq * a.out.head + 8 * q4;
#pragma unroll
          for (int cb = 0; cb < D / 32; cb++) {
            uint32_t u[4];
#pragma unroll
            for (int e = 0; e < 4; e++) u[e] = at_pack<F16>(w.o[4 * cb + e][2 * z] * inv, w.o[4 * cb + e][2 * z + 1] * inv);
            at_quad_transpose(u, q4);
            if (real) *reinterpret_cast<uint4 *>(dst + 32 * cb) = make_uint4(u[0], u[1], u[2], u[3]);
          }
          if (a.lse && real && q4 == 0)
            a.lse[(size_t)(it.first + i) * a.q_heads + hq] = w.l[z] == 0.f ? -INFINITY : w.m[z] * a.scale + logf(w.l[z]);
        }
      } else {
        const int z1 = x != x0;                    // the warp's first part, or its last
        if (lane == 0) {
          s.seg[warp][z1].item0 = item0;
          s.seg[warp][z1].at = sp;
        }
        w.put(part_of(warp, z1), s.stat[warp][z1]);
      }
      x = item0 + c1;
      sp.chunk = c1;
      if (x < x1) at_settle<kTok>(s.t, a, sp);
    }
    // copies in flight (after a wait ran out) land before the CTA ends
    if (!ok)
      for (uint32_t k = kp > kAtStages ? kp - kAtStages : 0; k < kp; k++)
        mbar_wait_bounded(&s.full[warp][k % kAtStages], (k / kAtStages) & 1u, a.wait_ns);
  }
  __syncthreads();

  // -------------------------------------------------------------------- join
  // A row for 16 lanes at a time, D / 16 elements a lane.
  constexpr int N = D / 16;
  const int hl = lane & 15;
  using Row = AtRow<N>;
  const long long y0 = start(blockIdx.x * kAtWarps), y1 = start((blockIdx.x + 1) * kAtWarps);   // the CTA's range
  // The parts of one item lie side by side, in the order of the context.  Lane q
  // looks at part q: one that is of another item than the last part before it
  // begins a run, and its lane works out what the run is.
  const AtSeg &sg = s.seg[(lane >> 1) & (kAtWarps - 1)][lane & 1];
  const long long item0 = lane < 2 * kAtWarps ? sg.item0 : -1;
  const unsigned valid = __ballot_sync(kFull, item0 >= 0), below = valid & ((1u << lane) - 1u);
  const long long prev0 = __shfl_sync(kFull, item0, below ? 31 - __clz(below) : 0);
  const bool lead = item0 >= 0 && (!below || prev0 != item0);
  const unsigned begins = __ballot_sync(kFull, lead);
  // rows of the run's item; whether other CTAs hold parts of it too (the first and the last item of the range, if
  // they start or end outside), and which: slot 0 is that of the item that the range begins with
  int rows = 0, c0 = 0, c1 = 0;                    // c0, c1: the CTAs that hold the item's first and last chunk
  bool out = false;
  if (lead) {
    rows = (int)min((long long)kAtRows, (long long)s.t.n[sg.at.b] * a.group - sg.at.rt * kAtRows);
    const long long end = item0 + sg.at.nch - 1;
    out = item0 < y0 || end >= y1;
    c0 = item0 >= y0 ? (int)blockIdx.x : cta_of(item0);
    c1 = end < y1 ? (int)blockIdx.x : cta_of(end);
  }
  const int which = item0 > y0;
  int incl = rows;
#pragma unroll
  for (int w = 1; w < 2 * kAtWarps; w <<= 1) {
    const int u = __shfl_up_sync(kFull, incl, w);
    if (lane >= w) incl += u;
  }
  const int units = __shfl_sync(kFull, incl, 2 * kAtWarps - 1);
  for (int ub = 2 * warp; ub < units; ub += 2 * kAtWarps) {
    const unsigned m0 = __ballot_sync(kFull, lead && ub < incl), m1 = __ballot_sync(kFull, lead && ub + 1 < incl);
    const bool real = lane < 16 || m1;             // the odd row of the last pair may be missing
    const int u = ub + (real ? lane >> 4 : 0), q0 = __ffs(lane >= 16 && m1 ? m1 : m0) - 1;
    const unsigned rest = begins & ~((2u << q0) - 1u);
    const int q1 = rest ? __ffs(rest) - 1 : 2 * kAtWarps, r = u - __shfl_sync(kFull, incl - rows, q0);
    const int w = __shfl_sync(kFull, which, q0), o = __shfl_sync(kFull, (int)out, q0);
    Row row;
    row.clear();
    for (int q = q0; q < q1; q += 4) {             // four at a time; past the run: no part
      float2 st[4];
      float4 v[4][N / 4];
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const int z = min(q + e, 2 * kAtWarps - 1);
        st[e] = q + e < q1 ? s.stat[z >> 1][z & 1][r] : make_float2(-INFINITY, kAtNoPart);
        const float4 *src = reinterpret_cast<const float4 *>(part_of(z >> 1, z & 1) + r * kLd + N * hl);
#pragma unroll
        for (int k = 0; k < N / 4; k++) v[e][k] = src[k];
      }
      row.add(st, v, c);
    }
    if (!real) continue;
    if (o) at_keep<D>(p, 2 * blockIdx.x + w, r, hl, row);
    else at_emit<N, F16>(p, AtItem(s.t, a, s.seg[q0 >> 1][q0 & 1].at), r, hl, row);
  }
  const unsigned outs = __ballot_sync(kFull, out);
  if (!outs) return;
  __syncthreads();
  if (warp == 0 && out) s.last[which] = at_ticket(p, c0, c1 - c0 + 1);
  __syncthreads();
  for (unsigned left = outs; left; left &= left - 1) {
    const int q0 = __ffs(left) - 1, w = __shfl_sync(kFull, which, q0);
    if (!s.last[w]) continue;
    const AtItem it(s.t, a, s.seg[q0 >> 1][q0 & 1].at);
    const int f = __shfl_sync(kFull, c0, q0), e = __shfl_sync(kFull, c1, q0);
    // CTA f's part is its last one, unless its range begins with the item; the others' is their first
    const int slot0 = 2 * f + (__shfl_sync(kFull, item0, q0) > start(f * kAtWarps));
    const int r = 2 * warp + (lane >> 4);          // all the rows at once
    if (r < it.rows) {
      Row row;
      row.clear();
      at_gather<D>(p, f, e, slot0, r, hl, c, row);
      at_emit<N, F16>(p, it, r, hl, row);
    }
  }
}

namespace {
typedef void (*AtKernel)(const AtArgs);
AtKernel at_kernel(int head_dim, int f16, bool many) {
  if (many) {
    if (head_dim == 64) return f16 ? attn_many_kernel<64, true> : attn_many_kernel<64, false>;
    return f16 ? attn_many_kernel<128, true> : attn_many_kernel<128, false>;
  }
  if (head_dim == 64) return f16 ? attn_few_kernel<64, true> : attn_few_kernel<64, false>;
  return f16 ? attn_few_kernel<128, true> : attn_few_kernel<128, false>;
}
int at_smem(int head_dim) { return head_dim == 64 ? AtGeom<64>::kSmem : AtGeom<128>::kSmem; }
}  // namespace

cudaError_t attn_tree_setup(int head_dim, int f16) {
  for (int many = 0; many < 2; many++) {
    const cudaError_t err = cudaFuncSetAttribute(at_kernel(head_dim, f16, many != 0), cudaFuncAttributeMaxDynamicSharedMemorySize,
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
  w.stat = take(8 * (size_t)(2 * num_sms) * kAtRows);
  w.part = take(4 * (size_t)(2 * num_sms) * kAtRows * head_dim);
  w.wide = attn_wide_ws(off, head_dim, num_sms);
  w.total = w.wide.total;
  return w;
}

cudaError_t launch_attn_tree(const AttnArgs &a, uint8_t *ws, int num_sms, cudaStream_t stream) {
  const AttnTreeWs w = attn_tree_ws(a.head_dim, num_sms);
  const long long rows = ((long long)a.T * a.group + a.B - 1) / a.B;   // of a request and kv head, on the average
  const long long items = (long long)a.B * a.kv_heads * ((rows + kAtRows - 1) / kAtRows);
  const long long most = ((long long)a.max_pages << a.page_shift) * a.head_dim / 2048;   // chunks of a context
  if (rows > kAtMostRows && items * most > (long long)kAtMostChunks * kAtWarps * num_sms)
    return launch_attn_wide_tree(a, ws, w.wide, num_sms, stream);
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
  const bool many = items > num_sms;
  at_kernel(a.head_dim, a.f16, many)<<<num_sms, kAtThreads, at_smem(a.head_dim), stream>>>(p);
  return cudaGetLastError();
}

}  // namespace moe
