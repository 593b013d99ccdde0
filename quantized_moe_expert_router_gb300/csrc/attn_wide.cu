// attn_wide.cu -- attention on the 5th-generation tensor cores: causal over
// whole packed prompts (moe_attn_prompt), and over the paged cache when a
// request brings many query rows (moe_attn_tree; attn_tree.cu has the other
// calls).
//
// The G query heads of a kv head are rows of one matrix (row = token * G + head of
// the group), so a key tile serves all of them and short prompts fill the 128-row
// tensor-core tiles: a row tile is floor(128 / G) whole tokens.  An item is
// (request, kv head, two row tiles): they share every key/value tile of 128 tokens.  With c =
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
//   warp 0          key/value tiles by tensor-map copies (128-byte swizzle)
//                   into a ring of stages: the key tile that S needs next with the
//                   value tile that PV needs; takes the items
//   warp 1          MMA issue: S of the next tile follows PV of this one, so one
//                   row tile's softmax runs while the other's MMAs do.  The tensor
//                   pipe's queue covers some 250 cycles of the issuer's way from
//                   one operation to the next, hence one stage, one barrier and
//                   few commits a tile (and not an issuer per row tile: their
//                   MMAs mix, and each change of accumulator costs)
//   warps 2-3       the scan below; warp 2 also Q rows by tensor-map boxes (64, G, tokens)
//   warps 4-7, 8-11 softmax of row tile 0 and 1: a thread owns a row, so the
//                   maximum and the sum need no exchange between threads;
//                   also the rare rescaling of O and the epilogue
// Tensor memory: S0, S1 (128 columns each, P over their first 64), O0, O1.
//
// A tile past the last token that all rows see holds keys that some rows, or
// all, may not see.  Their scores are replaced by -infinity, so P is 0; but 0
// times an infinite or NaN v is NaN, so warps 2-3 scan those tiles' v, zero
// such elements and note their tokens, and the epilogue adds them to the
// rows that do see the token.
//
// A wait knows its phase by parity alone, so no barrier may be two phases on when
// a waiter looks (it would wait for the next phase of that parity, or for ever).
// What keeps each from it:
//   sched_full    (item parity) item i + 2 is posted when sched_empty has all 11 arrivals
//                 of item i, each after that warp's last use of the item
//   kv_full       the stage is filled again after kv_empty, which the MMA warp commits
//                 after its own wait, and behind v_clean, which both helper warps
//                 give after theirs; v_posted says that the phase before is over
//   kv_empty      the copy warp waits before each filling; no lane copies before all
//                 lanes have passed
//   q_full        filled again by warp 2 behind q_empty, behind the MMA warp's wait
//   q_empty       waited for by warp 2 alone, whose lanes meet before the next Q is
//                 copied, and without that Q there is no next commit
//   v_posted, v_clean   (item parity) used again two items on, behind sched_empty
//   s_full, p_full, o_done   S, P and O of a row tile go to and fro between the MMA
//                 warp and the four softmax warps, which all arrive on p_full
// (tests/attn_barriers.py runs these roles with any one of them held back.)
//
// Prompts: items are taken from a counter, those with most key tiles first; an
// item's length depends on its row tile alone, so with the requests ranked by
// length the idx-th longest item has a closed form (prompt_item).
// Few prompts: items are single row tiles, and the two row tiles are the same rows
// over alternate key tiles (twins), joined through shared memory.
// Cache: the key tiles of all items stand in one line that the CTAs share
// (at_share).  A part of an item goes to the workspace (fp32 O, m, l) and
// attn_join_kernel joins the parts in the order of the context.  Parts of at most
// 128 rows are twins too, so that the softmax of one still runs beside the MMAs of
// the other.
//
// Bound, D = 128: the tensor pipe.  S and PV of a row tile and key tile take it 1025
// cycles when nothing else runs; beside the copies that write the same shared memory
// some 1250, and 100 to 150 pass until the next product's P is seen.  16384 tokens (2
// kv heads of 8): 630 us, 1745 TFLOP/s, where a library product has 1900; 4 x 4096 (4
// of 8): 350 us, 1570; 512 (8 of 4): 11.9 us, a chain of launch (2 us), items and first
// copies (3), two key tiles a twin (5) and the store.  D = 64: one product behind the other; the pipe takes 525 cycles, the
// exponentials 512 and the way from P to the next S the rest of 1140: 8192 tokens (4
// of 8) 259 us, 1060 TFLOP/s; 17 prompts of 62 to 1501 (8 of 3) 44 us.  A third S
// buffer with S three products ahead measured the same (267, 48).  Over the cache,
// 4 requests of 16 to 64 rows at 1125 to 9000 (4 of 8): 27 us: launch 2, lengths, shares and
// first copies 5.4, 6 key tiles a CTA 8.4 (2870 cycles for the 2050 of two row tiles, while
// the CTAs copy 64 KB each: 7.2 TB/s from L2), the part's store 2.5, the join 6.
#include <math.h>
#include <string.h>

#include "attn_tc.cuh"

namespace moe {

constexpr int kApThreads = 384;
constexpr int kApRows = 256, kApTile = 128;      // rows of an item; rows of a row tile, tokens of a key tile
constexpr int kApRegsSoft = 208, kApRegsRest = 88;
constexpr int kApWTma = 0, kApWMma = 1, kApWHelp = 2, kApWSoft = 4;
constexpr int kApMaxB = MOE_ATTN_MAX_REQUESTS;
constexpr int kApMaxSms = 1024;                  // CTAs of the wide kernel at most
constexpr float kApSlack = 8.f;                  // log2 of the largest P
constexpr int kApMinTiles = 2;                   // key tiles of a CTA at least (cache); us with 2, 6, 10: 512 rows at 9000 30.3, 30.3,
                                                 // 32.9; 64 rows of 2 requests at 4000 19.6, 20.2, 21.7

template <int D>
struct ApGeom {
  static constexpr int kTileBytes = kApTile * D * 2;
  static constexpr int kQTile = kTileBytes;
  static constexpr int kStages = D == 128 ? 2 : 4; // of a key and a value tile
  static constexpr int kSmem = 2 * kTileBytes + kStages * 2 * kTileBytes + 1024;
};
// Latent attention, expanded: keys of 192 elements, of which the heads share the last 64, and values of 128.  Two
// stages of 80 KB do not fit beside the 96 KB of Q, so the ring is of pieces, 128 tokens x 64 elements each: the value
// tile's two, then the three of the key tile that S needs next.  A slot is free when its piece has been read for the last
// time, so of the five pieces that a row tile's two products read, two of the next are there before and
// three come while the other row tile's products run.  A tile's pieces share a barrier (kv_full, four in turn):
// beside the products, which read shared memory all the time, each look at one costs 100 to 200 cycles.  8192 tokens of
// 32 heads 458 us, 1500 TFLOP/s (568 with a barrier a piece; for seconds on end 496, at the 1.9 GHz of the power cap).  A step, two
// row tiles and a key tile, is 2560 cycles of the tensor pipe and 2660 of shared memory (S reads 8 KB in 64 cycles, and the
// copies), and takes 3900 by clock reads: the issuing warp spends 2670 in the issue of its products, with that behind it, waits
// 440 for values, P and keys, and is 800 between those, where the pipe can run dry.
constexpr int kApPiece = kApTile * 128;
struct ApLatGeom {
  static constexpr int kTileBytes = 2 * kApPiece;
  static constexpr int kQTile = 3 * kApPiece;
  static constexpr int kStages = 7;                // pieces
  static constexpr int kSmem = 2 * kQTile + kStages * kApPiece + 1024;
};
template <int D, bool LAT>
struct ApGeomOf { using type = ApGeom<D>; };
template <int D>
struct ApGeomOf<D, true> { using type = ApLatGeom; };

struct ApArgs {
  CUtensorMap kmap, vmap;      // prompt: (64, 1, 128) boxes over [rows][kv_heads][D]; cache: (64, page, 1, 1) over
                               // [pages][kv_heads][page][D]; 128-byte swizzle
  CUtensorMap qmap;            // (64, group, per) boxes over [rows][q_heads][D]
  CUtensorMap rmap;            // latent: (64, 1, 128) boxes over [rows][1][64], the key part that the heads share
  AttnArgs a;
  int *ctrl;                   // workspace control words
  int magic;                   // ceil(2^16 / group)
  int per;                     // tokens of a row tile: floor(128 / group)
  int span;                    // prompts: tokens of an item, per (twins) or 2 * per
  // cache only
  int4 *desc;                  // per CTA, of the item whose first part it holds and others the rest:
                               // (first, hk, tok0, toks), (first CTA, last CTA, its slot, twin)
  float4 *part;                // [2 * grid][D / 4][256]  O of a part
  float2 *stat;                // [2 * grid][256]         (m, l)
};

struct ApItem {
  int b, hk;                   // request (-1: no more items), kv head
  int first;                   // the request's first packed row
  int tok0, toks;              // the item's tokens, among the request's fresh ones
  int j0, n;                   // first key tile and number of key tiles
  int n0, n1;                  // key tiles of the two row tiles
  int cached;                  // context before the fresh tokens
  int all, end;                // tokens that every row sees; tokens from `end` on are seen by none
  int m0;                      // tiles j0 + m0 .. are masked
  int twin;                    // the second row tile is the first one, over the odd tiles
  int slot;                    // where the part goes; -1: the item is whole
};

// What finds the items.  Prompts: requests by falling length.
template <bool PAGED>
struct ApSched {
  uint16_t order[kApMaxB];
  int tiles[kApMaxB];          // items per kv head of the k-th longest
  int before[kApMaxB + 1];     // items (per kv head) of row tiles in which fewer than k + 1 requests take part
};
// Cache: the line of key tiles.
template <>
struct ApSched<true> {
  long long work[kApMaxB + 1]; // tiles of the requests before
  int first[kApMaxB], n[kApMaxB], cached[kApMaxB];   // first packed row, fresh rows, cached tokens
  int cand[kApThreads / 32][32];
};

template <bool PAGED>
struct ApSmem : ApSched<PAGED> {
  uint64_t kv_full[7], kv_empty[7];
  uint64_t q_full, q_empty, s_full[2], p_full[2], o_done[2], v_posted[2][3], v_clean[2][3], x_full[2], sched_full[2], sched_empty[2], drain;
  uint32_t tmem;
  int wsum[kApThreads / 32];
  ApItem item[2];
  int v_pos[2][3], v_tile[2][3];   // by item parity: stages of the masked value tiles, counted from the CTA's start; latent:
                               // their first pieces, and their places among the tiles
  float2 stat[2][kApTile];     // (m, l) of the twins of a prompt
  uint32_t bad[2][2][3][4];    // by item parity, scanning warp and masked tile: tokens with a non-finite v
  long long wsum2[kApThreads / 32];
};

// Of a request of n fresh rows over the cache: items of a kv head, and key
// tiles that its rows may see.
__device__ __forceinline__ int cache_tiles(const ApArgs &p, int n) { return at_idiv(n + 2 * p.per - 1, 2 * p.per); }
__device__ __forceinline__ int cache_nch(const AttnArgs &a, int n, int cached) {
  const int ctx = min(cached + (a.tree_mask ? min(n, MOE_ATTN_MAX_TREE) : n), a.max_pages << a.page_shift);
  return (ctx + kApTile - 1) / kApTile;
}

// The idx-th item by falling row tile: row tiles [tiles[k], tiles[k - 1]) have
// the k longest requests.
__device__ __forceinline__ void prompt_item(const ApSmem<false> &s, const ApArgs &p, int idx, ApItem &it) {
  const AttnArgs &a = p.a;
  const int e = at_idiv(idx, a.kv_heads);
  it.hk = idx - e * a.kv_heads;
  int lo = 0, hi = a.B - 1;                        // largest k with before[k] <= e
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.before[mid] <= e) lo = mid; else hi = mid - 1;
  }
  const int k = lo + 1, off = e - s.before[lo];
  const int lvl = at_idiv(off, k);
  it.tok0 = (s.tiles[lo] - 1 - lvl) * p.span;
  it.b = s.order[off - lvl * k];
  it.first = __ldg(a.cu + it.b);
  it.toks = min(min(__ldg(a.cu + it.b + 1), a.T) - it.first - it.tok0, p.span);
  it.n = (it.tok0 + it.toks - 1) / kApTile + 1;
  it.twin = p.span == p.per;
  it.n0 = it.twin ? (it.n + 1) >> 1 : (it.tok0 + min(it.toks, p.per) - 1) / kApTile + 1;
  it.n1 = it.twin ? it.n >> 1 : (it.toks > p.per ? it.n : 0);
  it.j0 = it.cached = 0;
  it.all = it.tok0 + 1;
  it.end = it.tok0 + it.toks;                      // the causal limit alone cuts
  it.m0 = it.all / kApTile;
  it.slot = -1;
}

// The part of an item that starts at place x of the line of key tiles, up to
// the end of the CTA's share; returns the place after it.  n = 0: the rows need
// nothing of it (later tokens than theirs).
__device__ __forceinline__ long long cache_part(const ApSmem<true> &s, const ApArgs &p, long long x, const AtShare &share, ApItem &it) {
  const AttnArgs &a = p.a;
  int lo = 0, hi = a.B - 1;                        // largest b with work[b] <= x
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.work[mid] <= x) lo = mid; else hi = mid - 1;
  }
  it.b = lo;
  it.first = s.first[lo];
  it.cached = s.cached[lo];
  const int n = s.n[lo], tiles = cache_tiles(p, n), nch = cache_nch(a, n, it.cached);
  const int item = (int)at_div(x - s.work[lo], nch);
  const long long item0 = s.work[lo] + (long long)item * nch, xe = min(share.x1, item0 + nch);
  it.hk = at_idiv(item, tiles);
  it.tok0 = (item - it.hk * tiles) * 2 * p.per;
  it.toks = min(n - it.tok0, 2 * p.per);
  const int lim = min(a.max_pages << a.page_shift, it.cached + n);
  it.all = a.tree_mask ? it.cached : it.cached + it.tok0 + 1;
  it.end = min(lim, it.cached + (a.tree_mask ? min(n, MOE_ATTN_MAX_TREE) : it.tok0 + it.toks));
  const int need = (it.end + kApTile - 1) / kApTile;                          // key tiles of this row tile
  it.j0 = (int)(x - item0);
  it.n = max(0, min((int)(xe - item0), need) - it.j0);
  const bool whole = it.j0 == 0 && it.n == need;
  it.twin = !whole && it.toks <= p.per;
  it.slot = whole ? -1 : 2 * (int)blockIdx.x + (x > share.x0);
  it.n0 = it.twin ? (it.n + 1) >> 1 : it.n;
  it.n1 = it.twin ? it.n >> 1 : (it.toks > p.per ? it.n : 0);
  it.m0 = max(0, it.all / kApTile - it.j0);
  if (!whole && it.j0 == 0) {
    // for the join, at the CTA that holds the first part: the last part of a
    // CTA's share, so that there is one at most
    int c0, c1;
    share.ctas_of(item0, item0 + need - 1, c0, c1);
    if (share.len) c1 = c0 + (need - 1) / share.len;
    if ((threadIdx.x & 31) == 0) {
      int4 *d = p.desc + 2 * blockIdx.x;
      d[0] = make_int4(it.first, it.hk, it.tok0, it.toks);
      d[1] = make_int4(c0, c1, it.slot, it.twin);
    }
  }
  return xe;
}

// Bits of the tokens base .. base + 31 (word w of the tile) that a row sees.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u); }
template <bool PAGED>
__device__ __forceinline__ uint32_t visible_bits(const AttnArgs &a, const ApItem &it, uint64_t word, int lim, int base,
                                                 uint32_t held, int w) {
  if constexpr (!PAGED) return low_bits(lim + 1 - base);
  uint32_t bits;
  if (a.tree_mask) {
    const int f0 = base - it.cached;               // fresh row of the first bit
    const uint32_t fresh = f0 >= 64 || f0 <= -32 ? 0u : (f0 >= 0 ? (uint32_t)(word >> f0) : (uint32_t)(word << -f0));
    bits = low_bits(-f0) | fresh;
  } else {
    bits = low_bits(it.cached + lim + 1 - base);
  }
  bits &= low_bits(it.end - base);
  const uint32_t pages = a.page_shift == 4 ? ((held >> (2 * w)) & 1u ? 0xFFFFu : 0u) | ((held >> (2 * w)) & 2u ? 0xFFFF0000u : 0u)
                                           : ((held >> ((32 * w) >> a.page_shift)) & 1u ? ~0u : 0u);
  return bits & pages;
}

// exp2(c v + mc) of 32 scores: P as 16 packed words, and its sum added to acc.
template <bool F16>
__device__ __forceinline__ void ap_weights(const float *v, float2 c2, float2 mc2, uint32_t *pk, float2 (&acc)[2]) {
#pragma unroll
  for (int e = 0; e < 16; e++) {
    float2 t = ffma2(make_float2(v[2 * e], v[2 * e + 1]), c2, mc2);
    t.x = at_exp2(t.x);
    t.y = at_exp2(t.y);
    acc[e & 1] = at_add2(acc[e & 1], t);
    pk[e] = at_pack<F16>(t.x, t.y);
  }
}
__device__ __forceinline__ float ap_max(const float (&v)[128]) {
  float mx[4];
#pragma unroll
  for (int q = 0; q < 4; q++) {
    mx[q] = fmaxf(v[32 * q], v[32 * q + 1]);
#pragma unroll
    for (int e = 2; e < 32; e += 2) mx[q] = at_max3(mx[q], v[32 * q + e], v[32 * q + e + 1]);
  }
  return at_max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
}

// TWINS: prompts whose items are one row tile each, over alternate key tiles.  LAT: keys of 192 elements (D = 128).
template <int D, bool F16, bool PAGED, bool TWINS, bool LAT>
__global__ void __launch_bounds__(kApThreads, 1) attn_wide_kernel(const __grid_constant__ ApArgs p) {
  extern __shared__ uint8_t dsm[];
  __shared__ ApSmem<PAGED> s;
  using G = typename ApGeomOf<D, LAT>::type;
  constexpr int kStages = G::kStages, kTB = G::kTileBytes, kQT = G::kQTile, kHalves = D / 64, kQHalves = LAT ? 3 : kHalves;
  const AttnArgs &a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t smem0 = (smem_u32(dsm) + 1023u) & ~1023u;
  const uint32_t q_smem = smem0, ring = smem0 + 2 * kQT;
  uint8_t *const generic0 = dsm + (smem0 - smem_u32(dsm));

  // the first lengths: on their way while the barriers are set up
  int lo0 = 0, hi0 = 0;
  if (!PAGED && !LAT && tid < a.B) {
    lo0 = __ldg(a.cu + tid);
    hi0 = __ldg(a.cu + tid + 1);
  }
  if (warp == 0) {
    // a barrier a lane: one lane would take some 25 cycles for each of them
    if (lane < kStages) {
      mbar_init(&s.kv_full[lane], 1);
      mbar_init(&s.kv_empty[lane], 1);
    }
    if (lane < 2) {
      mbar_init(&s.s_full[lane], 1);
      mbar_init(&s.p_full[lane], 4);
      mbar_init(&s.o_done[lane], 1);
      mbar_init(&s.sched_full[lane], 1);
      mbar_init(&s.sched_empty[lane], 11);         // 8 softmax warps, MMA warp, 2 helper warps
    } else if (lane < 5) {
      mbar_init(&s.v_posted[0][lane - 2], 1);
      mbar_init(&s.v_posted[1][lane - 2], 1);
      mbar_init(&s.v_clean[0][lane - 2], 2);       // both helper warps
      mbar_init(&s.v_clean[1][lane - 2], 2);
    } else if (lane == 5) {
      mbar_init(&s.q_full, 1);
      mbar_init(&s.q_empty, 1);
      mbar_init(&s.x_full[0], 4);
      mbar_init(&s.x_full[1], 4);
      mbar_init(&s.drain, 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid == 32 * kApWHelp) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.kmap)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.vmap)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.qmap)) : "memory");
    if (LAT) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.rmap)) : "memory");
  }
  if (warp == kApWMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s.tmem)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if constexpr (LAT) pdl_wait();                   // the kernel before is done: what follows reads its results
  long long total = 0;                             // prompt: items; cache: key tiles
  AtShare share = {};
  if constexpr (PAGED) {
    int nitems = 0;
    for (int b0 = 0; b0 < a.B; b0 += kApThreads) {
      const int b = b0 + tid;
      int items = 0;
      long long v = 0;
      if (b < a.B) {
        const int lo = __ldg(a.cu + b), hi = __ldg(a.cu + b + 1);
        const int cached = min(max(__ldg(a.cached + b), 0), a.max_pages << a.page_shift);   // no sum with rows passes 2^31
        const int n = lo < 0 ? 0 : max(0, min(hi, a.T) - lo);
        s.first[b] = lo;
        s.n[b] = n;
        s.cached[b] = cached;
        items = cache_tiles(p, n) * a.kv_heads;
        v = (long long)items * cache_nch(a, n, cached);
      }
      long long incl = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += t;
      }
      items = __reduce_add_sync(kFull, items);
      if (lane == 31) {
        s.wsum2[warp] = incl;
        s.wsum[warp] = items;
      }
      __syncthreads();
      long long at = total;
#pragma unroll
      for (int w = 0; w < kApThreads / 32; w++) {
        at += w < warp ? s.wsum2[w] : 0;
        total += s.wsum2[w];
        nitems += s.wsum[w];
      }
      if (b < a.B) s.work[b] = at + incl - v;
      __syncthreads();
    }
    share = at_share<kApThreads / 32>(
        s.work, a.B, total, nitems, kApMinTiles, s.cand,
        [&](int b) { return cache_tiles(p, s.n[b]) * a.kv_heads; }, [&](int b) { return cache_nch(a, s.n[b], s.cached[b]); });
    if (tid == 0) p.desc[2 * blockIdx.x + 1] = make_int4(0, -1, 0, 0);   // nothing to join, unless cache_part finds it
  } else {
    // requests by falling number of row tiles (equal ones by index), every CTA alike
    for (int b = tid; b < a.B; b += kApThreads) {
      const bool there = !LAT && b == tid;
      const int lo = there ? lo0 : __ldg(a.cu + b), n = max(0, min(there ? hi0 : __ldg(a.cu + b + 1), a.T) - lo);
      s.before[b] = lo < 0 ? 0 : at_idiv(n + p.span - 1, p.span);
    }
    __syncthreads();
    for (int b = tid; b < a.B; b += kApThreads) {
      const int mine = s.before[b];
      int rank = 0;
      for (int o = 0; o < a.B; o++) rank += s.before[o] > mine || (s.before[o] == mine && o < b);
      s.order[rank] = (uint16_t)b;
      s.tiles[rank] = mine;
    }
    __syncthreads();
    int items = 0;                                   // per kv head
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
      if (lane == 31) s.wsum[warp] = incl;
      __syncthreads();
      int at = items;
#pragma unroll
      for (int w = 0; w < kApThreads / 32; w++) {
        at += w < warp ? s.wsum[w] : 0;
        items += s.wsum[w];
      }
      if (k < a.B) s.before[k] = at + incl;
      __syncthreads();
    }
    total = (long long)(items + a.B * s.tiles[a.B - 1]) * a.kv_heads;   // row tiles that every request has come last
  }
  at_fence_before();
  __syncthreads();
  at_fence_after();
  const uint32_t tb = s.tmem;
  const float c = a.scale * 1.44269504088896340736f;
  if constexpr (PAGED) pdl_launch_dependents();    // the join's CTAs take the SMs as they fall free, and wait

  if (warp >= kApWSoft) {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kApRegsSoft));
    const int h = (warp - kApWSoft) >> 2;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t ts = tb + lanes + 128u * h, to = tb + lanes + 256u + 128u * h;
    uint32_t ns = 0, ni = 0;                       // key tiles of this row tile, and items with any, so far
    bool ok = true;
    for (int i = 0;; i++) {
      if (!at_wait(&s.sched_full[i & 1], (uint32_t)(i >> 1) & 1u, a, p.ctrl)) break;
      const ApItem it = s.item[i & 1];
      if (it.b < 0) break;
      const int nt = h ? it.n1 : it.n0;
      const int r = tid & 127, dt = (r * p.magic) >> 16;                        // row of the row tile, its token there
      const bool twin = PAGED ? it.twin : TWINS;
      const int tl = (twin ? 0 : h * p.per) + dt;                               // token of the item
      const bool real = dt < p.per && tl < it.toks;
      const int lim = it.tok0 + min(tl, it.toks - 1);   // the row's token: of the prompt, or among the fresh ones
      uint64_t word = 0;
      if constexpr (PAGED)
        if (a.tree_mask) word = __ldg(a.tree_mask + it.first + lim);
      float m = -INFINITY;                         // the maximum that P is taken against
      bool far = false;                            // a row of the warp takes m off its scores before it scales them
      float2 l2 = make_float2(0.f, 0.f);
      for (int j = 0; j < nt; j++, ns++) {
        const int jl = twin ? 2 * j + h : j, tok0 = (it.j0 + jl) * kApTile;
        bool masked;
        uint32_t held = 0;                         // pages of the tile that are in the cache
        if constexpr (PAGED) {
          const int np = kApTile >> a.page_shift, col = (tok0 >> a.page_shift) + lane;
          const int id = lane < np && col < a.max_pages ? __ldg(a.block_table + (size_t)it.b * a.max_pages + col) : -1;
          held = __ballot_sync(kFull, (unsigned)id < (unsigned)a.num_pages);
          masked = jl >= it.m0 || held != (1u << np) - 1u;
        } else {
          masked = __any_sync(kFull, tok0 + kApTile - 1 > lim);
        }
        ok = at_wait(&s.s_full[h], ns & 1u, a, p.ctrl);
        if (!ok) break;
        at_fence_after();
        float v[128];
#pragma unroll
        for (int q = 0; q < 4; q++) at_ld32(ts + 32u * q, v + 32 * q);
        at_wait_ld(v);
        if (masked) {
#pragma unroll
          for (int w = 0; w < 4; w++) {
            const uint32_t bits = visible_bits<PAGED>(a, it, word, lim, tok0 + 32 * w, held, w);
            if (__any_sync(kFull, bits != ~0u)) {
#pragma unroll
              for (int e = 0; e < 32; e++) v[32 * w + e] = (bits >> e) & 1u ? v[32 * w + e] : -INFINITY;
            }
          }
        }
        const float top = ap_max(v);
        float ref = m;                             // what c takes off the scores with them
        if (j == 0 || far || __any_sync(kFull, (top - m) * c > kApSlack)) {
          if (j == 0) {
            m = real ? top : INFINITY;             // rows of no token hold anything: P = 0, and no say in the vote
          } else {
            const float m1 = fmaxf(m, top), f = m1 == -INFINITY ? 1.f : at_exp2((m - m1) * c);
            m = m1;
            l2.x *= f;
            l2.y *= f;
            // PV of the tile before is done: S of this one was issued behind it
#pragma unroll 1
            for (int q = 0; q < D / 32; q++) {
              float o[32];
              at_ld32(to + 32u * q, o);
              at_wait_ld(o);
#pragma unroll
              for (int e = 0; e < 32; e++) o[e] *= f;
              at_st32(to + 32u * q, o);
            }
            at_wait_st();
          }
          ref = m;
          far = __any_sync(kFull, at_far(m, c));
          if (far) {
            const float own = at_far(m, c) ? -m : 0.f;
            const float2 off = make_float2(own, own);
#pragma unroll
            for (int e = 0; e < 64; e++) {
              const float2 t = at_add2(make_float2(v[2 * e], v[2 * e + 1]), off);
              v[2 * e] = t.x;
              v[2 * e + 1] = t.y;
            }
            if (own != 0.f) ref = 0.f;
          }
        }
        const float mc = ref == -INFINITY ? 0.f : -ref * c;
        const float2 c2 = make_float2(c, c), mc2 = make_float2(mc, mc);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int q = 0; q < 4; q++) {
          uint32_t pk[16];
          ap_weights<F16>(v + 32 * q, c2, mc2, pk, sum);
          at_st16(ts + 16u * q, pk);
        }
        l2 = at_add2(l2, at_add2(sum[0], sum[1]));
        at_wait_st();
        at_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.p_full[h]);
      }
      if (!ok) break;
      float l = l2.x + l2.y;
      if (PAGED && it.slot >= 0) p.stat[(size_t)it.slot * kApRows + (kApTile * h + (tid & 127))] = make_float2(m, nt > 0 ? l : kAtNoPart);
      if (nt > 0) {
        // ---------------------------------------------------------- epilogue
        if (!at_wait(&s.o_done[h], ni++ & 1u, a, p.ctrl)) break;
        at_fence_after();
        // words of the masked tiles that this row tile's PV waited for: the others may be of an
        // earlier item, or not complete yet
        const int wend = 4 * ((twin ? it.n : nt) - it.m0);
        uint32_t anybad = 0;
#pragma unroll
        for (int w = 0; w < 12; w++)
          if (w < wend && !(twin && ((it.m0 + (w >> 2)) & 1) != h)) anybad |= s.bad[i & 1][0][w >> 2][w & 3] | s.bad[i & 1][1][w >> 2][w & 3];
        if (anybad) {
#pragma unroll 1
          for (int q = 0; q < D / 32; q++) {
            float o[32];
            at_ld32(to + 32u * q, o);
            at_wait_ld(o);
            for (int w = 0; w < wend; w++) {
              uint32_t bits = s.bad[i & 1][0][w >> 2][w & 3] | s.bad[i & 1][1][w >> 2][w & 3];
              for (; bits; bits &= bits - 1) {
                const int jl = it.m0 + (w >> 2);   // tile of the part
                if (twin && (jl & 1) != h) continue;
                const int tok = (it.j0 + jl) * kApTile + 32 * (w & 3) + __ffs(bits) - 1;
                const uint16_t *vp;
                if constexpr (PAGED) {
                  const int f = tok - it.cached;
                  if (tok >= it.end || !(a.tree_mask ? f < 64 && ((word >> (f & 63)) & 1) : f <= lim)) continue;
                  const long long page = __ldg(a.block_table + (size_t)it.b * a.max_pages + (tok >> a.page_shift));
                  vp = a.v_cache + (((page * a.kv_heads + it.hk) << a.page_shift) + (tok & ((1 << a.page_shift) - 1))) * D + 32 * q;
                } else {
                  if (tok > lim) continue;
                  vp = a.v.p + (long long)(it.first + tok) * a.v.row + (long long)it.hk * a.v.head + 32 * q;
                }
#pragma unroll
                for (int e = 0; e < 32; e++) {
                  const float u = at_value<F16>(__ldg(vp + e));
                  if (!isfinite(u)) o[e] += u;
                }
              }
            }
            __syncwarp();
            at_st32(to + 32u * q, o);
          }
          at_wait_st();
        }
        const bool halves = TWINS && it.n1 > 0;
        if (halves) {
          // Each twin gives the other the O of half of the columns, through shared memory
          // in the place of Q: a CTA has one item then, and its S are done.
          constexpr int kHalf = D / 2;
          float4 *const x = reinterpret_cast<float4 *>(generic0) + (tid & 127);   // [giver][element / 4 of the half][row]
          s.stat[h][tid & 127] = make_float2(m, l);
#pragma unroll 1
          for (int q = 0; q < kHalf / 32; q++) {
            float o[32];
            at_ld32(to + (uint32_t)(kHalf * (h ^ 1) + 32 * q), o);
            at_wait_ld(o);
#pragma unroll
            for (int e = 0; e < 8; e++)
              x[(kHalf / 4 * h + 8 * q + e) * kApTile] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.x_full[h]);
          if (!at_wait(&s.x_full[h ^ 1], 0u, a, p.ctrl)) break;
          const float2 other = s.stat[h ^ 1][tid & 127];
          const float top = fmaxf(m, other.x);
          const float f0 = m == top ? 1.f : at_exp2((m - top) * c), f1 = other.x == top ? 1.f : at_exp2((other.x - top) * c);
          m = top;
          l = h ? other.y * f1 + l * f0 : l * f0 + other.y * f1;
#pragma unroll 1
          for (int q = 0; q < kHalf / 32; q++) {
            float o[32];
            at_ld32(to + (uint32_t)(kHalf * h + 32 * q), o);
            at_wait_ld(o);
#pragma unroll
            for (int e = 0; e < 8; e++) {
              const float4 w = x[(kHalf / 4 * (h ^ 1) + 8 * q + e) * kApTile];
              o[4 * e] = o[4 * e] * f0 + w.x * f1;
              o[4 * e + 1] = o[4 * e + 1] * f0 + w.y * f1;
              o[4 * e + 2] = o[4 * e + 2] * f0 + w.z * f1;
              o[4 * e + 3] = o[4 * e + 3] * f0 + w.w * f1;
            }
            at_st32(to + (uint32_t)(kHalf * h + 32 * q), o);
          }
          at_wait_st();
        }
        if (PAGED && it.slot >= 0) {
          // [element / 4][row]: the 32 rows of a warp side by side
          float4 *part = p.part + (size_t)it.slot * (D / 4) * kApRows + (kApTile * h + (tid & 127));
#pragma unroll 1
          for (int q = 0; q < D / 32; q++) {
            float o[32];
            at_ld32(to + 32u * q, o);
            at_wait_ld(o);
#pragma unroll
            for (int e = 0; e < 8; e++)
              part[(8 * q + e) * kApRows] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        } else {
          const float inv = l == 0.f ? 0.f : 1.f / l;
          const int hq = it.hk * a.group + r - dt * a.group;
          if (a.lse && real && !(TWINS && h))
            a.lse[(size_t)(it.first + lim) * a.q_heads + hq] = l == 0.f ? -INFINITY : m * a.scale + logf(l);
          // A lane's row at a time would touch 32 lines a store; with the
          // fragment shape a quad holds 32 elements of a row (pairs 2 q4 of each
          // 8), and a transpose within the quad gives each lane 16 bytes of 64.
          const int qg = lane >> 2, q4 = lane & 3;
#pragma unroll 1
          for (int rb = 0; rb < 2; rb++) {
            float iv[2];
            uint16_t *dst[2];
            bool wr[2];
#pragma unroll
            for (int z = 0; z < 2; z++) {
              const int rl = 16 * rb + 8 * z + qg, rr = (r & ~31) + rl, dr = (rr * p.magic) >> 16;
              const int tr = tl - dt + dr;         // token of the item (not twins: they are parts)
              iv[z] = __shfl_sync(kFull, inv, rl);
              wr[z] = dr < p.per && tr < it.toks;
              dst[z] = a.out.p + (long long)(it.first + it.tok0 + tr) * a.out.row +
                       (long long)(it.hk * a.group + rr - dr * a.group) * a.out.head + 8 * q4;
            }
#pragma unroll
            for (int cz = 0; cz < D / 32; cz += 2) {   // blocks of 32 columns, two loads at a time; of twins their half
              const int blocks = halves ? D / 64 : D / 32, cb = (halves ? D / 64 * h : 0) + cz;
              if (cz >= blocks) break;
              float o[32];
              __syncwarp();                        // behind stores that some lanes leave out: the loads are the whole warp's
              at_ld_frag(to + ((uint32_t)(16 * rb) << 16) + 32u * cb, o);
              if (cz + 1 < blocks) at_ld_frag(to + ((uint32_t)(16 * rb) << 16) + 32u * (cb + 1), o + 16);
              at_wait_ld(o);
#pragma unroll
              for (int y = 0; y < 2; y++) {
                if (cz + y >= blocks) break;
#pragma unroll
                for (int z = 0; z < 2; z++) {
                  uint32_t w[4];
#pragma unroll
                  for (int e = 0; e < 4; e++)
                    w[e] = at_pack<F16>(o[16 * y + 4 * e + 2 * z] * iv[z], o[16 * y + 4 * e + 2 * z + 1] * iv[z]);
                  at_quad_transpose(w, q4);
                  if (wr[z]) *reinterpret_cast<uint4 *>(dst[z] + 32 * (cb + y)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
              }
            }
          }
        }
        at_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.sched_empty[i & 1]);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kApRegsRest));
    if (warp == kApWTma) {
      // ---------------------------------------------------------- items and key/value tiles
      // over the cache every lane copies a page of the tile; else lane 0 the whole tile
      if (PAGED || lane == 0) {
        int pos = 0, tiles = 0;                    // stages so far; latent: pieces, and tiles of keys and of values
        long long next = PAGED ? share.x0 : blockIdx.x;
        bool ok = true;
        // over the cache the warp waits as one; else lane 0 is alone
        auto wait = [&](uint64_t *bar, uint32_t parity) {
          if constexpr (PAGED) return at_wait(bar, parity, a, p.ctrl);
          const bool got = mbar_wait_bounded(bar, parity, a.wait_ns);
          if (!got) atomicOr(p.ctrl + kAttnCtrlFlags, MOE_FLAG_TIMEOUT);
          return got;
        };
        for (int i = 0; ok; i++) {
          ApItem it;
          it.b = -1;
          if constexpr (PAGED) {
            while (next < share.x1) {
              next = cache_part(s, p, next, share, it);
              if (it.n > 0) break;
              it.b = -1;
            }
          } else if (next < total) {
            prompt_item(s, p, (int)next, it);
          }
          if (i >= 2 && !wait(&s.sched_empty[i & 1], (uint32_t)((i >> 1) - 1) & 1u)) break;
          if (lane == 0) {
            s.item[i & 1] = it;
            mbar_arrive(&s.sched_full[i & 1]);
          }
          if (it.b < 0) break;
          if (TWINS) next = total;                 // a CTA an item
          else if (!PAGED) next = gridDim.x + atomicAdd(p.ctrl + kAttnCtrlNext, 1);
          // stage q: K[q] and V[q - ahead], as far as they are there
          const int n = it.n, ahead = (PAGED ? it.twin : TWINS) ? 2 : 1;
          if constexpr (LAT) {
            // pieces in the order of their use: V[q - ahead], K[q]
            auto take = [&](int z) {               // slot of piece pos + z, free
              const int at = pos + z;
              if (ok && at >= kStages) ok = wait(&s.kv_empty[at % kStages], (uint32_t)(at / kStages - 1) & 1u);
              return at % kStages;
            };
            for (int q = 0; q < n + ahead && ok; q++) {
              if (q >= ahead) {
                const int s0 = take(0), s1 = take(1), j = q - ahead, row = it.first + j * kApTile;
                if (!ok) break;
                uint64_t *bar = &s.kv_full[tiles & 3];
                mbar_arrive_expect_tx(bar, (uint32_t)(2 * kApPiece) + a.stall);
                if (j >= it.m0) {                  // the scan may wait for these pieces now, as below
                  s.v_pos[i & 1][j - it.m0] = pos;
                  s.v_tile[i & 1][j - it.m0] = tiles;
                  mbar_arrive(&s.v_posted[i & 1][j - it.m0]);
                }
                // elements 0 .. 63 lie in the lower slot
                at_tma_3d(ring + min(s0, s1) * kApPiece, &p.vmap, 0, it.hk, row, bar);
                at_tma_3d(ring + max(s0, s1) * kApPiece, &p.vmap, 64, it.hk, row, bar);
                pos += 2;
                tiles++;
              }
              if (q < n) {
                const int row = it.first + q * kApTile;
                uint64_t *bar = &s.kv_full[tiles & 3];
                int slot = take(0);                // behind it nothing waits for the barrier's last phase any more
                if (!ok) break;
                mbar_arrive_expect_tx(bar, (uint32_t)(3 * kApPiece) + a.stall);
                tiles++;
                for (int z = 0; z < 3; z++) {
                  if (z) slot = take(0);
                  if (!ok) break;
                  at_tma_3d(ring + slot * kApPiece, z == 2 ? &p.rmap : &p.kmap, z == 2 ? 0 : 64 * z, z == 2 ? 0 : it.hk, row, bar);
                  pos++;
                }
              }
            }
          } else for (int q = 0; q < n + ahead; q++) {
            if (q >= n && q < ahead) continue;
            const int slot = pos % kStages;
            int page[2] = {0, 0};
            if constexpr (PAGED) {
#pragma unroll
              for (int z = 0; z < 2; z++) {
                const int col = ((it.j0 + q - z * ahead) * kApTile >> a.page_shift) + lane;
                const bool here = (z ? q >= ahead : q < n) && lane < kApTile >> a.page_shift && col < a.max_pages;
                const int id = here ? __ldg(a.block_table + (size_t)it.b * a.max_pages + col) : -1;
                page[z] = (unsigned)id < (unsigned)a.num_pages ? id : a.num_pages;   // past the end: reads zeros
              }
            }
            if (pos >= kStages) ok = wait(&s.kv_empty[slot], (uint32_t)(pos / kStages - 1) & 1u);
            if (!ok) break;
            if (lane == 0) {
              mbar_arrive_expect_tx(&s.kv_full[slot], (uint32_t)(kTB * ((q < n) + (q >= ahead))) + a.stall);
              // the scan may wait for this stage now: before, the barrier may still
              // be in an earlier phase, which a wait cannot tell from this one
              if (q - ahead >= it.m0) {
                s.v_pos[i & 1][q - ahead - it.m0] = pos;
                mbar_arrive(&s.v_posted[i & 1][q - ahead - it.m0]);
              }
            }
            if constexpr (PAGED) __syncwarp();
#pragma unroll
            for (int z = 0; z < 2; z++) {
              if (!(z ? q >= ahead : q < n)) continue;
              const uint32_t dst = ring + (2 * slot + z) * kTB;
              for (int hf = 0; hf < kHalves; hf++) {
                if constexpr (PAGED) {
                  if (lane < kApTile >> a.page_shift)
                    at_tma_4d(dst + hf * (kApTile * 128) + ((uint32_t)lane << (a.page_shift + 7)), z ? &p.vmap : &p.kmap, 64 * hf, 0,
                              it.hk, page[z], &s.kv_full[slot]);
                } else {
                  at_tma_3d(dst + hf * (kApTile * 128), z ? &p.vmap : &p.kmap, 64 * hf, it.hk,
                            it.first + (it.j0 + q - z * ahead) * kApTile, &s.kv_full[slot]);
                }
              }
            }
            pos++;
          }
        }
        // copies in flight land before the CTA ends
        const int rounds = LAT ? tiles : pos, bars = LAT ? 4 : kStages;
        for (int q = (rounds > bars ? rounds - bars : 0); q < rounds; q++)
          mbar_wait_bounded(&s.kv_full[q % bars], (uint32_t)(q / bars) & 1u, a.wait_ns);
        if (!PAGED && !TWINS) {
          // the last CTA to have taken its last item leaves the counters at zero
          __threadfence();
          if (atomicAdd(p.ctrl + kAttnCtrlDone, 1) == (int)gridDim.x - 1) {
            p.ctrl[kAttnCtrlNext] = 0;
            p.ctrl[kAttnCtrlDone] = 0;
          }
        }
      }
      __syncwarp();
    } else if (warp == kApWMma) {
      // ---------------------------------------------------------- MMA issue
      // The whole warp goes through the loop, so that what the instructions take
      // (descriptors, tensor-memory columns) stays in uniform registers and costs
      // one addition; one elected lane issues.
      constexpr uint32_t id_s = at_idesc(F16, kApTile, false), id_o = at_idesc(F16, D, true);
      const uint32_t tu = __shfl_sync(kFull, tb, 0);
      const uint64_t dq0 = at_desc(q_smem, 16), dk0 = at_desc(ring, 16), dv0 = at_desc(ring + (LAT ? 0 : kTB), kApTile * 128);
      int slot = 0;                                // next stage and its phase
      uint32_t phase = 0, clean = 0, np0 = 0, np1 = 0;   // clean: a phase bit per item parity and masked tile
      bool ok = true;
      auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (ok && !mbar_wait_bounded(bar, parity, a.wait_ns)) {
          atomicOr(p.ctrl + kAttnCtrlFlags, MOE_FLAG_TIMEOUT);
          ok = false;
        }
      };
      // The lanes go on or end together.  With a wait that S or PV stands behind, the
      // vote comes after the issue: the lanes meet at the election anyway.
      auto all_ok = [&]() {
        ok = __all_sync(kFull, ok);
        return ok;
      };
      auto next_stage = [&]() {
        if (++slot == kStages) {
          slot = 0;
          phase ^= 1u;
        }
      };
      auto issue_s = [&](int h, int q) {           // S of row tile h = Q of row tile q K: by the elected lane
        const uint64_t da = dq0 + (uint64_t)(q * (kQT >> 4)), db = dk0 + (uint64_t)(slot * (2 * kTB >> 4));
#pragma unroll
        for (int k = 0; k < D / 16; k++) {
          const uint32_t off = (uint32_t)((k >> 2) * (kApTile * 128) + (k & 3) * 32) >> 4;
          at_mma_ss(tu + 128u * h, da + off, db + off, id_s, k > 0);
        }
        at_commit(&s.s_full[h]);
      };
      uint32_t pos = 0, tiles = 0;                 // latent: pieces and tiles so far
      auto wait_tile = [&](uint32_t t) { wait(&s.kv_full[t & 3u], (t >> 2) & 1u); };
      // Latent: S of row tile h from the pieces `at`, at + 1, at + 2, which are there; `last`: their last use.  By the elected lane.
      auto issue_s3 = [&](int h, int q, uint32_t at, bool last, bool q_last) {
        uint64_t da = dq0 + (uint64_t)(q * (kQT >> 4));
        uint32_t sl = at % kStages;
#pragma unroll 1
        for (int z = 0; z < 3; z++) {
          const uint64_t db = dk0 + (uint64_t)(sl * (kApPiece >> 4));
#pragma unroll
          for (int k = 0; k < 4; k++) at_mma_ss(tu + 128u * h, da + (uint64_t)(2 * k), db + (uint64_t)(2 * k), id_s, k > 0 ? 1u : (uint32_t)(z > 0));
          if (last) at_commit(&s.kv_empty[sl]);
          da += (uint64_t)(kApPiece >> 4);
          sl = sl + 1 == kStages ? 0 : sl + 1;
        }
        at_commit(&s.s_full[h]);
        if (q_last) at_commit(&s.q_empty);
      };
      for (int i = 0; ok; i++) {
        wait(&s.sched_full[i & 1], (uint32_t)(i >> 1) & 1u);
        if (!all_ok()) break;
        const ApItem &im = s.item[i & 1];
        if (__shfl_sync(kFull, im.b, 0) < 0) break;
        const int n = __shfl_sync(kFull, im.n, 0), m0 = __shfl_sync(kFull, im.m0, 0);
        const int n0 = __shfl_sync(kFull, im.n0, 0), n1 = __shfl_sync(kFull, im.n1, 0);
        const int end = __shfl_sync(kFull, im.end - im.j0 * kApTile, 0);   // tokens of the part from here on are seen by none
        const bool twin = PAGED ? __shfl_sync(kFull, im.twin, 0) : TWINS;
        const int ahead = twin ? 2 : 1;            // S of tile j + ahead follows PV of tile j
        wait(&s.q_full, (uint32_t)i & 1u);
        if constexpr (LAT) {
          for (int j = 0; j < ahead && j < n && ok; j++) {
            const bool q_last = j + 1 == n;
            wait_tile(tiles++);
            at_fence_after();
            if (at_elect() && ok) {
              if (twin) {
                issue_s3(j, 0, pos, true, q_last);
              } else {
                issue_s3(0, 0, pos, n1 == 0, q_last && n1 == 0);
                if (n1 > 0) issue_s3(1, 1, pos, true, q_last);
              }
            }
            if (!all_ok()) break;
            pos += 3;
          }
          for (int j = 0; j < n && ok; j++) {
            // V[j] at pieces pos, pos + 1, and K[j + ahead] behind it
            const uint32_t s0 = pos % kStages, s1 = s0 + 1 == kStages ? 0 : s0 + 1, lo = min(s0, s1), hi = max(s0, s1);
            wait_tile(tiles++);
            if (j >= m0) {
              const int z = j - m0, bit = 3 * (i & 1) + z;   // z: 0, 1 or 2
              wait(&s.v_clean[i & 1][z], (clean >> bit) & 1u);
              clean ^= 1u << bit;
            }
            const int left = end - j * kApTile;    // tokens of the tile that some row sees
            // the pair's second half of the elements is `hi - lo` slots on
            const uint64_t db = at_desc(ring + lo * kApPiece, (hi - lo) * kApPiece);
            const uint32_t add = j >= ahead;
            bool keys = false;                     // K[j + ahead] is known to be there: waited for behind the first PV
            pos += 2;
#pragma unroll
            for (int h = 0; h < 2; h++) {
              const int nh = h ? n1 : n0;
              if (twin ? (j & 1) == h : j < nh) {
                uint32_t &np = h ? np1 : np0;
                const bool more = twin ? j + 2 < n : j + 1 < nh, tail = twin || h || n1 == 0;   // the tile's last row tile
                const bool q_last = tail && j + ahead + 1 == n, at_once = more && keys;
                wait(&s.p_full[h], np);
                np ^= 1u;
                at_fence_after();
                if (at_elect() && ok) {
                  const uint32_t oc = tu + 256u + 128u * h, pc = tu + 128u * h;
                  if (left >= kApTile) {
#pragma unroll
                    for (int k = 0; k < kApTile / 16; k++) at_mma_ts(oc, pc + 8u * k, db + (uint64_t)(128u * k), id_o, k > 0 ? 1u : add);
                  } else {
#pragma unroll 1
                    for (int k = 0; 16 * k < left; k++) at_mma_ts(oc, pc + 8u * k, db + (uint64_t)(128u * k), id_o, k > 0 ? 1u : add);
                  }
                  if (tail) {
                    at_commit(&s.kv_empty[lo]);
                    at_commit(&s.kv_empty[hi]);
                  }
                  if (!more) at_commit(&s.o_done[h]);
                  if (at_once) issue_s3(h, twin ? 0 : h, pos, tail, q_last);
                }
                if (more && !at_once) {
                  wait_tile(tiles);
                  keys = true;
                  at_fence_after();
                  if (at_elect() && ok) issue_s3(h, twin ? 0 : h, pos, tail, q_last);
                }
                if (!all_ok()) break;
              }
            }
            if (j + ahead < n) {
              pos += 3;
              tiles++;
            }
          }
        } else {
          for (int j = 0; j < ahead && j < n; j++) {
            wait(&s.kv_full[slot], phase);
            if (!all_ok()) break;
            at_fence_after();
            if (at_elect()) {
              if (twin) {
                issue_s(j, 0);
              } else {
                issue_s(0, 0);
                if (n1 > 0) issue_s(1, 1);
              }
              at_commit(&s.kv_empty[slot]);
              if (j + 1 == n) at_commit(&s.q_empty);
            }
            __syncwarp();
            next_stage();
          }
          for (int j = 0; j < n && ok; j++) {
            wait(&s.kv_full[slot], phase);
            if (j >= m0) {
              const int z = j - m0, bit = 3 * (i & 1) + z;   // z: 0, 1 or 2
              wait(&s.v_clean[i & 1][z], (clean >> bit) & 1u);
              clean ^= 1u << bit;
            }
            const int left = end - j * kApTile;      // tokens of the tile that some row sees
            const uint64_t db = dv0 + (uint64_t)(slot * (2 * kTB >> 4));
            const uint32_t add = j >= ahead;
#pragma unroll
            for (int h = 0; h < 2; h++) {
              const int nh = h ? n1 : n0;
              if (twin ? (j & 1) == h : j < nh) {
                uint32_t &np = h ? np1 : np0;
                const bool more = twin ? j + 2 < n : j + 1 < nh;
                wait(&s.p_full[h], np);
                np ^= 1u;
                at_fence_after();
                if (at_elect() && ok) {
                  const uint32_t oc = tu + 256u + 128u * h, pc = tu + 128u * h;
                  if (left >= kApTile) {
#pragma unroll
                    for (int k = 0; k < kApTile / 16; k++) at_mma_ts(oc, pc + 8u * k, db + (uint64_t)(128u * k), id_o, k > 0 ? 1u : add);
                  } else {
#pragma unroll 1
                    for (int k = 0; 16 * k < left; k++) at_mma_ts(oc, pc + 8u * k, db + (uint64_t)(128u * k), id_o, k > 0 ? 1u : add);
                  }
                  if (more) issue_s(h, twin ? 0 : h);
                  else at_commit(&s.o_done[h]);      // the row tile's last
                  if (twin || h || n1 == 0) {        // and the tile's last
                    at_commit(&s.kv_empty[slot]);
                    if (j + ahead + 1 == n) at_commit(&s.q_empty);
                  }
                }
                if (!all_ok()) break;
              }
            }
            if (!ok) break;
            next_stage();
          }
        }
        if (lane == 0) mbar_arrive(&s.sched_empty[i & 1]);
      }
      // every MMA issued has completed before tensor memory is released
      if (at_elect()) at_commit(&s.drain);
      mbar_wait_bounded(&s.drain, 0u, a.wait_ns);
      __syncwarp();
    } else {
      // ---------------------------------------------------------- Q rows, and the scan of masked tiles' v
      const int ht = tid - 32 * kApWHelp;
      uint32_t posted[3] = {0u, 0u, 0u};
      int nq = 0;                                  // items whose Q has been copied
      bool ok = true;
      for (int i = 0; ok; i++) {
        if (!at_wait(&s.sched_full[i & 1], (uint32_t)(i >> 1) & 1u, a, p.ctrl)) break;
        const ApItem it = s.item[i & 1];
        if (it.b < 0) break;
        const int n = it.n;
        if (lane < 12) s.bad[i & 1][warp - kApWHelp][lane >> 2][lane & 3] = 0u;
        __syncwarp();
        // warp 3 has no part in Q: were it to wait here, the MMA warp could be done with the
        // next Q before it looks
        if (warp == kApWHelp && i > 0 && !at_wait(&s.q_empty, (uint32_t)(i - 1) & 1u, a, p.ctrl)) break;
        // a box (64, group, per) is a row tile; rows past the item's tokens are
        // others' or zeros, rows past the box what was there: none is stored
        if (ht == 0) {
          const int boxes = it.toks > p.per ? 2 : 1;
          mbar_arrive_expect_tx(&s.q_full, (uint32_t)(boxes * p.per * a.group * kQHalves * 128));
          for (int q = 0; q < boxes; q++)
            for (int hf = 0; hf < kQHalves; hf++)
              at_tma_3d(q_smem + q * kQT + hf * (kApTile * 128), &p.qmap, 64 * hf, it.hk * a.group, it.first + it.tok0 + q * p.per,
                        &s.q_full);
        }
        nq++;
        for (int j = it.m0; j < n; j++) {
          const int z = j - it.m0;
          const uint32_t ph = z == 0 ? posted[0] : (z == 1 ? posted[1] : posted[2]);   // by item parity: bit i & 1
          ok = at_wait(&s.v_posted[i & 1][z], (ph >> (i & 1)) & 1u, a, p.ctrl);
          if (!ok) break;
          const int pos = s.v_pos[i & 1][z], slot = pos % kStages;
          const int bar = LAT ? s.v_tile[i & 1][z] & 3 : slot;
          ok = at_wait(&s.kv_full[bar], (uint32_t)(LAT ? s.v_tile[i & 1][z] >> 2 : pos / kStages) & 1u, a, p.ctrl);
          if (!ok) break;
          const int next = (pos + 1) % kStages, lo = min(slot, next), hi = max(slot, next);   // latent: the slots of the tile's halves
          if (z == 0) posted[0] ^= 1u << (i & 1);
          else if (z == 1) posted[1] ^= 1u << (i & 1);
          else posted[2] ^= 1u << (i & 1);
          uint8_t *tile = generic0 + 2 * kQT + (LAT ? lo * kApPiece : (2 * slot + 1) * kTB);
          const int half = LAT ? (hi - lo) * kApPiece : kApTile * 128;
          // earlier tokens are seen by every row; PV leaves out the groups of 16 past the last one that is seen
          const int r0 = max(0, it.all - (it.j0 + j) * kApTile);
          const int r1 = min(kApTile, (it.end - (it.j0 + j) * kApTile + 15) & ~15);
          for (int hf = 0; hf < kHalves; hf++)
#pragma unroll 4
            for (int e = r0 * 8 + ht; e < r1 * 8; e += 64) {
              uint4 *at = reinterpret_cast<uint4 *>(tile + hf * half) + e;
              const uint4 w = *at;
              const uint32_t f[4] = {at_nonfinite<F16>(w.x), at_nonfinite<F16>(w.y), at_nonfinite<F16>(w.z), at_nonfinite<F16>(w.w)};
              if (f[0] | f[1] | f[2] | f[3]) {
                uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int w = 0; w < 4; w++) u[w] &= ~(((f[w] >> 15) & 0x00010001u) * 0xFFFFu);
                *at = make_uint4(u[0], u[1], u[2], u[3]);
                atomicOr(&s.bad[i & 1][warp - kApWHelp][z][(e >> 3) >> 5], 1u << ((e >> 3) & 31));
              }
            }
          at_fence_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.v_clean[i & 1][z]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.sched_empty[i & 1]);
      }
      // a copy in flight lands before the CTA ends
      if (warp == kApWHelp && nq > 0) mbar_wait_bounded(&s.q_full, (uint32_t)(nq - 1) & 1u, a.wait_ns);
      __syncwarp();
    }
  }
  at_fence_before();
  __syncthreads();
  if (warp == kApWMma) {
    at_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tb), "r"(512) : "memory");
  }
}

// Joins the parts of the items that several CTAs took, in the order of the
// context: o = sum_k 2^(c (m_k - m)) O_k / sum_k 2^(c (m_k - m)) l_k.  A unit is 1024 / D
// rows of an item, a thread one row and four of its elements, so that 8 or 16
// rows are read side by side and a long context's many parts are spread over as
// many CTAs as there are.  The items to join are few and anywhere among the CTAs'
// descriptions: every CTA looks all of them over and takes its units.  Latency bound:
// the parts (19 MB for the 4 requests above, from L2) take some 6 us behind the kernel
// above, which their bytes alone would in 3; more CTAs or more registers gave nothing.
template <int D, bool F16>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ ApArgs p, int sms) {
  __shared__ unsigned masks[kApMaxSms / 32];
  constexpr int kUnit = 1024 / D, kUnits = kApRows / kUnit;
  const AttnArgs &a = p.a;
  const int tid = threadIdx.x, words = (sms + 31) / 32;
  pdl_wait();
  for (int k = tid; k < 32 * words; k += 256) {
    const unsigned mask = __ballot_sync(kFull, k < sms && __ldcg(&p.desc[2 * k + 1].y) >= 0);
    if ((tid & 31) == 0) masks[k >> 5] = mask;
  }
  __syncthreads();
  int count = 0;
  for (int w = 0; w < words; w++) count += __popc(masks[w]);
  const float c = a.scale * 1.44269504088896340736f;
  for (int unit = blockIdx.x; unit < count * kUnits; unit += gridDim.x) {
    // the unit's item: the description of the (unit / kUnits)-th set bit
    int left = unit / kUnits, w = 0;
    while (left >= __popc(masks[w])) left -= __popc(masks[w++]);
    unsigned bits = masks[w];
    for (; left > 0; left--) bits &= bits - 1;
    const int which = 32 * w + __ffs(bits) - 1;
    const int4 d0 = __ldcg(p.desc + 2 * which), d1 = __ldcg(p.desc + 2 * which + 1);
    const int first = d0.x, hk = d0.y, tok0 = d0.z, toks = d0.w, c0 = d1.x, c1 = d1.y, slot0 = d1.z, twin = d1.w;
    const int r = unit % kUnits * kUnit + tid % kUnit, d4 = tid / kUnit;
    const int rt = r & (kApTile - 1), dt = (rt * p.magic) >> 16, tl = (r / kApTile) * p.per + dt;   // as in the kernel above
    if (dt >= p.per || tl >= toks) continue;
    const int nsrc = (c1 - c0 + 1) << twin;        // twins: two sources a part, 128 rows apart
    float top = kAtLeast, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int q0 = 0; q0 < nsrc; q0 += 8) {         // eight sources at a time, so that their loads wait together
      float2 st[8];
      float4 u[8];
      float t1 = top;
#pragma unroll
      for (int z = 0; z < 8; z++) {
        const int q = q0 + z, k = c0 + (q >> twin), slot = k == c0 ? slot0 : 2 * k;
        const int row = r + (twin && (q & 1) ? kApTile : 0);
        st[z] = make_float2(-INFINITY, kAtNoPart);
        if (q < nsrc) {
          st[z] = __ldcg(p.stat + (size_t)slot * kApRows + row);
          u[z] = __ldcg(p.part + ((size_t)slot * (D / 4) + d4) * kApRows + row);
        }
      }
#pragma unroll
      for (int z = 0; z < 8; z++) t1 = fmaxf(t1, st[z].x);
      const float f0 = top == t1 ? 1.f : at_exp2((top - t1) * c);
      top = t1;
      sum *= f0;
      acc.x *= f0;
      acc.y *= f0;
      acc.z *= f0;
      acc.w *= f0;
#pragma unroll
      for (int z = 0; z < 8; z++) {
        if (st[z].y < 0.f) continue;               // no part, or a twin without a tile
        const float f = at_exp2((st[z].x - t1) * c);
        sum = fmaf(st[z].y, f, sum);
        acc.x = fmaf(u[z].x, f, acc.x);
        acc.y = fmaf(u[z].y, f, acc.y);
        acc.z = fmaf(u[z].z, f, acc.z);
        acc.w = fmaf(u[z].w, f, acc.w);
      }
    }
    const int i = tok0 + tl, hq = hk * a.group + rt - dt * a.group;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    *reinterpret_cast<uint2 *>(a.out.p + (long long)(first + i) * a.out.row + (long long)hq * a.out.head + 4 * d4) =
        make_uint2(at_pack<F16>(acc.x * inv, acc.y * inv), at_pack<F16>(acc.z * inv, acc.w * inv));
    if (a.lse && d4 == 0) a.lse[(size_t)(first + i) * a.q_heads + hq] = sum == 0.f ? -INFINITY : top * a.scale + logf(sum);
  }
}

namespace {
typedef void (*ApKernel)(const ApArgs);
typedef void (*ApJoin)(const ApArgs, int);
template <bool PAGED, bool TWINS>
ApKernel ap_kernel(int head_dim, int f16) {
  if (head_dim == 64) return f16 ? attn_wide_kernel<64, true, PAGED, TWINS, false> : attn_wide_kernel<64, false, PAGED, TWINS, false>;
  return f16 ? attn_wide_kernel<128, true, PAGED, TWINS, false> : attn_wide_kernel<128, false, PAGED, TWINS, false>;
}
ApKernel ap_latent(bool twins, int f16) {
  if (twins) return f16 ? attn_wide_kernel<128, true, false, true, true> : attn_wide_kernel<128, false, false, true, true>;
  return f16 ? attn_wide_kernel<128, true, false, false, true> : attn_wide_kernel<128, false, false, false, true>;
}
ApJoin ap_join(int head_dim, int f16) {
  if (head_dim == 64) return f16 ? attn_join_kernel<64, true> : attn_join_kernel<64, false>;
  return f16 ? attn_join_kernel<128, true> : attn_join_kernel<128, false>;
}
int ap_smem(int head_dim) { return head_dim == 64 ? ApGeom<64>::kSmem : ApGeom<128>::kSmem; }

// Packed rows [T][heads][dim] in boxes of 64 elements x `heads_box` heads x `rows_box` rows.
cudaError_t encode_rows(CUtensorMap *map, const RowView &r, int T, int heads, int heads_box, int rows_box, int dim, const AttnArgs &a) {
  const AttnMapEncodeFn enc = attn_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)T};
  const cuuint64_t strides[2] = {(cuuint64_t)r.head * 2, (cuuint64_t)r.row * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)heads_box, (cuuint32_t)rows_box};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult e = enc(map, a.f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, r.p, dims, strides,
                         box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return e == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Row tiles of whole tokens, and their Q as boxes.
cudaError_t encode_q(ApArgs *p, int dim) {
  const AttnArgs &a = p->a;
  p->magic = (65536 + a.group - 1) / a.group;
  p->per = kApTile / a.group;
  return encode_rows(&p->qmap, a.q, a.T, a.q_heads, a.group, p->per, dim, a);
}
}  // namespace

namespace {
cudaError_t ap_setup(ApKernel k, int smem) {
  cudaFuncAttributes at;
  const cudaError_t err = cudaFuncGetAttributes(&at, k);
  if (err != cudaSuccess) return err;
  // the register shares of the warpgroups have to fit what the CTA is launched with
  if (at.numRegs * kApThreads < kApRegsSoft * 256 + kApRegsRest * 128) return cudaErrorInvalidConfiguration;
  return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}
}  // namespace

cudaError_t attn_wide_setup(int head_dim, int f16) {
  const ApKernel kernels[3] = {ap_kernel<false, false>(head_dim, f16), ap_kernel<false, true>(head_dim, f16), ap_kernel<true, false>(head_dim, f16)};
  for (const ApKernel k : kernels) {
    const cudaError_t err = ap_setup(k, ap_smem(head_dim));
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

cudaError_t attn_wide_latent_setup(int f16) {
  const cudaError_t err = ap_setup(ap_latent(false, f16), ApLatGeom::kSmem);
  return err == cudaSuccess ? ap_setup(ap_latent(true, f16), ApLatGeom::kSmem) : err;
}

AttnWideWs attn_wide_ws(size_t off, int head_dim, int num_sms) {
  AttnWideWs w;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = (off + bytes + 255) / 256 * 256;
    return at;
  };
  w.desc = take(32 * (size_t)num_sms);
  w.stat = take(8 * (size_t)(2 * num_sms) * kApRows);
  w.part = take(4 * (size_t)(2 * num_sms) * kApRows * head_dim);
  w.total = off;
  return w;
}

cudaError_t launch_attn_prompt(const AttnArgs &a, const RowView *k_rope, int *ctrl, int num_sms, cudaStream_t stream) {
  ApArgs p;
  memset(&p, 0, sizeof(p));
  p.a = a;
  p.ctrl = ctrl;
  cudaError_t err = encode_q(&p, k_rope ? a.head_dim + 64 : a.head_dim);
  if (err == cudaSuccess) err = encode_rows(&p.kmap, a.k, a.T, a.kv_heads, 1, kApTile, a.head_dim, a);
  if (err == cudaSuccess) err = encode_rows(&p.vmap, a.v, a.T, a.kv_heads, 1, kApTile, a.head_dim, a);
  if (err == cudaSuccess && k_rope) err = encode_rows(&p.rmap, *k_rope, a.T, 1, 1, kApTile, 64, a);
  if (err != cudaSuccess) return err;
  // Items at most: every request may end inside one.  Where row tiles are as few as
  // CTAs, an item is one row tile and the softmax warps of the other take every second
  // of its key tiles (us with twins, without): 1 prompt of 512, 8 kv heads of 4, D = 128
  // 11.5, 13.5; of 2000, 1 kv head of 8 20.3, 29.5; of 1000, 8 of 2, D = 64 11.5, 15.6.
  auto items_of = [&](int span) { return (a.T + (long long)a.B * (span - 1)) / span * a.kv_heads; };
  p.span = items_of(p.per) <= num_sms ? p.per : 2 * p.per;
  const long long items = items_of(p.span);
  const int grid = (int)(items < num_sms ? items : num_sms);
  const bool twins = p.span == p.per;
  const ApKernel k = k_rope ? ap_latent(twins, a.f16) : (twins ? ap_kernel<false, true> : ap_kernel<false, false>)(a.head_dim, a.f16);
  if (!k_rope) {
    k<<<grid, kApThreads, ap_smem(a.head_dim), stream>>>(p);
    return cudaGetLastError();
  }
  // its launch, and the setting up of its barriers, beside the end of the kernel before
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kApThreads);
  cfg.dynamicSmemBytes = ApLatGeom::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, p);
}

cudaError_t launch_attn_wide_tree(const AttnArgs &a, uint8_t *ws, const AttnWideWs &w, int num_sms, cudaStream_t stream) {
  ApArgs p;
  memset(&p, 0, sizeof(p));
  p.a = a;
  p.ctrl = reinterpret_cast<int *>(ws);
  p.desc = reinterpret_cast<int4 *>(ws + w.desc);
  p.stat = reinterpret_cast<float2 *>(ws + w.stat);
  p.part = reinterpret_cast<float4 *>(ws + w.part);
  cudaError_t err = encode_q(&p, a.head_dim);
  if (err == cudaSuccess) err = attn_encode_cache(&p.kmap, a.k_cache, a, 1 << a.page_shift);
  if (err == cudaSuccess) err = attn_encode_cache(&p.vmap, a.v_cache, a, 1 << a.page_shift);
  if (err != cudaSuccess) return err;
  if (num_sms > kApMaxSms) num_sms = kApMaxSms;
  ap_kernel<true, false>(a.head_dim, a.f16)<<<num_sms, kApThreads, ap_smem(a.head_dim), stream>>>(p);
  if ((err = cudaGetLastError()) != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * num_sms));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, ap_join(a.head_dim, a.f16), p, num_sms);
}

}  // namespace moe
