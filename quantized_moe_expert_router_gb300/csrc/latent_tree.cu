// latent_tree.cu -- absorbed latent attention over the paged cache on the 5th-generation
// tensor cores (moe_latent_tree): single tokens, drafted trees or the next part of a prompt.
//
// All heads of a token read the same cached vectors (c, r) of 512 + 64 elements, keys and
// values at once, so a tile of 64 tokens comes once and serves up to 64 query rows (tokens x
// heads).  Query rows are the N of both products, tokens and latent elements the M:
//   S^T = K Q^T                 M = 64 tokens, N rows, K = 576: A the tile as it lies, B = Q
//   m' = max(m, max S);  P = 2^(c (S - m'));  l = l 2^(c (m - m')) + sum P,  c = softmax_scale * log2(e)
//   O^T = O^T 2^(c (m - m')) + C^T P^T   M = 4 x 128 latent elements, N rows, K = 64 tokens: A the same tile
//                               transposed (M-major), B = P^T
// That way few rows cost little (N is 16, 32 or 64), the 512 x N fp32 of O^T fit tensor memory
// beside two S^T (6 N of 512 columns; rows as M would take 512 columns for O alone), and the tile is in
// shared memory once.  The price: the products read A and B from shared memory at 128 bytes a cycle, which
// bounds a step of 16 (measured: S 24, 25, 33 cycles at N = 16, 32, 64, O 39, 41, 49).
// The maximum of a row goes over tokens, which are lanes; so the maximum that P is taken against moves only
// when some score passes it by 2^8 (in P's terms), one vote of the four warps a tile tells, and the sums stay
// per lane to the item's end.  P is rounded to the element type because the tensor cores multiply equal types; m, l
// and O are fp32, l is summed from the unrounded values.
//
// An item is (request, whole tokens of it, a part of the heads): N rows at most.  More than 64
// heads are two parts.  One CTA per SM, 12 warps:
//   warp 0           tiles, 64 elements x a page a copy (128-byte swizzle): two halves of 64 x 256 elements into a
//                    ring of 4 or 5, and with the second the key part into one of 2 or 3; takes the items
//   warps 1, 3       MMA issue of S and of O: the products read shared memory all the time, which makes every wait's
//                    look at a barrier slow (100 to 200 cycles), so one's products fill the other's waits (one issuer that
//                    takes what is ready: 163 us where two have 154, 16 tokens at up to 100000 of 64 heads)
//   warp 2           Q rows by boxes (64, heads, tokens)
//   warps 4-7, 8-11  softmax of rows 0 .. N/2 - 1 and N/2 .. N - 1: a warp has 16 tokens, a thread two
//                    of them and a quarter of the warp's rows (the fragment shape: an accumulator of 64 rows fills 16 of a
//                    warp's 32 lanes); the rescaling of O and the epilogue, a thread a latent element
// A half is free when the products of its latent elements are done, P lies where the tile's key part was.  With
// N = 64 shared memory holds Q and two tiles, so that one comes while the other is worked on.  (One tile of 128 tokens
// instead: S needs 17 % fewer cycles, but nothing comes between S and the values' products, and all SMs then
// load and compute in step: 16 tokens at up to 100000 of 64 heads 204 us.)
//
// The tiles of all items stand in one line that the CTAs share (LtCursor); calls with two items
// over the same tokens (two parts of the heads, or more tokens than a tile has room for) give each place of
// the line to two CTAs, which read the same tiles at the same time: the second one from L2.  A
// part of an item goes to the workspace (fp32 O, m, l); lat_join_kernel joins them, always in the same order.
//
// Where contexts are short or items many, an item is not cut: there is nothing to join then.
//
// A token that a row does not see has P = 0, but 0 times an infinite or NaN latent is NaN: in
// tiles with tokens that not every row sees the softmax warps zero such elements after S, note the token, and
// the epilogue makes these elements NaN in the rows that do see it.
//
// A wait knows its phase by parity alone, so no barrier may be two phases on when a waiter looks:
//   sched_full    (item parity) item i + 2 is posted when sched_empty has all 11 arrivals of item i
//   kv_full       filled again behind kv_empty, which the O warp commits behind the tile's p_full,
//                 which every softmax warp gives after its scan.  The place of a second half is free only after that of
//                 the key part that comes with it.
//   kv_empty      waited for by the copy warp, whose lanes meet before they copy
//   q_full        filled again behind q_empty; q_empty is waited for by warp 2 alone, and without that Q there is no next
//   s_full        (tile parity) S of tile t + 2 is issued behind p_full of tile t
//   p_full        (tile parity) P of tile t + 2 follows its S.  That S comes after the S warp has waited for p_full of tile t,
//                 and needs the whole tile t + 2, whose second half lies where one of tile t lay: behind the O warp's wait
//                 for p_full of tile t.
//   pv_done       (tile parity) tile t lies, with its second half, where one of tile t - 3 or t - 2 lay, so with S of tile t the
//                 products of tile t - 3 are done: a warp that has it may wait for those of tile t - 1, and then for those
//                 of tile t; the next ones on these barriers need P that it has not given
// The softmax warps of a half also meet at a named barrier: a warp whose wait ran out goes on to
// the next vote, which tells the others, and all four end together.
//
// Bound: for up to 64 rows over long contexts HBM (16 tokens at up to 100000 of 64 heads 154 us, 5.2 TB/s; 16 heads,
// 16 at up to 60000, 84 us, 5.7); for more rows shared memory (a tile's products alone 1970 cycles at N = 64, 1490 at N = 16; by clock
// reads 2600 to 3300 beside one another and behind a ring of two tiles: 128 heads, 16 at up to 60000, 157 us, 730 TFLOP/s); for short
// contexts a chain of latencies: one token at 50 9 us, at 1000 12, join 3 of it.  Around the tiles the first scores come 5
// (one request) to 9 us after the start, an item's epilogue takes 1 (N = 16) to 2.3, the join 4 (N = 16) to 7.
#include <float.h>
#include <limits.h>
#include <math.h>
#include <stddef.h>
#include <string.h>

#include "attn_tc.cuh"
#include "latent.h"

namespace moe {

constexpr int kLtThreads = 384;
constexpr int kLtTile = 64;                       // tokens of a tile
constexpr int kLtWTma = 0, kLtWS = 1, kLtWQ = 2, kLtWO = 3, kLtWSoft = 4;
constexpr int kLtChunk = kLtTile * 128, kLtPair = 2 * kLtChunk, kLtHalf = 2 * kLtPair;   // bytes of 64, 128 and 256 elements of a tile
constexpr int kLtBlocks = kLatDim / 128;          // of 128 latent elements
constexpr int kLtMaxB = MOE_ATTN_MAX_REQUESTS;
constexpr int kLtMaxSms = 1024;
constexpr int kLtRows = 64;                       // rows of an item at most
constexpr float kLtSlack = 8.f;                   // log2 of the largest P
constexpr float kLtUnset = FLT_MAX;               // in place of -m before a row has seen anything: any finite score passes it

template <int N>
struct LtGeom {
  static constexpr int kHalves = N == 64 ? 4 : 5;
  static constexpr int kParts = N == 64 ? 2 : 3;  // key parts
  static constexpr int kRope = kHalves * kLtHalf; // a key part, then P in its place: 64 x 128 bytes, 64 x 2 N
  static constexpr int kQ = kRope + kParts * kLtChunk;
  static constexpr int kQChunk = N * 128;         // 64 elements of the rows
  static constexpr int kSmem = kQ + 9 * kQChunk + 1024;
};

struct LtArgs {
  CUtensorMap cmap;            // (64, page or 64) boxes over [num_pages * page][576]
  CUtensorMap qmap, rmap;      // (64, hh, per) boxes over [T][heads][512] and [T][heads][64]
  LatArgs a;
  int *ctrl;
  int hh, hp;                  // heads of a part, parts
  int per;                     // tokens of an item
  int gang;                    // CTAs (1 or 2) to a place of the line
  int magic;                   // ceil(2^16 / hh)
  int whole;                   // items are not cut: no parts, no join
  int slack;                   // tiles by which equal parts may be longer than the mean
  int4 *desc;                  // per CTA, of the item whose first part it holds and others the rest:
                               // (first, head part, tok0, toks), (first group, last group, its slot, place in the group)
  float *part;                 // [2 * grid][N][512]  O of a part
  float2 *stat;                // [2 * grid][N]       (m, l)
};

struct LtItem {
  int b;                       // request (-1: no more items)
  int first, tok0, toks, hpart;
  int j0, n;                   // first tile and number of tiles
  int cached, all, end;        // context before the fresh tokens; tokens that every row sees; tokens from `end` on are seen by none
  int m0;                      // tiles j0 + m0 .. are masked
  int slot;                    // where the part goes; -1: the item is whole
};

struct LtSmem {
  uint64_t kv_full[5], kv_empty[5];
  uint64_t q_full, q_empty, s_full[2], p_full[2], pv_done[2], sched_full[2], sched_empty[2], drain;
  uint32_t tmem;
  int fail[2];                 // the vote at which a wait was found to have run out
  LtItem item[2];
  uint32_t bad[2][3][2];       // by item parity and masked tile: tokens with a non-finite latent
  float wmax[2][4][32], wsum[2][4][32];
  alignas(16) float m[8][32];  // per softmax warp: -m of its rows
  alignas(16) float f[8][32];  // and their factors
};
static_assert(offsetof(LtSmem, m) % 16 == 0 && offsetof(LtSmem, f) % 16 == 0, "read four at a time");

// While the CTA's copy warp finds its share, in the place of the tiles: of each request its items and their tiles.
struct LtSetup {
  int items[kLtMaxB], nch[kLtMaxB];
};

__device__ __forceinline__ bool lt_wait(uint64_t *bar, uint32_t parity, const LtArgs &p) {
  const bool ok = __all_sync(kFull, mbar_wait_bounded(bar, parity, p.a.wait_ns));
  if (!ok && (threadIdx.x & 31) == 0) atomicOr(p.ctrl + kAttnCtrlFlags, MOE_FLAG_TIMEOUT);
  return ok;
}
// True in all of a half's 128 threads when it is in one of them.
__device__ __forceinline__ bool lt_any(int half, bool x) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %2, 0;\n\tbarrier.cta.red.or.pred.aligned p, %1, 128, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(1 + half), "r"((uint32_t)x)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void lt_sync(int half) {
  __syncwarp();
  asm volatile("barrier.cta.sync.aligned %0, 128;" ::"r"(1 + half) : "memory");
}
// 8, 16 or 32 columns of this warp's 32 tensor-memory lanes.
template <int C>
__device__ __forceinline__ void lt_ld(uint32_t at, float (&r)[C]) {
  if constexpr (C == 32) {
    at_ld32(at, r);
  } else if constexpr (C == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(at)
        : "memory");
  } else {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
                 : "r"(at)
                 : "memory");
  }
  at_wait_ld(r);
}
template <int C>
__device__ __forceinline__ void lt_st(uint32_t at, const float (&r)[C]) {
  if constexpr (C == 32) {
    at_st32(at, r);
  } else if constexpr (C == 16) {
    at_st16(at, reinterpret_cast<const uint32_t *>(r));
  } else {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "f"(r[0]), "f"(r[1]), "f"(r[2]),
                 "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7])
                 : "memory");
  }
}
// C / 2 columns of 16 of this warp's lanes as fragments: r[4 i + e] is column 8 i + 2 (lane & 3) + (e & 1) of row lane / 4 + 8 (e >> 1).
template <int C>
__device__ __forceinline__ void lt_frag(uint32_t at, float (&r)[C / 2]) {
  if constexpr (C == 32) {
    at_ld_frag(at, r);
  } else if constexpr (C == 16) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
                 : "r"(at)
                 : "memory");
  } else {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3])
                 : "r"(at)
                 : "memory");
  }
  at_wait_ld(r);
}

// Descriptor of P^T: rows of tokens, 2 N bytes under the swizzle of that width (N-major); 8 rows apart.
template <int N>
__device__ __forceinline__ uint64_t lt_desc_p(uint32_t addr) {
  constexpr uint64_t layout = N == 64 ? 2 : (N == 32 ? 4 : 6);
  return (uint64_t)((addr >> 4) & 0x3FFFu) | (1ull << 16) | ((uint64_t)((16u * N) >> 4) << 32) | (1ull << 46) | (layout << 61);
}
// Place of 16-byte piece c of row k of P^T under that swizzle.
template <int N>
__device__ __forceinline__ int lt_p_at(int k, int c) {
  return k * 2 * N + ((N == 64 ? c ^ (k & 7) : (N == 32 ? c ^ ((k >> 1) & 3) : c ^ ((k >> 2) & 1))) << 4);
}
// Instruction descriptors: S with M = 64 and both operands K-major, O with M = 128, A M-major and B N-major.
__device__ __forceinline__ constexpr uint32_t lt_idesc_s(bool f16, int n) { return (at_idesc(f16, n, false) & ~(31u << 24)) | ((64u >> 4) << 24); }
__device__ __forceinline__ constexpr uint32_t lt_idesc_o(bool f16, int n) { return at_idesc(f16, n, true) | (1u << 15); }

// Of a request of n fresh rows: items of a place of the line, and tiles that its rows may see.
__device__ __forceinline__ int lt_groups(const LtArgs &p, int n) { return p.hp * at_idiv(n + p.per - 1, p.per); }
__device__ __forceinline__ int lt_items(const LtArgs &p, int n) { return p.gang == 2 ? (lt_groups(p, n) + 1) >> 1 : lt_groups(p, n); }
__device__ __forceinline__ int lt_nch(const LatArgs &a, int n, int cached) {
  const int ctx = min(cached + (a.tree_mask ? min(n, MOE_ATTN_MAX_TREE) : n), a.max_pages << a.page_shift);
  return (ctx + kLtTile - 1) / kLtTile;
}
__device__ __forceinline__ void lt_request(const LatArgs &a, int b, int &first, int &n, int &cached) {
  first = __ldg(a.cu + b);
  n = first < 0 ? 0 : max(0, min(__ldg(a.cu + b + 1), a.T) - first);
  cached = min(max(__ldg(a.cached + b), 0), a.max_pages << a.page_shift);       // no sum with rows passes 2^31
}

// Walks the line of tiles from the CTA's share on.
struct LtCursor {
  AtShare share;
  int b, first, n, cached, items;
  int places;                  // of an item of b in the line
  bool few;                    // items that are not cut, at most one for a CTA
  long long work;              // places of the requests before b
  // of the last part, when it is the first of several: what the join has to know
  bool split;
  int need;
  long long item0;
  __device__ __forceinline__ void load(const LtArgs &p) {
    lt_request(p.a, b, first, n, cached);
    places = per_item(p, lt_nch(p.a, n, cached));
    items = lt_items(p, n);
  }
  // An item's places are its tiles.  One that is not cut is that CTA's in whose share it starts; it has three places more, its
  // epilogue's and its first copies' time, or a single place where there is a CTA for each.
  __device__ __forceinline__ int per_item(const LtArgs &p, int tiles) const { return !p.whole ? tiles : (few ? 1 : tiles + 3); }
  __device__ __forceinline__ int member(const LtArgs &p) const { return p.gang == 2 ? (int)blockIdx.x & 1 : 0; }
  // The share of this CTA, by one warp: a chain of a few hundred cycles a step, and of one look at each request, while the
  // other warps have nothing to do yet.  (lo, hi, held): cu, cu + 1 and cached of request `lane`.
  __device__ __forceinline__ void find(const LtArgs &p, LtSetup &u, int lo, int hi, int held) {
    const LatArgs &a = p.a;
    const int lane = threadIdx.x & 31, end = (a.B + 31) & ~31;
    const int grid = p.gang == 2 ? (int)gridDim.x >> 1 : (int)gridDim.x, me = p.gang == 2 ? (int)blockIdx.x >> 1 : (int)blockIdx.x;
    long long total = 0;
    int count = 0;
    for (int r = lane; r < end; r += 32) {
      if (r >= 32 && r < a.B) {
        lo = __ldg(a.cu + r);
        hi = __ldg(a.cu + r + 1);
        held = __ldg(a.cached + r);
      }
      const int rows = r < a.B && lo >= 0 ? max(0, min(hi, a.T) - lo) : 0, c = min(max(held, 0), a.max_pages << a.page_shift);
      const int i = rows ? lt_items(p, rows) : 0, t = rows ? lt_nch(a, rows, c) : 0;
      u.items[r] = i;
      u.nch[r] = t;
      total += (long long)i * (p.whole ? t + 3 : t);
      count += i;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kFull, total, o);
    count = __reduce_add_sync(kFull, count);
    few = p.whole && count <= grid;
    if (few) total = count;
    __syncwarp();
    AtShare r;
    r.me = me;
    r.len = r.c0 = r.c1 = 0;
    r.x0 = r.x1 = r.rem = 0;
    r.per = 1;
    r.ctas = (int)min(total, (long long)grid);
    if (total > grid) {
      r.per = at_div(total, grid);
      r.rem = total - r.per * grid;
      // A share of the line that ends within items is two parts and more, with an epilogue each (with 64 rows some two tiles' time)
      // and a source of the join: equal parts may be longer than the mean by that.
      const long long mean = r.per + (r.rem > 0);
      if (!p.whole && count <= grid && mean < (1 << 28)) {
        auto fits = [&](int len) {
          int parts = 0;
          for (int q = lane; q < end; q += 32) parts += u.items[q] * at_idiv(u.nch[q] + len - 1, len);
          return __reduce_add_sync(kFull, parts) <= grid;
        };
        int least = (int)mean, most = least + p.slack;
        if (fits(most)) {
          while (least < most) {
            const int mid = (least + most) >> 1;
            if (fits(mid)) most = mid; else least = mid + 1;
          }
          r.len = least;
        }
      }
    }
    if (!r.len && me < r.ctas) {
      r.x0 = r.start(me);
      r.x1 = r.start(me + 1);
    }
    b = first = n = cached = places = items = 0;
    work = 0;
    long long before = 0, at = r.len ? (long long)me : r.x0;   // what counts: parts, or tiles
    for (int q0 = 0; q0 < end; q0 += 32) {
      const int i = u.items[q0 + lane], t = i ? per_item(p, u.nch[q0 + lane]) : 0, unit = r.len ? at_idiv(t + r.len - 1, r.len) : t;
      const long long v = (long long)i * t, w = (long long)i * unit;
      long long incl = v, incl_w = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(kFull, incl, o), y = __shfl_up_sync(kFull, incl_w, o);
        if (lane >= o) {
          incl += x;
          incl_w += y;
        }
      }
      const long long place = at - before - (incl_w - w);
      const unsigned mine = __ballot_sync(kFull, place >= 0 && place < w);
      if (mine && (r.len || r.x0 < r.x1)) {
        const int src = __ffs(mine) - 1;
        b = q0 + src;
        work += __shfl_sync(kFull, incl - v, src);
        items = __shfl_sync(kFull, i, src);
        places = __shfl_sync(kFull, t, src);
        if (r.len) {
          const int pi = __shfl_sync(kFull, unit, src), k0 = (int)__shfl_sync(kFull, place, src), item = at_idiv(k0, pi), k = k0 - item * pi;
          const long long i0 = work + (long long)item * places;
          r.x0 = i0 + (long long)k * r.len;
          r.x1 = min(r.x0 + r.len, i0 + places);
          r.c0 = me - k;
          r.c1 = r.c0 + pi - 1;
        }
        lt_request(a, b, first, n, cached);
        break;
      }
      work += __shfl_sync(kFull, incl, 31);
      before += __shfl_sync(kFull, incl_w, 31);
    }
    share = r;
  }
  // The part of an item that starts at place x, up to the end of the CTA's share; returns the place after it.
  // it.n = 0: there is nothing to do here.
  __device__ __forceinline__ long long part(const LtArgs &p, long long x, LtItem &it) {
    const LatArgs &a = p.a;
    while (n == 0 || x >= work + (long long)items * places) {
      work += (long long)items * places;
      b++;
      load(p);
    }
    const int item = (int)at_div(x - work, places), group = p.gang * item + member(p);
    item0 = work + (long long)item * places;
    const long long xe = p.whole ? item0 + places : min(share.x1, item0 + places);
    const int tg = p.hp == 2 ? group >> 1 : group;
    it.b = b;
    it.first = first;
    it.hpart = p.hp == 2 ? group & 1 : 0;
    it.tok0 = tg * p.per;
    it.toks = min(n - it.tok0, p.per);
    it.n = 0;
    split = false;
    if (it.toks <= 0 || (p.whole && x > item0)) return xe;   // the place's second item is not there; the item is another CTA's
    it.cached = cached;
    const int lim = min(a.max_pages << a.page_shift, cached + n);
    it.all = a.tree_mask ? cached : cached + it.tok0 + 1;
    it.end = min(lim, cached + (a.tree_mask ? min(n, MOE_ATTN_MAX_TREE) : it.tok0 + it.toks));
    need = (it.end + kLtTile - 1) / kLtTile;       // tiles of these rows
    it.j0 = (int)(x - item0);
    it.n = p.whole ? need : max(0, min((int)(xe - item0), need) - it.j0);
    const bool whole = it.j0 == 0 && it.n == need;
    it.slot = whole ? -1 : 2 * (int)blockIdx.x + (x > share.x0);
    it.m0 = max(0, it.all / kLtTile - it.j0);
    split = !whole && it.j0 == 0;
    return xe;
  }
  // For the join, at the CTA that holds the first part: the last part of a CTA's share, so that there is one at most.
  __device__ __forceinline__ void describe(const LtArgs &p, const LtItem &it) {
    if (!split) return;
    int c0, c1;
    share.ctas_of(item0, item0 + need - 1, c0, c1);
    if (share.len) c1 = c0 + (need - 1) / share.len;
    if ((threadIdx.x & 31) == 0) {
      int4 *d = p.desc + 2 * blockIdx.x;
      d[0] = make_int4(it.first, it.hpart, it.tok0, it.toks);
      d[1] = make_int4(c0, c1, it.slot, member(p));
    }
  }
};

__device__ __forceinline__ void lt_tma_2d(uint32_t dst, const CUtensorMap *map, int c0, int c1, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
      : "memory");
}

template <int N, bool F16>
__global__ void __launch_bounds__(kLtThreads, 1) lat_tree_kernel(const __grid_constant__ LtArgs p) {
  extern __shared__ uint8_t dsm[];
  __shared__ LtSmem s;
  using G = LtGeom<N>;
  constexpr uint32_t NH = G::kHalves, NR = G::kParts;
  constexpr int NC = N / 2;
  const LatArgs &a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t smem0 = (smem_u32(dsm) + 1023u) & ~1023u;
  uint8_t *const generic0 = dsm + (smem0 - smem_u32(dsm));

  if (warp == kLtWO) {
    if (lane < (int)NH) {
      mbar_init(&s.kv_full[lane], 1);
      mbar_init(&s.kv_empty[lane], 1);
    } else if (lane >= 14 && lane < 16) {
      mbar_init(&s.s_full[lane - 14], 1);
      mbar_init(&s.p_full[lane - 14], 8);
      mbar_init(&s.pv_done[lane - 14], 1);
    } else if (lane >= 16 && lane < 18) {
      mbar_init(&s.sched_full[lane - 16], 1);
      mbar_init(&s.sched_empty[lane - 16], 11);    // 8 softmax warps, S, O and Q warps
      s.fail[lane - 16] = INT_MAX;
    } else if (lane == 18) {
      mbar_init(&s.q_full, 1);
      mbar_init(&s.q_empty, 1);
    } else if (lane == 19) {
      mbar_init(&s.drain, 2);                      // S and O warps
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid == 32 * kLtWQ) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.cmap)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.qmap)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.rmap)) : "memory");
  }
  if (warp == kLtWS) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s.tmem)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // rows of Q that no box fills
  for (int i = tid; i < 9 * (N - p.per * p.hh) * 8; i += kLtThreads) {
    const int row = p.per * p.hh + (i >> 3) / 9, chunk = (i >> 3) % 9;
    *reinterpret_cast<uint4 *>(generic0 + G::kQ + chunk * G::kQChunk + row * 128 + (i & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
  }

  pdl_wait();                                      // the kernel before is done: what follows reads its results
  int lo = 0, hi = 0, held0 = 0;
  if (warp == kLtWTma && lane < a.B) {
    lo = __ldg(a.cu + lane);
    hi = __ldg(a.cu + lane + 1);
    held0 = __ldg(a.cached + lane);
  }
  at_fence_async();                                // the MMAs read what was written here
  at_fence_before();
  __syncthreads();
  at_fence_after();
  const uint32_t tb = s.tmem;
  const float c = a.scale * 1.44269504088896340736f;
  pdl_launch_dependents();                         // the join's CTAs take the SMs as they fall free, and wait

  if (warp >= kLtWSoft) {
    // ------------------------------------------------------------ softmax
    const int h = (warp - kLtWSoft) >> 2, w4 = warp & 3;
    const uint32_t lanes = (uint32_t)(32 * w4) << 16;
    const uint32_t ts = tb + lanes + 4u * N + (uint32_t)(h * NC), to = tb + lanes + (uint32_t)(h * NC);
    float *const mw = s.m[warp - kLtWSoft], *const fw = s.f[warp - kLtWSoft];
    const int cl = lane & (NC - 1), rl = h * NC + cl;                           // the row whose maximum the lane keeps
    const int kt = 16 * w4 + (lane >> 2), qc = 2 * (lane & 3);                  // first of the thread's tokens of a tile; first of its rows of 8
    uint32_t ns = 0;                               // tiles so far
    int nv = 0;                                    // votes so far
    bool ok = true;
    // 0: nobody says yes; 1: somebody does; 2: a wait has run out, all four warps end here
    auto vote = [&](bool x) {
      if (!ok && lane == 0) atomicMin(&s.fail[h], nv);
      const bool any = lt_any(h, x || !ok);
      const int r = !any ? 0 : (*reinterpret_cast<volatile int *>(&s.fail[h]) <= nv ? 2 : 1);
      nv++;
      return r;
    };
    for (int i = 0;; i++) {
      ok = lt_wait(&s.sched_full[i & 1], (uint32_t)(i >> 1) & 1u, p);
      if (vote(false) == 2) break;
      const LtItem it = s.item[i & 1];
      if (it.b < 0) break;
      const int rows = it.toks * p.hh;
      const int tl_l = (rl * p.magic) >> 16, head_l = it.hpart * p.hh + rl - tl_l * p.hh;
      const bool valid_l = rl < rows && head_l < a.heads;
      float m_l = -INFINITY;                       // the maximum that P is taken against
      float l[NC / 4];
#pragma unroll
      for (int n = 0; n < NC / 4; n++) l[n] = 0.f;
      if (lane < NC) mw[lane] = valid_l ? kLtUnset : -kLtUnset;   // rows of no token have no say
      __syncwarp();
      bool dead = false;
      for (int j = 0; j < it.n; j++, ns++) {
        const int tile0 = (it.j0 + j) * kLtTile, col = (tile0 + 16 * w4) >> a.page_shift;   // the warp's tokens are of one page
        const int id = col < a.max_pages ? __ldg(a.block_table + (size_t)it.b * a.max_pages + col) : -1;
        const bool held = (unsigned)id < (unsigned)a.num_pages;
        const uint32_t sb = ts + (ns & 1u) * N;
        ok = lt_wait(&s.s_full[ns & 1u], (ns >> 1) & 1u, p);
        at_fence_after();
        float v[NC / 2];
        lt_frag<NC>(sb, v);
        uint32_t seen[2] = {~0u, ~0u};             // rows that see the thread's tokens
        auto hide = [&]() {
#pragma unroll
          for (int n = 0; n < NC / 2; n++) v[n] = (seen[(n >> 1) & 1] >> (8 * (n >> 2) + qc + (n & 1))) & 1u ? v[n] : -INFINITY;
        };
        const bool masked = j >= it.m0 || !held;
        if (masked) {
          const uint64_t ones = p.hh == 64 ? ~0ull : (1ull << p.hh) - 1ull;
#pragma unroll
          for (int z = 0; z < 2; z++) {
            const int tok = tile0 + kt + 8 * z, f = tok - it.cached;
            uint64_t sees = 0;                     // whole tokens' rows
            if (held && tok < it.end) {
              if (f < 0) {
                sees = ~0ull;
              } else if (a.tree_mask) {
                for (int t = 0; t < it.toks; t++)
                  if (f < 64 && (__ldg(a.tree_mask + it.first + it.tok0 + t) >> f) & 1ull) sees |= ones << (t * p.hh);
              } else {
                const int t0 = max(0, f - it.tok0);                            // rows from this token on
                sees = t0 * p.hh >= 64 ? 0ull : ~0ull << (t0 * p.hh);
              }
            }
            seen[z] = (uint32_t)(sees >> (h * NC));
          }
          hide();
          // The products take tokens in groups of 16, up to the last that some row sees: of those that not every row sees, all 256
          // threads look at 16 bytes each, so that a few tokens at a context's end cost one look.
          const int t0 = max(0, it.all - tile0), t1 = min(kLtTile, ((it.end + 15) & ~15) - tile0);
          if (ok && j >= it.m0 && t0 < t1) {
            const uint32_t pos = 2u * ns, slot[2] = {pos % NH, (pos + 1) % NH};
            // have completed: S needed them; orders the copies before the loads
            if (mbar_try_wait(&s.kv_full[slot[0]], (pos / NH) & 1u) && mbar_try_wait(&s.kv_full[slot[1]], ((pos + 1) / NH) & 1u)) {
#pragma unroll 4
              for (int e = 64 * t0 + tid - 32 * kLtWSoft; e < 64 * t1; e += 256) {
                const int t = e >> 6, z = e & 63;  // token, 16 bytes of its latent
                uint4 *at = reinterpret_cast<uint4 *>(generic0 + (z & 32 ? slot[1] : slot[0]) * kLtHalf + ((z >> 3) & 3) * kLtChunk + t * 128 +
                                                      ((z & 7) ^ (t & 7)) * 16);
                const uint4 w = *at;
                const uint32_t g[4] = {at_nonfinite<F16>(w.x), at_nonfinite<F16>(w.y), at_nonfinite<F16>(w.z), at_nonfinite<F16>(w.w)};
                if (g[0] | g[1] | g[2] | g[3]) {
                  uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                  for (int y = 0; y < 4; y++) u[y] &= ~(((g[y] >> 15) & 0x00010001u) * 0xFFFFu);
                  *at = make_uint4(u[0], u[1], u[2], u[3]);
                  atomicOr(&s.bad[i & 1][j - it.m0][t >> 5], 1u << (t & 31));
                }
              }
            }
          }
          __syncwarp();
        }
        // v becomes c (v - m), the arguments of the exponentials: 0 at the maximum however large the scores are
        auto arguments = [&]() {
          const float2 c2 = make_float2(c, c);
          float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int n = 0; n < NC / 8; n++) {
            const float2 m = *reinterpret_cast<const float2 *>(mw + 8 * n + qc);
#pragma unroll
            for (int z = 0; z < 2; z++) {
              const float2 t = ffma2(at_add2(make_float2(v[4 * n + 2 * z], v[4 * n + 2 * z + 1]), m), c2, make_float2(0.f, 0.f));
              v[4 * n + 2 * z] = t.x;
              v[4 * n + 2 * z + 1] = t.y;
              top[z] = at_max3(top[z], t.x, t.y);
            }
          }
          return fmaxf(top[0], top[1]);
        };
        const int moved = vote(arguments() > kLtSlack);
        if (moved == 2) {
          dead = true;
          break;
        }
        if (moved) {
          lt_frag<NC>(sb, v);                      // the scores again
          hide();
#pragma unroll
          for (int n = 0; n < NC / 8; n++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
              float x = fmaxf(v[4 * n + e], v[4 * n + 2 + e]);
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
              if (lane < 4) s.wmax[h][w4][8 * n + qc + e] = x;
            }
          lt_sync(h);
          const float m1 = fmaxf(fmaxf(m_l, fmaxf(s.wmax[h][0][cl], s.wmax[h][1][cl])), fmaxf(s.wmax[h][2][cl], s.wmax[h][3][cl]));
          const float f = m1 == m_l || m_l == -INFINITY || !valid_l ? 1.f : at_exp2((m_l - m1) * c);
          m_l = m1;
          if (lane < NC) {
            mw[lane] = valid_l ? (m1 == -INFINITY ? kLtUnset : -m1) : -kLtUnset;
            fw[lane] = f;
          }
          __syncwarp();
#pragma unroll
          for (int n = 0; n < NC / 4; n++) l[n] *= fw[8 * (n >> 1) + qc + (n & 1)];
          if (j > 0) {
            ok = lt_wait(&s.pv_done[(ns - 1) & 1u], ((ns - 1) >> 1) & 1u, p) && ok;   // the products of the tile before
            at_fence_after();
#pragma unroll 1
            for (int b = 0; b < kLtBlocks; b++) {
              float o[NC];
              lt_ld(to + (uint32_t)(b * N), o);
#pragma unroll
              for (int n = 0; n < NC; n++) o[n] *= fw[n];
              lt_st(to + (uint32_t)(b * N), o);
            }
            at_wait_st();
          }
          arguments();
        }
        uint8_t *const pt = generic0 + G::kRope + (ns % NR) * kLtChunk + 2 * qc;
#pragma unroll
        for (int n = 0; n < NC / 2; n++) v[n] = at_exp2(v[n]);
#pragma unroll
        for (int n = 0; n < NC / 8; n++)
#pragma unroll
          for (int z = 0; z < 2; z++)
            *reinterpret_cast<uint32_t *>(pt + lt_p_at<N>(kt + 8 * z, h * (NC / 8) + n)) = at_pack<F16>(v[4 * n + 2 * z], v[4 * n + 2 * z + 1]);
        at_fence_async();
        at_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.p_full[ns & 1u]);
        // beside the products
#pragma unroll
        for (int n = 0; n < NC / 4; n++) l[n] += v[4 * (n >> 1) + (n & 1)] + v[4 * (n >> 1) + 2 + (n & 1)];
      }
      if (dead) break;
      // -------------------------------------------------------------- epilogue
#pragma unroll
      for (int n = 0; n < NC / 4; n++) {
        float x = l[n];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(kFull, x, o);
        if (lane < 4) s.wsum[h][w4][8 * (n >> 1) + qc + (n & 1)] = x;
      }
      if (ns > 1) ok = lt_wait(&s.pv_done[ns & 1u], ((ns - 2) >> 1) & 1u, p);
      ok = lt_wait(&s.pv_done[(ns - 1) & 1u], ((ns - 1) >> 1) & 1u, p) && ok;
      if (vote(false) == 2) break;
      const int el = 32 * w4 + lane;               // latent element of a block
      at_fence_after();
      const float l_l = (s.wsum[h][0][cl] + s.wsum[h][1][cl]) + (s.wsum[h][2][cl] + s.wsum[h][3][cl]);
      if (w4 == 0 && lane < NC && valid_l) {
        if (it.slot >= 0) p.stat[(size_t)it.slot * N + rl] = make_float2(m_l, l_l);
        else if (a.lse) a.lse[(size_t)(it.first + it.tok0 + tl_l) * a.heads + head_l] = l_l == 0.f ? -INFINITY : m_l * a.scale + logf(l_l);
      }
      if (lane < NC) fw[lane] = l_l == 0.f ? 0.f : 1.f / l_l;
      __syncwarp();
      uint32_t anybad = 0;
      const int wend = min(6, 2 * (it.n - it.m0));
#pragma unroll
      for (int w = 0; w < 6; w++)
        if (w < wend) anybad |= s.bad[i & 1][w >> 1][w & 1];
#pragma unroll 1
      for (int b = 0; b < kLtBlocks; b++) {
        float o[NC];
        lt_ld(to + (uint32_t)(b * N), o);
        if (anybad) {
          for (int w = 0; w < wend; w++)
            for (uint32_t bits = s.bad[i & 1][w >> 1][w & 1]; bits; bits &= bits - 1) {
              const int tok = (it.j0 + it.m0) * kLtTile + 32 * w + __ffs(bits) - 1, f = tok - it.cached;
              if (tok >= it.end) continue;
              const long long page = __ldg(a.block_table + (size_t)it.b * a.max_pages + (tok >> a.page_shift));
              const long long at = ((page << a.page_shift) + (tok & ((1 << a.page_shift) - 1))) * kLatRow + 128 * b + el;
              if (isfinite(at_value<F16>(__ldg(a.cache + at)))) continue;
#pragma unroll
              for (int n = 0; n < NC; n++) {
                const int tl = ((h * NC + n) * p.magic) >> 16;
                if (tl >= it.toks) continue;
                const bool sees = f < 0 || (a.tree_mask ? f < 64 && (__ldg(a.tree_mask + it.first + it.tok0 + tl) >> f) & 1ull
                                                        : f <= it.tok0 + tl);
                if (sees) o[n] = __int_as_float(0x7FFFFFFF);
              }
            }
          __syncwarp();
        }
        if (it.slot >= 0) {
          float *part = p.part + ((size_t)it.slot * N + h * NC) * kLatDim + 128 * b + el;
#pragma unroll
          for (int n = 0; n < NC; n++)
            if (h * NC + n < rows) part[(size_t)n * kLatDim] = o[n];
        } else {
          // lanes are neighbouring elements: of two rows an even lane stores a pair of the first and an odd one of the second
#pragma unroll
          for (int n = 0; n < NC; n += 2) {
            const float x = o[n] * fw[n], y = o[n + 1] * fw[n + 1];
            const float got = __shfl_xor_sync(kFull, lane & 1 ? x : y, 1);
            const uint32_t w = lane & 1 ? at_pack<F16>(got, y) : at_pack<F16>(x, got);
            const int r = h * NC + n + (lane & 1), tl = (r * p.magic) >> 16, head = it.hpart * p.hh + r - tl * p.hh;
            if (r < rows && head < a.heads)
              *reinterpret_cast<uint32_t *>(a.out.p + (long long)(it.first + it.tok0 + tl) * a.out.row + (long long)head * a.out.head + 128 * b +
                                            (el & ~1)) = w;
          }
          __syncwarp();
        }
      }
      at_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.sched_empty[i & 1]);
    }
  } else if (warp == kLtWTma) {
    // ---------------------------------------------------------- items and tiles
    const int box = min(a.page_shift, 6), np = kLtTile >> box, pg = lane & (np - 1), part = lane >> (6 - box);   // copies of 2^box tokens, 64 elements
    const uint32_t place = (uint32_t)pg << (box + 7);
    uint32_t pos = 0, tiles = 0;                   // halves and tiles so far
    LtCursor cur;
    if (lane == 0 && !p.whole) p.desc[2 * blockIdx.x + 1] = make_int4(0, -1, 0, 0);   // nothing to join, unless the cursor finds it
    cur.find(p, *reinterpret_cast<LtSetup *>(generic0), lo, hi, held0);
    at_fence_async();                              // copies come where the requests' tiles were counted
    __syncwarp();
    long long next = cur.share.x0;
    bool ok = true;
    for (int i = 0; ok; i++) {
      LtItem it;
      it.b = -1;
      while (next < cur.share.x1) {
        next = cur.part(p, next, it);
        if (it.n > 0) break;
        it.b = -1;
      }
      if (i >= 2 && !lt_wait(&s.sched_empty[i & 1], (uint32_t)((i >> 1) - 1) & 1u, p)) break;
      if (lane < 6) s.bad[i & 1][lane >> 1][lane & 1] = 0u;
      __syncwarp();
      if (lane == 0) {
        s.item[i & 1] = it;
        mbar_arrive(&s.sched_full[i & 1]);
      }
      if (it.b < 0) break;
      const int32_t *table = a.block_table + (size_t)it.b * a.max_pages;
      auto page_row = [&](int j) {                 // the cache row of the lane's copy; past the end: reads zeros
        const int tok = (it.j0 + j) * kLtTile + (pg << box), col = tok >> a.page_shift;
        const int id = col < a.max_pages ? __ldg(table + col) : -1;
        return (unsigned)id < (unsigned)a.num_pages ? (id << a.page_shift) + (tok & ((1 << a.page_shift) - 1)) : a.num_pages << a.page_shift;
      };
      int row = page_row(0);
      for (int j = 0; j < it.n && ok; j++, tiles++) {
        const int ahead = j + 1 < it.n ? page_row(j + 1) : 0;
        for (int z = 0; z < 2; z++, pos++) {
          const uint32_t slot = pos % NH, to = smem0 + slot * kLtHalf + place;
          if (pos >= NH) ok = lt_wait(&s.kv_empty[slot], (pos / NH - 1) & 1u, p);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&s.kv_full[slot], (uint32_t)(kLtHalf + (z ? kLtChunk : 0)) + a.stall);
          __syncwarp();
          for (int e = part; e < 4 + z; e += 32 >> (6 - box))   // the second half's fifth is the key part
            lt_tma_2d(e < 4 ? to + (uint32_t)(e * kLtChunk) : smem0 + G::kRope + (tiles % NR) * kLtChunk + place, &p.cmap, 256 * z + 64 * e, row,
                      &s.kv_full[slot]);
        }
        if (!ok) break;
        if (j == 0) cur.describe(p, it);
        row = ahead;
      }
    }
    // copies in flight land before the CTA ends; nothing else may pass these barriers now
    for (uint32_t q = pos > NH ? pos - NH : 0; q < pos; q++) mbar_wait_bounded(&s.kv_full[q % NH], (q / NH) & 1u, a.wait_ns);
    __syncwarp();
  } else if (warp == kLtWS || warp == kLtWO) {
    // ---------------------------------------------------------- MMA issue
    // The whole warp goes through the loop, so that descriptors stay in uniform registers; one elected lane issues.
    const uint32_t tu = __shfl_sync(kFull, tb, 0);
    bool ok = true;
    // the lanes go on or end together
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      ok = __all_sync(kFull, ok && mbar_wait_bounded(bar, parity, a.wait_ns));
      if (!ok && lane == 0) atomicOr(p.ctrl + kAttnCtrlFlags, MOE_FLAG_TIMEOUT);
      at_fence_after();
    };
    if (warp == kLtWS) {
      constexpr uint32_t id_s = lt_idesc_s(F16, N);
      const uint64_t dq0 = at_desc(smem0 + G::kQ, 16), dr0 = at_desc(smem0 + G::kRope, 16), dk0 = at_desc(smem0, 16);
      uint32_t slot = 0, phase = 0, part = 0, t = 0;   // the next half's slot and phase, the tile's key part, tiles so far
      for (int i = 0; ok; i++) {
        wait(&s.sched_full[i & 1], (uint32_t)(i >> 1) & 1u);
        if (!ok) break;
        const LtItem &im = s.item[i & 1];
        if (__shfl_sync(kFull, im.b, 0) < 0) break;
        const int n = __shfl_sync(kFull, im.n, 0);
        wait(&s.q_full, (uint32_t)i & 1u);
        for (int j = 0; j < n && ok; j++, t++) {
          const uint32_t d = tu + 4u * N + (t & 1u) * N;
          if (t >= 2) wait(&s.p_full[t & 1u], ((t >> 1) - 1) & 1u);      // the scores of tile t - 2 have been read
#pragma unroll 1
          for (uint32_t z = 0; z < 2 && ok; z++) {
            wait(&s.kv_full[slot], phase);
            if (!ok) break;
            if (at_elect()) {
              uint64_t da = dk0 + (uint64_t)(slot * (kLtHalf >> 4)), db = dq0 + (uint64_t)(z * (4 * G::kQChunk >> 4));
              uint32_t acc = z;
#pragma unroll 1
              for (int e = 0; e < 4; e++) {
#pragma unroll
                for (int k = 0; k < 4; k++) {
                  at_mma_ss(d, da + (uint64_t)(2 * k), db + (uint64_t)(2 * k), id_s, acc);
                  acc = 1u;
                }
                da += (uint64_t)(kLtChunk >> 4);
                db += (uint64_t)(G::kQChunk >> 4);
              }
              if (z) {
                const uint64_t dr = dr0 + (uint64_t)(part * (kLtChunk >> 4));
#pragma unroll
                for (int k = 0; k < 4; k++) at_mma_ss(d, dr + (uint64_t)(2 * k), db + (uint64_t)(2 * k), id_s, 1u);
                at_commit(&s.s_full[t & 1u]);
                if (j + 1 == n) at_commit(&s.q_empty);
              }
            }
            __syncwarp();
            if (++slot == NH) {
              slot = 0;
              phase ^= 1u;
            }
          }
          part = part + 1 == NR ? 0 : part + 1;
        }
        if (lane == 0) mbar_arrive(&s.sched_empty[i & 1]);
      }
    } else {
      constexpr uint32_t id_o = lt_idesc_o(F16, N);
      const uint64_t dv0 = at_desc(smem0, kLtChunk), dp0 = lt_desc_p<N>(smem0 + G::kRope);
      uint32_t slot = 0, part = 0, t = 0;              // of the tile: its first half's slot, its key part; tiles so far
      for (int i = 0; ok; i++) {
        wait(&s.sched_full[i & 1], (uint32_t)(i >> 1) & 1u);
        if (!ok) break;
        const LtItem &im = s.item[i & 1];
        if (__shfl_sync(kFull, im.b, 0) < 0) break;
        const int n = __shfl_sync(kFull, im.n, 0), end = __shfl_sync(kFull, im.end - im.j0 * kLtTile, 0);
        for (int j = 0; j < n && ok; j++, t++) {
          // groups of 16 tokens up to the last that some row sees
          const int left = end - j * kLtTile, steps = left >= kLtTile ? kLtTile / 16 : (left + 15) >> 4;
          wait(&s.p_full[t & 1u], (t >> 1) & 1u);
          if (!ok) break;
          if (at_elect()) {
            const uint64_t dp = dp0 + (uint64_t)(part * (kLtChunk >> 4));
            const uint32_t add = j > 0;
            uint32_t sl = slot;
#pragma unroll 1
            for (int b = 0; b < kLtBlocks; b++) {
              const uint64_t da = dv0 + (uint64_t)(sl * (kLtHalf >> 4) + (b & 1) * (kLtPair >> 4));
#pragma unroll
              for (int k = 0; k < kLtTile / 16; k++)
                if (k < steps) at_mma_ss(tu + (uint32_t)(b * N), da + (uint64_t)(128u * k), dp + (uint64_t)(2u * N * k), id_o, k > 0 ? 1u : add);
              if (b & 1) {
                at_commit(&s.kv_empty[sl]);
                sl = sl + 1 == NH ? 0 : sl + 1;
              }
            }
            at_commit(&s.pv_done[t & 1u]);
          }
          __syncwarp();
          slot = slot + 2 >= NH ? slot + 2 - NH : slot + 2;
          part = part + 1 == NR ? 0 : part + 1;
        }
        if (lane == 0) mbar_arrive(&s.sched_empty[i & 1]);
      }
    }
    // every MMA issued has completed before tensor memory is released
    if (at_elect()) at_commit(&s.drain);
    mbar_wait_bounded(&s.drain, 0u, a.wait_ns);
    __syncwarp();
  } else if (warp == kLtWQ) {
    // ---------------------------------------------------------- Q rows
    int nq = 0;
    for (int i = 0;; i++) {
      if (!lt_wait(&s.sched_full[i & 1], (uint32_t)(i >> 1) & 1u, p)) break;
      const LtItem it = s.item[i & 1];
      if (it.b < 0) break;
      if (i > 0 && !lt_wait(&s.q_empty, (uint32_t)(i - 1) & 1u, p)) break;
      // a box (64, hh, per): rows past the item's tokens are others' or zeros, and are not stored
      if (lane == 0) mbar_arrive_expect_tx(&s.q_full, (uint32_t)(9 * 128 * p.hh * p.per));
      __syncwarp();
      if (lane < 9)
        at_tma_3d(smem0 + G::kQ + (uint32_t)(lane * G::kQChunk), lane < 8 ? &p.qmap : &p.rmap, lane < 8 ? 64 * lane : 0, it.hpart * p.hh,
                  it.first + it.tok0, &s.q_full);
      nq++;
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.sched_empty[i & 1]);
    }
    if (nq > 0) mbar_wait_bounded(&s.q_full, (uint32_t)(nq - 1) & 1u, a.wait_ns);   // a copy in flight lands before the CTA ends
    __syncwarp();
  }
  at_fence_before();
  __syncthreads();
  if (warp == kLtWS) {
    at_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tb), "r"(512) : "memory");
  }
}

// Joins the parts of the items that several CTAs took: o = sum_k 2^(c (m_k - m)) O_k / sum_k 2^(c (m_k - m)) l_k.  128
// threads have a row, four elements each.  Of items of up to 8 parts a CTA takes four rows at once, a fourth of its threads one each;
// of items of more parts one row at a time, the fourths of the threads every fourth part, summed up in
// that order at the end.  Latency bounds it: the parts lie in L2, and four loads of a thread wait together.
constexpr int kLtJoinFew = 8;
struct LtSum {
  float top, sum;
  float4 acc;
  // parts k0, k0 + step, ... c1 of row r
  template <int N>
  __device__ __forceinline__ void add(const LtArgs &p, int4 d1, int k0, int step, int r, int d4, float c) {
    for (; k0 <= d1.y; k0 += 4 * step) {
      float2 st[4];
      float4 u[4];
      float t1 = top;
#pragma unroll
      for (int z = 0; z < 4; z++) {
        const int k = k0 + step * z;
        const size_t slot = k == d1.x ? d1.z : 2 * (k * p.gang + d1.w);
        st[z] = make_float2(-INFINITY, 0.f);
        u[z] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k <= d1.y) {
          st[z] = __ldcg(p.stat + slot * N + r);
          u[z] = __ldcg(reinterpret_cast<const float4 *>(p.part + (slot * N + r) * kLatDim) + d4);
        }
      }
#pragma unroll
      for (int z = 0; z < 4; z++) t1 = fmaxf(t1, st[z].x);
      const float f0 = top == t1 ? 1.f : at_exp2((top - t1) * c);
      top = t1;
      sum *= f0;
      acc.x *= f0;
      acc.y *= f0;
      acc.z *= f0;
      acc.w *= f0;
#pragma unroll
      for (int z = 0; z < 4; z++) one(st[z], u[z], c);
    }
  }
  // a part whose maximum is not above `top`
  __device__ __forceinline__ void one(float2 st, float4 u, float c) {
    if (st.x == -INFINITY && st.y == 0.f) {        // no weight there: u is 0, or NaN by an infinite element of a latent
      acc = make_float4(acc.x + u.x, acc.y + u.y, acc.z + u.z, acc.w + u.w);
      return;
    }
    const float f = st.x == top ? 1.f : at_exp2((st.x - top) * c);
    sum = fmaf(st.y, f, sum);
    acc.x = fmaf(u.x, f, acc.x);
    acc.y = fmaf(u.y, f, acc.y);
    acc.z = fmaf(u.z, f, acc.z);
    acc.w = fmaf(u.w, f, acc.w);
  }
};

template <int N, bool F16>
__global__ void __launch_bounds__(512) lat_join_kernel(const __grid_constant__ LtArgs p, int ctas) {
  __shared__ unsigned masks[kLtMaxSms / 32];
  __shared__ float4 acc4[4][128];
  __shared__ float2 stat4[4];
  const LatArgs &a = p.a;
  const int tid = threadIdx.x, words = (ctas + 31) / 32, d4 = tid & 127, sg = tid >> 7;
  pdl_wait();
  for (int k = tid; k < 32 * words; k += 512) {
    const unsigned mask = __ballot_sync(kFull, k < ctas && __ldcg(&p.desc[2 * k + 1].y) >= 0);
    if ((tid & 31) == 0) masks[k >> 5] = mask;
  }
  __syncthreads();
  int count = 0;
  for (int w = 0; w < words; w++) count += __popc(masks[w]);
  const float c = a.scale * 1.44269504088896340736f;
  const int quads = count * (N / 4);
  for (int unit = blockIdx.x; unit < 4 * quads; unit += gridDim.x) {
    const int rr = unit / quads, quad = unit - rr * quads;
    int left = quad / (N / 4), w = 0;              // the item: the left-th set bit
    while (left >= __popc(masks[w])) left -= __popc(masks[w++]);
    unsigned bits = masks[w];
    for (; left > 0; left--) bits &= bits - 1;
    const int which = 32 * w + __ffs(bits) - 1;
    const int4 d0 = __ldcg(p.desc + 2 * which), d1 = __ldcg(p.desc + 2 * which + 1);
    const bool few = d1.y - d1.x < kLtJoinFew;
    if (few && rr > 0) continue;
    const int r = 4 * (quad % (N / 4)) + (few ? sg : rr), tl = (r * p.magic) >> 16, head = d0.y * p.hh + r - tl * p.hh;
    const bool valid = tl < p.per && tl < d0.w && head < a.heads;
    LtSum t = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    if (valid) t.add<N>(p, d1, few ? d1.x : d1.x + sg, few ? 1 : 4, r, d4, c);
    if (!few) {
      acc4[sg][d4] = t.acc;
      if (d4 == 0) stat4[sg] = make_float2(t.top, t.sum);
      __syncthreads();
      t = {fmaxf(fmaxf(stat4[0].x, stat4[1].x), fmaxf(stat4[2].x, stat4[3].x)), 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll
      for (int z = 0; z < 4; z++) t.one(stat4[z], acc4[z][d4], c);
      __syncthreads();
    }
    if (valid && (few || sg == 0)) {
      const float inv = t.sum == 0.f ? 0.f : 1.f / t.sum;
      const long long row = d0.x + d0.z + tl;
      *reinterpret_cast<uint2 *>(a.out.p + row * a.out.row + (long long)head * a.out.head + 4 * d4) =
          make_uint2(at_pack<F16>(t.acc.x * inv, t.acc.y * inv), at_pack<F16>(t.acc.z * inv, t.acc.w * inv));
      if (a.lse && d4 == 0) a.lse[row * a.heads + head] = t.sum == 0.f ? -INFINITY : t.top * a.scale + logf(t.sum);
    }
  }
}

namespace {
typedef void (*LtKernel)(const LtArgs);
typedef void (*LtJoin)(const LtArgs, int);
LtKernel lt_kernel(int n, int f16) {
  if (n == 16) return f16 ? lat_tree_kernel<16, true> : lat_tree_kernel<16, false>;
  if (n == 32) return f16 ? lat_tree_kernel<32, true> : lat_tree_kernel<32, false>;
  return f16 ? lat_tree_kernel<64, true> : lat_tree_kernel<64, false>;
}
LtJoin lt_join(int n, int f16) {
  if (n == 16) return f16 ? lat_join_kernel<16, true> : lat_join_kernel<16, false>;
  if (n == 32) return f16 ? lat_join_kernel<32, true> : lat_join_kernel<32, false>;
  return f16 ? lat_join_kernel<64, true> : lat_join_kernel<64, false>;
}
int lt_smem(int n) { return n == 16 ? LtGeom<16>::kSmem : (n == 32 ? LtGeom<32>::kSmem : LtGeom<64>::kSmem); }

cudaError_t lt_encode(CUtensorMap *map, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides, const cuuint32_t *box,
                      int f16) {
  const AttnMapEncodeFn enc = attn_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult e = enc(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void *>(base),
                         dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return e == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}
cudaError_t lt_encode_rows(CUtensorMap *map, const RowView &r, int dim, const LtArgs &p) {
  const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)p.a.heads, (cuuint64_t)p.a.T};
  const cuuint64_t strides[2] = {(cuuint64_t)r.head * 2, (cuuint64_t)r.row * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)p.hh, (cuuint32_t)p.per};
  return lt_encode(map, r.p, 3, dims, strides, box, p.a.f16);
}
}  // namespace

cudaError_t lat_tree_setup(int f16) {
  for (const int n : {16, 32, 64}) {
    const cudaError_t err = cudaFuncSetAttribute(lt_kernel(n, f16), cudaFuncAttributeMaxDynamicSharedMemorySize, lt_smem(n));
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

LatWs lat_ws(int num_sms) {
  LatWs w;
  size_t off = kAttnCtrlBytes;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = (off + bytes + 255) / 256 * 256;
    return at;
  };
  w.desc = take(32 * (size_t)num_sms);
  w.stat = take(8 * (size_t)(2 * num_sms) * kLtRows);
  w.part = take(4 * (size_t)(2 * num_sms) * kLtRows * kLatDim);
  w.total = off;
  return w;
}

cudaError_t launch_lat_tree(const LatArgs &a, uint8_t *ws, int num_sms, cudaStream_t stream) {
  LtArgs p;
  memset(&p, 0, sizeof(p));
  const LatWs w = lat_ws(num_sms);
  p.a = a;
  p.ctrl = reinterpret_cast<int *>(ws);
  p.desc = reinterpret_cast<int4 *>(ws + w.desc);
  p.stat = reinterpret_cast<float2 *>(ws + w.stat);
  p.part = reinterpret_cast<float *>(ws + w.part);
  p.hp = a.heads > kLtRows ? 2 : 1;
  p.hh = (a.heads + p.hp - 1) / p.hp;
  p.magic = (65536 + p.hh - 1) / p.hh;
  // room for the mean request's tokens, if there is
  const int mean = (int)(((long long)a.T + a.B - 1) / a.B), most = kLtRows / p.hh, rows = p.hh * (mean < most ? mean : most);
  const int n = rows <= 16 ? 16 : (rows <= 32 ? 32 : 64);
  p.per = n / p.hh;
  p.gang = p.hp == 2 || mean > p.per ? 2 : 1;
  if (num_sms > kLtMaxSms) num_sms = kLtMaxSms;
  const int grid = p.gang == 2 ? (num_sms < 2 ? 2 : num_sms & ~1) : num_sms;
  p.slack = 3 + n / 32;
  // Items stay whole where that costs less than parts and their join: in tiles' time (1.25 us) 2.4, and the parts' way
  // through L2, up to 4 for one of 64 rows on every SM and twice that where a CTA has several items.  It costs, where every item
  // has a CTA, the tiles of the longest above a CTA's share (the longest is what the block table has room for, the mean
  // taken to be 0.6 of it); else half of an item at the end, a fifth where a CTA has many.  us whole and cut:
  //   1 row of 16 heads at 120 tokens 10.1, 11.6, at 250 13.1, 11.4; 64 requests of up to 250 13.9, 16.3, of up to 500 20.0, 18.5
  //   64 heads, 64 requests of up to 500 24.5, 30.8, of up to 1000 36.9, 33.8; 512 of up to 2000 156, 181, of up to 4000 283, 268
  //   8 trees of 8 and 64 heads at up to 250 18.0, 20.6, at up to 500 24.4, 22.2; 64 of them at up to 2000 93, 110, 4000 186, 149
  // These tables were as wide as the longest context.  The rule knows the call's sizes only, the lengths are on the device: a table
  // of capacity counts as long contexts, whose items are cut, at the second figure of each pair.
  const double places = grid / p.gang, tiles = (double)(((long long)a.max_pages << a.page_shift) + kLtTile - 1) / kLtTile;
  const double items = (double)a.B * ((p.hp * ((mean + p.per - 1) / p.per) + p.gang - 1) / p.gang);
  const double share = 0.6 * items * tiles / places, parts = items > places ? 2 : (items * tiles < places ? items * tiles / places : 1);
  p.whole = (items > places ? (items > 2 * places ? 0.2 : 0.5) * tiles : tiles - (share > 1 ? share : 1)) <= 2.4 + 4 * (n / 64.) * parts;
  const cuuint64_t cdims[2] = {(cuuint64_t)kLatRow, (cuuint64_t)a.num_pages << a.page_shift};
  const cuuint64_t cstride[1] = {2 * kLatRow};
  const cuuint32_t cbox[2] = {64, (cuuint32_t)(a.page_shift < 6 ? 1 << a.page_shift : kLtTile)};
  cudaError_t err = lt_encode(&p.cmap, a.cache, 2, cdims, cstride, cbox, a.f16);
  if (err == cudaSuccess) err = lt_encode_rows(&p.qmap, a.q, kLatDim, p);
  if (err == cudaSuccess) err = lt_encode_rows(&p.rmap, a.q_rope, kLatRope, p);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kLtThreads);
  cfg.dynamicSmemBytes = (size_t)lt_smem(n);
  if ((err = cudaLaunchKernelEx(&cfg, lt_kernel(n, a.f16), p)) != cudaSuccess || p.whole) return err;
  cfg.gridDim = dim3((unsigned)(4 * num_sms));
  cfg.blockDim = dim3(512);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, lt_join(n, a.f16), p, grid);
}

}  // namespace moe
