// kv_cache.cu -- the paged key/value cache's bookkeeping (moe_kv_plan) and the
// writing of its rows (moe_kv_append).
#include "attn.h"
#include "gemv_core.cuh"

namespace moe {

constexpr int kPlanThreads = 256;
constexpr int kPlanMaxRequests = MOE_ATTN_MAX_REQUESTS;
constexpr int kPlanTree = MOE_ATTN_MAX_TREE;

struct KvPlanSmem {
  int cu[kPlanMaxRequests + 1];      // row offsets
  int first[kPlanMaxRequests + 1];   // new pages of the requests before
  int cached[kPlanMaxRequests];
  int wsum[2][kPlanThreads / 32];
  int top[kPlanThreads / 32];        // longest context
  int flags;
  int8_t parent[kPlanThreads + kPlanTree];
};

// Largest b of 0 .. n - 1 with first[b] <= x (first ascending, first[0] <= x).
__device__ __forceinline__ int last_at_most(const int *first, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// need = ceil((cached + fresh) / page), have = ceil(cached / page) pages per
// request; exclusive sums of the fresh rows (cu) and of need - have (the place
// of a request's first new page in the free list) over the requests.  Every
// CTA computes the same sums from the B lengths (at most 8 KB, in L2 after the
// first CTA's read) so that no second launch or grid barrier is needed, then
// takes kPlanThreads rows and its share of the new table entries.  The work
// is a chain of three dependent loads (lengths; a page id; the store), so
// launch latency bounds it; tree parents are staged in shared memory because
// walking them in global memory would add one load latency per tree level.
// 7 requests of drafted trees: 3.4 us; 48 prompts (31190 rows): 3.1 us.
__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const KvPlanArgs a) {
  __shared__ KvPlanSmem s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int page = 1 << a.page_shift;
  if (tid == 0) s.flags = 0;
  __syncthreads();
  int rows = 0, pages = 0, top = 0, bad = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int c = 0, f = 0;
    if (b < a.B) {
      c = __ldg(a.cached + b);
      f = __ldg(a.fresh + b);
      if (c < 0 || f < 0) bad |= MOE_KV_FLAG_LENGTH;
      c = min(max(c, 0), 1 << 30);
      f = min(max(f, 0), a.T);                          // no sum below passes 2^31: B * T is bounded by the host
      if (((long long)c + f + page - 1) >> a.page_shift > a.max_pages) bad |= MOE_KV_FLAG_TABLE;
      if (a.parents && f > kPlanTree) bad |= MOE_KV_FLAG_TREE;
    }
    const int need = min((c + f + page - 1) >> a.page_shift, a.max_pages);
    const int have = min((c + page - 1) >> a.page_shift, need);
    top = max(top, c + f);
    int v[2] = {f, need - have}, incl[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
      incl[i] = v[i];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(kFull, incl[i], o);
        if (lane >= o) incl[i] += t;
      }
      if (lane == 31) s.wsum[i][warp] = incl[i];
    }
    __syncthreads();
    int before[2] = {rows, pages};
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; w++) {
#pragma unroll
      for (int i = 0; i < 2; i++) before[i] += w < warp ? s.wsum[i][w] : 0;
      rows += s.wsum[0][w];
      pages += s.wsum[1][w];
    }
    if (b < a.B) {
      s.cu[b] = before[0] + incl[0] - v[0];
      s.first[b] = before[1] + incl[1] - v[1];
      s.cached[b] = c;
    }
    __syncthreads();
  }
  if (tid == 0) {
    s.cu[a.B] = rows;
    s.first[a.B] = pages;
  }
  if (rows > a.T) bad |= MOE_KV_FLAG_LENGTH;
  __syncthreads();

  // this CTA's rows
  const int t0 = blockIdx.x * kPlanThreads, t = t0 + tid;
  if (a.parents) {
    for (int i = tid; i < kPlanThreads + kPlanTree; i += kPlanThreads) {
      const int r = t0 - kPlanTree + i;
      const int p = r >= 0 && r < a.T ? __ldg(a.parents + r) : -1;
      s.parent[i] = (int8_t)(p < -1 || p >= kPlanTree ? kPlanTree : p);    // kPlanTree: not a row of a tree
    }
    __syncthreads();
  }
  if (t < a.T) {
    int slot = -1, pos = -1;
    uint64_t word = 0;
    if (t < rows) {
      const int b = last_at_most(s.cu, a.B, t), local = t - s.cu[b], c = s.cached[b];
      const int place = c + local, col = place >> a.page_shift, have = (c + page - 1) >> a.page_shift;
      pos = place;
      if (col < a.max_pages) {
        const int at = s.first[b] + col - have;
        const int id = col < have ? __ldg(a.block_table + (size_t)b * a.max_pages + col)
                                  : (at < a.num_free ? __ldg(a.free_pages + at) : -1);
        if ((unsigned)id < (unsigned)a.num_pages) slot = (id << a.page_shift) + (place & (page - 1));
        else bad |= MOE_KV_FLAG_PAGES;
      }
      if (a.parents) {
        // the path to the context, from the row down: parents are earlier
        // rows, so the walk ends after at most 64 steps
        int i = local, depth = 0;
        if (local < kPlanTree) {
          word = 1ull << i;
          for (;;) {
            const int p = s.parent[tid + kPlanTree - local + i];
            if (p == -1) break;
            if (p >= i) {                               // not an earlier row: the path ends here
              bad |= MOE_KV_FLAG_TREE;
              break;
            }
            i = p;
            word |= 1ull << i;
            depth++;
          }
        }
        pos = c + depth;
      }
    }
    a.slots[t] = slot;
    a.positions[t] = pos;
    if (a.tree_mask) a.tree_mask[t] = word;
  }
  // this CTA's share of the new table entries
  for (int i = t; i < pages; i += gridDim.x * kPlanThreads) {
    const int b = last_at_most(s.first, a.B, i);
    const int col = ((s.cached[b] + page - 1) >> a.page_shift) + i - s.first[b];
    const int id = i < a.num_free ? __ldg(a.free_pages + i) : -1;
    const bool ok = (unsigned)id < (unsigned)a.num_pages;
    if (!ok) bad |= MOE_KV_FLAG_PAGES;
    a.block_table[(size_t)b * a.max_pages + col] = ok ? id : -1;
  }
  if (blockIdx.x == 0) {
    for (int b = tid; b <= a.B; b += kPlanThreads) a.cu[b] = s.cu[b];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
    if (lane == 0) s.top[warp] = top;
  }
  if (bad) atomicOr(&s.flags, bad);
  __syncthreads();
  if (tid == 0) {
    if (s.flags) atomicOr(a.info + 3, s.flags);
    if (blockIdx.x == 0) {
      for (int w = 1; w < kPlanThreads / 32; w++) top = max(top, s.top[w]);
      a.info[0] = rows;
      a.info[1] = min(pages, a.num_free);
      a.info[2] = top;
    }
  }
}

cudaError_t launch_kv_plan(const KvPlanArgs &a, cudaStream_t stream) {
  int grid = (a.T + kPlanThreads - 1) / kPlanThreads;
  if (grid < 1) grid = 1;
  kv_plan_kernel<<<grid, kPlanThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

// One thread per 16 bytes of a row's keys and values: both sides of every copy are
// whole 128-byte lines whatever the slots' order, and HBM bounds it: 16384 rows of
// 8 heads of 128 take 19.8 us, 6.8 TB/s (a plain copy has 6.8); 56 rows 2.0 us, a
// launch.
__global__ void __launch_bounds__(256) kv_append_kernel(const KvAppendArgs a) {
  const int chunks = a.head_dim / 8, per_row = a.kv_heads * chunks;
  const long long n = (long long)a.T * per_row;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < n; i += gridDim.x * 256LL) {
    const int t = (int)(i / per_row), r = (int)(i - (long long)t * per_row), h = r / chunks, c = r - h * chunks;
    const int slot = __ldg(a.slots + t);
    if ((unsigned)slot >= (unsigned)a.num_slots) continue;
    const long long pg = slot >> a.page_shift, place = slot & ((1 << a.page_shift) - 1);
    const long long dst = (((pg * a.kv_heads + h) << a.page_shift) + place) * a.head_dim + 8 * c;
    *reinterpret_cast<uint4 *>(a.k_cache + dst) =
        __ldg(reinterpret_cast<const uint4 *>(a.k.p + t * a.k.row + h * a.k.head + 8 * c));
    *reinterpret_cast<uint4 *>(a.v_cache + dst) =
        __ldg(reinterpret_cast<const uint4 *>(a.v.p + t * a.v.row + h * a.v.head + 8 * c));
  }
}

cudaError_t launch_kv_append(const KvAppendArgs &a, int num_sms, cudaStream_t stream) {
  const long long n = (long long)a.T * a.kv_heads * (a.head_dim / 8);
  long long grid = (n + 255) / 256;
  if (grid > 16LL * num_sms) grid = 16LL * num_sms;
  kv_append_kernel<<<(unsigned)grid, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace moe
