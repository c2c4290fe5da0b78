// The pages of a paged K/V cache: grown, shared, freed and compacted, on the
// device and without a host copy of the tables.
//
// The state of a pool is refs[num_blocks], how many table entries hold each
// page (free: <= 0), next to the block tables and lengths that the attention
// calls read.  Freeing and sharing then only add to refs, in any order, with
// the same result; growing and compacting find free pages by a scan of refs
// (4 bytes a page, against the thousands of bytes a page holds), lowest ids
// first, so that they too give the same result in every run.
//
// * extend_plan_kernel: one cluster of two CTAs or more.  Its first sums up what
//   each request needs (a prefix sum over the requests), the others count the free
//   pages of their part of refs; after the cluster's barrier each hands the free
//   pages of its part, which are consecutive in rank, to the requests that those
//   ranks belong to.  page_copy_kernel then copies the shared, partly filled pages
//   that a request appends to (copy on write), in every cache.
// * compact_plan_kernel: one cluster.  Pages past the number of live ones move
//   to the free ids before it, both in ascending order; compact_move_kernel
//   moves their rows in every cache, their refs, and rewrites the tables.
// * fork_kernel, trim_kernel: a CTA per row.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "../../include/mvp.h"
#include "mvp_internal.cuh"
#include "ptx.cuh"

namespace mvp {

namespace {

constexpr int kMaxCaches = 256;
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kTile = 4 * kPlanThreads;  // pages of one step of a scan of refs: four per thread
constexpr int kCopyThreads = 256;
constexpr int kCopyChunks = 4;  // 16-byte chunks in flight per thread
constexpr int kCopyBytes = kCopyThreads * kCopyChunks * 16;
constexpr size_t kPagesHeader = 256;
constexpr unsigned kWarp = 0xffffffffu;

struct Caches {
  unsigned char* at[kMaxCaches];
  int n;
  long long row_bytes;   // of one token
  long long page_bytes;  // block_size rows
};

// Exclusive prefix sum over the CTA's threads, and the sum.
template <class T>
__device__ __forceinline__ T block_scan(T v, T* warp_sums, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(kWarp, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  T s = lane < kPlanWarps ? warp_sums[lane] : T(0);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(kWarp, s, o);
    if (lane >= o) s += y;
  }
  total = __shfl_sync(kWarp, s, 31);
  const T before = __shfl_sync(kWarp, s, (warp + 31) & 31);
  __syncthreads();  // warp_sums is free again
  return (warp > 0 ? before : T(0)) + x - v;
}

template <class T>
__device__ __forceinline__ T block_sum(T v, T* warp_sums) {
  T total;
  (void)block_scan(v, warp_sums, total);
  return total;
}

// refs of four consecutive pages, 1 (held) past the pool's end.
__device__ __forceinline__ int4 refs_of(const int32_t* refs, long long i, int num_blocks) {
  if (i + 3 < num_blocks && (reinterpret_cast<uintptr_t>(refs) & 15u) == 0) return *reinterpret_cast<const int4*>(refs + i);
  int4 r = make_int4(1, 1, 1, 1);
  if (i < num_blocks) r.x = refs[i];
  if (i + 1 < num_blocks) r.y = refs[i + 1];
  if (i + 2 < num_blocks) r.z = refs[i + 2];
  if (i + 3 < num_blocks) r.w = refs[i + 3];
  return r;
}
__device__ __forceinline__ int free_of(int4 r) { return (r.x <= 0) + (r.y <= 0) + (r.z <= 0) + (r.w <= 0); }

// This CTA's part of the pool: whole tiles.
__device__ __forceinline__ void part_of(int num_blocks, int rank, int ctas, long long& lo, long long& hi) {
  const long long tiles = (static_cast<long long>(num_blocks) + kTile - 1) / kTile;
  lo = tiles * rank / ctas * kTile;
  hi = tiles * (rank + 1) / ctas * kTile;
}

// Pages that n keys take.
__device__ __forceinline__ int pages_of(long long n, int shift) {
  return static_cast<int>((n + (1LL << shift) - 1) >> shift);
}

// ------------------------------------------------------------------ extend
// A request's part of the plan, and a page to copy.
struct ExtendRequest {
  int base;   // rank of its first new page among the call's
  int start;  // column of its table that takes it
  int cow;    // index of its page copy, or -1
};
struct PageCopy {
  int src, dst, rows;
};

struct ExtendParams {
  int32_t* refs;
  int32_t* bt;
  const int32_t* lens;
  const int32_t* add;
  int32_t* new_lens;
  int32_t* missing;
  int* n_copies;           // workspace
  ExtendRequest* reqs;     // [num_reqs]
  PageCopy* copies;        // [num_reqs]
  int num_blocks, num_reqs, max_blocks, shift;
};

// The last of n bases that is at most k.
template <class Base>
__device__ __forceinline__ int last_at_most(const Base& base, int n, long long k) {
  int b = 0;
  while (n > 1) {
    const int half = n >> 1;
    if (base(b + half) <= k) {
      b += half;
      n -= half;
    } else {
      n = half;
    }
  }
  return b;
}

// Bound by latency: four dependent loads (lengths, table, refs, refs again) and
// the barriers between them.  256 requests, 131072 pages: 10 us with eight CTAs;
// 15 with the bases searched in global memory and the first CTA counting too.
__global__ void __launch_bounds__(kPlanThreads) extend_plan_kernel(const ExtendParams p) {
  __shared__ long long s_sum[kPlanWarps];
  __shared__ int s_isum[kPlanWarps];
  __shared__ long long s_free[kMaxCluster];  // of every CTA of the cluster
  __shared__ long long s_need;               // pages that the call needs
  __shared__ int s_bad;
  __shared__ int s_base[kPlanThreads];  // the requests' bases, where they fit
  griddep_launch_dependents();
  const int ctas = static_cast<int>(cluster_ctas());
  const int rank = static_cast<int>(cluster_rank());
  const int t = threadIdx.x;
  cluster_sync_all();  // every CTA runs: its shared memory may be written

  // What each request needs (the first CTA).
  if (rank == 0) {
    long long need = 0;  // pages, and in the upper bits copies
    bool bad = false;
    for (int b0 = 0; b0 < p.num_reqs; b0 += kPlanThreads) {
      const int b = b0 + t;
      long long w = 0;
      int start = 0, old = -1, rows = 0;
      bool cow = false;
      if (b < p.num_reqs) {
        const long long n = p.lens[b], a = p.add[b];
        if (n < 0 || a < 0 || n + a > INT_MAX || ((n + a + (1LL << p.shift) - 1) >> p.shift) > p.max_blocks) {
          bad = true;
        } else {
          start = pages_of(n, p.shift);
          rows = static_cast<int>(n & ((1 << p.shift) - 1));
          w = pages_of(n + a, p.shift) - start;
          if (a > 0 && rows > 0) {
            old = p.bt[static_cast<size_t>(b) * p.max_blocks + start - 1];
            cow = old >= 0 && old < p.num_blocks && p.refs[old] > 1;
            if (cow) {
              --start;
              ++w;
            }
          }
        }
      }
      long long sum;
      const long long before = need + block_scan(w + (cow ? 1LL << 40 : 0LL), s_sum, sum);
      need += sum;
      if (b < p.num_reqs) {
        const int c = cow ? static_cast<int>(before >> 40) : -1;
        p.reqs[b] = {static_cast<int>(before), start, c};
        if (cow) p.copies[c] = {old, -1, rows};
      }
    }
    bad = __syncthreads_or(bad);
    if (t == 0) {
      *p.n_copies = static_cast<int>(need >> 40);
      for (int r = 0; r < ctas; ++r) {
        if (r == 0) {
          s_need = need & ((1LL << 40) - 1);
          s_bad = bad;
        } else {
          st_cluster_u64(mapa_shared(smem_u32(&s_need), r), need & ((1LL << 40) - 1));
          st_cluster_u32(mapa_shared(smem_u32(&s_bad), r), bad);
        }
      }
    }
  }
  // The free pages of this CTA's part (the first has none).
  long long lo = 0, hi = 0, count = 0;
  if (rank > 0) {
    part_of(p.num_blocks, rank - 1, ctas - 1, lo, hi);
#pragma unroll 4
    for (long long i = lo + 4 * t; i < hi; i += kTile) count += free_of(refs_of(p.refs, i, p.num_blocks));
    count = block_sum(count, s_sum);
  }
  if (t < ctas) {
    if (t == rank) s_free[rank] = count;
    else st_cluster_u64(mapa_shared(smem_u32(&s_free[rank]), t), count);
  }
  cluster_sync_all();

  long long total = 0, at = 0;
  for (int r = 0; r < ctas; ++r) {
    if (r < rank) at += s_free[r];
    total += s_free[r];
  }
  const long long need = s_need;
  const int missing = s_bad ? -1 : need > total ? static_cast<int>(min(need - total, static_cast<long long>(INT_MAX))) : 0;
  if (rank == 0) {
    if (t == 0) {
      *p.missing = missing;
      if (missing != 0) *p.n_copies = 0;
    }
    for (int b = t; b < p.num_reqs; b += kPlanThreads) p.new_lens[b] = p.lens[b] + (missing == 0 ? p.add[b] : 0);
  }
  if (missing != 0 || at >= need || lo >= hi) return;
  const bool in_shared = p.num_reqs <= kPlanThreads;
  if (in_shared) {
    if (t < p.num_reqs) s_base[t] = p.reqs[t].base;
    __syncthreads();
  }
  for (long long i0 = lo; i0 < hi && at < need; i0 += kTile) {
    const long long i = i0 + 4 * t;
    const int4 r = refs_of(p.refs, i, p.num_blocks);
    int sum;
    long long k = at + block_scan(free_of(r), s_isum, sum);
    at += sum;
    const int held[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (held[j] > 0) continue;
      if (k < need) {
        // the last request whose first new page has a rank of at most k
        const int b = in_shared ? last_at_most([&](int i) { return s_base[i]; }, p.num_reqs, k)
                                : last_at_most([&](int i) { return p.reqs[i].base; }, p.num_reqs, k);
        const ExtendRequest q = p.reqs[b];
        const int page = static_cast<int>(i) + j;
        p.bt[static_cast<size_t>(b) * p.max_blocks + q.start + (static_cast<int>(k) - q.base)] = page;
        p.refs[page] = 1;
        if (q.cow >= 0 && k == q.base) p.copies[q.cow].dst = page;
      }
      ++k;
    }
  }
}

// 16-byte chunks [first, first + kCopyThreads * kCopyChunks) of n: loads ahead of stores.
__device__ __forceinline__ void copy_part(unsigned char* dst, const unsigned char* src, long long first, long long n) {
  const uint4* s = reinterpret_cast<const uint4*>(src);
  uint4* d = reinterpret_cast<uint4*>(dst);
  uint4 x[kCopyChunks];
#pragma unroll
  for (int c = 0; c < kCopyChunks; ++c) {
    const long long i = first + threadIdx.x + c * kCopyThreads;
    if (i < n) x[c] = s[i];
  }
#pragma unroll
  for (int c = 0; c < kCopyChunks; ++c) {
    const long long i = first + threadIdx.x + c * kCopyThreads;
    if (i < n) d[i] = x[c];
  }
}

// The page copies of a plan, in every cache: a unit is kCopyBytes of a page, all
// of it in flight at once.  Bound by memory: 256 copies of parts of 128 KB pages
// in each of 32 caches, 459 MB read (mostly from L2: eight copies share a source)
// and written, 100 us.
__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const __grid_constant__ Caches caches,
                                                                 const PageCopy* copies, const int* n_copies,
                                                                 int32_t* refs) {
  griddep_wait();
  const int n = *n_copies;
  for (int i = blockIdx.x * kCopyThreads + threadIdx.x; i < n; i += gridDim.x * kCopyThreads)
    atomicSub(refs + copies[i].src, 1);
  const long long parts = (caches.page_bytes + kCopyBytes - 1) / kCopyBytes;
  const long long units = n * caches.n * parts;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int part = static_cast<int>(u % parts);
    const long long rest = u / parts;
    const PageCopy c = copies[rest / caches.n];
    unsigned char* base = caches.at[rest % caches.n];
    const long long n16 = c.rows * caches.row_bytes / 16, first = part * static_cast<long long>(kCopyBytes / 16);
    if (first < n16) copy_part(base + c.dst * caches.page_bytes, base + c.src * caches.page_bytes, first, n16);
  }
}

// ------------------------------------------------------------------ fork, trim
struct ForkParams {
  int32_t* refs;
  const int32_t* bt;
  const int32_t* lens;
  const int32_t* parents;
  int32_t* bt_out;
  int32_t* lens_out;
  int num_blocks, num_reqs, max_blocks, num_out, max_blocks_out, shift;
};

constexpr int kRowThreads = 256;

__device__ __forceinline__ int clamped_len(int n, int max_blocks, int shift) {
  return static_cast<int>(min(static_cast<long long>(max(n, 0)), static_cast<long long>(max_blocks) << shift));
}

// Bound by latency and, with long rows, by the atomics: 256 rows of some 1200
// pages each, 6.6 us.
// CTAs [0, num_reqs): a row of the old table, whose pages gain a holder for
// every new row beyond one that continues it.  CTAs after those: a new row.
__global__ void __launch_bounds__(kRowThreads) fork_kernel(const ForkParams p) {
  if (blockIdx.x < p.num_reqs) {
    const int b = blockIdx.x;
    int kids = 0;
    for (int i = threadIdx.x; i < p.num_out; i += kRowThreads) kids += __ldg(p.parents + i) == b;
    __shared__ int s_kids;
    if (threadIdx.x == 0) s_kids = 0;
    __syncthreads();
    kids = __reduce_add_sync(kWarp, kids);
    if ((threadIdx.x & 31) == 0 && kids != 0) atomicAdd(&s_kids, kids);
    __syncthreads();
    const int more = s_kids - 1;
    if (more == 0) return;
    const int n = pages_of(clamped_len(__ldg(p.lens + b), p.max_blocks, p.shift), p.shift);
    for (int i = threadIdx.x; i < n; i += kRowThreads) {
      const int page = __ldg(p.bt + static_cast<size_t>(b) * p.max_blocks + i);
      if (page >= 0 && page < p.num_blocks) atomicAdd(p.refs + page, more);
    }
  } else {
    const int i = blockIdx.x - p.num_reqs;
    const int b = __ldg(p.parents + i);
    const bool some = b >= 0 && b < p.num_reqs;
    const int len = some ? clamped_len(__ldg(p.lens + b), p.max_blocks, p.shift) : 0;
    if (threadIdx.x == 0) p.lens_out[i] = len;
    const int n = pages_of(len, p.shift);
    for (int j = threadIdx.x; j < n; j += kRowThreads)
      p.bt_out[static_cast<size_t>(i) * p.max_blocks_out + j] = __ldg(p.bt + static_cast<size_t>(b) * p.max_blocks + j);
  }
}

struct TrimParams {
  int32_t* refs;
  const int32_t* bt;
  int32_t* lens;
  const int32_t* keep;
  int num_blocks, max_blocks, shift;
};

// (3.5 us for 256 requests: a launch and three dependent loads.)
__global__ void __launch_bounds__(kRowThreads) trim_kernel(const TrimParams p) {
  const int b = blockIdx.x;
  const int keep = p.keep[b], len = p.lens[b];
  __syncthreads();  // every thread has read the length
  if (keep < 0 || keep >= len) return;
  if (threadIdx.x == 0) p.lens[b] = keep;
  const int lo = pages_of(keep, p.shift), hi = pages_of(clamped_len(len, p.max_blocks, p.shift), p.shift);
  for (int i = lo + threadIdx.x; i < hi; i += kRowThreads) {
    const int page = p.bt[static_cast<size_t>(b) * p.max_blocks + i];
    if (page >= 0 && page < p.num_blocks) atomicSub(p.refs + page, 1);
  }
}

// ------------------------------------------------------------------ compact
struct CompactParams {
  int32_t* refs;
  int32_t* bt;
  const int32_t* lens;
  int32_t* map;       // [num_blocks]
  int32_t* num_live;
  int* n_moves;       // workspace
  int32_t* src;       // [num_blocks / 2 + 1] each
  int32_t* dst;
  int num_blocks, num_reqs, max_blocks, shift;
};

// Three passes over refs (live pages; those among the first ids; the map), the
// last two from L2, between two cluster barriers: 7 us for 4096 pages.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const CompactParams p) {
  __shared__ long long s_sum[kPlanWarps];
  __shared__ int s_isum[kPlanWarps];
  __shared__ long long s_live[2][kMaxCluster];  // live pages of every CTA's part; those among the first `live` ids
  griddep_launch_dependents();
  const int ctas = static_cast<int>(cluster_ctas());
  const int rank = ctas > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int t = threadIdx.x;
  if (ctas > 1) cluster_sync_all();  // every CTA runs: its shared memory may be written
  long long lo, hi;
  part_of(p.num_blocks, rank, ctas, lo, hi);
  hi = min(hi, static_cast<long long>(p.num_blocks));
  auto publish = [&](int k, long long count) {
    count = block_sum(count, s_sum);
    if (t < ctas) {
      if (t == rank) s_live[k][rank] = count;
      else st_cluster_u64(mapa_shared(smem_u32(&s_live[k][rank]), t), count);
    }
    if (ctas > 1) cluster_sync_all();
    else __syncthreads();
  };
  long long count = 0;
  for (long long i = lo + 4 * t; i < hi; i += kTile)
    count += min(4LL, p.num_blocks - i) - free_of(refs_of(p.refs, i, p.num_blocks));
  publish(0, count);
  long long live = 0, before = 0;  // live pages in all, and in the parts before this one
  for (int r = 0; r < ctas; ++r) {
    if (r < rank) before += s_live[0][r];
    live += s_live[0][r];
  }
  count = 0;
  for (long long i = lo + 4 * t; i < min(hi, live); i += kTile) {
    const int4 r = refs_of(p.refs, i, static_cast<int>(live));  // (1 past the end)
    count += min(4LL, live - i) - free_of(r);
  }
  publish(1, count);
  long long stay = 0;  // live pages that are where they may stay
  for (int r = 0; r < ctas; ++r) stay += s_live[1][r];
  if (rank == 0 && t == 0) {
    *p.num_live = static_cast<int>(live);
    *p.n_moves = static_cast<int>(live - stay);
  }
  for (long long i0 = lo; i0 < hi; i0 += kTile) {
    const long long i = i0 + 4 * t;
    const int4 r = refs_of(p.refs, i, p.num_blocks);
    const int n = static_cast<int>(max(0LL, min(4LL, p.num_blocks - i)));
    int sum;
    long long k = before + block_scan(i < p.num_blocks ? n - free_of(r) : 0, s_isum, sum);  // live pages before page i
    before += sum;
    const int held[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j >= n) break;
      const int page = static_cast<int>(i) + j;
      if (held[j] > 0) {
        if (page < live) p.map[page] = page;
        else p.src[k - stay] = page;  // (its map entry is written when it moves)
        ++k;
      } else {
        p.map[page] = -1;
        if (page < live) p.dst[page - k] = page;
      }
    }
  }
}

// Metadata first: a table entry finds its page's new id by the page's rank in
// src (the moved pages' map entries are written meanwhile).  Then the pages, as
// in page_copy_kernel: 2.06 GB moved in 595 us, the rate of a plain copy.
__global__ void __launch_bounds__(kCopyThreads) compact_move_kernel(const __grid_constant__ Caches caches,
                                                                    const CompactParams p) {
  griddep_wait();
  const int n = *p.n_moves;
  const int live = *p.num_live;
  const int thread = blockIdx.x * kCopyThreads + threadIdx.x, threads = gridDim.x * kCopyThreads;
  for (int i = thread; i < n; i += threads) {
    const int from = p.src[i], to = p.dst[i];
    p.map[from] = to;
    p.refs[to] = p.refs[from];
    p.refs[from] = 0;
  }
  for (int b = blockIdx.x; b < p.num_reqs; b += gridDim.x) {
    const int m = pages_of(clamped_len(p.lens[b], p.max_blocks, p.shift), p.shift);
    int32_t* row = p.bt + static_cast<size_t>(b) * p.max_blocks;
    for (int i = threadIdx.x; i < m; i += kCopyThreads) {
      const int page = row[i];
      if (page < live || page >= p.num_blocks) continue;
      int k = 0, len = n;  // the last move whose source is at most page
      while (len > 1) {
        const int half = len >> 1;
        if (p.src[k + half] <= page) {
          k += half;
          len -= half;
        } else {
          len = half;
        }
      }
      if (n > 0 && p.src[k] == page) row[i] = p.dst[k];
    }
  }
  const long long parts = (caches.page_bytes + kCopyBytes - 1) / kCopyBytes;
  const long long units = static_cast<long long>(n) * caches.n * parts;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int part = static_cast<int>(u % parts);
    const long long rest = u / parts;
    const int move = static_cast<int>(rest / caches.n);
    unsigned char* base = caches.at[rest % caches.n];
    copy_part(base + p.dst[move] * caches.page_bytes, base + p.src[move] * caches.page_bytes,
              part * static_cast<long long>(kCopyBytes / 16), caches.page_bytes / 16);
  }
}

// ------------------------------------------------------------------ host
// CTAs of the cluster that scans refs.
int plan_ctas(int num_blocks) {
  int n = 1;
  while (n < kMaxCluster && static_cast<long long>(n) * 2 * kTile <= num_blocks) n *= 2;
  return n;
}

int page_shift(int block_size) {
  int shift = 0;
  while (shift < 30 && (1 << shift) < block_size) ++shift;
  return block_size < 16 || block_size > 256 || (1 << shift) != block_size ? -1 : shift;
}

int take_caches(Caches& c, void* const* caches, int num_caches, size_t row_bytes, int block_size) {
  if (num_caches < 0 || (num_caches > 0 && caches == nullptr)) return MVP_ERR_ARG;
  if (num_caches > kMaxCaches) return MVP_ERR_UNSUPPORTED;
  if (num_caches > 0 && (row_bytes == 0 || row_bytes % 16 != 0 || row_bytes > (size_t{1} << 24))) return MVP_ERR_UNSUPPORTED;
  c.n = num_caches;
  c.row_bytes = static_cast<long long>(row_bytes);
  c.page_bytes = c.row_bytes * block_size;
  for (int i = 0; i < num_caches; ++i) {
    if (caches[i] == nullptr) return MVP_ERR_ARG;
    if ((reinterpret_cast<uintptr_t>(caches[i]) & 15u) != 0) return MVP_ERR_UNSUPPORTED;
    c.at[i] = static_cast<unsigned char*>(caches[i]);
  }
  return MVP_OK;
}

template <class... Args>
cudaError_t launch(void (*kernel)(Args...), int grid, int block, int cluster, bool dependent, void* stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n++].val.clusterDim.z = 1;
  }
  if (dependent) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.stream = static_cast<cudaStream_t>(stream);
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Copying CTAs: so many per SM, or as many as there can be units.  One fewer, so
// that their number has no power of two in common with the parts of a page and each
// CTA takes all parts of pages in turn: pages that are copied in part end before
// their last parts (32 prompts shared by 8 samples, 32 caches, pages of 8 parts: 131
// us with 1216 CTAs, 112 with 1215).  1215 = 3^5 5: of pages of 3, 5, 6, .. parts a
// CTA still takes some parts only.
// A step's extension, which mostly copies nothing, takes eight (a launch that
// finds no work then costs 2.5 us); a compaction 64 (2 GB moved: 645 us with 8,
// 606 with 16, 595 with 64: units go to whichever SM is free).
constexpr int kExtendCopyCtas = 8, kCompactCtas = 64;
int copy_grid(const Caches& c, long long max_pages, int num_sms, int per_sm) {
  const long long parts = (c.page_bytes + kCopyBytes - 1) / kCopyBytes;
  const long long units = std::max<long long>(1, max_pages * std::max(1LL, c.n * parts));
  return static_cast<int>(std::min<long long>(units, static_cast<long long>(per_sm) * num_sms - 1));
}

}  // namespace

}  // namespace mvp

using namespace mvp;

extern "C" {

size_t mvp_kv_extend_workspace_size(int num_reqs) {
  if (num_reqs <= 0) return 0;
  return kPagesHeader + static_cast<size_t>(num_reqs) * (sizeof(ExtendRequest) + sizeof(PageCopy));
}

size_t mvp_kv_compact_workspace_size(int num_blocks) {
  if (num_blocks <= 0) return 0;
  return kPagesHeader + 2 * (static_cast<size_t>(num_blocks) / 2 + 1) * sizeof(int32_t);
}

int mvp_kv_extend_paged(void* const* caches, int num_caches, size_t row_bytes, int32_t* refs, int num_blocks,
                        int32_t* block_table, int max_blocks_per_seq, int block_size, const int32_t* seq_lens_k,
                        const int32_t* add_lens, int32_t* new_seq_lens, int num_reqs, int32_t* missing,
                        void* workspace, size_t workspace_bytes, void* stream) {
  set_last_launches(0);
  const int shift = page_shift(block_size);
  if (shift < 0 || num_reqs < 0 || num_blocks < 1 || max_blocks_per_seq < 1) return MVP_ERR_ARG;
  Caches c;
  const int st = take_caches(c, caches, num_caches, row_bytes, block_size);
  if (st != MVP_OK) return st;
  if (refs == nullptr || missing == nullptr) return MVP_ERR_ARG;
  if (num_reqs == 0) return cudaMemsetAsync(missing, 0, sizeof(int32_t), static_cast<cudaStream_t>(stream)) == cudaSuccess ? MVP_OK : MVP_ERR_CUDA;
  if (block_table == nullptr || seq_lens_k == nullptr || add_lens == nullptr || new_seq_lens == nullptr || workspace == nullptr)
    return MVP_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(workspace) & 15u) != 0) return MVP_ERR_UNSUPPORTED;
  if (workspace_bytes < mvp_kv_extend_workspace_size(num_reqs)) return MVP_ERR_CAPACITY;
  if (num_reqs > 65535) return MVP_ERR_UNSUPPORTED;  // (page counts and copies share 64 bits)
  int* err = nullptr;
  int num_sms = 1;
  if (device_error_word(&err, &num_sms) != cudaSuccess) return MVP_ERR_CUDA;
  ExtendParams p;
  p.refs = refs;
  p.bt = block_table;
  p.lens = seq_lens_k;
  p.add = add_lens;
  p.new_lens = new_seq_lens;
  p.missing = missing;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  p.n_copies = reinterpret_cast<int*>(ws);
  p.reqs = reinterpret_cast<ExtendRequest*>(ws + kPagesHeader);
  p.copies = reinterpret_cast<PageCopy*>(p.reqs + num_reqs);
  p.num_blocks = num_blocks;
  p.num_reqs = num_reqs;
  p.max_blocks = max_blocks_per_seq;
  p.shift = shift;
  const int ctas = std::min(kMaxCluster, plan_ctas(num_blocks) + 1);
  if (launch(extend_plan_kernel, ctas, kPlanThreads, ctas, false, stream, ExtendParams(p)) != cudaSuccess) return MVP_ERR_CUDA;
  if (launch(page_copy_kernel, copy_grid(c, num_reqs, num_sms, kExtendCopyCtas), kCopyThreads, 1, true, stream, Caches(c),
             static_cast<const PageCopy*>(p.copies), static_cast<const int*>(p.n_copies), refs) != cudaSuccess)
    return MVP_ERR_CUDA;
  set_last_launches(2);
  return MVP_OK;
}

int mvp_kv_fork_paged(int32_t* refs, int num_blocks, const int32_t* block_table, const int32_t* seq_lens_k,
                      int num_reqs, int max_blocks_per_seq, const int32_t* parents, int num_out,
                      int32_t* block_table_out, int max_blocks_out, int32_t* seq_lens_out, int block_size,
                      void* stream) {
  set_last_launches(0);
  const int shift = page_shift(block_size);
  if (shift < 0 || num_reqs < 0 || num_out < 0 || num_blocks < 1 || max_blocks_per_seq < 1) return MVP_ERR_ARG;
  if (max_blocks_out < max_blocks_per_seq) return MVP_ERR_ARG;
  if (num_reqs > (1 << 24) || num_out > (1 << 24)) return MVP_ERR_UNSUPPORTED;
  // (each old row reads all parents: the kernel would hold the GPU for minutes)
  if (static_cast<long long>(num_reqs) * num_out > 1LL << 40) return MVP_ERR_UNSUPPORTED;
  if (num_reqs + num_out == 0) return MVP_OK;
  if (refs == nullptr || (num_reqs > 0 && (block_table == nullptr || seq_lens_k == nullptr))) return MVP_ERR_ARG;
  if (num_out > 0 && (parents == nullptr || block_table_out == nullptr || seq_lens_out == nullptr)) return MVP_ERR_ARG;
  if (num_out > 0 && num_reqs > 0 && (block_table_out == block_table || seq_lens_out == seq_lens_k)) return MVP_ERR_ARG;
  const ForkParams p{refs,     block_table, seq_lens_k,         parents, block_table_out, seq_lens_out,
                     num_blocks, num_reqs,  max_blocks_per_seq, num_out, max_blocks_out,  shift};
  if (launch(fork_kernel, num_reqs + num_out, kRowThreads, 1, false, stream, ForkParams(p)) != cudaSuccess) return MVP_ERR_CUDA;
  set_last_launches(1);
  return MVP_OK;
}

int mvp_kv_trim_paged(int32_t* refs, int num_blocks, const int32_t* block_table, int max_blocks_per_seq,
                      int32_t* seq_lens_k, const int32_t* new_seq_lens, int num_reqs, int block_size, void* stream) {
  set_last_launches(0);
  const int shift = page_shift(block_size);
  if (shift < 0 || num_reqs < 0 || num_blocks < 1 || max_blocks_per_seq < 1) return MVP_ERR_ARG;
  if (num_reqs == 0) return MVP_OK;
  if (refs == nullptr || block_table == nullptr || seq_lens_k == nullptr || new_seq_lens == nullptr) return MVP_ERR_ARG;
  const TrimParams p{refs, block_table, seq_lens_k, new_seq_lens, num_blocks, max_blocks_per_seq, shift};
  if (launch(trim_kernel, num_reqs, kRowThreads, 1, false, stream, TrimParams(p)) != cudaSuccess) return MVP_ERR_CUDA;
  set_last_launches(1);
  return MVP_OK;
}

int mvp_kv_compact_paged(void* const* caches, int num_caches, size_t row_bytes, int32_t* refs, int num_blocks,
                         int32_t* block_table, int max_blocks_per_seq, int block_size, const int32_t* seq_lens_k,
                         int num_reqs, int32_t* block_map, int32_t* num_live, void* workspace,
                         size_t workspace_bytes, void* stream) {
  set_last_launches(0);
  const int shift = page_shift(block_size);
  if (shift < 0 || num_reqs < 0 || num_blocks < 1 || max_blocks_per_seq < 1) return MVP_ERR_ARG;
  Caches c;
  const int st = take_caches(c, caches, num_caches, row_bytes, block_size);
  if (st != MVP_OK) return st;
  if (refs == nullptr || block_map == nullptr || num_live == nullptr || workspace == nullptr) return MVP_ERR_ARG;
  if (num_reqs > 0 && (block_table == nullptr || seq_lens_k == nullptr)) return MVP_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(workspace) & 15u) != 0) return MVP_ERR_UNSUPPORTED;
  if (workspace_bytes < mvp_kv_compact_workspace_size(num_blocks)) return MVP_ERR_CAPACITY;
  int* err = nullptr;
  int num_sms = 1;
  if (device_error_word(&err, &num_sms) != cudaSuccess) return MVP_ERR_CUDA;
  CompactParams p;
  p.refs = refs;
  p.bt = block_table;
  p.lens = seq_lens_k;
  p.map = block_map;
  p.num_live = num_live;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  p.n_moves = reinterpret_cast<int*>(ws);
  p.src = reinterpret_cast<int32_t*>(ws + kPagesHeader);
  p.dst = p.src + num_blocks / 2 + 1;
  p.num_blocks = num_blocks;
  p.num_reqs = num_reqs;
  p.max_blocks = max_blocks_per_seq;
  p.shift = shift;
  const int ctas = plan_ctas(num_blocks);
  if (launch(compact_plan_kernel, ctas, kPlanThreads, ctas, false, stream, CompactParams(p)) != cudaSuccess) return MVP_ERR_CUDA;
  if (launch(compact_move_kernel, copy_grid(c, std::max<long long>(num_blocks / 2, num_reqs), num_sms, kCompactCtas),
             kCopyThreads, 1, true, stream, Caches(c), CompactParams(p)) != cudaSuccess)
    return MVP_ERR_CUDA;
  set_last_launches(2);
  return MVP_OK;
}

}  // extern "C"
