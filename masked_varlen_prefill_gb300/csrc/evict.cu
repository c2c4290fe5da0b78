// Eviction from a paged K/V cache by the attention weight each key received.
//
// Per request and KV head, of n keys the first `first`, the last `recent` and
// the heaviest of the others stay, `budget` in all (ties go to the lower
// index, NaN counts as -inf); they keep their order and move to
// the front of the request's blocks, K, V and weights alike.
//
// 1. evict_select_kernel finds, per (request, KV head), the weight of rank
//    budget - first - recent by a radix select over order-preserving integer
//    keys (11, 11 and 10 bits: three histograms in shared memory, or fewer
//    where all of a bin stays), then lists the kept keys in order: a bit per
//    key from warp votes, and a prefix sum of their counts.  Integer counts
//    only, so the result does not depend on the order of the atomics.  Long
//    requests are shared by a cluster of CTAs, which add their histograms
//    through distributed shared memory.  It reads 4 bytes of each key's
//    weight (from L2 after the first time), against 4 * D bytes of K and V
//    that the move reads and writes for a kept one.  Bound by its instructions
//    (about 40 per 32 keys) and by the latency of a pass whatever the keys (1500
//    cycles between its barriers): 48 requests of 4096 to 32768
//    keys, 8 KV heads, 40 us (four compares and a prefix sum per key in place
//    of the votes, and always three passes: 50).
// 2. evict_move_kernel copies the kept rows, 32 KB per CTA, all of it in flight
//    at once in registers (bulk copies of single rows measured slower: at 256
//    bytes each they queue for the copy engine).  It is bound by memory.  In
//    place it must not
//    overwrite a row that another CTA has still to read: a kept key never
//    moves to a higher index, so a segment of the result only overwrites rows
//    that the same or earlier segments read.  Each CTA takes its segment from
//    a ticket counter, loads it, publishes "loaded" and, before
//    it stores, waits for the earlier segments whose rows it is about to
//    overwrite.  Earlier tickets are held by CTAs that already run and reach
//    "loaded" without waiting for anyone, so the wait ends whatever the number
//    of CTAs on the GPU (and is bounded all the same).
#include <cuda_bf16.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <mutex>

#include "../../include/mvp.h"
#include "mvp_internal.cuh"
#include "ptx.cuh"

namespace mvp {

namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelKeys = 16384;  // keys a CTA holds in shared memory (the rest is read again from L2)
constexpr int kBins = 2048;
constexpr unsigned kFullWarp = 0xffffffffu;
constexpr uint32_t kStays = 0xffffffffu;  // order key of a key that stays whatever its weight
static_assert(kBins == 4 * kSelThreads, "four bins per thread");
constexpr int kMoveThreads = 256;
constexpr int kMoveWarps = kMoveThreads / 32;
constexpr int kMoveChunks = 4;  // 16-byte chunks of K, and of V, in flight per thread
constexpr int kMinSegRows = kMoveWarps * 32 * kMoveChunks / 64;  // rows of a segment at the largest head_dim
constexpr size_t kEvictHeader = 256;  // the ticket counter, ahead of the flags

struct EvictParams {
  __nv_bfloat16* k;
  __nv_bfloat16* v;
  const float* w;
  float* w_out;
  const int32_t* seq_k;
  const int32_t* bt;
  const int32_t* bt_out;
  const int32_t* slots;  // or null
  int32_t* new_lens;
  int32_t* kept;         // [num_reqs, hkv, budget]
  int* ticket;
  int* flags;            // [num_reqs * hkv, n_segs]
  int num_reqs, hkv, d, num_slots;
  long long w_stride;
  int block_shift, max_blocks, max_blocks_out, num_blocks;
  int max_k_len, budget, first, recent;
  int seg_rows, n_segs;
  int* err;
};

__device__ __forceinline__ int keys_of(const EvictParams& p, int b) {
  return min(max(__ldg(p.seq_k + b), 0), p.max_k_len);
}

// Index of (b, h)'s row of weights, or -1 (bounds-checked build: a slot outside).
__device__ __forceinline__ long long weight_row(const EvictParams& p, int b, int h) {
  const int slot = p.slots != nullptr ? __ldg(p.slots + b) : b;
  if (!in_bounds(slot, p.num_slots, p.err)) return -1;
  return (static_cast<long long>(slot) * p.hkv + h) * p.w_stride;
}

// Larger key, heavier weight; -0 and +0 are equal, NaN is -inf.
__device__ __forceinline__ uint32_t order_key(float w) {
  const uint32_t u = __float_as_uint(fmaxf(w, -INFINITY) + 0.0f);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ int ld_cluster_s32(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ int4 ld_cluster_v4(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p) {
  extern __shared__ __align__(16) uint32_t s_key[];  // [kSelKeys] order keys of the CTA's first keys
  __shared__ __align__(16) int s_hist[kBins];
  __shared__ int s_warp[kSelWarps][2];
  __shared__ int s_bin, s_need, s_in;
  __shared__ int s_count[2];
  const int cl = static_cast<int>(cluster_size()), c = static_cast<int>(cluster_rank());
  const int cl_shift = __popc(cl - 1);  // (a power of two)
  const int bh = blockIdx.x >> cl_shift, b = bh / p.hkv, h = bh - b * p.hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto sync = [&]() {
    if (cl > 1) cluster_sync_all();
    else __syncthreads();
  };
  if (c == 0) {
    for (int i = tid; i < p.n_segs; i += kSelThreads) p.flags[static_cast<size_t>(bh) * p.n_segs + i] = 0;
    if (bh == 0 && tid == 0) *p.ticket = 0;
  }
  const int n = keys_of(p, b);
  if (c == 0 && h == 0 && tid == 0) p.new_lens[b] = min(n, p.budget);
  int32_t* kept = p.kept + static_cast<size_t>(bh) * p.budget;
  const long long wrow = weight_row(p, b, h);
  if (n <= p.budget || wrow < 0) {
    for (int i = c * kSelThreads + tid; i < p.budget; i += cl * kSelThreads) kept[i] = i < n ? i : -1;
    return;
  }
  const float* w = p.w + wrow;
  const int lo = p.first, hi = n - p.recent;  // the keys that compete
  // This CTA's keys [s0, s1), each warp's a run of `per` of them.
  static_assert((kSelWarps & (kSelWarps - 1)) == 0, "a power of two");
  const int round = 128 * kSelWarps * cl;
  const int per = ((n + round - 1) >> (cl_shift + __popc(128 * kSelWarps - 1))) * 128;
  const int s0 = min(n, c * per * kSelWarps), s1 = min(n, s0 + per * kSelWarps);
  const int size = per * kSelWarps;
  const uint32_t span = static_cast<uint32_t>(hi - lo);
  // Order key of key k, of weight x: kStays for those that stay anyway, 0 past
  // the CTA's last one (order keys of weights lie strictly between).
  auto encode = [&](int k, float x) -> uint32_t {
    const uint32_t key = static_cast<uint32_t>(k - lo) < span ? order_key(x) : kStays;
    return k < s1 ? key : 0u;
  };
  auto read = [&](int i) -> uint32_t { return encode(s0 + i, w[min(s0 + i, n - 1)]); };

  // ------------------------------------------------ the weight of that rank
  // Every key once from memory, into shared memory and the first histogram.
  *reinterpret_cast<int4*>(&s_hist[4 * tid]) = make_int4(0, 0, 0, 0);
  __syncthreads();
  // Eight loads in flight per thread.
  constexpr int kAhead = 8;
  for (int i0 = 0; i0 < size; i0 += kAhead * kSelThreads) {
    const int k = s0 + i0 + tid;
    float x[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) x[u] = k + u * kSelThreads < s1 ? w[k + u * kSelThreads] : 0.f;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int at = i0 + u * kSelThreads;  // (the same for all threads; size and kSelKeys are multiples)
      if (at >= size) break;
      const uint32_t key = encode(k + u * kSelThreads, x[u]);
      if (at < kSelKeys) s_key[at + tid] = key;
      atomicAdd(&s_hist[key >> 21], 1);
    }
  }
  uint32_t prefix = kStays - 1u, mask = 0u;  // (no weight's key: none competes when none may stay)
  int need = p.budget - p.first - p.recent;
  if (need > 0) {
    prefix = 0u;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
      const uint32_t digit = pass == 2 ? 1023u : kBins - 1u;
      if (pass > 0) {
        if (cl > 1) {  // (a CTA alone has cleared them as it read them)
          *reinterpret_cast<int4*>(&s_hist[4 * tid]) = make_int4(0, 0, 0, 0);
          __syncthreads();
        }
        auto add = [&](uint4 k) {
          const bool in[4] = {(k.x & mask) == prefix, (k.y & mask) == prefix, (k.z & mask) == prefix,
                              (k.w & mask) == prefix};
          if (!(in[0] || in[1] || in[2] || in[3])) return;
          if (in[0]) atomicAdd(&s_hist[(k.x >> shift) & digit], 1);
          if (in[1]) atomicAdd(&s_hist[(k.y >> shift) & digit], 1);
          if (in[2]) atomicAdd(&s_hist[(k.z >> shift) & digit], 1);
          if (in[3]) atomicAdd(&s_hist[(k.w >> shift) & digit], 1);
        };
#pragma unroll 2
        for (int at = 0; at < min(size, kSelKeys); at += 4 * kSelThreads)
          add(*reinterpret_cast<const uint4*>(s_key + at + 4 * tid));
        for (int at = kSelKeys; at < size; at += 4 * kSelThreads) {
          const int i = at + tid;
          add(make_uint4(read(i), read(i + kSelThreads), read(i + 2 * kSelThreads), read(i + 3 * kSelThreads)));
        }
      }
      sync();
      // Bins from the heaviest down, four per thread; the cluster's counts are
      // added up by every CTA alike.
      const int bin0 = kBins - 4 - 4 * tid;
      int4 q;
      if (cl == 1) {
        q = *reinterpret_cast<const int4*>(&s_hist[bin0]);
        *reinterpret_cast<int4*>(&s_hist[bin0]) = make_int4(0, 0, 0, 0);
      } else {
        q = make_int4(0, 0, 0, 0);
        for (int r = 0; r < cl; ++r) {
          const int4 o = ld_cluster_v4(mapa_shared(smem_u32(&s_hist[bin0]), r));
          q = make_int4(q.x + o.x, q.y + o.y, q.z + o.z, q.w + o.w);
        }
      }
      if (pass == 0 && tid == 0) q.w = 0;                // keys that stay anyway
      if (pass == 0 && tid == kSelThreads - 1) q.x = 0;  // past the last key
      const int cnt[4] = {q.w, q.z, q.y, q.x}, sum = q.x + q.y + q.z + q.w;
      // The warp that the rank falls into finds the bin.
      const int warp_sum = __reduce_add_sync(kFullWarp, sum);
      if (lane == 0) s_warp[warp][0] = warp_sum;
      __syncthreads();
      const int warp_before = __reduce_add_sync(kFullWarp, lane < warp ? s_warp[lane & (kSelWarps - 1)][0] : 0);
      if (warp_before < need && need <= warp_before + warp_sum) {
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(kFullWarp, incl, o);
          if (lane >= o) incl += x;
        }
        const int before = warp_before + incl - sum;
        if (before < need && need <= before + sum) {  // one thread
          int at = before, i = 0;
          while (at + cnt[i] < need) at += cnt[i++];
          s_bin = bin0 + 3 - i;
          s_need = need - at;
          s_in = cnt[i];
        }
      }
      __syncwarp();
      sync();  // (also: every CTA has read the others' counts)
      prefix |= static_cast<uint32_t>(s_bin) << shift;
      mask |= digit << shift;
      need = s_need;
      if (need == s_in) {  // every key of the bin stays: no need to look into it
        prefix -= 1u;
        need = 0;
        break;
      }
    }
  } else {
    __syncthreads();  // s_key is complete
  }

  // ------------------------------------------------ the kept keys, in order
  // Keys above the prefix stay, and the first `need` of those equal to it.
  // 1024 of the warp's keys at a time: lane u takes the votes on the u-th 32 of
  // them, a bit per key.
  const int i0 = __shfl_sync(kFullWarp, warp, 0) * per;  // (known to be the warp's own)
  unsigned above = 0, equal = 0;
  auto vote = [&](int at) {
    above = equal = 0;
    const int words = min(32, (i0 + per - at) / 32);
    auto take = [&](int u, uint32_t k) {
      const unsigned g = __ballot_sync(kFullWarp, k > prefix), e = __ballot_sync(kFullWarp, k == prefix);
      if (lane == u) {
        above = g;
        equal = e;
      }
    };
    const int held = min(words, max(0, kSelKeys - at) / 32);  // (the first keys, in shared memory)
#pragma unroll 4
    for (int u = 0; u < held; ++u) take(u, s_key[at + 32 * u + lane]);
#pragma unroll 4
    for (int u = held; u < words; ++u) take(u, read(at + 32 * u + lane));
  };
  // Their numbers in this warp's run, then before it.
  int g = 0, tie = 0;
  for (int at = i0; at < i0 + per; at += 1024) {
    vote(at);
    g += __popc(above);
    tie += __popc(equal);
  }
  g = __reduce_add_sync(kFullWarp, g);
  tie = __reduce_add_sync(kFullWarp, tie);
  if (lane == 0) {
    s_warp[warp][0] = g;
    s_warp[warp][1] = tie;
  }
  __syncthreads();
  int gb = __reduce_add_sync(kFullWarp, lane < warp ? s_warp[lane & (kSelWarps - 1)][0] : 0);
  int tb = __reduce_add_sync(kFullWarp, lane < warp ? s_warp[lane & (kSelWarps - 1)][1] : 0);
  if (cl > 1) {
    if (tid == kSelThreads - 1) {
      s_count[0] = gb + g;
      s_count[1] = tb + tie;
    }
    __syncwarp();
    cluster_sync_all();
    for (int r = 0; r < c; ++r) {
      gb += ld_cluster_s32(mapa_shared(smem_u32(&s_count[0]), r));
      tb += ld_cluster_s32(mapa_shared(smem_u32(&s_count[1]), r));
    }
  }
  for (int at = i0; at < i0 + per; at += 1024) {
    if (per > 1024) vote(at);  // (else the votes are still here)
    const int own = __popc(above) | __popc(equal) << 16;
    int incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(kFullWarp, incl, o);
      if (lane >= o) incl += x;
    }
    const int t0 = tb + ((incl - own) >> 16), room = max(need - t0, 0);
    if (room == 0) equal = 0;
    while (__popc(equal) > room) equal &= ~(1u << (31 - __clz(equal)));  // the highest goes first
    // Listed in shared memory, where these keys were (nobody reads them again),
    // and from there to `kept` in whole lines: 16384 keys cut to 8192, 384 times,
    // take 72000 cycles with each lane storing its own.  Keys past those held
    // there are few words of long requests.
    const int all = __shfl_sync(kFullWarp, incl, 31);
    const int start = gb + min(tb, need), count = (all & 0xffff) + min(tb + (all >> 16), need) - min(tb, need);
    const bool held = at + 1024 <= kSelKeys;
    int to = ((incl - own) & 0xffff) + min(t0, need) - min(tb, need);
    __syncwarp();
    for (unsigned stay = above | equal; stay != 0; stay &= stay - 1, ++to) {
      const int k = s0 + at + 32 * lane + __ffs(stay) - 1;
      if (held) s_key[at + to] = k;
      else if (start + to < p.budget) kept[start + to] = k;
    }
    __syncwarp();
    if (held)
      for (int i = lane; i < min(count, p.budget - start); i += 32) kept[start + i] = s_key[at + i];
    gb += all & 0xffff;
    tb += all >> 16;
  }
  // (Here, not at the start: move CTAs waiting next to the second wave of these
  // cost 45 us of 400 on a batch of 384 (request, KV head) pairs.)
  griddep_launch_dependents();
  if (cl > 1) cluster_sync_all();  // no CTA leaves while another reads its counts
}

// Row of key j in the caches, or -1 (an id outside them).
__device__ __forceinline__ long long cache_row(const EvictParams& p, const int32_t* bt, int max_blocks, int b, int j) {
  const int blk = j >> p.block_shift;
  if (blk >= max_blocks) return -1;
  const int id = __ldg(bt + static_cast<size_t>(b) * max_blocks + blk);
  if (id < 0 || id >= p.num_blocks) return -1;
  return (static_cast<long long>(id) << p.block_shift) + (j & ((1 << p.block_shift) - 1));
}

__device__ __forceinline__ uint4 ld_stream(const void* ptr) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(ptr)
               : "memory");
  return r;
}

__device__ __forceinline__ int ld_acquire(const int* ptr) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(ptr) : "memory");
  return v;
}

__device__ __forceinline__ void add_release(int* ptr, int v) {
  asm volatile("red.release.gpu.global.add.s32 [%0], %1;" ::"l"(ptr), "r"(v) : "memory");
}

// A CTA per segment; its warps take wr rows each and share nothing but the
// ticket, so that each goes through kept keys -> block ids -> rows -> flag ->
// stores at its own pace.  A segment's flag counts the warps that have loaded.
// 48 requests cut to 4096 keys of 8 KV heads at D = 128 (1.6 GB moved): 284 us,
// 0.86 of the copy rate, with five CTAs per SM (296 with the four that 56
// registers allow).
__global__ void __launch_bounds__(kMoveThreads, 5) evict_move_kernel(const EvictParams p) {
  __shared__ int s_ticket;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_wait();
  if (threadIdx.x == 0) s_ticket = atomicAdd(p.ticket, 1);
  __syncthreads();
  const int bhs = p.num_reqs * p.hkv;
  if (s_ticket >= bhs * p.n_segs) {  // another call runs on this workspace
    if (threadIdx.x == 0) atomicCAS(p.err, 0, static_cast<int>(kDevQueueConflict));
    return;
  }
  // Tickets: KV head fastest (the heads of a key share DRAM pages), then
  // request, then segment, so that the segments in flight at one time belong to
  // many requests and have loaded long before the next ones of theirs store
  // (segments fastest: 8000 of 27000 cycles were spent waiting).
  const int s = s_ticket / bhs, bh = s_ticket % bhs;
  const int b = bh / p.hkv, h = bh % p.hkv;
  const int n = keys_of(p, b), m = min(n, p.budget);
  const int r0 = s * p.seg_rows, seg_end = min(r0 + p.seg_rows, m);
  if (r0 >= m) return;  // (no later segment waits for it)
  const int wr = p.seg_rows / kMoveWarps;
  const int w0 = r0 + warp * wr, rows = min(wr, seg_end - w0);  // this warp's rows (none: rows <= 0)
  const int32_t* kept = p.kept + static_cast<size_t>(bh) * p.budget;
  int* flags = p.flags + static_cast<size_t>(bh) * p.n_segs;
  const long long wrow = weight_row(p, b, h);
  const bool last = seg_end == m;
  const long long row_bytes = static_cast<long long>(p.hkv) * p.d * 2, head = static_cast<long long>(h) * p.d * 2;
  const unsigned char* kb = reinterpret_cast<const unsigned char*>(p.k) + head;
  const unsigned char* vb = reinterpret_cast<const unsigned char*>(p.v) + head;

  // Lane i: the warp's i-th row.  Rows that stay where they are (the keys
  // before the first evicted one, in place) are neither read nor written.
  long long src = -1, dst = -1;
  float wv = 0.f;
  bool moves = false;
  if (lane < rows) {
    const int j = __ldg(kept + w0 + lane);
    src = cache_row(p, p.bt, p.max_blocks, b, j);
    dst = cache_row(p, p.bt_out, p.max_blocks_out, b, w0 + lane);
    if (wrow >= 0) wv = *(volatile const float*)(p.w + wrow + j);
    moves = p.w_out != p.w || j != w0 + lane;
    if (src < 0 || dst < 0 || src == dst) src = -1;
    else moves = true;
  }
  // 16-byte chunks: slot x = lane + 32 u is chunk x % cpr of row x / cpr.
  const int cpr = p.d / 8;
  const bool pow2 = (cpr & (cpr - 1)) == 0;
  const int shift = 31 - __clz(cpr);
  auto row_of = [&](int u) { return pow2 ? (lane + 32 * u) >> shift : (lane + 32 * u) / cpr; };
  uint4 bk[kMoveChunks], bv[kMoveChunks];
  uint32_t seen = __float_as_uint(wv);
#pragma unroll
  for (int u = 0; u < kMoveChunks; ++u) {
    const int i = row_of(u);
    const long long from = __shfl_sync(0xffffffffu, src, i & 31);
    bk[u] = bv[u] = make_uint4(0, 0, 0, 0);
    if (i < rows && from >= 0) {
      const long long at = from * row_bytes + 16 * (lane + 32 * u - i * cpr);
      bk[u] = ld_stream(kb + at);
      bv[u] = ld_stream(vb + at);
    }
  }
#pragma unroll
  for (int u = 0; u < kMoveChunks; ++u) seen |= bk[u].x | bv[u].x;
  // Loaded: the vote takes a bit of every value that was loaded, so none is in
  // flight when the flag goes up (released after the warp's sync).
  asm volatile("" : "+r"(seen));
  const unsigned voted = __ballot_sync(0xffffffffu, seen == 0u);
  asm volatile("" ::"r"(voted));
  __syncwarp();
  if (lane == 0) add_release(flags + s, 1);
  if (!__any_sync(0xffffffffu, moves) && !last) return;

  // Wait for the earlier segments that read any of the rows this one writes
  // (or, the last one, clears): those whose last key is at or past r0.
  bool ok = true;
  for (int e = s - 1 - lane; e >= 0 && ok; e -= 32) {
    if (__ldg(kept + (e + 1) * p.seg_rows - 1) < r0) break;
    if (ld_acquire(flags + e) >= kMoveWarps) continue;
    const unsigned long long t0 = global_timer_ns();
    while (ld_acquire(flags + e) < kMoveWarps) {
      if (global_timer_ns() - t0 > 1000ull * kDefaultWaitLimitUs) {
        atomicCAS(p.err, 0, static_cast<int>(kDevTimeoutOther));
        ok = false;
        break;
      }
    }
  }
  // ... and for this segment's other warps.
  if (lane == 0 && ok) {
    const unsigned long long t0 = global_timer_ns();
    while (ld_acquire(flags + s) < kMoveWarps) {
      if (global_timer_ns() - t0 > 1000ull * kDefaultWaitLimitUs) {
        atomicCAS(p.err, 0, static_cast<int>(kDevTimeoutOther));
        ok = false;
        break;
      }
    }
  }
  if (!__all_sync(0xffffffffu, ok)) return;
  __syncwarp();  // what one lane acquired holds for the other lanes' stores (a vote does not order memory)
#pragma unroll
  for (int u = 0; u < kMoveChunks; ++u) {
    const int i = row_of(u);
    const long long from = __shfl_sync(0xffffffffu, src, i & 31), to = __shfl_sync(0xffffffffu, dst, i & 31);
    if (i < rows && from >= 0) {
      const long long at = to * row_bytes + 16 * (lane + 32 * u - i * cpr);
      *reinterpret_cast<uint4*>(const_cast<unsigned char*>(kb) + at) = bk[u];
      *reinterpret_cast<uint4*>(const_cast<unsigned char*>(vb) + at) = bv[u];
    }
  }
  if (wrow >= 0) {
    if (lane < rows) p.w_out[wrow + w0 + lane] = wv;
    if (last)
      for (int j = m + threadIdx.x; j < n; j += kMoveThreads) p.w_out[wrow + j] = 0.f;
  }
}

// The select kernel's dynamic shared memory attribute, once per device.
cudaError_t set_select_smem() {
  static std::mutex mutex;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mutex);
  if (done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelKeys * 4);
  if (e == cudaSuccess) done[dev] = true;
  return e;
}

int seg_rows_for(int d) { return kMoveWarps * std::min(32, 32 * kMoveChunks / (d / 8)); }

}  // namespace

}  // namespace mvp

using namespace mvp;

extern "C" {

size_t mvp_kv_evict_workspace_size(int num_reqs, int num_heads_kv, int budget) {
  if (num_reqs < 1 || num_heads_kv < 1 || budget < 1) return 0;
  const size_t segs = (static_cast<size_t>(budget) + kMinSegRows - 1) / kMinSegRows;
  return kEvictHeader + static_cast<size_t>(num_reqs) * num_heads_kv * segs * sizeof(int);
}

int mvp_kv_evict_paged(void* k_cache, void* v_cache, const float* weights, float* weights_out, int num_slots,
                       long long weight_stride, const int32_t* slots, const int32_t* seq_lens_k,
                       const int32_t* block_table, const int32_t* block_table_out, int block_size,
                       int max_blocks_per_seq, int max_blocks_out, int num_blocks, int num_reqs, int max_k_len,
                       int num_heads_kv, int head_dim, int budget, int first_tokens, int recent_tokens,
                       int32_t* new_seq_lens, int32_t* kept, void* workspace, size_t workspace_bytes, void* stream) {
  set_last_launches(0);
  if (num_reqs < 0 || num_heads_kv < 1 || max_k_len < 0 || num_slots < 0) return MVP_ERR_ARG;
  if (head_dim < 16 || head_dim > 512 || head_dim % 8 != 0) return MVP_ERR_UNSUPPORTED;
  if (budget < 1 || first_tokens < 0 || recent_tokens < 0) return MVP_ERR_ARG;
  if (static_cast<long long>(first_tokens) + recent_tokens > budget) return MVP_ERR_ARG;
  if (budget > (1 << 30) || max_k_len > (1 << 30)) return MVP_ERR_UNSUPPORTED;  // indices stay in an int
  int shift = 0;
  while (shift < 30 && (1 << shift) < block_size) ++shift;
  if (block_size < 16 || block_size > 256 || (1 << shift) != block_size) return MVP_ERR_ARG;
  if (num_blocks < 1 || max_blocks_per_seq < 1) return MVP_ERR_ARG;
  if (static_cast<long long>(max_blocks_per_seq) * block_size < max_k_len) return MVP_ERR_ARG;
  if (num_reqs == 0) return MVP_OK;
  if (k_cache == nullptr || v_cache == nullptr || weights == nullptr || seq_lens_k == nullptr ||
      block_table == nullptr || new_seq_lens == nullptr || kept == nullptr || workspace == nullptr)
    return MVP_ERR_ARG;
  if (new_seq_lens == seq_lens_k) return MVP_ERR_ARG;
  if (weight_stride < max_k_len || (slots == nullptr && num_slots < num_reqs)) return MVP_ERR_ARG;
  if (block_table_out == nullptr) {
    block_table_out = block_table;
    max_blocks_out = max_blocks_per_seq;
  }
  const long long longest = budget < max_k_len ? budget : max_k_len;
  if (max_blocks_out < 1 || static_cast<long long>(max_blocks_out) * block_size < longest) return MVP_ERR_ARG;
  if (((reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache) |
        reinterpret_cast<uintptr_t>(workspace)) & 15u) != 0)
    return MVP_ERR_UNSUPPORTED;
  if (workspace_bytes < mvp_kv_evict_workspace_size(num_reqs, num_heads_kv, budget)) return MVP_ERR_CAPACITY;
  EvictParams p;
  p.seg_rows = seg_rows_for(head_dim);
  p.n_segs = static_cast<int>((longest + p.seg_rows - 1) / p.seg_rows);
  if (p.n_segs < 1) p.n_segs = 1;
  const long long bh = static_cast<long long>(num_reqs) * num_heads_kv;
  if (bh * 8 > INT_MAX || bh * p.n_segs > INT_MAX) return MVP_ERR_UNSUPPORTED;
  int* err = nullptr;
  int num_sms = 1;
  if (device_error_word(&err, &num_sms) != cudaSuccess) return MVP_ERR_CUDA;
  p.k = static_cast<__nv_bfloat16*>(k_cache);
  p.v = static_cast<__nv_bfloat16*>(v_cache);
  p.w = weights;
  p.w_out = weights_out != nullptr ? weights_out : const_cast<float*>(weights);
  p.seq_k = seq_lens_k;
  p.bt = block_table;
  p.bt_out = block_table_out;
  p.slots = slots;
  p.new_lens = new_seq_lens;
  p.kept = kept;
  p.ticket = static_cast<int*>(workspace);
  p.flags = reinterpret_cast<int*>(static_cast<unsigned char*>(workspace) + kEvictHeader);
  p.num_reqs = num_reqs;
  p.hkv = num_heads_kv;
  p.d = head_dim;
  p.num_slots = num_slots;
  p.w_stride = weight_stride;
  p.block_shift = shift;
  p.max_blocks = max_blocks_per_seq;
  p.max_blocks_out = max_blocks_out;
  p.num_blocks = num_blocks;
  p.max_k_len = max_k_len;
  p.budget = budget;
  p.first = first_tokens;
  p.recent = recent_tokens;
  p.err = err;
  // CTAs per (request, KV head), at most eight: so many that shared memory
  // holds all keys of the longest request, and while the GPU has room for two
  // per SM, as few as 4096 keys each.
  int cl = 1;
  while (cl < 8 && (static_cast<long long>(cl) * kSelKeys < max_k_len ||
                    (bh * cl * 2 <= 2LL * num_sms && max_k_len / (2 * cl) >= 4096)))
    cl *= 2;
  if (set_select_smem() != cudaSuccess) return MVP_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cl;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cl > 1 ? 1 : 0;
  cfg.gridDim = dim3(static_cast<unsigned>(bh * cl));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = kSelKeys * 4;
  cfg.stream = static_cast<cudaStream_t>(stream);
  if (cudaLaunchKernelEx(&cfg, evict_select_kernel, p) != cudaSuccess) return MVP_ERR_CUDA;
  cfg.attrs = attr + 1;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(bh * p.n_segs));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.dynamicSmemBytes = 0;
  if (cudaLaunchKernelEx(&cfg, evict_move_kernel, p) != cudaSuccess) return MVP_ERR_CUDA;
  set_last_launches(2);
  return MVP_OK;
}

}  // extern "C"
