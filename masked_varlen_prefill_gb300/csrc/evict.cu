// Eviction from a paged K/V cache by the attention weight each key received.
//
// Per request and KV head, of n keys the first `first`, the last `recent` and
// the heaviest of the others stay, `budget` in all (ties go to the lower
// index, NaN counts as -inf); they keep their order and move to
// the front of the request's blocks, K, V and weights alike.
//
// 1. evict_select_kernel finds, per (request, KV head), the weight of rank
//    budget - first - recent by a radix select over order-preserving integer
//    keys (11, 11 and 10 bits: three histograms in shared memory), then lists
//    the kept keys in order with a block-wide prefix sum.  Integer counts
//    only, so the result does not depend on the order of the atomics.  Long
//    requests are shared by a cluster of CTAs, which add their histograms
//    through distributed shared memory.  It reads 4 bytes of each key's
//    weight (from L2 after the first time), against 4 * D bytes of K and V
//    that the move reads and writes for a kept one.
// 2. evict_move_kernel copies the kept rows, 64 KB per CTA, all of a CTA's
//    loads in flight at once.  It is bound by memory.  In place it must not
//    overwrite a row that another CTA has still to read: a kept key never
//    moves to a higher index, so a segment of the result only overwrites rows
//    that the same or earlier segments read.  Each CTA takes its segment from
//    a ticket counter, loads it into registers, publishes "loaded" and, before
//    it stores, waits for the earlier segments whose rows it is about to
//    overwrite.  Earlier tickets are held by CTAs that already run and reach
//    "loaded" without waiting for anyone, so the wait ends whatever the number
//    of CTAs on the GPU (and is bounded all the same).
#include <cuda_bf16.h>

#include <climits>
#include <cmath>

#include "../../include/mvp.h"
#include "mvp_internal.cuh"
#include "ptx.cuh"

namespace mvp {

namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelPer = 4;  // elements per thread and step of the ordered pass
constexpr int kBins = 2048;
constexpr int kMoveThreads = 512;
constexpr int kMoveChunks = 8;  // 16-byte chunks in flight per thread
constexpr int kMinSegRows = 32;  // rows of a segment at the largest head_dim
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
  const uint32_t u = __float_as_uint(w != w ? -INFINITY : w + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
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

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p) {
  __shared__ int s_hist[kBins];
  __shared__ int s_warp[2][kSelWarps][2];
  __shared__ int s_bin, s_need;
  __shared__ int s_count[2];
  const int cl = static_cast<int>(cluster_size()), c = static_cast<int>(cluster_rank());
  const int bh = blockIdx.x / cl, b = bh / p.hkv, h = bh % p.hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto sync = [&]() {
    if (cl > 1) cluster_sync_all();
    else __syncthreads();
  };
  griddep_launch_dependents();
  griddep_wait();
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
  constexpr int kTile = kSelThreads * kSelPer;
  const int seg = (n + cl * kTile - 1) / (cl * kTile) * kTile;
  const int s0 = min(n, c * seg), s1 = min(n, s0 + seg);

  // ------------------------------------------------ the weight of that rank
  uint32_t prefix = 0xffffffffu, mask = 0u;  // (no key is 0xffffffff: none competes when none may stay)
  int need = p.budget - p.first - p.recent;
  if (need > 0) {
    prefix = 0u;
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
      const int bins = pass == 2 ? 1024 : kBins;
      for (int i = tid; i < kBins; i += kSelThreads) s_hist[i] = 0;
      __syncthreads();
#pragma unroll 4
      for (int j = max(s0, lo) + tid; j < min(s1, hi); j += kSelThreads) {
        const uint32_t key = order_key(w[j]);
        if ((key & mask) == prefix) atomicAdd(&s_hist[(key >> shift) & (bins - 1)], 1);
      }
      sync();
      // Bins from the heaviest down, kBins / kSelThreads per thread; the
      // cluster's counts are added up by every CTA alike.
      constexpr int kPer = kBins / kSelThreads;
      int cnt[kPer], sum = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int bin = bins - 1 - (tid * kPer + i);
        cnt[i] = 0;
        if (bin >= 0) {
          if (cl == 1) cnt[i] = s_hist[bin];
          else
            for (int r = 0; r < cl; ++r) cnt[i] += ld_cluster_s32(mapa_shared(smem_u32(&s_hist[bin]), r));
        }
        sum += cnt[i];
      }
      int incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      if (lane == 31) s_warp[0][warp][0] = incl;
      __syncthreads();
      int before = incl - sum;
      for (int i = 0; i < warp; ++i) before += s_warp[0][i][0];
      if (before < need && need <= before + sum) {  // one thread
        int at = before, i = 0;
        while (at + cnt[i] < need) at += cnt[i++];
        s_bin = bins - 1 - (tid * kPer + i);
        s_need = need - at;
      }
      __syncwarp();
      sync();  // (also: every CTA has read the others' counts)
      prefix |= static_cast<uint32_t>(s_bin) << shift;
      mask |= static_cast<uint32_t>(bins - 1) << shift;
      need = s_need;
    }
  }

  // ------------------------------------------------ the kept keys, in order
  // Class of key j: 2 stays, 1 ties with the weight of that rank (the first
  // `need` of those stay), 0 goes.
  auto cls = [&](int j) -> int {
    if (j < lo || j >= hi) return 2;
    const uint32_t key = order_key(w[j]);
    return key > prefix ? 2 : (key == prefix ? 1 : 0);
  };
  int base_g = 0, base_t = 0;  // keys of class 2 and 1 before this CTA's
  if (cl > 1) {
    int g = 0, t = 0;
#pragma unroll 4
    for (int j = s0 + tid; j < s1; j += kSelThreads) {
      const int x = cls(j);
      g += x == 2;
      t += x == 1;
    }
    g = __reduce_add_sync(0xffffffffu, g);
    t = __reduce_add_sync(0xffffffffu, t);
    if (tid < 2) s_count[tid] = 0;
    __syncthreads();
    if (lane == 0) {
      atomicAdd(&s_count[0], g);
      atomicAdd(&s_count[1], t);
    }
    cluster_sync_all();
    for (int r = 0; r < c; ++r) {
      base_g += ld_cluster_s32(mapa_shared(smem_u32(&s_count[0]), r));
      base_t += ld_cluster_s32(mapa_shared(smem_u32(&s_count[1]), r));
    }
  }
  int step = 0;
  for (int j0 = s0; j0 < s1; j0 += kTile, step ^= 1) {
    unsigned g[kSelPer], t[kSelPer];
    int ng = 0, nt = 0;
#pragma unroll
    for (int i = 0; i < kSelPer; ++i) {
      const int j = j0 + warp * (32 * kSelPer) + i * 32 + lane;
      const int x = j < s1 ? cls(j) : 0;
      g[i] = __ballot_sync(0xffffffffu, x == 2);
      t[i] = __ballot_sync(0xffffffffu, x == 1);
      ng += __popc(g[i]);
      nt += __popc(t[i]);
    }
    if (lane == 0) {
      s_warp[step][warp][0] = ng;
      s_warp[step][warp][1] = nt;
    }
    __syncthreads();  // (two buffers: the next step's writes wait for the one after)
    int gb = base_g, tb = base_t;
    for (int i = 0; i < kSelWarps; ++i) {
      const int a = s_warp[step][i][0], q = s_warp[step][i][1];
      if (i < warp) {
        gb += a;
        tb += q;
      }
      base_g += a;
      base_t += q;
    }
    const unsigned below = (1u << lane) - 1u;
#pragma unroll
    for (int i = 0; i < kSelPer; ++i) {
      const int mine_t = tb + __popc(t[i] & below);
      const bool is_t = (t[i] >> lane) & 1u;
      const int at = gb + __popc(g[i] & below) + min(mine_t, need);
      if ((((g[i] >> lane) & 1u) || (is_t && mine_t < need)) && at < p.budget)
        kept[at] = j0 + warp * (32 * kSelPer) + i * 32 + lane;
      gb += __popc(g[i]);
      tb += __popc(t[i]);
    }
  }
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

__device__ __forceinline__ void st_release(int* ptr, int v) {
  asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(ptr), "r"(v) : "memory");
}

__global__ void __launch_bounds__(kMoveThreads, 2) evict_move_kernel(const EvictParams p) {
  extern __shared__ long long s_rows[];  // [seg_rows] source rows, then [seg_rows] destination rows
  __shared__ int s_ticket, s_ok;
  const int tid = threadIdx.x;
  griddep_wait();
  if (tid == 0) {
    s_ticket = atomicAdd(p.ticket, 1);
    s_ok = 1;
  }
  __syncthreads();
  if (s_ticket >= p.num_reqs * p.hkv * p.n_segs) {  // another call runs on this workspace
    if (tid == 0) atomicCAS(p.err, 0, static_cast<int>(kDevQueueConflict));
    return;
  }
  // tickets: KV head fastest (the heads of a key share DRAM pages), then segment, then request
  const int h = s_ticket % p.hkv, rest = s_ticket / p.hkv;
  const int s = rest % p.n_segs, b = rest / p.n_segs;
  const int bh = b * p.hkv + h;
  const int n = keys_of(p, b), m = min(n, p.budget);
  const int r0 = s * p.seg_rows, rows = min(p.seg_rows, m - r0);
  if (rows <= 0) return;  // (no later segment waits for it)
  const int32_t* kept = p.kept + static_cast<size_t>(bh) * p.budget;
  int* flags = p.flags + static_cast<size_t>(bh) * p.n_segs;
  const long long wrow = weight_row(p, b, h);
  const bool last = r0 + rows == m;

  // Rows that stay where they are (the keys before the first evicted one,
  // in place) are neither read nor written.
  int moves = 0;
  for (int i = tid; i < rows; i += kMoveThreads) {
    const int j = __ldg(kept + r0 + i);
    const long long src = cache_row(p, p.bt, p.max_blocks, b, j);
    const long long dst = cache_row(p, p.bt_out, p.max_blocks_out, b, r0 + i);
    const bool move = src >= 0 && dst >= 0 && src != dst;
    s_rows[i] = move ? src : -1;
    s_rows[p.seg_rows + i] = dst;
    moves |= move || (p.w_out != p.w) || j != r0 + i;
  }
  moves = __syncthreads_or(moves);
  if (!moves && !last) {
    if (tid == 0) st_release(flags + s, 1);
    return;
  }

  // Load: 16-byte chunks of the segment's K rows, then of its V rows.
  const int cpr = p.d / 8;  // chunks per row
  const int half = rows * cpr;
  const long long row_bytes = static_cast<long long>(p.hkv) * p.d * 2, head = static_cast<long long>(h) * p.d * 2;
  uint4 buf[kMoveChunks];
#pragma unroll
  for (int u = 0; u < kMoveChunks; ++u) {
    const int x = tid + u * kMoveThreads;
    if (x < 2 * half) {
      const int y = x < half ? x : x - half;
      const long long src = s_rows[y / cpr];
      if (src >= 0)
        buf[u] = ld_stream(reinterpret_cast<const unsigned char*>(x < half ? p.k : p.v) + src * row_bytes + head +
                           16 * (y % cpr));
    }
  }
  float wv[2] = {0.f, 0.f};  // (seg_rows <= 2 * kMoveThreads)
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = tid + u * kMoveThreads;
    if (i < rows && wrow >= 0) wv[u] = *(volatile const float*)(p.w + wrow + __ldg(kept + r0 + i));
  }
  // Loaded: every thread's loads are done before the flag is seen set.
  __threadfence();
  __syncthreads();
  if (tid == 0) st_release(flags + s, 1);

  // Wait for the earlier segments that read any of the rows this one writes
  // (or, the last one, clears): those whose last key is at or past r0.
  if (tid < 32) {
    bool ok = true;
    for (int e = s - 1 - tid; e >= 0 && ok; e -= 32) {
      if (__ldg(kept + (e + 1) * p.seg_rows - 1) < r0) break;
      if (ld_acquire(flags + e) != 0) continue;
      const unsigned long long t0 = global_timer_ns();
      while (ld_acquire(flags + e) == 0) {
        if (global_timer_ns() - t0 > 1000ull * kDefaultWaitLimitUs) {
          atomicCAS(p.err, 0, static_cast<int>(kDevTimeoutOther));
          ok = false;
          break;
        }
      }
    }
    if (!ok) s_ok = 0;
  }
  __syncthreads();
  if (!s_ok) return;
#pragma unroll
  for (int u = 0; u < kMoveChunks; ++u) {
    const int x = tid + u * kMoveThreads;
    if (x < 2 * half) {
      const int y = x < half ? x : x - half;
      const int i = y / cpr;
      if (s_rows[i] >= 0)
        *reinterpret_cast<uint4*>(reinterpret_cast<unsigned char*>(x < half ? p.k : p.v) +
                                  s_rows[p.seg_rows + i] * row_bytes + head + 16 * (y % cpr)) = buf[u];
    }
  }
  if (wrow >= 0) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = tid + u * kMoveThreads;
      if (i < rows) p.w_out[wrow + r0 + i] = wv[u];
    }
    if (last)
      for (int j = m + tid; j < n; j += kMoveThreads) p.w_out[wrow + j] = 0.f;
  }
}

int seg_rows_for(int d) { return kMoveThreads * kMoveChunks / 2 / (d / 8); }

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
  // CTAs per (request, KV head): enough to fill the GPU with two per SM, at
  // most eight, none with fewer than 4096 keys.
  int cl = 1;
  while (cl < 8 && bh * cl * 2 <= 2LL * num_sms && max_k_len / (2 * cl) >= 4096) cl *= 2;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cl;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(bh * cl));
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  if (cudaLaunchKernelEx(&cfg, evict_select_kernel, p) != cudaSuccess) return MVP_ERR_CUDA;
  cfg.attrs = attr + 1;
  cfg.gridDim = dim3(static_cast<unsigned>(bh * p.n_segs));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.dynamicSmemBytes = 2 * p.seg_rows * sizeof(long long);
  if (cudaLaunchKernelEx(&cfg, evict_move_kernel, p) != cudaSuccess) return MVP_ERR_CUDA;
  set_last_launches(2);
  return MVP_OK;
}

}  // extern "C"
