// The attention weight each key received, sm_103a.
//
//   w[h, j] (+)= sum over the rows i that see key j and the G query heads g of
//                KV head h of exp(scale q_ig . k_jh [+ sink_g if j = 0] - lse_ig)
//
// with the lse that the attention call left: the column sums of its
// probabilities, which an eviction policy accumulates per cached key.
//
// The scores are computed transposed, S^T = K Q^T, so that a TMEM lane is a
// key and its columns are (position, head) pairs: a thread owns a key, sums its
// own columns in fp32 registers, and nothing is reduced across threads.  No
// atomics: the sums are the same in every run.
//
// Prefill rows: a CTA keeps a 128-key block of one KV head in shared memory
// (the A operand, loaded once) and streams the query tiles that see any of it,
// 128 columns = 128 / G positions x G heads, through a ring of 64-dim chunks
// (the B operand).  Work: 2 D flops and one exponential per visible (row, key)
// and head; at D = 128 the exponentials (16384 per 128 x 128 tile) cost as much
// as the MMA, so both must overlap: S^T is double-buffered in TMEM, one thread
// issues the MMAs, two warpgroups of epilogue warps split each tile's columns.
// Visibility is a closed interval of columns per key (the causal and window
// rules solved for the row), so a masked tile costs one bit mask per 32
// columns; tiles seen whole skip it.  Only range-table rows need a test per
// column, in the tiles that hold such a row.
//
// Single-token rows: K is streamed (the A operand, 64-dim chunks of 128 keys),
// the row's G heads are the B operand (N = G rounded up to 16); bound by the
// one read of K.
#include <cuda_bf16.h>

#include <algorithm>
#include <climits>
#include <mutex>

#include "../../include/mvp.h"
#include "mask.cuh"
#include "mvp_internal.cuh"
#include "ptx.cuh"

namespace mvp {

namespace {

constexpr int kKeys = 128;        // keys of a block: the MMA's M
constexpr int kCols = 128;        // columns of a query tile: the MMA's N (prefill rows)
constexpr int kChunkBytes = 128 * 128;  // 128 rows x 64 dims of bf16, 128-byte swizzled
constexpr float kLog2e = 1.4426950408889634f;
constexpr unsigned kFull = 0xffffffffu;

struct KwParams {
  MaskParams m;
  const float* lse;        // [hq, total_q]
  float* w;                // [num_slots, hkv, w_stride]
  float* partial;          // [splits, num_reqs, hkv, n_kb * 128] or null (one split)
  const int32_t* slots;    // or null
  int num_slots;
  long long w_stride;
  int accumulate;
  int num_reqs, hq, hkv, group;
  int req_offset;          // prefill kernel: first request it covers
  int skip_decode;         // prefill kernel: leave single-token requests
  int npos;                // query positions per tile
  int n_kb;                // key blocks (prefill) or key chunks (decode) of max_k_len
  int splits;              // parts the query tiles of a key block are shared by
  int max_k_len;
  int* err;
};

// Geometry of request b.
struct Req {
  int q0, q_len, k0, k_len, ctx;
};

template <bool PAGED>
__device__ __forceinline__ Req load_req(const KwParams& p, int b) {
  Req r;
  r.q0 = __ldg(p.m.cu_q + b);
  r.q_len = __ldg(p.m.cu_q + b + 1) - r.q0;
  if constexpr (PAGED) {
    r.k0 = 0;
    r.k_len = __ldg(p.m.seq_k + b);
  } else {
    r.k0 = __ldg(p.m.cu_k + b);
    r.k_len = __ldg(p.m.cu_k + b + 1) - r.k0;
  }
  r.ctx = p.m.ctx_lens ? __ldg(p.m.ctx_lens + b) : (r.k_len - r.q_len);
  r.k_len = min(r.k_len, p.max_k_len);
  if (r.q_len > 0) (void)in_bounds(r.q0 + r.q_len - 1, p.m.total_q, p.err);
  return r;
}

__device__ __forceinline__ float* weight_row(const KwParams& p, int b, int h) {
  const int slot = p.slots != nullptr ? __ldg(p.slots + b) : b;
  if (!in_bounds(slot, p.num_slots, p.err)) return nullptr;
  return p.w + (static_cast<long long>(slot) * p.hkv + h) * p.w_stride;
}

// Positions that see key j by the causal / window / first-token rules, as a
// closed interval (64-bit: positions and windows may be any int32).
__device__ __forceinline__ void seen_by(const MaskParams& m, int j, long long& lo, long long& hi) {
  const long long far = 1LL << 40;
  lo = m.causal ? j : (m.window_right >= 0 ? static_cast<long long>(j) - m.window_right : -far);
  hi = (m.window_left >= 0 && j >= m.first_tokens) ? static_cast<long long>(j) + m.window_left : far;
}

// Range entry of packed row (q0 + i) at position pos, clamped as the mask
// does; empty (1, 0) without one.
__device__ __forceinline__ int2 range_of(const MaskParams& m, const Req& r, int i) {
  const RowVis v = row_visibility(m, r.ctx + i, r.k_len, true, r.q0 + i, 0);
  return make_int2(v.r_lo, v.r_hi);
}

// ------------------------------------------------------------------ prefill rows
constexpr int kPfThreads = 384;  // producer, MMA, column and idle warps, 8 epilogue warps
constexpr int kMaxTileBits = 4096;
constexpr int kInfo = 4;  // column-info slots

template <int NCH>
struct PfCfg {
  static constexpr int STAGES = NCH <= 2 ? 4 : (NCH == 4 ? 8 : 5);  // Q chunks in flight
  static constexpr int K_BYTES = NCH * kChunkBytes;
  static constexpr int SMEM = K_BYTES + STAGES * kChunkBytes + 1024;
  static constexpr int CTAS = SMEM <= 110 * 1024 ? 2 : 1;
};

struct ColInfo {
  float nl2[kCols];   // -lse * log2(e); -inf for columns without a row
  float sink[kCols];  // key-0 sinks in log2 units (key-0 mode)
  int2 rng[kCols];    // range interval of the column's row (tiles with ranges)
};

template <int NCH>
struct __align__(16) PfShared {
  ColInfo info[kInfo];
  uint32_t range_bits[kMaxTileBits / 32];  // tiles with a row whose range meets this key block
  float part[kKeys];                       // second epilogue warpgroup's sums
  uint64_t k_full;
  uint64_t q_full[8], q_empty[8];
  uint64_t s_full[2], s_empty[2];
  uint64_t col_full[kInfo], col_empty[kInfo];
  uint64_t final_mma;
  uint32_t tmem_base;
  WaitCtl wc;
};

// The query tiles a CTA visits: [t_lo, t_hi) by the closed-form rules and, with
// a range table, the earlier ones whose bit is set; every role walks them alike.
struct TileWalk {
  int t, t_lo, t_hi;
  const uint32_t* bits;  // null: no ranges
  bool all;              // more tiles than bits: visit every one
  __device__ __forceinline__ bool ranged(int x) const {
    return bits != nullptr && (all || ((bits[x >> 5] >> (x & 31)) & 1u));
  }
  __device__ __forceinline__ bool next() {  // t: the tile to visit
    ++t;
    while (t < t_hi && t < t_lo && !ranged(t)) ++t;
    return t < t_hi;
  }
};

template <int NCH, bool PAGED>
__global__ void __launch_bounds__(kPfThreads, PfCfg<NCH>::CTAS)
    key_weights_prefill_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                               const KwParams p) {
  using C = PfCfg<NCH>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = smem;
  uint8_t* sQ = smem + C::K_BYTES;
  __shared__ PfShared<NCH> sb;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  griddep_wait();
  int x = blockIdx.x;
  const int kb = x % p.n_kb;
  x /= p.n_kb;
  const int split = x % p.splits;
  x /= p.splits;
  const int h = x % p.hkv;
  const int b = x / p.hkv + p.req_offset;
  const Req r = load_req<PAGED>(p, b);
  const int ja = kb * kKeys, jb = min(ja + kKeys, r.k_len) - 1;
  if (jb < ja || (p.skip_decode && r.q_len == 1)) return;
  const bool use_table = table_active(p.m);

  // Tiles by the closed-form rules: positions [lo of the first key, hi of the
  // last], where a first token's hi is unbounded.
  TileWalk walk;
  const int n_tiles = (r.q_len + p.npos - 1) / p.npos;
  {
    long long lo_a, hi_a, lo_b, hi_b;
    seen_by(p.m, ja, lo_a, hi_a);
    seen_by(p.m, jb, lo_b, hi_b);
    const long long lo = max(lo_a - r.ctx, 0LL), hi = min(max(hi_a, hi_b) - r.ctx, static_cast<long long>(r.q_len) - 1);
    walk.t_lo = static_cast<int>(min(lo / p.npos, static_cast<long long>(n_tiles)));
    walk.t_hi = hi < 0 ? 0 : static_cast<int>(hi / p.npos) + 1;
    walk.bits = use_table ? sb.range_bits : nullptr;
    walk.all = n_tiles > kMaxTileBits;
  }
  if (use_table && !walk.all) {
    for (int i = threadIdx.x; i < kMaxTileBits / 32; i += kPfThreads) sb.range_bits[i] = 0;
    __syncthreads();
    const int rows = min(walk.t_hi * p.npos, r.q_len);
    for (int i = threadIdx.x; i < rows; i += kPfThreads) {
      const int2 e = range_of(p.m, r, i);
      if (max(e.x, ja) <= min(e.y, jb)) atomicOr(&sb.range_bits[(i / p.npos) >> 5], 1u << ((i / p.npos) & 31));
    }
  }
  // This split's part of the tiles (the closed-form ones and those before).
  {
    const int first = use_table ? 0 : walk.t_lo;
    const long long n = max(walk.t_hi - first, 0);
    const int a = first + static_cast<int>(n * split / p.splits), e = first + static_cast<int>(n * (split + 1) / p.splits);
    walk.t_hi = e;
    walk.t_lo = max(walk.t_lo, a);
    walk.t = a - 1;
  }

  if (threadIdx.x == 0) {
    mbar_init(&sb.k_full, 1);
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&sb.q_full[i], 1);
      mbar_init(&sb.q_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sb.s_full[i], 1);
      mbar_init(&sb.s_empty[i], 8);
    }
    for (int i = 0; i < kInfo; ++i) {
      mbar_init(&sb.col_full[i], 1);
      mbar_init(&sb.col_empty[i], 8);
    }
    mbar_init(&sb.final_mma, 1);
    sb.wc.abort = 0;
    sb.wc.limit_us = p.m.wait_limit_us;
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc(&sb.tmem_base, 2 * kCols);
    tmem_relinquish();
  }
  // Rows of a Q chunk that no copy writes (128 is not a multiple of the group):
  // zero, so that their columns are finite.
  const int ncol = p.npos * p.group;
  if (ncol < kCols) {
    const int words = (kCols - ncol) * 8;  // 16-byte words at the end of each chunk
    for (int i = threadIdx.x; i < C::STAGES * words; i += kPfThreads)
      reinterpret_cast<uint4*>(sQ + (i / words) * kChunkBytes + ncol * 128)[i % words] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sb.tmem_base;

  if (warp == 0) {
    // ---------------------------------------------------------------- loads
    if (lane == 0) {
      bool ok = true;
      int n = 0;  // chunks issued
      bool k_loaded = false;
      const uint32_t q_bytes = static_cast<uint32_t>(ncol) * 128;
      while (ok && walk.next()) {
        if (!k_loaded) {
          k_loaded = true;
          mbar_arrive_expect_tx(&sb.k_full, C::K_BYTES);
          const int run = PAGED ? min(kKeys, 1 << p.m.block_shift) : kKeys;
          for (int i = 0; i < kKeys; i += run) {
            const int row = PAGED ? kv_row(p.m, b, 0, r.k_len, ja + i) : r.k0 + ja;
#pragma unroll
            for (int c = 0; c < NCH; ++c)
              tma_load_3d(sK + c * kChunkBytes + i * 128, &map_k, &sb.k_full, c * 64, h, row);
          }
        }
        for (int c = 0; ok && c < NCH; ++c, ++n) {
          const int s = n % C::STAGES;
          if (n >= C::STAGES && !mbar_wait(&sb.q_empty[s], ((n / C::STAGES) - 1) & 1, &sb.wc, p.err, kDevTimeoutLoad)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&sb.q_full[s], q_bytes);
          tma_load_3d(sQ + s * kChunkBytes, &map_q, &sb.q_full[s], c * 64, h * p.group, r.q0 + walk.t * p.npos);
        }
      }
      if (!ok) sb.wc.abort = 1;
      WaitCtl own = own_wait_ctl(&sb.wc);  // copies in flight complete before the CTA leaves
      if (k_loaded) mbar_wait(&sb.k_full, 0, &own, nullptr, 0);
      for (int s = 0; s < C::STAGES && s < n; ++s) mbar_wait(&sb.q_full[s], ((n - 1 - s) / C::STAGES) & 1, &own, nullptr, 0);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMAs
    constexpr uint32_t idesc = idesc_bf16_f32(kKeys, kCols, false, false);
    const uint64_t dk = smem_desc_sw128(smem_u32(sK), 16, 1024);
    const uint64_t dq = smem_desc_sw128(smem_u32(sQ), 16, 1024);
    const bool issuer = elect_one();
    bool ok = true;
    int n = 0;  // chunks
    for (int i = 0; ok && walk.next(); ++i) {
      if (i == 0) ok = mbar_wait(&sb.k_full, 0, &sb.wc, p.err, kDevTimeoutLoad);
      if (ok && i >= 2) ok = mbar_wait(&sb.s_empty[i & 1], ((i >> 1) - 1) & 1, &sb.wc, p.err, kDevTimeoutSoftmax);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + (i & 1) * kCols;
      for (int c = 0; c < NCH; ++c, ++n) {
        const int s = n % C::STAGES;
        if (!mbar_wait_spin(&sb.q_full[s], (n / C::STAGES) & 1, &sb.wc, p.err, kDevTimeoutLoad)) {
          ok = false;
          break;
        }
        if (issuer) {
#pragma unroll
          for (int k16 = 0; k16 < 4; ++k16)
            mma_ss_one<1>(d, desc_add(dk, static_cast<uint32_t>((c * kChunkBytes + k16 * 32) >> 4)),
                          desc_add(dq, static_cast<uint32_t>((s * kChunkBytes + k16 * 32) >> 4)), idesc,
                          (c | k16) != 0 ? 1u : 0u);
        }
        __syncwarp();
        mma_commit_elect<1>(&sb.q_empty[s]);
      }
      if (ok) mma_commit_elect<1>(&sb.s_full[i & 1]);
    }
    if (!ok && lane == 0) sb.wc.abort = 1;
    mma_commit_elect<1>(&sb.final_mma);
    WaitCtl own = own_wait_ctl(&sb.wc);
    mbar_wait(&sb.final_mma, 0, &own, p.err, kDevTimeoutMma);
  } else if (warp == 2) {
    // ---------------------------------------------------------------- column info
    bool ok = true;
    const bool key0 = p.m.sink_mode == 1 && p.m.sinks != nullptr;
    // This lane's columns lane + 32 k: row within the tile, and the lse of it.
    int pos[4];
    const float* src[4];
    float sink[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = lane + 32 * k, g = c % p.group;
      pos[k] = c < ncol ? c / p.group : INT_MAX / 2;
      src[k] = p.lse + static_cast<size_t>(h * p.group + g) * p.m.total_q + r.q0 + c / p.group;
      sink[k] = key0 && c < ncol ? __ldg(p.m.sinks + h * p.group + g) * kLog2e : 0.f;
    }
    auto load = [&](int t, float (&nl)[4]) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int row = t * p.npos + pos[k];
        nl[k] = row < r.q_len && in_bounds(r.q0 + row, p.m.total_q, p.err) ? __ldg(src[k] + t * p.npos) : INFINITY;
      }
    };
    float nl[4], next_nl[4];
    bool have = walk.next();
    if (have) load(walk.t, nl);
    for (int i = 0; ok && have; ++i) {
      const int slot = i % kInfo, t = walk.t;
      // the next tile's loads are in flight while this one waits for its slot
      have = walk.next();
      if (have) load(walk.t, next_nl);
      if (i >= kInfo) ok = mbar_wait(&sb.col_empty[slot], ((i / kInfo) - 1) & 1, &sb.wc, p.err, kDevTimeoutOther);
      if (!__all_sync(kFull, ok)) break;
      ColInfo& f = sb.info[slot];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = lane + 32 * k, row = t * p.npos + pos[k];
        f.nl2[c] = -kLog2e * nl[k];
        if (key0) f.sink[c] = sink[k];
        if (walk.ranged(t)) f.rng[c] = row < r.q_len ? range_of(p.m, r, row) : make_int2(1, 0);
        nl[k] = next_nl[k];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sb.col_full[slot]);
    }
    if (!ok) sb.wc.abort = 1;
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- exponentials and sums
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const int row = quarter * 32 + lane, key = ja + row;
    const uint32_t base = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * (kCols / 2);
    const float sc = p.m.scale_log2;
    const uint64_t sc2 = f2_pack(sc, sc);
    const bool key0 = p.m.sink_mode == 1 && p.m.sinks != nullptr && ja == 0;
    long long p_lo, p_hi;
    seen_by(p.m, key, p_lo, p_hi);
    if (key > jb) p_hi = p_lo - 1;
    // tiles all of whose rows see every key of the block: positions [in_lo, in_hi]
    long long in_lo, in_hi, tmp;
    seen_by(p.m, jb, in_lo, tmp);
    seen_by(p.m, ja, tmp, in_hi);
    if (jb >= p.m.first_tokens && ja < p.m.first_tokens) in_hi = min(in_hi, static_cast<long long>(p.m.first_tokens) + p.m.window_left);
    uint64_t acc[2] = {0ull, 0ull};
    bool ok = true;
    for (int i = 0; walk.next(); ++i) {
      const int slot = i % kInfo;
      ok = mbar_wait(&sb.col_full[slot], (i / kInfo) & 1, &sb.wc, p.err, kDevTimeoutOther);
      if (ok) ok = mbar_wait(&sb.s_full[i & 1], (i >> 1) & 1, &sb.wc, p.err, kDevTimeoutMma);
      if (!ok) break;
      tc_fence_after();
      const ColInfo& f = sb.info[slot];
      const int row0 = walk.t * p.npos;             // the tile's first row
      const int valid = min(p.npos, r.q_len - row0);  // rows of the request in it
      const long long p0 = static_cast<long long>(r.ctx) + row0;
      const bool ranged = walk.ranged(walk.t);
      const bool whole = valid == p.npos && p0 >= in_lo && p0 + valid - 1 <= in_hi && !ranged && !key0;
      // columns of the tile that see this thread's key: [c_lo, c_hi]
      const int c_lo = static_cast<int>(min(max(p_lo - p0, 0LL), static_cast<long long>(valid))) * p.group;
      const int c_hi = static_cast<int>(min(max(p_hi - p0 + 1, 0LL), static_cast<long long>(valid))) * p.group - 1;
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        uint32_t s[32];
        tmem_ld_32x32b_x32(base + (i & 1) * kCols + cc * 32, s);
        tmem_ld_wait(s);
        if (cc == 1) {  // the scores are in registers: the buffer is free
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sb.s_empty[i & 1]);
        }
        const int col0 = half * (kCols / 2) + cc * 32;
        if (whole) {
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const float4 nl = *reinterpret_cast<const float4*>(&f.nl2[col0 + 4 * q]);
            float a0, a1, a2, a3;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(s[4 * q]), __uint_as_float(s[4 * q + 1])), sc2, f2_pack(nl.x, nl.y)), a0, a1);
            f2_unpack(f2_fma(f2_pack(__uint_as_float(s[4 * q + 2]), __uint_as_float(s[4 * q + 3])), sc2, f2_pack(nl.z, nl.w)), a2, a3);
            acc[0] = f2_add(acc[0], f2_pack(ex2_approx(a0), ex2_approx(a1)));
            acc[1] = f2_add(acc[1], f2_pack(ex2_approx(a2), ex2_approx(a3)));
          }
        } else {
          uint32_t bits = interval_bits(c_lo, c_hi, col0);
          if (ranged && key <= jb) {
#pragma unroll 8
            for (int q = 0; q < 32; ++q) {
              const int2 e = f.rng[col0 + q];
              bits |= static_cast<uint32_t>(key >= e.x && key <= e.y) << q;
            }
          }
          if (bits != 0u) {
            float sum = 0.f;
#pragma unroll
            for (int q = 0; q < 32; ++q) {
              float v = fmaf(__uint_as_float(s[q]), sc, f.nl2[col0 + q]);
              if (key0 && key == 0) v += f.sink[col0 + q];
              sum += ((bits >> q) & 1u) ? ex2_approx(v) : 0.f;
            }
            acc[0] = f2_add(acc[0], f2_pack(sum, 0.f));
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sb.col_empty[slot]);
    }
    if (!ok) sb.wc.abort = 1;
    float x0, x1, x2, x3;
    f2_unpack(acc[0], x0, x1);
    f2_unpack(acc[1], x2, x3);
    const float mine = (x0 + x1) + (x2 + x3);
    if (half == 1) sb.part[row] = mine;
    named_barrier(1, 256);
    if (half == 0 && key <= jb) {
      const float total = mine + sb.part[row];
      if (p.partial != nullptr) {
        p.partial[((static_cast<size_t>(split) * p.num_reqs + b) * p.hkv + h) * (static_cast<size_t>(p.n_kb) * kKeys) + key] = total;
      } else {
        float* w = weight_row(p, b, h);
        if (w != nullptr) w[key] = p.accumulate ? w[key] + total : total;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 2 * kCols);
}

// Adds the splits' partial sums up, in their order.
template <bool PAGED>
__global__ void __launch_bounds__(256) key_weights_combine_kernel(const KwParams p) {
  griddep_wait();
  const int h = blockIdx.y, b = blockIdx.z + p.req_offset;
  const Req r = load_req<PAGED>(p, b);
  if (p.skip_decode && r.q_len == 1) return;
  const int key = blockIdx.x * 256 + threadIdx.x;
  if (key >= r.k_len) return;
  const size_t row = static_cast<size_t>(p.n_kb) * kKeys;
  float total = 0.f;
  for (int s = 0; s < p.splits; ++s) total += p.partial[((static_cast<size_t>(s) * p.num_reqs + b) * p.hkv + h) * row + key];
  float* w = weight_row(p, b, h);
  if (w != nullptr) w[key] = p.accumulate ? w[key] + total : total;
}

// ------------------------------------------------------------------ single-token rows
constexpr int kDecTiles = 16;  // key tiles of a CTA
constexpr int kDecStages = 6;  // K chunks in flight
constexpr int kDecThreads = 192;  // producer, MMA and 4 epilogue warps

template <int NCH>
struct DecCfg {
  static constexpr int Q_BYTES(int n) { return NCH * n * 128; }
};

struct __align__(16) DecShared {
  float nl2[kCols];
  float sink[kCols];
  uint64_t q_full;
  uint64_t k_full[kDecStages], k_empty[kDecStages];
  uint64_t s_full[2], s_empty[2];
  uint64_t final_mma;
  uint32_t tmem_base;
  WaitCtl wc;
};

template <int NCH, bool PAGED>
__global__ void __launch_bounds__(kDecThreads)
    key_weights_decode_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                              const KwParams p, const int n, const int tmem_cols) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = smem;
  uint8_t* sQ = smem + kDecStages * kChunkBytes;
  __shared__ DecShared sb;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_wait();
  const int b = blockIdx.z, h = blockIdx.y;
  const Req r = load_req<PAGED>(p, b);
  if (r.q_len != 1) return;
  const int key_lo = blockIdx.x * (kDecTiles * kKeys);
  if (key_lo >= r.k_len) return;
  const int tiles = min(kDecTiles, (r.k_len - key_lo + kKeys - 1) / kKeys);
  const RowVis vis = row_visibility(p.m, r.ctx, r.k_len, table_active(p.m), r.q0, b);
  const int f_hi = p.m.first_tokens > 0 ? first_tokens_hi(p.m, r.ctx, r.k_len) : -1;
  auto meets = [&](int i) {  // the row sees a key of tile i
    const int a = key_lo + i * kKeys, e = a + kKeys - 1;
    return max(a, vis.b_lo) <= min(e, vis.b_hi) || max(a, vis.r_lo) <= min(e, vis.r_hi) || a <= f_hi;
  };
  if (threadIdx.x == 0) {
    mbar_init(&sb.q_full, 1);
    for (int i = 0; i < kDecStages; ++i) {
      mbar_init(&sb.k_full[i], 1);
      mbar_init(&sb.k_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sb.s_full[i], 1);
      mbar_init(&sb.s_empty[i], 4);
    }
    mbar_init(&sb.final_mma, 1);
    sb.wc.abort = 0;
    sb.wc.limit_us = p.m.wait_limit_us;
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc(&sb.tmem_base, tmem_cols);
    tmem_relinquish();
  }
  for (int g = threadIdx.x; g < p.group; g += kDecThreads) {
    sb.nl2[g] = -kLog2e * __ldg(p.lse + static_cast<size_t>(h * p.group + g) * p.m.total_q + r.q0);
    sb.sink[g] = p.m.sink_mode == 1 && p.m.sinks != nullptr ? __ldg(p.m.sinks + h * p.group + g) * kLog2e : 0.f;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sb.tmem_base;

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      int c = 0;
      const int run = PAGED ? min(kKeys, 1 << p.m.block_shift) : kKeys;
      mbar_arrive_expect_tx(&sb.q_full, static_cast<uint32_t>(NCH * p.group * 128));
      for (int x = 0; x < NCH; ++x) tma_load_3d(sQ + x * n * 128, &map_q, &sb.q_full, x * 64, h * p.group, r.q0);
      for (int i = 0; ok && i < tiles; ++i) {
        if (!meets(i)) continue;
        for (int x = 0; x < NCH; ++x, ++c) {
          const int s = c % kDecStages;
          if (c >= kDecStages && !mbar_wait(&sb.k_empty[s], ((c / kDecStages) - 1) & 1, &sb.wc, p.err, kDevTimeoutLoad)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&sb.k_full[s], kChunkBytes);
          for (int k = 0; k < kKeys; k += run) {
            const int key = key_lo + i * kKeys + k;
            const int row = PAGED ? kv_row(p.m, b, 0, r.k_len, key) : r.k0 + key;
            tma_load_3d(sK + s * kChunkBytes + k * 128, &map_k, &sb.k_full[s], x * 64, h, row);
          }
        }
      }
      if (!ok) sb.wc.abort = 1;
      WaitCtl own = own_wait_ctl(&sb.wc);
      mbar_wait(&sb.q_full, 0, &own, nullptr, 0);
      for (int s = 0; s < kDecStages && s < c; ++s) mbar_wait(&sb.k_full[s], ((c - 1 - s) / kDecStages) & 1, &own, nullptr, 0);
    }
  } else if (warp == 1) {
    const uint32_t idesc = idesc_bf16_f32(kKeys, n, false, false);
    const uint64_t dk = smem_desc_sw128(smem_u32(sK), 16, 1024);
    const uint64_t dq = smem_desc_sw128(smem_u32(sQ), 16, 1024);
    const bool issuer = elect_one();
    bool ok = mbar_wait(&sb.q_full, 0, &sb.wc, p.err, kDevTimeoutLoad);
    int c = 0, j = 0;
    for (int i = 0; ok && i < tiles; ++i) {
      if (!meets(i)) continue;
      if (j >= 2 && !mbar_wait(&sb.s_empty[j & 1], ((j >> 1) - 1) & 1, &sb.wc, p.err, kDevTimeoutSoftmax)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t d = tmem + (j & 1) * n;
      for (int x = 0; x < NCH; ++x, ++c) {
        const int s = c % kDecStages;
        if (!mbar_wait(&sb.k_full[s], (c / kDecStages) & 1, &sb.wc, p.err, kDevTimeoutLoad)) {
          ok = false;
          break;
        }
        if (issuer) {
#pragma unroll
          for (int k16 = 0; k16 < 4; ++k16)
            mma_ss_one<1>(d, desc_add(dk, static_cast<uint32_t>((s * kChunkBytes + k16 * 32) >> 4)),
                          desc_add(dq, static_cast<uint32_t>((x * n * 128 + k16 * 32) >> 4)), idesc,
                          (x | k16) != 0 ? 1u : 0u);
        }
        __syncwarp();
        mma_commit_elect<1>(&sb.k_empty[s]);
      }
      if (ok) mma_commit_elect<1>(&sb.s_full[j & 1]);
      ++j;
    }
    if (!ok && lane == 0) sb.wc.abort = 1;
    mma_commit_elect<1>(&sb.final_mma);
    WaitCtl own = own_wait_ctl(&sb.wc);
    mbar_wait(&sb.final_mma, 0, &own, p.err, kDevTimeoutMma);
  } else {
    const int quarter = warp & 3;
    const uint32_t base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    float* w = weight_row(p, b, h);
    bool ok = true;
    int j = 0;
    for (int i = 0; i < tiles; ++i) {
      const int key = key_lo + i * kKeys + quarter * 32 + lane;
      float total = 0.f;
      const bool visit = meets(i);
      if (visit) {
        ok = mbar_wait(&sb.s_full[j & 1], (j >> 1) & 1, &sb.wc, p.err, kDevTimeoutMma);
        if (!ok) break;
        tc_fence_after();
        const bool see = key < r.k_len && (vis.visible(key) || key <= f_hi);
        for (int n0 = 0; n0 < n; n0 += 16) {
          uint32_t s[16];
          tmem_ld_32x32b_x16(base + (j & 1) * n + n0, s);
          tmem_ld_wait16(s);
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            if (n0 + q < p.group) {
              float v = fmaf(__uint_as_float(s[q]), p.m.scale_log2, sb.nl2[n0 + q]);
              if (key == 0) v += sb.sink[n0 + q];
              total += ex2_approx(v);
            }
          }
        }
        if (!see) total = 0.f;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sb.s_empty[j & 1]);
        ++j;
      }
      if (w != nullptr && key < r.k_len) {
        if (!p.accumulate) w[key] = total;
        else if (visit) w[key] += total;
      }
    }
    if (!ok) sb.wc.abort = 1;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, tmem_cols);
}

std::mutex g_kw_mutex;

// Sets a kernel's dynamic shared memory attribute once per device.
template <class K>
cudaError_t set_smem(K kern, int bytes, bool (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_kw_mutex);
  if (done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done[dev] = true;
  return e;
}

template <int NCH, bool PAGED>
cudaError_t launch_prefill_rows(const KwParams& p, const CUtensorMap& mq, const CUtensorMap& mk, long long ctas,
                                cudaStream_t stream) {
  static bool done[64] = {};
  cudaError_t e = set_smem(key_weights_prefill_kernel<NCH, PAGED>, PfCfg<NCH>::SMEM, done);
  if (e != cudaSuccess) return e;
  key_weights_prefill_kernel<NCH, PAGED><<<static_cast<unsigned>(ctas), kPfThreads, PfCfg<NCH>::SMEM, stream>>>(mq, mk, p);
  return cudaGetLastError();
}

template <int NCH, bool PAGED>
cudaError_t launch_decode_rows(const KwParams& p, int reqs, const CUtensorMap& mq, const CUtensorMap& mk,
                               cudaStream_t stream) {
  static bool done[64] = {};
  constexpr int kMost = kDecStages * kChunkBytes + NCH * kCols * 128 + 1024;
  cudaError_t e = set_smem(key_weights_decode_kernel<NCH, PAGED>, kMost, done);
  if (e != cudaSuccess) return e;
  const int n = (p.group + 15) / 16 * 16;
  int cols = 32;
  while (cols < 2 * n) cols *= 2;
  const int smem = kDecStages * kChunkBytes + NCH * n * 128 + 1024;
  key_weights_decode_kernel<NCH, PAGED><<<dim3(p.n_kb, p.hkv, reqs), kDecThreads, smem, stream>>>(mq, mk, p, n, cols);
  return cudaGetLastError();
}

// Parts the query tiles of a key block are shared by: enough CTAs for two
// rounds, not fewer than eight tiles each.
int split_count(int num_reqs, int hkv, int max_q_len, int max_k_len, int npos, int num_sms) {
  const long long blocks = static_cast<long long>(num_reqs) * hkv * ((max_k_len + kKeys - 1) / kKeys);
  const int tiles = (max_q_len + npos - 1) / npos;
  int s = 1;
  while (s < 16 && blocks * s < 2LL * num_sms && tiles / (2 * s) >= 8) s *= 2;
  return s;
}

int key_weights_impl(const void* q, const void* k, const float* lse, float* weights, int num_slots,
                     long long weight_stride, const int32_t* slots, int accumulate, const int32_t* cu_seqlens_q,
                     const int32_t* context_lens, int num_reqs, int total_q, int max_q_len, int max_k_len,
                     int num_decode_reqs, int num_heads_q, int num_heads_kv, int head_dim, const int32_t* range_table,
                     const int32_t* range_covered, int causal, int window_left, int window_right, int first_tokens,
                     const float* sinks, int sink_mode, float scale, void* workspace, size_t workspace_bytes,
                     void* stream, const int32_t* cu_k, const int32_t* seq_k, const int32_t* block_table,
                     long long kv_rows, int block_shift, int max_blocks) {
  const bool paged = block_table != nullptr;
  if (num_reqs < 1 || num_reqs > 65535 || total_q < 0 || kv_rows < 0) return MVP_ERR_ARG;
  if (num_heads_q < 1 || num_heads_kv < 1 || num_heads_q % num_heads_kv != 0) return MVP_ERR_ARG;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256 && head_dim != 512) return MVP_ERR_UNSUPPORTED;
  if (num_heads_q / num_heads_kv > kCols || num_heads_kv > 65535) return MVP_ERR_UNSUPPORTED;
  if (sink_mode < 0 || sink_mode > 2 || (sink_mode != 0 && sinks == nullptr)) return MVP_ERR_ARG;
  if (window_left < -1 || window_right < -1 || first_tokens < 0) return MVP_ERR_ARG;
  if ((causal != 0 && causal != 1) || (accumulate != 0 && accumulate != 1)) return MVP_ERR_ARG;
  if (num_decode_reqs < -1 || num_decode_reqs > num_reqs) return MVP_ERR_ARG;
  if (!(scale > 0.f) || scale > 3.0e38f) return MVP_ERR_ARG;  // NaN, <= 0, inf
  if (max_q_len < 0 || max_k_len < 0 || num_slots < 0) return MVP_ERR_ARG;
  if (weight_stride < max_k_len || (slots == nullptr && num_slots < num_reqs)) return MVP_ERR_ARG;
  if (total_q == 0 && accumulate) return MVP_OK;  // nothing to add
  if (kv_rows < 1 || kv_rows > INT_MAX || max_q_len < 1 || max_k_len < 1 || total_q < 1) return MVP_ERR_ARG;
  if (q == nullptr || k == nullptr || lse == nullptr || weights == nullptr || cu_seqlens_q == nullptr ||
      (paged ? seq_k == nullptr : cu_k == nullptr))
    return MVP_ERR_ARG;
  if (((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k)) & 15u) != 0) return MVP_ERR_UNSUPPORTED;
  if (range_table != nullptr && (reinterpret_cast<uintptr_t>(range_table) & 7u) != 0) return MVP_ERR_UNSUPPORTED;
  int* err = nullptr;
  int num_sms = 1;
  if (device_error_word(&err, &num_sms) != cudaSuccess) return MVP_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);

  KwParams p{};
  MaskParams& m = p.m;
  m.cu_q = cu_seqlens_q;
  m.cu_k = paged ? nullptr : cu_k;
  m.seq_k = paged ? seq_k : nullptr;
  m.block_table = block_table;
  m.block_shift = paged ? block_shift : 0;
  m.max_blocks = paged ? max_blocks : 0;
  m.ctx_lens = context_lens;
  m.table = range_table;
  m.covered = range_table ? range_covered : nullptr;
  m.sinks = sink_mode ? sinks : nullptr;
  m.causal = causal;
  m.window_left = window_left;
  m.window_right = causal ? 0 : window_right;
  m.first_tokens = window_left < 0 ? 0 : first_tokens;
  m.sink_mode = sink_mode;
  m.scale_log2 = scale * kLog2e;
  m.scale = scale;
  m.wait_limit_us = kDefaultWaitLimitUs;
  m.total_q = total_q;
  m.err = err;
  p.lse = lse;
  p.w = weights;
  p.slots = slots;
  p.num_slots = num_slots;
  p.w_stride = weight_stride;
  p.accumulate = accumulate;
  p.num_reqs = num_reqs;
  p.hq = num_heads_q;
  p.hkv = num_heads_kv;
  p.group = num_heads_q / num_heads_kv;
  p.npos = kCols / p.group;
  p.max_k_len = max_k_len;
  p.err = err;

  const int decode_count = num_decode_reqs < 0 ? num_reqs : num_decode_reqs;
  const int first = num_decode_reqs < 0 ? 0 : num_decode_reqs;
  // Requests without queries (q_len 0) are set to 0 by the prefill kernel.
  const bool run_prefill = first < num_reqs && (max_q_len > 1 || !accumulate);
  const int box = paged ? std::min(kKeys, 1 << block_shift) : kKeys;
  CUtensorMap mq, mk;
  int launches = 0;
  if (!encode_bf16_3d(&mk, k, head_dim, num_heads_kv, static_cast<int>(kv_rows), 64, 1, box, true))
    return MVP_ERR_UNSUPPORTED;
  if (run_prefill) {
    if (!encode_bf16_3d(&mq, q, head_dim, num_heads_q, total_q, 64, p.group, p.npos, true)) return MVP_ERR_UNSUPPORTED;
    KwParams pp = p;
    pp.req_offset = first;
    pp.skip_decode = 1;
    pp.n_kb = (max_k_len + kKeys - 1) / kKeys;
    pp.splits = split_count(num_reqs - first, p.hkv, max_q_len, max_k_len, p.npos, num_sms);
    const size_t one = static_cast<size_t>(num_reqs) * p.hkv * pp.n_kb * kKeys * sizeof(float);
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0) pp.splits = 1;
    while (pp.splits > 1 && one * pp.splits > workspace_bytes) pp.splits /= 2;
    pp.partial = pp.splits > 1 ? static_cast<float*>(workspace) : nullptr;
    const long long ctas = static_cast<long long>(pp.n_kb) * pp.splits * p.hkv * (num_reqs - first);
    if (ctas > INT_MAX) return MVP_ERR_UNSUPPORTED;
    cudaError_t e = cudaErrorInvalidValue;
    switch (head_dim) {
      case 64: e = paged ? launch_prefill_rows<1, true>(pp, mq, mk, ctas, st) : launch_prefill_rows<1, false>(pp, mq, mk, ctas, st); break;
      case 128: e = paged ? launch_prefill_rows<2, true>(pp, mq, mk, ctas, st) : launch_prefill_rows<2, false>(pp, mq, mk, ctas, st); break;
      case 256: e = paged ? launch_prefill_rows<4, true>(pp, mq, mk, ctas, st) : launch_prefill_rows<4, false>(pp, mq, mk, ctas, st); break;
      case 512: e = paged ? launch_prefill_rows<8, true>(pp, mq, mk, ctas, st) : launch_prefill_rows<8, false>(pp, mq, mk, ctas, st); break;
    }
    if (e != cudaSuccess) return MVP_ERR_CUDA;
    ++launches;
    if (pp.partial != nullptr) {
      const dim3 grid((max_k_len + 255) / 256, p.hkv, num_reqs - first);
      if (paged) key_weights_combine_kernel<true><<<grid, 256, 0, st>>>(pp);
      else key_weights_combine_kernel<false><<<grid, 256, 0, st>>>(pp);
      if (cudaGetLastError() != cudaSuccess) return MVP_ERR_CUDA;
      ++launches;
    }
  }
  if (decode_count > 0) {
    if (!encode_bf16_3d(&mq, q, head_dim, num_heads_q, total_q, 64, p.group, 1, true)) return MVP_ERR_UNSUPPORTED;
    KwParams pd = p;
    pd.n_kb = (max_k_len + kDecTiles * kKeys - 1) / (kDecTiles * kKeys);
    cudaError_t e = cudaErrorInvalidValue;
    switch (head_dim) {
      case 64: e = paged ? launch_decode_rows<1, true>(pd, decode_count, mq, mk, st) : launch_decode_rows<1, false>(pd, decode_count, mq, mk, st); break;
      case 128: e = paged ? launch_decode_rows<2, true>(pd, decode_count, mq, mk, st) : launch_decode_rows<2, false>(pd, decode_count, mq, mk, st); break;
      case 256: e = paged ? launch_decode_rows<4, true>(pd, decode_count, mq, mk, st) : launch_decode_rows<4, false>(pd, decode_count, mq, mk, st); break;
      case 512: e = paged ? launch_decode_rows<8, true>(pd, decode_count, mq, mk, st) : launch_decode_rows<8, false>(pd, decode_count, mq, mk, st); break;
    }
    if (e != cudaSuccess) return MVP_ERR_CUDA;
    ++launches;
  }
  set_last_launches(launches);
  return MVP_OK;
}

}  // namespace

}  // namespace mvp

using namespace mvp;

extern "C" {

size_t mvp_key_weights_workspace_size(int num_reqs, int num_heads_kv, int max_q_len, int max_k_len) {
  if (num_reqs < 1 || num_heads_kv < 1 || max_q_len < 1 || max_k_len < 1) return 0;
  // the most splits any group size and GPU of up to 160 SMs asks for
  const int s = max_q_len == 1 ? 1 : split_count(num_reqs, num_heads_kv, max_q_len, max_k_len, 1, 160);
  if (s < 2) return 0;
  const size_t keys = (static_cast<size_t>(max_k_len) + kKeys - 1) / kKeys * kKeys;
  return static_cast<size_t>(s) * num_reqs * num_heads_kv * keys * sizeof(float);
}

int mvp_attn_key_weights_varlen(const void* q, const void* k, const float* lse, float* weights, int num_slots,
                                long long weight_stride, const int32_t* slots, int accumulate,
                                const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, const int32_t* context_lens,
                                int num_reqs, int total_q, int total_k, int max_q_len, int max_k_len,
                                int num_decode_reqs, int num_heads_q, int num_heads_kv, int head_dim,
                                const int32_t* range_table, const int32_t* range_covered, int causal, int window_left,
                                int window_right, int first_tokens, const float* sinks, int sink_mode, float scale,
                                void* workspace, size_t workspace_bytes, void* stream) {
  set_last_launches(0);
  return key_weights_impl(q, k, lse, weights, num_slots, weight_stride, slots, accumulate, cu_seqlens_q, context_lens,
                          num_reqs, total_q, max_q_len, max_k_len, num_decode_reqs, num_heads_q, num_heads_kv,
                          head_dim, range_table, range_covered, causal, window_left, window_right, first_tokens, sinks,
                          sink_mode, scale, workspace, workspace_bytes, stream, cu_seqlens_k, nullptr, nullptr,
                          total_k, 0, 0);
}

int mvp_attn_key_weights_paged(const void* q, const void* k_cache, const float* lse, float* weights, int num_slots,
                               long long weight_stride, const int32_t* slots, int accumulate,
                               const int32_t* cu_seqlens_q, const int32_t* seq_lens_k, const int32_t* block_table,
                               int block_size, int max_blocks_per_seq, int num_blocks, const int32_t* context_lens,
                               int num_reqs, int total_q, int max_q_len, int max_k_len, int num_decode_reqs,
                               int num_heads_q, int num_heads_kv, int head_dim, const int32_t* range_table,
                               const int32_t* range_covered, int causal, int window_left, int window_right,
                               int first_tokens, const float* sinks, int sink_mode, float scale, void* workspace,
                               size_t workspace_bytes, void* stream) {
  set_last_launches(0);
  int shift = 0;
  while (shift < 30 && (1 << shift) < block_size) ++shift;
  if (block_size < 16 || block_size > 256 || (1 << shift) != block_size) return MVP_ERR_ARG;
  if (num_blocks < 1 || max_blocks_per_seq < 1 || block_table == nullptr || seq_lens_k == nullptr)
    return MVP_ERR_ARG;
  if (static_cast<long long>(max_blocks_per_seq) * block_size < max_k_len) return MVP_ERR_ARG;
  if (static_cast<long long>(num_blocks) * block_size > INT_MAX) return MVP_ERR_UNSUPPORTED;
  return key_weights_impl(q, k_cache, lse, weights, num_slots, weight_stride, slots, accumulate, cu_seqlens_q,
                          context_lens, num_reqs, total_q, max_q_len, max_k_len, num_decode_reqs, num_heads_q,
                          num_heads_kv, head_dim, range_table, range_covered, causal, window_left, window_right,
                          first_tokens, sinks, sink_mode, scale, workspace, workspace_bytes, stream, nullptr,
                          seq_lens_k, block_table, static_cast<long long>(num_blocks) * block_size, shift,
                          max_blocks_per_seq);
}

}  // extern "C"
