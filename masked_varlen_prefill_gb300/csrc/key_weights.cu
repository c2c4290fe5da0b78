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
// Prefill rows: a CTA pair (.cta_group::2 MMAs, M = 256) keeps a 256-key block
// of one KV head in shared memory (the A operand, each CTA its 128 keys) and
// streams the query tiles that see any of it, N = 256 columns = 2 x floor(128 /
// G) positions x G heads, each CTA loading half of them, through a ring of
// 64-dim chunks (the B operand).  S^T is double-buffered in TMEM; two
// warpgroups of epilogue warps per CTA share the tiles.
// * -lse / scale is added by the tensor core, relative to one lse per tile (the
//   exponent's FFMA adds that): 16 more dims, three of them the bf16 terms of it
//   (hi + mid + lo, 24 bits) in the columns' operand against ones in the keys'.
//   Read from shared memory instead it cost a wavefront per column and warp
//   (with operands and copies the shared-memory pipe was full).  A key-0 sink
//   goes the same way, against ones in the row of key 0 alone: 3 prompts of
//   1061 tokens, 32/8 heads, D = 256 take 54 us with sinks and 52 without (164
//   when the epilogue added it, in its masked path).
// * Work: 2 D flops and one exponential per visible (row, key) and head; the
//   exponentials (32 per clock and SM) take half the MMA's time at D = 256 and
//   as long at D = 128.
// * Visibility is a closed interval of columns per key (the causal and window
//   rules solved for the row), so a masked tile costs one bit mask per 32
//   columns; tiles seen whole skip it.  Only range-table rows need a test per
//   column, in the tiles that hold such a row.
//
// Single tokens, and calls whose requests all have few rows (a drafted
// continuation to verify): K is streamed (the A operand, 64-dim chunks of 128
// keys), the rows' G heads are the B operand (N = rows x G rounded up to 16, at
// most 128); bound by the one read of K, and past some 48 columns by a chain of
// one exponential per column in four warps.  64 requests of 4096 .. 8192 keys,
// 32/8 heads, D = 128: 131 us with 1 or 4 rows, 239 with 16, 400 with 32
// (floor 124); 946 in the prefill kernel, whose tiles of 256 columns they leave
// mostly empty.
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
  float* partial;          // [splits, num_reqs, hkv, n_kb * 256] or null (one split)
  const int32_t* slots;    // or null
  int num_slots;
  long long w_stride;
  int accumulate;
  int num_reqs, hkv, group;
  int req_offset;          // prefill kernel: first request it covers
  int skip_decode;         // prefill kernel: leave single-token requests
  int npos;                // query positions per tile
  int n_kb;                // key blocks (prefill) or key chunks (decode) of max_k_len
  int blocks;              // key blocks one CTA pair takes, one after the other, of
  int grouped_rows;        // the first (request, KV head, split) rows; one of the others
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
constexpr int kEpi = 2;  // epilogue warpgroups
constexpr int kPfThreads = 128 + 128 * kEpi;  // producer, MMA, column and idle warps, epilogue warps
constexpr int kMaxTileBits = 4096;
constexpr int kTile = 2 * kCols;           // columns of a pair's tile
constexpr int kExtBytes = kCols * 16;      // 128 rows x 8 dims of bf16
// Slots of a tile's -lse / scale: the column warp runs up to three tiles ahead of
// the MMAs.
constexpr int kExt = 3;
constexpr float kHuge = 3.0e38f;           // (a bf16 value near it stays finite)

template <int NCH>
struct PfCfg {
  static constexpr int KBUF = NCH <= 4 ? 2 : 1;                  // K blocks in shared memory
  static constexpr int STAGES = NCH <= 2 ? 8 : 5;                // Q chunks in flight
  // The two epilogue warpgroups take the tiles in turn, a buffer each (TURNS),
  // or half of every tile's columns.  In turn a warp does a tile's bookkeeping
  // once per 256 columns instead of 128; by halves a buffer is free sooner,
  // which is what D = 256 needs, where a tile's MMAs take as long as its
  // exponentials.  Four requests of 16384 + 2048 keys, 16/8 heads, in turn and
  // by halves: D = 64 491 / 534 us, 128 521 / 543, 256 757 / 651, 512 (chunks over
  // 0 .. 16384 keys) 443 / 477.
  static constexpr bool TURNS = NCH != 4;
  static constexpr int HALVES = TURNS ? 2 : 1;  // halves of a tile a warpgroup takes
  static constexpr int K_BYTES = NCH * kChunkBytes;
  static constexpr int Q_OFF = KBUF * K_BYTES;
  static constexpr int EXT_OFF = Q_OFF + STAGES * kChunkBytes;   // the keys' two parts, the slots, zeros
  static constexpr int ZERO_OFF = EXT_OFF + (2 + kExt) * kExtBytes;
  static constexpr int RNG_OFF = ZERO_OFF + kExtBytes;           // two slots of kTile intervals
  static constexpr int SHARED_OFF = RNG_OFF + 2 * kTile * 8;
};

struct __align__(16) PfShared {
  uint32_t range_bits[kMaxTileBits / 32];  // tiles with a row whose range meets this key block
  uint64_t k_full[2], k_empty[2];
  uint64_t q_full[8], q_empty[8];
  uint64_t ext_full[kExt], ext_empty[kExt];
  uint64_t s_full[2], s_empty[2];
  uint64_t rng_full[2], rng_empty[2];
  uint64_t final_mma;
  uint32_t tmem_base;
  WaitCtl wc;
};
template <int NCH>
constexpr int pf_smem() {
  return PfCfg<NCH>::SHARED_OFF + static_cast<int>(sizeof(PfShared)) + 1024;
}
static_assert((kEpi - 1) * kKeys * 4 <= 2 * kTile * 8, "the sums fit the range slots");
static_assert(pf_smem<4>() <= 227 * 1024 && pf_smem<8>() <= 227 * 1024 && pf_smem<2>() <= 227 * 1024, "smem budget");

// Key block of the pair, and the query tiles that see any of it: [t_lo, t_hi)
// by the closed-form rules and, with a range table, the earlier ones whose bit
// is set.  Every role of both CTAs walks them alike.
struct TileWalk {
  int ja, jb;            // keys of the block
  int t, t_lo, t_hi;
  const uint32_t* bits;  // null: no ranges
  bool all;              // more tiles than bits: visit every one
  __device__ __forceinline__ bool ranged(int x) const {
    return bits != nullptr && (all || ((bits[x >> 5] >> (x & 31)) & 1u));
  }
  __device__ __forceinline__ bool next() {  // t: the tile to visit
    ++t;
    if (bits != nullptr)
      while (t < t_hi && t < t_lo && !ranged(t)) ++t;
    return t < t_hi;
  }
};

// (b > 0; a 64-bit division costs four of 32 bits, and most fit)
__device__ __forceinline__ long long floor_div(long long a, int b) {
  const unsigned long long u = a >= 0 ? a : -a + b - 1;
  const long long x = (u >> 32) == 0 ? static_cast<unsigned>(u) / static_cast<unsigned>(b) : u / b;
  return a >= 0 ? x : -x;
}

// bits: the block's range bits, or null; whole: before the split.
__device__ __forceinline__ TileWalk walk_of(const KwParams& p, const Req& r, int kb, int split, const uint32_t* bits,
                                            bool whole) {
  TileWalk w;
  w.ja = kb * kTile;
  w.jb = min(w.ja + kTile, r.k_len) - 1;
  const int rows = 2 * p.npos, n_tiles = (r.q_len + rows - 1) / rows;
  long long lo_a, hi_a, lo_b, hi_b;
  seen_by(p.m, w.ja, lo_a, hi_a);
  seen_by(p.m, w.jb, lo_b, hi_b);
  // positions [lo of the first key, hi of the last] (a first token's hi is unbounded)
  const long long lo = max(lo_a - r.ctx, 0LL), hi = min(max(hi_a, hi_b) - r.ctx, static_cast<long long>(r.q_len) - 1);
  w.t_lo = static_cast<int>(min(lo / rows, static_cast<long long>(n_tiles)));
  w.t_hi = hi < 0 ? 0 : static_cast<int>(hi / rows) + 1;
  w.bits = bits;
  w.all = n_tiles > kMaxTileBits;
  w.t = -1;
  if (w.jb < w.ja) w.t_hi = 0;
  if (!whole) {
    const int first = bits != nullptr ? 0 : w.t_lo;
    const long long n = max(w.t_hi - first, 0);
    const int a = first + static_cast<int>(n * split / p.splits);
    w.t_hi = first + static_cast<int>(n * (split + 1) / p.splits);
    w.t_lo = max(w.t_lo, a);
    w.t = a - 1;
  }
  return w;
}

// Descriptor of an operand of 16 dims without swizzle: 8-row x 16-byte core
// matrices, the row groups of dims 0 .. 7 128 bytes apart, dims 8 .. 15 (zeros,
// one block for all of them) `zeros` bytes behind.
__device__ __forceinline__ uint64_t ext_desc(uint32_t saddr, int zeros) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(zeros >> 4) << 16) |
         (static_cast<uint64_t>(128 >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
}

// What a tile's columns have their lse relative to: that of its first row and
// head.  lse / scale is 144 at lse 9 and D = 256, where an fp32 sum keeps 2^-17;
// its differences within a tile are a few units, like the scores.
__device__ __forceinline__ float tile_base(const KwParams& p, const Req& r, int h, int t) {
  const int row = r.q0 + 2 * t * p.npos;
  if (!in_bounds(row, p.m.total_q, p.err)) return 0.f;
  const float x = __ldg(p.lse + static_cast<size_t>(h * p.group) * p.m.total_q + row);
  return fabsf(x) <= kHuge ? x : 0.f;  // (not for an infinity or NaN)
}

template <int NCH, bool PAGED>
__global__ void __launch_bounds__(kPfThreads, 1)
    key_weights_prefill_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                               const KwParams p) {
  using C = PfCfg<NCH>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = smem;
  uint8_t* sQ = smem + C::Q_OFF;
  uint8_t* sE = smem + C::EXT_OFF;
  int2* sR = reinterpret_cast<int2*>(smem + C::RNG_OFF);
  PfShared& sb = *reinterpret_cast<PfShared*>(smem + C::SHARED_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());

  int x = blockIdx.x >> 1;
  const int n_groups = (p.n_kb + p.blocks - 1) / p.blocks;
  const bool grouped = x < p.grouped_rows * n_groups;
  const int per_row = grouped ? n_groups : p.n_kb, blocks = grouped ? p.blocks : 1;
  if (!grouped) x -= p.grouped_rows * n_groups;
  const int kb0 = (x % per_row) * blocks;
  x = x / per_row + (grouped ? 0 : p.grouped_rows);
  const int split = x % p.splits;
  x /= p.splits;
  const int h = x % p.hkv;
  const int b = x / p.hkv + p.req_offset;
  const Req r = load_req<PAGED>(p, b);
  if (kb0 * kTile >= r.k_len || (p.skip_decode && r.q_len == 1)) return;  // (both CTAs)
  const int kb1 = min(kb0 + blocks, (r.k_len + kTile - 1) / kTile);
  const bool use_table = table_active(p.m);
  const uint32_t* bits = use_table ? sb.range_bits : nullptr;
  const int ncol = p.npos * p.group;  // columns of a CTA's half of a tile that have rows

  // Tiles whose ranges meet the key block (with a table, one block per pair).
  if (use_table) {
    const TileWalk w = walk_of(p, r, kb0, 0, bits, true);
    if (!w.all) {
      for (int i = threadIdx.x; i < kMaxTileBits / 32; i += kPfThreads) sb.range_bits[i] = 0;
      __syncthreads();
      const int rows = min(w.t_hi * 2 * p.npos, r.q_len);
      for (int i = threadIdx.x; i < rows; i += kPfThreads) {
        const int2 e = range_of(p.m, r, i);
        const int t = i / (2 * p.npos);
        if (max(e.x, w.ja) <= min(e.y, w.jb)) atomicOr(&sb.range_bits[t >> 5], 1u << (t & 31));
      }
    }
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sb.k_full[i], 1);
      mbar_init(&sb.k_empty[i], 1);
      mbar_init(&sb.s_full[i], 1);
      mbar_init(&sb.s_empty[i], C::TURNS ? 8 : 16);  // both CTAs' epilogue warps of the buffer (rank 0's barrier)
      mbar_init(&sb.rng_full[i], 1);
      mbar_init(&sb.rng_empty[i], C::TURNS ? 4 : 8);  // this CTA's
    }
    for (int i = 0; i < kExt; ++i) {
      mbar_init(&sb.ext_full[i], 2);  // both CTAs' column warps
      mbar_init(&sb.ext_empty[i], 1);
    }
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&sb.q_full[i], 1);
      mbar_init(&sb.q_empty[i], 1);
    }
    mbar_init(&sb.final_mma, 1);
    sb.wc.abort = 0;
    sb.wc.limit_us = p.m.wait_limit_us;
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(&sb.tmem_base, 2 * kTile);
    tmem_relinquish_pair();
  }
  // Operand parts that nothing else writes: ones in the first three dims of the
  // keys' extension (and, for the block of key 0, in that key's next three,
  // which take the columns' sinks), the zeros of dims 8 .. 15, and zeros in the
  // rows of a Q chunk past the last column.
  for (int i = threadIdx.x; i < kCols; i += kPfThreads) {
    const bool first_key = rank == 0 && i == 0;
    *reinterpret_cast<uint4*>(sE + 16 * i) = make_uint4(0x3F803F80u, 0x00003F80u, 0u, 0u);
    *reinterpret_cast<uint4*>(sE + kExtBytes + 16 * i) =
        make_uint4(0x3F803F80u, first_key ? 0x3F803F80u : 0x00003F80u, first_key ? 0x3F803F80u : 0u, 0u);
    *reinterpret_cast<uint4*>(smem + C::ZERO_OFF + 16 * i) = make_uint4(0, 0, 0, 0);
  }
  if (ncol < kCols) {
    const int words = (kCols - ncol) * 8;  // 16-byte words at the end of each chunk
    for (int i = threadIdx.x; i < C::STAGES * words; i += kPfThreads)
      reinterpret_cast<uint4*>(sQ + (i / words) * kChunkBytes + ncol * 128)[i % words] = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the peer's barriers and operand parts are there
  tc_fence_after();
  const uint32_t tmem = sb.tmem_base;

  if (warp == 0) {
    // ---------------------------------------------------------------- loads
    // Each CTA loads its 128 keys of a block and its half of a tile's columns;
    // both complete on rank 0's barriers.
    if (lane == 0) {
      bool ok = true;
      int n = 0, nb = 0;  // Q chunks, K blocks issued
      const uint32_t q_bytes = static_cast<uint32_t>(ncol) * 128;
      const int run = PAGED ? min(kKeys, 1 << p.m.block_shift) : kKeys;
      for (int kb = kb0; ok && kb < kb1; ++kb) {
        TileWalk walk = walk_of(p, r, kb, split, bits, false);
        bool k_loaded = false;
        while (ok && walk.next()) {
          if (!k_loaded) {
            k_loaded = true;
            const int s = nb % C::KBUF;
            if (nb >= C::KBUF && !mbar_wait(&sb.k_empty[s], ((nb / C::KBUF) - 1) & 1, &sb.wc, p.err, kDevTimeoutLoad)) {
              ok = false;
              break;
            }
            if (rank == 0) mbar_arrive_expect_tx(&sb.k_full[s], 2 * C::K_BYTES);
            const uint32_t bar = mapa_shared(smem_u32(&sb.k_full[s]), 0);
            for (int i = 0; i < kKeys; i += run) {
              const int key = walk.ja + rank * kKeys + i;
              const int row = PAGED ? kv_row(p.m, b, 0, r.k_len, key) : r.k0 + key;
#pragma unroll
              for (int c = 0; c < NCH; ++c)
                tma_load_3d_pair(sK + s * C::K_BYTES + c * kChunkBytes + i * 128, &map_k, bar, c * 64, h, row);
            }
            ++nb;
          }
          const int q_row = r.q0 + (2 * walk.t + rank) * p.npos;
          for (int c = 0; c < NCH; ++c, ++n) {
            const int s = n % C::STAGES;
            if (n >= C::STAGES && !mbar_wait(&sb.q_empty[s], ((n / C::STAGES) - 1) & 1, &sb.wc, p.err, kDevTimeoutLoad)) {
              ok = false;
              break;
            }
            if (rank == 0) mbar_arrive_expect_tx(&sb.q_full[s], 2 * q_bytes);
            tma_load_3d_pair(sQ + s * kChunkBytes, &map_q, mapa_shared(smem_u32(&sb.q_full[s]), 0), c * 64, h * p.group,
                             q_row);
          }
        }
      }
      if (!ok) sb.wc.abort = 1;
      // Copies in flight complete before the CTAs leave (rank 1 stays until
      // rank 0 has drained: the final cluster barrier).
      if (rank == 0) {
        WaitCtl own = own_wait_ctl(&sb.wc);
        for (int s = 0; s < C::KBUF && s < nb; ++s) mbar_wait(&sb.k_full[s], ((nb - 1 - s) / C::KBUF) & 1, &own, nullptr, 0);
        for (int s = 0; s < C::STAGES && s < n; ++s) mbar_wait(&sb.q_full[s], ((n - 1 - s) / C::STAGES) & 1, &own, nullptr, 0);
      }
    }
  } else if (warp == 1 && rank == 0) {
    // ---------------------------------------------------------------- MMAs
    constexpr uint32_t idesc = idesc_bf16_f32(2 * kKeys, kTile, false, false);
    const uint64_t dk0 = smem_desc_sw128(smem_u32(sK), 16, 1024);
    const uint64_t dq = smem_desc_sw128(smem_u32(sQ), 16, 1024);
    const bool issuer = elect_one();
    bool ok = true;
    int n = 0, nb = 0, i = 0;  // chunks, K blocks, tiles
    for (int kb = kb0; ok && kb < kb1; ++kb) {
      TileWalk walk = walk_of(p, r, kb, split, bits, false);
      bool any = false;
      const int part = kb == 0 ? 1 : 0;  // the keys' extension
      const uint64_t keys = ext_desc(smem_u32(sE + part * kExtBytes), (2 + kExt - part) * kExtBytes);
      for (; ok && walk.next(); ++i) {
        const int ks = nb % C::KBUF;
        if (!any) ok = mbar_wait(&sb.k_full[ks], (nb / C::KBUF) & 1, &sb.wc, p.err, kDevTimeoutLoad);
        any = true;
        const int es = i % kExt;
        if (ok && i >= 2) ok = mbar_wait_spin(&sb.s_empty[i & 1], ((i >> 1) - 1) & 1, &sb.wc, p.err, kDevTimeoutSoftmax);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + (i & 1) * kTile;
        const uint64_t dk = desc_add(dk0, static_cast<uint32_t>((ks * C::K_BYTES) >> 4));
        for (int c = 0; c < NCH; ++c, ++n) {
          const int s = n % C::STAGES;
          if (!mbar_wait_spin(&sb.q_full[s], (n / C::STAGES) & 1, &sb.wc, p.err, kDevTimeoutLoad)) {
            ok = false;
            break;
          }
          if (issuer) {
#pragma unroll
            for (int k16 = 0; k16 < 4; ++k16)
              mma_ss_one<2>(d, desc_add(dk, static_cast<uint32_t>((c * kChunkBytes + k16 * 32) >> 4)),
                            desc_add(dq, static_cast<uint32_t>((s * kChunkBytes + k16 * 32) >> 4)), idesc,
                            (c | k16) != 0 ? 1u : 0u);
          }
          __syncwarp();
          mma_commit_elect<2>(&sb.q_empty[s]);
        }
        // the columns' lse last: the products add up among themselves first
        if (ok) ok = mbar_wait_spin(&sb.ext_full[es], (i / kExt) & 1, &sb.wc, p.err, kDevTimeoutOther);
        if (!ok) break;
        if (issuer)
          mma_ss_one<2>(d, keys, ext_desc(smem_u32(sE + (2 + es) * kExtBytes), (kExt - es) * kExtBytes), idesc, 1u);
        __syncwarp();
        mma_commit_elect<2>(&sb.ext_empty[es]);
        mma_commit_elect<2>(&sb.s_full[i & 1]);
      }
      if (any) {
        if (ok) mma_commit_elect<2>(&sb.k_empty[nb % C::KBUF]);
        ++nb;
      }
    }
    if (!ok && lane == 0) sb.wc.abort = 1;
    mma_commit_elect<2>(&sb.final_mma);
    WaitCtl own = own_wait_ctl(&sb.wc);
    mbar_wait(&sb.final_mma, 0, &own, p.err, kDevTimeoutMma);
  } else if (warp == 2) {
    // ---------------------------------------------------------------- columns
    // This lane's columns lane + 32 k of the CTA's half: row within the tile,
    // and the lse of it.  (base - lse) / scale goes into the column's extension
    // as three bf16 terms.
    bool ok = true;
    // The key-0 sinks (key-0-bias mode), in units of the score, go there the same
    // way, against the ones of key 0 alone.
    const float inv = -1.f / p.m.scale;
    int pos[4];
    const float* src[4];
    uint32_t sink1[4], sink2[4];  // terms (0, hi) and (mid, lo)
    auto bf16 = [](float x) { return __bfloat162float(__float2bfloat16_rn(x)); };
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = lane + 32 * k;
      float x = 0.f;
      if (p.m.sink_mode == 1 && p.m.sinks != nullptr && c < ncol) {
        const float s0 = __ldg(p.m.sinks + h * p.group + c % p.group);
        // (a NaN reaches the rows of key 0 through their lse; here it would
        // meet the other keys' zeros)
        x = isnan(s0) ? 0.f : fabsf(s0) == INFINITY ? copysignf(kHuge, s0) : -s0 * inv;
      }
      sink1[k] = pack_bf16x2(0.f, x);
      sink2[k] = pack_bf16x2(x - bf16(x), (x - bf16(x)) - bf16(x - bf16(x)));
      pos[k] = c < ncol ? rank * p.npos + c / p.group : INT_MAX / 2;
      src[k] = p.lse + static_cast<size_t>(h * p.group + c % p.group) * p.m.total_q + r.q0 + rank * p.npos + c / p.group;
    }
    auto load = [&](int t, float (&l)[4], float& base) {
      base = tile_base(p, r, h, t);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int row = 2 * t * p.npos + pos[k];
        l[k] = row < r.q_len && in_bounds(r.q0 + row, p.m.total_q, p.err) ? __ldg(src[k] + 2 * t * p.npos) : INFINITY;
      }
    };
    const uint32_t ext_bar = mapa_shared(smem_u32(&sb.ext_full[0]), 0);
    int i = 0;
    for (int kb = kb0; ok && kb < kb1; ++kb) {
      TileWalk walk = walk_of(p, r, kb, split, bits, false);
      float l[4], next_l[4], base = 0.f, next_base = 0.f;
      bool have = walk.next();
      if (have) load(walk.t, l, base);
      for (; ok && have; ++i) {
        const int slot = i & 1, es = i % kExt, t = walk.t;
        // the next tile's loads are in flight while this one waits for its slot
        have = walk.next();
        if (have) load(walk.t, next_l, next_base);
        if (i >= kExt) ok = mbar_wait(&sb.ext_empty[es], ((i / kExt) - 1) & 1, &sb.wc, p.err, kDevTimeoutMma);
        if (ok && use_table && i >= 2) ok = mbar_wait(&sb.rng_empty[slot], ((i >> 1) - 1) & 1, &sb.wc, p.err, kDevTimeoutOther);
        if (!__all_sync(kFull, ok)) break;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          // an infinite lse: a weight of zero whatever the score (of -inf too: its
          // row has no probabilities, whether it sees nothing or a key that a sink
          // of -inf closes)
          const float v = fabsf(l[k]) == INFINITY ? -kHuge : (l[k] - base) * inv;
          const float hi = bf16(v), mid = bf16(v - hi);
          const uint32_t w0 = pack_bf16x2(hi, mid), w1 = pack_bf16x2((v - hi) - mid, 0.f);
          *reinterpret_cast<uint4*>(sE + (2 + es) * kExtBytes + 16 * (lane + 32 * k)) =
              make_uint4(w0, w1 | sink1[k], sink2[k], 0u);
          l[k] = next_l[k];
        }
        base = next_base;
        fence_proxy_async_smem();
        __syncwarp();
        // (released at CTA scope: what the arrival publishes are this CTA's own
        // shared-memory writes, made visible to the tensor core by the fence
        // above; a release at cluster scope also waits for the loads in flight,
        // and took a tile from 1150 to 1300 ns)
        if (lane == 0) mbar_arrive_cluster(ext_bar + es * 8);
        if (use_table) {
          if (walk.ranged(t))
            for (int c = lane; c < kTile; c += 32) {
              const int half = c / kCols, cc = c % kCols, row0 = (2 * t + half) * p.npos;
              if ((r.q_len - row0) * static_cast<long long>(p.group) <= cc - lane) continue;  // (32 columns of no row: not read)
              const int row = row0 + cc / p.group;
              sR[slot * kTile + c] = (cc < ncol && row < r.q_len) ? range_of(p.m, r, row) : make_int2(1, 0);
            }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sb.rng_full[slot]);
        }
      }
    }
    if (!ok) sb.wc.abort = 1;
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- exponentials and sums
    const int quarter = warp & 3, part = (warp - 4) >> 2;  // the warpgroup
    const int row = quarter * 32 + lane;
    const uint32_t base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const float sc = p.m.scale_log2;
    const uint64_t sc2 = f2_pack(sc, sc);
    const uint32_t s_empty0 = mapa_shared(smem_u32(&sb.s_empty[0]), 0);
    float* w = p.partial != nullptr
                   ? p.partial + ((static_cast<size_t>(split) * p.num_reqs + b) * p.hkv + h) * (static_cast<size_t>(p.n_kb) * kTile)
                   : weight_row(p, b, h);
    const bool add = p.partial == nullptr && p.accumulate;
    bool ok = true;
    int i = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      TileWalk walk = walk_of(p, r, kb, split, bits, false);
      const int ja = walk.ja + rank * kKeys, jb = min(ja + kKeys - 1, walk.jb), key = ja + row;  // this CTA's keys
      long long p_lo, p_hi;
      seen_by(p.m, key, p_lo, p_hi);
      if (key > jb) p_hi = p_lo - 1;
      // rows at positions [in_lo, in_hi] see every key of the block
      long long in_lo, in_hi, tmp;
      seen_by(p.m, jb, in_lo, tmp);
      seen_by(p.m, ja, tmp, in_hi);
      if (jb >= p.m.first_tokens && ja < p.m.first_tokens)
        in_hi = min(in_hi, static_cast<long long>(p.m.first_tokens) + p.m.window_left);
      // ... that is, the tiles [w_lo, w_hi] all of whose npos rows of a half do
      // (64-bit divisions, once per block: done per tile they and the walk took
      // 700 of 2200 clocks a tile).
      const int rows2 = 2 * p.npos;
      int w_lo[C::HALVES], w_hi[C::HALVES];
#pragma unroll
      for (int e = 0; e < C::HALVES; ++e) {
        const int half = C::TURNS ? e : part;
        const long long at0 = static_cast<long long>(r.ctx) + half * p.npos;  // position of tile 0's first row of the half
        w_lo[e] = static_cast<int>(max(0LL, min(-floor_div(at0 - in_lo, rows2), 1LL << 30)));
        w_hi[e] = static_cast<int>(max(-1LL, min(floor_div(in_hi - at0 - p.npos + 1, rows2),
                                                    floor_div(r.q_len - p.npos - half * p.npos, rows2))));
      }
      uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
      int base_t = -1;  // the tile whose base is loaded, one of this warpgroup's ahead
      float base_next = 0.f;
      for (; walk.next(); ++i) {
        const int buf = i & 1;
        if (C::TURNS && buf != part) continue;
        const float shift = -kLog2e * (base_t == walk.t ? base_next : tile_base(p, r, h, walk.t));
        base_t = walk.t + C::HALVES;
        if (base_t < walk.t_hi) base_next = tile_base(p, r, h, base_t);
        const uint64_t shift2 = f2_pack(shift, shift);
        ok = mbar_wait(&sb.s_full[buf], (i >> 1) & 1, &sb.wc, p.err, kDevTimeoutMma);
        if (ok && use_table) ok = mbar_wait(&sb.rng_full[buf], (i >> 1) & 1, &sb.wc, p.err, kDevTimeoutOther);
        if (!ok) break;
        tc_fence_after();
        auto release = [&]() {  // the scores are in registers: the buffer is free
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(s_empty0 + buf * 8);
        };
        const bool ranged = walk.ranged(walk.t);
#pragma unroll
        for (int e = 0; e < C::HALVES; ++e) {
          const int half = C::TURNS ? e : part;
          const uint32_t col = base + buf * kTile + half * kCols;
          if (walk.t >= w_lo[e] && walk.t <= w_hi[e] && !ranged) {
            uint32_t s[2][32];
            tmem_ld_32x32b_x32(col, s[0]);
#pragma unroll
            for (int cc = 0; cc < kCols / 32; ++cc) {
              tmem_ld_wait(s[cc & 1]);
              if (cc < kCols / 32 - 1) tmem_ld_32x32b_x32(col + 32 * (cc + 1), s[(cc + 1) & 1]);
              else if (e == C::HALVES - 1) release();
#pragma unroll
              for (int q = 0; q < 16; ++q) {
                float a0, a1;
                f2_unpack(f2_fma(f2_pack(__uint_as_float(s[cc & 1][2 * q]), __uint_as_float(s[cc & 1][2 * q + 1])), sc2, shift2), a0, a1);
                acc[q & 3] = f2_add(acc[q & 3], f2_pack(ex2_approx(a0), ex2_approx(a1)));
              }
            }
          } else {
            const int row0 = (2 * walk.t + half) * p.npos;          // this half's first row
            const int valid = max(0, min(p.npos, r.q_len - row0));  // rows of the request in it
            const long long p0 = static_cast<long long>(r.ctx) + row0;
            // columns of the half that see this thread's key: [c_lo, c_hi]
            const int c_lo = static_cast<int>(min(max(p_lo - p0, 0LL), static_cast<long long>(valid))) * p.group;
            const int c_hi = static_cast<int>(min(max(p_hi - p0 + 1, 0LL), static_cast<long long>(valid))) * p.group - 1;
            const int n_cc = (valid * p.group + 31) / 32;  // (32 columns at a time, of rows)
            if (e == C::HALVES - 1 && n_cc == 0) release();
#pragma unroll 1
            for (int cc = 0; cc < n_cc; ++cc) {
              uint32_t s[32];
              tmem_ld_32x32b_x32(col + 32 * cc, s);
              uint32_t seen = interval_bits(c_lo, c_hi, 32 * cc);
              if (ranged && key <= jb) {
#pragma unroll 8
                for (int q = 0; q < 32; ++q) {
                  const int2 g = sR[buf * kTile + half * kCols + 32 * cc + q];
                  seen |= static_cast<uint32_t>(key >= g.x && key <= g.y) << q;
                }
              }
              tmem_ld_wait(s);
              if (e == C::HALVES - 1 && cc == n_cc - 1) release();
#pragma unroll
              for (int q = 0; q < 16; ++q) {
                const float e0 = ex2_approx(fmaf(__uint_as_float(s[2 * q]), sc, shift));
                const float e1 = ex2_approx(fmaf(__uint_as_float(s[2 * q + 1]), sc, shift));
                acc[q & 3] = f2_add(acc[q & 3], f2_pack((seen >> (2 * q)) & 1u ? e0 : 0.f, (seen >> (2 * q + 1)) & 1u ? e1 : 0.f));
              }
            }
          }
        }
        if (use_table) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&sb.rng_empty[buf]);
        }
      }
      // a block's sums: the warpgroups' parts, in their order
      float x0, x1, x2, x3;
      f2_unpack(f2_add(acc[0], acc[1]), x0, x1);
      f2_unpack(f2_add(acc[2], acc[3]), x2, x3);
      float total = (x0 + x1) + (x2 + x3);
      // (through the range intervals' slots, once every warp is done with those)
      float* parts = reinterpret_cast<float*>(sR);  // [kEpi - 1][kKeys]
      if (use_table) named_barrier(3, 128 * kEpi);
      if (part > 0) parts[(part - 1) * kKeys + row] = total;
      named_barrier(1, 128 * kEpi);
      if (part == 0 && key <= jb && w != nullptr) {
#pragma unroll
        for (int e = 0; e < kEpi - 1; ++e) total += parts[e * kKeys + row];
        w[key] = add ? w[key] + total : total;
      }
      named_barrier(2, 128 * kEpi);  // (they are read before the next block's)
    }
    if (!ok) sb.wc.abort = 1;
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // rank 0's MMAs and drain are complete
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 2 * kTile);
}

// Adds the splits' partial sums up, in their order.
template <bool PAGED>
__global__ void __launch_bounds__(256) key_weights_combine_kernel(const KwParams p) {
  const int h = blockIdx.y, b = blockIdx.z + p.req_offset;
  const Req r = load_req<PAGED>(p, b);
  if (p.skip_decode && r.q_len == 1) return;
  const int key = blockIdx.x * 256 + threadIdx.x;
  if (key >= r.k_len) return;
  const size_t row = static_cast<size_t>(p.n_kb) * kTile;
  float total = 0.f;
  for (int s = 0; s < p.splits; ++s) total += p.partial[((static_cast<size_t>(s) * p.num_reqs + b) * p.hkv + h) * row + key];
  float* w = weight_row(p, b, h);
  if (w != nullptr) w[key] = p.accumulate ? w[key] + total : total;
}

// ------------------------------------------------------------------ requests of few rows
constexpr int kFewCols = 128;  // columns (rows x heads) of a request this kernel takes, at most
constexpr int kDecTiles = 16;  // key tiles of a CTA
constexpr int kDecStages = 6;  // K chunks in flight
constexpr int kDecThreads = 192;  // producer, MMA and 4 epilogue warps

struct __align__(16) DecShared {
  float nl2[kCols];  // of a column
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
                              const KwParams p, const int max_rows, const int n, const int tmem_cols) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = smem;
  uint8_t* sQ = smem + kDecStages * kChunkBytes;
  // Base and range interval of a column's row, and the last first token it sees
  // (more than one row: the columns are few).
  int4* sV = reinterpret_cast<int4*>(sQ + NCH * n * 128);
  int* sF = reinterpret_cast<int*>(sV + kFewCols);
  __shared__ DecShared sb;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.z, h = blockIdx.y;
  const Req r = load_req<PAGED>(p, b);
  // All requests of the call have at most max_rows rows, or it is one and the
  // others are left to the prefill kernel.
  if (max_rows == 1 ? r.q_len != 1 : r.q_len < 1 && p.accumulate) return;
  const int rows = min(r.q_len, max_rows), ncol = rows * p.group;
  const int key_lo = blockIdx.x * (kDecTiles * kKeys);
  if (key_lo >= r.k_len) return;
  const int tiles = min(kDecTiles, (r.k_len - key_lo + kKeys - 1) / kKeys);
  // The hulls of what the rows see, and the keys that all of them do; each
  // column's own for the tiles between.
  const bool use_table = table_active(p.m);
  RowVis vis;
  int f_hi = -1, all_lo, all_hi;
  if (max_rows == 1) {
    vis = row_visibility(p.m, r.ctx, r.k_len, use_table, r.q0, b);
    if (p.m.first_tokens > 0) f_hi = first_tokens_hi(p.m, r.ctx, r.k_len);
    all_lo = vis.b_lo;
    all_hi = vis.b_hi;
  } else {
    vis.b_lo = vis.r_lo = INT_MAX;
    vis.b_hi = vis.r_hi = -1;
    all_lo = 0;
    all_hi = rows > 0 ? r.k_len - 1 : -1;
    for (int c = lane; c < ncol; c += 32) {
      const int i = c / p.group;
      const RowVis v = row_visibility(p.m, r.ctx + i, r.k_len, use_table, r.q0 + i, b);
      const int f = p.m.first_tokens > 0 ? first_tokens_hi(p.m, r.ctx + i, r.k_len) : -1;
      if (!v.base_empty()) {
        vis.b_lo = min(vis.b_lo, v.b_lo);
        vis.b_hi = max(vis.b_hi, v.b_hi);
      }
      if (!v.range_empty()) {
        vis.r_lo = min(vis.r_lo, v.r_lo);
        vis.r_hi = max(vis.r_hi, v.r_hi);
      }
      f_hi = max(f_hi, f);
      all_lo = max(all_lo, v.b_lo);
      all_hi = min(all_hi, v.b_hi);
      if (warp == 0) {
        sV[c] = make_int4(v.b_lo, v.b_hi, v.r_lo, v.r_hi);
        sF[c] = f;
      }
    }
    vis.b_lo = __reduce_min_sync(kFull, vis.b_lo);
    vis.b_hi = __reduce_max_sync(kFull, vis.b_hi);
    vis.r_lo = __reduce_min_sync(kFull, vis.r_lo);
    vis.r_hi = __reduce_max_sync(kFull, vis.r_hi);
    f_hi = __reduce_max_sync(kFull, f_hi);
    all_lo = __reduce_max_sync(kFull, all_lo);
    all_hi = __reduce_min_sync(kFull, all_hi);
  }
  auto meets = [&](int i) {  // a row may see a key of tile i
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
  for (int c = threadIdx.x; c < ncol; c += kDecThreads) {
    const int i = max_rows == 1 ? 0 : c / p.group, g = c - i * p.group;
    const float l = in_bounds(r.q0 + i, p.m.total_q, p.err)
                        ? __ldg(p.lse + static_cast<size_t>(h * p.group + g) * p.m.total_q + r.q0 + i)
                        : INFINITY;
    sb.nl2[c] = l == -INFINITY ? l : -kLog2e * l;  // (a row without probabilities: 0)
    sb.sink[c] = p.m.sink_mode == 1 && p.m.sinks != nullptr ? __ldg(p.m.sinks + h * p.group + g) * kLog2e : 0.f;
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
      mbar_arrive_expect_tx(&sb.q_full, static_cast<uint32_t>(NCH * max_rows * p.group * 128));
      for (int x = 0; x < NCH; ++x) tma_load_3d(sQ + x * n * 128, &map_q, &sb.q_full, x * 64, h * p.group, r.q0);
      // Cache rows of a tile's runs (paged), looked up a tile ahead: the block
      // ids' latency is then not in the way of a freed stage.
      constexpr int kRuns = PAGED ? kKeys / 16 : 1;
      int next[kRuns];
      auto look_up = [&](int i) {
        if constexpr (PAGED) {
#pragma unroll
          for (int k = 0; k < kRuns; ++k)
            if (k * run < kKeys) next[k] = kv_row(p.m, b, 0, r.k_len, key_lo + i * kKeys + k * run);
        }
      };
      auto next_tile = [&](int i) {
        while (i < tiles && !meets(i)) ++i;
        return i;
      };
      int i = next_tile(0);
      if (i < tiles) look_up(i);
      while (ok && i < tiles) {
        int rows[kRuns];
#pragma unroll
        for (int k = 0; k < kRuns; ++k) rows[k] = next[k];
        const int after = next_tile(i + 1);
        if (after < tiles) look_up(after);
        for (int x = 0; x < NCH; ++x, ++c) {
          const int s = c % kDecStages;
          if (c >= kDecStages && !mbar_wait(&sb.k_empty[s], ((c / kDecStages) - 1) & 1, &sb.wc, p.err, kDevTimeoutLoad)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&sb.k_full[s], kChunkBytes);
#pragma unroll
          for (int k = 0; k < kRuns; ++k) {
            if (k * run >= kKeys) break;
            const int row = PAGED ? rows[k] : r.k0 + key_lo + i * kKeys;
            tma_load_3d(sK + s * kChunkBytes + k * run * 128, &map_k, &sb.k_full[s], x * 64, h, row);
          }
        }
        i = after;
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
        const int a = key_lo + i * kKeys;
        const bool whole = a >= all_lo && a + kKeys - 1 <= all_hi;  // by all rows
        const bool one = vis.visible(key) || key <= f_hi;           // (one row: its own intervals)
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        for (int n0 = 0; n0 < ncol; n0 += 16) {
          uint32_t s[16];
          tmem_ld_32x32b_x16(base + (j & 1) * n + n0, s);
          tmem_ld_wait16(s);
          if (whole && a > 0 && n0 + 16 <= ncol) {  // every key is seen, and none is key 0
#pragma unroll
            for (int q = 0; q < 16; ++q)
              sum[q & 3] += ex2_approx(fmaf(__uint_as_float(s[q]), p.m.scale_log2, sb.nl2[n0 + q]));
            continue;
          }
          uint32_t seen = n0 + 16 <= ncol ? 0xffffu : (1u << (ncol - n0)) - 1u;
          if (!whole && max_rows == 1) seen = one ? seen : 0u;
          if (!whole && max_rows > 1) {
#pragma unroll 4
            for (int q = 0; q < min(16, ncol - n0); ++q) {
              const int4 x = sV[n0 + q];
              if (!((key >= x.x && key <= x.y) || (key >= x.z && key <= x.w) || key <= sF[n0 + q])) seen &= ~(1u << q);
            }
          }
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            const float nl2 = sb.nl2[n0 + q] + (key == 0 ? sb.sink[n0 + q] : 0.f);
            const float e = ex2_approx(fmaf(__uint_as_float(s[q]), p.m.scale_log2, nl2));
            sum[q & 3] += (seen >> q) & 1u ? e : 0.f;
          }
        }
        total = (sum[0] + sum[1]) + (sum[2] + sum[3]);
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
cudaError_t launch_prefill_rows(const KwParams& p, const CUtensorMap& mq, const CUtensorMap& mk, long long pairs,
                                cudaStream_t stream) {
  static bool done[64] = {};
  cudaError_t e = set_smem(key_weights_prefill_kernel<NCH, PAGED>, pf_smem<NCH>(), done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(kPfThreads);
  cfg.dynamicSmemBytes = pf_smem<NCH>();
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, key_weights_prefill_kernel<NCH, PAGED>, mq, mk, p);
}

template <int NCH, bool PAGED>
cudaError_t launch_decode_rows(const KwParams& p, int reqs, int rows, const CUtensorMap& mq, const CUtensorMap& mk,
                               cudaStream_t stream) {
  static bool done[64] = {};
  constexpr int kFewBytes = kFewCols * 20;
  constexpr int kMost = kDecStages * kChunkBytes + NCH * kCols * 128 + 1024 + (NCH < 8 ? kFewBytes : 0);
  static_assert(NCH < 8 || kFewBytes <= NCH * (kCols / 4) * 128, "D = 512: it has the room of a quarter of the columns");
  cudaError_t e = set_smem(key_weights_decode_kernel<NCH, PAGED>, kMost, done);
  if (e != cudaSuccess) return e;
  const int n = (rows * p.group + 15) / 16 * 16;
  int cols = 32;
  while (cols < 2 * n) cols *= 2;
  const int smem = kDecStages * kChunkBytes + NCH * n * 128 + 1024 + (rows > 1 ? kFewBytes : 0);
  key_weights_decode_kernel<NCH, PAGED><<<dim3(p.n_kb, p.hkv, reqs), kDecThreads, smem, stream>>>(mq, mk, p, rows, n, cols);
  return cudaGetLastError();
}

// Parts the query tiles of a key block are shared by: while half of the GPU's CTA
// pairs would have no block, not fewer than four tiles each.  Measured at D =
// 256: one 2048-row prompt of 16/8 heads (64 blocks for 76 pairs) 27 us alone,
// 31 in two parts, 40 in four (a pair's set-up, the second kernel); a 4096-row
// prompt of 8/2 heads (32 blocks) 80 us alone, 47 in two, 49 in four.
int split_count(int num_reqs, int hkv, int max_q_len, int max_k_len, int npos, int num_sms) {
  const long long blocks = static_cast<long long>(num_reqs) * hkv * ((max_k_len + kTile - 1) / kTile);
  const int tiles = (max_q_len + 2 * npos - 1) / (2 * npos);
  int s = 1;
  while (s < 16 && blocks * s < num_sms / 4 && tiles / (2 * s) >= 4) s *= 2;
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
  if (scale < 1e-30f) return MVP_ERR_UNSUPPORTED;              // lse / scale stays finite
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
  p.hkv = num_heads_kv;
  p.group = num_heads_q / num_heads_kv;
  p.npos = kCols / p.group;
  p.max_k_len = max_k_len;
  p.err = err;

  // Mixed in any order, but so many rows that every request has more than one
  // (unless rows are padding): the prefill kernel takes them all, right for
  // single tokens too, and the other one is not launched.  (Not where no request
  // has more than one: there all rows past the requests' are padding.)
  const bool no_single =
      num_decode_reqs < 0 && max_q_len > 1 && total_q > static_cast<long long>(num_reqs - 1) * max_q_len + 1;
  // No request of more than a few rows: the single tokens' kernel takes them
  // all, with a column per row and head (up to its 128, 33 rows of 4 heads take
  // 839 us in the other one and 32 rows 402 here; 96 at D = 512, where 33 rows
  // of 4 take 264 and 24 take 143).
  const int most = head_dim == 512 ? kFewCols * 3 / 4 : kFewCols;  // (what shared memory holds)
  const bool few = max_q_len > 1 && static_cast<long long>(max_q_len) * p.group <= most;
  const int decode_count = few ? num_reqs : no_single ? 0 : (num_decode_reqs < 0 ? num_reqs : num_decode_reqs);
  const int first = few ? num_reqs : num_decode_reqs < 0 ? 0 : num_decode_reqs;
  const int dec_rows = few ? max_q_len : 1;
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
    pp.skip_decode = no_single || num_decode_reqs >= 0 ? 0 : 1;  // (only where the other kernel covers them too)
    pp.n_kb = (max_k_len + kTile - 1) / kTile;
    pp.splits = split_count(num_reqs - first, p.hkv, max_q_len, max_k_len, p.npos, num_sms);
    const size_t one = static_cast<size_t>(num_reqs) * p.hkv * pp.n_kb * kTile * sizeof(float);
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0) pp.splits = 1;
    while (pp.splits > 1 && one * pp.splits > workspace_bytes) pp.splits /= 2;
    pp.partial = pp.splits > 1 ? static_cast<float*>(workspace) : nullptr;
    // Key blocks per CTA pair: as many as leave four rounds of pairs (the next
    // block's K loads behind this one's tiles; the pair's set-up, 2 us, is paid
    // once), at most eight, and single blocks for the last quarter of the rows,
    // so that the pairs end together (four 2048-row chunks over 0 .. 16384 keys:
    // 256 us; four blocks everywhere 272, eight 303, one 296).  With a range
    // table one block, whose tiles are listed at the start.
    const int rows = pp.splits * p.hkv * (num_reqs - first);
    const long long blocks = static_cast<long long>(pp.n_kb) * rows;
    pp.blocks = 1;
    if (range_table == nullptr) pp.blocks = static_cast<int>(std::max(1LL, std::min(8LL, blocks / (2LL * num_sms))));
    pp.grouped_rows = rows - rows / 4;
    const long long pairs = static_cast<long long>((pp.n_kb + pp.blocks - 1) / pp.blocks) * pp.grouped_rows +
                            static_cast<long long>(pp.n_kb) * (rows - pp.grouped_rows);
    if (2 * pairs > INT_MAX) return MVP_ERR_UNSUPPORTED;
    cudaError_t e = cudaErrorInvalidValue;
    switch (head_dim) {
      case 64:
        e = paged ? launch_prefill_rows<1, true>(pp, mq, mk, pairs, st)
                  : launch_prefill_rows<1, false>(pp, mq, mk, pairs, st);
        break;
      case 128:
        e = paged ? launch_prefill_rows<2, true>(pp, mq, mk, pairs, st)
                  : launch_prefill_rows<2, false>(pp, mq, mk, pairs, st);
        break;
      case 256:
        e = paged ? launch_prefill_rows<4, true>(pp, mq, mk, pairs, st)
                  : launch_prefill_rows<4, false>(pp, mq, mk, pairs, st);
        break;
      case 512:
        e = paged ? launch_prefill_rows<8, true>(pp, mq, mk, pairs, st)
                  : launch_prefill_rows<8, false>(pp, mq, mk, pairs, st);
        break;
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
    if (!encode_bf16_3d(&mq, q, head_dim, num_heads_q, total_q, 64, p.group, dec_rows, true)) return MVP_ERR_UNSUPPORTED;
    KwParams pd = p;
    pd.n_kb = (max_k_len + kDecTiles * kKeys - 1) / (kDecTiles * kKeys);
    cudaError_t e = cudaErrorInvalidValue;
    switch (head_dim) {
      case 64:
        e = paged ? launch_decode_rows<1, true>(pd, decode_count, dec_rows, mq, mk, st)
                  : launch_decode_rows<1, false>(pd, decode_count, dec_rows, mq, mk, st);
        break;
      case 128:
        e = paged ? launch_decode_rows<2, true>(pd, decode_count, dec_rows, mq, mk, st)
                  : launch_decode_rows<2, false>(pd, decode_count, dec_rows, mq, mk, st);
        break;
      case 256:
        e = paged ? launch_decode_rows<4, true>(pd, decode_count, dec_rows, mq, mk, st)
                  : launch_decode_rows<4, false>(pd, decode_count, dec_rows, mq, mk, st);
        break;
      case 512:
        e = paged ? launch_decode_rows<8, true>(pd, decode_count, dec_rows, mq, mk, st)
                  : launch_decode_rows<8, false>(pd, decode_count, dec_rows, mq, mk, st);
        break;
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
  const size_t keys = (static_cast<size_t>(max_k_len) + kTile - 1) / kTile * kTile;
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
