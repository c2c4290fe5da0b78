// Rotary positions with several axes, written into a paged K/V cache.
//
// Pair i of a head (i < rot_dim / 2) turns by pos[axis(i)] * f_i radians: the
// pair (x, y) becomes (x cos - y sin, x sin + y cos).  The axes are the
// coordinates a token has (time, height and width in images and video, one
// for text); each pair follows one of them.  Queries are rotated into q_out,
// keys into their cache rows, values copied into theirs.
//
// Angles.  pos * f in fp32 loses the angle of far positions (at a million
// tokens half an ulp of the product is 0.03 radians), so the table holds
// each frequency as turns per position, f / 2 pi, in 64-bit fixed point: the
// product with the position wraps modulo one turn by itself, exactly, and its
// upper 32 bits are the turn within 2^-32.  It is then rounded to fp32: an angle
// within 1e-7 radians at every int32 position, as fine as the fp32 rotation,
// which is rounded once to bf16 (what the attention kernels read).
//
// The kernel is bound by memory: (Hq + 2 Hkv) * D elements of each token are
// read and written once.  A CTA takes one token (up to eight small ones): a few
// threads turn the token's pairs' angles into shared memory, shared by all the
// heads, while every thread already has its first elements on their way.
// Measured, 12 thousand tokens of 16/8 heads at D 256 (0.4 GB): 65.6 us, 0.90 of
// the copy rate (67.3 with eight CTAs per SM instead of ten, 69.7 with 256
// threads, 73 with the loads behind the angles).
#include <cuda_bf16.h>

#include <climits>
#include <cmath>
#include <cstring>

#include "../../include/mvp.h"
#include "mvp_internal.cuh"
#include "ptx.cuh"

namespace mvp {

namespace {

constexpr int kRopeThreads = 128;
constexpr int kMaxPairs = 256;   // head_dim <= 512
constexpr int kMaxTokens = 8;    // tokens of a CTA
constexpr int kMaxAngles = 1024;  // tokens x pairs of a CTA

struct RopeParams {
  const void* q;
  const void* k;
  const void* v;
  __nv_bfloat16* q_out;
  __nv_bfloat16* k_cache;
  __nv_bfloat16* v_cache;
  const int32_t* positions;  // [num_axes, total_q]
  const uint4* table;        // per pair: turns per position (low word, high word), axis, 0
  const int32_t* cu_q;
  const int32_t* seq_k;
  const int32_t* block_table;
  long long q_stride, k_stride, v_stride;  // elements from one token to the next
  int num_reqs, total_q, num_axes;
  int tokens;  // tokens of a CTA: a power of two
  int hq, hkv, d, rot;
  int block_shift, max_blocks, num_blocks;
  int* err;
};

// Request b with cu_q[b] <= t < cu_q[b + 1], or -1 for a row past the batch
// (warp-collective: a 32-ary search, each step probing 32 offsets).
__device__ __forceinline__ int request_of_row(const int32_t* cu_q, int num_reqs, int t, int lane) {
  if (t >= __ldg(cu_q + num_reqs)) return -1;
  int lo = 0, n = num_reqs;  // the answer, the largest b with cu_q[b] <= t, lies in [lo, lo + n)
  while (n > 1) {
    const int c = lo + static_cast<int>(static_cast<long long>(lane) * n / 32);
    const unsigned m = __ballot_sync(0xffffffffu, __ldg(cu_q + c) <= t);
    const int k = m != 0u ? 31 - __clz(m) : 0;
    const int next = k == 31 ? lo + n : lo + static_cast<int>(static_cast<long long>(k + 1) * n / 32);
    lo += static_cast<int>(static_cast<long long>(k) * n / 32);
    n = next - lo;
  }
  return lo;
}

struct Eight {
  float x[8];
};

// 16 bytes of q, k or v, by an ordinary load: q_out may be q, and the read-only
// path is for memory that nothing writes during the kernel.  (Each 16 bytes are
// read and written by one thread, so loads need no order among the stores.)
__device__ __forceinline__ uint4 ld16(const void* p) {
  uint4 u;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p));
  return u;
}

// Eight elements as they lie in memory, and their values.
template <class T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = ld16(p); }
  __device__ __forceinline__ Eight get() const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    Eight e;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      e.x[2 * i] = __uint_as_float(w[i] << 16);
      e.x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    return e;
  }
};
template <>
struct Raw8<float> {
  uint4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = ld16(p);
    b = ld16(p + 4);
  }
  __device__ __forceinline__ Eight get() const {
    return {{__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z), __uint_as_float(a.w),
             __uint_as_float(b.x), __uint_as_float(b.y), __uint_as_float(b.z), __uint_as_float(b.w)}};
  }
};

__device__ __forceinline__ void store8(__nv_bfloat16* p, const Eight& e) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(e.x[0], e.x[1]), pack_bf16x2(e.x[2], e.x[3]),
                                            pack_bf16x2(e.x[4], e.x[5]), pack_bf16x2(e.x[6], e.x[7]));
}

// T: element type of q, k and v.  ADJ: pairs are (2 i, 2 i + 1), else
// (i, i + rot / 2).  MANY: a CTA takes several tokens.
template <class T, bool ADJ, bool MANY>
__global__ void __launch_bounds__(kRopeThreads, sizeof(T) == 2 && !MANY ? 10 : 6) rope_append_kernel(RopeParams p) {
  __shared__ __align__(16) float s_cos[MANY ? kMaxAngles : kMaxPairs], s_sin[MANY ? kMaxAngles : kMaxPairs];
  __shared__ long long s_row[kMaxTokens];
  const int half = p.rot / 2;
  const int tokens = MANY ? p.tokens : 1;
  const int group = MANY ? kRopeThreads / tokens : kRopeThreads;  // threads of a token
  const int mine = MANY ? static_cast<int>(threadIdx.x) / group : 0;
  const int tid = MANY ? static_cast<int>(threadIdx.x) % group : static_cast<int>(threadIdx.x);
  const int t0 = blockIdx.x * tokens, t = MANY ? min(t0 + mine, p.total_q - 1) : t0;
  griddep_launch_dependents();  // (an attention call behind this one sets up beside it)
  const T* q = static_cast<const T*>(p.q) + static_cast<size_t>(t) * p.q_stride;
  const T* k = static_cast<const T*>(p.k) + static_cast<size_t>(t) * p.k_stride;
  const T* v = static_cast<const T*>(p.v) + static_cast<size_t>(t) * p.v_stride;
  auto head_of = [&](int h) { return h < p.hq ? q + static_cast<size_t>(h) * p.d : k + static_cast<size_t>(h - p.hq) * p.d; };
  // The rotated part in units of 16 elements (8 pairs) of one head, of q's and
  // then k's heads, and v's part in units of 8: each thread's first ones are on
  // their way before the angles and the cache row are known.
  const int per_head = p.rot / 16, units = (p.hq + p.hkv) * per_head, v_units = p.hkv * p.d / 8;
  auto at_of = [&](int c, int second) { return ADJ ? 16 * c + 8 * second : 8 * c + half * second; };
  constexpr int kAhead = 2;
  Raw8<T> a[kAhead], b[kAhead], vr;
  auto load = [&](int u0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int u = u0 + i * group;
      if (u < units) {
        const T* src = head_of(u / per_head);
        a[i].load(src + at_of(u % per_head, 0));
        b[i].load(src + at_of(u % per_head, 1));
      }
    }
  };
  load(tid);
  if (tid < v_units) vr.load(v + 8 * tid);
  const int n_tokens = MANY ? min(tokens, p.total_q - t0) : 1;
  const int lane = threadIdx.x & 31;
  for (int x = threadIdx.x >> 5; x < n_tokens; x += kRopeThreads / 32) {
    // a token's cache row, -1 where it has none, -2 past the batch
    const int req = request_of_row(p.cu_q, p.num_reqs, t0 + x, lane);
    if (lane == 0) {
      long long row = -1;
      if (req >= 0) {
        const int j = __ldg(p.seq_k + req) - __ldg(p.cu_q + req + 1) + t0 + x;
        const int blk = j >> p.block_shift;
        if (j >= 0 && blk < p.max_blocks) {
          const int id = __ldg(p.block_table + static_cast<size_t>(req) * p.max_blocks + blk);
          if (id >= 0 && id < p.num_blocks)
            row = (static_cast<long long>(id) << p.block_shift) + (j & ((1 << p.block_shift) - 1));
        }
        (void)in_bounds(row, LLONG_MAX, p.err);  // a request's tokens are keys of its own (checked build)
      }
      s_row[x] = req >= 0 ? row : -2;
    }
  }
  // (from the last thread down: the first warp looks a row up)
  for (int i = kRopeThreads - 1 - threadIdx.x; i < n_tokens * half; i += kRopeThreads) {
    const int x = MANY ? i / half : 0, pair = i - x * half;
    const uint4 e = __ldg(p.table + pair);
    // (a table packed for more axes than the call gives positions of: the last)
    const int axis = static_cast<int>(min(e.z, static_cast<uint32_t>(p.num_axes - 1)));
    const long long pos = __ldg(p.positions + static_cast<size_t>(axis) * p.total_q + t0 + x);
    const unsigned long long f = (static_cast<unsigned long long>(e.y) << 32) | e.x;
    // turn in [-1/2, 1/2): the product's upper word as a signed fraction
    const int turn = static_cast<int>((static_cast<unsigned long long>(pos) * f) >> 32);
    float s, c;
    sincospif(static_cast<float>(turn) * 0x1p-31f, &s, &c);
    s_cos[i] = c;
    s_sin[i] = s;
  }
  __syncthreads();
  if (mine >= n_tokens) return;
  const long long row = s_row[mine];
  if (row == -2) return;  // a row past the batch (padding): nothing is written
  const float* my_cos = s_cos + mine * half;
  const float* my_sin = s_sin + mine * half;
  __nv_bfloat16* qo = p.q_out + static_cast<size_t>(t) * p.hq * p.d;
  __nv_bfloat16* ko = p.k_cache + static_cast<size_t>(row < 0 ? 0 : row) * p.hkv * p.d;
  __nv_bfloat16* vo = p.v_cache + static_cast<size_t>(row < 0 ? 0 : row) * p.hkv * p.d;
  auto out_of = [&](int h) { return h < p.hq ? qo + static_cast<size_t>(h) * p.d : ko + static_cast<size_t>(h - p.hq) * p.d; };
  const int heads = row < 0 ? p.hq : p.hq + p.hkv;

  for (int u0 = tid; u0 < units; u0 += kAhead * group) {
    if (u0 != tid) load(u0);
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      const int u = u0 + n * group, c = u % per_head;
      if (u >= heads * per_head) continue;
      Eight x = a[n].get(), y = b[n].get();
      const float4* cs = reinterpret_cast<const float4*>(my_cos + 8 * c);
      const float4* sn = reinterpret_cast<const float4*>(my_sin + 8 * c);
      const float4 c0 = cs[0], c1 = cs[1], n0 = sn[0], n1 = sn[1];
      const float co[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
      const float si[8] = {n0.x, n0.y, n0.z, n0.w, n1.x, n1.y, n1.z, n1.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float& e = ADJ ? (i < 4 ? x.x[2 * i] : y.x[2 * i - 8]) : x.x[i];
        float& o = ADJ ? (i < 4 ? x.x[2 * i + 1] : y.x[2 * i - 7]) : y.x[i];
        const float r = e * co[i] - o * si[i];
        o = e * si[i] + o * co[i];
        e = r;
      }
      __nv_bfloat16* dst = out_of(u / per_head);
      store8(dst + at_of(c, 0), x);
      store8(dst + at_of(c, 1), y);
    }
  }
  // The rest is copied: the unrotated dims of q and k, and v.
  const int tail = (p.d - p.rot) / 8;
  for (int u = tid; u < heads * tail; u += group) {
    const int h = u / tail, at = p.rot + 8 * (u % tail);
    Raw8<T> x;
    x.load(head_of(h) + at);
    store8(out_of(h) + at, x.get());
  }
  if (row >= 0)
    for (int u = tid; u < v_units; u += group) {
      if (u != tid) vr.load(v + 8 * u);
      store8(vo + 8 * u, vr.get());
    }
}

}  // namespace

}  // namespace mvp

using namespace mvp;

extern "C" {

int mvp_rope_table_pack(const double* inv_freq, const int32_t* axes, int pairs, int num_axes, void* table) {
  if (inv_freq == nullptr || table == nullptr || pairs < 1 || pairs > kMaxPairs || num_axes < 1 || num_axes > 4)
    return MVP_ERR_ARG;
  // 1 / (2 pi) as the sum of two doubles
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;
  for (int i = 0; i < pairs; ++i) {
    const int axis = axes != nullptr ? axes[i] : 0;
    if (axis < 0 || axis >= num_axes) return MVP_ERR_ARG;
    if (!(std::fabs(inv_freq[i]) <= 6.0)) return MVP_ERR_ARG;  // NaN, or a turn or more per position
    const double hi = inv_freq[i] * kHi;
    const double lo = std::fma(inv_freq[i], kHi, -hi) + inv_freq[i] * kLo;
    // |hi| < 1: hi * 2^62 is an integer below 2^62 or has its last bits cut exactly
    const double whole = std::floor(hi * 0x1p62);
    const double rest = (hi * 0x1p62 - whole) + lo * 0x1p62;  // |rest| < 2^10
    const uint64_t f = (static_cast<uint64_t>(static_cast<int64_t>(whole)) << 2) +
                       static_cast<uint64_t>(static_cast<int64_t>(std::nearbyint(rest * 4.0)));
    const uint32_t e[4] = {static_cast<uint32_t>(f), static_cast<uint32_t>(f >> 32), static_cast<uint32_t>(axis), 0u};
    std::memcpy(static_cast<unsigned char*>(table) + 16 * static_cast<size_t>(i), e, 16);
  }
  return MVP_OK;
}

int mvp_rope_append_paged(const void* q, const void* k, const void* v, int src_fp32, void* q_out, void* k_cache,
                          void* v_cache, const int32_t* positions, const void* rope_table, int num_axes, int rot_dim,
                          int adjacent, const int32_t* cu_seqlens_q, const int32_t* seq_lens_k,
                          const int32_t* block_table, int block_size, int max_blocks_per_seq, int num_blocks,
                          int num_reqs, int total_q, int num_heads_q, int num_heads_kv, int head_dim,
                          long long q_stride, long long k_stride, long long v_stride, void* stream) {
  set_last_launches(0);
  if (num_reqs < 1 || total_q < 0 || num_heads_q < 1 || num_heads_kv < 1) return MVP_ERR_ARG;
  if (head_dim < 16 || head_dim > 2 * kMaxPairs || head_dim % 8 != 0) return MVP_ERR_UNSUPPORTED;
  if (rot_dim < 16 || rot_dim > head_dim) return MVP_ERR_ARG;
  if (rot_dim % 16 != 0) return MVP_ERR_UNSUPPORTED;
  if (num_axes < 1 || num_axes > 4) return MVP_ERR_ARG;
  if ((src_fp32 != 0 && src_fp32 != 1) || (adjacent != 0 && adjacent != 1)) return MVP_ERR_ARG;
  int shift = 0;
  while (shift < 30 && (1 << shift) < block_size) ++shift;
  if (block_size < 16 || block_size > 256 || (1 << shift) != block_size) return MVP_ERR_ARG;
  if (num_blocks < 1 || max_blocks_per_seq < 1) return MVP_ERR_ARG;
  const long long rows_q = static_cast<long long>(num_heads_q) * head_dim;
  const long long rows_kv = static_cast<long long>(num_heads_kv) * head_dim;
  if (rows_q > INT_MAX / 2 || rows_kv > INT_MAX / 2) return MVP_ERR_UNSUPPORTED;
  if (total_q == 0) return MVP_OK;
  if (q == nullptr || k == nullptr || v == nullptr || q_out == nullptr || k_cache == nullptr || v_cache == nullptr ||
      positions == nullptr || rope_table == nullptr || cu_seqlens_q == nullptr || seq_lens_k == nullptr ||
      block_table == nullptr)
    return MVP_ERR_ARG;
  if (q_stride < rows_q || k_stride < rows_kv || v_stride < rows_kv) return MVP_ERR_ARG;
  const uintptr_t all = reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) |
                        reinterpret_cast<uintptr_t>(v) | reinterpret_cast<uintptr_t>(q_out) |
                        reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache) |
                        reinterpret_cast<uintptr_t>(rope_table);
  if ((all & 15u) != 0) return MVP_ERR_UNSUPPORTED;
  const int elem = src_fp32 ? 4 : 2;
  if (((q_stride | k_stride | v_stride) * elem) & 15) return MVP_ERR_UNSUPPORTED;
  int* err = nullptr;
  int num_sms = 1;
  if (device_error_word(&err, &num_sms) != cudaSuccess) return MVP_ERR_CUDA;
  RopeParams p;
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k_cache = static_cast<__nv_bfloat16*>(k_cache);
  p.v_cache = static_cast<__nv_bfloat16*>(v_cache);
  p.positions = positions;
  p.table = static_cast<const uint4*>(rope_table);
  p.cu_q = cu_seqlens_q;
  p.seq_k = seq_lens_k;
  p.block_table = block_table;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.num_reqs = num_reqs;
  p.total_q = total_q;
  p.num_axes = num_axes;
  p.hq = num_heads_q;
  p.hkv = num_heads_kv;
  p.d = head_dim;
  p.rot = rot_dim;
  p.block_shift = shift;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.err = err;
  cudaLaunchConfig_t cfg = {};
  // Tokens per CTA: one, or as many as have 1024 16-byte outputs between them
  // while the GPU gets two CTAs per SM (three fp32 requests of 8/2 heads at D 64,
  // 76 outputs a row: 6.3 us in a graph; 12.2 against 13.9 called one by one).
  const int outputs = (num_heads_q + num_heads_kv) * (rot_dim / 16 + (head_dim - rot_dim) / 8) + num_heads_kv * head_dim / 8;
  p.tokens = 1;
  while (p.tokens < kMaxTokens && 2 * p.tokens * outputs <= 1024 && 2 * p.tokens * (rot_dim / 2) <= kMaxAngles &&
         total_q / (2 * p.tokens) >= 2 * num_sms)
    p.tokens *= 2;
  cfg.gridDim = dim3((total_q + p.tokens - 1) / p.tokens);
  cfg.blockDim = dim3(kRopeThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  using Kern = void (*)(RopeParams);
  const Kern kerns[2][2][2] = {
      {{rope_append_kernel<__nv_bfloat16, false, false>, rope_append_kernel<__nv_bfloat16, false, true>},
       {rope_append_kernel<__nv_bfloat16, true, false>, rope_append_kernel<__nv_bfloat16, true, true>}},
      {{rope_append_kernel<float, false, false>, rope_append_kernel<float, false, true>},
       {rope_append_kernel<float, true, false>, rope_append_kernel<float, true, true>}}};
  const Kern kern = kerns[src_fp32][adjacent][p.tokens > 1];
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return MVP_ERR_CUDA;
  set_last_launches(1);
  return MVP_OK;
}

}  // extern "C"
