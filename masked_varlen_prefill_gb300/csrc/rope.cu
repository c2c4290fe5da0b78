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
// upper 32 bits are the turn within 2^-32.  sincospi of twice that turn is
// correct to fp32 at every int32 position.  Rotation is in fp32, rounded once
// to bf16 (what the attention kernels read).
//
// The kernel is bound by memory: (Hq + 2 Hkv) * D elements of each token are
// read and written once.  One CTA per token: a few threads turn the token's
// pairs' angles into shared memory, shared by all the heads, while every
// thread already has its first elements on their way.
#include <cuda_bf16.h>

#include <climits>
#include <cmath>
#include <cstring>

#include "../../include/mvp.h"
#include "mvp_internal.cuh"
#include "ptx.cuh"

namespace mvp {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxPairs = 256;  // head_dim <= 512

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

__device__ __forceinline__ Eight load8(const __nv_bfloat16* p) {
  const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  Eight e;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    e.x[2 * i] = __uint_as_float(w[i] << 16);
    e.x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  return e;
}

__device__ __forceinline__ Eight load8(const float* p) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const Eight& e) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(e.x[0], e.x[1]), pack_bf16x2(e.x[2], e.x[3]),
                                            pack_bf16x2(e.x[4], e.x[5]), pack_bf16x2(e.x[6], e.x[7]));
}

// T: element type of q, k and v.  ADJ: pairs are (2 i, 2 i + 1), else
// (i, i + rot / 2).
template <class T, bool ADJ>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeParams p) {
  __shared__ __align__(16) float s_cos[kMaxPairs], s_sin[kMaxPairs];
  __shared__ long long s_row;
  const int t = blockIdx.x;
  const int half = p.rot / 2;
  griddep_launch_dependents();
  griddep_wait();
  if (threadIdx.x < 32) {
    // the token's cache row, or -1 where it has none
    const int b = request_of_row(p.cu_q, p.num_reqs, t, threadIdx.x);
    if (threadIdx.x == 0) {
      long long row = -1;
      if (b >= 0) {
        const int j = __ldg(p.seq_k + b) - __ldg(p.cu_q + b + 1) + t;
        const int blk = j >> p.block_shift;
        if (j >= 0 && blk < p.max_blocks) {
          const int id = __ldg(p.block_table + static_cast<size_t>(b) * p.max_blocks + blk);
          if (id >= 0 && id < p.num_blocks)
            row = (static_cast<long long>(id) << p.block_shift) + (j & ((1 << p.block_shift) - 1));
        }
        (void)in_bounds(row, LLONG_MAX, p.err);  // a request's tokens are keys of its own (checked build)
      }
      s_row = b >= 0 ? row : -2;
    }
  }
  for (int i = threadIdx.x; i < half; i += kRopeThreads) {
    const uint4 e = __ldg(p.table + i);
    // (a table packed for more axes than the call gives positions of: the last)
    const int axis = static_cast<int>(min(e.z, static_cast<uint32_t>(p.num_axes - 1)));
    const long long pos = __ldg(p.positions + static_cast<size_t>(axis) * p.total_q + t);
    const unsigned long long f = (static_cast<unsigned long long>(e.y) << 32) | e.x;
    // turn in [-1/2, 1/2): the product's upper word as a signed fraction
    const int turn = static_cast<int>((static_cast<unsigned long long>(pos) * f) >> 32);
    float s, c;
    sincospif(static_cast<float>(turn) * 0x1p-31f, &s, &c);
    s_cos[i] = c;
    s_sin[i] = s;
  }
  __syncthreads();
  const long long row = s_row;
  if (row == -2) return;  // a row past the batch (padding): nothing is written

  const T* q = static_cast<const T*>(p.q) + static_cast<size_t>(t) * p.q_stride;
  const T* k = static_cast<const T*>(p.k) + static_cast<size_t>(t) * p.k_stride;
  const T* v = static_cast<const T*>(p.v) + static_cast<size_t>(t) * p.v_stride;
  __nv_bfloat16* qo = p.q_out + static_cast<size_t>(t) * p.hq * p.d;
  __nv_bfloat16* ko = p.k_cache + static_cast<size_t>(row < 0 ? 0 : row) * p.hkv * p.d;
  __nv_bfloat16* vo = p.v_cache + static_cast<size_t>(row < 0 ? 0 : row) * p.hkv * p.d;
  const int heads = row < 0 ? p.hq : p.hq + p.hkv;

  // Rotated part: units of 16 elements (8 pairs) of one head.
  const int per_head = p.rot / 16;
  for (int u = threadIdx.x; u < heads * per_head; u += kRopeThreads) {
    const int h = u / per_head, c = u % per_head;
    const T* src = h < p.hq ? q + static_cast<size_t>(h) * p.d : k + static_cast<size_t>(h - p.hq) * p.d;
    __nv_bfloat16* dst = h < p.hq ? qo + static_cast<size_t>(h) * p.d : ko + static_cast<size_t>(h - p.hq) * p.d;
    const int at0 = ADJ ? 16 * c : 8 * c, at1 = ADJ ? 16 * c + 8 : half + 8 * c;
    Eight a = load8(src + at0), b = load8(src + at1);
    const float4* cs = reinterpret_cast<const float4*>(s_cos + 8 * c);
    const float4* sn = reinterpret_cast<const float4*>(s_sin + 8 * c);
    const float4 c0 = cs[0], c1 = cs[1], n0 = sn[0], n1 = sn[1];
    const float co[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
    const float si[8] = {n0.x, n0.y, n0.z, n0.w, n1.x, n1.y, n1.z, n1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float& x = ADJ ? (i < 4 ? a.x[2 * i] : b.x[2 * i - 8]) : a.x[i];
      float& y = ADJ ? (i < 4 ? a.x[2 * i + 1] : b.x[2 * i - 7]) : b.x[i];
      const float rx = x * co[i] - y * si[i];
      y = x * si[i] + y * co[i];
      x = rx;
    }
    store8(dst + at0, a);
    store8(dst + at1, b);
  }
  // The rest is copied: the unrotated dims of q and k, and v.
  const int tail = (p.d - p.rot) / 8;
  for (int u = threadIdx.x; u < heads * tail; u += kRopeThreads) {
    const int h = u / tail, at = p.rot + 8 * (u % tail);
    const T* src = h < p.hq ? q + static_cast<size_t>(h) * p.d : k + static_cast<size_t>(h - p.hq) * p.d;
    __nv_bfloat16* dst = h < p.hq ? qo + static_cast<size_t>(h) * p.d : ko + static_cast<size_t>(h - p.hq) * p.d;
    store8(dst + at, load8(src + at));
  }
  if (row >= 0)
    for (int u = threadIdx.x; u < p.hkv * p.d / 8; u += kRopeThreads) store8(vo + 8 * u, load8(v + 8 * u));
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
  if (device_error_word(&err) != cudaSuccess) return MVP_ERR_CUDA;
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
  cfg.gridDim = dim3(total_q);
  cfg.blockDim = dim3(kRopeThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  auto kern = src_fp32 ? (adjacent ? rope_append_kernel<float, true> : rope_append_kernel<float, false>)
                       : (adjacent ? rope_append_kernel<__nv_bfloat16, true> : rope_append_kernel<__nv_bfloat16, false>);
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return MVP_ERR_CUDA;
  set_last_launches(1);
  return MVP_OK;
}

}  // extern "C"
