// Prefill attention under a cap past kWideCap, with or without any other function
// of the score and first tokens: instantiations of attn_prefill.cuh (2 x 8192 rows,
// 32/8 heads, D = 128, cap 1e8: 1493 us; 1193 with a cap of 50 and its kernel).  A
// translation unit of its own, so that the others stay what they are and all
// compile in parallel.
#include "attn_prefill.cuh"

namespace mvp {

cudaError_t launch_prefill_scored_wide(int head_dim, const PrefillParams& p, const CUtensorMap& mq, const CUtensorMap& mk,
                                       const CUtensorMap& mv, cudaStream_t stream) {
  switch (head_dim) {
    case 64: return launch_cfg<Cfg64, true, kScored | kCapped | kBiased | kWide>(p, mq, mk, mv, stream);
    case 128: return launch_cfg<Cfg128, true, kScored | kCapped | kBiased | kWide>(p, mq, mk, mv, stream);
    case 256: return launch_cfg<Cfg256, true, kScored | kCapped | kBiased | kWide>(p, mq, mk, mv, stream);
    case 512: return launch_cfg<Cfg512, true, kScored | kCapped | kBiased | kWide>(p, mq, mk, mv, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace mvp
