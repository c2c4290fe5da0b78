// Prefill attention with functions of the score (a tanh cap, a distance bias)
// and documents: the SCORED instantiations of attn_prefill.cuh, which also
// take first tokens.  A translation unit of their own, like
// attn_prefill_first.cu's, so that the others stay what they are.
#include "attn_prefill.cuh"

namespace mvp {

cudaError_t launch_prefill_scored(int head_dim, const PrefillParams& p, const CUtensorMap& mq, const CUtensorMap& mk,
                                  const CUtensorMap& mv, cudaStream_t stream) {
  switch (head_dim) {
    case 64: return launch_cfg<Cfg64, true, true>(p, mq, mk, mv, stream);
    case 128: return launch_cfg<Cfg128, true, true>(p, mq, mk, mv, stream);
    case 256: return launch_cfg<Cfg256, true, true>(p, mq, mk, mv, stream);
    case 512: return launch_cfg<Cfg512, true, true>(p, mq, mk, mv, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace mvp
