// Prefill attention under a window that leaves the first tokens visible: the
// FIRST instantiations of attn_prefill.cuh.  They are a translation unit of
// their own so that the others stay what they are (the extra interval costs
// registers in the softmax warps) and both compile in parallel.
#include "attn_prefill.cuh"

namespace mvp {

cudaError_t launch_prefill_first(int head_dim, const PrefillParams& p, const CUtensorMap& mq, const CUtensorMap& mk,
                                 const CUtensorMap& mv, cudaStream_t stream) {
  switch (head_dim) {
    case 64: return launch_cfg<Cfg64, true>(p, mq, mk, mv, stream);
    case 128: return launch_cfg<Cfg128, true>(p, mq, mk, mv, stream);
    case 256: return launch_cfg<Cfg256, true>(p, mq, mk, mv, stream);
    case 512: return launch_cfg<Cfg512, true>(p, mq, mk, mv, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace mvp
