// Single-token rows with functions of the score (a tanh cap, a distance bias)
// and documents, without first tokens: instantiations of attn_decode.cuh.
#include "attn_decode.cuh"

namespace mvp {

cudaError_t launch_decode_scored(int head_dim, const DecodeParams& p, const CUtensorMap& mk, const CUtensorMap& mv,
                                 cudaStream_t stream, int* launches) {
  return launch_decode_dim<false, true>(head_dim, p, mk, mv, stream, launches);
}

}  // namespace mvp
