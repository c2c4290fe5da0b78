// Single-token rows with functions of the score (a tanh cap, a distance bias)
// and documents, under a window that leaves the first tokens visible: instantiations of attn_decode.cuh.
#include "attn_decode.cuh"

namespace mvp {

cudaError_t launch_decode_scored_first(int head_dim, const DecodeParams& p, const CUtensorMap& mk, const CUtensorMap& mv,
                                 cudaStream_t stream, int* launches) {
  return launch_decode_dim<true, true>(head_dim, p, mk, mv, stream, launches);
}

}  // namespace mvp
