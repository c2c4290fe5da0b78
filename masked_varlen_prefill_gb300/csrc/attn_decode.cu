// Single-token rows: the plain instantiations of attn_decode.cuh, and the
// choice between them and those for functions of the score.
#include "attn_decode.cuh"

namespace mvp {

int decode_keys_per_tile(int head_dim) { return kt_for(head_dim); }
int decode_box_inner(int head_dim) { return box_for(head_dim); }
int scored_ctas_per_sm(int head_dim) {
  // (228 KB; a CTA takes 1 KB more and up to 4 KB for its probabilities)
  const auto held = [](int smem) { return 228 * 1024 / (smem + 5 * 1024); };
  switch (head_dim) {
    case 64: return held(DCfg<64, true>::SMEM);
    case 128: return held(DCfg<128, true>::SMEM);
    case 256: return held(DCfg<256, true>::SMEM);
    default: return held(DCfg<512, true>::SMEM);
  }
}

cudaError_t launch_decode(int head_dim, const DecodeParams& p, const CUtensorMap& mk, const CUtensorMap& mv,
                          cudaStream_t stream, int* launches) {
  const bool first = p.m.first_tokens > 0;
  if (p.m.sf.any())
    return first ? launch_decode_scored_first(head_dim, p, mk, mv, stream, launches)
                 : launch_decode_scored(head_dim, p, mk, mv, stream, launches);
  return first ? launch_decode_dim<true, false>(head_dim, p, mk, mv, stream, launches)
               : launch_decode_dim<false, false>(head_dim, p, mk, mv, stream, launches);
}

}  // namespace mvp
