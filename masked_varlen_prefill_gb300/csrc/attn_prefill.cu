// Prefill attention without first tokens: the instantiations of
// attn_prefill.cuh, and the choice between them by head dimension.
#include "attn_prefill.cuh"

namespace mvp {

template <class C>
PrefillShape shape_of() {
  return {C::BN, C::DV, C::DV_SPLIT, C::BN, C::KROWS, C::NCTA, C::ITEM_ROWS, C::SPLITD ? 2 : 1, C::DQ, C::OC,
          C::ITEM_ROWS, C::OCW - C::OC};
}

PrefillShape prefill_tile_shape(int head_dim, bool d512_head_split) {
  switch (head_dim) {
    case 64: return shape_of<Cfg64>();
    case 128: return shape_of<Cfg128>();
    case 256: return shape_of<Cfg256>();
    case 512: return d512_head_split ? shape_of<Cfg512S>() : shape_of<Cfg512>();
    default: return {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
  }
}

cudaError_t launch_prefill(int head_dim, bool d512_head_split, const PrefillParams& p, const CUtensorMap& mq,
                           const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t stream) {
  if (p.m.sf.any()) return launch_prefill_scored(head_dim, p, mq, mk, mv, stream);
  if (p.m.first_tokens > 0) return launch_prefill_first(head_dim, p, mq, mk, mv, stream);
  switch (head_dim) {
    case 64: return launch_cfg<Cfg64, false>(p, mq, mk, mv, stream);
    case 128: return launch_cfg<Cfg128, false>(p, mq, mk, mv, stream);
    case 256: return launch_cfg<Cfg256, false>(p, mq, mk, mv, stream);
    case 512:
      return d512_head_split ? launch_cfg<Cfg512S, false>(p, mq, mk, mv, stream) : launch_cfg<Cfg512, false>(p, mq, mk, mv, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace mvp
