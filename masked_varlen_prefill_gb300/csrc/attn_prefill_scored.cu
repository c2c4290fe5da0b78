// Prefill attention whose rows see their document alone: instantiations of
// attn_prefill.cuh.  Translation units of their own, like
// attn_prefill_first.cu, so that the others stay what they are and all
// compile in parallel.
#include "attn_prefill.cuh"

namespace mvp {

cudaError_t launch_prefill_docs(int head_dim, const PrefillParams& p, const CUtensorMap& mq, const CUtensorMap& mk,
                                const CUtensorMap& mv, cudaStream_t stream) {
  switch (head_dim) {
    case 64: return launch_cfg<Cfg64, false, kScored>(p, mq, mk, mv, stream);
    case 128: return launch_cfg<Cfg128, false, kScored>(p, mq, mk, mv, stream);
    case 256: return launch_cfg<Cfg256, false, kScored>(p, mq, mk, mv, stream);
    case 512: return launch_cfg<Cfg512, false, kScored>(p, mq, mk, mv, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_prefill_scored(int head_dim, const PrefillParams& p, const CUtensorMap& mq, const CUtensorMap& mk,
                                  const CUtensorMap& mv, cudaStream_t stream) {
  const bool cap = p.m.sf.cap_log2 > 0.f, bias = p.m.sf.slopes != nullptr;
  if (p.m.sf.wide) return launch_prefill_scored_wide(head_dim, p, mq, mk, mv, stream);
  if (p.m.first_tokens > 0) return launch_prefill_scored_first(head_dim, p, mq, mk, mv, stream);
  if (cap && bias) return launch_prefill_capped_biased(head_dim, p, mq, mk, mv, stream);
  if (cap) return launch_prefill_capped(head_dim, p, mq, mk, mv, stream);
  if (bias) return launch_prefill_biased(head_dim, p, mq, mk, mv, stream);
  return launch_prefill_docs(head_dim, p, mq, mk, mv, stream);
}

}  // namespace mvp
