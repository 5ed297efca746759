// attention_scored.cu -- the attention kernel's scored passes over every kind of
// cache: capped and distance-biased scores, document and prefix masks (ScoreMod in
// attention_impl.cuh).  Always the tensor-core maths, whose scores sit in registers
// between the two products.  Compiled apart, like the other instantiations.
#include "attention_byte.cuh"

namespace pkv {

cudaError_t launch_attention_scored(const AttnParams& p, int cache_kind, int gqa, const CUtensorMap& km,
                                    const CUtensorMap& vm, cudaStream_t st) {
    if (p.mode != kModeBalanced || p.num_new > 0 || is_cascade_pass(p)) return cudaErrorInvalidValue;
    if (cache_kind == PKV_CACHE_E4M3) return dispatch_byte<true, kScored>(p, km, vm, st);
    if (cache_kind == PKV_CACHE_I8) return dispatch_byte<false, kScored>(p, km, vm, st);
    return launch_attention_impl<false, kScored>(p, cache_kind, gqa, km, vm, st);
}

}  // namespace pkv
