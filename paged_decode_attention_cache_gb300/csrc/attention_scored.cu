// attention_scored.cu -- the attention kernel's scored passes over every kind of
// cache: capped and distance-biased scores, document and prefix masks (ScoreMod in
// attention_impl.cuh).  Always the tensor-core maths, whose scores sit in registers
// between the two products.  Compiled apart, like the other instantiations.
//
// Bound: HBM behind the start of the launch (plan, first copies) and the merges, about
// 7 us that every balanced call has (12 over the 8-bit caches); the cap's and the bias's
// dozen instructions a score hide behind it.  Measured on one GB300: bf16, 88 MB of
// capped scores in 19.5 us (19.1 without the cap), 68 MB behind a window and a prefix in
// 17.0 us (4.0 TB/s); int8, 88 MB with document starts in 29.5 us (0.5 less without cap and bias).
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
