// attention_byte.cu -- the attention kernel over the 8-bit caches with one scale
// per (block, kv head): the plain schedules and the cascade pass.  Compiled
// apart, like the other instantiations.
#include "attention_byte.cuh"

namespace pkv {

cudaError_t launch_attention_byte(const AttnParams& p, int cache_kind, const CUtensorMap& km, const CUtensorMap& vm,
                                  cudaStream_t st) {
    if (p.num_new > 0) return cudaErrorInvalidValue;   // no fused step: refused by the entry point
    if (cache_kind == PKV_CACHE_E4M3)
        return is_cascade_pass(p) ? dispatch_byte<true, kCascade>(p, km, vm, st) : dispatch_byte<true, kPlain>(p, km, vm, st);
    return is_cascade_pass(p) ? dispatch_byte<false, kCascade>(p, km, vm, st) : dispatch_byte<false, kPlain>(p, km, vm, st);
}

}  // namespace pkv
