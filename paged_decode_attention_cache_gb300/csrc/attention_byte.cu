// attention_byte.cu -- the attention kernel over the 8-bit caches with one scale
// per (block, kv head): the plain schedules and the cascade pass.  Compiled
// apart, like the other instantiations.
#include "attention_byte.cuh"

namespace pkv {

namespace {

template <bool E4M3, bool CASC>
cudaError_t dispatch_byte(const AttnParams& p, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t st) {
    const bool narrow = (p.num_heads / p.num_kv_heads) * p.q_len <= 8;
    if (p.head_dim == 128)
        return narrow ? launch_math<TeMath<E4M3, 128, 1>, false, CASC>(p, km, vm, st)
                      : launch_math<TeMath<E4M3, 128, 2>, false, CASC>(p, km, vm, st);
    return narrow ? launch_math<TeMath<E4M3, 64, 1>, false, CASC>(p, km, vm, st)
                  : launch_math<TeMath<E4M3, 64, 2>, false, CASC>(p, km, vm, st);
}

}  // namespace

cudaError_t launch_attention_byte(const AttnParams& p, int cache_kind, const CUtensorMap& km, const CUtensorMap& vm,
                                  cudaStream_t st) {
    if (p.num_new > 0) return cudaErrorInvalidValue;   // no fused step: refused by the entry point
    if (cache_kind == PKV_CACHE_E4M3)
        return is_cascade_pass(p) ? dispatch_byte<true, true>(p, km, vm, st) : dispatch_byte<true, false>(p, km, vm, st);
    return is_cascade_pass(p) ? dispatch_byte<false, true>(p, km, vm, st) : dispatch_byte<false, false>(p, km, vm, st);
}

}  // namespace pkv
