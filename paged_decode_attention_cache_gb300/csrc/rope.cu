// rope.cu -- rotary positions of queries and keys, with the cache write of the
// rotated keys and the values in the same launch.
//
//   angle(p, i) = p * f_i,  c = mscale cos, s = mscale sin
//   (a, b) -> (a c - b s, b c + a s) for the pairs (i, i + R/2) (half layout) or
//   (2i, 2i + 1) (interleaved) of the first R = rotary_dim dims of a head.
//
// The angle is exact whatever the position: f_i is held as a 64-bit fraction of
// a turn, so the product's low 64 bits are the phase (whole turns fall off the
// top), one integer multiply where fp32 loses the angle of a far position and
// fp64 runs at a small part of the fp32 rate.  The phase's top 32 bits are
// rounded to fp32 half-turns (2^-25 of a half-turn) for sincospif.
//
// Bound: HBM for prompts (each row read once, written once), launch and
// dependent-load latency for a few tokens.  A CTA takes a few tokens: its
// threads first work out the tokens' R/2 cosines and sines into shared memory,
// once for all the heads, then move 16-byte chunks.
#include <type_traits>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 64;    // R / 2 <= 64
constexpr int kMaxTokens = 4;    // tokens of a CTA

template <typename T>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
    uint32_t r;
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 v = __floats2half2_rn(a, b);
        memcpy(&r, &v, 4);
    } else {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        memcpy(&r, &v, 4);
    }
    return r;
}

// (a, b) turned by (c, s)
__device__ __forceinline__ float2 turn(float a, float b, float2 cs) {
    return make_float2(fmaf(a, cs.x, -(b * cs.y)), fmaf(b, cs.x, a * cs.y));
}

// cosines and sines of `ntok` tokens from t0 on, cs[tok * pairs + i]
__device__ __forceinline__ void angles(const RopeParams& p, int64_t t0, int ntok, float2* cs) {
    const int pairs = p.rotary_dim / 2;
    for (int x = threadIdx.x; x < ntok * pairs; x += kThreads) {
        const int tok = x / pairs, i = x - tok * pairs;
        const uint64_t phase = uint64_t(p.positions[t0 + tok]) * p.freq[i];
        float s, c;
        sincospif(float(int32_t(phase >> 32)) * 4.656612873077393e-10f, &s, &c);
        cs[x] = make_float2(c * p.mscale, s * p.mscale);
    }
}

// Where row h of token t goes: q heads to q_out, k heads to k_out and / or the cache slot.
struct Dest {
    uint16_t* a;
    uint16_t* b;
};

__device__ __forceinline__ int64_t token_slot(const RopeParams& p, int64_t t) {
    if (!p.slot_mapping) return -1;
    const int64_t slot = p.slot_mapping[t];
    return slot < int64_t(p.num_blocks) * 16 ? slot : -1;
}

__device__ __forceinline__ Dest row_dest(const RopeParams& p, int64_t t, int h, int64_t slot) {
    const int D = p.head_dim;
    if (h < p.num_heads) return {static_cast<uint16_t*>(p.q_out) + t * p.q_out_stride + int64_t(h) * D, nullptr};
    h -= p.num_heads;
    Dest d{nullptr, nullptr};
    if (h < p.num_kv_heads) {
        if (p.k_out) d.a = static_cast<uint16_t*>(p.k_out) + t * p.k_out_stride + int64_t(h) * D;
        if (slot >= 0) d.b = static_cast<uint16_t*>(p.k_cache) + (slot * p.num_kv_heads + h) * D;
    } else if (slot >= 0) {
        d.b = static_cast<uint16_t*>(p.v_cache) + (slot * p.num_kv_heads + h - p.num_kv_heads) * D;
    }
    return d;
}

__device__ __forceinline__ const uint16_t* row_src(const RopeParams& p, int64_t t, int h) {
    const int D = p.head_dim;
    if (h < p.num_heads) return static_cast<const uint16_t*>(p.q) + t * p.q_stride + int64_t(h) * D;
    h -= p.num_heads;
    if (h < p.num_kv_heads) return static_cast<const uint16_t*>(p.k) + t * p.k_stride + int64_t(h) * D;
    return static_cast<const uint16_t*>(p.v) + t * p.v_stride + int64_t(h - p.num_kv_heads) * D;
}

__device__ __forceinline__ void flag_slots(const RopeParams& p, int64_t t0, int ntok) {
    if (p.slot_mapping && threadIdx.x < ntok && p.slot_mapping[t0 + threadIdx.x] >= int64_t(p.num_blocks) * 16)
        flag_error(p.err, PKV_DEVERR_OOB_SLOT);
}

// One warp per row (a head of q, k or v of a token), any even rotary_dim: lane l takes pairs l, l + 32, then the
// dims past them one by one.
template <typename T>
__global__ void __launch_bounds__(kThreads) rope_rows_kernel(RopeParams p) {
    grid_dep_wait();
    grid_dep_launch();
    __shared__ float2 cs[kMaxTokens * kMaxPairs];
    const int64_t t0 = int64_t(blockIdx.x) * p.tokens_per_cta;
    const int ntok = int(min(int64_t(p.tokens_per_cta), p.num_tokens - t0));
    flag_slots(p, t0, ntok);
    angles(p, t0, ntok, cs);
    __syncthreads();
    const int lane = threadIdx.x & 31, pairs = p.rotary_dim / 2, D = p.head_dim;
    const int rows = p.num_heads + (p.slot_mapping ? 2 : 1) * p.num_kv_heads;
    for (int r = threadIdx.x >> 5; r < ntok * rows; r += kThreads / 32) {
        const int tok = r / rows, h = r - tok * rows;
        const int64_t t = t0 + tok;
        const Dest d = row_dest(p, t, h, token_slot(p, t));
        if (!d.a && !d.b) continue;
        const uint16_t* src = row_src(p, t, h);
        const int rot = h < p.num_heads + p.num_kv_heads ? pairs : 0;
        for (int i = lane; i < rot; i += 32) {
            const int ia = p.layout == PKV_ROPE_HALF ? i : 2 * i, ib = p.layout == PKV_ROPE_HALF ? i + pairs : 2 * i + 1;
            const float2 y = turn(Half16<T>::to_float(src[ia]), Half16<T>::to_float(src[ib]), cs[tok * pairs + i]);
            const uint32_t w = pack16<T>(y.x, y.y);
            if (d.a) {
                d.a[ia] = uint16_t(w);
                d.a[ib] = uint16_t(w >> 16);
            }
            if (d.b) {
                d.b[ia] = uint16_t(w);
                d.b[ib] = uint16_t(w >> 16);
            }
        }
        for (int i = 2 * rot + lane; i < D; i += 32) {
            const uint16_t x = src[i];
            if (d.a) d.a[i] = x;
            if (d.b) d.b[i] = x;
        }
    }
}

}  // namespace

cudaError_t launch_rope(RopeParams p, cudaStream_t stream) {
    p.tokens_per_cta = kMaxTokens;
    const int64_t ctas = (p.num_tokens + int64_t(p.tokens_per_cta) - 1) / p.tokens_per_cta;
    if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
    const dim3 grid{unsigned(ctas)};
    return p.dtype == PKV_BF16 ? launch_kernel(rope_rows_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, stream, p)
                               : launch_kernel(rope_rows_kernel<__half>, grid, dim3(kThreads), 0, stream, p);
}

}  // namespace pkv
