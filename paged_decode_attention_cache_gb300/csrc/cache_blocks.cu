// cache_blocks.cu -- the 8-bit caches with one scale per (16-token block, kv
// head): the append of new tokens, and the dequantising gather.
//
// A block's scale has to cover every token in it, so the append works on whole
// (sequence, block) pairs instead of single slots: one warp takes the new tokens
// of one (block, kv head), for K or for V, finds their largest magnitude, grows
// the scale if the block's own does not cover it, rewrites the block's older
// codes for the grown scale, and quantises the new rows.  No other warp touches
// that (block, kv head), so there is nothing to wait for and no atomic.
//
// Scales sit on a coarse grid: int8 scales have three significant bits, e4m3
// scales are powers of two.  A scale that grows does so by a quarter or more
// (int8) or doubles (e4m3), so a block filled token by token is re-rounded a few
// times at most where exact scales would re-round at every new maximum, and an
// e4m3 code keeps its value exactly unless it turns subnormal.  The price is up
// to one part in five of int8's range (a tenth on average).
//
// Bound: HBM for prompts (4 bytes read and 2 written per element of K + V: 83 MB in
// 16.2 us, 5.1 TB/s), dependent-load latency for a decode step (length -> table ->
// scale; 64 tokens of 8 heads in 2.4 us).
#include <cuda_fp8.h>

#include <type_traits>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

namespace {

constexpr int kBlock = 16;
constexpr int kThreads = 64;   // append: 83 MB in 17.2, 16.4, 16.2 us with 256, 128, 64

// The largest magnitude of two 16-bit floats in each half of a and b (packed).
template <typename Src>
__device__ __forceinline__ uint32_t absmax2(uint32_t a, uint32_t b) {
    using V = typename std::conditional<std::is_same<Src, __half>::value, __half2, __nv_bfloat162>::type;
    V x, y;
    memcpy(&x, &a, 4);
    memcpy(&y, &b, 4);
    const V z = __hmax2(x, __habs2(y));
    uint32_t r;
    memcpy(&r, &z, 4);
    return r;
}

// amax / qmax rounded up to the scale grid.  0 stays 0; nothing below 2^-126
// (so that 1 / scale is finite).
template <bool E4M3>
__device__ __forceinline__ float scale_for(float amax) {
    const float t = __fdiv_rn(amax, E4M3 ? 448.f : 127.f);
    constexpr uint32_t drop = E4M3 ? 0x007fffffu : 0x001fffffu;
    const float up = __uint_as_float((__float_as_uint(t) + drop) & ~drop);
    return t > 0.f ? fmaxf(up, 1.17549435e-38f) : 0.f;
}

// Four numbers already divided by the scale -> four codes.  int8: adding 1.5 x 2^23
// leaves the number rounded half to even in the low mantissa bits (|x| <= 127 by the
// scale's choice), one addition where rounding and converting take the slow pipe twice.
template <bool E4M3>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    if constexpr (E4M3) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
        return lo | (hi << 16);
    } else {
        auto q = [](float x) { return __float_as_uint(__fadd_rn(x, 12582912.f)); };
        return __byte_perm(__byte_perm(q(a), q(b), 0x0040), __byte_perm(q(c), q(d), 0x0040), 0x5410);
    }
}

template <bool E4M3>
__device__ __forceinline__ float code_value(uint32_t byte) {
    if constexpr (E4M3)
        return __half2float(__half(__nv_cvt_fp8_to_halfraw(__nv_fp8_storage_t(byte), __NV_E4M3)));
    return float(int(int8_t(byte)));
}

// What unit `u` of the work list belongs to: sequence s, whose units start at
// cu[s] / 16 + 2 s (at least as far apart as the blocks its tokens can touch), its
// rows [c0, c1) and its context.  All lanes probe the remaining range at once, and the
// last round brings what the caller needs next with it.
struct UnitSeq {
    int s, c0, c1, ctx;
};
__device__ __forceinline__ UnitSeq find_seq(const BlockWriteParams& p, int u, int lane) {
    int lo = 0, hi = p.num_seqs;   // start(lo) <= u, the answer is in [lo, hi)
    auto start = [&](int c, int s) { return min(max(c, 0), p.num_tokens) / kBlock + 2 * s; };
    while (hi - lo > 31) {
        const int step = (hi - lo + 31) / 32, s = lo + lane * step;
        const uint32_t m = __ballot_sync(0xffffffffu, s < hi && start(p.cu_new[min(s, p.num_seqs)], s) <= u) | 1u;
        lo += (31 - __clz(m)) * step;   // the last probe that starts at or before u
        hi = min(hi, lo + step);
    }
    const int s = lo + lane;
    const int c = min(max(p.cu_new[min(s, p.num_seqs)], 0), p.num_tokens);
    const int ctx = p.context_lens[min(s, p.num_seqs - 1)];
    const uint32_t m = __ballot_sync(0xffffffffu, s < hi && start(c, s) <= u) | 1u;
    const int last = 31 - __clz(m);
    return {lo + last, __shfl_sync(0xffffffffu, c, last), __shfl_sync(0xffffffffu, c, last + 1),
            __shfl_sync(0xffffffffu, ctx, last)};
}

template <typename Src, bool E4M3, int D>
__global__ void __launch_bounds__(kThreads, 1) append_blocks_kernel(BlockWriteParams p) {
    grid_dep_wait();
    grid_dep_launch();
    constexpr int LPR = D / 8;           // lanes per row, 8 values each
    constexpr int RPP = 32 / LPR;        // rows per pass
    constexpr int NP = kBlock / RPP;     // passes over the block
    const int lane = threadIdx.x & 31;
    const int H = p.num_kv_heads;
    const int64_t w = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (w >= int64_t(p.units) * H * 2) return;
    const int which = int(w & 1);        // 0: K, 1: V
    const int h = int((w >> 1) % H);
    const int u = int((w >> 1) / H);

    // ---- this unit's sequence, its new tokens and the block
    int s, i, n, row0, ctx;
    if (p.cu_new) {
        const UnitSeq q = find_seq(p, u, lane);
        s = q.s;
        i = u - (q.c0 / kBlock + 2 * s);
        n = q.c1 - q.c0;
        row0 = q.c0;
        ctx = q.ctx;
    } else {
        const int per = (p.q_len + 14) / kBlock + 1;
        s = u / per;
        i = u - s * per;
        n = p.q_len;
        row0 = s * p.q_len;
        ctx = p.context_lens[s];
    }
    if (i < 0 || n <= 0 || ctx <= 0) return;
    const int cap = p.max_blocks * kBlock;
    if (ctx > cap && i == 0 && h == 0 && which == 0 && lane == 0) flag_error(p.err, PKV_DEVERR_CAPACITY);
    const int p0 = max(ctx - n, 0), p1 = min(ctx, cap);   // positions written: [p0, p1)
    if (p0 >= p1) return;
    const int64_t b64 = int64_t(p0 / kBlock) + i;
    if (b64 * kBlock >= p1) return;
    const int b = int(b64);
    const int a = max(p0 - b * kBlock, 0), e = min(p1 - b * kBlock, kBlock);   // new rows [a, e) of the block
    const int pb = p.block_tables[int64_t(s) * p.max_blocks + b];
    const uint16_t* src = static_cast<const uint16_t*>(which ? p.v_new : p.k_new);
    const int64_t stride = which ? p.v_stride : p.k_stride;
    const int r0 = lane / LPR, d0 = (lane % LPR) * 8;

    // ---- the new rows, which do not wait for the table entry
    uint4 x[NP];
    const int64_t src_row = int64_t(row0) + int64_t(b) * kBlock - (int64_t(ctx) - n);   // row of offset 0
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        const int r = k * RPP + r0;
        x[k] = make_uint4(0u, 0u, 0u, 0u);
        if (r >= a && r < e) x[k] = __ldg(reinterpret_cast<const uint4*>(src + (src_row + r) * stride + h * D + d0));
    }
    if (pb < 0 || pb >= p.num_blocks) {
        if (h == 0 && which == 0 && lane == 0) flag_error(p.err, PKV_DEVERR_OOB_BLOCK);
        return;
    }
    const int64_t meta = int64_t(pb) * H + h;
    float* scale_at = (which ? p.v_scale : p.k_scale) + meta;
    uint8_t* codes = static_cast<uint8_t*>(which ? p.v_cache : p.k_cache) + (int64_t(pb) * kBlock * H + h) * D;

    // ---- the scale: the largest magnitude of the new rows, and the block's own
    uint32_t m2 = 0;
    float s_old = a > 0 ? *scale_at : 0.f;
    if (!(s_old > 0.f) || isinf(s_old)) s_old = 0.f;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        m2 = absmax2<Src>(m2, x[k].x);
        m2 = absmax2<Src>(m2, x[k].y);
        m2 = absmax2<Src>(m2, x[k].z);
        m2 = absmax2<Src>(m2, x[k].w);
    }
    const float2 mf = Half16<Src>::unpack2(m2);
    float amax = fmaxf(mf.x, mf.y);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float s_new = fmaxf(s_old, scale_for<E4M3>(amax));
    // a scale below 2^-126, which only the cache's owner can have put there, stays only for new rows of zeros: their codes
    // are 0, not 0 times its infinite reciprocal
    const float inv = s_new >= 1.17549435e-38f ? __fdiv_rn(1.f, s_new) : 0.f;

    // ---- the block's older rows, for a scale that grew
    if (a > 0 && s_new > s_old) {
        const float share = __fdiv_rn(s_old, s_new);
#pragma unroll 2
        for (int r = r0; r < a; r += RPP) {
            uint2* at = reinterpret_cast<uint2*>(codes + int64_t(r) * H * D + d0);
            const uint2 c = *at;
            float f[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) f[q] = code_value<E4M3>(((q < 4 ? c.x : c.y) >> (8 * (q & 3))) & 0xffu) * share;
            *at = make_uint2(codes4<E4M3>(f[0], f[1], f[2], f[3]), codes4<E4M3>(f[4], f[5], f[6], f[7]));
        }
    }
    // ---- the new rows
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        const int r = k * RPP + r0;
        if (r < a || r >= e) continue;
        const float2 f0 = Half16<Src>::unpack2(x[k].x), f1 = Half16<Src>::unpack2(x[k].y);
        const float2 f2 = Half16<Src>::unpack2(x[k].z), f3 = Half16<Src>::unpack2(x[k].w);
        *reinterpret_cast<uint2*>(codes + int64_t(r) * H * D + d0) =
            make_uint2(codes4<E4M3>(f0.x * inv, f0.y * inv, f1.x * inv, f1.y * inv),
                       codes4<E4M3>(f2.x * inv, f2.y * inv, f3.x * inv, f3.y * inv));
    }
    __syncwarp();   // every lane has read the old scale
    if (lane == 0) *scale_at = s_new;
}

// 16 codes -> 16 values of OutT.
template <typename OutT, bool E4M3>
__device__ __forceinline__ void expand16(uint4 c, float scale, uint4& lo, uint4& hi) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint32_t o[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const uint32_t two = (w[q / 2] >> (16 * (q & 1))) & 0xffffu;
        const float x = code_value<E4M3>(two & 0xffu) * scale, y = code_value<E4M3>(two >> 8) * scale;
        if constexpr (std::is_same<OutT, __nv_bfloat16>::value) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
            memcpy(o + q, &v, 4);
        } else {
            const __half2 v = __floats2half2_rn(x, y);
            memcpy(o + q, &v, 4);
        }
    }
    lo = make_uint4(o[0], o[1], o[2], o[3]);
    hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// A CTA expands kGatherItems items of logical block b of sequence s, an item being 16 dims
// of one (token, kv head), K and V: 16-byte loads, and 32-byte stores where the outputs are
// aligned for them (two 16-byte stores leave every 32-byte sector to two instructions).
// Bound by HBM, which writes two bytes for each it reads, where the outputs pass L2: 375 MB
// at 6.5 TB/s (of 6.8 measured for a copy), 149 MB at 6.0.  At 73 MB (13.4 us) the 49 MB of
// outputs stay in the 129 MB L2 (0.6 MB were written to DRAM while it ran): there the start of
// the launch and the issue of loads and stores count.  Measured on the way at
// 73 MB: 17.1 us with a CTA of 256 threads per block and 16-byte stores, 15.8 with halves of
// blocks, 14.7 with 32-byte stores too, 14.0 with one item per thread at a time and quarters
// of 8 heads of 128 dims (256 items), 15.3 with eighths.
constexpr int kGatherThreads = 128, kGatherItems = 256;

__device__ __forceinline__ void store32(uint4* at, uint4 lo, uint4 hi) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(lo.x), "r"(lo.y), "r"(lo.z),
                 "r"(lo.w), "r"(hi.x), "r"(hi.y), "r"(hi.z), "r"(hi.w)
                 : "memory");
}

template <typename OutT, bool E4M3, int D>
__global__ void __launch_bounds__(kGatherThreads) gather_blocks_kernel(GatherParams p) {
    grid_dep_wait();
    grid_dep_launch();
    constexpr int CPT = D / 16;
    const int H = p.num_kv_heads, parts = (kBlock * H * CPT + kGatherItems - 1) / kGatherItems;
    const int s = blockIdx.y, b = blockIdx.x / parts, part = blockIdx.x - b * parts;
    int ctx = p.context_lens[s];
    const int64_t row0 = p.cu_seq_lens[s];
    const int pb = p.block_tables[int64_t(s) * p.max_blocks + b];
    const int cap = p.max_blocks * kBlock;
    if (ctx > cap) {
        if (blockIdx.x == 0 && threadIdx.x == 0) flag_error(p.err, PKV_DEVERR_CAPACITY);
        ctx = cap;
    }
    const int t0 = b * kBlock;
    if (t0 >= ctx) return;
    const int ntok = min(kBlock, ctx - t0);
    if (pb < 0 || pb >= p.num_blocks) {
        if (part == 0 && threadIdx.x == 0) flag_error(p.err, PKV_DEVERR_OOB_BLOCK);
        return;
    }
    const int64_t src0 = int64_t(pb) * kBlock * H * D, dst0 = (row0 + t0) * H * D;
    const uint4* src[2] = {reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.k_cache) + src0),
                           reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.v_cache) + src0)};
    const float* scale[2] = {static_cast<const float*>(p.k_scale) + int64_t(pb) * H, static_cast<const float*>(p.v_scale) + int64_t(pb) * H};
    uint4* dst[2] = {reinterpret_cast<uint4*>(static_cast<OutT*>(p.k_out) + dst0), reinterpret_cast<uint4*>(static_cast<OutT*>(p.v_out) + dst0)};
    const bool wide = ((reinterpret_cast<uintptr_t>(p.k_out) | reinterpret_cast<uintptr_t>(p.v_out)) & 31u) == 0;
    // the block's first ntok token rows are contiguous on both sides
    const int i1 = min(ntok * H * CPT, (part + 1) * kGatherItems);
    for (int i = part * kGatherItems + threadIdx.x; i < i1; i += kGatherThreads) {
        uint4 c[2];
        float sc[2];
        const int h = (i / CPT) % H;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            c[w] = __ldcs(src[w] + i);
            sc[w] = __ldg(scale[w] + h);
        }
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            uint4 lo, hi;
            expand16<OutT, E4M3>(c[w], sc[w], lo, hi);
            if (wide) {
                store32(dst[w] + 2 * i, lo, hi);
            } else {
                dst[w][2 * i] = lo;
                dst[w][2 * i + 1] = hi;
            }
        }
    }
}

template <typename Src, bool E4M3>
cudaError_t append_d(const BlockWriteParams& p, dim3 grid, cudaStream_t st) {
    return p.head_dim == 128 ? launch_kernel(append_blocks_kernel<Src, E4M3, 128>, grid, dim3(kThreads), 0, st, p)
                             : launch_kernel(append_blocks_kernel<Src, E4M3, 64>, grid, dim3(kThreads), 0, st, p);
}

template <typename OutT, bool E4M3>
cudaError_t gather_d(const GatherParams& p, dim3 grid, cudaStream_t st) {
    return p.head_dim == 128 ? launch_kernel(gather_blocks_kernel<OutT, E4M3, 128>, grid, dim3(kGatherThreads), 0, st, p)
                             : launch_kernel(gather_blocks_kernel<OutT, E4M3, 64>, grid, dim3(kGatherThreads), 0, st, p);
}

}  // namespace

cudaError_t launch_append_blocks(BlockWriteParams p, cudaStream_t stream) {
    const int64_t units = p.cu_new ? int64_t(p.num_tokens) / kBlock + 2 * int64_t(p.num_seqs)
                                   : int64_t(p.num_seqs) * ((p.q_len + 14) / kBlock + 1);
    const int64_t ctas = (units * p.num_kv_heads * 2 + kThreads / 32 - 1) / (kThreads / 32);
    if (units > 0x7fffffff || ctas > 0x7fffffff) return cudaErrorInvalidValue;
    p.units = int32_t(units);
    const dim3 grid{unsigned(ctas)};
    const bool e4 = p.cache_kind == PKV_CACHE_E4M3;
    if (p.src_dtype == PKV_BF16)
        return e4 ? append_d<__nv_bfloat16, true>(p, grid, stream) : append_d<__nv_bfloat16, false>(p, grid, stream);
    return e4 ? append_d<__half, true>(p, grid, stream) : append_d<__half, false>(p, grid, stream);
}

cudaError_t launch_gather_blocks(const GatherParams& p, int cache_kind, cudaStream_t stream) {
    const int64_t parts = (int64_t(p.num_kv_heads) * p.head_dim + kGatherItems - 1) / kGatherItems;
    if (p.max_blocks * parts > 0x7fffffff) return cudaErrorInvalidValue;
    const dim3 grid(unsigned(p.max_blocks * parts), p.num_seqs);
    const bool e4 = cache_kind == PKV_CACHE_E4M3;
    if (p.out_dtype == PKV_BF16)
        return e4 ? gather_d<__nv_bfloat16, true>(p, grid, stream) : gather_d<__nv_bfloat16, false>(p, grid, stream);
    return e4 ? gather_d<__half, true>(p, grid, stream) : gather_d<__half, false>(p, grid, stream);
}

}  // namespace pkv
