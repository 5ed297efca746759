// attention_byte.cuh -- block math of the caches held in 8 bits with one scale
// per (16-token block, kv head): int8 (PKV_CACHE_I8) and fp8 e4m3
// (PKV_CACHE_E4M3) codes.  Included after attention_impl.cuh.
#pragma once

#include "attention_impl.cuh"

namespace pkv {

namespace {

__device__ __forceinline__ uint32_t hsub2_u32(uint32_t a, uint32_t b) {
    __half2 x, y;
    memcpy(&x, &a, 4);
    memcpy(&y, &b, 4);
    const __half2 z = __hsub2(x, y);
    uint32_t r;
    memcpy(&r, &z, 4);
    return r;
}

// Four codes (code i in byte i) -> fp16x2 of codes (0, 2) and (1, 3), exact.
// int8: the byte goes under the exponent of 1024 with its sign bit flipped, which
// is 1152 + code; subtract 1152.
// e4m3: the conversion instruction, on bytes put in that order.  Its NaN codes
// (0x7f, 0xff) come out NaN.
template <bool E4M3>
__device__ __forceinline__ void bytes_to_f16(uint32_t w, uint32_t& even, uint32_t& odd) {
    if constexpr (E4M3) {
        const uint32_t x = __byte_perm(w, 0u, 0x3120);
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
            : "=r"(even), "=r"(odd)
            : "r"(x));
    } else {
        even = hsub2_u32((w & 0x00ff00ffu) ^ 0x64806480u, 0x64806480u);
        odd = hsub2_u32(((w >> 8) & 0x00ff00ffu) ^ 0x64806480u, 0x64806480u);
    }
}

// As TqMath, the contraction is turned around: S^T = K Q^T puts the block's 16
// tokens on the MMA's M side and up to 8 (NT = 1) or 16 (NT = 2) query columns
// on N, and O^T = V^T P^T puts 16 head dims on M.
//   K: codes to exact fp16 in registers.  A thread's four k positions of a
//      k-step are four consecutive bytes of a row, paired (0, 2) and (1, 3); the
//      query operand uses the same dim order.  The block's one K scale
//      multiplies the scores.
//   Q: fp16 in the operand.  bf16 queries are first scaled by a power of two
//      per row (largest magnitude to [256, 512)), taken off the scores again, so
//      no bf16 query leaves fp16's range.
//   V: codes to fp16 in the A operand (ldmatrix.trans of 16-bit words = 2 dims x
//      2 tokens): the 16 dims of an M tile are a row's 16-byte chunk, even dims in
//      rows 0-7, odd dims in rows 8-15.  The block's one V scale goes into P,
//      relative to the largest scale seen so far (vref, a power of two; the
//      accumulators are rescaled when it grows, as for the running maximum) and
//      times 2^14, so that the operand P * scale / vref * 2^14 keeps its bits
//      down to 2^-28 of the largest; the accumulators stay in the MMA.  (A
//      multiply-add of each block's product onto the accumulators took 32 more
//      instructions and as many registers.)
//   P: fp16 hi + lo (two MMAs, P exact to ~2^-22): one fp16 P rounds each weight
//      by 2^-12, as large an error as the rounding of an fp16 output.
// 4 KB per block and kv head at D = 128: half the bf16 cache's bytes for about
// the same instructions, so the consumers' issue rate sits nearer the HBM rate.
template <bool E4M3, int D, int NT>
struct TeMath {
    static constexpr bool kTensor = true;
    static constexpr int kD = D;
    static constexpr int NCW = NT == 1 ? 11 : 7;
    static constexpr int kSegCost = pkv::kSegCost;
    static constexpr int kIssueGroup = 22;
    static constexpr int NKS = D / 16;     // k-steps of the score contraction
    static constexpr int NMT = D / 16;     // M tiles of O^T
    static constexpr int KT = kBS * D;
    static constexpr int OFF_V = align_up(KT, 1024);
    static constexpr int TX = 2 * KT;   // bytes the TMA copies deliver
    static constexpr int STAGE = 2 * KT;
    // {K scale, V scale} of each stage, in an array of their own: behind the tiles
    // they cost a stage 1 KB of padding, and the ring a quarter of its depth
    // (copies alone, 8 x 65536 tokens: 135 us against 111 us)
    static constexpr int kSide = 8;
    static constexpr int SCRATCH = 0;
    static constexpr bool kQ8 = true;
    static constexpr float kPUnit = 16384.f;   // 2^14, see V
    static_assert(OFF_V % 1024 == 0 && STAGE % 1024 == 0, "swizzled tiles need 1 KB alignment");

    uint32_t qb[NT][NKS][2];   // Q^T operand: query column g (+8), this thread's dims
    float o[NT][NMT][4];       // O^T: dims 16 mt + 2g, + 1 of query columns 2t, 2t + 1
    float m_run[NT][2], l_part[NT][2];   // query columns 2t, 2t + 1 (l: this thread's tokens)
    float vref;                // o holds sum P V / (vref 2^-14)
    float kcol[NT][2];         // what turns the column's products into base-2 scores, but for the K scale
    int lim[NT][2];
    int lo_;       // first visible token
    int lim_lo_;   // smallest lim over this thread's live columns (no live column: INT_MAX)
    ScoreMod<2 * NT> mod_;   // query columns 8 nt + 2t, + 1
    float scale_log2_;

    static __device__ __forceinline__ void issue(uint8_t* dst, uint8_t* side, const CUtensorMap* km,
                                                 const CUtensorMap* vm, const AttnParams& p, int kvh, int pb,
                                                 uint64_t* bar) {
        const size_t meta = size_t(pb) * p.num_kv_heads + kvh;
        cp_async_4(side, static_cast<const float*>(p.k_scale) + meta);
        cp_async_4(side + 4, static_cast<const float*>(p.v_scale) + meta);
        cp_async_mbar_arrive(bar);
        mbar_arrive_expect_tx(bar, TX);
        const uint64_t pol = l2_evict_first_policy();
        tma_load_2d_hint(dst, km, kvh * D, pb * kBS, bar, pol);
        tma_load_2d_hint(dst + OFF_V, vm, kvh * D, pb * kBS, bar, pol);
    }

    // the fused step does not take these caches (a new token may change its block's scale)
    __device__ __forceinline__ void patch(uint8_t*, int, int, const uint8_t*, int, const AttnParams&) const {}

    __device__ __forceinline__ void init(int) {}

    // query column n = head (n / q_len), draft (n % q_len)
    template <int VAR>
    __device__ __forceinline__ void begin(const AttnParams& p, int s, int kvh, int ctx, int lane) {
        const int g = lane >> 2, t = lane & 3;
        const int G = p.num_heads / p.num_kv_heads, QL = p.q_len, M = G * QL;
        lo_ = visible_lo<VAR>(p, s, ctx);
        if constexpr (VAR == kScored) mod_.begin(p, s, ctx);
        lim_lo_ = INT_MAX;
        vref = 1.17549435e-38f;   // 2^-126
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int n = 8 * nt + g;
            const int h = n < M ? n / QL : 0, j = n < M ? n % QL : 0;
            const int qr = n < M ? query_row<VAR>(p, s, j) : -1;
            const bool valid = qr >= 0;
            const size_t qoff = (size_t(valid ? qr : 0) * p.num_heads + kvh * G + h) * D;
            // this thread's dims t*D/4 .. t*D/4 + D/4 - 1: D/2 contiguous bytes, as 16-byte loads
            uint32_t qw[D / 8];
            const uint4* qv = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.q) + qoff + t * (D / 4));
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint4 x = valid ? qv[i] : make_uint4(0u, 0u, 0u, 0u);
                qw[4 * i] = x.x; qw[4 * i + 1] = x.y; qw[4 * i + 2] = x.z; qw[4 * i + 3] = x.w;
            }
            float back = 1.f;
            if (p.q_dtype == PKV_BF16) {
                // largest exponent field of the column: the power of two that brings it to 2^8
                uint32_t ex = 0;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) ex = max(ex, max((qw[i] >> 7) & 0xffu, (qw[i] >> 23) & 0xffu));
                ex = max(ex, __shfl_xor_sync(0xffffffffu, ex, 1));
                ex = max(ex, __shfl_xor_sync(0xffffffffu, ex, 2));
                // 2^(135 - ex) and its inverse stay normal fp32 numbers; a row of zeros or subnormals
                // (ex 0) and one with an infinity or NaN (ex 255) take the nearest of them
                const uint32_t e = min(max(ex, 16u), 254u);
                const float up = __uint_as_float((262u - e) << 23);
                back = __uint_as_float((e - 8u) << 23);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const float2 f = Half16<__nv_bfloat16>::unpack2(qw[i]);
                    qw[i] = pack2<false>(f.x * up, f.y * up);
                }
            }
#pragma unroll
            for (int kk = 0; kk < NKS; ++kk) {
                // dims d0 .. d0 + 3 (d0 = t*D/4 + 4*kk) as (d0, d0 + 2), (d0 + 1, d0 + 3)
                qb[nt][kk][0] = __byte_perm(qw[2 * kk], qw[2 * kk + 1], 0x5410);
                qb[nt][kk][1] = __byte_perm(qw[2 * kk], qw[2 * kk + 1], 0x7632);
            }
            // column 2t + e's factor sits in the lanes of g = 2t + e
            const float kc = scale_log2_ * back;
            kcol[nt][0] = __shfl_sync(0xffffffffu, kc, (2 * t) * 4);
            kcol[nt][1] = __shfl_sync(0xffffffffu, kc, (2 * t + 1) * 4);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int n2 = 8 * nt + 2 * t + e;
                const int j2 = n2 % QL;
                if constexpr (VAR == kScored) mod_.column(p, 2 * nt + e, kvh * G + (n2 < M ? n2 / QL : 0), j2, ctx);
                const bool ok2 = n2 < M && query_row<VAR>(p, s, j2) >= 0;
                // a cascade row (one decode query) sees the entry's whole context; verify rows are causal
                lim[nt][e] = ok2 ? (VAR == kCascade ? ctx : max(0, ctx - QL + j2 + 1)) : 0;
                if (lim[nt][e] > 0) lim_lo_ = min(lim_lo_, lim[nt][e]);
                m_run[nt][e] = -INFINITY;
                l_part[nt][e] = 0.f;
            }
#pragma unroll
            for (int mt = 0; mt < NMT; ++mt) o[nt][mt][0] = o[nt][mt][1] = o[nt][mt][2] = o[nt][mt][3] = 0.f;
        }
    }

    template <int VAR>
    __device__ __forceinline__ void block(const uint8_t* stg, const uint8_t* side, int pos0, int ntok, int lane) {
        const int g = lane >> 2, t = lane & 3;
        const uint32_t stg_a = smem_addr(stg);
        // ------------------------------------------------ S^T = K Q^T (rows = tokens g, g + 8)
        uint32_t w[2][NKS];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = g + 8 * r;
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const int c = t * (D / 64) + i;
                const uint4 v = *reinterpret_cast<const uint4*>(stg + row * D + 16 * swz<D>(c, row));
                w[r][4 * i] = v.x; w[r][4 * i + 1] = v.y; w[r][4 * i + 2] = v.z; w[r][4 * i + 3] = v.w;
            }
        }
        const float2 ss = *reinterpret_cast<const float2*>(side);
        float sc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
#pragma unroll
        for (int kk = 0; kk < NKS; ++kk) {
            uint32_t a[4];
            bytes_to_f16<E4M3>(w[0][kk], a[0], a[2]);
            bytes_to_f16<E4M3>(w[1][kk], a[1], a[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(sc[nt], a, qb[nt][kk][0], qb[nt][kk][1]);
        }
        // block scale, base-2 softmax scale, causal / context mask
        const int pg = pos0 + g, pg8 = pos0 + g + 8;
        const bool all = pos0 >= lo_ && pos0 + kBS <= lim_lo_;   // whole block visible to every live column
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float k = ss.x * kcol[nt][e];
                if constexpr (VAR == kScored) {
                    const bool v0 = pg < lim[nt][e] && (pg >= lo_ || pg < mod_.pre);
                    const bool v1 = pg8 < lim[nt][e] && (pg8 >= lo_ || pg8 < mod_.pre);
                    sc[nt][e] = v0 ? mod_(sc[nt][e] * k, pg, 2 * nt + e) : -INFINITY;
                    sc[nt][2 + e] = v1 ? mod_(sc[nt][2 + e] * k, pg8, 2 * nt + e) : -INFINITY;
                } else {
                    const bool v0 = all ? lim[nt][e] > 0 : (pg < lim[nt][e] && pg >= lo_);
                    const bool v1 = all ? lim[nt][e] > 0 : (pg8 < lim[nt][e] && pg8 >= lo_);
                    sc[nt][e] = v0 ? sc[nt][e] * k : -INFINITY;
                    sc[nt][2 + e] = v1 ? sc[nt][2 + e] * k : -INFINITY;
                }
            }
        // ------------------------------------------------ online softmax per query column
        float alpha[NT][2];
        bool rescale = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float bm = fmaxf(sc[nt][e], sc[nt][2 + e]);
                bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 4));
                bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 8));
                bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 16));
                const float mn = fmaxf(m_run[nt][e], bm);
                const float mu = (mn == -INFINITY) ? 0.f : mn;
                // nothing accumulated yet (padding columns stay so): no rescale
                alpha[nt][e] = (m_run[nt][e] == -INFINITY) ? 1.f : exp2_ftz(m_run[nt][e] - mu);
                const float p0 = exp2_ftz(sc[nt][e] - mu), p1 = exp2_ftz(sc[nt][2 + e] - mu);
                sc[nt][e] = p0;
                sc[nt][2 + e] = p1;
                l_part[nt][e] = l_part[nt][e] * alpha[nt][e] + (p0 + p1);
                m_run[nt][e] = mn;
                rescale |= alpha[nt][e] != 1.f;
            }
        float grow = 1.f;
        if (fabsf(ss.y) > vref) {   // the same in every lane
            const uint32_t up = min((__float_as_uint(fabsf(ss.y)) + 0x007fffffu) & 0xff800000u, 253u << 23);
            const float ref = __uint_as_float(up);
            grow = vref * __uint_as_float((254u << 23) - up);
            vref = ref;
            rescale = true;
        }
        if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float f0 = alpha[nt][0] * grow, f1 = alpha[nt][1] * grow;
#pragma unroll
                for (int mt = 0; mt < NMT; ++mt) {
                    o[nt][mt][0] *= f0; o[nt][mt][2] *= f0;
                    o[nt][mt][1] *= f1; o[nt][mt][3] *= f1;
                }
            }
        }
        // ------------------------------------------------ P^T operand (tokens 2t.., query column g), hi and lo
        uint32_t ph[NT][2], pl[NT][2];
        // scale / vref is exact but for a subnormal product: 1 / vref is a power of two
        const float ratio = ss.y * __uint_as_float((254u << 23) - __float_as_uint(vref)) * kPUnit;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float x = sc[nt][2 * r] * ratio, y = sc[nt][2 * r + 1] * ratio;
                const uint32_t h = pack2<false>(x, y);
                const float2 hf = Half16<__half>::unpack2(h);
                ph[nt][r] = movm_trans(h);
                pl[nt][r] = movm_trans(pack2<false>(x - hf.x, y - hf.y));
            }
        // ------------------------------------------------ O^T += V^T P^T
        // e4m3 V rows past the context may hold NaN codes: zero them in the operand
        const uint32_t m01 = (2 * t < ntok ? 0x0000ffffu : 0u) | (2 * t + 1 < ntok ? 0xffff0000u : 0u);
        const uint32_t m23 = (8 + 2 * t < ntok ? 0x0000ffffu : 0u) | (9 + 2 * t < ntok ? 0xffff0000u : 0u);
#pragma unroll
        for (int c0 = 0; c0 < NMT; c0 += 2) {
            // matrices (transposed 16-bit words): tokens 0-7, 8-15 of chunk c0, then of chunk c0 + 1
            const int mi = lane >> 3, r = lane & 7;
            const int tok = (mi & 1) * 8 + r, c = c0 + (mi >> 1);
            uint32_t X[4];
            ldsm_x4_t(stg_a + OFF_V + tok * D + 16 * swz<D>(c, tok), X);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t a[4];
                bytes_to_f16<E4M3>(X[2 * h], a[0], a[1]);
                bytes_to_f16<E4M3>(X[2 * h + 1], a[2], a[3]);
                if (E4M3 && ntok < kBS) {
                    a[0] &= m01; a[1] &= m01; a[2] &= m23; a[3] &= m23;
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma_f16(o[nt][c0 + h], a, ph[nt][0], ph[nt][1]);
                    mma_f16(o[nt][c0 + h], a, pl[nt][0], pl[nt][1]);
                }
            }
        }
    }

    __device__ __forceinline__ void finish(int) {
        const float unit = vref * (1.f / kPUnit);   // 0 if vref never grew: then every scale was 0, or no block came
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int mt = 0; mt < NMT; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[nt][mt][i] *= unit;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = l_part[nt][e];
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                l_part[nt][e] = l;
            }
    }

    // unnormalised rows [M][D] (ob_idx order) and per-row (m, l) of this warp
    __device__ __forceinline__ void store(float* ob, float* mw, float* lw, int M, int lane) const {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int q = 8 * nt + 2 * t + e;
                if (q >= M) continue;
#pragma unroll
                for (int mt = 0; mt < NMT; ++mt)
                    *reinterpret_cast<float2*>(ob + ob_idx(q, 16 * mt + 2 * g, D)) =
                        make_float2(o[nt][mt][e], o[nt][mt][2 + e]);
                if (g == 0) {
                    mw[q] = m_run[nt][e];
                    lw[q] = l_part[nt][e];
                }
            }
    }
};

template <bool E4M3, int VAR>
cudaError_t dispatch_byte(const AttnParams& p, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t st) {
    const bool narrow = (p.num_heads / p.num_kv_heads) * p.q_len <= 8;
    if (p.head_dim == 128)
        return narrow ? launch_math<TeMath<E4M3, 128, 1>, false, VAR>(p, km, vm, st)
                      : launch_math<TeMath<E4M3, 128, 2>, false, VAR>(p, km, vm, st);
    return narrow ? launch_math<TeMath<E4M3, 64, 1>, false, VAR>(p, km, vm, st)
                  : launch_math<TeMath<E4M3, 64, 2>, false, VAR>(p, km, vm, st);
}

}  // namespace

}  // namespace pkv
