// attention_byte.cuh -- attention over the caches held in 8 bits with one scale per
// (16-token block, kv head): int8 (PKV_CACHE_I8) and fp8 e4m3 (PKV_CACHE_E4M3)
// codes.  The work list, the balanced plan and the piece combine are those of
// attention_impl.cuh; the kernel around them is this file's own, for a block of
// half the size (4 KB at head_dim 128) and more instructions per byte:
//
//   - A CTA's range of blocks is cut once more, into one contiguous share per warp.
//     A warp streams its share by itself: it fills its own stages (ReadAhead), keeps
//     the softmax state across its blocks and stores the pairs that lie in its share
//     whole straight from registers.  The warps meet once, when all are through:
//     then the partials of the pairs cut between them are merged, and those cut
//     between CTAs published and combined as in attention_impl.cuh.
//   - A step is two blocks: 32 tokens share a wait, a maximum and a refill.
// What this replaced (one GB300, 32 x 4096 tokens e4m3): one producer warp issues
// copies of 4 KB blocks at about 85 % of the HBM rate, and with every pair spread
// over all the warps a barrier at each segment's end took a third of their time.
// Measured (one GB300, 8 kv heads of 128 dims): 8 x 65536 int8, 8 query rows a kv head,
// 703 MB in 120.6 us, 5.8 TB/s of 6.8 measured for a copy; 32 x 4096 e4m3, 4 rows,
// 172 MB in 36.9 us, 4.7 TB/s, of which the plan before the first copy takes about 5 us
// and the merges 4; half the MMAs (both halves of P in one) changed nothing there.
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

// e4m3 codes 0, 1 and 2, 3 of w -> fp16x2 each (exact; the NaN codes 0x7f and 0xff come out NaN).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& c01, uint32_t& c23) {
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(c01), "=r"(c23)
        : "r"(w));
}

// Four K codes -> two fp16x2 operand words.  e4m3: codes (0, 1), (2, 3) by the
// conversion instruction.  int8: codes (0, 2), (1, 3) as fp16 subnormals: the byte
// with its sign bit flipped, alone in a half, is (code + 128) 2^-24 exactly, and
// the MMA takes subnormals; 128 sum(q) comes off the score instead (one LOP a
// word, and two for the odd bytes).
template <bool E4M3>
__device__ __forceinline__ void k_operand(uint32_t w, uint32_t& x, uint32_t& y) {
    if constexpr (E4M3) {
        e4m3x4_to_f16(w, x, y);
    } else {
        x = (w & 0x00ff00ffu) ^ 0x00800080u;
        y = ((w >> 8) & 0x00ff00ffu) ^ 0x00800080u;
    }
}

// Four V codes -> fp16x2 of codes (0, 2) and (1, 3), exact.  int8: the byte goes
// under the exponent of 1024 with its sign bit flipped, which is 1152 + code, and
// 1152 is subtracted: V's sums run over the whole context, where a bias taken off
// at the end would leave the rounding of numbers several times their size.
template <bool E4M3>
__device__ __forceinline__ void v_operand(uint32_t w, uint32_t& even, uint32_t& odd) {
    if constexpr (E4M3) {
        e4m3x4_to_f16(__byte_perm(w, 0u, 0x3120), even, odd);
    } else {
        even = hsub2_u32((w & 0x00ff00ffu) ^ 0x64806480u, 0x64806480u);
        odd = hsub2_u32(((w >> 8) & 0x00ff00ffu) ^ 0x64806480u, 0x64806480u);
    }
}

// A step: up to two consecutive units (blocks) of one segment, one stage.
constexpr int kStepUnits = 2;
__device__ __forceinline__ int seg_steps(int units) { return (units + kStepUnits - 1) / kStepUnits; }

// A warp's next segment: of its share of the CTA's range (the iterator is cut to
// it), or, in the single pass, its share of the CTA's next pair (may be empty).
template <int NCW, int VAR>
__device__ __forceinline__ bool next_share(const AttnParams& p, SegIter<VAR>& it, Seg& sg, int warp) {
    if (!it.next(p, sg)) return false;
    if (p.mode == kModeSingle) {
        const int b0 = sg.b0, ns = seg_steps(sg.b1 - b0);
        sg.b1 = min(sg.b1, b0 + kStepUnits * (ns * (warp + 1) / NCW));
        sg.b0 = b0 + kStepUnits * (ns * warp / NCW);
    }
    return true;
}

// Where a warp reads ahead: its next step to load.  The segment iterator behind it
// is touched once per segment and lives in shared memory; the table entries are read
// a step's time before they are needed.
template <int NCW, int VAR>
struct ReadAhead {
    const int32_t* bt;   // the segment's block table
    int u, end;          // first unit of the next step, the segment's end; u >= end: none
    int kvh, pb0, pb1;   // the step's blocks; pb1 is kNone when it has one
    Span span;
    static constexpr int kNone = INT_MIN;

    __device__ __forceinline__ void walk(const AttnParams& p, SegIter<VAR>* at, int warp, int lane) {
        SegIter<VAR> it = *at;
        Seg g;
        u = end = 0;
        while (next_share<NCW>(p, it, g, warp)) {
            if (g.b0 >= g.b1) continue;
            bt = p.block_tables + size_t(VAR == kCascade ? p.item_seq[g.s] : g.s) * p.max_blocks;
            u = g.b0;
            end = g.b1;
            kvh = g.kvh;
            if constexpr (VAR == kScored) span = g.span;
            break;
        }
        __syncwarp();   // every lane has its copy
        if (lane == 0) *at = it;
        __syncwarp();
        entry();
    }
    __device__ __forceinline__ int block_of(int v) const {
        if constexpr (VAR == kScored) return v < span.npre ? v : v + span.hole;
        return v;
    }
    __device__ __forceinline__ void entry() {
        if (u >= end) return;
        pb0 = bt[block_of(u)];
        pb1 = u + 1 < end ? bt[block_of(u + 1)] : kNone;
    }
    __device__ __forceinline__ void advance(const AttnParams& p, SegIter<VAR>* at, int warp, int lane) {
        u += kStepUnits;
        if (u < end)
            entry();
        else
            walk(p, at, warp, lane);
    }
};

// As TqMath, the contraction is turned around: S^T = K Q^T puts the block's 16
// tokens on the MMA's M side and up to 8 (NT = 1) or 16 (NT = 2) query columns
// on N, and O^T = V^T P^T puts 16 head dims on M.
// Two blocks are one step: their 32 tokens share the maximum, the rescale and the
// bookkeeping (one block at a step took 559 instructions a block; see k_operand,
// v_operand and the V scale below for the rest of the way down).
//   K: codes to exact fp16 in registers.  A thread's four k positions of a
//      k-step are four consecutive bytes of a row; the query operand uses the
//      same dim order.  The block's one K scale multiplies the scores.
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
//   P: fp16 hi + lo (two MMAs, exact to ~2^-22): one operand would round each
//      weight by 2^-12, as large an error as an fp16 output's own rounding.
// 4 KB per block and kv head at D = 128, half the bf16 cache's bytes for more
// instructions: the issue rate of the consumers is what stands nearest the HBM
// rate.
template <bool E4M3, int D, int NT>
struct TeMath {
    static constexpr int kD = D;
    static constexpr int kRows = 8 * NT;
    // warps, three or two to a scheduler (11 left one scheduler's two warps through 4 us before the others' three)
    static constexpr int NCW = NT == 1 ? 12 : 8;
    // Where a warp leaves the partial of its share's first pair: rows 8 .. 15 of the pair's piece slot in the
    // workspace while a pair has at most 8 rows (a CTA has one such partial per sequence: the warp in which the
    // pair ends), which leaves shared memory for 24 stages; else its own slot in shared memory.
    static constexpr bool kHeadInPiece = NT == 1;
    static constexpr int kSegCost = 4;     // balanced: blocks' worth one more segment costs
    static constexpr int NKS = D / 16;     // k-steps of the score contraction
    static constexpr int NMT = D / 16;     // M tiles of O^T
    static constexpr int KT = kBS * D;
    static constexpr int OFF_V = align_up(KT, 1024);
    static constexpr int BLOCK = 2 * KT;   // a block's K and V
    static constexpr int STAGE = kStepUnits * BLOCK;
    // {K scale, V scale} of each block, in an array of their own: behind the tiles
    // they cost a block 1 KB of padding, and the ring a quarter of its depth
    // (copies alone, 8 x 65536 tokens: 135 us against 111 us)
    static constexpr int kSide = kStepUnits * 8;
    static constexpr float kPUnit = 16384.f;   // 2^14, see V
    static constexpr float kKUnit = E4M3 ? 1.f : 16777216.f;   // 2^24: int8 K operands are subnormals
    static_assert(OFF_V % 1024 == 0 && STAGE % 1024 == 0, "swizzled tiles need 1 KB alignment");

    uint32_t qb[NT][NKS][2];   // Q^T operand: query column g (+8), this thread's dims
    float o[NT][NMT][4];       // O^T: dims 16 mt + 2g, + 1 of query columns 2t, 2t + 1
    float m_run[NT][2], l_part[NT][2];   // query columns 2t, 2t + 1 (l: this thread's tokens)
    float vref;                // o holds sum P V / (vref 2^-14)
    float kcol[NT][2];         // what turns the column's products into base-2 scores, but for the K scale
    float kbias[NT][2];        // int8: 128 sum(q) in the products' unit
    int lim[NT][2];
    int lo_;       // first visible token
    int lim_lo_;   // smallest lim over the live columns of the warp (none: INT_MAX)
    ScoreMod<2 * NT> mod_;   // query columns 8 nt + 2t, + 1
    float scale_log2_;

    // A step's blocks pb0 (if ok0) and pb1 (if ok1) into one stage, by the whole warp:
    // lanes 0-3 copy a scale each, then lane 0 the tiles.
    static __device__ __forceinline__ void issue(uint8_t* dst, uint8_t* side, const CUtensorMap* km,
                                                 const CUtensorMap* vm, const AttnParams& p, int kvh, int pb0, bool ok0,
                                                 int pb1, bool ok1, uint64_t* bar, int lane) {
        if (lane < 4 && (lane < 2 ? ok0 : ok1)) {
            const size_t meta = size_t(lane < 2 ? pb0 : pb1) * p.num_kv_heads + kvh;
            cp_async_4(side + 4 * lane, static_cast<const float*>(lane & 1 ? p.v_scale : p.k_scale) + meta);
            cp_async_mbar_arrive(bar);
        }
        __syncwarp();   // the phase waits for those copies before lane 0's arrival can end it
        if (lane == 0) {
            const uint64_t pol = l2_evict_first_policy();
            mbar_arrive_expect_tx(bar, (int(ok0) + int(ok1)) * BLOCK);
            if (ok0) {
                tma_load_2d_hint(dst, km, kvh * D, pb0 * kBS, bar, pol);
                tma_load_2d_hint(dst + OFF_V, vm, kvh * D, pb0 * kBS, bar, pol);
            }
            if (ok1) {
                tma_load_2d_hint(dst + BLOCK, km, kvh * D, pb1 * kBS, bar, pol);
                tma_load_2d_hint(dst + BLOCK + OFF_V, vm, kvh * D, pb1 * kBS, bar, pol);
            }
        }
    }

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
            float qs = 0.f;   // this thread's share of the column's sum of q, as the MMA sees it
#pragma unroll
            for (int kk = 0; kk < NKS; ++kk) {
                // dims d0 .. d0 + 3 (d0 = t*D/4 + 4*kk) in the order of k_operand
                qb[nt][kk][0] = E4M3 ? qw[2 * kk] : __byte_perm(qw[2 * kk], qw[2 * kk + 1], 0x5410);
                qb[nt][kk][1] = E4M3 ? qw[2 * kk + 1] : __byte_perm(qw[2 * kk], qw[2 * kk + 1], 0x7632);
                if constexpr (!E4M3) {
                    const float2 f0 = Half16<__half>::unpack2(qw[2 * kk]), f1 = Half16<__half>::unpack2(qw[2 * kk + 1]);
                    qs += (f0.x + f0.y) + (f1.x + f1.y);
                }
            }
            // column 2t + e's factor sits in the lanes of g = 2t + e
            const float kc = scale_log2_ * back * kKUnit;
            kcol[nt][0] = __shfl_sync(0xffffffffu, kc, (2 * t) * 4);
            kcol[nt][1] = __shfl_sync(0xffffffffu, kc, (2 * t + 1) * 4);
            kbias[nt][0] = kbias[nt][1] = 0.f;
            if constexpr (!E4M3) {
                qs += __shfl_xor_sync(0xffffffffu, qs, 1);
                qs += __shfl_xor_sync(0xffffffffu, qs, 2);
                qs *= 128.f / kKUnit;
                kbias[nt][0] = __shfl_sync(0xffffffffu, qs, (2 * t) * 4);
                kbias[nt][1] = __shfl_sync(0xffffffffu, qs, (2 * t + 1) * 4);
            }
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
        lim_lo_ = min(lim_lo_, __shfl_xor_sync(0xffffffffu, lim_lo_, 1));
        lim_lo_ = min(lim_lo_, __shfl_xor_sync(0xffffffffu, lim_lo_, 2));
    }

    // blocks at positions posa, posb with na, nb stored tokens (0: none to take)
    template <int VAR>
    __device__ __forceinline__ void step(uint8_t* stg, const uint8_t* side, int posa, int na, int posb, int nb,
                                         int lane) {
        const int g = lane >> 2, t = lane & 3;
        const int pos0[2] = {posa, posb}, ntok[2] = {na, nb};
        float sc[2][NT][4];   // scores, then weights: block, query n-tile, tokens g, g + 8 x columns 2t, 2t + 1
        const float4 sraw = *reinterpret_cast<const float4*>(side);
        // a block that was not loaded left what was there before: scale 0, so that weight 0 stays 0
        const float ks[2] = {sraw.x, sraw.z}, vs[2] = {na > 0 ? sraw.y : 0.f, nb > 0 ? sraw.w : 0.f};
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            // -------------------------------------------- S^T = K Q^T (rows = tokens g, g + 8)
            const uint8_t* tile = stg + b * BLOCK;
            uint32_t w[2][NKS];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = g + 8 * r;
#pragma unroll
                for (int i = 0; i < D / 64; ++i) {
                    const int c = t * (D / 64) + i;
                    const uint4 v = *reinterpret_cast<const uint4*>(tile + row * D + 16 * swz<D>(c, row));
                    w[r][4 * i] = v.x; w[r][4 * i + 1] = v.y; w[r][4 * i + 2] = v.z; w[r][4 * i + 3] = v.w;
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[b][nt][i] = -kbias[nt][i & 1];
#pragma unroll
            for (int kk = 0; kk < NKS; ++kk) {
                uint32_t a[4];
                k_operand<E4M3>(w[0][kk], a[0], a[2]);
                k_operand<E4M3>(w[1][kk], a[1], a[3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_f16(sc[b][nt], a, qb[nt][kk][0], qb[nt][kk][1]);
            }
            // block scale, base-2 softmax scale, causal / context mask.  A block that is whole for every live
            // column needs none; a padding column's scores (zero query) then count as visible too, and
            // nobody reads its sums.
            const int pg = pos0[b] + g, pg8 = pos0[b] + g + 8;
            const bool all = VAR != kScored && ntok[b] > 0 && pos0[b] >= lo_ && pos0[b] + kBS <= lim_lo_;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float k = ks[b] * kcol[nt][e];
                    sc[b][nt][e] *= k;
                    sc[b][nt][2 + e] *= k;
                    if constexpr (VAR == kScored) {
                        sc[b][nt][e] = mod_(sc[b][nt][e], pg, 2 * nt + e);
                        sc[b][nt][2 + e] = mod_(sc[b][nt][2 + e], pg8, 2 * nt + e);
                    }
                    if (!all) {
                        const int pre = VAR == kScored ? mod_.pre : 0;
                        if (ntok[b] == 0 || pg >= lim[nt][e] || (pg < lo_ && pg >= pre)) sc[b][nt][e] = -INFINITY;
                        if (ntok[b] == 0 || pg8 >= lim[nt][e] || (pg8 < lo_ && pg8 >= pre)) sc[b][nt][2 + e] = -INFINITY;
                    }
                }
        }
        // ------------------------------------------------ online softmax per query column
        float f[NT][2];   // what the accumulators are multiplied by
        bool rescale = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float bm = fmaxf(fmaxf(sc[0][nt][e], sc[0][nt][2 + e]), fmaxf(sc[1][nt][e], sc[1][nt][2 + e]));
                bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 4));
                bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 8));
                bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 16));
                const float mn = fmaxf(m_run[nt][e], bm);
                const float mu = (mn == -INFINITY) ? 0.f : mn;
                // nothing accumulated yet: no rescale
                f[nt][e] = (m_run[nt][e] == -INFINITY) ? 1.f : exp2_ftz(m_run[nt][e] - mu);
                float sum = 0.f;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    sc[b][nt][e] = exp2_ftz(sc[b][nt][e] - mu);
                    sc[b][nt][2 + e] = exp2_ftz(sc[b][nt][2 + e] - mu);
                    sum += sc[b][nt][e] + sc[b][nt][2 + e];
                }
                l_part[nt][e] = l_part[nt][e] * f[nt][e] + sum;
                m_run[nt][e] = mn;
                rescale |= f[nt][e] != 1.f;
            }
        const float vmax = fmaxf(fabsf(vs[0]), fabsf(vs[1]));
        float grow = 1.f;
        if (vmax > vref) {   // the same in every lane
            const uint32_t up = min((__float_as_uint(vmax) + 0x007fffffu) & 0xff800000u, 253u << 23);
            grow = vref * __uint_as_float((254u << 23) - up);
            vref = __uint_as_float(up);
            rescale = true;
        }
        if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float f0 = f[nt][0] * grow, f1 = f[nt][1] * grow;
#pragma unroll
                for (int mt = 0; mt < NMT; ++mt) {
                    o[nt][mt][0] *= f0; o[nt][mt][2] *= f0;
                    o[nt][mt][1] *= f1; o[nt][mt][3] *= f1;
                }
            }
        }
        // (scale / vref) * 2^14, in this order: vref is 2^-126 .. 2^126, so 1 / vref is a normal power of two and the quotient
        // exact and at most 1 (for scales up to 2^126); it is 0 for a scale of 0, a block of zeros, also while vref is still
        // 2^-126, where 2^14 / vref would be infinite
        const float inv_ref = __uint_as_float((254u << 23) - __float_as_uint(vref));
        auto weigh = [&](uint8_t* tile, float vscale, int pos, int n, const float (&sb)[NT][4]) {
            if (E4M3 && (n < kBS || (VAR == kScored && pos < lo_))) {
                // rows past the context (scored: or masked for all) may hold NaN codes, which weight 0 would not stop:
                // the warp clears them in its own stage.  A test and masks at every operand instead cost 38.5 us at
                // 32 x 4096, this 36.8
                for (int i = lane; i < kBS * (D / 16); i += 32) {
                    const int r = i / (D / 16);
                    bool keep = r < n;
                    if constexpr (VAR == kScored) keep &= pos + r >= lo_ || pos + r < mod_.pre;
                    if (!keep) *reinterpret_cast<uint4*>(tile + OFF_V + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();   // before the next copy into this stage
                __syncwarp();
            }
            // -------------------------------------------- P^T operand (tokens 2t.., query column g)
            uint32_t ph[NT][2], pl[NT][2];
            const float ratio = (vscale * inv_ref) * kPUnit;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float x = sb[nt][2 * r] * ratio, y = sb[nt][2 * r + 1] * ratio;
                    const uint32_t h = pack2<false>(x, y);
                    ph[nt][r] = movm_trans(h);
                    const float2 hf = Half16<__half>::unpack2(h);
                    pl[nt][r] = movm_trans(pack2<false>(x - hf.x, y - hf.y));
                }
            // -------------------------------------------- O^T += V^T P^T
            const uint32_t tile_v = smem_addr(tile) + OFF_V;
#pragma unroll
            for (int c0 = 0; c0 < NMT; c0 += 2) {
                // matrices (transposed 16-bit words): tokens 0-7, 8-15 of chunk c0, then of chunk c0 + 1
                const int mi = lane >> 3, r = lane & 7;
                const int tok = (mi & 1) * 8 + r, c = c0 + (mi >> 1);
                uint32_t X[4];
                ldsm_x4_t(tile_v + tok * D + 16 * swz<D>(c, tok), X);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t a[4];
                    v_operand<E4M3>(X[2 * h], a[0], a[1]);
                    v_operand<E4M3>(X[2 * h + 1], a[2], a[3]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_f16(o[nt][c0 + h], a, ph[nt][0], ph[nt][1]);
                        mma_f16(o[nt][c0 + h], a, pl[nt][0], pl[nt][1]);
                    }
                }
            }
        };
        weigh(stg, vs[0], posa, na, sc[0]);
        weigh(stg + BLOCK, vs[1], posb, nb, sc[1]);
    }

    __device__ __forceinline__ void finish(int) {
        // subnormal (2^-140) if vref never grew: the sums it multiplies are then those of scales up to 2^-126, or zeros
        const float unit = vref * (1.f / kPUnit);
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

    // f(query row, dim, value, value of the next dim) for this lane's part of the sums
    template <class F>
    __device__ __forceinline__ void each(int M, int lane, F f) const {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int q = 8 * nt + 2 * t + e;
                if (q >= M) continue;
#pragma unroll
                for (int mt = 0; mt < NMT; ++mt)
                    f(q, 16 * mt + 2 * g, o[nt][mt][e], o[nt][mt][2 + e], m_run[nt][e], l_part[nt][e]);
            }
    }
};

// ---------------------------------------------------------------- the kernel

// What a warp keeps in shared memory: its iterators, and the segments whose partials
// it leaves: the first of its share ([0], it goes on after that) and the last ([1]).
template <int VAR>
struct WarpState {
    SegIter<VAR> it, ahead;
    Seg part[2];
};

// A pair that a CTA has a piece of: its sequence, the first lane that has one, how many have.
struct Job {
    int s, c_lo, np;
};

// Whether the warps have slots for partials in shared memory (see kHeadInPiece; in the single pass every warp
// leaves one while its stages are already loading the next pair).
template <class Math>
__host__ __device__ constexpr bool own_slots(int mode) {
    return mode == kModeSingle || (mode == kModeBalanced && !Math::kHeadInPiece);
}

// Two consecutive outputs from element i (even).
__device__ __forceinline__ void store_out2(void* out, int dtype, size_t i, float x, float y) {
    if (dtype == PKV_F32)
        reinterpret_cast<float2*>(out)[i >> 1] = make_float2(x, y);
    else if (dtype == PKV_BF16)
        reinterpret_cast<uint32_t*>(out)[i >> 1] = pack2<true>(x, y);
    else
        reinterpret_cast<uint32_t*>(out)[i >> 1] = pack2<false>(x, y);
}

// Cut the CTA's range [u0, u1) of its lane's list into NCW shares of equal cost and set
// `it` to the warp's.  A unit costs 1 and every sequence that begins behind u0 costs
// kShareSeg more (its queries' loads, and the partial or rows left before it: 2.5 us
// against 1.1 us that a warp takes per block at the HBM rate).  32 sequences at a time,
// one per lane.
constexpr int kShareSeg = 2;
template <int NCW, int VAR>
__device__ __forceinline__ void warp_share(const AttnParams& p, const Plan& pl, SegIter<VAR>& it, int warp, int lane) {
    const long long len = pl.u1 - pl.u0;
    long long begins = 0;   // sequences that begin in (u0, u1)
    long long start = pl.start0;
    for (int s0 = pl.s0; s0 < p.num_seqs && start < pl.u1; s0 += 32) {
        const int s = s0 + lane;
        long long n = s < p.num_seqs ? seq_units<VAR>(p, s, seq_ctx(p, s)) : 0, incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
        }
        const long long at = start + incl - n;
        begins += __popc(__ballot_sync(0xffffffffu, n > 0 && at > pl.u0 && at < pl.u1));
        start += __shfl_sync(0xffffffffu, incl, 31);
    }
    const long long total = len + kShareSeg * begins;
    const long long x0 = total * warp / NCW, x1 = total * (warp + 1) / NCW;
    // u(x): the first unit at or past cost position x; unit u of a sequence with b begins before it (its own too)
    // lies at u - u0 + kShareSeg b
    it.u = it.u1 = pl.u1;
    it.s = p.num_seqs;
    bool have0 = false, have1 = warp == NCW - 1;
    long long b0 = 0;
    int r0 = pl.r0;
    start = pl.start0;
    for (int s0 = pl.s0; s0 < p.num_seqs && start < pl.u1 && !(have0 && have1); s0 += 32) {
        const int s = s0 + lane;
        const int ctx = s < p.num_seqs ? seq_ctx(p, s) : 0;
        long long n = s < p.num_seqs ? seq_units<VAR>(p, s, ctx) : 0, incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
        }
        const long long at = start + incl - n;   // the sequence's first unit
        const long long lo = max(at, pl.u0), hi = min(at + n, pl.u1);
        const uint32_t live = __ballot_sync(0xffffffffu, n > 0), mine = 1u << lane;
        const uint32_t began = __ballot_sync(0xffffffffu, n > 0 && at > pl.u0 && at < pl.u1);
        const long long b = b0 + __popc(began & (mine | (mine - 1u)));
        const int r = r0 + __popc(live & (mine - 1u));
        const long long shift = kShareSeg * b - pl.u0;   // position of unit u: u + shift
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const long long x = k ? x1 : x0;
            if (k ? have1 : have0) continue;
            const uint32_t in = __ballot_sync(0xffffffffu, lo < hi && hi + shift > x);
            if (!in) continue;
            const int src = __ffs(in) - 1;
            const long long u = __shfl_sync(0xffffffffu, max(lo, x - shift), src);
            if (k) {
                it.u1 = u;
                have1 = true;
            } else {
                it.u = u;
                it.load_seq(p, s0 + src, __shfl_sync(0xffffffffu, at, src), __shfl_sync(0xffffffffu, ctx, src));
                it.r = __shfl_sync(0xffffffffu, r, src);
                have0 = true;
            }
        }
        b0 += __popc(began);
        r0 += __popc(live);
        start += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (it.u1 < it.u) it.u1 = it.u;
}

template <class Math, int VAR>
__global__ void __launch_bounds__(Math::NCW * 32, 1)
byte_attention_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                      const AttnParams p) {
    constexpr int NCW = Math::NCW, CT = NCW * 32, D = Math::kD, MR = Math::kRows;
    extern __shared__ uint8_t smem_raw[];
    // 1 KB aligned (the swizzled tiles need it), by an offset: shared loads below stay shared loads
    uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const int S = p.stages;
    const int G = p.num_heads / p.num_kv_heads, QL = p.q_len, M = G * QL, H = p.num_heads, Hkv = p.num_kv_heads;
    // shared-memory layout (byte_smem_bytes)
    uint8_t* side = smem + size_t(S) * Math::STAGE;                                // [S][kSide]
    float* ob = reinterpret_cast<float*>(side + S * Math::kSide);                   // [NCW][M][D] or none, ob_idx order
    float* mw = ob + (own_slots<Math>(p.mode) ? NCW * M * D : 0);                   // [2 NCW][MR] maxima of the partials
    float* lw = mw + 2 * NCW * MR;                                                  // [2 NCW][MR] sums
    long long* red = reinterpret_cast<long long*>(lw + 2 * NCW * MR);
    WarpState<VAR>* state = reinterpret_cast<WarpState<VAR>*>(red + kRedSlots);     // [NCW]
    uint64_t* full = reinterpret_cast<uint64_t*>(state + NCW);                      // [S]
    int* poison = reinterpret_cast<int*>(full + S);                                 // [S]
    int* flag = poison + S;                                                         // [4] plan scratch
    int* have = flag + 4;                                                           // [2 NCW] partials left
    Job* jobs = reinterpret_cast<Job*>(have + 2 * NCW);                             // [2]

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < S; ++i) mbar_init(&full[i], 1);
        fence_barrier_init();
    }
    if (tid < 2 * NCW) have[tid] = 0;
#ifdef PKV_TIMELINE
    // as in attention_kernel, but the segment words: 4 warp 0's share is through, 5 all shares, 6 merged, 7 end
    unsigned int tl_launch = 0;
    bool tl_first = true;
    if (tid == 0) {
        tl_launch = p.timeline ? unsigned(atomicAdd(p.timeline, 1ull) / gridDim.x) : 0u;
        PKV_TL(0);
    }
#endif

    // ---- this CTA's range of units (attention_impl.cuh)
    const int lane_kvh = blockIdx.x % Hkv, lane_idx = blockIdx.x / Hkv, nlanes = gridDim.x / Hkv;
    const bool single = p.mode == kModeSingle;
    if (VAR == kCascade || p.wait_first) grid_dep_wait();   // the plan reads what the previous kernel wrote
    Plan pl;
    if (single) {
        const long long total = (long long)p.num_seqs * Hkv;
        pl.chunk = (total + gridDim.x - 1) / gridDim.x;
        pl.u0 = blockIdx.x * pl.chunk;
        pl.u1 = pl.u0 + pl.chunk < total ? pl.u0 + pl.chunk : total;
        pl.s0 = 0;
        pl.ctx0 = -1;
        pl.r0 = 0;
        pl.start0 = 0;
        __syncthreads();
    } else {
        cta_plan<VAR>(p, lane_idx, nlanes, red, flag, pl);
    }
#ifdef PKV_TIMELINE
    if (tid == 0) PKV_TL(1);
#endif
    if (tid == 0) grid_dep_launch();
    if (pl.u1 < pl.u0) pl.u1 = pl.u0;
    WarpState<VAR>& ws = state[warp];
    {
        SegIter<VAR> it;
        it.u = pl.u0;
        it.u1 = pl.u1;
        it.kvh = lane_kvh;
        it.r = pl.r0;
        if (!single) warp_share<NCW>(p, pl, it, warp, lane);
        if (lane == 0) {
            prefetch_tensormap(&k_map);
            prefetch_tensormap(&v_map);
            ws.it = ws.ahead = it;
        }
        __syncwarp();
    }

    // ---- read ahead: fill the stages this warp owns
    ReadAhead<NCW, VAR> ahead;
    auto fill = [&](int st) {
        if (ahead.u >= ahead.end) return;
        // a block out of range is not loaded, and masked out (bit i of poison: unit i of the step)
        const bool two = ahead.pb1 != ahead.kNone;
        const bool ok0 = ahead.pb0 >= 0 && ahead.pb0 < p.num_blocks;
        const bool ok1 = two && ahead.pb1 >= 0 && ahead.pb1 < p.num_blocks;
        if (lane == 0) {
            if (!ok0 || (two && !ok1)) flag_error(p.err, PKV_DEVERR_OOB_BLOCK);
            poison[st] = (ok0 ? 0 : 1) | (ok1 ? 0 : 2);
        }
        Math::issue(smem + size_t(st) * Math::STAGE, side + st * Math::kSide, &k_map, &v_map, p, ahead.kvh, ahead.pb0, ok0,
                    ahead.pb1, ok1, &full[st], lane);
        ahead.advance(p, &ws.ahead, warp, lane);
    };
    ahead.walk(p, &ws.ahead, warp, lane);   // the first table entries: an input, read before the wait
    grid_dep_wait();
#ifdef PKV_TIMELINE
    if (tid == 0) PKV_TL(2);
#endif
    // One stage first: the copies of a launch's first stages all come at the end of their burst, so a warp with
    // two of them in it would start twice as late.  The others follow when the first is there.
    fill(warp);
    bool primed = false;

    // Partition (split) or cascade slot of row m of segment g, or the output row's first element.
    auto slot_of = [&](const Seg& g, int qrow, int hg) {
        const int slot_p = g.part + ((VAR == kCascade && g.s < p.num_items) ? p.part_offset : 0);
        return (size_t(qrow) * H + hg) * p.max_partitions + slot_p;
    };
    const bool to_parts = VAR == kCascade || p.mode == kModeSplit;

    constexpr int kPer = (MR * D / 4 + CT - 1) / CT;   // float4 sums a thread takes in a merge, at most
    const int n4 = (M * D) >> 2;
    // Final rows of segment g from merged sums: float4 i4 of the pair's M x D.
    auto store_final = [&](const Seg& g, int i4, float4 r, float Mx, float L) {
        const int m = (i4 << 2) / D, d = (i4 << 2) % D;
        const int h = m / QL, qrow = query_row<VAR>(p, g.s, m - h * QL), hg = g.kvh * G + h;
        if (VAR == kCascade && qrow < 0) return;   // a cascade item's padding column
        // a row whose sum is not positive (no visible token, or a NaN scale) is written as zeros
        const bool live = L > 0.f;
        const float inv = live ? 1.f / L : 0.f;
        const float4 x = live ? make_float4(r.x * inv, r.y * inv, r.z * inv, r.w * inv) : make_float4(0.f, 0.f, 0.f, 0.f);
        if (to_parts) {
            const size_t pi = slot_of(g, qrow, hg);
            reinterpret_cast<float4*>(p.tmp_out + pi * D)[d >> 2] = x;
            if (d == 0) {
                p.max_logits[pi] = live ? Mx * kLn2 : -INFINITY;
                p.exp_sums[pi] = L;
            }
        } else {
            store_out4(p.out, p.out_dtype, (size_t(qrow) * H + hg) * D + d, x);
        }
    };
    // Partial i of the CTA: 2 w + 1, the last segment of warp w's share, in its first stage, whose copies are
    // done by then; 2 w, the first, in its own slot or with the pair's piece (kHeadInPiece).  Single pass: 2 w for
    // every pair, in its own slot.  Element (m, d) at ob_idx(m, d).
    const bool in_slots = own_slots<Math>(p.mode);
    auto partial = [&](int i, int seq) -> float* {
        if (i & 1) return reinterpret_cast<float*>(smem + size_t(i >> 1) * Math::STAGE);
        if (in_slots) return ob + size_t(i >> 1) * M * D;
        return p.part_o + (size_t((lane_idx + seq) * Hkv + lane_kvh) * kMaxRows + 8) * D;
    };
    // The partials of `mask` (bit i: partial i), weighed and summed in their order, for float4 i4 of the pair; eight
    // at a time in flight.
    auto merge = [&](uint32_t mask, int seq, int i4, float4& r, float& Mx, float& L) {
        const int m = (i4 << 2) / D, at = ob_idx(m, (i4 << 2) % D, D);
        r = make_float4(0.f, 0.f, 0.f, 0.f);
        Mx = -INFINITY;
        L = 0.f;
        const int i0 = (__ffs(mask) - 1) & ~7, i1 = 32 - __clz(mask);
        for (int b = i0; b < i1; b += 8) {
            float mi[8], li[8];
            float4 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const bool in = (mask >> (b + k)) & 1u;
                mi[k] = in ? mw[(b + k) * MR + m] : -INFINITY;
                li[k] = in ? lw[(b + k) * MR + m] : 0.f;
                v[k] = in ? *reinterpret_cast<const float4*>(partial(b + k, seq) + at) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float Mn = Mx;
#pragma unroll
            for (int k = 0; k < 8; ++k) Mn = fmaxf(Mn, mi[k]);
            const float a = (Mx == -INFINITY) ? 0.f : exp2f(Mx - Mn);
            r.x *= a; r.y *= a; r.z *= a; r.w *= a;
            L *= a;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float f = (mi[k] == -INFINITY) ? 0.f : exp2f(mi[k] - Mn);
                L = fmaf(li[k], f, L);
                r.x = fmaf(v[k].x, f, r.x);
                r.y = fmaf(v[k].y, f, r.y);
                r.z = fmaf(v[k].z, f, r.z);
                r.w = fmaf(v[k].w, f, r.w);
            }
            Mx = Mn;
        }
    };

    Math mth;
    mth.scale_log2_ = p.scale_log2;
    int st = warp;       // this warp's next stage, and its phase
    uint32_t phase = 0;
    bool lost = false;   // a copy did not come: no later one is read, no stage filled
    while (true) {
        Seg sg;
        bool more, on;   // on: the share goes on behind this segment
        {
            SegIter<VAR> it = ws.it;
            more = next_share<NCW>(p, it, sg, warp);
            on = it.u < it.u1;
            __syncwarp();
            if (lane == 0) ws.it = it;
            __syncwarp();
        }
        if (!more) break;
        mth.template begin<VAR>(p, sg.s, sg.kvh, sg.ctx, lane);
        for (int u = sg.b0; u < sg.b1; u += kStepUnits) {
            const bool ok = !lost && __all_sync(0xffffffffu, mbar_wait(&full[st], phase));
#ifdef PKV_TIMELINE
            if (tl_first && tid == 0) PKV_TL(3);
            tl_first = false;
#endif
            if (!primed) {
                for (int more_st = warp + NCW; more_st < S; more_st += NCW) fill(more_st);
                primed = true;
            }
            if (ok) {
                const int ba = unit_block<VAR>(sg, u), bb = unit_block<VAR>(sg, u + 1);
                const int bad = poison[st];
                const int na = (bad & 1) ? 0 : min(kBS, sg.ctx - ba * kBS);
                const int nb = (bad & 2) ? 0 : min(kBS, sg.ctx - bb * kBS);
                if (na + nb > 0)
                    mth.template step<VAR>(smem + size_t(st) * Math::STAGE, side + st * Math::kSide, ba * kBS, na, bb * kBS,
                                           nb, lane);
                __syncwarp();
                fill(st);
            } else {
                lost = true;
                if (lane == 0) flag_error(p.err, PKV_DEVERR_TIMEOUT);
                break;   // st stays at the copy that did not come
            }
            st += NCW;
            if (st >= S) {
                st -= S;
                phase ^= 1u;
            }
        }
        mth.finish(lane);
        if (p.mode == kModeSplit || (p.mode == kModeBalanced && sg.whole)) {
            // all of the pair (or partition) is here: straight from registers
            mth.each(M, lane, [&](int q, int d, float x, float y, float Mx, float L) {
                const int h = q / QL, qrow = query_row<VAR>(p, sg.s, q - h * QL), hg = sg.kvh * G + h;
                if (VAR == kCascade && qrow < 0) return;
                const bool live = L > 0.f;
                const float inv = live ? 1.f / L : 0.f;
                x = live ? x * inv : 0.f;
                y = live ? y * inv : 0.f;
                if (to_parts) {
                    const size_t pi = slot_of(sg, qrow, hg);
                    reinterpret_cast<float2*>(p.tmp_out + pi * D)[d >> 1] = make_float2(x, y);
                    if (d == 0) {
                        p.max_logits[pi] = live ? Mx * kLn2 : -INFINITY;
                        p.exp_sums[pi] = L;
                    }
                } else {
                    store_out2(p.out, p.out_dtype, (size_t(qrow) * H + hg) * D + d, x, y);
                }
            });
            continue;
        }
        // ---- a part of the pair: left for the merge
        const int i = 2 * warp + ((single || on) ? 0 : 1);
        float* dst = partial(i, sg.s);
        const bool hold = lost && (i & 1);   // a copy may still be under way into that stage (see below)
        mth.each(M, lane, [&](int q, int d, float x, float y, float Mx, float L) {
            if (!hold) *reinterpret_cast<float2*>(dst + ob_idx(q, d, D)) = make_float2(x, y);
            if (d == 0) {
                mw[i * MR + q] = hold ? -INFINITY : Mx;
                lw[i * MR + q] = hold ? 0.f : L;
            }
        });
        if (lane == 0) {
            have[i] = 1;
            ws.part[i & 1] = sg;
        }
        if (single) {
            // every warp of the CTA has its share of this pair
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const int i4 = tid + k * CT;
                float4 r;
                float Mx, L;
                if (i4 < n4) {
                    merge(0x55555555u & ((1u << (2 * NCW)) - 1u), sg.s, i4, r, Mx, L);
                    store_final(sg, i4, r, Mx, L);
                }
            }
            __syncthreads();   // the slots are free again
        }
    }
    if (lost) {
        // The stages that were filled when a copy did not come, a ring of them from that one on, are waited for once more
        // (one that was not filled runs into the limit), so that no copy is under way when the CTA ends.  The partial that
        // was not written there counts for nothing.
        for (int n = S / NCW; n > 0; --n) {
            mbar_wait(&full[st], phase);
            st += NCW;
            if (st >= S) {
                st -= S;
                phase ^= 1u;
            }
        }
        __syncwarp();
        for (int i4 = lane; i4 < n4; i4 += 32)
            reinterpret_cast<float4*>(smem + size_t(warp) * Math::STAGE)[i4] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    // context longer than its table: flagged once per sequence
    for (int s = blockIdx.x * CT + tid; s < p.num_seqs; s += gridDim.x * CT)
        if (p.context_lens[s] > p.max_blocks * kBS) flag_error(p.err, PKV_DEVERR_CAPACITY);
    // balanced mode: sequences with nothing visible still get their zero rows
    // (cascade: an empty partial in the sequence's own slot)
    if (p.mode == kModeBalanced) {
        if constexpr (VAR == kCascade) {
            for (int s = p.num_items + blockIdx.x; s < p.num_seqs; s += gridDim.x)
                if (seq_units<VAR>(p, s, seq_ctx(p, s)) == 0)
                    for (int h = tid; h < H; h += CT) {
                        const size_t pi = (size_t(query_row<VAR>(p, s, 0)) * H + h) * p.max_partitions;
                        p.max_logits[pi] = -INFINITY;
                        p.exp_sums[pi] = 0.f;
                    }
        } else {
            for (int s = blockIdx.x; s < p.num_seqs; s += gridDim.x)
                if (VAR == kScored ? seq_units<VAR>(p, s, seq_ctx(p, s)) == 0 : seq_ctx(p, s) == 0)
                    for (int i = tid; i < QL * H * D; i += CT)
                        store_out(p.out, p.out_dtype, size_t(s) * QL * H * D + i, 0.f);
        }
    }
    if (p.mode != kModeBalanced) return;

    // ---- all shares are through: merge the pairs that were cut between the warps.  A run of partials of one
    // sequence is one pair; the first and the last may go on in other CTAs.
#ifdef PKV_TIMELINE
    if (tid == 0) PKV_TL(4);
#endif
    __syncthreads();
#ifdef PKV_TIMELINE
    if (tid == 0) PKV_TL(5);
#endif
    const long long chunk = pl.chunk;
    // every warp finds the runs for itself: lane i holds partial i's sequence
    const int my_seq = lane < 2 * NCW && have[lane] ? state[lane >> 1].part[lane & 1].s : -1;
    const uint32_t present = __ballot_sync(0xffffffffu, my_seq >= 0);
    const uint32_t below = present & ((1u << lane) - 1u);
    const int prev_seq = __shfl_sync(0xffffffffu, my_seq, below ? 31 - __clz(below) : lane);
    const uint32_t starts = __ballot_sync(0xffffffffu, my_seq >= 0 && (!below || prev_seq != my_seq));
    // the work: float4s of every run's pair, 32 to a warp at a time
    int njobs = 0, nrun = 0;
    const int per_run = (n4 + 31) / 32;
    for (uint32_t left = starts; left; left &= left - 1, ++nrun) {
        const int i0 = __ffs(left) - 1;
        const uint32_t later = left & (left - 1);
        const uint32_t mask = present & ~((1u << i0) - 1u) & (later ? (1u << (__ffs(later) - 1)) - 1u : 0xffffffffu);
        const Seg& g = state[i0 >> 1].part[i0 & 1];
        // the first and the last pair may have pieces in other CTAs
        const bool whole = g.pair_start >= pl.u0 && g.pair_start + g.nu <= pl.u1;
        for (int c = 0; c < per_run; ++c) {
            const int i4 = 32 * c + lane;
            if ((nrun * per_run + c) % NCW != warp || i4 >= n4) continue;
            float4 r;
            float Mx, L;
            merge(mask, g.s, i4, r, Mx, L);
            if (whole) {
                store_final(g, i4, r, Mx, L);
            } else {
                // piece slot: unique because (lane_idx + s) grows along a lane's pieces
                const size_t slot = size_t((lane_idx + g.s) * Hkv + g.kvh) * kMaxRows;
                reinterpret_cast<float4*>(p.part_o + slot * D)[i4] = r;
                const int m = (i4 << 2) / D;
                if ((i4 << 2) % D == 0) reinterpret_cast<float2*>(p.part_ml)[slot + m] = make_float2(Mx, L);
            }
        }
        if (!whole && tid == 0) {
            // what the pieces' combine needs of the pair
            Job& jb = jobs[njobs];
            jb.s = g.s;
            const long long c0 = g.pair_start + g.cost_base - p.seg_cost, c1 = c0 + g.nu - 1;
            if (c1 < INT_MAX && chunk < INT_MAX) {   // nearly always: a 64-bit division takes several times as long
                jb.c_lo = int(c0) / int(chunk);
                jb.np = int(c1) / int(chunk) - jb.c_lo + 1;
            } else {
                jb.c_lo = int(c0 / chunk);
                jb.np = int(c1 / chunk) - jb.c_lo + 1;
            }
        }
        njobs += !whole;
    }
#ifdef PKV_TIMELINE
    if (tid == 0) PKV_TL(6);
    if (tid == 0 && njobs == 0) PKV_TL(7);
#endif
    if (njobs == 0) return;
    // ---- publish the pieces; whoever finishes a pair's last one combines them (no waiting): the barrier, then
    // the count with release semantics at gpu scope
    __syncthreads();
    if (tid < njobs) {
        const int pair = jobs[tid].s * Hkv + lane_kvh;
        const bool last = atomic_add_acq_rel_gpu(&p.counters[pair], 1) == jobs[tid].np - 1;
        if (!last) jobs[tid].np = 0;
    }
    __syncthreads();
    // Pieces hold unnormalised sums relative to their own max m_c: O = sum_c 2^(m_c - M) O_c,
    // L = sum_c 2^(m_c - M) l_c; eight at a time in flight, folded in by an online rescale in piece order (the
    // same bits whoever combines).
    for (int x = tid; x < njobs * n4; x += CT) {
        const Job& jb = jobs[x >= n4];
        const int i4 = x >= n4 ? x - n4 : x, np = jb.np, m = (i4 << 2) / D;
        if (np == 0) continue;
        constexpr int kFly = 8;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float Mr = -INFINITY, Lr = 0.f;
        for (int c0 = 0; c0 < np; c0 += kFly) {
            float2 ml[kFly];
            float4 v[kFly];
#pragma unroll
            for (int w = 0; w < kFly; ++w) {
                ml[w] = make_float2(-INFINITY, 0.f);
                v[w] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (c0 + w < np) {
                    const size_t sl = size_t((jb.c_lo + c0 + w + jb.s) * Hkv + lane_kvh) * kMaxRows;
                    ml[w] = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + sl + m);
                    v[w] = __ldcg(reinterpret_cast<const float4*>(p.part_o + sl * D) + i4);
                }
            }
            float Mn = Mr;
#pragma unroll
            for (int w = 0; w < kFly; ++w)
                if (ml[w].y > 0.f) Mn = fmaxf(Mn, ml[w].x);
            const float a = (Mr == -INFINITY) ? 0.f : exp2f(Mr - Mn);
            acc.x *= a; acc.y *= a; acc.z *= a; acc.w *= a;
            Lr *= a;
#pragma unroll
            for (int w = 0; w < kFly; ++w) {
                const float f = (ml[w].y > 0.f) ? exp2f(ml[w].x - Mn) : 0.f;
                acc.x = fmaf(f, v[w].x, acc.x);
                acc.y = fmaf(f, v[w].y, acc.y);
                acc.z = fmaf(f, v[w].z, acc.z);
                acc.w = fmaf(f, v[w].w, acc.w);
                Lr = fmaf(f, ml[w].y, Lr);
            }
            Mr = Mn;
        }
        Seg g;
        g.s = jb.s;
        g.kvh = lane_kvh;
        g.part = 0;
        store_final(g, i4, acc, Mr, Lr);
    }
    if (tid < njobs && jobs[tid].np > 0) p.counters[jobs[tid].s * Hkv + lane_kvh] = 0;   // ready for the next launch
#ifdef PKV_TIMELINE
    if (tid == 0) PKV_TL(7);
#endif
}

template <class Math, int VAR>
int byte_smem_bytes(int stages, int M, int mode) {
    constexpr int NCW = Math::NCW;
    return stages * (Math::STAGE + Math::kSide + 8 + 4) + (own_slots<Math>(mode) ? NCW * M * Math::kD * 4 : 0) + 4 * NCW * Math::kRows * 4 +
           kRedSlots * 8 + NCW * int(sizeof(WarpState<VAR>)) + 16 + 2 * NCW * 4 +
           2 * int(sizeof(Job)) + 1024;
}

template <class Math, int VAR>
cudaError_t launch_byte(AttnParams p, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t stream) {
    int num_sms = 0;
    const cudaError_t e = prepare_device<byte_attention_kernel<Math, VAR>>(&num_sms);
    if (e != cudaSuccess) return e;
    const int M = (p.num_heads / p.num_kv_heads) * p.q_len;
    const int per_stage = byte_smem_bytes<Math, VAR>(1, M, p.mode) - byte_smem_bytes<Math, VAR>(0, M, p.mode);
    int stages = (kSmemLimit - byte_smem_bytes<Math, VAR>(0, M, p.mode)) / per_stage;
    if (stages > 6 * Math::NCW) stages = 6 * Math::NCW;
    stages = stages / Math::NCW * Math::NCW;   // every stage always belongs to the same warp
    if (stages < Math::NCW) return cudaErrorInvalidConfiguration;
    p.stages = stages;
    if (p.mode == kModeBalanced) {
        p.seg_cost = Math::kSegCost;
        p.min_chunk = kStepUnits * Math::NCW;   // one step for every warp: more CTAs would only add pieces
    }
    const int cap = num_sms < kMaxGrid ? num_sms : kMaxGrid;
    int grid;
    if (p.mode == kModeSingle) {
        const long long pairs = (long long)p.num_seqs * p.num_kv_heads;
        grid = pairs < cap ? int(pairs < 1 ? 1 : pairs) : cap;
    } else {
        // Hkv lanes of L CTAs each (at least one lane)
        int L = cap / p.num_kv_heads;
        if (L < 1) L = 1;
        const long long lane_units = (long long)p.num_seqs * p.max_blocks;   // upper bound of a lane's list
        if (lane_units < L) L = int(lane_units < 1 ? 1 : lane_units);
        grid = L * p.num_kv_heads;
    }
    return launch_kernel(byte_attention_kernel<Math, VAR>, dim3(grid), dim3(Math::NCW * 32),
                         size_t(byte_smem_bytes<Math, VAR>(stages, M, p.mode)), stream, km, vm, p);
}

template <bool E4M3, int VAR>
cudaError_t dispatch_byte(const AttnParams& p, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t st) {
    const bool narrow = (p.num_heads / p.num_kv_heads) * p.q_len <= 8;
    if (p.head_dim == 128)
        return narrow ? launch_byte<TeMath<E4M3, 128, 1>, VAR>(p, km, vm, st)
                      : launch_byte<TeMath<E4M3, 128, 2>, VAR>(p, km, vm, st);
    return narrow ? launch_byte<TeMath<E4M3, 64, 1>, VAR>(p, km, vm, st)
                  : launch_byte<TeMath<E4M3, 64, 2>, VAR>(p, km, vm, st);
}

}  // namespace

}  // namespace pkv
