// attention_selected.cuh -- attention of each (query token, kv head) over its own
// list of pages (16-token blocks), as a selection gives them: what the kernels for
// single tokens (attention_selected.cu) and for several neighbouring tokens of a
// sequence (attention_selected_rows.cu) have in common.
//
//   out[r, h] = sum_t softmax_t(scale q[r,h] . K[t]) V[t]  over the listed pages' visible tokens
//
// No two kv heads read the same pages, so the balanced plan over whole sequences
// (attention_impl.cuh) has nothing to cut: a cluster of 1 to 8 CTAs takes a kv head and
// one query token, or a few, its warps two pages each at a time, and they merge by the
// log-sum-exp identity, in shared memory and then across the cluster.
//
// A warp streams its pages by itself: it fills its own ring of stages by TMA, one tile of K and
// one of V a page, each with a barrier of its own, and nobody else waits for it.  8-bit codes and
// K8/V4 are widened to fp16 in registers.  P is split in two 16-bit halves (two MMAs), as one
// would round each weight by as much as the output's own rounding.
#pragma once

#include <cooperative_groups.h>

#include "attention_byte.cuh"
#include "pkv_rows.cuh"

namespace cg = cooperative_groups;

namespace pkv {

namespace {

constexpr int kSelWarps = 4, kSelThreads = kSelWarps * 32;
constexpr int kSelCluster = 8;   // CTAs of a cluster at most
constexpr int kSelTokens = 8;    // query tokens of a CTA at most: a bit each in a page's byte

// TMA loads that leave their lines in L2 as any load does: other CTAs read the same pages.
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int32_t x, int32_t y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}

// A page of one kv head in a stage: its K tile, its V tile, and beside the ring its scales.
template <int KIND, int D>
struct PageMath {
    static constexpr bool kHalf = KIND == PKV_CACHE_F16 || KIND == PKV_CACHE_BF16;
    static constexpr bool kByte = KIND == PKV_CACHE_I8 || KIND == PKV_CACHE_E4M3;
    static constexpr bool kBf = KIND == PKV_CACHE_BF16;      // the MMAs' 16-bit type
    static constexpr int KE = kHalf ? 2 : 1;                 // bytes of a K element
    static constexpr int VROW = KIND == PKV_CACHE_K8V4 ? D / 2 : D * KE;   // bytes of a V row
    static constexpr int KT = kBS * D * KE, VT = kBS * VROW;
    static constexpr int OFF_V = align_up(KT, 1024), STAGE = align_up(OFF_V + VT, 1024);
    static constexpr int STAGES = kHalf ? 2 : 4;             // of a warp: one or two steps
    static constexpr int NG = D / 32;                        // K8V4: groups of a row
    static constexpr int SIDE = kByte ? 16 : kHalf ? 0 : 32 + 64 * NG;   // {K, V scale}; K8V4: K scales, V scales, V zeros
    static constexpr int NKS = D / 16;                       // k steps of S
    static constexpr int NMT = D / 16;                       // M tiles of O^T
    // The running maximum that weights are relative to grows only when a score is above it by more than kSlack (base 2), so
    // that the sums are seldom rescaled.  Weights of up to 2^kSlack fit the operand; in fp16 they keep their bits down to 2^-38.
    static constexpr float kSlack = kBf ? 8.f : 1.f, kPUnit = kBf ? 1.f : 16384.f;

    // K, or V, of page pb and its scales into a stage, by the whole warp.  SHARED: other CTAs read the same pages.
    template <bool V, bool SHARED>
    static __device__ __forceinline__ void issue(uint8_t* dst, uint8_t* side, const CUtensorMap* map, const SelectedParams& p, int kvh,
                                                 int pb, uint64_t* bar, int lane) {
        const int64_t meta = int64_t(pb) * p.num_kv_heads + kvh;
        if constexpr (kByte) {
            if (lane == 0) {
                cp_async_4(side + (V ? 4 : 0), static_cast<const float*>(V ? p.v_scale : p.k_scale) + meta);
                cp_async_mbar_arrive(bar);
            }
        } else if constexpr (!kHalf) {
            if (lane < (V ? 4 * NG : 2)) {   // 16 bytes a lane: 32 of K scales; 32 NG of V scales, 32 NG of zeros
                const uint8_t* src = !V ? static_cast<const uint8_t*>(p.k_scale) + meta * 32
                                   : lane < 2 * NG ? static_cast<const uint8_t*>(p.v_scale) + meta * 32 * NG
                                                   : static_cast<const uint8_t*>(p.v_zero) + meta * 32 * NG - 32 * NG;
                cp_async_16(side + (V ? 32 : 0) + 16 * lane, src + 16 * lane);
                cp_async_mbar_arrive(bar);
            }
        }
        __syncwarp();   // the phase waits for those copies before lane 0's arrival can end it
        if (lane == 0) {
            uint8_t* to = dst + (V ? OFF_V : 0);
            mbar_arrive_expect_tx(bar, V ? VT : KT);
            if constexpr (kHalf) {
                if constexpr (SHARED) tma_load_3d(to, map, 0, pb * kBS, kvh * (D / 64), bar);
                else tma_load_3d_hint(to, map, 0, pb * kBS, kvh * (D / 64), bar, l2_evict_first_policy());
            } else {
                if constexpr (SHARED) tma_load_2d(to, map, kvh * (V ? VROW : D), pb * kBS, bar);
                else tma_load_2d_hint(to, map, kvh * (V ? VROW : D), pb * kBS, bar, l2_evict_first_policy());
            }
        }
    }

    // The first of the two dims that k step kk has at lane position t in each operand word: 16-bit caches in order, 8-bit
    // codes four neighbouring bytes of the thread's quarter of the row.
    static __device__ __forceinline__ int q_dim(int kk, int word, int t) {
        return kHalf ? 16 * kk + 8 * word + 2 * t : t * (D / 4) + 4 * kk + 2 * word;
    }

    // four codes -> fp16 pairs (0, 1) and (2, 3), exact
    static __device__ __forceinline__ void widen(uint32_t w, uint32_t& a, uint32_t& b) {
        if constexpr (KIND == PKV_CACHE_E4M3) e4m3x4_to_f16(w, a, b);
        else s8x4_to_f16x4(w, a, b);
    }

    // The K operands of two pages, k step by k step: f(kk, a), a[b] the MMA's A operand (tokens g, g + 8) of page b.
    template <class F>
    static __device__ __forceinline__ void keys(const uint8_t* const (&stage)[2], int lane, F f) {
        if constexpr (kHalf) {
            // 16-byte chunk c = 2 kk + (mi >> 1) of row tk, at chunk c ^ (tk & 7) of the 128 bytes: the lane's part of that
            // exclusive or is worked out once
            const int mi = lane >> 3, tk = (mi & 1) * 8 + (lane & 7);
            const uint32_t lane_at = tk * 128 + 16 * ((tk & 7) ^ (mi >> 1));
            const uint32_t at[2] = {smem_addr(stage[0]) + lane_at, smem_addr(stage[1]) + lane_at};
#pragma unroll
            for (int kk = 0; kk < NKS; ++kk) {
                uint32_t a[2][4];
                ldsm_x4((at[0] ^ (32 * (kk & 3))) + (kk >> 2) * 2048, a[0]);
                ldsm_x4((at[1] ^ (32 * (kk & 3))) + (kk >> 2) * 2048, a[1]);
                f(kk, a);
            }
        } else {
            const int g = lane >> 2, t = lane & 3;
            uint32_t w[2][2][NKS];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int i = 0; i < D / 64; ++i) {
                        const int row = g + 8 * r, c = t * (D / 64) + i;
                        const uint4 v = *reinterpret_cast<const uint4*>(stage[b] + row * D + 16 * swz<D>(c, row));
                        w[b][r][4 * i] = v.x; w[b][r][4 * i + 1] = v.y; w[b][r][4 * i + 2] = v.z; w[b][r][4 * i + 3] = v.w;
                    }
#pragma unroll
            for (int kk = 0; kk < NKS; ++kk) {
                uint32_t a[2][4];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    widen(w[b][0][kk], a[b][0], a[b][2]);
                    widen(w[b][1][kk], a[b][1], a[b][3]);
                }
                f(kk, a);
            }
        }
    }
    // a token's K scale
    static __device__ __forceinline__ float k_scale(const uint8_t* side, int token) {
        if constexpr (kByte) return *reinterpret_cast<const float*>(side);
        else if constexpr (!kHalf) return Half16<__half>::to_float(reinterpret_cast<const uint16_t*>(side)[token]);
        else return 1.f;
    }
    static __device__ __forceinline__ float v_scale(const uint8_t* side) { return reinterpret_cast<const float*>(side)[1]; }

    // The M tile mt of V^T: rows g are dim(mt, g), rows g + 8 kNext further.
    static constexpr int kNext = kHalf ? 8 : 1;
    static __device__ __forceinline__ int dim(int mt, int g) {
        return kHalf ? 16 * mt + g : kByte ? 16 * mt + 2 * g : 32 * (mt >> 1) + 4 * g + 2 * (mt & 1);
    }
    // f(first tile, operands) for each few tiles (the MMAs onto one tile's sums then lie apart).  CUT: without the tokens that
    // m01 (2t, 2t + 1) and m23 (8 further) leave out.
    template <bool CUT, int FEW, class F>
    static __device__ __forceinline__ void tiles(const uint8_t* stage, const uint8_t* side, uint32_t m01, uint32_t m23, int lane, F f) {
        const int mi = lane >> 3, r = lane & 7, t = lane & 3;
        const uint32_t base = smem_addr(stage) + OFF_V;
        if constexpr (kHalf) {
            const int tk = (mi >> 1) * 8 + r;
            const uint32_t at = base + tk * 128 + 16 * ((tk & 7) ^ (mi & 1));   // as in keys()
#pragma unroll
            for (int m0 = 0; m0 < NMT; m0 += FEW) {
                uint32_t a[FEW][4];
#pragma unroll
                for (int j = 0; j < FEW; ++j) {
                    ldsm_x4_t((at ^ (32 * ((m0 + j) & 3))) + ((m0 + j) >> 2) * 2048, a[j]);
                    if constexpr (CUT) {
                        a[j][0] &= m01; a[j][1] &= m01; a[j][2] &= m23; a[j][3] &= m23;
                    }
                }
                f(m0, a);
            }
        } else {
            const int tk = (mi & 1) * 8 + r;
#pragma unroll
            for (int c0 = 0; c0 < VROW / 16; c0 += 2) {
                uint32_t x[4];   // tokens 0-7, 8-15 of chunk c0, then of chunk c0 + 1
                ldsm_x4_t(base + tk * VROW + 16 * swz<VROW>(c0 + (mi >> 1), tk), x);
                if constexpr (CUT) {
                    x[0] &= m01; x[1] &= m23; x[2] &= m01; x[3] &= m23;
                }
                if constexpr (kByte) {
                    // a word is dims 2g, 2g + 1 of two tokens: one dim of both to a row
                    uint32_t a[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        widen(__byte_perm(x[2 * h], 0u, 0x3120), a[h][0], a[h][1]);
                        widen(__byte_perm(x[2 * h + 1], 0u, 0x3120), a[h][2], a[h][3]);
                    }
                    f(c0, a);
                } else {
                    // a word is dims 4g .. 4g + 3 of two tokens; code * scale + zero, rounded once to fp16 (2^-11 of the
                    // value, as an fp16 cache holds it)
                    uint32_t a[4][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint16_t* vs = reinterpret_cast<const uint16_t*>(side + 32) + c0 + h;
                        const uint16_t* vz = vs + kBS * NG;
                        uint32_t sc[2], ze[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int tok = (2 * t + 8 * i) * NG;
                            sc[i] = vs[tok] | uint32_t(vs[tok + NG]) << 16;
                            ze[i] = vz[tok] | uint32_t(vz[tok + NG]) << 16;
                            if constexpr (CUT) {
                                sc[i] &= i ? m23 : m01;
                                ze[i] &= i ? m23 : m01;
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t code = u4pair_to_f16x2(x[2 * h + (i >> 1)], 2 * j + (i & 1));
                                __half2 v, s2, z2;
                                memcpy(&v, &code, 4);
                                memcpy(&s2, &sc[i >> 1], 4);
                                memcpy(&z2, &ze[i >> 1], 4);
                                v = __hfma2(v, s2, z2);
                                memcpy(&a[2 * h + j][i], &v, 4);
                            }
                    }
                    f(2 * c0, a);
                }
            }
        }
    }
};

// The pages of a warp and its ring: entries warp, warp + 4, .. of the CTA's n (all with a block), page k of them in stage
// k % STAGES.
template <class Math, bool SHARED>
struct Ring {
    const SelectedParams& p;
    const CUtensorMap *k_map, *v_map;
    const int2* entry;
    int n, kvh, warp, lane;
    uint8_t *stages, *sides;      // this warp's
    uint64_t *k_full, *v_full;
    int k_ahead, v_ahead;         // the next entries to load
    uint32_t k_phase, v_phase;    // parities of the stages' next copies, a bit each

    __device__ __forceinline__ const uint8_t* stage(int st) const { return stages + st * Math::STAGE; }
    __device__ __forceinline__ const uint8_t* side(int st) const { return sides + st * Math::SIDE; }
    __device__ __forceinline__ void fill_k(int st) {
        if (k_ahead < n)
            Math::template issue<false, SHARED>(stages + st * Math::STAGE, sides + st * Math::SIDE, k_map, p, kvh, entry[k_ahead].y,
                                                k_full + st, lane);
        k_ahead += kSelWarps;
    }
    __device__ __forceinline__ void fill_v(int st) {
        if (v_ahead < n)
            Math::template issue<true, SHARED>(stages + st * Math::STAGE, sides + st * Math::SIDE, v_map, p, kvh, entry[v_ahead].y,
                                               v_full + st, lane);
        v_ahead += kSelWarps;
    }
    __device__ __forceinline__ void begin() {
        k_ahead = v_ahead = warp;
#pragma unroll
        for (int st = 0; st < Math::STAGES; ++st) {
            fill_k(st);
            fill_v(st);
        }
    }
    __device__ __forceinline__ bool wait_k(int st) {
        const bool came = mbar_wait(k_full + st, (k_phase >> st) & 1u);
        k_phase ^= 1u << st;
        return came;
    }
    __device__ __forceinline__ bool wait_v(int st) {
        const bool came = mbar_wait(v_full + st, (v_phase >> st) & 1u);
        v_phase ^= 1u << st;
        return came;
    }
    // A copy did not come: no copy is under way when the CTA ends (a stage that was not filled runs into the limit).
    __device__ __forceinline__ void give_up() {
        flag_error(p.err, PKV_DEVERR_TIMEOUT);
        for (int st = 0; st < Math::STAGES; ++st) {
            wait_k(st);
            wait_v(st);
        }
    }
};

// The cluster's barrier in two halves, by all its threads.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

// What a CTA's warps leave to merge, COLS query columns each: sums o in the warps' rings, [COLS][D + 4] (padded against
// bank conflicts), running maxima (base 2) and sums of weights here.
template <int COLS>
struct Partials {
    float m[kSelWarps][COLS], l[kSelWarps][COLS];
    float weight[kSelCluster][COLS], total[COLS];       // of the merges
    float from_m[kSelCluster][COLS], from_l[kSelCluster][COLS];   // the cluster's CTAs'
};

// Room for the other CTAs' sums of a CTA's share of the outputs (clusters only).
template <int COLS, int D>
constexpr size_t exchange_bytes() {
    return size_t(COLS * D / 4 + kSelCluster) * 16;
}

// A column's weight for one of n partials, by n neighbouring threads (n a power of two): the weighted sum L, the maximum M.
// 0 for a partial without a page alone: an infinity or NaN in another's sums stays, however small its weight.
__device__ __forceinline__ float weigh(int n, float m, float l, float& L, float& M) {
    M = l == 0.f ? -INFINITY : m;   // no page (a page has a token whose weight is 1)
    for (int o = 1; o < n; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float w = l == 0.f ? 0.f : fmaxf(exp2f(m - M), 1.4e-45f);
    L = l == 0.f ? 0.f : w * l;
    for (int o = 1; o < n; o <<= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    return w;
}

// The warps' partials, then the cluster's CTAs', into the outputs of rows r0 .. : column = row * G + head.  The weights of all
// partials first (a lane each), then the sums.  In a cluster each CTA sends every other its sums of that one's share of the
// outputs (`exchange`): one barrier, and nothing is read from another CTA.
template <int COLS, int D>
__device__ __forceinline__ void merge_and_store(const SelectedParams& p, cg::cluster_group& cl, Partials<COLS>& part, float* o,
                                                int warp_stride, float4* exchange, int r0, int cols, int kvh, int G) {
    constexpr int OW = D + 4;
    const int C = int(cl.num_blocks()), rank = int(cl.block_rank());
    const int items = cols * (D / 4), share = (items + C - 1) / C;   // four dims of a column; a CTA's share of them
    __syncthreads();
    if (C > 1) cluster_wait();   // the others have begun
    if (threadIdx.x < kSelWarps * COLS) {
        const int col = threadIdx.x / kSelWarps, k = threadIdx.x % kSelWarps;
        float L, M;
        part.weight[k][col] = weigh(kSelWarps, part.m[k][col], part.l[k][col], L, M);
        if (C == 1) {
            if (k == 0) part.total[col] = L;
        } else {
            for (int r = k; r < C; r += kSelWarps) {
                *cl.map_shared_rank(&part.from_m[rank][col], r) = M;
                *cl.map_shared_rank(&part.from_l[rank][col], r) = L;
            }
        }
    }
    __syncthreads();
    auto store = [&](int item, float4 sum) {
        const int col = item / (D / 4), d = (item % (D / 4)) * 4;
        const float L = part.total[col], inv = L > 0.f ? 1.f / L : (L == L ? 0.f : L);   // no visible token: zeros
        store_out4(p.out, p.out_dtype, (size_t(r0 + col / G) * p.num_heads + size_t(kvh) * G + col % G) * D + d,
                   make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv));
    };
    auto add = [](float4& sum, float w, float4 v) {
        if (w == 0.f) return;   // not 0 times what was never written
        sum.x += w * v.x;
        sum.y += w * v.y;
        sum.z += w * v.z;
        sum.w += w * v.w;
    };
    for (int i = threadIdx.x; i < items; i += kSelThreads) {
        const int col = i / (D / 4), d = (i % (D / 4)) * 4;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kSelWarps; ++k)
            add(sum, part.weight[k][col], *reinterpret_cast<const float4*>(o + k * warp_stride + col * OW + d));
        if (C == 1) {
            store(i, sum);
        } else {
            const int r = i / share;
            cl.map_shared_rank(exchange, r)[rank * share + (i - r * share)] = sum;
        }
    }
    if (C == 1) return;
    cl.sync();   // what was sent has come
    for (int i = threadIdx.x; i < kSelCluster * COLS; i += kSelThreads) {
        const int col = i / kSelCluster, k = i % kSelCluster;
        float L, M;
        part.weight[k][col] = weigh(kSelCluster, k < C ? part.from_m[k][col] : 0.f, k < C ? part.from_l[k][col] : 0.f, L, M);
        if (k == 0) part.total[col] = L;
    }
    __syncthreads();
    for (int j = threadIdx.x; j < share && rank * share + j < items; j += kSelThreads) {
        const int i = rank * share + j;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < C; ++k) add(sum, part.weight[k][i / (D / 4)], exchange[k * share + j]);
        store(i, sum);
    }
}

// What the query tokens of a CTA see and list.
struct SelectedTile {
    const SelectedParams& p;
    RowTile tile;
    int kvh, behind0;   // behind0: rows of the sequence from the tile's first on
    int64_t ctx;
    const int32_t* table;
    __device__ __forceinline__ SelectedTile(const SelectedParams& p_, RowTile t, int h) : p(p_), tile(t), kvh(h) {
        ctx = p.context_lens[t.s];
        behind0 = (p.cu_q ? min(p.cu_q[t.s + 1], p.num_rows) : (t.s + 1) * p.q_len) - t.r0;
        table = p.block_tables + int64_t(t.s) * p.max_blocks;
    }
    __device__ __forceinline__ bool over() const { return ctx > int64_t(p.max_blocks) * kBS; }
    __device__ __forceinline__ int visible(int i) const { return visible_tokens(ctx, p.max_blocks, behind0 - i); }
    __device__ __forceinline__ int pages(int i) const { return (visible(i) + kBS - 1) / kBS; }
    __device__ __forceinline__ const int32_t* list(int i) const {
        return p.lists + ((int64_t(tile.r0) + i) * p.num_kv_heads + kvh) * p.max_pages;
    }
    __device__ __forceinline__ int count(int i) const {
        return min(max(p.counts[(int64_t(tile.r0) + i) * p.num_kv_heads + kvh], 0), p.max_pages);
    }
    __device__ __forceinline__ int block(int page) const {   // -1: out of range
        const int b = table[page];
        if (b >= 0 && b < p.num_blocks) return b;
        flag_error(p.err, PKV_DEVERR_OOB_BLOCK);
        return -1;
    }
    // An entry is taken if it is in range and above every entry taken before it.  By a warp: f(index, in the list, taken, entry).
    template <class F>
    __device__ __forceinline__ void in_order(int row, int lane, F f) const {
        const int32_t* at = list(row);
        const int n = count(row), most_pages = pages(row);
        int top = -1;
        for (int j = 0; j < n; j += 32) {
            const int i = j + lane;
            const int e = i < n ? at[i] : -1;
            const bool in = e >= 0 && e < most_pages;
            int most = in ? e : -1;   // the largest entry in range up to this one, which is the largest taken too
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, most, o);
                if (lane >= o) most = max(most, x);
            }
            int before = __shfl_up_sync(0xffffffffu, most, 1);
            before = max(lane ? before : -1, top);
            f(i, i < n, in && e > before, e);
            top = max(top, __shfl_sync(0xffffffffu, most, 31));
        }
    }
    // Entries without a block leave the CTA's list (n, in shared memory), by a warp; the others keep their order.
    __device__ __forceinline__ int close_up(int2* entry, int n, int lane) const {
        int to = 0;
        for (int j = 0; j < n; j += 32) {
            const int2 e = j + lane < n ? entry[j + lane] : make_int2(0, -1);
            const uint32_t who = __ballot_sync(0xffffffffu, e.y >= 0);
            __syncwarp();
            if (e.y >= 0) entry[to + __popc(who & ((1u << lane) - 1u))] = e;
            to += __popc(who);
            __syncwarp();
        }
        return to;
    }
};

// The query operand into shared memory, for all warps: Q[item], item = (column tile, k step, lane), of column
// 8 * tile + lane / 4 the dims of lane position lane % 4.  8-bit caches take fp16: bf16 queries times the power of two that
// brings their column's largest magnitude to [256, 512); q_most [columns] holds the exponents (cleared before).
// With two column tiles their words lie side by side: Q[2 * (k step * 32 + lane)], the MMA's A operand {tile 0, 1 word 0; 0, 1 word 1}.
template <class Math, int COLS, int D>
struct Queries {
    static constexpr int NKS = D / 16, PER = COLS / 8 * NKS * 32 / kSelThreads;
    uint2 x[PER];
    static __device__ __forceinline__ int col(int k) {
        return 8 * (((threadIdx.x + k * kSelThreads) >> 5) / NKS) + (int(threadIdx.x & 31) >> 2);
    }
    // the loads, which depend on nothing but the rows
    __device__ __forceinline__ void load(const SelectedParams& p, int r0, int cols, int kvh, int G) {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int kk = ((threadIdx.x + k * kSelThreads) >> 5) % NKS, c = col(k), t = threadIdx.x & 3;
            x[k] = make_uint2(0u, 0u);
            if (c >= cols) continue;
            const uint16_t* src = static_cast<const uint16_t*>(p.q) + ((int64_t(r0) + c / G) * p.num_heads + int64_t(kvh) * G + c % G) * D;
            x[k].x = __ldg(reinterpret_cast<const uint32_t*>(src + Math::q_dim(kk, 0, t)));
            x[k].y = __ldg(reinterpret_cast<const uint32_t*>(src + Math::q_dim(kk, 1, t)));
        }
    }
    __device__ __forceinline__ void store(const SelectedParams& p, uint2* Q, uint32_t* q_most) {
        if (!Math::kHalf && p.q_dtype == PKV_BF16) {
#pragma unroll
            for (int k = 0; k < PER; ++k)
                atomicMax(&q_most[col(k)], max(max((x[k].x >> 7) & 0xffu, (x[k].x >> 23) & 0xffu),
                                               max((x[k].y >> 7) & 0xffu, (x[k].y >> 23) & 0xffu)));
            __syncthreads();
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                const float up = __uint_as_float((262u - min(max(q_most[col(k)], 16u), 254u)) << 23);
                const float2 a = Half16<__nv_bfloat16>::unpack2(x[k].x), b = Half16<__nv_bfloat16>::unpack2(x[k].y);
                x[k] = make_uint2(pack2<false>(a.x * up, a.y * up), pack2<false>(b.x * up, b.y * up));
            }
        }
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int item = threadIdx.x + k * kSelThreads;
            if constexpr (COLS == 8) {
                Q[item] = x[k];
            } else {
                const int nt = item / (NKS * 32);
                uint32_t* to = reinterpret_cast<uint32_t*>(Q) + 4 * (item - nt * NKS * 32) + nt;
                to[0] = x[k].x;
                to[2] = x[k].y;
            }
        }
    }
};
// what turns a column's products into base-2 scores
template <class Math>
__device__ __forceinline__ float column_scale(const SelectedParams& p, const uint32_t* q_most, int col) {
    if (Math::kHalf || p.q_dtype != PKV_BF16) return p.scale_log2;
    return p.scale_log2 * __uint_as_float((min(max(q_most[col], 16u), 254u) - 8u) << 23);
}

// 8-bit caches: the sums hold P V / vref times kPUnit, vref a power of two that grows with the V scales of the pages that the
// query lists.  Two pages' scales -> what their weights are multiplied by, and what the sums are.  The operand's two halves keep a
// weight to 2^-39 of vref over its page's scale (as byte_attention_kernel's do): what a query gets of a page whose scale is less than
// 2^-20 of the largest one that it lists loses bits, and of less than 2^-38 is lost.
template <class Math>
__device__ __forceinline__ float v_units(float (&vs)[2], float& vref) {
    float grow = 1.f;
    const float mag = fmaxf(fabsf(vs[0]), fabsf(vs[1]));
    if (mag > vref) {   // the same in every lane with the same query
        const uint32_t up = min((__float_as_uint(mag) + 0x007fffffu) & 0xff800000u, 253u << 23);
        grow = vref * __uint_as_float((254u << 23) - up);
        vref = __uint_as_float(up);
    }
    // (scale / vref) * kPUnit in this order: the quotient is exact and at most 1
    const float inv = __uint_as_float((254u << 23) - __float_as_uint(vref));
    vs[0] = (vs[0] * inv) * Math::kPUnit;
    vs[1] = (vs[1] * inv) * Math::kPUnit;
    return grow;
}

// A row's (or column's) new maximum of scores `most`: what the weights are relative to from here on, and the factor f of
// the sums so far; m_run is replaced.  At most kSlack below the maximum itself; 0 while there is no score.
template <class Math>
__device__ __forceinline__ float reference(float most, float& m_run, float& f) {
    const bool grow = most > m_run + Math::kSlack;   // also the first score (m_run is -inf)
    const float now = grow ? most : m_run, ref = now == -INFINITY ? 0.f : now;
    f = grow && m_run > -INFINITY ? exp2_ftz(m_run - ref) : 1.f;
    m_run = now;
    return ref;
}

// Two weights as the 16-bit pair of the operand, and the pair of what that leaves.
template <class Math>
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
    hi = pack2<Math::kBf>(x, y);
    const float2 back = Half16<typename std::conditional<Math::kBf, __nv_bfloat16, __half>::type>::unpack2(hi);
    lo = pack2<Math::kBf>(x - back.x, y - back.y);
}

// Shared memory of a CTA besides its lists: the rings and their scales.
template <class Math>
constexpr size_t ring_bytes() {
    return 1024 + size_t(kSelWarps) * Math::STAGES * (Math::STAGE + Math::SIDE);
}

// How many query tokens of a sequence a CTA of attention_rows_kernel takes: what fills the MMA's 16 rows.
inline int shared_tokens(const SelectedParams& p) {
    const int64_t each = (int64_t(p.num_rows) + p.num_seqs - 1) / p.num_seqs;   // of a sequence, on average
    const int G = p.num_heads / p.num_kv_heads, rows = 16 / G < kSelTokens ? 16 / G : kSelTokens;
    return rows < each ? rows : int(each);
}

// CTAs of an SM that the registers are shared out for; the rings, 64 KB at 128 16-bit dims, allow three there.  With three the
// kernel for several tokens spills 276 bytes (64 x 4 bf16 tokens over 64 pages of 8 heads: 86.9 us, with two 69.0).
constexpr int sel_ctas(int KIND, int D, bool rows) {
    const bool half = KIND == PKV_CACHE_F16 || KIND == PKV_CACHE_BF16;
    return rows && half && D == 128 ? 2 : D == 64 && !rows ? 4 : 3;
}

// Shared memory with which no SM takes a third CTA (a fourth) of a grid that two (three) to each hold: the GPU hands CTAs out
// unevenly while the kernel before ends.  256 CTAs, 8 heads, without it / with it: 32 tokens of 8192 over 64 e4m3 pages 22.9 / 18.4 us,
// of 16384 over 128 41.0 / 31.9 (int8 41.1 / 35.9, bf16 44.3 / 44.0); drafts, 32 x 3 over 64 e4m3 pages 36.2 / 32.4.
// Fewer CTAs are left alone: the next kernel's start beside them (1 token, 64 CTAs: 5.6 us, 6.0 with one CTA to an SM).
inline size_t spread(int64_t ctas, size_t smem) {
    const int64_t each = (ctas + 151) / 152;
    if (each != 2 && each != 3) return smem;
    const size_t least = 228 * 1024 / (each + 1);
    return smem < least ? least : smem;
}

}  // namespace

}  // namespace pkv
