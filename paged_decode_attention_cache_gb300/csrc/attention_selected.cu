// attention_selected.cu -- attention of each (query token, kv head) over its own
// list of pages (16-token blocks), as a selection gives them.
//
//   out[r, h] = sum_t softmax_t(scale q[r,h] . K[t]) V[t]  over the listed pages' visible tokens
//
// No two kv heads read the same pages, so the balanced plan over whole sequences
// (attention_impl.cuh) has nothing to cut: a cluster of 1 to 8 CTAs takes one
// (query token, kv head), its warps one page each at a time, and they merge by the
// log-sum-exp identity, in shared memory and then across the cluster.  Neighbouring
// query tokens of a sequence (drafts, a chunk of a prompt) have much of their lists in
// common: a CTA takes up to 16 / g of them, reads the union of their lists once, and
// masks by token.
//
// A page of one kv head is 16 rows of 128 to 256 bytes, found through the table: a warp loads
// it straight into registers in the layout that the MMAs want, with no stage in
// shared memory and no barrier:
//   S^T = K Q^T   (tokens on M, the group's query heads on N): a thread takes 16
//                 contiguous bytes of its token's row, and the query operand holds
//                 the same dims in the same places (the order of a contraction's
//                 terms is free);
//   O^T = V^T P^T (dims on M): a thread takes the same dims of tokens 2t, 2t + 1,
//                 2t + 8, 2t + 9 and pairs the tokens with byte permutes; rows g and
//                 g + 8 of an M tile are two neighbouring dims of its chunk.
// The next page's K is in flight while this one's weights are worked out, V while the
// scores are.  Two MMAs per V tile: P is split in two 16-bit halves, as one would
// round each weight by as much as the output's own rounding.
#include <cooperative_groups.h>

#include "attention_byte.cuh"
#include "pkv_rows.cuh"

namespace cg = cooperative_groups;

namespace pkv {

namespace {

constexpr int kSelWarps = 4, kSelThreads = kSelWarps * 32;
constexpr int kSelCluster = 8;   // CTAs of a cluster at most
constexpr int kSelTokens = 8;    // query tokens of a CTA at most: a bit each in a page's byte

// A page's K and V rows of one kv head, as a warp holds and uses them.
template <int KIND, int D>
struct PageMath {
    static constexpr bool kHalf = KIND == PKV_CACHE_F16 || KIND == PKV_CACHE_BF16;
    static constexpr bool kByte = KIND == PKV_CACHE_I8 || KIND == PKV_CACHE_E4M3;
    static constexpr bool kBf = KIND == PKV_CACHE_BF16;      // the MMAs' 16-bit type
    static constexpr int KE = kHalf ? 2 : 1;                 // bytes of a K element
    static constexpr int VROW = KIND == PKV_CACHE_K8V4 ? D / 2 : D * KE;   // bytes of a V row
    static constexpr int NKC = D * KE / 64;                  // 16-byte chunks of a K row that a thread takes
    static constexpr int NKS = D / 16;                       // k steps of S
    static constexpr int NVB = VROW / 8;                     // bytes of a V row that a thread takes
    static constexpr int NVW = NVB / 4;
    static constexpr int NMT = D / 16;                       // M tiles of O^T
    static constexpr float kPUnit = kBf ? 1.f : 16384.f;     // fp16 weights keep their bits down to 2^-38

    uint32_t k[2][NKC * 4];   // tokens g, g + 8
    uint32_t v[4][NVW];       // tokens 2t, 2t + 1, 2t + 8, 2t + 9
    float ks[2], vs;          // scales: K of the two tokens (8-bit caches: of the block), V of the block
    uint32_t vsc[2], vze[2];  // K8V4: fp16 pairs of tokens (2t, 2t + 1), (2t + 8, 2t + 9)

    static __device__ __forceinline__ uint4 ld16(const void* p) { return __ldg(static_cast<const uint4*>(p)); }

    __device__ __forceinline__ void load_k(const SelectedParams& p, int64_t pb, int kvh, int live, int g, int t) {
        const int64_t row = int64_t(p.num_kv_heads) * D * KE;
        const uint8_t* base = static_cast<const uint8_t*>(p.k) + pb * kBS * row + int64_t(kvh) * D * KE + 16 * t;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int tok = g + 8 * r;
#pragma unroll
            for (int c = 0; c < NKC; ++c) {
                const uint4 x = tok < live ? ld16(base + tok * row + 64 * c) : make_uint4(0u, 0u, 0u, 0u);
                k[r][4 * c] = x.x; k[r][4 * c + 1] = x.y; k[r][4 * c + 2] = x.z; k[r][4 * c + 3] = x.w;
            }
            if constexpr (KIND == PKV_CACHE_K8V4)
                ks[r] = tok < live ? Half16<__half>::to_float(__ldg(static_cast<const uint16_t*>(p.k_scale) +
                                                                    (pb * p.num_kv_heads + kvh) * kBS + tok))
                                   : 0.f;
        }
        if constexpr (kByte) ks[0] = ks[1] = __ldg(static_cast<const float*>(p.k_scale) + pb * p.num_kv_heads + kvh);
    }

    __device__ __forceinline__ void load_v(const SelectedParams& p, int64_t pb, int kvh, int live, int g, int t) {
        const int64_t row = int64_t(p.num_kv_heads) * VROW;
        const uint8_t* base = static_cast<const uint8_t*>(p.v) + pb * kBS * row + int64_t(kvh) * VROW;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int tok = 2 * t + (i & 1) + 8 * (i >> 1);
            const uint8_t* at = base + tok * row;
            const bool on = tok < live;
            if constexpr (NVB == 32) {   // two chunks of 16 bytes, half a row apart: full sectors in each load
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint4 x = on ? ld16(at + 128 * c + 16 * g) : make_uint4(0u, 0u, 0u, 0u);
                    v[i][4 * c] = x.x; v[i][4 * c + 1] = x.y; v[i][4 * c + 2] = x.z; v[i][4 * c + 3] = x.w;
                }
            } else if constexpr (NVB == 16) {
                const uint4 x = on ? ld16(at + 16 * g) : make_uint4(0u, 0u, 0u, 0u);
                v[i][0] = x.x; v[i][1] = x.y; v[i][2] = x.z; v[i][3] = x.w;
            } else if constexpr (NVB == 8) {
                const uint2 x = on ? __ldg(reinterpret_cast<const uint2*>(at + 8 * g)) : make_uint2(0u, 0u);
                v[i][0] = x.x; v[i][1] = x.y;
            } else {
                v[i][0] = on ? __ldg(reinterpret_cast<const uint32_t*>(at + 4 * g)) : 0u;
            }
        }
        if constexpr (kByte) vs = __ldg(static_cast<const float*>(p.v_scale) + pb * p.num_kv_heads + kvh);
        if constexpr (KIND == PKV_CACHE_K8V4) {
            constexpr int NG = D / 32;
            const int64_t m0 = (pb * p.num_kv_heads + kvh) * kBS * NG + g * (D / 8) / 32;
            const uint16_t *sc = static_cast<const uint16_t*>(p.v_scale), *ze = static_cast<const uint16_t*>(p.v_zero);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int tok = 2 * t + 8 * i;
                const int64_t m = m0 + tok * NG;
                const uint32_t s0 = tok < live ? __ldg(sc + m) : 0u, s1 = tok + 1 < live ? __ldg(sc + m + NG) : 0u;
                const uint32_t z0 = tok < live ? __ldg(ze + m) : 0u, z1 = tok + 1 < live ? __ldg(ze + m + NG) : 0u;
                vsc[i] = s0 | s1 << 16;
                vze[i] = z0 | z1 << 16;
            }
        }
    }

    // four codes -> fp16 pairs (0, 1) and (2, 3), exact
    static __device__ __forceinline__ void widen(uint32_t w, uint32_t& a, uint32_t& b) {
        if constexpr (KIND == PKV_CACHE_E4M3) e4m3x4_to_f16(w, a, b);
        else s8x4_to_f16x4(w, a, b);
    }

    // s = K Q^T: tokens g, g + 8 x query columns 8 nt + 2t, + 1
    template <int NT>
    __device__ __forceinline__ void scores(const uint32_t (&q)[NT][NKS][2], float (&s)[NT][4]) const {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
        for (int kk = 0; kk < NKS; ++kk) {
            uint32_t a[4];
            if constexpr (kHalf) {
                a[0] = k[0][2 * kk]; a[1] = k[1][2 * kk]; a[2] = k[0][2 * kk + 1]; a[3] = k[1][2 * kk + 1];
            } else {
                widen(k[0][kk], a[0], a[2]);
                widen(k[1][kk], a[1], a[3]);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816<kBf>(s[nt], a, q[nt][kk][0], q[nt][kk][1]);
        }
    }

    // the M tile mt of V^T: rows g and g + 8 are dims dim(mt, g) and one above
    static __device__ __forceinline__ int dim(int mt, int g) {
        return NVB == 32 ? (mt >> 2) * 64 + 8 * g + 2 * (mt & 3) : (D / 8) * g + 2 * mt;
    }
    // V as if the page had only its first `live` tokens
    __device__ __forceinline__ void cut_v(int live, int t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t keep = 2 * t + (i & 1) + 8 * (i >> 1) < live ? 0xffffffffu : 0u;
#pragma unroll
            for (int j = 0; j < NVW; ++j) v[i][j] &= keep;
            if constexpr (KIND == PKV_CACHE_K8V4) {
                const uint32_t half = keep | (i & 1 ? 0x0000ffffu : 0xffff0000u);
                vsc[i >> 1] &= half;
                vze[i >> 1] &= half;
            }
        }
    }
    // tiles 2 i and 2 i + 1, from the words that hold their four dims
    __device__ __forceinline__ void tiles(int i, uint32_t (&a)[2][4]) const {
#pragma unroll
        for (int half = 0; half < 2; ++half) {   // tokens 2t, 2t + 1; then 8 further
            const uint32_t *x = v[2 * half], *y = v[2 * half + 1];
            if constexpr (kHalf) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    a[j][2 * half] = __byte_perm(x[2 * i + j], y[2 * i + j], 0x5410);
                    a[j][2 * half + 1] = __byte_perm(x[2 * i + j], y[2 * i + j], 0x7632);
                }
            } else if constexpr (kByte) {
                widen(__byte_perm(x[i], y[i], 0x5140), a[0][2 * half], a[0][2 * half + 1]);
                widen(__byte_perm(x[i], y[i], 0x7362), a[1][2 * half], a[1][2 * half + 1]);
            } else {
                // 4-bit codes: code * scale + zero, rounded once to fp16 (2^-11 of the value, as an fp16 cache holds it)
                const uint32_t w = __byte_perm(x[i / 2], y[i / 2], i & 1 ? 0x7632 : 0x5410);
                __half2 s, z;
                memcpy(&s, &vsc[half], 4);
                memcpy(&z, &vze[half], 4);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t c = u4pair_to_f16x2(w, j);
                    __half2 h;
                    memcpy(&h, &c, 4);
                    h = __hfma2(h, s, z);
                    memcpy(&a[j >> 1][2 * half + (j & 1)], &h, 4);
                }
            }
        }
    }
};

// What is left to merge: a warp's, or a CTA's, sums over its pages, for COLS query columns.
template <int COLS, int D>
struct Partial {
    float m[COLS], l[COLS];   // running maximum (base 2) and sum
    float o[COLS][D];
};

// The query columns of a CTA are g heads of each of its tokens, column = token * g + head.
// UNION: several tokens.  NT: tiles of 8 columns.
template <int KIND, int D, int NT, bool UNION>
__global__ void __launch_bounds__(kSelThreads, NT == 1 ? 3 : 2) attention_selected_kernel(SelectedParams p) {
    using Math = PageMath<KIND, D>;
    constexpr int NKS = Math::NKS, NMT = Math::NMT, COLS = 8 * NT;
    extern __shared__ int2 entry[];   // this CTA's pages: page, block (-1: skipped)
    __shared__ Partial<COLS, D> part[kSelWarps + 1];
    __shared__ float weight[kSelCluster][COLS], total[COLS];   // of the merges
    __shared__ int scan[kSelWarps];
    cg::cluster_group cl = cg::this_cluster();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int C = int(cl.num_blocks()), rank = int(cl.block_rank());
    grid_dep_wait();
    grid_dep_launch();
    const int kvh = blockIdx.y, G = p.num_heads / p.num_kv_heads;
    const RowTile tile = find_tile(p.cu_q, p.num_seqs, p.num_rows, p.q_len, p.tile_rows, int(blockIdx.x / C), lane);
    if (tile.s < 0) return;   // no row: the same in every CTA of the cluster
    const int rows = UNION ? tile.rows : 1, cols = rows * G;
    const int64_t ctx = p.context_lens[tile.s];
    const int behind0 = (p.cu_q ? min(p.cu_q[tile.s + 1], p.num_rows) : (tile.s + 1) * p.q_len) - tile.r0;   // rows from the first on
    if (ctx > int64_t(p.max_blocks) * kBS && rank == 0 && kvh == 0 && threadIdx.x == 0) flag_error(p.err, PKV_DEVERR_CAPACITY);
    auto visible = [&](int i) { return visible_tokens(ctx, p.max_blocks, behind0 - i); };
    auto pages_of = [&](int i) { return (visible(i) + kBS - 1) / kBS; };
    auto list_of = [&](int i) { return p.lists + ((int64_t(tile.r0) + i) * p.num_kv_heads + kvh) * p.max_pages; };
    auto count_of = [&](int i) { return min(max(p.counts[(int64_t(tile.r0) + i) * p.num_kv_heads + kvh], 0), p.max_pages); };
    const int vis = visible(rows - 1), vis_all = visible(0);   // tokens that the last row, and that every row, sees
    const int32_t* table = p.block_tables + int64_t(tile.s) * p.max_blocks;
    auto block_of = [&](int page) {
        const int b = table[page];
        if (b >= 0 && b < p.num_blocks) return b;
        flag_error(p.err, PKV_DEVERR_OOB_BLOCK);
        return -1;
    };
    // An entry is taken if it is in range and above every entry taken before it.  By a warp: f(i, entry) of those.
    auto in_order = [&](int row, auto f) {
        const int32_t* list = list_of(row);
        const int count = count_of(row), pages = pages_of(row);
        int top = -1;
        for (int j = 0; j < count; j += 32) {
            const int i = j + lane;
            const int e = i < count ? list[i] : -1;
            const bool in = e >= 0 && e < pages;
            int most = in ? e : -1;   // the largest entry in range up to this one, which is the largest taken too
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, most, o);
                if (lane >= o) most = max(most, x);
            }
            int before = __shfl_up_sync(0xffffffffu, most, 1);
            before = max(lane ? before : -1, top);
            f(i, i < count, in && e > before, e);
            top = max(top, __shfl_sync(0xffffffffu, most, 31));
        }
    };

    // ---- the list: each entry in range and above the one before it, or the slow way
    int i0, i1;   // this CTA's part of the pages
    uint32_t* const bytes = reinterpret_cast<uint32_t*>(entry + p.entries);   // UNION: the rows that list a page, a bit each
    if constexpr (!UNION) {
        const int32_t* list = list_of(0);
        const int count = count_of(0), pages = pages_of(0);
        i0 = int(int64_t(count) * rank / C);
        i1 = int(int64_t(count) * (rank + 1) / C);
        bool fine = true;
        for (int i = threadIdx.x; i < count; i += kSelThreads) {
            const int e = list[i], before = i ? list[i - 1] : -1;
            fine &= e > before && e < pages;
            if (i >= i0 && i < i1) entry[i - i0] = make_int2(e, e >= 0 && e < pages ? block_of(e) : -1);
        }
        if (__syncthreads_or(!fine)) {
            if (warp == 0) {
                in_order(0, [&](int i, bool there, bool taken, int) {
                    if (there && !taken && i >= i0 && i < i1) entry[i - i0].y = -1;
                });
                if (lane == 0 && rank == 0) flag_error(p.err, PKV_DEVERR_PAGE_LIST);
            }
            __syncthreads();
        }
    } else {
        const int n = (vis + kBS - 1) / kBS, words = (n + 3) / 4;
        for (int i = threadIdx.x; i < words; i += kSelThreads) bytes[i] = 0;
        __syncthreads();
        bool fine = true;
        for (int row = warp; row < rows; row += kSelWarps) {
            const int32_t* list = list_of(row);
            const int count = count_of(row), pages = pages_of(row);
            for (int i = lane; i < count; i += 32) {
                const int e = list[i], before = i ? list[i - 1] : -1;
                const bool ok = e > before && e < pages;
                fine &= ok;
                if (ok) atomicOr(bytes + (e >> 2), 1u << (8 * (e & 3) + row));
            }
        }
        if (__syncthreads_or(!fine)) {
            for (int i = threadIdx.x; i < words; i += kSelThreads) bytes[i] = 0;
            __syncthreads();
            for (int row = warp; row < rows; row += kSelWarps)
                in_order(row, [&](int, bool, bool taken, int e) {
                    if (taken) atomicOr(bytes + (e >> 2), 1u << (8 * (e & 3) + row));
                });
            if (threadIdx.x == 0 && rank == 0) flag_error(p.err, PKV_DEVERR_PAGE_LIST);
            __syncthreads();
        }
        // the pages that some row lists, in order: a thread takes neighbouring words
        const int per = (words + kSelThreads - 1) / kSelThreads, w0 = min(int(threadIdx.x) * per, words), w1 = min(w0 + per, words);
        auto listed = [&](int w) {   // one bit for each of a word's pages: 0, 8, 16, 24
            uint32_t x = bytes[w];
            x |= x >> 4;
            x |= x >> 2;
            x |= x >> 1;
            return x & 0x01010101u;
        };
        int c = 0;
        for (int w = w0; w < w1; ++w) c += __popc(listed(w));
        int incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        if (lane == 31) scan[warp] = incl;
        __syncthreads();
        int at = incl - c, count = 0;
#pragma unroll
        for (int w = 0; w < kSelWarps; ++w) {
            if (w < warp) at += scan[w];
            count += scan[w];
        }
        i0 = int(int64_t(count) * rank / C);
        i1 = int(int64_t(count) * (rank + 1) / C);
        for (int w = w0; w < w1; ++w)
            for (uint32_t x = listed(w); x; x &= x - 1, ++at)
                if (at >= i0 && at < i1) entry[at - i0].x = 4 * w + (__ffs(x) - 1) / 8;
        __syncthreads();
        for (int i = threadIdx.x; i < i1 - i0; i += kSelThreads) entry[i].y = block_of(entry[i].x);
        __syncthreads();
    }
    auto rows_of_page = [&](int page) { return UNION ? (bytes[page >> 2] >> (8 * (page & 3))) & 0xffu : 1u; };

    // ---- the query operand: column 8 nt + g, the dims of this thread's K chunks
    uint32_t q[NT][NKS][2];
    float kcol[NT][2];   // what turns the products of columns 8 nt + 2t, + 1 into base-2 scores
    uint32_t bit[NT][2]; // the row of those columns, as a bit (0: no column)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        uint32_t w[D / 8];
        const int col = 8 * nt + g;
        const bool on = col < cols;
        const uint16_t* src = static_cast<const uint16_t*>(p.q) +
                              ((int64_t(tile.r0) + (on ? col / G : 0)) * p.num_heads + int64_t(kvh) * G + (on ? col % G : 0)) * D;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            // 16-byte pieces of the query row, in the chunks' order
            const int d = Math::kHalf ? 32 * i + 8 * t : 64 * (i / 2) + 16 * t + 8 * (i & 1);
            const uint4 x = on ? __ldg(reinterpret_cast<const uint4*>(src + d)) : make_uint4(0u, 0u, 0u, 0u);
            w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
        }
        float back = 1.f;
        if (!Math::kHalf && p.q_dtype == PKV_BF16) {
            // to fp16, times the power of two that brings the column's largest magnitude to [256, 512)
            uint32_t ex = 0;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) ex = max(ex, max((w[i] >> 7) & 0xffu, (w[i] >> 23) & 0xffu));
            ex = max(ex, __shfl_xor_sync(0xffffffffu, ex, 1));
            ex = max(ex, __shfl_xor_sync(0xffffffffu, ex, 2));
            const uint32_t e = min(max(ex, 16u), 254u);
            const float up = __uint_as_float((262u - e) << 23);
            back = __uint_as_float((e - 8u) << 23);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const float2 f = Half16<__nv_bfloat16>::unpack2(w[i]);
                w[i] = pack2<false>(f.x * up, f.y * up);
            }
        }
#pragma unroll
        for (int kk = 0; kk < NKS; ++kk) {
            q[nt][kk][0] = w[2 * kk];
            q[nt][kk][1] = w[2 * kk + 1];
        }
        const float kc = p.scale_log2 * back;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            kcol[nt][c] = __shfl_sync(0xffffffffu, kc, 8 * t + 4 * c);
            const int mine = 8 * nt + 2 * t + c;
            bit[nt][c] = mine < cols ? 1u << (mine / G) : 0u;
        }
    }

    // ---- the pages
    float o[NT][NMT][4], m_run[NT][2], l_part[NT][2];
    float vref = 1.17549435e-38f;   // 8-bit caches: o holds sum P V / vref (times kPUnit); a power of two
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int mt = 0; mt < NMT; ++mt) o[nt][mt][0] = o[nt][mt][1] = o[nt][mt][2] = o[nt][mt][3] = 0.f;
        m_run[nt][0] = m_run[nt][1] = -INFINITY;
        l_part[nt][0] = l_part[nt][1] = 0.f;
    }
    Math pg;
    const int n = i1 - i0;
    int at = warp;
    int2 e = make_int2(0, -1);
    auto next = [&] {   // the warp's next page with a block
        for (; at < n; at += kSelWarps) {
            e = entry[at];
            if (e.y >= 0) break;
        }
    };
    next();
    if (at < n) pg.load_k(p, e.y, kvh, min(vis - e.x * kBS, kBS), g, t);
    while (at < n) {
        const int page = e.x, live = min(vis - page * kBS, kBS);
        pg.load_v(p, e.y, kvh, live, g, t);
        float s[NT][4];
        pg.scores(q, s);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                s[nt][c] *= Math::kHalf ? kcol[nt][c] : pg.ks[0] * kcol[nt][c];
                s[nt][2 + c] *= Math::kHalf ? kcol[nt][c] : pg.ks[1] * kcol[nt][c];
            }
        at += kSelWarps;
        next();
        if (at < n) pg.load_k(p, e.y, kvh, min(vis - e.x * kBS, kBS), g, t);
        const uint32_t who = rows_of_page(page);
        const bool edge = page * kBS + kBS > vis_all;   // some row does not see all of its tokens
        if (edge || (UNION && who != (1u << rows) - 1u)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int row = UNION ? __ffs(bit[nt][c] | 0x100u) - 1 : 0;
                    const int sees = UNION && !(who & bit[nt][c]) ? 0 : visible(row < rows ? row : 0) - page * kBS;
                    if (g >= sees) s[nt][c] = -INFINITY;
                    if (g + 8 >= sees) s[nt][2 + c] = -INFINITY;
                }
        }
        float f[NT][2];
        bool rescale = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float bm = fmaxf(s[nt][c], s[nt][2 + c]);
                bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 4));
                bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 8));
                bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 16));
                const float mn = fmaxf(m_run[nt][c], bm), mu = mn == -INFINITY ? 0.f : mn;
                f[nt][c] = m_run[nt][c] == -INFINITY ? 1.f : exp2_ftz(m_run[nt][c] - mu);
                s[nt][c] = exp2_ftz(s[nt][c] - mu);
                s[nt][2 + c] = exp2_ftz(s[nt][2 + c] - mu);
                l_part[nt][c] = l_part[nt][c] * f[nt][c] + (s[nt][c] + s[nt][2 + c]);
                m_run[nt][c] = mn;
                rescale |= f[nt][c] != 1.f;
            }
        float ratio = Math::kPUnit;   // what the weights are multiplied by in the operand
        if constexpr (Math::kByte) {
            const float mag = fabsf(pg.vs);
            if (mag > vref) {   // the same in every lane
                const uint32_t up = min((__float_as_uint(mag) + 0x007fffffu) & 0xff800000u, 253u << 23);
                const float grow = vref * __uint_as_float((254u << 23) - up);
                vref = __uint_as_float(up);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    f[nt][0] *= grow;
                    f[nt][1] *= grow;
                }
                rescale = true;
            }
            // (scale / vref) * 2^14 in this order: the quotient is exact and at most 1
            ratio = (pg.vs * __uint_as_float((254u << 23) - __float_as_uint(vref))) * Math::kPUnit;
        }
        if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int mt = 0; mt < NMT; ++mt) {
                    o[nt][mt][0] *= f[nt][0]; o[nt][mt][2] *= f[nt][0];
                    o[nt][mt][1] *= f[nt][1]; o[nt][mt][3] *= f[nt][1];
                }
        }
        uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float x = s[nt][2 * h] * ratio, y = s[nt][2 * h + 1] * ratio;
                const uint32_t w = pack2<Math::kBf>(x, y);
                const float2 back = Half16<typename std::conditional<Math::kBf, __nv_bfloat16, __half>::type>::unpack2(w);
                hi[nt][h] = movm_trans(w);
                lo[nt][h] = movm_trans(pack2<Math::kBf>(x - back.x, y - back.y));
            }
        if (!UNION || (!edge && who == (1u << rows) - 1u)) {
#pragma unroll
            for (int i = 0; i < NMT / 2; ++i) {
                uint32_t a[2][4];
                pg.tiles(i, a);
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma16816<Math::kBf>(o[nt][2 * i + j], a[j], hi[nt][0], hi[nt][1]);
                        mma16816<Math::kBf>(o[nt][2 * i + j], a[j], lo[nt][0], lo[nt][1]);
                    }
            }
        } else {
            // Rows that do not list the page keep their sums (a weight of 0 would not stop an infinity or NaN in V); a page
            // that some row sees in part is taken for one row at a time, the last first, without the tokens it does not see.
            for (uint32_t left = who; left;) {
                const int row = 31 - __clz(left);
                const uint32_t now = edge ? 1u << row : who;
                left &= ~now;
                if (edge) pg.cut_v(visible(row) - page * kBS, t);
#pragma unroll
                for (int i = 0; i < NMT / 2; ++i) {
                    uint32_t a[2][4];
                    pg.tiles(i, a);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float x[4] = {o[nt][2 * i + j][0], o[nt][2 * i + j][1], o[nt][2 * i + j][2], o[nt][2 * i + j][3]};
                            mma16816<Math::kBf>(x, a[j], hi[nt][0], hi[nt][1]);
                            mma16816<Math::kBf>(x, a[j], lo[nt][0], lo[nt][1]);
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                if (now & bit[nt][c & 1]) o[nt][2 * i + j][c] = x[c];
                        }
                }
            }
        }
    }

    // ---- the warp's partial
    const float unit = (Math::kByte ? vref : 1.f) * (1.f / Math::kPUnit);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float l = l_part[nt][c];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            const int col = 8 * nt + 2 * t + c;
            if (g == 0) {
                part[warp].m[col] = m_run[nt][c];
                part[warp].l[col] = l;
            }
            if (col < cols) {
#pragma unroll
                for (int mt = 0; mt < NMT; ++mt)
                    *reinterpret_cast<float2*>(&part[warp].o[col][Math::dim(mt, g)]) =
                        make_float2(o[nt][mt][c] * unit, o[nt][mt][2 + c] * unit);
            }
        }
    __syncthreads();

    // ---- the CTA's, and the cluster's: a column's weights first, then its sums
    // a column's weight for one of n partials, by n neighbouring threads (n a power of two); the sum of weighted l
    auto weigh = [&](int n, float m, float l, float& L, float& M) {
        M = l == 0.f ? -INFINITY : m;   // no page (a page has a token whose weight is 1)
        for (int o = 1; o < n; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        const float w = l == 0.f ? 0.f : exp2f(m - M);
        L = l == 0.f ? 0.f : w * l;
        for (int o = 1; o < n; o <<= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
        return w;
    };
    Partial<COLS, D>& mine = part[kSelWarps];
    if (threadIdx.x < kSelWarps * COLS) {
        const int col = threadIdx.x / kSelWarps, k = threadIdx.x % kSelWarps;
        float L, M;
        weight[k][col] = weigh(kSelWarps, part[k].m[col], part[k].l[col], L, M);
        if (k == 0) {
            total[col] = mine.l[col] = L;
            mine.m[col] = M;
        }
    }
    __syncthreads();
    auto store = [&](int item, float4 sum) {
        const int col = item / (D / 4), d = (item % (D / 4)) * 4;
        const float L = total[col], inv = L > 0.f ? 1.f / L : (L == L ? 0.f : L);   // no visible token: zeros
        store_out4(p.out, p.out_dtype, (size_t(tile.r0 + col / G) * p.num_heads + size_t(kvh) * G + col % G) * D + d,
                   make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv));
    };
    auto add = [](float4& sum, float w, float4 v) {
        if (w == 0.f) return;   // not 0 times what was never written
        sum.x += w * v.x;
        sum.y += w * v.y;
        sum.z += w * v.z;
        sum.w += w * v.w;
    };
    const int items = cols * (D / 4);
    for (int i = threadIdx.x; i < items; i += kSelThreads) {
        const int col = i / (D / 4), d = (i % (D / 4)) * 4;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kSelWarps; ++k) add(sum, weight[k][col], *reinterpret_cast<const float4*>(&part[k].o[col][d]));
        if (C == 1) store(i, sum);
        else *reinterpret_cast<float4*>(&mine.o[col][d]) = sum;
    }
    if (C == 1) return;
    cl.sync();
    for (int i = threadIdx.x; i < kSelCluster * COLS; i += kSelThreads) {
        const int col = i / kSelCluster, k = i % kSelCluster;
        const Partial<COLS, D>* from = cl.map_shared_rank(&mine, k < C ? k : 0);
        const float m = from->m[col], l = k < C ? from->l[col] : 0.f;
        float L, M;
        weight[k][col] = weigh(kSelCluster, m, l, L, M);
        if (k == 0) total[col] = L;
    }
    __syncthreads();
    for (int i = rank * kSelThreads + threadIdx.x; i < items; i += C * kSelThreads) {
        const int col = i / (D / 4), d = (i % (D / 4)) * 4;
        float4 v[kSelCluster], sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kSelCluster; ++k)
            v[k] = *reinterpret_cast<const float4*>(&cl.map_shared_rank(&mine, k < C ? k : 0)->o[col][d]);
#pragma unroll
        for (int k = 0; k < kSelCluster; ++k) add(sum, weight[k][col], v[k]);
        store(i, sum);
    }
    cl.sync();   // no CTA leaves while another reads its partial
}

// The kernel may take kSelectedSmem of dynamic shared memory: said once per kernel and device.
template <int KIND, int D, int NT, bool UNION>
cudaError_t launch_nt(const SelectedParams& p, int64_t units, int cluster, size_t smem, cudaStream_t st) {
    static PerDevice ready;
    int dev = 0, one = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = cudaError_t(ready.get(dev, &one, [](int* v) {
        *v = 1;
        return int(cudaFuncSetAttribute(attention_selected_kernel<KIND, D, NT, UNION>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        kSelectedSmem));
    }));
    if (e != cudaSuccess) return e;
    return launch_cluster_kernel(attention_selected_kernel<KIND, D, NT, UNION>, dim3(unsigned(units * cluster), p.num_kv_heads),
                                 dim3(kSelThreads), unsigned(cluster), smem, st, p);
}

template <int KIND>
cudaError_t launch_kind(const SelectedParams& p, int64_t units, int cluster, size_t smem, cudaStream_t st) {
    if (p.tile_rows > 1)
        return p.head_dim == 128 ? launch_nt<KIND, 128, 2, true>(p, units, cluster, smem, st)
                                 : launch_nt<KIND, 64, 2, true>(p, units, cluster, smem, st);
    return p.head_dim == 128 ? launch_nt<KIND, 128, 1, false>(p, units, cluster, smem, st)
                             : launch_nt<KIND, 64, 1, false>(p, units, cluster, smem, st);
}

}  // namespace

cudaError_t launch_attention_selected(SelectedParams p, int cache_kind, cudaStream_t stream) {
    const int64_t hint = p.cu_q ? (int64_t(p.num_rows) + p.num_seqs - 1) / p.num_seqs : p.q_len;   // rows of a sequence
    const int G = p.num_heads / p.num_kv_heads;
    int C = 1;
    int64_t units = 0, most = 0;   // tiles, and the pages that one may have
    size_t smem = 0;
    auto size = [&] {   // the CTA's entries, and a byte for each page where rows share them
        p.entries = int((most + C - 1) / C);
        smem = size_t(p.entries) * 8 + (p.tile_rows > 1 ? (size_t(p.max_blocks) + 3) / 4 * 4 : 0);
        return smem <= kSelectedSmem;
    };
    auto tiles = [&](int rows) {
        p.tile_rows = rows;
        units = p.cu_q ? (rows > 1 ? int64_t(p.num_rows) / rows + p.num_seqs : int64_t(p.num_rows) + p.num_seqs)
                       : int64_t(p.num_seqs) * ((int64_t(p.q_len) + rows - 1) / rows);
        most = int64_t(rows) * p.max_pages;
        if (most > p.max_blocks) most = p.max_blocks;   // an entry beyond them is skipped
        if (rows == 1) most = p.max_pages;
        // three CTAs to an SM (two where rows share pages): as many clusters as run at once
        const int64_t room = rows > 1 ? 304 : 456;
        C = 1;
        while (C < kSelCluster && units * p.num_kv_heads * C * 2 <= room && most >= 2 * C * 2 * kSelWarps) C *= 2;
        while (!size() && C < kSelCluster) C *= 2;
        return size();
    };
    int rows = 16 / G < kSelTokens ? 16 / G : kSelTokens;
    if (rows > hint) rows = int(hint);
    if (!(rows > 1 && tiles(rows)) && !tiles(1)) return cudaErrorInvalidValue;
    if (units * C > 0x7fffffff) return cudaErrorInvalidValue;
    switch (cache_kind) {
        case PKV_CACHE_F16: return launch_kind<PKV_CACHE_F16>(p, units, C, smem, stream);
        case PKV_CACHE_BF16: return launch_kind<PKV_CACHE_BF16>(p, units, C, smem, stream);
        case PKV_CACHE_K8V4: return launch_kind<PKV_CACHE_K8V4>(p, units, C, smem, stream);
        case PKV_CACHE_I8: return launch_kind<PKV_CACHE_I8>(p, units, C, smem, stream);
        default: return launch_kind<PKV_CACHE_E4M3>(p, units, C, smem, stream);
    }
}

}  // namespace pkv
