// attention_selected.cu -- attention of each (query token, kv head) over its own
// list of pages (16-token blocks), as a selection gives them.
//
//   out[r, h] = sum_t softmax_t(scale q[r,h] . K[t]) V[t]  over the listed pages' visible tokens
//
// No two kv heads read the same pages, so the balanced plan over whole sequences
// (attention_impl.cuh) has nothing to cut: a cluster of 1 to 8 CTAs takes one
// (query token, kv head), its warps one page each at a time, and they merge by the
// log-sum-exp identity, in shared memory and then across the cluster.
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
constexpr int kSelRows = 8;      // query heads of a kv head at most

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

    // s = K Q^T: tokens g, g + 8 x query heads 2t, 2t + 1
    __device__ __forceinline__ void scores(const uint32_t (&q)[NKS][2], float (&s)[4]) const {
        s[0] = s[1] = s[2] = s[3] = 0.f;
#pragma unroll
        for (int kk = 0; kk < NKS; ++kk) {
            uint32_t a[4];
            if constexpr (kHalf) {
                a[0] = k[0][2 * kk]; a[1] = k[1][2 * kk]; a[2] = k[0][2 * kk + 1]; a[3] = k[1][2 * kk + 1];
            } else {
                widen(k[0][kk], a[0], a[2]);
                widen(k[1][kk], a[1], a[3]);
            }
            mma16816<kBf>(s, a, q[kk][0], q[kk][1]);
        }
    }

    // the M tile mt of V^T: rows g and g + 8 are dims dim(mt, g) and one above
    static __device__ __forceinline__ int dim(int mt, int g) {
        return NVB == 32 ? (mt >> 2) * 64 + 8 * g + 2 * (mt & 3) : (D / 8) * g + 2 * mt;
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

// What is left to merge: a warp's, or a CTA's, sums over its pages.
template <int D>
struct Partial {
    float m[kSelRows], l[kSelRows];   // running maximum (base 2) and sum of each query head
    float o[kSelRows][D];
};

template <int KIND, int D>
__global__ void __launch_bounds__(kSelThreads, 3) attention_selected_kernel(SelectedParams p) {
    using Math = PageMath<KIND, D>;
    constexpr int NKS = Math::NKS, NMT = Math::NMT;
    extern __shared__ int2 entry[];   // this CTA's entries of the list: page, block (-1: skipped)
    __shared__ Partial<D> part[kSelWarps + 1];
    cg::cluster_group cl = cg::this_cluster();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int C = int(cl.num_blocks()), rank = int(cl.block_rank());
    grid_dep_wait();
    grid_dep_launch();
    const int64_t r = blockIdx.x / C;
    const int kvh = blockIdx.y, G = p.num_heads / p.num_kv_heads;
    const Row row = find_row(p.cu_q, p.context_lens, p.num_seqs, p.q_len, p.max_blocks, int(r), lane);
    if (row.s < 0) return;   // behind the last sequence: the row keeps what it held
    if (row.over && rank == 0 && kvh == 0 && threadIdx.x == 0) flag_error(p.err, PKV_DEVERR_CAPACITY);

    // ---- the list: each entry in range and above the one before it, or the slow way below
    const int pages = (row.vis + kBS - 1) / kBS;
    const int64_t pair = r * p.num_kv_heads + kvh;
    const int32_t* list = p.lists + pair * p.max_pages;
    const int32_t* table = p.block_tables + int64_t(row.s) * p.max_blocks;
    const int count = min(max(p.counts[pair], 0), p.max_pages);
    const int i0 = int(int64_t(count) * rank / C), i1 = int(int64_t(count) * (rank + 1) / C);
    bool fine = true;
    for (int i = threadIdx.x; i < count; i += kSelThreads) {
        const int e = list[i], before = i ? list[i - 1] : -1;
        fine &= e > before && e < pages;
        if (i >= i0 && i < i1) {
            int b = e >= 0 && e < pages ? table[e] : -1;
            if (e >= 0 && e < pages && (b < 0 || b >= p.num_blocks)) {
                flag_error(p.err, PKV_DEVERR_OOB_BLOCK);
                b = -1;
            }
            entry[i - i0] = make_int2(e, b);
        }
    }
    if (__syncthreads_or(!fine)) {
        // an entry is taken if it is in range and above every entry taken before it
        if (warp == 0) {
            int top = -1;
            for (int j = 0; j < count; j += 32) {
                const int i = j + lane;
                const int e = i < count ? list[i] : -1;
                const bool in = e >= 0 && e < pages;
                int most = in ? e : -1;   // largest in-range entry up to this one: what is taken has that as its maximum too
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int x = __shfl_up_sync(0xffffffffu, most, o);
                    if (lane >= o) most = max(most, x);
                }
                int before = __shfl_up_sync(0xffffffffu, most, 1);
                before = max(lane ? before : -1, top);
                if (i >= i0 && i < i1 && !(in && e > before)) entry[i - i0].y = -1;
                top = max(top, __shfl_sync(0xffffffffu, most, 31));
            }
            if (lane == 0 && rank == 0) flag_error(p.err, PKV_DEVERR_PAGE_LIST);
        }
        __syncthreads();
    }

    // ---- the query operand: head g, the dims of this thread's K chunks
    uint32_t q[NKS][2];
    float kcol[2];   // what turns query head 2t's and 2t + 1's products into base-2 scores
    {
        uint32_t w[D / 8];
        const bool on = g < G;
        const uint16_t* src = static_cast<const uint16_t*>(p.q) + (r * p.num_heads + int64_t(kvh) * G + (on ? g : 0)) * D;
        constexpr int PER = Math::kHalf ? 8 : 16;   // dims of a chunk
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            // 16-byte pieces of the query row, in the chunks' order
            const int d = Math::kHalf ? 32 * i + 8 * t : 64 * (i / 2) + PER * t + 8 * (i & 1);
            const uint4 x = on ? __ldg(reinterpret_cast<const uint4*>(src + d)) : make_uint4(0u, 0u, 0u, 0u);
            w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
        }
        float back = 1.f;
        if (!Math::kHalf && p.q_dtype == PKV_BF16) {
            // to fp16, times the power of two that brings the head's largest magnitude to [256, 512)
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
            q[kk][0] = w[2 * kk];
            q[kk][1] = w[2 * kk + 1];
        }
        const float kc = p.scale_log2 * back;
        kcol[0] = __shfl_sync(0xffffffffu, kc, 8 * t);
        kcol[1] = __shfl_sync(0xffffffffu, kc, 8 * t + 4);
    }

    // ---- the pages
    float o[NMT][4], m_run[2] = {-INFINITY, -INFINITY}, l_part[2] = {0.f, 0.f};
    float vref = 1.17549435e-38f;   // 8-bit caches: o holds sum P V / vref (times kPUnit); a power of two
#pragma unroll
    for (int mt = 0; mt < NMT; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
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
    if (at < n) pg.load_k(p, e.y, kvh, min(row.vis - e.x * kBS, kBS), g, t);
    while (at < n) {
        const int live = min(row.vis - e.x * kBS, kBS);
        pg.load_v(p, e.y, kvh, live, g, t);
        float s[4];
        pg.scores(q, s);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            s[c] *= Math::kHalf ? kcol[c] : pg.ks[0] * kcol[c];
            s[2 + c] *= Math::kHalf ? kcol[c] : pg.ks[1] * kcol[c];
        }
        at += kSelWarps;
        next();
        if (at < n) pg.load_k(p, e.y, kvh, min(row.vis - e.x * kBS, kBS), g, t);
        if (live < kBS) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (g >= live) s[c] = -INFINITY;
                if (g + 8 >= live) s[2 + c] = -INFINITY;
            }
        }
        float f[2];
        bool rescale = false;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float bm = fmaxf(s[c], s[2 + c]);
            bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 4));
            bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 8));
            bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 16));
            const float mn = fmaxf(m_run[c], bm), mu = mn == -INFINITY ? 0.f : mn;
            f[c] = m_run[c] == -INFINITY ? 1.f : exp2_ftz(m_run[c] - mu);
            s[c] = exp2_ftz(s[c] - mu);
            s[2 + c] = exp2_ftz(s[2 + c] - mu);
            l_part[c] = l_part[c] * f[c] + (s[c] + s[2 + c]);
            m_run[c] = mn;
            rescale |= f[c] != 1.f;
        }
        float ratio = Math::kPUnit;   // what the weights are multiplied by in the operand
        if constexpr (Math::kByte) {
            const float mag = fabsf(pg.vs);
            if (mag > vref) {   // the same in every lane
                const uint32_t up = min((__float_as_uint(mag) + 0x007fffffu) & 0xff800000u, 253u << 23);
                const float grow = vref * __uint_as_float((254u << 23) - up);
                vref = __uint_as_float(up);
                f[0] *= grow;
                f[1] *= grow;
                rescale = true;
            }
            // (scale / vref) * 2^14 in this order: the quotient is exact and at most 1
            ratio = (pg.vs * __uint_as_float((254u << 23) - __float_as_uint(vref))) * Math::kPUnit;
        }
        if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
            for (int mt = 0; mt < NMT; ++mt) {
                o[mt][0] *= f[0]; o[mt][2] *= f[0];
                o[mt][1] *= f[1]; o[mt][3] *= f[1];
            }
        }
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float x = s[2 * h] * ratio, y = s[2 * h + 1] * ratio;
            const uint32_t w = pack2<Math::kBf>(x, y);
            const float2 back = Half16<typename std::conditional<Math::kBf, __nv_bfloat16, __half>::type>::unpack2(w);
            hi[h] = movm_trans(w);
            lo[h] = movm_trans(pack2<Math::kBf>(x - back.x, y - back.y));
        }
#pragma unroll
        for (int i = 0; i < NMT / 2; ++i) {
            uint32_t a[2][4];
            pg.tiles(i, a);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                mma16816<Math::kBf>(o[2 * i + j], a[j], hi[0], hi[1]);
                mma16816<Math::kBf>(o[2 * i + j], a[j], lo[0], lo[1]);
            }
        }
    }

    // ---- the warp's partial
    const float unit = (Math::kByte ? vref : 1.f) * (1.f / Math::kPUnit);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        float l = l_part[c];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        const int qh = 2 * t + c;
        if (g == 0) {
            part[warp].m[qh] = m_run[c];
            part[warp].l[qh] = l;
        }
        if (qh < G) {
#pragma unroll
            for (int mt = 0; mt < NMT; ++mt)
                *reinterpret_cast<float2*>(&part[warp].o[qh][Math::dim(mt, g)]) = make_float2(o[mt][c] * unit, o[mt][2 + c] * unit);
        }
    }
    __syncthreads();

    // ---- the CTA's, and the cluster's
    auto merge = [&](int n, auto from, int item, float& M, float& L) {
        const int qh = item / (D / 4), d = (item % (D / 4)) * 4;
        M = -INFINITY;
        for (int k = 0; k < n; ++k) M = fmaxf(M, from(k)->m[qh]);
        L = 0.f;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < n; ++k) {
            const Partial<D>* x = from(k);
            if (x->l[qh] == 0.f) continue;   // no page (a page has a token whose weight is 1)
            const float w = exp2f(x->m[qh] - M);
            const float4 v = *reinterpret_cast<const float4*>(&x->o[qh][d]);
            L += w * x->l[qh];
            sum.x += w * v.x;
            sum.y += w * v.y;
            sum.z += w * v.z;
            sum.w += w * v.w;
        }
        return sum;
    };
    auto store = [&](int item, float4 sum, float L) {
        const int qh = item / (D / 4), d = (item % (D / 4)) * 4;
        const float inv = L > 0.f ? 1.f / L : (L == L ? 0.f : L);   // no visible token: zeros
        store_out4(p.out, p.out_dtype, size_t(r * p.num_heads + int64_t(kvh) * G + qh) * D + d,
                   make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv));
    };
    const int items = G * (D / 4);
    auto warps = [&](int k) { return &part[k]; };
    float M, L;
    if (C == 1) {
        for (int i = threadIdx.x; i < items; i += kSelThreads) {
            const float4 sum = merge(kSelWarps, warps, i, M, L);
            store(i, sum, L);
        }
        return;
    }
    Partial<D>& mine = part[kSelWarps];
    for (int i = threadIdx.x; i < items; i += kSelThreads) {
        const float4 sum = merge(kSelWarps, warps, i, M, L);
        const int qh = i / (D / 4), d = (i % (D / 4)) * 4;
        *reinterpret_cast<float4*>(&mine.o[qh][d]) = sum;
        if (d == 0) {
            mine.m[qh] = M;
            mine.l[qh] = L;
        }
    }
    cl.sync();
    auto ranks = [&](int k) { return cl.map_shared_rank(&mine, k); };
    for (int i = rank * kSelThreads + threadIdx.x; i < items; i += C * kSelThreads) {
        const float4 sum = merge(C, ranks, i, M, L);
        store(i, sum, L);
    }
    cl.sync();   // no CTA leaves while another reads its partial
}

// The kernel may take kSelectedSmem of shared memory for list entries: said once per kernel and device.
template <int KIND, int D>
cudaError_t launch_d(const SelectedParams& p, int cluster, size_t smem, cudaStream_t st) {
    static PerDevice ready;
    int dev = 0, one = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = cudaError_t(ready.get(dev, &one, [](int* v) {
        *v = 1;
        return int(cudaFuncSetAttribute(attention_selected_kernel<KIND, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelectedSmem));
    }));
    if (e != cudaSuccess) return e;
    return launch_cluster_kernel(attention_selected_kernel<KIND, D>, dim3(unsigned(int64_t(p.num_rows) * cluster), p.num_kv_heads),
                                 dim3(kSelThreads), unsigned(cluster), smem, st, p);
}

template <int KIND>
cudaError_t launch_kind(const SelectedParams& p, int cluster, size_t smem, cudaStream_t st) {
    return p.head_dim == 128 ? launch_d<KIND, 128>(p, cluster, smem, st) : launch_d<KIND, 64>(p, cluster, smem, st);
}

}  // namespace

cudaError_t launch_attention_selected(const SelectedParams& p, int cache_kind, cudaStream_t stream) {
    const int64_t pairs = int64_t(p.num_rows) * p.num_kv_heads;
    int C = 1;
    while (C < kSelCluster && pairs * C < 304 && p.max_pages >= 4 * C * kSelWarps) C *= 2;
    while (C < kSelCluster && (int64_t(p.max_pages) + C - 1) / C * 8 > kSelectedSmem) C *= 2;
    const size_t smem = (size_t(p.max_pages) + C - 1) / C * 8;
    if (smem > kSelectedSmem || int64_t(p.num_rows) * C > 0x7fffffff) return cudaErrorInvalidValue;
    switch (cache_kind) {
        case PKV_CACHE_F16: return launch_kind<PKV_CACHE_F16>(p, C, smem, stream);
        case PKV_CACHE_BF16: return launch_kind<PKV_CACHE_BF16>(p, C, smem, stream);
        case PKV_CACHE_K8V4: return launch_kind<PKV_CACHE_K8V4>(p, C, smem, stream);
        case PKV_CACHE_I8: return launch_kind<PKV_CACHE_I8>(p, C, smem, stream);
        default: return launch_kind<PKV_CACHE_E4M3>(p, C, smem, stream);
    }
}

}  // namespace pkv
