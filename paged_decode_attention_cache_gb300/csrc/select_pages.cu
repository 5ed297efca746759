// select_pages.cu -- the bounds of each page's keys, and the selection of the
// pages that a query token attends by them (a page is a cache block, 16 tokens).
//
// Bounds: lo[d] and hi[d], the smallest and the largest key of a page's stored
// tokens, dim by dim and kv head by kv head.
//
// Score of a page for a query token and a kv head, over the head's G query heads:
//   sum_h sum_d max(q_hd lo_d, q_hd hi_d) = sum_d [ n_d lo_d + p_d hi_d ],
//   n_d = sum_h min(q_hd, 0),  p_d = sum_h max(q_hd, 0)
// since the maximum takes hi where q is positive and lo where it is negative: one
// product of length 2 D whatever the group, and the queries are folded once.
//
// The selection is that of the exact scores.  They are worked out in fp32, with
// a bound e on their error; the k-th largest of them, T, is found by a radix
// selection on their bits; a page above T + 2 e is in, one below T - 2 e is out, and
// only if more pages lie between than there are places left are those pages'
// scores worked out again in fp64 (the products are exact there).  fp64 runs at a
// sixtieth of the fp32 rate on this GPU; one row in some tens has two pages that near.
#include <cooperative_groups.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "per_device.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_rows.cuh"

namespace cg = cooperative_groups;

namespace pkv {

namespace {

// ---------------------------------------------------------------- bounds

// What the bounds are the smallest and largest of, 16 bytes at a time.
struct I8 {};
struct E4M3 {};
struct K8 {};   // int8 codes with a scale per token

// e4m3 codes as signed bytes in the numbers' order, and back (the map is its own inverse).
__device__ __forceinline__ uint32_t e4m3_order4(uint32_t w) {
    const uint32_t neg = (w >> 7) & 0x01010101u;
    return w ^ (neg * 0x7fu);
}

template <typename T>
struct Extremes {
    uint32_t lo[4], hi[4];
    static __device__ __forceinline__ uint32_t in(uint32_t w) {
        if constexpr (std::is_same<T, E4M3>::value) return e4m3_order4(w);
        return w;
    }
    static __device__ __forceinline__ uint32_t low(uint32_t a, uint32_t b) {
        if constexpr (std::is_same<T, I8>::value || std::is_same<T, E4M3>::value) {
            return __vmins4(a, b);
        } else {
            using V = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
            V x, y;
            memcpy(&x, &a, 4);
            memcpy(&y, &b, 4);
            const V z = __hmin2(x, y);
            uint32_t r;
            memcpy(&r, &z, 4);
            return r;
        }
    }
    static __device__ __forceinline__ uint32_t high(uint32_t a, uint32_t b) {
        if constexpr (std::is_same<T, I8>::value || std::is_same<T, E4M3>::value) {
            return __vmaxs4(a, b);
        } else {
            using V = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
            V x, y;
            memcpy(&x, &a, 4);
            memcpy(&y, &b, 4);
            const V z = __hmax2(x, y);
            uint32_t r;
            memcpy(&r, &z, 4);
            return r;
        }
    }
    __device__ __forceinline__ void take(uint4 v, bool first) {
        const uint32_t w[4] = {in(v.x), in(v.y), in(v.z), in(v.w)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = first ? w[i] : low(lo[i], w[i]);
            hi[i] = first ? w[i] : high(hi[i], w[i]);
        }
    }
    __device__ __forceinline__ uint4 lows() const { return make_uint4(in(lo[0]), in(lo[1]), in(lo[2]), in(lo[3])); }
    __device__ __forceinline__ uint4 highs() const { return make_uint4(in(hi[0]), in(hi[1]), in(hi[2]), in(hi[3])); }
};

constexpr int kBoundsThreads = 128;

// A thread takes 16 bytes of the keys' width (some dims of one kv head) of one
// touched page, over its stored rows: all rows' loads are in flight together, and
// neighbouring threads read neighbouring bytes.  CTAs of a sequence share its
// touched pages.
template <typename T>
__global__ void __launch_bounds__(kBoundsThreads) key_bounds_kernel(KeyBoundsParams p) {
    grid_dep_wait();
    grid_dep_launch();
    constexpr bool kK8 = std::is_same<T, K8>::value;
    constexpr int E = std::is_same<T, __half>::value || std::is_same<T, __nv_bfloat16>::value ? 2 : 1;   // bytes of a key
    const int s = blockIdx.y;
    const int64_t ctx64 = p.context_lens[s];
    int64_t n = p.q_len;
    if (p.cu_new) n = int64_t(p.cu_new[s + 1]) - p.cu_new[s];
    if (ctx64 <= 0 || n <= 0) return;
    const int cap = p.max_blocks * kBlockSize;
    if (ctx64 > cap && blockIdx.x == 0 && threadIdx.x == 0) flag_error(p.err, PKV_DEVERR_CAPACITY);
    const int64_t p0 = max(ctx64 - n, int64_t(0));
    const int ctx = int(min(ctx64, int64_t(cap)));
    if (p0 >= ctx) return;
    const int b0 = int(p0) / kBlockSize, pages = (ctx + kBlockSize - 1) / kBlockSize - b0;
    const int row = p.num_kv_heads * p.head_dim * E;   // bytes of a token's keys
    const int chunks = row / 16;
    const int64_t items = int64_t(pages) * chunks;
    for (int64_t i = int64_t(blockIdx.x) * kBoundsThreads + threadIdx.x; i < items; i += int64_t(gridDim.x) * kBoundsThreads) {
        const int page = b0 + int(i / chunks), c = int(i % chunks);
        const int pb = p.block_tables[int64_t(s) * p.max_blocks + page];
        if (pb < 0 || pb >= p.num_blocks) {
            if (c == 0) flag_error(p.err, PKV_DEVERR_OOB_BLOCK);
            continue;
        }
        const int rows = min(kBlockSize, ctx - page * kBlockSize);
        const uint8_t* src = static_cast<const uint8_t*>(p.k_cache) + int64_t(pb) * kBlockSize * row + 16 * c;
        uint4 x[kBlockSize];
#pragma unroll
        for (int r = 0; r < kBlockSize; ++r)
            if (r < rows) x[r] = __ldg(reinterpret_cast<const uint4*>(src + int64_t(r) * row));
        const int dim_bytes = p.head_dim * E, h = c * 16 / dim_bytes, at = c * 16 - h * dim_bytes;
        const int64_t head = int64_t(pb) * p.num_kv_heads + h;
        if constexpr (!kK8) {
            Extremes<T> m;
#pragma unroll
            for (int r = 0; r < kBlockSize; ++r)
                if (r < rows) m.take(x[r], r == 0);
            uint8_t* dst = static_cast<uint8_t*>(p.bounds) + head * 2 * dim_bytes + at;
            *reinterpret_cast<uint4*>(dst) = m.lows();
            *reinterpret_cast<uint4*>(dst + dim_bytes) = m.highs();
        } else {
            // code * scale is exact in fp32 (8 and 11 bits); fp16 takes it rounded outwards
            const uint16_t* sc = static_cast<const uint16_t*>(p.k_scale) + head * kBlockSize;
            float lo[16], hi[16];
#pragma unroll
            for (int r = 0; r < kBlockSize; ++r) {
                if (r >= rows) continue;
                const float f = Half16<__half>::to_float(sc[r]);
                const uint32_t w[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
#pragma unroll
                for (int d = 0; d < 16; ++d) {
                    const float v = float(int(int8_t(w[d / 4] >> (8 * (d & 3))))) * f;
                    lo[d] = r == 0 ? v : fminf(lo[d], v);
                    hi[d] = r == 0 ? v : fmaxf(hi[d], v);
                }
            }
            __half* dst = static_cast<__half*>(p.bounds) + head * 2 * p.head_dim + at;
            uint32_t wl[8], wh[8];
#pragma unroll
            for (int d = 0; d < 8; ++d) {
                const __half2 a = __halves2half2(__float2half_rd(lo[2 * d]), __float2half_rd(lo[2 * d + 1]));
                const __half2 b = __halves2half2(__float2half_ru(hi[2 * d]), __float2half_ru(hi[2 * d + 1]));
                memcpy(wl + d, &a, 4);
                memcpy(wh + d, &b, 4);
            }
            uint4* dl = reinterpret_cast<uint4*>(dst);
            uint4* dh = reinterpret_cast<uint4*>(dst + p.head_dim);
            dl[0] = make_uint4(wl[0], wl[1], wl[2], wl[3]);
            dl[1] = make_uint4(wl[4], wl[5], wl[6], wl[7]);
            dh[0] = make_uint4(wh[0], wh[1], wh[2], wh[3]);
            dh[1] = make_uint4(wh[4], wh[5], wh[6], wh[7]);
        }
    }
}

// ---------------------------------------------------------------- selection

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kLoads = 8;        // 16-byte loads in flight of a lane
constexpr int kSmallBand = 64;   // pages near the border whose fp64 scores are compared each with each

// 16 bytes of bounds as fp32 (exact).
template <typename T>
struct Chunk {
    static constexpr int kN = std::is_same<T, __half>::value || std::is_same<T, __nv_bfloat16>::value ? 8 : 16;
    static __device__ __forceinline__ void get(uint4 v, float (&f)[kN]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (kN == 8) {
                const float2 two = Half16<T>::unpack2(w[i]);
                f[2 * i] = two.x;
                f[2 * i + 1] = two.y;
            } else if constexpr (std::is_same<T, I8>::value) {
#pragma unroll
                for (int j = 0; j < 4; ++j) f[4 * i + j] = float(int(int8_t(w[i] >> (8 * j))));
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w[i] >> (16 * j)), __NV_E4M3));
                    const float2 two = __half22float2(h);
                    f[4 * i + 2 * j] = two.x;
                    f[4 * i + 2 * j + 1] = two.y;
                }
            }
        }
    }
    static __device__ __forceinline__ double one(const void* base, int64_t i) {
        if constexpr (kN == 8) return double(Half16<T>::to_float(static_cast<const uint16_t*>(base)[i]));
        else if constexpr (std::is_same<T, I8>::value) return double(static_cast<const int8_t*>(base)[i]);
        else
            return double(__half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(base)[i], __NV_E4M3))));
    }
};

// Order of fp32 numbers as unsigned integers, and back.
__device__ __forceinline__ uint32_t key32(float f) {
    const uint32_t u = __float_as_uint(f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_key32(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }
__device__ __forceinline__ uint64_t key64(double d) {
    const uint64_t u = uint64_t(__double_as_longlong(d + 0.0));   // -0 counts as 0
    return u >> 63 ? ~u : u | (uint64_t(1) << 63);
}

struct Shared {
    uint32_t hist[8][256];
    float amax[kWarps];
    float absum;                   // this CTA's largest sum of magnitudes
    int above, band;               // this CTA's pages above T + 2e, and between
    int taken, ties;               // pages that this CTA writes; pages that tie at the border
    int list_n;
    int list_page[kSmallBand];
    double list_score[kSmallBand];
    int scan[kWarps];
    int bin, rest;
    double w64[2 * 128];
};

// A CTA's share of the row's pages and what it reads them with.
template <typename T>
struct Share {
    const SelectParams& p;
    int s, kvh, p0, n;             // this CTA's pages [p0, p0 + n)

    // the page's score in fp64, by a warp; every lane gets it
    __device__ double exact(const Shared& sh, int page, int lane) const {
        const int pb = p.block_tables[int64_t(s) * p.max_blocks + page];
        if (pb < 0 || pb >= p.num_blocks) return -INFINITY;
        const int64_t head = int64_t(pb) * p.num_kv_heads + kvh, at = head * 2 * p.head_dim;
        double x = 0.0;
        for (int i = lane; i < 2 * p.head_dim; i += 32) x = fma(sh.w64[i], Chunk<T>::one(p.bounds, at + i), x);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (Chunk<T>::kN == 16) x *= double(p.k_scale[head]);
        return x == x ? x : -INFINITY;
    }
};

// Exclusive prefix sum of v over the CTA's threads; the total in `total`.
__device__ __forceinline__ int block_scan(int v, int* warps, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) warps[warp] = x;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += warps[w];
        total += warps[w];
    }
    return before + x - v;
}

// One digit of a radix selection over the cluster: the histograms are complete in
// every CTA; finds the bin, from the top, that holds the need-th number.  bin and
// rest (the place within the bin, from 1) come out the same in every CTA.
__device__ __forceinline__ void find_bin(cg::cluster_group& cl, Shared& sh, uint32_t (&hist)[256], int need, int& bin,
                                         int& rest) {
    cl.sync();
    const int t = threadIdx.x, b = 255 - t;   // thread t counts from the top
    int c = 0;
    for (unsigned r = 0; r < cl.num_blocks(); ++r) c += int(cl.map_shared_rank(&hist[0], r)[b]);
    int total;
    const int before = block_scan(c, sh.scan, total);
    if (before < need && before + c >= need) {
        sh.bin = b;
        sh.rest = need - before;
    }
    __syncthreads();
    bin = sh.bin;
    rest = sh.rest;
}

// A cluster of 1 to 8 CTAs per (query token, kv head): each scores a contiguous
// share of the pages, keeps the scores in its shared memory, and they select
// together through the others' histograms.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) select_pages_kernel(SelectParams p) {
    extern __shared__ float score[];
    __shared__ Shared sh;
    cg::cluster_group cl = cg::this_cluster();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int C = int(cl.num_blocks()), rank = int(cl.block_rank());
    grid_dep_wait();
    grid_dep_launch();
    const int64_t r = blockIdx.x / C;
    const int kvh = blockIdx.y;
    const Row row = find_row(p.cu_q, p.context_lens, p.num_seqs, p.q_len, p.max_blocks, int(r), lane);
    if (row.s < 0) return;   // behind the last sequence: the row keeps what it held (all CTAs of the cluster agree)
    if (row.over && rank == 0 && kvh == 0 && threadIdx.x == 0) flag_error(p.err, PKV_DEVERR_CAPACITY);
    const int n = (row.vis + kBlockSize - 1) / kBlockSize;
    int32_t* list = p.lists + (r * p.num_kv_heads + kvh) * p.max_pages;
    if (rank == 0 && threadIdx.x == 0) p.counts[r * p.num_kv_heads + kvh] = min(n, p.max_pages);
    if (n <= p.max_pages) {   // every page
        for (int i = rank * kThreads + threadIdx.x; i < p.max_pages; i += C * kThreads) list[i] = i < n ? i : -1;
        return;
    }
    const int share = (n + C - 1) / C;
    const Share<T> my{p, row.s, kvh, min(rank * share, n), min(share, max(0, n - rank * share))};
    const int c0 = p.keep_first, c1 = n - p.keep_last;   // the pages that scores decide about
    const int want = p.max_pages - p.keep_first - p.keep_last;

    // ---- the queries, folded
    constexpr int N = Chunk<T>::kN, LP = 2 * D / N, PP = 32 / LP;   // numbers of a lane, lanes of a page, pages of a load
    const int G = p.num_heads / p.num_kv_heads;
    float w[N];
    {
        const int i0 = (lane % LP) * N;
        const bool hi = i0 >= D;
        const int64_t q0 = (r * p.num_heads + int64_t(kvh) * G) * D + (hi ? i0 - D : i0);
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = 0.f;
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float q = load_q(p.q, p.q_dtype, q0 + int64_t(g) * D + i);
                w[i] += hi ? fmaxf(q, 0.f) : fminf(q, 0.f);
            }
    }
    for (int i = threadIdx.x; i < 8 * 256; i += kThreads) (&sh.hist[0][0])[i] = 0;
    if (threadIdx.x == 0) sh.list_n = sh.above = sh.band = 0;

    // ---- scores
    float amax = 0.f;   // of this lane's products, the largest sum of magnitudes
    constexpr int STEP = kLoads * PP;
    const int32_t* table = p.block_tables + int64_t(row.s) * p.max_blocks + my.p0;
    for (int i0 = warp * STEP; i0 < my.n; i0 += kWarps * STEP) {
        int pb = -1;
        if (lane < STEP && i0 + lane < my.n) {
            pb = table[i0 + lane];
            if (pb < 0 || pb >= p.num_blocks) {
                pb = -1;
                flag_error(p.err, PKV_DEVERR_OOB_BLOCK);
            }
        }
        float sc = 1.f;
        if (N == 16) sc = pb >= 0 ? p.k_scale[int64_t(pb) * p.num_kv_heads + kvh] : 0.f;
        uint4 x[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            const int b = __shfl_sync(0xffffffffu, pb, u * PP + lane / LP);
            x[u] = make_uint4(0u, 0u, 0u, 0u);
            if (b >= 0)
                x[u] = __ldg(static_cast<const uint4*>(p.bounds) + (int64_t(b) * p.num_kv_heads + kvh) * LP + lane % LP);
        }
        float v[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            float f[N], a = 0.f;
            Chunk<T>::get(x[u], f);
            v[u] = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                v[u] = fmaf(w[i], f[i], v[u]);
                a = fmaf(fabsf(w[i]), fabsf(f[i]), a);
            }
            if (N == 16) a *= fabsf(__shfl_sync(0xffffffffu, sc, u * PP + lane / LP));
            amax = a <= amax ? amax : a;   // a NaN stays
        }
        // sums over the page's lanes: each step halves the loads a lane holds, while there are any
        int held = kLoads, u = 0;
#pragma unroll
        for (int o = LP / 2; o >= 1; o >>= 1) {
            if (held > 1) {
                held /= 2;
                const bool up = lane & o;
#pragma unroll
                for (int i = 0; i < kLoads / 2; ++i)
                    if (i < held) {
                        const float give = up ? v[i] : v[i + held];
                        const float keep = up ? v[i + held] : v[i];
                        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                    }
                u += up ? held : 0;
            } else {
                v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
            }
        }
        constexpr int SPARE = LP / kLoads;   // lanes that hold the same sum
        const int at = u * PP + lane / LP;
        float sum = v[0];
        if (N == 16) sum *= __shfl_sync(0xffffffffu, sc, at);
        const int b = __shfl_sync(0xffffffffu, pb, at);
        if (lane % SPARE == 0 && i0 + at < my.n) score[i0 + at] = b >= 0 && sum == sum ? sum : -INFINITY;
    }
    {   // the largest sum of magnitudes: at most the sum of the lanes' largest
        float a = amax;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
        if (lane == 0) sh.amax[warp] = a;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        float a = 0.f;
        for (int k = 0; k < kWarps; ++k) a = sh.amax[k] <= a ? a : sh.amax[k];
        sh.absum = a;
    }
    const int l0 = max(c0 - my.p0, 0), l1 = min(c1 - my.p0, my.n);   // this CTA's candidates: [l0, l1)

    // ---- T, the want-th largest score
    uint32_t prefix = 0;
    int need = want, bin, rest;
    for (int d = 0; d < 4; ++d) {
        const int shift = 24 - 8 * d;
        for (int i = l0 + threadIdx.x; i < l1; i += kThreads) {
            const uint32_t k = key32(score[i]);
            if (d == 0 || k >> (shift + 8) == prefix) atomicAdd(&sh.hist[d][(k >> shift) & 255u], 1u);
        }
        if (want == 0) break;
        find_bin(cl, sh, sh.hist[d], need, bin, rest);
        prefix = (prefix << 8) | uint32_t(bin);
        need = rest;
    }
    if (want == 0) cl.sync();
    float absum = 0.f;
    for (int k = 0; k < C; ++k) {
        const float a = *cl.map_shared_rank(&sh.absum, k);
        absum = a <= absum ? absum : a;
    }
    // |fp32 score - score| <= 2^-19 of the sum of magnitudes: at most 16 products and 5 sums in a row, 7 roundings of the
    // folded queries and one of the scale, each 2^-24; and what underflows
    const float e2 = absum > 0.f ? 2.f * fmaf(absum, 1.9073486e-6f, 1.17549435e-38f) : absum == 0.f ? 0.f : INFINITY;
    const float T0 = want ? from_key32(prefix) : INFINITY;
    const float up = T0 + e2, down = T0 - e2;
    auto above = [&](float x) { return want && x > up; };
    auto near = [&](float x) { return want && !(x > up) && !(x < down); };
    {
        int a = 0, b = 0;
        for (int i = l0 + threadIdx.x; i < l1; i += kThreads) {
            a += above(score[i]);
            b += near(score[i]);
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        if (lane == 0) {
            atomicAdd(&sh.above, a);
            atomicAdd(&sh.band, b);
        }
    }
    cl.sync();
    int total_above = 0, total_band = 0;
    for (int k = 0; k < C; ++k) {
        total_above += *cl.map_shared_rank(&sh.above, k);
        total_band += *cl.map_shared_rank(&sh.band, k);
    }
    const int places = want - total_above;   // for the pages between
    const bool whole = total_band == places;
    // a page between is marked: in +inf, out -inf, NaN if it ties with the border and the lower page goes first
    constexpr float kTie = NAN;
    if (!whole) {
        int tie_places = places;
        if (e2 == 0.f) {   // every score is exactly 0
            for (int i = l0 + threadIdx.x; i < l1; i += kThreads)
                if (near(score[i])) score[i] = kTie;
        } else {
            for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
                const bool hi = i >= D;
                const int64_t q0 = (r * p.num_heads + int64_t(kvh) * G) * D + (hi ? i - D : i);
                double x = 0.0;
                for (int g = 0; g < G; ++g) {
                    const float q = load_q(p.q, p.q_dtype, q0 + int64_t(g) * D);
                    x += hi ? fmaxf(q, 0.f) : fminf(q, 0.f);
                }
                sh.w64[i] = x;
            }
            __syncthreads();
            if (total_band <= kSmallBand) {
                for (int i = l0 + threadIdx.x; i < l1; i += kThreads)
                    if (near(score[i])) sh.list_page[atomicAdd(&sh.list_n, 1)] = my.p0 + i;
                __syncthreads();
                for (int k = warp; k < sh.list_n; k += kWarps) {
                    const double x = my.exact(sh, sh.list_page[k], lane);
                    if (lane == 0) sh.list_score[k] = x;
                }
                cl.sync();
                if (threadIdx.x < sh.list_n) {
                    const int page = sh.list_page[threadIdx.x];
                    const double x = sh.list_score[threadIdx.x];
                    int better = 0;
                    for (int k = 0; k < C; ++k) {
                        const int m = *cl.map_shared_rank(&sh.list_n, k);
                        const int* pages = cl.map_shared_rank(&sh.list_page[0], k);
                        const double* xs = cl.map_shared_rank(&sh.list_score[0], k);
                        for (int i = 0; i < m; ++i) better += xs[i] > x || (xs[i] == x && pages[i] < page);
                    }
                    score[page - my.p0] = better < places ? INFINITY : -INFINITY;
                }
                tie_places = 0;
            } else {
                // many pages that near (the same text again and again): a radix selection on the bits of the fp64
                // scores, worked out again for each digit
                uint64_t top = 0;
                need = places;
                for (int d = 0; d < 8; ++d) {
                    const int shift = 56 - 8 * d;
                    cl.sync();   // the last digit's histogram has been read
                    for (int i = threadIdx.x; i < 256; i += kThreads) sh.hist[0][i] = 0;
                    __syncthreads();
                    for (int i = l0 + warp; i < l1; i += kWarps) {
                        if (!near(score[i])) continue;
                        const uint64_t k = key64(my.exact(sh, my.p0 + i, lane));
                        if (lane == 0 && (d == 0 || k >> (shift + 8) == top)) atomicAdd(&sh.hist[0][(k >> shift) & 255u], 1u);
                    }
                    find_bin(cl, sh, sh.hist[0], need, bin, rest);
                    top = (top << 8) | uint32_t(bin);
                    need = rest;
                }
                for (int i = l0 + warp; i < l1; i += kWarps) {
                    if (!near(score[i])) continue;
                    const uint64_t k = key64(my.exact(sh, my.p0 + i, lane));
                    __syncwarp();
                    if (lane == 0) score[i] = k > top ? INFINITY : k < top ? -INFINITY : kTie;
                    __syncwarp();
                }
                tie_places = need;
            }
        }
        __syncthreads();
        if (tie_places > 0) {   // the same in every CTA
            const int per = (my.n + kThreads - 1) / kThreads, a = min(int(threadIdx.x) * per, my.n), b = min(a + per, my.n);
            int t = 0, total;
            for (int i = max(a, l0); i < min(b, l1); ++i) t += score[i] != score[i];
            int before = block_scan(t, sh.scan, total);
            if (threadIdx.x == 0) sh.ties = total;
            cl.sync();
            for (int k = 0; k < rank; ++k) before += *cl.map_shared_rank(&sh.ties, k);
            for (int i = max(a, l0); i < min(b, l1); ++i)
                if (score[i] != score[i]) score[i] = before++ < tie_places ? INFINITY : -INFINITY;
        }
        __syncthreads();
    }

    // ---- the list, in rising order
    {
        const int per = (my.n + kThreads - 1) / kThreads, a = min(int(threadIdx.x) * per, my.n), b = min(a + per, my.n);
        auto in = [&](int i) {
            const float x = score[i];
            return i < l0 || i >= l1 || above(x) || (whole ? near(x) : x == INFINITY);
        };
        int t = 0, total;
        for (int i = a; i < b; ++i) t += in(i);
        int at = block_scan(t, sh.scan, total);
        if (threadIdx.x == 0) sh.taken = total;
        cl.sync();
        for (int k = 0; k < rank; ++k) at += *cl.map_shared_rank(&sh.taken, k);
        for (int i = a; i < b; ++i)
            if (in(i)) {
                if (at < p.max_pages) list[at] = my.p0 + i;
                ++at;
            }
    }
    cl.sync();   // no CTA leaves while another reads its shared memory
}

// The kernel may take kSelectSmem of shared memory: said once per kernel and device.
template <typename T, int D>
cudaError_t launch_select_d(const SelectParams& p, int cluster, size_t smem, cudaStream_t st) {
    static PerDevice ready;
    int dev = 0, one = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = cudaError_t(ready.get(dev, &one, [](int* v) {
        *v = 1;
        return int(cudaFuncSetAttribute(select_pages_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelectSmem));
    }));
    if (e != cudaSuccess) return e;
    return launch_cluster_kernel(select_pages_kernel<T, D>, dim3(unsigned(int64_t(p.num_rows) * cluster), p.num_kv_heads),
                                 dim3(kThreads), unsigned(cluster), smem, st, p);
}

template <typename T>
cudaError_t launch_select_t(const SelectParams& p, int cluster, size_t smem, cudaStream_t st) {
    return p.head_dim == 128 ? launch_select_d<T, 128>(p, cluster, smem, st) : launch_select_d<T, 64>(p, cluster, smem, st);
}

}  // namespace

cudaError_t launch_key_bounds(const KeyBoundsParams& p, int cache_kind, cudaStream_t stream) {
    const int chunks = p.num_kv_heads * p.head_dim * (cache_kind == PKV_CACHE_F16 || cache_kind == PKV_CACHE_BF16 ? 2 : 1) / 16;
    int64_t pages = p.max_blocks;
    if (!p.cu_new && (p.q_len + 14) / kBlockSize + 1 < pages) pages = (p.q_len + 14) / kBlockSize + 1;
    int64_t ctas = (pages * chunks + kBoundsThreads - 1) / kBoundsThreads;
    // lengths that only the device knows: enough CTAs to fill the GPU
    const int64_t most = (2048 + p.num_seqs - 1) / p.num_seqs;
    if (p.cu_new && ctas > most) ctas = most;
    const dim3 grid(unsigned(ctas < 65535 ? ctas : 65535), p.num_seqs), block(kBoundsThreads);
    switch (cache_kind) {
        case PKV_CACHE_F16: return launch_kernel(key_bounds_kernel<__half>, grid, block, 0, stream, p);
        case PKV_CACHE_BF16: return launch_kernel(key_bounds_kernel<__nv_bfloat16>, grid, block, 0, stream, p);
        case PKV_CACHE_I8: return launch_kernel(key_bounds_kernel<I8>, grid, block, 0, stream, p);
        case PKV_CACHE_E4M3: return launch_kernel(key_bounds_kernel<E4M3>, grid, block, 0, stream, p);
        default: return launch_kernel(key_bounds_kernel<K8>, grid, block, 0, stream, p);
    }
}

cudaError_t launch_select_pages(const SelectParams& p, int cache_kind, cudaStream_t stream) {
    const int64_t pairs = int64_t(p.num_rows) * p.num_kv_heads;
    int C = 1;
    while (C < kMaxCluster && pairs * C < 304 && p.max_blocks / (2 * C) >= 64) C *= 2;
    while (C < kMaxCluster && int64_t(p.max_blocks + C - 1) / C * 4 > kSelectSmem) C *= 2;
    const size_t smem = (size_t(p.max_blocks) + C - 1) / C * 4;
    if (smem > kSelectSmem || int64_t(p.num_rows) * C > 0x7fffffff) return cudaErrorInvalidValue;
    switch (cache_kind) {
        case PKV_CACHE_BF16: return launch_select_t<__nv_bfloat16>(p, C, smem, stream);
        case PKV_CACHE_I8: return launch_select_t<I8>(p, C, smem, stream);
        case PKV_CACHE_E4M3: return launch_select_t<E4M3>(p, C, smem, stream);
        default: return launch_select_t<__half>(p, C, smem, stream);   // fp16 caches, and K8V4's fp16 bounds
    }
}

}  // namespace pkv
