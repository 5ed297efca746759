// select_pages.cuh -- the selection of the pages that a query token attends, by the
// bounds of their keys (a page is a cache block, 16 tokens).
//
// Score of a page for a query token and a kv head, over the head's G query heads:
//   sum_h sum_d max(q_hd lo_d, q_hd hi_d) = sum_d [ n_d lo_d + p_d hi_d ],
//   n_d = sum_h min(q_hd, 0),  p_d = sum_h max(q_hd, 0)
// since the maximum takes hi where q is positive and lo where it is negative: one
// product of length 2 D whatever the group, and the queries are folded once.
//
// The selection is that of the exact scores.  They are worked out by 16-bit MMAs with
// fp32 sums, with a bound e on their error; T, the k-th largest of them, is found; a page
// above T + 2 e is in, one below T - 2 e is out (score_error.h), and only if more pages lie between than
// there are places left are those pages' scores worked out again in fp64 (the products
// are exact there), which runs at a sixtieth of the fp32 rate on this GPU.
#pragma once

#include <cooperative_groups.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "attention_byte.cuh"
#include "pkv_rows.cuh"
#include "score_error.h"

namespace cg = cooperative_groups;

namespace pkv {

// What the bounds hold: __half, __nv_bfloat16, or the codes of an 8-bit cache.
struct I8 {};
struct E4M3 {};

namespace {

constexpr int kMaxCluster = 8;

// Sum of two pairs of 16-bit floats.
template <bool BF>
__device__ __forceinline__ uint32_t add2(uint32_t a, uint32_t b) {
    using V = typename std::conditional<BF, __nv_bfloat162, __half2>::type;
    V x, y;
    memcpy(&x, &a, 4);
    memcpy(&y, &b, 4);
    const V z = __hadd2(x, y);
    uint32_t r;
    memcpy(&r, &z, 4);
    return r;
}

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

// How the bounds' numbers enter the MMAs.  The folded queries are fp32 and taken in two 16-bit terms, in two columns of
// the operand: bf16 (16 bits together) or, for fp16 and the 8-bit codes, which fp16 holds exactly, fp16 (22 bits),
// scaled by a power of two for each row.
template <typename T, int D>
struct ScoreMath {
    static constexpr bool kHalf = std::is_same<T, __half>::value || std::is_same<T, __nv_bfloat16>::value;
    static constexpr bool kBf = std::is_same<T, __nv_bfloat16>::value;
    static constexpr int E = kHalf ? 2 : 1;         // bytes of a number
    static constexpr int NKC = D * E / 64;          // 16-byte chunks of a lo or hi row that a thread takes
    static constexpr int NKS = D / 16;              // k steps of lo, and of hi

    // first of the four dims that lane position t has in k step ks: (0, 1) in one word, (2, 3) in the other
    static __device__ __forceinline__ int dim(int ks, int t) {
        return kHalf ? 32 * (ks >> 1) + 8 * t + 4 * (ks & 1) : 64 * (ks >> 2) + 16 * t + 4 * (ks & 3);
    }
    static __device__ __forceinline__ void widen(uint32_t w, uint32_t& a, uint32_t& b) {
        if constexpr (std::is_same<T, E4M3>::value) e4m3x4_to_f16(w, a, b);
        else s8x4_to_f16x4(w, a, b);
    }
    static constexpr int SPC = NKS / NKC;           // k steps of a chunk
    // the operand words of a chunk's k step j of pages g and g + 8
    static __device__ __forceinline__ void operand(const uint4 (&x)[2], int j, uint32_t (&a)[4]) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            if constexpr (kHalf) {
                a[r] = j ? x[r].z : x[r].x;
                a[2 + r] = j ? x[r].w : x[r].y;
            } else {
                widen(j == 0 ? x[r].x : j == 1 ? x[r].y : j == 2 ? x[r].z : x[r].w, a[r], a[2 + r]);
            }
        }
    }
    // a bound's number; SKIP: 0 in the place of an infinity that `skip` says has a weight of 0 (the maximum took the other bound)
    template <bool SKIP = false>
    static __device__ __forceinline__ double one(const void* base, int64_t i, bool skip = false) {
        if constexpr (kHalf) {
            uint16_t u = static_cast<const uint16_t*>(base)[i];
            if (SKIP && skip && (u & 0x7fffu) == (kBf ? 0x7f80u : 0x7c00u)) u = 0;
            return double(Half16<T>::to_float(u));
        }
        else if constexpr (std::is_same<T, I8>::value) return double(static_cast<const int8_t*>(base)[i]);
        else return double(__half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(base)[i], __NV_E4M3))));
    }
};

// Where a row's selection stands: the bins in which its want-th largest score lies, level by level.
constexpr int kLevels = 3;
struct RowState {
    float lo[kLevels], inv[kLevels];
    int bin[kLevels];
    int levels, need;       // levels that are done; the place within the last bin, from 1
    int in_bin;
    int lowest;             // the lowest bin at every level
    float e2;               // twice the bound on a score's error
    float above, below;     // pages above `above` are in; those below `below` are out
    float slack;            // how far the levels' roundings may have moved a bin's edge
    int r, n, vis;          // the row, its pages, its tokens
    int slow;               // left to the slow way
    int zero;               // no magnitude that fp32 holds: queries or bounds of zeros, or products that underflow
    int taken;              // near pages that are in (sel)
};

// ROWS query tokens to a CTA; CL: in clusters.
template <int ROWS, int NW, bool CL>
struct SelectShared {
    static constexpr int R = ROWS, kWarps = NW, kThreads = 32 * NW;
    static constexpr int NB = R <= 4 ? 256 : 128;    // bins of a level
    static constexpr int LT = R <= 4 ? 128 : 64;     // pages near the border that are ranked by each other
    RowState row[R];
    float back[R];                  // what a row's scaled sums are multiplied by
    uint32_t wmax[R];               // largest folded query (fp32 bits)
    uint32_t smin[R], smax[R];      // keys of the smallest (but -inf) and largest score
    uint32_t amax[R];               // largest sum of magnitudes (fp32 bits)
    alignas(8) uint32_t hist[R][NB];
    uint32_t hsum[CL ? R : 1][NB];      // of all CTAs
    int above[R][kWarps];           // pages above the border in each warp's part
    int list_n[R];
    int list_page[R][LT];
    float list_score[R][LT];
    int all_page[CL ? R : 1][LT];       // the lists of all CTAs
    float all_score[CL ? R : 1][LT];
    int sel[R][LT];                 // near pages that are in
    int scan[kWarps];
    int bin, rest, in_bin, ties, taken, count_a, some;
};

__device__ __forceinline__ int bin_of(float x, float lo, float inv, int bins) {
    return min(max(__float2int_rz((x - lo) * inv), 0), bins - 1);   // not a number: 0
}

// Whether x lies in the bins chosen so far.
template <int NB>
__device__ __forceinline__ bool in_bins(const RowState& s, float x) {
    for (int l = 0; l < s.levels; ++l)
        if (bin_of(x, s.lo[l], s.inv[l], NB) != s.bin[l]) return false;
    return true;
}

// x[k], x[k + 32], x[k + 64] and x[k + 96], as far as they lie in front of `end`.
__device__ __forceinline__ void read4(const float* x, int k, int end, float (&v)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = k + 32 * j < end ? x[k + 32 * j] : -INFINITY;
}

// Exclusive prefix sum of v over the CTA's threads; the total in `total`.
template <int kWarps>
__device__ __forceinline__ int block_scan(int v, int (&warps)[kWarps], int& total) {
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

__device__ __forceinline__ void team_sync(cg::cluster_group& cl, int C) {
    if (C > 1) cl.sync();
    else __syncthreads();
}

// The scores in fp64 of the pages in blocks b0 and b1 (out of range: none), whose loads and sums do not wait for one another, by a
// warp whose lanes hold the folded queries of dims lane, lane + 32, .. of lo, then of hi: the first's in lanes 0-15, the
// second's in the others.  INF: bounds may be infinite.
template <typename T, int D, bool INF>
__device__ __forceinline__ double exact_scores(const SelectParams& p, const double (&w)[2 * D / 32], int kvh, int b0, int b1, int lane) {
    using Math = ScoreMath<T, D>;
    const bool ok0 = b0 >= 0 && b0 < p.num_blocks, ok1 = b1 >= 0 && b1 < p.num_blocks, second = lane >= 16;
    const int64_t h0 = int64_t(ok0 ? b0 : 0) * p.num_kv_heads + kvh, h1 = int64_t(ok1 ? b1 : 0) * p.num_kv_heads + kvh;
    double x = 0.0, y = 0.0;
#pragma unroll
    for (int k = 0; k < 2 * D / 32; ++k) {
        const bool none = INF && (__double_as_longlong(w[k]) << 1) == 0;   // a weight of 0
        x = fma(w[k], Math::template one<INF>(p.bounds, h0 * 2 * D + lane + 32 * k, none), x);
        y = fma(w[k], Math::template one<INF>(p.bounds, h1 * 2 * D + lane + 32 * k, none), y);
    }
    const double other = __shfl_xor_sync(0xffffffffu, second ? x : y, 16);
    x = (second ? y : x) + other;
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (Math::E == 1) x *= double(p.k_scale[second ? h1 : h0]);
    return (second ? ok1 : ok0) && x == x ? x : -INFINITY;
}
// fp32's a + b is s + e exactly.
__device__ __forceinline__ float two_sum(float a, float b, float& e) {
    const float s = a + b, z = s - a;
    e = (a - (s - z)) + (b - z);
    return s;
}
// The folded queries in fp64.  A sum of up to 8 numbers of 16 bits nearly always is two fp32 numbers exactly, which takes a tenth
// of the time that fp64 does; else (a remainder of the remainders, or nothing finite) it is worked out in fp64.
template <int D>
__device__ __forceinline__ void exact_weights(const SelectParams& p, int r, int kvh, int lane, double (&w)[2 * D / 32]) {
    const int G = p.num_heads / p.num_kv_heads;
    const int64_t q0 = (int64_t(r) * p.num_heads + int64_t(kvh) * G) * D + lane;
    float hi[2 * D / 32], lo[2 * D / 32];
    bool more = false, small = false;
#pragma unroll
    for (int k = 0; k < 2 * D / 32; ++k) hi[k] = lo[k] = 0.f;
#pragma unroll 4
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int k = 0; k < 2 * D / 32; ++k) {
            const float q = load_q(p.q, p.q_dtype, q0 + int64_t(g) * D + 32 * (k % (D / 32)));
            float e, rest;
            hi[k] = two_sum(hi[k], (k < D / 32 ? q < 0.f : q > 0.f) ? q : 0.f * q, e);   // not a number stays so
            lo[k] = two_sum(lo[k], e, rest);
            more |= rest != 0.f;
        }
#pragma unroll
    for (int k = 0; k < 2 * D / 32; ++k) {
        w[k] = double(hi[k]);
        small |= lo[k] != 0.f;
    }
    if (__any_sync(0xffffffffu, small))
#pragma unroll
        for (int k = 0; k < 2 * D / 32; ++k) w[k] += double(lo[k]);
    if (!__any_sync(0xffffffffu, more)) return;
#pragma unroll
    for (int k = 0; k < 2 * D / 32; ++k) {
        w[k] = 0.0;
        for (int g = 0; g < G; ++g) {
            const float q = load_q(p.q, p.q_dtype, q0 + int64_t(g) * D + 32 * (k % (D / 32)));
            w[k] += (k < D / 32 ? q < 0.f : q > 0.f) ? q : 0.f * q;
        }
    }
}

// A row's selection in the general way, all CTAs together: T, the want-th largest fp32 score, by a radix selection on
// its bits; the pages between T - e2 and T + e2 by the same on the high words of their fp64 scores, and those whose high word is
// the border's on the low words, worked out again; ties by page.  For rows with hundreds of pages that near (the same text again
// and again, nothing but zeros, products that underflow) and for magnitudes that are not finite.  open: a bit for each of this
// CTA's pages.  zeros: whether all pages' bounds are 0; -1: not looked at yet.
// Bound: fp64, a row and page at a time.  All pages alike, 8 bf16 kv heads of 128 dims: 1 sequence of 512 92 us, 32 of up to 2048
// 1.76 ms, 1401 tokens over up to 1024 29 ms; an infinite bound a sequence 50 us, 0.9 and 14.5 ms; queries of zeros 21, 54, 506 us.
template <typename T, int D, bool CL, typename Sh>
__device__ __noinline__ void select_slow(const SelectParams& p, cg::cluster_group& cl, Sh& sh, const RowState& row, int seq, int kvh,
                                         float* score, uint32_t* open, int p0, int np, int& zeros, int32_t* list) {
    const int C = CL ? int(cl.num_blocks()) : 1, rank = CL ? int(cl.block_rank()) : 0, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kThreads = Sh::kThreads, kWarps = Sh::kWarps;
    const int n = row.n, want = p.max_pages - p.keep_first - p.keep_last;
    const float e2 = row.e2;
    const int mine = max(0, min(np, n - p0));   // this CTA's pages of the row
    const int l0 = min(max(p.keep_first - p0, 0), mine), l1 = max(min(n - p.keep_last - p0, mine), l0);
    uint32_t* const raw = reinterpret_cast<uint32_t*>(score);
    uint32_t* hist = &sh.hist[0][0];   // 128 bins or more; 7 bits a digit
    constexpr int BITS = 7, BINS = 1 << BITS;
    int need = want, in_bin = 0;   // the place among the numbers that equal the one found, and how many do
    // the need-th largest of the keys of pages that are counted
    auto radix = [&](auto counted, auto key) {
        uint32_t prefix = 0;
        for (int shift = 28; shift >= 0; shift -= BITS) {   // 4 bits, then 7 at a time
            team_sync(cl, C);   // the last histogram has been read
            for (int i = threadIdx.x; i < BINS; i += kThreads) hist[i] = 0;
            __syncthreads();
            for (int i = l0 + threadIdx.x; i < l1; i += kThreads) {
                if (!counted(i)) continue;
                const uint32_t k = key(i);
                if (shift == 28 || k >> (shift + BITS) == prefix) atomicAdd(&hist[(k >> shift) & (BINS - 1)], 1u);
            }
            team_sync(cl, C);
            // the bin, from the top, that holds the need-th number, and the place in it
            const int b = BINS - 1 - int(threadIdx.x);
            int c = 0;
            if (b >= 0)
                for (int k = 0; k < C; ++k) c += int(cl.map_shared_rank(hist, k)[b]);
            int total;
            const int before = block_scan(c, sh.scan, total);
            if (before < need && before + c >= need) {
                sh.bin = b;
                sh.rest = need - before;
                sh.in_bin = c;
            }
            __syncthreads();
            prefix = (prefix << BITS) | uint32_t(sh.bin);
            need = sh.rest;
            in_bin = sh.in_bin;
        }
        return prefix;
    };
    // with a bound that is not finite every page is near, and T is not needed
    const float T0 = e2 < INFINITY ? from_key32(radix([](int) { return true; }, [&](int i) { return key32(score[i]); })) : 0.f;
    const float up = T0 + e2, down = T0 - e2;
    auto near = [&](float x) { return !(x > up) && !(x < down); };
    if (threadIdx.x == 0) sh.count_a = 0;
    __syncthreads();
    int a = 0;
    for (int i = l0 + threadIdx.x; i < l1; i += kThreads) a += score[i] > up;
    if (a) atomicAdd(&sh.count_a, a);
    team_sync(cl, C);
    need = want;   // places for the pages between
    for (int k = 0; k < C; ++k) need -= *cl.map_shared_rank(&sh.count_a, k);
    // a page is marked: in +inf, out -inf, NaN if it ties with the border and the lower page goes first
    constexpr float kTie = NAN;
    double w64[2 * D / 32];
    exact_weights<D>(p, row.r, kvh, lane, w64);
    bool none = false, any = false;   // a query that is not finite: every score is not a number
#pragma unroll
    for (int k = 0; k < 2 * D / 32; ++k) {
        none |= w64[k] != w64[k];
        any |= w64[k] != 0.0;
    }
    any = __any_sync(0xffffffffu, any);
    const int32_t* table = p.block_tables + int64_t(seq) * p.max_blocks + p0;
    if (any && row.zero && zeros < 0) {
        constexpr int E = ScoreMath<T, D>::E;
        if (threadIdx.x == 0) sh.some = 0;
        __syncthreads();
        bool some = false;
        constexpr uint32_t kSigns = E == 2 ? 0x7fff7fffu : std::is_same<T, E4M3>::value ? 0x7f7f7f7fu : 0xffffffffu;   // all but them
        for (int i0 = 8 * warp; i0 < np; i0 += 8 * kWarps) {   // eight pages' loads in flight
            int pb[8];
            uint4 v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) pb[j] = i0 + j < np ? table[i0 + j] : -1;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = pb[j] >= 0 && pb[j] < p.num_blocks && lane < 2 * D * E / 16
                           ? __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.bounds) +
                                                                  (int64_t(pb[j]) * p.num_kv_heads + kvh) * 2 * D * E) + lane)
                           : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int j = 0; j < 8; ++j) some |= ((v[j].x | v[j].y | v[j].z | v[j].w) & kSigns) != 0;
        }
        if (some) sh.some = 1;
        team_sync(cl, C);
        zeros = 1;
        for (int k = 0; k < C; ++k) zeros &= *cl.map_shared_rank(&sh.some, k) == 0;
    }
    // queries or bounds of zeros: every score is 0, but where a bound is not finite, and e2 then neither
    if (__any_sync(0xffffffffu, none) || (e2 < INFINITY && (!any || (row.zero && zeros)))) {   // every score near the border is the same
        for (int i = l0 + threadIdx.x; i < l1; i += kThreads) score[i] = near(score[i]) ? kTie : score[i] > up ? INFINITY : -INFINITY;
    } else {
        // pages that stay open by f(i), the others marked by g(i); a word's pages to a warp
        auto close = [&](auto f, auto g) {
            for (int i0 = (l0 & ~31) + 32 * warp; i0 < l1; i0 += 32 * kWarps) {
                const int i = i0 + lane;
                const bool there = i >= l0 && i < l1, stays = there && f(i);
                if (there && !stays) score[i] = g(i);
                const uint32_t word = __ballot_sync(0xffffffffu, stays);
                if (lane == 0) open[i0 / 32] = word;
            }
            __syncthreads();
        };
        auto is_open = [&](int i) { return (open[i >> 5] >> (i & 31) & 1u) != 0; };
        // the words of the open pages' fp64 scores, two pages at a time
        auto exact = [&](int shift) {
            for (int i = l0 + 2 * warp; i < l1; i += 2 * kWarps) {
                const bool first = is_open(i), second = i + 1 < l1 && is_open(i + 1);
                if (!first && !second) continue;
                const double d = exact_scores<T, D, true>(p, w64, kvh, first ? table[i] : -1, second ? table[i + 1] : -1, lane);
                if ((lane & 15) == 0 && (lane ? second : first)) raw[i + (lane >> 4)] = uint32_t(key64(d) >> shift);
            }
            __syncthreads();
        };
        auto word = [&](int i) { return raw[i]; };
        close([&](int i) { return near(score[i]); }, [&](int i) { return score[i] > up ? INFINITY : -INFINITY; });
        exact(32);
        const uint32_t high = radix(is_open, word);
        const bool all = in_bin == need;   // of the pages with the border's high word
        close([&](int i) { return is_open(i) && raw[i] == high; },
              [&](int i) { return is_open(i) ? raw[i] > high ? INFINITY : -INFINITY : score[i]; });
        uint32_t low = 0;
        if (!all) {
            exact(0);
            low = radix(is_open, word);
        }
        close([](int) { return false; }, [&](int i) {
            return !is_open(i) ? score[i] : all || raw[i] > low ? INFINITY : raw[i] < low ? -INFINITY : kTie;
        });
    }
    const int tie_places = need;
    __syncthreads();
    // a thread takes neighbouring pages, so that both prefix sums below go by page
    const int per = (mine + kThreads - 1) / kThreads, b0 = min(int(threadIdx.x) * per, mine), b1 = min(b0 + per, mine);
    int c = 0, total;
    for (int i = max(b0, l0); i < min(b1, l1); ++i) c += score[i] != score[i];
    int before = block_scan(c, sh.scan, total);
    if (threadIdx.x == 0) sh.ties = total;
    team_sync(cl, C);
    for (int k = 0; k < rank; ++k) before += *cl.map_shared_rank(&sh.ties, k);
    for (int i = max(b0, l0); i < min(b1, l1); ++i)
        if (score[i] != score[i]) score[i] = before++ < tie_places ? INFINITY : -INFINITY;
    auto in = [&](int i) { return i < l0 || i >= l1 || score[i] == INFINITY; };
    c = 0;
    for (int i = b0; i < b1; ++i) c += in(i);
    int at = block_scan(c, sh.scan, total);
    if (threadIdx.x == 0) sh.taken = total;
    team_sync(cl, C);
    for (int k = 0; k < rank; ++k) at += *cl.map_shared_rank(&sh.taken, k);
    for (int i = b0; i < b1; ++i)
        if (in(i)) {
            if (at < p.max_pages) list[at] = p0 + i;
            ++at;
        }
}

// A cluster of 1 to 8 CTAs takes a tile of up to 4 NT query tokens of one sequence and a kv head.
//   Scores: pages on the MMA's M side, query tokens on N.  A warp takes 16 pages at a time straight from global
//   memory into the operand (the order of a contraction's terms is free: a thread takes 16 contiguous bytes); a CTA
//   takes a contiguous share of the pages and keeps the scores in its shared memory.
//   Selection, by the warps of all CTAs, a row for each or several warps to a row: a histogram between the
//   smallest and the largest score, the bin of the border, and again inside it while it holds many; the pages
//   in it, and those that the error may have moved across its edges, are ranked by each other.
// Bound: a wave of CTAs whose loads do not cover HBM's latency: two to an SM, 64 registers of a thread in flight.  32 sequences of
// 2048 bf16 pages, 8 heads of 128 dims, take 54.3 us for 269 MB, 6 of them before the first loads and 3 of selection: 5.9 TB/s
// between; of 512 to 2048 pages (172 MB) 44.5 us, the time of the longest ones' CTAs, 4.8 TB/s between, DRAM 43 % busy over
// the whole.  Few or long sequences: the clusters' barriers, about 1 us each with what is read across (1 x 512 pages 11.6 us; 4 x
// 8192 int8 pages, 2 tokens, 33.5 us, 52 MB), and fp64 where pages next to the border need it, 3 us.  Chunks of prompts: the
// MMAs and their operands' latency, half of the time, and the bins and lists of 16 rows (1401 tokens over up to 1024 pages, 126 us).
template <typename T, int D, int NT, int NW, bool CL>
__global__ void __launch_bounds__(32 * NW, 16 / NW) select_pages_kernel(SelectParams p) {
    using Math = ScoreMath<T, D>;
    using Sh = SelectShared<4 * NT, NW, CL>;
    constexpr int R = Sh::R, NB = Sh::NB, LT = Sh::LT, NKS = Math::NKS, kThreads = Sh::kThreads, kWarps = Sh::kWarps;
    constexpr int MT = (R + 7) / 8;                   // column tiles of the magnitudes: a column to a row
    extern __shared__ __align__(16) uint8_t dyn[];
    __shared__ Sh sh;
    uint2* const W = reinterpret_cast<uint2*>(dyn);   // [2 NKS][NT][32 lanes]: columns 2 i, 2 i + 1 are row i's terms
    uint2* const WM = W + 2 * NKS * NT * 32;          // [NKS][MT][32 lanes]: the larger magnitude of both parts
    float* const scores = reinterpret_cast<float*>(WM + NKS * MT * 32);   // [tile_rows][stride]
    const int words = (p.stride + 31) / 32;
    uint32_t* const bits = reinterpret_cast<uint32_t*>(scores + p.tile_rows * p.stride);   // [tile_rows][words]: pages that are in
    cg::cluster_group cl = cg::this_cluster();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int C = CL ? int(cl.num_blocks()) : 1, rank = CL ? int(cl.block_rank()) : 0;
    // No grid_dep_launch(): with it the next kernels' starts, ahead of this one's end, changed no time.
    grid_dep_wait();
    const int kvh = blockIdx.y, G = p.num_heads / p.num_kv_heads;
    const RowTile tile = find_tile(p.cu_q, p.num_seqs, p.num_rows, p.q_len, p.tile_rows, int(blockIdx.x / C), lane);
    if (tile.s < 0) return;   // the same in every CTA of the cluster
    const int rows = tile.rows;
    const int64_t ctx = p.context_lens[tile.s];
    const int behind0 = (p.cu_q ? min(p.cu_q[tile.s + 1], p.num_rows) : (tile.s + 1) * p.q_len) - tile.r0;   // rows from the first on
    if (ctx > int64_t(p.max_blocks) * kBlockSize && rank == 0 && kvh == 0 && threadIdx.x == 0) flag_error(p.err, PKV_DEVERR_CAPACITY);
    auto pages_of = [&](int i) { return (visible_tokens(ctx, p.max_blocks, behind0 - i) + kBlockSize - 1) / kBlockSize; };
    const int n_max = pages_of(rows - 1);   // the last row sees most
    auto out_list = [&](int i) { return p.lists + ((int64_t(tile.r0) + i) * p.num_kv_heads + kvh) * p.max_pages; };

    // ---- rows that take every page
    int first_row = 0;   // the first that does not: rows see more and more
    while (first_row < rows && pages_of(first_row) <= p.max_pages) ++first_row;
    for (int i = rank * kWarps + warp; i < rows; i += C * kWarps) {
        const int n = pages_of(i);
        if (lane == 0) p.counts[(int64_t(tile.r0) + i) * p.num_kv_heads + kvh] = min(n, p.max_pages);
        if (i < first_row)
            for (int k = lane; k < p.max_pages; k += 32) out_list(i)[k] = k < n ? k : -1;
    }
    if (first_row >= rows) return;
    const int share = ((n_max + C - 1) / C + 15) & ~15;
    const int p0 = min(rank * share, n_max), np = min(share, n_max - p0);   // this CTA's pages [p0, p0 + np)

    // ---- where the bounds come from
    const int32_t* table = p.block_tables + int64_t(tile.s) * p.max_blocks + p0;
    // block of page i0 + lane (lanes 0 .. 15); it is looked at a tile's time later, when it has come
    auto entry = [&](int i0) { return lane < 16 && i0 + lane < np ? table[i0 + lane] : -1; };
    struct Source {               // where pages g and g + 8 of a tile come from
        const uint8_t* at[2];     // null: not a page
        float scale[2];           // 8-bit caches
    };
    auto source = [&](int pb, int i0) {
        Source f;
        if (pb < 0 || pb >= p.num_blocks) {
            if (lane < 16 && i0 + lane < np) flag_error(p.err, PKV_DEVERR_OOB_BLOCK);
            pb = -1;
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int b = __shfl_sync(0xffffffffu, pb, g + 8 * r);
            const int64_t head = int64_t(b) * p.num_kv_heads + kvh;
            f.at[r] = b >= 0 ? static_cast<const uint8_t*>(p.bounds) + head * 2 * D * Math::E + 16 * t : nullptr;
            f.scale[r] = Math::E == 1 && b >= 0 ? __ldg(p.k_scale + head) : 1.f;
        }
        return f;
    };
    // chunks of lo and hi, of pages g and g + 8: all of a tile's, or (16 rows, for the registers) two ahead
    constexpr int AHEAD = NT == 1 || Math::NKC < 2 ? Math::NKC : 2;
    uint4 x[AHEAD][2][2];
    auto load = [&](const Source& f, int c) {
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int r = 0; r < 2; ++r)
                x[c % AHEAD][part][r] = f.at[r] ? __ldg(reinterpret_cast<const uint4*>(f.at[r] + part * D * Math::E + 64 * c))
                                        : make_uint4(0u, 0u, 0u, 0u);
    };
    // ---- the queries, folded
    if (threadIdx.x < R) {
        const int i = threadIdx.x;
        sh.wmax[i] = sh.smax[i] = sh.amax[i] = 0;
        sh.smin[i] = 0xffffffffu;
        sh.list_n[i] = 0;
        RowState& s = sh.row[i];
        s.r = tile.r0 + i;
        s.n = i < rows ? pages_of(i) : 0;
        s.levels = s.slow = s.taken = 0;
        s.in_bin = INT_MAX;
        s.need = p.max_pages - p.keep_first - p.keep_last;
    }
    for (int i = threadIdx.x; i < R * NB; i += kThreads) (&sh.hist[0][0])[i] = 0;
    // a thread takes four dims of a row: item = (k step, row, lane position)
    constexpr int ITEMS = NKS * R * 4, PER = (ITEMS + kThreads - 1) / kThreads;
    float w[PER][8];   // the sums of four dims' negative parts, then of their positive parts
    const int entry0 = entry(warp * 16);
    uint2 qv[NT == 1 ? PER : 1][8];   // a few rows: the queries' loads go first, then the first tile's bounds, then the sums
    auto queries = [&](int k, int h) {
        const int item = threadIdx.x + k * kThreads, tt = item & 3, i = (item >> 2) % R, ks = (item >> 2) / R;
        if (item >= ITEMS || i >= rows || h >= G) return make_uint2(0u, 0u);
        return __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.q) + ((int64_t(tile.r0) + i) * p.num_heads +
                                                                                         int64_t(kvh) * G + h) * D + Math::dim(ks, tt)));
    };
    if constexpr (NT == 1)
#pragma unroll
        for (int k = 0; k < PER; ++k)
#pragma unroll
            for (int h = 0; h < 8; ++h) qv[k][h] = queries(k, h);
    Source now = source(entry0, warp * 16);
    if constexpr (NT == 1)
#pragma unroll
        for (int c = 0; c < AHEAD; ++c) load(now, c);
    int next = entry((warp + kWarps) * 16);
#pragma unroll
    for (int k = 0; k < PER; ++k) {
#pragma unroll
        for (int d = 0; d < 8; ++d) w[k][d] = 0.f;
#pragma unroll
        for (int h = 0; h < 8; ++h) {
            if (h >= G) break;
            const uint2 v = NT == 1 ? qv[NT == 1 ? k : 0][h] : queries(k, h);
            float2 a, b;
            if (p.q_dtype == PKV_BF16) {
                a = Half16<__nv_bfloat16>::unpack2(v.x);
                b = Half16<__nv_bfloat16>::unpack2(v.y);
            } else {
                a = Half16<__half>::unpack2(v.x);
                b = Half16<__half>::unpack2(v.y);
            }
            const float f[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                w[k][d] += f[d] < 0.f ? f[d] : 0.f * f[d];   // not a number stays so
                w[k][4 + d] += f[d] > 0.f ? f[d] : 0.f * f[d];
            }
        }
    }
    if (!Math::kBf) {
        __syncthreads();   // wmax is cleared
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int item = threadIdx.x + k * kThreads, i = (item >> 2) % R;
            uint32_t m = 0;
#pragma unroll
            for (int d = 0; d < 8; ++d) m = max(m, __float_as_uint(fabsf(w[k][d])));
            if (item < ITEMS && i < rows) atomicMax(&sh.wmax[i], m);
        }
        __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int item = threadIdx.x + k * kThreads, tt = item & 3, i = (item >> 2) % R, ks = (item >> 2) / R;
        if (item >= ITEMS) break;
        float up = 1.f;
        if (!Math::kBf) {   // the row's largest to [2^14, 2^15)
            const uint32_t ex = min(max(sh.wmax[i] >> 23, 15u), 254u);
            up = __uint_as_float((268u - ex) << 23);
            if (ks == 0 && tt == 0) sh.back[i] = __uint_as_float((ex - 14u) << 23);
        }
        float most[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            most[d] = fmaxf(fabsf(w[k][d]), fabsf(w[k][4 + d])) * up;
            // fp16's second term is off by 2^-25 at most, however small the weight: 2^-18 of the magnitude counted for it
            if (!Math::kBf && sh.wmax[i] > 0) most[d] = most[d] < 0.0078125f ? 0.0078125f : most[d];   // a NaN stays
        }
        WM[(ks * MT + i / 8) * 32 + (i % 8) * 4 + tt] = make_uint2(pack2<Math::kBf>(most[0], most[1]), pack2<Math::kBf>(most[2], most[3]));
        if (R < 8) WM[ks * MT * 32 + (i + 4) * 4 + tt] = make_uint2(0u, 0u);   // columns of no row
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            float f[4];
#pragma unroll
            for (int d = 0; d < 4; ++d) f[d] = w[k][4 * part + d] * up;
#pragma unroll
            for (int term = 0; term < 2; ++term) {
                const uint2 v = make_uint2(pack2<Math::kBf>(f[0], f[1]), pack2<Math::kBf>(f[2], f[3]));
                W[((part * NKS + ks) * NT + i / 4) * 32 + ((i % 4) * 2 + term) * 4 + tt] = v;
                using U = typename std::conditional<Math::kBf, __nv_bfloat16, __half>::type;
                const float2 a = Half16<U>::unpack2(v.x), b = Half16<U>::unpack2(v.y);
                f[0] -= a.x; f[1] -= a.y; f[2] -= b.x; f[3] -= b.y;
            }
        }
    }
    __syncthreads();

    // ---- scores
    if constexpr (NT > 1)
#pragma unroll
        for (int c = 0; c < AHEAD; ++c) load(now, c);
    {
        float lo_[NT], hi_[NT];   // of rows 4 nt + t
        uint32_t am[MT][2];       // the largest magnitudes of rows 8 mt + 2 t, + 1, as bits: one that is not a number is above infinity
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            lo_[nt] = INFINITY;
            hi_[nt] = -INFINITY;
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) am[mt][0] = am[mt][1] = 0;
        for (int i0 = warp * 16; i0 < np; i0 += kWarps * 16) {
            const Source then = source(next, i0 + kWarps * 16);
            next = entry(i0 + 2 * kWarps * 16);
            // Four k steps to a chain of MMAs, and the chains' sums added in fp32: a chain's error is then 2^-18 of its own
            // terms'.  A chunk's registers take a later one as soon as its MMAs have read them.
            float sum[NT][2], mag[MT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) sum[nt][0] = sum[nt][1] = 0.f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) mag[mt][0] = mag[mt][1] = mag[mt][2] = mag[mt][3] = 0.f;
#pragma unroll
            for (int c = 0; c < Math::NKC; ++c) {
#pragma unroll
                for (int j0 = 0; j0 < Math::SPC; j0 += 2) {
                    float acc[NT][4];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
#pragma unroll
                    for (int j = j0; j < j0 + 2; ++j) {
                        const int ks = c * Math::SPC + j;
                        uint32_t a[2][4];
                        Math::operand(x[c % AHEAD][0], j, a[0]);
                        Math::operand(x[c % AHEAD][1], j, a[1]);
#pragma unroll
                        for (int part = 0; part < 2; ++part)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                const uint2 v = W[((part * NKS + ks) * NT + nt) * 32 + lane];
                                mma16816<Math::kBf>(acc[nt], a[part], v.x, v.y);
                            }
                        // |lo| + |hi|, for the sum of magnitudes
#pragma unroll
                        for (int i = 0; i < 4; ++i) a[0][i] = add2<Math::kBf>(a[0][i] & 0x7fff7fffu, a[1][i] & 0x7fff7fffu);
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            const uint2 v = WM[(ks * MT + mt) * 32 + lane];
                            mma16816<Math::kBf>(mag[mt], a[0], v.x, v.y);
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        sum[nt][0] += acc[nt][0] + acc[nt][1];
                        sum[nt][1] += acc[nt][2] + acc[nt][3];
                    }
                }
                if (c + AHEAD < Math::NKC) load(now, c + AHEAD);
                else load(then, c + AHEAD - Math::NKC);
            }
            const float scale[2] = {now.scale[0], now.scale[1]};
            const bool ok[2] = {now.at[0] != nullptr, now.at[1] != nullptr};
            now = then;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int page = i0 + g + 8 * r, at = p0 + page;
                if (page >= np) continue;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int row = 4 * nt + t;
                    if (row >= rows) continue;
                    float v = sum[nt][r];
                    if (!Math::kBf) v *= sh.back[row];
                    if (Math::E == 1) v *= scale[r];
                    if (!ok[r] || v != v) v = -INFINITY;
                    scores[row * p.stride + page] = v;
                    if (at >= p.keep_first && at < sh.row[row].n - p.keep_last) {   // of the pages that scores decide about
                        if (v > -INFINITY) lo_[nt] = fminf(lo_[nt], v);
                        hi_[nt] = fmaxf(hi_[nt], v);
                    }
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float a = Math::E == 1 ? mag[mt][2 * r + e] * fabsf(scale[r]) : mag[mt][2 * r + e];
                        am[mt][e] = max(am[mt][e], __float_as_uint(a));
                    }
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = 4 * nt + t;
            uint32_t a = key32(lo_[nt]), b = key32(hi_[nt]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                a = min(a, __shfl_xor_sync(0xffffffffu, a, o));
                b = max(b, __shfl_xor_sync(0xffffffffu, b, o));
            }
            if (g == 0 && row < rows) {
                atomicMin(&sh.smin[row], a);
                atomicMax(&sh.smax[row], b);
            }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = 8 * mt + 2 * t + e;
                uint32_t c = am[mt][e];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) c = max(c, __shfl_xor_sync(0xffffffffu, c, o));
                if (g == 0 && row < rows) atomicMax(&sh.amax[row], c);
            }
    }
    team_sync(cl, C);

    // ---- the first level's bins: between the smallest and the largest score
    for (int i = first_row + warp; i < rows; i += kWarps) {
        uint32_t a = sh.smin[i], b = sh.smax[i], c = sh.amax[i];
        if (CL) {
            const int k = lane < C ? lane : 0;   // a lane for each CTA
            a = __reduce_min_sync(0xffffffffu, *cl.map_shared_rank(&sh.smin[i], k));
            b = __reduce_max_sync(0xffffffffu, *cl.map_shared_rank(&sh.smax[i], k));
            c = __reduce_max_sync(0xffffffffu, *cl.map_shared_rank(&sh.amax[i], k));
        }
        RowState& s = sh.row[i];
        const float lo = from_key32(a), hi = from_key32(b), A = __uint_as_float(c) * (Math::kBf ? 1.f : sh.back[i]);
        const float inv = float(NB) / (hi - lo);
        // twice the bound on a score's error.  Magnitudes that are not finite (an infinite bound beside a query of the other sign
        // is a 0 times infinity in the MMAs) leave the row to the slow way
        // 8-bit caches: as do folded queries of 2^109 and more or below 2^-98, whose scores leave fp32 before the scale brings
        // them back, or lose bits that the scale makes large.
        const bool far = Math::E == 1 && sh.wmax[i] > 0 && (sh.wmax[i] >= 236u << 23 || sh.wmax[i] < 29u << 23);
        const float e2 = A < INFINITY && !far ? 2.f * fmaf(A, ScoreError<Math::kBf>::kRelative, ScoreError<Math::kBf>::kUnderflow) : INFINITY;
        __syncwarp();
        if (lane == 0) {
            s.lo[0] = lo;
            s.inv[0] = inv < 1e30f && hi - lo < 1e30f ? inv : 0.f;   // all the same, or not finite: one bin
            s.slack = 0.f;
            s.lowest = 1;
            s.e2 = e2;
            s.zero = A == 0.f;
            s.slow = s.need > 0 && !(e2 < INFINITY);
        }
    }
    __syncthreads();

    // A row's warps: 8, 4, 2 or 1; their part of this CTA's pages of the row.
    int wpr = kWarps;
    while (wpr > 1 && kWarps / wpr < rows - first_row) wpr /= 2;
    const int team = warp / wpr, teams = kWarps / wpr, member = warp % wpr;
    const int part = ((np + wpr - 1) / wpr + 31) & ~31, a0 = min(member * part, np), a1 = min(a0 + part, np);
    auto decided = [&](const RowState& s, int& l0, int& l1) {   // the pages of this part that scores decide about
        l0 = max(p.keep_first - p0, a0);
        l1 = min(s.n - p.keep_last - p0, a1);
    };
    const bool none = p.max_pages == p.keep_first + p.keep_last;   // scores decide about nothing
    for (int level = 0; !none; ++level) {
        for (int i = first_row + team; i < rows; i += teams) {
            const RowState& s = sh.row[i];
            if (s.slow || s.levels != level || s.in_bin <= LT / 2) continue;
            int l0, l1;
            decided(s, l0, l1);
            const float lo = s.lo[level], inv = s.inv[level];
            const float* x = scores + i * p.stride;
            if (level == 0)
                for (int k0 = l0; k0 < l1; k0 += 128) {
                    float v[4];
                    read4(x, k0 + lane, l1, v);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (k0 + 32 * j + lane < l1) atomicAdd(&sh.hist[i][bin_of(v[j], lo, inv, NB)], 1u);
                }
            else
                for (int k = l0 + lane; k < l1; k += 32)
                    if (in_bins<NB>(s, x[k])) atomicAdd(&sh.hist[i][bin_of(x[k], lo, inv, NB)], 1u);
        }
        team_sync(cl, C);
        if (CL) {
            for (int k = threadIdx.x; k < (rows - first_row) * NB; k += kThreads) {
                const int at = first_row * NB + k;
                uint32_t c = 0;
#pragma unroll
                for (int j = 0; j < kMaxCluster; ++j)
                    if (j < C) c += cl.map_shared_rank(&sh.hist[0][0], j)[at];
                (&sh.hsum[0][0])[at] = c;
            }
            __syncthreads();
        }
        bool more = false;
        for (int i = first_row + warp; i < rows; i += kWarps) {
            RowState& s = sh.row[i];
            if (s.slow || s.levels != level || s.in_bin <= LT / 2) continue;
            // lane 0 has the highest bins
            constexpr int BL = NB / 32;
            const uint32_t* h = CL ? &sh.hsum[CL ? i : 0][NB - BL * (lane + 1)] : &sh.hist[i][NB - BL * (lane + 1)];
            int c = 0;
#pragma unroll
            for (int j = 0; j < BL; ++j) c += int(h[j]);
            int incl = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            const int need = s.need;
            const uint32_t m = __ballot_sync(0xffffffffu, incl >= need);
            const int src = m ? __ffs(m) - 1 : 31;   // its bins hold the border
            if (lane == src) {
                int before = incl - c, j = BL - 1;
                while (j > 0 && before + int(h[j]) < need) before += int(h[j--]);
                const int b = NB - BL * (lane + 1) + j;
                s.bin[level] = b;
                s.need = need - before;
                s.in_bin = int(h[j]);
                s.levels = level + 1;
                const float inv = s.inv[level], lo = s.lo[level], wide = inv > 0.f ? 1.f / inv : INFINITY;
                const float low = fmaf(float(b), wide, lo), high = fmaf(float(b + 1), wide, lo);
                s.slack += NB * wide * 3.8e-6f + (fabsf(lo) + fabsf(high)) * 4.8e-7f;   // 2^-18 of the range, 2^-21 of the numbers
                s.above = high + s.slack + s.e2;
                s.lowest &= b == 0;   // scores of -infinity lie there
                s.below = s.lowest ? -INFINITY : low - s.slack - s.e2;
                if (level + 1 < kLevels) {
                    s.lo[level + 1] = low;
                    s.inv[level + 1] = inv * NB < 1e30f ? inv * NB : 0.f;
                }
                if (!(s.above < INFINITY)) s.slow = 1;
            }
            __syncwarp();
            more |= !s.slow && s.in_bin > LT / 2;
        }
        if (!__syncthreads_or(more) || level + 1 == kLevels) break;   // the same in every CTA
        team_sync(cl, C);   // the histograms have been read
        for (int i = threadIdx.x; i < R * NB; i += kThreads) (&sh.hist[0][0])[i] = 0;
        __syncthreads();
    }

    // ---- the pages above the border and those always taken, marked, the former counted, and the pages near the border, listed
    {
        for (int i = first_row + team; i < rows; i += teams) {
            const RowState& s = sh.row[i];
            if (s.slow) continue;
            int l0, l1, c = 0;
            decided(s, l0, l1);
            const float* x = scores + i * p.stride;
            const float above = s.above, below = s.below;
            const int end = min(a1, s.n - p0);
            for (int k0 = a0; k0 < end; k0 += 128) {
                float v[4];
                read4(x, k0 + lane, end, v);
                uint32_t who[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int k = k0 + 32 * j + lane;
                    const bool open = k >= l0 && k < l1 && !none, in = open && v[j] > above;
                    c += in;
                    who[j] = __ballot_sync(0xffffffffu, in || (k < end && (k < l0 || k >= l1)));
                    if (open && !in && v[j] >= below) {
                        const int at = atomicAdd(&sh.list_n[i], 1);
                        if (at < LT) {
                            sh.list_page[i][at] = p0 + k;
                            sh.list_score[i][at] = v[j];
                        }
                    }
                }
                if (lane < 4 && k0 + 32 * lane < end)
                    bits[i * words + k0 / 32 + lane] = lane < 2 ? (lane ? who[1] : who[0]) : lane == 2 ? who[2] : who[3];
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
            if (lane == 0) sh.above[i][member] = c;
        }
    }
    if (none) {
        __syncthreads();
    } else {
        team_sync(cl, C);
        // ---- their ranks
        for (int i = first_row + warp; i < rows; i += kWarps) {
            RowState& s = sh.row[i];
            if (s.slow) continue;
            int m = 0, above = 0;
            int* pages = sh.list_page[i];
            float* xs = sh.list_score[i];
            if (CL) {
                pages = sh.all_page[CL ? i : 0];
                xs = sh.all_score[CL ? i : 0];
                const int k = lane < C ? lane : 0;   // a lane for each CTA's list, then for each of its entries
                const int mk = lane < C ? *cl.map_shared_rank(&sh.list_n[i], k) : 0;
                for (int j = lane; j < C * wpr; j += 32) above += cl.map_shared_rank(&sh.above[i][0], j / wpr)[j % wpr];
                above = __reduce_add_sync(0xffffffffu, above);
                int upto = mk;
#pragma unroll
                for (int o = 1; o < kMaxCluster; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += y;
                }
                m = __shfl_sync(0xffffffffu, upto, C - 1);
                if (m <= LT)
#pragma unroll
                    for (int j = 0; j < LT; j += 32) {
                        int r = 0, first = 0;   // the entry's CTA, and that one's first entry
#pragma unroll
                        for (int k2 = 0; k2 < kMaxCluster - 1; ++k2) {
                            const int end = __shfl_sync(0xffffffffu, upto, k2);
                            if (k2 < C - 1 && j + lane >= end) {
                                r = k2 + 1;
                                first = end;
                            }
                        }
                        if (j + lane < m) {
                            pages[j + lane] = cl.map_shared_rank(&sh.list_page[i][0], r)[j + lane - first];
                            xs[j + lane] = cl.map_shared_rank(&sh.list_score[i][0], r)[j + lane - first];
                        }
                    }
            } else {
                m = sh.list_n[i];
                for (int j = 0; j < wpr; ++j) above += sh.above[i][j];
            }
            __syncwarp();
            const int places = p.max_pages - p.keep_first - p.keep_last - above;
            if (m > LT) {   // too many
                if (lane == 0) s.slow = 1;
                continue;
            }
            // by fp32 scores: the places-th largest, T
            constexpr int EL = LT / 32;
            float T0 = 0.f;
            bool found = false;
#pragma unroll
            for (int j = 0; j < EL; ++j) {
                const int e = lane + 32 * j;
                if (32 * j >= m) break;
                int better = 0;
                const float v = e < m ? xs[e] : 0.f;
                const int pg = e < m ? pages[e] : 0;
                for (int k = 0; k < m; ++k) better += xs[k] > v || (xs[k] == v && pages[k] < pg);
                if (e < m && better == places - 1) {
                    T0 = v;
                    found = true;
                }
            }
            const uint32_t who = __ballot_sync(0xffffffffu, found);
            T0 = __shfl_sync(0xffffffffu, T0, who ? __ffs(who) - 1 : 0);
            const float up = T0 + s.e2, down = T0 - s.e2;
            int hi = 0, band = 0;
#pragma unroll
            for (int j = 0; j < EL; ++j) {
                const int e = lane + 32 * j;
                hi += e < m && xs[e] > up;
                band += e < m && !(xs[e] > up) && !(xs[e] < down);
            }
            hi = __reduce_add_sync(0xffffffffu, hi);
            band = __reduce_add_sync(0xffffffffu, band);
            const bool whole = band == places - hi;
            double* exact = reinterpret_cast<double*>(&sh.hist[i][0]);   // its bins have been read, by all CTAs
            static_assert(NB * 4 >= LT * 8, "fp64 scores in the row's histogram");
            if (!whole) {
                int block[EL];   // of this lane's entries, all at once
#pragma unroll
                for (int j = 0; j < EL; ++j) {
                    const int e = lane + 32 * j;
                    block[j] = e < m ? p.block_tables[int64_t(tile.s) * p.max_blocks + pages[e]] : -1;
                }
                double w64[2 * D / 32];
                exact_weights<D>(p, s.r, kvh, lane, w64);
#pragma unroll
                for (int j = 0; j < EL; ++j) {
                    const int e = lane + 32 * j;
                    uint32_t left = __ballot_sync(0xffffffffu, e < m && !(xs[e] > up) && !(xs[e] < down));
                    while (left) {   // two at a time
                        const int e0 = __ffs(left) - 1;
                        left &= left - 1;
                        const int e1 = left ? __ffs(left) - 1 : e0;
                        left &= left - 1;
                        const double d = exact_scores<T, D, false>(p, w64, kvh, __shfl_sync(0xffffffffu, block[j], e0),
                                                            __shfl_sync(0xffffffffu, block[j], e1), lane);
                        if ((lane & 15) == 0) exact[32 * j + (lane ? e1 : e0)] = d;
                    }
                }
                __syncwarp();
            }
            int taken = 0;
#pragma unroll
            for (int j = 0; j < EL; ++j) {
                const int e = lane + 32 * j;
                if (32 * j >= m) break;
                bool in = e < m && !(xs[e] < down);
                if (in && !whole && !(xs[e] > up)) {
                    int better = 0;
                    for (int k = 0; k < m; ++k)
                        if (!(xs[k] > up) && !(xs[k] < down))
                            better += exact[k] > exact[e] || (exact[k] == exact[e] && pages[k] < pages[e]);
                    in = better < places - hi;
                }
                const uint32_t who2 = __ballot_sync(0xffffffffu, in);
                if (in) sh.sel[i][taken + __popc(who2 & ((1u << lane) - 1u))] = pages[e];
                taken += __popc(who2);
                const int k = in ? pages[e] - p0 : -1;
                if (k >= 0 && k < np) atomicOr(&bits[i * words + k / 32], 1u << (k & 31));
            }
            if (lane == 0) s.taken = taken;
        }
        __syncthreads();
    }

    // ---- the lists, in rising order
    for (int i = first_row + team; i < rows; i += teams) {
        const RowState& s = sh.row[i];
        if (s.slow) continue;
        // in front of this part: pages always taken, pages above the border in other parts, near pages that are in
        const int from = p0 + a0;
        int at = 0;
        if (!none) {
            for (int j = lane; j < s.taken; j += 32) at += sh.sel[i][j] < from;
            for (int j = lane; j < rank * wpr + member; j += 32)
                at += CL ? cl.map_shared_rank(&sh.above[i][0], j / wpr)[j % wpr] : sh.above[i][j];
            at = __reduce_add_sync(0xffffffffu, at);
        }
        at += min(from, p.keep_first) + max(0, from - (s.n - p.keep_last));
        int32_t* list = out_list(i);
        const int end = min(a1, s.n - p0);
        // us, 64 x 256 pages of single tokens (64 to a warp), 4 chunks of 256 tokens over 1024 e4m3 pages: a word to a lane
        // 20.3 / 99.8, a bit to a lane 19.6 / 103.3 (with both, and what came later, 16.5 / 98.2)
        if (end - a0 > 256) {
            for (int k0 = a0; k0 < end; k0 += 1024) {   // a word to a lane
                const int k = k0 + 32 * lane;
                uint32_t m = k < end ? bits[i * words + k / 32] : 0u;
                int to = __popc(m);
                const int mine = to;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, to, o);
                    if (lane >= o) to += y;
                }
                const int all = __shfl_sync(0xffffffffu, to, 31);
                to += at - mine;
                for (; m; m &= m - 1, ++to)
                    if (to < p.max_pages) list[to] = p0 + k + __ffs(m) - 1;
                at += all;
            }
        } else {
            for (int k0 = a0; k0 < end; k0 += 128) {   // a bit to a lane
                uint32_t m[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) m[j] = k0 + 32 * j < end ? bits[i * words + k0 / 32 + j] : 0u;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int to = at + __popc(m[j] & ((1u << lane) - 1u));
                    if ((m[j] >> lane & 1u) && to < p.max_pages) list[to] = p0 + k0 + 32 * j + lane;
                    at += __popc(m[j]);
                }
            }
        }
    }

    // ---- rows left to the slow way, all CTAs together
    int zeros = -1;
    for (int i = first_row; i < rows; ++i)
        if (sh.row[i].slow)
            select_slow<T, D, CL>(p, cl, sh, sh.row[i], tile.s, kvh, scores + i * p.stride, bits + i * words, p0, np, zeros, out_list(i));
    if (C > 1) cl.sync();   // no CTA leaves while another reads its shared memory
}

// The kernel may take kSelectSmem of dynamic shared memory: said once per kernel and device.
template <typename T, int D, int NT, int NW, bool CL>
cudaError_t launch_select_nt(const SelectParams& p, int64_t units, int cluster, size_t smem, cudaStream_t st) {
    static PerDevice ready;
    int dev = 0, one = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = cudaError_t(ready.get(dev, &one, [](int* v) {
        *v = 1;
        return int(cudaFuncSetAttribute(select_pages_kernel<T, D, NT, NW, CL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        kSelectSmem));
    }));
    if (e != cudaSuccess) return e;
    return launch_cluster_kernel(select_pages_kernel<T, D, NT, NW, CL>, dim3(unsigned(units * cluster), p.num_kv_heads), dim3(32 * NW),
                                 unsigned(cluster), smem, st, p);
}

template <typename T, int D>
cudaError_t launch_select_d(SelectParams p, cudaStream_t st) {
    int C = 1;
    auto bytes = [&](int nt) {   // the queries' operand and the scores
        p.stride = ((p.max_blocks + C - 1) / C + 15) & ~15;
        return size_t(D / 16 * 32 * 8) * (2 * nt + (nt + 1) / 2) + size_t(p.tile_rows) * (p.stride + (p.stride + 31) / 32) * 4;
    };
    auto units = [&] {
        return p.cu_q ? int64_t(p.num_rows) / p.tile_rows + p.num_seqs
                      : int64_t(p.num_seqs) * ((int64_t(p.q_len) + p.tile_rows - 1) / p.tile_rows);
    };
    // 16 query tokens to a CTA where 4 to one would be more than three rounds of the GPU (two CTAs to an SM), else 4.  us with
    // 4 / 16, 64 of up to 1024 pages, 8 kv heads of 128 dims: 1 seq x 32 tokens 20.2 / 41.6, 4 x 32 26.7 / 41.5, 32 x 8
    // 39.5 / 57.5, 32 x 16 64.0 / 68.3, 4 x 128 66.4 / 52.3, 4 x 512 206 / 166; 4 heads of 64 dims: 4 x 128 26.6 / 32.4,
    // 4 x 256 47.8 / 38.3.  The host knows the rows of all sequences together and the table's width, no lengths: one chunk of 512
    // with 63 single tokens takes 80 us (apart 38 and 27).  Shared memory goes by the width: at 128 dims two CTAs of 16 to an SM up
    // to 1072 columns, one up to 2480, then tiles of 4; 1401 tokens over 1024 pages 126 us in a table of 1072 columns, 178 of 1088
    // and 2048, 220 of 4096, 367 of 8192, 553 of 20480.
    const int64_t all = p.num_rows, each = (all + p.num_seqs - 1) / p.num_seqs;
    if (each > 4 && all * p.num_kv_heads > 4 * 912) {
        p.tile_rows = 16;
        if (bytes(4) <= kSelectSmem)
            return units() > 0x7fffffff ? cudaErrorInvalidValue : launch_select_nt<T, D, 4, 8, false>(p, units(), 1, bytes(4), st);
    }
    p.tile_rows = int(p.cu_q || each > 4 ? 4 : each);
    // As many clusters as run at once (two CTAs of 8 warps to an SM), of 128 pages or more to a CTA, which pay from 512
    // pages on.  8 kv heads of 128 dims, us with C = 1 / 2 / 4 / 8: 1 x 512 pages 11.8 / 12.5 / 11.6 / 11.4, a step of
    // 8 x 256 26.2 / 28.9 / 29.4 / 38.7, 32 x 2048 44.1 / 50.7 / 67.9 / 109, 4 x 8192 (int8) 120 / 64.5 / 41.9 / 34.4.
    const int64_t pairs = units() * p.num_kv_heads;
    if (p.max_blocks >= 512)
        while (C < kMaxCluster && pairs * C * 2 <= 304 && p.max_blocks / (2 * C) >= 128) C *= 2;
    // CTAs of 4 warps where there are more.  us with 4 / 8: 64 x 256 pages, 8 heads 16.5 / 22.0, 128 x 1024 68.8 / 74.2, a step
    // of 64 x 125 32.3 / 37.5; but 32 x 256 14.8 / 14.3, 32 x 2048 54.9 / 44.2.
    const bool narrow = pairs > 304;
    // what a CTA's shared memory does not hold is spread over more CTAs, then taken in smaller tiles
    while (bytes(1) > kSelectSmem) {
        if (C < kMaxCluster) C *= 2;
        else if (p.tile_rows > 1) p.tile_rows /= 2;
        else return cudaErrorInvalidValue;
    }
    const size_t smem = bytes(1);
    if (units() * C > 0x7fffffff) return cudaErrorInvalidValue;
    if (C > 1) return launch_select_nt<T, D, 1, 8, true>(p, units(), C, smem, st);
    return narrow ? launch_select_nt<T, D, 1, 4, false>(p, units(), C, smem, st) : launch_select_nt<T, D, 1, 8, false>(p, units(), C, smem, st);
}

template <typename T>
cudaError_t launch_select_t(const SelectParams& p, cudaStream_t st) {
    return p.head_dim == 128 ? launch_select_d<T, 128>(p, st) : launch_select_d<T, 64>(p, st);
}

}  // namespace

}  // namespace pkv
