// rope.cu -- rotary positions of queries and keys, with the cache write of the
// rotated keys and the values in the same launch.
//
//   angle(p, i) = p * f_i,  c = mscale cos, s = mscale sin
//   (a, b) -> (a c - b s, b c + a s) for the pairs (i, i + R/2) (half layout) or
//   (2i, 2i + 1) (interleaved) of the first R = rotary_dim dims of a head.
//
// The product is exact whatever the position: f_i is held as a 64-bit fraction of
// a turn, so the product's low 64 bits are the phase (whole turns fall off the
// top), one integer multiply where fp32 loses the angle of a far position and
// fp64 runs at a small part of the fp32 rate.  The phase's top 32 bits are
// rounded to fp32 half-turns for sincospif: 2^-25 of a half-turn, and 2^-31 for the
// bits below them.  The table is fp64's: its entries' 2^-53 of a turn count as often as
// the position says.
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

// Threads of a CTA: half layout 256 (8192 tokens of 32 + 8 heads of 128 dims 32.5 us, with 128 32.7; 512 tokens 3.1
// and 4.0), interleaved 128 (34.0, with 256 35.9), half with chunks that do not match 128 (43.4, with 256 68).
constexpr int kHalfThreads = 256, kPairThreads = 128, kAnyThreads = 128;
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

// cosine and sine of pair i of token t
__device__ __forceinline__ float2 angle(const RopeParams& p, int64_t t, int i) {
    const uint64_t phase = uint64_t(p.positions[t]) * p.freq[i];
    float s, c;
    sincospif(float(int32_t(phase >> 32)) * 4.656612873077393e-10f, &s, &c);
    return make_float2(c * p.mscale, s * p.mscale);
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

// 16-byte chunks: the interleaved layout (a pair is a word), and the half layout where
// rotary_dim % 16 == 0, so that a pair's elements lie at the same place of two chunks.
// A thread moves two chunks of a row: the two that turn with one another (half), or
// one from each half of what is left (interleaved, and dims that are kept), so that the
// threads of a row always read and write side by side.  D / 16 threads
// are a row, so a CTA of 256 has 32 (D = 128) or 64 rows in its hands at once (of 128, half), and
// loads four such sets before it stores the first.
// The angles' table in shared memory keeps the four or two float4 (cos, sin, cos, sin)
// of a chunk apart, so that the threads of a row read 16 bytes side by side.
// 8192 tokens of 32 + 8 + 8 heads, bf16, D = 128: 32.4 us (6.1 TB/s, of 6.8 measured);
// one warp per row with 2-byte accesses took 84.  Interleaved 34.0; 37.7 with 256 threads and
// two chunks side by side to a thread, whose halves of a 32-byte sector two stores write.
template <typename T, bool HALF, int D>
__global__ void __launch_bounds__(HALF ? kHalfThreads : kPairThreads) rope_chunks_kernel(RopeParams p) {
    constexpr int kT = HALF ? kHalfThreads : kPairThreads;
    constexpr int TPR = D / 16;                 // threads per row
    constexpr int RPB = kT / TPR;               // rows of a CTA at once
    constexpr int Q4 = HALF ? 4 : 2;            // float4s of a chunk's angles
    constexpr int U = 4;                        // rows a thread loads ahead
    __shared__ float4 cs[kMaxTokens][Q4][HALF ? 8 : 16];
    grid_dep_wait();
    grid_dep_launch();
    const int64_t t0 = int64_t(blockIdx.x) * p.tokens_per_cta;
    const int ntok = int(min(int64_t(p.tokens_per_cta), p.num_tokens - t0));
    const int rows = p.num_heads + (p.slot_mapping ? 2 : 1) * p.num_kv_heads, turned = p.num_heads + p.num_kv_heads;
    const int x = threadIdx.x % TPR, pairs = p.rotary_dim / 2;
    // this thread's two chunks, and which of them turn
    const int nrot = p.rotary_dim / 16;         // half: chunk pairs that turn
    const int ca = HALF && x >= nrot ? nrot + x : x, cb = HALF && x < nrot ? x + nrot : TPR + x;
    const bool ta = HALF ? x < nrot : 8 * ca < p.rotary_dim, tb = HALF ? x < nrot : 8 * cb < p.rotary_dim;

    int tok = 0, row = threadIdx.x / TPR;       // the next row to load
    auto settle = [&]() {
        while (row >= rows && tok < ntok) {
            row -= rows;
            ++tok;
        }
    };
    settle();
    bool ready = false;
    while (true) {
        uint4 a[U], b[U];
        int rt[U], rr[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            rt[k] = tok;
            rr[k] = row;
            if (tok < ntok) {
                const uint4* src = reinterpret_cast<const uint4*>(row_src(p, t0 + tok, row));
                a[k] = __ldcs(src + ca);
                b[k] = __ldcs(src + cb);
                row += RPB;
                settle();
            }
        }
        if (!ready) {
            // the first rows are on their way; the angles meanwhile
            flag_slots(p, t0, ntok);
            for (int y = threadIdx.x; y < ntok * pairs; y += kT) {
                const int at = y / pairs, i = y - at * pairs;
                const int c = i / (2 * Q4), j = (i / 2) % Q4;
                reinterpret_cast<float2*>(&cs[at][j][c])[i & 1] = angle(p, t0 + at, i);
            }
            __syncthreads();
            ready = true;
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (rt[k] >= ntok) break;
            const int64_t t = t0 + rt[k];
            const Dest d = row_dest(p, t, rr[k], token_slot(p, t));
            if (rr[k] < turned) {
                if constexpr (HALF) {
                    if (ta) {
                        uint32_t* wa = &a[k].x;
                        uint32_t* wb = &b[k].x;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float4 f = cs[rt[k]][j][x];
                            const float2 u = Half16<T>::unpack2(wa[j]), v = Half16<T>::unpack2(wb[j]);
                            const float2 y0 = turn(u.x, v.x, make_float2(f.x, f.y)), y1 = turn(u.y, v.y, make_float2(f.z, f.w));
                            wa[j] = pack16<T>(y0.x, y1.x);
                            wb[j] = pack16<T>(y0.y, y1.y);
                        }
                    }
                } else {
                    auto spin = [&](uint4& v, int c) {
                        const uint4 kept = v;
                        uint32_t* w = &v.x;
                        const int words = pairs - 4 * c;   // pairs of this chunk that turn
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const float4 f = cs[rt[k]][j][c];
                            const float2 u0 = Half16<T>::unpack2(w[2 * j]), u1 = Half16<T>::unpack2(w[2 * j + 1]);
                            const float2 y0 = turn(u0.x, u0.y, make_float2(f.x, f.y)), y1 = turn(u1.x, u1.y, make_float2(f.z, f.w));
                            w[2 * j] = pack16<T>(y0.x, y0.y);
                            w[2 * j + 1] = pack16<T>(y1.x, y1.y);
                        }
                        if (words < 4) {
                            v.y = words > 1 ? v.y : kept.y;
                            v.z = words > 2 ? v.z : kept.z;
                            v.w = kept.w;
                        }
                    };
                    if (ta) spin(a[k], ca);
                    if (tb) spin(b[k], cb);
                }
            }
            if (d.a) {
                reinterpret_cast<uint4*>(d.a)[ca] = a[k];
                reinterpret_cast<uint4*>(d.a)[cb] = b[k];
            }
            if (d.b) {
                reinterpret_cast<uint4*>(d.b)[ca] = a[k];
                reinterpret_cast<uint4*>(d.b)[cb] = b[k];
            }
        }
        if (tok >= ntok) break;
    }
}

// Half layout with any other rotary_dim: a pair's elements lie at different places of
// their chunks.  As above, two chunks side by side to a thread; the chunks that turn go
// through shared memory, where a thread finds its elements' partners (a row lies in one
// warp).  One warp per row, or a thread per pair, spend more on addresses than on this.
template <typename T, int D>
__global__ void __launch_bounds__(kAnyThreads, 6) rope_any_kernel(RopeParams p) {
    constexpr int TPR = D / 16, RPB = kAnyThreads / TPR, U = 4;
    __shared__ float2 cs[kMaxTokens * 64];
    __shared__ uint4 held[RPB][D / 8 + 1];      // a row set's chunks (rows of a warp in different banks)
    grid_dep_wait();
    grid_dep_launch();
    const int64_t t0 = int64_t(blockIdx.x) * p.tokens_per_cta;
    const int ntok = int(min(int64_t(p.tokens_per_cta), p.num_tokens - t0));
    const int rows = p.num_heads + (p.slot_mapping ? 2 : 1) * p.num_kv_heads, turned = p.num_heads + p.num_kv_heads;
    const int x = threadIdx.x % TPR, mine = threadIdx.x / TPR, pairs = p.rotary_dim / 2, ca = 2 * x;
    flag_slots(p, t0, ntok);
    for (int y = threadIdx.x; y < ntok * pairs; y += kAnyThreads) cs[y] = angle(p, t0 + y / pairs, y % pairs);
    __syncthreads();
    int tok = 0, row = mine;
    auto settle = [&]() {
        while (row >= rows && tok < ntok) {
            row -= rows;
            ++tok;
        }
    };
    settle();
    while (__any_sync(0xffffffffu, tok < ntok)) {
        uint4 a[U], b[U];
        int rt[U], rr[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            rt[k] = tok;
            rr[k] = row;
            if (tok < ntok) {
                const uint4* src = reinterpret_cast<const uint4*>(row_src(p, t0 + tok, row));
                a[k] = __ldcs(src + ca);
                b[k] = __ldcs(src + ca + 1);
                row += RPB;
                settle();
            }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const bool there = rt[k] < ntok, turns = there && rr[k] < turned && 8 * ca < 2 * pairs;
            __syncwarp();   // the set before has been read (and every row of this one loaded)
            if (turns) {
                held[mine][ca] = a[k];
                held[mine][ca + 1] = b[k];
            }
            __syncwarp();
            if (turns) {
                const uint16_t* at = reinterpret_cast<const uint16_t*>(held[mine]);
                const float2* f = cs + rt[k] * pairs;
                auto mix = [&](uint4& v, int c) {
                    uint32_t* w = &v.x;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int dim = 8 * c + 2 * j;
                        if (dim >= 2 * pairs) break;   // rotary_dim is even: a word turns whole or not at all
                        const float2 own = Half16<T>::unpack2(w[j]);
                        auto one = [&](float u, int d) {
                            const float o = Half16<T>::to_float(at[d < pairs ? d + pairs : d - pairs]);
                            return d < pairs ? turn(u, o, f[d]).x : turn(o, u, f[d - pairs]).y;
                        };
                        w[j] = pack16<T>(one(own.x, dim), one(own.y, dim + 1));
                    }
                };
                mix(a[k], ca);
                mix(b[k], ca + 1);
            }
            if (there) {
                const Dest d = row_dest(p, t0 + rt[k], rr[k], token_slot(p, t0 + rt[k]));
                if (d.a) {
                    reinterpret_cast<uint4*>(d.a)[ca] = a[k];
                    reinterpret_cast<uint4*>(d.a)[ca + 1] = b[k];
                }
                if (d.b) {
                    reinterpret_cast<uint4*>(d.b)[ca] = a[k];
                    reinterpret_cast<uint4*>(d.b)[ca + 1] = b[k];
                }
            }
        }
    }
}

template <typename T, int D>
cudaError_t launch_layout(const RopeParams& p, dim3 grid, cudaStream_t st) {
    const bool half = p.layout == PKV_ROPE_HALF;
    if (half && p.rotary_dim % 16 != 0) return launch_kernel(rope_any_kernel<T, D>, grid, dim3(kAnyThreads), 0, st, p);
    return half ? launch_kernel(rope_chunks_kernel<T, true, D>, grid, dim3(kHalfThreads), 0, st, p)
                : launch_kernel(rope_chunks_kernel<T, false, D>, grid, dim3(kPairThreads), 0, st, p);
}

}  // namespace

cudaError_t launch_rope(RopeParams p, cudaStream_t stream) {
    // A CTA's table of angles and start-up are worth about 24 KB of rows: two tokens of 48 heads of 128 dims (8192
    // tokens: 39.9, 32.3, 33.5 us with 1, 2, 4), four of 48 of 64 dims (33.0, 24.6, 18.2 us).  But no fewer
    // than 256 CTAs for it (256 tokens of 24 heads of 64: 2.1 us with 256 CTAs, 2.3 with 64).
    const int64_t row_elems = (int64_t(p.num_heads) + 2 * int64_t(p.num_kv_heads)) * p.head_dim;
    p.tokens_per_cta = row_elems * 4 <= 12288 ? 4 : row_elems * 2 <= 12288 ? 2 : 1;
    while (p.tokens_per_cta > 1 && p.num_tokens / p.tokens_per_cta < 256) p.tokens_per_cta /= 2;
    const int64_t ctas = (p.num_tokens + int64_t(p.tokens_per_cta) - 1) / p.tokens_per_cta;
    if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
    const dim3 grid{unsigned(ctas)};
    if (p.head_dim == 128)
        return p.dtype == PKV_BF16 ? launch_layout<__nv_bfloat16, 128>(p, grid, stream) : launch_layout<__half, 128>(p, grid, stream);
    return p.dtype == PKV_BF16 ? launch_layout<__nv_bfloat16, 64>(p, grid, stream) : launch_layout<__half, 64>(p, grid, stream);
}

}  // namespace pkv
