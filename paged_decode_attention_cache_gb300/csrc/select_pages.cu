// select_pages.cu -- the bounds of each page's keys (the smallest and the largest of a
// cache block's stored tokens, dim by dim and kv head by kv head), and the selection
// over them for bf16 (select_pages.cuh; the other types: select_half.cu, select_i8.cu, select_e4m3.cu).
//
// Bound of the bounds: dependent loads (length -> table -> keys) for a step (64 sequences, 2.4 us with the launch); for
// prompts the same and then HBM (7 of up to 4000 tokens of e4m3, 18.5 MB in 7.4 us, of which HBM's rate would take 2.7).
#include "select_pages.cuh"

namespace pkv {

namespace {

struct K8 {};   // int8 codes with a scale per token

// e4m3 codes as signed bytes in the numbers' order, and back (the map is its own inverse).
__device__ __forceinline__ uint32_t e4m3_order4(uint32_t w) {
    const uint32_t neg = (w >> 7) & 0x01010101u;
    return w ^ (neg * 0x7fu);
}

// The smallest and the largest of rows of 16 bytes.
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

}  // namespace

cudaError_t launch_key_bounds(const KeyBoundsParams& p, int cache_kind, cudaStream_t stream) {
    const int chunks = p.num_kv_heads * p.head_dim * (cache_kind == PKV_CACHE_F16 || cache_kind == PKV_CACHE_BF16 ? 2 : 1) / 16;
    int64_t pages = p.max_blocks;
    const int64_t touched = (int64_t(p.q_len) + 14) / kBlockSize + 1;   // by q_len tokens, at most
    if (!p.cu_new && touched < pages) pages = touched;
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
    switch (cache_kind) {
        case PKV_CACHE_BF16: return launch_select_t<__nv_bfloat16>(p, stream);
        case PKV_CACHE_I8: return launch_select_i8(p, stream);
        case PKV_CACHE_E4M3: return launch_select_e4m3(p, stream);
        default: return launch_select_half(p, stream);   // fp16 caches, and K8V4's fp16 bounds
    }
}

}  // namespace pkv
