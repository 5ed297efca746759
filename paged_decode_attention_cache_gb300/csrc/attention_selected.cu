// attention_selected.cu -- attention over lists of pages, one query token to a cluster
// (attention_selected.cuh), and the choice between it and several (attention_selected_rows.cu).
//
// As TtMath and TeMath: S^T = K Q^T has a page's tokens on the MMA's M side and the kv head's
// query heads on its 8 columns, O^T = V^T P^T the dims on M.
//
// Bound: HBM where 16-bit pages fill the GPU (32 tokens over 128 pages of 8 bf16 heads of 128 dims:
// 269 MB in 44 us, 6.1 TB/s); 8-bit pages by the latency of their widening and MMAs (64 tokens of 8192 over
// 64 of their pages, 8 heads: e4m3, 134 MB, 38 us, int8 38, K8/V4 41); one token over 64 pages, 5.6 us, by the
// chain count -> list -> table -> page and the merge's two barriers.
#include "attention_selected.cuh"

namespace pkv {

namespace {

template <int KIND, int D>
__global__ void __launch_bounds__(kSelThreads, sel_ctas(KIND, D, false))
attention_selected_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map, const SelectedParams p) {
    constexpr int COLS = 8;
    using Math = PageMath<KIND, D>;
    constexpr int NKS = Math::NKS, NMT = Math::NMT, STAGES = Math::STAGES, RING = STAGES * Math::STAGE, OW = D + 4;
    static_assert(COLS * OW * 4 <= RING, "a warp's partial lies in its ring");
    extern __shared__ uint8_t smem_raw[];
    // 1 KB aligned (the swizzled tiles need it)
    uint8_t* const smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t* const sides = smem + kSelWarps * RING;
    int2* const entry = reinterpret_cast<int2*>(sides + kSelWarps * STAGES * Math::SIDE);   // this CTA's pages: page, block
    __shared__ uint64_t k_full[kSelWarps * STAGES], v_full[kSelWarps * STAGES];
    __shared__ Partials<COLS> part;
    __shared__ uint2 Q[COLS / 8 * NKS * 32];
    __shared__ uint32_t q_most[COLS];
    __shared__ int kept;
    cg::cluster_group cl = cg::this_cluster();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int C = int(cl.num_blocks()), rank = int(cl.block_rank());
    if (C > 1) cluster_arrive();   // waited for before anything is sent to another CTA
    if (threadIdx.x < COLS) q_most[threadIdx.x] = 0;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kSelWarps * STAGES; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&v_full[i], 1);
        }
        fence_barrier_init();
        prefetch_tensormap(&k_map);
        prefetch_tensormap(&v_map);
    }
    grid_dep_wait();
    const int kvh = blockIdx.y, G = p.num_heads / p.num_kv_heads;
    const RowTile tile = find_tile(p.cu_q, p.num_seqs, p.num_rows, p.q_len, 1, int(blockIdx.x / C), lane);
    if (tile.s < 0) {   // no row: the same in every CTA of the cluster
        if (C > 1) cluster_wait();
        return;
    }
    Queries<Math, COLS, D> queries;
    queries.load(p, tile.r0, G, kvh, G);
    const SelectedTile mine(p, tile, kvh);
    if (mine.over() && rank == 0 && kvh == 0 && threadIdx.x == 0) flag_error(p.err, PKV_DEVERR_CAPACITY);
    const int vis = mine.visible(0);

    // ---- the list: each entry in range and above the one before it, with a block, or the slow way
    const int32_t* list = mine.list(0);
    // the first entries come with the count, not after it
    int e = int(threadIdx.x) < p.max_pages ? list[threadIdx.x] : -1;
    int before = threadIdx.x > 0 && int(threadIdx.x) < p.max_pages ? list[threadIdx.x - 1] : -1;
    const int count = mine.count(0), pages = mine.pages(0);
    const int i0 = int(int64_t(count) * rank / C), i1 = int(int64_t(count) * (rank + 1) / C);
    int n = i1 - i0;
    bool rising = true, whole = true;
    for (int i = threadIdx.x; i < count; i += kSelThreads) {
        if (i >= kSelThreads) {
            e = list[i];
            before = list[i - 1];
        }
        rising &= e > before && e < pages;
        if (i >= i0 && i < i1) {
            const int b = e >= 0 && e < pages ? mine.block(e) : -1;
            whole &= b >= 0;
            entry[i - i0] = make_int2(e, b);
        }
    }
    if (__syncthreads_or(!rising || !whole)) {
        const bool bad = __syncthreads_or(!rising);
        if (warp == 0) {
            if (bad) {
                mine.in_order(0, lane, [&](int i, bool there, bool taken, int) {
                    if (there && !taken && i >= i0 && i < i1) entry[i - i0].y = -1;
                });
                __syncwarp();
                if (lane == 0 && rank == 0) flag_error(p.err, PKV_DEVERR_PAGE_LIST);
            }
            const int k = mine.close_up(entry, n, lane);
            if (lane == 0) kept = k;
        }
        __syncthreads();
        n = kept;
    }

    // ---- the first pages, on their way; the query operand
    Ring<Math, false> ring{p, &k_map, &v_map, entry, n, kvh, warp, lane, smem + warp * RING, sides + warp * STAGES * Math::SIDE,
                           k_full + warp * STAGES, v_full + warp * STAGES, 0, 0, 0u, 0u};
    ring.begin();
    queries.store(p, Q, q_most);
    __syncthreads();
    uint2 q[NKS];
#pragma unroll
    for (int kk = 0; kk < NKS; ++kk) q[kk] = Q[kk * 32 + lane];
    const float kcol[2] = {column_scale<Math>(p, q_most, 2 * t), column_scale<Math>(p, q_most, 2 * t + 1)};

    // ---- the pages: a step is two (the second may be missing), whose MMAs and softmaxes do not wait for one another.  K's
    // stages are filled again while the weights are worked out, V's while the next step's scores are.
    float o[NMT][4], m_run[2] = {-INFINITY, -INFINITY}, l_part[2] = {0.f, 0.f}, vref = 1.17549435e-38f;
#pragma unroll
    for (int mt = 0; mt < NMT; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
    int st = 0;
    for (int at = warp; at < n; at += 2 * kSelWarps) {
        const bool two = at + kSelWarps < n;
        const int page[2] = {entry[at].x, two ? entry[at + kSelWarps].x : 0};
        const uint8_t *const stage[2] = {ring.stage(st), ring.stage(st + 1)}, *const side[2] = {ring.side(st), ring.side(st + 1)};
        bool came = ring.wait_k(st);
        if (two) came &= ring.wait_k(st + 1);
        float s[2][4];   // tokens g, g + 8 x query heads 2t, 2t + 1
#pragma unroll
        for (int b = 0; b < 2; ++b) s[b][0] = s[b][1] = s[b][2] = s[b][3] = 0.f;
        // a page that is missing: of what its stage held, and left out below
        Math::keys(stage, lane, [&](int kk, const uint32_t (&a)[2][4]) {
            mma16816<Math::kBf>(s[0], a[0], q[kk].x, q[kk].y);
            mma16816<Math::kBf>(s[1], a[1], q[kk].x, q[kk].y);
        });
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const float k0 = Math::k_scale(side[b], g), k8 = Math::k_scale(side[b], g + 8);
            const int live = b && !two ? 0 : vis - page[b] * kBS;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                s[b][c] = g < live ? s[b][c] * (k0 * kcol[c]) : -INFINITY;
                s[b][2 + c] = g + 8 < live ? s[b][2 + c] * (k8 * kcol[c]) : -INFINITY;
            }
        }
        __syncwarp();   // the K tiles have been read
        ring.fill_k(st);
        ring.fill_k(st + 1);
        float f[2];
        bool rescale = false;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float bm = fmaxf(fmaxf(s[0][c], s[0][2 + c]), fmaxf(s[1][c], s[1][2 + c]));
            bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 4));
            bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 8));
            bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 16));
            const float mu = reference<Math>(bm, m_run[c], f[c]);
            float sum = 0.f;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                s[b][c] = exp2_ftz(s[b][c] - mu);
                s[b][2 + c] = exp2_ftz(s[b][2 + c] - mu);
                sum += s[b][c] + s[b][2 + c];
            }
            l_part[c] = l_part[c] * f[c] + sum;
            rescale |= f[c] != 1.f;
        }
        came &= ring.wait_v(st);
        if (two) came &= ring.wait_v(st + 1);
        if (!came) {
            ring.give_up();
            break;
        }
        float unit[2] = {Math::kPUnit, Math::kPUnit};   // what the weights are multiplied by in the operand
        if constexpr (Math::kByte) {
            unit[0] = Math::v_scale(side[0]);
            unit[1] = two ? Math::v_scale(side[1]) : 0.f;
            const float grow = v_units<Math>(unit, vref);
            f[0] *= grow;
            f[1] *= grow;
            rescale |= grow != 1.f;
        }
        if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
            for (int mt = 0; mt < NMT; ++mt) {
                o[mt][0] *= f[0]; o[mt][2] *= f[0];
                o[mt][1] *= f[1]; o[mt][3] *= f[1];
            }
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            if (b && !two) break;
            uint32_t hi[2], lo[2];   // P^T operand: tokens 2t, 2t + 1 (and 8 further) of query head g
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                split2<Math>(s[b][2 * h] * unit[b], s[b][2 * h + 1] * unit[b], hi[h], lo[h]);
                hi[h] = movm_trans(hi[h]);
                lo[h] = movm_trans(lo[h]);
            }
            auto add = [&](int m0, auto& a) {
                constexpr int N = sizeof(a) / 16;
#pragma unroll
                for (int j = 0; j < N; ++j) mma16816<Math::kBf>(o[m0 + j], a[j], hi[0], hi[1]);
#pragma unroll
                for (int j = 0; j < N; ++j) mma16816<Math::kBf>(o[m0 + j], a[j], lo[0], lo[1]);
            };
            const int live = vis - page[b] * kBS, k = 2 * t;
            if (live >= kBS) {
                Math::template tiles<false, 4>(stage[b], side[b], 0u, 0u, lane, add);
            } else {   // the tokens behind the last one may hold anything
                const uint32_t m01 = (k < live ? 0xffffu : 0u) | (k + 1 < live ? 0xffff0000u : 0u);
                const uint32_t m23 = (k + 8 < live ? 0xffffu : 0u) | (k + 9 < live ? 0xffff0000u : 0u);
                Math::template tiles<true, 4>(stage[b], side[b], m01, m23, lane, add);
            }
        }
        __syncwarp();   // the V tiles have been read
        ring.fill_v(st);
        ring.fill_v(st + 1);
        st = st + 2 == STAGES ? 0 : st + 2;
    }

    // The next kernel may come now: its CTAs, were they here from the start, would take the places beside some of these
    // CTAs and leave others alone, and this grid's successor would run as unevenly (32 tokens of 8192 over 64 pages of 8 e4m3 heads, without
    // spread(): 32.9 us early, 22.9 late).
    grid_dep_launch();
    // ---- the warp's partial, and the merges
    const float back = (Math::kByte ? vref : 1.f) * (1.f / Math::kPUnit);
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        float l = l_part[c];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        const int col = 2 * t + c;
        if (g == 0) {
            part.m[warp][col] = m_run[c];
            part.l[warp][col] = l;
        }
        if (col < G) {
            float* to = reinterpret_cast<float*>(smem + warp * RING) + col * OW;
#pragma unroll
            for (int mt = 0; mt < NMT; ++mt) {
                to[Math::dim(mt, g)] = o[mt][c] * back;
                to[Math::dim(mt, g) + Math::kNext] = o[mt][2 + c] * back;
            }
        }
    }
    merge_and_store<COLS, D>(p, cl, part, reinterpret_cast<float*>(smem), RING / 4,
                             reinterpret_cast<float4*>(reinterpret_cast<uint8_t*>(entry) + p.list_bytes), tile.r0, G, kvh, G);
}

// The kernel may take kSelectedSmem of dynamic shared memory: said once per kernel and device.
template <int KIND, int D>
cudaError_t launch_one(const SelectedParams& p, int64_t units, int cluster, size_t lists, const CUtensorMap& km, const CUtensorMap& vm,
                       cudaStream_t st) {
    static PerDevice ready;
    int dev = 0, one = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = cudaError_t(ready.get(dev, &one, [](int* v) {
        *v = 1;
        return int(cudaFuncSetAttribute(attention_selected_kernel<KIND, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelectedSmem));
    }));
    if (e != cudaSuccess) return e;
    const size_t smem = ring_bytes<PageMath<KIND, D>>() + lists + (cluster > 1 ? exchange_bytes<8, D>() : 0);
    return launch_cluster_kernel(attention_selected_kernel<KIND, D>, dim3(unsigned(units * cluster), p.num_kv_heads), dim3(kSelThreads),
                                 unsigned(cluster), spread(units * cluster * p.num_kv_heads, smem), st, km, vm, p);
}

template <int KIND>
cudaError_t launch_kind(const SelectedParams& p, int64_t units, int cluster, size_t lists, const CUtensorMap& km,
                        const CUtensorMap& vm, cudaStream_t st) {
    return p.head_dim == 128 ? launch_one<KIND, 128>(p, units, cluster, lists, km, vm, st)
                             : launch_one<KIND, 64>(p, units, cluster, lists, km, vm, st);
}

}  // namespace

cudaError_t launch_attention_selected(SelectedParams p, int cache_kind, const CUtensorMap& km, const CUtensorMap& vm,
                                      cudaStream_t stream) {
    int C = 1;
    int64_t units = 0, most = 0;   // tiles, and the pages that one may have
    size_t lists = 0;
    auto size = [&] {   // the CTA's entries, and a byte for each page where rows share them
        p.entries = int((most + C - 1) / C);
        lists = (size_t(p.entries) * 8 + (p.tile_rows > 1 ? (size_t(p.max_blocks) + 3) / 4 * 4 : 0) + 15) / 16 * 16;
        p.list_bytes = int(lists);
        return lists <= kSelectedLists;
    };
    auto tiles = [&](int rows) {
        p.tile_rows = rows;
        units = p.cu_q ? int64_t(p.num_rows) / rows + p.num_seqs : int64_t(p.num_seqs) * ((int64_t(p.q_len) + rows - 1) / rows);
        most = int64_t(rows) * p.max_pages;
        if (rows > 1 && most > p.max_blocks) most = p.max_blocks;
        // as many clusters as run at once
        const int64_t room = 152 * (rows > 1 ? 2 : sel_ctas(cache_kind, p.head_dim, false));
        C = 1;
        while (C < kSelCluster && units * p.num_kv_heads * C * 2 <= room && most >= 2 * C * 2 * kSelWarps) C *= 2;
        while (!size() && C < kSelCluster) C *= 2;
        return size();
    };
    // Neighbouring tokens together, if all lists have more than 96 pages for each SM, which single tokens' clusters, being more,
    // read sooner; and where a page's K row has 256 bytes, four tokens or more: two or three read that much from L2 about as
    // soon as they find the union of their lists.  us alone / together, 8 kv heads, 64 pages: bf16 of 4 query heads of 128 dims,
    // 8 seqs x 4 tokens 14.6 / 15.1, 16 x 4 31.7 / 24.4, 64 x 4 84.9 / 69.1, 64 x 8 151 / 106, but 16 x 3 19.2 / 23.4, 32 x 3
    // 40.3 / 35.0, 64 x 2 60.2 / 60.9; e4m3 8 x 2 12.1 / 14.0, 16 x 3 34.8 / 22.5, 64 x 2 66.8 / 60.7; bf16 of 64 dims 64 x 2
    // 61.8 / 45.7.  16 x 3 e4m3 tokens, 4 kv heads, 101 pages: 28.9 / 19.0.
    int rows = shared_tokens(p);
    const bool half = cache_kind == PKV_CACHE_F16 || cache_kind == PKV_CACHE_BF16;
    if (int64_t(p.num_rows) * p.num_kv_heads * p.max_pages <= 96 * 152 || (rows < 4 && half && p.head_dim == 128)) rows = 1;
    if (!(rows > 1 && tiles(rows)) && !tiles(1)) return cudaErrorInvalidValue;
    if (units * C > 0x7fffffff) return cudaErrorInvalidValue;
    if (p.tile_rows > 1) return launch_attention_rows(p, cache_kind, units, C, lists, km, vm, stream);
    switch (cache_kind) {
        case PKV_CACHE_F16: return launch_kind<PKV_CACHE_F16>(p, units, C, lists, km, vm, stream);
        case PKV_CACHE_BF16: return launch_kind<PKV_CACHE_BF16>(p, units, C, lists, km, vm, stream);
        case PKV_CACHE_K8V4: return launch_kind<PKV_CACHE_K8V4>(p, units, C, lists, km, vm, stream);
        case PKV_CACHE_I8: return launch_kind<PKV_CACHE_I8>(p, units, C, lists, km, vm, stream);
        default: return launch_kind<PKV_CACHE_E4M3>(p, units, C, lists, km, vm, stream);
    }
}

}  // namespace pkv
