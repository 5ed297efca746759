// attention_selected_rows.cu -- attention over lists of pages, several neighbouring query tokens
// of a sequence to a cluster (attention_selected.cuh): drafts, a chunk of a prompt.
//
// Their lists have much in common: a CTA takes up to 16 / g tokens, which with the kv head's g query
// heads are 16 query rows, reads the union of their lists once, and masks by row.
//
// With 16 rows the queries take the MMA's M side, S = Q K^T and O = P V: P's accumulators are then
// its operand as they lie, and a thread has two rows' statistics where it would have four columns'.
//
// Bound: latency, in three parts one after the other (16 x 3 tokens over 101 pages of 4 e4m3 heads, 27 MB in
// 19.0 us: the union of the lists 5.6 thousand clocks, the pages 15, the merges 7.7; issue slots 25 % used).
#include "attention_selected.cuh"

namespace pkv {

namespace {

template <int KIND, int D>
__global__ void __launch_bounds__(kSelThreads, sel_ctas(KIND, D, true))
attention_rows_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map, const SelectedParams p) {
    constexpr int COLS = 16;   // query rows
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
    __shared__ __align__(16) uint2 Q[COLS / 8 * NKS * 32];
    __shared__ uint32_t q_most[COLS];
    __shared__ int scan[kSelWarps], kept;
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
    const RowTile tile = find_tile(p.cu_q, p.num_seqs, p.num_rows, p.q_len, p.tile_rows, int(blockIdx.x / C), lane);
    if (tile.s < 0) {   // no row: the same in every CTA of the cluster
        if (C > 1) cluster_wait();
        return;
    }
    Queries<Math, COLS, D> queries;
    queries.load(p, tile.r0, tile.rows * G, kvh, G);
    const SelectedTile mine(p, tile, kvh);
    if (mine.over() && rank == 0 && kvh == 0 && threadIdx.x == 0) flag_error(p.err, PKV_DEVERR_CAPACITY);
    const int rows = tile.rows, cols = rows * G;
    const int vis_all = mine.visible(0);   // tokens that every row sees

    // ---- the union of the lists, if every entry is in range and above the one before it; else the slow way
    uint32_t* const bytes = reinterpret_cast<uint32_t*>(entry + p.entries);   // the rows that list a page, a bit each
    const int words = (mine.pages(rows - 1) + 3) / 4;
    for (int i = threadIdx.x; i < words; i += kSelThreads) bytes[i] = 0;
    __syncthreads();
    bool rising = true;
    for (int row = warp; row < rows; row += kSelWarps) {
        const int32_t* list = mine.list(row);
        int e = lane < p.max_pages ? list[lane] : -1;   // comes with the count, not after it
        const int count = mine.count(row), pages = mine.pages(row);
        int last = -1;   // the entry before this 32
        for (int i = lane; i - lane < count; i += 32) {
            const int ahead = i + 32 < p.max_pages ? list[i + 32] : -1;
            int before = __shfl_up_sync(0xffffffffu, e, 1);
            if (lane == 0) before = last;
            const bool ok = e > before && e < pages;
            if (i < count) {
                rising &= ok;
                if (ok) atomicOr(bytes + (e >> 2), 1u << (8 * (e & 3) + row));
            }
            last = __shfl_sync(0xffffffffu, e, 31);
            e = ahead;
        }
    }
    if (__syncthreads_or(!rising)) {
        for (int i = threadIdx.x; i < words; i += kSelThreads) bytes[i] = 0;
        __syncthreads();
        for (int row = warp; row < rows; row += kSelWarps)
            mine.in_order(row, lane, [&](int, bool, bool taken, int e) {
                if (taken) atomicOr(bytes + (e >> 2), 1u << (8 * (e & 3) + row));
            });
        if (threadIdx.x == 0 && rank == 0) flag_error(p.err, PKV_DEVERR_PAGE_LIST);
        __syncthreads();
    }
    // the pages that some row lists, in order: a thread takes neighbouring words
    int n;
    {
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
        const int i0 = int(int64_t(count) * rank / C), i1 = int(int64_t(count) * (rank + 1) / C);   // this CTA's
        for (int w = w0; w < w1; ++w)
            for (uint32_t x = listed(w); x; x &= x - 1, ++at)
                if (at >= i0 && at < i1) entry[at - i0].x = 4 * w + (__ffs(x) - 1) / 8;
        n = i1 - i0;
        __syncthreads();
        bool whole = true;
        for (int i = threadIdx.x; i < n; i += kSelThreads) {
            entry[i].y = mine.block(entry[i].x);
            whole &= entry[i].y >= 0;
        }
        if (__syncthreads_or(!whole)) {
            if (warp == 0) {
                const int k = mine.close_up(entry, n, lane);
                if (lane == 0) kept = k;
            }
            __syncthreads();
            n = kept;
        }
    }

    // ---- the first pages, on their way; the query operand (rows g, g + 8 in Q's column tiles 0, 1)
    Ring<Math, true> ring{p, &k_map, &v_map, entry, n, kvh, warp, lane, smem + warp * RING, sides + warp * STAGES * Math::SIDE,
                          k_full + warp * STAGES, v_full + warp * STAGES, 0, 0, 0u, 0u};
    ring.begin();
    queries.store(p, Q, q_most);
    __syncthreads();
    float krow[2];       // what turns the products of rows g, g + 8 into base-2 scores
    uint32_t bit[2];     // their query token, as a bit (0: no row)
    int seen[2];         // what it sees
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = g + 8 * r;
        krow[r] = column_scale<Math>(p, q_most, row);
        bit[r] = row < cols ? 1u << (row / G) : 0u;
        seen[r] = row < cols ? mine.visible(row / G) : 0;
    }
    const uint32_t every = (1u << rows) - 1u;

    // ---- the pages, two at a step.  Rows that do not list a page have weights of 0 in it, which would not stop an infinity
    // or NaN in V.  The first pass takes them so; a warp whose sums are not all finite takes its pages again, with care:
    // those rows then keep their sums.
    float o[NMT][2][4];  // rows g, g + 8 x dims dim(mt, 2t), dim(mt, 2t + 1), and kNext further
    float m_run[2], l_part[2], vref[2];
    for (bool care = false;; care = true) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            m_run[r] = -INFINITY;
            l_part[r] = 0.f;
            vref[r] = 1.17549435e-38f;
        }
#pragma unroll
        for (int mt = 0; mt < NMT; ++mt)
#pragma unroll
            for (int j = 0; j < 2; ++j) o[mt][j][0] = o[mt][j][1] = o[mt][j][2] = o[mt][j][3] = 0.f;
        bool came = true;
        int st = 0;
        for (int at = warp; at < n; at += 2 * kSelWarps) {
            const bool two = at + kSelWarps < n;
            const int page[2] = {entry[at].x, two ? entry[at + kSelWarps].x : 0};
            const uint8_t *const stage[2] = {ring.stage(st), ring.stage(st + 1)}, *const side[2] = {ring.side(st), ring.side(st + 1)};
            came &= ring.wait_k(st);
            if (two) came &= ring.wait_k(st + 1);
            float s[2][2][4];   // page, token half: rows g, g + 8 x tokens 8 half + 2t, + 1
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int h = 0; h < 2; ++h) s[b][h][0] = s[b][h][1] = s[b][h][2] = s[b][h][3] = 0.f;
            // a page that is missing: of what its stage held, and left out below
            Math::keys(stage, lane, [&](int kk, const uint32_t (&a)[2][4]) {
                const uint4 x = reinterpret_cast<const uint4*>(Q)[kk * 32 + lane];
                const uint32_t q[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int h = 0; h < 2; ++h) mma16816<Math::kBf>(s[b][h], q, a[b][h], a[b][2 + h]);
            });
            uint32_t who[2];
            bool edge[2];   // some row does not see all of the page's tokens
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                who[b] = b && !two ? 0u : (bytes[page[b] >> 2] >> (8 * (page[b] & 3))) & 0xffu;
                edge[b] = page[b] * kBS + kBS > vis_all;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float k = Math::kHalf ? krow[c >> 1] : krow[c >> 1] * Math::k_scale(side[b], 8 * h + 2 * t + (c & 1));
                        s[b][h][c] *= k;
                    }
                if (edge[b] || who[b] != every) {
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int live = who[b] & bit[r] ? seen[r] - page[b] * kBS : 0;
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                if (8 * h + 2 * t + c >= live) s[b][h][2 * r + c] = -INFINITY;
                    }
                }
            }
            __syncwarp();   // the K tiles have been read
            ring.fill_k(st);
            ring.fill_k(st + 1);
            float f[2];
            bool rescale = false;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float bm = -INFINITY;
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int h = 0; h < 2; ++h) bm = fmaxf(bm, fmaxf(s[b][h][2 * r], s[b][h][2 * r + 1]));
                bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 1));
                bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 2));
                const float mu = reference<Math>(bm, m_run[r], f[r]);
                float sum = 0.f;
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        s[b][h][2 * r] = exp2_ftz(s[b][h][2 * r] - mu);
                        s[b][h][2 * r + 1] = exp2_ftz(s[b][h][2 * r + 1] - mu);
                        sum += s[b][h][2 * r] + s[b][h][2 * r + 1];
                    }
                l_part[r] = l_part[r] * f[r] + sum;
                rescale |= f[r] != 1.f;
            }
            came &= ring.wait_v(st);
            if (two) came &= ring.wait_v(st + 1);
            if (!came) {
                ring.give_up();
                break;
            }
            // What a row's weights are multiplied by in the operand.  8-bit caches: the V scales that a row's unit grows with are
            // those of the pages it lists, so that another row's page, however large, takes no bits of its weights.
            float unit[2][2] = {{Math::kPUnit, Math::kPUnit}, {Math::kPUnit, Math::kPUnit}};   // row, page
            if constexpr (Math::kByte) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
#pragma unroll
                    for (int b = 0; b < 2; ++b) unit[r][b] = who[b] & bit[r] ? Math::v_scale(side[b]) : 0.f;
                    const float grow = v_units<Math>(unit[r], vref[r]);
                    f[r] *= grow;
                    rescale |= grow != 1.f;
                }
            }
            if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
                for (int mt = 0; mt < NMT; ++mt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        o[mt][j][0] *= f[0]; o[mt][j][1] *= f[0];
                        o[mt][j][2] *= f[1]; o[mt][j][3] *= f[1];
                    }
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                if (b && !two) break;
                uint32_t hi[4], lo[4];   // P operand
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        split2<Math>(s[b][h][2 * r] * unit[r][b], s[b][h][2 * r + 1] * unit[r][b], hi[2 * h + r], lo[2 * h + r]);
                if (!edge[b] && (!care || who[b] == every)) {
                    Math::template tiles<false, 2>(stage[b], side[b], 0u, 0u, lane, [&](int m0, auto& a) {
                        constexpr int N = sizeof(a) / 16;
#pragma unroll
                        for (int i = 0; i < N; ++i)
#pragma unroll
                            for (int j = 0; j < 2; ++j) mma16816<Math::kBf>(o[m0 + i][j], hi, a[i][j], a[i][2 + j]);
#pragma unroll
                        for (int i = 0; i < N; ++i)
#pragma unroll
                            for (int j = 0; j < 2; ++j) mma16816<Math::kBf>(o[m0 + i][j], lo, a[i][j], a[i][2 + j]);
                    });
                } else {
                    // rows that do not list the page keep their sums; a page that some row sees in part is taken for one query
                    // token at a time, without the tokens it does not see
                    for (uint32_t left = who[b]; left;) {
                        const uint32_t now = edge[b] ? left & (0u - left) : who[b];
                        left &= ~now;
                        const int live = edge[b] ? mine.visible(__ffs(now) - 1) - page[b] * kBS : kBS, k = 2 * t;
                        const uint32_t m01 = (k < live ? 0xffffu : 0u) | (k + 1 < live ? 0xffff0000u : 0u);
                        const uint32_t m23 = (k + 8 < live ? 0xffffu : 0u) | (k + 9 < live ? 0xffff0000u : 0u);
                        Math::template tiles<true, 1>(stage[b], side[b], m01, m23, lane, [&](int m0, auto& a) {
                            constexpr int N = sizeof(a) / 16;
#pragma unroll
                            for (int i = 0; i < N; ++i)
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    float(&to)[4] = o[m0 + i][j];
                                    float x[4] = {to[0], to[1], to[2], to[3]};
                                    mma16816<Math::kBf>(x, hi, a[i][j], a[i][2 + j]);
                                    mma16816<Math::kBf>(x, lo, a[i][j], a[i][2 + j]);
#pragma unroll
                                    for (int c = 0; c < 4; ++c)
                                        if (now & bit[c >> 1]) to[c] = x[c];
                                }
                        });
                    }
                }
            }
            __syncwarp();   // the V tiles have been read
            ring.fill_v(st);
            ring.fill_v(st + 1);
            st = st + 2 == STAGES ? 0 : st + 2;
        }
        if (care || !came) break;
        bool finite = true;
#pragma unroll
        for (int mt = 0; mt < NMT; ++mt)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) finite &= fabsf(o[mt][j][c]) < INFINITY;
        if (__all_sync(0xffffffffu, finite)) break;
        ring.begin();
    }

    // The next kernel may come now: its CTAs, were they here from the start, would take the places beside some of these
    // CTAs and leave others alone, and this grid's successor would run as unevenly (as in attention_selected.cu; 16 x 3 tokens over 101 pages of 4 e4m3
    // heads: 19.2 us early, 19.1 late).
    grid_dep_launch();
    // ---- the warp's partial, and the merges
    __syncwarp();
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const float back = (Math::kByte ? vref[r] : 1.f) * (1.f / Math::kPUnit);
        float l = l_part[r];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        const int row = g + 8 * r;
        if (t == 0) {
            part.m[warp][row] = m_run[r];
            part.l[warp][row] = l;
        }
        if (row < cols) {
            float* to = reinterpret_cast<float*>(smem + warp * RING) + row * OW;
#pragma unroll
            for (int mt = 0; mt < NMT; ++mt)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int c = 0; c < 2; ++c) to[Math::dim(mt, 2 * t + c) + j * Math::kNext] = o[mt][j][2 * r + c] * back;
        }
    }
    merge_and_store<COLS, D>(p, cl, part, reinterpret_cast<float*>(smem), RING / 4,
                             reinterpret_cast<float4*>(reinterpret_cast<uint8_t*>(entry) + p.list_bytes), tile.r0, cols, kvh, G);
}

// The kernel may take kSelectedSmem of dynamic shared memory: said once per kernel and device.
template <int KIND, int D>
cudaError_t launch_rows(const SelectedParams& p, int64_t units, int cluster, size_t lists, const CUtensorMap& km, const CUtensorMap& vm,
                        cudaStream_t st) {
    static PerDevice ready;
    int dev = 0, one = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = cudaError_t(ready.get(dev, &one, [](int* v) {
        *v = 1;
        return int(cudaFuncSetAttribute(attention_rows_kernel<KIND, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelectedSmem));
    }));
    if (e != cudaSuccess) return e;
    const size_t smem = ring_bytes<PageMath<KIND, D>>() + lists + (cluster > 1 ? exchange_bytes<16, D>() : 0);
    return launch_cluster_kernel(attention_rows_kernel<KIND, D>, dim3(unsigned(units * cluster), p.num_kv_heads), dim3(kSelThreads),
                                 unsigned(cluster), spread(units * cluster * p.num_kv_heads, smem), st, km, vm, p);
}

template <int KIND>
cudaError_t launch_kind(const SelectedParams& p, int64_t units, int cluster, size_t lists, const CUtensorMap& km,
                        const CUtensorMap& vm, cudaStream_t st) {
    return p.head_dim == 128 ? launch_rows<KIND, 128>(p, units, cluster, lists, km, vm, st)
                             : launch_rows<KIND, 64>(p, units, cluster, lists, km, vm, st);
}

}  // namespace

cudaError_t launch_attention_rows(const SelectedParams& p, int cache_kind, int64_t units, int C, size_t lists, const CUtensorMap& km,
                                  const CUtensorMap& vm, cudaStream_t stream) {
    switch (cache_kind) {
        case PKV_CACHE_F16: return launch_kind<PKV_CACHE_F16>(p, units, C, lists, km, vm, stream);
        case PKV_CACHE_BF16: return launch_kind<PKV_CACHE_BF16>(p, units, C, lists, km, vm, stream);
        case PKV_CACHE_K8V4: return launch_kind<PKV_CACHE_K8V4>(p, units, C, lists, km, vm, stream);
        case PKV_CACHE_I8: return launch_kind<PKV_CACHE_I8>(p, units, C, lists, km, vm, stream);
        default: return launch_kind<PKV_CACHE_E4M3>(p, units, C, lists, km, vm, stream);
    }
}

}  // namespace pkv
