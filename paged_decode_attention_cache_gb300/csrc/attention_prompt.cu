// attention_prompt.cu -- attention over lists of pages for chunks of prompts over fp16 and
// bf16 caches (attention_selected.cuh): 128 query rows to a CTA on tcgen05.
//
// 128 / g neighbouring query tokens with a kv head's g query heads are the M side of the MMAs; the
// CTA reads the union of their lists once, 4 pages (64 tokens) at a step, and masks by row:
//   S = Q K^T   both operands in shared memory (K-major, 128-byte swizzle), S in TMEM;
//   softmax     a thread owns a row: no shuffles, its maximum and sum stay with it;
//   O += P V    P from TMEM, where it takes S's place 32 columns at a time, as two 16-bit halves
//               (hi, lo) and so two MMAs a k step; V as the cache has it (N-major); O in TMEM.
// One thread issues the copies, one the MMAs, four warps do the softmax.  K, V and S have two
// buffers each: the next step's S is there when a softmax ends, and its O += P V runs under the
// next one.  256 columns of TMEM to a CTA; at 128 dims 96 KB of tiles, 8 bytes for each page that its
// lists may hold together, and 4 bytes (groups of 2 and 1: 8 and 16) for each column of the block table.
// Two CTAs to an SM as far as that goes: with lists of 64 up to 1,260 columns (20 thousand tokens) for
// groups of 4, 630 for groups of 1; the chunks below take 149 us, not 94, in a table of 1280 columns.
//
// Whatever the lists have in common, the union is no larger than what smaller tiles would read
// together, and a page costs 128 rows here what 16 rows cost mma.sync.
//
// Bound: the chain S -> softmax -> P -> O of a step, 2.7 thousand clocks of which the MMAs of an SM's two CTAs
// take 1.5, after a prologue of 20 (the union).  1001 tokens of 3 sequences, 32 query heads over 8 kv heads of
// 128 dims, 64 of 1024 pages each: 94 us (attention_selected_rows.cu: 174); tensor pipes 34 % busy.
#include <algorithm>

#include "attention_selected.cuh"

namespace pkv {

namespace {

constexpr int kRows = 128, kStepPages = 4, kStepTokens = kStepPages * kBS;
constexpr int kSoftWarps = 4, kPromptWarps = kSoftWarps + 2, kPromptThreads = kPromptWarps * 32;

// ---------------------------------------------------------------- tcgen05

__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t at, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols) : "memory");
}
__device__ __forceinline__ void fence_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// mbar_wait without the long suspension, whose end costs more than these waits last (the limit is the same).
__device__ __forceinline__ bool wait_soon(uint64_t* bar, uint32_t parity) {
    const uint32_t a = smem_addr(bar);
    if (mbar_try_wait(a, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (mbar_try_wait(a, parity)) return true;
        if (global_timer_ns() - t0 > kWaitLimitNs) return false;
    }
}

// The barrier's phase completes when this thread's MMAs so far have.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// d (+)= A B, A in shared memory
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a),
        "l"(b), "r"(idesc), "r"(uint32_t(add))
        : "memory");
}
// d (+)= A B, A in TMEM
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a),
        "l"(b), "r"(idesc), "r"(uint32_t(add))
        : "memory");
}

#define PKV_R32(X) \
    X(0), X(1), X(2), X(3), X(4), X(5), X(6), X(7), X(8), X(9), X(10), X(11), X(12), X(13), X(14), X(15), X(16), X(17), X(18), X(19), \
        X(20), X(21), X(22), X(23), X(24), X(25), X(26), X(27), X(28), X(29), X(30), X(31)

// 32 columns of this warp's 32 lanes of TMEM, a lane to a thread
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&r)[32]) {
#define PKV_OUT(i) "=r"(r[i])
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, "
        "%19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : PKV_R32(PKV_OUT)
        : "r"(at)
        : "memory");
#undef PKV_OUT
}
// The loads so far have come: r may be used behind it.
__device__ __forceinline__ void wait_ld(uint32_t (&r)[32]) {
#define PKV_TIE(i) "+r"(r[i])
    asm volatile("tcgen05.wait::ld.sync.aligned;" : PKV_R32(PKV_TIE)::"memory");
#undef PKV_TIE
}
__device__ __forceinline__ void tmem_store(uint32_t at, const uint32_t (&r)[32]) {
#define PKV_IN(i) "r"(r[i])
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
        "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::PKV_R32(PKV_IN),
        "r"(at)
        : "memory");
#undef PKV_IN
}
#undef PKV_R32

// Shared-memory operand with the 128-byte swizzle: address, and the strides in bytes between its 8-row (K-major) or
// 8-k (N-major) groups and, N-major, between its 64-element groups along N.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return uint64_t((addr >> 4) & 0x3fffu) | uint64_t((lbo >> 4) & 0x3fffu) << 16 | uint64_t((sbo >> 4) & 0x3fffu) << 32 |
           uint64_t(1) << 46 | uint64_t(2) << 61;
}
// fp32 sums of 16-bit products, M = 128
template <bool BF>
__device__ __forceinline__ constexpr uint32_t instruction(int n, bool b_n_major) {
    return 1u << 4 | (BF ? 1u << 7 | 1u << 10 : 0u) | (b_n_major ? 1u << 16 : 0u) | uint32_t(n / 8) << 17 | uint32_t(kRows / 16) << 24;
}

// ---------------------------------------------------------------- the kernel

template <bool BF, int D>
__global__ void __launch_bounds__(kPromptThreads, 2)
attention_prompt_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map, const SelectedParams p) {
    using T = typename std::conditional<BF, __nv_bfloat16, __half>::type;
    constexpr int NC = D / 64;                      // 64-dim chunks of a row
    constexpr int CHUNK = kRows * 128, TILE = NC * CHUNK;               // bytes of a chunk of Q, and of all
    constexpr int KV_CHUNK = kStepTokens * 128, KV_TILE = NC * KV_CHUNK;   // of a step's K, or V
    // as PageMath's; here the sums of the weights have fp16's unit too, 2^kShift
    constexpr float kSlack = BF ? 8.f : 1.f, kShift = BF ? 0.f : 14.f;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t *const sq = smem, *const sk = smem + TILE, *const sv = sk + 2 * KV_TILE;
    int2* const entry = reinterpret_cast<int2*>(sv + 2 * KV_TILE);            // the union's pages: page, block
    uint32_t* const marks = reinterpret_cast<uint32_t*>(entry + p.entries);   // [pages][mark words]: the tokens that list a page
    __shared__ uint64_t k_full[2], v_full[2], s_done[2], p_done[2], o_done[2];   // of the two buffers
    __shared__ uint32_t tmem_at;
    __shared__ int scan[kPromptWarps], kept, failed, counts[kRows], limits[kRows];
    __shared__ uint32_t redo[kRows / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int b = 0; b < 2; ++b) {
            mbar_init(&k_full[b], 1);
            mbar_init(&v_full[b], 1);
            mbar_init(&s_done[b], 1);
            mbar_init(&p_done[b], kSoftWarps);
            mbar_init(&o_done[b], 1);
        }
        fence_barrier_init();
        prefetch_tensormap(&k_map);
        prefetch_tensormap(&v_map);
        failed = 0;
    }
    if (threadIdx.x < kRows / 32) redo[threadIdx.x] = 0;
    grid_dep_wait();
    const int kvh = blockIdx.y, G = p.num_heads / p.num_kv_heads;
    const RowTile tile = find_tile(p.cu_q, p.num_seqs, p.num_rows, p.q_len, p.tile_rows, int(blockIdx.x), lane);
    if (tile.s < 0) return;
    const SelectedTile mine(p, tile, kvh);
    if (mine.over() && kvh == 0 && threadIdx.x == 0) flag_error(p.err, PKV_DEVERR_CAPACITY);
    const int rows = tile.rows, MW = (p.tile_rows + 31) / 32;   // query tokens; words of a page's marks
    const int pages = mine.pages(rows - 1);

    // ---- the queries, swizzled as TMA would have them; rows of no token are zeros
    for (int i0 = threadIdx.x; i0 < kRows * NC * 8; i0 += 8 * kPromptThreads) {
        uint4 x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = i0 + j * kPromptThreads, c = i % (NC * 8), row = i / (NC * 8);
            x[j] = make_uint4(0u, 0u, 0u, 0u);
            if (row < rows * G)
                x[j] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) +
                                                            ((int64_t(tile.r0) + row / G) * p.num_heads + int64_t(kvh) * G + row % G) * D) + c);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = i0 + j * kPromptThreads, c = i % (NC * 8), row = i / (NC * 8);
            if (i < kRows * NC * 8) *reinterpret_cast<uint4*>(sq + (c >> 3) * CHUNK + row * 128 + 16 * ((c & 7) ^ (row & 7))) = x[j];
        }
    }
    fence_proxy_async_smem();

    // ---- the union of the lists, if every entry is in range and above the one before it; else the slow way
    for (int i = threadIdx.x; i < pages * MW; i += kPromptThreads) marks[i] = 0;
    if (threadIdx.x < rows) {
        counts[threadIdx.x] = mine.count(threadIdx.x);
        limits[threadIdx.x] = mine.pages(threadIdx.x);
    }
    if (warp == 0) tmem_alloc(&tmem_at, 256);
    __syncthreads();
    // a warp takes four rows at a time, 64 entries of each: their loads are in flight together
    bool rising = true;
    for (int r0 = warp; r0 < rows; r0 += 4 * kPromptWarps) {
        int count[4], last[4], most = 0;   // last: the entry before these 64
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = r0 + j * kPromptWarps;
            count[j] = row < rows ? counts[row] : 0;
            most = max(most, count[j]);
            last[j] = -1;
        }
        for (int k0 = 0; k0 < most; k0 += 64) {
            int e[4][2];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int k = k0 + 32 * h + lane;
                    e[j][h] = k < count[j] ? mine.list(r0 + j * kPromptWarps)[k] : INT_MAX;
                }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int k = k0 + 32 * h + lane, row = r0 + j * kPromptWarps;
                    int before = __shfl_up_sync(0xffffffffu, e[j][h], 1);
                    if (lane == 0) before = last[j];
                    last[j] = __shfl_sync(0xffffffffu, e[j][h], 31);
                    if (k >= count[j]) continue;
                    const bool ok = e[j][h] > before && e[j][h] < limits[row];
                    rising &= ok;
                    if (ok) atomicOr(marks + e[j][h] * MW + (row >> 5), 1u << (row & 31));
                }
        }
    }
    if (__syncthreads_or(!rising)) {
        for (int i = threadIdx.x; i < pages * MW; i += kPromptThreads) marks[i] = 0;
        __syncthreads();
        for (int row = warp; row < rows; row += kPromptWarps)
            mine.in_order(row, lane, [&](int, bool, bool taken, int e) {
                if (taken) atomicOr(marks + e * MW + (row >> 5), 1u << (row & 31));
            });
        if (threadIdx.x == 0) flag_error(p.err, PKV_DEVERR_PAGE_LIST);
        __syncthreads();
    }
    int n;
    {
        const int per = (pages + kPromptThreads - 1) / kPromptThreads, a = min(int(threadIdx.x) * per, pages), b = min(a + per, pages);
        auto listed = [&](int page) {
            uint32_t any = 0;
            for (int w = 0; w < MW; ++w) any |= marks[page * MW + w];
            return any != 0;
        };
        int c = 0;
        for (int i = a; i < b; ++i) c += listed(i);
        int incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        if (lane == 31) scan[warp] = incl;
        __syncthreads();
        int at = incl - c;
        n = 0;
        for (int w = 0; w < kPromptWarps; ++w) {
            if (w < warp) at += scan[w];
            n += scan[w];
        }
        for (int i = a; i < b; ++i)
            if (listed(i)) entry[at++].x = i;
        __syncthreads();
        bool whole = true;
#pragma unroll 4
        for (int i = threadIdx.x; i < n; i += kPromptThreads) {
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
    const uint32_t tmem = tmem_at, tmem_s = tmem, tmem_o = tmem + 128;
    fence_after_sync();
    const int steps = (n + kStepPages - 1) / kStepPages;

    if (warp == kSoftWarps + 1) {
        // ---- the copies, by one thread: K's tile is free when S has been worked out, V's when it has been added
        if (lane == 0) {
            auto copy = [&](const CUtensorMap* map, uint8_t* dst, uint64_t* bar, int step) {
                const int first = step * kStepPages, k = min(kStepPages, n - first);
                mbar_arrive_expect_tx(bar, k * kBS * D * 2);
                for (int i = 0; i < k; ++i)
#pragma unroll
                    for (int c = 0; c < NC; ++c)
                        tma_load_2d(dst + c * KV_CHUNK + i * kBS * 128, map, kvh * D * 2 + c * 128, entry[first + i].y * kBS, bar);
            };
            for (int i = 0; i < steps; ++i) {
                const int b = i & 1;
                const uint32_t before = ((i >> 1) & 1) ^ 1u;   // the parity of the buffer's last use
                if (i > 1 && !wait_soon(&s_done[b], before)) break;
                copy(&k_map, sk + b * KV_TILE, &k_full[b], i);
                if (i > 1 && !wait_soon(&o_done[b], before)) break;
                copy(&v_map, sv + b * KV_TILE, &v_full[b], i);
            }
        }
    } else if (warp == kSoftWarps) {
        // ---- the MMAs, by one thread
        if (lane == 0) {
            // the operands' descriptors: an offset is added to their address field
            const uint64_t q0 = operand(smem_addr(sq), 16, 1024), k0 = operand(smem_addr(sk), 16, 1024);
            const uint64_t v0 = operand(smem_addr(sv), KV_CHUNK, 1024);
            auto scores = [&](int i) {   // S of step i
                const int b = i & 1;
                const uint32_t parity = (i >> 1) & 1;
                if (!wait_soon(&k_full[b], parity)) return false;
                if (i > 1 && !wait_soon(&o_done[b], parity ^ 1u)) return false;   // P of step i - 2 was there
                fence_after_sync();
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    mma_ss(tmem_s + b * kStepTokens, q0 + (((ks >> 2) * CHUNK + (ks & 3) * 32) >> 4),
                           k0 + ((b * KV_TILE + (ks >> 2) * KV_CHUNK + (ks & 3) * 32) >> 4), instruction<BF>(kStepTokens, false), ks > 0);
                mma_commit(&s_done[b]);
                return true;
            };
            bool came = steps > 0 ? scores(0) : true;
            for (int i = 0; i < steps && came; ++i) {
                const int b = i & 1;
                const uint32_t parity = (i >> 1) & 1;
                if (i + 1 < steps && !(came = scores(i + 1))) break;
                if (!(came = wait_soon(&v_full[b], parity) && wait_soon(&p_done[b], parity))) break;
                fence_after_sync();
                const uint32_t pa = tmem_s + b * kStepTokens;
                const uint64_t vb = v0 + ((b * KV_TILE) >> 4);
                mma_ts(tmem_o, pa, vb, instruction<BF>(D, true), i > 0);
                mma_ts(tmem_o, pa + 16, vb, instruction<BF>(D, true), true);
#pragma unroll
                for (int ks = 1; ks < kStepTokens / 16; ++ks) {
                    const uint32_t at = pa + 32 * (ks >> 1) + 8 * (ks & 1);   // hi; lo is 16 columns on
                    mma_ts(tmem_o, at, vb + ks * 128, instruction<BF>(D, true), true);
                    mma_ts(tmem_o, at + 16, vb + ks * 128, instruction<BF>(D, true), true);
                }
                mma_commit(&o_done[b]);
            }
            if (!came) {
                // something did not come: nothing is under way when the CTA ends (what was not started runs into the limit)
                flag_error(p.err, PKV_DEVERR_TIMEOUT);
                failed = 1;
                for (int b = 0; b < 2; ++b) {
                    mbar_wait(&k_full[b], 0);
                    mbar_wait(&k_full[b], 1);
                    mbar_wait(&v_full[b], 0);
                    mbar_wait(&v_full[b], 1);
                }
                mma_commit(&s_done[0]);
                mbar_wait(&s_done[0], 0);
                mbar_wait(&s_done[0], 1);
            }
        }
    } else {
        // ---- a row to a thread
        const int row = warp * 32 + lane, token = min(row / G, rows - 1);
        const bool on = row < rows * G;
        const int vis = mine.visible(token), vis_all = mine.visible(0), vis_most = mine.visible(rows - 1);
        const uint32_t lanes = uint32_t(warp * 32) << 16;   // this warp's lanes of TMEM
        const uint32_t* my_marks = marks + (token >> 5);
        const uint32_t my_bit = on ? 1u << (token & 31) : 0u;
        float m = -INFINITY, l = 0.f;
        bool came = true;
        for (int i = 0; i < steps; ++i) {
            const int first = i * kStepPages, k = min(kStepPages, n - first);
            // What is added to the scores of the step's pages: 0, or -inf where the row does not list the page.  Where some row
            // sees a page in part, or there are fewer than 4, tokens are left out one by one instead.
            float bias[kStepPages];
            bool cut = k < kStepPages, edge = cut;
#pragma unroll
            for (int b = 0; b < kStepPages; ++b) {
                const int page = entry[b < k ? first + b : first].x;
                bias[b] = b < k && (my_marks[page * MW] & my_bit) ? 0.f : -INFINITY;
                cut |= page * kBS + kBS > vis_most;
                edge |= page * kBS + kBS > vis_all;
            }
            const int buf = i & 1;
            const uint32_t parity = (i >> 1) & 1, tmem_p = tmem_s + buf * kStepTokens + lanes;
            came = __all_sync(0xffffffffu, wait_soon(&s_done[buf], parity));
            if (!came) break;
            fence_after_sync();
            // A chunk is 32 tokens, two pages; the next one's scores are on their way while one is worked on.
            constexpr int CH = kStepTokens / 32;
            uint32_t r[2][32];
            float most = -INFINITY, ref = 0.f, f = 1.f;
            auto reference = [&] {
                const bool grow = most > m + kSlack;
                const float now = grow ? most : m;
                ref = now == -INFINITY ? 0.f : now;
                f = grow && m > -INFINITY ? exp2_ftz(m - ref) : 1.f;
                m = now;
                l *= f;
                if (__any_sync(0xffffffffu, f != 1.f)) {   // the sums so far, when the last step's have been added
                    came = __all_sync(0xffffffffu, wait_soon(&o_done[buf ^ 1], ((i - 1) >> 1) & 1));
                    fence_after_sync();
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        tmem_load(tmem_o + lanes + 32 * c, r[0]);
                        wait_ld(r[0]);
#pragma unroll
                        for (int j = 0; j < 32; ++j) r[0][j] = __float_as_uint(__uint_as_float(r[0][j]) * f);
                        tmem_store(tmem_o + lanes + 32 * c, r[0]);
                    }
                }
            };
            // the weights of two tokens in the place of their scores: the pair's 16-bit halves, and what they leave
            auto weights = [&](float x, float y, uint32_t& hi, uint32_t& lo) {
                x = exp2_ftz(x);
                y = exp2_ftz(y);
                l += x + y;
                hi = pack2<BF>(x, y);
                const float2 back = Half16<T>::unpack2(hi);
                lo = pack2<BF>(x - back.x, y - back.y);
            };
            if (!edge) {
                tmem_load(tmem_p, r[0]);
                wait_ld(r[0]);
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    if (c + 1 < CH) tmem_load(tmem_p + 32 * (c + 1), r[(c + 1) & 1]);
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        most = fmaxf(most, fmaf(__uint_as_float(r[c & 1][j]), p.scale_log2, bias[2 * c + (j >> 4)]));
                    if (c + 1 < CH) wait_ld(r[(c + 1) & 1]);
                }
                reference();
                tmem_load(tmem_p, r[0]);
#pragma unroll
                for (int b = 0; b < kStepPages; ++b) bias[b] += kShift - ref;
                wait_ld(r[0]);
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    if (c + 1 < CH) tmem_load(tmem_p + 32 * (c + 1), r[(c + 1) & 1]);
                    uint32_t w[32];
#pragma unroll
                    for (int j = 0; j < 32; j += 2)
                        weights(fmaf(__uint_as_float(r[c & 1][j]), p.scale_log2, bias[2 * c + (j >> 4)]),
                                fmaf(__uint_as_float(r[c & 1][j + 1]), p.scale_log2, bias[2 * c + (j >> 4)]), w[j / 2], w[16 + j / 2]);
                    if (c + 1 < CH) wait_ld(r[(c + 1) & 1]);
                    tmem_store(tmem_p + 32 * c, w);
                }
            } else {
                // what the row sees of a chunk's pages
                auto live = [&](int c, int h) {
                    if (2 * c + h >= k) return 0;
                    const int page = entry[first + 2 * c + h].x;
                    return my_marks[page * MW] & my_bit ? vis - page * kBS : 0;
                };
                auto score = [&](uint32_t bits, int j, int lo, int hi) {
                    return (j & 15) < (j < 16 ? lo : hi) ? __uint_as_float(bits) * p.scale_log2 : -INFINITY;
                };
#pragma unroll 1
                for (int c = 0; c < CH; ++c) {
                    const int lo = live(c, 0), hi = live(c, 1);
                    tmem_load(tmem_p + 32 * c, r[0]);
                    wait_ld(r[0]);
#pragma unroll
                    for (int j = 0; j < 32; ++j) most = fmaxf(most, score(r[0][j], j, lo, hi));
                }
                reference();
#pragma unroll 1
                for (int c = 0; c < CH; ++c) {
                    const int lo = live(c, 0), hi = live(c, 1);
                    tmem_load(tmem_p + 32 * c, r[0]);
                    wait_ld(r[0]);
                    uint32_t w[32];
#pragma unroll
                    for (int j = 0; j < 32; j += 2)
                        weights(score(r[0][j], j, lo, hi) + (kShift - ref), score(r[0][j + 1], j + 1, lo, hi) + (kShift - ref), w[j / 2],
                                w[16 + j / 2]);
                    tmem_store(tmem_p + 32 * c, w);
                }
            }
            if (cut) {   // tokens behind the last one, and pages that are none, may hold anything: 0 times it would not be 0
                came &= __all_sync(0xffffffffu, mbar_wait(&v_full[buf], parity)) != 0;
                for (int j = threadIdx.x; j < kStepTokens * NC * 8; j += kSoftWarps * 32) {
                    const int tok = j / (NC * 8), c = j % (NC * 8), b = tok / kBS;
                    const bool keep = b < k && entry[first + b].x * kBS + tok % kBS < vis_most;
                    if (!keep) *reinterpret_cast<uint4*>(sv + buf * KV_TILE + (c >> 3) * KV_CHUNK + tok * 128 + 16 * (c & 7)) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
            }
            if (!came) break;
            wait_st();
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_done[buf]);
        }
        // ---- the outputs
        if (came && steps > 0) came = __all_sync(0xffffffffu, mbar_wait(&o_done[(steps - 1) & 1], ((steps - 1) >> 1) & 1));
        if (came) {
            fence_after_sync();
            const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);   // no visible token: zeros
            const size_t at = (size_t(tile.r0 + token) * p.num_heads + size_t(kvh) * G + row % G) * D;
            bool finite = true;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t r[32];
                if (steps > 0) {
                    tmem_load(tmem_o + lanes + 32 * c, r);
                    wait_ld(r);
                }
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (steps > 0 && l != 0.f)
                        v = make_float4(__uint_as_float(r[j]) * inv, __uint_as_float(r[j + 1]) * inv, __uint_as_float(r[j + 2]) * inv,
                                        __uint_as_float(r[j + 3]) * inv);
                    finite &= fabsf(v.x) < INFINITY && fabsf(v.y) < INFINITY && fabsf(v.z) < INFINITY && fabsf(v.w) < INFINITY;
                    if (on) store_out4(p.out, p.out_dtype, at + 32 * c + j, v);
                }
            }
            if (on && !finite) atomicOr(&redo[row >> 5], 1u << (row & 31));
            fence_before_sync();
        } else {
            failed = 1;
        }
    }
    // The next kernel may come now: its CTAs, were they here from the start, would take the places beside some of these
    // CTAs and leave others alone, and this grid's successor would run as unevenly (as in attention_selected.cu; no difference measured here).
    grid_dep_launch();
    __syncthreads();
    if (warp == 0) {
        fence_after_sync();
        tmem_free(tmem, 256);
    }
    if (failed) return;

    // ---- rows that are not finite, again one by one: an infinity or NaN in V that the row does not see, times its weight of 0,
    // may have reached it
    for (int row = warp; row < rows * G; row += kPromptWarps) {
        if (!(redo[row >> 5] >> (row & 31) & 1u)) continue;
        const int token = row / G, vis = mine.visible(token);
        const int64_t head = (int64_t(tile.r0) + token) * p.num_heads + int64_t(kvh) * G + row % G;
        constexpr int E = D / 32;
        float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
        for (int d = 0; d < E; ++d) {
            q[d] = load_q(p.q, p.q_dtype, head * D + lane * E + d) * p.scale_log2;
            o[d] = 0.f;
        }
        for (int i = 0; i < n; ++i) {
            const int2 e = entry[i];
            if (!(marks[e.x * MW + (token >> 5)] >> (token & 31) & 1u)) continue;
            const int live = min(vis - e.x * kBS, kBS);
            for (int t = 0; t < live; ++t) {
                const int64_t at = ((int64_t(e.y) * kBS + t) * p.num_kv_heads + kvh) * D + lane * E;
                float s = 0.f;
#pragma unroll
                for (int d = 0; d < E; ++d) s = fmaf(q[d], Half16<T>::to_float(static_cast<const uint16_t*>(p.k)[at + d]), s);
#pragma unroll
                for (int x = 16; x >= 1; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
                // the maximum so far; 0 while there is no score above -infinity, whose weight is 0.  A sum that is infinite or not
                // a number stays so, however small its factor
                const float now = fmaxf(m, s), to = now == -INFINITY ? 0.f : now, f = m == -INFINITY ? 1.f : exp2f(m - to), w = exp2f(s - to);
                m = now;
                l = l * f + w;
#pragma unroll
                for (int d = 0; d < E; ++d) o[d] = o[d] * f + w * Half16<T>::to_float(static_cast<const uint16_t*>(p.v)[at + d]);
            }
        }
        for (int d = 0; d < E; ++d)
            store_out(p.out, p.out_dtype, size_t(head) * D + lane * E + d, l == 0.f ? 0.f : o[d] / l);
    }
}

// The kernel may take kPromptSmem of dynamic shared memory: said once per kernel and device.
constexpr int kPromptSmem = 220 * 1024;
template <bool BF, int D>
cudaError_t launch_prompt(const SelectedParams& p, int64_t units, size_t smem, const CUtensorMap& km, const CUtensorMap& vm,
                          cudaStream_t st) {
    static PerDevice ready;
    int dev = 0, one = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = cudaError_t(ready.get(dev, &one, [](int* v) {
        *v = 1;
        return int(cudaFuncSetAttribute(attention_prompt_kernel<BF, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPromptSmem));
    }));
    if (e != cudaSuccess) return e;
    return launch_kernel(attention_prompt_kernel<BF, D>, dim3(unsigned(units), p.num_kv_heads), dim3(kPromptThreads), smem, st, km, vm, p);
}

// Query tokens to a CTA, and its shared memory.
int prompt_tokens(const SelectedParams& p) { return kRows / (p.num_heads / p.num_kv_heads); }
size_t prompt_smem(const SelectedParams& p) {
    int64_t most = int64_t(prompt_tokens(p)) * p.max_pages;
    if (most > p.max_blocks) most = p.max_blocks;
    const int64_t words = (prompt_tokens(p) + 31) / 32;
    return 1024 + size_t(kRows + 4 * kStepTokens) * p.head_dim * 2 + size_t(most) * 8 + size_t(p.max_blocks) * words * 4;
}

}  // namespace

// 16-bit caches, lists that fit, sequences of two of attention_rows_kernel's tiles or more, and more than 608 of those tiles,
// two rounds of the GPU: a CTA here takes the time of several, and with fewer the GPU is not filled.  us there / here, 8 kv
// heads of 128 dims, 4 query heads each, 64 pages of 1024: 1 seq x 128 tokens (256 tiles) 30.9 / 73.6, 4 x 64 (512) 58.7 / 80.2,
// 32 x 8 (512) 59.2 / 59.9, 4 x 128 (1024) 112 / 78.9, 32 x 16 (1024) 111 / 65.5, 32 x 128 744 / 313; of 256 pages, 16 x 16
// (512) 51.2 / 45.3, 6 x 64 (768) 73.9 / 52.4; 32 pages of 256, 128 x 4 (1024, one tile a sequence) 83.7 / 114.
bool prompt_tiles(const SelectedParams& p, int cache_kind) {
    if (cache_kind != PKV_CACHE_F16 && cache_kind != PKV_CACHE_BF16) return false;
    const int64_t rows = p.num_rows, tokens = shared_tokens(p);
    return rows >= 2 * tokens * p.num_seqs && rows * p.num_kv_heads > 608 * tokens && prompt_smem(p) <= kPromptSmem;
}

cudaError_t launch_attention_prompt(SelectedParams p, int cache_kind, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t stream) {
    const size_t smem = prompt_smem(p);
    p.tile_rows = prompt_tokens(p);
    p.entries = int(std::min<int64_t>(int64_t(p.tile_rows) * p.max_pages, p.max_blocks));
    const int64_t units = p.cu_q ? int64_t(p.num_rows) / p.tile_rows + p.num_seqs
                                 : int64_t(p.num_seqs) * ((int64_t(p.q_len) + p.tile_rows - 1) / p.tile_rows);
    if (units > 0x7fffffff) return cudaErrorInvalidValue;
    if (cache_kind == PKV_CACHE_BF16)
        return p.head_dim == 128 ? launch_prompt<true, 128>(p, units, smem, km, vm, stream)
                                 : launch_prompt<true, 64>(p, units, smem, km, vm, stream);
    return p.head_dim == 128 ? launch_prompt<false, 128>(p, units, smem, km, vm, stream)
                             : launch_prompt<false, 64>(p, units, smem, km, vm, stream);
}

}  // namespace pkv
