// pkv_rows.cuh -- which sequence a query token belongs to and what it sees.
#pragma once

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

// A tile of up to R query tokens of one sequence: its sequence (-1: none), its first row and how many.
struct RowTile {
    int s, r0, rows;
};

// Tile u of R rows each, by a whole warp.  Without cu a sequence has ceil(q_len / R) tiles; with it, its tiles begin at
// cu[s] / R + s, which is at least as far apart as the tiles it needs (num_rows / R + num_seqs in all).
__device__ __forceinline__ RowTile find_tile(const int32_t* cu, int num_seqs, int num_rows, int q_len, int R, int u, int lane) {
    if (!cu) {
        const int per = (q_len + R - 1) / R, s = u / per, i = u - s * per;
        if (s >= num_seqs) return {-1, 0, 0};
        return {s, s * q_len + i * R, min(R, q_len - i * R)};
    }
    auto start = [&](int s) { return min(max(cu[s], 0), num_rows) / R + s; };
    int lo = 0, hi = num_seqs;   // start(lo) <= u; the answer is in [lo, hi)
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, at = lo + lane * step;
        const uint32_t m = __ballot_sync(0xffffffffu, at < hi && start(at < hi ? at : lo) <= u) | 1u;
        lo += (31 - __clz(m)) * step;   // the last probe that begins at or before u
        hi = min(hi, lo + step);
    }
    const int c0 = min(max(cu[lo], 0), num_rows), c1 = min(max(cu[lo + 1], 0), num_rows);
    const int64_t r0 = int64_t(c0) + int64_t(u - (c0 / R + lo)) * R;
    if (r0 < c0 || r0 >= c1) return {-1, 0, 0};
    return {lo, int(r0), min(R, c1 - int(r0))};
}

// The tokens that a query token sees, `behind` being how many of the sequence's there are from it on (itself one): the last
// one sees the whole context, as far as the block table goes.
__device__ __forceinline__ int visible_tokens(int64_t ctx, int max_blocks, int behind) {
    return int(min(max(ctx - behind + 1, int64_t(0)), int64_t(max_blocks) * kBlockSize));
}

}  // namespace pkv
