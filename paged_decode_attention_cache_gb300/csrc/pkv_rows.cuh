// pkv_rows.cuh -- which sequence a query token belongs to and what it sees.
#pragma once

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

// A query token: its sequence (-1: none, a row behind the last sequence's), its visible tokens (0: none), and
// whether the sequence's context is longer than its block table (vis is then cut to the table).
struct Row {
    int s, vis;
    bool over;
};

// Query token r, by a whole warp: sequence s's tokens are rows cu[s] .. cu[s + 1] - 1 (or, without cu, q_len each),
// and the last of them sees the sequence's whole context.  All lanes probe the remaining range of cu at once.
__device__ __forceinline__ Row find_row(const int32_t* cu, const int32_t* context_lens, int num_seqs, int q_len,
                                        int max_blocks, int r, int lane) {
    int s, behind;   // behind: the sequence's query tokens from this one on
    if (!cu) {
        s = r / q_len;
        behind = q_len - (r - s * q_len);
        if (s >= num_seqs) return {-1, 0, false};
    } else {
        if (num_seqs < 1 || r >= cu[num_seqs] || r < cu[0]) return {-1, 0, false};
        int lo = 0, hi = num_seqs;   // cu[lo] <= r; the answer is in [lo, hi)
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32, at = lo + lane * step;
            const uint32_t m = __ballot_sync(0xffffffffu, at < hi && cu[at < hi ? at : lo] <= r) | 1u;
            lo += (31 - __clz(m)) * step;   // the last probe that begins at or before r
            hi = min(hi, lo + step);
        }
        s = lo;
        behind = cu[s + 1] - r;
        if (behind < 1) return {-1, 0, false};   // lengths that do not rise
    }
    const int64_t ctx = context_lens[s];
    const int64_t cap = int64_t(max_blocks) * kBlockSize;
    return {s, int(min(max(ctx - behind + 1, int64_t(0)), cap)), ctx > cap};
}

}  // namespace pkv
