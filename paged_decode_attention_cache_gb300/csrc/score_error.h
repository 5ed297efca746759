// score_error.h -- how far a page's score, worked out by MMAs in fp32 (select_pages.cuh), may be from the exact one:
// kRelative of the page's sum of magnitudes as the kernel counts it, and kUnderflow.  Plain C++.
#pragma once

namespace pkv {

// BF: bounds and folded queries in bf16; else in fp16, queries scaled to at most 2^15.
template <bool BF>
struct ScoreError {
    // Four MMAs to a chain, of 17 addends each (16 products and the sum so far): an addend loses less than 2^-24 of the largest
    // (measured on a GB300: 2^-25, and the sum once 2^-23, 21 / 34 of this).
    static constexpr double kChain = 4 * 17 / 16777216.0;
    // What two 16-bit terms leave of a folded query.  bf16: the first at most half a step, 2^-8 of the query's power of two, and
    // the second half a step of that, 2^-17.  fp16: 2^-23 so, but never less than half of the smallest step, 2^-25, and a
    // weight counts as at least 2^-7 in the sum of magnitudes: 2^-18 of it.
    static constexpr double kTerms = BF ? 1 / 131072.0 : 1 / 262144.0;
    static constexpr double kChains = 1 / 2097152.0;   // up to 4 chains' two columns added in fp32: 5 roundings of 2^-24 at most
    static constexpr double kFold = 1 / 2097152.0;     // a folded query: the fp32 sum of up to 8 of one sign
    static constexpr double kScale = 1 / 8388608.0;    // the power of two, and an 8-bit cache's scale
    // The sum of magnitudes is short by up to 2^-7 of itself: each weight and each |lo| + |hi| are rounded to 16 bits once.
    static constexpr double kShort = 1 / 128.0;
    static constexpr float kRelative = BF ? 1.29e-5f : 9.1e-6f;
    static_assert(double(kRelative) * (1 - kShort) >= kChain + kTerms + kChains + kFold + kScale, "a bound on the score's error");

    // 2^-126 for each product: 2 D of them, in both terms.
    static constexpr float kUnderflow = 6.1e-36f;
    static_assert(double(kUnderflow) >= 2 * 2 * 128 * 1.1754943508222875e-38, "a bound on what underflows");
};

}  // namespace pkv
