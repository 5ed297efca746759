// The pieces of the bound on a page score's error, and the bound: one line for bf16, one for fp16.
#include <cstdio>

#include "score_error.h"

template <bool BF>
static void line() {
    using E = pkv::ScoreError<BF>;
    std::printf("%.17g %.17g %.17g %.17g\n", E::kTerms, E::kChain + E::kChains + E::kFold + E::kScale, E::kShort, double(E::kRelative));
}

int main() {
    line<true>();
    line<false>();
}
