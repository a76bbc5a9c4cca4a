// Specialisations of the received-weight kernels for one head dim, D = FA_HEAD_DIM
// (compiled once per supported D, in parallel).
#ifndef FA_HEAD_DIM
#error "compile with -DFA_HEAD_DIM=<16|32|64|128|256>"
#endif
#include "fa_score_rows_kernel.cuh"

#include <algorithm>

namespace fa {

template <bool BF16, int NT>
static cudaError_t launch_rows(const ScoreLaunch& a) {
    using T = ScoreRows<FA_HEAD_DIM>;
    ScoreParams p = a.params;
    // no more warps than there can be steps
    const int64_t steps = (int64_t)p.Z * p.Hkv * ((p.cap + T::KT - 1) / T::KT);
    p.workers = (int)std::max<int64_t>(1, std::min<int64_t>(steps, (int64_t)a.sms * T::CTAS * SCORE_WARPS));
    return launch_dependent(fa_score_rows_kernel<FA_HEAD_DIM, BF16, NT>, dim3((unsigned)((p.workers + SCORE_WARPS - 1) / SCORE_WARPS)),
                            32 * SCORE_WARPS, 0, a.stream, p);
}

#define FA_CAT2(a, b) a##b
#define FA_CAT(a, b) FA_CAT2(a, b)
cudaError_t FA_CAT(launch_score_d, FA_HEAD_DIM)(const ScoreLaunch& a, bool bf16) {
    const bool one = (int64_t)a.params.T * a.params.G <= 8;
    if (bf16) return one ? launch_rows<true, 1>(a) : launch_rows<true, 2>(a);
    return one ? launch_rows<false, 1>(a) : launch_rows<false, 2>(a);
}

}  // namespace fa
