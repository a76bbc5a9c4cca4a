// Specialisations of the received-weight kernels for one head dim, D = FA_HEAD_DIM
// (compiled once per supported D, in parallel).
#ifndef FA_HEAD_DIM
#error "compile with -DFA_HEAD_DIM=<16|32|64|128|256>"
#endif
#include "fa_launch.h"
#include "fa_score_rows_kernel.cuh"
#include "fa_score_tile_kernel.cuh"

#include <algorithm>

namespace fa {

template <bool BF16, int NT>
static cudaError_t launch_rows(const ScoreLaunch& a) {
    using T = ScoreRows<FA_HEAD_DIM>;
    ScoreParams p = a.params;
    // no more warps than there can be steps
    const int64_t steps = (int64_t)p.Z * p.Hkv * ((p.cap + T::KT - 1) / T::KT);
    p.workers = (int)std::max<int64_t>(1, std::min<int64_t>(steps, (int64_t)a.sms * T::ctas(NT) * SCORE_WARPS));
    return launch_dependent(fa_score_rows_kernel<FA_HEAD_DIM, BF16, NT>, dim3((unsigned)((p.workers + SCORE_WARPS - 1) / SCORE_WARPS)),
                            32 * SCORE_WARPS, 0, a.stream, p);
}

template <bool BF16>
static cudaError_t launch_tiles(const ScoreLaunch& a) {
    using T = ScoreTile<FA_HEAD_DIM>;
    static_assert(T::BR == score_tile_facts(FA_HEAD_DIM).rows && T::KB == score_tile_facts(FA_HEAD_DIM).block,
                  "the host's facts");
    static_assert(sizeof(scoret::Cut) == 48 && T::KB <= 256, "workspace");
    auto kernel = fa_score_tile_kernel<FA_HEAD_DIM, BF16>;
    static std::atomic<uint64_t> configured{0};  // context the opt-in shared memory size was set in
    cudaError_t err = set_smem_for_context(kernel, T::SMEM_BYTES, configured);
    if (err != cudaSuccess) return err;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.sms);
    cfg.blockDim = dim3(T::THREADS);
    cfg.dynamicSmemBytes = T::SMEM_BYTES;
    cfg.stream = a.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, kernel, *a.tmQ, *a.tmK, a.params);
    if (err != cudaSuccess || a.params.parts == nullptr || a.sms < 2) return err;
    return launch_dependent(fa_score_merge_kernel<FA_HEAD_DIM>, dim3((unsigned)(a.sms - 1)), T::KB, 0, a.stream, a.params);
}

#define FA_CAT2(a, b) a##b
#define FA_CAT(a, b) FA_CAT2(a, b)
cudaError_t FA_CAT(launch_score_d, FA_HEAD_DIM)(const ScoreLaunch& a, bool bf16) {
    if (a.tiles) return bf16 ? launch_tiles<true>(a) : launch_tiles<false>(a);
    const int64_t rows = (int64_t)a.params.T * a.params.G;
    if (rows <= 8) return bf16 ? launch_rows<true, 1>(a) : launch_rows<false, 1>(a);
    if constexpr (FA_HEAD_DIM <= 128)
        if (rows > 16) return bf16 ? launch_rows<true, 4>(a) : launch_rows<false, 4>(a);
    return bf16 ? launch_rows<true, 2>(a) : launch_rows<false, 2>(a);
}

}  // namespace fa
