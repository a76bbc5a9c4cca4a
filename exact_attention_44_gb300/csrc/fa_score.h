// Parameters and launchers of the received attention weight (fa_cache_score).
#pragma once

#include <cuda_runtime_api.h>

#include <cstdint>

#include "fa_paged.h"

namespace fa {

struct ScoreParams {
    const uint16_t* q;
    int64_t sq_z, sq_h, sq_n;
    const float* lse;          // (Z, Hq, T) contiguous
    const uint16_t* k;         // strides in elements: page, head, slot
    int64_t sk_p, sk_h, sk_n;
    const int32_t* table;
    int64_t st_z;
    const int32_t *lens, *news;
    float* scores;             // (Z, Hkv, >= cap)
    int64_t ss_z, ss_h;
    int Z, Hq, Hkv, G, T;
    int page, M, P, cap;       // cap = M * page: positions a sequence can have
    FastDiv by_g, by_page;
    float scale, decay;
    int workers;               // warps of the launch
    uint32_t* status;
};

struct ScoreLaunch {
    ScoreParams params;
    int sms;
    cudaStream_t stream;
};

cudaError_t launch_score_d16(const ScoreLaunch& a, bool bf16);
cudaError_t launch_score_d32(const ScoreLaunch& a, bool bf16);
cudaError_t launch_score_d64(const ScoreLaunch& a, bool bf16);
cudaError_t launch_score_d128(const ScoreLaunch& a, bool bf16);
cudaError_t launch_score_d256(const ScoreLaunch& a, bool bf16);

}  // namespace fa
