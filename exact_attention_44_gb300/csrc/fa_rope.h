// Parameters and launchers of rotary positions (fa_rope.cu).
#pragma once

#include <cuda_runtime_api.h>

#include <cstdint>

#include "fa_cache.h"

namespace fa {

// Rows (z, h, n) of 16-bit elements, strides in elements, D contiguous.
struct RopeParams {
    const uint16_t *q, *k, *v;       // rows in
    int64_t q_z, q_h, q_n, k_z, k_h, k_n, v_z, v_h, v_n;
    uint16_t *qo, *ko;               // rows out; ko unused where a cache takes them
    int64_t qo_z, qo_h, qo_n, ko_z, ko_h, ko_n;
    bool q_in_place, k_in_place;     // elements that do not turn stay where they are
    const int32_t* positions;        // nullptr: the row's index (a cache: its slot)
    int64_t pos_z;
    int64_t turns[128];              // (R / 2) turns a position in units of 2^-64
    int Z, Hq, Hk, N, D, R;
    int heads;                       // of a thread (set by the launch)
    int token_shift;                 // log2 of the tokens of a sequence that a CTA takes (set by the launch)
    float cos_factor, sin_factor;    // factor; its sign turns back
    // a cache (fa_cache_append_rope): k and v rows go to their slots
    CacheView kc, vc;
    const int32_t* table;
    int64_t st_z;
    const int32_t *lens, *news;
    int page, M, P;
    uint32_t* status;
};

cudaError_t launch_rope(const RopeParams& p, bool bf16, bool interleaved, bool cache, int sms, cudaStream_t stream);

}  // namespace fa
