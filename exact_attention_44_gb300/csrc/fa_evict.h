// Parameters and launcher of fa_cache_evict (fa_evict.cu).
#pragma once

#include <cuda_runtime_api.h>

#include <cstdint>

#include "fa_cache.h"
#include "fa_paged.h"

namespace fa {

struct EvictParams {
    CacheView k, v;
    int32_t* table;
    int64_t st_z;
    int32_t *lens, *refs;
    float* scores;                   // (L, Z, H, >= M * page)
    int64_t ss_l, ss_z, ss_h;
    const int32_t* keep;             // or nullptr: budget for all
    int32_t* missing;
    int Z, L, H, D, page, M, P;
    int budget, first, recent;       // budget <= M * page
    FastDiv by_page;
    int32_t* ws;                     // evict_workspace_ints(L, Z, H, M, budget)
    uint32_t* status;
};
// per sequence: length it is cut to (-1: it stays as it is), first page it needs of its own,
// place in the page list; the number of pages lacking (-1: none is replaced); each sequence's
// table row as it was and as it will be; the page list; per (layer, sequence, head) the first
// row that moves and the positions that stay
inline int64_t evict_workspace_ints(int64_t L, int64_t Z, int64_t H, int64_t M, int64_t budget) {
    return 3 * Z + 1 + 3 * Z * M + L * Z * H * (1 + budget);
}

cudaError_t launch_cache_evict(const EvictParams& p, int sms, cudaStream_t stream);

}  // namespace fa
