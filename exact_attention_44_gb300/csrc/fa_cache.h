// Parameters and launchers of the paged cache's own operations (fa_cache.cu).
#pragma once

#include <cuda_runtime_api.h>

#include <cstdint>

namespace fa {

// One cache (K or V): 16-bit elements, strides in elements, D contiguous.
struct CacheView {
    uint16_t* base;
    int64_t l, p, h, n;  // layer, page, head, slot
};

struct AppendParams {
    CacheView k, v;
    const uint16_t *ks, *vs;        // the new rows
    int64_t ks_z, ks_h, ks_n, vs_z, vs_h, vs_n;
    const int32_t* table;
    int64_t st_z;
    const int32_t *lens, *news;     // news may be nullptr
    int Z, H, T, D, page, M, P;
    int lanes;                      // of a token (set by the launch)
    uint32_t* status;
};

struct CommitParams {
    CacheView k, v;
    const int32_t* table;
    int64_t st_z;
    const int32_t *lens, *path, *kept;
    int64_t sp_z;                   // row stride of path
    int Z, L, H, A, D, page, M, P;
    uint32_t* status;
};

struct ForkParams {
    CacheView k, v;
    int32_t* table;
    int64_t st_z;
    int32_t *lens, *refs;
    const int32_t* source;          // nullptr: every sequence stays
    int32_t* missing;               // or nullptr
    int Z, L, H, D, page, M, P, room;
    int whole;                      // all or nothing
    int32_t* ws;                    // fork_workspace_ints(Z, M)
    uint32_t* status;
};
// per sequence: source, length after, first column to fill, columns to fill,
// place in the page list, partly filled page of the source; the list of tails (3
// each), the number of pages found (-1: nothing is to be changed) and of tails;
// the page list
inline int64_t fork_workspace_ints(int64_t Z, int64_t M) { return 9 * Z + 2 + Z * M; }

cudaError_t launch_cache_append(AppendParams p, cudaStream_t stream);
cudaError_t launch_cache_commit(const CommitParams& p, cudaStream_t stream);
cudaError_t launch_cache_fork(const ForkParams& p, int sms, cudaStream_t stream);

}  // namespace fa
