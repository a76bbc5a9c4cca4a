// Parameters and launchers of the paged-cache operators: attention over a
// paged cache (fa_fwd_paged) and the cache's own operations (append, commit,
// fork).  Host and device.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime_api.h>

#include <cstdint>

namespace fa {

constexpr uint32_t STATUS_PAGE = 8;  // FA_ERR_PAGE: a block table entry outside the cache was needed
constexpr int PAGE_WORD = 1;         // its place behind the status word of waits and checks, which it must not hide

// Where a bad page was met; recorded in bits 8-15 of its status word.
enum PageSite : uint32_t {
    SITE_PAGE_ATTENTION = 60,
    SITE_PAGE_APPEND = 61,
    SITE_PAGE_COMMIT = 62,
    SITE_PAGE_FORK = 63,
    SITE_PAGE_SCORE = 64,
    SITE_PAGE_EVICT = 65,
};

// Division of 0 <= n < 2^31 by a positive divisor fixed for the launch, in four
// instructions: with s = ceil(log2 d) and m = floor(2^32 (2^s - d) / d) + 1, the
// quotient is (m n / 2^32 + n) / 2^s (Granlund and Montgomery 1994, figure 4.1).
struct FastDiv {
    uint32_t m = 1, s1 = 0, s2 = 0;
    FastDiv() = default;
    explicit FastDiv(uint32_t d) {
        uint32_t s = 0;
        while ((uint64_t(1) << s) < d) ++s;
        m = (uint32_t)(((uint64_t(1) << 32) * ((uint64_t(1) << s) - d)) / d + 1);
        s1 = s < 1 ? s : 1;
        s2 = s > 0 ? s - 1 : 0;
    }
#ifdef __CUDACC__
    __device__ __forceinline__ int operator()(int n) const {
        const uint32_t t = __umulhi(m, (uint32_t)n);
        return (int)((t + (((uint32_t)n - t) >> s1)) >> s2);
    }
#endif
};

// Attention over a paged cache.  Strides are in elements; the cache's are
// (page, head, slot) with the head dim contiguous.
struct PagedParams {
    const void* q;
    const void* kc;
    const void* vc;
    void* o;
    float* lse;                // (Z, Hq, T) fp32 contiguous, or nullptr
    int64_t sq_z, sq_h, sq_n;
    int64_t so_z, so_h, so_n;
    int64_t sk_p, sk_h, sk_n;
    int64_t sv_p, sv_h, sv_n;
    const int32_t* table;      // page of positions page * i .. page * i + page - 1 of sequence z at [z * st_z + i]
    int64_t st_z;
    const int32_t* lens;       // (Z) positions before the new tokens
    const int32_t* news;       // (Z) new tokens, or nullptr: T each
    const uint32_t* mask;      // bit j of words [z * sm_z + t * words ..]: new token t sees new token j; nullptr: j <= t
    int64_t sm_z;
    int words;                 // ceil(T / 32)
    int Z, Hq, Hkv, G, T;      // G = Hq / Hkv
    int page, M, P;            // slots a page, table columns, pages of the cache
    FastDiv by_g, by_page, by_tile_rows, by_team;
    bool wide_o;               // every row of O starts at a multiple of 32 bytes
    bool few;                  // at most 32 sequences, and all block counts fit in 31 bits
    int cap;                   // M * page: positions a sequence can have
    int tile_rows;             // query rows of a tile (a row is a (token, head of the group) pair, heads innermost)
    int box_rows;              // positions a TMA box holds: gcd(page, positions a block)
    int snap;                  // tile groups of at most this many key blocks are not cut
    int tiles;                 // tiles of one (z, kv head): ceil(T * G / tile_rows)
    float scale_log2;          // scale * log2(e) (rows kernel: signed; tile kernel: its magnitude)
    int negate_s;              // tile kernel: the scale is negative
    float* scratch;            // two partial-result slots a worker, slot_floats floats each
    int64_t slot_floats;
    void* cuts;                // PagedCut of each team
    int team, teams;           // workers of a team; teams (team * teams workers)
    uint32_t* status;
    uint64_t wait_limit_ns;
    int inject_stall;
};

struct PagedLaunch {
    PagedParams params;
    bool tiles;                // the tile kernel, else the rows kernel
    const CUtensorMap* tmK;
    const CUtensorMap* tmV;
    const CUtensorMap* tmQ;    // tile kernel only
    cudaStream_t stream;
};

cudaError_t launch_paged_d16(const PagedLaunch& a, bool bf16);
cudaError_t launch_paged_d32(const PagedLaunch& a, bool bf16);
cudaError_t launch_paged_d64(const PagedLaunch& a, bool bf16);
cudaError_t launch_paged_d128(const PagedLaunch& a, bool bf16);
cudaError_t launch_paged_d256(const PagedLaunch& a, bool bf16);
void paged_facts_d16(int* workers, int* block);
void paged_facts_d32(int* workers, int* block);
void paged_facts_d64(int* workers, int* block);
void paged_facts_d128(int* workers, int* block);
void paged_facts_d256(int* workers, int* block);

// What a launch needs from the library's per-device state (fa_api.cu).
struct DeviceFacts {
    int sms;
    uint32_t* status;
    uint64_t wait_limit_ns;
    int inject_stall;
};
cudaError_t device_facts(DeviceFacts* out);
// |scale| log2(e) and the scale's sign; false for a scale that cannot be taken
bool split_scale(float scale, float* c, int* negate);
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

}  // namespace fa
