// Parameters and launchers of the received attention weight (fa_cache_score).
#pragma once

#include <cuda.h>
#include <cuda_runtime_api.h>

#include <cstddef>
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
    int workers;               // rows kernel: warps of the launch
    // tile kernel
    int tokens, token_shift;   // new tokens of a tile (a power of two), its log2
    int tile_rows, tile_cols;  // tokens * G, and that rounded up to 16
    int box_rows;              // positions a TMA box holds
    int long_q;                // many tiles a unit: one slot for K, more for Q
    float* parts;              // two slots of sums a CTA, or nullptr: no unit is cut
    void* cuts;
    uint64_t wait_limit_ns;
    int inject_stall;
    uint32_t* status;
};

struct ScoreLaunch {
    ScoreParams params;
    bool tiles;                // the tile kernel, else the rows kernel
    const CUtensorMap* tmQ;    // tile kernel only
    const CUtensorMap* tmK;
    int sms;
    cudaStream_t stream;
};

// Facts of the tile kernel: query rows of a tile, positions of a unit.
struct ScoreTileFacts {
    int rows, block;
};
constexpr ScoreTileFacts score_tile_facts(int D) { return D == 256 ? ScoreTileFacts{64, 128} : ScoreTileFacts{128, 256}; }
// Workspace: two slots of a unit's sums, and where its range starts, a CTA.
constexpr size_t score_slot_bytes(int sms) { return (size_t)sms * 2 * 256 * sizeof(float); }
constexpr size_t score_workspace_bytes(int sms) { return score_slot_bytes(sms) + (size_t)sms * 48; }

cudaError_t launch_score_d16(const ScoreLaunch& a, bool bf16);
cudaError_t launch_score_d32(const ScoreLaunch& a, bool bf16);
cudaError_t launch_score_d64(const ScoreLaunch& a, bool bf16);
cudaError_t launch_score_d128(const ScoreLaunch& a, bool bf16);
cudaError_t launch_score_d256(const ScoreLaunch& a, bool bf16);

}  // namespace fa
