// Argument checks and tensor maps that the paged-cache entry points share (host only).
#pragma once

#include <cuda_runtime_api.h>

#include <cstdint>
#include <utility>

#include "fa.h"
#include "fa_cache.h"
#include "fa_paged.h"

namespace fa {

fa_status report_cuda(const char* what, cudaError_t e);  // fa_api.cu

namespace checks {

inline bool head_dim_ok(int D) { return D == 16 || D == 32 || D == 64 || D == 128 || D == 256; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool misaligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

// d-stride 1, 16-byte aligned base, the other strides multiples of 8 elements
// in every dimension of extent > 1; outputs must not fold rows together
// (stride 0).
inline fa_status check_strided(const void* ptr, const fa_strides* s, int64_t nb, int64_t nh, int64_t nn, bool written) {
    if (s == nullptr) return FA_ERR_INVALID_ARG;
    if (nb * nh * nn == 0) return FA_OK;  // nothing there: the pointer is not used
    if (ptr == nullptr) return FA_ERR_INVALID_ARG;
    if (s->d != 1 || misaligned(ptr, 16)) return FA_ERR_ALIGNMENT;
    const int64_t st[3] = {s->b, s->h, s->n}, ext[3] = {nb, nh, nn};
    for (int i = 0; i < 3; ++i) {
        if (ext[i] <= 1) continue;
        if (st[i] < 0 || st[i] % 8 != 0 || st[i] >= (int64_t(1) << 38)) return FA_ERR_ALIGNMENT;
        if (written && st[i] == 0) return FA_ERR_INVALID_ARG;
    }
    return FA_OK;
}

// The cache's geometry and its block table.
inline fa_status check_cache(const fa_paged_cache& c, bool table_written) {
    if (c.Z < 0 || c.L < 0 || c.P < 0 || c.Hkv < 0 || c.max_pages < 0 || c.table_stride < 0) return FA_ERR_INVALID_ARG;
    if (!head_dim_ok(c.D) || c.page_size < 16 || c.page_size % 16 != 0) return FA_ERR_UNSUPPORTED;
    if ((int64_t)c.max_pages * c.page_size > (int64_t(1) << 30) || c.Z > 65535) return FA_ERR_UNSUPPORTED;
    if ((int64_t)c.Z * c.max_pages > 0) {
        if (c.block_table == nullptr) return FA_ERR_INVALID_ARG;
        if (misaligned(c.block_table, 4)) return FA_ERR_ALIGNMENT;
        if (table_written && c.Z > 1 && c.table_stride < c.max_pages) return FA_ERR_INVALID_ARG;
    }
    if (c.L > 1)
        for (const int64_t s : {c.k_layer, c.v_layer})
            if (s <= 0 || s % 8 != 0 || s >= (int64_t(1) << 42)) return FA_ERR_ALIGNMENT;
    return FA_OK;
}
// Its tensors (where a call has work for them) and lengths.
inline fa_status check_cache_data(const fa_paged_cache& c, bool written) {
    if (c.L > 0)
        for (const auto& t : {std::make_pair(c.k, &c.sk), std::make_pair(c.v, &c.sv)}) {
            const fa_status st = check_strided(t.first, t.second, c.P, c.Hkv, c.page_size, written);
            if (st != FA_OK) return st;
        }
    if (c.seq_lens == nullptr) return FA_ERR_INVALID_ARG;
    return misaligned(c.seq_lens, 4) ? FA_ERR_ALIGNMENT : FA_OK;
}
inline fa_status check_ints(const void* p, bool needed) {
    if (p == nullptr) return needed ? FA_ERR_INVALID_ARG : FA_OK;
    return misaligned(p, 4) ? FA_ERR_ALIGNMENT : FA_OK;
}

inline CacheView view(void* base, const fa_strides& s, int64_t layer) {
    return CacheView{static_cast<uint16_t*>(base), layer, s.b, s.h, s.n};
}

}  // namespace checks

// 4-D tensor map with the head dim innermost (dims: D, then `dims` outermost
// last) and boxes of one swizzle chunk x the given extents.
struct PagedMapDim {
    int64_t extent, stride;  // stride in elements
    int box;
};
inline CUresult make_paged_map(CUtensorMap* map, const void* ptr, bool bf16, int D, const PagedMapDim (&dims)[3]) {
    const int swe = D < 64 ? D : 64;
    const CUtensorMapSwizzle sw = swe == 64   ? CU_TENSOR_MAP_SWIZZLE_128B
                                  : swe == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                              : CU_TENSOR_MAP_SWIZZLE_32B;
    cuuint64_t ext[4] = {(cuuint64_t)D, 0, 0, 0}, str[3];
    cuuint32_t box[4] = {(cuuint32_t)swe, 0, 0, 0}, ones[4] = {1, 1, 1, 1};
    for (int i = 0; i < 3; ++i) {
        ext[i + 1] = (cuuint64_t)dims[i].extent;
        // a dimension of extent 1 is never stepped along; give it a harmless stride
        str[i] = dims[i].extent > 1 ? (cuuint64_t)dims[i].stride * 2 : (cuuint64_t)D * 2;
        box[i + 1] = (cuuint32_t)dims[i].box;
    }
    const auto fn = tensor_map_encoder();
    if (fn == nullptr) return CUDA_ERROR_NOT_SUPPORTED;
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void*>(ptr),
              ext, str, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// Largest box of whole page rows that tiles a block of `bn` positions.
inline int paged_box_rows(int page, int bn) {
    int r = 16;
    while (r < bn && page % (2 * r) == 0) r *= 2;
    return r;
}

}  // namespace fa
