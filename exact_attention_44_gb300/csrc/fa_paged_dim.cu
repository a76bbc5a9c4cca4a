// Specialisations of the paged attention kernels for one head dim, D =
// FA_HEAD_DIM (compiled once per supported D, in parallel).
#ifndef FA_HEAD_DIM
#error "compile with -DFA_HEAD_DIM=<16|32|64|128|256>"
#endif
#include "fa_launch.h"
#include "fa_paged.h"
#include "fa_paged_rows_kernel.cuh"
#include "fa_paged_tile_kernel.cuh"

namespace fa {

template <int BK, bool BF16, bool COLS>
static cudaError_t launch_merge(const PagedLaunch& a, cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)a.params.Z * a.params.Hkv * a.params.tiles * a.merge_slices));
    cfg.blockDim = dim3(PAGED_MERGE_THREADS);
    cfg.stream = a.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fa_paged_merge_kernel<FA_HEAD_DIM, BK, BF16, COLS>, a.params, a.grid,
                              a.merge_slices);
}

template <int RT, bool BF16>
static cudaError_t launch_rows(const PagedLaunch& a) {
    using T = RowsTraits<FA_HEAD_DIM, RT>;
    auto kernel = fa_paged_rows_kernel<FA_HEAD_DIM, RT, BF16>;
    static std::atomic<uint64_t> configured{0};
    cudaError_t err = set_smem_for_context(kernel, T::SMEM, configured);
    if (err != cudaSuccess) return err;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.grid);
    cfg.blockDim = dim3(32 * ROWS_WARPS);
    cfg.dynamicSmemBytes = T::SMEM;
    cfg.stream = a.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, kernel, a.params);
    return err == cudaSuccess ? launch_merge<ROWS_BK, BF16, false>(a, attr) : err;
}

template <bool BF16>
static cudaError_t launch_tile(const PagedLaunch& a) {
    using T = TileTraits<FA_HEAD_DIM>;
    auto kernel = fa_paged_tile_kernel<FA_HEAD_DIM, BF16>;
    static std::atomic<uint64_t> configured{0};
    cudaError_t err = set_smem_for_context(kernel, T::SMEM_BYTES, configured);
    if (err != cudaSuccess) return err;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.grid);
    cfg.blockDim = dim3(T::THREADS);
    cfg.dynamicSmemBytes = T::SMEM_BYTES;
    cfg.stream = a.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, kernel, *a.tmQ, *a.tmK, *a.tmV, a.params);
    return err == cudaSuccess ? launch_merge<T::BN, BF16, true>(a, attr) : err;
}

#define FA_CAT2(a, b) a##b
#define FA_CAT(a, b) FA_CAT2(a, b)
cudaError_t FA_CAT(launch_paged_d, FA_HEAD_DIM)(const PagedLaunch& a, bool bf16) {
    if (a.rows == 0) return bf16 ? launch_tile<true>(a) : launch_tile<false>(a);
#if FA_HEAD_DIM <= 128
    if (a.rows == 32) return bf16 ? launch_rows<32, true>(a) : launch_rows<32, false>(a);
#endif
    return bf16 ? launch_rows<16, true>(a) : launch_rows<16, false>(a);
}

}  // namespace fa
