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

// Programmatic dependent launch: a kernel's set-up may overlap the tail of the
// one before it on the stream (it waits for it before any global memory access).
struct Dependent {
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = {};
    Dependent(unsigned grid, unsigned threads, size_t smem, cudaStream_t stream) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.gridDim = dim3(grid);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
};

// sub: blocks per cut and member
template <int BK, bool BF16>
static cudaError_t launch_merge(const PagedLaunch& a, int sub) {
    if (a.params.teams < 2) return cudaSuccess;  // no cuts
    Dependent d((unsigned)((a.params.teams - 1) * a.params.team * sub), PAGED_MERGE_THREADS, 0, a.stream);
    return cudaLaunchKernelEx(&d.cfg, fa_paged_merge_kernel<FA_HEAD_DIM, BK, BF16>, a.params, sub);
}

template <bool BF16>
static cudaError_t launch_rows(const PagedLaunch& a) {
    using T = RowsTraits<FA_HEAD_DIM>;
    auto kernel = fa_paged_rows_kernel<FA_HEAD_DIM, BF16>;
    static std::atomic<uint64_t> configured{0};  // context the opt-in shared memory size was set in
    cudaError_t err = set_smem_for_context(kernel, T::SMEM, configured);
    if (err != cudaSuccess) return err;
    Dependent d((unsigned)((a.params.teams + ROWS_WARPS - 1) / ROWS_WARPS), 32 * ROWS_WARPS, T::SMEM, a.stream);
    err = cudaLaunchKernelEx(&d.cfg, kernel, *a.tmK, *a.tmV, a.params);
    return err == cudaSuccess ? launch_merge<T::KT, BF16>(a, 1) : err;
}

template <bool BF16>
static cudaError_t launch_tile(const PagedLaunch& a) {
    using T = TileTraits<FA_HEAD_DIM>;
    auto kernel = fa_paged_tile_kernel<FA_HEAD_DIM, BF16>;
    static std::atomic<uint64_t> configured{0};
    cudaError_t err = set_smem_for_context(kernel, T::SMEM_BYTES, configured);
    if (err != cudaSuccess) return err;
    Dependent d((unsigned)(a.params.team * a.params.teams), T::THREADS, T::SMEM_BYTES, a.stream);
    err = cudaLaunchKernelEx(&d.cfg, kernel, *a.tmQ, *a.tmK, *a.tmV, a.params);
    return err == cudaSuccess ? launch_merge<T::BN, BF16>(a, 8) : err;
}

#define FA_CAT2(a, b) a##b
#define FA_CAT(a, b) FA_CAT2(a, b)
cudaError_t FA_CAT(launch_paged_d, FA_HEAD_DIM)(const PagedLaunch& a, bool bf16) {
    if (a.tiles) return bf16 ? launch_tile<true>(a) : launch_tile<false>(a);
    return bf16 ? launch_rows<true>(a) : launch_rows<false>(a);
}

// Host-side facts of the rows kernel: workers (warps) an SM, positions a block.
void FA_CAT(paged_facts_d, FA_HEAD_DIM)(int* workers, int* block) {
    using T = RowsTraits<FA_HEAD_DIM>;
    *workers = T::CTAS * ROWS_WARPS;
    *block = T::KT;
}

}  // namespace fa
