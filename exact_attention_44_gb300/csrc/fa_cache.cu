// The paged cache's own operations: new rows in (append), accepted drafted
// rows moved together (commit), sequences forked, freed and given room (fork).
// All of them move 16-bit data without looking at it, in 16-byte pieces, and
// are bounded by those bytes at large sizes and by launch latency at small
// ones.  A block table entry outside the cache is never followed: the rows
// are skipped and STATUS_PAGE is recorded.
#include "fa_cache.h"

#include "fa_paged.h"
#include "fa_ptx.cuh"

namespace fa {

namespace {

// Small integers through L2: the kernels are programmatic dependents (see
// fa_paged_sched.cuh), and fork rewrites tables in place.
__device__ __forceinline__ int ldi(const int32_t* p) { return __ldcg(p); }

__device__ __forceinline__ void bad_page(uint32_t* status, uint32_t site) {
    atomicCAS(status, 0u, STATUS_PAGE | (site << 8) | ((blockIdx.x & 0xFFFFu) << 16));
}

template <typename K, typename P>
cudaError_t launch_dependent(K kernel, int64_t grid, int threads, size_t smem, cudaStream_t stream, const P& p) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// ------------------------------------------------------------ append --------
// Row (z, t, h) of the new K and V, t < news[z], to position lens[z] + t.  A
// thread moves one 16-byte piece of K and the same one of V; pieces of a row
// are neighbours, then heads, then tokens.
constexpr int APPEND_THREADS = 256;

__global__ void __launch_bounds__(APPEND_THREADS) fa_cache_append_kernel(const AppendParams p) {
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int pieces = p.D / 8;
    const uint32_t per_z = (uint32_t)p.T * p.H * pieces;  // < 2^31 (checked on the host)
    const int z = blockIdx.y;
    const int len = max(ldi(p.lens + z), 0);
    const int nl = p.news != nullptr ? min(ldi(p.news + z), p.T) : p.T;
    const uint32_t i = blockIdx.x * APPEND_THREADS + threadIdx.x;
    if (i >= per_z) return;
    const uint32_t row = i / pieces, c = i - row * pieces;
    const int t = (int)(row / p.H), h = (int)(row - (uint32_t)t * p.H);
    if (t >= nl) return;
    const int64_t pos = (int64_t)len + t;
    const int64_t col = pos / p.page;
    const int e = col < p.M ? ldi(p.table + z * p.st_z + col) : -1;
    if ((unsigned)e >= (unsigned)p.P) {
        bad_page(p.status, SITE_PAGE_APPEND);
        return;
    }
    const int slot = (int)(pos - col * p.page);
    const uint4 a = __ldcg(reinterpret_cast<const uint4*>(p.ks + z * p.ks_z + h * p.ks_h + t * p.ks_n + c * 8));
    const uint4 b = __ldcg(reinterpret_cast<const uint4*>(p.vs + z * p.vs_z + h * p.vs_h + t * p.vs_n + c * 8));
    *reinterpret_cast<uint4*>(p.k.base + e * p.k.p + h * p.k.h + slot * p.k.n + c * 8) = a;
    *reinterpret_cast<uint4*>(p.v.base + e * p.v.p + h * p.v.h + slot * p.v.n + c * 8) = b;
}

// ------------------------------------------------------------ commit --------
// Position lens[z] + path[z][i] to lens[z] + i for i < kept[z], in place.  One
// thread takes a 16-byte piece through all of the path's steps: with the path
// strictly increasing a step writes only where the same thread has already
// read (position lens[z] + i is read by no step after i), so steps need no
// barrier, and the reads of eight steps may go ahead of their writes.
constexpr int COMMIT_THREADS = 256;

__global__ void __launch_bounds__(COMMIT_THREADS) fa_cache_commit_kernel(const CommitParams p) {
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int pieces = p.D / 8;
    const uint32_t per_z = (uint32_t)p.L * 2 * p.H * pieces;  // < 2^31 (checked on the host)
    const uint32_t i = blockIdx.x * COMMIT_THREADS + threadIdx.x;
    const int z = blockIdx.y;
    if (i >= per_z) return;
    const uint32_t c = i % pieces;
    uint32_t r = i / pieces;
    const uint32_t h = r % p.H;
    r /= p.H;
    const bool is_v = r & 1u;
    const uint32_t layer = r >> 1;
    const CacheView& cache = is_v ? p.v : p.k;
    uint16_t* base = cache.base + layer * cache.l + h * cache.h + c * 8;
    const int64_t len = max(ldi(p.lens + z), 0), cap = (int64_t)p.M * p.page;
    const int n = min(ldi(p.kept + z), p.A);
    const int32_t* row = p.table + z * p.st_z;
    auto at = [&](int64_t pos) -> uint16_t* {
        if (pos < 0 || pos >= cap) return nullptr;
        const int64_t col = pos / p.page;
        const int e = ldi(row + col);
        return (unsigned)e < (unsigned)p.P ? base + e * cache.p + (pos - col * p.page) * cache.n : nullptr;
    };
    constexpr int U = 8;
    for (int s0 = 0; s0 < n; s0 += U) {
        uint4 v[U];
        uint16_t* to[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            to[u] = nullptr;
            if (s0 + u < n) {
                const int from = ldi(p.path + z * p.sp_z + s0 + u);
                if (from != s0 + u) {
                    const uint16_t* src = at(len + from);
                    to[u] = at(len + s0 + u);
                    if (src == nullptr || to[u] == nullptr) {
                        bad_page(p.status, SITE_PAGE_COMMIT);
                        to[u] = nullptr;
                    } else {
                        v[u] = __ldcg(reinterpret_cast<const uint4*>(src));
                    }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (to[u] != nullptr) *reinterpret_cast<uint4*>(to[u]) = v[u];
    }
}

// ------------------------------------------------------------ fork ----------
// Two kernels.  The first, one CTA, decides everything from the state as it
// was: each sequence's length after, which columns of its row need a page of
// its own, and which pages those are -- the lowest ones whose count is 0, in
// the order of sequences and columns (so the result does not depend on
// timing).  The second rewrites the table and counts, and copies the partly
// filled pages.
constexpr int PLAN_THREADS = 1024;

struct ForkWs {
    int32_t *src, *len, *first, *count, *off, *tail, *found, *pages;
};
__device__ __forceinline__ ForkWs fork_ws(const ForkParams& p) {
    ForkWs w;
    w.src = p.ws;
    w.len = w.src + p.Z;
    w.first = w.len + p.Z;
    w.count = w.first + p.Z;
    w.off = w.count + p.Z;
    w.tail = w.off + p.Z;         // 3 per sequence: from page, to page, rows (0: none)
    w.found = w.tail + 3 * p.Z;   // pages found
    w.pages = w.found + 2;
    return w;
}

// exclusive prefix sum over the CTA; total in *sum
__device__ __forceinline__ int block_scan(int v, int* red, int* sum) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int x = v;
    for (int d = 1; d < 32; d *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 31) red[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int y = lane < (int)blockDim.x / 32 ? red[lane] : 0;
        for (int d = 1; d < 32; d *= 2) {
            const int u = __shfl_up_sync(0xffffffffu, y, d);
            if (lane >= d) y += u;
        }
        red[lane] = y;
    }
    __syncthreads();
    *sum = red[31];
    return x - v + (warp > 0 ? red[warp - 1] : 0);
}

__global__ void __launch_bounds__(PLAN_THREADS) fa_cache_fork_plan_kernel(const ForkParams p) {
    __shared__ int red[32];
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const ForkWs w = fork_ws(p);
    const int tid = threadIdx.x;
    const int cap = p.M * p.page;
    int wanted = 0, excess = 0;
    for (int z0 = 0; z0 < p.Z; z0 += PLAN_THREADS) {
        const int z = z0 + tid;
        int count = 0, over = 0;
        if (z < p.Z) {
            int src = p.source != nullptr ? ldi(p.source + z) : z;
            if (src < -1 || src >= p.Z) {  // not a sequence: left as it is
                bad_page(p.status, SITE_PAGE_FORK);
                src = z;
            }
            const int len = src >= 0 ? min(max(ldi(p.lens + src), 0), cap) : 0;
            const int need = src >= 0 ? (int)(((int64_t)len + p.room + p.page - 1) / p.page) : 0;
            int first = src == z ? (len + p.page - 1) / p.page : len / p.page;
            if (src == z)
                while (first < min(need, p.M) && ldi(p.table + z * p.st_z + first) >= 0) ++first;  // room it has
            count = max(0, min(need, p.M) - first);
            over = max(0, need - p.M);
            w.src[z] = src;
            w.len[z] = len;
            w.first[z] = first;
            w.count[z] = count;
        }
        int sum, off = block_scan(count, red, &sum);
        if (z < p.Z) w.off[z] = wanted + off;
        wanted += sum;
        int unused = block_scan(over, red, &sum);
        (void)unused;
        excess += sum;
    }
    // the first `wanted` pages with count 0
    int found = 0;
    for (int p0 = 0; p0 < p.P && found < wanted; p0 += 4 * PLAN_THREADS) {
        const int i = p0 + 4 * tid;
        int c[4], k = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            c[u] = i + u < p.P ? ldi(p.refs + i + u) : 1;
            k += c[u] == 0;
        }
        int sum, at = found + block_scan(k, red, &sum);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (c[u] == 0) {
                if (at < wanted) w.pages[at] = i + u;
                ++at;
            }
        found += sum;
    }
    found = min(found, wanted);
    __syncthreads();
    // tails: the partly filled last page of a source goes to the copy's first own page
    for (int z = tid; z < p.Z; z += PLAN_THREADS) {
        const int src = w.src[z], len = w.len[z], tail = len % p.page;
        int rows = 0, from = 0, to = 0;
        if (src >= 0 && src != z && tail > 0 && w.off[z] < found && w.count[z] > 0) {
            from = ldi(p.table + src * p.st_z + len / p.page);
            to = w.pages[w.off[z]];
            if ((unsigned)from < (unsigned)p.P) rows = tail;
            else bad_page(p.status, SITE_PAGE_FORK);
        }
        w.tail[3 * z] = from;
        w.tail[3 * z + 1] = to;
        w.tail[3 * z + 2] = rows;
    }
    if (tid == 0) {
        w.found[0] = found;
        if (p.missing != nullptr) *p.missing = wanted - found + excess;
    }
}

// Table, lengths and counts: a CTA takes `cols` columns of every row, reads
// them all before it writes any (a source row may be rewritten in the same
// call), and counts one reference less for what a changed row held and one
// more for what it holds.  The other CTAs copy tails: rows of all heads of one
// (sequence, layer, K or V) each.
constexpr int FORK_THREADS = 256;

struct ForkApply {
    ForkParams p;
    int cols, table_ctas;
};

__global__ void __launch_bounds__(FORK_THREADS) fa_cache_fork_apply_kernel(const ForkApply a) {
    extern __shared__ int old[];  // [Z][cols]
    const ForkParams& p = a.p;
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const ForkWs w = fork_ws(p);
    const int tid = threadIdx.x;
    if ((int)blockIdx.x < a.table_ctas) {
        const int c0 = blockIdx.x * a.cols, nc = min(a.cols, p.M - c0), n = p.Z * a.cols;
        const int found = ldi(w.found);
        for (int i = tid; i < n; i += FORK_THREADS) {
            const int z = i / a.cols, c = i - z * a.cols;
            old[i] = c < nc ? ldi(p.table + z * p.st_z + c0 + c) : -1;
        }
        __syncthreads();
        for (int i = tid; i < n; i += FORK_THREADS) {
            const int z = i / a.cols, c = i - z * a.cols, col = c0 + c;
            if (c >= nc) continue;
            const int src = ldi(w.src + z), first = ldi(w.first + z), count = ldi(w.count + z);
            const int was = old[i];
            int now = was;
            if (src != z) now = src >= 0 && col < ldi(w.len + z) / p.page ? old[src * a.cols + c] : -1;
            if (col >= first && col < first + count) {
                const int at = ldi(w.off + z) + col - first;
                if (at < found) now = ldi(w.pages + at);
            }
            if (now == was) continue;
            if ((unsigned)was < (unsigned)p.P) atomicAdd(p.refs + was, -1);
            else if (was >= 0) bad_page(p.status, SITE_PAGE_FORK);
            if ((unsigned)now < (unsigned)p.P) atomicAdd(p.refs + now, 1);
            p.table[z * p.st_z + col] = now;
        }
        if (blockIdx.x == 0)
            for (int z = tid; z < p.Z; z += FORK_THREADS) p.lens[z] = ldi(w.len + z);
        return;
    }
    const int pieces = p.D / 8;
    const int64_t jobs = (int64_t)p.Z * p.L * 2;
    for (int64_t j = blockIdx.x - a.table_ctas; j < jobs; j += gridDim.x - a.table_ctas) {
        const int z = (int)(j / (2 * p.L)), r = (int)(j - (int64_t)z * 2 * p.L);
        const int rows = ldi(w.tail + 3 * z + 2);
        if (rows == 0) continue;
        const int64_t from = ldi(w.tail + 3 * z), to = ldi(w.tail + 3 * z + 1);
        const CacheView& cache = r & 1 ? p.v : p.k;
        uint16_t* base = cache.base + (int64_t)(r >> 1) * cache.l;
        for (int i = tid; i < p.H * rows * pieces; i += FORK_THREADS) {
            const int c = i % pieces, row = i / pieces, h = row / rows, slot = row - h * rows;
            const int64_t at = h * cache.h + slot * cache.n + c * 8;
            *reinterpret_cast<uint4*>(base + to * cache.p + at) =
                __ldcg(reinterpret_cast<const uint4*>(base + from * cache.p + at));
        }
    }
}

}  // namespace

cudaError_t launch_cache_append(const AppendParams& p, cudaStream_t stream) {
    const int64_t per_z = (int64_t)p.T * p.H * (p.D / 8);
    const int64_t gx = (per_z + APPEND_THREADS - 1) / APPEND_THREADS;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)gx, (unsigned)p.Z);
    cfg.blockDim = dim3(APPEND_THREADS);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fa_cache_append_kernel, p);
}

cudaError_t launch_cache_commit(const CommitParams& p, cudaStream_t stream) {
    const int64_t per_z = (int64_t)p.L * 2 * p.H * (p.D / 8);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((per_z + COMMIT_THREADS - 1) / COMMIT_THREADS), (unsigned)p.Z);
    cfg.blockDim = dim3(COMMIT_THREADS);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fa_cache_commit_kernel, p);
}

cudaError_t launch_cache_fork(const ForkParams& p, int sms, cudaStream_t stream) {
    cudaError_t err = launch_dependent(fa_cache_fork_plan_kernel, 1, PLAN_THREADS, 0, stream, p);
    if (err != cudaSuccess) return err;
    ForkApply a{p, 1, 0};
    // columns a CTA: as many as 32 KB of shared memory hold, but enough CTAs to spread the rows
    a.cols = (int)(8192 / p.Z);
    a.cols = a.cols < 1 ? 1 : a.cols > 32 ? 32 : a.cols;
    a.table_ctas = p.M > 0 ? (p.M + a.cols - 1) / a.cols : 1;  // the first writes the lengths
    const int64_t jobs = (int64_t)p.Z * p.L * 2;
    const int64_t copies = p.source == nullptr ? 0 : jobs < 4 * sms ? jobs : 4 * sms;
    return launch_dependent(fa_cache_fork_apply_kernel, a.table_ctas + copies, FORK_THREADS,
                            (size_t)p.Z * a.cols * sizeof(int), stream, a);
}

}  // namespace fa
