// The paged cache's own operations: new rows in (append), accepted drafted
// rows moved together (commit), sequences forked, freed and given room (fork).
// All of them move 16-bit data without looking at it, in 16-byte pieces, and
// are bounded by those bytes at large sizes and by launch latency at small
// ones.  A block table entry outside the cache is never followed: the rows
// are skipped and STATUS_PAGE is recorded.
#include "fa_cache.h"

#include <climits>

#include "fa_paged.h"
#include "fa_ptx.cuh"

namespace fa {

namespace {

// Small integers through L2: the kernels are programmatic dependents (see
// fa_paged_sched.cuh), and fork rewrites tables in place.
__device__ __forceinline__ int ldi(const int32_t* p) { return __ldcg(p); }

__device__ __forceinline__ void bad_page(uint32_t* status, uint32_t site) {
    atomicCAS(status + PAGE_WORD, 0u, STATUS_PAGE | (site << 8) | ((blockIdx.x & 0xFFFFu) << 16));
}

template <typename K, typename P>
cudaError_t launch_dependent(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, const P& p) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// ------------------------------------------------------------ append --------
// Row (z, t, h) of the new K and V, t < news[z], to position lens[z] + t.  A
// group of up to 32 lanes takes a token: one block table entry for all of its
// heads, then the 16-byte pieces of its K and V rows, four of each in flight a
// lane.  (A thread a piece, each with its own table entry, took 17.5 us where
// this takes 8.8 to 9.5: five prompts of up to 2011 tokens, 8 heads of D = 128, 62 MB
// read and written, repeated in a graph, where the L2 cache keeps part; 12.6 on new
// inputs, 4.9 TB/s.)  One token for each of 64 sequences: 2.1 us in a graph, 3.0 a
// call, a launch and three dependent loads.
constexpr int APPEND_THREADS = 128;

__global__ void __launch_bounds__(APPEND_THREADS) fa_cache_append_kernel(const AppendParams p) {
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int z = blockIdx.y, lane = threadIdx.x & (p.lanes - 1);
    const int t = (int)((blockIdx.x * APPEND_THREADS + threadIdx.x) / p.lanes);
    if (t >= p.T) return;
    const int len = max(ldi(p.lens + z), 0);
    const int nl = p.news != nullptr ? ldi(p.news + z) : p.T;
    if (t >= nl) return;
    const uint32_t pos = (uint32_t)len + (uint32_t)t, col = pos / (uint32_t)p.page;  // below 2^32
    const int e = col < (uint32_t)p.M ? ldi(p.table + z * p.st_z + col) : -1;
    if ((unsigned)e >= (unsigned)p.P) {
        bad_page(p.status, SITE_PAGE_APPEND);
        return;
    }
    const int64_t slot = pos - col * (uint32_t)p.page;
    const uint16_t* ks = p.ks + z * p.ks_z + t * p.ks_n;
    const uint16_t* vs = p.vs + z * p.vs_z + t * p.vs_n;
    uint16_t* kd = p.k.base + e * p.k.p + slot * p.k.n;
    uint16_t* vd = p.v.base + e * p.v.p + slot * p.v.n;
    const int shift = 31 - __clz(p.D / 8), n = p.H << shift;  // pieces of a row: a power of two
    constexpr int U = 4;
    for (int i0 = lane; i0 < n; i0 += U * p.lanes) {
        uint4 a[U], b[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * p.lanes, h = i >> shift, c = (i & ((1 << shift) - 1)) * 8;
            if (i < n) {
                a[u] = __ldcg(reinterpret_cast<const uint4*>(ks + h * p.ks_h + c));
                b[u] = __ldcg(reinterpret_cast<const uint4*>(vs + h * p.vs_h + c));
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * p.lanes, h = i >> shift, c = (i & ((1 << shift) - 1)) * 8;
            if (i < n) {
                *reinterpret_cast<uint4*>(kd + h * p.k.h + c) = a[u];
                *reinterpret_cast<uint4*>(vd + h * p.v.h + c) = b[u];
            }
        }
    }
}

// ------------------------------------------------------------ commit --------
// Position lens[z] + path[z][i] to lens[z] + i for i < kept[z], in place.  A
// CTA first turns a batch of steps into offsets within K and V; then one thread
// takes a 16-byte piece (of a layer, K or V, head) through the steps: with the
// path strictly increasing a step writes only where the same thread has
// already read (position lens[z] + i is read by no step after i), so steps need
// no barrier, and the reads of eight steps may go ahead of their writes.  64
// sequences x 9 tokens x 16 layers x 8 heads of D = 128 (33.6 MB): 9.0 us on new
// inputs, 3.7 TB/s, 7.2 to 8.0 repeated in a graph (16.5 with table look-ups in every
// thread); 4 sequences x 5 tokens: 2.8 to 3.1 us.
constexpr int COMMIT_THREADS = 256;
constexpr int COMMIT_BATCH = 64;

__global__ void __launch_bounds__(COMMIT_THREADS) fa_cache_commit_kernel(const CommitParams p) {
    __shared__ int64_t move[2][2][COMMIT_BATCH];  // [K, V][from, to][step]; from -1: nothing to do
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int tid = threadIdx.x, z = blockIdx.y;
    const int shift = 31 - __clz(p.D / 8);
    const uint32_t per_z = ((uint32_t)p.L * 2 * p.H) << shift;  // < 2^31 (checked on the host)
    const uint32_t i = blockIdx.x * COMMIT_THREADS + tid;
    const uint32_t c = i & ((1u << shift) - 1);
    uint32_t r = i >> shift;
    const uint32_t h = r % p.H;
    r /= p.H;
    const int is_v = r & 1u;
    const CacheView& cache = is_v ? p.v : p.k;
    uint16_t* base = cache.base + (int64_t)(r >> 1) * cache.l + h * cache.h + c * 8;
    const int n = min(ldi(p.kept + z), p.A);
    const int len = max(ldi(p.lens + z), 0);
    const int32_t* row = p.table + z * p.st_z;
    for (int b0 = 0; b0 < n; b0 += COMMIT_BATCH) {
        const int count = min(COMMIT_BATCH, n - b0);
        if (b0 > 0) __syncthreads();
        if (tid < 2 * count) {  // two threads a step: where it is, where it goes
            const int step = tid >> 1, to = tid & 1;
            const int from = ldi(p.path + z * p.sp_z + b0 + step), j = to ? b0 + step : from;
            const int64_t pos = (int64_t)len + j;
            int64_t k = -1, v = -1;
            if (from != b0 + step) {
                const uint32_t col = pos >= 0 && pos < (int64_t)p.M * p.page ? (uint32_t)pos / (uint32_t)p.page : 0u;
                const int e = pos >= 0 && pos < (int64_t)p.M * p.page ? ldi(row + col) : -1;
                if ((unsigned)e < (unsigned)p.P) {
                    const int64_t slot = (uint32_t)pos - col * (uint32_t)p.page;
                    k = e * p.k.p + slot * p.k.n;
                    v = e * p.v.p + slot * p.v.n;
                } else {
                    bad_page(p.status, SITE_PAGE_COMMIT);
                }
            }
            move[0][to][step] = k;
            move[1][to][step] = v;
        }
        __syncthreads();
        if (i >= per_z) continue;
        constexpr int U = 8;
        for (int s0 = 0; s0 < count; s0 += U) {
            uint4 v[U];
            bool go[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                go[u] = s0 + u < count && move[is_v][0][s0 + u] >= 0 && move[is_v][1][s0 + u] >= 0;
                if (go[u]) v[u] = __ldcg(reinterpret_cast<const uint4*>(base + move[is_v][0][s0 + u]));
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (go[u]) *reinterpret_cast<uint4*>(base + move[is_v][1][s0 + u]) = v[u];
        }
    }
}

// ------------------------------------------------------------ fork ----------
// Two kernels.  The first, one CTA, decides everything from the state as it
// was: each sequence's length after, which columns of its row need a page of
// its own, and which pages those are -- the lowest ones whose count is 0, in
// the order of sequences and columns (so the result does not depend on
// timing).  The second rewrites the table and counts, and copies the partly
// filled pages.  Bounded by latency in small pools: 6.3 us for 8 beams over 16 layers,
// 8.1 to 8.8 us for a batch of 96, about half for each kernel; a page of room that a
// sequence still has costs a dependent load, and used pages in front of the free ones
// 22 us per 100 000.  One cluster of eight CTAs with
// barriers between the phases instead took 14.0 and 22.4 us: too few loads in
// flight for the table and the tails.
constexpr int PLAN_THREADS = 1024;

struct ForkWs {
    int32_t *src, *len, *first, *count, *off, *from, *tail, *found, *pages;
};
__device__ __forceinline__ ForkWs fork_ws(const ForkParams& p) {
    ForkWs w;
    w.src = p.ws;
    w.len = w.src + p.Z;
    w.first = w.len + p.Z;
    w.count = w.first + p.Z;
    w.off = w.count + p.Z;
    w.from = w.off + p.Z;
    w.tail = w.from + p.Z;        // list of tails: from page, to page, rows
    w.found = w.tail + 3 * p.Z;   // pages found, tails
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
    __shared__ int tails;
    __shared__ unsigned long long excess;
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const ForkWs w = fork_ws(p);
    const int tid = threadIdx.x;
    if (tid == 0) {
        tails = 0;
        excess = 0;
    }
    __syncthreads();
    const int cap = p.M * p.page;
    int wanted = 0;
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
            const int full = len / p.page, rows = len - full * p.page;
            const int from = rows > 0 ? ldi(p.table + src * p.st_z + full) : -1;  // (full < M)
            int first = full + (src == z && rows > 0);
            if (src == z)
                while (first < min(need, p.M) && ldi(p.table + z * p.st_z + first) >= 0) ++first;  // room it has
            // The rows of a partly filled page that is not in the table are lost (a call that
            // ran short has left it uncopied).  No page can bring them back: what they and
            // all behind them need goes on lacking, in copies too.
            const bool lost = rows > 0 && (unsigned)from >= (unsigned)p.P;
            count = lost ? 0 : max(0, min(need, p.M) - first);
            over = lost ? need - full : max(0, need - p.M);
            if (lost && src != z) bad_page(p.status, SITE_PAGE_FORK);
            w.src[z] = src;
            w.from[z] = from;
            w.len[z] = len;
            w.first[z] = first;
            w.count[z] = count;
        }
        int sum, off = block_scan(count, red, &sum);
        if (z < p.Z) w.off[z] = wanted + off;
        wanted += sum;
        if (over > 0) atomicAdd(&excess, (unsigned long long)over);
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
    // tails: the partly filled last page of a source goes to the copy's first own
    // page (the list's order is of no account: no page is in it twice as a target,
    // and no target is a source)
    for (int z = tid; z < p.Z; z += PLAN_THREADS) {
        const int src = w.src[z], rows = w.len[z] % p.page;
        if (src < 0 || src == z || rows == 0 || w.off[z] >= found || w.count[z] == 0) continue;
        int32_t* t = w.tail + 3 * atomicAdd(&tails, 1);
        t[0] = w.from[z];
        t[1] = w.pages[w.off[z]];
        t[2] = rows;
    }
    __syncthreads();
    if (tid == 0) {
        const long long lack = (long long)wanted - found + (long long)excess;
        const bool none = p.whole && lack > 0;
        w.found[0] = none ? -1 : found;
        w.found[1] = none ? 0 : tails;
        if (p.missing != nullptr) *p.missing = (int)min(lack, (long long)INT_MAX);
    }
}

// Table, lengths and counts: a CTA takes `cols` columns of every row, reads
// them all before it writes any (a source row may be rewritten in the same
// call), and counts one reference less for what a changed row held and one
// more for what it holds.  The warps of the other CTAs copy tails, a (tail,
// layer, K or V, head) at a time.
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
        if (found < 0) return;  // all or nothing, and pages lack
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
    // a warp per (tail, layer, K or V, head)
    const int shift = 31 - __clz(p.D / 8), lane = tid % 32, per_tail = p.L * 2 * p.H;
    const int64_t jobs = (int64_t)ldi(w.found + 1) * per_tail;
    const int64_t warps = (int64_t)(gridDim.x - a.table_ctas) * (FORK_THREADS / 32);
    for (int64_t j = (int64_t)(blockIdx.x - a.table_ctas) * (FORK_THREADS / 32) + tid / 32; j < jobs; j += warps) {
        const int i = (int)(j / per_tail), r = (int)(j - (int64_t)i * per_tail), lk = r / p.H, h = r - lk * p.H;
        const int64_t from = ldi(w.tail + 3 * i), to = ldi(w.tail + 3 * i + 1);
        const int n = ldi(w.tail + 3 * i + 2) << shift;
        const CacheView& cache = lk & 1 ? p.v : p.k;
        uint16_t* base = cache.base + (int64_t)(lk >> 1) * cache.l + h * cache.h;
        constexpr int U = 8;
        for (int i0 = lane; i0 < n; i0 += 32 * U) {
            uint4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int x = i0 + 32 * u;
                if (x < n)
                    v[u] = __ldcg(reinterpret_cast<const uint4*>(base + from * cache.p + (x >> shift) * cache.n +
                                                                 (x & ((1 << shift) - 1)) * 8));
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int x = i0 + 32 * u;
                if (x < n)
                    *reinterpret_cast<uint4*>(base + to * cache.p + (x >> shift) * cache.n + (x & ((1 << shift) - 1)) * 8) = v[u];
            }
        }
    }
}

}  // namespace

cudaError_t launch_cache_append(AppendParams p, cudaStream_t stream) {
    p.lanes = 1;
    while (p.lanes < 32 && p.lanes < p.H * (p.D / 8)) p.lanes *= 2;
    return launch_dependent(fa_cache_append_kernel, dim3((unsigned)(((int64_t)p.T * p.lanes + APPEND_THREADS - 1) / APPEND_THREADS), (unsigned)p.Z),
                            APPEND_THREADS, 0, stream, p);
}

cudaError_t launch_cache_commit(const CommitParams& p, cudaStream_t stream) {
    const int64_t per_z = (int64_t)p.L * 2 * p.H * (p.D / 8);
    return launch_dependent(fa_cache_commit_kernel, dim3((unsigned)((per_z + COMMIT_THREADS - 1) / COMMIT_THREADS), (unsigned)p.Z),
                            COMMIT_THREADS, 0, stream, p);
}

cudaError_t launch_cache_fork(const ForkParams& p, int sms, cudaStream_t stream) {
    cudaError_t err = launch_dependent(fa_cache_fork_plan_kernel, dim3(1), PLAN_THREADS, 0, stream, p);
    if (err != cudaSuccess) return err;
    ForkApply a{p, 1, 0};
    // columns a CTA: about two table entries a thread (32 KB of shared memory at most, Z <= 8192)
    a.cols = 2 * FORK_THREADS / p.Z;
    a.cols = a.cols < 1 ? 1 : a.cols > 32 ? 32 : a.cols;
    a.table_ctas = p.M > 0 ? (p.M + a.cols - 1) / a.cols : 1;  // the first writes the lengths
    const int64_t jobs = ((int64_t)p.Z * p.L * 2 * p.H + FORK_THREADS / 32 - 1) / (FORK_THREADS / 32);  // at most
    const int64_t copies = p.source == nullptr ? 0 : jobs < 8 * sms ? jobs : 8 * sms;
    return launch_dependent(fa_cache_fork_apply_kernel, dim3((unsigned)(a.table_ctas + copies)), FORK_THREADS,
                            (size_t)p.Z * a.cols * sizeof(int), stream, a);
}

}  // namespace fa
