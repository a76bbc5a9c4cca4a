// Cutting the sequences of a paged cache back to a budget: of each (layer, sequence, kv
// head) the positions with the highest scores stay, in their order, and move together.
//
// Three kernels.  The first, a CTA a (layer, sequence, head), selects: a histogram of the
// keys' upper 11 bits finds where the n-th highest score lies, the few keys there are
// ranked against one another (or, if they are many, 11 and 10 bits more are counted), and
// then the positions that stay are listed.  The second, one CTA, does the books: pages that are
// rewritten but shared with other sequences are replaced by free ones, lowest first in
// the order of sequences and columns (so the result does not depend on timing).  The
// third moves the rows, in place, and writes tables, counts and lengths.
//
// What bounds it is the rows that move: 8 D bytes each, against 4 to 12 bytes of
// selection a position.  32 sequences of 1500-2900 positions cut to 1024, 8 layers x 8 heads
// of D = 128 (2.2 GB): 36 us to select, 19 for the books, 326 to move (6.6 TB/s, nearly a
// plain copy's rate), in all, since the launches overlap, 366.  One sequence of 1200, 16 layers
// (134 MB): 6.4, 6.7 and 25 us, in all 32.5, of which the books are one CTA's chain of dependent
// loads.  (In all: repeated in a graph, without the copies that put the sequences back.)  Every
// row behind the first one that goes moves: from 1025 positions to 1024 the one sequence takes
// 27 us and the 32 take 214, where 1200 and 1500-2900 take 31 and 410 on the same pages of 16.
#include "fa_evict.h"

#include <climits>

#include "fa_cache.cuh"
#include "fa_paged.h"
#include "fa_ptx.cuh"

namespace fa {

namespace {

struct EvictWs {
    int32_t *target, *own, *off, *lack, *before, *after, *pages, *first, *idx;
};
__device__ __forceinline__ EvictWs evict_ws(const EvictParams& p) {
    EvictWs w;
    const int64_t zm = (int64_t)p.Z * p.M;
    w.target = p.ws;
    w.own = w.target + p.Z;
    w.off = w.own + p.Z;
    w.lack = w.off + p.Z;
    w.before = w.lack + 1;
    w.after = w.before + zm;
    w.pages = w.after + zm;
    w.first = w.pages + zm;
    w.idx = w.first + (int64_t)p.L * p.Z * p.H;
    return w;
}

// What a sequence is cut to; -1: it stays as it is.
__device__ __forceinline__ int cut_to(const EvictParams& p, int z, int len) {
    int n = p.budget;
    if (p.keep != nullptr) {
        const int k = ldi(p.keep + z);
        if (k < 0) return -1;
        n = min(n, k);
    }
    return len > n ? n : -1;
}
__device__ __forceinline__ int held_len(const EvictParams& p, int z) { return min(max(ldi(p.lens + z), 0), p.P > 0 ? p.M * p.page : 0); }

// ------------------------------------------------------------ select --------
constexpr int SELECT_THREADS = 256;
constexpr int SELECT_WARPS = SELECT_THREADS / 32;
constexpr int BINS = 2048;
constexpr int LISTED = 512;  // keys that are ranked against one another

// Unsigned keys in the order of the scores; -0 is 0, a NaN is above everything.
__device__ __forceinline__ uint32_t score_key(float x) {
    if (x != x) return 0xffffffffu;
    const uint32_t b = __float_as_uint(x == 0.f ? 0.f : x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__global__ void __launch_bounds__(SELECT_THREADS, 6) fa_evict_select_kernel(const EvictParams p, int held) {
    extern __shared__ uint32_t keys_held[];  // the candidates' keys, if they fit
    __shared__ __align__(16) int hist[BINS];  // the highest digit first
    __shared__ uint32_t list[LISTED];
    __shared__ int red[SELECT_WARPS], red2[SELECT_WARPS], found[3], listed, first_moved;
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const EvictWs w = evict_ws(p);
    const int h = blockIdx.x, z = blockIdx.y, l = blockIdx.z;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int len = held_len(p, z), target = cut_to(p, z, len);
    if (h == 0 && l == 0 && tid == 0) w.target[z] = target;
    if (target < 0) return;
    // the sequence's table row, a share of it each (p.M may be large where sequences are short)
    for (int64_t c = ((int64_t)l * p.H + h) * SELECT_THREADS + tid; c < p.M; c += (int64_t)p.L * p.H * SELECT_THREADS)
        w.before[(int64_t)z * p.M + c] = ldi(p.table + z * p.st_z + c);
    const int64_t unit = ((int64_t)l * p.Z + z) * p.H + h;
    const int front = min(p.first, target), back = min(p.recent, target - front);
    const int n = len - back - front, m = target - back - front;  // candidates, and how many of them stay: m < n
    const float* from = p.scores + l * p.ss_l + z * p.ss_z + h * p.ss_h + front;
    const bool fits = n <= held;
    if (fits) {
        constexpr int U = 8;
        for (int i0 = tid; i0 < n; i0 += U * SELECT_THREADS) {
            float v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = i0 + u * SELECT_THREADS < n ? __ldcg(from + i0 + u * SELECT_THREADS) : 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i0 + u * SELECT_THREADS < n) keys_held[i0 + u * SELECT_THREADS] = score_key(v[u]);
        }
    }
    auto key = [&](int i) { return fits ? keys_held[i] : score_key(__ldcg(from + i)); };

    // the m-th highest key: its bits from the top, 11, 11 and 10 at a time; `want` is how
    // many keys with these upper bits stay
    uint32_t prefix = 0;
    int want = m;
    if (m > 0)
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
            const uint32_t above = pass == 0 ? 0u : ~0u << (shift + bits);
            for (int i = tid; i < BINS / 4; i += SELECT_THREADS) reinterpret_cast<int4*>(hist)[i] = make_int4(0, 0, 0, 0);
            if (tid == 0) listed = 0;
            __syncthreads();
            for (int i = tid; i < n; i += SELECT_THREADS) {
                const uint32_t k = key(i);
                if ((k & above) == prefix) atomicAdd(&hist[BINS - 1 - ((k >> shift) & ((1u << bits) - 1))], 1);
            }
            __syncthreads();
            // a thread sums eight bins
            static_assert(BINS == 8 * SELECT_THREADS, "bins of a thread");
            const int4 lo = reinterpret_cast<const int4*>(hist)[2 * tid], hi = reinterpret_cast<const int4*>(hist)[2 * tid + 1];
            const int bin[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            const int mine = ((bin[0] + bin[1]) + (bin[2] + bin[3])) + ((bin[4] + bin[5]) + (bin[6] + bin[7]));
            int x = mine;
            for (int d = 1; d < 32; d *= 2) {
                const int y = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += y;
            }
            if (lane == 31) red[warp] = x;
            __syncthreads();
            for (int i = 0; i < warp; ++i) x += red[i];
            if (x >= want && x - mine < want) {  // one thread
                int before = x - mine;
                bool done = false;
#pragma unroll
                for (int b = 0; b < 8; ++b)
                    if (!done) {
                        if (before + bin[b] >= want) {
                            found[0] = BINS - 1 - (8 * tid + b);
                            found[1] = want - before;
                            found[2] = bin[b];
                            done = true;
                        }
                        before += bin[b];
                    }
            }
            __syncthreads();
            prefix |= (uint32_t)found[0] << shift;
            want = found[1];
            const int same = found[2];
            if (pass == 0 && same <= LISTED) {
                for (int i = tid; i < n; i += SELECT_THREADS) {
                    const uint32_t k = key(i);
                    if (k >> 21 == prefix >> 21) list[atomicAdd(&listed, 1)] = k;
                }
                __syncthreads();
                for (int i = tid; i < same; i += SELECT_THREADS) {
                    const uint32_t k = list[i];
                    int higher = 0, equal = 0;
#pragma unroll 4
                    for (int j = 0; j < same; ++j) {
                        higher += list[j] > k;
                        equal += list[j] == k;
                    }
                    if (higher < want && want <= higher + equal) {  // (equal ones write the same)
                        found[0] = (int)k;
                        found[1] = want - higher;
                    }
                }
                __syncthreads();
                prefix = (uint32_t)found[0];
                want = found[1];
                break;
            }
        }
    __syncthreads();
    // Keys above the prefix stay, and of those equal to it the first `want`.  A warp takes
    // a contiguous share of the candidates.
    const int share = ((n + SELECT_WARPS - 1) / SELECT_WARPS + 31) / 32 * 32;
    const int i0 = min(warp * share, n), i1 = min(i0 + share, n);
    int higher = 0, equal = 0;
    if (m > 0)
        for (int i = i0; i < i1; i += 32) {
            const bool in = i + lane < i1;
            const uint32_t k = in ? key(i + lane) : 0u;
            higher += __popc(__ballot_sync(0xffffffffu, in && k > prefix));
            equal += __popc(__ballot_sync(0xffffffffu, in && k == prefix));
        }
    if (lane == 0) {
        red[warp] = higher;
        red2[warp] = equal;
    }
    if (tid == 0) first_moved = target;
    __syncthreads();
    int to = front, ties = want;  // where this warp's first one goes, and how many equal ones are left for it
    for (int i = 0; i < warp; ++i) {
        to += red[i] + min(ties, red2[i]);
        ties -= min(ties, red2[i]);
    }
    int32_t* idx = w.idx + unit * p.budget;
    int moved = target;
    if (m > 0)
        for (int i = i0; i < i1; i += 32) {
            const bool in = i + lane < i1;
            const uint32_t k = in ? key(i + lane) : 0u;
            const uint32_t hi = __ballot_sync(0xffffffffu, in && k > prefix), eq = __ballot_sync(0xffffffffu, in && k == prefix);
            const uint32_t below = (1u << lane) - 1;
            const bool stays = in && (k > prefix || (k == prefix && __popc(eq & below) < ties));
            if (stays) {
                const int at = to + __popc(hi & below) + min(ties, __popc(eq & below));
                idx[at] = front + i + lane;
                if (at != front + i + lane) moved = min(moved, at);
            }
            to += __popc(hi) + min(ties, __popc(eq));
            ties -= min(ties, __popc(eq));
        }
    for (int i = tid; i < front; i += SELECT_THREADS) idx[i] = i;
    for (int i = tid; i < back; i += SELECT_THREADS) idx[front + m + i] = len - back + i;
    if (tid == 0 && back > 0) moved = min(moved, front + m);  // (len - back > front + m)
    for (int d = 16; d > 0; d /= 2) moved = min(moved, __shfl_xor_sync(0xffffffffu, moved, d));
    if (lane == 0) atomicMin(&first_moved, moved);
    __syncthreads();
    if (tid == 0) w.first[unit] = first_moved;
}

// ------------------------------------------------------------ plan ----------
constexpr int EVICT_PLAN_THREADS = 1024;

// exclusive prefix sum over the CTA; total in *sum
__device__ __forceinline__ int cta_scan(int v, int* red, int* sum) {
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

__global__ void __launch_bounds__(EVICT_PLAN_THREADS) fa_evict_plan_kernel(const EvictParams p) {
    __shared__ int red[32];
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const EvictWs w = evict_ws(p);
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    constexpr int WARPS = EVICT_PLAN_THREADS / 32;
    // a warp a sequence: its first page that is rewritten, and how many from there on are shared
    bool any = false;
    for (int z = warp; z < p.Z; z += WARPS) {
        const int target = ldi(w.target + z);
        int count = 0, own = 0;
        if (target >= 0) {
            int first = target;
            for (int i = lane; i < p.L * p.H; i += 32) {
                const int l = i / p.H, h = i - l * p.H;
                first = min(first, ldi(w.first + ((int64_t)l * p.Z + z) * p.H + h));
            }
            for (int d = 16; d > 0; d /= 2) first = min(first, __shfl_xor_sync(0xffffffffu, first, d));
            own = first / p.page;
            const int need = (target + p.page - 1) / p.page;
            for (int c = own + lane; c < need; c += 32) {
                const int e = ldi(w.before + (int64_t)z * p.M + c);
                count += (unsigned)e < (unsigned)p.P && ldi(p.refs + e) > 1;
            }
            for (int d = 16; d > 0; d /= 2) count += __shfl_xor_sync(0xffffffffu, count, d);
        }
        if (lane == 0) {
            w.own[z] = own;
            w.off[z] = count;
        }
        any |= count > 0;
    }
    if (!__syncthreads_or(any)) {  // each page is its sequence's own: the rows of the table only get shorter
        if (tid == 0) {
            *w.lack = -1;
            *p.missing = 0;
        }
        return;
    }
    int wanted = 0;
    for (int z0 = 0; z0 < p.Z; z0 += EVICT_PLAN_THREADS) {
        const int z = z0 + tid;
        int sum, off = cta_scan(z < p.Z ? ldi(w.off + z) : 0, red, &sum);
        if (z < p.Z) w.off[z] = wanted + off;
        wanted += sum;
    }
    // the first `wanted` pages with count 0
    int found = 0;
    for (int p0 = 0; p0 < p.P && found < wanted; p0 += 4 * EVICT_PLAN_THREADS) {
        const int i = p0 + 4 * tid;
        int c[4], k = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            c[u] = i + u < p.P ? ldi(p.refs + i + u) : 1;
            k += c[u] == 0;
        }
        int sum, at = found + cta_scan(k, red, &sum);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (c[u] == 0) {
                if (at < wanted) w.pages[at] = i + u;
                ++at;
            }
        found += sum;
    }
    const int lack = max(0, wanted - found);
    if (tid == 0) {
        *w.lack = lack;
        *p.missing = lack;
    }
    __syncthreads();
    if (lack > 0) return;
    // the rows as they will be
    for (int z = warp; z < p.Z; z += WARPS) {
        const int target = ldi(w.target + z);
        if (target < 0) continue;
        const int own = ldi(w.own + z), need = (target + p.page - 1) / p.page;
        int off = ldi(w.off + z);
        for (int c0 = 0; c0 < need; c0 += 32) {
            const int c = c0 + lane, e = c < need ? ldi(w.before + (int64_t)z * p.M + c) : -1;
            const bool shared = c >= own && (unsigned)e < (unsigned)p.P && ldi(p.refs + e) > 1;
            const uint32_t all = __ballot_sync(0xffffffffu, shared);
            if (c < need) w.after[(int64_t)z * p.M + c] = shared ? ldi(w.pages + off + __popc(all & ((1u << lane) - 1))) : e;
            off += __popc(all);
        }
    }
}

// ------------------------------------------------------------ move ----------
// Row idx[i] to row i of each (layer, sequence, head), K and V, and its score.  idx[i] >=
// i increases with i, so what a row overwrites is read by no later row: within a CTA the
// rows go in chunks, the reads of a chunk before its writes, and those of the next chunk
// go ahead of the writes of this one.  Where the rows are is looked up for 256 of them at
// a time, a batch ahead.
constexpr int MOVE_THREADS = 256;

struct EvictMove {
    EvictParams p;
    int table_ctas;
    int parts;       // CTAs that share the columns of a (layer, sequence, head, K or V)
    int64_t movers;  // CTAs that move K and V
};

__global__ void __launch_bounds__(MOVE_THREADS, 4) fa_evict_move_kernel(const __grid_constant__ EvictMove a) {
    const EvictParams& p = a.p;
    constexpr int U = 4;
    __shared__ int64_t where[2][2][MOVE_THREADS];  // [batch parity][from, to][row]; from -1: it stays
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const EvictWs w = evict_ws(p);
    const int tid = threadIdx.x;
    const int lack = ldi(w.lack);
    if (lack > 0) return;
    const int32_t* rows_after = lack < 0 ? w.before : w.after;
    if ((int)blockIdx.x < a.table_ctas) {  // the books
        const int chunks = (p.M + MOVE_THREADS - 1) / MOVE_THREADS;
        for (int64_t i = blockIdx.x; i < (int64_t)p.Z * chunks; i += a.table_ctas) {
            const int z = (int)(i / chunks), k = (int)(i - (int64_t)z * chunks), c = k * MOVE_THREADS + tid;
            const int target = ldi(w.target + z);
            if (target < 0) continue;
            const int need = (target + p.page - 1) / p.page;
            if (c < p.M) {
                const int was = ldi(w.before + (int64_t)z * p.M + c);
                const int now = c < need ? ldi(rows_after + (int64_t)z * p.M + c) : -1;
                if (now != was) {
                    if ((unsigned)was < (unsigned)p.P) atomicAdd(p.refs + was, -1);
                    if ((unsigned)now < (unsigned)p.P) atomicAdd(p.refs + now, 1);
                    p.table[z * p.st_z + c] = now;
                }
            }
            if (k == 0 && tid == 0) p.lens[z] = target;
        }
        return;
    }
    const int64_t block = (int64_t)blockIdx.x - a.table_ctas;
    const bool moves = block < a.movers;  // else the scores of a (layer, sequence, head)
    const int64_t both = moves ? block / a.parts : 2 * (block - a.movers), unit = both / 2;
    const int h = (int)(unit % p.H), z = (int)(unit / p.H % p.Z), l = (int)(unit / p.H / p.Z);
    const int target = ldi(w.target + z);
    if (target < 0) return;
    const int32_t *idx = w.idx + unit * p.budget, *before = w.before + (int64_t)z * p.M, *after = rows_after + (int64_t)z * p.M;
    const int unmoved = ldi(w.first + unit);
    if (!moves) {
        float* s = p.scores + l * p.ss_l + z * p.ss_z + h * p.ss_h;
        for (int i0 = unmoved; i0 < target; i0 += U * MOVE_THREADS) {
            float v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * MOVE_THREADS + tid;
                if (i < target) v[u] = __ldcg(s + ldi(idx + i));
            }
            __syncthreads();
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * MOVE_THREADS + tid;
                if (i < target) s[i] = v[u];
            }
        }
        return;
    }
    const CacheView& cache = both % 2 == 0 ? p.k : p.v;
    // this CTA's columns of a row, in 16-byte pieces a lane; all powers of two
    const int per = p.D / 8 / a.parts, shift = 31 - __clz(per), side = MOVE_THREADS >> shift;
    uint16_t* base = cache.base + l * cache.l + h * cache.h + ((int)(block % a.parts) * per + (tid & (per - 1))) * 8;
    const int row = tid >> shift;
    const int start = min(ldi(w.own + z) * p.page, target);
    bool bad = false;
    auto find = [&](int i, int half) {  // row i, by thread i - the batch's first row
        int64_t from = -1, to = -1;
        if (i < target) {
            const int j = i < unmoved ? i : ldi(idx + i);
            const int cf = p.by_page(j), ct = p.by_page(i);
            const int ef = ldi(before + cf), et = ldi(after + ct);
            if (j != i || ef != et) {
                if ((unsigned)ef < (unsigned)p.P && (unsigned)et < (unsigned)p.P) {
                    from = ef * cache.p + (j - cf * p.page) * cache.n;
                    to = et * cache.p + (i - ct * p.page) * cache.n;
                } else {
                    bad = true;
                }
            }
        }
        where[half][0][tid] = from;
        where[half][1][tid] = to;
    };
    const int chunk = min(U * side, MOVE_THREADS), chunks = (target - start + chunk - 1) / chunk;
    const int a_batch = MOVE_THREADS / chunk;  // chunks: a power of two
    uint4 now[U], then[U];
    auto load = [&](int k, uint4 (&v)[U]) {
        const int r0 = (k & (a_batch - 1)) * chunk, half = (k / a_batch) & 1;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * side + row;
            if (u * side < chunk && where[half][0][r] >= 0) v[u] = __ldcg(reinterpret_cast<const uint4*>(base + where[half][0][r]));
        }
    };
    auto store = [&](int k, const uint4 (&v)[U]) {
        const int r0 = (k & (a_batch - 1)) * chunk, half = (k / a_batch) & 1;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * side + row;
            if (u * side < chunk && where[half][0][r] >= 0) *reinterpret_cast<uint4*>(base + where[half][1][r]) = v[u];
        }
    };
    if (chunks > 0) {
        find(start + tid, 0);
        __syncthreads();
        load(0, now);
    }
    for (int k = 0; k < chunks; ++k) {
        __syncthreads();  // this chunk has been read, and the batch before is done
        const int next = k / a_batch + 1;
        if (k % a_batch == 0 && next * a_batch < chunks) {
            find(start + next * MOVE_THREADS + tid, next & 1);
            if (a_batch == 1) __syncthreads();
        }
        if (k + 1 < chunks) load(k + 1, then);
        store(k, now);
#pragma unroll
        for (int u = 0; u < U; ++u) now[u] = then[u];
    }
    if (bad) bad_page(p.status, SITE_PAGE_EVICT);
}

}  // namespace

cudaError_t launch_cache_evict(const EvictParams& p, int sms, cudaStream_t stream) {
    // keys of up to 8192 candidates are held in shared memory
    const int64_t cap = (int64_t)p.M * p.page;
    const int held = (int)(cap < 8192 ? cap : 8192);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.H, (unsigned)p.Z, (unsigned)p.L);
    cfg.blockDim = dim3(SELECT_THREADS);
    cfg.dynamicSmemBytes = (size_t)held * sizeof(uint32_t);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t err = cudaLaunchKernelEx(&cfg, fa_evict_select_kernel, p, held);
    if (err != cudaSuccess) return err;
    err = launch_dependent(fa_evict_plan_kernel, dim3(1), EVICT_PLAN_THREADS, 0, stream, p);
    if (err != cudaSuccess) return err;
    const int64_t chunks = (int64_t)p.Z * ((p.M + MOVE_THREADS - 1) / MOVE_THREADS);
    EvictMove a{p, (int)(chunks < sms ? chunks : sms), 1, 0};
    const int64_t units = (int64_t)p.L * p.Z * p.H;
    // few units: their columns in up to four parts of 64 bytes at least, until every SM has
    // its four CTAs
    while (a.parts < 4 && p.D / 8 / a.parts > 4 && units * 2 * a.parts * 2 <= 4 * (int64_t)sms) a.parts *= 2;
    a.movers = units * 2 * a.parts;
    return launch_dependent(fa_evict_move_kernel, dim3((unsigned)(a.table_ctas + a.movers + units)), MOVE_THREADS, 0, stream, a);
}

}  // namespace fa
