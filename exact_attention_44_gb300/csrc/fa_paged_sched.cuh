// Work division of the paged attention kernels, computed on the device: the
// lengths live there, and a call reads nothing back.
//
// A tile is up to p.tile_rows query rows of one (sequence, kv head); a row is
// a (new token, query head of the group) pair with the heads innermost, so
// that the rows of a sequence with fewer new tokens than T are a prefix and
// the K/V rows are read once for the whole group.  A worker is a warp of the
// rows kernel or a CTA of the tile kernel.  p.team workers form a team that
// takes p.team neighbouring tiles of a kv head at the same time, one each,
// over the same key blocks, so that the blocks come from DRAM once and from L2
// for the others.  The (tile group, key block) pairs, in the order sequence,
// kv head, group, block, are laid end to end and cut into one equal range per
// team, whatever the lengths are (a cut inside a group of at most p.snap blocks
// moves to the group's end); a tile that a cut crosses leaves partial results
// (O / l in fp32 and the base-2 log-sum-exp) in slots of the workspace, two per
// worker, and fa_paged_merge_kernel joins them in the order of the keys.
// Nothing depends on timing: the same inputs give the same bits.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_paged.h"
#include "fa_ptx.cuh"

namespace fa {

// Loads through L2.  The kernels are launched as programmatic dependents, so
// they may be resident before the kernel that writes their inputs has
// finished; a line of the L1 cache could then be older than the data.
__device__ __forceinline__ int ldi(const int32_t* p) { return __ldcg(p); }

// Lengths of a sequence, clamped to what its block table can hold: `len`
// positions before the new tokens, `nl` new tokens.
struct SeqLen {
    int len, nl;
};
__device__ __forceinline__ SeqLen seq_len(const PagedParams& p, int z) {
    SeqLen s;
    const int n = ldi(p.lens + z);
    const int m = p.news != nullptr ? ldi(p.news + z) : p.T;
    s.len = min(max(n, 0), p.cap);
    s.nl = min(max(m, 0), min(p.T, p.cap - s.len));
    return s;
}

// Key blocks of BK positions that tile mt sees.  With the chain rule (no
// mask) a tile stops at the block of its last token; with a mask any token may
// be seen.
template <int BK>
__device__ __forceinline__ int tile_blocks(const PagedParams& p, const SeqLen& s, int mt) {
    int end = s.len + s.nl;
    if (p.mask == nullptr) {
        const int last = min((mt + 1) * p.tile_rows, s.nl * p.G) - 1;
        end = s.len + p.by_g(last) + 1;
    }
    return (end + BK - 1) / BK;
}
__device__ __forceinline__ int live_tiles(const PagedParams& p, const SeqLen& s) {
    return p.by_tile_rows(s.nl * p.G + p.tile_rows - 1);
}
__device__ __forceinline__ int live_groups(const PagedParams& p, const SeqLen& s) {
    return p.by_team(live_tiles(p, s) + p.team - 1);
}
// blocks of tile group gi: those of its last tile (a tile of a chain sees at
// least what the one before it sees; tile_blocks stops at the live rows)
template <int BK>
__device__ __forceinline__ int group_blocks(const PagedParams& p, const SeqLen& s, int gi) {
    return tile_blocks<BK>(p, s, (gi + 1) * p.team - 1);
}
// blocks of all groups of one (sequence, kv head)
template <int BK>
__device__ __forceinline__ int64_t head_blocks(const PagedParams& p, const SeqLen& s) {
    if (s.nl == 0) return 0;
    const int n = live_groups(p, s);
    if (p.mask != nullptr) return (int64_t)n * group_blocks<BK>(p, s, 0);
    int64_t sum = 0;
    for (int i = 0; i < n; ++i) sum += group_blocks<BK>(p, s, i);
    return sum;
}

// Sum over the block's threads; `red` holds one value per warp.
__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* red) {
    for (int m = 16; m > 0; m /= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
    __syncthreads();
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    int64_t s = 0;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) s += red[w];
    return s;
}

// A team's place in the order, and the lengths of its sequence.
struct PagedWalk {
    int z, hk, gi;   // tile group
    int jb;          // its first block in this range
    int groups;      // of its sequence
    int64_t left;    // blocks left in the range
    SeqLen s;
};
// A worker's part of it: one tile's key blocks.
struct PagedSeg {
    int z, hk;
    int jb, je;      // key blocks
    int slot;        // -1: the whole tile; else where its part goes
    int len, nl;
    int row0, rows;  // first query row of the tile and its live rows
};
// On to the next tile group (sequences without new tokens have none).
template <int BK>
__device__ __forceinline__ void paged_next(const PagedParams& p, PagedWalk& w) {
    w.left -= group_blocks<BK>(p, w.s, w.gi) - w.jb;
    w.jb = 0;
    if (w.left <= 0) return;
    if (++w.gi < w.groups) return;
    w.gi = 0;
    if (++w.hk < p.Hkv) return;
    w.hk = 0;
    do {
        if (++w.z >= p.Z) {
            w.left = 0;
            return;
        }
        w.s = seq_len(p, w.z);
    } while (w.s.nl == 0);
    w.groups = live_groups(p, w.s);
}

// Unsigned division that takes the 32-bit route where both fit: the 64-bit one
// costs a few hundred cycles, which a short call would feel.
__device__ __forceinline__ int64_t fast_div(int64_t a, int64_t b) {
    return ((uint64_t)(a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// The cut of `total` blocks into `teams` ranges: q blocks each, one more for
// the first rem.  There are no empty ranges (the merge reads the slots of every
// range between a tile's first and last).
struct PagedCuts {
    int64_t q;
    int rem, teams;
    __device__ __forceinline__ int64_t start(int c) const { return q * c + min(c, rem); }
    __device__ __forceinline__ int team_of(int64_t x) const {
        const int64_t big = (q + 1) * rem;
        return x < big ? (int)fast_div(x, q + 1) : rem + (int)fast_div(x - big, q);
    }
};
__device__ __forceinline__ PagedCuts paged_cuts(const PagedParams& p, int64_t total) {
    PagedCuts c{0, 0, (int)min((int64_t)p.teams, total)};
    if (total > 0) {
        c.q = fast_div(total, c.teams);
        c.rem = (int)(total - c.q * c.teams);
    }
    return c;
}

// Where a team's range starts, for the merge (z = -1: it has none).
struct alignas(16) PagedCut {
    int z, hk, gi, jb;
    int len, nl, rem, teams;
    int64_t q;
};

template <int RANGES>
struct PagedFind {
    int64_t red[32];
    int64_t z_before[RANGES];  // blocks before sequence z
    int64_t lo[RANGES];
    int z[RANGES], len[RANGES], nl[RANGES];
};

// Where the range of team first + mine starts (RANGES teams a CTA, mine the same
// in all threads of a warp), recorded for the merge by the thread that
// `records`.  pads: some sequence has fewer than T new tokens.  Called by every
// thread of the CTA; with few sequences (p.few) the warps need not all call it.
template <int BK, int RANGES>
__device__ __forceinline__ PagedWalk paged_range(const PagedParams& p, PagedFind<RANGES>* f, int first, int mine,
                                              bool records, bool& pads) {
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid % 32;
    const int c = first + mine;
    PagedWalk w{-1, 0, 0, 0, 0, 0, {0, 0}};
    PagedCuts cuts{0, 0, 0};
    if (p.few) {
        // Few sequences: each warp by itself, one sequence a lane, in 32 bits.  This
        // stands between the launch and the first copy.
        SeqLen s{0, 0};
        int per = 0;
        if (lane < p.Z) {
            s = seq_len(p, lane);
            per = (int)head_blocks<BK>(p, s);
        }
        pads = __any_sync(0xffffffffu, lane < p.Z && s.nl < p.T);
        const int v = per * p.Hkv;
        int x = v;
        for (int d = 1; d < 32; d *= 2) {
            const int y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        const int total = __shfl_sync(0xffffffffu, x, 31);
        cuts = paged_cuts(p, total);
        if (c < cuts.teams) {
            const int lo = (int)cuts.start(c);
            w.z = __ffs(__ballot_sync(0xffffffffu, lo < x)) - 1;
            per = __shfl_sync(0xffffffffu, per, w.z);
            w.s = SeqLen{__shfl_sync(0xffffffffu, s.len, w.z), __shfl_sync(0xffffffffu, s.nl, w.z)};
            int rem = lo - __shfl_sync(0xffffffffu, x - v, w.z);
            w.hk = p.Hkv <= 32 ? __popc(__ballot_sync(0xffffffffu, (lane + 1) * (int64_t)per <= rem)) : rem / per;
            rem -= w.hk * per;
            for (int n; rem >= (n = group_blocks<BK>(p, w.s, w.gi)); ++w.gi) rem -= n;
            w.jb = rem;
            w.left = (int)cuts.start(c + 1) - lo;
            w.groups = live_groups(p, w.s);
        }
    } else {
        SeqLen s{0, 0};
        int64_t own = 0, v = 0;
        bool pad = false;
#pragma unroll 4
        for (int z = tid; z < p.Z; z += nt) {
            s = seq_len(p, z);
            v = p.Hkv * head_blocks<BK>(p, s);
            own += v;
            pad |= s.nl < p.T;
        }
        cuts = paged_cuts(p, block_sum(own, f->red));
        if (tid < RANGES) f->lo[tid] = first + tid < cuts.teams ? cuts.start(first + tid) : -1;
        pads = __syncthreads_or(pad);
        int64_t base = 0;
        for (int z0 = 0; z0 < p.Z; z0 += nt) {
            const int z = z0 + tid;
            if (p.Z > nt) {  // (with at most one sequence a thread its lengths are read once)
                s = z < p.Z ? seq_len(p, z) : SeqLen{0, 0};
                v = p.Hkv * head_blocks<BK>(p, s);
            }
            int64_t x = v;
            for (int d = 1; d < 32; d *= 2) {
                const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += y;
            }
            __syncthreads();
            if (lane == 31) f->red[tid / 32] = x;
            __syncthreads();
            int64_t sum = 0;
            x += base;
            for (int i = 0; i < nt / 32; ++i) {
                if (i < tid / 32) x += f->red[i];
                sum += f->red[i];
            }
#pragma unroll
            for (int r = 0; r < RANGES; ++r)
                if (x - v <= f->lo[r] && f->lo[r] < x) {
                    f->z[r] = z;
                    f->len[r] = s.len;
                    f->nl[r] = s.nl;
                    f->z_before[r] = x - v;
                }
            base += sum;
        }
        __syncthreads();
        if (c < cuts.teams) {
            w.z = f->z[mine];
            w.s = SeqLen{f->len[mine], f->nl[mine]};
            int64_t rem = cuts.start(c) - f->z_before[mine];
            const int64_t per = head_blocks<BK>(p, w.s);
            w.hk = (int)fast_div(rem, per);
            rem -= w.hk * per;
            for (int64_t n; rem >= (n = group_blocks<BK>(p, w.s, w.gi)); ++w.gi) rem -= n;
            w.jb = (int)rem;
            w.left = cuts.start(c + 1) - cuts.start(c);
            w.groups = live_groups(p, w.s);
        }
    }
    // a short group is not cut: the team before has it whole
    if (w.left > 0 && w.jb > 0 && group_blocks<BK>(p, w.s, w.gi) <= p.snap) paged_next<BK>(p, w);
    if (records && c < p.teams)
        static_cast<PagedCut*>(p.cuts)[c] = PagedCut{w.z, w.hk, w.gi, w.jb, w.s.len, w.s.nl, cuts.rem, cuts.teams, cuts.q};
    return w;
}

// The tile of a group that a member takes: in turn from the first and from the
// last, so that the chain's longer later tiles do not all fall to one member (a
// group counts as many blocks as its last tile has: prompts of 1024 tokens, 4 x 16
// heads of D = 128, 49.6 -> 39.3 us).
__device__ __forceinline__ int member_tile(const PagedParams& p, int hk, int gi, int member) {
    return gi * p.team + ((hk + gi) & 1 ? p.team - 1 - member : member);
}

// The next segment of member `member` of a team at or after w's place (worker:
// its number in the launch); false when the range is done.
template <int BK>
__device__ __forceinline__ bool paged_seg(const PagedParams& p, PagedWalk& w, PagedSeg& g, int worker, int member) {
    for (; w.left > 0; paged_next<BK>(p, w)) {
        const int mt = member_tile(p, w.hk, w.gi, member);
        g.row0 = mt * p.tile_rows;
        g.rows = min(p.tile_rows, w.s.nl * p.G - g.row0);
        if (g.rows <= 0) continue;
        const int own = tile_blocks<BK>(p, w.s, mt);
        g.z = w.z;
        g.hk = w.hk;
        g.jb = w.jb;
        const bool whole = own - w.jb <= w.left || group_blocks<BK>(p, w.s, w.gi) <= p.snap;
        g.je = whole ? own : w.jb + (int)w.left;
        if (g.je <= g.jb) continue;
        g.slot = g.jb == 0 && g.je == own ? -1 : 2 * worker + (g.jb > 0 ? 0 : 1);
        g.len = w.s.len;
        g.nl = w.s.nl;
        return true;
    }
    return false;
}

// O = 0 and lse = -inf for the rows of tokens t >= nl: one (sequence, query
// head) pair a warp, the pairs dealt to all warps of the launch (this one is
// number `warp` of `warps`).
template <int D>
__device__ __forceinline__ void paged_fill(const PagedParams& p, int warp, int warps) {
    const int lane = threadIdx.x % 32;
    const int64_t pairs = (int64_t)p.Z * p.Hq;
    for (int64_t i0 = warp; i0 < pairs; i0 += (int64_t)warps * 32) {
        const int64_t i = i0 + (int64_t)warps * lane;
        const int z = i < pairs ? (int)(i / p.Hq) : 0, h = (int)(i - (int64_t)z * p.Hq);
        const int nl = i < pairs ? seq_len(p, z).nl : p.T;
        for (uint32_t todo = __ballot_sync(0xffffffffu, nl < p.T); todo != 0; todo &= todo - 1) {
            const int src = __ffs(todo) - 1;
            const int64_t zz = __shfl_sync(0xffffffffu, z, src), hh = __shfl_sync(0xffffffffu, h, src);
            const int first = __shfl_sync(0xffffffffu, nl, src);
            for (int64_t k = lane; k < (int64_t)(p.T - first) * (D / 8); k += 32) {
                const int t = first + (int)(k / (D / 8)), c = (int)(k % (D / 8));
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + zz * p.so_z + hh * p.so_h + t * p.so_n + 8 * c) =
                    make_uint4(0u, 0u, 0u, 0u);
                if (c == 0 && p.lse != nullptr) p.lse[(zz * p.Hq + hh) * p.T + t] = -INFINITY;
            }
        }
    }
}

__device__ __forceinline__ void record_bad_page(uint32_t* status, uint32_t site) {
    atomicCAS(status + PAGE_WORD, 0u, STATUS_PAGE | (site << 8) | ((blockIdx.x & 0xFFFFu) << 16));
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
    if constexpr (BF16) {
        __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<uint32_t*>(&h);
    } else {
        __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<uint32_t*>(&h);
    }
}

// ------------------------------------------------------------ merge ---------
// Blocks ((b - 1) * team + member) * sub + 0 .. sub - 1 look at the cut between
// the ranges of teams b - 1 and b.  If it falls inside a tile group, the
// member's tile of it has its parts with the teams c0 (slot 2c + 1) and c0 + 1
// .. c1 (slots 2c); the cuts inside the tile are c0 + 1 .. c1, and each of
// their blocks merges one share of the tile's (eight columns, row) items.  A
// part is [D / 8][tile_rows][8] floats of O / l, as both kernels' threads hold
// it, then a log-sum-exp per row; items follow that order, so that a warp's
// loads are contiguous.  With
// lambda_s the base-2 log-sum-exp of part s and O_s its O / l,
//     lambda = log2 sum_s 2^lambda_s,   O = sum_s 2^(lambda_s - lambda) O_s.
// in one pass with a running maximum, so that a part's lambda and its O are one
// round of loads; with few items up to 32 neighbouring lanes share one, split
// the parts and join by shuffles.
// What bounds it is latency: a launch behind the kernel that writes the parts,
// one round of loads for the cut, one or two for the parts, which lie in L2.  It
// takes 4 to 5 us of a call on either kernel (2 MB of parts: one sequence of 1024,
// 128 parts a tile; 14 MB: 8 sequences x 32 tokens).  Blocks a cut, each with a
// share of the tile: one in the rows kernel (two: 10.5 -> 10.7 us for one sequence
// of 1024, 45.7 -> 46.7 for two of 30000), 8 in the tile kernel, whose parts are
// eight times as large (1 / 4 / 8 / 16: 36.1 / 23.6 / 21.7 / 23.0 us for 8 sequences
// x 32 tokens).  Eight columns an item rather than four: half the index arithmetic,
// 23.0 -> 21.7 and 11.1 -> 10.5 us.  The loads of four parts in flight a thread: with
// two, whose 48 registers leave room for a block beside those of the rows kernel,
// 10.5 -> 11.0 and 21.7 -> 22.4, but 97.8 -> 96.2 for 64 sequences of 256-4096.
constexpr int PAGED_MERGE_THREADS = 128;

// Eight floats, a whole sector, through L2.
__device__ __forceinline__ void ld_part(const float* from, float (&v)[8]) {
    asm volatile("ld.global.cg.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "l"(from)
                 : "memory");
}

template <int D, int BK, bool BF16>
__global__ void __launch_bounds__(PAGED_MERGE_THREADS) fa_paged_merge_kernel(const PagedParams p, int sub) {
    constexpr int W = D / 8, NT = PAGED_MERGE_THREADS;
    // (no early launch of the next kernel: its set-up would take issue slots from the merge, 187 against
    // 194 us for 32 sequences x 64 drafted tokens)
    ptx::grid_dependency_wait();
    const int tid = threadIdx.x;
    const int member = (int)(blockIdx.x / sub) % p.team;
    // One warp works out the block's share for all (the arithmetic in every warp took
    // longer than the loads): {first and last item, parts, z, kv head, row0, first slot}.
    __shared__ int what[8];
    if (tid < 32) {
        const int b = 1 + (int)blockIdx.x / (p.team * sub);
        const int4* rec = reinterpret_cast<const int4*>(static_cast<const PagedCut*>(p.cuts) + b);
        const int4 cut = __ldcg(rec), more = __ldcg(rec + 1);
        const PagedCuts cuts{__ldcg(reinterpret_cast<const long long*>(rec + 2)), more.z, more.w};
        int first = 0, last = 0, parts = 0, c0 = 0;
        const int mt = member_tile(p, cut.y, cut.z, member), row0 = mt * p.tile_rows;
        const SeqLen s{more.x, more.y};
        const int live = cut.x < 0 ? 0 : min(p.tile_rows, s.nl * p.G - row0);
        if (live > 0 && cut.w > 0) {  // there is such a range, and it does not start with a tile
            const int64_t t0 = cuts.start(b) - cut.w, t1 = t0 + tile_blocks<BK>(p, s, mt) - 1;
            c0 = cuts.team_of(t0);
            const int c1 = cuts.team_of(t1);
            if (b <= c1) {  // (else the cut is behind this tile's last block)
                parts = c1 - c0 + 1;
                // as many of the cut's blocks as leave a thread about four loads
                const int cuts_in = c1 - c0, loads = cuts_in * NT * 4;
                const int use = min(sub, (live * W * parts + loads - 1) / loads);
                const int mine = (int)blockIdx.x % sub, shares = cuts_in * use, share = (live * W + shares - 1) / shares;
                if (mine < use) {
                    first = ((b - 1 - c0) * use + mine) * share;
                    last = min(first + share, live * W);
                }
            }
        }
        if (tid == 0) {
            what[0] = first, what[1] = last, what[2] = parts, what[3] = cut.x, what[4] = cut.y, what[5] = row0;
            what[6] = 2 * (c0 * p.team + member), what[7] = live;
        }
    }
    __syncthreads();
    const int first = what[0], last = what[1], parts = what[2];
    if (first >= last) return;
    const int z = what[3], hk = what[4], row0 = what[5], live = what[7];
    // the first part is in slot 2 c + 1 of its worker, the others in slots 2 c: offsets in
    // floats, below 2^32 (two slots a worker, at most 1280 x 33 KB or 152 x 132 KB each)
    const float* base = p.scratch + (int64_t)what[6] * p.slot_floats;
    const uint32_t slot0 = (uint32_t)p.slot_floats, step = 2u * (uint32_t)p.team * slot0, lses = (uint32_t)(p.tile_rows * D);
    int spl = 1;
    while (spl < 32 && spl < parts && (last - first) * spl * 2 <= NT) spl *= 2;
    const int sl = tid % spl;
    for (int i0 = first; i0 < last; i0 += NT / spl) {
        const int i = i0 + tid / spl;
        const bool ok = i < last;
        // items: eight-column groups, in each the live rows
        const int kg = ok ? i / live : 0, r = ok ? i - kg * live : 0, at = (kg * p.tile_rows + r) * 8;
        float mx = -INFINITY, den = 0.f, acc[8];
#pragma unroll
        for (int y = 0; y < 8; ++y) acc[y] = 0.f;
        constexpr int U = 4;
        for (int x0 = sl; ok && x0 < parts; x0 += U * spl) {
            float l[U], v[U][8];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                l[u] = -INFINITY;
#pragma unroll
                for (int y = 0; y < 8; ++y) v[u][y] = 0.f;
                const int x = x0 + u * spl;
                if (x < parts) {
                    const float* from = base + (x == 0 ? slot0 : (uint32_t)x * step);
                    ld_part(from + at, v[u]);
                    l[u] = __ldcg(from + lses + r);
                }
            }
            float top = mx;
#pragma unroll
            for (int u = 0; u < U; ++u) top = fmaxf(top, l[u]);
            const float a = mx == -INFINITY ? 0.f : ptx::ex2(mx - top);
            mx = top;
            den *= a;
#pragma unroll
            for (int y = 0; y < 8; ++y) acc[y] *= a;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float w = l[u] == -INFINITY ? 0.f : ptx::ex2(l[u] - top);
                den += w;
#pragma unroll
                for (int y = 0; y < 8; ++y) acc[y] += w * v[u][y];
            }
        }
        for (int k = spl / 2; k > 0; k /= 2) {
            const float other = __shfl_xor_sync(0xffffffffu, mx, k), top = fmaxf(mx, other);
            const float a = mx == -INFINITY ? 0.f : ptx::ex2(mx - top);
            mx = top;
            den *= a;
            den += __shfl_xor_sync(0xffffffffu, den, k);
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                acc[y] *= a;
                acc[y] += __shfl_xor_sync(0xffffffffu, acc[y], k);
            }
        }
        if (!ok || sl != 0) continue;
        const int row = row0 + r, t = p.by_g(row), h = hk * p.G + row - t * p.G;
        const float inv = den == 0.f ? 0.f : 1.f / den;  // (a NaN score reaches O)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + (int64_t)z * p.so_z + h * p.so_h + t * p.so_n + 8 * kg) =
            make_uint4(pack_pair<BF16>(acc[0] * inv, acc[1] * inv), pack_pair<BF16>(acc[2] * inv, acc[3] * inv),
                       pack_pair<BF16>(acc[4] * inv, acc[5] * inv), pack_pair<BF16>(acc[6] * inv, acc[7] * inv));
        if (kg == 0 && p.lse != nullptr)
            p.lse[((int64_t)z * p.Hq + h) * p.T + t] = den == 0.f ? -INFINITY : (mx + log2f(den)) * 0.6931471805599453f;
    }
}

}  // namespace fa
