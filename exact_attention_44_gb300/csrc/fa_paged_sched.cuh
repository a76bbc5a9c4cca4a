// Work division of the paged attention kernels, computed on the device: the
// lengths live there, and a call reads nothing back.
//
// A tile is up to p.tile_rows query rows of one (sequence, kv head); a row is
// a (new token, query head of the group) pair with the heads innermost, so
// that the rows of a sequence with fewer new tokens than T are a prefix and
// the K/V rows are read once for the whole group.  The (tile, key block)
// pairs, in the order sequence, kv head, tile, block, are laid end to end and
// cut into one equal range per CTA, whatever the lengths are; a tile that a cut
// crosses leaves partial results (O / l in fp32 and the base-2 log-sum-exp) in
// slots of the workspace, two per CTA, and fa_paged_merge_kernel joins them in
// the order of the keys.  Nothing depends on timing: the same inputs give the
// same bits.
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
        end = s.len + last / p.G + 1;
    }
    return (end + BK - 1) / BK;
}
__device__ __forceinline__ int live_tiles(const PagedParams& p, const SeqLen& s) {
    return (s.nl * p.G + p.tile_rows - 1) / p.tile_rows;
}
// blocks of one (sequence, kv head), of tiles 0 .. mt - 1
template <int BK>
__device__ __forceinline__ int64_t head_blocks_before(const PagedParams& p, const SeqLen& s, int mt) {
    if (s.nl == 0) return 0;
    if (p.mask != nullptr) return (int64_t)mt * tile_blocks<BK>(p, s, 0);
    int64_t n = 0;
    for (int m = 0; m < mt; ++m) n += tile_blocks<BK>(p, s, m);
    return n;
}
template <int BK>
__device__ __forceinline__ int64_t seq_blocks(const PagedParams& p, int z) {
    const SeqLen s = seq_len(p, z);
    return p.Hkv * head_blocks_before<BK>(p, s, live_tiles(p, s));
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

// A CTA's place in the order: the segments of its range, one after another.
struct PagedWalk {
    int z, hk, mt;   // tile
    int jb;          // its first block in this range
    int64_t left;    // blocks left in the range
};
struct PagedSeg {
    int z, hk, mt;
    int jb, je;      // key blocks
    int slot;        // -1: the whole tile; else where its part goes
    int len, nl;
    int row0, rows;  // first query row of the tile and its live rows
};

struct PagedFind {
    int64_t red[32];
    int64_t z_before;  // blocks before sequence z
    int z;
};

// Every thread of the CTA: total blocks, and the start of CTA c's range.
template <int BK>
__device__ __forceinline__ PagedWalk paged_range(const PagedParams& p, int c, int grid, PagedFind* f) {
    const int tid = threadIdx.x, nt = blockDim.x;
    int64_t own = 0;
    for (int z = tid; z < p.Z; z += nt) own += seq_blocks<BK>(p, z);
    const int64_t total = block_sum(own, f->red);
    PagedWalk w{p.Z, 0, 0, 0, 0};
    if (total < grid) grid = (int)total;  // no empty ranges between the others: the merge reads each one's slot
    if (c >= grid) return w;              // the same answer in every thread
    const int64_t lo = total * c / grid, hi = total * (c + 1) / grid;
    int64_t base = 0;
    for (int z0 = 0; z0 < p.Z; z0 += nt) {
        const int z = z0 + tid;
        const int64_t v = z < p.Z ? seq_blocks<BK>(p, z) : 0;
        int64_t x = v;
        for (int d = 1; d < 32; d *= 2) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
            if (tid % 32 >= d) x += y;
        }
        __syncthreads();
        if (tid % 32 == 31) f->red[tid / 32] = x;
        if (tid == 0) f->z = -1;
        __syncthreads();
        int64_t before = base, sum = 0;
        for (int i = 0; i < nt / 32; ++i) {
            if (i < tid / 32) before += f->red[i];
            sum += f->red[i];
        }
        x += before;
        if (x - v <= lo && lo < x) {
            f->z = z;
            f->z_before = x - v;
        }
        __syncthreads();
        if (f->z >= 0) break;
        base += sum;
    }
    w.z = f->z;
    int64_t rem = lo - f->z_before;
    const SeqLen s = seq_len(p, w.z);
    const int64_t per = head_blocks_before<BK>(p, s, live_tiles(p, s));
    w.hk = (int)(rem / per);
    rem -= w.hk * per;
    w.mt = 0;
    for (int64_t n; rem >= (n = tile_blocks<BK>(p, s, w.mt)); ++w.mt) rem -= n;
    w.jb = (int)rem;
    w.left = hi - lo;
    return w;
}

template <int BK>
__device__ __forceinline__ PagedSeg paged_seg(const PagedParams& p, const PagedWalk& w) {
    PagedSeg g;
    const SeqLen s = seq_len(p, w.z);
    const int n = tile_blocks<BK>(p, s, w.mt);
    g.z = w.z;
    g.hk = w.hk;
    g.mt = w.mt;
    g.jb = w.jb;
    g.je = n - w.jb <= w.left ? n : w.jb + (int)w.left;
    g.slot = g.jb == 0 && g.je == n ? -1 : 2 * (int)blockIdx.x + (g.jb > 0 ? 0 : 1);
    g.len = s.len;
    g.nl = s.nl;
    g.row0 = w.mt * p.tile_rows;
    g.rows = min(p.tile_rows, s.nl * p.G - g.row0);
    return g;
}

// On to the next segment (sequences without new tokens have no tiles).
__device__ __forceinline__ void paged_next(const PagedParams& p, const PagedSeg& g, PagedWalk& w) {
    w.left -= g.je - g.jb;
    w.jb = 0;
    if (w.left <= 0) return;
    if (++w.mt * p.tile_rows < g.nl * p.G) return;
    w.mt = 0;
    if (++w.hk < p.Hkv) return;
    w.hk = 0;
    for (++w.z; w.z < p.Z && seq_len(p, w.z).nl == 0; ++w.z) {
    }
    if (w.z >= p.Z) w.left = 0;
}

__device__ __forceinline__ void record_bad_page(uint32_t* status, uint32_t site) {
    atomicCAS(status, 0u, STATUS_PAGE | (site << 8) | ((blockIdx.x & 0xFFFFu) << 16));
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
// `slices` blocks per (sequence, kv head, tile), each a share of its rows.  A tile that the cuts crossed has
// its parts in slots 2 c0 + 1 (the CTA c0 of its first block) and 2 c (CTAs
// c0 + 1 .. c1); with lambda_s the base-2 log-sum-exp of part s and O_s its O / l,
//     lambda = log2 sum_s 2^lambda_s,   O = sum_s 2^(lambda_s - lambda) O_s,
// taken in one pass with a running maximum.  Rows of new tokens that the
// sequence does not have get O = 0 and lse = -inf.  A thread takes four
// columns of a row; with few rows several threads share them and split the
// parts, and join through shared memory.  COLS: a slot holds float4 column
// groups [D / 4][128] (the tile kernel's threads each own a row), else rows
// [tile_rows][D].
constexpr int PAGED_MERGE_THREADS = 512;

template <int D, int BK, bool BF16, bool COLS>
__global__ void __launch_bounds__(PAGED_MERGE_THREADS) fa_paged_merge_kernel(const PagedParams p, int grid, int slices) {
    __shared__ int64_t red[32];
    __shared__ float sh[PAGED_MERGE_THREADS * 6];
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int tid = threadIdx.x;
    const int per_z = p.Hkv * p.tiles;
    const int tile = blockIdx.x / slices, slice = blockIdx.x - tile * slices;
    const int z = tile / per_z, r = tile - z * per_z;
    const int hk = r / p.tiles, mt = r - hk * p.tiles;
    const SeqLen s = seq_len(p, z);
    const int row0 = mt * p.tile_rows;
    // this block's rows of the tile, the live ones first
    const int share = (p.tile_rows + slices - 1) / slices, lo = slice * share, hi = min(lo + share, p.tile_rows);
    const int live = min(hi, s.nl * p.G - row0);
    const int rows = live - lo;  // may be <= 0
    constexpr int W = D / 4;
    auto row_at = [&](int row, int64_t& lse_at, int64_t& o_at) {  // row of the (sequence, kv head)
        const int t = row / p.G, h = hk * p.G + row - t * p.G;
        lse_at = ((int64_t)z * p.Hq + h) * p.T + t;
        o_at = (int64_t)z * p.so_z + h * p.so_h + t * p.so_n;
    };
    // rows without a token
    {
        const int first = max(live, lo), last = min(hi, p.T * p.G - row0);
        for (int i = first * W + tid; i < last * W; i += PAGED_MERGE_THREADS) {
            const int row = i / W, c = i - row * W;
            int64_t la, oa;
            row_at(row0 + row, la, oa);
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + oa + 4 * c) = make_uint2(0u, 0u);
            if (c == 0 && p.lse != nullptr) p.lse[la] = -INFINITY;
        }
    }
    if (rows <= 0) return;
    int64_t before = 0, all = 0;
    for (int i = tid; i < p.Z; i += PAGED_MERGE_THREADS) {
        const int64_t n = seq_blocks<BK>(p, i);
        all += n;
        if (i < z) before += n;
    }
    const int64_t total = block_sum(all, red);
    if (total < grid) grid = (int)total;
    const int64_t per = head_blocks_before<BK>(p, s, live_tiles(p, s));
    const int64_t t0 = block_sum(before, red) + hk * per + head_blocks_before<BK>(p, s, mt);
    const int64_t t1 = t0 + tile_blocks<BK>(p, s, mt) - 1;
    // the CTA whose range [total c / grid, total (c + 1) / grid) holds position x
    const int c0 = (int)(((t0 + 1) * grid + total - 1) / total - 1);
    const int c1 = (int)(((t1 + 1) * grid + total - 1) / total - 1);
    if (c0 == c1) return;  // the whole tile went straight to O
    const int items = rows * W;
    int spl = 1;
    while (spl < 32 && items * spl * 2 <= PAGED_MERGE_THREADS) spl *= 2;
    const int per_round = PAGED_MERGE_THREADS / spl;
    const int g = tid / per_round;  // this thread's share of the parts
    for (int i0 = 0; i0 < items; i0 += per_round) {
        const int i = i0 + tid - g * per_round;
        const bool ok = g < spl && i < items;
        const int row = !ok ? 0 : lo + (COLS ? i % rows : i / W), c = !ok ? 0 : COLS ? i / rows : i % W;
        float mx = -INFINITY, den = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (ok) {
#pragma unroll 4
            for (int x = c0 + g; x <= c1; x += spl) {
                const float* slot = p.scratch + (int64_t)(x == c0 ? 2 * x + 1 : 2 * x) * p.slot_floats;
                const float l = __ldcg(slot + (COLS ? 128 : p.tile_rows) * D + row);
                const float4 v = __ldcg(reinterpret_cast<const float4*>(slot) + (COLS ? c * 128 + row : row * W + c));
                const float top = fmaxf(mx, l);
                const float a = mx == -INFINITY ? 0.f : exp2f(mx - top), b = l == -INFINITY ? 0.f : exp2f(l - top);
                mx = top;
                den = den * a + b;
                acc.x = acc.x * a + b * v.x;
                acc.y = acc.y * a + b * v.y;
                acc.z = acc.z * a + b * v.z;
                acc.w = acc.w * a + b * v.w;
            }
        }
        if (spl > 1) {
            __syncthreads();
            float* m = sh + tid;
            m[0] = mx;
            m[PAGED_MERGE_THREADS] = den;
            m[2 * PAGED_MERGE_THREADS] = acc.x;
            m[3 * PAGED_MERGE_THREADS] = acc.y;
            m[4 * PAGED_MERGE_THREADS] = acc.z;
            m[5 * PAGED_MERGE_THREADS] = acc.w;
            __syncthreads();
            if (g == 0 && ok) {
                for (int k = 1; k < spl; ++k) {
                    const float* n = sh + tid + k * per_round;
                    const float top = fmaxf(mx, n[0]);
                    const float a = mx == -INFINITY ? 0.f : exp2f(mx - top), b = n[0] == -INFINITY ? 0.f : exp2f(n[0] - top);
                    mx = top;
                    den = den * a + b * n[PAGED_MERGE_THREADS];
                    acc.x = acc.x * a + b * n[2 * PAGED_MERGE_THREADS];
                    acc.y = acc.y * a + b * n[3 * PAGED_MERGE_THREADS];
                    acc.z = acc.z * a + b * n[4 * PAGED_MERGE_THREADS];
                    acc.w = acc.w * a + b * n[5 * PAGED_MERGE_THREADS];
                }
            }
        }
        if (!ok || g != 0) continue;
        int64_t la, oa;
        row_at(row0 + row, la, oa);
        const float inv = den == 0.f ? 0.f : 1.f / den;  // a NaN score reaches O
        uint2 out;
        out.x = pack_pair<BF16>(acc.x * inv, acc.y * inv);
        out.y = pack_pair<BF16>(acc.z * inv, acc.w * inv);
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + oa + 4 * c) = out;
        if (c == 0 && p.lse != nullptr) p.lse[la] = den == 0.f ? -INFINITY : (mx + log2f(den)) * 0.6931471805599453f;
    }
}

}  // namespace fa
