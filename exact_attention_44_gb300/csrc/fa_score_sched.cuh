// Work division of the received-weight kernels, on the device, where the lengths are:
// the steps of all sequences, laid end to end, are cut into one equal range a worker.
#pragma once

#include "fa_cache.cuh"
#include "fa_score.h"

namespace fa {

// Positions before the new tokens and new tokens of a sequence, clamped to what its
// block table can hold.
struct ScoreLen {
    int len, nl;
};
__device__ __forceinline__ ScoreLen score_len(const ScoreParams& p, int z) {
    const int n = ldi(p.lens + z), m = p.news != nullptr ? ldi(p.news + z) : p.T;
    ScoreLen s;
    s.len = min(max(n, 0), p.cap);
    s.nl = min(max(m, 0), min(p.T, p.cap - s.len));
    return s;
}

// Where a worker's range starts: step `at` of sequence z, `left` steps in all (0: none).
struct ScorePlace {
    int z;
    ScoreLen s;
    int64_t at, left;
};

template <int RANGES>
struct ScoreFind {
    int64_t red[32], lo[RANGES], at[RANGES];
    int z[RANGES], len[RANGES], nl[RANGES];
};

// The place of range first + mine of `ranges` (RANGES of them a CTA, mine the same in
// all threads of a warp).  count(s): steps of a sequence.  Called by every thread of
// the CTA; with up to 32 sequences the warps need not all call it.  *start: the first
// step of the range, *all: the steps of all sequences.
template <int RANGES, typename Count>
__device__ __forceinline__ ScorePlace score_place(const ScoreParams& p, ScoreFind<RANGES>* f, int first, int mine,
                                                  int ranges, Count count, int64_t* start = nullptr,
                                                  int64_t* all = nullptr) {
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid % 32, c = first + mine;
    ScorePlace w{0, {0, 0}, 0, 0};
    auto cut = [&](int64_t total, int i, int64_t& lo, int64_t& n) {
        // total / ranges steps each, one more for the first of them
        const bool small = (uint64_t)total >> 32 == 0;
        const int64_t q = small ? (int64_t)((uint32_t)total / (uint32_t)ranges) : total / ranges;
        const int64_t rem = total - q * ranges;
        lo = q * i + (i < rem ? i : rem);
        n = i < ranges ? q + (i < rem) : 0;
    };
    auto report = [&](int64_t lo, int64_t total) {
        if (start != nullptr) {
            *start = lo;
            *all = total;
        }
    };
    if (p.Z <= 32) {  // each warp by itself, one sequence a lane
        ScoreLen s{0, 0};
        int64_t v = 0;
        if (lane < p.Z) {
            s = score_len(p, lane);
            v = count(s);
        }
        int64_t x = v;
        for (int d = 1; d < 32; d *= 2) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        int64_t lo;
        const int64_t total = __shfl_sync(0xffffffffu, x, 31);
        cut(total, c, lo, w.left);
        report(lo, total);
        if (w.left > 0) {
            w.z = __ffs(__ballot_sync(0xffffffffu, lo < x)) - 1;
            w.at = lo - __shfl_sync(0xffffffffu, x - v, w.z);
            w.s = ScoreLen{__shfl_sync(0xffffffffu, s.len, w.z), __shfl_sync(0xffffffffu, s.nl, w.z)};
        }
        return w;
    }
    int64_t own = 0;
    for (int z = tid; z < p.Z; z += nt) own += count(score_len(p, z));
    for (int d = 16; d > 0; d /= 2) own += __shfl_xor_sync(0xffffffffu, own, d);
    if (lane == 0) f->red[tid / 32] = own;
    __syncthreads();
    int64_t total = 0, lo;
    for (int i = 0; i < nt / 32; ++i) total += f->red[i];
    cut(total, c, lo, w.left);
    report(lo, total);
    if (tid < RANGES) {
        int64_t l, n;
        cut(total, first + tid, l, n);
        f->lo[tid] = n > 0 ? l : -1;
    }
    int64_t base = 0;
    for (int z0 = 0; z0 < p.Z; z0 += nt) {
        const int z = z0 + tid;
        const ScoreLen s = z < p.Z ? score_len(p, z) : ScoreLen{0, 0};
        const int64_t v = z < p.Z ? count(s) : 0;
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
                f->at[r] = f->lo[r] - (x - v);
            }
        base += sum;
    }
    __syncthreads();
    if (w.left > 0) {
        w.z = f->z[mine];
        w.s = ScoreLen{f->len[mine], f->nl[mine]};
        w.at = f->at[mine];
    }
    return w;
}

}  // namespace fa
