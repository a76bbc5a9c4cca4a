// The weight that cached positions receive from few query rows:
//     score_j = decay score_j + sum over rows i that see j of exp(q_i k_j scale - lse_i).
//
// What bounds it is reading K once (2 D bytes a position and kv head), so the work is
// organised around loads in flight.  A warp takes an equal range of the launch's steps
// of KT positions and holds K in registers: the products run on mma.sync m16n8k16 with
// K as A -- 16 positions -- and the query rows as B, and since a product does not care
// in which order its D terms are taken, a thread's share of A's columns can be any as
// long as B's is the same: 16 contiguous bytes of its two rows, which it loads straight
// from the cache.  Nothing goes through shared memory.  A position's weights lie in
// four neighbouring lanes and are summed there, in fp32.  Rows that do not fit in registers
// (more than 32, groups wider than a tile) are loaded again for every step: right for any
// number, but slow for many (512 tokens of 136 heads after 1000 positions, one kv head, D =
// 128: 1.7 ms, against 33 us for 128 heads on the tile kernel).
//
// What hides the way to memory is the number of warps: one step of K in 32 registers, 20
// warps an SM for up to 8 rows.  Measured: 64 sequences of 256-4096 positions, one token,
// 32 query heads on 8 of D = 128 (294 MB with the scores): 51 to 52 us repeated in a graph,
// 52 to 53 called on new inputs, 5.6 to 5.8 TB/s (8000-12000: 214 us, 6.3 TB/s); with two steps
// in registers and 16 warps 54 in a graph, with 12 warps an SM 61, 28 (72 registers, spilled)
// 65.  One sequence of 1024: 2.9 to 3.1 us in a graph.  A sequence without a new token is no
// work with decay 1, else a read and a write of its scores: 64 of 2000, half of them idle, 25 and
// 35 us, none 48.
#pragma once

#include "fa_ptx.cuh"
#include "fa_score_sched.cuh"

namespace fa {

constexpr int SCORE_WARPS = 4;  // a CTA

template <int D_>
struct ScoreRows {
    static constexpr int D = D_;
    static constexpr int U = D >= 128 ? 1 : 128 / D;   // groups of 16 positions a step
    static constexpr int KT = 16 * U;
    static constexpr int PW = D >= 32 ? 4 : 2;         // words a thread loads of a row at a time
    static constexpr int NP = D / (8 * PW);            // such pieces of a row
    static constexpr int ctas(int nt) { return D == 256 || (D == 128 && nt == 4) ? 3 : nt == 1 ? 5 : 4; }  // an SM
};

namespace score {

template <bool BF16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    if constexpr (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// PW words of a row from `from`.
template <int PW>
__device__ __forceinline__ void load_piece(const uint16_t* from, uint32_t* w) {
    if constexpr (PW == 4) {
        const uint4 x = __ldcg(reinterpret_cast<const uint4*>(from));
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    } else {
        const uint2 x = __ldcg(reinterpret_cast<const uint2*>(from));
        w[0] = x.x, w[1] = x.y;
    }
}

// A step: KT positions of a kv head.
struct Step {
    int z, hk, j;   // j: which KT positions
    ScoreLen s;
};

// What a warp holds of a step's K: rows lane / 4 and lane / 4 + 8 of each group, and the
// scores so far of the positions that its lane writes.
template <int D>
struct Keys {
    using T = ScoreRows<D>;
    uint32_t w[T::U][2][T::NP][T::PW];
    float old[T::U];
};

}  // namespace score

template <int D, bool BF16, int NT>
__global__ void __launch_bounds__(32 * SCORE_WARPS, ScoreRows<D>::ctas(NT)) fa_score_rows_kernel(const ScoreParams p) {
    using T = ScoreRows<D>;
    using namespace score;
    __shared__ ScoreFind<SCORE_WARPS> find;
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, c = lane % 4;
    // (without a new token K has no say, and with decay 1 the scores stay as they are)
    auto steps = [&](const ScoreLen& s) { return s.nl == 0 && p.decay == 1.f ? 0 : (s.len + s.nl + T::KT - 1) / T::KT; };
    const ScorePlace place = score_place<SCORE_WARPS>(p, &find, blockIdx.x * SCORE_WARPS, warp, p.workers,
                                                      [&](const ScoreLen& s) { return (int64_t)steps(s) * p.Hkv; });
    int64_t left = place.left;
    if (left == 0) return;

    Step cur{place.z, 0, 0, place.s};
    cur.hk = (int)(place.at / steps(place.s));
    cur.j = (int)(place.at - (int64_t)cur.hk * steps(place.s));
    auto advance = [&](Step& x) {
        if (++x.j < steps(x.s)) return;
        x.j = 0;
        if (++x.hk < p.Hkv) return;
        x.hk = 0;
        do {
            if (++x.z >= p.Z) return;
            x.s = score_len(p, x.z);
        } while (steps(x.s) == 0);
    };
    // lane u's table entry of group u of a step
    auto ask = [&](const Step& x) -> int {
        const int pos = x.j * T::KT + lane * 16;
        return lane < T::U && x.s.nl > 0 && pos < x.s.len + x.s.nl ? ldi(p.table + x.z * p.st_z + p.by_page(pos)) : 0;
    };
    auto load = [&](const Step& x, int entries, Keys<D>& k) {
        const int end = x.s.len + x.s.nl;
#pragma unroll
        for (int u = 0; u < T::U; ++u) {
            const int e = __shfl_sync(0xffffffffu, entries, u), pos = x.j * T::KT + u * 16;
            const bool asked = x.s.nl > 0 && pos < end, there = asked && (unsigned)e < (unsigned)p.P;
            if (asked && !there && lane == 0) bad_page(p.status, SITE_PAGE_SCORE);
            const int slot = pos - p.by_page(pos) * p.page;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int r = g + 8 * y;
                const uint16_t* row = p.k + e * p.sk_p + x.hk * p.sk_h + (slot + r) * p.sk_n + c * 2 * T::PW;
#pragma unroll
                for (int i = 0; i < T::NP; ++i) {
#pragma unroll
                    for (int w = 0; w < T::PW; ++w) k.w[u][y][i][w] = 0u;
                    if (there && pos + r < end) load_piece<T::PW>(row + i * 8 * T::PW, k.w[u][y][i]);
                }
            }
            const int mine = pos + g + 8 * (c & 1);
            k.old[u] = 0.f;
            if (p.decay != 0.f && c < 2 && mine < x.s.len)
                k.old[u] = __ldcg(p.scores + x.z * p.ss_z + x.hk * p.ss_h + mine) * p.decay;
        }
    };

    // Query rows r0 .. r0 + 8 NT - 1 of the step's group, a row a (token, head) pair with
    // the heads innermost: their elements as B, and for this lane's two columns of each 8
    // their lse and the last position that they see (-1: nothing).
    uint32_t q[NT][T::NP][T::PW];
    float lse[NT][2];
    int last[NT][2];
    auto load_q = [&](const Step& x, int r0) {
        const int rows = x.s.nl * p.G;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = r0 + 8 * n + g, t = p.by_g(r), h = x.hk * p.G + r - t * p.G;
            const uint16_t* row = p.q + x.z * p.sq_z + h * p.sq_h + t * p.sq_n + c * 2 * T::PW;
#pragma unroll
            for (int i = 0; i < T::NP; ++i) {
#pragma unroll
                for (int w = 0; w < T::PW; ++w) q[n][i][w] = 0u;
                if (r < rows) load_piece<T::PW>(row + i * 8 * T::PW, q[n][i]);
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int rc = r0 + 8 * n + 2 * c + y, tc = p.by_g(rc), hc = x.hk * p.G + rc - tc * p.G;
                lse[n][y] = -INFINITY;
                if (rc < rows) lse[n][y] = __ldcg(p.lse + ((int64_t)x.z * p.Hq + hc) * p.T + tc);
                last[n][y] = lse[n][y] == -INFINITY ? -1 : x.s.len + tc;
            }
        }
    };
    int q_z = -1, q_hk = -1;

    auto use = [&](const Step& x, const Keys<D>& k) {
        float sum[T::U][2];
#pragma unroll
        for (int u = 0; u < T::U; ++u) sum[u][0] = sum[u][1] = 0.f;
        const int rows = x.s.nl * p.G;
        const bool once = rows <= 8 * NT;
        for (int r0 = 0; r0 < rows; r0 += 8 * NT) {
            if (!once || q_z != x.z || q_hk != x.hk) load_q(x, r0);
#pragma unroll
            for (int u = 0; u < T::U; ++u) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < T::NP; ++i)
#pragma unroll
                        for (int w = 0; w < T::PW; w += 2)
                            mma<BF16>(d, k.w[u][0][i][w], k.w[u][1][i][w], k.w[u][0][i][w + 1], k.w[u][1][i][w + 1],
                                      q[n][i][w], q[n][i][w + 1]);
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const int pos = x.j * T::KT + u * 16 + g + 8 * (y / 2);
                        const float e = ptx::ex2(fmaf(d[y], p.scale, -lse[n][y & 1]) * 1.4426950408889634f);
                        sum[u][y / 2] += pos <= last[n][y & 1] ? e : 0.f;
                    }
                }
            }
        }
        q_z = once ? x.z : -1;
        q_hk = x.hk;
#pragma unroll
        for (int u = 0; u < T::U; ++u) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                sum[u][y] += __shfl_xor_sync(0xffffffffu, sum[u][y], 1);
                sum[u][y] += __shfl_xor_sync(0xffffffffu, sum[u][y], 2);
            }
            const int mine = x.j * T::KT + u * 16 + g + 8 * (c & 1);
            if (c < 2 && mine < x.s.len + x.s.nl)
                p.scores[x.z * p.ss_z + x.hk * p.ss_h + mine] = k.old[u] + (c == 0 ? sum[u][0] : sum[u][1]);
        }
    };

    // table entries a step ahead
    int entries = ask(cur);
    Keys<D> k;
    for (; left > 0; --left) {
        load(cur, entries, k);
        Step next = cur;
        if (left > 1) {
            advance(next);
            entries = ask(next);
        }
        use(cur, k);
        cur = next;
    }
}

}  // namespace fa
