// Attention over a paged cache for few query rows (a decode step, a small
// tree): O = softmax(Q Kᵀ · scale) V for up to RT rows of one (sequence, kv
// head) -- the new tokens of the sequence times the query heads that share the
// kv head -- against all of its cached positions.
//
// What bounds it is reading K and V once: with R rows a position costs
// 4 D R multiply-adds' flops for 4 D bytes, far below what the tensor cores
// could do.  So the work is organised around loads in flight, not around the
// products:
//   * four warps a CTA, each with its own ring of NST 16-position stages of K
//     and V in shared memory, filled by its own 16-byte cp.async copies through
//     the block table; no barrier between warps in the loop, so a late page
//     holds up one warp only;
//   * the products run on mma.sync m16n8k16: a tile of 16 or 32 rows is far
//     too small for a 128-row tcgen05 tile (see fa_paged_tile_kernel.cuh for
//     the calls with many rows), and S, P and O stay in registers;
//   * warps take the 16-position tiles of a segment in turn, keep a running
//     maximum and sum of their own, and join once at the end of the segment.
// Positions past the sequence's end are never read: their copies have source
// size 0, which fills zeros, so whatever a page holds behind the last token
// (NaN included) has no effect.
#pragma once

#include "fa_paged_sched.cuh"

namespace fa {

constexpr int ROWS_WARPS = 4;
constexpr int ROWS_BK = 16 * ROWS_WARPS;  // positions per key block of the schedule

template <int D_, int RT_>
struct RowsTraits {
    static constexpr int D = D_, RT = RT_;
    static constexpr int CTAS = D <= 128 ? 2 : 1;  // per SM
    static constexpr int CPR = D / 8;                    // 16-byte chunks per row
    static constexpr int HALF = 16 * D * 2;              // bytes of 16 rows of K (or V)
    static constexpr int NST = D >= 128 ? 3 : D == 64 ? 6 : 8;
    static constexpr int RING = NST * 2 * HALF;          // per warp
    static constexpr int OFF_Q = ROWS_WARPS * RING;
    static constexpr int OFF_ML = OFF_Q + RT * D * 2;
    static constexpr int OFF_FIND = OFF_ML + 2 * ROWS_WARPS * RT * 4;
    static constexpr int SMEM = OFF_FIND + (int)sizeof(PagedFind);
    static_assert(RT * D * 4 <= RING, "a warp's O fits its ring");
    static_assert(SMEM * CTAS <= 227 * 1024 - CTAS * 1024, "shared memory budget");
    static_assert(OFF_FIND % 8 == 0, "alignment");
};

namespace rowsk {

// 16-byte chunk c of row r of a [rows][D] 16-bit tile: chunks are permuted so
// that eight consecutive rows of one chunk lie in different bank groups.
template <int D>
__device__ __forceinline__ uint32_t swz(int r, int c) {
    constexpr int CPR = D / 8;
    if constexpr (CPR >= 8) return (uint32_t)(r * CPR + (c ^ (r & 7))) * 16u;
    else if constexpr (CPR == 4) return (uint32_t)(r * CPR + (c ^ ((r >> 1) & 3))) * 16u;
    else return (uint32_t)(r * CPR + (c ^ ((r >> 2) & 1))) * 16u;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A running maximum may lag behind the largest score by this much (log2
// units) before O and l are rescaled: probabilities stay <= 2^8, exact in
// fp16 and bf16 range, and O / l and lse do not depend on the reference.
constexpr float LAG = 8.0f;

}  // namespace rowsk

template <int D, int RT, bool BF16>
__global__ void __launch_bounds__(32 * ROWS_WARPS, RowsTraits<D, RT>::CTAS)
    fa_paged_rows_kernel(const PagedParams p) {
    using T = RowsTraits<D, RT>;
    using namespace rowsk;
    constexpr int MT = RT / 16;                 // 16-row groups
    constexpr int KS = D / 16;                  // 16-wide steps along the head dim
    constexpr bool QREG = RT == 16 && D <= 128; // Q fragments stay in registers
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sbase = ptx::smem_addr(smem);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    float* ml = reinterpret_cast<float*>(smem + T::OFF_ML);  // [2][warps][RT]: m, l
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();

    const uint32_t ring = sbase + warp * T::RING;
    const uint16_t* kc = static_cast<const uint16_t*>(p.kc);
    const uint16_t* vc = static_cast<const uint16_t*>(p.vc);
    PagedWalk walk = paged_range<ROWS_BK>(p, blockIdx.x, gridDim.x, reinterpret_cast<PagedFind*>(smem + T::OFF_FIND));

    while (walk.left > 0) {
        const PagedSeg sg = paged_seg<ROWS_BK>(p, walk);
        paged_next(p, sg, walk);
        const int end = sg.len + sg.nl;
        // this warp's 16-position tiles: t0, t0 + 4, ...
        const int t0 = sg.jb * ROWS_WARPS + warp;
        const int t1 = min(sg.je * ROWS_WARPS, (end + 15) / 16);
        const int n = t0 < t1 ? (t1 - t0 + ROWS_WARPS - 1) / ROWS_WARPS : 0;
        const int32_t* row_of_table = p.table + (int64_t)sg.z * p.st_z;

        auto load = [&](int i) {
            const int k0 = (t0 + i * ROWS_WARPS) * 16;
            const int pi = k0 / p.page, slot = k0 - pi * p.page;  // page is a multiple of 16: one page a tile
            const int e = ldi(row_of_table + pi);
            const bool good = (unsigned)e < (unsigned)p.P;
            if (!good && lane == 0) record_bad_page(p.status, SITE_PAGE_ATTENTION);
            const uint16_t* ks = kc;
            const uint16_t* vs = vc;
            if (good) {
                ks += e * p.sk_p + sg.hk * p.sk_h + slot * p.sk_n;
                vs += e * p.sv_p + sg.hk * p.sv_h + slot * p.sv_n;
            }
            const int live = good ? end - k0 : 0;  // rows of the tile that exist
            const uint32_t dst = ring + (i % T::NST) * 2 * T::HALF;
#pragma unroll
            for (int x = 0; x < 16 * T::CPR / 32; ++x) {
                const int id = x * 32 + lane, r = id / T::CPR, c = id % T::CPR;
                const bool there = r < live;
                const uint32_t at = swz<D>(r, c);
                cp_async16(dst + at, there ? ks + r * p.sk_n + c * 8 : kc, there ? 16 : 0);
                cp_async16(dst + T::HALF + at, there ? vs + r * p.sv_n + c * 8 : vc, there ? 16 : 0);
            }
        };
#pragma unroll
        for (int i = 0; i < T::NST - 1; ++i) {
            if (i < n) load(i);
            cp_commit();
        }
        // Q rows of the tile (zeros past the live ones)
        for (int x = tid; x < RT * T::CPR; x += 32 * ROWS_WARPS) {
            const int r = x / T::CPR, c = x % T::CPR;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (r < sg.rows) {
                const int row = sg.row0 + r, t = row / p.G, h = sg.hk * p.G + row - t * p.G;
                v = __ldcg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + (int64_t)sg.z * p.sq_z +
                                                          h * p.sq_h + t * p.sq_n + c * 8));
            }
            ptx::st_shared_v4(sbase + T::OFF_Q + swz<D>(r, c), v.x, v.y, v.z, v.w);
        }
        __syncthreads();
        // ldmatrix addresses: A fragments (rows lane % 16, chunk half lane / 16)
        uint32_t qf[QREG ? KS : 1][4];
        if constexpr (QREG) {
#pragma unroll
            for (int k = 0; k < KS; ++k) ldsm4(sbase + T::OFF_Q + swz<D>(lane % 16, 2 * k + lane / 16), qf[k]);
        }
        float o[MT][D / 8][4];
        float m[MT][2], l[MT][2];
        int tok[MT][2];
#pragma unroll
        for (int a = 0; a < MT; ++a) {
#pragma unroll
            for (int x = 0; x < D / 8; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y) o[a][x][y] = 0.f;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                m[a][y] = -INFINITY;
                l[a][y] = 0.f;
                tok[a][y] = min((sg.row0 + a * 16 + y * 8 + lane / 4) / p.G, p.T - 1);
            }
        }

        for (int i = 0; i < n; ++i) {
            cp_wait<T::NST - 2>();
            __syncwarp();
            const uint32_t ks = ring + (i % T::NST) * 2 * T::HALF, vs = ks + T::HALF;
            float s[MT][2][4];
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int y = 0; y < 4; ++y) s[a][x][y] = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t b[4];  // keys 0-7: d 0-7, d 8-15; keys 8-15: the same
                ldsm4(ks + swz<D>(lane % 8 + (lane / 16) * 8, 2 * k + (lane / 8) % 2), b);
#pragma unroll
                for (int a = 0; a < MT; ++a) {
                    uint32_t qa[4];
                    if constexpr (QREG) {
#pragma unroll
                        for (int y = 0; y < 4; ++y) qa[y] = qf[k][y];
                    } else {
                        ldsm4(sbase + T::OFF_Q + swz<D>(a * 16 + lane % 16, 2 * k + lane / 16), qa);
                    }
                    mma16816<BF16>(s[a][0], qa, b[0], b[1]);
                    mma16816<BF16>(s[a][1], qa, b[2], b[3]);
                }
            }
            const int k0 = (t0 + i * ROWS_WARPS) * 16;
            const bool masked = k0 + 16 > sg.len;
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        float v = s[a][x][y] * p.scale_log2;
                        if (masked) {
                            const int j = k0 + x * 8 + 2 * (lane % 4) + (y & 1) - sg.len, t = tok[a][y / 2];
                            bool seen = j < 0;
                            if (!seen && j < sg.nl)
                                seen = p.mask == nullptr
                                           ? j <= t
                                           : (__ldcg(p.mask + sg.z * p.sm_z + (int64_t)t * p.words + (j >> 5)) >> (j & 31)) & 1u;
                            if (!seen) v = -INFINITY;
                        }
                        s[a][x][y] = v;
                    }
            uint32_t pf[MT][4];
            bool grow = false;
            float top[MT][2];
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    float t = fmaxf(fmaxf(s[a][0][2 * y], s[a][0][2 * y + 1]), fmaxf(s[a][1][2 * y], s[a][1][2 * y + 1]));
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
                    top[a][y] = t;
                    grow |= t > m[a][y] + LAG;
                }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int a = 0; a < MT; ++a)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float mn = fmaxf(m[a][y], top[a][y]);
                        const float alpha = m[a][y] == -INFINITY ? 0.f : ptx::ex2(m[a][y] - mn);
                        m[a][y] = mn;
                        l[a][y] *= alpha;
#pragma unroll
                        for (int x = 0; x < D / 8; ++x) {
                            o[a][x][2 * y] *= alpha;
                            o[a][x][2 * y + 1] *= alpha;
                        }
                    }
            }
#pragma unroll
            for (int a = 0; a < MT; ++a) {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const float ref = m[a][y] == -INFINITY ? 0.f : m[a][y];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float p0 = ptx::ex2(s[a][x][2 * y] - ref), p1 = ptx::ex2(s[a][x][2 * y + 1] - ref);
                        l[a][y] += p0 + p1;
                        // P in the input type for the product (the sum keeps fp32): half a unit of
                        // the last place of each weight, as the other forward kernels round it
                        pf[a][x * 2 + y] = pack_pair<BF16>(p0, p1);
                    }
                }
            }
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {
                uint32_t b[4];  // d 0-7: keys 0-7, 8-15; d 8-15: the same
                ldsm4t(vs + swz<D>(lane % 16, 2 * x + lane / 16), b);
#pragma unroll
                for (int a = 0; a < MT; ++a) {
                    mma16816<BF16>(o[a][2 * x], pf[a], b[0], b[1]);
                    mma16816<BF16>(o[a][2 * x + 1], pf[a], b[2], b[3]);
                }
            }
            __syncwarp();
            if (i + T::NST - 1 < n) load(i + T::NST - 1);
            cp_commit();
        }

        // Join the warps: m, l and O through shared memory (a warp's O over its own, now idle, ring).
        cp_wait<0>();
        __syncwarp();
        float* mine = reinterpret_cast<float*>(smem + warp * T::RING);
        constexpr int XM = D / 8 < 8 ? D / 8 - 1 : 7;  // column permutation against bank conflicts
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                float t = l[a][y];
                t += __shfl_xor_sync(0xffffffffu, t, 1);
                t += __shfl_xor_sync(0xffffffffu, t, 2);
                const int r = a * 16 + y * 8 + lane / 4;
                if (lane % 4 == 0) {
                    ml[warp * RT + r] = m[a][y];
                    ml[(ROWS_WARPS + warp) * RT + r] = t;
                }
#pragma unroll
                for (int x = 0; x < D / 8; ++x)
                    *reinterpret_cast<float2*>(mine + r * D + ((x ^ (r & XM)) * 8) + 2 * (lane % 4)) =
                        make_float2(o[a][x][2 * y], o[a][x][2 * y + 1]);
            }
        __syncthreads();
        for (int x = tid; x < sg.rows * (D / 4); x += 32 * ROWS_WARPS) {
            const int r = x / (D / 4), c = x % (D / 4);
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < ROWS_WARPS; ++w) top = fmaxf(top, ml[w * RT + r]);
            float den = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < ROWS_WARPS; ++w) {
                const float mw = ml[w * RT + r];
                const float f = mw == -INFINITY ? 0.f : ptx::ex2(mw - top);
                den += f * ml[(ROWS_WARPS + w) * RT + r];
                const float4 v = *reinterpret_cast<const float4*>(
                    reinterpret_cast<const float*>(smem + w * T::RING) + r * D + (((c / 2) ^ (r & XM)) * 8) + (c % 2) * 4);
                if (mw != -INFINITY) {
                    acc.x += f * v.x;
                    acc.y += f * v.y;
                    acc.z += f * v.z;
                    acc.w += f * v.w;
                }
            }
            const float inv = den == 0.f ? 0.f : 1.f / den;  // nothing seen: O = 0, lse = -inf
            const float lse2 = den == 0.f ? -INFINITY : top + log2f(den);
            if (sg.slot >= 0) {
                float* slot = p.scratch + (int64_t)sg.slot * p.slot_floats;
                *reinterpret_cast<float4*>(slot + r * D + 4 * c) =
                    make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
                if (c == 0) slot[RT * D + r] = lse2;
            } else {
                const int row = sg.row0 + r, t = row / p.G, h = sg.hk * p.G + row - t * p.G;
                uint2 out;
                out.x = pack_pair<BF16>(acc.x * inv, acc.y * inv);
                out.y = pack_pair<BF16>(acc.z * inv, acc.w * inv);
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + (int64_t)sg.z * p.so_z + h * p.so_h +
                                          t * p.so_n + 4 * c) = out;
                if (c == 0 && p.lse != nullptr)
                    p.lse[((int64_t)sg.z * p.Hq + h) * p.T + t] = lse2 * 0.6931471805599453f;
            }
        }
        __syncthreads();  // before the next segment fills the rings and Q
    }
}

}  // namespace fa
