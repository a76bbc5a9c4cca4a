// Attention over a paged cache for few query rows (a decode step, a small
// tree): O = softmax(Q Kᵀ · scale) V for up to 16 rows of one (sequence, kv
// head) -- the new tokens of the sequence times the query heads that share the
// kv head -- against all of its cached positions.
//
// What bounds it is reading K and V once: with R rows a position costs 4 D R
// flops for 4 D bytes, far below what the tensor cores could do.  So the work
// is organised around loads in flight, not around the products:
//   * a warp is a worker of its own: it takes one equal range of the launch's
//     key blocks (KT positions each), with a private ring of NST blocks of K
//     and V in shared memory that it fills by TMA through the block table, one
//     lane per box of min(page, KT) rows of a 64-column chunk.  No warp waits
//     for another one anywhere, so a late page holds up one warp only, and
//     there is nothing to join at the end of a tile but the parts that the
//     merge kernel joins anyway;
//   * the ring runs across the ends of tiles and sequences: the copies of the
//     next tile are in flight while the last one is finished, and the block
//     table entry of the copies after those is on its way too;
//   * the products run on mma.sync m16n8k16: 16 rows are far too few for a
//     128-row tcgen05 tile (fa_paged_tile_kernel.cuh takes the calls with more
//     rows), and Q, S, P and O stay in registers.
// Measured: 64 sequences of 256-4096 positions, one token, 32 query heads on 8 of
// D = 128 (572 MB): 91 us without the merge, 6.3 TB/s, 94 % of a plain copy's
// rate; two of 30000-32768, 16 heads of D = 64 (257 MB): 41.7 us, 6.2 TB/s.  Two
// CTAs of four warps an SM (231 registers a thread) have rings of 192 KB, two
// thirds of them in flight at a time.  One sequence of 1024: 6.2 us, the way from
// launch to lengths, table entry, copies and one block a warp.  The merge adds 4
// to 5 us to each.  At D = 256 there is room for one CTA an SM, and the tile
// kernel is level or better from one row on: there this kernel has only the
// groups of more than 128 query heads.
// What a page holds behind the sequence's last position has no effect: its
// scores are masked, and its V rows are zeroed in shared memory (0 · NaN would
// reach O).  Waits for copies are bounded as in fa_fwd_kernel.cuh.
#pragma once

#include "fa_fwd_kernel.cuh"
#include "fa_paged_sched.cuh"

namespace fa {

constexpr int ROWS_WARPS = 4;  // per CTA

template <int D_>
struct RowsTraits {
    static constexpr int D = D_, RT = 16;
    static constexpr int CTAS = D <= 128 ? 2 : 1;        // per SM
    static constexpr int U = D <= 64 ? 2 : 1;            // 16-position steps per key block
    static constexpr int KT = 16 * U;                    // positions per key block
    static constexpr int CPR = D / 8;                    // 16-byte pieces per row
    static constexpr int SW = D >= 64 ? 128 : D * 2;     // bytes per swizzled row chunk
    static constexpr int NCHUNK = D * 2 / SW;
    static constexpr int HALF = KT * D * 2;              // bytes of a block of K (or V)
    static constexpr int NST = D >= 64 ? 3 : 4;
    static constexpr int RING = NST * 2 * HALF;          // per warp
    static constexpr bool QREG = D <= 128;               // Q fragments in registers, else in shared memory
    static constexpr int QB = QREG ? 0 : RT * D * 2;     // per warp
    static constexpr int OFF_Q = ROWS_WARPS * RING;
    static constexpr int OFF_BAR = OFF_Q + ROWS_WARPS * QB;  // NST barriers a warp: copies landed
    static constexpr int OFF_ABORT = OFF_BAR + ROWS_WARPS * NST * 8;
    static constexpr int OFF_FIND = OFF_ABORT + 16;
    static constexpr int SMEM = OFF_FIND + (int)sizeof(PagedFind<ROWS_WARPS>) + 1024;  // (+ alignment)
    static_assert(SMEM * CTAS <= 228 * 1024 - CTAS * 1024 && SMEM <= 227 * 1024, "shared memory budget");
    static_assert(OFF_FIND % 8 == 0 && HALF % 1024 == 0, "alignment");
    static_assert(2 * NCHUNK * U <= 32, "a lane per box");
};

namespace rowsk {

// 16-byte piece c of row r of a tile of ROWS rows as TMA lays it out: chunks of
// up to 128 bytes a row, [chunk][row], the pieces of a row permuted so that
// eight consecutive rows of one piece lie in different banks.
template <int D, int ROWS>
__device__ __forceinline__ uint32_t swz(int r, int c) {
    constexpr int CPR = D / 8;
    if constexpr (CPR >= 8) return (uint32_t)((c / 8) * ROWS * 128 + r * 128 + (((c % 8) ^ (r & 7)) << 4));
    else if constexpr (CPR == 4) return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
    else return (uint32_t)(r * 32 + ((c ^ ((r >> 2) & 1)) << 4));
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

// The copies of one worker: its place in the range, a few blocks ahead of the
// products.  A lane has one box of each block: rows piece * box_rows .. of chunk
// `chunk` of K or V, and loads the block table entry of its next box ahead.
template <int D>
struct RowsLoader {
    using T = RowsTraits<D>;
    PagedWalk w;
    PagedSeg g;
    int j;          // next block to copy
    bool more;
    bool there;     // this lane's box of it exists
    int page, slot;

    __device__ __forceinline__ int piece() const { return (int)(threadIdx.x % 32) / (2 * T::NCHUNK); }
    __device__ __forceinline__ void request(const PagedParams& p) {
        const int k = j * T::KT + piece() * p.box_rows;
        there = piece() * p.box_rows < T::KT && k < g.len + g.nl;
        if (there) {
            const int col = p.by_page(k);
            page = ldi(p.table + (int64_t)g.z * p.st_z + col);
            slot = k - col * p.page;
        }
    }
    __device__ __forceinline__ void start(const PagedParams& p, const PagedWalk& walk, int worker) {
        w = walk;
        more = paged_seg<T::KT>(p, w, g, worker, 0);
        if (more) {
            j = g.jb;
            request(p);
        }
    }
    // Copy the next block to `dst`, completing on `bar`, and go on to the one after.
    __device__ __forceinline__ void load(const PagedParams& p, const CUtensorMap* tmK, const CUtensorMap* tmV,
                                         uint32_t dst, uint32_t bar, int worker, uint64_t policy) {
        const int lane = threadIdx.x % 32;
        const uint32_t bytes = (uint32_t)p.box_rows * T::SW;
        const uint32_t n = __popc(__ballot_sync(0xffffffffu, there));
        if (lane == 0) ptx::mbar_arrive_expect_tx(bar, n * bytes);
        __syncwarp();
        if (there) {
            if ((unsigned)page >= (unsigned)p.P) {
                record_bad_page(p.status, SITE_PAGE_ATTENTION);
                page = p.P;  // outside the map: zeros
            }
            const int which = lane % (2 * T::NCHUNK), chunk = which / 2;
            ptx::tma_load_4d(dst + (which & 1) * T::HALF + chunk * (T::KT * T::SW) + piece() * bytes,
                             which & 1 ? tmV : tmK, bar, chunk * (T::SW / 2), slot, g.hk, page, policy);
        }
        if (++j == g.je) {
            paged_next<T::KT>(p, w);
            more = paged_seg<T::KT>(p, w, g, worker, 0);
            j = g.jb;
        }
        if (more) request(p);
    }
};

}  // namespace rowsk

template <int D, bool BF16>
__global__ void __launch_bounds__(32 * ROWS_WARPS, RowsTraits<D>::CTAS)
    fa_paged_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const PagedParams p) {
    using T = RowsTraits<D>;
    using namespace rowsk;
    constexpr int KS = D / 16, U = T::U;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = ptx::smem_addr(smem);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int worker = blockIdx.x * ROWS_WARPS + warp;
    const uint32_t ring = sbase + warp * T::RING, bars = sbase + T::OFF_BAR + warp * T::NST * 8;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + T::OFF_ABORT);
    if (lane == 0) {
        for (int i = 0; i < T::NST; ++i) ptx::mbar_init(bars + 8 * i, 1);
        if (warp == 0) *abort_flag = 0;
        ptx::fence_mbar_init();
        if (p.P > 0) {
            ptx::prefetch_tmap(&tmK);
            ptx::prefetch_tmap(&tmV);
        }
    }
    __syncthreads();
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();

    const Ctl ctl{abort_flag, p.status, p.wait_limit_ns};
    const uint64_t policy = ptx::policy_evict_first();  // (each position is read once)
    auto* find = reinterpret_cast<PagedFind<ROWS_WARPS>*>(smem + T::OFF_FIND);
    bool pads;
    PagedWalk walk = paged_range<T::KT, ROWS_WARPS>(p, find, blockIdx.x * ROWS_WARPS, warp, lane == 0, pads);
    RowsLoader<D> ld;
    ld.start(p, walk, worker);
    int loads = 0, used = 0;  // blocks asked for and used up
    // the next block into slot loads % NST; test hook: the first worker's first one is withheld
    auto load = [&](int slot) {
        const bool withheld = p.inject_stall && worker == 0 && loads == 0;
        if (!withheld) ld.load(p, &tmK, &tmV, ring + slot * 2 * T::HALF, bars + 8 * slot, worker, policy);
        ++loads;
    };
#pragma unroll
    for (int i = 0; i < T::NST - 1; ++i)
        if (ld.more) load(i);
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;

    PagedSeg sg;
    for (; ok && paged_seg<T::KT>(p, walk, sg, worker, 0); paged_next<T::KT>(p, walk)) {
        // Q fragments of the tile's rows (zeros past the live ones); a thread
        // holds rows lane / 4 and lane / 4 + 8
        auto q_row = [&](int r) -> const uint16_t* {
            const int row = sg.row0 + r, t = p.by_g(row), h = sg.hk * p.G + row - t * p.G;
            return static_cast<const uint16_t*>(p.q) + (int64_t)sg.z * p.sq_z + h * p.sq_h + t * p.sq_n;
        };
        uint32_t qf[T::QREG ? KS : 1][4];
        const uint32_t qs = sbase + T::OFF_Q + warp * T::QB;
        if constexpr (T::QREG) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int r = lane / 4 + 8 * y;
                const uint16_t* src = q_row(min(r, sg.rows - 1)) + 2 * (lane % 4);
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    const uint32_t a = __ldcg(reinterpret_cast<const uint32_t*>(src + 16 * k));
                    const uint32_t b = __ldcg(reinterpret_cast<const uint32_t*>(src + 16 * k + 8));
                    qf[k][y] = r < sg.rows ? a : 0u;
                    qf[k][2 + y] = r < sg.rows ? b : 0u;
                }
            }
        } else {
            __syncwarp();
            for (int x = lane; x < T::RT * T::CPR; x += 32) {
                const int r = x / T::CPR, c = x % T::CPR;
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (r < sg.rows) v = __ldcg(reinterpret_cast<const uint4*>(q_row(r) + c * 8));
                ptx::st_shared_v4(qs + swz<D, 16>(r, c), v.x, v.y, v.z, v.w);
            }
            __syncwarp();
        }
        float o[D / 8][4];
        float m[2], l[2];
        int tok[2];
#pragma unroll
        for (int x = 0; x < D / 8; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) o[x][y] = 0.f;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            m[y] = -INFINITY;
            l[y] = 0.f;
            tok[y] = min(p.by_g(sg.row0 + y * 8 + lane / 4), p.T - 1);
        }

        for (int j = sg.jb; j < sg.je; ++j) {
            if (!warp_wait_phase(bars + 8 * stage, phase, ctl, SITE_K_FULL)) { ok = false; break; }
            const uint32_t ks = ring + stage * 2 * T::HALF, vs = ks + T::HALF;
            const int behind = sg.len + sg.nl - j * T::KT;  // first row behind the sequence's end
            if (behind < T::KT) {
                for (int i = lane; i < (T::KT - behind) * T::CPR; i += 32)
                    ptx::st_shared_v4(vs + swz<D, T::KT>(behind + i / T::CPR, i % T::CPR), 0u, 0u, 0u, 0u);
                ptx::fence_proxy_async_smem();  // before a later copy into the slot
                __syncwarp();
            }
            float s[2 * U][4];
#pragma unroll
            for (int x = 0; x < 2 * U; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y) s[x][y] = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t qa[4];
                if constexpr (T::QREG) {
#pragma unroll
                    for (int y = 0; y < 4; ++y) qa[y] = qf[k][y];
                } else {
                    ldsm4(qs + swz<D, 16>(lane % 16, 2 * k + lane / 16), qa);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    uint32_t b[4];  // keys 0-7: d 0-7, d 8-15; keys 8-15: the same
                    ldsm4(ks + swz<D, T::KT>(16 * u + lane % 8 + (lane / 16) * 8, 2 * k + (lane / 8) % 2), b);
                    mma16816<BF16>(s[2 * u], qa, b[0], b[1]);
                    mma16816<BF16>(s[2 * u + 1], qa, b[2], b[3]);
                }
            }
            const int k0 = j * T::KT;
#pragma unroll
            for (int x = 0; x < 2 * U; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y) s[x][y] *= p.scale_log2;
            if (k0 + T::KT > sg.len) {
#pragma unroll
                for (int x = 0; x < 2 * U; ++x)
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const int i = k0 + x * 8 + 2 * (lane % 4) + (y & 1) - sg.len, t = tok[y / 2];
                        bool seen = i < 0;
                        if (!seen && i < sg.nl)
                            seen = p.mask == nullptr
                                       ? i <= t
                                       : (__ldcg(p.mask + sg.z * p.sm_z + (int64_t)t * p.words + (i >> 5)) >> (i & 31)) & 1u;
                        if (!seen) s[x][y] = -INFINITY;
                    }
            }
            float top[2];
            bool grow = false;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                float t = fmaxf(s[0][2 * y], s[0][2 * y + 1]);
#pragma unroll
                for (int x = 1; x < 2 * U; ++x) t = ptx::fmax3(t, s[x][2 * y], s[x][2 * y + 1]);
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
                top[y] = t;
                grow |= t > m[y] + LAG;
            }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const float mn = fmaxf(m[y], top[y]);
                    const float alpha = m[y] == -INFINITY ? 0.f : ptx::ex2(m[y] - mn);
                    m[y] = mn;
                    l[y] *= alpha;
#pragma unroll
                    for (int x = 0; x < D / 8; ++x) {
                        o[x][2 * y] *= alpha;
                        o[x][2 * y + 1] *= alpha;
                    }
                }
            }
            uint32_t pf[U][4];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const float ref = m[y] == -INFINITY ? 0.f : m[y];  // nothing seen so far: p = 0
#pragma unroll
                for (int x = 0; x < 2 * U; ++x) {
                    const float p0 = ptx::ex2(s[x][2 * y] - ref), p1 = ptx::ex2(s[x][2 * y + 1] - ref);
                    l[y] += p0 + p1;
                    // P in the input type for the product (the sum keeps fp32): half a unit of
                    // the last place of each weight, as the other forward kernels round it
                    pf[x / 2][(x % 2) * 2 + y] = pack_pair<BF16>(p0, p1);
                }
            }
#pragma unroll
            for (int x = 0; x < D / 16; ++x)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    uint32_t b[4];  // d 0-7: keys 0-7, 8-15; d 8-15: the same
                    ldsm4t(vs + swz<D, T::KT>(16 * u + lane % 16, 2 * x + lane / 16), b);
                    mma16816<BF16>(o[2 * x], pf[u], b[0], b[1]);
                    mma16816<BF16>(o[2 * x + 1], pf[u], b[2], b[3]);
                }
            __syncwarp();
            // the block NST - 1 ahead goes to the slot that the last block has left
            ++used;
            if (ld.more) load(stage == 0 ? T::NST - 1 : stage - 1);
            if (++stage == T::NST) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if (!ok) break;

#pragma unroll
        for (int y = 0; y < 2; ++y) {
            float den = l[y];
            den += __shfl_xor_sync(0xffffffffu, den, 1);
            den += __shfl_xor_sync(0xffffffffu, den, 2);
            const int r = y * 8 + lane / 4;
            if (r >= sg.rows) continue;
            const float inv = den == 0.f ? 0.f : 1.f / den;  // nothing seen: O = 0, lse = -inf
            const float lse2 = den == 0.f ? -INFINITY : m[y] + log2f(den);
            if (sg.slot >= 0) {
                float* slot = p.scratch + (int64_t)sg.slot * p.slot_floats;
#pragma unroll
                for (int x = 0; x < D / 8; ++x)
                    *reinterpret_cast<float2*>(slot + (x * p.tile_rows + r) * 8 + 2 * (lane % 4)) =
                        make_float2(o[x][2 * y] * inv, o[x][2 * y + 1] * inv);
                if (lane % 4 == 0) slot[p.tile_rows * D + r] = lse2;
            } else {
                const int row = sg.row0 + r, t = p.by_g(row), h = sg.hk * p.G + row - t * p.G;
                uint16_t* dst = static_cast<uint16_t*>(p.o) + (int64_t)sg.z * p.so_z + h * p.so_h + t * p.so_n;
#pragma unroll
                for (int x = 0; x < D / 8; ++x)
                    *reinterpret_cast<uint32_t*>(dst + 8 * x + 2 * (lane % 4)) =
                        pack_pair<BF16>(o[x][2 * y] * inv, o[x][2 * y + 1] * inv);
                if (lane % 4 == 0 && p.lse != nullptr)
                    p.lse[((int64_t)sg.z * p.Hq + h) * p.T + t] = lse2 * 0.6931471805599453f;
            }
        }
    }
    if (!ok) {
        // let every copy still in flight land before shared memory is released (a withheld one never does)
        for (int i = used; i < loads; ++i)
            drain_phase(bars + 8 * (i % T::NST), (uint32_t)(i / T::NST) & 1u, p.inject_stall ? ctl.limit_ns / 64 : ctl.limit_ns);
    }
    if (pads) paged_fill<D>(p, worker, (int)gridDim.x * ROWS_WARPS);
}

}  // namespace fa
