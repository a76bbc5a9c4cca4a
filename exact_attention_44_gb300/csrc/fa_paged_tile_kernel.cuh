// Attention over a paged cache for many query rows (a wide tree, a chunk of a
// prompt): the forward of fa_fwd_kernel.cuh -- S = Q Kᵀ and O += P V on
// tcgen05 with S, P and O in tensor memory, K and V through TMA rings, an
// online softmax over four column groups -- with
//   * a tile of up to 128 (new token, query head) rows of one (sequence, kv
//     head), so that K and V of a position are loaded and multiplied once for
//     the whole group;
//   * K and V blocks gathered from their pages: a block of BN positions is
//     BN / RB boxes of RB = gcd(page, BN) rows, one lane of the producer warp
//     per box, each through its own block table entry (out of range: the
//     tensor map fills zeros);
//   * the device-side division of the work of fa_paged_sched.cuh;
//   * the tree's bits as one 32-bit word per thread and block (a thread holds
//     32 positions of a row);
//   * V rows behind the sequence's end zeroed in shared memory before the
//     product reads them: whatever the page holds there (NaN included) must
//     not meet the zero weights.
// Warps whose 32 rows hold no token skip the softmax and only keep the
// barriers' counts.  Every wait is bounded as in fa_fwd_kernel.cuh.
//
// Rows of a tile that hold no token (behind the last new token, and behind
// tile_rows where the group does not divide 128: there Q's slot is whatever
// shared memory held before) go through the products and the softmax of their
// warp, but must not decide anything for it: when O is rescaled, the lanes of
// the live rows move their reference too, and P is rounded against another one.
// So their reference is +inf from the first block on: they never ask for it.
//
// What bounds it.  With one tile a kv head (up to 128 rows), DRAM: a block's K
// and V are 64 KB at D = 128, 1.49 us of an SM's share of 6.7 TB/s (1.31 us
// measured), against 0.8 us that the chain S -> softmax -> P takes a block, as
// in the contiguous forward (1.06 us with 16-position pages, whose 32 boxes a
// block the copy unit takes one after another).  With two tiles the two bounds
// meet: 32 sequences of 4096-8192 positions x 64 tokens x 4 heads (848 MB, 207
// GFLOP) take 188 to 195 us a call (175 to 192 as one input repeated in a graph),
// 4.4 TB/s and 1.08 PFLOP/s at 1.2 kW, where the clock
// has fallen from 2.07 to 1.85 GHz (168 us with all pages in L2; a third slot
// in the rings of K and V instead of Q's second changes nothing).  Between two
// tiles a softmax warp loses 2.6 us (its last product 0.6, the output 1.2, the
// next tile's first scores 0.5), which short contexts feel: 128 sequences of
// 300-400 x 128 tokens x 4 heads take 183 us.  Short calls are bounded by the way
// from launch to the first products (about 8 us: lengths, block table, first
// copies, first block) and by the merge of the parts (about 5 us; 8 sequences of
// 500-3000 x 32 tokens: 22.0 us in all, 10 us of DRAM time).
#pragma once

#include "fa_fwd_kernel.cuh"
#include "fa_paged_sched.cuh"

namespace fa {

template <int D_>
struct TileTraits : Traits<D_> {
    using Base = Traits<D_>;
    static constexpr int B_VFIX = Base::NUM_BARS;             // [2] V slot's rows behind the end zeroed
    static constexpr int SEGS = 4;                            // segments in the ring
    static constexpr int B_SEGFULL = B_VFIX + 2;              // [SEGS] segment written (K producer)
    static constexpr int B_SEGFREE = B_SEGFULL + SEGS;        // [SEGS] read by every other warp
    static constexpr int NUM_BARS = B_SEGFREE + SEGS;
    static constexpr int OFF_BAR = Base::OFF_OST;             // (O is not staged)
    static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
    static constexpr int OFF_SEG = OFF_MISC + 16;
    static constexpr int SMEM_USED = OFF_SEG + SEGS * 48;
    static constexpr int SMEM_BYTES = (SMEM_USED + 1024) > 120 * 1024 ? SMEM_USED + 1024 : 120 * 1024;
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
    // four warps for the copies and products, then the softmax warps, which also write O
    static constexpr int THREADS = 32 * (4 + 4 * Base::NG);
    static __device__ __forceinline__ uint32_t bar_count(int i) {
        if (i >= B_SEGFREE && i < B_SEGFREE + SEGS) return THREADS / 32 - 1;
        if (i == Base::B_OFREE) return 4 * Base::NG;  // one arrival a warp
        if (i >= B_VFIX) return 1;
        return Base::bar_count(i);
    }
    static_assert((int)sizeof(PagedFind<1>) <= 2 * Base::HAND_ROWS * BM * 4, "the range search fits the hand-over area");
};

// The K producer's warp walks the range and hands the segments to the other
// warps through a ring in shared memory, a few ahead of them.  (Every role
// walking by itself cost registers -- 0.99 against 0.81 us a block in the
// softmax loop -- and 24 warps doing the same arithmetic at the start of every
// segment got in each other's way.)
struct SegMsg {
    int z, hk, jb, je, slot, len, nl, row0, rows, pads, unused[2];  // je = 0: the end
};
template <int D, typename Bar>
__device__ __forceinline__ void seg_put(volatile int* ring, const PagedSeg& g, bool have, bool pads,
                                         uint32_t n, Bar bar) {
    using T = TileTraits<D>;
    volatile int* s = ring + (n % T::SEGS) * (sizeof(SegMsg) / 4);
    if (threadIdx.x % 32 == 0) {
        s[0] = g.z, s[1] = g.hk, s[2] = g.jb, s[3] = have ? g.je : 0, s[4] = g.slot;
        s[5] = g.len, s[6] = g.nl, s[7] = g.row0, s[8] = g.rows, s[9] = pads;
        ptx::mbar_arrive(bar(T::B_SEGFULL + n % T::SEGS));
    }
    __syncwarp();
}
template <int D>
__device__ __forceinline__ void seg_read(volatile const int* ring, PagedSeg& g, uint32_t n) {
    volatile const int* s = ring + (n % TileTraits<D>::SEGS) * (sizeof(SegMsg) / 4);
    g.z = s[0], g.hk = s[1], g.jb = s[2], g.je = s[3], g.slot = s[4];
    g.len = s[5], g.nl = s[6], g.row0 = s[7], g.rows = s[8];
}
// WARP: the whole warp calls, else its one active lane.
template <int D, bool WARP, typename Bar>
__device__ __forceinline__ void seg_release(uint32_t n, Bar bar) {
    if (WARP) __syncwarp();
    if (!WARP || threadIdx.x % 32 == 0) ptx::mbar_arrive(bar(TileTraits<D>::B_SEGFREE + n % TileTraits<D>::SEGS));
}
// Waits for segment n of the ring; false when the wait ran out or another role gave up.
template <int D, bool WARP, typename Bar>
__device__ __forceinline__ bool seg_wait(uint32_t n, Bar bar, const Ctl& ctl) {
    using T = TileTraits<D>;
    const uint32_t full = bar(T::B_SEGFULL + n % T::SEGS), parity = (n / T::SEGS) & 1u;
    return WARP ? warp_wait_phase(full, parity, ctl, SITE_SEG_FULL) : wait_phase(full, parity, ctl, SITE_SEG_FULL);
}
// The next segment of a role that needs it no longer once it has read it; false
// at the end of the range, or (ok false) when the wait ran out.
template <int D, bool WARP, typename Bar>
__device__ __forceinline__ bool seg_get(volatile const int* ring, PagedSeg& g, uint32_t n, Bar bar, const Ctl& ctl,
                                        bool& ok) {
    ok = seg_wait<D, WARP>(n, bar, ctl);
    if (!ok) return false;
    seg_read<D>(ring, g, n);
    seg_release<D, WARP>(n, bar);
    return g.je > 0;
}

// A block's boxes: lane b of the producer warp has the box of positions
// kj * BN + b * rb .. (b * rb < BN), if the sequence has any of them.
struct PageBox {
    int page, slot;
    bool there;
};
__device__ __forceinline__ PageBox page_box(const PagedParams& p, const int32_t* row, int k0, int rb, int bn, int end,
                                            int lane) {
    PageBox b{p.P, 0, false};
    const int k = k0 + lane * rb;
    if (lane * rb < bn && k < end) {
        const int col = p.by_page(k);
        b.slot = k - col * p.page;
        b.page = ldi(row + col);
        b.there = true;
    }
    return b;
}
// Called by the warp: one block into shared memory at dst, completing on bar.
template <int D>
__device__ __forceinline__ void load_boxes(const PagedParams& p, PageBox b, const CUtensorMap* tm, uint32_t dst,
                                           uint32_t bar, int hk, int rb, int lane, uint64_t policy) {
    using T = Traits<D>;
    if (b.there && (unsigned)b.page >= (unsigned)p.P) {
        record_bad_page(p.status, SITE_PAGE_ATTENTION);
        b.page = p.P;  // outside the map: zeros
    }
    const uint32_t n = __popc(__ballot_sync(0xffffffffu, b.there));
    if (lane == 0) ptx::mbar_arrive_expect_tx(bar, n * rb * T::SW * T::NCHUNK);
    __syncwarp();
    if (b.there)
        for (int c = 0; c < T::NCHUNK; ++c)
            ptx::tma_load_4d(dst + c * (T::BN * T::SW) + lane * rb * T::SW, tm, bar, c * T::SWE, b.slot, hk, b.page,
                             policy);
}

template <int D>
__device__ void tile_producer_qk(const CUtensorMap* tmQ, const CUtensorMap* tmK, const PagedParams& p, PagedWalk w,
                                 bool pads, volatile int* ring, uint32_t sbase, uint32_t bar0, const Ctl& ctl) {
    using T = TileTraits<D>;
    auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    const int lane = threadIdx.x % 32;
    // K and V pass once (the members of a team read them at the same time), unless there
    // are more tiles than a team has members: evict first 165 against last 170 us for 16
    // sequences x 512 rows, 650 against 633 for 4 x 8192
    const uint64_t pol_q = ptx::policy_evict_first();
    const uint64_t pol_kv = p.tiles > p.team ? ptx::policy_evict_last() : ptx::policy_evict_first();
    uint32_t qi = 0, ki = 0;
    bool ok = true, withheld = false;
    auto load_q = [&](const PagedSeg& sg) -> bool {
        const uint32_t s = qi % T::Q_STAGES, ph = (qi / T::Q_STAGES) & 1u;
        if (!warp_wait_phase(bar(T::B_QEMPTY + s), ph ^ 1u, ctl, SITE_Q_EMPTY)) return false;
        if (lane == 0) {
            ptx::mbar_arrive_expect_tx(bar(T::B_QFULL + s), (uint32_t)p.tile_rows * T::SW * T::NCHUNK);
            const uint32_t dst = sbase + T::OFF_Q + s * T::Q_BYTES;
            for (int c = 0; c < T::NCHUNK; ++c)
                ptx::tma_load_4d(dst + c * (BM * T::SW), tmQ, bar(T::B_QFULL + s), c * T::SWE, sg.hk * p.G,
                                 p.by_g(sg.row0), sg.z, pol_q);
        }
        __syncwarp();
        ++qi;
        return true;
    };
    uint32_t nseg = 0;  // segments put into the ring
    auto put = [&](const PagedSeg& sg, bool have) -> bool {
        const uint32_t slot = nseg % T::SEGS;
        if (nseg >= (uint32_t)T::SEGS &&
            !warp_wait_phase(bar(T::B_SEGFREE + slot), (nseg / T::SEGS - 1) & 1u, ctl, SITE_SEG_FREE)) return false;
        seg_put<D>(ring, sg, have, pads, nseg, bar);
        ++nseg;
        return true;
    };
    const int member = (int)blockIdx.x - (int)(blockIdx.x / p.team) * p.team;
    PagedSeg sg{};
    bool have = paged_seg<T::BN>(p, w, sg, (int)blockIdx.x, member);
    ok = put(sg, have);
    bool first = true;
    while (ok && have) {
        const int jb = sg.jb, je = sg.je, hk = sg.hk, end = sg.len + sg.nl;
        const int32_t* row = p.table + (int64_t)sg.z * p.st_z;
        PageBox b = page_box(p, row, jb * T::BN, p.box_rows, T::BN, end, lane);
        // the first tile's Q goes while its first table entries are on their way
        if (first && !load_q(sg)) { ok = false; break; }
        first = false;
        for (int j = jb; j < je; ++j) {
            PageBox after = b;
            if (j + 1 < je) after = page_box(p, row, (j + 1) * T::BN, p.box_rows, T::BN, end, lane);
            const uint32_t s = ki & 1u;
            if (ki >= 2 && !warp_wait_phase(bar(T::B_SFULL + rslot<T::SR>(ki - 2)), rphase<T::SR>(ki - 2), ctl,
                                            SITE_K_EMPTY)) { ok = false; break; }
            if (p.inject_stall && blockIdx.x == 0 && !withheld) {
                withheld = true;  // never issued: the S issuer's wait for this block must time out
            } else {
                load_boxes<D>(p, b, tmK, sbase + T::OFF_K + s * T::KV_BYTES, bar(T::B_KFULL + s), hk, p.box_rows,
                              lane, pol_kv);
            }
            ++ki;
            b = after;
            // the next segment, after the first K; its Q then if there are two Q slots,
            // else after the last K
            if (j == jb) {
                paged_next<T::BN>(p, w);
                have = paged_seg<T::BN>(p, w, sg, (int)blockIdx.x, member);
                if (!put(sg, have)) { ok = false; break; }
            }
            if (j == (T::Q_STAGES >= 2 ? jb : je - 1) && have && !load_q(sg)) { ok = false; break; }
        }
    }
    if (!ok) {
        const uint64_t lim = ctl.limit_ns;
        for (uint32_t i = qi > (uint32_t)T::Q_STAGES ? qi - T::Q_STAGES : 0; i < qi; ++i)
            drain_phase(bar(T::B_QFULL + i % T::Q_STAGES), (i / T::Q_STAGES) & 1u, lim);
        for (uint32_t i = ki > 2u ? ki - 2u : 0u; i < ki; ++i)
            drain_phase(bar(T::B_KFULL + (i & 1u)), (i >> 1) & 1u, withheld ? lim / 64 : lim);
    }
}

template <int D>
__device__ void tile_producer_v(const CUtensorMap* tmV, const PagedParams& p, volatile int* ring, uint32_t sbase,
                                uint32_t bar0, const Ctl& ctl) {
    using T = TileTraits<D>;
    auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    const int lane = threadIdx.x % 32;
    const uint64_t pol_kv = p.tiles > p.team ? ptx::policy_evict_last() : ptx::policy_evict_first();
    uint32_t vi = 0;
    bool ok = true;
    for (uint32_t n = 0;; ++n) {
        int jb, je, hk, end;
        const int32_t* row;
        {
            PagedSeg sg;
            if (!ok || !seg_get<D, true>(ring, sg, n, bar, ctl, ok)) break;
            jb = sg.jb, je = sg.je, hk = sg.hk, end = sg.len + sg.nl;
            row = p.table + (int64_t)sg.z * p.st_z;
        }
        PageBox b = page_box(p, row, jb * T::BN, p.box_rows, T::BN, end, lane);
        for (int j = jb; j < je; ++j) {
            PageBox after = b;
            if (j + 1 < je) after = page_box(p, row, (j + 1) * T::BN, p.box_rows, T::BN, end, lane);
            const uint32_t s = vi & 1u;
            if (vi >= 2 && !warp_wait_phase(bar(T::B_PVDONE + rslot<T::SR>(vi - 2)), rphase<T::SR>(vi - 2), ctl,
                                            SITE_V_EMPTY)) { ok = false; break; }
            const uint32_t dst = sbase + T::OFF_V + s * T::KV_BYTES;
            load_boxes<D>(p, b, tmV, dst, bar(T::B_VFULL + s), hk, p.box_rows, lane, pol_kv);
            ++vi;
            b = after;
            if ((j + 1) * T::BN > end) {
                // zero the rows behind the end, once the copies have landed
                if (!warp_wait_phase(bar(T::B_VFULL + s), ((vi - 1) >> 1) & 1u, ctl, SITE_V_FULL)) { ok = false; break; }
                const int first = end - j * T::BN;  // 1 .. BN - 1
                constexpr int PR = T::SW / 16;      // 16-byte pieces of a row's chunk
                for (int c = 0; c < T::NCHUNK; ++c)
                    for (int i = first * PR + lane; i < T::BN * PR; i += 32)
                        ptx::st_shared_v4(dst + c * (T::BN * T::SW) + i * 16, 0u, 0u, 0u, 0u);
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(T::B_VFIX + s));
            }
        }
    }
    if (!ok)
        for (uint32_t i = vi > 2u ? vi - 2u : 0u; i < vi; ++i)
            drain_phase(bar(T::B_VFULL + (i & 1u)), (i >> 1) & 1u, ctl.limit_ns);
}

template <int D, bool BF16>
__device__ void tile_mma_qk(const PagedParams& p, volatile int* ring, uint32_t sbase, uint32_t bar0, uint32_t tmem,
                            const Ctl& ctl) {
    using T = TileTraits<D>;
    auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    const uint32_t IDESC = ptx::idesc_f16(BM, T::BN, BF16, false, false) | (p.negate_s ? ptx::IDESC_NEGATE_A : 0u);
    constexpr uint32_t HI = ptx::smem_desc_hi(8 * T::SW, T::SWIZZLE_CODE);
    const uint32_t q_lo0 = ptx::smem_desc_lo(sbase + T::OFF_Q, 16);
    const uint32_t k_lo0 = ptx::smem_desc_lo(sbase + T::OFF_K, 16);
    uint32_t qi = 0, g = 0;
    bool ok = true;
    for (uint32_t n = 0;; ++n) {
        int jb, je;
        {
            PagedSeg sg;
            if (!ok || !seg_get<D, false>(ring, sg, n, bar, ctl, ok)) break;
            jb = sg.jb, je = sg.je;
        }
        const uint32_t qs = qi % T::Q_STAGES;
        if (!wait_phase(bar(T::B_QFULL + qs), (qi / T::Q_STAGES) & 1u, ctl, SITE_Q_FULL)) { ok = false; break; }
        const uint32_t q_lo = q_lo0 + qs * (T::Q_BYTES >> 4);
        for (int j = jb; j < je; ++j, ++g) {
            const uint32_t kb = g & 1u, r = rslot<T::SR>(g);
            if (!wait_phase(bar(T::B_KFULL + kb), (g >> 1) & 1u, ctl, SITE_K_FULL)) { ok = false; break; }
            if (g >= (uint32_t)T::SR && !wait_phase(bar(T::B_PVDONE + r), rphase<T::SR>(g - T::SR), ctl, SITE_S_FREE)) {
                ok = false;
                break;
            }
            ptx::tc_fence_after();
            const uint32_t k_lo = k_lo0 + kb * (T::KV_BYTES >> 4);
            const uint32_t d_tmem = tmem + T::TM_S + r * T::BN;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t a_off = (((kk * 16) / T::SWE) * (BM * T::SW) + ((kk * 16) % T::SWE) * 2) >> 4;
                const uint32_t b_off = (((kk * 16) / T::SWE) * (T::BN * T::SW) + ((kk * 16) % T::SWE) * 2) >> 4;
                ptx::mma_ss(d_tmem, ptx::desc64(q_lo + a_off, HI), ptx::desc64(k_lo + b_off, HI), IDESC,
                            kk > 0 ? 1u : 0u);
            }
            ptx::tc_commit(bar(T::B_SFULL + r));
            if (j == je - 1) {
                ptx::tc_commit(bar(T::B_QEMPTY + qs));
                ++qi;
            }
        }
    }
    if (!ok) {
        ptx::tc_commit(bar(T::B_DRAIN));
        drain_phase(bar(T::B_DRAIN), 0u, ctl.limit_ns);
    }
}

template <int D, bool BF16>
__device__ void tile_mma_pv(const PagedParams& p, volatile int* ring, uint32_t sbase, uint32_t bar0, uint32_t tmem,
                            const Ctl& ctl) {
    using T = TileTraits<D>;
    auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    constexpr uint32_t IDESC = ptx::idesc_f16(BM, D, BF16, false, true);
    constexpr uint32_t HI = ptx::smem_desc_hi(8 * T::SW, T::SWIZZLE_CODE);
    const uint32_t v_lo0 = ptx::smem_desc_lo(sbase + T::OFF_V, T::BN * T::SW);
    uint32_t g = 0, ntile = 0, fixes[2] = {0, 0};
    bool ok = true;
    for (;; ++ntile) {
        int jb, je, end;
        {
            PagedSeg sg;
            if (!ok || !seg_get<D, false>(ring, sg, ntile, bar, ctl, ok)) break;
            jb = sg.jb, je = sg.je, end = sg.len + sg.nl;
        }
        for (int j = jb; j < je; ++j, ++g) {
            const uint32_t vb = g & 1u, r = rslot<T::SR>(g);
            if (j == jb && ntile > 0 &&
                !wait_phase(bar(T::B_OFREE), (ntile - 1) & 1u, ctl, SITE_O_FREE)) { ok = false; break; }
            if (!wait_phase(bar(T::B_PFULL + r), rphase<T::SR>(g), ctl, SITE_P_FULL)) { ok = false; break; }
            if (!wait_phase(bar(T::B_VFULL + vb), (g >> 1) & 1u, ctl, SITE_V_FULL)) { ok = false; break; }
            if ((j + 1) * T::BN > end) {
                const uint32_t n = vb == 0 ? fixes[0]++ : fixes[1]++;
                if (!wait_phase(bar(T::B_VFIX + vb), n & 1u, ctl, SITE_V_FULL)) { ok = false; break; }
            }
            ptx::tc_fence_after();
            const uint32_t v_lo = v_lo0 + vb * (T::KV_BYTES >> 4);
            const uint32_t a_tmem = tmem + T::TM_S + r * T::BN;
            const uint32_t acc0 = j > jb ? 1u : 0u;
#pragma unroll
            for (int kk = 0; kk < T::BN / 16; ++kk)
                ptx::mma_ts(tmem + T::TM_O, a_tmem + kk * 8, ptx::desc64(v_lo + ((kk * 16 * T::SW) >> 4), HI), IDESC,
                            kk > 0 ? 1u : acc0);
            ptx::tc_commit(bar(T::B_PVDONE + r));
        }
    }
    if (!ok) {
        ptx::tc_commit(bar(T::B_DRAIN + 1));
        drain_phase(bar(T::B_DRAIN + 1), 0u, ctl.limit_ns);
    }
}

// Which of positions k0 .. k0 + 31 new token t sees, as bits (row: its mask words, or nullptr).
__device__ __forceinline__ uint32_t seen_bits(const PagedParams& p, int len, int nl, const uint32_t* row, int t, int k0) {
    const int j0 = k0 - len;  // new token of the first position (negative: before the new tokens)
    const int lim = (row == nullptr ? min(t + 1, nl) : nl) - j0;
    if (lim <= 0) return 0u;
    uint32_t bits = lim >= 32 ? 0xffffffffu : (1u << lim) - 1u;
    if (row != nullptr && j0 > -32) {
        if (j0 >= 0) {
            const int i = j0 >> 5;
            const uint32_t lo = i < p.words ? __ldcg(row + i) : 0u, hi = i + 1 < p.words ? __ldcg(row + i + 1) : 0u;
            bits &= __funnelshift_r(lo, hi, j0 & 31);
        } else {
            bits &= (__ldcg(row) << -j0) | ((1u << -j0) - 1u);
        }
    }
    return bits;
}

// 32 bytes, a whole sector, in one store.
__device__ __forceinline__ void st_global_v8(void* to, const uint32_t* r) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void st_global_v4(void* to, const uint32_t* r) {
    *reinterpret_cast<uint4*>(to) = make_uint4(r[0], r[1], r[2], r[3]);
}

// One softmax warp's share of a finished tile or part: its 32 rows (one a
// lane), columns h * D / NG .. of O / l in the output type, or in fp32 with the
// base-2 log-sum-exps for the merge.  Both go out as the registers hold them,
// 32 bytes of a row at a time.  What does not need O (the sums, the addresses)
// comes before the wait for its last product, done(); false if that ran out.
template <int D, bool BF16, typename Done>
__device__ __forceinline__ bool tile_output(const PagedParams& p, const PagedSeg& sg, uint32_t bar0, uint32_t tmem,
                                            const float* ls, float m, int h, Done done) {
    using T = TileTraits<D>;
    constexpr int COLS = D / T::NG, STEP = COLS < 32 ? COLS : 32;  // columns of this warp, and of a round
    const int lane = threadIdx.x % 32, quad = (threadIdx.x / 32) % 4, row = quad * 32 + lane;
    const uint32_t o_addr = tmem + ((uint32_t)(quad * 32) << 16) + T::TM_O + h * COLS;
    float l = 0.f;
#pragma unroll
    for (int g = 0; g < T::NG; ++g) l += ls[g * BM + row];
    const float inv = l == 0.f ? 0.f : 1.f / l;  // nothing seen: O = 0, lse = -inf
    const bool part = sg.slot >= 0, live = row < sg.rows;
    uint8_t* dst;  // this lane's row: of O, or of the part's first column group
    float* lse;
    if (part) {
        float* slot = p.scratch + (int64_t)sg.slot * p.slot_floats;
        dst = reinterpret_cast<uint8_t*>(slot + ((h * COLS / 8) * p.tile_rows + row) * 8 + h * COLS % 8);
        lse = slot + p.tile_rows * D + row;
    } else {
        const int grow = sg.row0 + row, t = p.by_g(grow), hq = sg.hk * p.G + grow - t * p.G;
        dst = reinterpret_cast<uint8_t*>(static_cast<uint16_t*>(p.o) + (int64_t)sg.z * p.so_z + hq * p.so_h + t * p.so_n + h * COLS);
        lse = p.lse == nullptr ? nullptr : p.lse + ((int64_t)sg.z * p.Hq + hq) * p.T + t;
    }
    if (h == 0 && live && lse != nullptr) {
        const float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
        *lse = part ? lse2 : lse2 * 0.6931471805599453f;
    }
    if (!done()) return false;
    ptx::tc_fence_after();
#pragma unroll 1
    for (int c = 0; c < COLS; c += STEP) {
        uint32_t r[STEP];
        __syncwarp();
        if constexpr (STEP == 32) ptx::tmem_ld32(o_addr + c, r);
        else if constexpr (STEP == 16) ptx::tmem_ld16(o_addr + c, r);
        else if constexpr (STEP == 8) ptx::tmem_ld8(o_addr + c, r);
        else ptx::tmem_ld4(o_addr + c, r);
        if (c + STEP == COLS) {
            // all of this warp's O has been read: the next tile may overwrite it
            ptx::tc_fence_before();
            ptx::mbar_arrive_warp(bar0 + 8u * T::B_OFREE);
        }
        if (!live) continue;
        if (part) {
#pragma unroll
            for (int x = 0; x < STEP; ++x) r[x] = __float_as_uint(__uint_as_float(r[x]) * inv);
            if constexpr (STEP >= 8) {
#pragma unroll
                for (int x = 0; x < STEP; x += 8) st_global_v8(dst + ((c + x) / 8 * p.tile_rows) * 32, r + x);
            } else {
                st_global_v4(dst, r);
            }
        } else {
            uint32_t w[STEP / 2];
#pragma unroll
            for (int x = 0; x < STEP / 2; ++x)
                w[x] = pack2<BF16>(__uint_as_float(r[2 * x]) * inv, __uint_as_float(r[2 * x + 1]) * inv);
            if constexpr (STEP >= 16) {
#pragma unroll
                for (int x = 0; x < STEP / 2; x += 8) {
                    if (p.wide_o) {
                        st_global_v8(dst + c * 2 + x * 4, w + x);
                    } else {
                        st_global_v4(dst + c * 2 + x * 4, w + x);
                        st_global_v4(dst + c * 2 + x * 4 + 16, w + x + 4);
                    }
                }
            } else if constexpr (STEP == 8) {
                st_global_v4(dst, w);
            } else {
                *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
            }
        }
    }
    return true;
}

template <int D, bool BF16>
__device__ void tile_softmax(const PagedParams& p, volatile int* ring, uint32_t bar0, uint32_t tmem,
                             float* hand, float* red, int h, const Ctl& ctl) {
    using T = TileTraits<D>;
    constexpr int BN = T::BN, NG = T::NG, HC = BN / NG;
    static_assert(HC == 32, "a thread holds 32 positions");
    auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    const int quad = (threadIdx.x / 32) % 4;
    const int row = quad * 32 + threadIdx.x % 32;
    const uint32_t lane_addr = (uint32_t)(quad * 32) << 16;
    const float c = p.scale_log2;
    const uint64_t c2 = ptx::pack_f32x2(c, c);
    uint32_t step = 0, ntile = 0;
    for (;; ++ntile) {
        int jb, je, len, nl, tok;
        bool idle;
        const uint32_t* bits_row;
        {
            PagedSeg sg;
            if (!seg_wait<D, true>(ntile, bar, ctl)) return;
            seg_read<D>(ring, sg, ntile);  // (read again for the output: it is not kept in registers)
            if (sg.je == 0) break;
            jb = sg.jb, je = sg.je, len = sg.len, nl = sg.nl;
            tok = min(p.by_g(sg.row0 + row), p.T - 1);
            idle = quad * 32 >= sg.rows;  // none of the warp's rows holds a token
            bits_row = p.mask == nullptr ? nullptr : p.mask + sg.z * p.sm_z + (int64_t)tok * p.words;
        }
        const int masked = len / BN;  // first block that holds a new token, or ends behind the sequence
        float m = -INFINITY, l = 0.f;
        for (int j = jb; j < je; ++j) {
            const uint32_t r = rslot<T::SR>(step);
            const uint32_t b = step & 1u, ph = (step >> 1) & 1u;
            if (!warp_wait_phase(bar(T::B_SFULL + r), rphase<T::SR>(step), ctl, SITE_S_FULL)) return;
            if (idle) {
                // (P of these rows stays what S left there: rows do not mix)
                ptx::mbar_arrive(bar(T::B_RED + b));
                ptx::mbar_arrive(bar(T::B_PFULL + r));
                // not ahead of the others: an arrival for block step + 2 must not count for this one
                if (!warp_wait_phase(bar(T::B_RED + b), ph, ctl, SITE_MAX_XCHG)) return;
                ++step;
                continue;
            }
            ptx::tc_fence_after();
            const uint32_t s_addr = tmem + lane_addr + T::TM_S + r * BN;
            float s[HC];
            {
                uint32_t rr[HC];
                ptx::tmem_ld32(s_addr + h * HC, rr);
#pragma unroll
                for (int x = 0; x < HC; ++x) s[x] = __uint_as_float(rr[x]);
            }
            if (j >= masked) {
                const uint32_t bits = seen_bits(p, len, nl, bits_row, tok, j * BN + h * HC);
#pragma unroll
                for (int x = 0; x < HC; ++x)
                    if (!((bits >> x) & 1u)) s[x] = -INFINITY;
            }
            float mx0 = fmaxf(s[0], s[1]), mx1 = fmaxf(s[2], s[3]);
#pragma unroll
            for (int x = 4; x < HC; x += 4) {
                mx0 = ptx::fmax3(mx0, s[x], s[x + 1]);
                mx1 = ptx::fmax3(mx1, s[x + 2], s[x + 3]);
            }
            const float pmax = fmaxf(mx0, mx1);
            red[(b * NG + h) * BM + row] = pmax;
            ptx::mbar_arrive(bar(T::B_RED + b));
            auto block_max = [&]() {
                float mm = pmax;
#pragma unroll
                for (int g2 = 0; g2 < NG; ++g2) mm = fmaxf(mm, red[(b * NG + g2) * BM + row]);
                return mm * c;
            };
            if (j == jb) {
                if (!warp_wait_phase(bar(T::B_RED + b), ph, ctl, SITE_MAX_XCHG)) return;
                m = row < ring[(ntile % T::SEGS) * (sizeof(SegMsg) / 4) + 8] ? block_max() : INFINITY;
            }
            constexpr int NP = HC / 2;
            uint32_t pk[NP];
            auto exps = [&](float ref) -> uint64_t {
                ref = ref == -INFINITY ? 0.f : ref;  // nothing seen so far: p = 0, not 2^(-inf + inf)
                const uint64_t negm2 = ptx::pack_f32x2(-ref, -ref);
                uint64_t sum2 = ptx::pack_f32x2(0.f, 0.f);
#pragma unroll
                for (int x = 0; x < NP; ++x) {
                    float a0, a1;
                    ptx::unpack_f32x2(ptx::ffma2(ptx::pack_f32x2(s[2 * x], s[2 * x + 1]), c2, negm2), a0, a1);
                    const float p0 = ptx::ex2(a0), p1 = ptx::ex2(a1);
                    sum2 = ptx::fadd2(sum2, ptx::pack_f32x2(p0, p1));
                    pk[x] = pack2<BF16>(p0, p1);
                }
                return sum2;
            };
            uint64_t sum2 = exps(m);
            float alpha = 1.f;
            if (j > jb) {
                if (!warp_wait_phase(bar(T::B_RED + b), ph, ctl, SITE_MAX_XCHG)) return;
                const float m_tile = block_max();
                if (__any_sync(0xffffffffu, m_tile > m + RESCALE_LOG2)) {
                    const float m_new = fmaxf(m, m_tile);
                    alpha = m == -INFINITY ? 0.f : ptx::ex2(m - m_new);
                    m = m_new;
                    sum2 = exps(m);
                    const uint32_t g = step - 1;
                    if (!warp_wait_phase(bar(T::B_PVDONE + rslot<T::SR>(g)), rphase<T::SR>(g), ctl, SITE_PV_DONE))
                        return;
                    ptx::tc_fence_after();
                    rescale_o<D / NG>(tmem + lane_addr + T::TM_O + h * (D / NG), alpha);
                }
            }
            ptx::tmem_st16(s_addr + h * NP, pk);
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            ptx::mbar_arrive(bar(T::B_PFULL + r));
            float sl, sh;
            ptx::unpack_f32x2(sum2, sl, sh);
            l = l * alpha + (sl + sh);
            ++step;
        }
        // The groups share m (the reference is the same for all) and add their l.
        const uint32_t slot = ntile & 1u;
        float* ls = hand + slot * NG * BM;
        ls[h * BM + row] = l;
        ptx::mbar_arrive(bar(T::B_EPIFULL + slot));
        if (!warp_wait_phase(bar(T::B_EPIFULL + slot), (ntile >> 1) & 1u, ctl, SITE_EPI_FULL)) return;
        PagedSeg sg;
        seg_read<D>(ring, sg, ntile);
        const bool written = tile_output<D, BF16>(p, sg, bar0, tmem, ls, m, h, [&]() {
            const uint32_t g = step - 1;
            return warp_wait_phase(bar(T::B_PVDONE + rslot<T::SR>(g)), rphase<T::SR>(g), ctl, SITE_PV_DONE);
        });
        if (!written) return;
        seg_release<D, true>(ntile, bar);
    }
    if (ring[(ntile % T::SEGS) * (sizeof(SegMsg) / 4) + 9] != 0)  // pads, from the end's message
        paged_fill<D>(p, (int)blockIdx.x * 4 * NG + (int)threadIdx.x / 32 - 4, (int)gridDim.x * 4 * NG);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(TileTraits<D>::THREADS, 1)
    fa_paged_tile_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const PagedParams p) {
    using T = TileTraits<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = ptx::smem_addr(smem);
    const uint32_t bar0 = sbase + T::OFF_BAR;
    float* hand = reinterpret_cast<float*>(smem + T::OFF_HAND);
    float* red = reinterpret_cast<float*>(smem + T::OFF_RED);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + T::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + T::OFF_MISC + 4);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (threadIdx.x == 0) {
        for (int i = 0; i < T::NUM_BARS; ++i) ptx::mbar_init(bar0 + 8u * i, T::bar_count(i));
        *abort_flag = 0;
        ptx::fence_mbar_init();
        if (p.P > 0) {
            ptx::prefetch_tmap(&tmQ);
            ptx::prefetch_tmap(&tmK);
            ptx::prefetch_tmap(&tmV);
        }
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_addr(const_cast<uint32_t*>(tmem_slot)), T::TMEM_COLS);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Ctl ctl{abort_flag, p.status, p.wait_limit_ns};
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    volatile int* ring = reinterpret_cast<volatile int*>(smem + T::OFF_SEG);
    PagedWalk walk{};
    bool pads = false;
    // With few sequences the K producer's warp finds the range by itself; else
    // the CTA together.  (The search's area is the roles' hand-over area.)
    if (!p.few || warp == 0)
        walk = paged_range<T::BN, 1>(p, reinterpret_cast<PagedFind<1>*>(hand), (int)blockIdx.x / p.team, 0,
                                     threadIdx.x == 0 && blockIdx.x % p.team == 0, pads);
    if (!p.few) __syncthreads();

    if (warp == 0) {
        tile_producer_qk<D>(&tmQ, &tmK, p, walk, pads, ring, sbase, bar0, ctl);
    } else if (warp == 3) {
        tile_producer_v<D>(&tmV, p, ring, sbase, bar0, ctl);
    } else if (warp == 1) {
        if (lane == 0) tile_mma_qk<D, BF16>(p, ring, sbase, bar0, tmem, ctl);
    } else if (warp == 2) {
        if (lane == 0) tile_mma_pv<D, BF16>(p, ring, sbase, bar0, tmem, ctl);
    } else {
        tile_softmax<D, BF16>(p, ring, bar0, tmem, hand, red, (warp - 4) / 4, ctl);
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, T::TMEM_COLS);
    }
}

}  // namespace fa
