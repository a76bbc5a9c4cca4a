// The weight that cached positions receive from many query rows (a chunk of a prompt, the
// last tokens of one, the accepted tokens of a batch): see fa_score_rows_kernel.cuh.
//
// Sᵀ = K Qᵀ on tcgen05 with the positions as the rows of the product, so that a position
// is a lane of tensor memory and one thread's: the weights that it receives are summed in
// that thread's registers, tile after tile of query rows, and nothing is exchanged until
// the position's tiles are done.  A query row's lse belongs to a column, so every thread
// would need every lse; read from shared memory as broadcasts they took as long as the
// exponentials (both return 128 bytes a cycle to an SM's registers), so -lse / scale goes
// into the product: as three 16-bit pieces, 24 bits and more, against three constants, in
// one more step of 16 of the contraction, the last one (its rounding then is that of the
// result).  A unit of work is a block of KB positions of one (sequence, kv head):
// its K stays in shared memory while the tiles of up to BR query rows that see it stream
// by.  Units are laid end to end, counted in tiles and UNIT_COST for each (a prompt's last
// blocks are seen by few tiles: without it 96 us for the prompts below, with one tile 95), and
// cut into one equal range a CTA (fa_score_sched.cuh); a unit that a cut crosses leaves its
// sums in slots of the workspace, and fa_score_merge_kernel joins them in order.  Units of up
// to four tiles are counted whole and not cut (p.parts is nullptr): the merge costs more than
// it evens out.
//
// Roles: warp 0 walks the range, hands the units on and loads K through the block table
// (a lane a box of rows) and Q; warps 1 and 3 issue the products of every second tile each
// (a thread's waits in front of a tile take as long as the tile's products, and the tensor
// cores' queue does not reach across them); warp 2 stages the lse;
// sixteen warps take the exponentials: a quarter of the lanes each (a warp reaches only its
// own quarter of tensor memory), of one half of the positions, of a group of columns.
// Every wait is bounded as in fa_fwd_kernel.cuh.
//
// What bounds it.  With one tile a unit, DRAM: 32 sequences of 4096-8192 x 128 rows (417 MB)
// take 74 to 77 us, 5.5 to 5.7 TB/s, about 6 of them from launch to the first weights.  With
// many, the sixteen warps: 1600 cycles a tile of 256 positions x 128 rows, of which the two
// warps of a pair spend 1050 on 64 exponentials a thread each and the rest on the wait, the
// load of the scores and the loop; the products take 1150 of them, and the special function
// units, which give a warp's exponential in 4 cycles, 1024.  Four prompts of 1000 to 2000
// tokens after 0 to 3000 positions, 111 GFLOP: 93 us repeated in a graph, 100 to 112 on new
// inputs, 1.19 to 0.99 PFLOP/s, 0.61 to 0.51 of the measured bf16 peak (tensor pipe 56 % busy).  On
// the way there, in us, four prompts of 2000 tokens each (164 GFLOP, 84 us at that peak,
// constant lse, 32 heads): 228 with lse from shared memory and one issuer; 214 with the
// comparisons in a loop of their own; 200 with the halves' slots apart; 186 with two issuers
// and one barrier for scores and lse; 177 with lse in the product and the scores read at once;
// 168 with four slots for Q; 156 with a quarter of the instructions where lse is staged; 136
// with comparisons decided by each warp; 130 with UNIT_COST.  Not multiplying halves that a
// tile does not see: no gain.
//
// These are groups of 4, whose tiles of 32 tokens fill the 128 columns.  A group that does not
// (a tile's tokens are a power of two) pays for the columns left empty, and the warps whose
// column group is not full compare for every tile, since the way without comparisons is laid
// out for 64 columns: four prompts of 2000 tokens, 8 kv heads of D = 128, in us, groups of 4 and 8
// 63 and 115, of 3, 5, 6, 7 and 12 85, 143, 157, 138 and 308.
#pragma once

#include <climits>

#include "fa_fwd_kernel.cuh"
#include "fa_score_sched.cuh"

namespace fa {

template <int D_>
struct ScoreTile {
    static constexpr int D = D_;
    static constexpr int BR = D == 256 ? 64 : 128;       // query rows of a tile, at most
    static constexpr int KH = D == 256 ? 1 : 2;          // products of 128 positions a tile
    static constexpr int KB = 128 * KH;                  // positions of a unit
    static constexpr int SWE = D < 64 ? D : 64;          // elements of a swizzled row chunk
    static constexpr int SW = SWE * 2;
    static constexpr int NCHUNK = D / SWE;
    static constexpr uint32_t SWIZZLE_CODE = SW == 128 ? 2u : SW == 64 ? 4u : 6u;
    static constexpr int HALF_BYTES = 128 * D * 2;
    static constexpr int K_BYTES = KH * HALF_BYTES;
    static constexpr int Q_BYTES = BR * D * 2;
    static constexpr int K_STAGES = 2;
    static constexpr int Q_STAGES = D >= 128 ? 2 : 4;
    // with one slot for K its second one's room holds more of Q (p.long_q)
    static constexpr int Q_MORE = Q_STAGES + K_BYTES / Q_BYTES;
    static constexpr int SR = 512 / (KH * BR) < 4 ? 512 / (KH * BR) : 4;  // score slots in tensor memory
    static constexpr int WARPS = 16;                     // of the exponentials
    static constexpr int LR = 4;                         // lse slots
    static constexpr int NCG = WARPS / 4 / KH;           // column groups
    static constexpr int THREADS = 32 * (4 + WARPS);
    static constexpr int SEGS = 4;
    static constexpr int OFF_K = 0;
    static constexpr int OFF_Q = OFF_K + K_STAGES * K_BYTES;
    static constexpr int QL_BYTES = BR * 32;
    static constexpr int OFF_KL = OFF_Q + Q_STAGES * Q_BYTES;       // [128] the constants of the lse step
    static constexpr int OFF_QL = OFF_KL + 128 * 32;                // [LR][BR] the pieces of -lse / scale
    static constexpr int OFF_LSE = OFF_QL + LR * QL_BYTES;          // [LR][BR] -lse log2 e, where it has no pieces
    static constexpr int OFF_LAST = OFF_LSE + LR * BR * 4;          // [LR][BR] last position seen
    static constexpr int OFF_SUM = OFF_LAST + LR * BR * 4;          // [2][NCG][KB]
    static constexpr int OFF_FLAG = OFF_SUM + 2 * NCG * KB * 4;     // [LR] last position that a tile's first token sees
    static constexpr int OFF_SEG = OFF_FLAG + LR * 4;
    static constexpr int OFF_BAR = OFF_SEG + SEGS * 48;
    static constexpr int B_KFULL = 0;
    static constexpr int B_KEMPTY = B_KFULL + K_STAGES;
    static constexpr int B_QFULL = B_KEMPTY + K_STAGES;
    static constexpr int B_QEMPTY = B_QFULL + Q_MORE;
    static constexpr int B_SFULL = B_QEMPTY + Q_MORE;   // [SR][KH] product done (commit), lse staged (its issuer)
    static constexpr int B_SEMPTY = B_SFULL + SR * KH;    // [SR][KH] scores read (its warps)
    static constexpr int B_LFULL = B_SEMPTY + SR * KH;    // [LR] lse staged
    static constexpr int B_LEMPTY = B_LFULL + LR;         // [LR] lse used (every warp)
    static constexpr int B_SEGFULL = B_LEMPTY + LR;
    static constexpr int B_SEGFREE = B_SEGFULL + SEGS;
    static constexpr int B_SUM = B_SEGFREE + SEGS;        // [2] the groups' sums are there
    static constexpr int B_DRAIN = B_SUM + 2;             // [2] issuers
    static constexpr int NUM_BARS = B_DRAIN + 2;
    static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
    static constexpr int SMEM_USED = OFF_MISC + 16;
    // >= 120 KB keeps one CTA per SM, so no CTA ever waits on another's TMEM
    static constexpr int SMEM_BYTES = (SMEM_USED + 1024) > 120 * 1024 ? SMEM_USED + 1024 : 120 * 1024;
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
    static_assert(SR * KH * BR <= 512, "tensor memory budget");
    static __device__ __forceinline__ uint32_t bar_count(int i) {
        if (i >= B_SEMPTY && i < B_SEMPTY + SR * KH) return WARPS / KH;
        if (i >= B_SFULL && i < B_SFULL + SR * KH) return 2;
        if (i >= B_LEMPTY && i < B_LEMPTY + LR) return WARPS;
        if ((i >= B_KEMPTY && i < B_KEMPTY + K_STAGES) || (i >= B_QEMPTY && i < B_QEMPTY + Q_MORE)) return 2;  // issuers
        if (i >= B_SEGFREE && i < B_SEGFREE + SEGS) return 3 + WARPS;
        if (i >= B_SUM && i < B_SUM + 2) return WARPS;
        return 1;
    }
};

namespace scoret {

// The slots of K and Q: two and Q_STAGES, or (p.long_q) one and Q_MORE; Q's come behind K's.
template <int D>
struct Slots {
    using T = ScoreTile<D>;
    uint32_t k, q;
    int off_q;
    __device__ __forceinline__ explicit Slots(const ScoreParams& p)
        : k(p.long_q ? 1 : T::K_STAGES), q(p.long_q ? T::Q_MORE : T::Q_STAGES), off_q(T::OFF_K + (int)k * T::K_BYTES) {}
};
// A place in a ring of n slots: its slot, and how often it has come around.
struct Place {
    uint32_t slot = 0, round = 0;
    __device__ __forceinline__ void next(uint32_t n) {
        if (++slot == n) {
            slot = 0;
            ++round;
        }
    }
};

// A unit's part in a range: tiles i0 .. i1 - 1 of those that see its block.
struct Unit {
    int z, hk, j, i0, i1, slot, len, nl;  // i1 = 0: the end; slot -1: all of the unit's tiles
    int keep;                             // the next unit starts with the Q tile that this one ends with
};

// What a unit costs besides its tiles, in tiles: the way of its K to the first product.
constexpr int UNIT_COST = 2;
// Tiles of a sequence's rows, and which of them is the first that sees block j: the one
// with token j KB - len.
template <int D>
struct Shape {
    using T = ScoreTile<D>;
    int nb, nt, lag;  // blocks, tiles, ceil(len / tokens)
    __device__ __forceinline__ Shape(const ScoreParams& p, const ScoreLen& s) {
        nb = (s.len + s.nl + T::KB - 1) / T::KB;
        nt = (s.nl + p.tokens - 1) >> p.token_shift;
        lag = (s.len + p.tokens - 1) >> p.token_shift;
        if (s.nl == 0) {
            nt = 1;                       // only the scores so far
            lag = INT_MAX;
            if (p.decay == 1.f) nb = 0;   // which stay as they are
        }
    }
    // r = KB / tokens tiles from a block to the next
    __device__ __forceinline__ int first(const ScoreParams& p, int j) const {
        return (int)max((int64_t)0, (int64_t)j * (T::KB >> p.token_shift) - lag);
    }
    // cost of blocks 0 .. j - 1, in tiles and UNIT_COST for each, or (units are not cut) the blocks
    __device__ __forceinline__ int64_t before(const ScoreParams& p, int j) const {
        if (p.parts == nullptr) return j;
        const int64_t r = T::KB >> p.token_shift, j0 = lag / r + 1;  // the first block with first() > 0
        int64_t n = (int64_t)j * (nt + UNIT_COST);
        if (j > j0) n -= r * ((int64_t)(j - 1) * j - j0 * (j0 - 1)) / 2 - (int64_t)lag * (j - j0);
        return n;
    }
};

// Where a range starts, for the merge.
struct alignas(16) Cut {
    int z, hk, j, skip;   // tiles of the unit in front of the range
    int tiles, len, end, pad;
    int64_t start, total; // the unit's next tile and the end of all, in cost
};

}  // namespace scoret

template <int D>
struct ScoreWalk {
    using T = ScoreTile<D>;
    ScorePlace w;
    int hk, j, i;  // the next one of the unit's cost: UNIT_COST, then its tiles from first()
    __device__ __forceinline__ void start(const ScoreParams& p, const ScorePlace& place) {
        w = place;
        if (w.left == 0) return;
        const scoret::Shape<D> s(p, w.s);
        const int64_t per = s.before(p, s.nb);
        hk = (int)(w.at / per);
        const int64_t rem = w.at - hk * per;
        int lo = 0, hi = s.nb;  // before(lo) <= rem < before(hi)
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (s.before(p, mid) <= rem) lo = mid;
            else hi = mid;
        }
        j = lo;
        i = (int)(rem - s.before(p, lo));
    }
    // the next unit of the range; false at its end
    __device__ __forceinline__ bool next(const ScoreParams& p, scoret::Unit& u) {
        while (w.left > 0) {
            const scoret::Shape<D> s(p, w.s);
            const int first = s.first(p, j), tiles = s.nt - first, ahead = p.parts == nullptr ? 0 : scoret::UNIT_COST;
            const int take = p.parts == nullptr ? tiles : (int)min((int64_t)(ahead + tiles - i), w.left);
            const int lo = max(i - ahead, 0), hi = max(i + take - ahead, 0);
            u.z = w.z, u.hk = hk, u.j = j, u.len = w.s.len, u.nl = w.s.nl;
            u.i0 = first + lo;
            u.i1 = first + hi;
            u.slot = lo == 0 && hi == tiles ? -1 : 2 * (int)blockIdx.x + (lo > 0 ? 0 : 1);
            w.left -= p.parts == nullptr ? 1 : take;
            i = 0;
            if (w.left > 0 && ++j == s.nb) {
                j = 0;
                if (++hk == p.Hkv) {
                    hk = 0;
                    do w.s = score_len(p, ++w.z);
                    while (scoret::Shape<D>(p, w.s).nb == 0);
                }
            }
            if (hi > lo) return true;  // (a range may end in front of a unit's first tile)
        }
        return false;
    }
};

namespace scoret {

template <int D, typename Bar>
__device__ __forceinline__ void put(volatile int* ring, const Unit& u, uint32_t n, Bar bar) {
    using T = ScoreTile<D>;
    volatile int* s = ring + (n % T::SEGS) * 12;
    if (threadIdx.x % 32 == 0) {
        s[0] = u.z, s[1] = u.hk, s[2] = u.j, s[3] = u.i0, s[4] = u.i1, s[5] = u.slot, s[6] = u.len, s[7] = u.nl, s[8] = u.keep;
        ptx::mbar_arrive(bar(T::B_SEGFULL + n % T::SEGS));
    }
    __syncwarp();
}
// The n-th unit, for a whole warp (WARP) or its one active lane; false at the end, or (ok
// false) when the wait ran out.
template <int D, bool WARP, typename Bar>
__device__ __forceinline__ bool get(volatile const int* ring, Unit& u, uint32_t n, Bar bar, const Ctl& ctl, bool& ok) {
    using T = ScoreTile<D>;
    const uint32_t full = bar(T::B_SEGFULL + n % T::SEGS), parity = (n / T::SEGS) & 1u;
    ok = WARP ? warp_wait_phase(full, parity, ctl, SITE_SEG_FULL) : wait_phase(full, parity, ctl, SITE_SEG_FULL);
    if (!ok) return false;
    volatile const int* s = ring + (n % T::SEGS) * 12;
    u.z = s[0], u.hk = s[1], u.j = s[2], u.i0 = s[3], u.i1 = s[4], u.slot = s[5], u.len = s[6], u.nl = s[7], u.keep = s[8];
    if (WARP) __syncwarp();
    if (!WARP || threadIdx.x % 32 == 0) ptx::mbar_arrive(bar(T::B_SEGFREE + n % T::SEGS));
    return u.i1 > 0;
}

// A tile's Q is loaded unless it is the one before (blocks of a head whose rows are one tile).
template <int D>
__device__ void walk_and_load(const CUtensorMap* tmQ, const CUtensorMap* tmK, const ScoreParams& p, ScoreWalk<D> walk,
                              volatile int* ring, uint32_t sbase, uint32_t bar0, const Ctl& ctl) {
    using T = ScoreTile<D>;
    auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    const int lane = threadIdx.x % 32;
    // K passes once where all rows are one tile; else the units of a head are not far apart
    const uint64_t policy = ptx::policy_evict_first(), policy_q = ptx::policy_evict_last();
    const Slots<D> slots(p);
    uint32_t n = 0;
    Place k, q;
    bool ok = true, withheld = false, loaded = false;  // loaded: the unit's first Q tile is there
    Unit u{}, after{};
    bool have = walk.next(p, u);
    while (ok) {
        const bool more = have && walk.next(p, after);
        u.keep = more && after.z == u.z && after.hk == u.hk && after.i0 == u.i1 - 1;
        if (n >= (uint32_t)T::SEGS &&
            !warp_wait_phase(bar(T::B_SEGFREE + n % T::SEGS), (n / T::SEGS - 1) & 1u, ctl, SITE_SEG_FREE)) {
            ok = false;
            break;
        }
        if (!have) u.i1 = 0;
        put<D>(ring, u, n++, bar);
        if (!have) break;
        // lane b: the box of positions j KB + b box_rows .. (without a new token K has no say: its
        // products, with whatever is in its slot, are of rows that see nothing)
        const int end = u.nl > 0 ? u.len + u.nl : 0, k0 = u.j * T::KB + lane * p.box_rows;
        const bool there = lane * p.box_rows < T::KB && k0 < end;
        int page = p.P, slot = 0;
        if (there) {
            const int col = p.by_page(k0);
            slot = k0 - col * p.page;
            page = ldi(p.table + (int64_t)u.z * p.st_z + col);
            if ((unsigned)page >= (unsigned)p.P) {
                bad_page(p.status, SITE_PAGE_SCORE);
                page = p.P;  // outside the map: zeros
            }
        }
        if (!warp_wait_phase(bar(T::B_KEMPTY + k.slot), (k.round & 1u) ^ 1u, ctl, SITE_K_EMPTY)) { ok = false; break; }
        if (p.inject_stall && blockIdx.x == 0 && !withheld) {
            withheld = true;  // never issued: the wait for this block must time out
        } else {
            const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, there));
            if (lane == 0) ptx::mbar_arrive_expect_tx(bar(T::B_KFULL + k.slot), boxes * p.box_rows * T::SW * T::NCHUNK);
            __syncwarp();
            if (there) {
                const int r = lane * p.box_rows;
                const uint32_t dst = sbase + T::OFF_K + k.slot * T::K_BYTES + (r / 128) * T::HALF_BYTES + (r % 128) * T::SW;
                for (int c = 0; c < T::NCHUNK; ++c)
                    ptx::tma_load_4d(dst + c * (128 * T::SW), tmK, bar(T::B_KFULL + k.slot), c * T::SWE, slot, u.hk, page, policy);
            }
        }
        k.next(slots.k);
        for (int i = u.i0 + (loaded ? 1 : 0); i < u.i1; ++i) {
            if (!warp_wait_phase(bar(T::B_QEMPTY + q.slot), (q.round & 1u) ^ 1u, ctl, SITE_Q_EMPTY)) { ok = false; break; }
            if (lane == 0) {
                ptx::mbar_arrive_expect_tx(bar(T::B_QFULL + q.slot), (uint32_t)p.tile_rows * T::SW * T::NCHUNK);
                const uint32_t dst = sbase + slots.off_q + q.slot * T::Q_BYTES;
                for (int c = 0; c < T::NCHUNK; ++c)
                    ptx::tma_load_4d(dst + c * (T::BR * T::SW), tmQ, bar(T::B_QFULL + q.slot), c * T::SWE, u.hk * p.G,
                                     i << p.token_shift, u.z, policy_q);
            }
            __syncwarp();
            q.next(slots.q);
        }
        loaded = u.keep;
        u = after;
        have = more;
    }
    if (!ok) {
        // every slot's last copy
        for (uint32_t i = 0; i < slots.q; ++i)
            if (i < q.slot || q.round > 0)
                drain_phase(bar(T::B_QFULL + i), (i < q.slot ? q.round : q.round - 1) & 1u, ctl.limit_ns);
        for (uint32_t i = 0; i < slots.k; ++i)
            if (i < k.slot || k.round > 0)
                drain_phase(bar(T::B_KFULL + i), (i < k.slot ? k.round : k.round - 1) & 1u, withheld ? ctl.limit_ns / 64 : ctl.limit_ns);
    }
}

// The products of every second tile (issuer 0 or 1).  K and Q are released by both: a
// commit waits for the products of its own thread only.  Both also wait for every copy of
// K and Q, whoever's tile it is for: an issuer that did not could release a slot's next
// round before the other one has released this one.
template <int D, bool BF16>
__device__ void multiply(const ScoreParams& p, volatile int* ring, uint32_t sbase, uint32_t bar0, uint32_t tmem,
                         uint32_t issuer, const Ctl& ctl) {
    using T = ScoreTile<D>;
    auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    const uint32_t IDESC = ptx::idesc_f16(128, p.tile_cols, BF16, false, false);
    constexpr uint32_t HI = ptx::smem_desc_hi(8 * T::SW, T::SWIZZLE_CODE), HI_L = ptx::smem_desc_hi(8 * 32, 6);
    const Slots<D> slots(p);
    const uint32_t k_lo0 = ptx::smem_desc_lo(sbase + T::OFF_K, 16), q_lo0 = ptx::smem_desc_lo(sbase + slots.off_q, 16);
    const uint64_t kl = ptx::desc64(ptx::smem_desc_lo(sbase + T::OFF_KL, 16), HI_L);
    const uint32_t ql_lo = ptx::smem_desc_lo(sbase + T::OFF_QL, 16);
    uint32_t g = 0;  // tiles
    Place k, q;
    bool ok = true;
    Unit u;
    for (uint32_t n = 0; get<D, false>(ring, u, n, bar, ctl, ok); ++n) {
        if (!wait_phase(bar(T::B_KFULL + k.slot), k.round & 1u, ctl, SITE_K_FULL)) { ok = false; break; }
        for (int i = u.i0; i < u.i1; ++i, ++g) {
            if (!wait_phase(bar(T::B_QFULL + q.slot), q.round & 1u, ctl, SITE_Q_FULL)) { ok = false; break; }
            if ((g & 1u) == issuer) {
                const uint32_t r = g % T::SR, lr = g % T::LR;
                if (!wait_phase(bar(T::B_LFULL + lr), (g / T::LR) & 1u, ctl, SITE_EPI_FULL)) { ok = false; break; }
                const uint32_t q_lo = q_lo0 + q.slot * (T::Q_BYTES >> 4);
                const uint64_t ql = ptx::desc64(ql_lo + lr * (T::QL_BYTES >> 4), HI_L);
#pragma unroll
                for (int h = 0; h < T::KH; ++h) {
                    const uint32_t full = bar(T::B_SFULL + r * T::KH + h);
                    if (!wait_phase(bar(T::B_SEMPTY + r * T::KH + h), ((g / T::SR) & 1u) ^ 1u, ctl, SITE_S_FREE)) { ok = false; break; }
                    ptx::tc_fence_after();
                    const uint32_t k_lo = k_lo0 + ((k.slot * T::K_BYTES + h * T::HALF_BYTES) >> 4);
                    const uint32_t d = tmem + (r * T::KH + h) * T::BR;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t in = ((kk * 16) % T::SWE) * 2, chunk = (kk * 16) / T::SWE;
                        ptx::mma_ss(d, ptx::desc64(k_lo + ((chunk * (128 * T::SW) + in) >> 4), HI),
                                    ptx::desc64(q_lo + ((chunk * (T::BR * T::SW) + in) >> 4), HI), IDESC, kk > 0 ? 1u : 0u);
                    }
                    ptx::mma_ss(d, kl, ql, IDESC, 1u);
                    ptx::mbar_arrive(full);  // (hands on what stage_lse wrote)
                    ptx::tc_commit(full);
                }
                if (!ok) break;
            }
            if (i + 1 < u.i1 || u.keep == 0) {
                ptx::tc_commit(bar(T::B_QEMPTY + q.slot));
                q.next(slots.q);
            }
        }
        if (!ok) break;
        ptx::tc_commit(bar(T::B_KEMPTY + k.slot));
        k.next(slots.k);
    }
    // everything issued here has arrived before the CTA ends
    ptx::tc_commit(bar(T::B_DRAIN + issuer));
    drain_phase(bar(T::B_DRAIN + issuer), 0u, ctl.limit_ns);
}

// The lse step of the contraction: 32 bytes a row, in the 32-byte swizzle's order; this is
// where the first 16 of row r are (the others are zeros).
__device__ __forceinline__ uint32_t l_piece(int r) { return (uint32_t)(r * 32 + (((r >> 2) & 1) << 4)); }
// x as a + f b + f f c with 16-bit a, b, c: bf16 has fp32's range (f = 1); fp16 pieces keep
// their magnitude (f = 2^-11).  {a | b << 16, c}
template <bool BF16>
__device__ __forceinline__ void split3(float x, uint32_t& w0, uint32_t& w1) {
    if constexpr (BF16) {
        const __nv_bfloat16 a = __float2bfloat16_rn(x);
        const float r = x - __bfloat162float(a);
        const __nv_bfloat16 b = __float2bfloat16_rn(r), c = __float2bfloat16_rn(r - __bfloat162float(b));
        w0 = __bfloat16_as_ushort(a) | (uint32_t)__bfloat16_as_ushort(b) << 16;
        w1 = __bfloat16_as_ushort(c);
    } else {
        const __half a = __float2half_rn(x);
        const float r = (x - __half2float(a)) * 2048.f;
        const __half b = __float2half_rn(r), c = __float2half_rn((r - __half2float(b)) * 2048.f);
        w0 = __half_as_ushort(a) | (uint32_t)__half_as_ushort(b) << 16;
        w1 = __half_as_ushort(c);
    }
}
template <bool BF16>
__device__ __forceinline__ void constants3(uint32_t& w0, uint32_t& w1) {  // 1, f, f f
    w0 = BF16 ? 0x3f803f80u : 0x10003c00u;
    w1 = BF16 ? 0x3f80u : 0x0004u;
}

// Each tile's lse and the last position that each of its rows sees, a warp, the loads two
// tiles ahead.  A row that does not count (no token, nothing seen) sees nothing; columns
// behind the tile's rows are products with zeros.  A tile all of whose rows are tokens, their
// lse in pieces, hands on the last position that its first token sees: a warp whose positions
// are all seen by its columns' first token needs no comparisons, and one whose positions are
// seen by none has nothing to add (on a prompt's diagonal most warps are either: with one
// answer for the whole block the ranges there took 159000 cycles, the others 110000).
template <int D, bool BF16>
__device__ void stage_lse(const ScoreParams& p, volatile int* ring, uint8_t* smem, uint32_t bar0, const Ctl& ctl) {
    using T = ScoreTile<D>;
    auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    const int lane = threadIdx.x % 32;
    constexpr int N = T::BR / 32;
    struct Tile {
        float l[N];
        int j, i, len;
        bool there, whole;  // whole: each of its rows has a token
    };
    // this lane's columns: row c of a tile is head c % G of token c / G
    int tok[N];
    int64_t off[N];
#pragma unroll
    for (int x = 0; x < N; ++x) {
        const int c = x * 32 + lane;
        tok[x] = c < p.tile_rows ? p.by_g(c) : INT_MAX;
        off[x] = c < p.tile_rows ? (int64_t)(c - tok[x] * p.G) * p.T + tok[x] : 0;
    }
    uint32_t n = 0, g = 0;
    bool ok = true;
    Unit u{};
    const float* from = p.lse;
    auto fetch = [&](Tile& t) {
        if (u.i0 == u.i1) {
            t.there = ok && (n == 0 || u.i1 > 0) && get<D, true>(ring, u, n++, bar, ctl, ok);
            if (!t.there) return;
            from = p.lse + ((int64_t)u.z * p.Hq + u.hk * p.G) * p.T;
        }
        t.there = true;
        t.j = u.j, t.i = u.i0++, t.len = u.len;
        const int t0 = t.i << p.token_shift, left = u.nl - t0;
        t.whole = left >= p.tokens;
#pragma unroll
        for (int x = 0; x < N; ++x) {
            t.l[x] = -INFINITY;
            if (tok[x] < left) t.l[x] = __ldcg(from + off[x] + t0);
        }
    };
    // -lse / scale in three pieces, unless it is out of the type's range, infinite or NaN, or the
    // scale so large that what the last piece leaves out matters: in fp16 up to 2^-25 f f = 2^-47,
    // at LARGEST 2^-31 of an exponent; bf16 has bits down to 2^-133.
    const float per_scale = -1.f / p.scale;
    constexpr float LARGEST = BF16 ? 0x1p96f : 0x1p16f;
    const float limit = fabsf(p.scale) <= LARGEST ? (BF16 ? 1e38f : 60000.f) : -1.f;
    int* flags = reinterpret_cast<int*>(smem + T::OFF_FLAG);
    auto finish = [&](const Tile& t) -> bool {
        const int last0 = t.len + (t.i << p.token_shift), need = (t.j + 1) * T::KB - 1;
        bool pure = p.tile_rows == p.tile_cols && t.whole;  // every row a token, its lse in pieces
        uint32_t w0[N], w1[N];
#pragma unroll
        for (int x = 0; x < N; ++x) {
            const float q = t.l[x] * per_scale;
            const bool pieces = fabsf(q) <= limit;
            w0[x] = w1[x] = 0u;
            if (pieces) split3<BF16>(q, w0[x], w1[x]);
            pure &= pieces || tok[x] == INT_MAX;
        }
        pure = __all_sync(0xffffffffu, pure);
        const uint32_t r = g % T::LR;
        if (!warp_wait_phase(bar(T::B_LEMPTY + r), ((g / T::LR) & 1u) ^ 1u, ctl, SITE_S_FREE)) return false;
        const uint32_t ql = ptx::smem_addr(smem + T::OFF_QL) + r * T::QL_BYTES;
#pragma unroll
        for (int x = 0; x < N; ++x) ptx::st_shared_v4(ql + l_piece(x * 32 + lane), w0[x], w1[x], 0u, 0u);
        // (a group with fewer columns takes the comparisons' way)
        if (!pure || last0 < need || p.tile_cols < T::BR) {
            float* ls = reinterpret_cast<float*>(smem + T::OFF_LSE) + r * T::BR;
            int* la = reinterpret_cast<int*>(smem + T::OFF_LAST) + r * T::BR;
#pragma unroll
            for (int x = 0; x < N; ++x) {
                const int c = x * 32 + lane;
                const bool pieces = fabsf(t.l[x] * per_scale) <= limit;
                ls[c] = pieces ? 0.f : -t.l[x] * 1.4426950408889634f;
                la[c] = t.l[x] != -INFINITY ? last0 + tok[x] : -1;
            }
        }
        if (lane == 0) flags[r] = pure ? last0 : INT_MIN / 2;
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive_warp(bar(T::B_LFULL + r));
        ++g;
        return true;
    };
    Tile a, b;
    fetch(a);
    fetch(b);
    while (a.there) {
        if (!finish(a)) return;
        fetch(a);
        if (!b.there) break;
        if (!finish(b)) return;
        fetch(b);
    }
}

// The weights of 16 columns of a position's scores, added to two pairs of sums.
__device__ __forceinline__ void add16(const uint32_t (&s)[16], const float4* ls, const int4* la, int pos, uint64_t c2,
                                      uint64_t& sum0, uint64_t& sum1) {
#pragma unroll
    for (int x = 0; x < 16; x += 4) {
        const float4 l = ls[x / 4];
        const int4 t = la[x / 4];
        float a[4];
        ptx::unpack_f32x2(ptx::ffma2(ptx::pack_f32x2(__uint_as_float(s[x]), __uint_as_float(s[x + 1])), c2,
                                     ptx::pack_f32x2(l.x, l.y)), a[0], a[1]);
        ptx::unpack_f32x2(ptx::ffma2(ptx::pack_f32x2(__uint_as_float(s[x + 2]), __uint_as_float(s[x + 3])), c2,
                                     ptx::pack_f32x2(l.z, l.w)), a[2], a[3]);
        a[0] = pos <= t.x ? a[0] : -INFINITY;
        a[1] = pos <= t.y ? a[1] : -INFINITY;
        a[2] = pos <= t.z ? a[2] : -INFINITY;
        a[3] = pos <= t.w ? a[3] : -INFINITY;
        sum0 = ptx::fadd2(sum0, ptx::pack_f32x2(ptx::ex2(a[0]), ptx::ex2(a[1])));
        sum1 = ptx::fadd2(sum1, ptx::pack_f32x2(ptx::ex2(a[2]), ptx::ex2(a[3])));
    }
}
__device__ __forceinline__ void load_scores(uint32_t s_addr, uint32_t (&s)[64]) { ptx::tmem_ld64(s_addr, s); }
__device__ __forceinline__ void load_scores(uint32_t s_addr, uint32_t (&s)[16]) { ptx::tmem_ld16(s_addr, s); }

template <int D>
__device__ void weigh(const ScoreParams& p, volatile int* ring, uint8_t* smem, uint32_t bar0, uint32_t tmem, const Ctl& ctl) {
    using T = ScoreTile<D>;
    constexpr int COLS = T::BR / T::NCG;  // columns of a group, at most
    auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    const int w = threadIdx.x / 32 - 4, lane = threadIdx.x % 32;
    const int quad = w % 4, half = w / 4 % T::KH, cg = w / 4 / T::KH;
    const int key = half * 128 + quad * 32 + lane;
    const uint32_t lane_addr = (uint32_t)(quad * 32) << 16;
    const float c = p.scale * 1.4426950408889634f;
    const uint64_t c2 = ptx::pack_f32x2(c, c);
    // columns of a group, a multiple of 16, and this one's (the last may have fewer)
    const int group = (p.tile_cols + 16 * T::NCG - 1) / (16 * T::NCG) * 16;
    const int col0 = min(cg * group, p.tile_cols), cols = min(group, p.tile_cols - col0);
    // A block at `at` of a tile whose first token sees `last`: at <= last + plain_by, the group's
    // first token sees the warp's last position; at > last + none_by, its last token not the first.
    const int plain_by = cols == COLS ? p.by_g(col0) - half * 128 - quad * 32 - 31 : INT_MIN / 2;
    const int none_by = p.by_g(col0 + max(cols, 1) - 1) - half * 128 - quad * 32;
    float* sums = reinterpret_cast<float*>(smem + T::OFF_SUM);
    const int* flags = reinterpret_cast<const int*>(smem + T::OFF_FLAG);
    uint32_t g = 0;
    bool ok = true, ready = false;  // ready: the next scores were there when last asked
    Unit u;
    for (uint32_t n = 0; get<D, true>(ring, u, n, bar, ctl, ok); ++n) {
        const int pos = u.j * T::KB + key;
        float* score = p.scores + (int64_t)u.z * p.ss_z + u.hk * p.ss_h + pos;
        float old = 0.f;
        if (cg == 0 && u.slot < 0 && p.decay != 0.f && pos < u.len) old = __ldcg(score) * p.decay;
        uint64_t sum0 = ptx::pack_f32x2(0.f, 0.f), sum1 = sum0;
        for (int i = u.i0; i < u.i1; ++i, ++g) {
            const uint32_t r = g % T::SR, lr = g % T::LR;
            const uint32_t s_addr = tmem + lane_addr + (r * T::KH + half) * T::BR + col0;
            const float4* ls = reinterpret_cast<const float4*>(smem + T::OFF_LSE + (lr * T::BR + col0) * 4);
            const int4* la = reinterpret_cast<const int4*>(smem + T::OFF_LAST + (lr * T::BR + col0) * 4);
            if (!__all_sync(0xffffffffu, ready) &&
                !warp_wait_phase(bar(T::B_SFULL + r * T::KH + half), (g / T::SR) & 1u, ctl, SITE_S_FULL)) return;
            ptx::tc_fence_after();
            const int last = flags[lr], at = u.j * T::KB;
            const bool plain = at <= last + plain_by;
            const uint32_t next = bar(T::B_SFULL + (g + 1) % T::SR * T::KH + half), next_ph = ((g + 1) / T::SR) & 1u;
            if (plain) {
                // All of this warp's scores at once, so that their slot is free before they
                // are used, and no comparisons (in one loop with the others they took 6.9
                // instructions a weight).
                uint32_t s[COLS];
                load_scores(s_addr, s);
                ptx::tc_fence_before();
                __syncwarp();
                if (lane < 2) ptx::mbar_arrive(lane == 0 ? bar(T::B_SEMPTY + r * T::KH + half) : bar(T::B_LEMPTY + lr));
                // (asked now, looked at after the exponentials)
                ready = ptx::mbar_test_wait(next, next_ph);
#pragma unroll
                for (int x = 0; x < COLS; x += 4) {
                    float a[4];
                    ptx::unpack_f32x2(ptx::fmul2(ptx::pack_f32x2(__uint_as_float(s[x]), __uint_as_float(s[x + 1])), c2), a[0], a[1]);
                    ptx::unpack_f32x2(ptx::fmul2(ptx::pack_f32x2(__uint_as_float(s[x + 2]), __uint_as_float(s[x + 3])), c2), a[2], a[3]);
                    sum0 = ptx::fadd2(sum0, ptx::pack_f32x2(ptx::ex2(a[0]), ptx::ex2(a[1])));
                    sum1 = ptx::fadd2(sum1, ptx::pack_f32x2(ptx::ex2(a[2]), ptx::ex2(a[3])));
                }
            } else if (last >= 0 && at > last + none_by) {
                __syncwarp();
                if (lane < 2) ptx::mbar_arrive(lane == 0 ? bar(T::B_SEMPTY + r * T::KH + half) : bar(T::B_LEMPTY + lr));
                ready = ptx::mbar_test_wait(next, next_ph);
            } else {
#pragma unroll 1
                for (int c0 = 0; c0 < cols; c0 += 16) {
                    uint32_t s[16];
                    ptx::tmem_ld16(s_addr + c0, s);
                    add16(s, ls + c0 / 4, la + c0 / 4, pos, c2, sum0, sum1);
                }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane < 2) ptx::mbar_arrive(lane == 0 ? bar(T::B_SEMPTY + r * T::KH + half) : bar(T::B_LEMPTY + lr));
                ready = ptx::mbar_test_wait(next, next_ph);
            }
        }
        float s0, s1, s2, s3;
        ptx::unpack_f32x2(sum0, s0, s1);
        ptx::unpack_f32x2(sum1, s2, s3);
        float all = (s0 + s1) + (s2 + s3);
        if constexpr (T::NCG > 1) {
            // the groups' sums, in order; the slot's parity and this wait keep a warp from
            // writing where another has not read yet
            float* mine = sums + (n & 1u) * T::NCG * T::KB + key;
            mine[cg * T::KB] = all;
            ptx::mbar_arrive_warp(bar(T::B_SUM + (n & 1u)));
            if (!warp_wait_phase(bar(T::B_SUM + (n & 1u)), (n >> 1) & 1u, ctl, SITE_MAX_XCHG)) return;
            all = mine[0];
#pragma unroll
            for (int x = 1; x < T::NCG; ++x) all += mine[x * T::KB];
        }
        if (cg == 0) {
            if (u.slot >= 0) p.parts[(int64_t)u.slot * T::KB + key] = all;
            else if (pos < u.len + u.nl) *score = old + all;
        }
    }
}

}  // namespace scoret

template <int D, bool BF16>
__global__ void __launch_bounds__(ScoreTile<D>::THREADS, 1)
    fa_score_tile_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ ScoreParams p) {
    using T = ScoreTile<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = ptx::smem_addr(smem), bar0 = sbase + T::OFF_BAR;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + T::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + T::OFF_MISC + 4);
    volatile int* ring = reinterpret_cast<volatile int*>(smem + T::OFF_SEG);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        for (int i = 0; i < T::NUM_BARS; ++i) ptx::mbar_init(bar0 + 8u * i, T::bar_count(i));
        *abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&tmQ);
        ptx::prefetch_tmap(&tmK);
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_addr(const_cast<uint32_t*>(tmem_slot)), 512);
        ptx::tmem_relinquish();
    }
    // the lse step's constants and zeros
    for (int i = threadIdx.x; i < 128 * 2 + T::LR * T::BR * 2; i += T::THREADS)
        ptx::st_shared_v4(sbase + T::OFF_KL + i * 16, 0u, 0u, 0u, 0u);
    // rows of Q's slots behind the tile's: zeros (no copy writes them)
    if (p.tile_rows < p.tile_cols) {
        constexpr int PR = T::SW / 16;
        const scoret::Slots<D> slots(p);
        const int n = (p.tile_cols - p.tile_rows) * PR;
        for (int i = threadIdx.x; i < n * (int)slots.q * T::NCHUNK; i += T::THREADS)
            ptx::st_shared_v4(sbase + slots.off_q + (i / n) * (T::BR * T::SW) + p.tile_rows * T::SW + (i % n) * 16, 0u, 0u, 0u, 0u);
    }
    __syncthreads();
    if (threadIdx.x < 128) {
        uint32_t w0, w1;
        scoret::constants3<BF16>(w0, w1);
        ptx::st_shared_v4(sbase + T::OFF_KL + scoret::l_piece(threadIdx.x), w0, w1, 0u, 0u);
    }
    ptx::fence_proxy_async_smem();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Ctl ctl{abort_flag, p.status, p.wait_limit_ns};
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    // (the search's area is that of the sums)
    auto* find = reinterpret_cast<ScoreFind<1>*>(smem + T::OFF_SUM);
    static_assert(sizeof(ScoreFind<1>) <= 2 * T::NCG * T::KB * 4, "the range search fits the sums' area");
    auto count = [&](const ScoreLen& s) {
        const scoret::Shape<D> x(p, s);
        return x.before(p, x.nb) * p.Hkv;
    };
    ScoreWalk<D> walk{};
    if (p.Z > 32 || warp == 0) {
        int64_t start, total;
        const ScorePlace place = score_place<1>(p, find, (int)blockIdx.x, 0, (int)gridDim.x, count, &start, &total);
        walk.start(p, place);
        if (p.parts != nullptr && threadIdx.x == 0) {
            scoret::Cut cut{};
            cut.z = -1;
            if (place.left > 0) {
                const scoret::Shape<D> s(p, place.s);
                const int past = walk.i - scoret::UNIT_COST;  // tiles in front, or (negative) cost before the first
                cut = scoret::Cut{place.z, walk.hk, walk.j, max(past, 0), s.nt - s.first(p, walk.j), place.s.len,
                                  place.s.len + place.s.nl, 0, start, total};
            }
            static_cast<scoret::Cut*>(p.cuts)[blockIdx.x] = cut;
        }
    }
    if (p.Z > 32) __syncthreads();

    if (warp == 0) scoret::walk_and_load<D>(&tmQ, &tmK, p, walk, ring, sbase, bar0, ctl);
    else if (warp == 2) scoret::stage_lse<D, BF16>(p, ring, smem, bar0, ctl);
    else if (warp < 4) { if (lane == 0) scoret::multiply<D, BF16>(p, ring, sbase, bar0, tmem, warp / 2, ctl); }
    else scoret::weigh<D>(p, ring, smem, bar0, tmem, ctl);

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// Block b - 1 looks at the cut between ranges b - 1 and b.  If it is the first one inside
// its unit, the unit's parts -- slot 2 c + 1 of the range c that it starts in, slots 2 c
// of the following ones -- are added in order.
template <int D>
__global__ void __launch_bounds__(ScoreTile<D>::KB) fa_score_merge_kernel(const ScoreParams p) {
    using T = ScoreTile<D>;
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int b = 1 + (int)blockIdx.x, ranges = (int)gridDim.x + 1;
    const scoret::Cut* at = static_cast<const scoret::Cut*>(p.cuts) + b;
    const int4 u = __ldcg(reinterpret_cast<const int4*>(at)), v = __ldcg(reinterpret_cast<const int4*>(at) + 1);
    if (u.x < 0 || u.w == 0) return;  // no such range, or it starts with a unit
    const int64_t start = __ldcg(reinterpret_cast<const long long*>(at) + 4), total = __ldcg(reinterpret_cast<const long long*>(at) + 5);
    const int64_t q = total / ranges, rem = total - q * ranges;
    auto range_of = [&](int64_t x) {  // the range of tile x
        const int64_t big = (q + 1) * rem;
        return (int)(x < big ? x / (q + 1) : rem + (x - big) / q);
    };
    const int64_t t0 = start - u.w;
    const int c0 = range_of(t0), c1 = range_of(t0 + v.x - 1);
    if (b != c0 + 1) return;
    const int key = threadIdx.x, pos = u.z * T::KB + key;
    if (pos >= v.z) return;
    float all = __ldcg(p.parts + (int64_t)(2 * c0 + 1) * T::KB + key);
    for (int c = c0 + 1; c <= c1; ++c) all += __ldcg(p.parts + (int64_t)(2 * c) * T::KB + key);
    float* score = p.scores + (int64_t)u.x * p.ss_z + u.y * p.ss_h + pos;
    *score = (p.decay != 0.f && pos < v.y ? __ldcg(score) * p.decay : 0.f) + all;
}

}  // namespace fa
