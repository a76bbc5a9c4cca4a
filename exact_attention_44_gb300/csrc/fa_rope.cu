// Rotary positions: the first R elements of a row are R / 2 pairs -- (i, i + R / 2),
// or (2 i, 2 i + 1) interleaved -- and pair i of a row at position p turns by the
// angle p f_i:
//     (a, b) -> factor (a cos - b sin, a sin + b cos),
// the rest of the row stays.  The gradient is the turn back, times the same factor.
// With a cache (fa_cache_append_rope) the turned K rows and the V rows go to their
// slots through the block table.
//
// The angle.  p f in fp32 would be off by p 2^-24 radians (0.06 at a million), so f is
// given in turns as a 64-bit fixed-point fraction and the product with the integer p
// is taken modulo a whole turn by letting it wrap: what is left is off by f's own roundings,
// p (2^-65 + f 2^-54) turns for f radians a position (a quotient of 53 bits, then 64 fixed ones).
// Its upper 32 bits, as an fp32 number (2^-26 turns), go to sincospi.
//
// What bounds it is reading and writing each row once.  A thread takes 8 pairs (two
// 16-byte pieces) of a token through some of its heads, so that a sine and cosine serve
// several heads; the loads go out before the sines are worked out, and where the rows go is
// only looked at when they are there.  671 MB (32 + 8 heads of D = 128, 32768 tokens): 98
// us, 6.8 TB/s, a plain copy's rate; five prompts of 1006 to 2011 tokens into the cache (124
// MB) 24 us called on new inputs, 5.2 TB/s.  The turns come with the launch's arguments: read
// from one place in global memory by every warp, through L2, they took 367 us (one L2 slice
// serves them all).  One token: 1.9 us, 64 tokens into the cache 2.8 (in L2).
#include "fa_rope.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_cache.cuh"
#include "fa_paged.h"
#include "fa_ptx.cuh"

namespace fa {

namespace {

constexpr int ROPE_THREADS = 128;

template <bool BF16>
__device__ __forceinline__ float2 widen(uint32_t w) {
    if constexpr (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <bool BF16>
__device__ __forceinline__ uint32_t narrow(float lo, float hi) {
    if constexpr (BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

// V pairs as a thread holds them: V = 8, two 16-byte pieces; V = 1, two elements in
// the low halves of a word each.
template <int V>
struct Pairs {
    uint4 a, b;
};
template <>
struct Pairs<1> {
    uint32_t a, b;
};
// `from` and `apart`: the first element of the piece, and of its second half
template <int V>
__device__ __forceinline__ Pairs<V> load_pairs(const uint16_t* from, int apart) {
    Pairs<V> x;
    if constexpr (V == 8) {
        x.a = __ldcg(reinterpret_cast<const uint4*>(from));
        x.b = __ldcg(reinterpret_cast<const uint4*>(from + apart));
    } else {
        x.a = __ldcg(from);
        x.b = __ldcg(from + apart);
    }
    return x;
}
template <int V>
__device__ __forceinline__ void store_pairs(uint16_t* to, int apart, const Pairs<V>& x) {
    if constexpr (V == 8) {
        *reinterpret_cast<uint4*>(to) = x.a;
        *reinterpret_cast<uint4*>(to + apart) = x.b;
    } else {
        to[0] = (uint16_t)x.a;
        to[apart] = (uint16_t)x.b;
    }
}
template <bool BF16, bool INTER, int V>
__device__ __forceinline__ void turn(Pairs<V>& x, const float (&c)[V], const float (&s)[V]) {
    if constexpr (V == 1) {
        const float a = widen<BF16>(x.a).x, b = widen<BF16>(x.b).x;
        const uint32_t w = narrow<BF16>(fmaf(a, c[0], -(b * s[0])), fmaf(a, s[0], b * c[0]));
        x.a = w & 0xffffu;
        x.b = w >> 16;
    } else {
        uint32_t w[8] = {x.a.x, x.a.y, x.a.z, x.a.w, x.b.x, x.b.y, x.b.z, x.b.w};
        if constexpr (INTER) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 p = widen<BF16>(w[i]);
                w[i] = narrow<BF16>(fmaf(p.x, c[i], -(p.y * s[i])), fmaf(p.x, s[i], p.y * c[i]));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 a = widen<BF16>(w[i]), b = widen<BF16>(w[i + 4]);
                w[i] = narrow<BF16>(fmaf(a.x, c[2 * i], -(b.x * s[2 * i])), fmaf(a.y, c[2 * i + 1], -(b.y * s[2 * i + 1])));
                w[i + 4] = narrow<BF16>(fmaf(a.x, s[2 * i], b.x * c[2 * i]), fmaf(a.y, s[2 * i + 1], b.y * c[2 * i + 1]));
            }
        }
        x.a = make_uint4(w[0], w[1], w[2], w[3]);
        x.b = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// U: heads whose loads a thread has in flight
template <bool BF16, bool INTER, int V, bool CACHE, int U>
__global__ void __launch_bounds__(ROPE_THREADS) fa_rope_kernel(const __grid_constant__ RopeParams p) {
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    // pieces of a row: a power of two
    const int shift = 31 - __clz(p.D / (2 * V)), turning = p.R / (2 * V);
    const int piece = threadIdx.x & ((1 << shift) - 1), token = threadIdx.x >> shift;
    const int z = blockIdx.z * ((ROPE_THREADS >> shift) >> p.token_shift) + (token >> p.token_shift);
    const int n = (int)(blockIdx.x << p.token_shift) + (token & ((1 << p.token_shift) - 1));
    if (n >= p.N || z >= p.Z) return;
    uint32_t position = (uint32_t)n, col = 0;
    int page = -1;
    if constexpr (CACHE) {
        const int nl = p.news != nullptr ? ldi(p.news + z) : p.N, len = ldi(p.lens + z);
        if (n >= nl) return;
        position += (uint32_t)max(len, 0);  // below 2^32: the slot
        col = position / (uint32_t)p.page;
        page = col < (uint32_t)p.M ? ldi(p.table + z * p.st_z + col) : -1;
    }
    int64_t at = position;
    if (p.positions != nullptr) at = ldi(p.positions + z * p.pos_z + n);
    const bool turns = piece < turning;
    uint64_t f[V];
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = (uint64_t)p.turns[turns ? piece * V + i : 0];
    // where a piece starts, and its second half
    const int first = INTER || !turns ? piece * 2 * V : piece * V;
    const int apart = INTER || !turns ? V : p.R / 2;
    const int h0 = blockIdx.y * p.heads, h1 = min(h0 + p.heads, p.Hq + p.Hk + (CACHE ? p.Hk : 0));
    Pairs<V> x[U];
    // head i: of q, then of k, then (into a cache) of v
    auto load = [&](int h) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = h + u;
            if (i >= h1) continue;
            const uint16_t* from;
            if (i < p.Hq) from = p.q + z * p.q_z + i * p.q_h + n * p.q_n;
            else if (!CACHE || i < p.Hq + p.Hk) from = p.k + z * p.k_z + (i - p.Hq) * p.k_h + n * p.k_n;
            else from = p.v + z * p.v_z + (i - p.Hq - p.Hk) * p.v_h + n * p.v_n;
            x[u] = load_pairs<V>(from + first, apart);
        }
    };
    load(h0);  // (the table entry and the position are on their way too)
    float c[V], s[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        // the fraction of a turn, in half turns for sincospi
        const int32_t frac = (int32_t)(uint32_t)((f[i] * (uint64_t)at) >> 32);
        sincospif((float)frac * 0x1p-31f, &s[i], &c[i]);
        c[i] *= p.cos_factor;
        s[i] *= p.sin_factor;
    }
    int64_t slot = 0;
    if constexpr (CACHE) {
        slot = position - col * (uint32_t)p.page;
        if ((unsigned)page >= (unsigned)p.P) {
            bad_page(p.status, SITE_PAGE_APPEND);
            page = -1;
        }
    }
    for (int h = h0; h < h1; h += U) {
        if (h > h0) load(h);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = h + u;
            if (i >= h1) continue;
            uint16_t* to = nullptr;
            bool rope = turns;
            if (i < p.Hq) {
                if (turns || !p.q_in_place) to = p.qo + z * p.qo_z + i * p.qo_h + n * p.qo_n;
            } else if (!CACHE) {
                if (turns || !p.k_in_place) to = p.ko + z * p.ko_z + (i - p.Hq) * p.ko_h + n * p.ko_n;
            } else if (i < p.Hq + p.Hk) {
                if (page >= 0) to = p.kc.base + page * p.kc.p + (i - p.Hq) * p.kc.h + slot * p.kc.n;
            } else {
                if (page >= 0) to = p.vc.base + page * p.vc.p + (i - p.Hq - p.Hk) * p.vc.h + slot * p.vc.n;
                rope = false;
            }
            if (to != nullptr) {
                if (rope) turn<BF16, INTER, V>(x[u], c, s);
                store_pairs<V>(to + first, apart, x[u]);
            }
        }
    }
}

template <bool BF16, bool INTER, int V>
cudaError_t launch_v(RopeParams p, bool cache, int sms, cudaStream_t stream) {
    const int heads = p.Hq + p.Hk * (cache ? 2 : 1);
    const int tokens = ROPE_THREADS / (p.D / (2 * V));  // of a CTA: of several sequences if they have few
    p.token_shift = 0;
    while ((1 << p.token_shift) < tokens && (1 << p.token_shift) < p.N) ++p.token_shift;
    const int64_t x = ((int64_t)p.N + (1 << p.token_shift) - 1) >> p.token_shift;
    const int64_t zs = tokens >> p.token_shift, z = (p.Z + zs - 1) / zs;
    auto blocks = [&](int n) { return x * z * ((heads + n - 1) / n); };
    auto launch = [&](auto with_cache, auto without, int n) {
        p.heads = n;
        const dim3 grid((unsigned)x, (unsigned)((heads + n - 1) / n), (unsigned)z);
        return launch_dependent(cache ? with_cache : without, grid, ROPE_THREADS, 0, stream, p);
    };
    // Eight heads a thread, all in flight, where that leaves 16 CTAs an SM, else four, and with
    // few tokens fewer, so that there are CTAs for every SM.  Eight against four, inputs from
    // DRAM, D = 128, by CTAs of eight heads: 40 heads x 32768 tokens (10240) 99.5 / 99.8 us, 40 x
    // 8192 (2560) 27.5 / 26.9, 40 x 4096 (1280) 14.9 / 14.5, 32 x 4096 (1024) 12.4 / 12.0; into the
    // cache, q, k and v, 5 x 2011 tokens of 48 heads (3780) 37.2 / 39.9, of 32 (2520) 25.3 / 27.1, 8 x
    // 1000 of 32 (2016) 21.0 / 22.0, 64 x 17 of 48 (768) 9.3 / 8.4.  (With tensors in L2 eight is
    // ahead from 1000 CTAs on: 32 x 4096 8.3 / 9.4.)  One head against four: 40 x 1 1.8 / 2.2, 40 x
    // 256 3.8 / 3.0.
    if constexpr (V == 8)
        if (blocks(8) >= 16 * (int64_t)sms)
            return launch(fa_rope_kernel<BF16, INTER, V, true, 8>, fa_rope_kernel<BF16, INTER, V, false, 8>, 8);
    int n = 4;
    while (n > 1 && blocks(n) < sms) n /= 2;
    return launch(fa_rope_kernel<BF16, INTER, V, true, 4>, fa_rope_kernel<BF16, INTER, V, false, 4>, n);
}
template <bool BF16, bool INTER>
cudaError_t launch_layout(const RopeParams& p, bool cache, int sms, cudaStream_t stream) {
    // 16-byte pieces hold 8 pairs of one half: R a multiple of 16; other R go pair by pair
    return p.R % 16 == 0 ? launch_v<BF16, INTER, 8>(p, cache, sms, stream) : launch_v<BF16, INTER, 1>(p, cache, sms, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, bool bf16, bool interleaved, bool cache, int sms, cudaStream_t stream) {
    if (bf16) return interleaved ? launch_layout<true, true>(p, cache, sms, stream) : launch_layout<true, false>(p, cache, sms, stream);
    return interleaved ? launch_layout<false, true>(p, cache, sms, stream) : launch_layout<false, false>(p, cache, sms, stream);
}

}  // namespace fa
