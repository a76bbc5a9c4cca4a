// C ABI of rotary positions and of a cache held to a budget (fa_rope,
// fa_cache_append_rope, fa_cache_score, fa_cache_evict): argument validation, launch.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "fa.h"
#include "fa_checks.h"
#include "fa_evict.h"
#include "fa_paged.h"
#include "fa_rope.h"
#include "fa_score.h"

namespace {

using namespace fa::checks;

constexpr double kTwoPi = 6.283185307179586476925286766559;

bool flag_ok(int x) { return x == 0 || x == 1; }

// What fa_rope and fa_cache_append_rope share.
fa_status check_rope(int D, int rotary_dim, int interleaved, float factor, int dtype) {
    if (!flag_ok(interleaved) || !std::isfinite(factor)) return FA_ERR_INVALID_ARG;
    if (dtype != FA_DTYPE_F16 && dtype != FA_DTYPE_BF16) return FA_ERR_UNSUPPORTED;
    if (!head_dim_ok(D)) return FA_ERR_UNSUPPORTED;
    return rotary_dim < 2 || rotary_dim > D || rotary_dim % 2 != 0 ? FA_ERR_INVALID_ARG : FA_OK;
}
fa_status check_turns(const void* turns, const void* positions, int64_t positions_stride) {
    if (turns == nullptr || positions_stride < 0) return FA_ERR_INVALID_ARG;
    return check_ints(positions, false);
}
// The same rows: one address and the same strides where there is more than one row to step to.
bool same_place(const void* a, const fa_strides& sa, const void* b, const fa_strides& sb, int64_t Z, int64_t H, int64_t N) {
    return a == b && (Z <= 1 || sa.b == sb.b) && (H <= 1 || sa.h == sb.h) && (N <= 1 || sa.n == sb.n);
}

fa_status launch_score(int D, const fa::ScoreLaunch& a, bool bf16) {
    cudaError_t err;
    switch (D) {
        case 16: err = fa::launch_score_d16(a, bf16); break;
        case 32: err = fa::launch_score_d32(a, bf16); break;
        case 64: err = fa::launch_score_d64(a, bf16); break;
        case 128: err = fa::launch_score_d128(a, bf16); break;
        default: err = fa::launch_score_d256(a, bf16); break;
    }
    return err == cudaSuccess ? FA_OK : fa::report_cuda("cache score launch", err);
}

}  // namespace

extern "C" {

fa_status fa_rope_frequencies(int rotary_dim, const fa_rope_scaling* scaling, double* inv_freq) {
    if (inv_freq == nullptr || rotary_dim < 2 || rotary_dim % 2 != 0) return FA_ERR_INVALID_ARG;
    const fa_rope_scaling s = scaling != nullptr ? *scaling : fa_rope_scaling{FA_ROPE_PLAIN, 10000.0, 1.0, 0.0, 1.0, 32.0};
    if (s.kind < FA_ROPE_PLAIN || s.kind > FA_ROPE_RAMP) return FA_ERR_UNSUPPORTED;
    if (!std::isfinite(s.base) || s.base <= 0.0) return FA_ERR_INVALID_ARG;
    if (s.kind != FA_ROPE_PLAIN && (!std::isfinite(s.stretch) || s.stretch <= 0.0)) return FA_ERR_INVALID_ARG;
    if (s.kind == FA_ROPE_RAMP && (!std::isfinite(s.context) || s.context <= 0.0 || !std::isfinite(s.slow) ||
                                   !std::isfinite(s.fast) || s.fast <= s.slow))
        return FA_ERR_INVALID_ARG;
    const double R = rotary_dim;
    double base = s.base;
    if (s.kind == FA_ROPE_BASE && rotary_dim > 2) base *= std::pow(s.stretch, R / (R - 2.0));
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / R);
        if (s.kind == FA_ROPE_LINEAR) f /= s.stretch;
        if (s.kind == FA_ROPE_RAMP) {
            const double stay = std::min(1.0, std::max(0.0, (s.context * f / kTwoPi - s.slow) / (s.fast - s.slow)));
            f *= stay + (1.0 - stay) / s.stretch;
        }
        inv_freq[i] = f;
    }
    return FA_OK;
}

fa_status fa_rope_turns(int pairs, const double* inv_freq, int64_t* turns) {
    if (pairs < 0 || (pairs > 0 && (inv_freq == nullptr || turns == nullptr))) return FA_ERR_INVALID_ARG;
    for (int i = 0; i < pairs; ++i)
        if (!std::isfinite(inv_freq[i])) return FA_ERR_INVALID_ARG;
    for (int i = 0; i < pairs; ++i) {
        double t = inv_freq[i] / kTwoPi;
        t -= std::nearbyint(t);                         // exact; -1/2 .. 1/2
        const double u = std::ldexp(t, 64);
        turns[i] = u >= 0x1p63 ? INT64_MIN : (int64_t)std::nearbyint(u);  // (half a turn either way)
    }
    return FA_OK;
}

fa_status fa_rope(const fa_rope_args* args, cudaStream_t stream) {
    if (args == nullptr) return FA_ERR_INVALID_ARG;
    const fa_rope_args& x = *args;
    if (x.Z < 0 || x.Hq < 0 || x.Hk < 0 || x.N < 0 || !flag_ok(x.inverse)) return FA_ERR_INVALID_ARG;
    fa_status st = check_rope(x.D, x.rotary_dim, x.interleaved, x.factor, x.dtype);
    if (st != FA_OK) return st;
    if (x.Z > 65535 || x.N > (1 << 30) || (int64_t)x.Hq + x.Hk > 65535) return FA_ERR_UNSUPPORTED;
    if ((int64_t)x.Z * x.N * ((int64_t)x.Hq + x.Hk) == 0) return FA_OK;
    if ((st = check_strided(x.q, &x.sq, x.Z, x.Hq, x.N, false)) != FA_OK) return st;
    if ((st = check_strided(x.q_out, &x.sq_out, x.Z, x.Hq, x.N, true)) != FA_OK) return st;
    if ((st = check_strided(x.k, &x.sk, x.Z, x.Hk, x.N, false)) != FA_OK) return st;
    if ((st = check_strided(x.k_out, &x.sk_out, x.Z, x.Hk, x.N, true)) != FA_OK) return st;
    if ((st = check_turns(x.turns, x.positions, x.positions_stride)) != FA_OK) return st;
    // one tensor's output in place of the other tensor, or of its own in another layout
    if (x.Hq > 0 && x.Hk > 0 && (x.q_out == x.k_out || x.q_out == x.k || x.k_out == x.q)) return FA_ERR_INVALID_ARG;
    const bool q_same = x.Hq > 0 && same_place(x.q, x.sq, x.q_out, x.sq_out, x.Z, x.Hq, x.N);
    const bool k_same = x.Hk > 0 && same_place(x.k, x.sk, x.k_out, x.sk_out, x.Z, x.Hk, x.N);
    if ((x.Hq > 0 && x.q == x.q_out && !q_same) || (x.Hk > 0 && x.k == x.k_out && !k_same)) return FA_ERR_INVALID_ARG;
    fa::DeviceFacts f;
    const cudaError_t err = fa::device_facts(&f);
    if (err != cudaSuccess) return fa::report_cuda("device query", err);
    fa::RopeParams p{};
    p.q = static_cast<const uint16_t*>(x.q);
    p.k = static_cast<const uint16_t*>(x.k);
    p.qo = static_cast<uint16_t*>(x.q_out);
    p.ko = static_cast<uint16_t*>(x.k_out);
    p.q_z = x.sq.b, p.q_h = x.sq.h, p.q_n = x.sq.n;
    p.k_z = x.sk.b, p.k_h = x.sk.h, p.k_n = x.sk.n;
    p.qo_z = x.sq_out.b, p.qo_h = x.sq_out.h, p.qo_n = x.sq_out.n;
    p.ko_z = x.sk_out.b, p.ko_h = x.sk_out.h, p.ko_n = x.sk_out.n;
    p.q_in_place = q_same;
    p.k_in_place = k_same;
    p.positions = x.positions;
    p.pos_z = x.positions_stride;
    std::memcpy(p.turns, x.turns, (size_t)x.rotary_dim / 2 * sizeof(int64_t));  // (at most 128: D is 256 at most)
    p.Z = x.Z, p.Hq = x.Hq, p.Hk = x.Hk, p.N = x.N, p.D = x.D, p.R = x.rotary_dim;
    p.cos_factor = x.factor;
    p.sin_factor = x.inverse ? -x.factor : x.factor;
    p.status = f.status;
    const cudaError_t e = fa::launch_rope(p, x.dtype == FA_DTYPE_BF16, x.interleaved != 0, false, f.sms, stream);
    return e == cudaSuccess ? FA_OK : fa::report_cuda("rope launch", e);
}

fa_status fa_cache_append_rope(const fa_cache_append_rope_args* args, cudaStream_t stream) {
    if (args == nullptr) return FA_ERR_INVALID_ARG;
    const fa_cache_append_rope_args& x = *args;
    const fa_paged_cache& c = x.cache;
    if (x.T < 0 || x.Hq < 0 || c.L != 1) return FA_ERR_INVALID_ARG;
    fa_status st = check_cache(c, false);
    if (st != FA_OK) return st;
    if ((st = check_rope(c.D, x.rotary_dim, x.interleaved, x.factor, x.dtype)) != FA_OK) return st;
    if (x.T > (1 << 30) || (int64_t)x.Hq + 2 * (int64_t)c.Hkv > 65535) return FA_ERR_UNSUPPORTED;
    if ((int64_t)c.Z * x.T * ((int64_t)x.Hq + c.Hkv) == 0) return FA_OK;
    if ((st = check_strided(x.q, &x.sq, c.Z, x.Hq, x.T, false)) != FA_OK) return st;
    if ((st = check_strided(x.q_out, &x.sq_out, c.Z, x.Hq, x.T, true)) != FA_OK) return st;
    if ((st = check_strided(x.k, &x.sk, c.Z, c.Hkv, x.T, false)) != FA_OK) return st;
    if ((st = check_strided(x.v, &x.sv, c.Z, c.Hkv, x.T, false)) != FA_OK) return st;
    if ((st = check_cache_data(c, true)) != FA_OK) return st;
    if ((st = check_ints(x.new_lens, false)) != FA_OK) return st;
    if ((st = check_turns(x.turns, x.positions, x.positions_stride)) != FA_OK) return st;
    if (x.Hq > 0 && c.Hkv > 0 && (x.q_out == x.k || x.q_out == x.v)) return FA_ERR_INVALID_ARG;
    const bool q_same = x.Hq > 0 && same_place(x.q, x.sq, x.q_out, x.sq_out, c.Z, x.Hq, x.T);
    if (x.Hq > 0 && x.q == x.q_out && !q_same) return FA_ERR_INVALID_ARG;
    fa::DeviceFacts f;
    const cudaError_t err = fa::device_facts(&f);
    if (err != cudaSuccess) return fa::report_cuda("device query", err);
    fa::RopeParams p{};
    p.q = static_cast<const uint16_t*>(x.q);
    p.k = static_cast<const uint16_t*>(x.k);
    p.v = static_cast<const uint16_t*>(x.v);
    p.qo = static_cast<uint16_t*>(x.q_out);
    p.q_z = x.sq.b, p.q_h = x.sq.h, p.q_n = x.sq.n;
    p.k_z = x.sk.b, p.k_h = x.sk.h, p.k_n = x.sk.n;
    p.v_z = x.sv.b, p.v_h = x.sv.h, p.v_n = x.sv.n;
    p.qo_z = x.sq_out.b, p.qo_h = x.sq_out.h, p.qo_n = x.sq_out.n;
    p.q_in_place = q_same;
    p.positions = x.positions;
    p.pos_z = x.positions_stride;
    std::memcpy(p.turns, x.turns, (size_t)x.rotary_dim / 2 * sizeof(int64_t));  // (at most 128: D is 256 at most)
    p.Z = c.Z, p.Hq = x.Hq, p.Hk = c.Hkv, p.N = x.T, p.D = c.D, p.R = x.rotary_dim;
    p.cos_factor = p.sin_factor = x.factor;
    p.kc = view(c.k, c.sk, 0);
    p.vc = view(c.v, c.sv, 0);
    p.table = c.block_table;
    p.st_z = c.table_stride;
    p.lens = c.seq_lens;
    p.news = x.new_lens;
    p.page = c.page_size, p.M = c.max_pages, p.P = c.P;
    p.status = f.status;
    const cudaError_t e = fa::launch_rope(p, x.dtype == FA_DTYPE_BF16, x.interleaved != 0, true, f.sms, stream);
    return e == cudaSuccess ? FA_OK : fa::report_cuda("cache append rope launch", e);
}

fa_status fa_cache_score_workspace_size(size_t* bytes) {
    if (bytes == nullptr) return FA_ERR_INVALID_ARG;
    fa::DeviceFacts f;
    const cudaError_t err = fa::device_facts(&f);
    if (err != cudaSuccess) return fa::report_cuda("device query", err);
    *bytes = fa::score_workspace_bytes(f.sms);
    return FA_OK;
}

fa_status fa_cache_score(const fa_cache_score_args* args, cudaStream_t stream) {
    if (args == nullptr) return FA_ERR_INVALID_ARG;
    const fa_cache_score_args& x = *args;
    const fa_paged_cache& c = x.cache;
    if (x.Hq < 0 || c.Hkv < 1 || x.T < 0 || x.Hq % c.Hkv != 0 || c.L != 1 || x.score_seq < 0 || x.score_head < 0)
        return FA_ERR_INVALID_ARG;
    if (x.dtype != FA_DTYPE_F16 && x.dtype != FA_DTYPE_BF16) return FA_ERR_UNSUPPORTED;
    float magnitude = 0.f;
    int negative = 0;
    if (!fa::split_scale(x.scale, &magnitude, &negative) || !std::isfinite(x.decay)) return FA_ERR_INVALID_ARG;
    fa_status st = check_cache(c, false);
    if (st != FA_OK) return st;
    const int G = x.Hq / c.Hkv;
    if ((int64_t)x.T * G > (int64_t(1) << 30)) return FA_ERR_UNSUPPORTED;
    const int64_t cap = c.P > 0 ? (int64_t)c.max_pages * c.page_size : 0;
    if ((int64_t)c.Z * cap == 0) return FA_OK;  // no position, no score
    if ((st = check_strided(x.q, &x.sq, c.Z, x.Hq, x.T, false)) != FA_OK) return st;
    if ((st = check_strided(c.k, &c.sk, c.P, c.Hkv, c.page_size, false)) != FA_OK) return st;
    if (c.seq_lens == nullptr || x.scores == nullptr || ((int64_t)x.Hq * x.T > 0 && x.lse == nullptr)) return FA_ERR_INVALID_ARG;
    for (const void* ptr : {(const void*)c.seq_lens, (const void*)x.new_lens, (const void*)x.lse, (const void*)x.scores})
        if (misaligned(ptr, 4)) return FA_ERR_ALIGNMENT;
    // rows of scores must not fold together
    if ((c.Hkv > 1 && x.score_head < cap) || (c.Z > 1 && x.score_seq < cap)) return FA_ERR_INVALID_ARG;
    if (x.workspace == nullptr || misaligned(x.workspace, 256)) return FA_ERR_WORKSPACE;
    fa::DeviceFacts f;
    const cudaError_t err = fa::device_facts(&f);
    if (err != cudaSuccess) return fa::report_cuda("device query", err);
    if (x.workspace_bytes < fa::score_workspace_bytes(f.sms)) return FA_ERR_WORKSPACE;
    fa::ScoreLaunch a{};
    fa::ScoreParams& p = a.params;
    p.q = static_cast<const uint16_t*>(x.q);
    p.sq_z = x.sq.b, p.sq_h = x.sq.h, p.sq_n = x.sq.n;
    p.lse = x.lse;
    p.k = static_cast<const uint16_t*>(c.k);
    p.sk_p = c.sk.b, p.sk_h = c.sk.h, p.sk_n = c.sk.n;
    p.table = c.block_table;
    p.st_z = c.table_stride;
    p.lens = c.seq_lens;
    p.news = x.new_lens;
    p.scores = x.scores;
    p.ss_z = x.score_seq, p.ss_h = x.score_head;
    p.Z = c.Z, p.Hq = x.Hq, p.Hkv = c.Hkv, p.G = G, p.T = x.T;
    p.page = c.page_size, p.M = c.max_pages, p.P = c.P, p.cap = (int)cap;
    p.by_g = fa::FastDiv(std::max(G, 1));
    p.by_page = fa::FastDiv(p.page);
    p.scale = x.scale, p.decay = x.decay;
    p.status = f.status;
    p.wait_limit_ns = f.wait_limit_ns;
    p.inject_stall = f.inject_stall;
    a.sms = f.sms;
    a.stream = stream;
    const bool bf16 = x.dtype == FA_DTYPE_BF16;
    const fa::ScoreTileFacts tile = fa::score_tile_facts(c.D);
    // Up to 32 rows of a (sequence, kv head), 16 at D = 256, run on the rows kernel, the
    // others on the tile kernel, which needs a whole group in a tile.  Both sides, rows
    // against tile kernel, repeated in a graph, 16 sequences of 1000-4000, Hkv 8: 32 rows
    // 18.7 / 25.5 us at D 128, 14.7 / 23.8 at D 64, 12.9 / 23.7 at D 16; 32 rows of one
    // sequence of 1024 3.7 / 7.4, of 64 of 256-4096 67.8 / 75.2; 16 rows, D 256 and Hkv 4,
    // 13.6 / 20.4, 32 rows 25.2 / 20.
    a.tiles = G <= tile.rows && (int64_t)x.T * G > (c.D == 256 ? 16 : 32);
    CUtensorMap mq{}, mk{};
    if (a.tiles) {
        while (G << (p.token_shift + 1) <= tile.rows) ++p.token_shift;
        p.tokens = 1 << p.token_shift;
        p.tile_rows = p.tokens * G;
        p.tile_cols = (int)cdiv(p.tile_rows, 16) * 16;
        p.box_rows = fa::paged_box_rows(c.page_size, 128);
        const fa::PagedMapDim dq[3] = {{x.Hq, x.sq.h, G}, {x.T, x.sq.n, p.tokens}, {c.Z, x.sq.b, 1}};
        const fa::PagedMapDim dk[3] = {{c.page_size, c.sk.n, p.box_rows}, {c.Hkv, c.sk.h, 1}, {c.P, c.sk.b, 1}};
        if (fa::make_paged_map(&mq, x.q, bf16, c.D, dq) != CUDA_SUCCESS ||
            fa::make_paged_map(&mk, c.k, bf16, c.D, dk) != CUDA_SUCCESS)
            return FA_ERR_CUDA;
        a.tmQ = &mq;
        a.tmK = &mk;
        p.long_q = x.T >= 8 * p.tokens;
        // Units of up to four tiles are not cut: the merge takes about 3 us, as long as
        // the tiles that it could spare the busiest CTA.
        if (x.T > 4 * p.tokens) {
            p.parts = static_cast<float*>(x.workspace);
            p.cuts = static_cast<char*>(x.workspace) + fa::score_slot_bytes(f.sms);
        }
    }
    return launch_score(c.D, a, bf16);
}

fa_status fa_cache_evict_workspace_size(int L, int Z, int Hkv, int max_pages, int budget, size_t* bytes) {
    if (bytes == nullptr || L < 0 || Z < 0 || Hkv < 0 || max_pages < 0 || budget < 0) return FA_ERR_INVALID_ARG;
    if ((double)L * Z * Hkv * ((double)budget + 1) > 0x1p60) return FA_ERR_UNSUPPORTED;
    *bytes = (size_t)fa::evict_workspace_ints(L, Z, Hkv, max_pages, budget) * sizeof(int32_t);
    return FA_OK;
}

fa_status fa_cache_evict(const fa_cache_evict_args* args, cudaStream_t stream) {
    if (args == nullptr) return FA_ERR_INVALID_ARG;
    const fa_cache_evict_args& x = *args;
    const fa_paged_cache& c = x.cache;
    if (x.budget < 0 || x.first < 0 || x.recent < 0 || x.score_layer < 0 || x.score_seq < 0 || x.score_head < 0 ||
        x.missing == nullptr)
        return FA_ERR_INVALID_ARG;
    fa_status st = check_cache(c, true);
    if (st != FA_OK) return st;
    if (c.P > (1 << 30) || (int64_t)c.Z * c.max_pages > INT32_MAX || c.L > 65535 ||
        (int64_t)c.L * c.Hkv > INT32_MAX || (int64_t)c.L * c.Hkv * c.Z > (1 << 26))
        return FA_ERR_UNSUPPORTED;
    if ((st = check_ints(x.missing, true)) != FA_OK) return st;
    const int64_t cap = (int64_t)c.max_pages * c.page_size;
    if (c.Z == 0 || c.L == 0 || c.Hkv == 0 || c.P == 0 || cap == 0) {  // no position, no row
        const cudaError_t err = cudaMemsetAsync(x.missing, 0, sizeof(int32_t), stream);
        return err == cudaSuccess ? FA_OK : fa::report_cuda("cache evict", err);
    }
    if ((st = check_cache_data(c, true)) != FA_OK) return st;
    if ((st = check_ints(x.ref_counts, true)) != FA_OK) return st;
    if ((st = check_ints(x.keep, false)) != FA_OK) return st;
    if ((st = check_ints(x.scores, true)) != FA_OK) return st;
    if ((c.Hkv > 1 && x.score_head < cap) || (c.Z > 1 && x.score_seq < cap) || (c.L > 1 && x.score_layer < cap))
        return FA_ERR_INVALID_ARG;
    const int budget = (int)std::min<int64_t>(x.budget, cap);
    if (x.workspace == nullptr || misaligned(x.workspace, 256) ||
        x.workspace_bytes < (size_t)fa::evict_workspace_ints(c.L, c.Z, c.Hkv, c.max_pages, budget) * sizeof(int32_t))
        return FA_ERR_WORKSPACE;
    fa::DeviceFacts f;
    cudaError_t err = fa::device_facts(&f);
    if (err != cudaSuccess) return fa::report_cuda("device query", err);
    fa::EvictParams p{};
    p.k = view(c.k, c.sk, c.k_layer);
    p.v = view(c.v, c.sv, c.v_layer);
    p.table = c.block_table;
    p.st_z = c.table_stride;
    p.lens = c.seq_lens;
    p.refs = x.ref_counts;
    p.scores = x.scores;
    p.ss_l = x.score_layer, p.ss_z = x.score_seq, p.ss_h = x.score_head;
    p.keep = x.keep;
    p.missing = x.missing;
    p.Z = c.Z, p.L = c.L, p.H = c.Hkv, p.D = c.D, p.page = c.page_size, p.M = c.max_pages, p.P = c.P;
    p.budget = budget, p.first = x.first, p.recent = x.recent;
    p.by_page = fa::FastDiv(p.page);
    p.ws = static_cast<int32_t*>(x.workspace);
    p.status = f.status;
    err = fa::launch_cache_evict(p, f.sms, stream);
    return err == cudaSuccess ? FA_OK : fa::report_cuda("cache evict launch", err);
}

}  // extern "C"
