// C ABI of the paged-cache operators (fa_fwd_paged, fa_cache_append,
// fa_cache_commit, fa_cache_fork): argument validation, the choice of kernel,
// launch.
#include <algorithm>
#include <cstdint>
#include <utility>

#include "fa.h"
#include "fa_cache.h"
#include "fa_paged.h"

namespace fa {
fa_status report_cuda(const char* what, cudaError_t e);  // fa_api.cu
}

namespace {

bool head_dim_ok(int D) { return D == 16 || D == 32 || D == 64 || D == 128 || D == 256; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool misaligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

// d-stride 1, 16-byte aligned base, the other strides multiples of 8 elements
// in every dimension of extent > 1; outputs must not fold rows together
// (stride 0).
fa_status check_strided(const void* ptr, const fa_strides* s, int64_t nb, int64_t nh, int64_t nn, bool written) {
    if (s == nullptr) return FA_ERR_INVALID_ARG;
    if (nb * nh * nn == 0) return FA_OK;  // nothing there: the pointer is not used
    if (ptr == nullptr) return FA_ERR_INVALID_ARG;
    if (s->d != 1 || misaligned(ptr, 16)) return FA_ERR_ALIGNMENT;
    const int64_t st[3] = {s->b, s->h, s->n}, ext[3] = {nb, nh, nn};
    for (int i = 0; i < 3; ++i) {
        if (ext[i] <= 1) continue;
        if (st[i] < 0 || st[i] % 8 != 0 || st[i] >= (int64_t(1) << 38)) return FA_ERR_ALIGNMENT;
        if (written && st[i] == 0) return FA_ERR_INVALID_ARG;
    }
    return FA_OK;
}

// The cache's geometry and its block table.
fa_status check_cache(const fa_paged_cache& c, bool table_written) {
    if (c.Z < 0 || c.L < 0 || c.P < 0 || c.Hkv < 0 || c.max_pages < 0 || c.table_stride < 0) return FA_ERR_INVALID_ARG;
    if (!head_dim_ok(c.D) || c.page_size < 16 || c.page_size % 16 != 0) return FA_ERR_UNSUPPORTED;
    if ((int64_t)c.max_pages * c.page_size > (int64_t(1) << 30) || c.Z > 65535) return FA_ERR_UNSUPPORTED;
    if ((int64_t)c.Z * c.max_pages > 0) {
        if (c.block_table == nullptr) return FA_ERR_INVALID_ARG;
        if (misaligned(c.block_table, 4)) return FA_ERR_ALIGNMENT;
        if (table_written && c.Z > 1 && c.table_stride < c.max_pages) return FA_ERR_INVALID_ARG;
    }
    if (c.L > 1)
        for (const int64_t s : {c.k_layer, c.v_layer})
            if (s <= 0 || s % 8 != 0 || s >= (int64_t(1) << 42)) return FA_ERR_ALIGNMENT;
    return FA_OK;
}
// Its tensors (where a call has work for them) and lengths.
fa_status check_cache_data(const fa_paged_cache& c, bool written) {
    if (c.L > 0)
        for (const auto& t : {std::make_pair(c.k, &c.sk), std::make_pair(c.v, &c.sv)}) {
            const fa_status st = check_strided(t.first, t.second, c.P, c.Hkv, c.page_size, written);
            if (st != FA_OK) return st;
        }
    if (c.seq_lens == nullptr) return FA_ERR_INVALID_ARG;
    return misaligned(c.seq_lens, 4) ? FA_ERR_ALIGNMENT : FA_OK;
}
fa_status check_ints(const void* p, bool needed) {
    if (p == nullptr) return needed ? FA_ERR_INVALID_ARG : FA_OK;
    return misaligned(p, 4) ? FA_ERR_ALIGNMENT : FA_OK;
}

// Workers of the rows kernel an SM (warps), and the positions of its key block.
struct RowsFacts {
    int workers, block;
};
RowsFacts rows_facts(int D) {
    RowsFacts f{};
    switch (D) {
        case 16: fa::paged_facts_d16(&f.workers, &f.block); break;
        case 32: fa::paged_facts_d32(&f.workers, &f.block); break;
        case 64: fa::paged_facts_d64(&f.workers, &f.block); break;
        case 128: fa::paged_facts_d128(&f.workers, &f.block); break;
        default: fa::paged_facts_d256(&f.workers, &f.block); break;
    }
    return f;
}
constexpr int kMaxTeams = 1280;  // eight workers an SM on up to 160 SMs; fewer an SM beyond

// A partial-result slot holds the rows of O / l of a tile (16 in the rows
// kernel, 128 in the tile kernel) and their base-2 log-sum-exps, padded to 256
// bytes; two slots a worker.  Behind the slots: where each team's range
// starts, 48 bytes.
int64_t slot_floats(int rows, int D) { return ((int64_t)rows * (D + 1) + 63) / 64 * 64; }
size_t paged_slot_bytes(int D, int sms) {
    const int64_t rows = std::min(rows_facts(D).workers * sms, kMaxTeams) * slot_floats(16, D);
    return (size_t)(2 * std::max(rows, sms * slot_floats(128, D))) * sizeof(float);
}
size_t paged_workspace_bytes(int D, int sms) { return paged_slot_bytes(D, sms) + 48 * kMaxTeams; }

// 4-D tensor map with the head dim innermost (dims: D, then `dims` outermost
// last) and boxes of one swizzle chunk x the given extents.
struct MapDim {
    int64_t extent, stride;  // stride in elements
    int box;
};
CUresult make_paged_map(CUtensorMap* map, const void* ptr, bool bf16, int D, const MapDim (&dims)[3]) {
    const int swe = D < 64 ? D : 64;
    const CUtensorMapSwizzle sw = swe == 64   ? CU_TENSOR_MAP_SWIZZLE_128B
                                  : swe == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                              : CU_TENSOR_MAP_SWIZZLE_32B;
    cuuint64_t ext[4] = {(cuuint64_t)D, 0, 0, 0}, str[3];
    cuuint32_t box[4] = {(cuuint32_t)swe, 0, 0, 0}, ones[4] = {1, 1, 1, 1};
    for (int i = 0; i < 3; ++i) {
        ext[i + 1] = (cuuint64_t)dims[i].extent;
        // a dimension of extent 1 is never stepped along; give it a harmless stride
        str[i] = dims[i].extent > 1 ? (cuuint64_t)dims[i].stride * 2 : (cuuint64_t)D * 2;
        box[i + 1] = (cuuint32_t)dims[i].box;
    }
    const auto fn = fa::tensor_map_encoder();
    if (fn == nullptr) return CUDA_ERROR_NOT_SUPPORTED;
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void*>(ptr),
              ext, str, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// Largest box of whole page rows that tiles a block of `bn` positions.
int box_rows_for(int page, int bn) {
    int r = 16;
    while (r < bn && page % (2 * r) == 0) r *= 2;
    return r;
}

cudaError_t launch_paged(int D, const fa::PagedLaunch& a, bool bf16) {
    switch (D) {
        case 16: return fa::launch_paged_d16(a, bf16);
        case 32: return fa::launch_paged_d32(a, bf16);
        case 64: return fa::launch_paged_d64(a, bf16);
        case 128: return fa::launch_paged_d128(a, bf16);
        default: return fa::launch_paged_d256(a, bf16);
    }
}

fa::CacheView view(void* base, const fa_strides& s, int64_t layer) {
    return fa::CacheView{static_cast<uint16_t*>(base), layer, s.b, s.h, s.n};
}

}  // namespace

extern "C" {

fa_status fa_fwd_paged_workspace_size(int D, size_t* bytes) {
    if (bytes == nullptr) return FA_ERR_INVALID_ARG;
    if (!head_dim_ok(D)) return FA_ERR_UNSUPPORTED;
    fa::DeviceFacts f;
    const cudaError_t err = fa::device_facts(&f);
    if (err != cudaSuccess) return fa::report_cuda("device query", err);
    *bytes = paged_workspace_bytes(D, f.sms);
    return FA_OK;
}

fa_status fa_fwd_paged(const fa_fwd_paged_args* args, cudaStream_t stream) {
    if (args == nullptr) return FA_ERR_INVALID_ARG;
    const fa_fwd_paged_args& x = *args;
    const fa_paged_cache& cache = x.cache;
    const int Z = cache.Z, Hq = x.Hq, Hkv = cache.Hkv, T = x.T, D = cache.D, P = cache.P;
    if (Hq < 0 || Hkv < 1 || T < 0 || Hq % Hkv != 0 || x.mask_stride < 0 || cache.L != 1) return FA_ERR_INVALID_ARG;
    if (x.dtype != FA_DTYPE_F16 && x.dtype != FA_DTYPE_BF16) return FA_ERR_UNSUPPORTED;
    float c = 0.f;
    int negate = 0;
    if (!fa::split_scale(x.scale, &c, &negate)) return FA_ERR_INVALID_ARG;
    fa_status st = check_cache(cache, false);
    if (st != FA_OK) return st;
    const int G = Hq / Hkv;
    // (row and tile indices fit in 32 bits)
    if ((int64_t)T * G > (int64_t(1) << 30) || (int64_t)Z * Hkv * cdiv((int64_t)T * G, 16) > INT32_MAX)
        return FA_ERR_UNSUPPORTED;
    if ((int64_t)Z * Hq * T == 0) return FA_OK;
    if ((st = check_strided(x.q, &x.sq, Z, Hq, T, false)) != FA_OK) return st;
    if ((st = check_strided(x.o, &x.so, Z, Hq, T, true)) != FA_OK) return st;
    if ((st = check_cache_data(cache, false)) != FA_OK) return st;
    if ((st = check_ints(x.new_lens, false)) != FA_OK) return st;
    if ((st = check_ints(x.tree_mask, false)) != FA_OK) return st;
    if ((st = check_ints(x.lse, false)) != FA_OK) return st;
    if (x.workspace == nullptr || misaligned(x.workspace, 256)) return FA_ERR_WORKSPACE;

    fa::DeviceFacts f;
    cudaError_t err = fa::device_facts(&f);
    if (err != cudaSuccess) return fa::report_cuda("device query", err);
    if (x.workspace_bytes < paged_workspace_bytes(D, f.sms)) return FA_ERR_WORKSPACE;

    fa::PagedLaunch a{};
    fa::PagedParams& p = a.params;
    p.q = x.q;
    p.o = x.o;
    p.lse = x.lse;
    p.sq_z = x.sq.b, p.sq_h = x.sq.h, p.sq_n = x.sq.n;
    p.so_z = x.so.b, p.so_h = x.so.h, p.so_n = x.so.n;
    p.table = cache.block_table;
    p.st_z = cache.table_stride;
    p.lens = cache.seq_lens;
    p.news = x.new_lens;
    p.mask = reinterpret_cast<const uint32_t*>(x.tree_mask);
    p.sm_z = x.mask_stride;
    p.words = (T + 31) / 32;
    p.Z = Z, p.Hq = Hq, p.Hkv = Hkv, p.G = G, p.T = T;
    p.page = cache.page_size, p.M = cache.max_pages, p.P = P;
    p.cap = P > 0 ? p.M * p.page : 0;
    p.scratch = static_cast<float*>(x.workspace);
    p.status = f.status;
    p.wait_limit_ns = f.wait_limit_ns;
    p.inject_stall = f.inject_stall;
    a.stream = stream;

    const bool bf16 = x.dtype == FA_DTYPE_BF16;
    // Up to 16 rows of a (sequence, kv head) run on the rows kernel up to D = 128, the
    // others on the tile kernel, which needs a whole group in a tile.  Both sides, rows
    // against tile kernel, repeated in a graph: 16 rows, 16 sequences of 1000-4000, Hkv 8:
    // 35.0 / 36.1 us at D 128, 21.9 / 30.1 at D 64, 19.2 / 28.6 at D 16; 4 rows, 64
    // sequences of 256-4096, D 128: 96 / 101; 12 to 16 rows of one sequence of 1024, D 128:
    // 13.9 / 13.4, 14.7 / 13.4; 32 rows (two tiles of 16): 178 / 106.  At D = 256, where the
    // rows kernel has four warps an SM: 4 rows 22.7 / 19.8, 8 rows 25.1 / 19.9, 1 row 98.5 /
    // 98.8 and 13.8 / 15.0.
    a.tiles = G <= 128 && (D == 256 || T * (int64_t)G > 16);
    CUtensorMap mq{}, mk{}, mv{};
    int bk, workers;
    if (a.tiles) {
        const int tokens = 128 / G;
        bk = D == 256 ? 64 : 128;
        workers = f.sms;
        p.tile_rows = tokens * G;
        p.scale_log2 = c;
        p.negate_s = negate;
        p.slot_floats = slot_floats(128, D);
        const MapDim dq[3] = {{Hq, x.sq.h, G}, {T, x.sq.n, tokens}, {Z, x.sq.b, 1}};
        if (make_paged_map(&mq, x.q, bf16, D, dq) != CUDA_SUCCESS) return FA_ERR_CUDA;
        a.tmQ = &mq;
    } else {
        const RowsFacts rf = rows_facts(D);
        bk = rf.block;
        workers = std::min(rf.workers * f.sms, kMaxTeams);
        p.tile_rows = 16;
        p.scale_log2 = negate ? -c : c;
        p.slot_floats = slot_floats(16, D);
    }
    p.box_rows = box_rows_for(p.page, bk);
    if (P > 0) {
        const fa_strides &sk = cache.sk, &sv = cache.sv;
        const MapDim dk[3] = {{p.page, sk.n, p.box_rows}, {Hkv, sk.h, 1}, {P, sk.b, 1}};
        const MapDim dv[3] = {{p.page, sv.n, p.box_rows}, {Hkv, sv.h, 1}, {P, sv.b, 1}};
        if (make_paged_map(&mk, cache.k, bf16, D, dk) != CUDA_SUCCESS ||
            make_paged_map(&mv, cache.v, bf16, D, dv) != CUDA_SUCCESS)
            return FA_ERR_CUDA;
    }
    a.tmK = &mk;
    a.tmV = &mv;
    p.tiles = (int)cdiv((int64_t)T * G, p.tile_rows);
    // Teams of up to 8, as many members as leave the groups of a kv head equally large:
    // 8 sequences of 1000-3000, 9 tiles: 106 us as 8 + 1, 90 as 5 + 4.  (Of up to 4: 482
    // -> 508 us for a prompt of 8192 tokens, which reads K and V twice as often from L2;
    // 1: 561.)
    p.team = a.tiles ? (int)cdiv(p.tiles, cdiv(p.tiles, 8)) : 1;
    // more teams than there can be blocks would find no work
    const int64_t blocks = (int64_t)Z * Hkv * cdiv(p.tiles, p.team) * cdiv(p.cap, bk);
    p.teams = (int)std::max<int64_t>(1, std::min<int64_t>(blocks, workers / p.team));
    // Groups of up to 512 positions are not cut: a part costs its write and a share of
    // the merge (8 x 32 tokens over 50-250 positions 16.1 against 13.8 us).  Not in the
    // rows kernel, whose warps take 16 positions in turn: whole tiles of up to 256 took
    // 16.9 us where cut ones took 9.5 (8 sequences of 20-200).
    p.snap = a.tiles ? 512 / bk : 0;
    p.by_g = fa::FastDiv(G);
    p.by_page = fa::FastDiv(p.page);
    p.by_tile_rows = fa::FastDiv(p.tile_rows);
    p.by_team = fa::FastDiv(p.team);
    p.wide_o = !misaligned(x.o, 32) && (Z == 1 || p.so_z % 16 == 0) && (Hq == 1 || p.so_h % 16 == 0) &&
               (T == 1 || p.so_n % 16 == 0);
    p.few = Z <= 32 && blocks < (int64_t(1) << 30);
    p.cuts = static_cast<char*>(x.workspace) + paged_slot_bytes(D, f.sms);
    err = launch_paged(D, a, bf16);
    return err == cudaSuccess ? FA_OK : fa::report_cuda("paged attention launch", err);
}

fa_status fa_cache_append(const fa_cache_append_args* args, cudaStream_t stream) {
    if (args == nullptr) return FA_ERR_INVALID_ARG;
    const fa_cache_append_args& x = *args;
    const fa_paged_cache& c = x.cache;
    if (x.T < 0 || c.L != 1) return FA_ERR_INVALID_ARG;
    fa_status st = check_cache(c, false);
    if (st != FA_OK) return st;
    if ((int64_t)c.Hkv * x.T * (c.D / 8) >= INT32_MAX) return FA_ERR_UNSUPPORTED;
    if ((int64_t)c.Z * c.Hkv * x.T == 0) return FA_OK;
    if ((st = check_strided(x.k, &x.sk, c.Z, c.Hkv, x.T, false)) != FA_OK) return st;
    if ((st = check_strided(x.v, &x.sv, c.Z, c.Hkv, x.T, false)) != FA_OK) return st;
    if ((st = check_cache_data(c, true)) != FA_OK) return st;
    if ((st = check_ints(x.new_lens, false)) != FA_OK) return st;
    fa::DeviceFacts f;
    cudaError_t err = fa::device_facts(&f);
    if (err != cudaSuccess) return fa::report_cuda("device query", err);
    fa::AppendParams p{};
    p.k = view(c.k, c.sk, 0);
    p.v = view(c.v, c.sv, 0);
    p.ks = static_cast<const uint16_t*>(x.k);
    p.vs = static_cast<const uint16_t*>(x.v);
    p.ks_z = x.sk.b, p.ks_h = x.sk.h, p.ks_n = x.sk.n;
    p.vs_z = x.sv.b, p.vs_h = x.sv.h, p.vs_n = x.sv.n;
    p.table = c.block_table;
    p.st_z = c.table_stride;
    p.lens = c.seq_lens;
    p.news = x.new_lens;
    p.Z = c.Z, p.H = c.Hkv, p.T = x.T, p.D = c.D, p.page = c.page_size, p.M = c.max_pages, p.P = c.P;
    p.status = f.status;
    err = fa::launch_cache_append(p, stream);
    return err == cudaSuccess ? FA_OK : fa::report_cuda("cache append launch", err);
}

fa_status fa_cache_commit(const fa_cache_commit_args* args, cudaStream_t stream) {
    if (args == nullptr) return FA_ERR_INVALID_ARG;
    const fa_cache_commit_args& x = *args;
    const fa_paged_cache& c = x.cache;
    if (x.A < 0 || x.accepted_stride < 0) return FA_ERR_INVALID_ARG;
    fa_status st = check_cache(c, false);
    if (st != FA_OK) return st;
    if ((int64_t)c.L * 2 * c.Hkv * (c.D / 8) >= INT32_MAX) return FA_ERR_UNSUPPORTED;
    if ((int64_t)c.Z * c.L * c.Hkv * x.A == 0) return FA_OK;
    if ((st = check_cache_data(c, true)) != FA_OK) return st;
    if ((st = check_ints(x.accepted, true)) != FA_OK) return st;
    if ((st = check_ints(x.accepted_lens, true)) != FA_OK) return st;
    fa::DeviceFacts f;
    cudaError_t err = fa::device_facts(&f);
    if (err != cudaSuccess) return fa::report_cuda("device query", err);
    fa::CommitParams p{};
    p.k = view(c.k, c.sk, c.k_layer);
    p.v = view(c.v, c.sv, c.v_layer);
    p.table = c.block_table;
    p.st_z = c.table_stride;
    p.lens = c.seq_lens;
    p.path = x.accepted;
    p.kept = x.accepted_lens;
    p.sp_z = x.accepted_stride;
    p.Z = c.Z, p.L = c.L, p.H = c.Hkv, p.A = x.A, p.D = c.D, p.page = c.page_size, p.M = c.max_pages, p.P = c.P;
    p.status = f.status;
    err = fa::launch_cache_commit(p, stream);
    return err == cudaSuccess ? FA_OK : fa::report_cuda("cache commit launch", err);
}

fa_status fa_cache_fork_workspace_size(int Z, int max_pages, size_t* bytes) {
    if (bytes == nullptr || Z < 0 || max_pages < 0) return FA_ERR_INVALID_ARG;
    *bytes = (size_t)fa::fork_workspace_ints(Z, max_pages) * sizeof(int32_t);
    return FA_OK;
}

fa_status fa_cache_fork(const fa_cache_fork_args* args, cudaStream_t stream) {
    if (args == nullptr) return FA_ERR_INVALID_ARG;
    const fa_cache_fork_args& x = *args;
    const fa_paged_cache& c = x.cache;
    if (x.room < 0 || (x.all_or_nothing != 0 && x.all_or_nothing != 1)) return FA_ERR_INVALID_ARG;
    if (x.all_or_nothing && x.missing == nullptr) return FA_ERR_INVALID_ARG;  // whether it happened could not be told
    fa_status st = check_cache(c, true);
    if (st != FA_OK) return st;
    if (c.Z > 8192 || c.P > (1 << 30) || x.room > (1 << 30) || (int64_t)c.Z * c.max_pages > INT32_MAX ||
        (int64_t)c.L * 2 * c.Hkv > INT32_MAX || (int64_t)c.page_size * (c.D / 8) > INT32_MAX)
        return FA_ERR_UNSUPPORTED;
    if ((st = check_ints(x.missing, false)) != FA_OK) return st;
    if (c.Z == 0) {  // nothing to do, and nothing lacks
        const cudaError_t err = x.missing != nullptr ? cudaMemsetAsync(x.missing, 0, sizeof(int32_t), stream) : cudaSuccess;
        return err == cudaSuccess ? FA_OK : fa::report_cuda("cache fork", err);
    }
    if ((st = check_cache_data(c, true)) != FA_OK) return st;
    if ((st = check_ints(x.ref_counts, c.P > 0)) != FA_OK) return st;
    if ((st = check_ints(x.source, false)) != FA_OK) return st;
    if (x.workspace == nullptr || misaligned(x.workspace, 256) ||
        x.workspace_bytes < (size_t)fa::fork_workspace_ints(c.Z, c.max_pages) * sizeof(int32_t))
        return FA_ERR_WORKSPACE;
    fa::DeviceFacts f;
    cudaError_t err = fa::device_facts(&f);
    if (err != cudaSuccess) return fa::report_cuda("device query", err);
    fa::ForkParams p{};
    p.k = view(c.k, c.sk, c.k_layer);
    p.v = view(c.v, c.sv, c.v_layer);
    p.table = c.block_table;
    p.st_z = c.table_stride;
    p.lens = c.seq_lens;
    p.refs = x.ref_counts;
    p.source = x.source;
    p.missing = x.missing;
    p.Z = c.Z, p.L = c.L, p.H = c.Hkv, p.D = c.D, p.page = c.page_size, p.M = c.max_pages, p.P = c.P, p.room = x.room;
    p.whole = x.all_or_nothing;
    p.ws = static_cast<int32_t*>(x.workspace);
    p.status = f.status;
    err = fa::launch_cache_fork(p, f.sms, stream);
    return err == cudaSuccess ? FA_OK : fa::report_cuda("cache fork launch", err);
}

}  // extern "C"
