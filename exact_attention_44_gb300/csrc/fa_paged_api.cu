// C ABI of the paged-cache operators (fa_fwd_paged, fa_cache_append,
// fa_cache_commit, fa_cache_fork): argument validation, the choice of kernel,
// launch.
#include <algorithm>
#include <cmath>
#include <cstdint>

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
fa_status check_cache(int Z, int P, int page_size, int max_pages, const int32_t* table, int64_t table_stride,
                      bool written) {
    if (Z < 0 || P < 0 || max_pages < 0 || table_stride < 0) return FA_ERR_INVALID_ARG;
    if (page_size < 16 || page_size % 16 != 0) return FA_ERR_UNSUPPORTED;
    if ((int64_t)max_pages * page_size > (int64_t(1) << 30) || Z > 65535) return FA_ERR_UNSUPPORTED;
    if ((int64_t)Z * max_pages > 0) {
        if (table == nullptr) return FA_ERR_INVALID_ARG;
        if (misaligned(table, 4)) return FA_ERR_ALIGNMENT;
        if (written && Z > 1 && table_stride < max_pages) return FA_ERR_INVALID_ARG;
    }
    return FA_OK;
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

fa::CacheView view(void* base, const fa_strides* s, int64_t layer) {
    return fa::CacheView{static_cast<uint16_t*>(base), layer, s->b, s->h, s->n};
}

fa_status check_layers(int L, int64_t layer_stride) {
    if (L < 0) return FA_ERR_INVALID_ARG;
    if (L > 1 && (layer_stride <= 0 || layer_stride % 8 != 0 || layer_stride >= (int64_t(1) << 42)))
        return FA_ERR_ALIGNMENT;
    return FA_OK;
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

fa_status fa_fwd_paged(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse,
                       const int32_t* block_table, const int32_t* seq_lens, const int32_t* new_lens,
                       const int32_t* tree_mask, int Z, int Hq, int Hkv, int T, int D, int P, int page_size,
                       int max_pages, int64_t table_stride, int64_t mask_stride, const fa_strides* sq,
                       const fa_strides* sk, const fa_strides* sv, const fa_strides* so, float scale, fa_dtype dtype,
                       void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (Hq < 0 || Hkv < 1 || T < 0 || Hq % Hkv != 0 || mask_stride < 0) return FA_ERR_INVALID_ARG;
    if (!head_dim_ok(D) || (dtype != FA_DTYPE_F16 && dtype != FA_DTYPE_BF16)) return FA_ERR_UNSUPPORTED;
    float c = 0.f;
    int negate = 0;
    if (!fa::split_scale(scale, &c, &negate)) return FA_ERR_INVALID_ARG;
    fa_status st = check_cache(Z, P, page_size, max_pages, block_table, table_stride, false);
    if (st != FA_OK) return st;
    const int G = Hq / Hkv;
    const int64_t rows = (int64_t)Z * Hq * T;
    // (row and tile indices fit in 32 bits)
    if ((int64_t)T * G > (int64_t(1) << 30) || (int64_t)Z * Hkv * cdiv((int64_t)T * G, 16) > INT32_MAX)
        return FA_ERR_UNSUPPORTED;
    if (rows == 0) return FA_OK;
    if ((st = check_strided(q, sq, Z, Hq, T, false)) != FA_OK) return st;
    if ((st = check_strided(o, so, Z, Hq, T, true)) != FA_OK) return st;
    if ((st = check_strided(k_cache, sk, P, Hkv, page_size, false)) != FA_OK) return st;
    if ((st = check_strided(v_cache, sv, P, Hkv, page_size, false)) != FA_OK) return st;
    if ((st = check_ints(seq_lens, true)) != FA_OK) return st;
    if ((st = check_ints(new_lens, false)) != FA_OK) return st;
    if ((st = check_ints(tree_mask, false)) != FA_OK) return st;
    if ((st = check_ints(lse, false)) != FA_OK) return st;
    if (workspace == nullptr || misaligned(workspace, 256)) return FA_ERR_WORKSPACE;

    fa::DeviceFacts f;
    cudaError_t err = fa::device_facts(&f);
    if (err != cudaSuccess) return fa::report_cuda("device query", err);
    if (workspace_bytes < paged_workspace_bytes(D, f.sms)) return FA_ERR_WORKSPACE;

    fa::PagedLaunch a{};
    fa::PagedParams& p = a.params;
    p.q = q;
    p.kc = k_cache;
    p.vc = v_cache;
    p.o = o;
    p.lse = lse;
    p.sq_z = sq->b, p.sq_h = sq->h, p.sq_n = sq->n;
    p.so_z = so->b, p.so_h = so->h, p.so_n = so->n;
    p.sk_p = sk->b, p.sk_h = sk->h, p.sk_n = sk->n;
    p.sv_p = sv->b, p.sv_h = sv->h, p.sv_n = sv->n;
    p.table = block_table;
    p.st_z = table_stride;
    p.lens = seq_lens;
    p.news = new_lens;
    p.mask = reinterpret_cast<const uint32_t*>(tree_mask);
    p.sm_z = mask_stride;
    p.words = (T + 31) / 32;
    p.Z = Z, p.Hq = Hq, p.Hkv = Hkv, p.G = G, p.T = T;
    p.page = page_size, p.M = max_pages, p.P = P;
    p.cap = P > 0 ? max_pages * page_size : 0;  // a cache without pages holds nothing
    p.scratch = static_cast<float*>(workspace);
    p.status = f.status;
    p.wait_limit_ns = f.wait_limit_ns;
    p.inject_stall = f.inject_stall;
    a.stream = stream;

    const bool bf16 = dtype == FA_DTYPE_BF16;
    // Few rows of a (sequence, kv head) run on the rows kernel.  The tile
    // kernel needs a whole group in a tile.
    a.tiles = T * (int64_t)G > 16 && G <= 128;
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
        const MapDim dq[3] = {{Hq, sq->h, G}, {T, sq->n, tokens}, {Z, sq->b, 1}};
        if (make_paged_map(&mq, q, bf16, D, dq) != CUDA_SUCCESS) return FA_ERR_CUDA;
        a.tmQ = &mq;
    } else {
        const RowsFacts rf = rows_facts(D);
        bk = rf.block;
        workers = std::min(rf.workers * f.sms, kMaxTeams);
        p.tile_rows = 16;
        p.scale_log2 = negate ? -c : c;
        p.slot_floats = slot_floats(16, D);
    }
    p.box_rows = box_rows_for(page_size, bk);
    if (P > 0) {
        const MapDim dk[3] = {{page_size, sk->n, p.box_rows}, {Hkv, sk->h, 1}, {P, sk->b, 1}};
        const MapDim dv[3] = {{page_size, sv->n, p.box_rows}, {Hkv, sv->h, 1}, {P, sv->b, 1}};
        if (make_paged_map(&mk, k_cache, bf16, D, dk) != CUDA_SUCCESS || make_paged_map(&mv, v_cache, bf16, D, dv) != CUDA_SUCCESS)
            return FA_ERR_CUDA;
    }
    a.tmK = &mk;
    a.tmV = &mv;
    p.tiles = (int)cdiv((int64_t)T * G, p.tile_rows);
    p.team = a.tiles ? std::min(p.tiles, 8) : 1;
    // more teams than there can be blocks would find no work
    const int64_t blocks = (int64_t)Z * Hkv * cdiv(p.tiles, p.team) * cdiv(p.cap, bk);
    p.teams = (int)std::max<int64_t>(1, std::min<int64_t>(blocks, workers / p.team));
    p.cuts = static_cast<char*>(workspace) + paged_slot_bytes(D, f.sms);
    err = launch_paged(D, a, bf16);
    return err == cudaSuccess ? FA_OK : fa::report_cuda("paged attention launch", err);
}

fa_status fa_cache_append(const void* k, const void* v, void* k_cache, void* v_cache, const int32_t* block_table,
                          const int32_t* seq_lens, const int32_t* new_lens, int Z, int Hkv, int T, int D, int P,
                          int page_size, int max_pages, int64_t table_stride, const fa_strides* sk,
                          const fa_strides* sv, const fa_strides* skc, const fa_strides* svc, cudaStream_t stream) {
    if (Hkv < 0 || T < 0) return FA_ERR_INVALID_ARG;
    if (!head_dim_ok(D)) return FA_ERR_UNSUPPORTED;
    fa_status st = check_cache(Z, P, page_size, max_pages, block_table, table_stride, false);
    if (st != FA_OK) return st;
    if ((int64_t)Hkv * T * (D / 8) >= INT32_MAX) return FA_ERR_UNSUPPORTED;
    if ((int64_t)Z * Hkv * T == 0) return FA_OK;
    if ((st = check_strided(k, sk, Z, Hkv, T, false)) != FA_OK) return st;
    if ((st = check_strided(v, sv, Z, Hkv, T, false)) != FA_OK) return st;
    if ((st = check_strided(k_cache, skc, P, Hkv, page_size, true)) != FA_OK) return st;
    if ((st = check_strided(v_cache, svc, P, Hkv, page_size, true)) != FA_OK) return st;
    if ((st = check_ints(seq_lens, true)) != FA_OK) return st;
    if ((st = check_ints(new_lens, false)) != FA_OK) return st;
    fa::DeviceFacts f;
    cudaError_t err = fa::device_facts(&f);
    if (err != cudaSuccess) return fa::report_cuda("device query", err);
    fa::AppendParams p{};
    p.k = view(k_cache, skc, 0);
    p.v = view(v_cache, svc, 0);
    p.ks = static_cast<const uint16_t*>(k);
    p.vs = static_cast<const uint16_t*>(v);
    p.ks_z = sk->b, p.ks_h = sk->h, p.ks_n = sk->n;
    p.vs_z = sv->b, p.vs_h = sv->h, p.vs_n = sv->n;
    p.table = block_table;
    p.st_z = table_stride;
    p.lens = seq_lens;
    p.news = new_lens;
    p.Z = Z, p.H = Hkv, p.T = T, p.D = D, p.page = page_size, p.M = max_pages, p.P = P;
    p.status = f.status;
    err = fa::launch_cache_append(p, stream);
    return err == cudaSuccess ? FA_OK : fa::report_cuda("cache append launch", err);
}

fa_status fa_cache_commit(void* k_cache, void* v_cache, const int32_t* block_table, const int32_t* seq_lens,
                          const int32_t* accepted, const int32_t* accepted_lens, int Z, int L, int Hkv, int A, int D,
                          int P, int page_size, int max_pages, int64_t table_stride, int64_t accepted_stride,
                          int64_t k_layer_stride, int64_t v_layer_stride, const fa_strides* skc, const fa_strides* svc,
                          cudaStream_t stream) {
    if (Hkv < 0 || A < 0 || accepted_stride < 0) return FA_ERR_INVALID_ARG;
    if (!head_dim_ok(D)) return FA_ERR_UNSUPPORTED;
    fa_status st = check_cache(Z, P, page_size, max_pages, block_table, table_stride, false);
    if (st != FA_OK) return st;
    if ((st = check_layers(L, k_layer_stride)) != FA_OK || (st = check_layers(L, v_layer_stride)) != FA_OK) return st;
    if ((int64_t)L * 2 * Hkv * (D / 8) >= INT32_MAX) return FA_ERR_UNSUPPORTED;
    if ((int64_t)Z * L * Hkv * A == 0) return FA_OK;
    if ((st = check_strided(k_cache, skc, P, Hkv, page_size, true)) != FA_OK) return st;
    if ((st = check_strided(v_cache, svc, P, Hkv, page_size, true)) != FA_OK) return st;
    if ((st = check_ints(seq_lens, true)) != FA_OK) return st;
    if ((st = check_ints(accepted, true)) != FA_OK) return st;
    if ((st = check_ints(accepted_lens, true)) != FA_OK) return st;
    fa::DeviceFacts f;
    cudaError_t err = fa::device_facts(&f);
    if (err != cudaSuccess) return fa::report_cuda("device query", err);
    fa::CommitParams p{};
    p.k = view(k_cache, skc, k_layer_stride);
    p.v = view(v_cache, svc, v_layer_stride);
    p.table = block_table;
    p.st_z = table_stride;
    p.lens = seq_lens;
    p.path = accepted;
    p.kept = accepted_lens;
    p.sp_z = accepted_stride;
    p.Z = Z, p.L = L, p.H = Hkv, p.A = A, p.D = D, p.page = page_size, p.M = max_pages, p.P = P;
    p.status = f.status;
    err = fa::launch_cache_commit(p, stream);
    return err == cudaSuccess ? FA_OK : fa::report_cuda("cache commit launch", err);
}

fa_status fa_cache_fork_workspace_size(int Z, int max_pages, size_t* bytes) {
    if (bytes == nullptr || Z < 0 || max_pages < 0) return FA_ERR_INVALID_ARG;
    *bytes = (size_t)fa::fork_workspace_ints(Z, max_pages) * sizeof(int32_t);
    return FA_OK;
}

fa_status fa_cache_fork(void* k_cache, void* v_cache, int32_t* block_table, int32_t* seq_lens, int32_t* ref_counts,
                        const int32_t* source, int32_t* missing, int Z, int L, int Hkv, int D, int P, int page_size,
                        int max_pages, int room, int64_t table_stride, int64_t k_layer_stride, int64_t v_layer_stride,
                        const fa_strides* skc, const fa_strides* svc, void* workspace, size_t workspace_bytes,
                        cudaStream_t stream) {
    if (Hkv < 0 || room < 0) return FA_ERR_INVALID_ARG;
    if (!head_dim_ok(D)) return FA_ERR_UNSUPPORTED;
    fa_status st = check_cache(Z, P, page_size, max_pages, block_table, table_stride, true);
    if (st != FA_OK) return st;
    if ((st = check_layers(L, k_layer_stride)) != FA_OK || (st = check_layers(L, v_layer_stride)) != FA_OK) return st;
    if (Z > 8192 || room > (1 << 30) || (int64_t)Z * max_pages > INT32_MAX || (int64_t)Hkv * page_size * (D / 8) > INT32_MAX)
        return FA_ERR_UNSUPPORTED;
    if (Z == 0) return FA_OK;
    if ((int64_t)L * Hkv > 0) {
        if ((st = check_strided(k_cache, skc, P, Hkv, page_size, true)) != FA_OK) return st;
        if ((st = check_strided(v_cache, svc, P, Hkv, page_size, true)) != FA_OK) return st;
    }
    if ((st = check_ints(seq_lens, true)) != FA_OK) return st;
    if ((st = check_ints(ref_counts, P > 0)) != FA_OK) return st;
    if ((st = check_ints(source, false)) != FA_OK) return st;
    if ((st = check_ints(missing, false)) != FA_OK) return st;
    if (workspace == nullptr || misaligned(workspace, 256) ||
        workspace_bytes < (size_t)fa::fork_workspace_ints(Z, max_pages) * sizeof(int32_t))
        return FA_ERR_WORKSPACE;
    fa::DeviceFacts f;
    cudaError_t err = fa::device_facts(&f);
    if (err != cudaSuccess) return fa::report_cuda("device query", err);
    fa::ForkParams p{};
    static const fa_strides none{0, 0, 0, 1};
    p.k = view(k_cache, skc != nullptr ? skc : &none, k_layer_stride);
    p.v = view(v_cache, svc != nullptr ? svc : &none, v_layer_stride);
    p.table = block_table;
    p.st_z = table_stride;
    p.lens = seq_lens;
    p.refs = ref_counts;
    p.source = source;
    p.missing = missing;
    p.Z = Z, p.L = L, p.H = Hkv, p.D = D, p.page = page_size, p.M = max_pages, p.P = P, p.room = room;
    p.ws = static_cast<int32_t*>(workspace);
    p.status = f.status;
    err = fa::launch_cache_fork(p, f.sms, stream);
    return err == cudaSuccess ? FA_OK : fa::report_cuda("cache fork launch", err);
}

}  // extern "C"
