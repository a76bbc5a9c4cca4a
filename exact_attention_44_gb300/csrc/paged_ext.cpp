// Python binding of the paged-cache entry points and of rotary positions: argument
// checks and marshalling only.  A decode step makes two or three of these calls a layer,
// each a few microseconds of GPU time; through ctypes and Python the host side
// of one took 7 to 16 us, so it is a CPython extension over torch's tensors.
// The functions of libfa are handed over by address (bind), so the extension
// calls whichever build of the library the package has loaded.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_strided.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/function.h>
#include <torch/csrc/autograd/functions/utils.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/autograd/saved_variable.h>

#include <climits>
#include <cmath>
#include <initializer_list>
#include <memory>
#include <mutex>
#include <stdexcept>
#include <string>
#include <utility>

#include "fa.h"

namespace {

struct Library {
    decltype(&fa_fwd_paged) fwd = nullptr;
    decltype(&fa_fwd_paged_workspace_size) fwd_size = nullptr;
    decltype(&fa_cache_append) append = nullptr;
    decltype(&fa_cache_commit) commit = nullptr;
    decltype(&fa_cache_fork) fork = nullptr;
    decltype(&fa_cache_fork_workspace_size) fork_size = nullptr;
    decltype(&fa_rope) rope = nullptr;
    decltype(&fa_cache_append_rope) append_rope = nullptr;
    decltype(&fa_cache_score) score = nullptr;
    decltype(&fa_cache_score_workspace_size) score_size = nullptr;
    decltype(&fa_cache_evict) evict = nullptr;
    decltype(&fa_cache_evict_workspace_size) evict_size = nullptr;
    PyObject* error = nullptr;  // the package's FaError
} lib;

// A refused argument: the Python exception to raise.
struct Refused : std::runtime_error {
    PyObject* type;
    Refused(PyObject* t, const std::string& text) : std::runtime_error(text), type(t) {}
};
[[noreturn]] void value_error(std::string text) { throw Refused(PyExc_ValueError, text); }
[[noreturn]] void type_error(std::string text) { throw Refused(PyExc_TypeError, text); }

std::string shape_of(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}

// A tensor argument; null for None.
const at::Tensor* maybe_tensor(PyObject* o, const char* name) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
    return &THPVariable_Unpack(o);
}
const at::Tensor& tensor(PyObject* o, const char* name) {
    const at::Tensor* t = maybe_tensor(o, name);
    if (t == nullptr) type_error(std::string(name) + " must be a tensor");
    return *t;
}
int to_int(int64_t x, const char* name) {
    if (x > INT_MAX || x < INT_MIN) value_error(std::string(name) + " is out of range");
    return (int)x;
}
int int_arg(PyObject* o, const char* name) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw python_error();
    return to_int(x, name);
}

void check_ints(const at::Tensor& t, const char* name, std::initializer_list<int64_t> shape) {
    if (t.scalar_type() != at::kInt) type_error(std::string(name) + " must be int32");
    const at::IntArrayRef want(shape);
    if (t.sizes() != want) value_error(std::string(name) + " must have shape " + shape_of(want) + ", got " + shape_of(t.sizes()));
    if (want.back() > 1 && t.stride(-1) != 1) value_error(std::string(name) + "'s last dimension must be contiguous");
}
int32_t* ints(const at::Tensor* t) { return t == nullptr ? nullptr : static_cast<int32_t*>(t->data_ptr()); }

fa_strides strides4(const at::Tensor& t) {
    const auto s = t.strides();
    return fa_strides{s[0], s[1], s[2], s[3]};
}

// The cache's fields; layers: whether 5-D caches are allowed.
fa_paged_cache cache_of(const at::Tensor& k, const at::Tensor& v, const at::Tensor& table, const at::Tensor& lens,
                        int64_t Z, bool layers) {
    const auto shape = k.sizes();
    const size_t n = shape.size();
    if (shape != v.sizes() || !(n == 4 || (layers && n == 5)))
        value_error(std::string("k_cache and v_cache must both be (pages, Hkv, page_size, D)") +
                    (layers ? " or (layers, pages, Hkv, page_size, D)" : "") + ", got " + shape_of(shape) + ", " +
                    shape_of(v.sizes()));
    if (k.scalar_type() != v.scalar_type() || k.element_size() != 2)
        type_error("k_cache and v_cache must share one 16-bit dtype");
    if (table.scalar_type() != at::kInt) type_error("block_table must be int32");
    if (table.dim() != 2 || table.size(0) != Z)
        value_error("block_table must be (Z, max_pages) = (" + std::to_string(Z) + ", ...), got " + shape_of(table.sizes()));
    if (table.size(1) > 1 && table.stride(1) != 1) value_error("block_table rows must be contiguous");
    check_ints(lens, "seq_lens", {Z});
    const size_t d = n - 4;
    const auto ks = k.strides(), vs = v.strides();
    fa_paged_cache c{};
    c.k = k.data_ptr();
    c.v = v.data_ptr();
    c.sk = fa_strides{ks[d], ks[d + 1], ks[d + 2], ks[d + 3]};
    c.sv = fa_strides{vs[d], vs[d + 1], vs[d + 2], vs[d + 3]};
    if (d) {
        c.k_layer = ks[0];
        c.v_layer = vs[0];
    }
    c.block_table = ints(&table);
    c.table_stride = table.stride(0);
    c.seq_lens = ints(&lens);
    c.Z = to_int(Z, "the batch");
    c.L = d ? to_int(shape[0], "the layers") : 1;
    c.P = to_int(shape[d], "the pages");
    c.Hkv = to_int(shape[d + 1], "the heads");
    c.page_size = to_int(shape[d + 2], "page_size");
    c.D = to_int(shape[d + 3], "the head dim");
    c.max_pages = to_int(table.size(1), "max_pages");
    return c;
}

int cuda_device(const char* call, const at::Tensor& lead, std::initializer_list<const at::Tensor*> others) {
    for (const at::Tensor* t : others)
        if (t != nullptr && t->device() != lead.device())
            value_error(std::string(call) + ": every tensor must be on " + lead.device().str() + ", got one on " +
                        t->device().str());
    if (!lead.is_cuda()) value_error(std::string(call) + " takes CUDA tensors");
    return lead.get_device();
}

// The device and stream of a call: the given stream (its handle, an int), else
// torch's current one.  What is allocated meanwhile belongs to that stream, and
// the tensors of a call on another stream than the current one are kept from
// reuse until that stream has passed the call.
class Place {
  public:
    Place(PyObject* o, int device, std::initializer_list<const at::Tensor*> used)
        : device_((c10::DeviceIndex)device), stream_(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device)) {
        if (o == Py_None) return;
        void* p = PyLong_AsVoidPtr(o);
        if (p == nullptr && PyErr_Occurred()) throw python_error();
        if (static_cast<cudaStream_t>(p) == stream_.stream()) return;
        stream_ = c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(p), (c10::DeviceIndex)device);
        guard_.reset_stream(stream_);
        for (const at::Tensor* t : used)
            if (t != nullptr && t->has_storage())
                c10::cuda::CUDACachingAllocator::recordStream(t->storage().data_ptr(), stream_);
    }
    cudaStream_t stream() const { return stream_.stream(); }

  private:
    c10::cuda::CUDAGuard device_;
    c10::cuda::CUDAStream stream_;
    c10::cuda::OptionalCUDAStreamGuard guard_;
};

void check(fa_status st, const char* call) {
    if (st == FA_OK) return;
    if (PyObject* e = PyObject_CallFunction(lib.error, "is", (int)st, call)) {
        PyErr_SetObject(lib.error, e);
        Py_DECREF(e);
    }
    throw python_error();
}

// Runs fn without the interpreter lock (a launch can wait for the queue).
template <typename F>
fa_status unlocked(F&& fn) {
    PyThreadState* state = PyEval_SaveThread();
    const fa_status st = fn();
    PyEval_RestoreThread(state);
    return st;
}

// A call has written these: autograd may have saved them, and compares versions.
void written(std::initializer_list<const at::Tensor*> tensors) {
    for (const at::Tensor* t : tensors)
        if (t != nullptr && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

// A workspace argument: its bytes are counted, so they must lie together.
void check_workspace(const at::Tensor* t) {
    if (t != nullptr && !t->is_contiguous()) value_error("workspace must be contiguous");
}

at::Tensor scratch(size_t bytes, const at::Tensor& like) {
    return at::empty({(int64_t)bytes}, like.options().dtype(at::kByte));
}

template <typename F>
PyObject* guarded(F&& fn) {
    HANDLE_TH_ERRORS
    try {
        if (lib.fwd == nullptr) throw Refused(PyExc_ImportError, "libfa is not loaded");
        return fn();
    } catch (const Refused& r) {
        PyErr_SetString(r.type, r.what());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

bool expect(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return false;
}

// (q, k_cache, v_cache, block_table, seq_lens, o, lse, new_lens, tree_mask, scale, workspace, stream, want_lse)
PyObject* fwd_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!expect(n, 13)) return nullptr;
    return guarded([&]() -> PyObject* {
        const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k_cache"), &v = tensor(a[2], "v_cache");
        const at::Tensor &table = tensor(a[3], "block_table"), &lens = tensor(a[4], "seq_lens");
        const at::Tensor *o_arg = maybe_tensor(a[5], "o"), *lse_arg = maybe_tensor(a[6], "lse");
        const at::Tensor *news = maybe_tensor(a[7], "new_lens"), *mask = maybe_tensor(a[8], "tree_mask");
        const at::Tensor* ws_arg = maybe_tensor(a[10], "workspace");
        if (q.dim() != 4) value_error("q must be 4-D (Z, Hq, T, D)");
        const int64_t Z = q.size(0), Hq = q.size(1), T = q.size(2), D = q.size(3);
        fa_fwd_paged_args x{};
        x.cache = cache_of(k, v, table, lens, Z, false);
        if (x.cache.D != D)
            value_error("head dims differ: q has " + std::to_string(D) + ", the cache " + std::to_string(x.cache.D));
        if (q.scalar_type() == at::kBFloat16) x.dtype = FA_DTYPE_BF16;
        else if (q.scalar_type() == at::kHalf) x.dtype = FA_DTYPE_F16;
        else type_error("fa_fwd_paged takes float16 or bfloat16 tensors");
        if (k.scalar_type() != q.scalar_type()) type_error("q and the caches must share one dtype");
        if (news != nullptr) check_ints(*news, "new_lens", {Z});
        if (mask != nullptr) {
            const int64_t words = (T + 31) / 32;
            if (mask->dim() == 3) {
                check_ints(*mask, "tree_mask", {Z, T, words});
                x.mask_stride = mask->stride(0);
            } else {
                check_ints(*mask, "tree_mask", {T, words});
            }
            if (T > 1 && mask->stride(-2) != words) value_error("tree_mask's words must be contiguous within a sequence");
        }
        if (o_arg != nullptr && (o_arg->sizes() != q.sizes() || o_arg->scalar_type() != q.scalar_type()))
            value_error("o must match q's shape and dtype");
        if (lse_arg != nullptr && (lse_arg->scalar_type() != at::kFloat || lse_arg->dim() != 3 ||
                                   lse_arg->sizes() != q.sizes().slice(0, 3) || !lse_arg->is_contiguous()))
            value_error("lse must be a contiguous float32 (Z, Hq, T) tensor");
        double scale = 1.0 / std::sqrt((double)D);
        if (a[9] != Py_None) {
            scale = PyFloat_AsDouble(a[9]);
            if (scale == -1.0 && PyErr_Occurred()) throw python_error();
        }
        const int want = PyObject_IsTrue(a[12]);
        if (want < 0) throw python_error();
        check_workspace(ws_arg);
        const int dev = cuda_device("fa_fwd_paged", q, {&k, &v, &table, &lens, o_arg, lse_arg, news, mask, ws_arg});
        const Place place(a[11], dev, {&q, &k, &v, &table, &lens, o_arg, lse_arg, news, mask, ws_arg});
        at::Tensor o = o_arg != nullptr ? *o_arg : at::empty(q.sizes(), q.options());
        at::Tensor lse, ws;
        if (lse_arg != nullptr) lse = *lse_arg;
        else if (want) lse = at::empty(q.sizes().slice(0, 3), q.options().dtype(at::kFloat));
        if (ws_arg != nullptr) {
            ws = *ws_arg;
        } else {
            size_t bytes = 0;
            check(lib.fwd_size((int)D, &bytes), "fa_fwd_paged");
            ws = scratch(bytes, q);
        }
        x.q = q.data_ptr();
        x.o = o.data_ptr();
        x.lse = lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr;
        x.sq = strides4(q);
        x.so = strides4(o);
        x.new_lens = ints(news);
        x.tree_mask = ints(mask);
        x.workspace = ws.data_ptr();
        x.workspace_bytes = ws.nbytes();
        x.Hq = to_int(Hq, "the heads");
        x.T = to_int(T, "T");
        x.scale = (float)scale;
        check(unlocked([&] { return lib.fwd(&x, place.stream()); }), "fa_fwd_paged");
        PyObject* result = PyTuple_New(2);
        if (result == nullptr) throw python_error();
        PyTuple_SET_ITEM(result, 0, THPVariable_Wrap(o));
        if (lse.defined()) PyTuple_SET_ITEM(result, 1, THPVariable_Wrap(lse));
        else PyTuple_SET_ITEM(result, 1, (Py_INCREF(Py_None), Py_None));
        return result;
    });
}

// (k, v, k_cache, v_cache, block_table, seq_lens, new_lens, stream)
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!expect(n, 8)) return nullptr;
    return guarded([&]() -> PyObject* {
        const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
        const at::Tensor &kc = tensor(a[2], "k_cache"), &vc = tensor(a[3], "v_cache");
        const at::Tensor &table = tensor(a[4], "block_table"), &lens = tensor(a[5], "seq_lens");
        const at::Tensor* news = maybe_tensor(a[6], "new_lens");
        if (k.dim() != 4 || k.sizes() != v.sizes())
            value_error("k and v must both be (Z, Hkv, T, D), got " + shape_of(k.sizes()) + ", " + shape_of(v.sizes()));
        const int64_t Z = k.size(0);
        fa_cache_append_args x{};
        x.cache = cache_of(kc, vc, table, lens, Z, false);
        if (x.cache.Hkv != k.size(1) || x.cache.D != k.size(3))
            value_error("k and v must both be (Z, " + std::to_string(x.cache.Hkv) + ", T, " + std::to_string(x.cache.D) +
                        "), got " + shape_of(k.sizes()));
        if (k.scalar_type() != kc.scalar_type() || v.scalar_type() != kc.scalar_type())
            type_error("k and v must have the cache's dtype");
        if (news != nullptr) check_ints(*news, "new_lens", {Z});
        const int dev = cuda_device("fa_cache_append", k, {&v, &kc, &vc, &table, &lens, news});
        const Place place(a[7], dev, {&k, &v, &kc, &vc, &table, &lens, news});
        x.k = k.data_ptr();
        x.v = v.data_ptr();
        x.sk = strides4(k);
        x.sv = strides4(v);
        x.new_lens = ints(news);
        x.T = to_int(k.size(2), "T");
        check(unlocked([&] { return lib.append(&x, place.stream()); }), "fa_cache_append");
        Py_RETURN_NONE;
    });
}

// (k_cache, v_cache, block_table, seq_lens, accepted, accepted_lens, stream)
PyObject* cache_commit(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!expect(n, 7)) return nullptr;
    return guarded([&]() -> PyObject* {
        const at::Tensor &kc = tensor(a[0], "k_cache"), &vc = tensor(a[1], "v_cache");
        const at::Tensor &table = tensor(a[2], "block_table"), &lens = tensor(a[3], "seq_lens");
        const at::Tensor &path = tensor(a[4], "accepted"), &kept = tensor(a[5], "accepted_lens");
        if (path.dim() != 2) value_error("accepted must be (Z, A)");
        const int64_t Z = path.size(0);
        check_ints(path, "accepted", {Z, path.size(1)});
        check_ints(kept, "accepted_lens", {Z});
        fa_cache_commit_args x{};
        x.cache = cache_of(kc, vc, table, lens, Z, true);
        const int dev = cuda_device("fa_cache_commit", kc, {&vc, &table, &lens, &path, &kept});
        const Place place(a[6], dev, {&kc, &vc, &table, &lens, &path, &kept});
        x.accepted = ints(&path);
        x.accepted_stride = path.stride(0);
        x.accepted_lens = ints(&kept);
        x.A = to_int(path.size(1), "A");
        check(unlocked([&] { return lib.commit(&x, place.stream()); }), "fa_cache_commit");
        Py_RETURN_NONE;
    });
}

// (k_cache, v_cache, block_table, seq_lens, ref_counts, source, room, missing, workspace, stream, all_or_nothing)
PyObject* cache_fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!expect(n, 11)) return nullptr;
    return guarded([&]() -> PyObject* {
        const at::Tensor &kc = tensor(a[0], "k_cache"), &vc = tensor(a[1], "v_cache");
        const at::Tensor &table = tensor(a[2], "block_table"), &lens = tensor(a[3], "seq_lens");
        const at::Tensor &refs = tensor(a[4], "ref_counts"), *source = maybe_tensor(a[5], "source");
        const at::Tensor *missing = maybe_tensor(a[7], "missing"), *ws_arg = maybe_tensor(a[8], "workspace");
        if (lens.dim() != 1) value_error("seq_lens must be (Z)");
        const int64_t Z = lens.size(0);
        fa_cache_fork_args x{};
        x.cache = cache_of(kc, vc, table, lens, Z, true);
        check_ints(refs, "ref_counts", {x.cache.P});
        if (source != nullptr) check_ints(*source, "source", {Z});
        if (missing != nullptr) check_ints(*missing, "missing", {1});
        const int whole = PyObject_IsTrue(a[10]);
        if (whole < 0) throw python_error();
        if (whole && missing == nullptr) value_error("all_or_nothing needs missing, which says whether anything was done");
        x.room = int_arg(a[6], "room");
        x.all_or_nothing = whole;
        check_workspace(ws_arg);
        const int dev = cuda_device("fa_cache_fork", kc, {&vc, &table, &lens, &refs, source, missing, ws_arg});
        const Place place(a[9], dev, {&kc, &vc, &table, &lens, &refs, source, missing, ws_arg});
        at::Tensor ws;
        if (ws_arg != nullptr) {
            ws = *ws_arg;
        } else {
            size_t bytes = 0;
            check(lib.fork_size(x.cache.Z, x.cache.max_pages, &bytes), "fa_cache_fork");
            ws = scratch(bytes, kc);
        }
        x.ref_counts = ints(&refs);
        x.source = ints(source);
        x.missing = ints(missing);
        x.workspace = ws.data_ptr();
        x.workspace_bytes = ws.nbytes();
        check(unlocked([&] { return lib.fork(&x, place.stream()); }), "fa_cache_fork");
        Py_RETURN_NONE;
    });
}

fa_dtype dtype_of(const at::Tensor& t, const char* call) {
    if (t.scalar_type() == at::kBFloat16) return FA_DTYPE_BF16;
    if (t.scalar_type() == at::kHalf) return FA_DTYPE_F16;
    type_error(std::string(call) + " takes float16 or bfloat16 tensors");
}
float float_arg(PyObject* o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw python_error();
    return (float)x;
}
int flag_arg(PyObject* o) {
    const int x = PyObject_IsTrue(o);
    if (x < 0) throw python_error();
    return x;
}
// The frequencies' pairs.
int pairs_of(const at::Tensor& turns) {
    if (turns.scalar_type() != at::kLong || turns.dim() != 1 || !turns.is_contiguous() || !turns.device().is_cpu())
        value_error("turns must be a contiguous int64 tensor of rotary_dim / 2 entries on the host (fa_rope_turns)");
    return to_int(2 * turns.size(0), "rotary_dim");
}
// (N,) for all sequences or (Z, N); the stride between sequences
int64_t positions_stride(const at::Tensor& t, int64_t Z, int64_t N) {
    if (t.dim() == 1) {
        check_ints(t, "positions", {N});
        return 0;
    }
    check_ints(t, "positions", {Z, N});
    return t.stride(0);
}
void check_out(const at::Tensor* out, const at::Tensor& like, const char* name) {
    if (out != nullptr && (out->sizes() != like.sizes() || out->scalar_type() != like.scalar_type()))
        value_error(std::string(name) + " must match its input's shape and dtype");
}
// A tensor for the outputs of `like`: its layout if that is dense with the last dimension contiguous.
at::Tensor out_like(const at::Tensor& like) {
    const bool keep = like.is_non_overlapping_and_dense() && (like.size(3) <= 1 || like.stride(3) == 1);
    return keep ? at::empty_strided(like.sizes(), like.strides(), like.options()) : at::empty(like.sizes(), like.options());
}

// A call that failed where there may be no interpreter (the gradient's thread).
struct Failed : std::runtime_error {
    fa_status status;
    Failed(fa_status st, const char* call)
        : std::runtime_error(std::string(call) + ": status " + std::to_string((int)st)), status(st) {}
};

// Arguments of fa_rope but for the outputs; k may be null.
fa_rope_args rope_args(const at::Tensor& q, const at::Tensor* k, const at::Tensor& turns, const at::Tensor* pos, bool interleaved,
                       bool inverse, double factor) {
    if (q.dim() != 4) value_error("q must be 4-D (Z, H, N, D)");
    fa_rope_args x{};
    x.dtype = dtype_of(q, "fa_rope");
    if (k != nullptr) {
        if (k->dim() != 4 || k->size(0) != q.size(0) || k->size(2) != q.size(2) || k->size(3) != q.size(3))
            value_error("k must be (Z, Hk, N, D) like q, got " + shape_of(k->sizes()) + " for " + shape_of(q.sizes()));
        if (k->scalar_type() != q.scalar_type()) type_error("q and k must share one dtype");
        x.k = k->data_ptr();
        x.sk = strides4(*k);
        x.Hk = to_int(k->size(1), "the heads");
    }
    x.rotary_dim = pairs_of(turns);
    if (pos != nullptr) x.positions_stride = positions_stride(*pos, q.size(0), q.size(2));
    x.interleaved = interleaved;
    x.inverse = inverse;
    x.factor = (float)factor;
    x.q = q.data_ptr();
    x.sq = strides4(q);
    x.positions = ints(pos);
    x.turns = static_cast<const int64_t*>(turns.data_ptr());
    x.Z = to_int(q.size(0), "the batch");
    x.Hq = to_int(q.size(1), "the heads");
    x.N = to_int(q.size(2), "the rows");
    x.D = to_int(q.size(3), "the head dim");
    return x;
}
void rope_outputs(fa_rope_args& x, const at::Tensor& qo, const at::Tensor& ko) {
    x.q_out = qo.data_ptr();
    x.sq_out = strides4(qo);
    if (ko.defined()) {
        x.k_out = ko.data_ptr();
        x.sk_out = strides4(ko);
    }
}
PyObject* pair(const at::Tensor& a, const at::Tensor& b) {
    PyObject* result = PyTuple_New(2);
    if (result == nullptr) throw python_error();
    PyTuple_SET_ITEM(result, 0, THPVariable_Wrap(a));
    if (b.defined()) PyTuple_SET_ITEM(result, 1, THPVariable_Wrap(b));
    else PyTuple_SET_ITEM(result, 1, (Py_INCREF(Py_None), Py_None));
    return result;
}

// (q, k, turns, positions, interleaved, inverse, factor, q_out, k_out, stream)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!expect(n, 10)) return nullptr;
    return guarded([&]() -> PyObject* {
        const at::Tensor &q = tensor(a[0], "q"), &turns = tensor(a[2], "turns");
        const at::Tensor *k = maybe_tensor(a[1], "k"), *pos = maybe_tensor(a[3], "positions");
        const at::Tensor *qo_arg = maybe_tensor(a[7], "q_out"), *ko_arg = maybe_tensor(a[8], "k_out");
        if (k == nullptr && ko_arg != nullptr) value_error("k_out without k");
        fa_rope_args x = rope_args(q, k, turns, pos, flag_arg(a[4]), flag_arg(a[5]), float_arg(a[6]));
        check_out(qo_arg, q, "q_out");
        if (k != nullptr) check_out(ko_arg, *k, "k_out");
        const int dev = cuda_device("fa_rope", q, {k, pos, qo_arg, ko_arg});
        const Place place(a[9], dev, {&q, k, pos, qo_arg, ko_arg});
        const at::Tensor qo = qo_arg != nullptr ? *qo_arg : out_like(q);
        at::Tensor ko;
        if (k != nullptr) ko = ko_arg != nullptr ? *ko_arg : out_like(*k);
        rope_outputs(x, qo, ko);
        check(unlocked([&] { return lib.rope(&x, place.stream()); }), "fa_rope");
        written({qo_arg, ko_arg});
        return pair(qo, ko);
    });
}

// A gradient comes with any strides: itself where fa_rope takes them, else a copy.
at::Tensor rows_of(const at::Tensor& t) {
    if (t.numel() == 0) return t;
    bool fine = t.stride(3) == 1 && reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0;
    for (int i = 0; i < 3; ++i) fine = fine && (t.size(i) <= 1 || t.stride(i) % 8 == 0);
    return fine ? t : t.contiguous();
}

// fa_rope with autograd.  The gradient is the turn back, by this same function, so that it
// has gradients of its own.  A graph node in C++: a step's Python side took 160 us of 21 us
// of kernels (4 x 32 heads x 1024 rows of D = 128, both directions).
using torch::autograd::variable_list;
struct Turn {  // how rows turn, but for the rows
    at::Tensor turns;
    int64_t version;  // of turns when the graph was made
    bool interleaved, inverse;
    double factor;
};
int64_t version_of(const at::Tensor& t) { return t.is_inference() ? 0 : (int64_t)t._version(); }
std::pair<at::Tensor, at::Tensor> turn_rows(const at::Tensor& q, const at::Tensor& k, const at::Tensor& pos, const Turn& how);

struct TurnBackward : public torch::autograd::Node {  // of q and k, or of the one that needs a gradient
    Turn how;
    torch::autograd::SavedVariable positions;
    bool has_positions = false;
    std::string name() const override { return "RotaryBackward"; }
    variable_list apply(variable_list&& grads) override {
        // an input with an edge, a gradient, and somebody who asked for it
        auto wanted = [&](size_t i) { return i < grads.size() && grads[i].defined() && task_should_compute_output(i); };
        const bool first = wanted(0), second = wanted(1);
        variable_list out(grads.size());
        if (!first && !second) return out;
        at::Tensor pos;
        {
            std::lock_guard<std::mutex> lock(mutex_);
            if (has_positions) pos = positions.unpack();
        }
        if (version_of(how.turns) != how.version)
            throw std::runtime_error("rotary: turns, needed for the gradient, has been modified by an inplace operation");
        const Turn back{how.turns, how.version, how.interleaved, !how.inverse, how.factor};
        const auto r = turn_rows(rows_of(grads[first ? 0 : 1]), first && second ? rows_of(grads[1]) : at::Tensor(), pos, back);
        if (first) out[0] = r.first;
        if (second) out[1] = first ? r.second : r.first;
        return out;
    }
    void release_variables() override {
        std::lock_guard<std::mutex> lock(mutex_);
        positions.reset_data();
    }
};

// k and pos may be undefined; so is the second result then.
std::pair<at::Tensor, at::Tensor> turn_rows(const at::Tensor& q, const at::Tensor& k, const at::Tensor& pos, const Turn& how) {
    // (the outputs would have none, which reads as a derivative of zero)
    for (const at::Tensor* t : {&q, &k})
        TORCH_CHECK_NOT_IMPLEMENTED(!t->defined() || !t->_fw_grad(0).defined(),
                                    "rotary has no forward-mode gradient: an input carries a tangent");
    const at::Tensor *kp = k.defined() ? &k : nullptr, *pp = pos.defined() ? &pos : nullptr;
    fa_rope_args x = rope_args(q, kp, how.turns, pp, how.interleaved, how.inverse, how.factor);
    const int dev = cuda_device("rotary", q, {kp, pp});
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    const at::Tensor qo = out_like(q), ko = kp != nullptr ? out_like(k) : at::Tensor();
    rope_outputs(x, qo, ko);
    const fa_status st = PyGILState_Check() ? unlocked([&] { return lib.rope(&x, stream); }) : lib.rope(&x, stream);
    if (st != FA_OK) throw Failed(st, "fa_rope");
    // an input that needs no gradient is not in the graph, nor is its output
    const bool q_needs = at::GradMode::is_enabled() && q.requires_grad();
    const bool k_needs = at::GradMode::is_enabled() && kp != nullptr && k.requires_grad();
    if (q_needs || k_needs) {
        std::shared_ptr<TurnBackward> node(new TurnBackward(), torch::autograd::deleteNode);
        node->how = how;
        if (pp != nullptr) {
            node->positions = torch::autograd::SavedVariable(pos, false);
            node->has_positions = true;
        }
        if (q_needs && k_needs) node->set_next_edges(torch::autograd::collect_next_edges(q, k));
        else node->set_next_edges(torch::autograd::collect_next_edges(q_needs ? q : k));
        if (q_needs) torch::autograd::set_history(qo, node);
        if (k_needs) torch::autograd::set_history(ko, node);
    }
    return {qo, ko};
}

// (q, k, turns, positions, interleaved, factor)
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!expect(n, 6)) return nullptr;
    return guarded([&]() -> PyObject* {
        const at::Tensor &q = tensor(a[0], "q"), &turns = tensor(a[2], "turns");
        const at::Tensor *k = maybe_tensor(a[1], "k"), *pos = maybe_tensor(a[3], "positions");
        try {
            const Turn how{turns, version_of(turns), flag_arg(a[4]) != 0, false, (double)float_arg(a[5])};
            const auto out = turn_rows(q, k != nullptr ? *k : at::Tensor(), pos != nullptr ? *pos : at::Tensor(), how);
            return pair(out.first, out.second);
        } catch (const Failed& f) {
            check(f.status, "fa_rope");
            throw;
        }
    });
}

// (q, k, v, k_cache, v_cache, block_table, seq_lens, turns, positions, new_lens, interleaved, factor, q_out, stream)
PyObject* cache_append_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!expect(n, 14)) return nullptr;
    return guarded([&]() -> PyObject* {
        const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
        const at::Tensor &kc = tensor(a[3], "k_cache"), &vc = tensor(a[4], "v_cache");
        const at::Tensor &table = tensor(a[5], "block_table"), &lens = tensor(a[6], "seq_lens"), &turns = tensor(a[7], "turns");
        const at::Tensor *pos = maybe_tensor(a[8], "positions"), *news = maybe_tensor(a[9], "new_lens");
        const at::Tensor* qo_arg = maybe_tensor(a[12], "q_out");
        if (q.dim() != 4) value_error("q must be 4-D (Z, Hq, T, D)");
        if (k.dim() != 4 || k.sizes() != v.sizes())
            value_error("k and v must both be (Z, Hkv, T, D), got " + shape_of(k.sizes()) + ", " + shape_of(v.sizes()));
        const int64_t Z = k.size(0), T = k.size(2);
        fa_cache_append_rope_args x{};
        x.cache = cache_of(kc, vc, table, lens, Z, false);
        if (x.cache.Hkv != k.size(1) || x.cache.D != k.size(3))
            value_error("k and v must both be (Z, " + std::to_string(x.cache.Hkv) + ", T, " + std::to_string(x.cache.D) +
                        "), got " + shape_of(k.sizes()));
        if (q.size(0) != Z || q.size(2) != T || q.size(3) != k.size(3))
            value_error("q must be (Z, Hq, T, D) of k's tokens, got " + shape_of(q.sizes()) + " for " + shape_of(k.sizes()));
        x.dtype = dtype_of(q, "fa_cache_append_rope");
        if (k.scalar_type() != kc.scalar_type() || v.scalar_type() != kc.scalar_type() || q.scalar_type() != kc.scalar_type())
            type_error("q, k and v must have the cache's dtype");
        if (news != nullptr) check_ints(*news, "new_lens", {Z});
        check_out(qo_arg, q, "q_out");
        x.rotary_dim = pairs_of(turns);
        if (pos != nullptr) x.positions_stride = positions_stride(*pos, Z, T);
        x.interleaved = flag_arg(a[10]);
        x.factor = float_arg(a[11]);
        const int dev = cuda_device("fa_cache_append_rope", q, {&k, &v, &kc, &vc, &table, &lens, pos, news, qo_arg});
        const Place place(a[13], dev, {&q, &k, &v, &kc, &vc, &table, &lens, pos, news, qo_arg});
        const at::Tensor qo = qo_arg != nullptr ? *qo_arg : out_like(q);
        x.q = q.data_ptr();
        x.q_out = qo.data_ptr();
        x.k = k.data_ptr();
        x.v = v.data_ptr();
        x.sq = strides4(q);
        x.sq_out = strides4(qo);
        x.sk = strides4(k);
        x.sv = strides4(v);
        x.new_lens = ints(news);
        x.positions = ints(pos);
        x.turns = static_cast<const int64_t*>(turns.data_ptr());
        x.Hq = to_int(q.size(1), "the heads");
        x.T = to_int(T, "T");
        check(unlocked([&] { return lib.append_rope(&x, place.stream()); }), "fa_cache_append_rope");
        written({qo_arg, &kc, &vc});
        return THPVariable_Wrap(qo);
    });
}

// Scores: (..., positions) float32, the positions contiguous and at least the table's.
void check_scores(const at::Tensor& t, std::initializer_list<int64_t> shape, const fa_paged_cache& c) {
    const at::IntArrayRef want(shape);
    if (t.scalar_type() != at::kFloat) type_error("scores must be float32");
    if (t.dim() != (int64_t)want.size() + 1 || t.sizes().slice(0, want.size()) != want)
        value_error("scores must be " + shape_of(want) + " and the positions, got " + shape_of(t.sizes()));
    const int64_t cap = (int64_t)c.max_pages * c.page_size;
    if (t.size(-1) < cap) value_error("scores must have a place for each of " + std::to_string(cap) + " positions");
    if (t.size(-1) > 1 && t.stride(-1) != 1) value_error("scores' last dimension must be contiguous");
}

// (q, lse, k_cache, block_table, seq_lens, scores, new_lens, scale, decay, workspace, stream)
PyObject* cache_score(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!expect(n, 11)) return nullptr;
    return guarded([&]() -> PyObject* {
        const at::Tensor &q = tensor(a[0], "q"), &lse = tensor(a[1], "lse"), &kc = tensor(a[2], "k_cache");
        const at::Tensor &table = tensor(a[3], "block_table"), &lens = tensor(a[4], "seq_lens"), &scores = tensor(a[5], "scores");
        const at::Tensor *news = maybe_tensor(a[6], "new_lens"), *ws_arg = maybe_tensor(a[9], "workspace");
        if (q.dim() != 4) value_error("q must be 4-D (Z, Hq, T, D)");
        const int64_t Z = q.size(0), D = q.size(3);
        fa_cache_score_args x{};
        x.cache = cache_of(kc, kc, table, lens, Z, false);
        if (x.cache.D != D)
            value_error("head dims differ: q has " + std::to_string(D) + ", the cache " + std::to_string(x.cache.D));
        x.dtype = dtype_of(q, "fa_cache_score");
        if (kc.scalar_type() != q.scalar_type()) type_error("q and the cache must share one dtype");
        if (lse.scalar_type() != at::kFloat || lse.dim() != 3 || lse.sizes() != q.sizes().slice(0, 3) || !lse.is_contiguous())
            value_error("lse must be a contiguous float32 (Z, Hq, T) tensor");
        if (news != nullptr) check_ints(*news, "new_lens", {Z});
        check_scores(scores, {Z, (int64_t)x.cache.Hkv}, x.cache);
        x.scale = a[7] == Py_None ? (float)(1.0 / std::sqrt((double)D)) : float_arg(a[7]);
        x.decay = float_arg(a[8]);
        check_workspace(ws_arg);
        const int dev = cuda_device("fa_cache_score", q, {&lse, &kc, &table, &lens, &scores, news, ws_arg});
        const Place place(a[10], dev, {&q, &lse, &kc, &table, &lens, &scores, news, ws_arg});
        at::Tensor ws;
        if (ws_arg != nullptr) {
            ws = *ws_arg;
        } else {
            size_t bytes = 0;
            check(lib.score_size(&bytes), "fa_cache_score");
            ws = scratch(bytes, q);
        }
        x.q = q.data_ptr();
        x.lse = static_cast<const float*>(lse.data_ptr());
        x.scores = static_cast<float*>(scores.data_ptr());
        x.score_seq = scores.stride(0);
        x.score_head = scores.stride(1);
        x.sq = strides4(q);
        x.new_lens = ints(news);
        x.workspace = ws.data_ptr();
        x.workspace_bytes = ws.nbytes();
        x.Hq = to_int(q.size(1), "the heads");
        x.T = to_int(q.size(2), "T");
        check(unlocked([&] { return lib.score(&x, place.stream()); }), "fa_cache_score");
        written({&scores});
        Py_RETURN_NONE;
    });
}

// (k_cache, v_cache, block_table, seq_lens, ref_counts, scores, budget, missing, keep, first, recent, workspace, stream)
PyObject* cache_evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!expect(n, 13)) return nullptr;
    return guarded([&]() -> PyObject* {
        const at::Tensor &kc = tensor(a[0], "k_cache"), &vc = tensor(a[1], "v_cache");
        const at::Tensor &table = tensor(a[2], "block_table"), &lens = tensor(a[3], "seq_lens");
        const at::Tensor &refs = tensor(a[4], "ref_counts"), &scores = tensor(a[5], "scores"), &missing = tensor(a[7], "missing");
        const at::Tensor *keep = maybe_tensor(a[8], "keep"), *ws_arg = maybe_tensor(a[11], "workspace");
        if (lens.dim() != 1) value_error("seq_lens must be (Z)");
        const int64_t Z = lens.size(0);
        fa_cache_evict_args x{};
        x.cache = cache_of(kc, vc, table, lens, Z, true);
        check_ints(refs, "ref_counts", {x.cache.P});
        check_ints(missing, "missing", {1});
        if (keep != nullptr) check_ints(*keep, "keep", {Z});
        const bool layers = kc.dim() == 5;
        if (layers) check_scores(scores, {(int64_t)x.cache.L, Z, (int64_t)x.cache.Hkv}, x.cache);
        else check_scores(scores, {Z, (int64_t)x.cache.Hkv}, x.cache);
        x.budget = int_arg(a[6], "budget");
        x.first = int_arg(a[9], "first");
        x.recent = int_arg(a[10], "recent");
        check_workspace(ws_arg);
        const int dev = cuda_device("fa_cache_evict", kc, {&vc, &table, &lens, &refs, &scores, &missing, keep, ws_arg});
        const Place place(a[12], dev, {&kc, &vc, &table, &lens, &refs, &scores, &missing, keep, ws_arg});
        at::Tensor ws;
        if (ws_arg != nullptr) {
            ws = *ws_arg;
        } else {
            size_t bytes = 0;
            const int64_t cap = (int64_t)x.cache.max_pages * x.cache.page_size;
            const int budget = x.budget < cap ? x.budget : (int)cap;
            check(lib.evict_size(x.cache.L, x.cache.Z, x.cache.Hkv, x.cache.max_pages, budget, &bytes), "fa_cache_evict");
            ws = scratch(bytes, kc);
        }
        x.ref_counts = ints(&refs);
        x.scores = static_cast<float*>(scores.data_ptr());
        x.score_layer = layers ? scores.stride(0) : 0;
        x.score_seq = scores.stride(layers ? 1 : 0);
        x.score_head = scores.stride(layers ? 2 : 1);
        x.keep = ints(keep);
        x.missing = ints(&missing);
        x.workspace = ws.data_ptr();
        x.workspace_bytes = ws.nbytes();
        check(unlocked([&] { return lib.evict(&x, place.stream()); }), "fa_cache_evict");
        written({&kc, &vc, &table, &lens, &refs, &scores, &missing});
        Py_RETURN_NONE;
    });
}

// (FaError, the addresses of the entry points)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    constexpr int COUNT = 12;
    if (!expect(n, COUNT + 1)) return nullptr;
    void* p[COUNT];
    for (int i = 0; i < COUNT; ++i) {
        p[i] = PyLong_AsVoidPtr(a[1 + i]);
        if (p[i] == nullptr) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
            return nullptr;
        }
    }
    Py_INCREF(a[0]);
    Py_XDECREF(lib.error);
    lib.error = a[0];
    lib.fwd = reinterpret_cast<decltype(lib.fwd)>(p[0]);
    lib.fwd_size = reinterpret_cast<decltype(lib.fwd_size)>(p[1]);
    lib.append = reinterpret_cast<decltype(lib.append)>(p[2]);
    lib.commit = reinterpret_cast<decltype(lib.commit)>(p[3]);
    lib.fork = reinterpret_cast<decltype(lib.fork)>(p[4]);
    lib.fork_size = reinterpret_cast<decltype(lib.fork_size)>(p[5]);
    lib.rope = reinterpret_cast<decltype(lib.rope)>(p[6]);
    lib.append_rope = reinterpret_cast<decltype(lib.append_rope)>(p[7]);
    lib.score = reinterpret_cast<decltype(lib.score)>(p[8]);
    lib.score_size = reinterpret_cast<decltype(lib.score_size)>(p[9]);
    lib.evict = reinterpret_cast<decltype(lib.evict)>(p[10]);
    lib.evict_size = reinterpret_cast<decltype(lib.evict_size)>(p[11]);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(bind), METH_FASTCALL, nullptr},
    {"fwd_paged", reinterpret_cast<PyCFunction>(fwd_paged), METH_FASTCALL, nullptr},
    {"cache_append", reinterpret_cast<PyCFunction>(cache_append), METH_FASTCALL, nullptr},
    {"cache_commit", reinterpret_cast<PyCFunction>(cache_commit), METH_FASTCALL, nullptr},
    {"cache_fork", reinterpret_cast<PyCFunction>(cache_fork), METH_FASTCALL, nullptr},
    {"rope", reinterpret_cast<PyCFunction>(rope), METH_FASTCALL, nullptr},
    {"rotary", reinterpret_cast<PyCFunction>(rotary), METH_FASTCALL, nullptr},
    {"cache_append_rope", reinterpret_cast<PyCFunction>(cache_append_rope), METH_FASTCALL, nullptr},
    {"cache_score", reinterpret_cast<PyCFunction>(cache_score), METH_FASTCALL, nullptr},
    {"cache_evict", reinterpret_cast<PyCFunction>(cache_evict), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_ext", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_ext() { return PyModule_Create(&module); }
