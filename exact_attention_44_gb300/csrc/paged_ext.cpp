// Python binding of the paged-cache entry points: argument checks and
// marshalling only.  A decode step makes two or three of these calls a layer,
// each a few microseconds of GPU time; through ctypes and Python the host side
// of one took 7 to 16 us, so it is a CPython extension over torch's tensors.
// The functions of libfa are handed over by address (bind), so the extension
// calls whichever build of the library the package has loaded.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <initializer_list>
#include <string>

#include "fa.h"

namespace {

struct Library {
    decltype(&fa_fwd_paged) fwd = nullptr;
    decltype(&fa_fwd_paged_workspace_size) fwd_size = nullptr;
    decltype(&fa_cache_append) append = nullptr;
    decltype(&fa_cache_commit) commit = nullptr;
    decltype(&fa_cache_fork) fork = nullptr;
    decltype(&fa_cache_fork_workspace_size) fork_size = nullptr;
    PyObject* error = nullptr;  // the package's FaError
} lib;

// A refused argument: the Python exception to raise.
struct Refused {
    PyObject* type;
    std::string text;
};
[[noreturn]] void value_error(std::string text) { throw Refused{PyExc_ValueError, std::move(text)}; }
[[noreturn]] void type_error(std::string text) { throw Refused{PyExc_TypeError, std::move(text)}; }

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
        if (lib.fwd == nullptr) throw Refused{PyExc_ImportError, "libfa is not loaded"};
        return fn();
    } catch (const Refused& r) {
        PyErr_SetString(r.type, r.text.c_str());
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

// (FaError, the addresses of the six entry points)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!expect(n, 7)) return nullptr;
    void* p[6];
    for (int i = 0; i < 6; ++i) {
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
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(bind), METH_FASTCALL, nullptr},
    {"fwd_paged", reinterpret_cast<PyCFunction>(fwd_paged), METH_FASTCALL, nullptr},
    {"cache_append", reinterpret_cast<PyCFunction>(cache_append), METH_FASTCALL, nullptr},
    {"cache_commit", reinterpret_cast<PyCFunction>(cache_commit), METH_FASTCALL, nullptr},
    {"cache_fork", reinterpret_cast<PyCFunction>(cache_fork), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_ext", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_ext() { return PyModule_Create(&module); }
