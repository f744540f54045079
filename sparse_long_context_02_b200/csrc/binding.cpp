// Argument checks and marshalling of the rotary and 8-bit cache calls, as a
// CPython module.  A decode step calls them once per layer on microseconds of
// GPU work, and the same checks in Python cost more than the kernels: for 64
// rows, dsa_rope with two fresh outputs took 16.2 us of host time through
// ctypes, 5.9 of them in the library and the CUDA launch.
//
// The module computes nothing: it reads tensors' metadata, takes the current
// stream, allocates outputs and workspaces the caller did not bring (on the
// launch stream, so that their memory is not handed out again before the
// stream is done with it) and calls the C ABI of libdsa_b200.so.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <stdexcept>
#include <string>

#include "dsa.h"

namespace {

// What a Python caller gets as ValueError.
struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};

PyObject* g_check = nullptr;  // the package's _check(status, name)

decltype(&dsa_rope) f_rope;
decltype(&dsa_rope_backward) f_rope_backward;
decltype(&dsa_kv8_append) f_append;
decltype(&dsa_attn_kv8_workspace_size) f_workspace;
decltype(&dsa_sparse_attn_kv8) f_sparse;
decltype(&dsa_attn_kv8) f_dense;

std::string shape_of(const at::Tensor& t) {
    std::string s = "(";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + ")";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a CUDA tensor");
    return THPVariable_Unpack(o);
}

void on_device(const at::Tensor& t, const char* name, int dev) {
    if (!t.is_cuda()) throw Refused(std::string(name) + " must be a CUDA tensor");
    if (t.get_device() != dev)
        throw Refused(std::string(name) + " is on cuda:" + std::to_string(t.get_device()) +
                      ", but the library launches on the current device cuda:" +
                      std::to_string(dev));
}

void* dense(const at::Tensor& t, const char* name, int dev) {
    on_device(t, name, dev);
    if (!t.is_contiguous()) throw Refused(std::string(name) + " must be contiguous");
    return t.data_ptr();
}

template <typename T = void>
T* dense_or_null(PyObject* o, const char* name, int dev, at::ScalarType type, int64_t least) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != type || t.numel() < least)
        throw Refused(std::string(name) + " must be " + c10::toString(type) + " of at least " +
                      std::to_string(least) + " element(s)");
    return static_cast<T*>(dense(t, name, dev));
}

struct Heads {
    void* p = nullptr;
    int64_t stride = 0;
    int64_t heads = 0;
};

// An array [L][heads][d] whose heads are dense; tokens may lie apart.
Heads heads(const at::Tensor& t, const char* name, int dev, int64_t L, int64_t d,
            at::ScalarType type) {
    on_device(t, name, dev);
    if (t.scalar_type() != type)
        throw Refused(std::string(name) + " must be " + c10::toString(type) + ", got " +
                      c10::toString(t.scalar_type()));
    if (t.dim() != 3 || t.size(0) != L || t.size(2) != d)
        throw Refused(std::string(name) + " must be [" + std::to_string(L) + "][heads][" +
                      std::to_string(d) + "], got " + shape_of(t));
    const int64_t H = t.size(1);
    if ((t.stride(2) != 1 && d > 1) || (t.stride(1) != d && H > 1))
        throw Refused(std::string(name) + ": each token's heads must be dense");
    return {t.data_ptr(), L > 1 ? t.stride(0) : H * d, H};
}

// Other Python threads run meanwhile: a launch waits where the GPU's queue is full, an
// allocation where the memory has to come from the driver.
struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    Unlocked() = default;
    Unlocked(const Unlocked&) = delete;
    ~Unlocked() { PyEval_RestoreThread(state); }
};

template <typename... P, typename... A>
int call(dsa_status_t (*f)(P...), A... args) {
    const Unlocked unlocked;
    return f(args...);
}

// The launch stream: None is the current one, else a torch.cuda.Stream or a handle.
struct Launch {
    int dev;
    cudaStream_t handle;
    std::optional<c10::cuda::CUDAStream> other;

    // `first` is the call's first tensor: without a GPU there is no current device to ask for.
    Launch(PyObject* o, const at::Tensor& first, const char* name) {
        if (!first.is_cuda()) throw Refused(std::string(name) + " must be a CUDA tensor");
        dev = c10::cuda::current_device();
        if (o == Py_None) {
            handle = c10::cuda::getCurrentCUDAStream(dev).stream();
            return;
        }
        PyObject* h = PyObject_HasAttrString(o, "cuda_stream")
                          ? PyObject_GetAttrString(o, "cuda_stream")
                          : PyNumber_Index(o);
        if (h == nullptr) throw Refused("stream must be a torch.cuda.Stream or a stream handle");
        handle = static_cast<cudaStream_t>(PyLong_AsVoidPtr(h));
        Py_DECREF(h);
        if (PyErr_Occurred())
            throw Refused("stream must be a torch.cuda.Stream or a stream handle");
        other = handle != nullptr
                    ? c10::cuda::getStreamFromExternal(handle, static_cast<c10::DeviceIndex>(dev))
                    : c10::cuda::getDefaultCUDAStream(static_cast<c10::DeviceIndex>(dev));
    }

    at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
        const Unlocked unlocked;
        c10::cuda::OptionalCUDAStreamGuard guard;
        if (other) guard.reset_stream(*other);
        return at::empty(shape, at::TensorOptions()
                                    .dtype(type)
                                    .device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)));
    }
};

// Raises the package's DSAError for a status that is not DSA_OK.
bool done(int status, const char* name) {
    if (status == DSA_OK) return true;
    PyObject* r = PyObject_CallFunction(g_check, "is", status, name);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, name);
    return false;
}

// Runs a call's body; C++ exceptions end here, torch's as the Python exceptions that it
// has for them (an allocation that does not fit as torch.OutOfMemoryError).
template <typename F>
PyObject* guarded(F&& body) {
    try {
        return body();
    } catch (const Refused& e) {
        PyErr_Clear();
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (...) {
        if (!PyErr_Occurred()) torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

bool count(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return false;
}

double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw std::runtime_error("not a number");
    return v;
}

int integer(PyObject* o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw std::runtime_error("not an integer");
    return v > INT32_MAX || v < INT32_MIN ? -1 : static_cast<int>(v);
}

int type_code(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return DSA_TYPE_BF16;
        case at::kFloat: return DSA_TYPE_F32;
        case at::kFloat8_e4m3fn: return DSA_TYPE_E4M3;
        default: return -1;
    }
}

// (backward, q, k, positions, freqs, rot_scale, out_scale, offset, interleaved, out_dtype,
//  q_out, k_out, stream, err) -> (q_out, k_out)
PyObject* py_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!count(n, 14)) return nullptr;
    return guarded([&]() -> PyObject* {
        const bool backward = a[0] == Py_True;
        const std::string name = backward ? "dsa_rope_backward" : "dsa_rope";
        const at::Tensor& q = tensor(a[1], "q");
        if (q.dim() != 3) throw Refused("q must be [L][heads][d], got " + shape_of(q));
        const int64_t L = q.size(0), Hq = q.size(1), d = q.size(2);
        const at::ScalarType in = q.scalar_type();
        if (type_code(in) < 0)
            throw Refused(name + ": unsupported dtype " + c10::toString(in));
        at::ScalarType out = in;
        if (a[9] != Py_None) {
            if (!THPDtype_Check(a[9])) throw Refused(name + ": out_dtype must be a torch.dtype");
            out = reinterpret_cast<THPDtype*>(a[9])->scalar_type;
        } else if (a[10] != Py_None) {
            out = tensor(a[10], "q_out").scalar_type();
        }
        if (type_code(out) < 0)
            throw Refused(name + ": unsupported out_dtype " + c10::toString(out));
        const at::Tensor &pos = tensor(a[3], "positions"), &freqs = tensor(a[4], "freqs");
        if (pos.scalar_type() != at::kLong || pos.numel() != L)
            throw Refused(name + ": positions must be " + std::to_string(L) + " int64");
        if (freqs.scalar_type() != at::kLong)
            throw Refused(name + ": freqs must be int64 (rope_freqs)");
        if (a[2] == Py_None && a[11] != Py_None) throw Refused(name + ": k_out without k");
        if (Hq > INT32_MAX || d > INT32_MAX || freqs.numel() > INT32_MAX / 2)
            throw Refused(name + ": too many heads or elements");

        const Launch at_(a[12], q, "q");
        const Heads hq = heads(q, "q", at_.dev, L, d, in);
        Heads hk, ko;
        if (a[2] != Py_None) hk = heads(tensor(a[2], "k"), "k", at_.dev, L, d, in);
        const void* pp = dense(pos, "positions", at_.dev);
        const void* fp = dense(freqs, "freqs", at_.dev);
        int32_t* err = dense_or_null<int32_t>(a[13], "err", at_.dev, at::kInt, 1);

        at::Tensor q_out, k_out;
        q_out = a[10] != Py_None ? tensor(a[10], "q_out") : at_.empty({L, Hq, d}, out);
        const Heads qo = heads(q_out, "q_out", at_.dev, L, d, out);
        if (qo.heads != Hq)
            throw Refused(name + ": q_out has " + std::to_string(qo.heads) + " heads, q " +
                          std::to_string(Hq));
        if (a[2] != Py_None) {
            k_out = a[11] != Py_None ? tensor(a[11], "k_out") : at_.empty({L, hk.heads, d}, out);
            ko = heads(k_out, "k_out", at_.dev, L, d, out);
            if (ko.heads != hk.heads)
                throw Refused(name + ": k_out has " + std::to_string(ko.heads) + " heads, k " +
                              std::to_string(hk.heads));
        }
        const float rs = static_cast<float>(number(a[5])), os = static_cast<float>(number(a[6]));
        const int off = integer(a[7]), inter = PyObject_IsTrue(a[8]);
        if (inter < 0) throw std::runtime_error("interleaved has no truth value");
        const int rot = 2 * static_cast<int>(freqs.numel());
        const auto* positions = static_cast<const int64_t*>(pp);
        const auto* table = static_cast<const uint64_t*>(fp);
        const int st =
            backward
                ? call(f_rope_backward, hq.p, hk.p, positions, table, L, (int)Hq, (int)hk.heads,
                       (int)d, off, rot, inter, rs, type_code(in), type_code(out), hq.stride,
                       hk.stride, qo.stride, ko.stride, qo.p, ko.p, err, at_.handle)
                : call(f_rope, hq.p, hk.p, positions, table, L, (int)Hq, (int)hk.heads, (int)d, off,
                       rot, inter, rs, os, type_code(in), type_code(out), hq.stride, hk.stride,
                       qo.stride, ko.stride, qo.p, ko.p, err, at_.handle);
        if (!done(st, name.c_str())) return nullptr;
        PyObject* r = PyTuple_New(2);
        if (r == nullptr) return nullptr;
        PyObject* first = a[10] != Py_None ? Py_NewRef(a[10]) : THPVariable_Wrap(q_out);
        PyObject* second = a[2] == Py_None    ? Py_NewRef(Py_None)
                           : a[11] != Py_None ? Py_NewRef(a[11])
                                              : THPVariable_Wrap(k_out);
        PyTuple_SET_ITEM(r, 0, first);
        PyTuple_SET_ITEM(r, 1, second);
        return r;
    });
}

// A paged cache: (k8, v8, k_scale, v_scale, block_table, seq_lens).
struct Cache {
    void *k8, *v8;
    float *ks, *vs;
    int32_t *table, *lens;
    int64_t pages, page, Hkv, d, B, M;

    // Shapes and types, before anything that needs a device.
    explicit Cache(PyObject* const* a) {
        const at::Tensor &k = tensor(a[0], "k8"), &v = tensor(a[1], "v8");
        if (k.dim() != 4 || v.sizes() != k.sizes())
            throw Refused("k8 and v8 must be [pages][page][Hkv][d] of one shape, got " +
                          shape_of(k) + " and " + shape_of(v));
        pages = k.size(0);
        page = k.size(1);
        Hkv = k.size(2);
        d = k.size(3);
        const char* names[] = {"k8", "v8", "k_scale", "v_scale"};
        for (int i = 0; i < 2; ++i) {
            const at::ScalarType t = tensor(a[i], names[i]).scalar_type();
            if (t != at::kFloat8_e4m3fn && t != at::kByte)
                throw Refused(std::string(names[i]) + " must be float8_e4m3fn or uint8, got " +
                              c10::toString(t));
        }
        for (int i = 2; i < 4; ++i) {
            const at::Tensor& t = tensor(a[i], names[i]);
            if (t.scalar_type() != at::kFloat || t.dim() != 2 || t.size(0) != pages ||
                t.size(1) != Hkv)
                throw Refused(std::string(names[i]) + " must be [" + std::to_string(pages) + "][" +
                              std::to_string(Hkv) + "] float32");
        }
        const at::Tensor &bt = tensor(a[4], "block_table"), &sl = tensor(a[5], "seq_lens");
        if (bt.scalar_type() != at::kInt || bt.dim() != 2)
            throw Refused("block_table must be int32 with 2 dimensions");
        B = bt.size(0);
        M = bt.size(1);
        if (sl.scalar_type() != at::kInt || sl.dim() != 1 || sl.size(0) != B)
            throw Refused("seq_lens must be " + std::to_string(B) +
                          " int32, one per block_table row");
        if (page > INT32_MAX || Hkv > INT32_MAX || d > INT32_MAX || B > INT32_MAX || M > INT32_MAX)
            throw Refused("the cache's dimensions are too large");
    }

    void pointers(PyObject* const* a, int dev) {
        k8 = dense(tensor(a[0], "k8"), "k8", dev);
        v8 = dense(tensor(a[1], "v8"), "v8", dev);
        ks = static_cast<float*>(dense(tensor(a[2], "k_scale"), "k_scale", dev));
        vs = static_cast<float*>(dense(tensor(a[3], "v_scale"), "v_scale", dev));
        table = static_cast<int32_t*>(dense(tensor(a[4], "block_table"), "block_table", dev));
        lens = static_cast<int32_t*>(dense(tensor(a[5], "seq_lens"), "seq_lens", dev));
    }
};

int32_t* offsets(PyObject* o, const char* name, int64_t B, int dev) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != at::kInt || t.numel() != B + 1)
        throw Refused(std::string(name) + " must be " + std::to_string(B + 1) + " int32");
    return static_cast<int32_t*>(dense(t, name, dev));
}

// (K, V, k8, v8, k_scale, v_scale, block_table, seq_lens, new_off, stream, err) -> None
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!count(n, 11)) return nullptr;
    return guarded([&]() -> PyObject* {
        Cache c(a + 2);
        const at::Tensor &K = tensor(a[0], "K"), &V = tensor(a[1], "V");
        if (K.dim() != 3) throw Refused("K must be [T][heads][d], got " + shape_of(K));
        const Launch at_(a[9], tensor(a[2], "k8"), "k8");
        c.pointers(a + 2, at_.dev);
        const int64_t T = K.size(0);
        const Heads k = heads(K, "K", at_.dev, T, c.d, at::kBFloat16);
        const Heads v = heads(V, "V", at_.dev, T, c.d, at::kBFloat16);
        if (k.heads != c.Hkv || v.heads != c.Hkv)
            throw Refused("K and V must have " + std::to_string(c.Hkv) + " heads");
        const int32_t* new_off = offsets(a[8], "new_off", c.B, at_.dev);
        int32_t* err = dense_or_null<int32_t>(a[10], "err", at_.dev, at::kInt, 1);
        const int st = call(f_append, k.p, v.p, T, k.stride, v.stride, c.k8, c.v8, c.ks, c.vs,
                            c.pages, (int)c.page, c.table, (int)c.M, c.lens, new_off, (int)c.B,
                            (int)c.Hkv, (int)c.d, err, at_.handle);
        if (!done(st, "dsa_kv8_append")) return nullptr;
        Py_RETURN_NONE;
    });
}

// (Q, k8, v8, k_scale, v_scale, block_table, seq_lens, idx, scale, row_off, O, lse, workspace,
//  stream, err) -> O; idx None: every key
PyObject* py_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!count(n, 15)) return nullptr;
    return guarded([&]() -> PyObject* {
        Cache c(a + 1);
        const bool sparse = a[7] != Py_None;
        const at::Tensor& Q = tensor(a[0], "Q");
        if (Q.dim() != 3 || Q.size(2) != c.d || Q.scalar_type() != at::kBFloat16 ||
            Q.size(1) > INT32_MAX)
            throw Refused("Q must be [T][Hq][" + std::to_string(c.d) + "] bfloat16, got " +
                          shape_of(Q) + " " + c10::toString(Q.scalar_type()));
        const int64_t T = Q.size(0), Hq = Q.size(1);
        if (a[10] != Py_None) {
            const at::Tensor& O = tensor(a[10], "O");
            if (O.sizes() != Q.sizes() || O.scalar_type() != at::kBFloat16)
                throw Refused("O must have Q's shape, in bfloat16");
        }
        if (a[11] != Py_None) {
            const at::Tensor& lse = tensor(a[11], "lse");
            if (lse.dim() != 2 || lse.size(0) != T || lse.size(1) != Hq ||
                lse.scalar_type() != at::kFloat)
                throw Refused("lse must be [" + std::to_string(T) + "][" + std::to_string(Hq) +
                              "] float32");
        }
        int64_t keys = c.M * c.page;
        if (sparse) {
            const at::Tensor& idx = tensor(a[7], "idx");
            if (idx.dim() != 2 || idx.size(0) != T || idx.scalar_type() != at::kInt ||
                idx.size(1) > INT32_MAX)
                throw Refused("idx must be [" + std::to_string(T) + "][k] int32");
            keys = idx.size(1);
        }
        const Launch at_(a[13], Q, "Q");
        c.pointers(a + 1, at_.dev);
        const void* q = dense(Q, "Q", at_.dev);
        const int32_t* idx =
            sparse ? static_cast<int32_t*>(dense(tensor(a[7], "idx"), "idx", at_.dev)) : nullptr;
        const int32_t* row_off = offsets(a[9], "row_off", c.B, at_.dev);
        float* lse = nullptr;
        if (a[11] != Py_None) lse = static_cast<float*>(dense(tensor(a[11], "lse"), "lse", at_.dev));
        int32_t* err = dense_or_null<int32_t>(a[14], "err", at_.dev, at::kInt, 1);

        at::Tensor O =
            a[10] != Py_None ? tensor(a[10], "O") : at_.empty({T, Hq, c.d}, at::kBFloat16);
        void* o = dense(O, "O", at_.dev);
        at::Tensor ws;
        if (a[12] != Py_None) {
            ws = tensor(a[12], "workspace");
        } else if (sparse || T <= DSA_ATTN_KV8_CUT_ROWS) {
            const size_t need = f_workspace(T, keys, (int)Hq, (int)c.Hkv, (int)c.d);
            if (need > 0) ws = at_.empty({(int64_t)need}, at::kByte);
        }
        void* wp = ws.defined() ? dense(ws, "workspace", at_.dev) : nullptr;
        const size_t wb = ws.defined() ? ws.nbytes() : 0;
        const float scale = static_cast<float>(number(a[8]));
        const int st =
            sparse ? call(f_sparse, q, c.k8, c.v8, c.ks, c.vs, c.pages, (int)c.page, c.table,
                          (int)c.M, c.lens, row_off, (int)c.B, T, idx, (int)keys, (int)Hq,
                          (int)c.Hkv, (int)c.d, scale, o, lse, wp, wb, err, at_.handle)
                   : call(f_dense, q, c.k8, c.v8, c.ks, c.vs, c.pages, (int)c.page, c.table,
                          (int)c.M, c.lens, row_off, (int)c.B, T, (int)Hq, (int)c.Hkv, (int)c.d,
                          scale, o, lse, wp, wb, err, at_.handle);
        if (!done(st, sparse ? "dsa_sparse_attn_kv8" : "dsa_attn_kv8")) return nullptr;
        return a[10] != Py_None ? Py_NewRef(a[10]) : THPVariable_Wrap(O);
    });
}

// (library path, check): finds the C ABI's functions in the library that ctypes loaded.
PyObject* py_bind(PyObject*, PyObject* args) {
    const char* path;
    PyObject* check;
    if (!PyArg_ParseTuple(args, "sO", &path, &check)) return nullptr;
    void* h = dlopen(path, RTLD_NOW | RTLD_LOCAL);
    if (h == nullptr) {
        PyErr_Format(PyExc_RuntimeError, "%s", dlerror());
        return nullptr;
    }
    auto find = [&](auto& f, const char* name) {
        f = reinterpret_cast<std::remove_reference_t<decltype(f)>>(dlsym(h, name));
        if (f == nullptr && !PyErr_Occurred())
            PyErr_Format(PyExc_RuntimeError, "%s has no %s", path, name);
    };
    find(f_rope, "dsa_rope");
    find(f_rope_backward, "dsa_rope_backward");
    find(f_append, "dsa_kv8_append");
    find(f_workspace, "dsa_attn_kv8_workspace_size");
    find(f_sparse, "dsa_sparse_attn_kv8");
    find(f_dense, "dsa_attn_kv8");
    if (PyErr_Occurred()) return nullptr;
    Py_INCREF(check);
    Py_XDECREF(g_check);
    g_check = check;
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", py_bind, METH_VARARGS, nullptr},
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_rope)), METH_FASTCALL, nullptr},
    {"kv8_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_append)), METH_FASTCALL,
     nullptr},
    {"attn_kv8", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_attn)), METH_FASTCALL,
     nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() {
    PyObject* m = PyModule_Create(&module);
    // the torch and the Python that it was compiled against; the package checks it
    if (m != nullptr && PyModule_AddStringConstant(m, "built_for", DSA_BUILT_FOR) != 0)
        Py_CLEAR(m);
    return m;
}
