// The paged entry points and windows with sinks for torch tensors, as a Python extension
// module.
//
// Their kernels can take a few microseconds, less than a ctypes call with its checks and
// allocations takes in Python, so checks, output allocation and the call itself run here:
// the C ABI is unchanged and holds all of the computation.  The module finds the library's
// functions by name (load), so it links only against torch.
#include <Python.h>

#include <dlfcn.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <exception>
#include <optional>
#include <stdexcept>
#include <string>
#include <utility>

#include "../../include/fa.h"

namespace {

decltype(&fa_kv_append) g_append[2];  // bf16, e4m3
decltype(&fa_fwd_paged) g_paged[2];
decltype(&fa_paged_workspace_size) g_workspace;
decltype(&fa_fwd_sinks) g_fwd_sinks;
decltype(&fa_bwd_sinks) g_bwd_sinks;
decltype(&fa_bwd_workspace_size) g_bwd_workspace;
PyObject* g_error = nullptr;  // FAError(code, where)
PyObject* g_oom = nullptr;    // torch.OutOfMemoryError

struct ValueError : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct PyErr {};  // a Python exception is set

void require(bool ok, const char* what) {
    if (!ok) throw ValueError(what);
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
        throw PyErr{};
    }
    return THPVariable_Unpack(o);
}
const at::Tensor* tensor_or_none(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }

int64_t integer(PyObject* o) {
    PyObject* i = PyNumber_Index(o);
    if (!i) throw PyErr{};
    const long long v = PyLong_AsLongLong(i);
    Py_DECREF(i);
    if (v == -1 && PyErr_Occurred()) throw PyErr{};
    return v;
}
// Sizes go to the library as int; what does not fit is refused here.
int to_int(int64_t v) {
    require(v >= INT_MIN && v <= INT_MAX, "a size does not fit 32 bits");
    return static_cast<int>(v);
}

struct Cache {
    fa_paged_cache c;
    at::Device dev;
    bool fp8;
};

Cache check_cache(const at::Tensor& k, const at::Tensor& v, const at::Tensor& table, const at::Tensor& lens,
                  const at::Tensor* ks, const at::Tensor* vs) {
    const at::Device dev = k.device();
    require(k.dim() == 4 && v.sizes() == k.sizes() && v.scalar_type() == k.scalar_type(),
            "caches must be [num_pages, H_kv, page_size, d], alike");
    require((ks != nullptr) == (vs != nullptr), "an 8-bit cache has both scales, a bf16 cache none");
    const at::ScalarType t = k.scalar_type();
    require(ks ? t == at::kByte || t == at::kFloat8_e4m3fn : t == at::kBFloat16,
            "a cache is bf16, or with scales e4m3 (uint8 or float8_e4m3fn)");
    if (ks)
        for (const at::Tensor* s : {ks, vs}) {
            require(s->dim() == 2 && s->size(0) == k.size(0) && s->size(1) == k.size(1) && s->scalar_type() == at::kFloat,
                    "scales must be fp32 [num_pages, H_kv]");
            require(s->device() == dev && s->is_contiguous(), "scales must be contiguous, on the cache's device");
        }
    require(table.dim() == 2 && lens.dim() == 1 && lens.size(0) == table.size(0),
            "page_table must be [B, max_pages] and lens [B]");
    require(table.scalar_type() == at::kInt && lens.scalar_type() == at::kInt, "page_table and lens must be int32");
    require(k.is_cuda() && v.device() == dev && table.device() == dev && lens.device() == dev && k.is_contiguous() &&
                v.is_contiguous() && table.is_contiguous() && lens.is_contiguous(),
            "caches, page_table and lens must be contiguous, on one CUDA device");
    Cache out{{k.data_ptr(), v.data_ptr(), ks ? static_cast<float*>(ks->data_ptr()) : nullptr,
               vs ? static_cast<float*>(vs->data_ptr()) : nullptr, static_cast<const int*>(table.data_ptr()),
               static_cast<const int*>(lens.data_ptr()), to_int(table.size(0)), to_int(k.size(1)), to_int(k.size(3)),
               to_int(k.size(0)), to_int(k.size(2)), to_int(table.size(1))},
              dev, ks != nullptr};
    return out;
}

// bf16 rows of contiguous columns, of the given shape, on the cache's device.
void check_rows(const at::Tensor& t, at::IntArrayRef shape, const Cache& c, const char* name) {
    if (t.sizes() == shape && t.scalar_type() == at::kBFloat16 && t.device() == c.dev && t.stride(-1) == 1) return;
    std::string what = std::string(name) + " must be bf16 [";
    for (size_t i = 0; i < shape.size(); ++i) what += (i ? ", " : "") + std::to_string(shape[i]);
    throw ValueError(what + "] on the cache's device, columns contiguous");
}

void check_status(int code, const char* where) {
    if (code == FA_OK) return;
    PyObject* e = PyObject_CallFunction(g_error, "is", code, where);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw PyErr{};
}

float scale_of(PyObject* o, int64_t d) {
    if (o == Py_None) return static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)));
    const double tau = PyFloat_AsDouble(o);
    if (tau == -1.0 && PyErr_Occurred()) throw PyErr{};
    return static_cast<float>(tau);
}

// A tuple of tensors, each wrapped, or the argument that it came as.
PyObject* results(std::initializer_list<std::pair<const std::optional<at::Tensor>*, PyObject*>> rs) {
    PyObject* all = PyTuple_New(static_cast<Py_ssize_t>(rs.size()));
    if (!all) throw PyErr{};
    Py_ssize_t i = 0;
    for (const auto& [made, given] : rs) {
        PyObject* o = *made ? THPVariable_Wrap(**made) : Py_NewRef(given);
        if (!o) {
            Py_DECREF(all);
            throw PyErr{};
        }
        PyTuple_SET_ITEM(all, i++, o);
    }
    return all;
}

// Every Python function's frame: no C++ exception passes into the interpreter.
template <typename F>
PyObject* guarded(Py_ssize_t have, Py_ssize_t want, F&& f) {
    if (have != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, have);
        return nullptr;
    }
    try {
        return f();
    } catch (const PyErr&) {
    } catch (const ValueError& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const c10::OutOfMemoryError& e) {
        PyErr_SetString(g_oom, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// kv_append(k, v, k_cache, v_cache, page_table, lens, cu_new, q, inv_freq, interleaved,
//           k_scale, v_scale, q_out) -> rotated queries or None
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 13, [&]() -> PyObject* {
        const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
        const at::Tensor *cu = tensor_or_none(a[6], "cu_new"), *q = tensor_or_none(a[7], "q");
        const at::Tensor *freq = tensor_or_none(a[8], "inv_freq"), *given = tensor_or_none(a[12], "q_out");
        const int interleaved = PyObject_IsTrue(a[9]);
        if (interleaved < 0) throw PyErr{};
        const Cache c = check_cache(tensor(a[2], "k_cache"), tensor(a[3], "v_cache"), tensor(a[4], "page_table"),
                                    tensor(a[5], "lens"), tensor_or_none(a[10], "k_scale"),
                                    tensor_or_none(a[11], "v_scale"));
        require(k.dim() == 3, "k and v must be [T, H_kv, d]");
        const int64_t T = k.size(0), d = c.c.d;
        check_rows(k, {T, c.c.H_kv, d}, c, "k");
        check_rows(v, {T, c.c.H_kv, d}, c, "v");
        if (cu)
            require(cu->dim() == 1 && cu->size(0) == int64_t{c.c.B} + 1 && cu->scalar_type() == at::kInt &&
                        cu->device() == c.dev && cu->is_contiguous(),
                    "cu_new must be contiguous int32 [B + 1] on the cache's device");
        int rot = 0;
        if (freq) {
            require(freq->dim() == 1 && freq->scalar_type() == at::kDouble && freq->device() == c.dev &&
                        freq->is_contiguous(),
                    "inv_freq must be contiguous float64 [rot / 2] on the cache's device");
            require(freq->size(0) > 0, "inv_freq is empty");
            rot = to_int(2 * freq->size(0));
        }
        require(q || !given, "q_out without q");
        const c10::cuda::OptionalCUDAGuard guard(c.dev);
        std::optional<at::Tensor> made;
        const at::Tensor* out = given;
        int64_t H = 0;
        if (q) {
            require(q->dim() == 3, "q must be [T, H, d]");
            H = q->size(1);
            check_rows(*q, {T, H, d}, c, "q");
            if (given) check_rows(*given, {T, H, d}, c, "q_out");
            else out = &made.emplace(at::empty({T, H, d}, q->options()));
        }
        const bool has_q = H > 0;
        check_status(g_append[c.fp8](&c.c, k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0), v.stride(1),
                                     to_int(T), cu ? static_cast<const int*>(cu->data_ptr()) : nullptr,
                                     has_q ? q->data_ptr() : nullptr, has_q ? q->stride(0) : 0, has_q ? q->stride(1) : 0,
                                     has_q ? out->data_ptr() : nullptr, has_q ? out->stride(0) : 0,
                                     has_q ? out->stride(1) : 0, to_int(H),
                                     freq ? static_cast<const double*>(freq->data_ptr()) : nullptr, rot, interleaved,
                                     c10::cuda::getCurrentCUDAStream(c.dev.index()).stream()),
                     c.fp8 ? "fa_kv_append_fp8" : "fa_kv_append");
        if (!q) Py_RETURN_NONE;
        if (given) return Py_NewRef(a[12]);
        return THPVariable_Wrap(*made);
    });
}

// fwd_paged(q, k_cache, v_cache, page_table, lens, tau, window, sinks, k_scale, v_scale,
//           out, lse, workspace) -> (O, LSE)
PyObject* fwd_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 13, [&]() -> PyObject* {
        const at::Tensor& q = tensor(a[0], "q");
        const Cache c = check_cache(tensor(a[1], "k_cache"), tensor(a[2], "v_cache"), tensor(a[3], "page_table"),
                                    tensor(a[4], "lens"), tensor_or_none(a[8], "k_scale"),
                                    tensor_or_none(a[9], "v_scale"));
        const at::Tensor *out = tensor_or_none(a[10], "out"), *lse = tensor_or_none(a[11], "lse");
        const at::Tensor* ws = tensor_or_none(a[12], "workspace");
        require(q.dim() == 4, "expected [B, H, Nq, d] queries");
        const int sinks = to_int(integer(a[7]));
        int window = 0;
        if (a[6] == Py_None) {
            require(sinks == 0, "sinks need a window");
        } else {
            window = to_int(integer(a[6]));
            require(window >= 1, "a window holds at least one key");
        }
        const float tau = scale_of(a[5], c.c.d);
        const int64_t H = q.size(1), Nq = q.size(2);
        check_rows(q, {c.c.B, H, Nq, c.c.d}, c, "q");
        const c10::cuda::OptionalCUDAGuard guard(c.dev);
        std::optional<at::Tensor> made_out, made_lse, made_ws;
        if (out) check_rows(*out, q.sizes(), c, "out");
        else out = &made_out.emplace(at::empty(q.sizes(), q.options()));
        if (lse)
            require(lse->sizes() == q.sizes().slice(0, 3) && lse->scalar_type() == at::kFloat && lse->device() == c.dev &&
                        lse->is_contiguous(),
                    "lse must be contiguous fp32 [B, H, Nq] on the cache's device");
        else lse = &made_lse.emplace(at::empty(q.sizes().slice(0, 3), q.options().dtype(at::kFloat)));
        size_t bytes;
        if (ws) {
            require(ws->device() == c.dev && ws->is_contiguous(), "workspace must be contiguous, on the cache's device");
            bytes = ws->nbytes();
        } else {
            bytes = g_workspace(&c.c, to_int(H), to_int(Nq), window, sinks);
            if (bytes) ws = &made_ws.emplace(at::empty({static_cast<int64_t>(bytes)}, q.options().dtype(at::kByte)));
        }
        check_status(g_paged[c.fp8](&c.c, q.data_ptr(), q.stride(0), q.stride(1), q.stride(2), out->data_ptr(),
                                    out->stride(0), out->stride(1), out->stride(2), static_cast<float*>(lse->data_ptr()),
                                    to_int(H), to_int(Nq), tau, window, sinks, ws ? ws->data_ptr() : nullptr, bytes,
                                    c10::cuda::getCurrentCUDAStream(c.dev.index()).stream()),
                     c.fp8 ? "fa_fwd_paged_fp8" : "fa_fwd_paged");
        return results({{&made_out, a[10]}, {&made_lse, a[11]}});
    });
}

// Contiguous bf16 [B, H, N, d] tensors of one shape and CUDA device, as fa_fwd takes them.
void check_attention(std::initializer_list<const at::Tensor*> ts) {
    const at::Tensor& ref = **ts.begin();
    require(ref.dim() == 4, "expected [B, H, N, d] tensors");
    for (const at::Tensor* t : ts) {
        require(t->is_cuda() && t->scalar_type() == at::kBFloat16 && t->is_contiguous(),
                "inputs must be contiguous CUDA bf16 tensors");
        require(t->sizes() == ref.sizes() && t->device() == ref.device(), "inputs must share shape and device");
    }
}
void check_lse(const at::Tensor& lse, const at::Tensor& q) {
    require(lse.scalar_type() == at::kFloat && lse.is_contiguous() && lse.device() == q.device() &&
                lse.sizes() == q.sizes().slice(0, 3),
            "lse must be contiguous fp32 [B, H, N]");
}
// fwd_sinks(q, k, v, tau, window, sinks, out, lse) -> (O, LSE)
PyObject* fwd_sinks(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 8, [&]() -> PyObject* {
        const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
        const at::Tensor *out = tensor_or_none(a[6], "out"), *lse = tensor_or_none(a[7], "lse");
        check_attention({&q, &k, &v});
        const int B = to_int(q.size(0)), H = to_int(q.size(1)), N = to_int(q.size(2)), d = to_int(q.size(3));
        const int window = to_int(integer(a[4])), sinks = to_int(integer(a[5]));
        const float tau = scale_of(a[3], d);
        const c10::cuda::OptionalCUDAGuard guard(q.device());
        std::optional<at::Tensor> made_out, made_lse;
        if (out) check_attention({&q, out});
        else out = &made_out.emplace(at::empty(q.sizes(), q.options()));
        if (lse) check_lse(*lse, q);
        else lse = &made_lse.emplace(at::empty(q.sizes().slice(0, 3), q.options().dtype(at::kFloat)));
        check_status(g_fwd_sinks(q.data_ptr(), k.data_ptr(), v.data_ptr(), out->data_ptr(),
                                 static_cast<float*>(lse->data_ptr()), B, H, N, d, tau, window, sinks,
                                 c10::cuda::getCurrentCUDAStream(q.device().index()).stream()),
                     "fa_fwd_sinks");
        return results({{&made_out, a[6]}, {&made_lse, a[7]}});
    });
}

// bwd_sinks(q, k, v, o, do, lse, tau, window, sinks, dq, dk, dv, workspace) -> (dQ, dK, dV)
PyObject* bwd_sinks(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 13, [&]() -> PyObject* {
        const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &o = tensor(a[3], "o");
        const at::Tensor &go = tensor(a[4], "do"), &lse = tensor(a[5], "lse");
        check_attention({&q, &k, &v, &o, &go});
        check_lse(lse, q);
        const int B = to_int(q.size(0)), H = to_int(q.size(1)), N = to_int(q.size(2)), d = to_int(q.size(3));
        const int window = to_int(integer(a[7])), sinks = to_int(integer(a[8]));
        const float tau = scale_of(a[6], d);
        const c10::cuda::OptionalCUDAGuard guard(q.device());
        std::optional<at::Tensor> made[3], made_ws;
        void* grads[3];
        for (int i = 0; i < 3; ++i) {
            const at::Tensor* g = tensor_or_none(a[9 + i], "a gradient");
            if (g) check_attention({&q, g});
            else g = &made[i].emplace(at::empty(q.sizes(), q.options()));
            grads[i] = g->data_ptr();
        }
        const at::Tensor* ws = tensor_or_none(a[12], "workspace");
        if (ws) require(ws->device() == q.device() && ws->is_contiguous(), "workspace must be contiguous, on the inputs' device");
        else {
            const size_t need = g_bwd_workspace(B, H, N, d);
            ws = &made_ws.emplace(at::empty({static_cast<int64_t>(need ? need : 1)}, q.options().dtype(at::kByte)));
        }
        check_status(g_bwd_sinks(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), go.data_ptr(),
                                 static_cast<const float*>(lse.data_ptr()), grads[0], grads[1], grads[2], ws->data_ptr(),
                                 ws->nbytes(), B, H, N, d, tau, window, sinks,
                                 c10::cuda::getCurrentCUDAStream(q.device().index()).stream()),
                     "fa_bwd_sinks");
        return results({{&made[0], a[9]}, {&made[1], a[10]}, {&made[2], a[11]}});
    });
}

// load(path of the library, FAError, torch.OutOfMemoryError)
PyObject* load(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 3, [&]() -> PyObject* {
        const char* path = PyUnicode_AsUTF8(a[0]);
        if (!path) throw PyErr{};
        void* lib = dlopen(path, RTLD_NOW | RTLD_LOCAL);
        if (!lib) throw std::runtime_error(std::string("cannot load the library: ") + dlerror());
        const auto find = [&](const char* name) {
            void* f = dlsym(lib, name);
            if (!f) throw std::runtime_error(std::string("the library lacks ") + name);
            return f;
        };
        g_append[0] = reinterpret_cast<decltype(&fa_kv_append)>(find("fa_kv_append"));
        g_append[1] = reinterpret_cast<decltype(&fa_kv_append)>(find("fa_kv_append_fp8"));
        g_paged[0] = reinterpret_cast<decltype(&fa_fwd_paged)>(find("fa_fwd_paged"));
        g_paged[1] = reinterpret_cast<decltype(&fa_fwd_paged)>(find("fa_fwd_paged_fp8"));
        g_workspace = reinterpret_cast<decltype(&fa_paged_workspace_size)>(find("fa_paged_workspace_size"));
        g_fwd_sinks = reinterpret_cast<decltype(&fa_fwd_sinks)>(find("fa_fwd_sinks"));
        g_bwd_sinks = reinterpret_cast<decltype(&fa_bwd_sinks)>(find("fa_bwd_sinks"));
        g_bwd_workspace = reinterpret_cast<decltype(&fa_bwd_workspace_size)>(find("fa_bwd_workspace_size"));
        Py_XDECREF(g_error);
        Py_XDECREF(g_oom);
        g_error = Py_NewRef(a[1]);
        g_oom = Py_NewRef(a[2]);
        Py_RETURN_NONE;
    });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<kv_append>("kv_append"), method<fwd_paged>("fwd_paged"),
                           method<fwd_sinks>("fwd_sinks"), method<bwd_sinks>("bwd_sinks"), method<load>("load"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "fa_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_fa_binding() { return PyModule_Create(&g_module); }
