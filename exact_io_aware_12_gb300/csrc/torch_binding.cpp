// The paged entry points, windows with sinks and attention with capped, biased or masked scores
// for torch tensors, as a Python extension module.
//
// Their kernels can take a few microseconds, less than a ctypes call with its checks and
// allocations takes in Python, so checks, output allocation and the call itself run here:
// the C ABI is unchanged and holds all of the computation.  The module finds the library's
// functions by name (load), so it links only against torch.
#include <Python.h>

#include <dlfcn.h>

#include <ATen/cuda/EmptyTensor.h>
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
decltype(&fa_fwd_score) g_fwd_score;
decltype(&fa_bwd_score) g_bwd_score;
decltype(&fa_fwd_score_workspace_size) g_fwd_score_workspace;
decltype(&fa_bwd_score_workspace_size) g_bwd_score_workspace[2];  // [whether a bias's gradient is wanted]
decltype(&fa_fwd_paged_score) g_paged_score[2];
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

// An uninitialised tensor, made without the dispatcher (which took 1.2 us of the 3.5 that a call's two
// results cost).
at::Tensor make(at::IntArrayRef sizes, at::ScalarType type, const at::Device& dev) {
    return at::Tensor(at::detail::empty_cuda(sizes, type, dev, std::nullopt));
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
            else out = &made.emplace(make({T, H, d}, at::kBFloat16, c.dev));
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

// A fa_score from Python's arguments softcap, slopes, bias and buckets, for H heads on a device.
fa_score check_score(PyObject* const* a, int64_t H, const at::Device& dev) {
    fa_score s{};
    if (a[0] != Py_None) {
        const double cap = PyFloat_AsDouble(a[0]);
        if (cap == -1.0 && PyErr_Occurred()) throw PyErr{};
        s.softcap = static_cast<float>(cap);
        require(s.softcap > 0.f, "softcap must be above 0");
    }
    const at::Tensor *slopes = tensor_or_none(a[1], "slopes"), *bias = tensor_or_none(a[2], "bias");
    const at::Tensor* buckets = tensor_or_none(a[3], "buckets");
    require((bias != nullptr) == (buckets != nullptr), "a bias needs buckets, and buckets a bias");
    require(!bias || !slopes, "slopes or a bias, not both");
    if (slopes) {
        require(slopes->dim() == 1 && slopes->size(0) == H && slopes->scalar_type() == at::kFloat && slopes->device() == dev &&
                    slopes->is_contiguous(),
                "slopes must be contiguous fp32 [H] on the queries' device");
        s.slopes = static_cast<const float*>(slopes->data_ptr());
    }
    if (bias) {
        require(bias->dim() == 2 && bias->size(1) == H && bias->device() == dev && bias->is_contiguous() &&
                    (bias->scalar_type() == at::kFloat || bias->scalar_type() == at::kBFloat16),
                "bias must be contiguous fp32 or bf16 [num_buckets, H] on the queries' device");
        require(buckets->dim() == 1 && buckets->size(0) % 2 == 1 && buckets->scalar_type() == at::kInt &&
                    buckets->device() == dev && buckets->is_contiguous(),
                "buckets must be contiguous int32 [2 * max_distance + 1] on the queries' device");
        if (H == 0) return s;  // (biases of no heads have no address)
        s.bias = bias->data_ptr();
        s.buckets = static_cast<const int*>(buckets->data_ptr());
        s.bias_f32 = bias->scalar_type() == at::kFloat;
        s.num_buckets = to_int(bias->size(0));
        s.max_distance = to_int(buckets->size(0) / 2);
    }
    return s;
}

// fwd_paged(q, k_cache, v_cache, page_table, lens, tau, window, sinks, k_scale, v_scale,
//           out, lse, workspace[, softcap, slopes, bias, buckets]) -> (O, LSE)
PyObject* fwd_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, n == 13 ? 13 : 17, [&]() -> PyObject* {
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
        fa_score score{};
        if (n > 13) score = check_score(a + 13, H, c.dev);
        const c10::cuda::OptionalCUDAGuard guard(c.dev);
        std::optional<at::Tensor> made_out, made_lse, made_ws;
        if (out) check_rows(*out, q.sizes(), c, "out");
        else out = &made_out.emplace(make(q.sizes(), at::kBFloat16, c.dev));
        if (lse)
            require(lse->sizes() == q.sizes().slice(0, 3) && lse->scalar_type() == at::kFloat && lse->device() == c.dev &&
                        lse->is_contiguous(),
                    "lse must be contiguous fp32 [B, H, Nq] on the cache's device");
        else lse = &made_lse.emplace(make(q.sizes().slice(0, 3), at::kFloat, c.dev));
        size_t bytes;
        if (ws) {
            require(ws->device() == c.dev && ws->is_contiguous(), "workspace must be contiguous, on the cache's device");
            bytes = ws->nbytes();
        } else {
            bytes = g_workspace(&c.c, to_int(H), to_int(Nq), window, sinks);
            if (bytes) ws = &made_ws.emplace(make({static_cast<int64_t>(bytes)}, at::kByte, c.dev));
        }
        const auto call = [&](auto f, auto... more) {
            return f(&c.c, q.data_ptr(), q.stride(0), q.stride(1), q.stride(2), out->data_ptr(), out->stride(0),
                     out->stride(1), out->stride(2), static_cast<float*>(lse->data_ptr()), to_int(H), to_int(Nq), tau,
                     window, sinks, more..., ws ? ws->data_ptr() : nullptr, bytes,
                     c10::cuda::getCurrentCUDAStream(c.dev.index()).stream());
        };
        if (n > 13)
            check_status(call(g_paged_score[c.fp8], static_cast<const fa_score*>(&score)),
                         c.fp8 ? "fa_fwd_paged_score_fp8" : "fa_fwd_paged_score");
        else
            check_status(call(g_paged[c.fp8]), c.fp8 ? "fa_fwd_paged_fp8" : "fa_fwd_paged");
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
        else out = &made_out.emplace(make(q.sizes(), at::kBFloat16, q.device()));
        if (lse) check_lse(*lse, q);
        else lse = &made_lse.emplace(make(q.sizes().slice(0, 3), at::kFloat, q.device()));
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
            else g = &made[i].emplace(make(q.sizes(), at::kBFloat16, q.device()));
            grads[i] = g->data_ptr();
        }
        const at::Tensor* ws = tensor_or_none(a[12], "workspace");
        if (ws) require(ws->device() == q.device() && ws->is_contiguous(), "workspace must be contiguous, on the inputs' device");
        else {
            const size_t need = g_bwd_workspace(B, H, N, d);
            ws = &made_ws.emplace(make({static_cast<int64_t>(need ? need : 1)}, at::kByte, q.device()));
        }
        check_status(g_bwd_sinks(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), go.data_ptr(),
                                 static_cast<const float*>(lse.data_ptr()), grads[0], grads[1], grads[2], ws->data_ptr(),
                                 ws->nbytes(), B, H, N, d, tau, window, sinks,
                                 c10::cuda::getCurrentCUDAStream(q.device().index()).stream()),
                     "fa_bwd_sinks");
        return results({{&made[0], a[9]}, {&made[1], a[10]}, {&made[2], a[11]}});
    });
}

// Queries [B, H, N, d] and keys and values [B, H_kv, N, d] of attention with changed scores, and the
// rest of its fa_score: documents, prefixes and window.
struct Scored {
    int B, H, H_kv, N, d;
    fa_score f;
};
Scored check_scored(const at::Tensor& q, const at::Tensor& k, const at::Tensor& v, PyObject* const* a, int causal) {
    check_attention({&q});
    check_attention({&k, &v});
    require(k.device() == q.device() && k.size(0) == q.size(0) && k.size(2) == q.size(2) && k.size(3) == q.size(3),
            "keys and values must be [B, H_kv, N, d] on the queries' device");
    Scored s{to_int(q.size(0)), to_int(q.size(1)), to_int(k.size(1)), to_int(q.size(2)), to_int(q.size(3)),
             check_score(a, q.size(1), q.device())};
    require(s.H_kv == 0 ? s.H == 0 : s.H % s.H_kv == 0, "the query heads must be a multiple of the key heads");
    const at::Tensor *docs = tensor_or_none(a[4], "docs"), *prefix = tensor_or_none(a[5], "prefix");
    if (docs) {
        require(docs->dim() == 2 && docs->size(0) == s.B && docs->size(1) == s.N && docs->scalar_type() == at::kInt &&
                    docs->device() == q.device() && docs->is_contiguous(),
                "docs must be contiguous int32 [B, N] on the queries' device");
        s.f.docs = static_cast<const int*>(docs->data_ptr());
    }
    if (prefix) {
        require(causal, "a prefix needs causal=True");
        require(prefix->dim() == 1 && prefix->size(0) == s.B && prefix->scalar_type() == at::kInt &&
                    prefix->device() == q.device() && prefix->is_contiguous(),
                "prefix must be contiguous int32 [B] on the queries' device");
        s.f.prefix = static_cast<const int*>(prefix->data_ptr());
    }
    if (a[6] != Py_None) {
        require(causal, "a window needs causal=True");
        s.f.window = to_int(integer(a[6]));
        require(s.f.window >= 1, "a window holds at least one key");
    }
    return s;
}
// A workspace as given, or one of `need` bytes.
const at::Tensor* workspace_of(PyObject* o, size_t need, const at::Tensor& q, std::optional<at::Tensor>& made) {
    const at::Tensor* ws = tensor_or_none(o, "workspace");
    if (ws) require(ws->device() == q.device() && ws->is_contiguous(), "workspace must be contiguous, on the inputs' device");
    else if (need) ws = &made.emplace(make({static_cast<int64_t>(need)}, at::kByte, q.device()));
    return ws;
}
int truth(PyObject* o) {
    const int t = PyObject_IsTrue(o);
    if (t < 0) throw PyErr{};
    return t;
}

// fwd_score(q, k, v, causal, tau, softcap, slopes, bias, buckets, docs, prefix, window, out, lse,
//           workspace) -> (O, LSE)
PyObject* fwd_score(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 15, [&]() -> PyObject* {
        const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
        const at::Tensor *out = tensor_or_none(a[12], "out"), *lse = tensor_or_none(a[13], "lse");
        const int causal = truth(a[3]);
        const Scored s = check_scored(q, k, v, a + 5, causal);
        const float tau = scale_of(a[4], s.d);
        const c10::cuda::OptionalCUDAGuard guard(q.device());
        std::optional<at::Tensor> made_out, made_lse, made_ws;
        if (out) check_attention({&q, out});
        else out = &made_out.emplace(make(q.sizes(), at::kBFloat16, q.device()));
        if (lse) check_lse(*lse, q);
        else lse = &made_lse.emplace(make(q.sizes().slice(0, 3), at::kFloat, q.device()));
        const at::Tensor* ws = workspace_of(a[14], g_fwd_score_workspace(s.B, s.N, &s.f), q, made_ws);
        check_status(g_fwd_score(q.data_ptr(), k.data_ptr(), v.data_ptr(), out->data_ptr(), static_cast<float*>(lse->data_ptr()),
                                 s.B, s.H, s.H_kv, s.N, s.d, tau, causal, &s.f, ws ? ws->data_ptr() : nullptr,
                                 ws ? ws->nbytes() : 0, c10::cuda::getCurrentCUDAStream(q.device().index()).stream()),
                     "fa_fwd_score");
        return results({{&made_out, a[12]}, {&made_lse, a[13]}});
    });
}

// bwd_score(q, k, v, o, do, lse, causal, tau, softcap, slopes, bias, buckets, docs, prefix, window,
//           dq, dk, dv, dbias, workspace) -> (dQ, dK, dV, dBias); dbias False: not computed, None back
PyObject* bwd_score(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 20, [&]() -> PyObject* {
        const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &o = tensor(a[3], "o");
        const at::Tensor &go = tensor(a[4], "do"), &lse = tensor(a[5], "lse");
        const int causal = truth(a[6]);
        const Scored s = check_scored(q, k, v, a + 8, causal);
        check_attention({&q, &o, &go});
        check_lse(lse, q);
        const float tau = scale_of(a[7], s.d);
        const c10::cuda::OptionalCUDAGuard guard(q.device());
        std::optional<at::Tensor> made[4], made_ws;
        void* grads[4] = {nullptr, nullptr, nullptr, nullptr};
        for (int i = 0; i < 3; ++i) {
            const at::Tensor* g = tensor_or_none(a[15 + i], "a gradient");
            const at::Tensor& of = i == 0 ? q : k;
            if (g) check_attention({&of, g});
            else g = &made[i].emplace(make(of.sizes(), at::kBFloat16, q.device()));
            grads[i] = g->data_ptr();
        }
        const bool wanted = a[10] != Py_None && a[18] != Py_False;
        if (wanted) {
            const at::Tensor *g = tensor_or_none(a[18], "dbias"), &bias = tensor(a[10], "bias");
            if (g)
                require(g->sizes() == bias.sizes() && g->scalar_type() == bias.scalar_type() && g->device() == q.device() &&
                            g->is_contiguous(),
                        "dbias must be contiguous and like bias");
            else g = &made[3].emplace(make(bias.sizes(), bias.scalar_type(), q.device()));
            if (s.f.bias) grads[3] = g->data_ptr();
        }
        const at::Tensor* ws = workspace_of(a[19], g_bwd_score_workspace[grads[3] != nullptr](s.B, s.H, s.N, s.d, causal, &s.f), q, made_ws);
        check_status(g_bwd_score(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), go.data_ptr(),
                                 static_cast<const float*>(lse.data_ptr()), grads[0], grads[1], grads[2], grads[3], s.B, s.H,
                                 s.H_kv, s.N, s.d, tau, causal, &s.f, ws ? ws->data_ptr() : nullptr, ws ? ws->nbytes() : 0,
                                 c10::cuda::getCurrentCUDAStream(q.device().index()).stream()),
                     "fa_bwd_score");
        return results({{&made[0], a[15]}, {&made[1], a[16]}, {&made[2], a[17]}, {&made[3], wanted ? a[18] : Py_None}});
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
        g_fwd_score = reinterpret_cast<decltype(&fa_fwd_score)>(find("fa_fwd_score"));
        g_bwd_score = reinterpret_cast<decltype(&fa_bwd_score)>(find("fa_bwd_score"));
        g_fwd_score_workspace = reinterpret_cast<decltype(&fa_fwd_score_workspace_size)>(find("fa_fwd_score_workspace_size"));
        g_bwd_score_workspace[0] =
            reinterpret_cast<decltype(&fa_bwd_score_workspace_size)>(find("fa_bwd_score_frozen_workspace_size"));
        g_bwd_score_workspace[1] = reinterpret_cast<decltype(&fa_bwd_score_workspace_size)>(find("fa_bwd_score_workspace_size"));
        g_paged_score[0] = reinterpret_cast<decltype(&fa_fwd_paged_score)>(find("fa_fwd_paged_score"));
        g_paged_score[1] = reinterpret_cast<decltype(&fa_fwd_paged_score)>(find("fa_fwd_paged_score_fp8"));
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
                           method<fwd_sinks>("fwd_sinks"), method<bwd_sinks>("bwd_sinks"),
                           method<fwd_score>("fwd_score"), method<bwd_score>("bwd_score"), method<load>("load"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "fa_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_fa_binding() { return PyModule_Create(&g_module); }
