// rrf_torch.cpp -- the Python binding of the calls of a layer around its
// attention (see layer.py): checks of torch tensors, new outputs, the current
// stream, and a call of the C ABI.  No arithmetic.
//
// These calls are short: a decode step's kernels take 2 to 12 us, and looking
// at a dozen tensors and passing thirty arguments from Python took 9 to 17 us
// a call.  The module calls the C functions of the library that the package
// has loaded (bind(), called once), so there is one librrf.so in a process.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <stdexcept>
#include <string>

#include "rrf.h"

namespace {

// The C functions, by address, and what raises a status as an exception.
decltype(&rrf_scaled_mm_fp8_act) f_mm_fp8;
decltype(&rrf_scaled_mm_mxfp8_act) f_mm_mx;
decltype(&rrf_qk_norm_rope) f_norm;
decltype(&rrf_kv_cache_write_fp8) f_write;
decltype(&rrf_qk_norm_rope_kv_cache_fp8) f_fused;
decltype(&rrf_kv_cache_read_fp8) f_read;
PyObject* g_raise = nullptr;

// A refused argument: ValueError with this text.
struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};

void need(bool ok, const char* name, const char* what) {
    if (!ok) throw Refused(std::string(name) + " must be " + what);
}

// (These calls have no backward pass and are not seen by torch's dispatcher: a
// tensor whose gradient autograd would record is refused, not dropped from the
// graph without a word.)
const at::Tensor& tensor(PyObject* o, const char* name) {
    need(THPVariable_Check(o), name, "a tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    need(!t.requires_grad() || !at::GradMode::is_enabled(), name,
         "a tensor that does not require grad (this call has no gradient; call it under "
         "torch.no_grad())");
    return t;
}

// A tensor or None (an undefined one).
const at::Tensor& optional(PyObject* o, const char* name) {
    static const at::Tensor none;
    return o == Py_None ? none : tensor(o, name);
}

double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused("a number is wanted");
    return v;
}

int64_t integer(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused("an integer is wanted");
    return v;
}

int truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused("a truth value is wanted");
    return v;
}

// The call has written t: autograd, which may have saved it, is to know.
void written(const at::Tensor& t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

bool on(const at::Tensor& t, int index) { return t.is_cuda() && t.get_device() == index; }

// A dense vector of n values (any shape).
const void* vector(const at::Tensor& t, const char* name, at::ScalarType type, int64_t n,
                   int index) {
    need(t.defined() && t.scalar_type() == type && t.numel() == n && t.is_contiguous(), name,
         "a contiguous tensor of the type and the number of values that the call names");
    need(on(t, index), name, "on the inputs' device");
    return t.data_ptr();
}

// bf16 [tokens, heads, dim], a head's values contiguous.
struct Heads {
    void* p;
    int64_t token, head;
};

Heads heads(const at::Tensor& t, const char* name, int64_t tokens, int64_t n, int64_t dim,
            int index) {
    need(t.scalar_type() == at::kBFloat16 && t.dim() == 3 && t.size(0) == tokens &&
             t.size(1) == n && t.size(2) == dim && t.stride(2) == 1,
         name, "bf16 [tokens, heads, head_dim] with contiguous heads");
    need(on(t, index), name, "on the inputs' device");
    return Heads{t.data_ptr(), t.stride(0), t.stride(1)};
}

int device_of(const at::Tensor& t, const char* name) {
    need(t.is_cuda(), name, "a CUDA tensor");
    return t.get_device();
}

at::Tensor fresh(at::IntArrayRef shape, int index) {
    return at::detail::empty_cuda(shape, at::kBFloat16,
                                  at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(index)),
                                  c10::nullopt);
}

// call(stream) on the device and its current stream.
template <class Call>
bool launch(int index, Call call) {
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
    const rrf_status st = call(c10::cuda::getCurrentCUDAStream(index).stream());
    if (st == RRF_OK) return true;
    PyObject* r = PyObject_CallFunction(g_raise, "i", (int)st);
    Py_XDECREF(r);  // (it raises)
    return false;
}

// A binding's body: refusals and C++ errors as Python exceptions.
template <class Body>
PyObject* guarded(Py_ssize_t nargs, Py_ssize_t want, Body body) {
    if (nargs != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return body();
    } catch (const Refused& e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.what());
    } catch (...) {  // torch's own (out of memory, a CUDA error) as torch raises them
        torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

// --------------------------------------------------------------- products ---

// (a, sa, b, sb, bias, activation, residual, out), MX or not
template <bool MX>
PyObject* scaled_mm(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
    return guarded(nargs, 8, [&]() -> PyObject* {
        const at::Tensor &a = tensor(v[0], "a"), &sa = tensor(v[1], MX ? "sa" : "a_scale");
        const at::Tensor &b = tensor(v[2], "b"), &sb = tensor(v[3], MX ? "sb" : "b_scale");
        const at::Tensor &bias = optional(v[4], "bias"), &res = optional(v[6], "residual");
        at::Tensor out = optional(v[7], "out");
        const int index = device_of(a, "a");
        need(a.scalar_type() == at::kFloat8_e4m3fn && a.dim() == 2 && a.is_contiguous(), "a",
             "a contiguous 2-D float8_e4m3fn tensor");
        const int64_t m = a.size(0), k = a.size(1);
        need(b.scalar_type() == at::kFloat8_e4m3fn && b.dim() == 2 && b.is_contiguous() &&
                 b.size(1) == k && on(b, index),
             "b", "a contiguous float8_e4m3fn [N, K] tensor on a's device");
        const int64_t n = b.size(0);
        const auto scales = [](int64_t rows, int64_t cols) {
            return MX ? (rows + 127) / 128 * 128 * (cols / 32) : rows;
        };
        const at::ScalarType type = MX ? at::kByte : at::kFloat;
        const void* pa = vector(sa, MX ? "sa" : "a_scale", type, scales(m, k), index);
        const void* pb = vector(sb, MX ? "sb" : "b_scale", type, scales(n, k), index);
        const void* pbias =
            bias.defined() ? vector(bias, "bias", at::kBFloat16, n, index) : nullptr;
        const auto matrix = [&](const at::Tensor& t, const char* name) {
            need(t.scalar_type() == at::kBFloat16 && t.dim() == 2 && t.size(0) == m &&
                     t.size(1) == n && t.is_contiguous() && on(t, index),
                 name, "a contiguous bf16 [M, N] tensor on a's device");
            return t.data_ptr();
        };
        const void* pres = res.defined() ? matrix(res, "residual") : nullptr;
        if (!out.defined()) out = fresh({m, n}, index);
        void* po = matrix(out, "out");
        const int act = (int)integer(v[5]);
        const bool ok = launch(index, [&](rrf_stream_t s) {
            if constexpr (MX)
                return f_mm_mx(a.data_ptr(), pa, b.data_ptr(), pb, pbias, act, pres, po, m, n, k,
                               s);
            else
                return f_mm_fp8(a.data_ptr(), static_cast<const float*>(pa), b.data_ptr(),
                                static_cast<const float*>(pb), pbias, act, pres, po, m, n, k, s);
        });
        if (!ok) return nullptr;
        written(out);
        return THPVariable_Wrap(out);
    });
}

// --------------------------------------------------------- heads and cache ---

// The norm's weights and the rotation, from (q_gamma, k_gamma, eps,
// weight_offset, cos_sin, positions, interleaved).
struct Norm {
    const void *q_gamma, *k_gamma;
    float eps, weight_offset;
    const float* cos_sin = nullptr;
    int64_t rows = 0, rot = 0;
    const int64_t* positions = nullptr;
    int interleaved;

    Norm(PyObject* const* v, int64_t tokens, int64_t dim, int index) {
        q_gamma = vector(tensor(v[0], "q_gamma"), "q_gamma", at::kBFloat16, dim, index);
        k_gamma = vector(tensor(v[1], "k_gamma"), "k_gamma", at::kBFloat16, dim, index);
        eps = (float)number(v[2]);
        weight_offset = (float)number(v[3]);
        interleaved = truth(v[6]);
        const at::Tensor& table = optional(v[4], "cos_sin");
        if (!table.defined()) return;
        need(table.scalar_type() == at::kFloat && table.dim() == 2 && table.size(1) > 0 &&
                 table.is_contiguous() && on(table, index),
             "cos_sin", "a contiguous float32 [max_positions, rot_dim] tensor on the inputs' "
                        "device, or None (the norm alone)");
        cos_sin = static_cast<const float*>(table.data_ptr());
        rows = table.size(0);
        rot = table.size(1);
        positions = static_cast<const int64_t*>(
            vector(tensor(v[5], "positions"), "positions", at::kLong, tokens, index));
    }
};

// (k_cache, k_scales, v_cache, v_scales)
rrf_kv_cache cache_of(PyObject* const* v, int64_t n, int64_t dim, int index) {
    const at::Tensor &kc = tensor(v[0], "k_cache"), &ks = tensor(v[1], "k_scales");
    const at::Tensor &vc = tensor(v[2], "v_cache"), &vs = tensor(v[3], "v_scales");
    rrf_kv_cache c;
    need(kc.dim() == 4 && kc.size(2) == n && kc.size(3) == dim && kc.stride(3) == 1, "k_cache",
         "[pages, page_size, kv_heads, head_dim] with contiguous heads");
    c.num_pages = kc.size(0);
    c.page_size = kc.size(1);
    need(vc.sizes() == kc.sizes() && vc.strides() == kc.strides(), "v_cache",
         "of k_cache's shape and strides");
    need(ks.dim() == 3 && ks.size(0) == c.num_pages && ks.size(1) == c.page_size &&
             ks.size(2) == n,
         "k_scales", "[pages, page_size, kv_heads]");
    need(vs.sizes() == ks.sizes() && vs.strides() == ks.strides(), "v_scales",
         "of k_scales' shape and strides");
    need(kc.scalar_type() == at::kFloat8_e4m3fn && vc.scalar_type() == at::kFloat8_e4m3fn &&
             ks.scalar_type() == at::kFloat && vs.scalar_type() == at::kFloat,
         "the cache", "float8_e4m3fn codes and float32 scales");
    need(on(kc, index) && on(vc, index) && on(ks, index) && on(vs, index), "the cache",
         "on the inputs' device");
    c.k_codes = kc.data_ptr();
    c.v_codes = vc.data_ptr();
    c.k_scales = static_cast<float*>(ks.data_ptr());
    c.v_scales = static_cast<float*>(vs.data_ptr());
    for (int i = 0; i < 3; ++i) {
        c.code_strides[i] = kc.stride(i);
        c.scale_strides[i] = ks.stride(i);
    }
    return c;
}

// (k_cache, k_scales, v_cache, v_scales), looked at before
void written_cache(PyObject* const* v) {
    for (int i = 0; i < 4; ++i) written(THPVariable_Unpack(v[i]));
}

const at::Tensor& heads_tensor(PyObject* o, const char* name) {
    const at::Tensor& t = tensor(o, name);
    need(t.dim() == 3, name, "[tokens, heads, head_dim]");
    return t;
}

// (q, k, q_gamma, k_gamma, eps, weight_offset, cos_sin, positions, interleaved,
//  q_out, k_out)
PyObject* qk_norm_rope(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
    return guarded(nargs, 11, [&]() -> PyObject* {
        const at::Tensor &q = heads_tensor(v[0], "q"), &k = heads_tensor(v[1], "k");
        const int index = device_of(q, "q");
        const int64_t t = q.size(0), hq = q.size(1), d = q.size(2), hk = k.size(1);
        const Heads qh = heads(q, "q", t, hq, d, index), kh = heads(k, "k", t, hk, d, index);
        const Norm norm(v + 2, t, d, index);
        at::Tensor qo = optional(v[9], "q_out"), ko = optional(v[10], "k_out");
        if (!qo.defined()) qo = fresh({t, hq, d}, index);
        if (!ko.defined()) ko = fresh({t, hk, d}, index);
        const Heads qoh = heads(qo, "q_out", t, hq, d, index);
        const Heads koh = heads(ko, "k_out", t, hk, d, index);
        if (!launch(index, [&](rrf_stream_t s) {
                return f_norm(qh.p, qh.token, qh.head, kh.p, kh.token, kh.head, qoh.p, qoh.token,
                              qoh.head, koh.p, koh.token, koh.head, norm.q_gamma, norm.k_gamma,
                              norm.eps, norm.weight_offset, norm.cos_sin, norm.rows, norm.rot,
                              norm.interleaved, norm.positions, t, hq, hk, d, s);
            }))
            return nullptr;
        written(qo);
        written(ko);
        PyObject* a = THPVariable_Wrap(qo);
        PyObject* b = THPVariable_Wrap(ko);
        PyObject* pair = a && b ? PyTuple_Pack(2, a, b) : nullptr;
        Py_XDECREF(a);
        Py_XDECREF(b);
        return pair;
    });
}

// (k, v, slots, k_cache, k_scales, v_cache, v_scales, scale_ub)
PyObject* kv_cache_write(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
    return guarded(nargs, 8, [&]() -> PyObject* {
        const at::Tensor &k = heads_tensor(v[0], "k"), &x = heads_tensor(v[1], "v");
        const int index = device_of(k, "k");
        const int64_t t = k.size(0), h = k.size(1), d = k.size(2);
        const Heads kh = heads(k, "k", t, h, d, index), vh = heads(x, "v", t, h, d, index);
        const auto* slots = static_cast<const int64_t*>(
            vector(tensor(v[2], "slots"), "slots", at::kLong, t, index));
        const rrf_kv_cache cache = cache_of(v + 3, h, d, index);
        const float ub = (float)number(v[7]);
        if (!launch(index, [&](rrf_stream_t s) {
                return f_write(kh.p, kh.token, kh.head, vh.p, vh.token, vh.head, slots, ub,
                               &cache, t, h, d, s);
            }))
            return nullptr;
        written_cache(v + 3);
        Py_RETURN_NONE;
    });
}

// (q, k, v, q_gamma, k_gamma, eps, weight_offset, cos_sin, positions,
//  interleaved, slots, k_cache, k_scales, v_cache, v_scales, scale_ub, q_out)
PyObject* qk_norm_rope_kv_cache(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
    return guarded(nargs, 17, [&]() -> PyObject* {
        const at::Tensor &q = heads_tensor(v[0], "q"), &k = heads_tensor(v[1], "k");
        const at::Tensor& x = heads_tensor(v[2], "v");
        const int index = device_of(q, "q");
        const int64_t t = q.size(0), hq = q.size(1), d = q.size(2), hk = k.size(1);
        const Heads qh = heads(q, "q", t, hq, d, index), kh = heads(k, "k", t, hk, d, index);
        const Heads vh = heads(x, "v", t, hk, d, index);
        const Norm norm(v + 3, t, d, index);
        const auto* slots = static_cast<const int64_t*>(
            vector(tensor(v[10], "slots"), "slots", at::kLong, t, index));
        const rrf_kv_cache cache = cache_of(v + 11, hk, d, index);
        const float ub = (float)number(v[15]);
        at::Tensor qo = optional(v[16], "q_out");
        if (!qo.defined()) qo = fresh({t, hq, d}, index);
        const Heads qoh = heads(qo, "q_out", t, hq, d, index);
        const bool ok = launch(index, [&](rrf_stream_t s) {
            return f_fused(qh.p, qh.token, qh.head, kh.p, kh.token, kh.head, vh.p, vh.token,
                           vh.head, qoh.p, qoh.token, qoh.head, norm.q_gamma, norm.k_gamma,
                           norm.eps, norm.weight_offset, norm.cos_sin, norm.rows, norm.rot,
                           norm.interleaved, norm.positions, slots, ub, &cache, t, hq, hk, d, s);
        });
        if (!ok) return nullptr;
        written(qo);
        written_cache(v + 11);
        return THPVariable_Wrap(qo);
    });
}

// (k_cache, k_scales, v_cache, v_scales, block_table, seq_starts, k_out, v_out)
PyObject* kv_cache_read(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
    return guarded(nargs, 8, [&]() -> PyObject* {
        const at::Tensor &table = tensor(v[4], "block_table"), &starts = tensor(v[5], "seq_starts");
        const at::Tensor &ko = heads_tensor(v[6], "k_out"), &vo = tensor(v[7], "v_out");
        const int index = device_of(ko, "k_out");
        const int64_t rows = ko.size(0), h = ko.size(1), d = ko.size(2);
        need(ko.scalar_type() == at::kBFloat16 && ko.is_contiguous(), "k_out",
             "contiguous bf16 [rows, kv_heads, head_dim]");
        need(vo.scalar_type() == at::kBFloat16 && vo.sizes() == ko.sizes() &&
                 vo.is_contiguous() && on(vo, index),
             "v_out", "contiguous bf16 of k_out's shape, on its device");
        need(table.scalar_type() == at::kInt && table.dim() == 2 && on(table, index) &&
                 (table.size(1) <= 1 || table.stride(1) == 1),
             "block_table", "an int32 [sequences, pages] tensor on the outputs' device");
        const int64_t n = table.size(0);
        const auto* first = static_cast<const int32_t*>(
            vector(starts, "seq_starts", at::kInt, n + 1, index));
        const rrf_kv_cache cache = cache_of(v, h, d, index);
        if (!launch(index, [&](rrf_stream_t s) {
                return f_read(&cache, static_cast<const int32_t*>(table.data_ptr()),
                              table.stride(0), table.size(1), first, n, ko.data_ptr(),
                              vo.data_ptr(), rows, h, d, s);
            }))
            return nullptr;
        written(ko);
        written(vo);
        return PyTuple_Pack(2, v[6], v[7]);
    });
}

// (raise, addresses of the six functions)
PyObject* bind(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
    return guarded(nargs, 7, [&]() -> PyObject* {
        void* at[6];
        for (int i = 0; i < 6; ++i) {
            at[i] = PyLong_AsVoidPtr(v[1 + i]);
            if (at[i] == nullptr) throw Refused("an address of a function is wanted");
        }
        Py_INCREF(v[0]);
        Py_XDECREF(g_raise);
        g_raise = v[0];
        f_mm_fp8 = reinterpret_cast<decltype(f_mm_fp8)>(at[0]);
        f_mm_mx = reinterpret_cast<decltype(f_mm_mx)>(at[1]);
        f_norm = reinterpret_cast<decltype(f_norm)>(at[2]);
        f_write = reinterpret_cast<decltype(f_write)>(at[3]);
        f_fused = reinterpret_cast<decltype(f_fused)>(at[4]);
        f_read = reinterpret_cast<decltype(f_read)>(at[5]);
        Py_RETURN_NONE;
    });
}

#define RRF_METHOD(name, f) \
    {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}

PyMethodDef g_methods[] = {RRF_METHOD("bind", bind),
                           RRF_METHOD("scaled_mm_fp8_act", scaled_mm<false>),
                           RRF_METHOD("scaled_mm_mxfp8_act", scaled_mm<true>),
                           RRF_METHOD("qk_norm_rope", qk_norm_rope),
                           RRF_METHOD("kv_cache_write_fp8", kv_cache_write),
                           RRF_METHOD("qk_norm_rope_kv_cache_fp8", qk_norm_rope_kv_cache),
                           RRF_METHOD("kv_cache_read_fp8", kv_cache_read),
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_rrf_torch", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__rrf_torch() { return PyModule_Create(&g_module); }
