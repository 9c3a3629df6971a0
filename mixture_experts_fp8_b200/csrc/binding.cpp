// binding.cpp -- the marshalling of the operators around the layer for Python: checks of the tensors,
// allocation of outputs and temporaries, the caller's stream, and the call of libmoefp8.so.  Nothing is
// computed here.  These operators run in 3 to 10 us at decode sizes, where the same steps in Python took
// 8 to 18 us a call (two a tensor allocated, half one a tensor checked) and take 3.5 to 10 here.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cstdint>
#include <string>

#include "moefp8.h"

namespace {

// libmoefp8.so's entry points, as the package has loaded it.
struct Lib {
    decltype(&moe_last_error) last_error;
    decltype(&moe_add_rms_norm) add_rms_norm;
    decltype(&moe_linear) linear;
    decltype(&moe_linear_workspace_size) linear_workspace_size;
    decltype(&moe_balance_loss) balance_loss;
    decltype(&moe_balance_workspace_size) balance_workspace_size;
    decltype(&moe_route_backward) route_backward;
} g_lib;
PyObject* g_error = nullptr;                            // MoeError

// Set MoeError(code, message); returns false.
bool refuse(int code, const std::string& msg) {
    PyObject* e = PyObject_CallFunction(g_error, "is", code, msg.c_str());
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    return false;
}
bool refuse(const std::string& msg) { return refuse(MOE_ERR_INVALID_ARG, msg); }

bool check(int rc) { return rc == MOE_OK || refuse(rc, g_lib.last_error()); }

const char* type_name(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return "torch.bfloat16";
        case at::kFloat: return "torch.float32";
        case at::kDouble: return "torch.float64";
        case at::kHalf: return "torch.float16";
        case at::kByte: return "torch.uint8";
        case at::kInt: return "torch.int32";
        case at::kLong: return "torch.int64";
        case at::kBool: return "torch.bool";
        default: return at::toString(t);
    }
}

std::string shape_name(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}

bool tensor(PyObject* o, const char* name, const at::Tensor** out) {
    if (!THPVariable_Check(o)) return refuse(std::string(name) + " must be a tensor");
    *out = &THPVariable_Unpack(o);
    return true;
}

// One call: its device (the current one, that of its first tensor) and stream.
struct Call {
    int dev = -1;
    cudaStream_t stream = nullptr;
    c10::optional<c10::Stream> other, ambient;         // the caller's, and then the current one, for the allocator

    bool begin(PyObject* first, const char* name, PyObject* stream_) {
        const at::Tensor* t;
        if (!tensor(first, name, &t)) return false;
        if (!t->is_cuda()) return refuse(std::string(name) + " is on " + t->device().str() + ", not on the current device");
        const int current = c10::cuda::current_device();
        dev = t->get_device();
        if (dev != current)
            return refuse(std::string(name) + " is on cuda:" + std::to_string(dev) + ", the current device is cuda:" +
                          std::to_string(current));
        if (stream_ == Py_None) {
            stream = c10::cuda::getCurrentCUDAStream(dev).stream();
            return true;
        }
        long long v[4];
        const char* names[4] = {"cuda_stream", "stream_id", "device_index", "device_type"};
        for (int i = 0; i < 4; ++i) {
            PyObject* a = PyObject_GetAttrString(stream_, names[i]);
            if (!a) return false;
            v[i] = PyLong_AsLongLong(a);
            Py_DECREF(a);
            if (v[i] == -1 && PyErr_Occurred()) return false;
        }
        if (v[2] != dev)
            return refuse("stream is on cuda:" + std::to_string(v[2]) + ", " + name + " on cuda:" + std::to_string(dev));
        stream = reinterpret_cast<cudaStream_t>(v[0]);
        other = c10::Stream::unpack3(v[1], static_cast<c10::DeviceIndex>(v[2]), static_cast<c10::DeviceType>(v[3]));
        ambient = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).unwrap();
        return true;
    }

    // A tensor that the call allocates, from the pool of the stream that it runs on: a block of the current stream's
    // pool may still be in use by kernels pending there, which another stream does not wait for.  A result that the
    // current stream uses too is kept, once freed, until that stream has passed.
    at::Tensor make(at::IntArrayRef shape, at::ScalarType type, bool result = true) const {
        const at::Device device(at::kCUDA, static_cast<c10::DeviceIndex>(dev));
        if (!other) return at::detail::empty_cuda(shape, type, device, c10::nullopt);
        const c10::cuda::CUDAStreamGuard guard(*other);
        at::Tensor t = at::detail::empty_cuda(shape, type, device, c10::nullopt);
        if (result) t.record_stream(*ambient);
        return t;
    }

    // Pointer of tensor o (None: NULL); anything but a contiguous tensor of this shape, type and device is refused.
    bool arg(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type, void** out) const {
        *out = nullptr;
        if (o == Py_None) return true;
        const at::Tensor* t;
        if (!tensor(o, name, &t)) return false;
        return arg(*t, name, shape, type, out);
    }
    bool arg(const at::Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type, void** out) const {
        if (t.scalar_type() == type && t.is_cuda() && t.get_device() == dev && t.sizes() == shape && t.is_contiguous()) {
            *out = t.data_ptr();
            return true;
        }
        return refuse(std::string(name) + " must be a contiguous " + type_name(type) + " tensor of shape " + shape_name(shape) +
                      " on cuda:" + std::to_string(dev) + ", got " + type_name(t.scalar_type()) + " " + shape_name(t.sizes()) +
                      " on " + t.device().str() + (t.is_contiguous() ? "" : ", not contiguous"));
    }

    // The caller's workspace, or (None) one of `bytes` bytes for this call, kept alive by `own`.
    bool workspace(PyObject* o, size_t bytes, at::Tensor& own, void** out, size_t* have) const {
        if (o == Py_None) {
            own = make({static_cast<int64_t>(bytes)}, at::kByte, false);
            *out = own.data_ptr();
            *have = bytes;
            return true;
        }
        const at::Tensor* t;
        if (!tensor(o, "workspace", &t)) return false;
        if (!t->is_cuda() || t->get_device() != dev || !t->is_contiguous())
            return refuse("workspace must be a contiguous tensor on cuda:" + std::to_string(dev));
        *out = t->data_ptr();
        *have = t->nbytes();
        return true;
    }

    // The caller's output, or a new one where it passed None: a new reference.
    bool output(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type, void** out, PyObject** ref) const {
        if (o == Py_None) {
            at::Tensor t = make(shape, type);
            *out = t.data_ptr();
            *ref = THPVariable_Wrap(std::move(t));
            return *ref != nullptr;
        }
        if (!arg(o, name, shape, type, out)) return false;
        Py_INCREF(o);
        *ref = o;
        return true;
    }
};

// References that a function drops when it fails.
struct Refs {
    PyObject* p[4] = {nullptr, nullptr, nullptr, nullptr};
    ~Refs() {
        for (PyObject* o : p) Py_XDECREF(o);
    }
    PyObject* take(int i) {
        PyObject* o = p[i];
        p[i] = nullptr;
        return o;
    }
};

bool get_int(PyObject* cfg, const char* name, int32_t* out) {
    PyObject* a = PyObject_GetAttrString(cfg, name);
    if (!a) return false;
    PyObject* n = PyLong_Check(a) ? a : PyNumber_Long(a);
    if (n != a) Py_DECREF(a);
    if (!n) return false;
    const long v = PyLong_AsLong(n);
    Py_DECREF(n);
    if (v == -1 && PyErr_Occurred()) return false;
    if (v < INT32_MIN || v > INT32_MAX) return refuse(std::string(name) + " does not fit 32 bits");
    *out = static_cast<int32_t>(v);
    return true;
}

bool get_config(PyObject* o, moe_config_t* c) {
    struct {
        const char* name;
        int32_t* to;
    } f[] = {{"num_tokens", &c->num_tokens}, {"hidden", &c->hidden}, {"inter", &c->inter}, {"num_experts", &c->num_experts},
             {"top_k", &c->top_k}, {"routing", &c->routing}, {"renormalize", &c->renormalize},
             {"group_count", &c->group_count}, {"k_group", &c->k_group}, {"group_select_mode", &c->group_select_mode},
             {"recipe", &c->recipe}, {"shared_experts", &c->shared_experts}};
    for (auto& e : f)
        if (!get_int(o, e.name, e.to)) return false;
    PyObject* a = PyObject_GetAttrString(o, "routed_scaling_factor");
    if (!a) return false;
    c->routed_scaling_factor = static_cast<float>(PyFloat_AsDouble(a));
    Py_DECREF(a);
    return !PyErr_Occurred();
}

bool get_linear_config(PyObject* o, moe_linear_config_t* c) {
    return get_int(o, "num_tokens", &c->num_tokens) && get_int(o, "in_features", &c->in_features) &&
           get_int(o, "out_features", &c->out_features) && get_int(o, "recipe", &c->recipe) &&
           get_int(o, "activation", &c->activation);
}

int64_t scale_rows(int64_t rows) { return (rows + 135) / 4 * 4; }

// A pair (codes [rows, cols], scale words [cols/128, scale_rows]), or None; held keeps the two.
bool quantized_args(const Call& c, PyObject* q, int64_t rows, int64_t cols, void** codes, void** scales, Refs& held) {
    *codes = *scales = nullptr;
    if (q == Py_None) return true;
    if (!PyTuple_Check(q) && !PyList_Check(q)) return refuse("quantized must be a pair (codes, scale words)");
    if (PySequence_Size(q) != 2) return refuse("quantized must be a pair (codes, scale words)");
    held.p[0] = PySequence_GetItem(q, 0);
    held.p[1] = PySequence_GetItem(q, 1);
    return held.p[0] && held.p[1] && c.arg(held.p[0], "codes", {rows, cols}, at::kByte, codes) &&
           c.arg(held.p[1], "scales", {cols / 128, scale_rows(rows)}, at::kInt, scales);
}

// The sequences' mask and offsets; n: how many sequences.
bool seq_args(const Call& c, PyObject* mask, PyObject* off, int64_t T, void** m, void** o, int32_t* n) {
    *n = 1;
    *o = *m = nullptr;
    if (off != Py_None) {
        const at::Tensor* t;
        if (!tensor(off, "seq_offsets", &t)) return false;
        if (t->numel() < 2) return refuse("seq_offsets must hold at least two offsets");
        *n = static_cast<int32_t>(t->numel() - 1);
        if (!c.arg(*t, "seq_offsets", {t->numel()}, at::kInt, o)) return false;
    }
    if (mask == Py_None) return true;
    const at::Tensor* t;
    if (!tensor(mask, "token_mask", &t)) return false;
    return c.arg(*t, "token_mask", {T}, t->scalar_type() == at::kBool ? at::kBool : at::kByte, m);
}

bool count_args(Py_ssize_t n, Py_ssize_t want, const char* who) {
    if (!g_error) {
        PyErr_SetString(PyExc_RuntimeError, "not initialised: call through the package");
        return false;
    }
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", who, want, n);
    return false;
}

#define LIB_CALL(rc, expr)            \
    Py_BEGIN_ALLOW_THREADS rc = expr; \
    Py_END_ALLOW_THREADS

PyObject* add_rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count_args(n, 11, "add_rms_norm")) return nullptr;
    PyObject *x = a[1], *res = a[4], *res_out = a[5], *quantized = a[7];
    moe_config_t cfg{};
    Call c;
    Refs out, held;
    if (!get_config(a[0], &cfg) || !c.begin(x, "x", a[10])) return nullptr;
    const double eps = PyFloat_AsDouble(a[3]);
    if (eps == -1.0 && PyErr_Occurred()) return nullptr;
    const int want_y = PyObject_IsTrue(a[8]), want_q = PyObject_IsTrue(a[9]);
    if (want_y < 0 || want_q < 0) return nullptr;
    const int64_t T = cfg.num_tokens, H = cfg.hidden;
    void *px, *pw, *pr, *pro = nullptr, *py = nullptr, *pq = nullptr, *ps = nullptr;
    at::ScalarType rt = at::kBFloat16;
    if (!c.arg(x, "x", {T, H}, at::kBFloat16, &px) || !c.arg(a[2], "norm_weight", {H}, at::kFloat, &pw)) return nullptr;
    if (res == Py_None) {
        if (res_out != Py_None) {
            refuse("residual_out needs a residual");
            return nullptr;
        }
        pr = nullptr;
        Py_INCREF(x);
        out.p[0] = x;
    } else {
        const at::Tensor* t;
        if (!tensor(res, "residual", &t)) return nullptr;
        rt = t->scalar_type();
        if (rt != at::kBFloat16 && rt != at::kFloat) {
            refuse(std::string("residual must be torch.bfloat16 or torch.float32, got ") + type_name(rt));
            return nullptr;
        }
        if (!c.arg(*t, "residual", {T, H}, rt, &pr) || !c.output(res_out, "residual_out", {T, H}, rt, &pro, &out.p[0]))
            return nullptr;
    }
    if (a[6] != Py_None || want_y) {
        if (!c.output(a[6], "y", {T, H}, at::kBFloat16, &py, &out.p[1])) return nullptr;
    }
    if (quantized != Py_None) {
        if (!quantized_args(c, quantized, T, H, &pq, &ps, held)) return nullptr;
        Py_INCREF(quantized);
        out.p[2] = quantized;
    } else if (want_q) {
        Refs q;
        if (!c.output(Py_None, "codes", {T, H}, at::kByte, &pq, &q.p[0]) ||
            !c.output(Py_None, "scales", {H / 128, scale_rows(T)}, at::kInt, &ps, &q.p[1]) ||
            !(out.p[2] = PyTuple_Pack(2, q.p[0], q.p[1])))
            return nullptr;
    }
    int rc;
    LIB_CALL(rc, g_lib.add_rms_norm(&cfg, px, pr, rt == at::kFloat, static_cast<const float*>(pw), static_cast<float>(eps),
                                    pro, py, pq, ps, c.stream));
    if (!check(rc)) return nullptr;
    return PyTuple_Pack(3, out.p[0], out.p[1] ? out.p[1] : Py_None, out.p[2] ? out.p[2] : Py_None);
    END_HANDLE_TH_ERRORS
}

PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count_args(n, 9, "linear")) return nullptr;
    PyObject *weights = a[1], *x = a[2], *quantized = a[3];
    if ((x == Py_None) == (quantized == Py_None)) {
        refuse("pass exactly one of x and quantized");
        return nullptr;
    }
    moe_linear_config_t cfg{};
    Call c;
    Refs out;
    at::Tensor own;
    if (!get_linear_config(a[0], &cfg)) return nullptr;
    PyObject* first = x;
    if (x == Py_None) {
        if (!PyTuple_Check(quantized) && !PyList_Check(quantized)) {
            refuse("quantized must be a pair (codes, scale words)");
            return nullptr;
        }
        first = PySequence_Size(quantized) ? PySequence_GetItem(quantized, 0) : nullptr;
        if (!first) {
            refuse("quantized must be a pair (codes, scale words)");
            return nullptr;
        }
        Py_DECREF(first);                               // the pair keeps it
    }
    if (!c.begin(first, "x", a[8])) return nullptr;
    const int64_t T = cfg.num_tokens, K = cfg.in_features, N = cfg.out_features;
    if ((!PyTuple_Check(weights) && !PyList_Check(weights)) || PySequence_Size(weights) != 2) {
        refuse("weights must be the pair (w_t, ws_t) of transform_linear_weights");
        return nullptr;
    }
    Refs w, held;
    w.p[0] = PySequence_GetItem(weights, 0);
    w.p[1] = PySequence_GetItem(weights, 1);
    void *px, *pq, *ps, *pw, *pws, *pb, *pr, *py, *pk;
    size_t have, need = MOE_LINEAR_STATUS_BYTES;
    if (!c.arg(x, "x", {T, K}, at::kBFloat16, &px) || !quantized_args(c, quantized, T, K, &pq, &ps, held) ||
        !c.arg(w.p[0], "w_t", {K * N / (cfg.recipe == 2 ? 2 : 1)}, at::kByte, &pw) ||
        !c.arg(w.p[1], "ws_t", {K / 128 * ((N + 255) / 256 * 256) * 4}, at::kByte, &pws) ||
        !c.arg(a[4], "bias", {N}, at::kBFloat16, &pb) || !c.arg(a[5], "residual", {T, N}, at::kBFloat16, &pr))
        return nullptr;
    if (x != Py_None && a[7] == Py_None && !check(g_lib.linear_workspace_size(&cfg, &need))) return nullptr;
    if (!c.output(a[6], "y", {T, N}, at::kBFloat16, &py, &out.p[0]) || !c.workspace(a[7], need, own, &pk, &have))
        return nullptr;
    int rc;
    LIB_CALL(rc, g_lib.linear(&cfg, px, pq, ps, pw, pws, pb, pr, py, pk, have, c.stream));
    if (!check(rc)) return nullptr;
    return out.take(0);
    END_HANDLE_TH_ERRORS
}

PyObject* balance_loss(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count_args(n, 8, "balance_loss")) return nullptr;
    moe_config_t cfg{};
    Call c;
    Refs out;
    at::Tensor own;
    if (!get_config(a[0], &cfg) || !c.begin(a[1], "router_logits", a[7])) return nullptr;
    const double coef = PyFloat_AsDouble(a[3]);
    if (coef == -1.0 && PyErr_Occurred()) return nullptr;
    const int64_t T = cfg.num_tokens, E = cfg.num_experts;
    void *pl, *pi, *pm, *po, *loss, *counts, *tokens, *mean, *pk;
    int32_t S;
    size_t have, need = 0;
    if (!c.arg(a[1], "router_logits", {T, E}, at::kFloat, &pl) ||
        !c.arg(a[2], "topk_idx", {T, cfg.top_k}, at::kInt, &pi) || !seq_args(c, a[5], a[4], T, &pm, &po, &S))
        return nullptr;
    if (a[6] == Py_None && !check(g_lib.balance_workspace_size(&cfg, S, &need))) return nullptr;
    if (!c.output(Py_None, "loss", {1}, at::kFloat, &loss, &out.p[0]) ||
        !c.output(Py_None, "expert_counts", {S, E}, at::kInt, &counts, &out.p[1]) ||
        !c.output(Py_None, "seq_tokens", {S + 1}, at::kInt, &tokens, &out.p[2]) ||
        !c.output(Py_None, "mean_probs", {S, E}, at::kFloat, &mean, &out.p[3]) || !c.workspace(a[6], need, own, &pk, &have))
        return nullptr;
    int rc;
    LIB_CALL(rc, g_lib.balance_loss(&cfg, static_cast<const float*>(pl), static_cast<const int32_t*>(pi),
                                    static_cast<const uint8_t*>(pm), static_cast<const int32_t*>(po), S,
                                    static_cast<float>(coef), static_cast<int32_t*>(counts), static_cast<int32_t*>(tokens),
                                    static_cast<float*>(mean), static_cast<float*>(loss), pk, have, c.stream));
    if (!check(rc)) return nullptr;
    return PyTuple_Pack(4, out.p[0], out.p[1], out.p[2], out.p[3]);
    END_HANDLE_TH_ERRORS
}

PyObject* route_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count_args(n, 14, "route_backward")) return nullptr;
    moe_config_t cfg{};
    Call c;
    Refs out;
    at::Tensor own;
    if (!get_config(a[0], &cfg) || !c.begin(a[1], "router_logits", a[13])) return nullptr;
    const double coef = PyFloat_AsDouble(a[6]);
    if (coef == -1.0 && PyErr_Occurred()) return nullptr;
    const int64_t T = cfg.num_tokens, E = cfg.num_experts, k = cfg.top_k;
    void *pl, *pi, *pdw, *pes, *pdl, *pc, *pt, *pm, *po, *dl, *dpes = nullptr, *pk = nullptr;
    int32_t S;
    size_t have = 0, need = 0;
    if (!c.arg(a[1], "router_logits", {T, E}, at::kFloat, &pl) || !c.arg(a[2], "topk_idx", {T, k}, at::kInt, &pi) ||
        !c.arg(a[3], "d_topk_weights", {T, k}, at::kFloat, &pdw) || !c.arg(a[4], "per_expert_scale", {E}, at::kFloat, &pes) ||
        !c.arg(a[5], "d_loss", {1}, at::kFloat, &pdl) || !seq_args(c, a[10], a[9], T, &pm, &po, &S) ||
        !c.arg(a[7], "expert_counts", {S, E}, at::kInt, &pc) || !c.arg(a[8], "seq_tokens", {S + 1}, at::kInt, &pt) ||
        !c.output(a[11], "d_logits", {T, E}, at::kFloat, &dl, &out.p[0]))
        return nullptr;
    if (pes) {
        if (a[12] == Py_None && !check(g_lib.balance_workspace_size(&cfg, S, &need))) return nullptr;
        if (!c.output(Py_None, "d_per_expert_scale", {E}, at::kFloat, &dpes, &out.p[1]) ||
            !c.workspace(a[12], need, own, &pk, &have))
            return nullptr;
    }
    int rc;
    LIB_CALL(rc, g_lib.route_backward(&cfg, static_cast<const float*>(pl), static_cast<const float*>(pes),
                                      static_cast<const int32_t*>(pi), static_cast<const float*>(pdw),
                                      static_cast<const float*>(pdl), static_cast<float>(coef),
                                      static_cast<const int32_t*>(pc), static_cast<const int32_t*>(pt),
                                      static_cast<const uint8_t*>(pm), static_cast<const int32_t*>(po), S,
                                      static_cast<float*>(dl), static_cast<float*>(dpes), pk, have, c.stream));
    if (!check(rc)) return nullptr;
    return PyTuple_Pack(2, out.p[0], out.p[1] ? out.p[1] : Py_None);
    END_HANDLE_TH_ERRORS
}

// init(MoeError, addresses of the entry points in Lib's order)
PyObject* init(PyObject*, PyObject* args) {
    unsigned long long p[7];
    PyObject* e;
    if (!PyArg_ParseTuple(args, "OKKKKKKK", &e, &p[0], &p[1], &p[2], &p[3], &p[4], &p[5], &p[6])) return nullptr;
    Py_INCREF(e);
    Py_XDECREF(g_error);
    g_error = e;
    g_lib = {reinterpret_cast<decltype(g_lib.last_error)>(p[0]),
             reinterpret_cast<decltype(g_lib.add_rms_norm)>(p[1]),
             reinterpret_cast<decltype(g_lib.linear)>(p[2]),
             reinterpret_cast<decltype(g_lib.linear_workspace_size)>(p[3]),
             reinterpret_cast<decltype(g_lib.balance_loss)>(p[4]),
             reinterpret_cast<decltype(g_lib.balance_workspace_size)>(p[5]),
             reinterpret_cast<decltype(g_lib.route_backward)>(p[6])};
    Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"init", init, METH_VARARGS, nullptr},
    {"add_rms_norm", reinterpret_cast<PyCFunction>(add_rms_norm), METH_FASTCALL, nullptr},
    {"linear", reinterpret_cast<PyCFunction>(linear), METH_FASTCALL, nullptr},
    {"balance_loss", reinterpret_cast<PyCFunction>(balance_loss), METH_FASTCALL, nullptr},
    {"route_backward", reinterpret_cast<PyCFunction>(route_backward), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&kModule); }
