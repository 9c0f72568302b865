// marshal.cpp -- Python module _marshal: the arguments of the gate, the few-token
// experts, the adapter projection, the grouped products, the activation and the norm, from
// tensors to the C entry points.
//
// Small ones take 2 to 20 us of the GPU's time. In Python, checks of a dozen
// tensors, two or three outputs to allocate and up to 25 arguments to convert made
// them 12 (a gate) to 21 us of the host's; from here they are 5 to 11, launches
// included. Each function takes an entry point's address
// first, so that another build of the library can be called, and returns its
// status and the outputs.
#include <climits>
#include <initializer_list>
#include <string>

#include <ATen/Context.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/impl/LocalDispatchKeySet.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "moe_get.h"

namespace {

using at::Tensor;
using Shape = std::initializer_list<int64_t>;

[[noreturn]] void refuse(PyObject *type, const std::string &what) {
    PyErr_SetString(type, what.c_str());
    throw python_error();
}

std::string text(at::IntArrayRef shape) {
    std::string s = "(";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    return s + (shape.size() == 1 ? ",)" : ")");
}
std::string text(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return "torch.float32";
        case at::kBFloat16: return "torch.bfloat16";
        case at::kLong: return "torch.int64";
        case at::kInt: return "torch.int32";
        case at::kByte: return "torch.uint8";
        default: return c10::toString(t);
    }
}

// The entry points take sizes as int.
void check_sizes(std::initializer_list<int64_t> sizes) {
    for (int64_t n : sizes)
        if (n > INT_MAX) refuse(PyExc_ValueError, "a size of " + std::to_string(n) + " does not fit in 32 bits");
}

// A call's positional arguments, taken in order; the stream is the last.
class Args {
  public:
    Args(PyObject *const *args, Py_ssize_t n, Py_ssize_t want) : at_(args) {
        if (n != want) refuse(PyExc_TypeError, "wrong number of arguments");
        if (args[n - 1] == Py_None) return;
        given_ = PyLong_AsVoidPtr(args[n - 1]);
        if (given_ == nullptr && PyErr_Occurred()) throw python_error();
        stream_given_ = true;
    }
    template <class F>
    F *entry() {
        void *p = PyLong_AsVoidPtr(*at_++);
        if (p == nullptr) throw python_error();
        return reinterpret_cast<F *>(p);
    }
    int integer(const char *name) {
        const long long v = PyLong_AsLongLong(*at_++);
        if (v == -1 && PyErr_Occurred()) throw python_error();
        if (v < INT_MIN || v > INT_MAX)
            refuse(PyExc_OverflowError, std::string(name) + " is " + std::to_string(v) + ", which does not fit in 32 bits");
        return (int)v;
    }
    float real() {
        const double v = PyFloat_AsDouble(*at_++);
        if (v == -1.0 && PyErr_Occurred()) throw python_error();
        return (float)v;
    }
    // the handle, or None for the current stream; the call goes to the current device
    void *stream() const {
        const int current = c10::cuda::current_device();
        if (device_ != current)
            refuse(PyExc_ValueError, "tensors on cuda:" + std::to_string(device_) + ", the current device is cuda:" +
                                         std::to_string(current));
        return stream_given_ ? given_ : (void *)c10::cuda::getCurrentCUDAStream(current).stream();
    }
    const Tensor &tensor(const char *name, int64_t dims = -1) {
        PyObject *o = *at_++;
        if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " is not a tensor");
        const Tensor &t = THPVariable_Unpack(o);
        if (dims >= 0 && t.dim() != dims)
            refuse(PyExc_ValueError, std::string(name) + " has " + std::to_string(dims) + " dimensions, not " +
                                         std::to_string(t.dim()));
        if (!t.is_cuda()) refuse(PyExc_ValueError, "libmoe_get takes CUDA tensors only");
        if (!t.is_contiguous()) refuse(PyExc_ValueError, "libmoe_get takes contiguous tensors only");
        if (device_ < 0) device_ = t.device().index();
        if (t.device().index() != device_)
            refuse(PyExc_ValueError, std::string(name) + " is on " + t.device().str() + ", other tensors on cuda:" +
                                         std::to_string(device_));
        return t;
    }
    const Tensor &tensor(const char *name, at::ScalarType type, Shape shape) {
        PyObject *o = *at_;
        if (THPVariable_Check(o)) {
            const Tensor &t = THPVariable_Unpack(o);
            if (t.scalar_type() != type || t.sizes() != at::IntArrayRef(shape))
                refuse(PyExc_ValueError, std::string(name) + " is " + text(type) + " " + text(at::IntArrayRef(shape)) +
                                             ", not " + text(t.scalar_type()) + " " + text(t.sizes()));
        }
        return tensor(name);
    }
    // the word that kernels report to
    int32_t *status() {
        const Tensor &t = tensor("status");
        if (t.scalar_type() != at::kInt || t.numel() < 1)
            refuse(PyExc_ValueError, "status is torch.int32 of one element, not " + text(t.scalar_type()) + " " +
                                         text(t.sizes()));
        return static_cast<int32_t *>(t.data_ptr());
    }
    // null for None
    void *pointer_or_null(const char *name, at::ScalarType type, Shape shape) {
        if (*at_ == Py_None) return ++at_, nullptr;
        return tensor(name, type, shape).data_ptr();
    }
    // an output: allocated for None, under the stream that writes it, as torch.empty does. By the allocator's own entry,
    // which takes 0.6 us less, where nobody can tell: not with deterministic algorithms, which fill what is allocated, nor
    // where more than the ordinary keys are on (dispatch modes, tracing, function transforms).
    Tensor output(const char *name, at::ScalarType type, Shape shape, const Tensor &like) {
        if (*at_ != Py_None) return tensor(name, type, shape);
        ++at_;
        c10::cuda::OptionalCUDAStreamGuard under;
        if (stream_given_)
            under.reset_stream(c10::cuda::getStreamFromExternal((cudaStream_t)given_, like.device().index()));
        if (at::globalContext().deterministicAlgorithms() ||
            !(c10::impl::tls_local_dispatch_key_set().included_ - c10::default_included_set).empty())
            return at::empty(at::IntArrayRef(shape), at::TensorOptions().dtype(type).device(like.device()));
        return at::Tensor(at::detail::empty_cuda(at::IntArrayRef(shape), type, like.device(), std::nullopt));
    }
    // an output that is left out: an undefined tensor, None in Python
    Tensor optional_output(bool wanted, const char *name, at::ScalarType type, Shape shape, const Tensor &like) {
        if (wanted) return output(name, type, shape, like);
        if (*at_ != Py_None) refuse(PyExc_ValueError, std::string(name) + " is not written by this call");
        ++at_;
        return Tensor();
    }
    bool flag() { return integer("flag") != 0; }
    bool none() const { return *at_ == Py_None; }

  private:
    PyObject *const *at_;
    void *given_ = nullptr;
    bool stream_given_ = false;
    int device_ = -1;   // of the tensors so far
};

void *data_or_null(const Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

// {status, outputs...}
PyObject *result(int code, std::initializer_list<const Tensor *> outputs) {
    PyObject *tuple = PyTuple_New(1 + (Py_ssize_t)outputs.size());
    if (tuple == nullptr) throw python_error();
    PyTuple_SET_ITEM(tuple, 0, PyLong_FromLong(code));
    Py_ssize_t i = 1;
    for (const Tensor *t : outputs) PyTuple_SET_ITEM(tuple, i++, THPVariable_Wrap(*t));
    return tuple;
}

// The call itself, which may wait for room in a stream, without the interpreter's lock.
template <class F>
int unlocked(F call) {
    int code;
    Py_BEGIN_ALLOW_THREADS
    code = call();
    Py_END_ALLOW_THREADS
    return code;
}

int logits_type(const Tensor &logits) {
    if (logits.scalar_type() == at::kFloat) return MOE_LOGITS_F32;
    if (logits.scalar_type() != at::kBFloat16) refuse(PyExc_ValueError, "the router's logits are float32 or bfloat16");
    return MOE_LOGITS_BF16;
}

// (entry, logits, num_topk, bias, mode, scale, topk_idx, topk_weights, status, stream)
PyObject *topk_gate(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Args a(args, n, 10);
    auto *entry = a.entry<decltype(moe_topk_gate)>();
    const Tensor &logits = a.tensor("logits", 2);
    const int64_t T = logits.size(0), E = logits.size(1);
    check_sizes({T, E});
    const int type = logits_type(logits), k = a.integer("num_topk");
    const void *bias = a.pointer_or_null("bias", at::kFloat, {E});
    const int mode = a.integer("mode");
    const float scale = a.real();
    const Tensor idx = a.output("topk_idx", at::kLong, {T, k}, logits);
    const Tensor weights = a.output("topk_weights", at::kFloat, {T, k}, logits);
    int32_t *const status = a.status();
    void *const stream = a.stream();
    const int code = unlocked([&] {
        return entry(logits.data_ptr(), type, (const float *)bias, (int)T, k, (int)E, mode, scale,
                     (int64_t *)idx.data_ptr(), (float *)weights.data_ptr(), status, stream);
    });
    return result(code, {&idx, &weights});
    END_HANDLE_TH_ERRORS
}

// (entry, logits, topk_idx, grad_weights, mode, scale, out, status, stream)
PyObject *topk_gate_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Args a(args, n, 9);
    auto *entry = a.entry<decltype(moe_topk_gate_backward)>();
    const Tensor &logits = a.tensor("logits", 2);
    const int64_t T = logits.size(0), E = logits.size(1);
    const int type = logits_type(logits);
    const Tensor &idx = a.tensor("topk_idx", 2);
    const int64_t k = idx.size(1);
    check_sizes({T, E, k});
    if (idx.scalar_type() != at::kLong || idx.size(0) != T)
        refuse(PyExc_ValueError, "topk_idx is torch.int64 " + text(at::IntArrayRef{T, k}) + ", not " +
                                     text(idx.scalar_type()) + " " + text(idx.sizes()));
    const Tensor &grad = a.tensor("grad_weights", at::kFloat, {T, k});
    const int mode = a.integer("mode");
    const float scale = a.real();
    const Tensor out = a.output("out", logits.scalar_type(), {T, E}, logits);
    int32_t *const status = a.status();
    void *const stream = a.stream();
    const int code = unlocked([&] {
        return entry(logits.data_ptr(), type, (const int64_t *)idx.data_ptr(), (const float *)grad.data_ptr(), (int)T,
                     (int)k, (int)E, mode, scale, out.data_ptr(), status, stream);
    });
    return result(code, {&out});
    END_HANDLE_TH_ERRORS
}

// A layer's experts: (w13, w2, w13_scales, w2_scales) for rows of `hidden` channels.
struct Experts {
    const void *w13, *w2;
    const float *w13_scales = nullptr, *w2_scales = nullptr;
    int64_t E, I;
    int type;
    Experts(Args &a, int64_t H) {
        const Tensor &up = a.tensor("w13", 3), &down = a.tensor("w2", 3);
        const bool e4m3 = up.scalar_type() == at::kByte;
        const at::ScalarType dtype = e4m3 ? at::kByte : at::kBFloat16;
        E = down.size(0), I = down.size(2);
        check_sizes({E, I});
        auto check = [&](const Tensor &t, const char *name, Shape shape) {
            if (t.scalar_type() != dtype || t.sizes() != at::IntArrayRef(shape))
                refuse(PyExc_ValueError, std::string(name) + " is " + text(dtype) + " " + text(at::IntArrayRef(shape)) +
                                             ", not " + text(t.scalar_type()) + " " + text(t.sizes()));
        };
        check(up, "w13", {E, 2 * I, H});
        check(down, "w2", {E, H, I});
        w13 = up.data_ptr(), w2 = down.data_ptr();
        type = e4m3 ? MOE_WEIGHTS_E4M3 : MOE_WEIGHTS_BF16;
        auto scales = [&](const char *name, Shape shape) {
            if (a.none() == e4m3)
                refuse(PyExc_ValueError, e4m3 ? "E4M3 weights need w13_scales and w2_scales" : "bf16 weights take no scales");
            return (const float *)a.pointer_or_null(name, at::kFloat, shape);
        };
        w13_scales = scales("w13_scales", {E, 2 * I, H / 128});
        w2_scales = scales("w2_scales", {E, H, I / 128});
    }
};

// (entry, x, w13, w2, w13_scales, w2_scales, topk_idx, topk_weights, out, workspace, status, stream)
PyObject *experts(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Args a(args, n, 12);
    auto *entry = a.entry<decltype(moe_experts)>();
    const Tensor &x = a.tensor("x", 2);
    const int64_t T = x.size(0), H = x.size(1);
    if (x.scalar_type() != at::kBFloat16)
        refuse(PyExc_ValueError, "x is torch.bfloat16, not " + text(x.scalar_type()));
    const Experts w(a, H);
    const Tensor &idx = a.tensor("topk_idx", 2);
    const int64_t k = idx.size(1);
    check_sizes({T, H, k});
    if (idx.scalar_type() != at::kLong || idx.size(0) != T)
        refuse(PyExc_ValueError, "topk_idx is torch.int64 " + text(at::IntArrayRef{T, k}) + ", not " +
                                     text(idx.scalar_type()) + " " + text(idx.sizes()));
    const Tensor &weights = a.tensor("topk_weights", at::kFloat, {T, k});
    const Tensor out = a.output("out", at::kBFloat16, {T, H}, x);
    const Tensor &workspace = a.tensor("workspace");
    int32_t *const status = a.status();
    void *const stream = a.stream();
    const int code = unlocked([&] {
        return entry(x.data_ptr(), (int)T, (int)H, (const int64_t *)idx.data_ptr(), (const float *)weights.data_ptr(),
                     (int)k, (int)w.E, w.w13, w.w13_scales, w.w2, w.w2_scales, (int)w.I, w.type, out.data_ptr(),
                     workspace.data_ptr(), workspace.nbytes(), status, stream);
    });
    return result(code, {&out});
    END_HANDLE_TH_ERRORS
}

// (entry, x, w13, w2, w13_scales, w2_scales, logits, num_topk, bias, mode, scale, topk_idx, topk_weights, out, workspace,
//  status, stream)
PyObject *layer(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Args a(args, n, 17);
    auto *entry = a.entry<decltype(moe_layer)>();
    const Tensor &x = a.tensor("x", 2);
    const int64_t T = x.size(0), H = x.size(1);
    check_sizes({T, H});
    if (x.scalar_type() != at::kBFloat16)
        refuse(PyExc_ValueError, "x is torch.bfloat16, not " + text(x.scalar_type()));
    const Experts w(a, H);
    const Tensor &logits = a.tensor("logits", 2);
    if (logits.size(0) != T || logits.size(1) != w.E)
        refuse(PyExc_ValueError, "logits are " + text(at::IntArrayRef{T, w.E}) + ", not " + text(logits.sizes()));
    const int type = logits_type(logits), k = a.integer("num_topk");
    const void *bias = a.pointer_or_null("bias", at::kFloat, {w.E});
    const int mode = a.integer("mode");
    const float scale = a.real();
    const Tensor idx = a.output("topk_idx", at::kLong, {T, k}, x);
    const Tensor weights = a.output("topk_weights", at::kFloat, {T, k}, x);
    const Tensor out = a.output("out", at::kBFloat16, {T, H}, x);
    const Tensor &workspace = a.tensor("workspace");
    int32_t *const status = a.status();
    void *const stream = a.stream();
    const int code = unlocked([&] {
        return entry(x.data_ptr(), (int)T, (int)H, logits.data_ptr(), type, (const float *)bias, k, (int)w.E, mode, scale,
                     (int64_t *)idx.data_ptr(), (float *)weights.data_ptr(), w.w13, w.w13_scales, w.w2, w.w2_scales,
                     (int)w.I, w.type, out.data_ptr(), workspace.data_ptr(), workspace.nbytes(),
                     status, stream);
    });
    return result(code, {&out, &idx, &weights});
    END_HANDLE_TH_ERRORS
}

// (entry, x, w, adapter_idx, a, b, scales, out, workspace, status, stream)
PyObject *adapter_linear(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Args a(args, n, 11);
    auto *entry = a.entry<decltype(moe_adapter_linear)>();
    const Tensor &x = a.tensor("x", 2), &w = a.tensor("w", 2);
    const int64_t T = x.size(0), K = x.size(1), N = w.size(0);
    if (x.scalar_type() != at::kBFloat16 || w.scalar_type() != at::kBFloat16 || w.size(1) != K)
        refuse(PyExc_ValueError, "x and w are torch.bfloat16 [T, K] and [N, K], not " + text(x.scalar_type()) + " " +
                                     text(x.sizes()) + " and " + text(w.scalar_type()) + " " + text(w.sizes()));
    const Tensor &idx = a.tensor("adapter_idx", at::kInt, {T});
    const Tensor &down = a.tensor("a", 3);
    const int64_t L = down.size(0), r = down.size(1);
    check_sizes({T, K, N, L, r});
    if (down.scalar_type() != at::kBFloat16 || down.size(2) != K)
        refuse(PyExc_ValueError, "a is torch.bfloat16 " + text(at::IntArrayRef{L, r, K}) + ", not " +
                                     text(down.scalar_type()) + " " + text(down.sizes()));
    const Tensor &up = a.tensor("b", at::kBFloat16, {L, N, r}), &scales = a.tensor("scales", at::kFloat, {L});
    const Tensor out = a.output("out", at::kBFloat16, {T, N}, x);
    const Tensor &workspace = a.tensor("workspace");
    int32_t *const status = a.status();
    void *const stream = a.stream();
    const int code = unlocked([&] {
        return entry(x.data_ptr(), (int)T, (int)K, w.data_ptr(), (int)N, (const int32_t *)idx.data_ptr(), down.data_ptr(),
                     up.data_ptr(), (const float *)scales.data_ptr(), (int)L, (int)r, out.data_ptr(),
                     workspace.data_ptr(), workspace.nbytes(), status, stream);
    });
    return result(code, {&out});
    END_HANDLE_TH_ERRORS
}

// Rows [M, columns] of a grouped product or its gradient, bf16 unless `codes`.
const Tensor &rows_of(Args &a, const char *name, bool codes_too) {
    const Tensor &t = a.tensor(name, 2);
    if (t.scalar_type() != at::kBFloat16 && !(codes_too && t.scalar_type() == at::kByte))
        refuse(PyExc_ValueError, std::string(name) + (codes_too ? " is torch.bfloat16 or torch.uint8, not " : " is torch.bfloat16, not ") +
                                     text(t.scalar_type()));
    return t;
}

// (entry, x, w, expert_prefix, x_scales, w_scales, out, status, stream)
PyObject *grouped_linear(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Args a(args, n, 9);
    auto *entry = a.entry<decltype(moe_grouped_linear)>();
    const Tensor &x = rows_of(a, "x", true), &w = a.tensor("w", 3);
    const int64_t M = x.size(0), K = x.size(1), E = w.size(0), N = w.size(1);
    check_sizes({M, K, E, N});
    const bool e4m3 = x.scalar_type() == at::kByte;
    if (w.scalar_type() != x.scalar_type() || w.size(2) != K)
        refuse(PyExc_ValueError, "w is " + text(x.scalar_type()) + " " + text(at::IntArrayRef{E, N, K}) + ", not " +
                                     text(w.scalar_type()) + " " + text(w.sizes()));
    const Tensor &prefix = a.tensor("expert_prefix", at::kInt, {E + 1});
    auto scales = [&](const char *name, Shape shape) {
        if (a.none() == e4m3)
            refuse(PyExc_ValueError, e4m3 ? "E4M3 codes need x_scales and w_scales" : "bf16 rows and weights take no scales");
        return (const float *)a.pointer_or_null(name, at::kFloat, shape);
    };
    const float *x_scales = scales("x_scales", {M, K / 128});
    const float *w_scales = scales("w_scales", {E, N, K / 128});
    const Tensor out = a.output("out", at::kBFloat16, {M, N}, x);
    int32_t *const status = a.status();
    void *const stream = a.stream();
    const int code = unlocked([&] {
        return entry(x.data_ptr(), x_scales, (int)M, (int)K, w.data_ptr(), w_scales, (int)E, (int)N,
                     (const int32_t *)prefix.data_ptr(), e4m3 ? MOE_WEIGHTS_E4M3 : MOE_WEIGHTS_BF16, out.data_ptr(), status,
                     stream);
    });
    return result(code, {&out});
    END_HANDLE_TH_ERRORS
}

// (entry, grad, w, expert_prefix, out, status, stream)
PyObject *grouped_linear_grad_x(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Args a(args, n, 7);
    auto *entry = a.entry<decltype(moe_grouped_linear_grad_x)>();
    const Tensor &grad = rows_of(a, "grad", false), &w = a.tensor("w", 3);
    const int64_t M = grad.size(0), N = grad.size(1), E = w.size(0), K = w.size(2);
    check_sizes({M, K, E, N});
    if (w.scalar_type() != at::kBFloat16 || w.size(1) != N)
        refuse(PyExc_ValueError, "w is torch.bfloat16 " + text(at::IntArrayRef{E, N, K}) + ", not " + text(w.scalar_type()) +
                                     " " + text(w.sizes()));
    const Tensor &prefix = a.tensor("expert_prefix", at::kInt, {E + 1});
    const Tensor out = a.output("out", at::kBFloat16, {M, K}, grad);
    int32_t *const status = a.status();
    void *const stream = a.stream();
    const int code = unlocked([&] {
        return entry(grad.data_ptr(), (int)M, (int)N, w.data_ptr(), (int)E, (int)K, (const int32_t *)prefix.data_ptr(),
                     out.data_ptr(), status, stream);
    });
    return result(code, {&out});
    END_HANDLE_TH_ERRORS
}

// (entry, grad, x, expert_prefix, bf16, accumulate, out, status, stream)
PyObject *grouped_linear_grad_w(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Args a(args, n, 9);
    auto *entry = a.entry<decltype(moe_grouped_linear_grad_w)>();
    const Tensor &grad = rows_of(a, "grad", false), &x = rows_of(a, "x", false);
    const int64_t M = grad.size(0), N = grad.size(1), K = x.size(1);
    if (x.size(0) != M)
        refuse(PyExc_ValueError, "x is torch.bfloat16 " + text(at::IntArrayRef{M, K}) + ", not " + text(x.sizes()));
    const Tensor &prefix = a.tensor("expert_prefix", 1);
    const int64_t E = prefix.size(0) - 1;
    check_sizes({M, K, E, N});
    if (prefix.scalar_type() != at::kInt || E < 1)
        refuse(PyExc_ValueError, "expert_prefix is torch.int32 of at least two elements, not " + text(prefix.scalar_type()) +
                                     " " + text(prefix.sizes()));
    const bool bf16 = a.flag(), accumulate = a.flag();
    const Tensor out = a.output("out", bf16 ? at::kBFloat16 : at::kFloat, {E, N, K}, x);
    int32_t *const status = a.status();
    void *const stream = a.stream();
    const int code = unlocked([&] {
        return entry(grad.data_ptr(), x.data_ptr(), (int)M, (int)N, (int)K, (int)E, (const int32_t *)prefix.data_ptr(),
                     bf16 ? MOE_GRAD_BF16 : MOE_GRAD_F32, accumulate, out.data_ptr(), status, stream);
    });
    return result(code, {&out});
    END_HANDLE_TH_ERRORS
}

// gate_up [M, 2 I]
const Tensor &gate_up_of(Args &a) {
    const Tensor &t = rows_of(a, "gate_up", false);
    if (t.size(1) % 2 != 0) refuse(PyExc_ValueError, "gate_up has an odd number of columns");
    return t;
}

// (entry, gate_up, row_weights, num_rows, quantize, out, out_scales, status, stream)
PyObject *swiglu(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Args a(args, n, 9);
    auto *entry = a.entry<decltype(moe_swiglu)>();
    const Tensor &gate_up = gate_up_of(a);
    const int64_t M = gate_up.size(0), I = gate_up.size(1) / 2;
    check_sizes({M, I});
    const void *weights = a.pointer_or_null("row_weights", at::kFloat, {M});
    const void *rows = a.pointer_or_null("num_rows", at::kInt, {1});
    const bool codes = a.flag();
    if (codes && I % 128 != 0) refuse(PyExc_ValueError, "E4M3 codes need a multiple of 128 channels, not " + std::to_string(I));
    const Tensor out = a.output("out", codes ? at::kByte : at::kBFloat16, {M, I}, gate_up);
    const Tensor scales = a.optional_output(codes, "out_scales", at::kFloat, {M, I / 128}, gate_up);
    int32_t *const status = a.status();
    void *const stream = a.stream();
    const int code = unlocked([&] {
        return codes && M == 0 ? (int)MOE_OK   // scales without an element have no address
                               : entry(gate_up.data_ptr(), (int)M, (int)I, (const float *)weights, (const int32_t *)rows,
                                       out.data_ptr(), (float *)data_or_null(scales), status, stream);
    });
    return result(code, {&out, &scales});
    END_HANDLE_TH_ERRORS
}

// (entry, gate_up, grad, row_weights, num_rows, weights_too, out, grad_row_weights, status, stream)
PyObject *swiglu_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Args a(args, n, 10);
    auto *entry = a.entry<decltype(moe_swiglu_backward)>();
    const Tensor &gate_up = gate_up_of(a);
    const int64_t M = gate_up.size(0), I = gate_up.size(1) / 2;
    check_sizes({M, I});
    const Tensor &grad = a.tensor("grad", at::kBFloat16, {M, I});
    const void *weights = a.pointer_or_null("row_weights", at::kFloat, {M});
    const void *rows = a.pointer_or_null("num_rows", at::kInt, {1});
    const bool too = a.flag();
    const Tensor out = a.output("out", at::kBFloat16, {M, 2 * I}, gate_up);
    const Tensor grad_weights = a.optional_output(too, "grad_row_weights", at::kFloat, {M}, gate_up);
    int32_t *const status = a.status();
    void *const stream = a.stream();
    const int code = unlocked([&] {
        return entry(gate_up.data_ptr(), grad.data_ptr(), (int)M, (int)I, (const float *)weights, (const int32_t *)rows,
                     out.data_ptr(), (float *)data_or_null(grad_weights), status, stream);
    });
    return result(code, {&out, &grad_weights});
    END_HANDLE_TH_ERRORS
}

// weight [H], bf16 or fp32
const Tensor &norm_weight(Args &a, int64_t H, int &type) {
    const Tensor &w = a.tensor("weight", 1);
    if ((w.scalar_type() != at::kBFloat16 && w.scalar_type() != at::kFloat) || w.size(0) != H)
        refuse(PyExc_ValueError, "weight is torch.bfloat16 or torch.float32 " + text(at::IntArrayRef{H}) + ", not " +
                                     text(w.scalar_type()) + " " + text(w.sizes()));
    type = w.scalar_type() == at::kFloat ? MOE_NORM_WEIGHT_F32 : MOE_NORM_WEIGHT_BF16;
    return w;
}

// (entry, x, residual, weight, eps, bf16_out, quantize, out, residual_out, codes, scales, status, stream)
PyObject *add_rms_norm(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Args a(args, n, 13);
    auto *entry = a.entry<decltype(moe_add_rms_norm)>();
    const Tensor &x = rows_of(a, "x", false);
    const int64_t T = x.size(0), H = x.size(1);
    check_sizes({T, H});
    const bool add = !a.none();
    const void *residual = a.pointer_or_null("residual", at::kBFloat16, {T, H});
    int type;
    const Tensor &weight = norm_weight(a, H, type);
    const float eps = a.real();
    const bool wide = a.flag(), quantize = a.flag();
    if (quantize && H % 128 != 0) refuse(PyExc_ValueError, "E4M3 codes need a multiple of 128 channels, not " + std::to_string(H));
    const Tensor out = a.optional_output(wide, "out", at::kBFloat16, {T, H}, x);
    const Tensor residual_out = a.optional_output(add, "residual_out", at::kBFloat16, {T, H}, x);
    const Tensor codes = a.optional_output(quantize, "codes", at::kByte, {T, H}, x);
    const Tensor scales = a.optional_output(quantize, "scales", at::kFloat, {T, H / 128}, x);
    int32_t *const status = a.status();
    void *const stream = a.stream();
    const int code = unlocked([&] {
        return entry(x.data_ptr(), residual, (int)T, (int)H, weight.data_ptr(), type, eps, data_or_null(out),
                     data_or_null(residual_out), data_or_null(codes), (float *)data_or_null(scales), status, stream);
    });
    return result(code, {&out, &residual_out, &codes, &scales});
    END_HANDLE_TH_ERRORS
}

// (entry, h, weight, grad, grad_residual, eps, out, grad_weight, workspace, status, stream)
PyObject *add_rms_norm_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Args a(args, n, 11);
    auto *entry = a.entry<decltype(moe_add_rms_norm_backward)>();
    const Tensor &h = rows_of(a, "h", false);
    const int64_t T = h.size(0), H = h.size(1);
    check_sizes({T, H});
    int type;
    const Tensor &weight = norm_weight(a, H, type);
    const Tensor &grad = a.tensor("grad", at::kBFloat16, {T, H});
    const void *grad_residual = a.pointer_or_null("grad_residual", at::kBFloat16, {T, H});
    const float eps = a.real();
    const Tensor out = a.output("out", at::kBFloat16, {T, H}, h);
    const Tensor grad_weight = a.output("grad_weight", at::kFloat, {H}, h);
    const Tensor &workspace = a.tensor("workspace");
    int32_t *const status = a.status();
    void *const stream = a.stream();
    const int code = unlocked([&] {
        return entry(h.data_ptr(), weight.data_ptr(), type, grad.data_ptr(), grad_residual, (int)T, (int)H, eps,
                     out.data_ptr(), (float *)grad_weight.data_ptr(), workspace.data_ptr(), workspace.nbytes(), status,
                     stream);
    });
    return result(code, {&out, &grad_weight});
    END_HANDLE_TH_ERRORS
}

#define MARSHAL_METHOD(f) {#f, (PyCFunction)(void (*)())f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {MARSHAL_METHOD(topk_gate), MARSHAL_METHOD(topk_gate_backward), MARSHAL_METHOD(experts),
                         MARSHAL_METHOD(layer), MARSHAL_METHOD(adapter_linear),
                         MARSHAL_METHOD(grouped_linear), MARSHAL_METHOD(grouped_linear_grad_x),
                         MARSHAL_METHOD(grouped_linear_grad_w), MARSHAL_METHOD(swiglu), MARSHAL_METHOD(swiglu_backward),
                         MARSHAL_METHOD(add_rms_norm), MARSHAL_METHOD(add_rms_norm_backward), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
