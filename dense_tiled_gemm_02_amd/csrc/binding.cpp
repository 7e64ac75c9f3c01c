// Native side of the torch calls that grouped.py, w4.py, i8.py, norm.py and
// router.py have already checked once: from the arguments' types, shapes, strides
// and devices to the plan and the launch, without Python in between.  A
// decode-sized product is bound by its host time: 4.1 to 4.9 us here, 3.4 of them
// the library's call, against 7.4 where the call is checked (out given) and passed
// on by ctypes.
//
//   remember(kind, owner, plan, run, workspace, sizes, dtype, extra, tensors)
//       a call that passed the checks: its gemm_*_run address, plan handle (kept
//       alive by `owner`), workspace bytes, output sizes and type.  `extra`: the
//       call's other arguments (an int, a float, a dtype, None, or a tuple of these).
//       The row operators (norm, int8 rows, routing) have no plan: that the checks
//       were passed is all there is to remember.
//   call(kind, extra, *tensors)
//       the outputs; None for a call not remembered (or on a device that is not
//       the current one): the caller then takes the checked path; a non-zero
//       gemm_status as an int if the library refused.
//   forget()
//   norm(x, weight, residual, eps), norm_i8(...), i8_rows(X), route(logits, bias, parameters)
//       these operators on arguments that have been checked, with their gradients
//       (one Function each, which records itself where a gradient is needed)
//   functions(addresses)
//       where the library's entry points are, in the order of `Library`
//
// Only plain torch.Tensor and Parameter objects on a GPU are looked up.  The
// interpreter's lock guards the table; it is released for the allocations and
// the launch, which waits while the GPU's queue is full.
#include <Python.h>
#include <ATen/ATen.h>
#include <c10/core/AutogradState.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPGraphsC10Utils.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/autograd/variable.h>

#include <algorithm>
#include <cstring>
#include <initializer_list>
#include <unordered_map>
#include <utility>

#include "../../include/gemm.h"

namespace {

enum Kind { kMatmul = 0, kWgrad, kRows, kW4, kNorm, kNormI8, kI8Rows, kI8, kRoute, kKinds };
bool has_plan(int kind) { return kind <= kW4 || kind == kI8; }
constexpr int kMaxWords = 64;
constexpr size_t kMostCalls = 4096;

struct Key {
    int n = 0;
    int64_t w[kMaxWords];
    bool push(int64_t v) {
        if (n == kMaxWords) return false;
        w[n++] = v;
        return true;
    }
    bool operator==(const Key& o) const { return n == o.n && std::memcmp(w, o.w, n * sizeof(int64_t)) == 0; }
};

struct KeyHash {
    size_t operator()(const Key& k) const {
        uint64_t h = 0x9E3779B97F4A7C15ull;
        for (int i = 0; i < k.n; ++i) {
            h ^= static_cast<uint64_t>(k.w[i]);
            h *= 0xD6E8FEB86659FD93ull;
            h ^= h >> 32;
        }
        return static_cast<size_t>(h);
    }
};

struct Entry {
    int device;
    PyObject* owner;   // a reference
    void* run;
    void* plan;
    int64_t workspace;
    int64_t sizes[3];   // of the output, `dims` of them; rows: {groups, R, id bytes}
    int dims;
    at::ScalarType dtype;
};

std::unordered_map<Key, Entry, KeyHash>& table(int kind) {
    static std::unordered_map<Key, Entry, KeyHash> tables[kKinds];
    return tables[kind];
}

void forget(int kind) {
    std::unordered_map<Key, Entry, KeyHash> old;
    old.swap(table(kind));   // dropping an owner can run Python code
    for (auto& c : old) Py_XDECREF(c.second.owner);
}

// Appends what the checks look at; false for anything but a plain GPU tensor
// (None is an absent operand).
bool push_tensor(Key* k, PyObject* o, int* device) {
    if (o == Py_None) return k->push(-1);
    if (!THPVariable_CheckExact(o)) return false;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.layout() != at::kStrided || !t.has_storage() || t.is_conj() || t.is_neg()) return false;
    const int dev = t.device().index();
    if (*device < 0) *device = dev;
    const int64_t dims = t.dim();
    if (!k->push(static_cast<int64_t>(t.scalar_type()) | dims << 8 | static_cast<int64_t>(dev) << 16)) return false;
    const auto sizes = t.sizes(), strides = t.strides();
    for (int64_t i = 0; i < dims; ++i)
        if (!k->push(sizes[i]) || !k->push(strides[i])) return false;
    return true;
}

// `extra`: dtypes and None are singletons, known by address.
bool push_extra(Key* k, PyObject* o) {
    if (PyTuple_CheckExact(o)) {
        if (!k->push(4) || !k->push(PyTuple_GET_SIZE(o))) return false;
        for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(o); ++i)
            if (PyTuple_CheckExact(PyTuple_GET_ITEM(o, i)) || !push_extra(k, PyTuple_GET_ITEM(o, i))) return false;
        return true;
    }
    if (PyFloat_CheckExact(o)) {
        const double v = PyFloat_AS_DOUBLE(o);
        int64_t bits;
        std::memcpy(&bits, &v, sizeof bits);
        return k->push(3) && k->push(bits);
    }
    if (PyLong_CheckExact(o)) {
        const int64_t v = PyLong_AsLongLong(o);
        if (v == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            return false;
        }
        return k->push(1) && k->push(v);
    }
    if (o != Py_None && !THPDtype_Check(o)) return false;
    return k->push(2) && k->push(static_cast<int64_t>(reinterpret_cast<intptr_t>(o)));
}

const void* data(PyObject* o) { return o == Py_None ? nullptr : THPVariable_Unpack(o).const_data_ptr(); }

at::Tensor make(at::IntArrayRef sizes, at::ScalarType dtype, const at::Tensor& like) {
    return at::empty(sizes, at::TensorOptions().dtype(dtype).device(like.device()));
}

struct Unlocked {   // the interpreter's lock, released
    PyThreadState* state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

// The exception in flight as torch raises it: an allocation's by its own type, one
// that a Python hook raised as it is.
PyObject* raised() {
    try {
        throw;
    } catch (python_error& ex) {
        if (!PyErr_Occurred()) ex.restore();
    } catch (const c10::OutOfMemoryError& ex) {
        PyObject* const torch = PyImport_ImportModule("torch");
        PyObject* const type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        if (type) PyErr_SetString(type, ex.what_without_backtrace());
        Py_XDECREF(type);
        Py_XDECREF(torch);
    } catch (const std::exception& ex) {
        PyErr_SetString(PyExc_RuntimeError, ex.what());
    }
    return nullptr;
}

struct Held {   // a reference
    PyObject* o;
    explicit Held(PyObject* owner) : o(owner) { Py_INCREF(o); }
    ~Held() { Py_DECREF(o); }
};

// The outputs of one launch (`order`: of the rows) and its status.
struct Result {
    at::Tensor out, order;
    int status;
};

Result launch(int kind, const Entry& e, const at::Tensor& like, const void* const* in) {
    Result r;
    at::Tensor ws;   // released on return: later work of this stream may reuse it, in order
    void* const stream = c10::hip::getCurrentHIPStream(static_cast<c10::DeviceIndex>(e.device)).stream();
    if (kind == kRows) {
        typedef int (*fn)(const void*, int32_t, int64_t, int64_t, void*, void*, void*, size_t, void*);
        r.out = make({e.sizes[0] + 1}, at::kInt, like);
        r.order = make({e.sizes[1]}, at::kInt, like);
        if (e.workspace > 0) ws = make({e.workspace}, at::kByte, like);
        r.status = reinterpret_cast<fn>(e.run)(in[0], static_cast<int32_t>(e.sizes[2]), e.sizes[1], e.sizes[0],
                                               r.out.data_ptr(), r.order.data_ptr(),
                                               e.workspace > 0 ? ws.data_ptr() : nullptr, e.workspace, stream);
        return r;
    }
    r.out = make(at::IntArrayRef(e.sizes, e.dims), e.dtype, like);
    if (kind == kI8) {
        typedef int (*fn)(void*, const void*, const void*, const void*, const void*, const void*, void*, void*);
        r.status = reinterpret_cast<fn>(e.run)(e.plan, in[0], in[1], in[2], in[3], in[4], r.out.data_ptr(), stream);
    } else if (kind == kW4) {
        typedef int (*fn)(void*, const void*, const void*, const void*, const void*, const void*, void*, void*);
        r.status = reinterpret_cast<fn>(e.run)(e.plan, in[0], in[1], in[2], in[3], in[4], r.out.data_ptr(), stream);
    } else {
        typedef int (*fn)(void*, const void*, const void*, const void*, void*, void*, size_t, void*);
        if (e.workspace > 0) ws = make({e.workspace}, at::kByte, like);
        r.status = reinterpret_cast<fn>(e.run)(e.plan, in[0], in[1], in[2], r.out.data_ptr(),
                                               e.workspace > 0 ? ws.data_ptr() : nullptr, e.workspace, stream);
    }
    return r;
}

constexpr int kMostOperands = 5;
int operands(int kind) {
    switch (kind) {
        case kRows:
        case kI8Rows: return 1;
        case kRoute: return 2;
        case kW4:
        case kI8: return 5;
        default: return 3;
    }
}

// ---------------------------------------------------------------- the row operators

struct Library {
    gemm_status (*norm)(const gemm_norm_problem*, const void*, const void*, const void*, void*, void*, float*, void*);
    gemm_status (*norm_i8)(const gemm_norm_problem*, const void*, const void*, const void*, void*, int8_t*, float*, void*);
    gemm_status (*norm_grad_workspace)(const gemm_norm_problem*, size_t*);
    gemm_status (*norm_grad)(const gemm_norm_problem*, const void*, const void*, const void*, const void*, const float*, void*,
                             void*, void*, size_t, void*);
    gemm_status (*quantize)(const void*, gemm_dtype, int64_t, int64_t, int64_t, int8_t*, int64_t, float*, void*);
    gemm_status (*route)(const gemm_route_problem*, const void*, const float*, float*, int32_t*, void*);
    gemm_status (*route_grad)(const gemm_route_problem*, const void*, const int32_t*, const float*, void*, void*);
    const char* (*last_error)();
};
Library library;

struct Refused {   // by the library, with this status
    int status;
};
void check(gemm_status st) {
    if (st != GEMM_OK) throw Refused{static_cast<int>(st)};
}
// In a backward pass there is no Python to hand a status to.
void check_backward(gemm_status st) {
    if (st != GEMM_OK) throw std::runtime_error(library.last_error());
}

using torch::autograd::AutogradContext;
using torch::autograd::variable_list;

gemm_dtype code(const at::Tensor& t) {
    return t.scalar_type() == at::kHalf ? GEMM_F16 : t.scalar_type() == at::kBFloat16 ? GEMM_BF16 : GEMM_F32;
}
void* stream_of(const at::Tensor& t) { return c10::hip::getCurrentHIPStream(t.device().index()).stream(); }
void* data(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// A gradient whose rows are contiguous (a sum's is expanded from one value).
at::Tensor as_rows(const at::Tensor& t) {
    return !t.defined() || t.size(1) <= 1 || t.stride(1) == 1 ? t : t.contiguous();
}

// A saved tensor as it was: hooks may give back another layout, which is taken, and
// anything else, which must not reach a kernel.
at::Tensor as_saved(const at::Tensor& t, const at::Tensor& like, at::IntArrayRef sizes, std::initializer_list<at::ScalarType> types) {
    if (!t.defined() || t.layout() != at::kStrided || t.device() != like.device() || t.sizes() != sizes ||
        std::find(types.begin(), types.end(), t.scalar_type()) == types.end())
        throw std::runtime_error("a saved tensor came back from a hook on another device, of another type or of another shape");
    const at::Tensor r = t.resolve_neg();
    return r.size(-1) <= 1 || r.stride(-1) == 1 ? r : r.contiguous();
}

// These gradients have none of their own: whoever differentiates them is told.
variable_list once(variable_list grads, const char* what) {
    if (!at::GradMode::is_enabled()) return grads;
    for (auto& g : grads)
        if (g.defined()) g = g.detach().set_requires_grad(true);
    auto error = std::make_shared<torch::autograd::DelayedError>(std::string("the gradient of ") + what + " is not differentiable",
                                                                 static_cast<int64_t>(grads.size()));
    return (*error)(std::move(grads));
}

// There is no forward-mode derivative: whoever asks for one is told, whether or
// not the tensor requires a gradient (a dual number need not).
void no_tangent(const at::Tensor& t, const char* what) {
    if (t.defined() && c10::AutogradState::get_tls_state().get_fw_grad_mode() && t._fw_grad(0).defined())
        throw std::runtime_error(std::string(what) + " has no forward-mode derivative");
}

gemm_norm_problem norm_problem(const at::Tensor& x, const at::Tensor& w, const at::Tensor& r, double eps, int64_t sy) {
    gemm_norm_problem p = {};
    p.R = x.size(0);
    p.K = x.size(1);
    p.sx = x.stride(0);
    p.sy = sy;
    if (r.defined()) {
        p.sr = r.stride(0);
        p.sh = p.K;
        p.has_residual = 1;
    }
    p.dtype = code(x);
    p.weight = code(w);
    p.eps = static_cast<float>(eps);
    return p;
}

// y (into), h where there is a residual, rstd where it is wanted
struct Normed {
    at::Tensor y, h, rstd;
};
Normed norm_rows(const at::Tensor& x, const at::Tensor& w, const at::Tensor& r, double eps, bool want_rstd) {
    Normed n;
    n.y = make({x.size(0), x.size(1)}, x.scalar_type(), x);
    if (r.defined()) n.h = make({x.size(0), x.size(1)}, x.scalar_type(), x);
    if (want_rstd) n.rstd = make({x.size(0)}, at::kFloat, x);
    const gemm_norm_problem p = norm_problem(x, w, r, eps, x.size(1));
    check(library.norm(&p, data(x), data(r), data(w), data(n.h), data(n.y), static_cast<float*>(data(n.rstd)), stream_of(x)));
    return n;
}

struct NormFunction : torch::autograd::Function<NormFunction> {
    static variable_list forward(AutogradContext* ctx, const at::Tensor& x, const at::Tensor& w, const std::optional<at::Tensor>& r,
                                 double eps) {
        const Normed n = norm_rows(x, w, r ? *r : at::Tensor(), eps, true);
        ctx->set_materialize_grads(false);
        ctx->save_for_backward({n.h.defined() ? n.h : x, w, n.rstd});
        if (n.h.defined()) return {n.y, n.h};
        return {n.y};
    }

    static variable_list backward(AutogradContext* ctx, variable_list grads) {
        const auto saved = ctx->get_saved_variables();
        for (const at::Tensor& g : grads) no_tangent(g, "the gradient of rms_norm");
        const at::Tensor dy = as_rows(grads[0]), dh = grads.size() > 1 ? as_rows(grads[1]) : at::Tensor();
        at::Tensor dx = dh, dw;
        if (dy.defined()) {
            const at::Tensor h = as_saved(saved[0], dy, dy.sizes(), {dy.scalar_type()});
            const at::Tensor w = as_saved(saved[1], dy, {dy.size(1)}, {dy.scalar_type(), at::kFloat});
            const at::Tensor rstd = as_saved(saved[2], dy, {dy.size(0)}, {at::kFloat});
            const c10::DeviceGuard guard(h.device());
            dx = make({h.size(0), h.size(1)}, h.scalar_type(), h);
            gemm_norm_problem p = norm_problem(dx, w, dh, 1.0, dy.stride(0));
            p.sh = h.stride(0);
            at::Tensor ws;
            size_t need = 0;
            if (ctx->needs_input_grad(1)) {
                dw = make({w.size(0)}, w.scalar_type(), w);
                check_backward(library.norm_grad_workspace(&p, &need));
                if (need > 0) ws = make({static_cast<int64_t>(need)}, at::kByte, h);
            }
            check_backward(library.norm_grad(&p, data(dy), data(dh), data(h), data(w), static_cast<const float*>(data(rstd)), data(dx),
                                             data(dw), data(ws), need, stream_of(h)));
        }
        const bool residual = grads.size() > 1;
        return once({ctx->needs_input_grad(0) ? dx : at::Tensor(), dw,
                     residual && ctx->needs_input_grad(2) ? dx : at::Tensor(), at::Tensor()}, "rms_norm");
    }
};

bool wants_grad(const at::Tensor& t) { return t.defined() && t.requires_grad(); }

// A leaf's gradient is collected on the stream that its first live graph was
// recorded on, which a captured backward pass draws into the capture.  The default
// stream cannot be drawn in, and the process ends.
void not_on_default_stream(const at::Tensor& leaf, const char* what) {
    if (!wants_grad(leaf) || !leaf.is_leaf()) return;
    const auto collector = torch::autograd::impl::try_get_grad_accumulator(leaf);
    if (!collector) return;
    const auto stream = collector->stream();
    const c10::Stream bad = c10::hip::getDefaultHIPStream(leaf.device().index()).unwrap();
    if (stream && stream->id() == bad.id())
        throw std::runtime_error(std::string(what) + ": in a graph's capture, while a graph of the same leaf recorded on the default "
                                 "stream is alive; let go of that one first (its outputs, too), or record it on another stream");
}
void capturable(const at::Tensor& a, const at::Tensor& b, const at::Tensor& c, const char* what) {
    if (c10::hip::currentStreamCaptureStatusMayInitCtx() == c10::hip::CaptureStatus::None) return;
    for (const at::Tensor* t : {&a, &b, &c}) not_on_default_stream(*t, what);
}

// The outputs of an operator, in order.
variable_list norm_call(const at::Tensor& x, const at::Tensor& w, const at::Tensor& r, double eps) {
    for (const at::Tensor* t : {&x, &w, &r}) no_tangent(*t, "rms_norm");
    if (at::GradMode::is_enabled() && (wants_grad(x) || wants_grad(w) || wants_grad(r))) {
        capturable(x, w, r, "rms_norm");
        return NormFunction::apply(x, w, r.defined() ? std::optional<at::Tensor>(r) : std::nullopt, eps);
    }
    const Normed n = norm_rows(x, w, r, eps, false);
    if (n.h.defined()) return {n.y, n.h};
    return {n.y};
}

variable_list norm_i8_call(const at::Tensor& x, const at::Tensor& w, const at::Tensor& r, double eps) {
    at::Tensor q = make({x.size(0), x.size(1)}, at::kChar, x), scale = make({x.size(0)}, at::kFloat, x), h;
    if (r.defined()) h = make({x.size(0), x.size(1)}, x.scalar_type(), x);
    const gemm_norm_problem p = norm_problem(x, w, r, eps, x.size(1));
    check(library.norm_i8(&p, data(x), data(r), data(w), data(h), static_cast<int8_t*>(data(q)), static_cast<float*>(data(scale)),
                          stream_of(x)));
    if (h.defined()) return {q, scale, h};
    return {q, scale};
}

variable_list i8_rows_call(const at::Tensor& x) {
    at::Tensor q = make({x.size(0), x.size(1)}, at::kChar, x), scale = make({x.size(0)}, at::kFloat, x);
    check(library.quantize(data(x), code(x), x.size(0), x.size(1), x.stride(0), static_cast<int8_t*>(data(q)), x.size(1),
                           static_cast<float*>(data(scale)), stream_of(x)));
    return {q, scale};
}

// The parameters of a routing: top, score, groups, top_groups, group_best, renormalize, scale.
constexpr int kRouteInts = 6;
struct RouteParameters {
    int64_t v[kRouteInts];
    double scale;
};

gemm_route_problem route_problem(const at::Tensor& logits, bool bias, const RouteParameters& a) {
    gemm_route_problem p = {};
    p.R = logits.size(0);
    p.E = static_cast<int32_t>(std::min<int64_t>(logits.size(1), INT32_MAX));
    p.sl = logits.stride(0);
    p.top = static_cast<int32_t>(a.v[0]);
    p.score = static_cast<gemm_score>(a.v[1]);
    p.groups = static_cast<int32_t>(a.v[2]);
    p.top_groups = static_cast<int32_t>(a.v[3]);
    p.group_best = static_cast<int32_t>(a.v[4]);
    p.renormalize = static_cast<int32_t>(a.v[5]);
    p.has_bias = bias ? 1 : 0;
    p.scale = static_cast<float>(a.scale);
    p.dtype = code(logits);
    return p;
}

variable_list route_rows(const at::Tensor& logits, const at::Tensor& bias, const RouteParameters& a) {
    const int64_t top = a.v[0] >= 0 && a.v[0] <= logits.size(1) ? a.v[0] : 0;   // others are refused
    at::Tensor w = make({logits.size(0), top}, at::kFloat, logits), ids = make({logits.size(0), top}, at::kInt, logits);
    const gemm_route_problem p = route_problem(logits, bias.defined(), a);
    check(library.route(&p, data(logits), static_cast<const float*>(data(bias)), static_cast<float*>(data(w)),
                        static_cast<int32_t*>(data(ids)), stream_of(logits)));
    return {w, ids};
}

struct RouteFunction : torch::autograd::Function<RouteFunction> {
    static variable_list forward(AutogradContext* ctx, const at::Tensor& logits, const std::optional<at::Tensor>& bias,
                                 const std::vector<int64_t>& v, double scale) {
        RouteParameters a;
        std::copy(v.begin(), v.end(), a.v);
        a.scale = scale;
        variable_list out = route_rows(logits, bias ? *bias : at::Tensor(), a);
        ctx->set_materialize_grads(false);
        ctx->mark_non_differentiable({out[1]});
        ctx->save_for_backward({logits, out[1]});
        ctx->saved_data["v"] = v;
        ctx->saved_data["scale"] = scale;
        return out;
    }

    static variable_list backward(AutogradContext* ctx, variable_list grads) {
        if (!grads[0].defined()) return {at::Tensor(), at::Tensor(), at::Tensor(), at::Tensor()};
        no_tangent(grads[0], "the gradient of route");
        const auto saved = ctx->get_saved_variables();
        const at::Tensor dw = grads[0].contiguous().resolve_neg();
        const int64_t experts = saved[0].defined() && saved[0].dim() == 2 ? saved[0].size(1) : 0;
        const at::Tensor logits = as_saved(saved[0], dw, {dw.size(0), experts}, {at::kHalf, at::kBFloat16, at::kFloat});
        const at::Tensor ids = as_saved(saved[1], dw, dw.sizes(), {at::kInt}).contiguous();
        const auto v = ctx->saved_data["v"].toIntVector();
        RouteParameters a;
        std::copy(v.begin(), v.end(), a.v);
        a.scale = ctx->saved_data["scale"].toDouble();
        const c10::DeviceGuard guard(logits.device());
        at::Tensor dl = make({logits.size(0), logits.size(1)}, logits.scalar_type(), logits);
        const gemm_route_problem p = route_problem(logits, false, a);
        check_backward(library.route_grad(&p, data(logits), static_cast<const int32_t*>(data(ids)), static_cast<const float*>(data(dw)),
                                          data(dl), stream_of(logits)));
        return once({dl, at::Tensor(), at::Tensor(), at::Tensor()}, "route");
    }
};

variable_list route_call(const at::Tensor& logits, const at::Tensor& bias, const RouteParameters& a) {
    no_tangent(logits, "route");
    if (at::GradMode::is_enabled() && wants_grad(logits)) {
        capturable(logits, at::Tensor(), at::Tensor(), "route");
        return RouteFunction::apply(logits, bias.defined() ? std::optional<at::Tensor>(bias) : std::nullopt,
                                    std::vector<int64_t>(a.v, a.v + kRouteInts), a.scale);
    }
    return route_rows(logits, bias, a);
}

at::Tensor tensor_or_none(PyObject* o) { return o == Py_None ? at::Tensor() : THPVariable_Unpack(o); }

bool route_parameters(PyObject* o, RouteParameters* a) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != kRouteInts + 1) {
        PyErr_SetString(PyExc_TypeError, "route: seven parameters");
        return false;
    }
    for (int i = 0; i < kRouteInts; ++i) {
        a->v[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(o, i));
        if (a->v[i] == -1 && PyErr_Occurred()) return false;
        if (a->v[i] != static_cast<int32_t>(a->v[i])) a->v[i] = -1;   // no 32-bit value: refused as negative ones are
    }
    a->scale = PyFloat_AsDouble(PyTuple_GET_ITEM(o, kRouteInts));
    return !(a->scale == -1.0 && PyErr_Occurred());
}

// One of these on checked arguments: a tensor, a tuple of them, or the library's
// status as an int.
PyObject* row_operator(int kind, PyObject* extra, PyObject* const* t) {
    variable_list out;
    RouteParameters a;
    double eps = 0.0;
    if (kind == kRoute && !route_parameters(extra, &a)) return nullptr;
    if (kind == kNorm || kind == kNormI8) {
        eps = PyFloat_AsDouble(extra);
        if (eps == -1.0 && PyErr_Occurred()) return nullptr;
    }
    at::Tensor in[3];
    for (int i = 0; i < operands(kind); ++i) in[i] = tensor_or_none(t[i]);
    try {
        const Unlocked unlocked;
        out = kind == kNorm     ? norm_call(in[0], in[1], in[2], eps)
              : kind == kNormI8 ? norm_i8_call(in[0], in[1], in[2], eps)
              : kind == kI8Rows ? i8_rows_call(in[0])
                                : route_call(in[0], in[1], a);
    } catch (const Refused& r) {
        return PyLong_FromLong(r.status);
    }
    if (out.size() == 1) return THPVariable_Wrap(std::move(out[0]));
    PyObject* tuple = PyTuple_New(static_cast<Py_ssize_t>(out.size()));
    for (size_t i = 0; i < out.size(); ++i) PyTuple_SET_ITEM(tuple, static_cast<Py_ssize_t>(i), THPVariable_Wrap(std::move(out[i])));
    return tuple;
}

// The same from Python: norm(x, weight, residual, eps) and its like.
template <int KIND>
PyObject* py_row_operator(PyObject*, PyObject* const* args, Py_ssize_t n) {
    const int tensors = operands(KIND);
    bool fits = n == tensors + (KIND == kI8Rows ? 0 : 1);
    for (int i = 0; fits && i < tensors; ++i)
        fits = (args[i] == Py_None && i > 0) || (THPVariable_Check(args[i]) && THPVariable_Unpack(args[i]).is_cuda());
    if (!fits) {
        PyErr_SetString(PyExc_TypeError, "checked GPU tensors, and the operator's parameters");
        return nullptr;
    }
    try {
        return row_operator(KIND, n > tensors ? args[tensors] : Py_None, args);
    } catch (const std::exception&) {
        return raised();
    }
}

PyObject* py_functions(PyObject*, PyObject* args) {
    constexpr int count = sizeof(Library) / sizeof(void*);
    if (PyTuple_GET_SIZE(args) != count) {
        PyErr_SetString(PyExc_TypeError, "functions: as many addresses as entry points");
        return nullptr;
    }
    void* at[count];
    for (int i = 0; i < count; ++i) {
        at[i] = reinterpret_cast<void*>(static_cast<uintptr_t>(PyLong_AsUnsignedLongLong(PyTuple_GET_ITEM(args, i))));
        if (PyErr_Occurred()) return nullptr;
    }
    std::memcpy(&library, at, sizeof library);
    Py_RETURN_NONE;
}

bool read_key(Key* key, PyObject* extra, PyObject* const* t, int n, int* device) {
    *device = -1;
    if (!push_extra(key, extra)) return false;
    for (int i = 0; i < n; ++i)
        if (!push_tensor(key, t[i], device)) return false;
    return true;
}

PyObject* py_call(PyObject*, PyObject* const* args, Py_ssize_t n) {
    const long kind = n > 0 ? PyLong_AsLong(args[0]) : -1;
    if (kind < 0 || kind >= kKinds || n != 2 + operands(static_cast<int>(kind))) {
        PyErr_SetString(PyExc_TypeError, "call(kind, extra, *tensors)");
        return nullptr;
    }
    try {
        Key key;
        int device;
        if (!read_key(&key, args[1], args + 2, operands(kind), &device)) Py_RETURN_NONE;
        const auto& calls = table(kind);
        const auto hit = calls.find(key);
        if (hit == calls.end() || c10::hip::current_device() != hit->second.device) Py_RETURN_NONE;
        if (!has_plan(static_cast<int>(kind))) return row_operator(static_cast<int>(kind), args[1], args + 2);
        const Entry e = hit->second;   // the table may change while the lock is released
        const Held plan(e.owner);
        const at::Tensor like = THPVariable_Unpack(args[2]);
        const void* in[kMostOperands];
        for (int i = 0; i < operands(kind); ++i) in[i] = data(args[2 + i]);
        Result r;
        {
            const Unlocked unlocked;
            r = launch(static_cast<int>(kind), e, like, in);
        }
        if (r.status != 0) return PyLong_FromLong(r.status);
        if (kind != kRows) return THPVariable_Wrap(std::move(r.out));
        PyObject* pair = PyTuple_New(2);
        PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(std::move(r.out)));
        PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(std::move(r.order)));
        return pair;
    } catch (const std::exception&) {
        return raised();
    }
}

PyObject* py_remember(PyObject*, PyObject* args) {
    int kind;
    unsigned long long plan, run;
    long long workspace;
    PyObject *owner, *sizes, *dtype, *extra, *tensors;
    if (!PyArg_ParseTuple(args, "iOKKLO!OOO!", &kind, &owner, &plan, &run, &workspace, &PyTuple_Type, &sizes, &dtype, &extra,
                          &PyTuple_Type, &tensors))
        return nullptr;
    if (kind < 0 || kind >= kKinds || PyTuple_GET_SIZE(tensors) != operands(kind) || !THPDtype_Check(dtype) ||
        PyTuple_GET_SIZE(sizes) > 3) {
        PyErr_SetString(PyExc_TypeError, "remember: kind, sizes, dtype or tensors do not fit");
        return nullptr;
    }
    try {
        Key key;
        Entry e;
        PyObject* t[kMostOperands];
        for (int i = 0; i < operands(kind); ++i) t[i] = PyTuple_GET_ITEM(tensors, i);
        if (!read_key(&key, extra, t, operands(kind), &e.device) || e.device < 0) Py_RETURN_NONE;
        e.plan = reinterpret_cast<void*>(static_cast<uintptr_t>(plan));
        e.run = reinterpret_cast<void*>(static_cast<uintptr_t>(run));
        e.workspace = workspace;
        e.dtype = reinterpret_cast<THPDtype*>(dtype)->scalar_type;
        e.dims = static_cast<int>(PyTuple_GET_SIZE(sizes));
        for (int i = 0; i < e.dims; ++i) {
            e.sizes[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(sizes, i));
            if (PyErr_Occurred()) return nullptr;
        }
        auto& calls = table(kind);
        if (calls.size() >= kMostCalls) forget(kind);   // ragged row counts: one entry each
        e.owner = owner;
        if (calls.emplace(key, std::move(e)).second) Py_INCREF(owner);
    } catch (const std::exception&) {
        return raised();
    }
    Py_RETURN_NONE;
}

PyObject* py_forget(PyObject*, PyObject*) {
    for (int k = 0; k < kKinds; ++k) forget(k);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"call", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(py_call)), METH_FASTCALL, nullptr},
    {"remember", py_remember, METH_VARARGS, nullptr},
    {"forget", py_forget, METH_NOARGS, nullptr},
    {"functions", py_functions, METH_VARARGS, nullptr},
#define DTG_ROW(NAME, KIND) \
    {NAME, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&py_row_operator<KIND>)), METH_FASTCALL, nullptr}
    DTG_ROW("norm", kNorm),
    DTG_ROW("norm_i8", kNormI8),
    DTG_ROW("i8_rows", kI8Rows),
    DTG_ROW("route", kRoute),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
