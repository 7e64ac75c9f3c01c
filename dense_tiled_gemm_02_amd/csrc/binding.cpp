// Native side of the torch calls that grouped.py and w4.py have already checked
// once: from the arguments' types, shapes, strides and devices to the plan and
// the launch, without Python in between.  A decode-sized product is bound by
// its host time: 4.1 to 4.9 us here, 3.4 of them the library's call, against 7.4
// where the call is checked (out given) and passed on by ctypes.
//
//   remember(kind, owner, plan, run, workspace, sizes, dtype, extra, tensors)
//       a call that passed the checks: its gemm_*_run address, plan handle (kept
//       alive by `owner`), workspace bytes, output sizes and type.  `extra`: the
//       call's other argument (an int, a dtype or None).
//   call(kind, extra, *tensors)
//       the outputs; None for a call not remembered (or on a device that is not
//       the current one): the caller then takes the checked path; a non-zero
//       gemm_status as an int if the library refused.
//   forget()
//
// Only plain torch.Tensor and Parameter objects on a GPU are looked up.  The
// interpreter's lock guards the table; it is released for the allocations and
// the launch, which waits while the GPU's queue is full.
#include <Python.h>
#include <ATen/ATen.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <unordered_map>
#include <utility>

namespace {

enum Kind { kMatmul = 0, kWgrad = 1, kRows = 2, kW4 = 3, kKinds };
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
    if (kind == kW4) {
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
int operands(int kind) { return kind == kRows ? 1 : kind == kW4 ? 5 : 3; }

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
    } catch (const std::exception& ex) {
        PyErr_SetString(PyExc_RuntimeError, ex.what());
        return nullptr;
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
    } catch (const std::exception& ex) {
        PyErr_SetString(PyExc_RuntimeError, ex.what());
        return nullptr;
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
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
