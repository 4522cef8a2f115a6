// A planned C-ABI call on torch tensors (CPython module `_call`): what the Python classes do
// around such a call (checking each tensor, allocating outputs and workspace, finding the
// stream, collecting addresses) without the interpreter's share, about 1 us instead of 8. A
// decoding step makes a few such calls for kernels of a few microseconds.
//
// plan(function address, handle, device index, slots) makes the plan. A slot is an argument of the C
// function, in its order; the handle comes first and the stream last:
//   ("in" | "maybe", shape, strides or None, dtype)   a tensor (or None) that the caller gives
//   ("out", shape, dtype)                             an output, allocated here
//   ("storage", ((shape, dtype), ...))                a tuple of tensors; the address of a
//                                                     struct of theirs
//   ("workspace", bytes)                              device memory and its size: given as the
//                                                     last argument, or allocated here
// call(plan, ...) takes the tensors of the "in", "maybe" and "storage" slots in order, then the
// workspace or None. It returns the tuple of outputs, an int status other than 0 of the C
// function, or None if an argument is not what the plan says (the caller then finds out what
// is wrong and says so). All tensors have to be on the plan's device.
#include <ATen/ATen.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <vector>

namespace {

struct Spec {
    std::vector<int64_t> shape, strides;   // no strides: contiguous
    bool dense = true;
    at::ScalarType dtype = at::kByte;
};
enum Kind { kIn, kMaybe, kOut, kStorage, kWorkspace };
struct Slot {
    Kind kind;
    std::vector<Spec> specs;
    int64_t bytes = 0;
};
constexpr int kMostArgs = 14, kMostStorage = 8;
struct Plan {
    uintptr_t fn, handle;
    at::Device device;
    std::vector<Slot> slots;
    Py_ssize_t given = 0;   // arguments of call() behind the plan
    int outs = 0, args = 0;
};

PyObject* g_raw_stream = nullptr;   // device index -> address of torch's current stream

bool sizes_of(PyObject* o, std::vector<int64_t>* to) {
    PyObject* seq = PySequence_Fast(o, "a shape is a sequence");
    if (!seq) return false;
    for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(seq); ++i)
        to->push_back(PyLong_AsLongLong(PySequence_Fast_GET_ITEM(seq, i)));
    Py_DECREF(seq);
    return !PyErr_Occurred();
}
bool spec_of(PyObject* shape, PyObject* strides, PyObject* dtype, Spec* s) {
    if (!THPDtype_Check(dtype)) {
        PyErr_SetString(PyExc_TypeError, "a torch.dtype is wanted");
        return false;
    }
    s->dtype = reinterpret_cast<THPDtype*>(dtype)->scalar_type;
    if (!sizes_of(shape, &s->shape)) return false;
    s->dense = strides == Py_None;
    return s->dense || sizes_of(strides, &s->strides);
}

void free_plan(PyObject* capsule) { delete static_cast<Plan*>(PyCapsule_GetPointer(capsule, "planned call")); }

bool add_slot(Plan* p, PyObject* t) {
    const char* kind = PyTuple_Check(t) && PyTuple_GET_SIZE(t) > 0 ? PyUnicode_AsUTF8(PyTuple_GET_ITEM(t, 0)) : nullptr;
    if (!kind) return false;
    const std::string k = kind;
    const auto item = [&](Py_ssize_t i) { return PyTuple_GetItem(t, i); };
    Slot s;
    if (k == "in" || k == "maybe") {
        s.kind = k == "in" ? kIn : kMaybe;
        s.specs.emplace_back();
        if (PyTuple_GET_SIZE(t) != 4 || !spec_of(item(1), item(2), item(3), &s.specs[0])) return false;
        ++p->given;
        p->args += 1;
    } else if (k == "out") {
        s.kind = kOut;
        s.specs.emplace_back();
        if (PyTuple_GET_SIZE(t) != 3 || !spec_of(item(1), Py_None, item(2), &s.specs[0])) return false;
        ++p->outs;
        p->args += 1;
    } else if (k == "storage") {
        s.kind = kStorage;
        PyObject* parts = PyTuple_GET_SIZE(t) == 2 ? item(1) : nullptr;
        if (!parts || !PyTuple_Check(parts) || PyTuple_GET_SIZE(parts) > kMostStorage) return false;
        for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(parts); ++i) {
            PyObject* part = PyTuple_GET_ITEM(parts, i);
            s.specs.emplace_back();
            if (!PyTuple_Check(part) || PyTuple_GET_SIZE(part) != 2 ||
                !spec_of(PyTuple_GET_ITEM(part, 0), Py_None, PyTuple_GET_ITEM(part, 1), &s.specs.back()))
                return false;
        }
        ++p->given;
        p->args += 1;
    } else if (k == "workspace") {
        s.kind = kWorkspace;
        if (PyTuple_GET_SIZE(t) != 2) return false;
        s.bytes = PyLong_AsLongLong(item(1));
        p->args += 2;
    } else {
        return false;
    }
    p->slots.push_back(std::move(s));
    return !PyErr_Occurred();
}

PyObject* plan(PyObject*, PyObject* args) {
    unsigned long long fn = 0, handle = 0;
    int device = 0;
    PyObject* slots = nullptr;
    if (!PyArg_ParseTuple(args, "KKiO!:plan", &fn, &handle, &device, &PyTuple_Type, &slots)) return nullptr;
    Plan* p = new Plan{(uintptr_t)fn, (uintptr_t)handle, at::Device(at::kCUDA, (at::DeviceIndex)device), {}, 0, 0, 2};
    try {
        for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(slots); ++i)
            if (!add_slot(p, PyTuple_GET_ITEM(slots, i))) {
                delete p;
                if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "not a slot of a planned call");
                return nullptr;
            }
    } catch (const std::exception& e) {
        delete p;
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
    if (p->args > kMostArgs) {
        delete p;
        PyErr_SetString(PyExc_ValueError, "too many arguments for a planned call");
        return nullptr;
    }
    ++p->given;   // the workspace
    return PyCapsule_New(p, "planned call", free_plan);
}

bool fits(PyObject* o, const Spec& s, at::Device device, uintptr_t* address) {
    if (!THPVariable_Check(o)) return false;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() != s.dtype || t.layout() != at::kStrided || t.sizes() != s.shape) return false;
    if (s.dense ? !t.is_contiguous() : t.strides() != s.strides) return false;
    if (t.device() != device) return false;
    *address = reinterpret_cast<uintptr_t>(t.data_ptr());
    return true;
}

// Every argument is an address or a size: 64 bits each, in the order of the C function's.
int invoke(uintptr_t fn, int n, const uintptr_t* a) {
    using U = uintptr_t;
#define CALL(...) reinterpret_cast<int (*)(__VA_ARGS__)>(fn)
    switch (n) {
        case 7: return CALL(U, U, U, U, U, U, U)(a[0], a[1], a[2], a[3], a[4], a[5], a[6]);
        case 8: return CALL(U, U, U, U, U, U, U, U)(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7]);
        case 10:
            return CALL(U, U, U, U, U, U, U, U, U, U)(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9]);
        case 11:
            return CALL(U, U, U, U, U, U, U, U, U, U, U)(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9],
                                                         a[10]);
        case 14:
            return CALL(U, U, U, U, U, U, U, U, U, U, U, U, U, U)(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9],
                                                                  a[10], a[11], a[12], a[13]);
    }
#undef CALL
    return INT32_MIN;
}

PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
    const Plan* p = n > 0 ? static_cast<Plan*>(PyCapsule_GetPointer(args[0], "planned call")) : nullptr;
    if (!p) return nullptr;
    if (n - 1 != p->given) {
        PyErr_SetString(PyExc_TypeError, "a planned call takes its plan's arguments");
        return nullptr;
    }
    try {
        uintptr_t a[kMostArgs], storage[kMostStorage];
        at::Tensor outs[4], workspace;
        Py_ssize_t next = 1;
        // the given tensors first: nothing is allocated for a call that is not the plan's
        int at = 1;
        for (const Slot& s : p->slots) {
            if (s.kind == kIn || s.kind == kMaybe) {
                PyObject* o = args[next++];
                if (s.kind == kMaybe && o == Py_None)
                    a[at] = 0;
                else if (!fits(o, s.specs[0], p->device, &a[at]))
                    Py_RETURN_NONE;
            } else if (s.kind == kStorage) {
                PyObject* o = args[next++];
                if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != (Py_ssize_t)s.specs.size()) Py_RETURN_NONE;
                for (size_t i = 0; i < s.specs.size(); ++i)
                    if (!fits(PyTuple_GET_ITEM(o, i), s.specs[i], p->device, &storage[i])) Py_RETURN_NONE;
                a[at] = reinterpret_cast<uintptr_t>(storage);
            } else if (s.kind == kWorkspace) {
                ++at;
            }
            ++at;
        }
        int n_out = 0;
        at = 1;
        for (const Slot& s : p->slots) {
            if (s.kind == kOut) {
                outs[n_out] = at::empty(s.specs[0].shape, at::TensorOptions().dtype(s.specs[0].dtype).device(p->device));
                a[at] = reinterpret_cast<uintptr_t>(outs[n_out++].data_ptr());
            } else if (s.kind == kWorkspace) {
                PyObject* o = args[n - 1];
                int64_t bytes = s.bytes;
                if (o == Py_None && bytes == 0) {
                    a[at++] = 0;
                    a[at++] = 0;
                    continue;
                }
                if (o == Py_None) {
                    workspace = at::empty({bytes}, at::TensorOptions().dtype(at::kByte).device(p->device));
                } else {
                    if (!THPVariable_Check(o)) Py_RETURN_NONE;
                    workspace = THPVariable_Unpack(o);
                    if (workspace.device() != p->device || !workspace.is_contiguous()) Py_RETURN_NONE;
                    bytes = (int64_t)workspace.nbytes();
                }
                a[at++] = reinterpret_cast<uintptr_t>(workspace.data_ptr());
                a[at] = (uintptr_t)bytes;
            }
            ++at;
        }
        PyObject* index = PyLong_FromLong(p->device.index());
        if (!index) return nullptr;
        PyObject* stream = PyObject_CallOneArg(g_raw_stream, index);
        Py_DECREF(index);
        if (!stream) return nullptr;
        a[0] = p->handle;
        a[p->args - 1] = (uintptr_t)PyLong_AsUnsignedLongLong(stream);
        Py_DECREF(stream);
        if (PyErr_Occurred()) return nullptr;
        const int rc = invoke(p->fn, p->args, a);
        if (rc != 0) return PyLong_FromLong(rc);
        PyObject* result = PyTuple_New(p->outs);
        if (!result) return nullptr;
        for (int i = 0; i < p->outs; ++i) {
            PyObject* o = THPVariable_Wrap(std::move(outs[i]));
            if (!o) {
                Py_DECREF(result);
                return nullptr;
            }
            PyTuple_SET_ITEM(result, i, o);
        }
        return result;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

PyObject* set_raw_stream(PyObject*, PyObject* f) {
    Py_INCREF(f);
    Py_XDECREF(g_raw_stream);
    g_raw_stream = f;
    Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"plan", plan, METH_VARARGS, "plan(function address, handle, device index, slots): a planned call."},
    {"call", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call)), METH_FASTCALL,
     "call(plan, tensors..., workspace or None): outputs, a status, or None."},
    {"set_raw_stream", set_raw_stream, METH_O, "The function from a device's index to its current stream's address."},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_call", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__call(void) { return PyModule_Create(&kModule); }
