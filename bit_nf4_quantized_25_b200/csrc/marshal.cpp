// marshal.cpp -- the plain calls of the 8-bit activations and the 4-bit integer weights from Python: operands checked, results
// allocated on the current stream and the C ABI called in one step. At a few tokens a call takes the host longer than
// the GPU; from Python, with the tensors allocated one by one and the arguments through ctypes, act8_quantize took 9.5 us
// instead of 4.5, of which the library's call is 2.5.
//
// Each function returns what was asked for, the status if the library refused, or None for operands that are not plainly
// right: binding.py then takes its own, general way, which names what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <initializer_list>

#include "qlora_nf4.h"

namespace {

using at::ScalarType;

// The library's functions, by the addresses that the ctypes handle has.
struct Lib {
    decltype(&::act8_quantize) quantize8;
    decltype(&::act8_dequantize) dequantize8;
    decltype(&::qlora_lora_grads_act8_workspace_size) grads_size;
    decltype(&::qlora_lora_grads_act8) grads;
    decltype(&::swiglu_act8_fwd) swiglu_fwd;
    decltype(&::swiglu_act8_bwd) swiglu_bwd;
    decltype(&::int4_quantize) quantize4;
    decltype(&::int4_dequantize) dequantize4;
    decltype(&::int4_linear_fwd) linear4;
} lib = {};

constexpr int kFunctions = 9;
static_assert(sizeof(Lib) == kFunctions * sizeof(void *), "");

struct NoGil {
    PyThreadState *state = PyEval_SaveThread();
    ~NoGil() { PyEval_RestoreThread(state); }
};

// The current device's contiguous 2-D tensor of this type in o, or null.
const at::Tensor *matrix(PyObject *o, ScalarType type, c10::DeviceIndex dev) {
    if (!THPVariable_Check(o)) return nullptr;
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.layout() != at::kStrided || !t.is_cuda() || t.get_device() != dev || t.scalar_type() != type || t.dim() != 2 ||
        !t.is_contiguous())
        return nullptr;
    return &t;
}
const at::Tensor *matrix(PyObject *o, ScalarType type, c10::DeviceIndex dev, int64_t rows, int64_t cols) {
    const at::Tensor *t = matrix(o, type, dev);
    return t && t->size(0) == rows && t->size(1) == cols ? t : nullptr;
}

// What torch.empty ends up in; going there directly saves half a microsecond a tensor.
at::Tensor make(int64_t rows, int64_t cols, ScalarType type, c10::DeviceIndex dev) {
    return at::Tensor(at::detail::empty_cuda({rows, cols}, type, at::Device(at::kCUDA, dev), std::nullopt));
}

bool number(PyObject *o, int64_t &v) {
    if (!PyLong_CheckExact(o)) return false;
    v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    return v > 0;
}

PyObject *pack(std::initializer_list<at::Tensor> ts) {
    PyObject *out = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
    if (!out) return nullptr;
    Py_ssize_t i = 0;
    for (const at::Tensor &t : ts) {
        PyObject *o = t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
        if (!o) {
            Py_DECREF(out);
            return nullptr;
        }
        PyTuple_SET_ITEM(out, i++, o);
    }
    return out;
}

constexpr ScalarType kBf = ScalarType::BFloat16, kI8 = ScalarType::Char, kU8 = ScalarType::Byte, kF32 = ScalarType::Float;

struct Here {
    c10::DeviceIndex dev = c10::cuda::current_device();
    void *stream() const { return c10::cuda::getCurrentCUDAStream(dev).stream(); }
};

// An activation in 8 bits: rows, cols, codes, absmax, the first four of o.
bool act8(PyObject *const *o, const Here &here, qn_act8 &a) {
    if (!number(o[0], a.rows) || !number(o[1], a.cols) || a.cols % 64) return false;
    const at::Tensor *codes = matrix(o[2], kI8, here.dev, a.rows, a.cols), *absmax = matrix(o[3], kBf, here.dev, a.rows, a.cols / 64);
    if (!codes || !absmax) return false;
    a.codes = static_cast<int8_t *>(codes->data_ptr());
    a.absmax = static_cast<uint16_t *>(absmax->data_ptr());
    return true;
}
// A new one.
struct New8 {
    at::Tensor codes, absmax;
    qn_act8 c;
    New8(int64_t rows, int64_t cols, const Here &here)
        : codes(make(rows, cols, kI8, here.dev)),
          absmax(make(rows, cols / 64, kBf, here.dev)),
          c{rows, cols, static_cast<int8_t *>(codes.data_ptr()), static_cast<uint16_t *>(absmax.data_ptr())} {}
};

// A weight in 4-bit integers: n_out, k_in, group, codes, scale, zero_point, the first six of o.
bool int4(PyObject *const *o, const Here &here, qn_int4_weight &w) {
    int64_t group;
    if (!number(o[0], w.n_out) || !number(o[1], w.k_in) || !number(o[2], group)) return false;
    if ((group != 32 && group != 64 && group != 128) || w.k_in % group || w.k_in % 64) return false;
    w.group = static_cast<int32_t>(group);
    const at::Tensor *codes = matrix(o[3], kU8, here.dev, w.n_out, w.k_in / 2);
    const at::Tensor *scale = matrix(o[4], kBf, here.dev, w.n_out, w.k_in / group);
    const at::Tensor *zero = o[5] == Py_None ? nullptr : matrix(o[5], kU8, here.dev, w.n_out, w.k_in / group);
    if (!codes || !scale || (!zero && o[5] != Py_None)) return false;
    w.codes = static_cast<uint8_t *>(codes->data_ptr());
    w.scale = static_cast<uint16_t *>(scale->data_ptr());
    w.zero_point = zero ? static_cast<uint8_t *>(zero->data_ptr()) : nullptr;
    return true;
}

template <typename F>
qn_status run(F &&f) {
    NoGil free;
    return f();
}

// `first`: an operand that is a tensor. The current device is asked for only when it lies on a GPU.
#define FUNCTION(name, count, first)                                                           \
    PyObject *name(PyObject *, PyObject *const *o, Py_ssize_t n) {                             \
        HANDLE_TH_ERRORS                                                                       \
        if (n != (count)) {                                                                    \
            PyErr_SetString(PyExc_TypeError, #name " takes " #count " arguments");             \
            return nullptr;                                                                    \
        }                                                                                      \
        if (!THPVariable_Check(o[first]) || !THPVariable_Unpack(o[first]).is_cuda()) Py_RETURN_NONE; \
        const Here here;
#define END_FUNCTION   \
    END_HANDLE_TH_ERRORS \
    }
#define RETURN(status, result) return (status) == QN_OK ? (result) : PyLong_FromLong(status)

FUNCTION(act8_quantize, 1, 0)  // x
    const at::Tensor *x = matrix(o[0], kBf, here.dev);
    if (!x || x->numel() == 0 || x->size(1) % 64) Py_RETURN_NONE;
    New8 out(x->size(0), x->size(1), here);
    const qn_status s = run([&] { return lib.quantize8(x->data_ptr(), &out.c, here.stream()); });
    RETURN(s, pack({out.codes, out.absmax}));
END_FUNCTION

FUNCTION(act8_dequantize, 4, 2)  // an activation
    qn_act8 a;
    if (!act8(o, here, a)) Py_RETURN_NONE;
    at::Tensor out = make(a.rows, a.cols, kBf, here.dev);
    const qn_status s = run([&] { return lib.dequantize8(&a, out.data_ptr(), here.stream()); });
    RETURN(s, THPVariable_Wrap(out));
END_FUNCTION

FUNCTION(lora_grads, 8, 2)  // an activation, grad_h, A, B, alpha
    qn_act8 x;
    if (!act8(o, here, x) || !PyFloat_Check(o[7])) Py_RETURN_NONE;
    const at::Tensor *gh = matrix(o[4], kBf, here.dev), *A = matrix(o[5], kBf, here.dev), *B = matrix(o[6], kBf, here.dev);
    if (!gh || !A || !B) Py_RETURN_NONE;
    const int64_t n_out = gh->size(1), r = A->size(0);
    if (gh->size(0) != x.rows || A->size(1) != x.cols || B->size(0) != n_out || B->size(1) != r || n_out == 0 || r == 0 ||
        r > QN_MAX_RANK)
        Py_RETURN_NONE;
    size_t bytes = 0;
    qn_status s = lib.grads_size(x.rows, n_out, static_cast<int>(r), &bytes);
    if (s != QN_OK) return PyLong_FromLong(s);
    at::Tensor grad_A = make(r, x.cols, kF32, here.dev), grad_B = make(n_out, r, kF32, here.dev);
    at::Tensor ws = make(1, static_cast<int64_t>(bytes), kU8, here.dev);
    const float alpha = static_cast<float>(PyFloat_AS_DOUBLE(o[7]));
    s = run([&] {
        return lib.grads(&x, gh->data_ptr(), n_out, A->data_ptr(), B->data_ptr(), static_cast<int>(r), alpha, nullptr,
                         static_cast<float *>(grad_A.data_ptr()), static_cast<float *>(grad_B.data_ptr()), ws.data_ptr(), bytes,
                         here.stream());
    });
    RETURN(s, pack({grad_A, grad_B}));
END_FUNCTION

FUNCTION(swiglu_fwd, 2, 0)  // gate, up
    const at::Tensor *gate = matrix(o[0], kBf, here.dev);
    if (!gate || gate->numel() == 0 || gate->size(1) % 64) Py_RETURN_NONE;
    const int64_t rows = gate->size(0), cols = gate->size(1);
    const at::Tensor *up = matrix(o[1], kBf, here.dev, rows, cols);
    if (!up) Py_RETURN_NONE;
    at::Tensor y = make(rows, cols, kBf, here.dev);
    New8 g(rows, cols, here), u(rows, cols, here);
    const qn_status s = run([&] { return lib.swiglu_fwd(gate->data_ptr(), up->data_ptr(), y.data_ptr(), &g.c, &u.c, here.stream()); });
    RETURN(s, pack({y, g.codes, g.absmax, u.codes, u.absmax}));
END_FUNCTION

FUNCTION(swiglu_bwd, 9, 2)  // two activations, grad_y
    qn_act8 g, u;
    if (!act8(o, here, g) || !act8(o + 4, here, u) || g.rows != u.rows || g.cols != u.cols) Py_RETURN_NONE;
    const at::Tensor *dy = matrix(o[8], kBf, here.dev, g.rows, g.cols);
    if (!dy) Py_RETURN_NONE;
    at::Tensor dg = make(g.rows, g.cols, kBf, here.dev), du = make(g.rows, g.cols, kBf, here.dev);
    New8 y(g.rows, g.cols, here);
    const qn_status s = run([&] { return lib.swiglu_bwd(&g, &u, dy->data_ptr(), dg.data_ptr(), du.data_ptr(), &y.c, here.stream()); });
    RETURN(s, pack({dg, du, y.codes, y.absmax}));
END_FUNCTION

FUNCTION(int4_quantize, 3, 0)  // W, group, whether with zero points
    const at::Tensor *W = matrix(o[0], kBf, here.dev);
    int64_t group;
    if (!W || W->numel() == 0 || !number(o[1], group) || !PyBool_Check(o[2])) Py_RETURN_NONE;
    const int64_t n_out = W->size(0), k_in = W->size(1);
    if ((group != 32 && group != 64 && group != 128) || k_in % group || k_in % 64) Py_RETURN_NONE;
    at::Tensor codes = make(n_out, k_in / 2, kU8, here.dev), scale = make(n_out, k_in / group, kBf, here.dev), zero;
    if (o[2] == Py_True) zero = make(n_out, k_in / group, kU8, here.dev);
    const qn_int4_weight w{n_out, k_in, static_cast<int32_t>(group), static_cast<uint8_t *>(codes.data_ptr()),
                           static_cast<uint16_t *>(scale.data_ptr()),
                           zero.defined() ? static_cast<uint8_t *>(zero.data_ptr()) : nullptr};
    const qn_status s = run([&] { return lib.quantize4(W->data_ptr(), &w, here.stream()); });
    RETURN(s, pack({codes, scale, zero}));
END_FUNCTION

FUNCTION(int4_dequantize, 6, 3)  // a weight
    qn_int4_weight w;
    if (!int4(o, here, w)) Py_RETURN_NONE;
    at::Tensor out = make(w.n_out, w.k_in, kBf, here.dev);
    const qn_status s = run([&] { return lib.dequantize4(&w, out.data_ptr(), here.stream()); });
    RETURN(s, THPVariable_Wrap(out));
END_FUNCTION

FUNCTION(int4_linear, 7, 3)  // a weight, x
    qn_int4_weight w;
    if (!int4(o, here, w)) Py_RETURN_NONE;
    const at::Tensor *x = matrix(o[6], kBf, here.dev);
    if (!x || x->size(1) != w.k_in || x->size(0) == 0) Py_RETURN_NONE;
    const int64_t M = x->size(0);
    at::Tensor h = make(M, w.n_out, kBf, here.dev);
    const qn_status s = run([&] { return lib.linear4(&w, x->data_ptr(), M, h.data_ptr(), here.stream()); });
    RETURN(s, THPVariable_Wrap(h));
END_FUNCTION

// The addresses of the library's functions, in the order of Lib.
PyObject *bind(PyObject *, PyObject *const *o, Py_ssize_t n) {
    if (n != kFunctions) {
        PyErr_SetString(PyExc_TypeError, "bind takes the library's functions");
        return nullptr;
    }
    void *at[kFunctions];
    for (int i = 0; i < kFunctions; ++i) {
        at[i] = PyLong_AsVoidPtr(o[i]);
        if (!at[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
            return nullptr;
        }
    }
    std::memcpy(&lib, at, sizeof(lib));
    Py_RETURN_NONE;
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind), METHOD(act8_quantize), METHOD(act8_dequantize), METHOD(lora_grads), METHOD(swiglu_fwd),
                         METHOD(swiglu_bwd), METHOD(int4_quantize), METHOD(int4_dequantize), METHOD(int4_linear), {nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
