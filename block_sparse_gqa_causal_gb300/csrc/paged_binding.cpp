// paged_binding.cpp -- argument marshalling of the paged-cache calls and the
// rotary ones for Python: checks dtypes, shapes, layouts and devices, allocates the outputs
// that were not given and passes raw pointers and the current CUDA stream to
// the C-ABI.  The calls' kernels take a few microseconds for a decoding step;
// the same checks written in Python took three times as long.
#include <Python.h>

#include <ATen/DeviceGuard.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <sstream>
#include <string>
#include <vector>

#include "msa.h"

namespace {

enum Kind { kRequired = 0, kOptional = 1, kOutput = 2 };   // kOutput: allocated when None, and returned

struct Arg {
    std::string name;
    std::vector<int64_t> shape;     // a first dimension of -1: of any size (an input's)
    at::ScalarType dtype;
    int kind;
};
struct Call {
    int op;
    msa_paged_shape shape;
    std::vector<Arg> args;
};
constexpr int kMostArgs = 16;
constexpr const char *kCapsule = "msa_paged_call";

at::ScalarType dtype_of(int code)
{
    switch (code) {
    case 0: return at::kInt;
    case 1: return at::kFloat;
    case 2: return at::kBFloat16;
    default: return at::kFloat8_e4m3fn;
    }
}

void destroy(PyObject *capsule) { delete static_cast<Call *>(PyCapsule_GetPointer(capsule, kCapsule)); }

// prepare(op, (R, T, max_blocks, n_pages, Hq, Hkv, d, d_idx, topk, scale, scale_idx),
//         [(name, shape, dtype code, kind), ...]) -> handle of a call
PyObject *prepare(PyObject *, PyObject *args)
{
    HANDLE_TH_ERRORS
    int op;
    PyObject *list;
    msa_paged_shape s;
    if (!PyArg_ParseTuple(args, "i(iiiiiiiiiff)O!", &op, &s.R, &s.T, &s.max_blocks, &s.n_pages, &s.Hq, &s.Hkv, &s.d, &s.d_idx,
                          &s.topk, &s.scale, &s.scale_idx, &PyList_Type, &list))
        return nullptr;
    auto call = std::make_unique<Call>();
    call->op = op;
    call->shape = s;
    for (Py_ssize_t i = 0; i < PyList_GET_SIZE(list); ++i) {
        const char *name;
        PyObject *shape;
        int dtype, kind;
        if (!PyArg_ParseTuple(PyList_GET_ITEM(list, i), "sO!ii", &name, &PyTuple_Type, &shape, &dtype, &kind)) return nullptr;
        Arg a{name, {}, dtype_of(dtype), kind};
        for (Py_ssize_t j = 0; j < PyTuple_GET_SIZE(shape); ++j) {
            a.shape.push_back(PyLong_AsLongLong(PyTuple_GET_ITEM(shape, j)));
            if (PyErr_Occurred()) return nullptr;
        }
        call->args.push_back(std::move(a));
    }
    if (call->args.size() > kMostArgs) {
        PyErr_SetString(PyExc_ValueError, "too many arguments");
        return nullptr;
    }
    PyObject *capsule = PyCapsule_New(call.get(), kCapsule, destroy);
    if (capsule) call.release();
    return capsule;
    END_HANDLE_TH_ERRORS
}

std::string described(const at::Tensor &t)
{
    std::ostringstream s;
    s << t.scalar_type() << " " << t.sizes() << " contiguous=" << t.is_contiguous() << " on " << t.device();
    return s.str();
}

// any: the size of a first dimension that may be any
int launch(const Call &c, void *const *p, int any, void *ws, size_t n, void *stream)
{
    auto i32 = [&](int i) { return static_cast<int32_t *>(p[i]); };
    auto f32 = [&](int i) { return static_cast<float *>(p[i]); };
    switch (c.op) {
    case MSA_OP_PAGED_PLAN:
        return msa_paged_plan_held(&c.shape, i32(0), i32(1), i32(2), i32(3), i32(4), i32(5), i32(6), i32(7), i32(8), i32(9),
                                   i32(10), i32(11), i32(12), i32(13), ws, n, stream);
    case MSA_OP_PAGED_APPEND:
        return msa_paged_append(&c.shape, p[0], p[1], p[2], i32(3), i32(4), p[5], p[6], f32(7), f32(8), p[9], ws, n, stream);
    case MSA_OP_PAGED_BLOCK_SCORES:
        return msa_paged_block_scores(&c.shape, p[0], p[1], i32(2), i32(3), i32(4), i32(5), f32(6), ws, n, stream);
    case MSA_OP_PAGED_BLOCK_TOPK:
        return msa_paged_block_topk(&c.shape, f32(0), i32(1), i32(2), ws, n, stream);
    case MSA_OP_PAGED_FORK:
        return msa_paged_fork(&c.shape, i32(0), i32(1), i32(2), i32(3), i32(4), i32(5), i32(6), i32(7), i32(8), ws, n, stream);
    case MSA_OP_PAGED_COMPACT:
        return msa_paged_compact(&c.shape, i32(0), i32(1), i32(2), i32(3), i32(4), i32(5), i32(6), i32(7), i32(8), ws, n, stream);
    case MSA_OP_PAGED_COPY:
        return msa_paged_copy(&c.shape, i32(0), any, p[1], p[2], f32(3), f32(4), p[5], ws, n, stream);
    case MSA_OP_PAGED_CHUNK_SCORES:
        return msa_paged_chunk_scores(&c.shape, p[0], p[1], i32(2), i32(3), i32(4), f32(5), ws, n, stream);
    case MSA_OP_PAGED_CHUNK_ATTN:
        return msa_paged_chunk_attn(&c.shape, p[0], p[1], p[2], f32(3), f32(4), i32(5), i32(6), i32(7), i32(8), p[9], f32(10), ws, n, stream);
    default:
        return msa_paged_attn(&c.shape, p[0], p[1], p[2], f32(3), f32(4), i32(5), i32(6), i32(7), i32(8), p[9], f32(10), ws, n,
                              stream);
    }
}

// call(handle, workspace, *tensors) -> the outputs, or the C call's status where that is not MSA_OK
PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    HANDLE_TH_ERRORS
    if (nargs < 2) {
        PyErr_SetString(PyExc_TypeError, "call(handle, workspace, *tensors)");
        return nullptr;
    }
    const Call *c = static_cast<const Call *>(PyCapsule_GetPointer(args[0], kCapsule));
    if (!c) return nullptr;
    const size_t n = c->args.size();
    if ((size_t)nargs != n + 2) {
        PyErr_Format(PyExc_TypeError, "%zu tensors expected, %zd given", n, nargs - 2);
        return nullptr;
    }
    void *ptr[kMostArgs];
    c10::optional<at::Device> dev;
    auto complain = [](const std::string &what) {
        PyErr_SetString(PyExc_ValueError, what.c_str());
        return static_cast<PyObject *>(nullptr);
    };
    int made = 0, outputs = 0, any = 0;
    for (size_t i = 0; i < n; ++i) {
        const Arg &a = c->args[i];
        PyObject *obj = args[2 + i];
        outputs += a.kind == kOutput;
        ptr[i] = nullptr;
        if (obj == Py_None) {
            if (a.kind == kRequired) return complain(a.name + " is None");
            made += a.kind == kOutput;
            continue;
        }
        if (!THPVariable_Check(obj)) return complain(a.name + ": need a tensor");
        const at::Tensor &t = THPVariable_Unpack(obj);
        if (!dev) dev = t.device();
        const at::IntArrayRef want(a.shape);
        const bool free = !want.empty() && want[0] < 0;
        if (free && t.dim() > 0) any = (int)std::min<int64_t>(t.size(0), INT_MAX);
        const bool fits = free ? t.dim() == (int64_t)want.size() && t.sizes().slice(1) == want.slice(1) : t.sizes() == want;
        if (t.scalar_type() != a.dtype || !fits || !t.is_contiguous() || t.device() != *dev) {
            std::ostringstream s;
            s << a.name << ": need a contiguous " << a.dtype << " tensor of shape " << at::IntArrayRef(a.shape) << " on " << *dev
              << ", got " << described(t);
            return complain(s.str());
        }
        ptr[i] = t.data_ptr();
    }
    if (!dev || !dev->is_cuda()) return complain("need CUDA tensors" + (dev ? ", got " + dev->str() : std::string()));
    if (!THPVariable_Check(args[1])) return complain("workspace: need a tensor");
    const at::Tensor &ws = THPVariable_Unpack(args[1]);
    if (ws.device() != *dev || ws.scalar_type() != at::kByte || !ws.is_contiguous())
        return complain("workspace: need a contiguous uint8 tensor on " + dev->str() + ", got " + described(ws));

    const at::DeviceGuard guard(*dev);
    at::Tensor fresh[kMostArgs];
    if (made) {
        // several outputs of one type share an allocation (a plan has seven, and allocating them took longer than the plan)
        bool together = made > 1;
        int64_t total = 0, start[kMostArgs];
        const Arg *one = nullptr;
        for (size_t i = 0; i < n; ++i) {
            const Arg &a = c->args[i];
            if (a.kind != kOutput || args[2 + i] != Py_None) continue;
            if (!one) one = &a;
            together = together && a.dtype == one->dtype;
            start[i] = total;
            total += (c10::multiply_integers(a.shape) + 63) / 64 * 64;
        }
        at::Tensor all;
        if (together) all = at::empty({total}, at::TensorOptions().dtype(one->dtype).device(*dev));
        for (size_t i = 0; i < n; ++i) {
            const Arg &a = c->args[i];
            if (a.kind != kOutput || args[2 + i] != Py_None) continue;
            if (together) {
                fresh[i] = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
                fresh[i].unsafeGetTensorImpl()->set_storage_offset(start[i]);
                fresh[i].unsafeGetTensorImpl()->set_sizes_contiguous(a.shape);
            } else {
                fresh[i] = at::empty(a.shape, at::TensorOptions().dtype(a.dtype).device(*dev));
            }
            ptr[i] = fresh[i].data_ptr();
        }
    }
    const int status = launch(*c, ptr, any, ws.data_ptr(), (size_t)ws.numel(), c10::cuda::getCurrentCUDAStream(dev->index()).stream());
    if (status != MSA_OK) return PyLong_FromLong(status);
    PyObject *out = PyTuple_New(outputs);
    if (!out) return nullptr;
    Py_ssize_t at = 0;
    for (size_t i = 0; i < n; ++i) {
        if (c->args[i].kind != kOutput) continue;
        PyObject *obj = args[2 + i];
        if (obj == Py_None) {
            obj = THPVariable_Wrap(std::move(fresh[i]));
            if (!obj) {
                Py_DECREF(out);
                return nullptr;
            }
        } else {
            Py_INCREF(obj);
        }
        PyTuple_SET_ITEM(out, at++, obj);
    }
    return out;
    END_HANDLE_TH_ERRORS
}

constexpr const char *kRotaryCapsule = "msa_rotary_call";

void destroy_rotary(PyObject *capsule) { delete static_cast<msa_rotary_shape *>(PyCapsule_GetPointer(capsule, kRotaryCapsule)); }

// prepare_rotary(T, Hq, Hkv, d, d_rot, interleaved, period, offset, scale) -> handle of the calls
PyObject *prepare_rotary(PyObject *, PyObject *args)
{
    HANDLE_TH_ERRORS
    auto s = std::make_unique<msa_rotary_shape>();
    *s = msa_rotary_shape{};
    if (!PyArg_ParseTuple(args, "iiiiipiif", &s->T, &s->Hq, &s->Hkv, &s->d, &s->d_rot, &s->interleaved, &s->period, &s->offset, &s->scale))
        return nullptr;
    PyObject *capsule = PyCapsule_New(s.get(), kRotaryCapsule, destroy_rotary);
    if (capsule) s.release();
    return capsule;
    END_HANDLE_TH_ERRORS
}

// The distance between the T tokens of a bf16 tensor [.., heads, d], a token's heads one after another; -1 where there is none.
int64_t token_stride(const at::Tensor &t, int64_t T, int64_t heads, int64_t d)
{
    const int64_t n = t.dim();
    if (n < 2 || t.scalar_type() != at::kBFloat16 || t.size(n - 1) != d || t.size(n - 2) != heads || t.numel() != T * heads * d) return -1;
    if (t.stride(n - 1) != 1 || (heads > 1 && t.stride(n - 2) != d)) return -1;
    int64_t stride = 0, next = 0;
    for (int64_t i = n - 3; i >= 0; --i) {
        if (t.size(i) == 1) continue;
        if (t.stride(i) <= 0) return -1;     // (an expanded tensor: tokens that share their memory)
        if (!stride) stride = t.stride(i);
        else if (t.stride(i) != next) return -1;
        next = t.stride(i) * t.size(i);
    }
    return stride ? stride : heads * d;      // one token
}

// rotary(handle, backward, q, k, positions, freqs, q_out, k_out) -> (q_out, k_out), or the C call's status where that is not MSA_OK
PyObject *rotary(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    HANDLE_TH_ERRORS
    if (nargs != 8) {
        PyErr_SetString(PyExc_TypeError, "rotary(handle, backward, q, k, positions, freqs, q_out, k_out)");
        return nullptr;
    }
    const auto *given = static_cast<const msa_rotary_shape *>(PyCapsule_GetPointer(args[0], kRotaryCapsule));
    if (!given) return nullptr;
    msa_rotary_shape s = *given;
    auto complain = [](const std::string &what) {
        PyErr_SetString(PyExc_ValueError, what.c_str());
        return static_cast<PyObject *>(nullptr);
    };
    static const char *const names[] = {"q", "k", "positions", "freqs", "q_out", "k_out"};
    const at::Tensor *t[6];
    c10::optional<at::Device> dev;
    for (int i = 0; i < 6; ++i) {
        t[i] = nullptr;
        if (args[2 + i] == Py_None) continue;
        if (!THPVariable_Check(args[2 + i])) return complain(std::string(names[i]) + ": need a tensor");
        t[i] = &THPVariable_Unpack(args[2 + i]);
        if (!dev) dev = t[i]->device();
        if (t[i]->device() != *dev) return complain(std::string(names[i]) + ": need a tensor on " + dev->str() + ", got " + described(*t[i]));
    }
    if (!dev || !dev->is_cuda()) return complain("need CUDA tensors" + (dev ? ", got " + dev->str() : std::string()));
    if (!t[0] && !t[1]) return complain("q and k are None");
    if (!t[3] || t[3]->scalar_type() != at::kLong || t[3]->sizes() != at::IntArrayRef({s.d_rot / 2}) || !t[3]->is_contiguous())
        return complain("freqs: need a contiguous Long tensor of " + std::to_string(s.d_rot / 2) + " numbers" + (t[3] ? ", got " + described(*t[3]) : std::string()));
    if (t[2] && (t[2]->scalar_type() != at::kInt || t[2]->numel() != s.T || !t[2]->is_contiguous()))
        return complain("positions: need a contiguous Int tensor of " + std::to_string(s.T) + " numbers, got " + described(*t[2]));
    const at::DeviceGuard guard(*dev);
    long long *strides[4] = {&s.q_stride, &s.k_stride, &s.q_out_stride, &s.k_out_stride};
    at::Tensor fresh[2];
    void *ptr[4] = {};
    for (int i = 0; i < 4; ++i) {
        const int io = i & 1, heads = io ? s.Hkv : s.Hq, at = i < 2 ? i : 2 + i;
        if (i >= 2 && !t[io]) {
            if (t[at]) return complain(std::string(names[at]) + " without its input");
            continue;
        }
        if (!t[at] && i >= 2) {
            fresh[io] = at::empty(t[io]->sizes(), at::TensorOptions().dtype(at::kBFloat16).device(*dev));
            ptr[i] = fresh[io].data_ptr();
            s.zeros |= 1 << io;          // there is nothing in it that could be left as it was
            continue;
        }
        if (!t[at]) continue;
        const int64_t stride = token_stride(*t[at], s.T, heads, s.d);
        if (stride < 0)
            return complain(std::string(names[at]) + ": need BFloat16 [.., " + std::to_string(heads) + ", " + std::to_string(s.d) + "] of " +
                            std::to_string(s.T) + " evenly spaced tokens, each contiguous, got " + described(*t[at]));
        *strides[i] = stride;
        ptr[i] = t[at]->data_ptr();
    }
    const int back = PyObject_IsTrue(args[1]);
    if (back < 0) return nullptr;
    const int status = (back ? msa_rotary_bwd : msa_rotary_fwd)(
        &s, ptr[0], ptr[1], t[2] ? static_cast<int32_t *>(t[2]->data_ptr()) : nullptr, static_cast<unsigned long long *>(t[3]->data_ptr()), ptr[2], ptr[3],
        c10::cuda::getCurrentCUDAStream(dev->index()).stream());
    if (status != MSA_OK) return PyLong_FromLong(status);
    PyObject *out = PyTuple_New(2);
    if (!out) return nullptr;
    for (int io = 0; io < 2; ++io) {
        PyObject *obj = args[6 + io];
        if (fresh[io].defined()) {
            obj = THPVariable_Wrap(std::move(fresh[io]));
            if (!obj) {
                Py_DECREF(out);
                return nullptr;
            }
        } else {
            Py_INCREF(obj);
        }
        PyTuple_SET_ITEM(out, io, obj);
    }
    return out;
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"prepare_rotary", prepare_rotary, METH_VARARGS, nullptr},
    {"rotary", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rotary)), METH_FASTCALL, nullptr},
    {"prepare", prepare, METH_VARARGS, nullptr},
    {"call", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_binding(void) { return PyModule_Create(&module); }
