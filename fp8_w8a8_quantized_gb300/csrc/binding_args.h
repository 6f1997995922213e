// What the binding's extension modules share: checks of a call's arguments
// (ValueError), where a call runs, and the memory of its results.
#pragma once

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/Exception.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <optional>
#include <sstream>
#include <string>

#include "fp8w8a8.h"

namespace {

using at::Tensor;

std::string shape_text(at::IntArrayRef s) {
    std::ostringstream o;
    o << "(";
    for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
    o << (s.size() == 1 ? ",)" : ")");
    return o.str();
}

const char* dtype_text(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return "torch.bfloat16";
        case at::kFloat: return "torch.float32";
        case at::kInt: return "torch.int32";
        case at::kLong: return "torch.int64";
        case at::kByte: return "torch.uint8";
        default: return c10::toString(t);
    }
}

// Wants `t` to be a CUDA tensor of that dtype and shape (-1: any size).
void expect(const Tensor& t, const char* name, at::ScalarType dtype, at::IntArrayRef shape,
            bool contiguous = true) {
    bool ok = t.defined() && t.is_cuda() && t.scalar_type() == dtype &&
              t.dim() == static_cast<int64_t>(shape.size()) && (!contiguous || t.is_contiguous());
    for (size_t i = 0; ok && i < shape.size(); ++i) ok = shape[i] < 0 || t.size(i) == shape[i];
    if (ok) return;
    std::ostringstream o;
    o << name << " must be a CUDA " << dtype_text(dtype) << " tensor of shape " << shape_text(shape)
      << (contiguous ? ", contiguous" : "") << " (-1: any size)";
    if (t.defined())
        o << "; got " << dtype_text(t.scalar_type()) << " " << shape_text(t.sizes()) << " on "
          << t.device().str() << (t.is_contiguous() ? "" : ", not contiguous");
    TORCH_CHECK_VALUE(false, o.str());
}

Tensor tensor_of(PyObject* o, const char* name) {
    if (o == Py_None) return Tensor();
    TORCH_CHECK_VALUE(THPVariable_Check(o), name, " must be a CUDA tensor; got ", Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}

int64_t int_of(PyObject* o, const char* name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        TORCH_CHECK_VALUE(false, name, " must be a whole number of 64 bits");
    }
    return v;
}

float float_of(PyObject* o, const char* name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        TORCH_CHECK_VALUE(false, name, " must be a number");
    }
    return static_cast<float>(v);
}

bool bool_of(PyObject* o, const char* name) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) {
        PyErr_Clear();
        TORCH_CHECK_VALUE(false, name, " must be true or false");
    }
    return v != 0;
}

void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// Where a call runs: on the device of its first tensor, on the given stream
// (None: the device's current one), which is current while it allocates, so
// that memory that the caller lets go of is only used again behind the call.
struct Place {
    c10::cuda::CUDAGuard device;
    std::optional<c10::cuda::CUDAStreamGuard> guard;
    void* stream;
    Place(const Tensor& first, PyObject* s) : device(first.device()) {
        const auto index = first.device().index();
        if (s == Py_None) {
            stream = c10::cuda::getCurrentCUDAStream(index).stream();
        } else {
            cudaStream_t raw = reinterpret_cast<cudaStream_t>(int_of(s, "stream"));
            guard.emplace(raw ? c10::cuda::getStreamFromExternal(raw, index)
                              : c10::cuda::getDefaultCUDAStream(index));
            stream = raw;
        }
    }
};

void same_device(const Tensor& first, std::initializer_list<const Tensor*> others) {
    for (const Tensor* t : others)
        TORCH_CHECK_VALUE(!t->defined() || t->device() == first.device(),
                          "all tensors of a call must be on one device: ", first.device().str(), " and ",
                          t->device().str());
}

// (straight from the caching allocator: at::empty's dispatch costs as much again)
Tensor make(at::IntArrayRef shape, at::ScalarType dtype, const Tensor& like) {
    return at::detail::empty_cuda(shape, dtype, like.device(), std::nullopt);
}

// A contiguous tensor in a block that make() gave, from byte `offset` on.
Tensor carve(const Tensor& block, int64_t offset, at::IntArrayRef shape, at::ScalarType dtype) {
    Tensor t = at::detail::make_tensor<c10::TensorImpl>(
        c10::Storage(block.storage()), c10::DispatchKeySet(c10::DispatchKey::CUDA),
        c10::scalarTypeToTypeMeta(dtype));
    t.unsafeGetTensorImpl()->set_storage_offset(offset / static_cast<int64_t>(c10::elementSize(dtype)));
    t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    return t;
}

PyObject* status(fp8_status_t s) { return PyLong_FromLong(s); }

#define NARGS(want)                                                          \
    TORCH_CHECK_TYPE(nargs == (want), "internal call with ", nargs, " arguments")

}  // namespace
