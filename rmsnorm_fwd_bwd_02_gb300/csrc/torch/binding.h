// binding.h -- what the library's Python bindings in C++ share: the checks of
// torch tensors, the allocation of the outputs that a caller did not pass, and
// the raising of a status.
#pragma once

#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <string>

#include "rmsnorm.h"

namespace {

using at::ScalarType;
using at::Tensor;

PyObject *g_check = nullptr;          // check(status, where): raises

// A Python ValueError.
[[noreturn]] void refuse(const std::string &why) { C10_THROW_ERROR(ValueError, why); }

const Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o))
        refuse(c10::str(name, " must be a tensor"));
    return THPVariable_Unpack(o);
}

// The tensor of an optional argument, or nullptr for None.
const Tensor *optional(PyObject *o, const char *name)
{
    return o == Py_None ? nullptr : &tensor(o, name);
}

// rmsnorm_dtype of a row tensor
int row_code(ScalarType t)
{
    switch (t) {
    case at::kFloat: return RMSNORM_F32;
    case at::kBFloat16: return RMSNORM_BF16;
    case at::kHalf: return RMSNORM_F16;
    default: refuse(c10::str("unsupported dtype ", t));
    }
}

void on_device(const Tensor &t, const char *name, at::Device dev)
{
    if (t.device() != dev)
        refuse(c10::str(name, " must be on ", dev, ", got ", t.device()));
}

float *fp32(const Tensor &t, const char *name, at::IntArrayRef shape, at::Device dev)
{
    on_device(t, name, dev);
    if (t.scalar_type() != at::kFloat || t.sizes() != shape || !t.is_contiguous())
        refuse(c10::str(name, " must be a contiguous float32 tensor of shape ", shape, ", got ",
                        t.scalar_type(), " ", t.sizes()));
    return static_cast<float *>(t.data_ptr());
}

// The outputs of one call that the caller did not pass, from torch's CUDA
// allocator (without the dispatcher, which takes as long as the allocation).
// Up to kShared bytes together they are pieces of one allocation, each at a
// multiple of 256 bytes: the norm with the residual takes 3.9 us of a Grace
// core that way and 6.0 with four allocations, beside a launch of 2. That
// memory is free again when the last of them is; larger outputs have an
// allocation each, so that none holds back another's. So do those of the
// quantisation, of any size: a program keeps and saves them as a model's
// weights, and torch.save refuses tensors of two types in one storage (a
// small call takes 3.8 us on the host, 3.4 where the two share). The calls on
// heads share one for outputs of one type only.
class Outputs {
    static constexpr size_t kShared = 256 * 1024, kAlign = 256;
    c10::Storage shared_;
    size_t at_ = 0;

    static c10::Storage storage(size_t bytes)
    {
        c10::Allocator *a = c10::cuda::CUDACachingAllocator::get();
        return c10::Storage(c10::Storage::use_byte_size_t(), bytes, a->allocate(bytes), a,
                            /*resizable=*/true);
    }

public:
    // The bytes of an output of these rows and row stride.
    static size_t bytes(int64_t rows, int64_t ld, ScalarType t)
    {
        const size_t n = (size_t)rows * (size_t)ld * c10::elementSize(t);
        return (n + kAlign - 1) / kAlign * kAlign;
    }
    // An allocation each, on the current device.
    Outputs() = default;
    // One for all where total, the sum of their bytes(), allows it.
    explicit Outputs(size_t total)
    {
        if (total <= kShared)
            shared_ = storage(total);
    }
    // rows x cols, rows ld elements apart; rows < 0: a vector of cols.
    Tensor take(int64_t rows, int64_t cols, int64_t ld, ScalarType t)
    {
        const int skip = rows < 0;
        const size_t n = bytes(skip ? 1 : rows, ld, t);
        Tensor out = at::detail::make_tensor<c10::TensorImpl>(
            shared_ ? c10::Storage(shared_) : storage(n), c10::DispatchKeySet(c10::DispatchKey::CUDA),
            c10::scalarTypeToTypeMeta(t));
        c10::TensorImpl *impl = out.unsafeGetTensorImpl();
        const int64_t sizes[2] = {rows, cols}, strides[2] = {ld, 1};
        impl->set_storage_offset((int64_t)(at_ / c10::elementSize(t)));
        impl->set_sizes_and_strides(at::IntArrayRef(sizes + skip, 2 - skip),
                                    at::IntArrayRef(strides + skip, 2 - skip));
        if (shared_)
            at_ += n;
        return out;
    }
    // A dense tensor of up to four dimensions.
    Tensor dense(at::IntArrayRef sizes, ScalarType t)
    {
        int64_t n = 1, strides[4] = {1, 1, 1, 1};
        for (size_t i = sizes.size(); i-- > 0; n *= sizes[i])
            strides[i] = n;
        Tensor out = take(-1, n, n, t);
        out.unsafeGetTensorImpl()->set_sizes_and_strides(sizes, at::IntArrayRef(strides, sizes.size()));
        return out;
    }
};

PyObject *raised(int status, const char *where)
{
    PyObject *r = PyObject_CallFunction(g_check, "is", status, where);
    if (r != nullptr) {                 // it did not raise
        Py_DECREF(r);
        PyErr_Format(PyExc_RuntimeError, "%s: status %d", where, status);
    }
    return nullptr;
}

bool count(Py_ssize_t n, Py_ssize_t want)
{
    if (n == want && g_check != nullptr)
        return true;
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments, or init() was not called");
    return false;
}

} // namespace
