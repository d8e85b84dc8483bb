// fp8_torch.cpp -- the Python binding of the 8-bit entry points (module
// _fp8_torch): checks torch tensors, allocates the outputs that the caller
// did not pass, and calls the C ABI on the current stream.
//
// Why not ctypes, as for the other entry points: a decode step's 8-bit calls
// run for 2 to 4 us on the GPU, while checking, allocating and marshalling a
// call's tensors in Python takes 13 (the product) to 18 us (the norm with the
// residual) on a Grace core. The arithmetic is all behind the C ABI either
// way.
//
// The module does not link the library: rmsnorm.py hands it the functions'
// addresses and the Python function that raises a status.
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

constexpr int64_t kGroup = 128;

decltype(&rmsnorm_fwd_fp8) g_fwd = nullptr;
decltype(&rmsnorm_quant_fp8) g_quant = nullptr;
decltype(&rmsnorm_gemm_fp8) g_gemm = nullptr;
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

ScalarType dtype_of(PyObject *o, const char *name)
{
    if (!THPDtype_Check(o))
        refuse(c10::str(name, " must be a torch.dtype"));
    return reinterpret_cast<THPDtype *>(o)->scalar_type;
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

int fp8_code(ScalarType t, const char *name)
{
    switch (t) {
    case at::kFloat8_e4m3fn: return RMSNORM_E4M3;
    case at::kFloat8_e5m2: return RMSNORM_E5M2;
    default:
        refuse(c10::str(name, " must be float8_e4m3fn or float8_e5m2, got ", t));
    }
}

void on_device(const Tensor &t, const char *name, at::Device dev)
{
    if (t.device() != dev)
        refuse(c10::str(name, " must be on ", dev, ", got ", t.device()));
}

void two_d(const Tensor &t, const char *name)
{
    if (t.dim() != 2)
        refuse(c10::str(name, " must be 2-D, got ", t.sizes()));
    if (!t.is_cuda())
        refuse(c10::str(name, " must be a CUDA tensor, got ", t.device()));
}

// Row stride (elements) of a [M, H] tensor with unit column stride; H for
// one row.
int64_t row_stride(const Tensor &t, const char *name, int64_t M, int64_t H, ScalarType dtype,
                   at::Device dev)
{
    on_device(t, name, dev);
    if (t.scalar_type() != dtype)
        refuse(c10::str(name, " must be ", dtype, ", got ", t.scalar_type()));
    if (t.dim() != 2 || t.size(0) != M || t.size(1) != H)
        refuse(c10::str(name, " must be of shape [", M, ", ", H, "], got ", t.sizes()));
    if (t.stride(1) != 1 && H > 1)
        refuse(c10::str(name, " must have unit column stride"));
    return M > 1 ? t.stride(0) : H;
}

float *fp32(const Tensor &t, const char *name, at::IntArrayRef shape, at::Device dev)
{
    on_device(t, name, dev);
    if (t.scalar_type() != at::kFloat || t.sizes() != shape || !t.is_contiguous())
        refuse(c10::str(name, " must be a contiguous float32 tensor of shape ", shape, ", got ",
                        t.scalar_type(), " ", t.sizes()));
    return static_cast<float *>(t.data_ptr());
}

// The row stride of an 8-bit [M, H] output: rows start at multiples of 16
// bytes (as the product reads them).
int64_t row_pitch(int64_t H) { return (H + 15) / 16 * 16; }

// The outputs of one call that the caller did not pass, from torch's CUDA
// allocator (without the dispatcher, which takes as long as the allocation).
// Up to kShared bytes together they are pieces of one allocation, each at a
// multiple of 256 bytes: the norm with the residual takes 3.9 us of a Grace
// core that way and 6.0 with four allocations, beside a launch of 2. That
// memory is free again when the last of them is; larger outputs have an
// allocation each, so that none holds back another's. So do those of the
// quantisation, of any size: a program keeps and saves them as a model's
// weights, and torch.save refuses tensors of two types in one storage (a
// small call takes 3.8 us on the host, 3.4 where the two share).
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

// fwd_fp8(x, w, r, q, scale, h, rstd, eps, qdtype, want_rstd)
PyObject *fwd_fp8(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!count(n, 10))
        return nullptr;
    const Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "w");
    const Tensor *r = optional(a[2], "r"), *q_in = optional(a[3], "q"),
                 *scale_in = optional(a[4], "scale"), *h_in = optional(a[5], "h"),
                 *rstd_in = optional(a[6], "rstd");
    const double eps = PyFloat_AsDouble(a[7]);
    if (eps == -1.0 && PyErr_Occurred())
        return nullptr;
    const ScalarType qtype = dtype_of(a[8], "qdtype"), dtype = x.scalar_type();
    const int want_rstd = PyObject_IsTrue(a[9]);
    if (want_rstd < 0)
        return nullptr;
    two_d(x, "x");
    const int64_t M = x.size(0), H = w.numel(), G = (H + kGroup - 1) / kGroup;
    const at::Device dev = x.device();
    const int code = row_code(dtype), qcode = fp8_code(qtype, "qdtype");
    const int64_t ldx = row_stride(x, "x", M, H, dtype, dev);
    on_device(w, "w", dev);
    if (w.scalar_type() != dtype || !w.is_contiguous())
        refuse(c10::str("w must be a contiguous ", dtype, " tensor"));
    if (r == nullptr && h_in != nullptr)
        refuse("h is the residual variant's output: pass r too");
    const int64_t ldr = r ? row_stride(*r, "r", M, H, dtype, dev) : H;
    int64_t ldh = h_in ? row_stride(*h_in, "h", M, H, dtype, dev) : H;
    int64_t ldq = q_in ? row_stride(*q_in, "q", M, H, qtype, dev) : H;
    if (scale_in)
        fp32(*scale_in, "scale", {M, G}, dev);
    if (rstd_in)
        fp32(*rstd_in, "rstd", {M}, dev);

    const c10::cuda::CUDAGuard guard(dev);
    const bool new_h = r && !h_in, new_rstd = want_rstd && !rstd_in;
    if (!q_in)
        ldq = row_pitch(H);
    Outputs made((new_h ? Outputs::bytes(M, H, dtype) : 0) +
                 (q_in ? 0 : Outputs::bytes(M, ldq, qtype)) +
                 (scale_in ? 0 : Outputs::bytes(M, G, at::kFloat)) +
                 (new_rstd ? Outputs::bytes(1, M, at::kFloat) : 0));
    const Tensor h = h_in ? *h_in : new_h ? made.take(M, H, H, dtype) : Tensor();
    const Tensor q = q_in ? *q_in : made.take(M, H, ldq, qtype);
    const Tensor scale = scale_in ? *scale_in : made.take(M, G, G, at::kFloat);
    const Tensor rstd = rstd_in    ? *rstd_in
                        : new_rstd ? made.take(-1, M, M, at::kFloat)
                                   : Tensor();
    const int st = g_fwd(x.data_ptr(), ldx, r ? r->data_ptr() : nullptr, ldr, w.data_ptr(),
                         q.data_ptr(), ldq, static_cast<float *>(scale.data_ptr()),
                         r ? h.data_ptr() : nullptr, ldh,
                         rstd.defined() ? static_cast<float *>(rstd.data_ptr()) : nullptr, M, H,
                         (float)eps, code, qcode, c10::cuda::getCurrentCUDAStream(dev.index()).stream());
    if (st != RMSNORM_OK)
        return raised(st, "rmsnorm_fwd_fp8");
    // (h,) q, scale, rstd or None; an output that was passed comes back itself
    PyObject *out = PyTuple_New(r ? 4 : 3);
    if (out == nullptr)
        return nullptr;
    Py_ssize_t i = 0;
    auto put = [&](PyObject *in, const Tensor &t) {
        PyTuple_SET_ITEM(out, i++, in != Py_None ? Py_NewRef(in) : THPVariable_Wrap(t));
    };
    if (r)
        put(a[5], h);
    put(a[3], q);
    put(a[4], scale);
    put(a[6], rstd);
    return out;
    END_HANDLE_TH_ERRORS
}

// quant_fp8(x, q, scale, block_rows, qdtype)
PyObject *quant_fp8(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!count(n, 5))
        return nullptr;
    const Tensor &x = tensor(a[0], "x");
    const Tensor *q_in = optional(a[1], "q"), *scale_in = optional(a[2], "scale");
    const long rows = PyLong_AsLong(a[3]);
    if (rows == -1 && PyErr_Occurred())
        return nullptr;
    const ScalarType qtype = dtype_of(a[4], "qdtype");
    two_d(x, "x");
    const int64_t M = x.size(0), H = x.size(1);
    const at::Device dev = x.device();
    const int code = row_code(x.scalar_type()), qcode = fp8_code(qtype, "qdtype");
    const int64_t ldx = row_stride(x, "x", M, H, x.scalar_type(), dev);
    if (rows != 1 && rows != kGroup)
        refuse(c10::str("block_rows must be 1 or ", kGroup, ", got ", rows));
    const int64_t R = (M + rows - 1) / rows, G = (H + kGroup - 1) / kGroup;
    int64_t ldq = q_in ? row_stride(*q_in, "q", M, H, qtype, dev) : H;
    if (scale_in)
        fp32(*scale_in, "scale", {R, G}, dev);

    const c10::cuda::CUDAGuard guard(dev);
    if (!q_in)
        ldq = row_pitch(H);
    Outputs made;
    const Tensor q = q_in ? *q_in : made.take(M, H, ldq, qtype);
    const Tensor scale = scale_in ? *scale_in : made.take(R, G, G, at::kFloat);
    const int st = g_quant(x.data_ptr(), ldx, q.data_ptr(), ldq,
                           static_cast<float *>(scale.data_ptr()), M, H, (int)rows, code, qcode,
                           c10::cuda::getCurrentCUDAStream(dev.index()).stream());
    if (st != RMSNORM_OK)
        return raised(st, "rmsnorm_quant_fp8");
    PyObject *out = PyTuple_New(2);
    if (out == nullptr)
        return nullptr;
    PyTuple_SET_ITEM(out, 0, q_in ? Py_NewRef(a[1]) : THPVariable_Wrap(q));
    PyTuple_SET_ITEM(out, 1, scale_in ? Py_NewRef(a[2]) : THPVariable_Wrap(scale));
    return out;
    END_HANDLE_TH_ERRORS
}

// gemm_fp8(a, a_scale, b, b_scale, out, out_dtype, static_weights)
PyObject *gemm_fp8(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!count(n, 7))
        return nullptr;
    const Tensor &a = tensor(v[0], "a"), &sa = tensor(v[1], "a_scale"), &b = tensor(v[2], "b"),
                 &sb = tensor(v[3], "b_scale");
    const Tensor *out_in = optional(v[4], "out");
    const ScalarType dtype = out_in ? out_in->scalar_type() : dtype_of(v[5], "out_dtype");
    const int static_w = PyObject_IsTrue(v[6]);
    if (static_w < 0)
        return nullptr;
    two_d(a, "a");
    two_d(b, "b");
    const int64_t M = a.size(0), K = a.size(1), N = b.size(0), G = (K + kGroup - 1) / kGroup;
    if (b.size(1) != K)
        refuse(c10::str("a [M, K] and b [N, K] must have one K, got ", a.sizes(), " and ", b.sizes()));
    const at::Device dev = a.device();
    const int acode = fp8_code(a.scalar_type(), "a"), bcode = fp8_code(b.scalar_type(), "b");
    const int code = row_code(dtype);
    const int64_t lda = row_stride(a, "a", M, K, a.scalar_type(), dev);
    const int64_t ldb = row_stride(b, "b", N, K, b.scalar_type(), dev);
    const float *sap = fp32(sa, "a_scale", {M, G}, dev);
    const float *sbp = fp32(sb, "b_scale", {(N + kGroup - 1) / kGroup, G}, dev);
    const int64_t ldo = out_in ? row_stride(*out_in, "out", M, N, dtype, dev) : N;

    const c10::cuda::CUDAGuard guard(dev);
    const Tensor out = out_in ? *out_in : Outputs().take(M, N, N, dtype);
    const int st = g_gemm(a.data_ptr(), lda, sap, acode, b.data_ptr(), ldb, sbp, bcode,
                          out.data_ptr(), ldo, M, N, K, code,
                          static_w ? RMSNORM_GEMM_FP8_STATIC_WEIGHTS : 0,
                          c10::cuda::getCurrentCUDAStream(dev.index()).stream());
    if (st != RMSNORM_OK)
        return raised(st, "rmsnorm_gemm_fp8");
    return out_in ? Py_NewRef(v[4]) : THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

// init(address of rmsnorm_fwd_fp8, of rmsnorm_quant_fp8, of rmsnorm_gemm_fp8, check)
PyObject *init(PyObject *, PyObject *args)
{
    unsigned long long fwd, quant, gemm;
    PyObject *check;
    if (!PyArg_ParseTuple(args, "KKKO", &fwd, &quant, &gemm, &check))
        return nullptr;
    g_fwd = reinterpret_cast<decltype(g_fwd)>((uintptr_t)fwd);
    g_quant = reinterpret_cast<decltype(g_quant)>((uintptr_t)quant);
    g_gemm = reinterpret_cast<decltype(g_gemm)>((uintptr_t)gemm);
    Py_INCREF(check);
    Py_XSETREF(g_check, check);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"init", init, METH_VARARGS, nullptr},
    {"fwd_fp8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(fwd_fp8)), METH_FASTCALL,
     nullptr},
    {"quant_fp8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(quant_fp8)),
     METH_FASTCALL, nullptr},
    {"gemm_fp8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(gemm_fp8)), METH_FASTCALL,
     nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fp8_torch", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit__fp8_torch() { return PyModule_Create(&module); }
