// py_binding.cpp -- argument marshalling of the operators' torch wrappers
// (module _binding): checks tensors and fills in the C ABI's argument structs.
//
// A norm of one row takes 3 us on the GPU; reading five properties of each of
// six tensors took the wrapper as long in Python.  The C entry points are
// called by the addresses that init() is given, so they are those of the
// library that the package has loaded.  Nothing is kept from call to call.
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>
#include <string>

#include "ar.h"

namespace {

decltype(&ar_rmsnorm) p_rmsnorm = nullptr;
decltype(&ar_reduce_scatter_rmsnorm) p_reduce_scatter_rmsnorm = nullptr;
decltype(&ar_rmsnorm_backward) p_rmsnorm_backward = nullptr;

// A refused argument: becomes a ValueError.
struct Refused : std::exception {
    std::string text;
    explicit Refused(std::string t) : text(std::move(t)) {}
    const char* what() const noexcept override { return text.c_str(); }
};
// A Python error that is set already.
struct Raised : std::exception {};

const at::Tensor* tensor_or_none(PyObject* o, const char* what)
{
    if (o == Py_None)
        return nullptr;
    if (!THPVariable_Check(o))
        throw Refused(std::string(what) + " must be a tensor");
    return &THPVariable_Unpack(o);
}

const at::Tensor& tensor(PyObject* o, const char* what)
{
    const at::Tensor* t = tensor_or_none(o, what);
    if (!t)
        throw Refused(std::string(what) + " must be a tensor");
    return *t;
}

int64_t integer(PyObject* o)
{
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw Raised();
    return v;
}

float real(PyObject* o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw Raised();
    return (float)v;
}

// A stream's handle or a communicator's (None: NULL).
void* handle(PyObject* o)
{
    if (o == Py_None)
        return nullptr;
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred())
        throw Raised();
    return p;
}

std::string shape_text(at::IntArrayRef s)
{
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i)
        t += (i ? ", " : "") + std::to_string(s[i]);
    return t + ")";
}

std::string type_text(at::ScalarType t)
{
    switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    default: return c10::toString(t);
    }
}

// The AR_* code of a type, -1 for one that is not the library's.
int code_of(at::ScalarType t)
{
    switch (t) {
    case at::kInt: return AR_INT32;
    case at::kFloat: return AR_FLOAT32;
    case at::kBFloat16: return AR_BF16;
    case at::kFloat8_e4m3fn: return AR_E4M3;
    default: return -1;
    }
}

void check(const at::Tensor& t, int64_t device, at::IntArrayRef shape, at::ScalarType type,
           const char* what)
{
    if (!t.is_cuda() || t.get_device() != device)
        throw Refused(std::string(what) + " must be on cuda:" + std::to_string(device) + ", not " +
                      t.device().str());
    if (t.scalar_type() != type)
        throw Refused(std::string(what) + " has dtype " + type_text(t.scalar_type()) + ", not " +
                      type_text(type));
    if (t.sizes() != shape)
        throw Refused(std::string(what) + " must have shape " + shape_text(shape) + ", not " +
                      shape_text(t.sizes()));
}

// Address and row distance of a [rows, cols] tensor.
void* rows_of(const at::Tensor& t, int64_t device, at::IntArrayRef shape, at::ScalarType type,
              const char* what, size_t* stride)
{
    check(t, device, shape, type, what);
    if (t.stride(1) != 1 && shape[1] > 1)
        throw Refused(std::string("the last dimension of ") + what + " must be contiguous");
    *stride = (size_t)t.stride(0);
    return t.data_ptr();
}

// Address of a contiguous tensor.
void* block_of(const at::Tensor& t, int64_t device, at::IntArrayRef shape, at::ScalarType type,
               const char* what)
{
    check(t, device, shape, type, what);
    if (!t.is_contiguous())
        throw Refused(std::string(what) + " must be contiguous");
    return t.data_ptr();
}

// Codes of a norm's stream and weight.
void norm_types(const at::Tensor& x, const at::Tensor& weight, const char* what, int* dtype,
                int* weight_dtype)
{
    *dtype = code_of(x.scalar_type());
    *weight_dtype = code_of(weight.scalar_type());
    if (*dtype != AR_FLOAT32 && *dtype != AR_BF16)
        throw Refused(std::string(what) + " has dtype " + type_text(x.scalar_type()) +
                      ": float32 or bfloat16 is wanted");
    if (*weight_dtype != *dtype && *weight_dtype != AR_FLOAT32)
        throw Refused("weight has dtype " + type_text(weight.scalar_type()) + ": " +
                      type_text(x.scalar_type()) + " or torch.float32 is wanted");
    if (!x.is_cuda())
        throw Refused(std::string(what) + " must be on the GPU");
}

// A norm's output code, and its scales per row (0: no e4m3).
int64_t norm_output(const at::Tensor& x, const at::Tensor& y, const at::Tensor* scale, int64_t group,
                    int64_t cols, int dtype, int* out_dtype)
{
    *out_dtype = code_of(y.scalar_type());
    if (*out_dtype == dtype) {
        if (scale || group)
            throw Refused("scale and group belong to an e4m3 output");
        return 0;
    }
    if (*out_dtype != AR_E4M3)
        throw Refused("y has dtype " + type_text(y.scalar_type()) + ": " +
                      type_text(x.scalar_type()) + " or torch.float8_e4m3fn is wanted");
    if (!scale)
        throw Refused("an e4m3 output needs scale");
    if (group != 0 && group != 32 && group != 64 && group != 128 && group != 256)
        throw Refused("group must be 0 (a whole row), 32, 64, 128 or 256, got " +
                      std::to_string(group));
    return group ? (cols + group - 1) / group : 1;
}

template <class Call>
PyObject* guarded(Call call)
{
    try {
        return call();
    } catch (const Refused& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const Raised&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// An entry point's status.  Other Python threads run meanwhile: a launch may
// have to wait for room in its stream's queue.
template <class F, class... Args>
PyObject* status_of(F entry, Args... args)
{
    int rc = 0;
    Py_BEGIN_ALLOW_THREADS
    rc = entry(args...);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

void expect(Py_ssize_t got, Py_ssize_t want)
{
    if (got != want)
        throw Refused("wrong number of arguments");
    if (!p_rmsnorm)
        throw Refused("the binding has not been given the library's entry points");
}

// init(ar_rmsnorm, ar_reduce_scatter_rmsnorm, ar_rmsnorm_backward): addresses.
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        if (n != 3)
            throw Refused("wrong number of arguments");
        p_rmsnorm = reinterpret_cast<decltype(p_rmsnorm)>(handle(a[0]));
        p_reduce_scatter_rmsnorm = reinterpret_cast<decltype(p_reduce_scatter_rmsnorm)>(handle(a[1]));
        p_rmsnorm_backward = reinterpret_cast<decltype(p_rmsnorm_backward)>(handle(a[2]));
        Py_RETURN_NONE;
    });
}

// rmsnorm(x, weight, y, eps, residual, sum, scale, group, rstd, stream) -> status
PyObject* rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        expect(n, 10);
        const at::Tensor &x = tensor(a[0], "x"), &weight = tensor(a[1], "weight"),
                         &y = tensor(a[2], "y");
        const at::Tensor *residual = tensor_or_none(a[4], "residual"),
                         *sum = tensor_or_none(a[5], "sum"), *scale = tensor_or_none(a[6], "scale"),
                         *rstd = tensor_or_none(a[8], "rstd");
        if (x.dim() != 2)
            throw Refused("x must have shape (rows, cols), got " + shape_text(x.sizes()));
        const int64_t rows = x.size(0), cols = x.size(1), group = integer(a[7]);
        ar_rmsnorm_t p = {};
        norm_types(x, weight, "x", &p.dtype, &p.weight_dtype);
        const int64_t groups = norm_output(x, y, scale, group, cols, p.dtype, &p.out_dtype);
        const int64_t dev = x.get_device();
        const at::ScalarType type = x.scalar_type();
        const int64_t shape[] = {rows, cols}, scales[] = {rows, groups};
        p.eps = real(a[3]);
        p.rows = (size_t)rows;
        p.cols = (size_t)cols;
        p.group = (size_t)group;
        p.x = rows_of(x, dev, shape, type, "x", &p.x_stride);
        p.weight = block_of(weight, dev, {cols}, weight.scalar_type(), "weight");
        p.y = rows_of(y, dev, shape, y.scalar_type(), "y", &p.y_stride);
        if (residual)
            p.residual = rows_of(*residual, dev, shape, type, "residual", &p.residual_stride);
        if (sum)
            p.sum = rows_of(*sum, dev, shape, type, "sum", &p.sum_stride);
        if (scale)
            p.scale = static_cast<float*>(block_of(*scale, dev, scales, at::kFloat, "scale"));
        if (rstd)
            p.rstd = static_cast<float*>(block_of(*rstd, dev, {rows}, at::kFloat, "rstd"));
        return status_of(p_rmsnorm, &p, handle(a[9]));
    });
}

// reduce_scatter_rmsnorm(comm, send, weight, y, eps, residual, sum, scale, group, rstd, stream,
// ranks, dtype, device) -> status; the last three are the comm's
PyObject* reduce_scatter_rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        expect(n, 14);
        const at::Tensor &send = tensor(a[1], "send"), &weight = tensor(a[2], "weight"),
                         &y = tensor(a[3], "y");
        const at::Tensor *residual = tensor_or_none(a[5], "residual"),
                         *sum = tensor_or_none(a[6], "sum"), *scale = tensor_or_none(a[7], "scale"),
                         *rstd = tensor_or_none(a[9], "rstd");
        const int64_t cols = weight.dim() == 1 ? weight.size(0) : 0, group = integer(a[8]);
        const int64_t R = integer(a[11]);
        if (y.dim() != 2 || y.size(0) != R || (cols ? y.size(1) % cols : y.size(1)))
            throw Refused("y must have shape (" + std::to_string(R) + ", tokens * " +
                          std::to_string(cols) + "), got " + shape_text(y.sizes()));
        const int64_t tokens = cols ? y.size(1) / cols : 0;
        ar_rmsnorm_t p = {};
        norm_types(send, weight, "send", &p.dtype, &p.weight_dtype);
        if (p.dtype != integer(a[12]))
            throw Refused("send has dtype " + type_text(send.scalar_type()) + ", the comm another");
        const int64_t all[] = {R, R * y.size(1)};
        const void* from = block_of(send, integer(a[13]), all, send.scalar_type(), "send");
        const int64_t groups = norm_output(send, y, scale, group, cols, p.dtype, &p.out_dtype);
        const int64_t dev = send.get_device();
        const at::ScalarType type = send.scalar_type();
        const int64_t shape[] = {R, y.size(1)}, scales[] = {R, tokens * groups}, per[] = {R, tokens};
        p.eps = real(a[4]);
        p.rows = (size_t)tokens;
        p.cols = (size_t)cols;
        p.group = (size_t)group;
        p.weight = block_of(weight, dev, {cols}, weight.scalar_type(), "weight");
        p.y = block_of(y, dev, shape, y.scalar_type(), "y");
        if (residual)
            p.residual = block_of(*residual, dev, shape, type, "residual");
        if (sum)
            p.sum = block_of(*sum, dev, shape, type, "sum");
        if (scale)
            p.scale = static_cast<float*>(block_of(*scale, dev, scales, at::kFloat, "scale"));
        if (rstd)
            p.rstd = static_cast<float*>(block_of(*rstd, dev, per, at::kFloat, "rstd"));
        return status_of(p_reduce_scatter_rmsnorm, static_cast<ar_comm_t>(handle(a[0])), from, &p,
                         handle(a[10]));
    });
}

// rmsnorm_backward(dy, x, weight, rstd, dx, dweight, dsum, workspace, stream) -> status
PyObject* rmsnorm_backward(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        expect(n, 9);
        const at::Tensor &dy = tensor(a[0], "dy"), &x = tensor(a[1], "x"),
                         &weight = tensor(a[2], "weight"), &rstd = tensor(a[3], "rstd"),
                         &dx = tensor(a[4], "dx"), &dweight = tensor(a[5], "dweight"),
                         &workspace = tensor(a[7], "workspace");
        const at::Tensor* dsum = tensor_or_none(a[6], "dsum");
        if (x.dim() != 2 || dweight.dim() != 2)
            throw Refused("x must have shape (rows, cols) and dweight (ranks, cols)");
        const int64_t rows = x.size(0), cols = x.size(1), ranks = dweight.size(0);
        ar_rmsnorm_backward_t p = {};
        norm_types(x, weight, "x", &p.dtype, &p.weight_dtype);
        if (ranks < 1 || rows % ranks)
            throw Refused(std::to_string(rows) + " rows are not " + std::to_string(ranks) +
                          " equal shards");
        const int64_t dev = x.get_device();
        if (!workspace.is_cuda() || workspace.get_device() != dev || !workspace.is_contiguous())
            throw Refused("workspace must be a contiguous tensor on cuda:" + std::to_string(dev));
        const at::ScalarType type = x.scalar_type();
        const int64_t shape[] = {rows, cols}, wshape[] = {ranks, cols};
        p.ranks = ranks > 1 << 20 ? 1 << 20 : (int)ranks;  // refused all the same
        p.rows = (size_t)rows;
        p.cols = (size_t)cols;
        p.dy = rows_of(dy, dev, shape, type, "dy", &p.dy_stride);
        p.x = rows_of(x, dev, shape, type, "x", &p.x_stride);
        p.weight = block_of(weight, dev, {cols}, weight.scalar_type(), "weight");
        p.rstd = static_cast<float*>(block_of(rstd, dev, {rows}, at::kFloat, "rstd"));
        if (dsum)
            p.dsum = rows_of(*dsum, dev, shape, type, "dsum", &p.dsum_stride);
        p.dx = rows_of(dx, dev, shape, type, "dx", &p.dx_stride);
        p.dweight = static_cast<float*>(block_of(dweight, dev, wshape, at::kFloat, "dweight"));
        p.workspace = workspace.data_ptr();
        p.workspace_bytes = (size_t)workspace.nbytes();
        return status_of(p_rmsnorm_backward, &p, handle(a[8]));
    });
}

// Whether a tensor's elements fill one block of memory, in any order of its
// dimensions: smallest stride first, each is the product of the sizes before.
bool dense(const at::Tensor& t) { return t.is_non_overlapping_and_dense(); }

// spans(tensors, address, room) -> device index (-1: no tensors).  Fills the
// ar_span_t array at `address` from a list of tensors as they are now.
PyObject* spans(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        if (n != 3 || !PyList_Check(a[0]))
            throw Refused("wrong arguments");
        ar_span_t* to = static_cast<ar_span_t*>(handle(a[1]));
        const Py_ssize_t count = PyList_GET_SIZE(a[0]);
        if (count > integer(a[2]))
            throw Refused("the list has grown");
        int64_t device = -1;
        for (Py_ssize_t i = 0; i < count; ++i) {
            const at::Tensor& t = tensor(PyList_GET_ITEM(a[0], i), "a gradient");
            const auto which = [&] { return "tensor " + std::to_string(i); };
            const int dtype = code_of(t.scalar_type());
            if (dtype != AR_FLOAT32 && dtype != AR_BF16)
                throw Refused(which() + " has dtype " + type_text(t.scalar_type()) +
                              ": float32 or bfloat16 is wanted");
            if (!t.is_cuda() || (i && t.get_device() != device))
                throw Refused(which() + " is on " + t.device().str() + ": all must be on one GPU");
            if (!dense(t))
                throw Refused(which() + " is not dense in memory");
            device = t.get_device();
            to[i] = {t.data_ptr(), (size_t)t.numel(), dtype};
        }
        return PyLong_FromLongLong(device);
    });
}

// same_layout(tensors, tensors): equal types, shapes and strides, one by one.
PyObject* same_layout(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        if (n != 2 || !PyList_Check(a[0]) || !PyList_Check(a[1]))
            throw Refused("wrong arguments");
        const Py_ssize_t count = PyList_GET_SIZE(a[0]);
        if (count != PyList_GET_SIZE(a[1]))
            Py_RETURN_FALSE;
        for (Py_ssize_t i = 0; i < count; ++i) {
            const at::Tensor& s = tensor(PyList_GET_ITEM(a[0], i), "a gradient");
            const at::Tensor& t = tensor(PyList_GET_ITEM(a[1], i), "an output");
            if (s.scalar_type() != t.scalar_type() || s.sizes() != t.sizes() ||
                s.strides() != t.strides())
                Py_RETURN_FALSE;
        }
        Py_RETURN_TRUE;
    });
}

// dense(tensor)
PyObject* is_dense(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        if (n != 1)
            throw Refused("wrong number of arguments");
        return PyBool_FromLong(dense(tensor(a[0], "the argument")));
    });
}

#define METHOD(f) {#f, (PyCFunction)(void*)f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(init), METHOD(rmsnorm), METHOD(reduce_scatter_rmsnorm),
                         METHOD(rmsnorm_backward), METHOD(spans), METHOD(same_layout),
                         {"dense", (PyCFunction)(void*)is_dense, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
