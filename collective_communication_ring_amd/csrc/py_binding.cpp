// py_binding.cpp -- argument marshalling of the operators' torch wrappers
// (module _binding): checks tensors and fills in the C ABI's argument structs.
//
// A norm of one row takes 3 us on the GPU; reading five properties of each of
// six tensors took the wrapper as long in Python.  The C entry points are
// called by the addresses that init() and init_heads() are given, so they are
// those of the library that the package has loaded.  Nothing is kept from call to call.
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdint>
#include <exception>
#include <initializer_list>
#include <string>
#include <vector>

#include "ar.h"

namespace {

decltype(&ar_rmsnorm) p_rmsnorm = nullptr;
decltype(&ar_reduce_scatter_rmsnorm) p_reduce_scatter_rmsnorm = nullptr;
decltype(&ar_rmsnorm_backward) p_rmsnorm_backward = nullptr;
decltype(&ar_rotary) p_rotary = nullptr;
decltype(&ar_head_rmsnorm) p_head_rmsnorm = nullptr;
decltype(&ar_head_rmsnorm_backward) p_head_rmsnorm_backward = nullptr;
decltype(&ar_orthogonalize) p_orthogonalize = nullptr;

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

// An entry point's status.  The tensors' GPU is the current one during the call: a
// default stream's handle is 0 on every GPU and stands for the current one's.  Other
// Python threads run meanwhile: a launch may have to wait for room in its stream's
// queue.
template <class F, class... Args>
PyObject* status_of(int64_t device, F entry, Args... args)
{
    int rc = 0;
    const c10::DeviceGuard on(c10::Device(c10::DeviceType::CUDA, (c10::DeviceIndex)device));
    Py_BEGIN_ALLOW_THREADS
    rc = entry(args...);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

void expect(Py_ssize_t got, Py_ssize_t want, bool given = p_rmsnorm)
{
    if (got != want)
        throw Refused("wrong number of arguments");
    if (!given)
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

// init_heads(ar_rotary, ar_head_rmsnorm, ar_head_rmsnorm_backward, ar_orthogonalize): addresses.
PyObject* init_heads(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        if (n != 4)
            throw Refused("wrong number of arguments");
        p_rotary = reinterpret_cast<decltype(p_rotary)>(handle(a[0]));
        p_head_rmsnorm = reinterpret_cast<decltype(p_head_rmsnorm)>(handle(a[1]));
        p_head_rmsnorm_backward = reinterpret_cast<decltype(p_head_rmsnorm_backward)>(handle(a[2]));
        p_orthogonalize = reinterpret_cast<decltype(p_orthogonalize)>(handle(a[3]));
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
        return status_of(dev, p_rmsnorm, &p, handle(a[9]));
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
        return status_of(dev, p_reduce_scatter_rmsnorm, static_cast<ar_comm_t>(handle(a[0])), from, &p,
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
        return status_of(dev, p_rmsnorm_backward, &p, handle(a[8]));
    });
}

// ---- attention heads -----------------------------------------------------------

// What a call's arrays of heads have in common: [batch, tokens, heads, dim], or
// [tokens, heads, dim].
struct HeadShape {
    int64_t device, batch, tokens, dim;
    at::ScalarType type;
    bool three;
};

HeadShape head_shape(const at::Tensor& q, int* dtype)
{
    *dtype = code_of(q.scalar_type());
    if (*dtype != AR_FLOAT32 && *dtype != AR_BF16)
        throw Refused("q has dtype " + type_text(q.scalar_type()) +
                      ": float32 or bfloat16 is wanted");
    if (!q.is_cuda())
        throw Refused("q must be on the GPU");
    if (q.dim() != 3 && q.dim() != 4)
        throw Refused("q must have shape ([batch,] tokens, heads, dim), got " + shape_text(q.sizes()));
    const bool three = q.dim() == 3;
    return {q.get_device(), three ? 1 : q.size(0), q.size(three ? 0 : 1), q.size(three ? 2 : 3),
            q.scalar_type(), three};
}

// An array of `heads` heads (-1: as many as it has, which are returned).
int64_t heads_of(const at::Tensor& t, const HeadShape& s, int64_t heads, const char* what,
                 ar_heads_t* out)
{
    const int64_t d = s.three ? 3 : 4;
    if (t.dim() == d && heads < 0)
        heads = t.size(d - 2);
    const int64_t four[] = {s.batch, s.tokens, heads, s.dim};
    check(t, s.device, s.three ? at::IntArrayRef(four + 1, 3) : at::IntArrayRef(four, 4), s.type, what);
    if (s.dim > 1 && t.stride(d - 1) != 1)
        throw Refused(std::string("the last dimension of ") + what + " must be contiguous");
    *out = {t.data_ptr(), s.three ? 0 : (size_t)t.stride(0), (size_t)t.stride(d - 3),
            (size_t)t.stride(d - 2)};
    return heads;
}

// positions, frequencies (None: no rotation), layout, factor
void rotation_of(PyObject* const* a, const HeadShape& s, ar_rotation_t* r)
{
    const at::Tensor *positions = tensor_or_none(a[0], "positions"),
                     *frequencies = tensor_or_none(a[1], "frequencies");
    if (!frequencies && !positions)
        return;
    if (!frequencies || !positions)
        throw Refused("a rotation needs positions and frequencies");
    if (frequencies->dim() != 1)
        throw Refused("frequencies must have shape (rot_dim / 2,), got " +
                      shape_text(frequencies->sizes()));
    r->frequencies = static_cast<const double*>(block_of(
        *frequencies, s.device, frequencies->sizes(), at::kDouble, "the rotation's frequencies"));
    r->rot_dim = 2 * (size_t)frequencies->size(0);
    r->layout = (int)integer(a[2]);
    r->factor = real(a[3]);
    const at::ScalarType type = positions->scalar_type();
    if (type != at::kInt && type != at::kLong)
        throw Refused("positions have dtype " + type_text(type) + ": int32 or int64 is wanted");
    r->position_bytes = type == at::kInt ? 4 : 8;
    const bool shared = positions->dim() == 1;
    const int64_t two[] = {s.batch, s.tokens};
    check(*positions, s.device, shared ? at::IntArrayRef(two + 1, 1) : at::IntArrayRef(two, 2), type,
          "positions");
    if (s.tokens > 1 && positions->stride(shared ? 0 : 1) != 1)
        throw Refused("the last dimension of positions must be contiguous");
    r->positions = positions->data_ptr();
    r->position_stride = shared || s.batch == 1 ? 0 : (size_t)positions->stride(0);
}

const void* head_weight(PyObject* o, const HeadShape& s, const char* what, int* weight_dtype)
{
    const at::Tensor& w = tensor(o, what);
    const int code = code_of(w.scalar_type());
    if ((code != AR_FLOAT32 && w.scalar_type() != s.type) || (*weight_dtype >= 0 && code != *weight_dtype))
        throw Refused(std::string(what) + " has dtype " + type_text(w.scalar_type()) + ": " +
                      (*weight_dtype >= 0 ? "that of q_weight" : type_text(s.type) + " or torch.float32") +
                      " is wanted");
    *weight_dtype = code;
    return block_of(w, s.device, {s.dim}, w.scalar_type(), what);
}

// The keys' arguments come all together or not at all.
bool all_or_none(PyObject* const* a, std::initializer_list<int> which, const char* names)
{
    int given = 0;
    for (int i : which)
        given += a[i] != Py_None;
    if (given && given != (int)which.size())
        throw Refused(std::string("the keys need all of ") + names);
    return given;
}

// rotary(q, q_out, k, k_out, positions, frequencies, layout, factor, inverse, stream) -> status
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        expect(n, 10, p_rotary);
        ar_rotary_t p = {};
        const at::Tensor& q = tensor(a[0], "q");
        const HeadShape s = head_shape(q, &p.dtype);
        p.batch = (size_t)s.batch;
        p.tokens = (size_t)s.tokens;
        p.dim = (size_t)s.dim;
        p.q_heads = (size_t)heads_of(q, s, -1, "q", &p.q);
        heads_of(tensor(a[1], "q_out"), s, (int64_t)p.q_heads, "q_out", &p.q_out);
        if (all_or_none(a, {2, 3}, "k and k_out")) {
            p.k_heads = (size_t)heads_of(tensor(a[2], "k"), s, -1, "k", &p.k);
            heads_of(tensor(a[3], "k_out"), s, (int64_t)p.k_heads, "k_out", &p.k_out);
        }
        rotation_of(a + 4, s, &p.rotation);
        p.inverse = (int)integer(a[8]);
        return status_of(s.device, p_rotary, &p, handle(a[9]));
    });
}

// head_rmsnorm(q, q_weight, q_out, eps, k, k_weight, k_out, positions, frequencies, layout, factor,
// stream) -> status
PyObject* head_rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        expect(n, 12, p_head_rmsnorm);
        ar_head_rmsnorm_t p = {};
        const at::Tensor& q = tensor(a[0], "q");
        const HeadShape s = head_shape(q, &p.dtype);
        p.weight_dtype = -1;
        p.eps = real(a[3]);
        p.batch = (size_t)s.batch;
        p.tokens = (size_t)s.tokens;
        p.dim = (size_t)s.dim;
        p.q_heads = (size_t)heads_of(q, s, -1, "q", &p.q);
        p.q_weight = head_weight(a[1], s, "q_weight", &p.weight_dtype);
        heads_of(tensor(a[2], "q_out"), s, (int64_t)p.q_heads, "q_out", &p.q_out);
        if (all_or_none(a, {4, 5, 6}, "k, k_weight and k_out")) {
            p.k_heads = (size_t)heads_of(tensor(a[4], "k"), s, -1, "k", &p.k);
            p.k_weight = head_weight(a[5], s, "k_weight", &p.weight_dtype);
            heads_of(tensor(a[6], "k_out"), s, (int64_t)p.k_heads, "k_out", &p.k_out);
        }
        rotation_of(a + 7, s, &p.rotation);
        return status_of(s.device, p_head_rmsnorm, &p, handle(a[11]));
    });
}

// head_rmsnorm_backward(dq_out, q, q_weight, dq, q_dweight, eps, dk_out, k, k_weight, dk, k_dweight,
// positions, frequencies, layout, factor, workspace, stream) -> status
PyObject* head_rmsnorm_backward(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        expect(n, 17, p_head_rmsnorm_backward);
        ar_head_rmsnorm_backward_t p = {};
        const at::Tensor &q = tensor(a[1], "q"), &q_dweight = tensor(a[4], "q_dweight"),
                         &workspace = tensor(a[15], "workspace");
        const HeadShape s = head_shape(q, &p.dtype);
        if (q_dweight.dim() != 2)
            throw Refused("q_dweight must have shape (ranks, dim), got " + shape_text(q_dweight.sizes()));
        const int64_t ranks = q_dweight.size(0), shape[] = {ranks, s.dim};
        if (ranks < 1 || s.batch % ranks)
            throw Refused(std::to_string(s.batch) + " batches are not " + std::to_string(ranks) +
                          " equal shards");
        p.ranks = ranks > 1 << 20 ? 1 << 20 : (int)ranks;  // refused all the same
        p.weight_dtype = -1;
        p.eps = real(a[5]);
        p.batch = (size_t)s.batch;
        p.tokens = (size_t)s.tokens;
        p.dim = (size_t)s.dim;
        p.q_heads = (size_t)heads_of(q, s, -1, "q", &p.q);
        heads_of(tensor(a[0], "dq_out"), s, (int64_t)p.q_heads, "dq_out", &p.dq_out);
        heads_of(tensor(a[3], "dq"), s, (int64_t)p.q_heads, "dq", &p.dq);
        p.q_weight = head_weight(a[2], s, "q_weight", &p.weight_dtype);
        p.q_dweight = static_cast<float*>(block_of(q_dweight, s.device, shape, at::kFloat, "q_dweight"));
        if (all_or_none(a, {6, 7, 8, 9, 10}, "dk_out, k, k_weight, dk and k_dweight")) {
            p.k_heads = (size_t)heads_of(tensor(a[7], "k"), s, -1, "k", &p.k);
            heads_of(tensor(a[6], "dk_out"), s, (int64_t)p.k_heads, "dk_out", &p.dk_out);
            heads_of(tensor(a[9], "dk"), s, (int64_t)p.k_heads, "dk", &p.dk);
            p.k_weight = head_weight(a[8], s, "k_weight", &p.weight_dtype);
            p.k_dweight = static_cast<float*>(
                block_of(tensor(a[10], "k_dweight"), s.device, shape, at::kFloat, "k_dweight"));
        }
        rotation_of(a + 11, s, &p.rotation);
        if (!workspace.is_cuda() || workspace.get_device() != s.device || !workspace.is_contiguous())
            throw Refused("workspace must be a contiguous tensor on cuda:" + std::to_string(s.device));
        p.workspace = workspace.data_ptr();
        p.workspace_bytes = (size_t)workspace.nbytes();
        return status_of(s.device, p_head_rmsnorm_backward, &p, handle(a[16]));
    });
}

// How many matrices a list of them, or a tensor [count, rows, cols] or [rows, cols], holds.
Py_ssize_t matrix_count(PyObject* o, const char* what)
{
    if (PyList_Check(o))
        return PyList_GET_SIZE(o);
    const at::Tensor& t = tensor(o, what);
    return t.dim() == 3 ? (Py_ssize_t)t.size(0) : 1;
}

// Their addresses, and the distance of their rows.
template <class P>
void matrices_of(PyObject* o, int64_t device, const int64_t (&shape)[2], at::ScalarType type,
                 const char* what, std::vector<P>* at, size_t* stride)
{
    if (!PyList_Check(o)) {
        const at::Tensor& t = tensor(o, what);
        if (t.dim() != 3) {
            (*at)[0] = rows_of(t, device, shape, type, what, stride);
            return;
        }
        const int64_t all[] = {(int64_t)at->size(), shape[0], shape[1]};
        check(t, device, all, type, what);
        if (t.stride(2) != 1 && shape[1] > 1)
            throw Refused(std::string("the last dimension of ") + what + " must be contiguous");
        *stride = (size_t)t.stride(1);
        for (size_t i = 0; i < at->size(); ++i)
            (*at)[i] = static_cast<char*>(t.data_ptr()) + i * (size_t)t.stride(0) * t.element_size();
        return;
    }
    for (size_t i = 0; i < at->size(); ++i) {
        size_t own = 0;
        (*at)[i] = rows_of(tensor(PyList_GET_ITEM(o, (Py_ssize_t)i), what), device, shape, type, what, &own);
        if (i && shape[0] > 1 && own != *stride)
            throw Refused(std::string("the rows of all of ") + what + " must be equally far apart");
        *stride = own;
    }
}

// orthogonalize(x, y, coefficients, eps, scale, workspace, stream) -> status; x and y are lists of
// matrices, or tensors [count, rows, cols] or [rows, cols]; coefficients a list of 3 numbers for
// each step
PyObject* orthogonalize(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        expect(n, 7, p_orthogonalize);
        if (!PyList_Check(a[2]))
            throw Refused("wrong arguments");
        const Py_ssize_t count = matrix_count(a[0], "x");
        if (!count || matrix_count(a[1], "y") != count)
            throw Refused("x and y must be as many matrices, one at least");
        ar_orthogonalize_t p = {};
        const at::Tensor &x0 = tensor(PyList_Check(a[0]) ? PyList_GET_ITEM(a[0], 0) : a[0], "x"),
                         &workspace = tensor(a[5], "workspace");
        const at::ScalarType type = x0.scalar_type();
        p.dtype = code_of(type);
        if (p.dtype != AR_FLOAT32 && p.dtype != AR_BF16)
            throw Refused("x has dtype " + type_text(type) + ": float32 or bfloat16 is wanted");
        if (!x0.is_cuda())
            throw Refused("x must be on the GPU");
        const int64_t d = x0.dim();
        if (d != 2 && (d != 3 || PyList_Check(a[0])))
            throw Refused("a matrix must have shape (rows, cols), got " + shape_text(x0.sizes()));
        const int64_t dev = x0.get_device(), rows = x0.size(d - 2), cols = x0.size(d - 1);
        const int64_t shape[] = {rows, cols};
        std::vector<const void*> x((size_t)count);
        std::vector<void*> y((size_t)count);
        matrices_of(a[0], dev, shape, type, "x", &x, &p.x_stride);
        matrices_of(a[1], dev, shape, type, "y", &y, &p.out_stride);
        const Py_ssize_t numbers = PyList_GET_SIZE(a[2]);
        if (numbers % 3)
            throw Refused("each step has three coefficients");
        std::vector<float> coefficients((size_t)numbers);
        for (Py_ssize_t i = 0; i < numbers; ++i)
            coefficients[(size_t)i] = real(PyList_GET_ITEM(a[2], i));
        if (!workspace.is_cuda() || workspace.get_device() != dev || !workspace.is_contiguous())
            throw Refused("workspace must be a contiguous tensor on cuda:" + std::to_string(dev));
        p.steps = (int)std::min<Py_ssize_t>(numbers / 3, 1 << 20);
        p.eps = real(a[3]);
        p.scale = real(a[4]);
        p.count = (size_t)count;
        p.rows = (size_t)rows;
        p.cols = (size_t)cols;
        p.x = x.data();
        p.out = y.data();
        p.coefficients = coefficients.data();
        p.workspace = workspace.data_ptr();
        p.workspace_bytes = (size_t)workspace.nbytes();
        return status_of(dev, p_orthogonalize, &p, handle(a[6]));
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
PyMethodDef methods[] = {METHOD(init), METHOD(init_heads), METHOD(rmsnorm), METHOD(reduce_scatter_rmsnorm),
                         METHOD(rmsnorm_backward), METHOD(rotary), METHOD(head_rmsnorm),
                         METHOD(head_rmsnorm_backward), METHOD(orthogonalize), METHOD(spans),
                         METHOD(same_layout),
                         {"dense", (PyCFunction)(void*)is_dense, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
