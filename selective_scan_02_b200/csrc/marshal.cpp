// marshal.cpp -- the operators' Python calls (module _marshal): checks of torch tensors, outputs and workspaces
// that are not given, and one call of the C ABI of include/ss2d.h.  Nothing is computed here.
//
// The operators serve single tokens, where a call's time on the GPU is a few microseconds; the same checks and
// allocations made from Python take three times as long as the call.  Everything runs on the current stream of
// the tensors' device, which need not be the current device.
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/types.h>

#include <optional>
#include <string>

#include "ss2d.h"

namespace {

constexpr int64_t kBlock = 128;  // columns of one e4m3 scale

struct Refused {
    std::string what;
};

[[noreturn]] void refuse(const std::string &what) { throw Refused{what}; }

std::string shape_text(c10::IntArrayRef s)
{
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i)
        t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}

// A tensor argument; None gives an undefined tensor where `optional`.
at::Tensor tensor(PyObject *o, const char *name, bool optional = false)
{
    if (optional && o == Py_None)
        return {};
    if (!THPVariable_Check(o))
        refuse(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

at::ScalarType type_of(PyObject *o)
{
    if (!THPDtype_Check(o))
        refuse("out_dtype must be a torch.dtype");
    return reinterpret_cast<THPDtype *>(o)->scalar_type;
}

// The type code of float32, bfloat16 and (where `e4m3`) float8_e4m3fn.
int code_of(at::ScalarType t, const char *name, bool e4m3)
{
    if (t == at::kFloat)
        return SS2D_F32;
    if (t == at::kBFloat16)
        return SS2D_BF16;
    if (e4m3 && t == at::kFloat8_e4m3fn)
        return SS2D_E4M3;
    refuse(std::string(name) + (e4m3 ? " must be float32, bfloat16 or float8_e4m3fn" : " must be float32 or bfloat16"));
}

// The device and stream of one call.
struct Call {
    at::Device device;
    c10::cuda::CUDAGuard guard;
    cudaStream_t stream;

    static at::Device device_of(const at::Tensor &t)
    {
        if (!t.is_cuda())
            refuse("libss2d takes device tensors");
        return t.device();
    }
    explicit Call(const at::Tensor &t)
        : device(device_of(t)), guard(device), stream(c10::cuda::getCurrentCUDAStream(device.index()).stream())
    {
    }

    at::Tensor make(c10::IntArrayRef shape, at::ScalarType type) const
    {
        return at::Tensor(at::detail::empty_cuda(shape, type, device, std::nullopt));
    }
    void check(const at::Tensor &t, const char *name, at::ScalarType type, c10::IntArrayRef shape) const
    {
        if (t.device() != device)
            refuse(std::string(name) + " is on " + t.device().str() + ", not on " + device.str());
        if (t.scalar_type() != type)
            refuse(std::string(name) + " must be " + c10::toString(type) + ", not " + c10::toString(t.scalar_type()));
        if (t.sizes() != shape)
            refuse(std::string(name) + " must have shape " + shape_text(shape) + ", not " + shape_text(t.sizes()));
    }
    // The pointer of a dense tensor of this device, type and shape; of none, null.
    void *dense(const at::Tensor &t, const char *name, at::ScalarType type, c10::IntArrayRef shape) const
    {
        if (!t.defined())
            return nullptr;
        check(t, name, type, shape);
        if (!t.is_contiguous())
            refuse(std::string(name) + " must be contiguous");
        return t.data_ptr();
    }
    template <class T>
    T *dense(const at::Tensor &t, const char *name, at::ScalarType type, c10::IntArrayRef shape) const
    {
        return static_cast<T *>(dense(t, name, type, shape));
    }
    // Pointer and leading strides of a bf16 tensor with a dense last dimension.
    const void *strided(const at::Tensor &t, const char *name, c10::IntArrayRef shape, long long *strides) const
    {
        check(t, name, at::kBFloat16, shape);
        const size_t last = shape.size() - 1;
        if (shape[last] > 1 && t.stride(last) != 1)
            refuse(std::string("the last dimension of ") + name + " must be dense");
        for (size_t i = 0; i < last; ++i)
            strides[i] = t.stride(i);
        return t.data_ptr();
    }
    // A workspace of `need` bytes, or the given one (whose size the call checks).
    at::Tensor workspace(const at::Tensor &given, size_t need) const
    {
        if (!given.defined())
            return make({(int64_t)need}, at::kByte);
        if (given.device() != device || !given.is_contiguous())
            refuse("workspace must be a contiguous tensor on " + device.str());
        return given;
    }
};

int fit(int64_t n)
{
    if (n < 0 || n > 0x7fffffff)
        refuse("sizes must fit 32 bits");
    return (int)n;
}

at::DimVector with_last(c10::IntArrayRef shape, int64_t last)
{
    at::DimVector s(shape.begin(), shape.end());
    s.back() = last;
    return s;
}

// A call of the C ABI without the interpreter's lock, as ctypes makes the library's other calls: a launch waits where the
// queue of launches is full, and the status for its stream, while other threads (and the stream's host callbacks) go on.
template <class F>
int unlocked(const F &call)
{
    PyThreadState *const state = PyEval_SaveThread();
    const int status = call();
    PyEval_RestoreThread(state);
    return status;
}

// Python values of a call: the status where it is not SS2D_OK, else the tensors.
PyObject *result(int status, std::initializer_list<at::Tensor> tensors)
{
    if (status != SS2D_OK)
        return PyLong_FromLong(status);
    Py_ssize_t n = 0;
    for (const at::Tensor &t : tensors)
        n += t.defined();
    if (n == 1) {
        for (const at::Tensor &t : tensors)
            if (t.defined())
                return THPVariable_Wrap(t);
    }
    PyObject *all = PyTuple_New(n);
    if (!all)
        return nullptr;
    n = 0;
    for (const at::Tensor &t : tensors)
        if (t.defined())
            PyTuple_SET_ITEM(all, n++, THPVariable_Wrap(t));
    return all;
}

// rms_norm(x, weight, residual, eps, out_dtype, y, scales, residual_out)
PyObject *rms_norm(PyObject *const *a)
{
    const at::Tensor x = tensor(a[0], "x"), weight = tensor(a[1], "weight"), residual = tensor(a[2], "residual", true);
    const double eps = PyFloat_AsDouble(a[3]);
    if (PyErr_Occurred())
        return nullptr;
    at::Tensor y = tensor(a[5], "y", true), scales = tensor(a[6], "scales", true),
               residual_out = tensor(a[7], "residual_out", true);
    const Call c(x);
    if (x.dim() == 0)
        refuse("x must have a last dimension");
    const int64_t D = x.size(-1), rows = D ? x.numel() / D : 0;
    const int x_code = code_of(x.scalar_type(), "x", false);
    const void *xp = c.dense(x, "x", x.scalar_type(), x.sizes());
    const float *wp = c.dense<float>(weight, "weight", at::kFloat, {D});
    int r_code = 0;
    const void *rp = nullptr;
    void *rop = nullptr;
    if (residual.defined()) {
        r_code = code_of(residual.scalar_type(), "residual", false);
        rp = c.dense(residual, "residual", residual.scalar_type(), x.sizes());
        if (!residual_out.defined())
            residual_out = c.make(x.sizes(), residual.scalar_type());
        rop = c.dense(residual_out, "residual_out", residual.scalar_type(), x.sizes());
    } else if (residual_out.defined()) {
        refuse("residual_out is given without a residual");
    }
    const at::ScalarType type = y.defined() ? y.scalar_type() : type_of(a[4]);
    const int y_code = code_of(type, y.defined() ? "y" : "out_dtype", true);
    if (!y.defined())
        y = c.make(x.sizes(), type);
    void *yp = c.dense(y, "y", type, x.sizes());
    float *sp = nullptr;
    if (y_code == SS2D_E4M3) {
        const at::DimVector groups = with_last(x.sizes(), (D + kBlock - 1) / kBlock);
        if (!scales.defined())
            scales = c.make(groups, at::kFloat);
        sp = c.dense<float>(scales, "scales", at::kFloat, groups);
    } else if (scales.defined()) {
        refuse("scales is given without a float8_e4m3fn y");
    }
    const int columns = fit(D);
    const int status = unlocked(
        [&] { return ss2d_rms_norm(xp, x_code, rp, r_code, wp, (float)eps, yp, y_code, sp, rop, rows, columns, c.stream); });
    return result(status, {y, scales, residual_out});
}

// matmul_fp8(a, a_scales, w, w_scales, bias, out_dtype, out, workspace)
PyObject *matmul_fp8(PyObject *const *o)
{
    const at::Tensor a = tensor(o[0], "a"), a_scales = tensor(o[1], "a_scales"), w = tensor(o[2], "w"),
                     w_scales = tensor(o[3], "w_scales"), bias = tensor(o[4], "bias", true),
                     given = tensor(o[7], "workspace", true);
    at::Tensor out = tensor(o[6], "out", true);
    const Call c(a);
    if (a.dim() < 1 || w.dim() != 2)
        refuse("a must be (..., K) and w (N, K)");
    const int64_t K = a.size(-1), N = w.size(0), M = K ? a.numel() / K : 0;
    const int64_t kb = (K + kBlock - 1) / kBlock, nb = (N + kBlock - 1) / kBlock;
    const at::ScalarType type = out.defined() ? out.scalar_type() : type_of(o[5]);
    ss2d_matmul_fp8_args args{};
    args.struct_size = sizeof(args);
    args.M = fit(M);
    args.N = fit(N);
    args.K = fit(K);
    args.c_dtype = code_of(type, "out", false);
    args.a = c.dense(a, "a", at::kFloat8_e4m3fn, a.sizes());
    args.a_scales = c.dense<float>(a_scales, "a_scales", at::kFloat, with_last(a.sizes(), kb));
    args.w = c.dense(w, "w", at::kFloat8_e4m3fn, {N, K});
    args.w_scales = c.dense<float>(w_scales, "w_scales", at::kFloat, {nb, kb});
    args.bias = c.dense<float>(bias, "bias", at::kFloat, {N});
    const at::DimVector shape = with_last(a.sizes(), N);
    if (!out.defined())
        out = c.make(shape, type);
    args.c = c.dense(out, "out", type, shape);
    const size_t need = ss2d_matmul_fp8_workspace(&args);
    if (need == (size_t)-1)  // the call says what is wrong with its arguments
        return result(ss2d_matmul_fp8(&args, nullptr, 0, c.stream), {});
    const at::Tensor ws = c.workspace(given, need);
    return result(unlocked([&] { return ss2d_matmul_fp8(&args, ws.data_ptr(), ws.nbytes(), c.stream); }), {out});
}

void heads(const at::Tensor &q, const at::Tensor &v, int64_t dims, const char *shapes)
{
    if (q.dim() != dims || v.dim() != dims)
        refuse(std::string("q, k and v must be ") + shapes);
}

// linear_attention(q, k, v, log_decay, scale, h0, lengths, return_last_state, out, h_last, workspace)
PyObject *linear_attention(PyObject *const *o)
{
    const at::Tensor q = tensor(o[0], "q"), k = tensor(o[1], "k"), v = tensor(o[2], "v"),
                     log_decay = tensor(o[3], "log_decay"), h0 = tensor(o[5], "h0", true),
                     lengths = tensor(o[6], "lengths", true), given = tensor(o[10], "workspace", true);
    const double scale = PyFloat_AsDouble(o[4]);
    const int last_state = PyObject_IsTrue(o[7]);
    if (PyErr_Occurred())
        return nullptr;
    at::Tensor out = tensor(o[8], "out", true), h_last = tensor(o[9], "h_last", true);
    const Call c(q);
    heads(q, v, 4, "(B, L, G, Dk) and (B, L, H, Dv)");
    const int64_t B = q.size(0), L = q.size(1), G = q.size(2), Dk = q.size(3), H = v.size(2), Dv = v.size(3);
    ss2d_linear_attention_args args{};
    args.struct_size = sizeof(args);
    args.B = fit(B), args.L = fit(L), args.G = fit(G), args.H = fit(H), args.Dk = fit(Dk), args.Dv = fit(Dv);
    args.q = c.strided(q, "q", {B, L, G, Dk}, args.q_stride);
    args.k = c.strided(k, "k", {B, L, G, Dk}, args.k_stride);
    args.v = c.strided(v, "v", {B, L, H, Dv}, args.v_stride);
    args.decay_per_token = log_decay.dim() == 3;
    args.log_decay = args.decay_per_token ? c.dense<float>(log_decay, "log_decay", at::kFloat, {B, L, H})
                                          : c.dense<float>(log_decay, "log_decay", at::kFloat, {H});
    args.lengths = c.dense<int>(lengths, "lengths", at::kInt, {B});
    args.scale = (float)scale;
    args.h0 = c.dense<float>(h0, "h0", at::kFloat, {B, H, Dk, Dv});
    if (!h_last.defined() && last_state)
        h_last = c.make({B, H, Dk, Dv}, at::kFloat);
    args.h_last = c.dense<float>(h_last, "h_last", at::kFloat, {B, H, Dk, Dv});
    if (!out.defined())
        out = c.make({B, L, H, Dv}, at::kBFloat16);
    args.out = c.dense(out, "out", at::kBFloat16, {B, L, H, Dv});
    const size_t need = ss2d_linear_attention_workspace(&args);
    if (need == (size_t)-1)
        return result(ss2d_linear_attention(&args, nullptr, 0, c.stream), {});
    const at::Tensor ws = c.workspace(given, need);
    return result(unlocked([&] { return ss2d_linear_attention(&args, ws.data_ptr(), ws.nbytes(), c.stream); }), {out, h_last});
}

// linear_attention_step(q, k, v, log_decay, state, slots, scale, out)
PyObject *linear_attention_step(PyObject *const *o)
{
    const at::Tensor q = tensor(o[0], "q"), k = tensor(o[1], "k"), v = tensor(o[2], "v"),
                     log_decay = tensor(o[3], "log_decay"), state = tensor(o[4], "state"),
                     slots = tensor(o[5], "slots", true);
    const double scale = PyFloat_AsDouble(o[6]);
    if (PyErr_Occurred())
        return nullptr;
    at::Tensor out = tensor(o[7], "out", true);
    const Call c(q);
    heads(q, v, 3, "(B, G, Dk) and (B, H, Dv)");
    if (state.dim() != 4)
        refuse("state must be (pool, H, Dk, Dv)");
    const int64_t B = q.size(0), G = q.size(1), Dk = q.size(2), H = v.size(1), Dv = v.size(2), pool = state.size(0);
    ss2d_linear_attention_step_args args{};
    args.struct_size = sizeof(args);
    args.B = fit(B), args.pool = fit(pool), args.G = fit(G), args.H = fit(H), args.Dk = fit(Dk), args.Dv = fit(Dv);
    args.q = c.strided(q, "q", {B, G, Dk}, args.q_stride);
    args.k = c.strided(k, "k", {B, G, Dk}, args.k_stride);
    args.v = c.strided(v, "v", {B, H, Dv}, args.v_stride);
    args.decay_per_token = log_decay.dim() == 2;
    args.log_decay = args.decay_per_token ? c.dense<float>(log_decay, "log_decay", at::kFloat, {B, H})
                                          : c.dense<float>(log_decay, "log_decay", at::kFloat, {H});
    args.slots = c.dense<int>(slots, "slots", at::kInt, {B});
    args.scale = (float)scale;
    args.state = c.dense<float>(state, "state", at::kFloat, {pool, H, Dk, Dv});
    if (!out.defined())
        out = c.make({B, H, Dv}, at::kBFloat16);
    args.out = c.dense(out, "out", at::kBFloat16, {B, H, Dv});
    return result(unlocked([&] { return ss2d_linear_attention_step(&args, c.stream); }), {out});
}

// workspace_status(workspace)
PyObject *workspace_status(PyObject *const *o)
{
    const at::Tensor ws = tensor(o[0], "workspace");
    const Call c(ws);
    if (!ws.is_contiguous() || ws.nbytes() < sizeof(int))
        refuse("workspace must be a contiguous tensor that holds the error word (4 bytes)");
    return PyLong_FromLong(unlocked([&] { return ss2d_workspace_status(ws.data_ptr(), c.stream); }));
}

template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refused &e) {
        PyErr_SetString(PyExc_ValueError, e.what.c_str());
    } catch (const c10::OutOfMemoryError &e) {
        PyObject *cuda = PyImport_ImportModule("torch.cuda");
        PyObject *type = cuda ? PyObject_GetAttrString(cuda, "OutOfMemoryError") : nullptr;
        if (type)
            PyErr_SetString(type, e.what_without_backtrace());
        Py_XDECREF(type);
        Py_XDECREF(cuda);
    } catch (const c10::Error &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyMethodDef method(const char *name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<rms_norm, 8>("rms_norm"),
                         method<matmul_fp8, 8>("matmul_fp8"),
                         method<linear_attention, 11>("linear_attention"),
                         method<linear_attention_step, 8>("linear_attention_step"),
                         method<workspace_status, 1>("workspace_status"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
