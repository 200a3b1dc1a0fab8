// The Python binding of the training-step operators: looks each tensor over and
// calls the C entry point, whose status it returns.
//
// Argument marshalling only, like the rest of the binding, but in C++: the
// smallest calls run for 2 to 4 us on the GPU, and through ctypes and tensor
// attributes the checks alone took 4 to 7 us of host time a call (layer norm
// forward 7.9 us in all, gradient norm 5.5).
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAStream.h>

#include <cstdarg>
#include <cstdio>
#include <exception>

#include "fc.h"

namespace {

decltype(&fc_grad_norm) p_grad_norm;
decltype(&fc_adamw_step) p_adamw_step;
decltype(&fc_adamw8_step) p_adamw8_step;
decltype(&fc_layernorm_forward) p_layernorm_forward;
decltype(&fc_layernorm_backward) p_layernorm_backward;

// Thrown with a Python error set.
struct Refused {};

[[noreturn]] void refuse(const char *fmt, ...)
{
    char text[256];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(text, sizeof(text), fmt, ap);
    va_end(ap);
    PyErr_SetString(PyExc_ValueError, text);
    throw Refused{};
}

const at::Tensor *tensor(PyObject *o, const char *name)
{
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse("%s must be a tensor", name);
    return &THPVariable_Unpack(o);
}

const at::Tensor &needed(PyObject *o, const char *name)
{
    const at::Tensor *t = tensor(o, name);
    if (!t) refuse("%s must be a tensor", name);
    return *t;
}

void on_gpu(const at::Tensor &t, int dev, const char *name)
{
    if (!t.is_cuda() || t.get_device() != dev)
        refuse("%s must be on the GPU of the other tensors, not on %s", name,
               t.device().str().c_str());
}

int type_of(at::ScalarType s)
{
    switch (s) {
    case at::kFloat: return FC_TYPE_F32;
    case at::kHalf: return FC_TYPE_F16;
    case at::kBFloat16: return FC_TYPE_BF16;
    default: return -1;
    }
}

int type_of(const at::Tensor &t, const char *name)
{
    const int kind = type_of(t.scalar_type());
    if (kind < 0)
        refuse("%s must be float32, float16 or bfloat16, not %s", name,
               c10::toString(t.scalar_type()));
    return kind;
}

// Address of a contiguous tensor of n elements of type a, b or c (null stays).
void *flat(PyObject *o, int64_t n, const char *name, int dev, at::ScalarType a,
           at::ScalarType b = at::ScalarType::Undefined,
           at::ScalarType c = at::ScalarType::Undefined)
{
    const at::Tensor *t = tensor(o, name);
    if (!t) return nullptr;
    on_gpu(*t, dev, name);
    if (t->numel() != n || !t->is_contiguous())
        refuse("%s must be contiguous with %lld elements", name, (long long)n);
    const at::ScalarType s = t->scalar_type();
    if (s != a && s != b && s != c) refuse("%s must not be %s", name, c10::toString(s));
    return t->data_ptr();
}

float *flat32(PyObject *o, int64_t n, const char *name, int dev)
{
    return static_cast<float *>(flat(o, n, name, dev, at::kFloat));
}

// Address of a matrix like x with contiguous rows, and the elements between them.
void *matrix(const at::Tensor &t, const at::Tensor &x, const char *name, int dev, int64_t *ld)
{
    on_gpu(t, dev, name);
    if (t.dim() != 2 || t.scalar_type() != x.scalar_type() || t.size(0) != x.size(0) ||
        t.size(1) != x.size(1))
        refuse("%s must be of two dimensions, of the shape and type of x", name);
    if (t.size(1) > 1 && t.stride(1) != 1) refuse("the rows of %s must be contiguous", name);
    // the stride of a single row says nothing
    *ld = t.size(0) > 1 ? t.stride(0) : t.size(1);
    return t.data_ptr();
}

// Scratch of any type: its bytes are its elements', one after another.
void *scratch(const at::Tensor &t, int dev)
{
    on_gpu(t, dev, "workspace");
    if (!t.is_contiguous()) refuse("workspace must be contiguous");
    return t.data_ptr();
}

int64_t integer(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    return v;
}

double number(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{};
    return v;
}

// An integer, or None for the current stream of the GPU.
void *stream(PyObject *o, int dev)
{
    if (o == Py_None)
        return (void *)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    return (void *)(intptr_t)integer(o);
}

// What a table of layers carries: (pointers, type, layers, sizes, decay, N, device),
// the arrays as addresses.
struct Layers {
    const void *const *grads;
    int32_t type, L;
    const int64_t *sizes;
    const float *decay;
    int64_t N;
    int dev;

    explicit Layers(PyObject *o)
    {
        if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 7) refuse("not a table of layers");
        grads = (const void *const *)(intptr_t)integer(PyTuple_GET_ITEM(o, 0));
        type = (int32_t)integer(PyTuple_GET_ITEM(o, 1));
        L = (int32_t)integer(PyTuple_GET_ITEM(o, 2));
        sizes = (const int64_t *)(intptr_t)integer(PyTuple_GET_ITEM(o, 3));
        decay = (const float *)(intptr_t)integer(PyTuple_GET_ITEM(o, 4));
        N = integer(PyTuple_GET_ITEM(o, 5));
        dev = (int)integer(PyTuple_GET_ITEM(o, 6));
    }
};

// Runs f(args) and turns what it throws into a Python error.
template <class F>
PyObject *call(PyObject *const *args, Py_ssize_t n, Py_ssize_t want, F f)
{
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, %zd wanted", n, want);
        return nullptr;
    }
    try {
        return PyLong_FromLong((long)f(args));
    } catch (const Refused &) {
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
        return nullptr;
    }
}

// layers, loss_scale, max_norm, norm, scale, workspace, stream
PyObject *grad_norm(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return call(args, n, 7, [](PyObject *const *a) {
        const Layers l(a[0]);
        const at::Tensor &ws = needed(a[5], "workspace");
        void *const p = scratch(ws, l.dev);
        return p_grad_norm(l.grads, l.type, l.L, l.sizes, (float)number(a[1]),
                           (float)number(a[2]), flat32(a[3], 1, "norm", l.dev),
                           flat32(a[4], 1, "scale", l.dev), p, ws.nbytes(),
                           stream(a[6], l.dev));
    });
}

int32_t low_type(PyObject *o)
{
    return o == Py_None ? 0 : type_of(THPVariable_Unpack(o).scalar_type());
}

// layers, grad_scale, lr, beta1, beta2, eps, weight_decay, weights, weights_low,
// exp_avg, exp_avg_sq, steps, stream
PyObject *adamw_step(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return call(args, n, 13, [](PyObject *const *a) {
        const Layers l(a[0]);
        const float *scale = flat32(a[1], 1, "grad_scale", l.dev);
        float *w = flat32(a[7], l.N, "weights", l.dev);
        void *low = flat(a[8], l.N, "weights_low", l.dev, at::kHalf, at::kBFloat16);
        return p_adamw_step(l.grads, l.type, l.L, l.sizes, l.decay, scale, number(a[2]),
                            number(a[3]), number(a[4]), number(a[5]), number(a[6]), w, low,
                            low_type(a[8]), flat32(a[9], l.N, "exp_avg", l.dev),
                            flat32(a[10], l.N, "exp_avg_sq", l.dev),
                            (int32_t *)flat(a[11], 2, "steps", l.dev, at::kInt),
                            stream(a[12], l.dev));
    });
}

// An e4m3 state has N elements, or fills its last block.
void *codes(PyObject *o, int64_t N, int64_t whole, const char *name, int dev)
{
    const at::Tensor &t = needed(o, name);
    return flat(o, t.numel() == N ? N : whole, name, dev, at::kFloat8_e4m3fn);
}

// layers, grad_scale, lr, beta1, beta2, eps, weight_decay, weights, weights_low,
// exp_avg_q, exp_avg_scale, exp_rms_q, exp_rms_scale, steps, seed, stream
PyObject *adamw8_step(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return call(args, n, 16, [](PyObject *const *a) {
        const Layers l(a[0]);
        const int64_t blocks = (l.N + FC_STATE_BLOCK - 1) / FC_STATE_BLOCK;
        const int64_t whole = blocks * FC_STATE_BLOCK;
        const float *scale = flat32(a[1], 1, "grad_scale", l.dev);
        float *w = flat32(a[7], l.N, "weights", l.dev);
        void *low = flat(a[8], l.N, "weights_low", l.dev, at::kHalf, at::kBFloat16);
        const uint64_t seed = PyLong_AsUnsignedLongLongMask(a[14]);
        if (PyErr_Occurred()) throw Refused{};
        return p_adamw8_step(l.grads, l.type, l.L, l.sizes, l.decay, scale, number(a[2]),
                             number(a[3]), number(a[4]), number(a[5]), number(a[6]), w, low,
                             low_type(a[8]), codes(a[9], l.N, whole, "exp_avg_q", l.dev),
                             flat32(a[10], blocks, "exp_avg_scale", l.dev),
                             codes(a[11], l.N, whole, "exp_rms_q", l.dev),
                             flat32(a[12], blocks, "exp_rms_scale", l.dev),
                             (int32_t *)flat(a[13], 2, "steps", l.dev, at::kInt), seed,
                             stream(a[15], l.dev));
    });
}

// The matrix x: its GPU, shape and type.
struct Rows {
    const at::Tensor &x;
    int dev, type;
    int64_t rows, cols, ld;
    void *p;

    explicit Rows(PyObject *o) : x(needed(o, "x"))
    {
        if (x.dim() != 2) refuse("x must have two dimensions, not %d", (int)x.dim());
        type = type_of(x, "x");
        if (!x.is_cuda()) refuse("x must be on a GPU, not on %s", x.device().str().c_str());
        dev = (int)x.get_device();
        rows = x.size(0);
        cols = x.size(1);
        p = matrix(x, x, "x", dev, &ld);
    }
};

// x, weight, bias, eps, y, mean, rstd, stream
PyObject *layernorm_forward(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return call(args, n, 8, [](PyObject *const *a) {
        const Rows x(a[0]);
        int64_t ldy;
        void *y = matrix(needed(a[4], "y"), x.x, "y", x.dev, &ldy);
        const at::ScalarType own = x.x.scalar_type();
        const void *w = flat(a[1], x.cols, "weight", x.dev, at::kFloat, own);
        const void *b = flat(a[2], x.cols, "bias", x.dev, at::kFloat, own);
        int ptype = FC_TYPE_F32;
        if (w || a[1] != Py_None) ptype = type_of(THPVariable_Unpack(a[1]).scalar_type());
        if (a[2] != Py_None) {
            const int kind = type_of(THPVariable_Unpack(a[2]).scalar_type());
            if (a[1] != Py_None && kind != ptype) refuse("weight and bias must have one type");
            ptype = kind;
        }
        return p_layernorm_forward(x.p, x.rows, x.cols, x.ld, x.type, w, b, ptype,
                                   (float)number(a[3]), y, ldy,
                                   flat32(a[5], x.rows, "mean", x.dev),
                                   flat32(a[6], x.rows, "rstd", x.dev), stream(a[7], x.dev));
    });
}

// dy, x, weight, mean, rstd, dx, dweight, dbias, workspace, stream
PyObject *layernorm_backward(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return call(args, n, 10, [](PyObject *const *a) {
        const Rows x(a[1]);
        int64_t lddy, lddx;
        void *dy = matrix(needed(a[0], "dy"), x.x, "dy", x.dev, &lddy);
        void *dx = matrix(needed(a[5], "dx"), x.x, "dx", x.dev, &lddx);
        const void *w = flat(a[2], x.cols, "weight", x.dev, at::kFloat, x.x.scalar_type());
        const int ptype = a[2] == Py_None ? FC_TYPE_F32
                                          : type_of(THPVariable_Unpack(a[2]).scalar_type());
        void *dw = flat(a[6], x.cols, "dweight", x.dev, at::kFloat, at::kHalf, at::kBFloat16);
        void *db = flat(a[7], x.cols, "dbias", x.dev, at::kFloat, at::kHalf, at::kBFloat16);
        int gtype = FC_TYPE_F32;
        if (a[6] != Py_None) gtype = type_of(THPVariable_Unpack(a[6]).scalar_type());
        if (a[7] != Py_None) {
            const int kind = type_of(THPVariable_Unpack(a[7]).scalar_type());
            if (a[6] != Py_None && kind != gtype) refuse("dweight and dbias must have one type");
            gtype = kind;
        }
        const at::Tensor *ws = tensor(a[8], "workspace");
        void *const p = ws ? scratch(*ws, x.dev) : nullptr;
        return p_layernorm_backward(dy, lddy, x.p, x.ld, x.type, w, ptype,
                                    flat32(a[3], x.rows, "mean", x.dev),
                                    flat32(a[4], x.rows, "rstd", x.dev), x.rows, x.cols, dx,
                                    lddx, dw, db, gtype, p, ws ? ws->nbytes() : 0, stream(a[9], x.dev));
    });
}

// The addresses of the five C entry points, in the order of the pointers above.
PyObject *connect(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return call(args, n, 5, [](PyObject *const *a) {
        p_grad_norm = (decltype(p_grad_norm))(intptr_t)integer(a[0]);
        p_adamw_step = (decltype(p_adamw_step))(intptr_t)integer(a[1]);
        p_adamw8_step = (decltype(p_adamw8_step))(intptr_t)integer(a[2]);
        p_layernorm_forward = (decltype(p_layernorm_forward))(intptr_t)integer(a[3]);
        p_layernorm_backward = (decltype(p_layernorm_backward))(intptr_t)integer(a[4]);
        return 0;
    });
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(connect),           METHOD(grad_norm),
                         METHOD(adamw_step),        METHOD(adamw8_step),
                         METHOD(layernorm_forward), METHOD(layernorm_backward),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef definition = {PyModuleDef_HEAD_INIT, "_fcbind", nullptr, -1, methods,
                          nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__fcbind()
{
    return PyModule_Create(&definition);
}
