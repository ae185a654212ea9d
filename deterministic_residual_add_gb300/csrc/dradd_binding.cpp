// dradd_binding.cpp -- the Python binding of include/dradd_train.h and
// include/dradd_linear.h: checks of tensors, allocation of outputs, and the
// call, in one C function each.
//
// A decode step's kernels take two or three microseconds.  With the same
// checks and allocations in Python, a call through ctypes took 15 to 40 us on
// the GPU's host (rotation of 8 tokens 15.7, the norm + rotation gradient
// 39); from here 5.1 and 12.8.  The functions take every argument by
// position; train.py and linear.py give them their names, defaults and
// documentation.
#include <Python.h>

#include <cstdint>
#include <initializer_list>
#include <sstream>
#include <string>
#include <vector>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "dradd_linear.h"
#include "dradd_train.h"

namespace {

// Thrown with the Python error already set.
struct ErrorSet {};

[[noreturn]] void fail(PyObject* type, const std::string& what)
{
    PyErr_SetString(type, what.c_str());
    throw ErrorSet{};
}

// The interpreter's lock is free while one lives: a launch or an allocation
// may wait for the device, and the device for a host function in the
// interpreter.
struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

// Makes a call into the library; `f` must not touch Python.
template <typename F>
void run(const char* where, F f)
{
    dradd_status status;
    {
        const Unlocked unlocked;
        status = f();
    }
    if (status == DRADD_OK)
        return;
    PyObject* package = PyImport_ImportModule("deterministic_residual_add_gb300");
    PyObject* type = package ? PyObject_GetAttrString(package, "DraddError") : nullptr;
    PyObject* error = type ? PyObject_CallFunction(type, "is", status, where) : nullptr;
    if (error)
        PyErr_SetObject(type, error);
    Py_XDECREF(error);
    Py_XDECREF(type);
    Py_XDECREF(package);
    throw ErrorSet{};
}

// ---------------------------------------------------------------- arguments
// A tensor, or null for None.
const at::Tensor* optional_tensor(PyObject* o, const char* name)
{
    if (o == Py_None)
        return nullptr;
    if (!THPVariable_Check(o))
        fail(PyExc_TypeError, std::string(name) + " must be a tensor (got " + Py_TYPE(o)->tp_name + ")");
    return &THPVariable_Unpack(o);
}

const at::Tensor& tensor(PyObject* o, const char* name)
{
    const at::Tensor* t = optional_tensor(o, name);
    if (!t)
        fail(PyExc_TypeError, std::string(name) + " must be a tensor (got None)");
    return *t;
}

double number(PyObject* o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw ErrorSet{};
    return v;
}

uint64_t bits64(PyObject* o)
{
    const unsigned long long v = PyLong_AsUnsignedLongLongMask(o);
    if (v == static_cast<unsigned long long>(-1) && PyErr_Occurred())
        throw ErrorSet{};
    return v;
}

bool truth(PyObject* o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0)
        throw ErrorSet{};
    return v != 0;
}

// The call's type and device, those of its leading tensor.
struct Call {
    at::ScalarType type;
    int dtype;  // DRADD_*
    c10::Device device;
    c10::cuda::OptionalCUDAGuard guard;
    cudaStream_t stream;

    Call(const at::Tensor& x, const char* name) : type(x.scalar_type()), device(x.device())
    {
        switch (type) {
        case at::kBFloat16: dtype = DRADD_BF16; break;
        case at::kHalf: dtype = DRADD_F16; break;
        case at::kFloat: dtype = DRADD_F32; break;
        default:
            fail(PyExc_TypeError, std::string(name) + " must be bfloat16, float16 or float32 (got " +
                                      c10::toString(type) + ")");
        }
        if (!x.is_cuda())
            fail(PyExc_ValueError, std::string(name) + " must be a CUDA tensor");
        if (device.index() != c10::cuda::current_device())
            guard.set_device(device);
        stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
    }
};

void check(const at::Tensor& t, const char* name, at::ScalarType type, c10::Device device, at::IntArrayRef shape)
{
    if (t.scalar_type() != type)
        fail(PyExc_TypeError,
             std::string(name) + " must hold " + c10::toString(type) + " (got " + c10::toString(t.scalar_type()) + ")");
    if (t.device() != device)
        fail(PyExc_ValueError, std::string(name) + " is on " + t.device().str() + ", expected " + device.str());
    if (t.sizes() != shape) {
        std::ostringstream s;
        s << name << " has shape " << t.sizes() << ", expected " << shape;
        fail(PyExc_ValueError, s.str());
    }
}

// The address of a contiguous tensor of this type, device and shape.
void* flat(const at::Tensor& t, const char* name, at::ScalarType type, c10::Device device, at::IntArrayRef shape)
{
    check(t, name, type, device, shape);
    if (!t.is_contiguous())
        fail(PyExc_ValueError, std::string(name) + " must be contiguous");
    return t.data_ptr();
}

at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, c10::Device device)
{
    const Unlocked unlocked;
    return at::empty(shape, at::TensorOptions().dtype(type).device(device));
}

// An output: the tensor given, or a new contiguous one.
at::Tensor output(PyObject* o, const char* name, at::IntArrayRef shape, const Call& c)
{
    const at::Tensor* t = optional_tensor(o, name);
    return t ? *t : fresh(shape, c.type, c.device);
}

struct Workspace {
    at::Tensor keep;
    void* data = nullptr;
    size_t bytes = 0;

    Workspace(PyObject* o, size_t need, const Call& c)
    {
        const at::Tensor* t = optional_tensor(o, "workspace");
        if (t) {
            if (t->device() != c.device || !t->is_contiguous())
                fail(PyExc_ValueError, "workspace must be a contiguous tensor on " + c.device.str());
            keep = *t;
        } else {
            keep = fresh({static_cast<int64_t>(need)}, at::kByte, c.device);
        }
        data = keep.data_ptr();
        bytes = keep.nbytes();
    }
};

dradd_dropout dropout_of(PyObject* p, PyObject* seed, PyObject* offset, PyObject* step, const Call& c)
{
    dradd_dropout d = {static_cast<float>(number(p)), bits64(seed), bits64(offset), nullptr};
    const at::Tensor* s = optional_tensor(step, "step");
    if (s) {
        if (s->numel() != 1)
            fail(PyExc_ValueError, "step must hold one int64");
        d.step = static_cast<const int64_t*>(flat(*s, "step", at::kLong, c.device, s->sizes()));
    }
    return d;
}

PyObject* tuple_of(std::initializer_list<const at::Tensor*> ts)
{
    PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
    if (!r)
        throw ErrorSet{};
    Py_ssize_t i = 0;
    for (const at::Tensor* t : ts) {
        PyObject* o = Py_None;
        if (t && t->defined())
            o = THPVariable_Wrap(*t);
        else
            Py_INCREF(o);
        if (!o) {
            Py_DECREF(r);
            throw ErrorSet{};
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

// ------------------------------------------------------------------ dropout
// A contiguous tensor as [rows, last dimension], or a 2-D one with unit
// column stride.
struct Rows {
    void* data;
    int64_t n, cols, stride;

    Rows(const at::Tensor& t, const char* name, at::IntArrayRef shape, const Call& c)
    {
        check(t, name, c.type, c.device, shape);
        data = t.data_ptr();
        if (t.is_contiguous()) {
            cols = t.dim() ? t.size(-1) : 1;
            n = cols ? t.numel() / cols : 0;
            stride = cols;
        } else if (t.dim() == 2 && (t.size(1) <= 1 || t.stride(1) == 1)) {
            n = t.size(0);
            cols = t.size(1);
            stride = n > 1 ? t.stride(0) : cols;
        } else {
            fail(PyExc_ValueError, std::string(name) + " must be contiguous, or 2-D with unit column stride");
        }
    }
};

// dropout(x, residual | None, p, seed, offset, step | None, out | None)
PyObject* dropout(PyObject* const* a)
{
    const at::Tensor& x = tensor(a[0], "x");
    const at::Tensor* residual = optional_tensor(a[1], "residual");
    const Call c(x, "x");
    const at::IntArrayRef shape = x.sizes();
    const Rows xr(x, "x", shape, c);
    const at::Tensor out = output(a[6], residual ? "residual_out" : "out", shape, c);
    const Rows o(out, residual ? "residual_out" : "out", shape, c);
    const dradd_dropout d = dropout_of(a[2], a[3], a[4], a[5], c);
    if (residual) {
        const Rows r(*residual, "residual", shape, c);
        if (xr.cols)
            run("dropout_add_fwd", [&] {
                return dropout_add_fwd(o.data, o.stride, xr.data, xr.stride, r.data, r.stride, xr.n, xr.cols, &d,
                                       c.dtype, c.stream);
            });
    } else if (xr.cols) {
        run("dropout_fwd", [&] {
            return dropout_fwd(o.data, o.stride, xr.data, xr.stride, xr.n, xr.cols, &d, c.dtype, c.stream);
        });
    }
    return THPVariable_Wrap(out);
}

// ------------------------------------- dropout + residual add + RMSNorm
int64_t rows_of(const at::Tensor& x)
{
    if (x.dim() == 0 || x.size(-1) == 0)
        fail(PyExc_ValueError, "the last dimension must not be empty");
    return x.numel() / x.size(-1);
}

// drop_norm_fwd(x, residual, weight, p, eps, seed, offset, step, out, residual_out)
PyObject* drop_norm_fwd(PyObject* const* a)
{
    const at::Tensor& x = tensor(a[0], "x");
    const at::Tensor& residual = tensor(a[1], "residual");
    const at::Tensor& weight = tensor(a[2], "weight");
    const Call c(x, "x");
    const at::IntArrayRef shape = x.sizes();
    const int64_t n = rows_of(x), hidden = x.size(-1);
    void* xp = flat(x, "x", c.type, c.device, shape);
    void* rp = flat(residual, "residual", c.type, c.device, shape);
    void* wp = flat(weight, "weight", c.type, c.device, {hidden});
    const at::Tensor out = output(a[8], "out", shape, c);
    const at::Tensor residual_out = output(a[9], "residual_out", shape, c);
    const dradd_dropout d = dropout_of(a[3], a[5], a[6], a[7], c);
    void* op = flat(out, "out", c.type, c.device, shape);
    void* hp = flat(residual_out, "residual_out", c.type, c.device, shape);
    const float eps = static_cast<float>(number(a[4]));
    run("dropout_add_rmsnorm_fwd", [&] {
        return dropout_add_rmsnorm_fwd(op, hp, xp, rp, wp, eps, n, hidden, &d, c.dtype, c.stream);
    });
    return tuple_of({&out, &residual_out});
}

// drop_norm_bwd(dout, dresidual_out | None, h, weight, drop, p, eps, seed, offset, step, dx, dresidual, dweight,
//               weight_grad, workspace): drop false is add_rmsnorm_bwd, whose dresidual is dh and which has no dx
PyObject* drop_norm_bwd(PyObject* const* a)
{
    const at::Tensor& dout = tensor(a[0], "dout");
    const at::Tensor* dro = optional_tensor(a[1], "dresidual_out");
    const at::Tensor& h = tensor(a[2], "residual_out");
    const at::Tensor& weight = tensor(a[3], "weight");
    const bool drop = truth(a[4]), sums = truth(a[13]);
    const Call c(h, "residual_out");
    const at::IntArrayRef shape = h.sizes();
    const int64_t n = rows_of(h), hidden = h.size(-1);
    void* hp = flat(h, "residual_out", c.type, c.device, shape);
    void* gp = flat(dout, "dout", c.type, c.device, shape);
    void* dp = dro ? flat(*dro, "dresidual_out", c.type, c.device, shape) : nullptr;
    void* wp = flat(weight, "weight", c.type, c.device, {hidden});
    if (!sums && a[12] != Py_None)
        fail(PyExc_ValueError, "dweight is given but weight_grad is False");
    const char* name = drop ? "dresidual" : "dh";
    at::Tensor dx, dweight;
    if (drop)
        dx = output(a[10], "dx", shape, c);
    const at::Tensor dresidual = output(a[11], name, shape, c);
    void* op = flat(dresidual, name, c.type, c.device, shape);
    void* xp = drop ? flat(dx, "dx", c.type, c.device, shape) : nullptr;
    float* sp = nullptr;
    void* ws = nullptr;
    size_t bytes = 0;
    at::Tensor keep;
    if (sums) {
        const at::Tensor* given = optional_tensor(a[12], "dweight");
        dweight = given ? *given : fresh({hidden}, at::kFloat, c.device);
        sp = static_cast<float*>(flat(dweight, "dweight", at::kFloat, c.device, {hidden}));
        const Workspace w(a[14], rmsnorm_bwd_workspace_bytes(n, hidden, c.dtype), c);
        keep = w.keep;
        ws = w.data;
        bytes = w.bytes;
    }
    const float eps = static_cast<float>(number(a[6]));
    if (drop) {
        const dradd_dropout d = dropout_of(a[5], a[7], a[8], a[9], c);
        run("dropout_add_rmsnorm_bwd", [&] {
            return dropout_add_rmsnorm_bwd(xp, op, sp, gp, dp, hp, wp, eps, n, hidden, &d, c.dtype, ws, bytes,
                                           c.stream);
        });
    } else {
        run("add_rmsnorm_bwd", [&] {
            return add_rmsnorm_bwd(op, sp, gp, dp, hp, wp, eps, n, hidden, c.dtype, ws, bytes, c.stream);
        });
    }
    return tuple_of({&dx, &dresidual, &dweight});
}

// ------------------------------------------------------------------- rotary
dradd_heads heads(const at::Tensor& t, const char* name, const Call& c, at::IntArrayRef shape)
{
    check(t, name, c.type, c.device, shape);
    if (t.stride(3) != 1 && shape[3] > 1)
        fail(PyExc_ValueError, std::string(name) + " must have unit stride in its last dimension");
    return {t.data_ptr(), t.stride(0), t.stride(1), t.stride(2)};
}

// a: inv_freq, positions | None, position0, interleaved, scale
dradd_rope rope_of(const at::Tensor& q, const at::Tensor* k, PyObject* const* a, const Call& c)
{
    if (q.dim() != 4 || (k && (k->dim() != 4 || k->size(0) != q.size(0) || k->size(1) != q.size(1) ||
                               k->size(3) != q.size(3))))
        fail(PyExc_ValueError, "q and k must be [batch, seq, heads, head_dim], alike but for their heads");
    const at::Tensor& f = tensor(a[0], "inv_freq");
    if (f.dim() != 1)
        fail(PyExc_ValueError, "inv_freq must be 1-D: one frequency per pair");
    dradd_rope r = {};
    r.batch = q.size(0);
    r.seq = q.size(1);
    r.q_heads = q.size(2);
    r.k_heads = k ? k->size(2) : 0;
    r.head_dim = q.size(3);
    r.rot_dim = 2 * f.size(0);
    r.interleaved = truth(a[3]);
    r.inv_freq = static_cast<const double*>(flat(f, "inv_freq", at::kDouble, c.device, f.sizes()));
    r.position0 = static_cast<int64_t>(bits64(a[2]));
    const at::Tensor* pos = optional_tensor(a[1], "positions");
    if (pos) {
        if (r.position0)
            fail(PyExc_ValueError, "give positions or position0, not both");
        r.positions = static_cast<const int64_t*>(flat(*pos, "positions", at::kLong, c.device, {r.batch, r.seq}));
    }
    r.scale = static_cast<float>(number(a[4]));
    return r;
}

// One of q and k in a rotary call.
struct Side {
    at::Tensor out;
    dradd_heads to, from;

    Side(const at::Tensor& x, const char* name, PyObject* o, const char* out_name, const Call& c)
        : out(output(o, out_name, x.sizes(), c)), to(heads(out, out_name, c, x.sizes())),
          from(heads(x, name, c, x.sizes()))
    {
    }
};

// rope(inverse, q, k | None, inv_freq, positions, position0, interleaved, scale, q_out, k_out)
PyObject* rope(PyObject* const* a)
{
    const bool inverse = truth(a[0]);
    const at::Tensor& q = tensor(a[1], "q");
    const at::Tensor* k = optional_tensor(a[2], "k");
    const Call c(q, "q");
    const dradd_rope r = rope_of(q, k, a + 3, c);
    const Side sq(q, "q", a[8], inverse ? "dq" : "q_out", c);
    at::Tensor k_out;
    dradd_heads ko = {}, ki = {};
    if (k) {
        const Side sk(*k, "k", a[9], inverse ? "dk" : "k_out", c);
        k_out = sk.out;
        ko = sk.to;
        ki = sk.from;
    }
    run(inverse ? "rope_bwd" : "rope_fwd", [&] {
        return (inverse ? rope_bwd : rope_fwd)(&sq.to, &ko, &sq.from, &ki, &r, c.dtype, c.stream);
    });
    return tuple_of({&sq.out, &k_out});
}

// norm_rope_fwd(q, k | None, q_weight, k_weight | None, q_eps, k_eps, inv_freq, positions, position0, interleaved,
//               scale, q_out, k_out)
PyObject* norm_rope_fwd(PyObject* const* a)
{
    const at::Tensor& q = tensor(a[0], "q");
    const at::Tensor* k = optional_tensor(a[1], "k");
    const Call c(q, "q");
    const dradd_rope r = rope_of(q, k, a + 6, c);
    const void* qw = flat(tensor(a[2], "q_weight"), "q_weight", c.type, c.device, {r.head_dim});
    const Side sq(q, "q", a[11], "q_out", c);
    const void* kw = nullptr;
    at::Tensor k_out;
    dradd_heads ko = {}, ki = {};
    if (k) {
        kw = flat(tensor(a[3], "k_weight"), "k_weight", c.type, c.device, {r.head_dim});
        const Side sk(*k, "k", a[12], "k_out", c);
        k_out = sk.out;
        ko = sk.to;
        ki = sk.from;
    }
    const float q_eps = static_cast<float>(number(a[4])), k_eps = static_cast<float>(number(a[5]));
    run("qk_rmsnorm_rope_fwd", [&] {
        return qk_rmsnorm_rope_fwd(&sq.to, &ko, &sq.from, &ki, qw, kw, q_eps, k_eps, &r, c.dtype, c.stream);
    });
    return tuple_of({&sq.out, &k_out});
}

// norm_rope_bwd(dq_out, dk_out | None, q, k | None, q_weight, k_weight | None, q_eps, k_eps, inv_freq, positions,
//               position0, interleaved, scale, dq, dk, dq_weight, dk_weight, weight_grad, workspace)
PyObject* norm_rope_bwd(PyObject* const* a)
{
    const at::Tensor& q = tensor(a[2], "q");
    const at::Tensor* k = optional_tensor(a[3], "k");
    const bool sums = truth(a[17]);
    const Call c(q, "q");
    const dradd_rope r = rope_of(q, k, a + 8, c);
    if (!sums && (a[15] != Py_None || a[16] != Py_None))
        fail(PyExc_ValueError, "a weight's gradient is given but weight_grad is False");
    const void* qw = flat(tensor(a[4], "q_weight"), "q_weight", c.type, c.device, {r.head_dim});
    const dradd_heads gq = heads(tensor(a[0], "dq_out"), "dq_out", c, q.sizes());
    const Side sq(q, "q", a[13], "dq", c);
    const void* kw = nullptr;
    at::Tensor dk, dqw, dkw, keep;
    dradd_heads ko = {}, ki = {}, gk = {};
    if (k) {
        kw = flat(tensor(a[5], "k_weight"), "k_weight", c.type, c.device, {r.head_dim});
        gk = heads(tensor(a[1], "dk_out"), "dk_out", c, k->sizes());
        const Side sk(*k, "k", a[14], "dk", c);
        dk = sk.out;
        ko = sk.to;
        ki = sk.from;
    }
    float *qs = nullptr, *ks = nullptr;
    void* ws = nullptr;
    size_t bytes = 0;
    if (sums) {
        const auto sum = [&](PyObject* o, const char* name, at::Tensor& t) {
            const at::Tensor* given = optional_tensor(o, name);
            t = given ? *given : fresh({r.head_dim}, at::kFloat, c.device);
            return static_cast<float*>(flat(t, name, at::kFloat, c.device, {r.head_dim}));
        };
        qs = sum(a[15], "dq_weight", dqw);
        if (k)
            ks = sum(a[16], "dk_weight", dkw);
        const Workspace w(a[18], qk_rmsnorm_rope_bwd_workspace_bytes(&r, c.dtype), c);
        keep = w.keep;
        ws = w.data;
        bytes = w.bytes;
    }
    const float q_eps = static_cast<float>(number(a[6])), k_eps = static_cast<float>(number(a[7]));
    run("qk_rmsnorm_rope_bwd", [&] {
        return qk_rmsnorm_rope_bwd(&sq.to, &ko, qs, ks, &gq, &gk, &sq.from, &ki, qw, kw, q_eps, k_eps, &r, c.dtype, ws,
                                   bytes, c.stream);
    });
    return tuple_of({&sq.out, &dk, &dqw, &dkw});
}

// ---------------------------------------------------------- matrix products
// The call's type, one of the 16-bit ones.
Call product_call(const at::Tensor& x)
{
    if (x.scalar_type() != at::kBFloat16 && x.scalar_type() != at::kHalf)
        fail(PyExc_TypeError,
             std::string("x must be bfloat16 or float16 (got ") + c10::toString(x.scalar_type()) + ")");
    return Call(x, "x");
}

int64_t inner_of(const at::Tensor& x)
{
    if (x.dim() == 0 || x.size(-1) == 0)
        fail(PyExc_ValueError, "x must have a last dimension that is not empty");
    return x.size(-1);
}

// A 2-D weight [anything, inner].
const at::Tensor& weight_of(PyObject* o, int64_t inner)
{
    const at::Tensor& w = tensor(o, "weight");
    if (w.dim() != 2 || w.size(1) != inner) {
        std::ostringstream s;
        s << "weight has shape " << w.sizes() << ", expected [*, " << inner << "]";
        fail(PyExc_ValueError, s.str());
    }
    return w;
}

dradd_matrix matrix(const Rows& r) { return {r.data, r.stride}; }

std::vector<int64_t> with_last(at::IntArrayRef shape, int64_t n)
{
    std::vector<int64_t> v(shape.begin(), shape.end());
    v.back() = n;
    return v;
}

// linear_fwd(x, weight, bias | None, residual | None, act, out | None, workspace | None)
PyObject* linear_fwd(PyObject* const* a)
{
    const at::Tensor& x = tensor(a[0], "x");
    const Call c = product_call(x);
    const int64_t inner = inner_of(x);
    const at::Tensor& weight = weight_of(a[1], inner);
    const int64_t cols = weight.size(0);
    const at::Tensor* bias = optional_tensor(a[2], "bias");
    const at::Tensor* residual = optional_tensor(a[3], "residual");
    const int act = static_cast<int>(bits64(a[4]));
    const std::vector<int64_t> shape = with_last(x.sizes(), cols);
    const Rows xr(x, "x", x.sizes(), c), wr(weight, "weight", weight.sizes(), c);
    const void* bp = bias ? flat(*bias, "bias", c.type, c.device, {cols}) : nullptr;
    dradd_matrix rm = {nullptr, 0};
    if (residual)
        rm = matrix(Rows(*residual, "residual", shape, c));
    const at::Tensor out = output(a[5], "out", shape, c);
    const Rows o(out, "out", shape, c);
    const dradd_matrix om = matrix(o), xm = matrix(xr), wm = matrix(wr);
    const size_t need = linear_act_add_fwd_workspace_bytes(xr.n, inner, cols);
    void* ws = nullptr;
    size_t bytes = 0;
    at::Tensor keep;
    if (need) {
        const Workspace w(a[6], need, c);
        keep = w.keep;
        ws = w.data;
        bytes = w.bytes;
    }
    run("linear_act_add_fwd", [&] {
        return linear_act_add_fwd(&om, &xm, &wm, bp, &rm, act, xr.n, inner, cols, c.dtype, ws, bytes, c.stream);
    });
    return THPVariable_Wrap(out);
}

// linear_bwd(dout, x, weight, bias | None, act, dx, dweight, dbias, input_grad, weight_grad, workspace)
PyObject* linear_bwd(PyObject* const* a)
{
    const at::Tensor& dout = tensor(a[0], "dout");
    const at::Tensor& x = tensor(a[1], "x");
    const Call c = product_call(x);
    const int64_t inner = inner_of(x);
    const at::Tensor& weight = weight_of(a[2], inner);
    const int64_t cols = weight.size(0);
    const at::Tensor* bias = optional_tensor(a[3], "bias");
    const int act = static_cast<int>(bits64(a[4]));
    const bool want_x = truth(a[8]), want_w = truth(a[9]), want_b = want_w && bias;
    if ((!want_x && a[5] != Py_None) || (!want_w && a[6] != Py_None) || (!want_b && a[7] != Py_None))
        fail(PyExc_ValueError, "an output is given for a gradient that is not asked for");
    const std::vector<int64_t> shape = with_last(x.sizes(), cols);
    const Rows xr(x, "x", x.sizes(), c), wr(weight, "weight", weight.sizes(), c), gr(dout, "dout", shape, c);
    const void* bp = bias ? flat(*bias, "bias", c.type, c.device, {cols}) : nullptr;
    at::Tensor dx, dw, db;
    if (want_x)
        dx = output(a[5], "dx", x.sizes(), c);
    if (want_w)
        dw = output(a[6], "dweight", weight.sizes(), c);
    if (want_b)
        db = output(a[7], "dbias", {cols}, c);
    void* xp = want_x ? flat(dx, "dx", c.type, c.device, x.sizes()) : nullptr;
    void* wp = want_w ? flat(dw, "dweight", c.type, c.device, weight.sizes()) : nullptr;
    void* dbp = want_b ? flat(db, "dbias", c.type, c.device, {cols}) : nullptr;
    const dradd_matrix gm = matrix(gr), xm = matrix(xr), wm = matrix(wr);
    const Workspace w(a[10], linear_act_add_bwd_workspace_bytes(xr.n, inner, cols, act, want_x, want_w, want_b), c);
    run("linear_act_add_bwd", [&] {
        return linear_act_add_bwd(xp, wp, dbp, &gm, &xm, &wm, bp, act, xr.n, inner, cols, c.dtype, w.data, w.bytes,
                                  c.stream);
    });
    return tuple_of({&dx, &dw, &db});
}

// A row's words: int64 targets, or a teacher's index and logits.
struct LossWords {
    const int64_t* target = nullptr;
    int64_t ignore_index = 0;
    dradd_teacher teacher = {};
    bool distill = false;

    // a: target | index, teacher logits | None, ignore_index, temperature
    LossWords(PyObject* const* a, at::IntArrayRef rows, const Call& c)
    {
        const at::Tensor* logits = optional_tensor(a[1], "teacher_logits");
        distill = logits != nullptr;
        if (!distill) {
            const at::Tensor& t = tensor(a[0], "target");
            target = static_cast<const int64_t*>(flat(t, "target", at::kLong, c.device, rows));
            ignore_index = static_cast<int64_t>(bits64(a[2]));
            return;
        }
        const at::Tensor& t = tensor(a[0], "teacher_index");
        if (t.dim() == 0)
            fail(PyExc_ValueError, "teacher_index must have a last dimension: the entries of a row");
        std::vector<int64_t> shape(rows.begin(), rows.end());
        shape.push_back(t.size(-1));
        teacher.index = static_cast<const int64_t*>(flat(t, "teacher_index", at::kLong, c.device, shape));
        switch (logits->scalar_type()) {
        case at::kBFloat16: teacher.logits_dtype = DRADD_BF16; break;
        case at::kHalf: teacher.logits_dtype = DRADD_F16; break;
        case at::kFloat: teacher.logits_dtype = DRADD_F32; break;
        default: fail(PyExc_TypeError, "teacher_logits must be bfloat16, float16 or float32");
        }
        teacher.logits = flat(*logits, "teacher_logits", logits->scalar_type(), c.device, shape);
        teacher.top = t.size(-1);
        teacher.temperature = static_cast<float>(number(a[3]));
    }
};

// A row's fp32 number: contiguous, or one value for all rows.
struct RowNumbers {
    const float* data;
    int64_t stride;

    RowNumbers(const at::Tensor& t, const char* name, at::IntArrayRef rows, const Call& c)
    {
        bool one = true;
        for (int64_t i = 0; i < t.dim(); ++i)
            one = one && (t.stride(i) == 0 || t.size(i) == 1);
        check(t, name, at::kFloat, c.device, t.dim() == 0 ? t.sizes() : rows);
        if (!one && !t.is_contiguous())
            fail(PyExc_ValueError, std::string(name) + " must be contiguous, or one value for all rows");
        data = static_cast<const float*>(t.data_ptr());
        stride = one ? 0 : 1;
    }
};

// loss_fwd(x, weight, target | index, teacher_logits | None, ignore_index, temperature, loss, lse, workspace)
PyObject* loss_fwd(PyObject* const* a)
{
    const at::Tensor& x = tensor(a[0], "x");
    const Call c = product_call(x);
    const int64_t hidden = inner_of(x);
    const at::Tensor& weight = weight_of(a[1], hidden);
    const int64_t vocab = weight.size(0);
    const at::IntArrayRef rows = x.sizes().slice(0, x.dim() - 1);
    const Rows xr(x, "x", x.sizes(), c), wr(weight, "weight", weight.sizes(), c);
    const LossWords words(a + 2, rows, c);
    const auto numbers = [&](PyObject* o, const char* name) {
        const at::Tensor* t = optional_tensor(o, name);
        return t ? *t : fresh(rows, at::kFloat, c.device);
    };
    const at::Tensor loss = numbers(a[6], "loss"), lse = numbers(a[7], "lse");
    float* lp = static_cast<float*>(flat(loss, "loss", at::kFloat, c.device, rows));
    float* ep = static_cast<float*>(flat(lse, "lse", at::kFloat, c.device, rows));
    const Workspace w(a[8],
                      words.distill ? linear_distill_fwd_workspace_bytes(xr.n, hidden, vocab, words.teacher.top)
                                    : linear_cross_entropy_fwd_workspace_bytes(xr.n, hidden, vocab),
                      c);
    const dradd_matrix xm = matrix(xr), wm = matrix(wr);
    if (words.distill)
        run("linear_distill_fwd", [&] {
            return linear_distill_fwd(lp, ep, &xm, &wm, &words.teacher, xr.n, hidden, vocab, c.dtype, w.data, w.bytes,
                                      c.stream);
        });
    else
        run("linear_cross_entropy_fwd", [&] {
            return linear_cross_entropy_fwd(lp, ep, &xm, &wm, words.target, words.ignore_index, xr.n, hidden, vocab,
                                            c.dtype, w.data, w.bytes, c.stream);
        });
    return tuple_of({&loss, &lse});
}

// loss_bwd(dloss, dlse | None, x, weight, target | index, teacher_logits | None, ignore_index, temperature, lse, dx,
//          dweight, input_grad, weight_grad, workspace)
PyObject* loss_bwd(PyObject* const* a)
{
    const at::Tensor& x = tensor(a[2], "x");
    const Call c = product_call(x);
    const int64_t hidden = inner_of(x);
    const at::Tensor& weight = weight_of(a[3], hidden);
    const int64_t vocab = weight.size(0);
    const at::IntArrayRef rows = x.sizes().slice(0, x.dim() - 1);
    const Rows xr(x, "x", x.sizes(), c), wr(weight, "weight", weight.sizes(), c);
    const LossWords words(a + 4, rows, c);
    const RowNumbers dloss(tensor(a[0], "dloss"), "dloss", rows, c);
    const at::Tensor* given = optional_tensor(a[1], "dlse");
    const float* dlse = nullptr;
    int64_t dlse_stride = 0;
    if (given) {
        const RowNumbers n(*given, "dlse", rows, c);
        dlse = n.data;
        dlse_stride = n.stride;
    }
    const float* lse = static_cast<const float*>(flat(tensor(a[8], "lse"), "lse", at::kFloat, c.device, rows));
    const bool want_x = truth(a[11]), want_w = truth(a[12]);
    if ((!want_x && a[9] != Py_None) || (!want_w && a[10] != Py_None))
        fail(PyExc_ValueError, "an output is given for a gradient that is not asked for");
    at::Tensor dx, dw;
    if (want_x)
        dx = output(a[9], "dx", x.sizes(), c);
    if (want_w)
        dw = output(a[10], "dweight", weight.sizes(), c);
    void* xp = want_x ? flat(dx, "dx", c.type, c.device, x.sizes()) : nullptr;
    void* wp = want_w ? flat(dw, "dweight", c.type, c.device, weight.sizes()) : nullptr;
    const Workspace w(a[13],
                      words.distill ? linear_distill_bwd_workspace_bytes(xr.n, hidden, vocab, words.teacher.top)
                                    : linear_cross_entropy_bwd_workspace_bytes(xr.n, hidden, vocab),
                      c);
    const dradd_matrix xm = matrix(xr), wm = matrix(wr);
    if (words.distill)
        run("linear_distill_bwd", [&] {
            return linear_distill_bwd(xp, wp, dloss.data, dloss.stride, dlse, dlse_stride, &xm, &wm, &words.teacher,
                                      lse, xr.n, hidden, vocab, c.dtype, w.data, w.bytes, c.stream);
        });
    else
        run("linear_cross_entropy_bwd", [&] {
            return linear_cross_entropy_bwd(xp, wp, dloss.data, dloss.stride, dlse, dlse_stride, &xm, &wm,
                                            words.target, words.ignore_index, lse, xr.n, hidden, vocab, c.dtype,
                                            w.data, w.bytes, c.stream);
        });
    return tuple_of({&dx, &dw});
}

// ------------------------------------------------------------------- module
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const ErrorSet&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyMethodDef method(const char* name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<dropout, 7>("dropout"),
                         method<drop_norm_fwd, 10>("drop_norm_fwd"),
                         method<drop_norm_bwd, 15>("drop_norm_bwd"),
                         method<rope, 10>("rope"),
                         method<norm_rope_fwd, 13>("norm_rope_fwd"),
                         method<norm_rope_bwd, 19>("norm_rope_bwd"),
                         method<linear_fwd, 7>("linear_fwd"),
                         method<linear_bwd, 11>("linear_bwd"),
                         method<loss_fwd, 9>("loss_fwd"),
                         method<loss_bwd, 14>("loss_bwd"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
