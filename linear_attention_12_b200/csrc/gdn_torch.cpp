// gdn_torch.cpp -- argument checks, output allocation and the call itself for the binding's
// short calls (scan, norm, front-end gradients): what ``linear_attention_12_b200/gdn.py`` does
// for the others in Python.  A decode step's kernel takes 2 us and its call through Python
// and ctypes took 10; here it is half of that.
//
// It holds no arithmetic: tensors are checked, outputs and workspaces come from PyTorch's
// allocator on the current stream of the first tensor's device, and the C ABI of include/gdn.h
// is called through the addresses that ``bind`` was given.  Every function returns its results,
// or the gdn_status of a call that failed.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "../../include/gdn.h"

namespace {

struct Table {
    decltype(&gdn_scan) scan;
    decltype(&gdn_scan_backward) scan_backward;
    decltype(&gdn_scan_step) scan_step;
    decltype(&gdn_group_norm) group_norm;
    decltype(&gdn_group_norm_backward) group_norm_backward;
    decltype(&gdn_group_norm_backward_workspace_size) group_norm_backward_workspace_size;
    decltype(&gdn_frontend_backward) frontend_backward;
    decltype(&gdn_frontend_backward_workspace_size) frontend_backward_workspace_size;
};
Table lib;

using at::Tensor;
using torch::TypeError;
struct ValueError : torch::PyTorchError {
    using PyTorchError::PyTorchError;
    explicit ValueError(std::string m) : PyTorchError(std::move(m)) {}
    PyObject* python_type() override { return PyExc_ValueError; }
};

std::string shape_text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}

const Tensor& cuda_tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda())
        throw TypeError(std::string(name) + " must be a CUDA tensor");
    return THPVariable_Unpack(o);
}

gdn_dtype io_type(const Tensor& t, const char* name) {
    if (t.scalar_type() == at::kBFloat16) return GDN_BF16;
    if (t.scalar_type() == at::kFloat) return GDN_F32;
    throw TypeError(std::string(name) + " must be a bfloat16 or float32 tensor");
}

void expect(const Tensor& t, const char* name, at::ScalarType dtype, at::IntArrayRef shape,
            const at::Device& device) {
    if (t.scalar_type() != dtype)
        throw TypeError(std::string(name) + " must be " + c10::toString(dtype) + ", got " +
                        c10::toString(t.scalar_type()));
    if (t.sizes() != shape)
        throw ValueError(std::string(name) + " must have shape " + shape_text(shape) + ", got " +
                         shape_text(t.sizes()));
    if (t.device() != device)
        throw ValueError(std::string(name) + " is on " + t.device().str() + ", expected " +
                         device.str());
}

// Row stride of a token-major tensor whose rows of `cols` elements are dense (a column slice of
// a wider tensor will do).
int64_t rows(const Tensor& t, const char* name, at::ScalarType dtype, at::IntArrayRef shape,
             const at::Device& device, int64_t cols) {
    expect(t, name, dtype, shape, device);
    if (t.is_contiguous()) return cols;
    int64_t dense = 1;
    for (int64_t i = (int64_t)shape.size() - 1; i > 0; --i) {
        if (shape[i] != 1 && t.stride(i) != dense)
            throw ValueError("the rows of " + std::string(name) + " must be dense, got strides " +
                             shape_text(t.strides()));
        dense *= shape[i];
    }
    if (shape[0] <= 1) return cols;
    if (t.stride(0) < cols)
        throw ValueError("the rows of " + std::string(name) + " overlap: strides " +
                         shape_text(t.strides()));
    return t.stride(0);
}

const Tensor& dense(PyObject* o, const char* name, at::ScalarType dtype, at::IntArrayRef shape,
                    const at::Device& device) {
    const Tensor& t = cuda_tensor(o, name);
    expect(t, name, dtype, shape, device);
    if (!t.is_contiguous()) throw ValueError(std::string(name) + " must be contiguous");
    return t;
}
// The same for an argument that may be None: its data, or null.
float* dense_f32(PyObject* o, const char* name, at::IntArrayRef shape, const at::Device& device) {
    return o == Py_None ? nullptr
                        : static_cast<float*>(dense(o, name, at::kFloat, shape, device).data_ptr());
}

Tensor fresh(at::IntArrayRef shape, at::ScalarType dtype, const at::Device& device) {
    return Tensor(at::detail::empty_cuda(shape, dtype, device, std::nullopt));
}

// An output: the one given (its rows checked), or a fresh dense one.
Tensor output(PyObject* o, const char* name, at::ScalarType dtype, at::IntArrayRef shape,
              const at::Device& device, int64_t cols, int64_t& stride) {
    if (o == Py_None) {
        stride = cols;
        return fresh(shape, dtype, device);
    }
    const Tensor& t = cuda_tensor(o, name);
    stride = rows(t, name, dtype, shape, device, cols);
    return t;
}

Tensor workspace(PyObject* o, size_t need, const at::Device& device) {
    if (o == Py_None) return fresh({(int64_t)need}, at::kByte, device);
    const Tensor& t = cuda_tensor(o, "workspace");
    if (t.device() != device)
        throw ValueError("workspace is on " + t.device().str() + ", expected " + device.str());
    if (!t.is_contiguous()) throw ValueError("workspace must be contiguous");
    return t;
}

int32_t size32(int64_t n, const char* name) {
    if (n > 0x7fffffff) throw ValueError(std::string(name) + " is too large");
    return (int32_t)n;
}

void* here(const at::Device& device) {
    return c10::cuda::getCurrentCUDAStream(device.index()).stream();
}

// N and the data of cu_seqlens (None: one sequence).
int32_t sequences(PyObject* o, const at::Device& device, const int32_t*& cu) {
    cu = nullptr;
    if (o == Py_None) return 1;
    const Tensor& t = cuda_tensor(o, "cu_seqlens");
    if (t.dim() != 1 || t.numel() < 2)
        throw ValueError("cu_seqlens must be [N + 1] with N >= 1");
    expect(t, "cu_seqlens", at::kInt, t.sizes(), device);
    if (!t.is_contiguous()) throw ValueError("cu_seqlens must be contiguous");
    cu = static_cast<const int32_t*>(t.data_ptr());
    return size32(t.numel() - 1, "N");
}

// [N, ...channels] of a [T, ...channels] tensor.
c10::SmallVector<int64_t, 4> states_shape(const Tensor& x, int64_t N) {
    c10::SmallVector<int64_t, 4> s(x.sizes().begin(), x.sizes().end());
    s[0] = N;
    return s;
}

int64_t channels(const Tensor& x) {
    if (x.dim() < 2) throw ValueError("expected [T, ...channels], got " + shape_text(x.sizes()));
    int64_t C = 1;
    for (int64_t i = 1; i < x.dim(); ++i) C *= x.size(i);
    return C;
}

bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}

PyObject* status(gdn_status st) { return PyLong_FromLong(st); }

// A tuple of tensors (an undefined one: None).
PyObject* tuple_of(std::initializer_list<Tensor> ts) {
    PyObject* t = PyTuple_New((Py_ssize_t)ts.size());
    if (!t) return nullptr;
    Py_ssize_t i = 0;
    for (const Tensor& x : ts) {
        PyObject* o;
        if (x.defined()) {
            o = THPVariable_Wrap(x);
        } else {
            o = Py_None;
            Py_INCREF(o);
        }
        if (!o) {
            Py_DECREF(t);
            return nullptr;
        }
        PyTuple_SET_ITEM(t, i++, o);
    }
    return t;
}

#define GDN_ARGS(count)                                                             \
    HANDLE_TH_ERRORS if (n != (count)) throw TypeError(std::string(__func__) + ": wrong number of arguments")

// scan(x, log_alpha, h0, cu_seqlens, h, h_final, want_state) -> (h, h_final)
PyObject* scan(PyObject*, PyObject* const* a, Py_ssize_t n) {
    GDN_ARGS(7);
    const Tensor &x = cuda_tensor(a[0], "x"), &la = cuda_tensor(a[1], "log_alpha");
    const at::Device dev = x.device();
    const c10::cuda::CUDAGuard guard(dev);
    const gdn_dtype io = io_type(x, "x"), gate = io_type(la, "log_alpha");
    const int64_t C = channels(x);
    const int32_t* cu;
    const int32_t N = sequences(a[3], dev, cu);
    const int64_t xs = rows(x, "x", x.scalar_type(), x.sizes(), dev, C);
    const int64_t las = rows(la, "log_alpha", la.scalar_type(), x.sizes(), dev, C);
    const auto states = states_shape(x, N);
    const float* h0 = dense_f32(a[2], "h0", states, dev);
    int64_t hs;
    const Tensor h = output(a[4], "h", x.scalar_type(), x.sizes(), dev, C, hs);
    Tensor hf;
    if (a[5] != Py_None)
        hf = dense(a[5], "h_final", at::kFloat, states, dev);
    else if (truth(a[6]))
        hf = fresh(states, at::kFloat, dev);
    const gdn_status st =
        lib.scan(x.data_ptr(), xs, la.data_ptr(), las, h0, cu, N, size32(x.size(0), "T"),
                 size32(C, "C"), io, gate, h.data_ptr(), hs,
                 hf.defined() ? static_cast<float*>(hf.data_ptr()) : nullptr, here(dev));
    return st == GDN_OK ? tuple_of({h, hf}) : status(st);
    END_HANDLE_TH_ERRORS
}

// scan_backward(log_alpha, h, dh, h0, dh_final, cu_seqlens, dx, dlog_alpha, want_dh0)
//     -> (dx, dlog_alpha, dh0)
PyObject* scan_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    GDN_ARGS(9);
    const Tensor &la = cuda_tensor(a[0], "log_alpha"), &h = cuda_tensor(a[1], "h"),
                 &dh = cuda_tensor(a[2], "dh");
    const at::Device dev = h.device();
    const c10::cuda::CUDAGuard guard(dev);
    const gdn_dtype io = io_type(h, "h"), gate = io_type(la, "log_alpha");
    const int64_t C = channels(h);
    const int32_t* cu;
    const int32_t N = sequences(a[5], dev, cu);
    const at::IntArrayRef shape = h.sizes();
    const int64_t las = rows(la, "log_alpha", la.scalar_type(), shape, dev, C);
    const int64_t hs = rows(h, "h", h.scalar_type(), shape, dev, C);
    const int64_t dhs = rows(dh, "dh", h.scalar_type(), shape, dev, C);
    const auto states = states_shape(h, N);
    const float* h0 = dense_f32(a[3], "h0", states, dev);
    const float* dhf = dense_f32(a[4], "dh_final", states, dev);
    int64_t dxs, dlas;
    const Tensor dx = output(a[6], "dx", h.scalar_type(), shape, dev, C, dxs);
    const Tensor dla = output(a[7], "dlog_alpha", la.scalar_type(), shape, dev, C, dlas);
    const Tensor dh0 = truth(a[8]) ? fresh(states, at::kFloat, dev) : Tensor();
    const gdn_status st = lib.scan_backward(
        la.data_ptr(), las, h.data_ptr(), hs, dh.data_ptr(), dhs, h0, dhf, cu, N,
        size32(h.size(0), "T"), size32(C, "C"), io, gate, dx.data_ptr(), dxs, dla.data_ptr(), dlas,
        dh0.defined() ? static_cast<float*>(dh0.data_ptr()) : nullptr, here(dev));
    return st == GDN_OK ? tuple_of({dx, dla, dh0}) : status(st);
    END_HANDLE_TH_ERRORS
}

// scan_step(x, log_alpha, state, h) -> h
PyObject* scan_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
    GDN_ARGS(4);
    const Tensor &x = cuda_tensor(a[0], "x"), &la = cuda_tensor(a[1], "log_alpha");
    const at::Device dev = x.device();
    const c10::cuda::CUDAGuard guard(dev);
    const gdn_dtype io = io_type(x, "x"), gate = io_type(la, "log_alpha");
    const int64_t C = channels(x);
    const int64_t xs = rows(x, "x", x.scalar_type(), x.sizes(), dev, C);
    const int64_t las = rows(la, "log_alpha", la.scalar_type(), x.sizes(), dev, C);
    const Tensor& state = dense(a[2], "state", at::kFloat, x.sizes(), dev);
    int64_t hs;
    const Tensor h = output(a[3], "h", x.scalar_type(), x.sizes(), dev, C, hs);
    const gdn_status st = lib.scan_step(
        x.data_ptr(), xs, la.data_ptr(), las, static_cast<float*>(state.data_ptr()),
        size32(x.size(0), "B"), size32(C, "C"), io, gate, h.data_ptr(), hs, here(dev));
    return st == GDN_OK ? THPVariable_Wrap(h) : status(st);
    END_HANDLE_TH_ERRORS
}

// What both directions of the norm check.
struct NormArgs {
    const Tensor &x, &w;
    at::Device dev;
    gdn_dtype io;
    int32_t T, H, d, weight_heads;
    int64_t C, xs, zs = 0;
    const float* b;
    const Tensor* z = nullptr;

    NormArgs(PyObject* px, PyObject* pw, PyObject* pb, PyObject* pz)
        : x(cuda_tensor(px, "x")), w(cuda_tensor(pw, "weight")), dev(x.device()) {
        io = io_type(x, "x");
        if (x.dim() != 3) throw ValueError("x must be [T, H, d], got " + shape_text(x.sizes()));
        T = size32(x.size(0), "T"), H = size32(x.size(1), "H"), d = size32(x.size(2), "d");
        C = (int64_t)H * d;
        const bool shared = w.dim() == 1 && w.size(0) == d;
        if (!shared && !(w.dim() == 2 && w.size(0) == H && w.size(1) == d))
            throw ValueError("weight must have shape (" + std::to_string(d) + ",) or (" +
                             std::to_string(H) + ", " + std::to_string(d) + ")");
        weight_heads = shared ? 1 : H;
        dense(pw, "weight", at::kFloat, w.sizes(), dev);
        b = dense_f32(pb, "bias", w.sizes(), dev);
        xs = rows(x, "x", x.scalar_type(), x.sizes(), dev, C);
        if (pz != Py_None) {
            z = &cuda_tensor(pz, "z");
            zs = rows(*z, "z", x.scalar_type(), x.sizes(), dev, C);
        }
    }
    const float* weight() const { return static_cast<const float*>(w.data_ptr()); }
    const void* gate() const { return z ? z->data_ptr() : nullptr; }
};

// group_norm(x, weight, bias, z, norm, act, eps, y) -> y
PyObject* group_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    GDN_ARGS(8);
    const NormArgs p(a[0], a[1], a[2], a[3]);
    const c10::cuda::CUDAGuard guard(p.dev);
    const long norm = PyLong_AsLong(a[4]), act = PyLong_AsLong(a[5]);
    const double eps = PyFloat_AsDouble(a[6]);
    if (PyErr_Occurred()) return nullptr;
    int64_t ys;
    const Tensor y = output(a[7], "y", p.x.scalar_type(), p.x.sizes(), p.dev, p.C, ys);
    const gdn_status st = lib.group_norm(
        p.x.data_ptr(), p.xs, p.gate(), p.zs, p.weight(), p.b, p.T, p.H, p.d, p.weight_heads,
        (gdn_norm_kind)norm, (gdn_activation)act, (float)eps, p.io, y.data_ptr(), ys, here(p.dev));
    return st == GDN_OK ? THPVariable_Wrap(y) : status(st);
    END_HANDLE_TH_ERRORS
}

// group_norm_backward(dy, x, weight, bias, z, norm, act, eps, dx, dz, workspace)
//     -> (dx, dweight, dbias, dz)
PyObject* group_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    GDN_ARGS(11);
    const Tensor& dy = cuda_tensor(a[0], "dy");
    const NormArgs p(a[1], a[2], a[3], a[4]);
    const c10::cuda::CUDAGuard guard(p.dev);
    const long norm = PyLong_AsLong(a[5]), act = PyLong_AsLong(a[6]);
    const double eps = PyFloat_AsDouble(a[7]);
    if (PyErr_Occurred()) return nullptr;
    const at::ScalarType dt = p.x.scalar_type();
    const int64_t dys = rows(dy, "dy", dt, p.x.sizes(), p.dev, p.C);
    int64_t dxs, dzs = 0;
    const Tensor dx = output(a[8], "dx", dt, p.x.sizes(), p.dev, p.C, dxs);
    if (!p.z && a[9] != Py_None) throw ValueError("dz without z");
    const Tensor dz =
        p.z ? output(a[9], "dz", dt, p.x.sizes(), p.dev, p.C, dzs) : Tensor();
    const Tensor dw = fresh(p.w.sizes(), at::kFloat, p.dev);
    const Tensor db = p.b ? fresh(p.w.sizes(), at::kFloat, p.dev) : Tensor();
    const Tensor ws = workspace(
        a[10], lib.group_norm_backward_workspace_size(p.T, p.H, p.d, p.weight_heads, p.io), p.dev);
    const gdn_status st = lib.group_norm_backward(
        dy.data_ptr(), dys, p.x.data_ptr(), p.xs, p.gate(), p.zs, p.weight(), p.b, p.T, p.H, p.d,
        p.weight_heads, (gdn_norm_kind)norm, (gdn_activation)act, (float)eps, p.io, dx.data_ptr(),
        dxs, p.z ? dz.data_ptr() : nullptr, dzs, static_cast<float*>(dw.data_ptr()),
        p.b ? static_cast<float*>(db.data_ptr()) : nullptr, ws.data_ptr(), ws.nbytes(), here(p.dev));
    return st == GDN_OK ? tuple_of({dx, dw, db, dz}) : status(st);
    END_HANDLE_TH_ERRORS
}

// frontend_backward(q_raw, k_raw, v_raw, conv_w, a, b, dq, dk, dv, dlog_alpha, dbeta, cu_seqlens,
//     act, eps, workspace) -> (dq_raw, dk_raw, dv_raw, dconv_w, da, db)
PyObject* frontend_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    GDN_ARGS(15);
    const Tensor &q = cuda_tensor(a[0], "q_raw"), &v = cuda_tensor(a[2], "v_raw");
    const at::Device dev = q.device();
    const c10::cuda::CUDAGuard guard(dev);
    const gdn_dtype io = io_type(q, "q_raw");
    if (q.dim() != 3 || v.dim() != 3)
        throw ValueError("q_raw, k_raw and v_raw must be [T, H, d]");
    const at::ScalarType dt = q.scalar_type();
    const int64_t T = q.size(0), H_qk = q.size(1), dk = q.size(2), H_v = v.size(1), dv = v.size(2);
    const int64_t vs[3] = {T, H_v, dv}, gs[2] = {T, H_v}, wshape[2] = {(2 * H_qk + H_v) * dk, 4};
    const int32_t* cu;
    const int32_t N = sequences(a[11], dev, cu);
    const auto at_qk = [&](int i, const char* name) {
        return dense(a[i], name, dt, q.sizes(), dev).data_ptr();
    };
    const auto at_v = [&](int i, const char* name) { return dense(a[i], name, dt, vs, dev).data_ptr(); };
    const auto gate = [&](int i, const char* name) {
        return static_cast<const float*>(dense(a[i], name, at::kFloat, gs, dev).data_ptr());
    };
    const void *pq = at_qk(0, "q_raw"), *pk = at_qk(1, "k_raw"), *pv = at_v(2, "v_raw");
    const void *gq = at_qk(6, "dq"), *gk = at_qk(7, "dk"), *gv = at_v(8, "dv");
    const float *ga = gate(4, "a"), *gb = gate(5, "b"), *gla = gate(9, "dlog_alpha"),
                *gbe = gate(10, "dbeta");
    const float* w =
        static_cast<const float*>(dense(a[3], "conv_w", at::kFloat, wshape, dev).data_ptr());
    const long act = PyLong_AsLong(a[12]);
    const double eps = PyFloat_AsDouble(a[13]);
    if (PyErr_Occurred()) return nullptr;
    const Tensor dq = fresh(q.sizes(), dt, dev), dkr = fresh(q.sizes(), dt, dev),
                 dvr = fresh(vs, dt, dev), dw = fresh(wshape, at::kFloat, dev),
                 da = fresh(gs, at::kFloat, dev), db = fresh(gs, at::kFloat, dev);
    const int32_t T32 = size32(T, "T"), hq = size32(H_qk, "H_qk"), hv = size32(H_v, "H_v"),
                  d1 = size32(dk, "d"), d2 = size32(dv, "d");
    const Tensor ws = workspace(
        a[14], lib.frontend_backward_workspace_size(T32, hq, hv, d1, d2, io), dev);
    const gdn_status st = lib.frontend_backward(
        pq, pk, pv, w, ga, gb, cu, gq, gk, gv, gla, gbe, N, T32, hq, hv, d1, d2, io,
        (gdn_activation)act, (float)eps, dq.data_ptr(), dkr.data_ptr(), dvr.data_ptr(),
        static_cast<float*>(dw.data_ptr()), static_cast<float*>(da.data_ptr()),
        static_cast<float*>(db.data_ptr()), ws.data_ptr(), ws.nbytes(), here(dev));
    return st == GDN_OK ? tuple_of({dq, dkr, dvr, dw, da, db}) : status(st);
    END_HANDLE_TH_ERRORS
}

// bind(address, ...): the C ABI's functions, in the order of Table.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    GDN_ARGS(8);
    void* p[8];
    for (int i = 0; i < 8; ++i) p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
    static_assert(sizeof(Table) == sizeof(p), "one address per entry");
    memcpy(&lib, p, sizeof(p));
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

#define GDN_METHOD(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {GDN_METHOD(bind), GDN_METHOD(scan), GDN_METHOD(scan_backward),
                         GDN_METHOD(scan_step), GDN_METHOD(group_norm),
                         GDN_METHOD(group_norm_backward), GDN_METHOD(frontend_backward),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_gdn_torch", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__gdn_torch() { return PyModule_Create(&module); }
