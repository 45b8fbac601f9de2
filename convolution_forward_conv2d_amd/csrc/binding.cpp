// binding.cpp -- the feed-forward operators on torch tensors of the plain
// layout: contiguous, of matching types, on the current device.
//
// A call on one token is over in 4 us on the GPU; marshalling it in Python took
// 9 to 12.  Each function here checks whether its arguments are of the plain
// layout, allocates the outputs and calls the C ABI on torch's current stream;
// for anything else, wrong arguments among them, it returns None, and the
// Python function of the same name goes through its own checks.
#include <Python.h>

#include <initializer_list>
#include <unordered_map>

#include <ATen/ATen.h>
#include <ATen/EmptyTensor.h>
#include <ATen/record_function.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "miconv.h"

namespace {

using at::Tensor;

// This thread's handle on a device, bound to torch's current stream there.
mic_handle handle_on(int device)
{
    struct Bound {
        mic_handle handle = nullptr;
        hipStream_t stream = nullptr;
        ~Bound()
        {
            if (handle) mic_destroy(handle);
        }
    };
    static thread_local std::unordered_map<int, Bound> bound;
    Bound& b = bound[device];
    if (!b.handle && mic_create(&b.handle) != MIC_STATUS_SUCCESS) return nullptr;
    const hipStream_t stream = c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream();
    if (stream != b.stream) {
        if (mic_set_stream(b.handle, stream) != MIC_STATUS_SUCCESS) return nullptr;
        b.stream = stream;
    }
    return b.handle;
}

const Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// An argument that may be None; false: neither that nor a tensor.
bool maybe(PyObject* o, const Tensor*& t)
{
    t = o == Py_None ? nullptr : tensor(o);
    return o == Py_None || t;
}

bool dtype_of(const Tensor& t, mic_dtype& d)
{
    switch (t.scalar_type()) {
    case at::kFloat: d = MIC_DTYPE_F32; return true;
    case at::kBFloat16: d = MIC_DTYPE_BF16; return true;
    case at::kFloat8_e4m3fn: d = MIC_DTYPE_F8_E4M3; return true;
    default: return false;
    }
}

// The rows x features a call starts from.
bool plain_rows(const Tensor* t, int64_t& rows, int64_t& cols)
{
    if (!t || !t->is_cuda() || t->dim() < 1 || !t->is_contiguous() || t->numel() == 0) return false;
    if (t->get_device() != c10::hip::current_device()) return false;
    cols = t->size(-1);
    rows = t->numel() / cols;
    return rows < INT32_MAX && cols < INT32_MAX;
}

// Of that type and shape, contiguous, on like's device.
bool plain(const Tensor& t, at::ScalarType type, const Tensor& like, std::initializer_list<int64_t> shape)
{
    if (t.scalar_type() != type || t.device() != like.device() || !t.is_contiguous()) return false;
    return t.sizes() == at::IntArrayRef(shape.begin(), shape.size());
}

// The same with any leading dimensions of `rows` rows together.
bool plain_matrix(const Tensor& t, at::ScalarType type, const Tensor& like, int64_t rows, int64_t cols)
{
    return t.scalar_type() == type && t.device() == like.device() && t.is_contiguous() && t.dim() >= 1
           && t.size(-1) == cols && t.numel() == rows * cols;
}

bool plain_scale(const Tensor& t, const Tensor& like, int64_t rows)
{
    return t.scalar_type() == at::kFloat && t.device() == like.device() && t.is_contiguous() && t.numel() == rows;
}

void* data(const Tensor* t) { return t ? t->data_ptr() : nullptr; }
float* floats(const Tensor* t) { return t ? static_cast<float*>(t->data_ptr()) : nullptr; }

// An uninitialised tensor on the current device.  From torch's own allocator, without the dispatcher's way to it, which
// takes longer than the allocation (a norm of one token allocates four); through the dispatcher where something there
// looks at allocations or fills them: a dispatch mode, a profiler, deterministic algorithms.
Tensor fresh(at::IntArrayRef sizes, at::ScalarType type)
{
    if (c10::impl::TorchDispatchModeTLS::any_modes_set() || at::hasCallbacks() || at::globalContext().deterministicAlgorithms())
        return at::empty(sizes, at::TensorOptions().dtype(type).device(at::kCUDA));
    static c10::Allocator* const from = at::empty({0}, at::TensorOptions().dtype(at::kByte).device(at::kCUDA)).storage().allocator();
    return Tensor(at::detail::empty_generic(sizes, from, c10::DispatchKeySet(c10::DispatchKey::CUDA), type, std::nullopt));
}

Tensor rows_of(const Tensor& x, int64_t cols, at::ScalarType type)
{
    auto shape = x.sizes().vec();
    shape.back() = cols;
    return fresh(shape, type);
}

Tensor like(const Tensor& t, at::ScalarType type) { return fresh(t.sizes(), type); }

// Whether the rows of a contiguous matrix count as aligned: a call on such operands copies none.
bool even(const Tensor& t)
{
    const int64_t pitch = t.size(-1) * (int64_t)t.element_size();
    return (reinterpret_cast<uintptr_t>(t.data_ptr()) | (uintptr_t)pitch) % 16 == 0 && pitch < int64_t(1) << 22;
}

// A workspace of the size the library asks for; sizes are kept by call and shape.
template <class Ask> bool workspace(int call, mic_dtype d, int64_t m, int64_t n, int64_t k, const Tensor& x, Tensor& space,
                                    size_t& bytes, Ask ask)
{
    struct Key {
        int64_t call, m, n, k;
        bool operator==(const Key& o) const { return call == o.call && m == o.m && n == o.n && k == o.k; }
    };
    struct Hash {
        size_t operator()(const Key& v) const
        {
            return (size_t)(((v.m * 1000003 + v.n) * 1000003 + v.k) * 1000003 + v.call);
        }
    };
    static thread_local std::unordered_map<Key, size_t, Hash> sizes;
    const Key key = {(call * 8 + (int)d) * 64 + x.get_device(), m, n, k};
    const auto at_key = sizes.find(key);
    if (at_key != sizes.end()) {
        bytes = at_key->second;
    } else {
        if (ask(&bytes) != MIC_STATUS_SUCCESS) return false;
        if (sizes.size() > 4096) sizes.clear();
        sizes.emplace(key, bytes);
    }
    if (bytes) space = fresh({(int64_t)bytes}, at::kByte);
    return true;
}

// A truth value; false, with the exception set: it has none, as a tensor has not unless it is one bool.
bool flag(PyObject* o, const char* name, bool& v)
{
    const Tensor* t = tensor(o);
    if (t && (t->scalar_type() != at::kBool || t->numel() != 1)) {
        PyErr_Format(PyExc_TypeError, "%s must be True or False, not a tensor", name);
        return false;
    }
    const int is = PyObject_IsTrue(o);
    v = is > 0;
    return is >= 0;
}

PyObject* wrap(Tensor t) { return THPVariable_Wrap(std::move(t)); }

PyObject* none()
{
    Py_INCREF(Py_None);
    return Py_None;
}

PyObject* pack(std::initializer_list<PyObject*> items)
{
    PyObject* t = PyTuple_New((Py_ssize_t)items.size());
    Py_ssize_t i = 0;
    for (PyObject* o : items) PyTuple_SET_ITEM(t, i++, o);
    return t;
}

// (x, weight, residual, eps, e4m3) -> (y, sum, rstd, scale)
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    const Tensor *x, *w, *residual;
    int64_t rows, cols;
    mic_dtype d;
    if (n_args != 5 || !plain_rows(x = tensor(a[0]), rows, cols) || !(w = tensor(a[1])) || !maybe(a[2], residual))
        return none();
    const double eps = PyFloat_AsDouble(a[3]);
    if (PyErr_Occurred()) return nullptr;
    bool e4m3;
    if (!flag(a[4], "e4m3", e4m3)) return nullptr;
    const auto type = x->scalar_type();
    if (!dtype_of(*x, d) || d == MIC_DTYPE_F8_E4M3 || !plain(*w, type, *x, {cols})) return none();
    if (residual && (residual->sizes() != x->sizes() || !plain_matrix(*residual, type, *x, rows, cols))) return none();
    const mic_handle h = handle_on(x->get_device());
    if (!h) return none();
    Tensor y = like(*x, e4m3 ? at::kFloat8_e4m3fn : type), sum, scale;
    if (residual) sum = like(*x, type);
    Tensor rstd = fresh(x->sizes().slice(0, x->dim() - 1), at::kFloat);
    if (e4m3) scale = like(rstd, at::kFloat);
    if (mic_rms_norm(h, d, e4m3 ? MIC_DTYPE_F8_E4M3 : d, (int)rows, (int)cols, eps, x->data_ptr(), cols, data(residual), cols,
                     w->data_ptr(), y.data_ptr(), cols, residual ? sum.data_ptr() : nullptr, cols,
                     static_cast<float*>(rstd.data_ptr()), e4m3 ? static_cast<float*>(scale.data_ptr()) : nullptr)
        != MIC_STATUS_SUCCESS)
        return none();
    PyObject* s = a[0];
    if (residual) s = wrap(sum);
    else Py_INCREF(s);
    return pack({wrap(y), s, wrap(rstd), e4m3 ? wrap(scale) : none()});
    END_HANDLE_TH_ERRORS
}

// (dy, sum, weight, rstd, dsum, need_dweight) -> (dx, dweight or None)
PyObject* rms_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    const Tensor *dy, *sum, *w, *rstd, *dsum;
    int64_t rows, cols;
    mic_dtype d;
    if (n_args != 6 || !plain_rows(dy = tensor(a[0]), rows, cols) || !(sum = tensor(a[1])) || !(w = tensor(a[2]))
        || !(rstd = tensor(a[3])) || !maybe(a[4], dsum))
        return none();
    bool need_dw;
    if (!flag(a[5], "need_dweight", need_dw)) return nullptr;
    const auto type = dy->scalar_type();
    if (!dtype_of(*dy, d) || d == MIC_DTYPE_F8_E4M3 || !plain_matrix(*sum, type, *dy, rows, cols)
        || !plain(*w, type, *dy, {cols}) || !plain_scale(*rstd, *dy, rows)
        || (dsum && !plain_matrix(*dsum, type, *dy, rows, cols)))
        return none();
    const mic_handle h = handle_on(dy->get_device());
    Tensor space;
    size_t bytes = 0;
    if (!h || (need_dw && !workspace(0, d, rows, cols, 0, *dy, space, bytes, [&](size_t* b) {
            return mic_rms_norm_backward_workspace(h, (int)rows, (int)cols, b);
        })))
        return none();
    Tensor dx = like(*dy, type), dw;
    if (need_dw) dw = like(*w, type);
    if (mic_rms_norm_backward(h, d, (int)rows, (int)cols, dy->data_ptr(), cols, sum->data_ptr(), cols, w->data_ptr(),
                              floats(rstd), data(dsum), cols, dx.data_ptr(), cols, need_dw ? dw.data_ptr() : nullptr,
                              bytes ? space.data_ptr() : nullptr, bytes)
        != MIC_STATUS_SUCCESS)
        return none();
    return pack({wrap(dx), need_dw ? wrap(dw) : none()});
    END_HANDLE_TH_ERRORS
}

// The scales of a forward call, there where the operands are e4m3 and only there, and the output's type.
bool layer_types(mic_dtype d, bool wide, std::initializer_list<const Tensor*> scales, at::ScalarType type,
                 at::ScalarType& out, mic_dtype& out_d)
{
    for (const Tensor* s : scales)
        if ((d == MIC_DTYPE_F8_E4M3) != (s != nullptr)) return false;
    if (d != MIC_DTYPE_F8_E4M3) out = type, out_d = d;
    else out = wide ? at::kFloat : at::kBFloat16, out_d = wide ? MIC_DTYPE_F32 : MIC_DTYPE_BF16;
    return true;
}

// (x, w, bias, residual, act, x_scale, w_scale, out in fp32, preact, fast_sums) -> (y, z or None)
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    const Tensor *x, *w, *bias, *residual, *xs, *ws;
    int64_t m, k;
    mic_dtype d, out_d;
    at::ScalarType out;
    if (n_args != 10 || !plain_rows(x = tensor(a[0]), m, k) || !(w = tensor(a[1])) || !maybe(a[2], bias)
        || !maybe(a[3], residual) || !maybe(a[5], xs) || !maybe(a[6], ws) || !dtype_of(*x, d) || w->dim() != 2)
        return none();
    bool wide, keep, fast;
    if (!flag(a[7], "out in fp32", wide) || !flag(a[8], "return_preact", keep) || !flag(a[9], "fast_sums", fast)) return nullptr;
    const int64_t n = w->size(0);
    if (!n || n >= INT32_MAX || !layer_types(d, wide, {xs, ws}, x->scalar_type(), out, out_d)
        || !plain(*w, x->scalar_type(), *x, {n, k}) || (bias && !plain(*bias, out, *x, {n}))
        || (residual && !plain_matrix(*residual, out, *x, m, n)) || (xs && !plain_scale(*xs, *x, m))
        || (ws && (!plain_scale(*ws, *x, n) || ws->dim() != 1)))
        return none();
    const long act = PyLong_AsLong(a[4]);
    if (act == -1 && PyErr_Occurred()) return nullptr;
    const mic_handle h = handle_on(x->get_device());
    const bool aligned = even(*x) && even(*w);
    Tensor space;
    size_t bytes;
    if (!h || !workspace(aligned ? 5 : 1, d, m, n, k, *x, space, bytes, [&](size_t* b) {
            return aligned ? mic_linear_forward_workspace_aligned(h, d, (int)m, (int)n, (int)k, b)
                           : mic_linear_forward_workspace(h, d, (int)m, (int)n, (int)k, b);
        }))
        return none();
    Tensor y = rows_of(*x, n, out), z;
    if (keep) z = like(y, out);
    if (mic_linear_forward(h, d, out_d, (mic_activation)act, fast, (int)m, (int)n, (int)k, x->data_ptr(), k,
                           w->data_ptr(), k, floats(xs), floats(ws), data(bias), data(residual), n, y.data_ptr(), n,
                           keep ? z.data_ptr() : nullptr, n, bytes ? space.data_ptr() : nullptr, bytes)
        != MIC_STATUS_SUCCESS)
        return none();
    return pack({wrap(y), keep ? wrap(z) : none()});
    END_HANDLE_TH_ERRORS
}

// (dy, x, w, preact, act, bias, need_dx, need_dw) -> (dx, dw, dbias), each None where not asked for
PyObject* linear_backward(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    const Tensor *dy, *x, *w, *pre;
    int64_t m, n;
    mic_dtype d;
    if (n_args != 8 || !plain_rows(dy = tensor(a[0]), m, n) || !(x = tensor(a[1])) || !(w = tensor(a[2]))
        || !maybe(a[3], pre) || !dtype_of(*dy, d) || d == MIC_DTYPE_F8_E4M3 || x->dim() < 1)
        return none();
    bool bias, need_dx, need_dw;
    if (!flag(a[5], "bias", bias) || !flag(a[6], "need_dx", need_dx) || !flag(a[7], "need_dw", need_dw)) return nullptr;
    const long act = PyLong_AsLong(a[4]);
    if (act == -1 && PyErr_Occurred()) return nullptr;
    const auto type = dy->scalar_type();
    const int64_t k = x->size(-1);
    if (!k || k >= INT32_MAX || !plain_matrix(*x, type, *dy, m, k) || !plain(*w, type, *dy, {n, k})
        || (act && (!pre || !plain_matrix(*pre, type, *dy, m, n))))
        return none();
    const mic_handle h = handle_on(dy->get_device());
    const bool aligned = even(*x) && even(*w) && (act || even(*dy));
    Tensor space;
    size_t bytes;
    if (!h || !workspace(aligned ? act ? 6 : 7 : 2, d, m, n, k, *dy, space, bytes, [&](size_t* b) {
            return aligned ? mic_linear_backward_workspace_aligned(h, d, (mic_activation)act, (int)m, (int)n, (int)k, b)
                           : mic_linear_backward_workspace(h, d, (int)m, (int)n, (int)k, b);
        }))
        return none();
    Tensor dx, dw, db;
    if (need_dx) dx = like(*x, type);
    if (need_dw) dw = like(*w, type);
    if (bias) db = fresh({n}, type);
    if (mic_linear_backward(h, d, (mic_activation)act, (int)m, (int)n, (int)k, dy->data_ptr(), n, x->data_ptr(), k,
                            w->data_ptr(), k, act ? data(pre) : nullptr, n, need_dx ? dx.data_ptr() : nullptr, k,
                            need_dw ? dw.data_ptr() : nullptr, k,
                            bias ? db.data_ptr() : nullptr, bytes ? space.data_ptr() : nullptr, bytes)
        != MIC_STATUS_SUCCESS)
        return none();
    return pack({need_dx ? wrap(dx) : none(), need_dw ? wrap(dw) : none(), bias ? wrap(db) : none()});
    END_HANDLE_TH_ERRORS
}

// (x, w_gate, w_up, act, x_scale, w_gate_scale, w_up_scale, out in fp32, products, fast_sums) -> (y, gate, up)
PyObject* gated_linear(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    const Tensor *x, *wg, *wu, *xs, *gs, *us;
    int64_t m, k;
    mic_dtype d, out_d;
    at::ScalarType out;
    if (n_args != 10 || !plain_rows(x = tensor(a[0]), m, k) || !(wg = tensor(a[1])) || !(wu = tensor(a[2]))
        || !maybe(a[4], xs) || !maybe(a[5], gs) || !maybe(a[6], us) || !dtype_of(*x, d) || wg->dim() != 2)
        return none();
    bool wide, keep, fast;
    if (!flag(a[7], "out in fp32", wide) || !flag(a[8], "return_products", keep) || !flag(a[9], "fast_sums", fast)) return nullptr;
    const int64_t n = wg->size(0);
    const auto type = x->scalar_type();
    if (!n || n >= INT32_MAX || !layer_types(d, wide, {xs, gs, us}, type, out, out_d) || !plain(*wg, type, *x, {n, k})
        || !plain(*wu, type, *x, {n, k}) || (xs && !plain_scale(*xs, *x, m))
        || (gs && (!plain_scale(*gs, *x, n) || gs->dim() != 1)) || (us && (!plain_scale(*us, *x, n) || us->dim() != 1)))
        return none();
    const long act = PyLong_AsLong(a[3]);
    if (act == -1 && PyErr_Occurred()) return nullptr;
    const mic_handle h = handle_on(x->get_device());
    const bool aligned = even(*x) && even(*wg) && even(*wu);
    Tensor space;
    size_t bytes;
    if (!h || !workspace(aligned ? 8 : 3, d, m, n, k, *x, space, bytes, [&](size_t* b) {
            return aligned ? mic_gated_linear_forward_workspace_aligned(h, d, (int)m, (int)n, (int)k, b)
                           : mic_gated_linear_forward_workspace(h, d, (int)m, (int)n, (int)k, b);
        }))
        return none();
    Tensor y = rows_of(*x, n, out), gate, up;
    if (keep) gate = like(y, out), up = like(y, out);
    if (mic_gated_linear_forward(h, d, out_d, (mic_activation)act, fast, (int)m, (int)n, (int)k, x->data_ptr(),
                                 k, wg->data_ptr(), k, wu->data_ptr(), k, floats(xs), floats(gs), floats(us), y.data_ptr(),
                                 n, keep ? gate.data_ptr() : nullptr, n, keep ? up.data_ptr() : nullptr, n,
                                 bytes ? space.data_ptr() : nullptr, bytes)
        != MIC_STATUS_SUCCESS)
        return none();
    return pack({wrap(y), keep ? wrap(gate) : none(), keep ? wrap(up) : none()});
    END_HANDLE_TH_ERRORS
}

// (dy, x, w_gate, w_up, gate, up, act, need_dx, need_dw) -> (dx, dw_gate, dw_up), each None where not asked for
PyObject* gated_linear_backward(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    const Tensor *dy, *x, *wg, *wu, *gate, *up;
    int64_t m, n;
    mic_dtype d;
    if (n_args != 9 || !plain_rows(dy = tensor(a[0]), m, n) || !(x = tensor(a[1])) || !(wg = tensor(a[2]))
        || !(wu = tensor(a[3])) || !(gate = tensor(a[4])) || !(up = tensor(a[5])) || !dtype_of(*dy, d)
        || d == MIC_DTYPE_F8_E4M3 || x->dim() < 1)
        return none();
    bool need_dx, need_dw;
    if (!flag(a[7], "need_dx", need_dx) || !flag(a[8], "need_dw", need_dw)) return nullptr;
    const long act = PyLong_AsLong(a[6]);
    if (act == -1 && PyErr_Occurred()) return nullptr;
    const auto type = dy->scalar_type();
    const int64_t k = x->size(-1);
    if (!k || k >= INT32_MAX || !plain_matrix(*x, type, *dy, m, k) || !plain(*wg, type, *dy, {n, k})
        || !plain(*wu, type, *dy, {n, k}) || !plain_matrix(*gate, type, *dy, m, n) || !plain_matrix(*up, type, *dy, m, n))
        return none();
    const mic_handle h = handle_on(dy->get_device());
    const bool aligned = even(*x) && even(*wg) && even(*wu);
    Tensor space;
    size_t bytes;
    if (!h || !workspace(aligned ? 9 : 4, d, m, n, k, *dy, space, bytes, [&](size_t* b) {
            return aligned ? mic_gated_linear_backward_workspace_aligned(h, d, (int)m, (int)n, (int)k, b)
                           : mic_gated_linear_backward_workspace(h, d, (int)m, (int)n, (int)k, b);
        }))
        return none();
    Tensor dx, dg, du;
    if (need_dx) dx = like(*x, type);
    if (need_dw) dg = like(*wg, type), du = like(*wu, type);
    if (mic_gated_linear_backward(h, d, (mic_activation)act, (int)m, (int)n, (int)k, dy->data_ptr(), n, x->data_ptr(), k,
                                  wg->data_ptr(), k, wu->data_ptr(), k, gate->data_ptr(), n, up->data_ptr(), n,
                                  need_dx ? dx.data_ptr() : nullptr, k, need_dw ? dg.data_ptr() : nullptr, k,
                                  need_dw ? du.data_ptr() : nullptr, k,
                                  bytes ? space.data_ptr() : nullptr, bytes)
        != MIC_STATUS_SUCCESS)
        return none();
    return pack({need_dx ? wrap(dx) : none(), need_dw ? wrap(dg) : none(), need_dw ? wrap(du) : none()});
    END_HANDLE_TH_ERRORS
}

// (x, weight, bias, residual, eps, e4m3) -> (y, sum, mean, rstd, scale)
PyObject* layer_norm(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    const Tensor *x, *w, *bias, *residual;
    int64_t rows, cols;
    mic_dtype d;
    if (n_args != 6 || !plain_rows(x = tensor(a[0]), rows, cols) || !(w = tensor(a[1])) || !maybe(a[2], bias)
        || !maybe(a[3], residual))
        return none();
    const double eps = PyFloat_AsDouble(a[4]);
    if (PyErr_Occurred()) return nullptr;
    bool e4m3;
    if (!flag(a[5], "e4m3", e4m3)) return nullptr;
    const auto type = x->scalar_type();
    if (!dtype_of(*x, d) || d == MIC_DTYPE_F8_E4M3 || !plain(*w, type, *x, {cols}) || (bias && !plain(*bias, type, *x, {cols})))
        return none();
    if (residual && (residual->sizes() != x->sizes() || !plain_matrix(*residual, type, *x, rows, cols))) return none();
    const mic_handle h = handle_on(x->get_device());
    if (!h) return none();
    Tensor y = like(*x, e4m3 ? at::kFloat8_e4m3fn : type), sum, scale;
    if (residual) sum = like(*x, type);
    Tensor mean = fresh(x->sizes().slice(0, x->dim() - 1), at::kFloat);
    Tensor rstd = like(mean, at::kFloat);
    if (e4m3) scale = like(mean, at::kFloat);
    if (mic_layer_norm(h, d, e4m3 ? MIC_DTYPE_F8_E4M3 : d, (int)rows, (int)cols, eps, x->data_ptr(), cols, data(residual), cols,
                       w->data_ptr(), data(bias), y.data_ptr(), cols, residual ? sum.data_ptr() : nullptr, cols,
                       floats(&mean), floats(&rstd), e4m3 ? floats(&scale) : nullptr)
        != MIC_STATUS_SUCCESS)
        return none();
    PyObject* s = a[0];
    if (residual) s = wrap(sum);
    else Py_INCREF(s);
    return pack({wrap(y), s, wrap(mean), wrap(rstd), e4m3 ? wrap(scale) : none()});
    END_HANDLE_TH_ERRORS
}

// (dy, sum, weight, mean, rstd, dsum, bias, need_dweight) -> (dx, dweight, dbias), the last two None where not asked for
PyObject* layer_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    const Tensor *dy, *sum, *w, *mean, *rstd, *dsum;
    int64_t rows, cols;
    mic_dtype d;
    if (n_args != 8 || !plain_rows(dy = tensor(a[0]), rows, cols) || !(sum = tensor(a[1])) || !(w = tensor(a[2]))
        || !(mean = tensor(a[3])) || !(rstd = tensor(a[4])) || !maybe(a[5], dsum))
        return none();
    bool bias, need_dw;
    if (!flag(a[6], "bias", bias) || !flag(a[7], "need_dweight", need_dw)) return nullptr;
    const auto type = dy->scalar_type();
    if (!dtype_of(*dy, d) || d == MIC_DTYPE_F8_E4M3 || !plain_matrix(*sum, type, *dy, rows, cols)
        || !plain(*w, type, *dy, {cols}) || !plain_scale(*mean, *dy, rows) || !plain_scale(*rstd, *dy, rows)
        || (dsum && !plain_matrix(*dsum, type, *dy, rows, cols)))
        return none();
    const mic_handle h = handle_on(dy->get_device());
    Tensor space;
    size_t bytes = 0;
    if (!h || ((need_dw || bias) && !workspace(10, d, rows, cols, 0, *dy, space, bytes, [&](size_t* b) {
            return mic_layer_norm_backward_workspace(h, (int)rows, (int)cols, b);
        })))
        return none();
    Tensor dx = like(*dy, type), dw, db;
    if (need_dw) dw = like(*w, type);
    if (bias) db = like(*w, type);
    if (mic_layer_norm_backward(h, d, (int)rows, (int)cols, dy->data_ptr(), cols, sum->data_ptr(), cols, w->data_ptr(),
                                floats(mean), floats(rstd), data(dsum), cols, dx.data_ptr(), cols,
                                need_dw ? dw.data_ptr() : nullptr, bias ? db.data_ptr() : nullptr,
                                bytes ? space.data_ptr() : nullptr, bytes)
        != MIC_STATUS_SUCCESS)
        return none();
    return pack({wrap(dx), need_dw ? wrap(dw) : none(), bias ? wrap(db) : none()});
    END_HANDLE_TH_ERRORS
}

// (x, p, seed, offset, residual) -> y; any shape, everything contiguous
PyObject* dropout(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    const Tensor *x, *residual;
    mic_dtype d;
    if (n_args != 5 || !(x = tensor(a[0])) || !maybe(a[4], residual)) return none();
    if (!x->is_cuda() || !x->is_contiguous() || x->numel() == 0 || x->get_device() != c10::hip::current_device()
        || !dtype_of(*x, d) || d == MIC_DTYPE_F8_E4M3)
        return none();
    const auto type = x->scalar_type();
    if (residual
        && (residual->scalar_type() != type || residual->device() != x->device() || !residual->is_contiguous()
            || residual->sizes() != x->sizes()))
        return none();
    if (!(PyFloat_Check(a[1]) || (PyLong_Check(a[1]) && !PyBool_Check(a[1])))) return none();
    const double p = PyFloat_AsDouble(a[1]);
    uint64_t number[2] = {0, 0};
    const uint64_t* state = nullptr;
    for (int i = 0; i < 2; ++i) {
        if (const Tensor* t = i ? nullptr : tensor(a[2])) {
            if (t->scalar_type() != at::kLong || t->device() != x->device() || t->dim() != 1 || t->size(0) != 2
                || !t->is_contiguous())
                return none();
            state = static_cast<const uint64_t*>(t->data_ptr());
            continue;
        }
        if (!PyLong_Check(a[2 + i]) || PyBool_Check(a[2 + i])) return none();
        number[i] = PyLong_AsUnsignedLongLong(a[2 + i]);
        if (PyErr_Occurred()) {
            PyErr_Clear();                                     // out of range: the Python checks say so
            return none();
        }
    }
    const mic_handle h = handle_on(x->get_device());
    if (!h) return none();
    Tensor y = like(*x, type);
    const int64_t n = x->numel();
    if (mic_dropout(h, d, 1, n, p, number[0], number[1], state, x->data_ptr(), n, data(residual), n, y.data_ptr(), n)
        != MIC_STATUS_SUCCESS)
        return none();
    return wrap(y);
    END_HANDLE_TH_ERRORS
}

// Numbers of a loss; false: to be looked at by the Python checks.
bool loss_numbers(PyObject* index, PyObject* share, int64_t& ignore, double& smoothing)
{
    if (!PyLong_Check(index) || PyBool_Check(index) || !(PyFloat_Check(share) || (PyLong_Check(share) && !PyBool_Check(share))))
        return false;
    ignore = PyLong_AsLongLong(index);
    smoothing = PyFloat_AsDouble(share);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    return true;
}

// The operands of a loss: w (n, k), target of x's leading shape, bias (n) or none.
bool loss_operands(const Tensor& x, const Tensor& w, const Tensor& target, const Tensor* bias, int64_t n, int64_t k)
{
    const auto type = x.scalar_type();
    return n > 0 && n < INT32_MAX && plain(w, type, x, {n, k}) && target.scalar_type() == at::kLong
           && target.device() == x.device() && target.is_contiguous() && target.sizes() == x.sizes().slice(0, x.dim() - 1)
           && (!bias || plain(*bias, type, x, {n}));
}

// (x, w, target, bias, reduction, ignore_index, label_smoothing) -> (loss, lse, count)
PyObject* linear_cross_entropy(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    const Tensor *x, *w, *target, *bias;
    int64_t m, k, ignore;
    double smoothing;
    mic_dtype d;
    if (n_args != 7 || !plain_rows(x = tensor(a[0]), m, k) || !(w = tensor(a[1])) || !(target = tensor(a[2]))
        || !maybe(a[3], bias) || !dtype_of(*x, d) || d == MIC_DTYPE_F8_E4M3 || w->dim() != 2
        || !loss_numbers(a[5], a[6], ignore, smoothing))
        return none();
    const long reduction = PyLong_AsLong(a[4]);
    if (reduction == -1 && PyErr_Occurred()) return nullptr;
    const int64_t n = w->size(0);
    if (!loss_operands(*x, *w, *target, bias, n, k)) return none();
    const mic_handle h = handle_on(x->get_device());
    const bool aligned = even(*x) && even(*w);
    Tensor space;
    size_t bytes;
    if (!h || !workspace(aligned ? 11 : 12, d, m, n, k, *x, space, bytes, [&](size_t* b) {
            return aligned ? mic_linear_cross_entropy_workspace_aligned(h, d, (int)m, (int)n, (int)k, b)
                           : mic_linear_cross_entropy_workspace(h, d, (int)m, (int)n, (int)k, b);
        }))
        return none();
    const bool each = reduction == MIC_REDUCTION_NONE;
    Tensor lse = fresh(target->sizes(), at::kFloat), loss, count;
    if (each) loss = like(lse, at::kFloat);
    else loss = fresh({}, at::kFloat), count = fresh({}, at::kFloat);
    if (mic_linear_cross_entropy(h, d, (mic_reduction)reduction, (int)m, (int)n, (int)k, x->data_ptr(), k, w->data_ptr(), k,
                                 data(bias), static_cast<const int64_t*>(target->data_ptr()), ignore, smoothing, floats(&loss),
                                 floats(&lse), each ? nullptr : floats(&count), bytes ? space.data_ptr() : nullptr, bytes)
        != MIC_STATUS_SUCCESS)
        return none();
    return pack({wrap(loss), wrap(lse), each ? none() : wrap(count)});
    END_HANDLE_TH_ERRORS
}

// (dloss, x, w, target, lse, bias, count, ignore_index, label_smoothing, need_dx, need_dw, need_dbias) -> (dx, dw, dbias)
PyObject* linear_cross_entropy_backward(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    const Tensor *dloss, *x, *w, *target, *lse, *bias, *count;
    int64_t m, k, ignore;
    double smoothing;
    mic_dtype d;
    if (n_args != 12 || !(dloss = tensor(a[0])) || !plain_rows(x = tensor(a[1]), m, k) || !(w = tensor(a[2]))
        || !(target = tensor(a[3])) || !(lse = tensor(a[4])) || !maybe(a[5], bias) || !maybe(a[6], count) || !dtype_of(*x, d)
        || d == MIC_DTYPE_F8_E4M3 || w->dim() != 2 || !loss_numbers(a[7], a[8], ignore, smoothing))
        return none();
    bool need_dx, need_dw, need_db;
    if (!flag(a[9], "need_dx", need_dx) || !flag(a[10], "need_dw", need_dw) || !flag(a[11], "need_dbias", need_db)) return nullptr;
    const int64_t n = w->size(0);
    const bool each = dloss->dim() > 0 && dloss->sizes() == target->sizes();
    if (!loss_operands(*x, *w, *target, bias, n, k) || !plain_scale(*lse, *x, m) || !plain_scale(*dloss, *x, each ? m : 1)
        || (count && !plain_scale(*count, *x, 1)))
        return none();
    const mic_handle h = handle_on(x->get_device());
    const bool aligned = even(*x) && even(*w);
    Tensor space;
    size_t bytes;
    if (!h || !workspace(aligned ? 13 : 14, d, m, n, k, *x, space, bytes, [&](size_t* b) {
            return aligned ? mic_linear_cross_entropy_backward_workspace_aligned(h, d, (int)m, (int)n, (int)k, b)
                           : mic_linear_cross_entropy_backward_workspace(h, d, (int)m, (int)n, (int)k, b);
        }))
        return none();
    const auto type = x->scalar_type();
    need_db = need_db && bias;
    Tensor dx, dw, db;
    if (need_dx) dx = like(*x, type);
    if (need_dw) dw = like(*w, type);
    if (need_db) db = like(*bias, type);
    if (mic_linear_cross_entropy_backward(h, d, (int)m, (int)n, (int)k, floats(dloss), each, x->data_ptr(), k, w->data_ptr(), k,
                                          data(bias), static_cast<const int64_t*>(target->data_ptr()), ignore, smoothing,
                                          floats(lse), floats(count), need_dx ? dx.data_ptr() : nullptr, k,
                                          need_dw ? dw.data_ptr() : nullptr, k, need_db ? db.data_ptr() : nullptr,
                                          bytes ? space.data_ptr() : nullptr, bytes)
        != MIC_STATUS_SUCCESS)
        return none();
    return pack({need_dx ? wrap(dx) : none(), need_dw ? wrap(dw) : none(), need_db ? wrap(db) : none()});
    END_HANDLE_TH_ERRORS
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(rms_norm), FAST(rms_norm_backward), FAST(linear), FAST(linear_backward),
                         FAST(gated_linear), FAST(gated_linear_backward), FAST(layer_norm),
                         FAST(layer_norm_backward), FAST(dropout), FAST(linear_cross_entropy), FAST(linear_cross_entropy_backward), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", "The feed-forward operators on plainly laid out tensors.", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&module); }
