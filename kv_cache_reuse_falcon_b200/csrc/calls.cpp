// The Python binding's paged and windowed calls: checks of the tensors, the device and its current stream, and
// the call of the C entry point (include/unipin.h).  Serving makes these calls once per layer and step on small
// inputs; checked property by property from Python one took 12 us, of which the kernel's launch was 3.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <initializer_list>
#include <optional>
#include <stdexcept>
#include <string>

#include "unipin.h"

namespace {

struct ValueError : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct PythonError {};   // already set

using Sizes = std::initializer_list<int64_t>;

bool given(PyObject* o) { return o != nullptr && o != Py_None; }

const at::Tensor& tensor(PyObject* o, const char* name)
{
    if (!THPVariable_Check(o)) throw ValueError(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

long long integer(PyObject* o)
{
    PyObject* i = PyNumber_Index(o);
    if (!i) throw PythonError();
    const long long v = PyLong_AsLongLong(i);
    Py_DECREF(i);
    if (v == -1 && PyErr_Occurred()) throw PythonError();
    return v;
}

// As a C int; values outside its range, which no call accepts, become the nearest one.
int as_int(PyObject* o)
{
    const long long v = integer(o);
    return v > INT_MAX ? INT_MAX : (v < INT_MIN ? INT_MIN : (int)v);
}

double real(PyObject* o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError();
    return v;
}

bool truth(PyObject* o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw PythonError();
    return v != 0;
}

const char* type_name(at::ScalarType t)
{
    return t == at::kBFloat16 ? "bfloat16" : (t == at::kFloat ? "float32" : "int32");
}

void fits(const at::Tensor& t, const char* name, at::ScalarType type, Sizes shape)
{
    if (t.scalar_type() == type && t.sizes() == at::IntArrayRef(shape) && t.is_contiguous()) return;
    std::string s;
    for (int64_t n : shape) s += (s.empty() ? "" : ", ") + std::to_string(n);
    throw ValueError(std::string(name) + " must be a contiguous CUDA " + type_name(type) + " tensor [" + s + "]");
}

// A contiguous bfloat16 tensor [T, H, D].
const at::Tensor& token_rows(PyObject* o, const char* name)
{
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != at::kBFloat16 || t.dim() != 3 || !t.is_contiguous())
        throw ValueError(std::string(name) + " must be a contiguous CUDA bfloat16 tensor [T, H, D]");
    return t;
}

// An int32 vector with an entry per request.
const at::Tensor& batch(PyObject* o, const char* name)
{
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != at::kInt || t.dim() != 1 || !t.is_contiguous())
        throw ValueError(std::string(name) + " must be a contiguous CUDA int32 vector");
    return t;
}

const at::Tensor& page_table(PyObject* o, int64_t rows)
{
    const at::Tensor& t = tensor(o, "page_table");
    if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != rows || !t.is_contiguous())
        throw ValueError("page_table must be a contiguous CUDA int32 tensor [" + std::to_string(rows) + ", max_pages]");
    return t;
}

// C ints hold every size of a call.
int small(int64_t n, const char* name)
{
    if (n > INT_MAX) throw ValueError(std::string(name) + " is too long");
    return (int)n;
}

unipin_kvpool pool_of(const at::Tensor& k, const at::Tensor& v, PyObject* scales)
{
    for (const at::Tensor* t : {&k, &v}) {
        const at::ScalarType s = t->scalar_type();
        if ((s != at::kBFloat16 && s != at::kFloat8_e4m3fn && s != at::kByte) || t->dim() != 5 || !t->is_contiguous() ||
            !t->is_cuda())
            throw ValueError(std::string(t == &k ? "pool_k" : "pool_v") +
                             " must be a contiguous CUDA tensor [L, S, H, n_cap, D] of bfloat16 or E4M3 codes "
                             "(float8_e4m3fn or uint8)");
    }
    const bool bf16 = k.scalar_type() == at::kBFloat16;
    if (k.sizes() != v.sizes() || bf16 != (v.scalar_type() == at::kBFloat16))
        throw ValueError("pool_k and pool_v differ in shape or element type");
    unipin_kvpool p;
    p.k = k.data_ptr();
    p.v = v.data_ptr();
    p.L = small(k.size(0), "pool_k"), p.S = small(k.size(1), "pool_k"), p.H = small(k.size(2), "pool_k");
    p.n_cap = small(k.size(3), "pool_k"), p.D = small(k.size(4), "pool_k");
    p.dtype = bf16 ? UNIPIN_POOL_BF16 : UNIPIN_POOL_E4M3;
    p.k_scale = p.v_scale = 1.f;
    if (!bf16 && given(scales)) {
        for (int i = 0; i < 2; ++i) {
            PyObject* s = PySequence_GetItem(scales, i);
            if (!s) throw PythonError();
            const double x = PyFloat_AsDouble(s);
            Py_DECREF(s);
            if (x == -1.0 && PyErr_Occurred()) throw PythonError();
            (i ? p.v_scale : p.k_scale) = (float)x;
        }
    }
    return p;
}

void key_weights_fit(const at::Tensor& w, const unipin_kvpool& p)
{
    fits(w, "key_weights", at::kFloat, {p.L, p.S, p.H, p.n_cap});
}

struct Window {
    int window, n_sinks;
};

Window window_of(PyObject* window, PyObject* n_sinks)
{
    const long long w = given(window) ? integer(window) : INT_MAX, s = integer(n_sinks);
    if (w < 1 || w > INT_MAX || s < 0 || s > INT_MAX)
        throw ValueError("window must be at least 1 (None: no window) and n_sinks at least 0");
    return {(int)w, (int)s};
}

float scale_of(PyObject* scale, int64_t D) { return given(scale) ? (float)real(scale) : (float)(1.0 / std::sqrt((double)D)); }

// The tensors lie on one CUDA device.  While this lives that device is current on the thread, and on it the stream
// of the call: what the call allocates then belongs to that stream.  (Memory from the caller's current stream may
// still have work queued there, which the call's stream does not wait for.)
class Place {
public:
    Place(std::initializer_list<const at::Tensor*> tensors, PyObject* stream) : device_((*tensors.begin())->device())
    {
        bool one = device_.is_cuda();
        for (const at::Tensor* t : tensors) one = one && (!t || t->device() == device_);
        if (!one) {
            std::string s;
            for (const at::Tensor* t : tensors)
                if (t) s += (s.empty() ? "" : ", ") + t->device().str();
            throw ValueError("the tensors must lie on one CUDA device: " + s);
        }
        guard_.set_device(device_);
        const at::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream(device_.index());
        raw_ = current.stream();
        if (given(stream)) {
            PyObject* raw = PyObject_GetAttrString(stream, "cuda_stream");
            if (!raw) throw PythonError();
            raw_ = reinterpret_cast<cudaStream_t>(PyLong_AsUnsignedLongLong(raw));
            Py_DECREF(raw);
            if (PyErr_Occurred()) throw PythonError();
            if (raw_ != current.stream()) {
                caller_ = current;
                stream_guard_.reset_stream(c10::cuda::getStreamFromExternal(raw_, device_.index()));
            }
        }
    }
    void* stream() const { return raw_; }
    // An output: the caller goes on with it on the stream that was current.
    void handed_out(const at::Tensor& t) const
    {
        if (caller_) t.record_stream(caller_->unwrap());
    }

private:
    c10::Device device_;
    c10::cuda::OptionalCUDAGuard guard_;
    c10::cuda::OptionalCUDAStreamGuard stream_guard_;
    cudaStream_t raw_ = nullptr;
    std::optional<c10::cuda::CUDAStream> caller_;   // where the call's stream is another
};

template <typename T = void>
T* address(const at::Tensor* t) { return t ? static_cast<T*>(t->data_ptr()) : nullptr; }

const at::Tensor* optional(PyObject* o, const char* name) { return given(o) ? &tensor(o, name) : nullptr; }

// An output argument of up to three dimensions: the tensor given, or one that is made under the call's stream.
class Output {
public:
    Output(PyObject* o, const char* name, Sizes shape, at::ScalarType type) : type_(type), dims_(shape.size())
    {
        std::copy(shape.begin(), shape.end(), shape_);
        if (!given(o)) return;
        t_ = tensor(o, name);
        fits(t_, name, type, shape);
    }
    const at::Tensor* lent() const { return t_.defined() ? &t_ : nullptr; }
    const at::Tensor& in(const Place& at_, const at::Tensor& like)
    {
        if (!t_.defined()) {
            t_ = at::empty(at::IntArrayRef(shape_, dims_), like.options().dtype(type_));
            at_.handed_out(t_);
        }
        return t_;
    }

private:
    at::Tensor t_;
    at::ScalarType type_;
    size_t dims_;
    int64_t shape_[3];
};

// The workspace argument: "auto" (a fresh buffer of `bytes`, of the current stream: the call's), None, or a contiguous
// tensor.
struct Space {
    at::Tensor made;
    const at::Tensor* tensor = nullptr;
    size_t bytes = 0;
    template <typename F>
    Space(PyObject* o, const at::Tensor& like, F need)
    {
        if (PyUnicode_Check(o)) {
            if (PyUnicode_CompareWithASCIIString(o, "auto") != 0)
                throw ValueError("workspace must be 'auto', None or a CUDA tensor");
            bytes = need();
            if (bytes == 0) return;
            bytes = (bytes + 15) / 16 * 16;
            made = at::empty({(int64_t)bytes}, like.options().dtype(at::kByte));
            tensor = &made;
        } else if (given(o)) {
            tensor = &::tensor(o, "workspace");
            if (!tensor->is_cuda() || !tensor->is_contiguous())
                throw ValueError("workspace must be a contiguous CUDA tensor");
            bytes = tensor->nbytes();
        }
    }
};

PyObject* answer(int rc) { return PyLong_FromLong(rc); }

template <typename... Ts>
PyObject* answer(int rc, const Ts&... ts)
{
    PyObject* r = PyTuple_New(1 + sizeof...(ts));
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, PyLong_FromLong(rc));
    int i = 1;
    (PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(ts)), ...);
    return r;
}

// A method: kArgs arguments by position.
template <PyObject* (*F)(PyObject* const*), int kArgs>
PyObject* guarded(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    if (n != kArgs) {
        PyErr_Format(PyExc_TypeError, "%d arguments by position, got %zd", kArgs, n);
        return nullptr;
    }
    try {
        return F(a);
    } catch (const ValueError& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const PythonError&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// (pool_k, pool_v, layer, k, v, cu_seqlens, new_lens, page_table, first_rows, max_new, key_weights, dev_status, stream,
// pool_scales)
PyObject* pool_write(PyObject* const* a)
{
    const at::Tensor &pk = tensor(a[0], "pool_k"), &pv = tensor(a[1], "pool_v");
    const unipin_kvpool pool = pool_of(pk, pv, a[13]);
    const at::Tensor &k = token_rows(a[3], "k"), &v = token_rows(a[4], "v");
    const int64_t T = k.size(0);
    fits(k, "k", at::kBFloat16, {T, pool.H, pool.D});
    fits(v, "v", at::kBFloat16, {T, pool.H, pool.D});
    const at::Tensor& n = batch(a[6], "new_lens");
    const int64_t B = n.size(0);
    const at::Tensor &cu = tensor(a[5], "cu_seqlens"), &first = tensor(a[8], "first_rows");
    fits(cu, "cu_seqlens", at::kInt, {B + 1});
    fits(first, "first_rows", at::kInt, {B});
    const at::Tensor& table = page_table(a[7], B);
    const at::Tensor *w = optional(a[10], "key_weights"), *status = optional(a[11], "dev_status");
    if (w) key_weights_fit(*w, pool);
    const int layer = as_int(a[2]), max_new = as_int(a[9]);
    const Place at_({&pk, &pv, &k, &v, &cu, &n, &table, &first, w, status}, a[12]);
    return answer(unipin_paged_pool_write(&pool, layer, k.data_ptr(), v.data_ptr(), address<int>(&cu), address<int>(&n),
                                          address<int>(&table), small(table.size(1), "page_table"), address<int>(&first),
                                          small(B, "new_lens"), max_new, small(T, "k"), address<float>(w),
                                          address<int>(status), at_.stream()));
}

// (q, page_table, lens, pool_k, pool_v, layer, max_len, k_self, v_self, window, n_sinks, key_weights, out, out_fp32, scale,
// workspace, dev_status, stream, pool_scales)
PyObject* decode(PyObject* const* a)
{
    const at::Tensor& q = token_rows(a[0], "q");
    const int64_t R = q.size(0), H = q.size(1), D = q.size(2);
    const at::Tensor &pk = tensor(a[3], "pool_k"), &pv = tensor(a[4], "pool_v");
    const unipin_kvpool pool = pool_of(pk, pv, a[18]);
    if (pool.D != D || pool.H < 1 || H % pool.H != 0)
        throw ValueError("q must have the pool's head dim and a multiple of its " + std::to_string(pool.H) + " heads");
    const at::Tensor *ks = optional(a[7], "k_self"), *vs = optional(a[8], "v_self");
    if (!ks != !vs) throw ValueError("k_self and v_self go together");
    if (ks) {
        fits(*ks, "k_self", at::kBFloat16, {R, pool.H, D});
        fits(*vs, "v_self", at::kBFloat16, {R, pool.H, D});
    }
    const at::Tensor& lens = tensor(a[2], "lens");
    fits(lens, "lens", at::kInt, {R});
    const at::Tensor& table = page_table(a[1], R);
    const at::Tensor *w = optional(a[11], "key_weights"), *status = optional(a[16], "dev_status");
    if (w) key_weights_fit(*w, pool);
    const Window win = window_of(a[9], a[10]);
    const int layer = as_int(a[5]), max_len = as_int(a[6]);
    const bool fp32 = truth(a[13]);
    const float scale = scale_of(a[14], D);
    Output made(a[12], "out", {R, H, D}, fp32 ? at::kFloat : at::kBFloat16);
    const Place at_({&q, ks, vs, &table, &lens, &pk, &pv, w, made.lent(), status}, a[17]);
    const at::Tensor& out = made.in(at_, q);
    const Space ws(a[15], q, [&] {
        return unipin_paged_decode_workspace_size(&pool, small(R, "q"), small(H, "q"), max_len, win.window, win.n_sinks,
                                                  w != nullptr);
    });
    if (ws.tensor && ws.tensor->device() != q.device()) throw ValueError("workspace is on another device");
    const int rc = unipin_paged_decode_attn(
        q.data_ptr(), address(ks), address(vs), out.data_ptr(), fp32, address<int>(&table),
        small(table.size(1), "page_table"), address<int>(&lens), small(R, "q"), small(H, "q"), small(D, "q"), max_len,
        win.window, win.n_sinks, scale, &pool, layer, address<float>(w), address(ws.tensor), ws.bytes, address<int>(status),
        at_.stream());
    return answer(rc, out);
}

// (pool_k, pool_v, key_weights, layer, page_table, lens, max_len, budget, n_sinks, n_recent, kept, new_lens, dev_status,
// stream)
PyObject* evict(PyObject* const* a)
{
    const at::Tensor &pk = tensor(a[0], "pool_k"), &pv = tensor(a[1], "pool_v");
    const unipin_kvpool pool = pool_of(pk, pv, nullptr);
    if (!given(a[2])) throw ValueError("key_weights is required");
    const at::Tensor& w = tensor(a[2], "key_weights");
    key_weights_fit(w, pool);
    const at::Tensor& lens = batch(a[5], "lens");
    const int64_t R = lens.size(0);
    const at::Tensor& table = page_table(a[4], R);
    const at::Tensor* status = optional(a[12], "dev_status");
    const int layer = as_int(a[3]), max_len = as_int(a[6]), budget = as_int(a[7]);
    // (a budget that the call refuses gets no memory)
    const int64_t places = budget > 0 && budget <= (1 << 30) ? budget : 0;
    Output rows(a[10], "kept", {R, pool.H, places}, at::kInt), left(a[11], "new_lens", {R}, at::kInt);
    const Place at_({&pk, &pv, &w, &table, &lens, rows.lent(), left.lent(), status}, a[13]);
    const at::Tensor &kept = rows.in(at_, lens), &fewer = left.in(at_, lens);
    const int rc = unipin_paged_evict(&pool, layer, address<float>(&w), address<int>(&table),
                                      small(table.size(1), "page_table"), address<int>(&lens), small(R, "lens"), max_len,
                                      budget, as_int(a[8]), as_int(a[9]), address<int>(&kept), address<int>(&fewer),
                                      address<int>(status), at_.stream());
    return answer(rc, kept, fewer);
}

// What both windowed calls check of q, k and v.
struct Rows {
    const at::Tensor &q, &k, &v;
    int64_t T, H, D, Hkv;
    Rows(PyObject* q_, PyObject* k_, PyObject* v_) : q(token_rows(q_, "q")), k(token_rows(k_, "k")), v(token_rows(v_, "v"))
    {
        T = q.size(0), H = q.size(1), D = q.size(2), Hkv = k.size(1);
        fits(k, "k", at::kBFloat16, {T, Hkv, D});
        fits(v, "v", at::kBFloat16, {T, Hkv, D});
    }
};

// (q, k, v, cu_seqlens, past_lens, max_seqlen, window, n_sinks, out, out_fp32, scale, dev_status, stream, lse)
PyObject* prefill(PyObject* const* a)
{
    const Rows x(a[0], a[1], a[2]);
    const at::Tensor &past = batch(a[4], "past_lens"), &cu = tensor(a[3], "cu_seqlens");
    const int64_t B = past.size(0);
    fits(cu, "cu_seqlens", at::kInt, {B + 1});
    const Window win = window_of(a[6], a[7]);
    const bool fp32 = truth(a[9]);
    const at::Tensor *lse = optional(a[13], "lse"), *status = optional(a[11], "dev_status");
    if (lse) fits(*lse, "lse", at::kFloat, {x.T, x.H});
    Output made(a[8], "out", {x.T, x.H, x.D}, fp32 ? at::kFloat : at::kBFloat16);
    const Place at_({&x.q, &x.k, &x.v, &cu, &past, made.lent(), lse, status}, a[12]);
    const at::Tensor& out = made.in(at_, x.q);
    const int rc = unipin_windowed_prefill_attn(
        x.q.data_ptr(), x.k.data_ptr(), x.v.data_ptr(), out.data_ptr(), fp32, address<float>(lse), address<int>(&cu),
        address<int>(&past), small(B, "past_lens"), small(x.H, "q"), small(x.Hkv, "k"), small(x.D, "q"), as_int(a[5]),
        small(x.T, "q"), win.window, win.n_sinks, scale_of(a[10], x.D), address<int>(status), at_.stream());
    return answer(rc, out);
}

// (q, k, v, out, dout, lse, cu_seqlens, past_lens, max_seqlen, window, n_sinks, scale, grad_fp32, dq, dk, dv, workspace,
// dev_status, stream)
PyObject* prefill_bwd(PyObject* const* a)
{
    const Rows x(a[0], a[1], a[2]);
    const at::Tensor &o = tensor(a[3], "out"), &g = tensor(a[4], "dout"), &lse = tensor(a[5], "lse");
    fits(o, "out", at::kBFloat16, {x.T, x.H, x.D});
    fits(g, "dout", at::kBFloat16, {x.T, x.H, x.D});
    fits(lse, "lse", at::kFloat, {x.T, x.H});
    const at::Tensor &past = batch(a[7], "past_lens"), &cu = tensor(a[6], "cu_seqlens");
    const int64_t B = past.size(0);
    fits(cu, "cu_seqlens", at::kInt, {B + 1});
    const Window win = window_of(a[9], a[10]);
    const bool fp32 = truth(a[12]);
    const at::ScalarType kind = fp32 ? at::kFloat : at::kBFloat16;
    const int max_seqlen = as_int(a[8]);
    const at::Tensor* status = optional(a[17], "dev_status");
    Output made_q(a[13], "dq", {x.T, x.H, x.D}, kind), made_k(a[14], "dk", {x.T, x.Hkv, x.D}, kind),
        made_v(a[15], "dv", {x.T, x.Hkv, x.D}, kind);
    const Place at_({&x.q, &x.k, &x.v, &o, &g, &lse, &cu, &past, made_q.lent(), made_k.lent(), made_v.lent(), status},
                    a[18]);
    const at::Tensor &dq = made_q.in(at_, x.q), &dk = made_k.in(at_, x.q), &dv = made_v.in(at_, x.q);
    const Space ws(a[16], x.q, [&] {
        return unipin_windowed_prefill_bwd_workspace_size(small(B, "past_lens"), small(x.H, "q"), small(x.Hkv, "k"),
                                                          small(x.D, "q"), max_seqlen, small(x.T, "q"), win.window,
                                                          win.n_sinks);
    });
    if (ws.tensor && ws.tensor->device() != x.q.device()) throw ValueError("workspace is on another device");
    const int rc = unipin_windowed_prefill_bwd(
        x.q.data_ptr(), x.k.data_ptr(), x.v.data_ptr(), o.data_ptr(), g.data_ptr(), address<float>(&lse), dq.data_ptr(),
        dk.data_ptr(), dv.data_ptr(), fp32, address<int>(&cu), address<int>(&past), small(B, "past_lens"), small(x.H, "q"),
        small(x.Hkv, "k"), small(x.D, "q"), max_seqlen, small(x.T, "q"), win.window, win.n_sinks, scale_of(a[11], x.D),
        address(ws.tensor), ws.bytes, address<int>(status), at_.stream());
    return answer(rc, dq, dk, dv);
}

// The binding passes every argument by position.
PyMethodDef methods[] = {
    {"pool_write", (PyCFunction)(void (*)())&guarded<pool_write, 14>, METH_FASTCALL, nullptr},
    {"decode", (PyCFunction)(void (*)())&guarded<decode, 19>, METH_FASTCALL, nullptr},
    {"evict", (PyCFunction)(void (*)())&guarded<evict, 14>, METH_FASTCALL, nullptr},
    {"prefill", (PyCFunction)(void (*)())&guarded<prefill, 14>, METH_FASTCALL, nullptr},
    {"prefill_bwd", (PyCFunction)(void (*)())&guarded<prefill_bwd, 19>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

#define CALLS_TEXT_(x) #x
#define CALLS_TEXT(x) CALLS_TEXT_(x)
#define CALLS_JOIN_(a, b) a##b
#define CALLS_JOIN(a, b) CALLS_JOIN_(a, b)

PyModuleDef module = {PyModuleDef_HEAD_INIT, CALLS_TEXT(CALLS_MODULE), nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// CALLS_MODULE: the module's name, which the build forms from torch's version
PyMODINIT_FUNC CALLS_JOIN(PyInit_, CALLS_MODULE)() { return PyModule_Create(&module); }
