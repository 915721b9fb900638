// Argument marshalling of the paged cache and packed-row attention for torch
// tensors: shape, stride, type and device checks, output and workspace
// allocation, current stream, then the C entry point.  Host only.  (In Python
// the same checks took 20 to 40 us a call, several times what a decode step's
// kernels run; here a call costs a few.)
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <limits>
#include <optional>
#include <string>

#include "sfa.h"

namespace {

// The library's entry points (the ones ctypes loaded).
struct {
    decltype(&::paged_append) append;
    decltype(&::paged_read) read;
    decltype(&::paged_run) run;
    decltype(&::paged_workspace_size) ws_size;
    decltype(&::varlen_run) varlen;
    decltype(&::paged_append_rotated) rotated;
    decltype(&::paged_run_window) window;
    decltype(&::varlen_run_window) varlen_window;
    decltype(&::paged_run_shared) shared;
    decltype(&::paged_shared_workspace_size) shared_ws_size;
} fn;

// An argument error, raised in Python as `type`.
struct Refused {
    PyObject* type;
    std::string what;
};
#define SFA_ENTER HANDLE_TH_ERRORS try {
#define SFA_LEAVE                                  \
    } catch (const Refused& e) {                   \
        PyErr_SetString(e.type, e.what.c_str());   \
        return nullptr;                            \
    }                                              \
    END_HANDLE_TH_ERRORS

[[noreturn]] void bad(const std::string& what) { throw Refused{PyExc_ValueError, what}; }
void expect(bool ok, const char* what) {
    if (!ok) bad(what);
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw Refused{PyExc_TypeError, std::string(name) + ": a torch tensor expected"};
    return THPVariable_Unpack(o);
}
// None or a tensor.
const at::Tensor* maybe(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }

int type_code(at::ScalarType t) {
    switch (t) {
        case at::kHalf: return SFA_DTYPE_F16;
        case at::kBFloat16: return SFA_DTYPE_BF16;
        case at::kFloat8_e4m3fn: return SFA_DTYPE_E4M3;
        case at::kFloat8_e5m2: return SFA_DTYPE_E5M2;
        default: bad(std::string("element type ") + c10::toString(t) + " is not one of f16, bf16, e4m3, e5m2");
    }
}

long integer(PyObject* o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}
// A count that the C entry points take as int.
int count(int64_t v, const char* name) {
    if (v < INT32_MIN || v > INT32_MAX) bad(std::string(name) + ": beyond 32 bits");
    return (int)v;
}
int count(PyObject* o, const char* name) { return count((int64_t)integer(o), name); }
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}
// A positive scale stays positive in fp32 (zero would select the default).
float softmax_scale(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v > 0.0 && (float)v == 0.f ? std::numeric_limits<float>::denorm_min() : (float)v;
}

// (tokens, heads, dim) rows whose heads are contiguous; returns the token stride.
int64_t rows(const at::Tensor& x, const char* name, int64_t heads, int64_t dim) {
    if (x.dim() != 3) bad(std::string(name) + ": (tokens, heads, head_dim) expected");
    const int64_t T = x.size(0), H = x.size(1), D = x.size(2);
    if ((heads >= 0 && H != heads) || (dim >= 0 && D != dim))
        bad(std::string(name) + ": other heads or head_dim than the keys'");
    if ((D > 1 && x.stride(2) != 1) || (H > 1 && x.stride(1) != D))
        bad(std::string(name) + ": the heads of a row must be contiguous");
    // the stride of a single row says nothing: its heads' extent serves
    return T > 1 ? x.stride(0) : H * D;
}

const int32_t* list(const at::Tensor& x, const char* name, at::Device dev, int64_t n) {
    if (x.scalar_type() != at::kInt || !x.is_contiguous() || x.device() != dev)
        bad(std::string(name) + ": contiguous int32 on the keys' device expected");
    if (n >= 0 && x.numel() != n) bad(std::string(name) + ": " + std::to_string(n) + " entries expected");
    return x.const_data_ptr<int32_t>();
}

const float* scales(const at::Tensor* x, const char* name, at::Device dev, int64_t heads) {
    if (!x) return nullptr;
    if (x->scalar_type() != at::kFloat || !x->is_contiguous() || x->device() != dev || x->numel() != heads)
        bad(std::string(name) + ": contiguous float32, one for each kv head, on the keys' device expected");
    return x->const_data_ptr<float>();
}

paged_kv cache(PyObject* const* o, long layout, PyObject* sk, PyObject* sv, at::Device& dev) {
    const at::Tensor &k = tensor(o[0], "k_pages"), &v = tensor(o[1], "v_pages");
    const at::Tensor &table = tensor(o[2], "page_table"), &lens = tensor(o[3], "kv_lens");
    expect(k.dim() == 4 && k.sizes() == v.sizes() && k.scalar_type() == v.scalar_type() &&
               k.device() == v.device() && k.is_contiguous() && v.is_contiguous(),
           "k_pages and v_pages: contiguous 4-D pools of one shape, type and device expected");
    expect(table.dim() == 2, "page_table: (num_seqs, max_pages) expected");
    dev = k.device();
    const bool hnd = layout == SFA_KV_LAYOUT_HND;
    paged_kv c{};
    c.num_seqs = count(table.size(0), "num_seqs");
    c.max_pages = count(table.size(1), "max_pages");
    c.num_pages = count(k.size(0), "num_pages");
    c.page_size = count(k.size(hnd ? 2 : 1), "page_size");
    c.num_kv_heads = count(k.size(hnd ? 1 : 2), "num_kv_heads");
    c.head_dim = count(k.size(3), "head_dim");
    c.k = k.data_ptr();
    c.v = v.data_ptr();
    c.page_table = list(table, "page_table", dev, -1);
    c.kv_lens = list(lens, "kv_lens", dev, c.num_seqs);
    c.kv_layout = (sfa_kv_layout)layout;
    c.dtype = (sfa_dtype)type_code(k.scalar_type());
    c.scale_k = scales(maybe(sk, "scale_k"), "scale_k", dev, c.num_kv_heads);
    c.scale_v = scales(maybe(sv, "scale_v"), "scale_v", dev, c.num_kv_heads);
    return c;
}

// Makes the tensors' device current, and the stream given (else torch's
// current one stays), so that outputs and workspace come from that stream's
// memory and nothing else reuses it while the call runs there.
struct On {
    c10::cuda::OptionalCUDAGuard device;
    c10::cuda::OptionalCUDAStreamGuard other;
    sfa_stream_t stream;
    On(at::Device dev, PyObject* given) {
        expect(dev.is_cuda(), "tensors on a CUDA device expected");
        device.set_device(dev);
        if (given == Py_None) {
            stream = (sfa_stream_t)c10::cuda::getCurrentCUDAStream(dev.index()).stream();
        } else {
            stream = (sfa_stream_t)PyLong_AsVoidPtr(given);
            if (PyErr_Occurred()) throw python_error();
            other.reset_stream(c10::cuda::getStreamFromExternal((cudaStream_t)stream, dev.index()));
        }
    }
};

// The interpreter lock is let go while outputs are allocated and kernels
// launched: both can wait for the GPU (a full launch queue, say), and what they
// wait for can be a host function on a stream that needs the lock.
struct Unlocked {
    PyThreadState* held = PyEval_SaveThread();
    Unlocked() = default;
    Unlocked(const Unlocked&) = delete;
    ~Unlocked() { PyEval_RestoreThread(held); }
};

// Straight from torch's allocator: through the dispatcher each of a call's
// tensors took about half a microsecond more.
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType t, at::Device dev) {
    return at::Tensor(at::detail::empty_cuda(shape, t, dev, std::nullopt));
}

// An output: the one given, checked, or a new one.
at::Tensor output(const at::Tensor* given, const char* name, at::IntArrayRef shape, at::ScalarType t, at::Device dev) {
    if (!given) return fresh(shape, t, dev);
    if (given->sizes() != shape || given->scalar_type() != t || !given->is_contiguous() || given->device() != dev)
        bad(std::string(name) + ": a contiguous tensor of the result's shape, type and device expected");
    return *given;
}

PyObject* wrap(int status, const at::Tensor& x, const at::Tensor& y) {
    PyObject* px = THPVariable_Wrap(x);
    PyObject* py = y.defined() ? THPVariable_Wrap(y) : Py_NewRef(Py_None);
    return Py_BuildValue("(iNN)", status, px, py);
}

void arity(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) throw Refused{PyExc_TypeError, std::to_string(want) + " arguments expected"};
}

// k_new, v_new, cu_seqlens, k_pages, v_pages, page_table, kv_lens, layout, scale_k, scale_v, stream
PyObject* py_append(PyObject*, PyObject* const* o, Py_ssize_t n) {
    SFA_ENTER
    arity(n, 11);
    at::Device dev(at::kCPU);
    const paged_kv c = cache(o + 3, integer(o[7]), o[8], o[9], dev);
    const at::Tensor &k = tensor(o[0], "k_new"), &v = tensor(o[1], "v_new");
    expect(k.sizes() == v.sizes() && k.scalar_type() == v.scalar_type() && k.device() == dev && v.device() == dev,
           "k_new and v_new: one shape and type, on the pools' device, expected");
    const int64_t ks = rows(k, "k_new", c.num_kv_heads, c.head_dim), vs = rows(v, "v_new", c.num_kv_heads, c.head_dim);
    const int32_t* cu = list(tensor(o[2], "cu_seqlens"), "cu_seqlens", dev, (int64_t)c.num_seqs + 1);
    const int t = type_code(k.scalar_type()), T = count(k.size(0), "tokens");
    On on(dev, o[10]);
    int st;
    {
        Unlocked here;
        st = fn.append(&c, k.const_data_ptr(), v.const_data_ptr(), ks, vs, cu, T, (sfa_dtype)t, on.stream);
    }
    return PyLong_FromLong(st);
    SFA_LEAVE
}

// k_new, v_new, cu_seqlens, k_pages, v_pages, page_table, kv_lens, layout, scale_k, scale_v, inv_freq, q, interleaved,
// q_out, stream
PyObject* py_rotated(PyObject*, PyObject* const* o, Py_ssize_t n) {
    SFA_ENTER
    arity(n, 15);
    at::Device dev(at::kCPU);
    const paged_kv c = cache(o + 3, integer(o[7]), o[8], o[9], dev);
    const at::Tensor &k = tensor(o[0], "k_new"), &v = tensor(o[1], "v_new"), &freq = tensor(o[10], "inv_freq");
    const at::Tensor *q = maybe(o[11], "q"), *given = maybe(o[13], "q_out");
    expect(k.sizes() == v.sizes() && k.scalar_type() == v.scalar_type() && k.device() == dev && v.device() == dev,
           "k_new and v_new: one shape and type, on the pools' device, expected");
    const int64_t ks = rows(k, "k_new", c.num_kv_heads, c.head_dim), vs = rows(v, "v_new", c.num_kv_heads, c.head_dim);
    const int32_t* cu = list(tensor(o[2], "cu_seqlens"), "cu_seqlens", dev, (int64_t)c.num_seqs + 1);
    expect(freq.scalar_type() == at::kFloat && freq.dim() == 1 && freq.is_contiguous() && freq.device() == dev,
           "inv_freq: contiguous float32 (rotary_dim / 2) on the keys' device expected");
    const int rotary = count(2 * freq.numel(), "rotary_dim"), t = type_code(k.scalar_type()), T = count(k.size(0), "tokens");
    const bool pairs = truth(o[12]);
    int64_t qs = 0, os = 0;
    int Hq = 0;
    expect(q || !given, "q_out: only with q");
    if (q) {
        expect(q->device() == dev && q->scalar_type() == k.scalar_type(), "q: the keys' type and device expected");
        qs = rows(*q, "q", -1, c.head_dim);
        expect(q->size(0) == T, "q: as many rows as k_new expected");
        Hq = count(q->size(1), "heads");
        if (given) {
            expect(given->sizes() == q->sizes() && given->scalar_type() == q->scalar_type() && given->device() == dev,
                   "q_out: q's shape, type and device expected");
            os = rows(*given, "q_out", Hq, c.head_dim);
            expect(given->const_data_ptr() != q->const_data_ptr() || os == qs, "q_out: in place of q with another stride");
        } else {
            os = (int64_t)Hq * c.head_dim;
        }
    }
    On on(dev, o[14]);
    at::Tensor out;
    int st;
    {
        Unlocked here;
        if (q) out = given ? *given : fresh(q->sizes(), q->scalar_type(), dev);
        st = fn.rotated(&c, q ? q->const_data_ptr() : nullptr, k.const_data_ptr(), v.const_data_ptr(),
                        q ? out.data_ptr() : nullptr, qs, ks, vs, os, cu, T, Hq, freq.const_data_ptr<float>(), rotary, pairs,
                        (sfa_dtype)t, on.stream);
    }
    return Py_BuildValue("(iN)", st, out.defined() ? THPVariable_Wrap(out) : Py_NewRef(Py_None));
    SFA_LEAVE
}

// k_pages, v_pages, page_table, kv_lens, cu_seqlens, num_tokens, dtype (-1: default), layout, scale_k, scale_v,
// k_out, v_out, stream
PyObject* py_read(PyObject*, PyObject* const* o, Py_ssize_t n) {
    SFA_ENTER
    arity(n, 13);
    at::Device dev(at::kCPU);
    const paged_kv c = cache(o, integer(o[7]), o[8], o[9], dev);
    const int32_t* cu = list(tensor(o[4], "cu_seqlens"), "cu_seqlens", dev, (int64_t)c.num_seqs + 1);
    const int T = count(o[5], "num_tokens");
    expect(T >= 0, "num_tokens: not negative");
    const at::Tensor *gk = maybe(o[10], "out"), *gv = maybe(o[11], "out");
    const long want = integer(o[6]);
    expect(want == -1 || want == SFA_DTYPE_F16 || want == SFA_DTYPE_BF16, "dtype: f16 or bf16 expected");
    const at::ScalarType t = want == SFA_DTYPE_F16                ? at::kHalf
                             : want == SFA_DTYPE_BF16             ? at::kBFloat16
                             : gk                                 ? gk->scalar_type()
                             : c.dtype == SFA_DTYPE_F16           ? at::kHalf
                                                                  : at::kBFloat16;
    On on(dev, o[12]);
    const int64_t shape[3] = {T, c.num_kv_heads, c.head_dim};
    at::Tensor k, v;
    int st;
    {
        Unlocked here;
        k = output(gk, "out", shape, t, dev);
        v = output(gv, "out", shape, t, dev);
        st = fn.read(&c, cu, T, (sfa_dtype)type_code(t), k.data_ptr(), v.data_ptr(), on.stream);
    }
    return wrap(st, k, v);
    SFA_LEAVE
}

// Outputs and workspace of an attention call: out, lse, workspace as given.
struct Outputs {
    const at::Tensor *given_out, *given_lse, *given_ws;
    bool want_lse;
    at::Tensor out, lse;
    at::DataPtr own;              // the workspace, unless one is given
    void* ws = nullptr;
    size_t ws_bytes = 0;
    Outputs(PyObject* const* o, bool want)
        : given_out(maybe(o[0], "out")), given_lse(maybe(o[1], "lse")), given_ws(maybe(o[2], "workspace")), want_lse(want) {}
    void make(const at::Tensor& q, size_t need) {
        const at::Device dev = q.device();
        out = output(given_out, "out", q.sizes(), q.scalar_type(), dev);
        if (given_lse || want_lse) lse = output(given_lse, "lse", q.sizes().slice(0, 2), at::kFloat, dev);
        if (given_ws) {
            expect(given_ws->device() == dev && given_ws->is_contiguous(),
                   "workspace: a contiguous tensor on q's device expected");
            ws = given_ws->data_ptr();
            ws_bytes = given_ws->nbytes();
        } else {
            own = c10::cuda::CUDACachingAllocator::get()->allocate(need);
            ws = own.get();
            ws_bytes = need;
        }
    }
    float* lse_ptr() const { return lse.defined() ? lse.data_ptr<float>() : nullptr; }
};

// Which keys a row sees: all (causally: up to its own), those in a window and the
// sinks, or a shared prefix's and its own.
enum Keys { ALL, WINDOW, SHARED };

void causal_window(bool causal) { expect(causal, "window: causal attention only"); }

// q, k_pages, v_pages, page_table, kv_lens, cu_seqlens_q, scale, causal, layout, scale_k, scale_v, return_lse,
// max_q_len, out, lse, workspace, stream; then window, sinks, or cu_shared, shared_lens
template <Keys K>
PyObject* py_paged(PyObject*, PyObject* const* o, Py_ssize_t n) {
    SFA_ENTER
    arity(n, K == ALL ? 17 : 19);
    at::Device dev(at::kCPU);
    const paged_kv c = cache(o + 1, integer(o[8]), o[9], o[10], dev);
    const at::Tensor& q = tensor(o[0], "q");
    expect(q.device() == dev, "q: on the pools' device expected");
    const int64_t qs = rows(q, "q", -1, c.head_dim);
    const int32_t* cu = list(tensor(o[5], "cu_seqlens_q"), "cu_seqlens_q", dev, (int64_t)c.num_seqs + 1);
    const float scale = softmax_scale(o[6]);
    const int T = count(q.size(0), "tokens"), Hq = count(q.size(1), "heads"), hint = count(o[12], "max_q_len");
    const int t = type_code(q.scalar_type());
    const bool causal = truth(o[7]);
    int window = 0, sinks = 0, groups = 0;
    const int32_t *cu_shared = nullptr, *shared_lens = nullptr;
    if constexpr (K == WINDOW) {
        window = count(o[17], "window");
        sinks = count(o[18], "sinks");
        causal_window(causal);
    } else if constexpr (K == SHARED) {
        const at::Tensor& lens = tensor(o[18], "shared_lens");
        shared_lens = list(lens, "shared_lens", dev, -1);
        groups = count(lens.numel(), "groups");
        cu_shared = list(tensor(o[17], "cu_shared"), "cu_shared", dev, (int64_t)groups + 1);
    }
    Outputs r(o + 13, truth(o[11]));
    On on(dev, o[16]);
    size_t need = 0;
    int st = (K == SHARED ? fn.shared_ws_size : fn.ws_size)(c.num_seqs, T, Hq, c.num_kv_heads, c.head_dim, &need);
    if (st != SFA_OK) return Py_BuildValue("(iOO)", st, Py_None, Py_None);
    {
        Unlocked here;
        r.make(q, need);
        if constexpr (K == WINDOW)
            st = fn.window(&c, q.const_data_ptr(), qs, cu, T, Hq, hint, window, sinks, scale, (sfa_dtype)t,
                           r.out.data_ptr(), r.lse_ptr(), r.ws, r.ws_bytes, on.stream);
        else if constexpr (K == SHARED)
            st = fn.shared(&c, q.const_data_ptr(), qs, cu, T, Hq, hint, cu_shared, shared_lens, groups, scale, causal,
                           (sfa_dtype)t, r.out.data_ptr(), r.lse_ptr(), r.ws, r.ws_bytes, on.stream);
        else
            st = fn.run(&c, q.const_data_ptr(), qs, cu, T, Hq, hint, scale, causal, (sfa_dtype)t,
                        r.out.data_ptr(), r.lse_ptr(), r.ws, r.ws_bytes, on.stream);
    }
    return wrap(st, r.out, r.lse);
    SFA_LEAVE
}

// q, k, v, cu_seqlens_q, cu_seqlens_k, scale, causal, return_lse, max_q_len, out, lse, workspace, stream; then
// window, sinks
template <Keys K>
PyObject* py_varlen(PyObject*, PyObject* const* o, Py_ssize_t n) {
    SFA_ENTER
    arity(n, K == ALL ? 13 : 15);
    const at::Tensor &q = tensor(o[0], "q"), &k = tensor(o[1], "k"), &v = tensor(o[2], "v");
    const at::Device dev = q.device();
    expect(k.device() == dev && v.device() == dev && k.scalar_type() == q.scalar_type() &&
               v.scalar_type() == q.scalar_type() && k.sizes() == v.sizes(),
           "q, k, v: one type and device, k and v of one shape, expected");
    const int64_t qs = rows(q, "q", -1, -1), D = q.size(2);
    const int64_t ks = rows(k, "k", -1, D), vs = rows(v, "v", -1, D);
    const at::Tensor& lq = tensor(o[3], "cu_seqlens_q");
    const int32_t* cq = list(lq, "cu_seqlens_q", dev, -1);
    const int32_t* ck = list(tensor(o[4], "cu_seqlens_k"), "cu_seqlens_k", dev, lq.numel());
    const float scale = softmax_scale(o[5]);
    const int B = count(lq.numel() - 1, "num_seqs"), T = count(q.size(0), "tokens"), Hq = count(q.size(1), "heads");
    const int N = count(k.size(0), "keys"), Hkv = count(k.size(1), "heads"), hint = count(o[8], "max_q_len");
    const int t = type_code(q.scalar_type());
    const bool causal = truth(o[6]);
    int window = 0, sinks = 0;
    if constexpr (K == WINDOW) {
        window = count(o[13], "window");
        sinks = count(o[14], "sinks");
        causal_window(causal);
    }
    Outputs r(o + 9, truth(o[7]));
    On on(dev, o[12]);
    size_t need = 0;
    int st = fn.ws_size(B, T, Hq, Hkv, (int)D, &need);
    if (st != SFA_OK) return Py_BuildValue("(iOO)", st, Py_None, Py_None);
    {
        Unlocked here;
        r.make(q, need);
        if constexpr (K == WINDOW)
            st = fn.varlen_window(q.const_data_ptr(), k.const_data_ptr(), v.const_data_ptr(), qs, ks, vs, cq, ck, B, T, N,
                                  Hq, Hkv, (int)D, hint, window, sinks, scale, (sfa_dtype)t, r.out.data_ptr(), r.lse_ptr(),
                                  r.ws, r.ws_bytes, on.stream);
        else
            st = fn.varlen(q.const_data_ptr(), k.const_data_ptr(), v.const_data_ptr(), qs, ks, vs, cq, ck, B, T, N, Hq, Hkv,
                           (int)D, hint, scale, causal, (sfa_dtype)t, r.out.data_ptr(), r.lse_ptr(),
                           r.ws, r.ws_bytes, on.stream);
    }
    return wrap(st, r.out, r.lse);
    SFA_LEAVE
}

// Addresses of paged_append, paged_read, paged_run, paged_workspace_size, varlen_run.
PyObject* py_bind(PyObject*, PyObject* const* o, Py_ssize_t n) {
    SFA_ENTER
    arity(n, 5);
    fn.append = reinterpret_cast<decltype(fn.append)>(PyLong_AsVoidPtr(o[0]));
    fn.read = reinterpret_cast<decltype(fn.read)>(PyLong_AsVoidPtr(o[1]));
    fn.run = reinterpret_cast<decltype(fn.run)>(PyLong_AsVoidPtr(o[2]));
    fn.ws_size = reinterpret_cast<decltype(fn.ws_size)>(PyLong_AsVoidPtr(o[3]));
    fn.varlen = reinterpret_cast<decltype(fn.varlen)>(PyLong_AsVoidPtr(o[4]));
    if (PyErr_Occurred()) throw python_error();
    Py_RETURN_NONE;
    SFA_LEAVE
}

// Addresses of paged_append_rotated, paged_run_window, varlen_run_window, paged_run_shared,
// paged_shared_workspace_size.
PyObject* py_bind_more(PyObject*, PyObject* const* o, Py_ssize_t n) {
    SFA_ENTER
    arity(n, 5);
    fn.rotated = reinterpret_cast<decltype(fn.rotated)>(PyLong_AsVoidPtr(o[0]));
    fn.window = reinterpret_cast<decltype(fn.window)>(PyLong_AsVoidPtr(o[1]));
    fn.varlen_window = reinterpret_cast<decltype(fn.varlen_window)>(PyLong_AsVoidPtr(o[2]));
    fn.shared = reinterpret_cast<decltype(fn.shared)>(PyLong_AsVoidPtr(o[3]));
    fn.shared_ws_size = reinterpret_cast<decltype(fn.shared_ws_size)>(PyLong_AsVoidPtr(o[4]));
    if (PyErr_Occurred()) throw python_error();
    Py_RETURN_NONE;
    SFA_LEAVE
}

#define SFA_FN(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {SFA_FN("bind", py_bind), SFA_FN("paged_append", py_append), SFA_FN("paged_read", py_read),
                         SFA_FN("paged_attention", py_paged<ALL>), SFA_FN("varlen_attention", py_varlen<ALL>),
                         SFA_FN("bind_more", py_bind_more), SFA_FN("paged_append_rotated", py_rotated),
                         SFA_FN("paged_attention_window", py_paged<WINDOW>),
                         SFA_FN("varlen_attention_window", py_varlen<WINDOW>),
                         SFA_FN("shared_prefix_attention", py_paged<SHARED>), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors(void) { return PyModule_Create(&module); }
