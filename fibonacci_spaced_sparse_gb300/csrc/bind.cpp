// bind.cpp -- the native half of the Python binding of the norm, paged-cache and
// 8-bit calls (api.py): looks at the tensors, allocates outputs and
// calls the C ABI.  These calls run once per layer and step of a serving loop
// on kernels of a few microseconds, where marshalling in Python (ctypes and
// tensor attributes, 19 to 27 us a call on the Grace cores of a GB300) would
// be most of a step.
//
// Every function takes positional arguments only (api.py has the signatures
// and defaults); None stands for an absent tensor.  Work goes to the current
// stream of the tensors' device; outputs come from torch's allocator on it.
#include <Python.h>

#include <algorithm>
#include <initializer_list>
#include <string>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "sfa.h"

namespace {

using at::Tensor;

constexpr int64_t kHq = 8, kHkv = 2, kD = 64;

struct Refused {  // a Python exception to raise
    PyObject* type;
    std::string text;
};
[[noreturn]] void refuse(const std::string& text) { throw Refused{PyExc_ValueError, text}; }

std::string shape_text(at::IntArrayRef s) {
    std::string t = "[";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + "]";
}

const Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw Refused{PyExc_TypeError, std::string(name) + " must be a tensor"};
    return THPVariable_Unpack(o);
}

sfa_dtype dtype_of(const Tensor& t) {
    if (t.scalar_type() == at::kBFloat16) return SFA_BF16;
    if (t.scalar_type() == at::kFloat) return SFA_F32;
    throw Refused{PyExc_TypeError, std::string("unsupported dtype ") + at::toString(t.scalar_type())};
}

// Token stride (elements) of t [*lead, heads, 64]: heads and dimensions
// contiguous, tokens at one stride, so that a part of a packed projection is
// taken as it is.
int64_t token_stride(const Tensor& t, const char* name, at::IntArrayRef lead, int64_t heads) {
    const int64_t n = (int64_t)lead.size();
    bool fits = t.dim() == n + 2 && t.size(n) == heads && t.size(n + 1) == kD;
    int64_t tokens = 1;
    for (int64_t i = 0; fits && i < n; ++i) {
        fits = t.size(i) == lead[i];
        tokens *= lead[i];
    }
    if (!fits) {
        std::vector<int64_t> want(lead.begin(), lead.end());
        want.push_back(heads);
        want.push_back(kD);
        refuse(std::string(name) + " must be " + shape_text(want) + ", got " + shape_text(t.sizes()));
    }
    if (tokens == 0) return heads * kD;
    const auto st = t.strides();
    int64_t step = st[n - 1];
    bool one = true;
    if (n == 2) {
        if (lead[1] == 1)
            step = st[0];
        else
            one = lead[0] == 1 || st[0] == step * lead[1];
    }
    if (tokens == 1) step = heads * kD;
    if (!one || st[n + 1] != 1 || (heads > 1 && st[n] != kD) || step < heads * kD ||
        step * t.element_size() % 16 != 0)
        refuse(std::string(name) +
               ": heads must be contiguous and tokens at one stride of a multiple of 16 bytes, got strides " +
               shape_text(st));
    return step;
}

void like(const Tensor& t, const char* name, const Tensor& ref) {
    if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
    if (t.scalar_type() != ref.scalar_type() || t.device() != ref.device())
        refuse(std::string(name) + " must share the other tensors' dtype and device");
}

// The pointer of a contiguous tensor of this shape and type on ref's device.
void* dense(const Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type, const Tensor& ref) {
    if (t.sizes() != shape || t.scalar_type() != type || t.device() != ref.device() || !t.is_contiguous())
        refuse(std::string(name) + " must be a contiguous " + at::toString(type) + " " + shape_text(shape) +
               " tensor on " + ref.device().str());
    return t.data_ptr();
}

template <typename T = void>
T* dense_or_null(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type, const Tensor& ref) {
    return o == Py_None ? nullptr : static_cast<T*>(dense(tensor(o, name), name, shape, type, ref));
}

unsigned* status_word(PyObject* o, const Tensor& ref) {
    if (o == Py_None) return nullptr;
    const Tensor& t = tensor(o, "status");
    if (t.scalar_type() != at::kInt || t.device() != ref.device() || t.numel() < 1)
        refuse("status must be an int32 word on " + ref.device().str());
    return static_cast<unsigned*>(t.data_ptr());
}

// The RoPE table (None without a rotation) and its rows.
const float* table(PyObject* o, const Tensor& ref, int64_t* rows) {
    *rows = 0;
    if (o == Py_None) return nullptr;
    const Tensor& t = tensor(o, "rope");
    if (t.dim() != 3 || t.size(1) != kD / 2 || t.size(2) != 2 || t.scalar_type() != at::kFloat || !t.is_contiguous() ||
        t.device() != ref.device())
        refuse("rope must be a contiguous fp32 [rows, 32, 2] table (rope_table) on " + ref.device().str());
    *rows = t.size(0);
    return static_cast<const float*>(t.data_ptr());
}

// Without the interpreter's lock: other threads run while this one allocates or
// waits for room in the launch queue.
struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    Unlocked() = default;
    Unlocked(const Unlocked&) = delete;
    ~Unlocked() { PyEval_RestoreThread(state); }
};

// A new tensor on ref's device (the allocator's own entry: a dispatched
// at::empty costs a microsecond on a Grace core).
Tensor empty(at::IntArrayRef shape, at::ScalarType type, const Tensor& ref) {
    return Tensor(at::detail::empty_cuda(shape, type, ref.device(), std::nullopt));
}

// An output: the given one, checked, or a new one, which make() allocates (without
// the interpreter's lock, beside the library's call).
struct Out {
    Tensor made;
    PyObject* given;
    at::DimVector shape;
    at::ScalarType type;
    const Tensor& ref;
    void* ptr = nullptr;
    Out(PyObject* o, const char* name, at::IntArrayRef sizes, at::ScalarType t, const Tensor& r)
        : given(o), shape(sizes), type(t), ref(r) {
        if (o != Py_None) ptr = dense(tensor(o, name), name, sizes, t, r);
    }
    void* make() {
        if (given == Py_None) {
            made = empty(shape, type, ref);
            ptr = made.data_ptr();
        }
        return ptr;
    }
    PyObject* object() {
        if (given != Py_None) return Py_NewRef(given);
        return THPVariable_Wrap(std::move(made));
    }
};

// A workspace: the given one, or a new one of the size that need() asks for.
struct Scratch {
    Tensor made;
    const Tensor& ref;
    const bool own;
    void* ptr = nullptr;
    size_t bytes = 0;
    Scratch(PyObject* o, const Tensor& r) : ref(r), own(o == Py_None) {
        if (own) return;
        const Tensor& t = tensor(o, "workspace");
        if (t.device() != r.device() || !t.is_contiguous())
            refuse("workspace must be a contiguous tensor on " + r.device().str());
        ptr = t.data_ptr();
        bytes = (size_t)t.nbytes();
    }
    void need(size_t n) {
        if (!own || n == 0) return;
        made = empty({(int64_t)n}, at::kByte, ref);
        ptr = made.data_ptr();
        bytes = n;
    }
};

double number(PyObject* o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw python_error();
    return x;
}

int64_t integer(PyObject* o) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw python_error();
    return x;
}

bool truth(PyObject* o) {
    const int x = PyObject_IsTrue(o);
    if (x < 0) throw python_error();
    return x != 0;
}

int small(int64_t x) { return (int)std::clamp<int64_t>(x, -1, 0x7fffffff); }  // the library refuses both

sfa_params params(int64_t B, int64_t T, sfa_dtype dt, double theta) {
    sfa_params p = {};
    p.B = small(B);
    p.T = small(T);
    p.Hq = (int)kHq;
    p.Hkv = (int)kHkv;
    p.D = (int)kD;
    p.alpha = 1.f;
    p.rope_theta = (float)theta;
    p.dtype = dt;
    return p;
}

// Makes a call of the library, and its allocations, without the interpreter's lock;
// raises SfaError for a status other than SFA_OK.
template <typename F>
void call(const char* where, F f) {
    sfa_status st;
    {
        const Unlocked here;
        st = f();
    }
    if (st == SFA_OK) return;
    PyObject* lib = PyImport_ImportModule("fibonacci_spaced_sparse_gb300._lib");
    if (lib) Py_XDECREF(PyObject_CallMethod(lib, "check", "is", (int)st, where));
    Py_XDECREF(lib);
    throw python_error();
}

template <typename F>
PyObject* guarded(const char* name, Py_ssize_t got, Py_ssize_t want, F body) {
    HANDLE_TH_ERRORS
    if (got != want) {
        PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, got);
        return nullptr;
    }
    try {
        return body();
    } catch (const Refused& r) {
        PyErr_SetString(r.type, r.text.c_str());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject* tuple_of(std::initializer_list<PyObject*> items) {
    PyObject* t = PyTuple_New((Py_ssize_t)items.size());
    Py_ssize_t i = 0;
    for (PyObject* o : items) PyTuple_SET_ITEM(t, i++, o);
    return t;
}

// ------------------------------------------------------- norm with rotation

struct NormIn {
    const Tensor &q, &k;
    int64_t qs, ks, rows;
    const float *wq, *wk, *rope;
    const int* positions;
    double eps, theta;
    sfa_params p;

    // a: q, k, wq, wk, eps, theta, positions, rope
    explicit NormIn(PyObject* const* a) : q(tensor(a[0], "q")), k(tensor(a[1], "k")) {
        if (q.dim() != 4) refuse("q must be [B, T, 8, 64], got " + shape_text(q.sizes()));
        const sfa_dtype dt = dtype_of(q);
        like(q, "q", q);
        like(k, "k", q);
        const int64_t lead[2] = {q.size(0), q.size(1)};
        qs = token_stride(q, "q", lead, kHq);
        ks = token_stride(k, "k", lead, kHkv);
        wq = static_cast<const float*>(dense(tensor(a[2], "wq"), "wq", {kD}, at::kFloat, q));
        wk = static_cast<const float*>(dense(tensor(a[3], "wk"), "wk", {kD}, at::kFloat, q));
        eps = number(a[4]);
        theta = number(a[5]);
        positions = dense_or_null<const int>(a[6], "positions", lead, at::kInt, q);
        rope = table(a[7], q, &rows);
        if (theta > 0 && !positions && rows < lead[1] && lead[0] > 0)
            refuse("rope has " + std::to_string(rows) + " rows, the sequence " + std::to_string(lead[1]));
        p = params(lead[0], lead[1], dt, theta);
    }
};

// q, k, wq, wk, eps, theta, positions, rope, qhat, khat, status
PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded("norm_rope", n, 11, [&]() -> PyObject* {
        const NormIn x(a);
        c10::cuda::OptionalCUDAGuard guard(x.q.device());
        Out qh(a[8], "out[0]", x.q.sizes(), x.q.scalar_type(), x.q), kh(a[9], "out[1]", x.k.sizes(), x.q.scalar_type(), x.q);
        unsigned* status = status_word(a[10], x.q);
        const auto stream = c10::cuda::getCurrentCUDAStream(x.q.device().index()).stream();
        call("sfa_qk_norm_rope", [&] {
            return sfa_qk_norm_rope(&x.p, x.q.data_ptr(), x.qs, x.k.data_ptr(), x.ks, x.wq, x.wk, (float)x.eps, x.positions,
                                    x.rope, small(x.rows), qh.make(), kh.make(), status, stream);
        });
        return tuple_of({qh.object(), kh.object()});
    });
}

// q, k, wq, wk, eps, theta, positions, rope, dqhat, dkhat, workspace, dq, dk, dwq, dwk, status
PyObject* norm_rope_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded("norm_rope_backward", n, 16, [&]() -> PyObject* {
        const NormIn x(a);
        c10::cuda::OptionalCUDAGuard guard(x.q.device());
        const auto type = x.q.scalar_type();
        const void* dqhat = dense(tensor(a[8], "dqhat"), "dqhat", x.q.sizes(), type, x.q);
        const void* dkhat = dense(tensor(a[9], "dkhat"), "dkhat", x.k.sizes(), type, x.q);
        Tensor scratch;
        void* ws = nullptr;
        size_t bytes = 0;
        const bool own_scratch = a[10] == Py_None;
        if (!own_scratch) {
            const Tensor& t = tensor(a[10], "workspace");
            if (t.device() != x.q.device() || !t.is_contiguous())
                refuse("workspace must be a contiguous tensor on " + x.q.device().str());
            ws = t.data_ptr();
            bytes = (size_t)t.nbytes();
        }
        Out dq(a[11], "out[0]", x.q.sizes(), type, x.q), dk(a[12], "out[1]", x.k.sizes(), type, x.q);
        Out dwq(a[13], "out[2]", {kD}, at::kFloat, x.q), dwk(a[14], "out[3]", {kD}, at::kFloat, x.q);
        unsigned* status = status_word(a[15], x.q);
        const auto stream = c10::cuda::getCurrentCUDAStream(x.q.device().index()).stream();
        call("sfa_qk_norm_rope_backward", [&] {
            if (own_scratch && (bytes = sfa_qk_norm_rope_backward_workspace_size(&x.p)) != 0) {
                scratch = empty({(int64_t)bytes}, at::kByte, x.q);
                ws = scratch.data_ptr();
            }
            return sfa_qk_norm_rope_backward(&x.p, x.q.data_ptr(), x.qs, x.k.data_ptr(), x.ks, x.wq, x.wk, (float)x.eps,
                                             x.positions, x.rope, small(x.rows), dqhat, dkhat, dq.make(), dk.make(),
                                             static_cast<float*>(dwq.make()), static_cast<float*>(dwk.make()), ws, bytes,
                                             status, stream);
        });
        return tuple_of({dq.object(), dk.object(), dwq.object(), dwk.object()});
    });
}

// ------------------------------------------------------------- paged cache

struct CacheIn {
    const Tensor& k;
    sfa_dtype dt;
    int64_t S, cap;
    sfa_paged_fp8 f = {};       // scales and block_size of 8-bit pages
    sfa_paged& c = f.pages;

    // a: k_pages, v_pages, (scales of 8-bit pages,) block_table, cu_q, seq_lens; token:
    // the step's queries or keys
    CacheIn(PyObject* const* a, const Tensor& token, bool fp8) : k(tensor(a[0], "k_pages")) {
        dt = dtype_of(fp8 ? token : k);
        if (fp8 && k.scalar_type() != at::kFloat8_e4m3fn)
            throw Refused{PyExc_TypeError, std::string("k_pages must be float8_e4m3fn, got ") + at::toString(k.scalar_type())};
        const int64_t N = token.size(0);
        if (!k.is_cuda()) refuse("k_pages must be a CUDA tensor");
        if (k.dim() != 4 || k.size(2) != kHkv || k.size(3) != kD || !k.is_contiguous())
            refuse("k_pages must be a contiguous [num_pages, page_size, 2, 64] tensor, got " + shape_text(k.sizes()));
        const int64_t page = k.size(1);
        PyObject* const v_pages = a[1];
        if (k.size(0) < 1 || page < 1 || (page & (page - 1)))
            refuse("page_size must be a power of two and num_pages at least 1, got " + shape_text(k.sizes()));
        if (fp8) blocks(tensor(a[2], "page_scales"), page);
        a += fp8 ? 1 : 0;
        const Tensor& t = tensor(a[2], "block_table");
        if (t.dim() != 2 || t.size(1) < 1) refuse("block_table must be [S, max_pages], got " + shape_text(t.sizes()));
        S = t.size(0);
        c.k_pages = k.data_ptr();
        c.v_pages = dense(tensor(v_pages, "v_pages"), "v_pages", k.sizes(), k.scalar_type(), k);
        c.num_pages = small(k.size(0));
        c.page_size = small(page);
        c.block_table = static_cast<const int*>(dense(t, "block_table", t.sizes(), at::kInt, k));
        c.max_pages = small(t.size(1));
        c.cu_q = static_cast<const int*>(dense(tensor(a[3], "cu_q"), "cu_q", {S + 1}, at::kInt, k));
        c.seq_lens = static_cast<const int*>(dense(tensor(a[4], "seq_lens"), "seq_lens", {S}, at::kInt, k));
        c.N = small(N);
        cap = std::min<int64_t>(t.size(1) * page, 1 << 24);
    }
    CacheIn(const CacheIn&) = delete;

    // The scales of 8-bit pages, a block of rows each.
    void blocks(const Tensor& t, int64_t page) {
        if (t.dim() != 4 || t.size(1) < 1 || page % t.size(1) != 0)
            refuse("page_scales must be [num_pages, page_size / block_size, 2, 2], got " + shape_text(t.sizes()));
        f.scales = static_cast<float*>(dense(t, "page_scales", {k.size(0), t.size(1), 2, kHkv}, at::kFloat, k));
        f.block_size = small(page / t.size(1));
    }

    // Refuses a tensor of token rows that is not like the first of them.
    void same(const Tensor& t, const char* name, const Tensor& token) const {
        like(t, name, token);
        if (t.device() != k.device()) refuse(std::string(name) + " must be on the pages' device");
    }
};

// k, v, k_pages, v_pages, (page_scales,) block_table, cu_q, seq_lens, q, wq, wk, eps, theta, rope, q_out, status
PyObject* append_to(const char* name, bool fp8, PyObject* const* a, Py_ssize_t n) {
    return guarded(name, n, fp8 ? 16 : 15, [&]() -> PyObject* {
        const std::string call_name = std::string("sfa_") + name;
        const Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
        if (k.dim() != 3) refuse("k must be [N, 2, 64], got " + shape_text(k.sizes()));
        const int64_t lead[1] = {k.size(0)};
        const CacheIn x(a + 2, k, fp8);
        const Tensor& kind = fp8 ? k : x.k;
        x.same(k, "k", kind);
        x.same(v, "v", kind);
        const int64_t ks = token_stride(k, "k", lead, kHkv), vs = token_stride(v, "v", lead, kHkv);
        a += fp8 ? 1 : 0;
        const bool with_q = a[7] != Py_None;
        if (!with_q && (a[8] != Py_None || a[13] != Py_None)) refuse("wq and q_out go with q");
        const float* wq = dense_or_null<const float>(a[8], "wq", {kD}, at::kFloat, x.k);
        const float* wk = dense_or_null<const float>(a[9], "wk", {kD}, at::kFloat, x.k);
        const double eps = number(a[10]), theta = number(a[11]);
        int64_t rows;
        const float* rope = table(a[12], x.k, &rows);
        const sfa_params p = params(x.S, rope ? std::min(x.cap, rows) : x.cap, x.dt, theta);
        unsigned* status = status_word(a[14], x.k);
        c10::cuda::OptionalCUDAGuard guard(x.k.device());
        const auto stream = c10::cuda::getCurrentCUDAStream(x.k.device().index()).stream();
        auto append = [&](const void* q, int64_t qs, void* out) {
            return fp8 ? sfa_paged_append_fp8(&p, &x.f, q, qs, k.data_ptr(), ks, v.data_ptr(), vs, wq, wk, (float)eps, rope, out,
                                              status, stream)
                       : sfa_paged_append(&p, &x.c, q, qs, k.data_ptr(), ks, v.data_ptr(), vs, wq, wk, (float)eps, rope, out,
                                          status, stream);
        };
        if (!with_q) {
            call(call_name.c_str(), [&] { return append(nullptr, 0, nullptr); });
            Py_RETURN_NONE;
        }
        const Tensor& q = tensor(a[7], "q");
        x.same(q, "q", kind);
        const int64_t qs = token_stride(q, "q", lead, kHq);
        Out out(a[13], "q_out", q.sizes(), q.scalar_type(), x.k);
        call(call_name.c_str(), [&] { return append(q.data_ptr(), qs, out.make()); });
        return out.object();
    });
}
PyObject* paged_append(PyObject*, PyObject* const* a, Py_ssize_t n) { return append_to("paged_append", false, a, n); }
PyObject* paged_append_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) { return append_to("paged_append_fp8", true, a, n); }

// q, k_pages, v_pages, (page_scales,) block_table, cu_q, seq_lens, alpha, W, rungs, scale, need_lse, out, lse, status,
// round_offsets(, workspace)
PyObject* forward_over(const char* name, bool fp8, PyObject* const* a, Py_ssize_t n) {
    return guarded(name, n, fp8 ? 17 : 15, [&]() -> PyObject* {
        const std::string call_name = std::string("sfa_") + name;
        const Tensor& q = tensor(a[0], "q");
        if (q.dim() != 3) refuse("q must be [N, 8, 64], got " + shape_text(q.sizes()));
        const int64_t lead[1] = {q.size(0)};
        const CacheIn x(a + 1, q, fp8);
        x.same(q, "q", fp8 ? q : x.k);
        const int64_t qs = token_stride(q, "q", lead, kHq);
        a += fp8 ? 1 : 0;
        sfa_params p = params(x.S, x.cap, x.dt, 0.0);
        p.alpha = (float)number(a[6]);
        p.W = small(integer(a[7]));
        PyObject* seq = PySequence_Fast(a[8], "rungs must be a sequence of base offsets");
        if (!seq) throw python_error();
        float rungs[SFA_MAX_RUNGS];
        p.K = (int)std::min<Py_ssize_t>(PySequence_Fast_GET_SIZE(seq), SFA_MAX_RUNGS + 1);  // one too many is refused
        for (int i = 0; i < std::min(p.K, SFA_MAX_RUNGS); ++i)
            rungs[i] = (float)PyFloat_AsDouble(PySequence_Fast_GET_ITEM(seq, i));
        Py_DECREF(seq);
        if (PyErr_Occurred()) throw python_error();
        p.rungs = rungs;
        p.scale = (float)number(a[9]);
        p.round_offsets = truth(a[14]);
        unsigned* status = status_word(a[13], x.k);
        c10::cuda::OptionalCUDAGuard guard(x.k.device());
        Out out(a[11], "out", q.sizes(), q.scalar_type(), x.k);
        const int64_t lse_shape[2] = {lead[0], kHq};
        const bool need_lse = truth(a[10]);
        Out lse(need_lse ? a[12] : Py_None, "lse", lse_shape, at::kFloat, x.k);
        const auto stream = c10::cuda::getCurrentCUDAStream(x.k.device().index()).stream();
        Scratch scratch(fp8 ? a[15] : Py_None, x.k);
        call(call_name.c_str(), [&] {
            void* o = out.make();
            float* l = need_lse ? static_cast<float*>(lse.make()) : nullptr;
            if (fp8) scratch.need(sfa_paged_forward_fp8_workspace_size(&p, &x.f));
            return fp8 ? sfa_paged_forward_fp8(&p, &x.f, q.data_ptr(), qs, o, l, scratch.ptr, scratch.bytes, status, stream)
                       : sfa_paged_forward(&p, &x.c, q.data_ptr(), qs, o, l, status, stream);
        });
        if (!need_lse) return tuple_of({out.object(), Py_NewRef(Py_None)});
        return tuple_of({out.object(), lse.object()});
    });
}
PyObject* paged_forward(PyObject*, PyObject* const* a, Py_ssize_t n) { return forward_over("paged_forward", false, a, n); }
PyObject* paged_forward_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return forward_over("paged_forward_fp8", true, a, n);
}

// ------------------------------------- residual addition, norm and 8-bit rows

// Rows of x [..., dim] at one stride.
struct RowsIn {
    const Tensor& x;
    sfa_dtype dt;
    int64_t N, dim, stride;

    RowsIn(PyObject* o, const char* name) : x(tensor(o, name)) {
        dt = dtype_of(x);
        if (!x.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
        if (x.dim() < 1 || x.size(-1) < 1) refuse(std::string(name) + " must be [..., dim], got " + shape_text(x.sizes()));
        dim = x.size(-1);
        N = x.numel() / dim;
        stride = row_stride(x, name, dim);
    }
    // The stride of its rows, which all leading dimensions share.
    static int64_t row_stride(const Tensor& t, const char* name, int64_t dim) {
        if (t.numel() <= dim) {
            if (t.numel() > 0 && t.stride(-1) != 1 && dim > 1) refuse(std::string(name) + ": rows must be contiguous");
            return dim;
        }
        bool one = t.stride(-1) == 1 || dim == 1;
        int64_t step = -1, rows = 1;
        for (int64_t i = t.dim() - 2; i >= 0; --i) {
            if (t.size(i) == 1) continue;
            if (step < 0) step = t.stride(i);
            one = one && t.stride(i) == step * rows;
            rows *= t.size(i);
        }
        if (!one || step < dim || step * t.element_size() % 16 != 0)
            refuse(std::string(name) + ": rows must be contiguous and at one stride of a multiple of 16 bytes, got strides " +
                   shape_text(t.strides()));
        return step;
    }
    at::IntArrayRef lead() const { return x.sizes().slice(0, x.dim() - 1); }
};

// x, residual, w, eps, fp8, h, y, scale
PyObject* add_rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded("add_rms_norm", n, 8, [&]() -> PyObject* {
        const RowsIn in(a[0], "x");
        const bool sum = a[1] != Py_None, fp8 = truth(a[4]);
        const Tensor& r = sum ? tensor(a[1], "residual") : in.x;
        like(r, "residual", in.x);
        if (r.sizes() != in.x.sizes()) refuse("residual must be " + shape_text(in.x.sizes()) + ", got " + shape_text(r.sizes()));
        const int64_t rs = RowsIn::row_stride(r, "residual", in.dim);
        const float* w = static_cast<const float*>(dense(tensor(a[2], "w"), "w", {in.dim}, at::kFloat, in.x));
        const double eps = number(a[3]);
        if (!sum && a[5] != Py_None) refuse("out[0] goes with a residual");
        if (!fp8 && a[7] != Py_None) refuse("out[2] goes with fp8");
        c10::cuda::OptionalCUDAGuard guard(in.x.device());
        Out h(sum ? a[5] : Py_None, "out[0]", in.x.sizes(), in.x.scalar_type(), in.x);
        Out y(a[6], "out[1]", in.x.sizes(), fp8 ? at::kFloat8_e4m3fn : in.x.scalar_type(), in.x);
        Out s(fp8 ? a[7] : Py_None, "out[2]", in.lead(), at::kFloat, in.x);
        const auto stream = c10::cuda::getCurrentCUDAStream(in.x.device().index()).stream();
        call("sfa_add_rms_norm", [&] {
            void* to_h = sum ? h.make() : nullptr;
            void* to_y = y.make();
            return sfa_add_rms_norm(in.dt, small(in.N), small(in.dim), in.x.data_ptr(), in.stride, sum ? r.data_ptr() : nullptr, rs,
                                    w, (float)eps, to_h, fp8 ? nullptr : to_y, fp8 ? to_y : nullptr,
                                    fp8 ? static_cast<float*>(s.make()) : nullptr, stream);
        });
        PyObject* first = sum ? h.object() : Py_NewRef(a[0]);
        if (!fp8) return tuple_of({first, y.object()});
        return tuple_of({first, y.object(), s.object()});
    });
}

// x, x8, scale
PyObject* quantize_rows_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded("quantize_rows_fp8", n, 3, [&]() -> PyObject* {
        const RowsIn in(a[0], "x");
        c10::cuda::OptionalCUDAGuard guard(in.x.device());
        Out y(a[1], "out[0]", in.x.sizes(), at::kFloat8_e4m3fn, in.x), s(a[2], "out[1]", in.lead(), at::kFloat, in.x);
        const auto stream = c10::cuda::getCurrentCUDAStream(in.x.device().index()).stream();
        call("sfa_quantize_rows_fp8", [&] {
            void* to = y.make();
            return sfa_quantize_rows_fp8(in.dt, small(in.N), small(in.dim), in.x.data_ptr(), in.stride, to,
                                         static_cast<float*>(s.make()), stream);
        });
        return tuple_of({y.object(), s.object()});
    });
}

// h, w, dy, dh, eps, workspace, dx, dw
PyObject* add_rms_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded("add_rms_norm_backward", n, 8, [&]() -> PyObject* {
        const RowsIn in(a[0], "h");
        const auto type = in.x.scalar_type();
        const void* h = dense(in.x, "h", in.x.sizes(), type, in.x);
        const float* w = static_cast<const float*>(dense(tensor(a[1], "w"), "w", {in.dim}, at::kFloat, in.x));
        const void* dy = dense(tensor(a[2], "dy"), "dy", in.x.sizes(), type, in.x);
        const void* dh = dense_or_null(a[3], "dh", in.x.sizes(), type, in.x);
        const double eps = number(a[4]);
        Scratch scratch(a[5], in.x);
        c10::cuda::OptionalCUDAGuard guard(in.x.device());
        Out dx(a[6], "out[0]", in.x.sizes(), type, in.x), dw(a[7], "out[1]", {in.dim}, at::kFloat, in.x);
        const auto stream = c10::cuda::getCurrentCUDAStream(in.x.device().index()).stream();
        call("sfa_add_rms_norm_backward", [&] {
            const int N = small(in.N), dim = small(in.dim);
            scratch.need(sfa_add_rms_norm_backward_workspace_size(in.dt, N, dim));
            void* to = dx.make();
            return sfa_add_rms_norm_backward(in.dt, N, dim, h, w, (float)eps, dy, dh, to, static_cast<float*>(dw.make()),
                                             scratch.ptr, scratch.bytes, stream);
        });
        return tuple_of({dx.object(), dw.object()});
    });
}

// x8, x_scale, w8, w_scale, theta, rope, q, k, v, status
PyObject* qkv_rope_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded("qkv_rope_fp8", n, 10, [&]() -> PyObject* {
        const Tensor& x = tensor(a[0], "x8");
        if (x.dim() != 3 || x.scalar_type() != at::kFloat8_e4m3fn || !x.is_cuda() || !x.is_contiguous())
            refuse("x8 must be a contiguous float8_e4m3fn [B, T, d_model] CUDA tensor, got " +
                   std::string(at::toString(x.scalar_type())) + " " + shape_text(x.sizes()));
        const int64_t B = x.size(0), T = x.size(1), dm = x.size(2), rows = (kHq + 2 * kHkv) * kD;
        const float* sx = static_cast<const float*>(dense(tensor(a[1], "x_scale"), "x_scale", {B, T}, at::kFloat, x));
        const void* w = dense(tensor(a[2], "w8"), "w8", {rows, dm}, at::kFloat8_e4m3fn, x);
        const float* sw = static_cast<const float*>(dense(tensor(a[3], "w_scale"), "w_scale", {rows}, at::kFloat, x));
        const double theta = number(a[4]);
        int64_t have;
        const float* rope = table(a[5], x, &have);
        if (theta > 0 && have < T && B > 0)
            refuse("rope has " + std::to_string(have) + " rows, the sequence " + std::to_string(T));
        const int64_t qs[4] = {B, T, kHq, kD}, ks[4] = {B, T, kHkv, kD};
        Out q(a[6], "out[0]", qs, at::kBFloat16, x), k(a[7], "out[1]", ks, at::kBFloat16, x), v(a[8], "out[2]", ks, at::kBFloat16, x);
        unsigned* status = status_word(a[9], x);
        const sfa_params p = params(B, T, SFA_BF16, theta);
        c10::cuda::OptionalCUDAGuard guard(x.device());
        const auto stream = c10::cuda::getCurrentCUDAStream(x.device().index()).stream();
        call("sfa_qkv_rope_fp8", [&] {
            void *to_q = q.make(), *to_k = k.make(), *to_v = v.make();
            return sfa_qkv_rope_fp8(&p, small(dm), x.data_ptr(), sx, w, sw, rope, to_q, to_k, to_v, status, stream);
        });
        return tuple_of({q.object(), k.object(), v.object()});
    });
}

// t, heads: the token stride of t [..., heads, 64], on any device.
PyObject* stride_of(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded("stride_of", n, 2, [&]() -> PyObject* {
        const Tensor& t = tensor(a[0], "t");
        if (t.dim() < 3) refuse("t must be [..., heads, 64]");
        return PyLong_FromLongLong(token_stride(t, "t", t.sizes().slice(0, t.dim() - 2), integer(a[1])));
    });
}

template <typename F>
PyCFunction fast(F f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"norm_rope", fast(norm_rope), METH_FASTCALL, nullptr},
                         {"norm_rope_backward", fast(norm_rope_backward), METH_FASTCALL, nullptr},
                         {"paged_append", fast(paged_append), METH_FASTCALL, nullptr},
                         {"paged_forward", fast(paged_forward), METH_FASTCALL, nullptr},
                         {"paged_append_fp8", fast(paged_append_fp8), METH_FASTCALL, nullptr},
                         {"paged_forward_fp8", fast(paged_forward_fp8), METH_FASTCALL, nullptr},
                         {"add_rms_norm", fast(add_rms_norm), METH_FASTCALL, nullptr},
                         {"add_rms_norm_backward", fast(add_rms_norm_backward), METH_FASTCALL, nullptr},
                         {"quantize_rows_fp8", fast(quantize_rows_fp8), METH_FASTCALL, nullptr},
                         {"qkv_rope_fp8", fast(qkv_rope_fp8), METH_FASTCALL, nullptr},
                         {"stride_of", fast(stride_of), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_sfa_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__sfa_bind() { return PyModule_Create(&module); }
