// pw_binding.cpp -- argument marshalling of the calls on new tokens for Python: tensors in, checked and
// turned into the pointers and strides of the C ABI.  In C++ because a decoding step makes these calls
// once a layer on a few kilobytes: marshalled by ctypes a call took 15 to 18 us of the host, of a kernel
// of 3 to 14 us.
//
// Each function takes its arguments by position, in the order of api.py's calls of it, and returns the
// status code.  A tensor of the wrong type, device or layout raises AssertionError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

#include "../../include/pw.h"

namespace {

// Thrown with a Python error set.
struct Raised {};

[[noreturn]] void refuse(const char *what)
{
    PyErr_SetString(PyExc_AssertionError, what);
    throw Raised{};
}

void require(bool ok, const char *what)
{
    if (!ok)
        refuse(what);
}

// The arguments of a call, taken one after the other.
struct Args {
    PyObject *const *at, *const *end;

    PyObject *next()
    {
        if (at == end) {
            PyErr_SetString(PyExc_TypeError, "too few arguments");
            throw Raised{};
        }
        return *at++;
    }

    // null for None
    const at::Tensor *tensor()
    {
        PyObject *o = next();
        if (o == Py_None)
            return nullptr;
        if (!THPVariable_Check(o)) {
            PyErr_SetString(PyExc_TypeError, "a tensor is expected");
            throw Raised{};
        }
        return &THPVariable_Unpack(o);
    }

    const at::Tensor &needed(const char *name)
    {
        const at::Tensor *t = tensor();
        require(t != nullptr, name);
        return *t;
    }

    int64_t integer()
    {
        const long long v = PyLong_AsLongLong(next());
        if (v == -1 && PyErr_Occurred())
            throw Raised{};
        return v;
    }

    int small()
    {
        const int64_t v = integer();
        require(v >= INT32_MIN && v <= INT32_MAX, "an integer argument lies outside 32 bits");
        return static_cast<int>(v);
    }

    bool truth()
    {
        const int v = PyObject_IsTrue(next());
        if (v < 0)
            throw Raised{};
        return v != 0;
    }

    float real()
    {
        const double v = PyFloat_AsDouble(next());
        if (v == -1.0 && PyErr_Occurred())
            throw Raised{};
        return static_cast<float>(v);
    }

    // The stream of the call: the last argument's, or the device's current one.
    void *stream(c10::Device dev)
    {
        PyObject *o = next();
        if (o == Py_None)
            return c10::cuda::getCurrentCUDAStream(dev.index()).stream();
        PyObject *h = PyObject_GetAttrString(o, "cuda_stream");
        if (h == nullptr)
            throw Raised{};
        void *s = PyLong_AsVoidPtr(h);
        Py_DECREF(h);
        if (s == nullptr && PyErr_Occurred())
            throw Raised{};
        return s;
    }
};

// bf16 rows of heads [T, H, 128]
struct Rows {
    void *p = nullptr;
    int64_t st = 0, sh = 0, T = 0;
    int H = 0;

    Rows(const at::Tensor *x, c10::Device dev, const char *name)
    {
        if (x == nullptr)
            return;
        require(x->dim() == 3 && x->scalar_type() == at::kBFloat16 && x->size(2) == 128 && x->stride(2) == 1 && x->device() == dev, name);
        require(x->size(1) <= INT32_MAX, name);
        T = x->size(0);
        H = static_cast<int>(x->size(1));
        st = T > 1 ? x->stride(0) : 128 * static_cast<int64_t>(H);
        sh = H > 1 ? x->stride(1) : 128;
        p = x->data_ptr();
    }
};

template <class T>
T *plain(const at::Tensor *t, at::ScalarType type, c10::Device dev, const char *name)
{
    if (t == nullptr)
        return nullptr;
    require(t->scalar_type() == type && t->device() == dev && t->is_contiguous(), name);
    return static_cast<T *>(t->data_ptr());
}

// A norm weight, bf16 [128] or [heads, 128].
struct Weight {
    const void *p;
    int stride = 0;

    Weight(const at::Tensor *w, int heads, c10::Device dev) : p(plain<void>(w, at::kBFloat16, dev, "norm weight: contiguous bf16 on the rows' device"))
    {
        if (w == nullptr)
            return;
        require((w->dim() == 1 && w->size(0) == 128) || (w->dim() == 2 && w->size(0) == heads && w->size(1) == 128),
                "norm weight: [128] or [heads, 128]");
        stride = w->dim() == 2 ? 128 : 0;
    }
};

struct Rope {
    const float *p;
    int max_pos = 0, rot = 0;

    Rope(const at::Tensor *r, c10::Device dev) : p(plain<float>(r, at::kFloat, dev, "rope: contiguous fp32 on the rows' device"))
    {
        if (r == nullptr)
            return;
        require(r->dim() == 2 && r->size(0) <= INT32_MAX && r->size(1) <= 1024, "rope: [max_pos, rot_dim]");
        max_pos = static_cast<int>(r->size(0));
        rot = static_cast<int>(r->size(1));
    }
};

// cu_seqlens [B + 1] and ctx_lens [B] or None
struct Batch {
    const int32_t *cu, *ctx;
    int B;

    Batch(const at::Tensor &c, const at::Tensor *x, c10::Device dev)
        : cu(plain<int32_t>(&c, at::kInt, dev, "cu_seqlens: contiguous int32 on the rows' device")),
          ctx(plain<int32_t>(x, at::kInt, dev, "ctx_lens: contiguous int32 on the rows' device"))
    {
        require(c.numel() >= 1 && c.numel() <= INT32_MAX, "cu_seqlens: [B + 1]");
        B = static_cast<int>(c.numel() - 1);
        require(x == nullptr || x->numel() == B, "ctx_lens: [B]");
    }
};

// The paged cache and its table.
struct Cache {
    void *k, *v;
    const int32_t *table;
    int n_phys, Hkv, max_pages;

    Cache(const at::Tensor &K, const at::Tensor &V, const at::Tensor &t, int B, c10::Device dev)
        : k(plain<void>(&K, at::kByte, dev, "K_pages: contiguous uint8 on the rows' device")),
          v(plain<void>(&V, at::kByte, dev, "V_pages: contiguous uint8 on the rows' device")),
          table(plain<int32_t>(&t, at::kInt, dev, "page_table: contiguous int32 on the rows' device"))
    {
        require(K.dim() == 4 && K.size(2) == 64 && K.size(3) == 128 && K.sizes() == V.sizes(), "pages: [n_phys, Hkv, 64, 128]");
        require(t.dim() == 2 && t.size(0) == B, "page_table: [B, max_pages]");
        require(K.size(0) <= INT32_MAX && K.size(1) <= INT32_MAX && t.size(1) <= INT32_MAX, "a size lies outside 32 bits");
        n_phys = static_cast<int>(K.size(0));
        Hkv = static_cast<int>(K.size(1));
        max_pages = static_cast<int>(t.size(1));
    }
};

// The tensors' device is made the current one for the call.
struct OnDevice {
    c10::DeviceIndex before = -1;

    explicit OnDevice(c10::Device dev)
    {
        const c10::DeviceIndex now = c10::cuda::current_device();
        if (now != dev.index()) {
            c10::cuda::set_device(dev.index());
            before = now;
        }
    }
    ~OnDevice()
    {
        try {
            if (before >= 0)
                c10::cuda::set_device(before);
        } catch (...) { // the next call on that device says why
        }
    }
};

template <class F>
PyObject *guarded(PyObject *const *args, Py_ssize_t n, F f)
{
    try {
        Args a{args, args + n};
        return PyLong_FromLong(f(a));
    } catch (const Raised &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

template <class F>
pw_status launch(c10::Device dev, F f)
{
    const OnDevice on(dev);
    PyThreadState *const state = PyEval_SaveThread();
    const pw_status s = f();
    PyEval_RestoreThread(state);
    return s;
}

// Q, K, cu_seqlens, ctx_lens, q_weight, k_weight, eps, rope, interleaved, Q_out, K_out, status, stream
PyObject *qk_norm_rope(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded(args, n, [](Args &a) {
        const at::Tensor *Q = a.tensor(), *K = a.tensor();
        const at::Tensor *x = Q != nullptr ? Q : K;
        require(x != nullptr && x->is_cuda(), "Q or K on a CUDA device");
        const c10::Device dev = x->device();
        const Rows q(Q, dev, "Q: bf16 [T, Hq, 128]"), k(K, dev, "K: bf16 [T, Hk, 128]");
        const int64_t T = Q != nullptr ? q.T : k.T;
        require(K == nullptr || k.T == T, "Q and K have the same rows");
        const at::Tensor &cu = a.needed("cu_seqlens");
        const Batch b(cu, a.tensor(), dev);
        const Weight qw(a.tensor(), q.H, dev), kw(a.tensor(), k.H, dev);
        const float eps = a.real();
        const Rope r(a.tensor(), dev);
        const bool interleaved = a.truth();
        const Rows qo(a.tensor(), dev, "Q_out: bf16 [T, Hq, 128]"), ko(a.tensor(), dev, "K_out: bf16 [T, Hk, 128]");
        require(qo.H == q.H && ko.H == k.H && (Q == nullptr || qo.T == T) && (K == nullptr || ko.T == T),
                "an output's shape differs from its input's");
        int32_t *const status = plain<int32_t>(a.tensor(), at::kInt, dev, "status: int32 on the rows' device");
        void *const stream = a.stream(dev);
        return launch(dev, [&] {
            return pw_qk_norm_rope(q.p, q.st, q.sh, q.H, k.p, k.st, k.sh, k.H, qw.p, qw.stride, kw.p, kw.stride, eps, r.p, r.max_pos, r.rot,
                                   interleaved, b.cu, b.ctx, b.B, T, qo.p, qo.st, qo.sh, ko.p, ko.st, ko.sh, status, stream);
        });
    });
}

// K, V, K_pages, V_pages, page_table, cu_seqlens, ctx_lens, k_scale, v_scale, k_weight, eps, rope, interleaved, status, stream
PyObject *append(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded(args, n, [](Args &a) {
        const at::Tensor &K = a.needed("K"), &V = a.needed("V");
        require(K.is_cuda(), "K on a CUDA device");
        const c10::Device dev = K.device();
        const Rows k(&K, dev, "K: bf16 [T, Hkv, 128]"), v(&V, dev, "V: bf16 [T, Hkv, 128]");
        const at::Tensor &Kp = a.needed("K_pages"), &Vp = a.needed("V_pages"), &table = a.needed("page_table"), &cu = a.needed("cu_seqlens");
        const Batch b(cu, a.tensor(), dev);
        const Cache c(Kp, Vp, table, b.B, dev);
        require(k.H == c.Hkv && v.H == c.Hkv && v.T == k.T, "K and V have the cache's heads and the same rows");
        const float ks = a.real(), vs = a.real();
        const Weight kw(a.tensor(), k.H, dev);
        const float eps = a.real();
        const Rope r(a.tensor(), dev);
        const bool interleaved = a.truth();
        int32_t *const status = plain<int32_t>(a.tensor(), at::kInt, dev, "status: int32 on the rows' device");
        void *const stream = a.stream(dev);
        return launch(dev, [&] {
            return pw_append(k.p, k.st, k.sh, v.p, v.st, v.sh, c.Hkv, kw.p, kw.stride, eps, r.p, r.max_pos, r.rot, interleaved, b.cu, b.ctx,
                             b.B, k.T, c.table, c.max_pages, c.n_phys, ks, vs, c.k, c.v, status, stream);
        });
    });
}

// Q, K_pages, V_pages, page_table, cu_seqlens, ctx_lens, max_q_len, window, k_scale, v_scale, sm_scale, O, lse, workspace, status, stream
PyObject *chunk_attn(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded(args, n, [](Args &a) {
        const at::Tensor &Q = a.needed("Q");
        require(Q.is_cuda(), "Q on a CUDA device");
        const c10::Device dev = Q.device();
        const Rows q(&Q, dev, "Q: bf16 [T, Hq, 128]");
        const at::Tensor &Kp = a.needed("K_pages"), &Vp = a.needed("V_pages"), &table = a.needed("page_table"), &cu = a.needed("cu_seqlens");
        const Batch b(cu, a.tensor(), dev);
        const Cache c(Kp, Vp, table, b.B, dev);
        const int max_q = a.small(), window = a.small();
        const float ks = a.real(), vs = a.real(), sm = a.real();
        const at::Tensor &O = a.needed("O");
        void *const o = plain<void>(&O, at::kBFloat16, dev, "O: contiguous bf16 on Q's device");
        require(O.sizes() == Q.sizes(), "O has Q's shape");
        const at::Tensor *l = a.tensor();
        float *const lse = plain<float>(l, at::kFloat, dev, "lse: contiguous fp32 on Q's device");
        require(l == nullptr || (l->dim() == 2 && l->size(0) == q.T && l->size(1) == q.H), "lse: [T, Hq]");
        const at::Tensor &w = a.needed("workspace");
        require(w.device() == dev && w.is_contiguous(), "workspace: contiguous, on Q's device");
        int32_t *const status = plain<int32_t>(a.tensor(), at::kInt, dev, "status: int32 on Q's device");
        void *const stream = a.stream(dev);
        return launch(dev, [&] {
            return pw_chunk_attn(q.p, q.st, q.sh, q.H, c.k, c.v, c.Hkv, c.table, c.max_pages, c.n_phys, b.cu, b.ctx, b.B, q.T, max_q, window, ks,
                                 vs, sm, o, lse, w.data_ptr(), w.nbytes(), status, stream);
        });
    });
}

#define PW_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL

PyMethodDef methods[] = {{"pw_qk_norm_rope", PW_FAST(qk_norm_rope), "pw_qk_norm_rope of include/pw.h on tensors"},
                         {"pw_append", PW_FAST(append), "pw_append of include/pw.h on tensors"},
                         {"pw_chunk_attn", PW_FAST(chunk_attn), "pw_chunk_attn of include/pw.h on tensors"},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pw_binding", "Argument marshalling of the calls on new tokens.", -1, methods};

} // namespace

// What it was compiled for: build.py looks for the text in the file, the loader at the attribute.
#ifndef PW_BUILT_FOR
#error "PW_BUILT_FOR: the versions of torch and Python (build.py sets it)"
#endif

PyMODINIT_FUNC PyInit__pw_binding(void)
{
    static const char text[] = "[built for " PW_BUILT_FOR "]";
    PyObject *const m = PyModule_Create(&module);
    if (m != nullptr && PyModule_AddStringConstant(m, "built_for", text) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
