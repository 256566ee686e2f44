// Marshals tensors into the C ABI for the calls that serving makes for every
// token, where the host's time per call counts: rotary.py and paged.py call it.
// It checks shapes, types and devices, allocates outputs and workspaces on the
// tensors' device and current stream, and calls libda.so. What depends on
// values and sizes alone the library checks itself. A whole call takes the host
// 6.5 us (rotary norm), 5.1 (append) and 6.5 (attention), launches among it; in
// Python it took 23, 27 and 32.
#include <Python.h>

#include <dlfcn.h>

#include <cmath>
#include <initializer_list>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "paged.h"

namespace {

using at::Tensor;

PyObject *g_error = nullptr;  // DaError
struct Library {
    decltype(&qkr_forward) qkr_forward_;
    decltype(&qkr_workspace_size) qkr_workspace_size_;
    decltype(&qkr_backward) qkr_backward_;
    decltype(&pg_append) pg_append_;
    decltype(&pg_path) pg_path_;
    decltype(&pg_workspace_size) pg_workspace_size_;
    decltype(&pg_attention) pg_attention_;
    decltype(&da_last_error) da_last_error_;
} g_lib{};

// bind(handle of libda.so, DaError)
PyObject *bind(PyObject *, PyObject *args)
{
    unsigned long long handle = 0;
    PyObject *error = nullptr;
    if (!PyArg_ParseTuple(args, "KO", &handle, &error)) return nullptr;
    void *h = reinterpret_cast<void *>(handle);
    const auto find = [&](auto &f, const char *name) { return (f = reinterpret_cast<std::decay_t<decltype(f)>>(dlsym(h, name))) != nullptr; };
    if (!find(g_lib.qkr_forward_, "qkr_forward") || !find(g_lib.qkr_workspace_size_, "qkr_workspace_size") ||
        !find(g_lib.qkr_backward_, "qkr_backward") || !find(g_lib.pg_append_, "pg_append") || !find(g_lib.pg_path_, "pg_path") ||
        !find(g_lib.pg_workspace_size_, "pg_workspace_size") || !find(g_lib.pg_attention_, "pg_attention") ||
        !find(g_lib.da_last_error_, "da_last_error")) {
        PyErr_SetString(PyExc_RuntimeError, "libda.so lacks an entry point; build it anew");
        return nullptr;
    }
    Py_INCREF(error);
    Py_XDECREF(g_error);
    g_error = error;
    Py_RETURN_NONE;
}

// Raised as DaError(status, message).
struct Status {
    da_status status;
};
void check(da_status st)
{
    if (st != DA_OK) throw Status{st};
}

template <typename F> PyObject *guarded(F &&f)
{
    HANDLE_TH_ERRORS
    try {
        return f();
    } catch (const Status &s) {
        if (PyObject *e = PyObject_CallFunction(g_error, "is", static_cast<int>(s.status), g_lib.da_last_error_())) {
            PyErr_SetObject(g_error, e);
            Py_DECREF(e);
        }
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// ---- arguments ---------------------------------------------------------------

// A tensor, or null for None.
const Tensor *tensor(PyObject *o, const char *name)
{
    if (o == Py_None) return nullptr;
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
    return &THPVariable_Unpack(o);
}
const Tensor &needed(PyObject *o, const char *name)
{
    const Tensor *t = tensor(o, name);
    TORCH_CHECK_TYPE(t, name, " must be a tensor");
    return *t;
}

bool is(const Tensor &t, std::initializer_list<int64_t> shape) { return t.sizes() == at::IntArrayRef(shape); }

int type_of(const Tensor &t, const char *what)
{
    switch (t.scalar_type()) {
    case at::kFloat: return DA_F32;
    case at::kBFloat16: return DA_BF16;
    case at::kHalf: return DA_F16;
    default: TORCH_CHECK_TYPE(false, what, " must be float32, bfloat16 or float16");
    }
}

// All tensors that are there and not empty live on the device of this index.
void together(std::initializer_list<const Tensor *> all, int index)
{
    for (const Tensor *t : all) {
        if (!t || t->numel() == 0) continue;
        TORCH_CHECK_VALUE(t->is_cuda(), "device tensors must live on a CUDA device");
        TORCH_CHECK_VALUE(t->get_device() == index, "tensors must all live on one CUDA device");
    }
}

// Data of a tensor whose last dimension is contiguous; null if it is empty.
void *strided(const Tensor &t, const char *name)
{
    if (t.numel() == 0) return nullptr;
    TORCH_CHECK_VALUE(t.stride(-1) == 1 || t.size(-1) == 1, name, "'s last dimension must be contiguous");
    return t.data_ptr();
}

void *plain(const Tensor &t)
{
    if (t.numel() == 0) return nullptr;
    TORCH_CHECK_VALUE(t.is_contiguous(), "tensors must be contiguous");
    return t.data_ptr();
}

// An optional tensor of this shape and type, and its data.
void shaped(const Tensor *t, const char *name, std::initializer_list<int64_t> shape, at::ScalarType type)
{
    TORCH_CHECK_VALUE(!t || (is(*t, shape) && t->scalar_type() == type), name, " must be ", type, " ", at::IntArrayRef(shape));
}
template <typename T> T *data(const Tensor *t) { return t ? static_cast<T *>(plain(*t)) : nullptr; }

void like(const Tensor &t, const char *name, const Tensor &of, at::IntArrayRef shape)
{
    TORCH_CHECK_VALUE(t.sizes() == shape && t.scalar_type() == of.scalar_type(), name, " must be ", of.scalar_type(), " ", shape);
}

// A new contiguous tensor of t's type and device.
Tensor fresh(const Tensor &t, at::IntArrayRef shape)
{
    return at::empty(shape, t.options().requires_grad(false), at::MemoryFormat::Contiguous);
}

Tensor scratch(const Tensor &like, size_t bytes)
{
    return at::empty({static_cast<int64_t>(bytes)}, like.options().dtype(at::kByte).requires_grad(false));
}

void strides(const Tensor &t, int64_t *to, int n)
{
    for (int i = 0; i < n; ++i) to[i] = t.stride(i);
}

// The tensors' device and its current stream, without Python's lock: allocations
// and launches can block.
struct On {
    struct Unlocked {
        PyThreadState *state = PyEval_SaveThread();
        ~Unlocked() { PyEval_RestoreThread(state); }
    } unlocked;
    c10::cuda::OptionalCUDAGuard guard;
    da_stream_t stream = nullptr;

    explicit On(const Tensor &t)
    {
        TORCH_CHECK_VALUE(t.is_cuda(), "device tensors must live on a CUDA device");
        guard.set_device(t.device());
        stream = reinterpret_cast<da_stream_t>(c10::cuda::getCurrentCUDAStream(t.get_device()).stream());
    }
};

double number(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}
bool truth(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}

// None for a tensor that is not there.
PyObject *wrap(const Tensor &t)
{
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}
template <int N> PyObject *wrap(const Tensor (&t)[N])
{
    PyObject *r = PyTuple_New(N);
    if (!r) throw python_error();
    for (int i = 0; i < N; ++i) PyTuple_SET_ITEM(r, i, wrap(t[i]));
    return r;
}

void count(Py_ssize_t n, Py_ssize_t wanted) { TORCH_CHECK_TYPE(n == wanted, "expected ", wanted, " arguments"); }

// ---- rotary norm -------------------------------------------------------------

// q, k, frequencies, q_weight, k_weight, pos_q, pos_k, eps, interleaved, magnitude
constexpr int kRotary = 10;

struct Rotary {
    qkr_problem p{};
    const Tensor *q, *k, *turns, *wq, *wk, *pq, *pk;
    int index;

    const Tensor &any() const { return q ? *q : *k; }

    // What shapes and types allow to check.
    explicit Rotary(PyObject *const *a)
        : q(tensor(a[0], "q")), k(tensor(a[1], "k")), turns(tensor(a[2], "frequencies")), wq(tensor(a[3], "q_weight")),
          wk(tensor(a[4], "k_weight")), pq(tensor(a[5], "pos_q")), pk(tensor(a[6], "pos_k"))
    {
        TORCH_CHECK_VALUE(q || k, "there must be q or k");
        TORCH_CHECK_VALUE(!q || (q->dim() == 5 && q->size(3) == 2), "q must be [B, L, heads, 2, D]");
        TORCH_CHECK_VALUE(!k || (k->dim() == 5 && k->size(3) == 2), "k must be [B, L, heads, 2, D]");
        p.dtype = type_of(any(), "q and k");
        if (q && k) {
            TORCH_CHECK_TYPE(q->scalar_type() == k->scalar_type(), "q and k must have one type");
            TORCH_CHECK_VALUE(q->size(0) == k->size(0) && q->size(4) == k->size(4), "q and k disagree on batch or width");
        }
        TORCH_CHECK_VALUE(q || (!wq && !pq), "q_weight and pos_q go with q");
        TORCH_CHECK_VALUE(k || (!wk && !pk), "k_weight and pos_k go with k");
        p.normed = a[7] != Py_None;
        p.eps = p.normed ? static_cast<float>(number(a[7])) : 0.f;
        TORCH_CHECK_VALUE(p.normed || (!wq && !wk), "a weight needs the norm (eps)");
        TORCH_CHECK_VALUE(!turns || (turns->dim() == 1 && turns->scalar_type() == at::kLong),
                          "frequencies must be int64 [rotated / 2] (rotary_frequencies)");
        p.interleaved = truth(a[8]);
        p.magnitude = static_cast<float>(number(a[9]));
        const int64_t B = any().size(0), D = any().size(4), Lq = q ? q->size(1) : 0, Lk = k ? k->size(1) : 0;
        const int64_t H = q ? q->size(2) : 1, Hkv = k ? k->size(2) : 1, R = turns ? 2 * turns->size(0) : 0;
        for (int64_t n : {B, D, Lq, Lk, H, Hkv, R}) TORCH_CHECK_VALUE(n <= INT32_MAX, "a size exceeds 2^31 - 1");
        p.batch = static_cast<int32_t>(B);
        p.width = static_cast<int32_t>(D);
        p.num_queries = static_cast<int32_t>(Lq);
        p.num_keys = static_cast<int32_t>(Lk);
        p.num_heads = static_cast<int32_t>(H);
        p.num_kv_heads = static_cast<int32_t>(Hkv);
        p.rotated = static_cast<int32_t>(R);
        shaped(wq, "q_weight", {D}, at::kFloat);
        shaped(wk, "k_weight", {D}, at::kFloat);
        shaped(pq, "pos_q", {B, Lq}, at::kInt);
        shaped(pk, "pos_k", {B, Lk}, at::kInt);
        index = static_cast<int>(any().get_device());
    }

    void fill()
    {
        together({q, k, turns, wq, wk, pq, pk}, index);
        p.q_weight = data<float>(wq);
        p.k_weight = data<float>(wk);
        p.pos_q = data<int32_t>(pq);
        p.pos_k = data<int32_t>(pk);
        p.turns = data<int64_t>(turns);
        if (q) {
            p.q = strided(*q, "q");
            strides(*q, p.q_stride, 4);
        }
        if (k) {
            p.k = strided(*k, "k");
            strides(*k, p.k_stride, 4);
        }
    }
};

// (the rotary arguments, out_q, out_k) -> (q, k)
PyObject *rotary_forward(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        count(n, kRotary + 2);
        Rotary r(a);
        const Tensor *given[2] = {tensor(a[kRotary], "out_q"), tensor(a[kRotary + 1], "out_k")}, *ins[2] = {r.q, r.k};
        static const char *names[2] = {"out_q", "out_k"};
        for (int i = 0; i < 2; ++i) {
            TORCH_CHECK_VALUE(ins[i] || !given[i], names[i], " has no input");
            if (given[i]) like(*given[i], names[i], *ins[i], ins[i]->sizes());
        }
        together({given[0], given[1]}, r.index);
        r.fill();
        Tensor out[2];
        {
            const On at(r.any());
            void *to[2] = {nullptr, nullptr};
            for (int i = 0; i < 2; ++i)
                if (ins[i]) {
                    out[i] = given[i] ? *given[i] : fresh(*ins[i], ins[i]->sizes());
                    to[i] = plain(out[i]);
                }
            check(g_lib.qkr_forward_(&r.p, to[0], to[1], at.stream));
        }
        return wrap(out);
    });
}

// (the rotary arguments, grad_out_q, grad_out_k) -> (grad_q, grad_k, grad_q_weight, grad_k_weight)
PyObject *rotary_backward(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        count(n, kRotary + 2);
        Rotary r(a);
        const Tensor *gs[2] = {tensor(a[kRotary], "grad_out_q"), tensor(a[kRotary + 1], "grad_out_k")}, *ins[2] = {r.q, r.k}, *ws[2] = {r.wq, r.wk};
        static const char *names[2] = {"grad_out_q", "grad_out_k"};
        for (int i = 0; i < 2; ++i) {
            TORCH_CHECK_VALUE(!ins[i] == !gs[i], names[i], " goes with its input");
            if (gs[i]) like(*gs[i], names[i], *ins[i], ins[i]->sizes());
        }
        together({gs[0], gs[1]}, r.index);
        r.fill();
        const void *g[2] = {data<void>(gs[0]), data<void>(gs[1])};
        Tensor out[4];
        {
            const On at(r.any());
            void *to[4] = {};
            for (int i = 0; i < 2; ++i) {
                if (ins[i]) out[i] = fresh(*ins[i], ins[i]->sizes());
                if (ws[i]) out[2 + i] = fresh(*ws[i], ws[i]->sizes());
            }
            for (int i = 0; i < 4; ++i)
                if (out[i].defined()) to[i] = plain(out[i]);
            size_t bytes = 0;
            check(g_lib.qkr_workspace_size_(&r.p, &bytes));
            const Tensor scratch_ = bytes ? scratch(r.any(), bytes) : Tensor();
            check(g_lib.qkr_backward_(&r.p, g[0], g[1], to[0], to[1], static_cast<float *>(to[2]), static_cast<float *>(to[3]),
                                      bytes ? scratch_.data_ptr() : nullptr, bytes, at.stream));
        }
        return wrap(out);
    });
}

// ---- paged cache -------------------------------------------------------------

// k_cache, v_cache, page_table, lengths, counts
struct Cache {
    const Tensor &k, &v, &table, &lengths;
    const Tensor *counts;
    int64_t L;  // places of a sequence

    explicit Cache(PyObject *const *a)
        : k(needed(a[0], "k_cache")), v(needed(a[1], "v_cache")), table(needed(a[2], "page_table")), lengths(needed(a[3], "lengths")),
          counts(tensor(a[4], "counts"))
    {
        TORCH_CHECK_VALUE(k.dim() == 5 && k.size(3) == 2, "k_cache must be [pages, page_size, Hkv, 2, D]");
        TORCH_CHECK_VALUE(v.dim() == 4, "v_cache must be [pages, page_size, Hkv, Dv]");
        TORCH_CHECK_VALUE(k.sizes().slice(0, 3) == v.sizes().slice(0, 3), "k_cache and v_cache disagree on pages, page_size or heads");
        TORCH_CHECK_VALUE(table.dim() == 2, "page_table must be [B, pages of a sequence]");
        for (int64_t n : {k.size(0), k.size(1), k.size(2), k.size(4), v.size(3), table.size(1)})
            TORCH_CHECK_VALUE(n <= INT32_MAX, "a size exceeds 2^31 - 1");
        L = table.size(1) * k.size(1);
    }

    void shapes(int64_t B, const Tensor &tokens) const
    {
        TORCH_CHECK_TYPE(k.scalar_type() == tokens.scalar_type() && v.scalar_type() == tokens.scalar_type(),
                         "the cache must have the new tokens' type");
        TORCH_CHECK_VALUE(table.size(0) == B, "page_table must be [B, pages of a sequence]");
        shaped(&table, "page_table", {B, table.size(1)}, at::kInt);
        shaped(&lengths, "lengths", {B}, at::kInt);
        shaped(counts, "counts", {B}, at::kInt);
    }

    void fill(pg_cache &c, int index) const
    {
        together({&k, &v, &table, &lengths, counts}, index);
        c.num_pages = static_cast<int32_t>(k.size(0));
        c.page_size = static_cast<int32_t>(k.size(1));
        c.table_pages = static_cast<int32_t>(table.size(1));
        c.page_table = data<int32_t>(&table);
        c.lengths = data<int32_t>(&lengths);
        c.counts = data<int32_t>(counts);
        c.k = strided(k, "k_cache");
        c.v = strided(v, "v_cache");
        strides(k, c.k_stride, 4);
        strides(v, c.v_stride, 3);
    }
};

// (the rotary arguments, v, k_cache, v_cache, page_table, lengths, counts, out_q) -> q
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        count(n, kRotary + 7);
        const Tensor &k = needed(a[1], "k"), &v = needed(a[kRotary], "v");
        const Tensor *q = tensor(a[0], "q"), *given = tensor(a[kRotary + 6], "out_q");
        const Cache cache(a + kRotary + 1);
        TORCH_CHECK_VALUE(k.dim() == 5 && v.dim() == 4, "k must be [B, T, Hkv, 2, D] and v [B, T, Hkv, Dv]");
        TORCH_CHECK_VALUE(!q || (q->dim() == 5 && q->sizes().slice(0, 2) == k.sizes().slice(0, 2)), "q and k disagree on batch or tokens");
        TORCH_CHECK_VALUE(v.sizes().slice(0, 3) == k.sizes().slice(0, 3) && v.scalar_type() == k.scalar_type(),
                          "v must be of k's type, [B, T, Hkv, Dv] of k's tokens and heads");
        TORCH_CHECK_VALUE(cache.k.sizes().slice(2) == k.sizes().slice(2) && cache.v.sizes().slice(2) == v.sizes().slice(2),
                          "the cache must hold the new tokens' heads and widths");
        TORCH_CHECK_VALUE(q || !given, "out_q has no input");
        cache.shapes(k.size(0), k);
        Rotary r(a);
        if (given) like(*given, "out_q", *q, q->sizes());
        together({&v, given}, r.index);
        pg_cache c{};
        cache.fill(c, r.index);
        r.fill();
        int64_t vs[3];
        strides(v, vs, 3);
        const void *vp = strided(v, "v");
        Tensor out;
        {
            const On at(k);
            if (q) out = given ? *given : fresh(*q, q->sizes());
            check(g_lib.pg_append_(&r.p, vp, vs, static_cast<int32_t>(v.size(3)), &c, q ? plain(out) : nullptr, at.stream));
        }
        return wrap(out);
    });
}

// q, k_cache, v_cache, page_table, key_lengths, counts, lam, tree, bias_table, bucket_map, pos_q, pos_k, key_mask, causal, scale
constexpr int kAttention = 15;

struct Attention {
    pg_problem p{};
    const Tensor &q;
    int64_t shape[4];  // of the output
    int index;

    Attention(PyObject *const *a, const Tensor *out) : q(needed(a[0], "q"))
    {
        const Cache cache(a + 1);
        const Tensor &lam = needed(a[6], "lam");
        const Tensor *tree = tensor(a[7], "tree"), *bias = tensor(a[8], "bias_table"), *map = tensor(a[9], "bucket_map");
        const Tensor *pq = tensor(a[10], "pos_q"), *pk = tensor(a[11], "pos_k"), *mask = tensor(a[12], "key_mask");
        TORCH_CHECK_VALUE(q.dim() == 5 && q.size(3) == 2, "q must be [B, T, H, 2, D]");
        p.dtype = type_of(q, "q and the cache");
        TORCH_CHECK_VALUE(cache.k.size(4) == q.size(4), "q and k_cache disagree on width");
        TORCH_CHECK_VALUE(!bias == !map, "bias_table and bucket_map go together");
        const int64_t B = q.size(0), T = q.size(1), H = q.size(2), L = cache.L;
        for (int64_t n : {B, T, H}) TORCH_CHECK_VALUE(n <= INT32_MAX, "a size exceeds 2^31 - 1");
        cache.shapes(B, q);
        shaped(&lam, "lam", {H}, at::kFloat);
        shaped(pq, "pos_q", {B, T}, at::kInt);
        shaped(pk, "pos_k", {B, L}, at::kInt);
        shaped(mask, "key_mask", {B, L}, at::kBool);
        shaped(tree, "tree", {B, T, T}, at::kBool);
        if (bias) {
            TORCH_CHECK_VALUE(bias->dim() == 2 && map->dim() == 1 && map->size(0) % 2 == 1 && map->size(0) <= INT32_MAX && bias->size(0) <= INT32_MAX,
                              "bias_table must be [num_buckets, H] and bucket_map [2 * reach + 1]");
            shaped(bias, "bias_table", {bias->size(0), H}, at::kFloat);
            shaped(map, "bucket_map", {map->size(0)}, at::kInt);
            p.num_buckets = static_cast<int32_t>(bias->size(0));
            p.reach = static_cast<int32_t>(map->size(0) / 2);
        }
        shape[0] = B;
        shape[1] = T;
        shape[2] = H;
        shape[3] = cache.v.size(3);
        if (out) like(*out, "out", q, at::IntArrayRef(shape, 4));
        p.batch = static_cast<int32_t>(B);
        p.num_tokens = static_cast<int32_t>(T);
        p.num_heads = static_cast<int32_t>(H);
        p.num_kv_heads = static_cast<int32_t>(cache.k.size(2));
        p.width = static_cast<int32_t>(q.size(4));
        p.value_width = static_cast<int32_t>(cache.v.size(3));
        p.causal = truth(a[13]);
        p.scale = static_cast<float>(a[14] == Py_None ? std::pow(static_cast<double>(q.size(4)), -0.5) : number(a[14]));
        index = static_cast<int>(q.get_device());
        together({&q, &lam, tree, bias, map, pq, pk, mask, out}, index);
        cache.fill(p.cache, index);
        p.bias_table = data<float>(bias);
        p.bucket_map = data<int32_t>(map);
        p.lam = data<float>(&lam);
        p.pos_q = data<int32_t>(pq);
        p.pos_k = data<int32_t>(pk);
        p.key_mask = data<uint8_t>(mask);
        p.tree = data<uint8_t>(tree);
        p.q = strided(q, "q");
        strides(q, p.q_stride, 4);
    }
};

// (the attention's arguments, out) -> out
PyObject *attention(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        count(n, kAttention + 1);
        const Tensor *given = tensor(a[kAttention], "out");
        const Attention r(a, given);
        Tensor out;
        {
            const On at(r.q);
            out = given ? *given : fresh(r.q, at::IntArrayRef(r.shape, 4));
            void *to = plain(out);
            size_t bytes = 0;
            check(g_lib.pg_workspace_size_(&r.p, &bytes));
            const Tensor ws = bytes ? scratch(r.q, bytes) : Tensor();
            check(g_lib.pg_attention_(&r.p, to, bytes ? ws.data_ptr() : nullptr, bytes, at.stream));
        }
        return wrap(out);
    });
}

// (the attention's arguments) -> whether the tensor cores take it
PyObject *path(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        count(n, kAttention);
        const Attention r(a, nullptr);
        size_t bytes = 0;
        check(g_lib.pg_workspace_size_(&r.p, &bytes));  // the status of an invalid problem
        return PyBool_FromLong(g_lib.pg_path_(&r.p) == 1);
    });
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)> PyCFunction fast() { return reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(F)); }

PyMethodDef g_methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    {"rotary_forward", fast<rotary_forward>(), METH_FASTCALL, nullptr},
    {"rotary_backward", fast<rotary_backward>(), METH_FASTCALL, nullptr},
    {"append", fast<append>(), METH_FASTCALL, nullptr},
    {"attention", fast<attention>(), METH_FASTCALL, nullptr},
    {"path", fast<path>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
