// kv4_binding.cpp -- Python module _kv4_binding: the calls of the paged caches (kv4_*,
// kv8_*) and of windowed attention on torch tensors.  It checks tensors, allocates what
// the caller did not give and calls libcp's entry points; it holds no arithmetic.  A
// decode step makes these calls once per layer, and in Python their checks and
// allocations took longer than the kernels (21 us of host time for an attention call of
// 9 us; 11 here).
//
// libcp is not linked: its functions come as addresses (table()), so that the caller
// chooses the build of the library.  Functions return their tensors, or the status
// code of the call where that is not CP_OK.
#include <Python.h>

#include <ATen/Functions.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <limits.h>
#include <string.h>

#include "cp.h"

namespace {

struct Table {
    decltype(&kv4_append) append;
    decltype(&kv4_gather) gather;
    decltype(&kv4_attn) attn;
    decltype(&kv4_attn_workspace) attn_workspace;
    decltype(&kv4_select) select;
    decltype(&kv4_select_workspace) select_workspace;
    decltype(&kv8_append) append8;
    decltype(&kv8_gather) gather8;
    decltype(&kv8_attn) attn8;
    decltype(&kv8_attn_workspace) attn8_workspace;
    decltype(&kv8_evict) evict8;
    decltype(&window_attn_fwd) window_fwd;
    decltype(&window_attn_bwd) window_bwd;
    decltype(&window_attn_bwd_workspace) window_bwd_workspace;
};
constexpr int CALLS = 14;

constexpr const char *TABLE = "libcp.kv4";

// What a call refuses: ends in a ValueError.
struct Refused {
    std::string what;
};

template <typename... T>
[[noreturn]] void refuse(T... parts)
{
    std::ostringstream s;
    (s << ... << parts);
    throw Refused{s.str()};
}

// The positional arguments of one call, in order.
struct Args {
    PyObject *const *at;
    const Table *table;
    int64_t index = 0;   // the call's CUDA device

    Args(PyObject *const *args, Py_ssize_t given, Py_ssize_t wanted) : at(args)
    {
        if (given != wanted) refuse("kv4: ", wanted, " arguments expected, got ", given);
        table = static_cast<const Table *>(PyCapsule_GetPointer(*at++, TABLE));
        if (!table) throw python_error();
    }
    // a tensor, or null for None
    const at::Tensor *tensor(const char *name)
    {
        PyObject *o = *at++;
        if (o == Py_None) return nullptr;
        if (!THPVariable_Check(o)) refuse(name, " must be a tensor");
        return &THPVariable_Unpack(o);
    }
    const at::Tensor &needed(const char *name)
    {
        const at::Tensor *t = tensor(name);
        if (!t) refuse(name, " must be a tensor");
        return *t;
    }
    int64_t integer()
    {
        const long long v = PyLong_AsLongLong(*at++);
        if (v == -1 && PyErr_Occurred()) throw python_error();
        return v;
    }
    int small(const char *name)
    {
        const int64_t v = integer();
        if (v < INT_MIN || v > INT_MAX) refuse(name, " is out of range: ", v);
        return (int)v;
    }
    bool truth()
    {
        const int v = PyObject_IsTrue(*at++);
        if (v < 0) throw python_error();
        return v != 0;
    }
    float number()
    {
        const double v = PyFloat_AsDouble(*at++);
        if (v == -1.0 && PyErr_Occurred()) throw python_error();
        return (float)v;
    }
    void *stream() { return reinterpret_cast<void *>(integer()); }

    void on_device(const char *name, const at::Tensor &t) const
    {
        if (!t.is_cuda() || t.get_device() != index) refuse(name, " must be on CUDA device ", index);
    }
    void check(const char *name, const at::Tensor *t, at::ScalarType type) const
    {
        if (!t) return;
        on_device(name, *t);
        if (t->scalar_type() != type) refuse(name, " must be ", c10::toString(type), ", not ", c10::toString(t->scalar_type()));
        if (!t->is_contiguous()) refuse(name, " must be contiguous");
    }
    void check(const char *name, const at::Tensor *t, at::ScalarType type, at::IntArrayRef shape) const
    {
        if (!t) return;
        check(name, t, type);
        if (t->sizes() != shape) refuse(name, " must have shape ", shape, ", not ", t->sizes());
    }
};

int status(const char *name, int64_t v)
{
    if (v < 0 || v > INT_MAX) refuse(name, " is out of range: ", v);
    return (int)v;
}

struct Pool {
    int n_pages, heads, page, D, max_pages;
};

Pool check_pool(const Args &a, const at::Tensor &cache, const at::Tensor &pages, const at::Tensor &lens, int64_t B)
{
    a.check("cache", &cache, at::kByte);
    if (cache.dim() != 4 || cache.size(3) % 5) refuse("cache must have shape [n_pages, Hkv, page, 5 D / 4], not ", cache.sizes());
    a.check("pages", &pages, at::kInt);
    if (pages.dim() != 2 || pages.size(0) != B) refuse("pages must have shape [", B, ", max_pages], not ", pages.sizes());
    a.check("lens", &lens, at::kInt, {B});
    return {status("n_pages", cache.size(0)), status("Hkv", cache.size(1)), status("page", cache.size(2)),
            status("D", cache.size(3) / 5 * 4), status("max_pages", pages.size(1))};
}

void *ptr(const at::Tensor *t) { return t ? t->data_ptr() : nullptr; }
void *ptr(const at::Tensor &t) { return t.data_ptr(); }
const int32_t *ints(const at::Tensor *t) { return static_cast<const int32_t *>(ptr(t)); }
const int32_t *ints(const at::Tensor &t) { return static_cast<const int32_t *>(ptr(t)); }
const float *floats(const at::Tensor *t) { return static_cast<const float *>(ptr(t)); }

int code_of(at::ScalarType t) { return t == at::kBFloat16 ? CP_BF16 : t == at::kFloat ? CP_F32 : -1; }

// Runs a call of the library without the interpreter's lock.
template <typename F>
int run(F &&f)
{
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = f();
    Py_END_ALLOW_THREADS;
    return rc;
}

// (table, k, v, cache, pages, lens, cos, sin, q, q_out, positions, n_new, summary, interleaved, device, stream)
PyObject *append(PyObject *const *args, Py_ssize_t n_args)
{
    Args a(args, n_args, 16);
    const at::Tensor &k = a.needed("k"), &v = a.needed("v"), &cache = a.needed("cache"), &pages = a.needed("pages"),
                     &lens = a.needed("lens");
    const at::Tensor *cos = a.tensor("cos"), *sin = a.tensor("sin"), *q = a.tensor("q"), *q_out = a.tensor("q_out"),
                     *positions = a.tensor("positions"), *n_new = a.tensor("n_new"), *summary = a.tensor("summary");
    const bool interleaved = a.truth();
    a.index = a.integer();
    void *stream = a.stream();
    if (k.dim() != 4 || v.sizes() != k.sizes()) refuse("k and v must have shape [B, n, Hkv, D]");
    const at::ScalarType type = k.scalar_type();
    if (code_of(type) < 0 || v.scalar_type() != type || (q && q->scalar_type() != type))
        refuse("q, k, v must share dtype float32 or bfloat16");
    const int64_t B = k.size(0), n = k.size(1), H = k.size(2), D = k.size(3);
    const Pool p = check_pool(a, cache, pages, lens, B);
    if (p.heads != H || p.D != D) refuse("cache and k must share Hkv and D");
    if (!cos != !sin || (cos && (cos->dim() != 2 || cos->sizes() != sin->sizes())))
        refuse("cos and sin must share shape [max_pos, rot / 2]");
    a.check("cos", cos, at::kFloat);
    a.check("sin", sin, at::kFloat);
    a.check("positions", positions, at::kInt, {B, n});
    a.check("n_new", n_new, at::kInt, {B});
    a.check("summary", summary, at::kBFloat16, {p.n_pages, H, 2, D});
    if (q && (q->dim() != 4 || q->size(0) != B || q->size(1) != n || q->size(3) != D)) refuse("q must have shape [B, n, Hq, D]");
    if (q_out && !q) refuse("q_out without q");
    if (q) a.check("q_out", q_out, type, q->sizes());
    // rows contiguous; an axis of one entry is not stepped along: its stride says nothing
    int64_t strides[9] = {};
    const char *names[3] = {"k", "v", "q"};
    const at::Tensor *rows[3] = {&k, &v, q};
    for (int i = 0; i < 3; ++i) {
        if (!rows[i]) continue;
        a.on_device(names[i], *rows[i]);
        if (rows[i]->numel() && rows[i]->stride(3) != 1) refuse(names[i], "'s rows must be contiguous");
        for (int x = 0; x < 3; ++x) strides[3 * i + x] = rows[i]->size(x) > 1 ? rows[i]->stride(x) : 0;
    }
    at::Tensor out;
    if (q) out = q_out ? *q_out : at::empty(q->sizes(), q->options());
    const int b = status("B", B), nn = status("n", n), hq = q ? status("Hq", q->size(2)) : 0;
    const int rot = cos ? status("rot", 2 * cos->size(1)) : 0, max_pos = cos ? status("max_pos", cos->size(0)) : 0;
    const int rc = run([&] {
        return a.table->append(ptr(k), ptr(v), ptr(q), q ? ptr(out) : nullptr, ptr(cache), ptr(summary), ints(pages), ints(lens),
                               ints(n_new), ints(positions), floats(cos), floats(sin), strides, b, nn, hq, p.heads, p.D,
                               p.n_pages, p.page, p.max_pages, rot, interleaved, max_pos, code_of(type), stream);
    });
    if (rc) return PyLong_FromLong(rc);
    if (!q) Py_RETURN_NONE;
    return THPVariable_Wrap(out);
}

// (table, cache, pages, lens, count, start, bf16, k, v, device, stream)
PyObject *gather(PyObject *const *args, Py_ssize_t n_args)
{
    Args a(args, n_args, 11);
    const at::Tensor &cache = a.needed("cache"), &pages = a.needed("pages"), &lens = a.needed("lens");
    const int count = a.small("count");
    const at::Tensor *start = a.tensor("start");
    const at::ScalarType type = a.truth() ? at::kBFloat16 : at::kFloat;
    const at::Tensor *k = a.tensor("k"), *v = a.tensor("v");
    a.index = a.integer();
    void *stream = a.stream();
    if (lens.dim() != 1) refuse("lens must have shape [B]");
    if (count < 0) return PyLong_FromLong(CP_EINVAL);
    const int64_t B = lens.size(0);
    const Pool p = check_pool(a, cache, pages, lens, B);
    const int64_t shape[4] = {B, count, p.heads, p.D};
    a.check("start", start, at::kInt, {B});
    a.check("k", k, type, shape);
    a.check("v", v, type, shape);
    const auto options = cache.options().dtype(type);
    const at::Tensor ko = k ? *k : at::empty(shape, options), vo = v ? *v : at::empty(shape, options);
    const int b = status("B", B);
    const int rc = run([&] {
        return a.table->gather(ptr(cache), ints(pages), ints(lens), ints(start), ptr(ko), ptr(vo), b, count, p.heads, p.D,
                               p.n_pages, p.page, p.max_pages, code_of(type), stream);
    });
    if (rc) return PyLong_FromLong(rc);
    return Py_BuildValue("(NN)", THPVariable_Wrap(ko), THPVariable_Wrap(vo));
}

// (table, q, cache, pages, lens, vis, causal, scale, sel, out, lse, workspace, device, stream)
PyObject *attn(PyObject *const *args, Py_ssize_t n_args)
{
    Args a(args, n_args, 14);
    const at::Tensor &q = a.needed("q"), &cache = a.needed("cache"), &pages = a.needed("pages"), &lens = a.needed("lens");
    const at::Tensor *vis = a.tensor("vis");
    const bool causal = a.truth();
    const float scale = a.number();
    const at::Tensor *sel = a.tensor("sel"), *out = a.tensor("out"), *lse = a.tensor("lse"), *ws = a.tensor("workspace");
    a.index = a.integer();
    void *stream = a.stream();
    if (q.dim() != 4) refuse("q must have shape [B, n, Hq, D]");
    a.check("q", &q, at::kBFloat16);
    const int64_t B = q.size(0), n = q.size(1), Hq = q.size(2), D = q.size(3);
    const Pool p = check_pool(a, cache, pages, lens, B);
    if (p.D != D) refuse("cache and q must share D");
    a.check("vis", vis, at::kInt, {B, n});
    if (sel && sel->dim() != 4) refuse("sel must have shape [B, n, Hkv, n_sel]");
    const int n_sel = sel ? status("n_sel", sel->size(3)) : 0;
    if (sel) a.check("sel", sel, at::kInt, {B, n, p.heads, n_sel});
    const at::ScalarType type = out ? out->scalar_type() : at::kBFloat16;
    if (code_of(type) < 0) refuse("out must be float32 or bfloat16");
    a.check("out", out, type, q.sizes());
    a.check("lse", lse, at::kFloat, {B, Hq, n});
    if (ws) a.check("workspace", ws, ws->scalar_type());
    const size_t need = a.table->attn_workspace(p.D);
    const at::Tensor o = out ? *out : at::empty(q.sizes(), q.options());
    const at::Tensor z = lse ? *lse : at::empty({B, Hq, n}, q.options().dtype(at::kFloat));
    const at::Tensor w = ws ? *ws : at::empty({(int64_t)need}, q.options().dtype(at::kByte));
    const int b = status("B", B), nn = status("n", n), hq = status("Hq", Hq);
    const int rc = run([&] {
        return a.table->attn(ptr(q), ptr(cache), ints(pages), ints(lens), ints(vis), ints(sel), ptr(o),
                             static_cast<float *>(ptr(z)), b, nn, hq, p.heads, p.D, p.n_pages, p.page, p.max_pages, n_sel,
                             causal, code_of(type), scale, ptr(w), w.nbytes(), stream);
    });
    if (rc) return PyLong_FromLong(rc);
    return Py_BuildValue("(NN)", THPVariable_Wrap(o), THPVariable_Wrap(z));
}

// (table, q, summary, pages, lens, page, n_sel, vis, causal, keep_first, keep_last, sel, workspace, device, stream)
PyObject *select(PyObject *const *args, Py_ssize_t n_args)
{
    Args a(args, n_args, 15);
    const at::Tensor &q = a.needed("q"), &summary = a.needed("summary"), &pages = a.needed("pages"), &lens = a.needed("lens");
    const int page = a.small("page"), n_sel = a.small("n_sel");
    const at::Tensor *vis = a.tensor("vis");
    const bool causal = a.truth();
    const int first = a.small("keep_first"), last = a.small("keep_last");
    const at::Tensor *sel = a.tensor("sel"), *ws = a.tensor("workspace");
    a.index = a.integer();
    void *stream = a.stream();
    if (q.dim() != 4 || summary.dim() != 4) refuse("q must have shape [B, n, Hq, D] and summary [n_pages, Hkv, 2, D]");
    a.check("q", &q, at::kBFloat16);
    const int64_t B = q.size(0), n = q.size(1), Hq = q.size(2), D = q.size(3), P = summary.size(0), H = summary.size(1);
    a.check("summary", &summary, at::kBFloat16, {P, H, 2, D});
    a.check("pages", &pages, at::kInt);
    if (pages.dim() != 2 || pages.size(0) != B) refuse("pages must have shape [", B, ", max_pages], not ", pages.sizes());
    a.check("lens", &lens, at::kInt, {B});
    a.check("vis", vis, at::kInt, {B, n});
    if (n_sel < 1) return PyLong_FromLong(CP_EINVAL);
    const int64_t shape[4] = {B, n, H, n_sel};
    a.check("sel", sel, at::kInt, shape);
    if (ws) a.check("workspace", ws, ws->scalar_type());
    const int b = status("B", B), nn = status("n", n), hq = status("Hq", Hq), h = status("Hkv", H), d = status("D", D),
              np = status("n_pages", P), m = status("max_pages", pages.size(1));
    const at::Tensor s = sel ? *sel : at::empty(shape, pages.options());
    const at::Tensor w =
        ws ? *ws : at::empty({(int64_t)a.table->select_workspace(b, nn, h, m)}, q.options().dtype(at::kByte));
    const int rc = run([&] {
        return a.table->select(ptr(q), ptr(summary), ints(pages), ints(lens), ints(vis), static_cast<int32_t *>(ptr(s)), b, nn,
                               hq, h, d, np, page, m, n_sel, causal, first, last, ptr(w), w.nbytes(), stream);
    });
    if (rc) return PyLong_FromLong(rc);
    return THPVariable_Wrap(s);
}

Pool check_pool8(const Args &a, const at::Tensor &cache, const at::Tensor &scales, const at::Tensor &pages,
                 const at::Tensor &lens, int64_t B)
{
    a.check("cache", &cache, at::kByte);
    if (cache.dim() != 5 || cache.size(2) != 2) refuse("cache must have shape [n_pages, Hkv, 2, page, D], not ", cache.sizes());
    a.check("scales", &scales, at::kFloat, {cache.size(0), cache.size(1), 2, cache.size(3) / 16});
    a.check("pages", &pages, at::kInt);
    if (pages.dim() != 2 || pages.size(0) != B) refuse("pages must have shape [", B, ", max_pages], not ", pages.sizes());
    a.check("lens", &lens, at::kInt, {B});
    return {status("n_pages", cache.size(0)), status("Hkv", cache.size(1)), status("page", cache.size(3)),
            status("D", cache.size(4)), status("max_pages", pages.size(1))};
}

// Element strides of [B, n, H, D] rows; an axis of one entry is not stepped along.
void row_strides(const Args &a, const char *name, const at::Tensor &t, int64_t *strides)
{
    a.on_device(name, t);
    if (t.numel() && t.stride(3) != 1) refuse(name, "'s rows must be contiguous");
    for (int x = 0; x < 3; ++x) strides[x] = t.size(x) > 1 ? t.stride(x) : 0;
}

// (table, k, v, cache, scales, pages, lens, n_new, device, stream)
PyObject *append8(PyObject *const *args, Py_ssize_t n_args)
{
    Args a(args, n_args, 10);
    const at::Tensor &k = a.needed("k"), &v = a.needed("v"), &cache = a.needed("cache"), &scales = a.needed("scales"),
                     &pages = a.needed("pages"), &lens = a.needed("lens");
    const at::Tensor *n_new = a.tensor("n_new");
    a.index = a.integer();
    void *stream = a.stream();
    if (k.dim() != 4 || v.sizes() != k.sizes()) refuse("k and v must have shape [B, n, Hkv, D]");
    const at::ScalarType type = k.scalar_type();
    if (code_of(type) < 0 || v.scalar_type() != type) refuse("k and v must share dtype float32 or bfloat16");
    const int64_t B = k.size(0);
    const Pool p = check_pool8(a, cache, scales, pages, lens, B);
    if (p.heads != k.size(2) || p.D != k.size(3)) refuse("cache and k must share Hkv and D");
    a.check("n_new", n_new, at::kInt, {B});
    int64_t strides[6];
    row_strides(a, "k", k, strides);
    row_strides(a, "v", v, strides + 3);
    const int b = status("B", B), n = status("n", k.size(1));
    const int rc = run([&] {
        return a.table->append8(ptr(k), ptr(v), ptr(cache), static_cast<float *>(ptr(scales)), ints(pages), ints(lens),
                                ints(n_new), strides, b, n, p.heads, p.D, p.n_pages, p.page, p.max_pages, code_of(type), stream);
    });
    if (rc) return PyLong_FromLong(rc);
    Py_RETURN_NONE;
}

// (table, cache, scales, pages, lens, count, start, bf16, k, v, device, stream)
PyObject *gather8(PyObject *const *args, Py_ssize_t n_args)
{
    Args a(args, n_args, 12);
    const at::Tensor &cache = a.needed("cache"), &scales = a.needed("scales"), &pages = a.needed("pages"), &lens = a.needed("lens");
    const int count = a.small("count");
    const at::Tensor *start = a.tensor("start");
    const at::ScalarType type = a.truth() ? at::kBFloat16 : at::kFloat;
    const at::Tensor *k = a.tensor("k"), *v = a.tensor("v");
    a.index = a.integer();
    void *stream = a.stream();
    if (lens.dim() != 1) refuse("lens must have shape [B]");
    if (count < 0) return PyLong_FromLong(CP_EINVAL);
    const int64_t B = lens.size(0);
    const Pool p = check_pool8(a, cache, scales, pages, lens, B);
    const int64_t shape[4] = {B, count, p.heads, p.D};
    a.check("start", start, at::kInt, {B});
    a.check("k", k, type, shape);
    a.check("v", v, type, shape);
    const auto options = cache.options().dtype(type);
    const at::Tensor ko = k ? *k : at::empty(shape, options), vo = v ? *v : at::empty(shape, options);
    const int b = status("B", B);
    const int rc = run([&] {
        return a.table->gather8(ptr(cache), floats(&scales), ints(pages), ints(lens), ints(start), ptr(ko), ptr(vo), b, count,
                                p.heads, p.D, p.n_pages, p.page, p.max_pages, code_of(type), stream);
    });
    if (rc) return PyLong_FromLong(rc);
    return Py_BuildValue("(NN)", THPVariable_Wrap(ko), THPVariable_Wrap(vo));
}

// (table, q, cache, scales, pages, lens, window, sinks, vis, causal, scale, mass, out, lse, workspace, device, stream)
PyObject *attn8(PyObject *const *args, Py_ssize_t n_args)
{
    Args a(args, n_args, 17);
    const at::Tensor &q = a.needed("q"), &cache = a.needed("cache"), &scales = a.needed("scales"), &pages = a.needed("pages"),
                     &lens = a.needed("lens");
    const int64_t window = a.integer(), sinks = a.integer();
    const at::Tensor *vis = a.tensor("vis");
    const bool causal = a.truth();
    const float scale = a.number();
    const at::Tensor *mass = a.tensor("mass"), *out = a.tensor("out"), *lse = a.tensor("lse"), *ws = a.tensor("workspace");
    a.index = a.integer();
    void *stream = a.stream();
    if (q.dim() != 4) refuse("q must have shape [B, n, Hq, D]");
    a.check("q", &q, at::kBFloat16);
    const int64_t B = q.size(0), n = q.size(1), Hq = q.size(2), D = q.size(3);
    const Pool p = check_pool8(a, cache, scales, pages, lens, B);
    if (p.D != D) refuse("cache and q must share D");
    a.check("vis", vis, at::kInt, {B, n});
    a.check("mass", mass, at::kFloat, {B, p.heads, (int64_t)p.max_pages * p.page});
    const at::ScalarType type = out ? out->scalar_type() : at::kBFloat16;
    if (code_of(type) < 0) refuse("out must be float32 or bfloat16");
    a.check("out", out, type, q.sizes());
    a.check("lse", lse, at::kFloat, {B, Hq, n});
    if (ws) a.check("workspace", ws, ws->scalar_type());
    const int b = status("B", B), nn = status("n", n), hq = status("Hq", Hq);
    const at::Tensor o = out ? *out : at::empty(q.sizes(), q.options());
    const at::Tensor z = lse ? *lse : at::empty({B, Hq, n}, q.options().dtype(at::kFloat));
    const at::Tensor w = ws ? *ws
                            : at::empty({(int64_t)a.table->attn8_workspace(b, nn, hq, p.heads, p.D, p.page, p.max_pages, mass != nullptr)},
                                        q.options().dtype(at::kByte));
    const int rc = run([&] {
        return a.table->attn8(ptr(q), ptr(cache), floats(&scales), ints(pages), ints(lens), ints(vis), ptr(o),
                              static_cast<float *>(ptr(z)), static_cast<float *>(ptr(mass)), b, nn, hq, p.heads, p.D, p.n_pages,
                              p.page, p.max_pages, window, sinks, causal, code_of(type), scale, ptr(w), w.nbytes(), stream);
    });
    if (rc) return PyLong_FromLong(rc);
    return Py_BuildValue("(NN)", THPVariable_Wrap(o), THPVariable_Wrap(z));
}

// (table, cache, scales, pages, lens, mass, pages_to, budget, keep_first, keep_last, kept, lens_to, mass_to, device, stream)
PyObject *evict8(PyObject *const *args, Py_ssize_t n_args)
{
    Args a(args, n_args, 15);
    const at::Tensor &cache = a.needed("cache"), &scales = a.needed("scales"), &pages = a.needed("pages"), &lens = a.needed("lens"),
                     &mass = a.needed("mass"), &to = a.needed("pages_to");
    const int budget = a.small("budget"), first = a.small("keep_first"), last = a.small("keep_last");
    const at::Tensor *kept = a.tensor("kept"), *lens_to = a.tensor("lens_to"), *mass_to = a.tensor("mass_to");
    a.index = a.integer();
    void *stream = a.stream();
    if (lens.dim() != 1) refuse("lens must have shape [B]");
    const int64_t B = lens.size(0);
    const Pool p = check_pool8(a, cache, scales, pages, lens, B);
    a.check("mass", &mass, at::kFloat, {B, p.heads, (int64_t)p.max_pages * p.page});
    a.check("pages_to", &to, at::kInt);
    if (to.dim() != 2 || to.size(0) != B) refuse("pages_to must have shape [", B, ", max_to], not ", to.sizes());
    const int max_to = status("max_to", to.size(1));
    if (budget < 1 || budget > (int64_t)max_to * p.page) return PyLong_FromLong(CP_EINVAL);   // before kept is made
    a.check("kept", kept, at::kInt, {B, p.heads, budget});
    a.check("lens_to", lens_to, at::kInt, {B});
    const int64_t slots[3] = {B, p.heads, (int64_t)max_to * p.page};
    a.check("mass_to", mass_to, at::kFloat, slots);
    const at::Tensor k = kept ? *kept : at::empty({B, p.heads, budget}, lens.options());
    const at::Tensor l = lens_to ? *lens_to : at::empty({B}, lens.options());
    const at::Tensor m = mass_to ? *mass_to : at::empty(slots, mass.options());
    const int b = status("B", B);
    const int rc = run([&] {
        return a.table->evict8(ptr(cache), static_cast<float *>(ptr(scales)), ints(pages), ints(lens), floats(&mass), ints(to),
                               static_cast<int32_t *>(ptr(k)), static_cast<int32_t *>(ptr(l)), static_cast<float *>(ptr(m)), b,
                               p.heads, p.D, p.n_pages, p.page, p.max_pages, max_to, budget, first, last, stream);
    });
    if (rc) return PyLong_FromLong(rc);
    return Py_BuildValue("(NNN)", THPVariable_Wrap(k), THPVariable_Wrap(l), THPVariable_Wrap(m));
}

// What the windowed calls are given: q, k, v.
struct Window {
    int B, Hq, Hkv, D, type;
    int64_t Sq, Sk;
    Window(const Args &a, const at::Tensor &q, const at::Tensor &k, const at::Tensor &v)
    {
        if (q.dim() != 4 || k.dim() != 4) refuse("q and k must have shape [B, S, H, D]");
        const at::ScalarType t = q.scalar_type();
        type = code_of(t);
        if (type < 0 || k.scalar_type() != t || v.scalar_type() != t) refuse("q, k, v must share dtype float32 or bfloat16");
        a.check("q", &q, t);
        a.check("k", &k, t, {q.size(0), k.size(1), k.size(2), q.size(3)});
        a.check("v", &v, t, k.sizes());
        B = status("B", q.size(0)), Hq = status("Hq", q.size(2)), Hkv = status("Hkv", k.size(2)), D = status("D", q.size(3));
        Sq = q.size(1), Sk = k.size(1);
    }
};

// (table, q, k, v, window, sinks, scale, out, lse, device, stream)
PyObject *window_fwd(PyObject *const *args, Py_ssize_t n_args)
{
    Args a(args, n_args, 11);
    const at::Tensor &q = a.needed("q"), &k = a.needed("k"), &v = a.needed("v");
    const int64_t window = a.integer(), sinks = a.integer();
    const float scale = a.number();
    const at::Tensor *out = a.tensor("out"), *lse = a.tensor("lse");
    a.index = a.integer();
    void *stream = a.stream();
    const Window w(a, q, k, v);
    a.check("out", out, q.scalar_type(), q.sizes());
    a.check("lse", lse, at::kFloat, {w.B, w.Hq, w.Sq});
    const at::Tensor o = out ? *out : at::empty(q.sizes(), q.options());
    const at::Tensor z = lse ? *lse : at::empty({w.B, w.Hq, w.Sq}, q.options().dtype(at::kFloat));
    const int rc = run([&] {
        return a.table->window_fwd(ptr(q), ptr(k), ptr(v), ptr(o), static_cast<float *>(ptr(z)), w.B, w.Hq, w.Hkv, w.Sq, w.Sk,
                                   w.D, window, sinks, w.type, scale, stream);
    });
    if (rc) return PyLong_FromLong(rc);
    return Py_BuildValue("(NN)", THPVariable_Wrap(o), THPVariable_Wrap(z));
}

// (table, q, k, v, out, lse, dout, window, sinks, scale, dq, dk, dv, workspace, device, stream)
PyObject *window_bwd(PyObject *const *args, Py_ssize_t n_args)
{
    Args a(args, n_args, 16);
    const at::Tensor &q = a.needed("q"), &k = a.needed("k"), &v = a.needed("v"), &out = a.needed("out"), &lse = a.needed("lse"),
                     &dout = a.needed("dout");
    const int64_t window = a.integer(), sinks = a.integer();
    const float scale = a.number();
    const at::Tensor *dq = a.tensor("dq"), *dk = a.tensor("dk"), *dv = a.tensor("dv"), *ws = a.tensor("workspace");
    a.index = a.integer();
    void *stream = a.stream();
    const Window w(a, q, k, v);
    const at::ScalarType t = q.scalar_type();
    a.check("out", &out, t, q.sizes());
    a.check("dout", &dout, t, q.sizes());
    a.check("lse", &lse, at::kFloat, {w.B, w.Hq, w.Sq});
    a.check("dq", dq, t, q.sizes());
    a.check("dk", dk, t, k.sizes());
    a.check("dv", dv, t, k.sizes());
    if (ws) a.check("workspace", ws, ws->scalar_type());
    const at::Tensor x = dq ? *dq : at::empty(q.sizes(), q.options()), y = dk ? *dk : at::empty(k.sizes(), k.options()),
                     z = dv ? *dv : at::empty(k.sizes(), k.options());
    const at::Tensor s = ws ? *ws
                            : at::empty({(int64_t)a.table->window_bwd_workspace(w.B, w.Hq, w.Hkv, w.Sq, w.Sk, w.D, window, sinks,
                                                                                w.type)},
                                        q.options().dtype(at::kByte));
    const int rc = run([&] {
        return a.table->window_bwd(ptr(q), ptr(k), ptr(v), ptr(out), floats(&lse), ptr(dout), ptr(x), ptr(y), ptr(z), w.B, w.Hq,
                                   w.Hkv, w.Sq, w.Sk, w.D, window, sinks, w.type, scale, ptr(s), s.nbytes(), stream);
    });
    if (rc) return PyLong_FromLong(rc);
    return Py_BuildValue("(NNN)", THPVariable_Wrap(x), THPVariable_Wrap(y), THPVariable_Wrap(z));
}

// The calls' addresses in libcp, in Table's order
PyObject *table(PyObject *const *args, Py_ssize_t n_args)
{
    if (n_args != CALLS) refuse("kv4: ", CALLS, " addresses expected");
    void *f[CALLS];
    for (int i = 0; i < CALLS; ++i) {
        f[i] = PyLong_AsVoidPtr(args[i]);
        if (!f[i]) {
            if (PyErr_Occurred()) throw python_error();
            refuse("kv4: null address");
        }
    }
    Table *t = new Table;
    static_assert(sizeof(Table) == sizeof(f), "Table holds the addresses and nothing else");
    memcpy(static_cast<void *>(t), f, sizeof(f));
    return PyCapsule_New(t, TABLE, [](PyObject *c) { delete static_cast<Table *>(PyCapsule_GetPointer(c, TABLE)); });
}

// C++ exceptions end here: a refusal is a ValueError, torch's errors are its own.
template <PyObject *(*F)(PyObject *const *, Py_ssize_t)>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    try {
        return F(args, n);
    } catch (const Refused &r) {
        PyErr_SetString(PyExc_ValueError, r.what.c_str());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

#define CP_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&entry<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CP_METHOD(append), CP_METHOD(gather), CP_METHOD(attn), CP_METHOD(select), CP_METHOD(append8),
                         CP_METHOD(gather8), CP_METHOD(attn8), CP_METHOD(evict8), CP_METHOD(window_fwd), CP_METHOD(window_bwd), CP_METHOD(table),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kv4_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kv4_binding(void) { return PyModule_Create(&module); }
