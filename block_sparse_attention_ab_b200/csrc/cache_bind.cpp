// cache_bind.cpp -- Python binding of the ab_cache_* calls (module _cache_bind). A decoding
// step is a few kernels of some microseconds each, and checking and marshalling their
// arguments from Python through ctypes took longer than they run (16 us for ab_cache_append
// of 32 tokens, 31 us for ab_cache_attn of one token), so this binding is compiled: it checks
// types, devices and shapes, allocates outputs and workspaces through torch's allocator on
// the current stream, and calls the C ABI. It holds no state beside the handles' tensors, whose
// addresses and shapes are read anew in every call.
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/extension.h>

#include <optional>
#include <string>

#include "../../include/ab_attn.h"

namespace py = pybind11;
using at::Tensor;
using OptTensor = std::optional<Tensor>;

namespace {

py::object g_error;  // the package's AbError(code, where)

void check(ab_status s, const char *where)
{
    if (s == AB_OK) return;
    py::object e = g_error((int)s, where);
    PyErr_SetObject((PyObject *)Py_TYPE(e.ptr()), e.ptr());
    throw py::error_already_set();
}

[[noreturn]] void bad_type(const std::string &m) { throw py::type_error(m); }
[[noreturn]] void bad_value(const std::string &m) { throw py::value_error(m); }

std::string shape_of(at::IntArrayRef s)
{
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + ")";
}

// A contiguous tensor of the given type and shape on `dev`.
void *array(const Tensor &t, at::ScalarType type, at::IntArrayRef shape, at::Device dev, const char *name)
{
    if (t.scalar_type() != type) bad_type(std::string(name) + " must be " + toString(type));
    if (t.device() != dev) bad_value(std::string(name) + " must be on " + dev.str());
    if (t.sizes() != shape)
        bad_value(std::string(name) + " must be " + shape_of(shape) + ", got " + shape_of(t.sizes()));
    if (!t.is_contiguous()) bad_value(std::string(name) + " must be contiguous");
    return t.data_ptr();
}

void *array(const OptTensor &t, at::ScalarType type, at::IntArrayRef shape, at::Device dev, const char *name)
{
    return t ? array(*t, type, shape, dev, name) : nullptr;
}

struct Cache {
    Tensor k, v, table, length;
    OptTensor ksum, mass, pos;
    ab_cache c{};
    at::Device dev = at::kCUDA;
    at::ScalarType type;

    Cache(Tensor k_, Tensor v_, Tensor table_, Tensor length_, OptTensor ksum_, OptTensor mass_, OptTensor pos_)
        : k(k_), v(v_), table(table_), length(length_), ksum(ksum_), mass(mass_), pos(pos_)
    {
        read();
    }

    // Check the tensors and take their addresses: at every call, because a tensor may have been set
    // to other memory since the last one (an emptied and refilled storage, set_, .data).
    void read()
    {
        for (const Tensor *t : {&k, &v}) {
            const char *n = t == &k ? "k" : "v";
            if (!t->is_cuda()) bad_type(std::string(n) + " must be a CUDA tensor");
            if (t->scalar_type() != at::kBFloat16 && t->scalar_type() != at::kHalf)
                bad_type(std::string(n) + " must be bfloat16 or float16");
            if (t->dim() != 4 || t->stride(3) != 1)
                bad_value(std::string(n) + " must be [n_pages, Hk, page, d] with contiguous rows");
        }
        if (v.scalar_type() != k.scalar_type() || v.sizes() != k.sizes() || v.device() != k.device())
            bad_value("k and v must have one shape, type and device");
        if (table.dim() != 2) bad_value("table must be [B, max_pages]");
        dev = k.device();
        type = k.scalar_type();
        for (int i = 0; i < 4; ++i)
            if (k.size(i) > INT32_MAX || (i < 2 && table.size(i) > INT32_MAX)) bad_value("a dimension is too large");
        c.n_pages = k.size(0);
        c.Hk = k.size(1);
        c.page = k.size(2);
        c.d = k.size(3);
        c.B = table.size(0);
        c.max_pages = table.size(1);
        c.dtype = type == at::kHalf ? AB_F16 : AB_BF16;
        c.k = k.data_ptr();
        c.v = v.data_ptr();
        c.ksum = (float *)array(ksum, at::kFloat, {c.n_pages, c.Hk, c.d}, dev, "ksum");
        c.mass = (float *)array(mass, at::kFloat, {c.n_pages, c.Hk, c.page}, dev, "mass");
        c.pos = (int32_t *)array(pos, at::kInt, {c.n_pages, c.Hk, c.page}, dev, "pos");
        c.table = (const int32_t *)array(table, at::kInt, {c.B, c.max_pages}, dev, "table");
        c.length = (int32_t *)array(length, at::kInt, {c.B}, dev, "length");
        // the stride of a dimension of one element is never used
        auto st = [](const Tensor &t, int i) { return t.size(i) > 1 ? t.stride(i) : 0; };
        c.k_page = st(k, 0), c.k_head = st(k, 1), c.k_row = st(k, 2);
        c.v_page = st(v, 0), c.v_head = st(v, 1), c.v_row = st(v, 2);
    }

    const int32_t *per_seq(const OptTensor &t, const char *name) const
    {
        return (const int32_t *)array(t, at::kInt, {c.B}, dev, name);
    }
    int *flag(const OptTensor &t) const { return (int *)array(t, at::kInt, {1}, dev, "dev_flag"); }

    // [B, heads, T, d]; heads < 0: any
    ab_tokens tokens(const Tensor &t, int64_t heads, const char *name) const
    {
        if (t.scalar_type() != type) bad_type(std::string(name) + " must be " + toString(type));
        if (t.device() != dev) bad_value(std::string(name) + " must be on " + dev.str());
        if (t.dim() != 4 || t.size(0) != c.B || t.size(3) != c.d || (heads >= 0 && t.size(1) != heads))
            bad_value(std::string(name) + " must be [" + std::to_string(c.B) + ", " +
                      (heads < 0 ? "Hq" : std::to_string(heads)) + ", T, " + std::to_string(c.d) + "], got " +
                      shape_of(t.sizes()));
        if (t.size(1) > INT32_MAX || t.size(2) > INT32_MAX)  // the C ABI's counts have 32 bits
            bad_value(std::string(name) + " has too many heads or tokens");
        if (t.stride(3) != 1) bad_value(std::string(name) + ": rows must be contiguous");
        auto st = [&](int i) { return t.size(i) > 1 ? t.stride(i) : (int64_t)0; };
        return {t.data_ptr(), st(0), st(1), st(2)};
    }

    // The current stream of the cache's device, made current for the call.
    struct On {
        c10::cuda::CUDAGuard guard;
        void *stream;
        explicit On(at::Device d) : guard(d), stream(c10::cuda::getCurrentCUDAStream(d.index()).stream()) {}
    };
    Tensor empty(at::IntArrayRef shape, at::ScalarType t) const
    {
        return at::empty(shape, at::TensorOptions().dtype(t).device(dev));
    }
};

struct Plan {
    const int32_t *idx = nullptr, *cnt = nullptr;
    const float *w = nullptr;
    int per_token = 0;
};

Plan plan_of(const Cache &x, int64_t T, const OptTensor &idx, const OptTensor &cnt, const OptTensor &w)
{
    Plan p;
    if (!idx) {
        if (cnt || w) bad_value("cnt and w go with idx");
        return p;
    }
    if (!cnt) bad_value("idx needs cnt");
    const int64_t Tp = idx->dim() == 4 ? idx->size(2) : -1;
    if (Tp != 1 && Tp != T) bad_value("idx must have 1 or " + std::to_string(T) + " rows per key head");
    const auto &c = x.c;
    p.idx = (const int32_t *)array(idx, at::kInt, {c.B, c.Hk, Tp, c.max_pages}, x.dev, "idx");
    p.cnt = (const int32_t *)array(cnt, at::kInt, {c.B, c.Hk, Tp}, x.dev, "cnt");
    p.w = (const float *)array(w, at::kFloat, {c.B, c.Hk, Tp, c.max_pages}, x.dev, "w");
    p.per_token = Tp == T;
    return p;
}

void append(Cache &x, const Tensor &k, const Tensor &v, const OptTensor &n_new, const OptTensor &sel,
            const OptTensor &start, const OptTensor &pos, const OptTensor &dev_flag)
{
    x.read();
    const ab_tokens tk = x.tokens(k, x.c.Hk, "k"), tv = x.tokens(v, x.c.Hk, "v");
    if (v.size(2) != k.size(2)) bad_value("k and v must have one shape");
    const int T = (int)k.size(2);
    Cache::On on(x.dev);
    check(ab_cache_append(x.c, tk, tv, T, x.per_seq(n_new, "n_new"),
                          (const int32_t *)array(sel, at::kInt, {x.c.B, T}, x.dev, "sel"), x.per_seq(start, "start"),
                          x.per_seq(pos, "pos"), x.flag(dev_flag), on.stream),
          "ab_cache_append");
}

Tensor score(Cache &x, const Tensor &q, const OptTensor &n_tok, bool per_token, int first, int recent,
             const OptTensor &out, const OptTensor &dev_flag)
{
    x.read();
    const ab_tokens tq = x.tokens(q, -1, "q");
    Cache::On on(x.dev);
    const int64_t T = q.size(2);
    const std::array<int64_t, 4> shape = {x.c.B, x.c.Hk, per_token ? T : 1, x.c.max_pages};
    Tensor o = out ? *out : x.empty(shape, at::kFloat);
    check(ab_cache_score(x.c, tq, (int)q.size(1), (int)T, x.per_seq(n_tok, "n_tok"), per_token, first, recent,
                         (float *)array(o, at::kFloat, shape, x.dev, "out"), x.flag(dev_flag), on.stream),
          "ab_cache_score");
    return o;
}

size_t workspace_size(const Cache &x, int Hq, int T, bool per_token)
{
    size_t n = 0;
    check(ab_cache_attn_workspace_size(x.c, Hq, T, per_token, &n), "ab_cache_attn_workspace_size");
    return n;
}

size_t attn_workspace(Cache &x, int Hq, int T, bool per_token)
{
    x.read();
    return workspace_size(x, Hq, T, per_token);
}

py::object attn(Cache &x, const Tensor &q, const OptTensor &k, const OptTensor &v, const OptTensor &n_tok,
                const OptTensor &tree, const OptTensor &idx, const OptTensor &cnt, const OptTensor &w, bool want_lse,
                const OptTensor &out, const std::optional<at::ScalarType> &out_type, const OptTensor &workspace,
                const OptTensor &dev_flag)
{
    x.read();
    const ab_tokens tq = x.tokens(q, -1, "q");
    const int64_t B = x.c.B, Hq = q.size(1), T = q.size(2), d = x.c.d;
    if (!k != !v) bad_value("k and v go together");
    ab_tokens tk{}, tv{};
    if (k) {
        tk = x.tokens(*k, x.c.Hk, "k");
        tv = x.tokens(*v, x.c.Hk, "v");
        if (k->size(2) != T || v->size(2) != T) bad_value("q, k and v must have the same number of tokens");
    }
    const Plan p = plan_of(x, T, idx, cnt, w);
    const at::ScalarType ot = out_type ? *out_type : out ? out->scalar_type() : x.type;
    if (ot != x.type && ot != at::kFloat) bad_type("out_dtype must be the cache's type or torch.float32");
    Cache::On on(x.dev);
    Tensor o = out ? *out : x.empty({B, Hq, T, d}, ot);
    void *po = array(o, ot, {B, Hq, T, d}, x.dev, "out");
    Tensor lse;
    if (want_lse) lse = x.empty({B, Hq, T}, at::kFloat);
    const void *pt = array(tree, at::kBool, {B, T, T}, x.dev, "tree");
    Tensor ws = workspace ? *workspace
                          : x.empty({(int64_t)workspace_size(x, (int)Hq, (int)T, p.per_token)}, at::kByte);
    array(ws, at::kByte, ws.sizes(), x.dev, "workspace");
    check(ab_cache_attn(x.c, tq, tk, tv, (int)Hq, (int)T, x.per_seq(n_tok, "n_tok"), (const uint8_t *)pt, p.idx,
                        p.cnt, p.w, p.per_token, po, ot == at::kFloat ? AB_F32 : (ab_dtype)x.c.dtype,
                        want_lse ? lse.data_ptr<float>() : nullptr, ws.data_ptr(), (size_t)ws.numel(),
                        x.flag(dev_flag), on.stream),
          "ab_cache_attn");
    if (want_lse) return py::make_tuple(o, lse);
    return py::cast(o);
}

Tensor mass(Cache &x, const Tensor &q, const Tensor &lse, const OptTensor &n_tok, const OptTensor &sel,
            const OptTensor &idx, const OptTensor &cnt, const OptTensor &w, const OptTensor &out,
            const OptTensor &dev_flag)
{
    x.read();
    const ab_tokens tq = x.tokens(q, -1, "q");
    if (!x.mass) bad_value("the cache has no mass");
    const int64_t B = x.c.B, Hq = q.size(1), T = q.size(2);
    const Plan p = plan_of(x, T, idx, cnt, w);
    Cache::On on(x.dev);
    check(ab_cache_mass(x.c, tq, (int)Hq, (int)T, x.per_seq(n_tok, "n_tok"),
                        (const int32_t *)array(sel, at::kInt, {B, T}, x.dev, "sel"),
                        (const float *)array(lse, at::kFloat, {B, Hq, T}, x.dev, "lse"), p.idx, p.cnt, p.w,
                        p.per_token, (float *)array(out, at::kFloat, x.mass->sizes(), x.dev, "out"),
                        x.flag(dev_flag), on.stream),
          "ab_cache_mass");
    return out ? *out : *x.mass;
}

py::tuple keep(Cache &x, int64_t budget, int64_t recent, const OptTensor &next_pos, const OptTensor &score,
               const OptTensor &pos, const OptTensor &length, const OptTensor &workspace, const OptTensor &dev_flag)
{
    x.read();
    // before they are cut to the 32 bits of the C ABI: src is allocated from the whole budget
    if (budget < 1 || budget > INT32_MAX) bad_value("budget must be 1 .. 2^31 - 1");
    if (recent < 0 || recent > INT32_MAX) bad_value("recent must be 0 .. 2^31 - 1");
    const int64_t B = x.c.B, Hk = x.c.Hk;
    const std::array<int64_t, 3> slots = {x.c.n_pages, Hk, x.c.page};
    Cache::On on(x.dev);
    Tensor src = x.empty({B, Hk, budget}, at::kInt), n = x.empty({B}, at::kInt);
    size_t need = 0;
    check(ab_cache_keep_workspace_size(x.c, (int)budget, &need), "ab_cache_keep");
    Tensor ws = workspace ? *workspace : x.empty({(int64_t)need}, at::kByte);
    array(ws, at::kByte, ws.sizes(), x.dev, "workspace");
    check(ab_cache_keep(x.c, (int)budget, (int)recent, x.per_seq(next_pos, "next_pos"),
                        (const float *)array(score, at::kFloat, slots, x.dev, "score"),
                        (const int32_t *)array(pos, at::kInt, slots, x.dev, "pos"), x.per_seq(length, "length"),
                        src.data_ptr<int32_t>(), n.data_ptr<int32_t>(), ws.data_ptr(), (size_t)ws.numel(),
                        x.flag(dev_flag), on.stream),
          "ab_cache_keep");
    return py::make_tuple(src, n);
}

void compact(Cache &x, const Tensor &src, const Tensor &n_keep, const OptTensor &dev_flag)
{
    x.read();
    if (src.dim() != 3 || src.size(2) > INT32_MAX) bad_value("src must be [B, Hk, budget]");
    Cache::On on(x.dev);
    check(ab_cache_compact(x.c, (int)src.size(2),
                           (const int32_t *)array(src, at::kInt, {x.c.B, x.c.Hk, src.size(2)}, x.dev, "src"),
                           x.per_seq(n_keep, "n_keep"), x.flag(dev_flag), on.stream),
          "ab_cache_compact");
}

}  // namespace

PYBIND11_MODULE(_cache_bind, m)
{
    m.def("set_error", [](py::object e) { g_error = std::move(e); });
    py::class_<Cache>(m, "Cache")
        .def(py::init<Tensor, Tensor, Tensor, Tensor, OptTensor, OptTensor, OptTensor>())
        .def("append", &append)
        .def("score", &score)
        .def("attn_workspace", &attn_workspace)
        .def("attn", &attn)
        .def("mass", &mass)
        .def("keep", &keep)
        .def("compact", &compact);
    // the class must not outlive the interpreter's error type
    m.add_object("_cleanup", py::capsule([]() { g_error.release(); }));
}
