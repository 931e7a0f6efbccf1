// kvq_binding.cpp -- argument marshalling of the block-scaled, windowed and
// page-copy calls: torch tensors in, the C ABI's pointers out.
//
// These calls take up to sixteen tensors and run for a few microseconds on the
// GPU when a batch is small; checked tensor by tensor in Python they cost 15
// to 90 us on the host, here 2.6 to 5.6 us (Grace).  The
// checks are those of the Python binding: type, shape, contiguity, and every
// tensor on one device, which the launch is made on whatever the current one
// is.  Each function takes the tensors of the Python wrapper of its name and
// returns the C call's status.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/core/ScalarType.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>
#include <vector>

#include "../../include/kvq.h"

namespace {

using at::ScalarType;

// Entry points of the library that the package loaded, set by bind().
struct Api {
    decltype(&kvq_decode_attn_window) decode_attn_window;
    decltype(&kvq_decode_attn_blocks) decode_attn_blocks;
    decltype(&kvq_tag_check_window) tag_check_window;
    decltype(&kvq_append_blocks) append_blocks;
    decltype(&kvq_copy_pages) copy_pages;
} api = {};

struct Refused {};                           // a Python exception is set

[[noreturn]] void refuse(PyObject *type, const std::string &what)
{
    PyErr_SetString(type, what.c_str());
    throw Refused();
}

std::string shape_text(at::IntArrayRef s)
{
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i)
        t += (i ? ", " : "") + std::to_string(s[i]);
    return t + ")";
}

// The tensors of one call: their checks, and the device they share.
class Args {
public:
    explicit Args(const char *fn) : fn_(fn) {}

    // Tensor object -> tensor; TypeError if it is none.
    const at::Tensor &tensor(PyObject *o, const char *name)
    {
        if (!THPVariable_Check(o))
            refuse(PyExc_TypeError, std::string(name) + ": expected a tensor, got " + Py_TYPE(o)->tp_name);
        return THPVariable_Unpack(o);
    }

    void expect(const at::Tensor &t, const char *name, std::initializer_list<ScalarType> types,
                std::initializer_list<int64_t> shape)
    {
        bool fits = false;
        for (ScalarType s : types)
            fits |= t.scalar_type() == s;
        if (!fits)
            refuse(types.size() > 1 ? PyExc_ValueError : PyExc_TypeError,
                   std::string(name) + ": expected " + c10::toString(*types.begin()) +
                       (types.size() > 1 ? std::string(" or ") + c10::toString(types.begin()[1]) : "") + ", got " +
                       c10::toString(t.scalar_type()));
        if (!t.sizes().equals(at::IntArrayRef(shape)))
            refuse(PyExc_ValueError, std::string(name) + ": expected shape " + shape_text(shape) + ", got " +
                                         shape_text(t.sizes()));
    }

    // The address of a contiguous tensor; where it lies is checked by device().
    void *at(const at::Tensor &t, const char *name)
    {
        if (!t.is_contiguous())
            refuse(PyExc_ValueError, std::string(name) + ": expected a contiguous tensor");
        const int dev = t.is_cuda() ? t.get_device() : kHost;
        if (dev_ == kNone)
            dev_ = dev;
        else if (dev != dev_ && other_ == kNone)
            other_ = dev;
        return t.data_ptr();
    }

    void *take(PyObject *o, const char *name, std::initializer_list<ScalarType> types,
               std::initializer_list<int64_t> shape)
    {
        const at::Tensor &t = tensor(o, name);
        expect(t, name, types, shape);
        return at(t, name);
    }

    void *take_or_none(PyObject *o, const char *name, std::initializer_list<ScalarType> types,
                       std::initializer_list<int64_t> shape)
    {
        return o == Py_None ? nullptr : take(o, name, types, shape);
    }

    // Any contiguous tensor of 4-byte elements of this shape.
    void *take_words(PyObject *o, const char *name, std::initializer_list<int64_t> shape)
    {
        const at::Tensor &t = tensor(o, name);
        if (t.element_size() != 4 || !t.sizes().equals(at::IntArrayRef(shape)))
            refuse(PyExc_ValueError, std::string(name) + ": expected 32-bit values of shape " + shape_text(shape));
        return at(t, name);
    }

    // The one CUDA device of every tensor taken.
    int device() const
    {
        if (dev_ == kHost || other_ == kHost)
            refuse(PyExc_ValueError, std::string(fn_) + ": expected CUDA tensors");
        if (other_ != kNone)
            refuse(PyExc_ValueError, std::string(fn_) + ": tensors on cuda:" + std::to_string(dev_) + " and cuda:" +
                                         std::to_string(other_));
        return dev_;
    }

    // The given stream (a torch stream or a handle), or the device's current one.
    kvq_stream_t stream(PyObject *o) const
    {
        const int dev = device();
        if (o == Py_None)
            return reinterpret_cast<kvq_stream_t>(
                c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream());
        PyObject *handle = o;
        Py_INCREF(handle);
        if (!PyLong_Check(o)) {
            Py_DECREF(handle);
            PyObject *index = PyObject_GetAttrString(o, "device_index");
            if (index == nullptr)
                throw Refused();
            const long on = PyLong_AsLong(index);
            Py_DECREF(index);
            if (on == -1 && PyErr_Occurred())
                throw Refused();
            if (on != dev)
                refuse(PyExc_ValueError, std::string(fn_) + ": a stream of cuda:" + std::to_string(on) +
                                             " for tensors on cuda:" + std::to_string(dev));
            handle = PyObject_GetAttrString(o, "cuda_stream");
            if (handle == nullptr)
                throw Refused();
        }
        void *p = PyLong_AsVoidPtr(handle);
        Py_DECREF(handle);
        if (p == nullptr && PyErr_Occurred())
            throw Refused();
        return reinterpret_cast<kvq_stream_t>(p);
    }

private:
    static constexpr int kNone = -2, kHost = -1;
    const char *fn_;
    int dev_ = kNone, other_ = kNone;
};

int32_t int_of(PyObject *o, const char *name)
{
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred())
        throw Refused();
    if (v < INT32_MIN || v > INT32_MAX)
        refuse(PyExc_OverflowError, std::string(name) + ": does not fit 32 bits");
    return static_cast<int32_t>(v);
}

kvq_cache_desc desc_of(PyObject *o)
{
    kvq_cache_desc d;
    const struct { const char *name; int32_t *to; } fields[] = {{"num_pages", &d.num_pages},
                                                                {"page_size", &d.page_size},
                                                                {"num_kv_heads", &d.num_kv_heads},
                                                                {"head_dim", &d.head_dim},
                                                                {"cache_dtype", &d.cache_dtype}};
    for (const auto &f : fields) {
        PyObject *v = PyObject_GetAttrString(o, f.name);
        if (v == nullptr)
            throw Refused();
        const long x = PyLong_AsLong(v);
        Py_DECREF(v);
        if (x == -1 && PyErr_Occurred())
            throw Refused();
        if (x < INT32_MIN || x > INT32_MAX)
            refuse(PyExc_OverflowError, std::string(f.name) + ": does not fit 32 bits");
        *f.to = static_cast<int32_t>(x);
    }
    return d;
}

ScalarType cache_type(const kvq_cache_desc &d)
{
    return d.cache_dtype == KVQ_CACHE_FP8_E4M3 ? ScalarType::Byte : ScalarType::BFloat16;
}

void *take_cache(Args &a, const kvq_cache_desc &d, PyObject *o, const char *name)
{
    return a.take(o, name, {cache_type(d)}, {d.num_pages, d.num_kv_heads, d.page_size, d.head_dim});
}

constexpr int kBlockTokens = 16;             // tokens that share an exponent

void *take_exps(Args &a, const kvq_cache_desc &d, PyObject *o, const char *name)
{
    return a.take(o, name, {ScalarType::Char}, {d.num_pages, d.num_kv_heads, d.page_size / kBlockTokens});
}

// (batch, entries per row) of a block table.
std::pair<int32_t, int32_t> take_table(Args &a, PyObject *o, const int32_t **table)
{
    const at::Tensor &t = a.tensor(o, "block_table");
    if (t.dim() != 2)
        refuse(PyExc_ValueError, "block_table: expected [batch][max_pages_per_seq]");
    a.expect(t, "block_table", {ScalarType::Int}, {t.size(0), t.size(1)});
    if (t.size(0) > INT32_MAX || t.size(1) > INT32_MAX)
        refuse(PyExc_ValueError, "block_table: too large");
    *table = static_cast<const int32_t *>(a.at(t, "block_table"));
    return {static_cast<int32_t>(t.size(0)), static_cast<int32_t>(t.size(1))};
}

// Run a call on its device without the interpreter lock.
template <typename Call>
PyObject *launch(int dev, const Call &call)
{
    kvq_status st;
    {
        const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
        Py_BEGIN_ALLOW_THREADS
        st = call();
        Py_END_ALLOW_THREADS
    }
    return PyLong_FromLong(st);
}

// No C++ exception leaves an entry.
template <typename Body>
PyObject *entry(const char *fn, Py_ssize_t nargs, Py_ssize_t want, const Body &body)
{
    if (nargs != want) {
        PyErr_Format(PyExc_TypeError, "%s: expected %zd arguments, got %zd", fn, want, nargs);
        return nullptr;
    }
    try {
        return body();
    } catch (const Refused &) {
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// (desc, q, k_cache, v_cache, k_scale | k_exp, v_scale | v_exp, block_table,
//  seq_lens, softmax_scale, window, num_sinks, abort_flags, out, workspace, num_splits, stream)
PyObject *decode_attn(const char *fn, bool blocks, PyObject *const *p, Py_ssize_t nargs)
{
    return entry(fn, nargs, 16, [&]() -> PyObject * {
        Args a(fn);
        const kvq_cache_desc d = desc_of(p[0]);
        const at::Tensor &qt = a.tensor(p[1], "q");
        if (qt.dim() != 4)
            refuse(PyExc_ValueError, "q: expected [batch][query tokens][query heads][head_dim]");
        const int64_t B = qt.size(0), n = qt.size(1), hq = qt.size(2);
        if (B > INT32_MAX || n > INT32_MAX || hq > INT32_MAX)
            refuse(PyExc_ValueError, "q: too large");
        a.expect(qt, "q", {ScalarType::BFloat16}, {B, n, hq, d.head_dim});
        const void *q = a.at(qt, "q");
        const void *k = take_cache(a, d, p[2], "k_cache"), *v = take_cache(a, d, p[3], "v_cache");
        const void *s0 = nullptr, *s1 = nullptr;
        if (blocks) {
            s0 = take_exps(a, d, p[4], "k_exp");
            s1 = take_exps(a, d, p[5], "v_exp");
        } else if (d.cache_dtype == KVQ_CACHE_FP8_E4M3) {  // ignored with a bf16 cache
            s0 = a.take(p[4], "k_scale", {ScalarType::Float}, {d.num_kv_heads});
            s1 = a.take(p[5], "v_scale", {ScalarType::Float}, {d.num_kv_heads});
        }
        const int32_t *table;
        const auto [rows, maxp] = take_table(a, p[6], &table);
        if (rows != B)
            refuse(PyExc_ValueError, "block_table: expected " + std::to_string(B) + " rows, got " +
                                         std::to_string(rows));
        const auto *seq = static_cast<const int32_t *>(a.take(p[7], "seq_lens", {ScalarType::Int}, {B}));
        const double scale = PyFloat_AsDouble(p[8]);
        if (scale == -1.0 && PyErr_Occurred())
            throw Refused();
        const int32_t window = int_of(p[9], "window"), sinks = int_of(p[10], "num_sinks");
        const auto *abort =
            static_cast<const uint8_t *>(a.take_or_none(p[11], "abort_flags", {ScalarType::Byte}, {B}));
        const at::Tensor &ot = a.tensor(p[12], "out");
        a.expect(ot, "out", {ScalarType::BFloat16, ScalarType::Float}, {B, n, hq, d.head_dim});
        void *out = a.at(ot, "out");
        void *ws = nullptr;
        size_t ws_bytes = 0;
        if (p[13] != Py_None) {
            const at::Tensor &wt = a.tensor(p[13], "workspace");
            ws = a.at(wt, "workspace");
            ws_bytes = static_cast<size_t>(wt.numel()) * wt.element_size();
        }
        const int32_t splits = int_of(p[14], "num_splits");
        const int dev = a.device();
        const kvq_stream_t stream = a.stream(p[15]);
        const int32_t type = ot.scalar_type() == ScalarType::Float ? KVQ_OUT_FP32 : KVQ_OUT_BF16;
        const int32_t b32 = static_cast<int32_t>(B), n32 = static_cast<int32_t>(n), h32 = static_cast<int32_t>(hq);
        const int32_t entries = maxp;
        return launch(dev, [&] {
            if (blocks)
                return api.decode_attn_blocks(&d, q, b32, n32, h32, k, v, static_cast<const int8_t *>(s0),
                                              static_cast<const int8_t *>(s1), table, entries, seq,
                                              static_cast<float>(scale), window, sinks, abort, out, type, ws, ws_bytes,
                                              splits, stream);
            return api.decode_attn_window(&d, q, b32, n32, h32, k, v, static_cast<const float *>(s0),
                                          static_cast<const float *>(s1), table, entries, seq,
                                          static_cast<float>(scale), window, sinks, abort, out, type, ws, ws_bytes,
                                          splits, stream);
        });
    });
}

PyObject *py_decode_attn_window(PyObject *, PyObject *const *p, Py_ssize_t n)
{
    return decode_attn("kvq_decode_attn_window", false, p, n);
}

PyObject *py_decode_attn_blocks(PyObject *, PyObject *const *p, Py_ssize_t n)
{
    return decode_attn("kvq_decode_attn_blocks", true, p, n);
}

// (block_table, expected_tags, seq_lens, page_size, page_tags, window, num_sinks,
//  num_query_tokens, abort_flags, stream)
PyObject *py_tag_check_window(PyObject *, PyObject *const *p, Py_ssize_t nargs)
{
    return entry("kvq_tag_check_window", nargs, 10, [&]() -> PyObject * {
        Args a("kvq_tag_check_window");
        const int32_t *table;
        const auto [B, maxp] = take_table(a, p[0], &table);
        const auto *want = static_cast<const uint32_t *>(a.take_words(p[1], "expected_tags", {B, maxp}));
        const auto *seq = static_cast<const int32_t *>(a.take(p[2], "seq_lens", {ScalarType::Int}, {B}));
        const int32_t ps = int_of(p[3], "page_size");
        const at::Tensor &tt = a.tensor(p[4], "page_tags");
        if (tt.dim() != 1 || tt.size(0) > INT32_MAX)
            refuse(PyExc_ValueError, "page_tags: expected 32-bit tags [num_pages]");
        const auto *tags = static_cast<const uint32_t *>(a.take_words(p[4], "page_tags", {tt.size(0)}));
        const int32_t pages = static_cast<int32_t>(tt.size(0));
        const int32_t window = int_of(p[5], "window"), sinks = int_of(p[6], "num_sinks");
        const int32_t n = int_of(p[7], "num_query_tokens");
        auto *flags = static_cast<uint8_t *>(a.take(p[8], "abort_flags", {ScalarType::Byte}, {B}));
        const int dev = a.device();
        const kvq_stream_t stream = a.stream(p[9]);
        const int32_t rows = B, entries = maxp;
        return launch(dev, [&] {
            return api.tag_check_window(table, want, seq, rows, entries, ps, tags, pages, window, sinks, n, flags,
                                        stream);
        });
    });
}

// (desc, k_new, v_new, token_offsets, block_table, seq_lens, abort_flags, k_cache,
//  v_cache, k_exp, v_exp, stream)
PyObject *py_append_blocks(PyObject *, PyObject *const *p, Py_ssize_t nargs)
{
    return entry("kvq_append_blocks", nargs, 12, [&]() -> PyObject * {
        Args a("kvq_append_blocks");
        const kvq_cache_desc d = desc_of(p[0]);
        const at::Tensor &kt = a.tensor(p[1], "k_new");
        if (kt.dim() != 3 || kt.size(0) > INT32_MAX)
            refuse(PyExc_ValueError, "k_new: expected [tokens][num_kv_heads][head_dim]");
        const int64_t T = kt.size(0);
        const void *k_new = a.take(p[1], "k_new", {ScalarType::BFloat16}, {T, d.num_kv_heads, d.head_dim});
        const void *v_new = a.take(p[2], "v_new", {ScalarType::BFloat16}, {T, d.num_kv_heads, d.head_dim});
        const int32_t *table;
        const auto [B, maxp] = take_table(a, p[4], &table);
        const auto *off = static_cast<const int32_t *>(
            a.take_or_none(p[3], "token_offsets", {ScalarType::Int}, {static_cast<int64_t>(B) + 1}));
        const auto *seq = static_cast<const int32_t *>(a.take(p[5], "seq_lens", {ScalarType::Int}, {B}));
        const auto *abort =
            static_cast<const uint8_t *>(a.take_or_none(p[6], "abort_flags", {ScalarType::Byte}, {B}));
        void *k = take_cache(a, d, p[7], "k_cache"), *v = take_cache(a, d, p[8], "v_cache");
        auto *ke = static_cast<int8_t *>(take_exps(a, d, p[9], "k_exp"));
        auto *ve = static_cast<int8_t *>(take_exps(a, d, p[10], "v_exp"));
        const int dev = a.device();
        const kvq_stream_t stream = a.stream(p[11]);
        const int32_t rows = B, entries = maxp;
        return launch(dev, [&] {
            return api.append_blocks(&d, k_new, v_new, static_cast<int32_t>(T), off, table, entries, seq, rows, abort,
                                     k, v, ke, ve, stream);
        });
    });
}

// (desc, caches, exps, src_pages, dst_pages, stream)
PyObject *py_copy_pages(PyObject *, PyObject *const *p, Py_ssize_t nargs)
{
    return entry("kvq_copy_pages", nargs, 6, [&]() -> PyObject * {
        Args a("kvq_copy_pages");
        const kvq_cache_desc d = desc_of(p[0]);
        struct Sequence {
            PyObject *o;
            explicit Sequence(PyObject *s) : o(PySequence_Fast(s, "expected a sequence of tensors"))
            {
                if (o == nullptr)
                    throw Refused();
            }
            ~Sequence() { Py_DECREF(o); }
            Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(o); }
            PyObject *operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(o, i); }
        } caches(p[1]), exps(p[2]);
        std::vector<void *> cp(static_cast<size_t>(caches.size())), ep(static_cast<size_t>(exps.size()));
        for (Py_ssize_t i = 0; i < caches.size(); ++i)
            cp[static_cast<size_t>(i)] = take_cache(a, d, caches[i], "caches");
        for (Py_ssize_t i = 0; i < exps.size(); ++i)
            ep[static_cast<size_t>(i)] = take_exps(a, d, exps[i], "exps");
        const at::Tensor &st = a.tensor(p[3], "src_pages");
        if (st.dim() != 1 || st.size(0) > INT32_MAX)
            refuse(PyExc_ValueError, "src_pages: expected page ids [num_listed]");
        const int64_t n = st.size(0);
        const auto *src = static_cast<const int32_t *>(a.take(p[3], "src_pages", {ScalarType::Int}, {n}));
        const auto *dst = static_cast<const int32_t *>(a.take(p[4], "dst_pages", {ScalarType::Int}, {n}));
        const int dev = a.device();
        const kvq_stream_t stream = a.stream(p[5]);
        return launch(dev, [&] {
            return api.copy_pages(&d, cp.data(), static_cast<int32_t>(cp.size()), ep.data(),
                                  static_cast<int32_t>(ep.size()), src, dst, static_cast<int32_t>(n), stream);
        });
    });
}

// bind(addresses): the five entry points of the loaded library, in the order of Api.
PyObject *py_bind(PyObject *, PyObject *const *p, Py_ssize_t nargs)
{
    return entry("bind", nargs, 5, [&]() -> PyObject * {
        void *f[5];
        for (int i = 0; i < 5; ++i) {
            f[i] = PyLong_AsVoidPtr(p[i]);
            if (f[i] == nullptr) {
                if (!PyErr_Occurred())
                    PyErr_SetString(PyExc_ValueError, "bind: null entry point");
                throw Refused();
            }
        }
        api.decode_attn_window = reinterpret_cast<decltype(api.decode_attn_window)>(f[0]);
        api.decode_attn_blocks = reinterpret_cast<decltype(api.decode_attn_blocks)>(f[1]);
        api.tag_check_window = reinterpret_cast<decltype(api.tag_check_window)>(f[2]);
        api.append_blocks = reinterpret_cast<decltype(api.append_blocks)>(f[3]);
        api.copy_pages = reinterpret_cast<decltype(api.copy_pages)>(f[4]);
        Py_RETURN_NONE;
    });
}

using FastCall = PyObject *(*)(PyObject *, PyObject *const *, Py_ssize_t);

PyMethodDef method(const char *name, FastCall f)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method("bind", py_bind),
                         method("decode_attn_window", py_decode_attn_window),
                         method("decode_attn_blocks", py_decode_attn_blocks),
                         method("tag_check_window", py_tag_check_window),
                         method("append_blocks", py_append_blocks),
                         method("copy_pages", py_copy_pages),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kvq_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit__kvq_native() { return PyModule_Create(&module); }
