// marshal.cpp -- argument marshalling of the calls that take strided tensors
// of several types (the rotating appends and the latent pool's), for torch.
//
// The same work as the ctypes binding's: check what the library cannot see
// from pointers (element types, shapes, strides, devices), read the pointers
// and sizes off the tensors, make the C call on the current stream of the
// tensors' device.  In Python the fourteen tensors of one append took 13 us a
// call and ctypes another 4, next to 2 us of kernel.
//
// Each function returns the call's pa_status, or raises ValueError.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <string>

#include "pa.h"

namespace {

decltype(&pa_rope_append) g_rope_append = nullptr;
decltype(&pa_latent_append) g_latent_append = nullptr;
decltype(&pa_latent_decode) g_latent_decode = nullptr;
decltype(&pa_latent_prefill) g_latent_prefill = nullptr;

struct Refused : std::exception {
    std::string text;
    explicit Refused(std::string t) : text(std::move(t)) {}
    const char* what() const noexcept override { return text.c_str(); }
};

[[noreturn]] void refuse(const char* fn, const char* what) { throw Refused(std::string(fn) + ": " + what); }

inline void need(const char* fn, bool ok, const char* what)
{
    if (!ok) refuse(fn, what);
}

// A tensor argument; None gives nullptr.
const at::Tensor* tensor(const char* fn, PyObject* o, const char* name, bool may_be_none = false)
{
    if (o == Py_None && may_be_none) return nullptr;
    if (!THPVariable_Check(o)) refuse(fn, (std::string(name) + " must be a tensor").c_str());
    return &THPVariable_Unpack(o);
}

double number(PyObject* o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused("a scalar argument is not a number");
    }
    return v;
}

int64_t whole(PyObject* o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused("a size or stream argument is not an integer");
    }
    return v;
}

bool truth(PyObject* o, const char* name)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) {                          // (an array of several elements)
        PyErr_Clear();
        throw Refused(std::string(name) + " is neither true nor false");
    }
    return v != 0;
}

// Sizes that the C call takes as int32.
int32_t narrow(int64_t v)
{
    if (v > 0x7fffffffLL || v < -0x80000000LL) throw Refused("a size passes 32 bits");
    return static_cast<int32_t>(v);
}

pa_dtype type_code(at::ScalarType t)
{
    switch (t) {
    case at::kHalf: return PA_DTYPE_F16;
    case at::kBFloat16: return PA_DTYPE_BF16;
    case at::kByte:
    case at::kFloat8_e4m3fn: return PA_DTYPE_FP8_E4M3;
    case at::kChar: return PA_DTYPE_INT8;
    case at::kFloat: return PA_DTYPE_F32;
    default: return static_cast<pa_dtype>(99);       // refused by the library
    }
}

void* ptr(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }

// [rows][heads][dim] with whole head rows side by side; the rows' stride is free.
bool head_rows(const at::Tensor& t, int64_t rows, int64_t heads, int64_t dim, at::ScalarType type)
{
    return t.scalar_type() == type && t.dim() == 3 && t.size(0) == rows && t.size(1) == heads &&
           t.size(2) == dim && t.stride(2) == 1 && (heads == 1 || t.stride(1) == dim);
}

bool vector_of(const at::Tensor& t, int64_t n, at::ScalarType type)
{
    return t.scalar_type() == type && t.dim() == 1 && t.size(0) == n && t.is_contiguous();
}

// The C calls run without the interpreter's lock, as through ctypes: other
// threads go on while a launch waits for the driver.  The arguments stay alive,
// their caller holds them.
struct Unlocked {
    PyThreadState* const state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

template <typename F, typename... Args>
int call_unlocked(F f, Args... args)
{
    const Unlocked unlocked;
    return f(args...);
}

// The device that all the tensors are on, made current for the call.
struct OnDevice {
    c10::cuda::CUDAGuard guard;
    cudaStream_t stream;
    OnDevice(c10::Device d, int64_t given) : guard(d)
    {
        stream = given == -1 ? c10::cuda::getCurrentCUDAStream(d.index()).stream()
                             : reinterpret_cast<cudaStream_t>(given);
    }
};

template <typename... Ts>
c10::Device one_device(const char* fn, const at::Tensor& first, const Ts*... rest)
{
    const c10::Device d = first.device();
    need(fn, d.is_cuda() && (... && (rest == nullptr || rest->device() == d)),
         "all tensors must be on one CUDA device");
    return d;
}

void check_status(const char* fn, const at::Tensor* t)
{
    need(fn, t == nullptr || (t->scalar_type() == at::kInt && t->numel() >= 1), "d_status must be int32");
}

int rope_append(PyObject* const* a)
{
    const char* fn = "pa_rope_append";
    const at::Tensor &query_out = *tensor(fn, a[0], "query_out"), &query = *tensor(fn, a[1], "query"),
                     &key = *tensor(fn, a[2], "key"), &value = *tensor(fn, a[3], "value"),
                     &k_cache = *tensor(fn, a[4], "k_cache"), &v_cache = *tensor(fn, a[5], "v_cache"),
                     &slots = *tensor(fn, a[6], "slot_mapping"), &pos = *tensor(fn, a[7], "positions"),
                     &table = *tensor(fn, a[8], "cos_sin");
    const at::Tensor *qw = tensor(fn, a[9], "q_weight", true), *kw = tensor(fn, a[10], "k_weight", true);
    const double eps = number(a[11]);
    const bool pairs = truth(a[12], "interleaved");
    const double k_scale = number(a[13]), v_scale = number(a[14]);
    const at::Tensor *ks = tensor(fn, a[15], "k_scales", true), *vs = tensor(fn, a[16], "v_scales", true),
                     *status = tensor(fn, a[17], "d_status", true);
    need(fn, query.dim() == 3 && k_cache.dim() == 4, "query is [T][Hq][D], k_cache [num_blocks][B][Hkv][D]");
    const at::ScalarType type = query.scalar_type();
    const int64_t tokens = query.size(0), hq = query.size(1), d = query.size(2);
    const int64_t blocks = k_cache.size(0), block = k_cache.size(1), hkv = k_cache.size(2);
    need(fn, head_rows(query, tokens, hq, d, type) && head_rows(query_out, tokens, hq, d, type),
         "query and query_out must be [T][Hq][D] of one type with contiguous heads");
    need(fn, head_rows(key, tokens, hkv, d, type) && head_rows(value, tokens, hkv, d, type),
         "key and value must be [T][Hkv][D] of the query's type with contiguous heads");
    need(fn, k_cache.sizes() == v_cache.sizes() && k_cache.size(3) == d &&
                 k_cache.scalar_type() == v_cache.scalar_type() && k_cache.is_contiguous() &&
                 v_cache.is_contiguous(),
         "k_cache and v_cache must be contiguous pools of one shape");
    need(fn, vector_of(slots, tokens, at::kLong) && vector_of(pos, tokens, at::kLong),
         "slot_mapping and positions must be contiguous int64 [T]");
    need(fn, table.scalar_type() == at::kFloat && table.dim() == 2 && table.is_contiguous(),
         "cos_sin must be contiguous float32 [max_position][rot_dim]");
    need(fn, (!qw || vector_of(*qw, d, type)) && (!kw || vector_of(*kw, d, type)),
         "norm weights must be contiguous [D] of the query's type");
    for (const at::Tensor* s : {ks, vs})
        need(fn, s == nullptr || (s->scalar_type() == at::kFloat && s->is_contiguous() && s->dim() == 3 &&
                                  s->size(0) == blocks && s->size(1) == hkv && s->size(2) == block),
             "scale pools must be contiguous float32 [num_blocks][Hkv][B]");
    check_status(fn, status);
    const OnDevice on(one_device(fn, query, &query_out, &key, &value, &k_cache, &v_cache, &slots, &pos, &table,
                                 qw, kw, ks, vs, status),
                      whole(a[18]));
    return call_unlocked(
        g_rope_append, ptr(&query_out), ptr(&query), ptr(&key), ptr(&value), ptr(&k_cache), ptr(&v_cache),
        static_cast<float*>(ptr(ks)), static_cast<float*>(ptr(vs)), static_cast<int64_t*>(ptr(&slots)),
        static_cast<int64_t*>(ptr(&pos)), static_cast<float*>(ptr(&table)), ptr(qw), ptr(kw),
        static_cast<float>(eps), narrow(tokens), narrow(hq), narrow(hkv), narrow(d), narrow(table.size(1)),
        table.size(0), pairs ? 1 : 0, query_out.stride(0), query.stride(0), key.stride(0), value.stride(0),
        narrow(block), blocks, type_code(type), type_code(k_cache.scalar_type()), static_cast<float>(k_scale),
        static_cast<float>(v_scale), static_cast<int32_t*>(ptr(status)), on.stream);
}

int latent_append(PyObject* const* a)
{
    const char* fn = "pa_latent_append";
    const at::Tensor *q_out = tensor(fn, a[0], "query_out", true), *q_in = tensor(fn, a[1], "query_rope", true);
    const at::Tensor &latent = *tensor(fn, a[2], "latent"), &cache = *tensor(fn, a[3], "cache"),
                     &slots = *tensor(fn, a[4], "slot_mapping"), &pos = *tensor(fn, a[5], "positions"),
                     &table = *tensor(fn, a[6], "cos_sin");
    const at::Tensor* weight = tensor(fn, a[7], "weight", true);
    const double eps = number(a[8]);
    const bool pairs = truth(a[9], "interleaved");
    const at::Tensor* status = tensor(fn, a[10], "d_status", true);
    need(fn, cache.dim() == 3 && cache.is_contiguous(), "cache must be contiguous [num_blocks][B][L + R]");
    need(fn, table.scalar_type() == at::kFloat && table.dim() == 2 && table.is_contiguous(),
         "cos_sin must be contiguous float32 [max_position][rope_dim]");
    const at::ScalarType type = cache.scalar_type();
    const int64_t width = cache.size(2), rope = table.size(1);
    need(fn, latent.scalar_type() == type && latent.dim() == 2 && latent.size(1) == width &&
                 latent.stride(1) == 1,
         "latent must be [T][L + R] of the cache's type with contiguous rows");
    const int64_t tokens = latent.size(0);
    need(fn, (q_out == nullptr) == (q_in == nullptr), "query_rope and query_out go together");
    int64_t heads = 0, q_t = 0, q_h = 0, o_t = 0, o_h = 0;
    if (q_in != nullptr) {
        need(fn, q_in->dim() == 3, "query_rope must be [T][H][R]");
        heads = q_in->size(1);
        for (const at::Tensor* t : {q_in, q_out})
            need(fn, t->scalar_type() == type && t->dim() == 3 && t->size(0) == tokens &&
                         t->size(1) == heads && t->size(2) == rope && t->stride(2) == 1,
                 "query_rope and query_out must be [T][H][R] of the cache's type with contiguous rows");
        q_t = q_in->stride(0);
        q_h = q_in->stride(1);
        o_t = q_out->stride(0);
        o_h = q_out->stride(1);
    }
    need(fn, vector_of(slots, tokens, at::kLong) && vector_of(pos, tokens, at::kLong),
         "slot_mapping and positions must be contiguous int64 [T]");
    need(fn, !weight || vector_of(*weight, width - rope, type),
         "weight must be contiguous [L] of the cache's type");
    check_status(fn, status);
    const OnDevice on(one_device(fn, cache, q_out, q_in, &latent, &slots, &pos, &table, weight, status),
                      whole(a[11]));
    return call_unlocked(
        g_latent_append, ptr(q_out), ptr(q_in), ptr(&latent), ptr(&cache), static_cast<int64_t*>(ptr(&slots)),
        static_cast<int64_t*>(ptr(&pos)), static_cast<float*>(ptr(&table)), ptr(weight),
        static_cast<float>(eps), narrow(tokens), narrow(heads), narrow(width - rope), narrow(rope),
        table.size(0), pairs ? 1 : 0, o_t, o_h, q_t, q_h, latent.stride(0), narrow(cache.size(1)),
        cache.size(0), type_code(type), static_cast<int32_t*>(ptr(status)), on.stream);
}

void check_tables(const char* fn, const at::Tensor& tables, const at::Tensor& lens, int64_t seqs)
{
    need(fn, tables.scalar_type() == at::kInt && tables.dim() == 2 && tables.size(0) == seqs &&
                 tables.is_contiguous(),
         "block_tables must be contiguous int32 [S][max_blocks_per_seq]");
    need(fn, vector_of(lens, seqs, at::kInt), "context_lens must be contiguous int32 [S]");
}

size_t bytes(const at::Tensor* t) { return t ? t->nbytes() : 0; }

int latent_decode(PyObject* const* a)
{
    const char* fn = "pa_latent_decode";
    const at::Tensor &out = *tensor(fn, a[0], "out"), &query = *tensor(fn, a[1], "query"),
                     &cache = *tensor(fn, a[2], "cache"), &tables = *tensor(fn, a[3], "block_tables"),
                     &lens = *tensor(fn, a[4], "context_lens");
    const int64_t max_context = whole(a[5]);
    const double scale = number(a[6]);
    const at::Tensor *ws = tensor(fn, a[7], "workspace", true), *status = tensor(fn, a[8], "d_status", true);
    need(fn, query.dim() == 3 && out.dim() == 3 && cache.dim() == 3 &&
                 query.scalar_type() == cache.scalar_type() && out.scalar_type() == cache.scalar_type() &&
                 cache.size(2) == query.size(2) && out.size(0) == query.size(0) &&
                 out.size(1) == query.size(1) && query.is_contiguous() && cache.is_contiguous() &&
                 out.is_contiguous(),
         "out [S][H][L], query [S][H][L + R] and cache [num_blocks][B][L + R] must be contiguous tensors "
         "of one type");
    const int64_t seqs = query.size(0), lat = out.size(2);
    check_tables(fn, tables, lens, seqs);
    need(fn, ws == nullptr || ws->is_contiguous(), "workspace must be contiguous");
    check_status(fn, status);
    const OnDevice on(one_device(fn, query, &out, &cache, &tables, &lens, ws, status), whole(a[9]));
    return call_unlocked(
        g_latent_decode, ptr(&out), ptr(&query), ptr(&cache), static_cast<int32_t*>(ptr(&tables)),
        static_cast<int32_t*>(ptr(&lens)), narrow(seqs), narrow(query.size(1)), narrow(lat),
        narrow(query.size(2) - lat), narrow(cache.size(1)), narrow(tables.size(1)), cache.size(0),
        narrow(max_context), static_cast<float>(scale), ptr(ws), bytes(ws), type_code(query.scalar_type()),
        static_cast<int32_t*>(ptr(status)), on.stream);
}

int latent_prefill(PyObject* const* a)
{
    const char* fn = "pa_latent_prefill";
    const at::Tensor &out = *tensor(fn, a[0], "out"), &query = *tensor(fn, a[1], "query"),
                     &cache = *tensor(fn, a[2], "cache"), &w = *tensor(fn, a[3], "w_kv"),
                     &tables = *tensor(fn, a[4], "block_tables"), &starts = *tensor(fn, a[5], "query_starts"),
                     &lens = *tensor(fn, a[6], "context_lens");
    const int64_t max_query = whole(a[7]), max_context = whole(a[8]);
    const double scale = number(a[9]);
    const at::Tensor *ws = tensor(fn, a[10], "workspace", true), *status = tensor(fn, a[11], "d_status", true);
    const at::ScalarType type = query.scalar_type();
    need(fn, query.dim() == 3 && out.dim() == 3 && cache.dim() == 3 && w.dim() == 3 && lens.dim() == 1 &&
                 cache.scalar_type() == type && out.scalar_type() == type && w.scalar_type() == type &&
                 out.size(0) == query.size(0) && out.size(1) == query.size(1) && w.size(0) == query.size(1) &&
                 query.is_contiguous() && cache.is_contiguous() && out.is_contiguous() && w.is_contiguous(),
         "out [T][H][value], query [T][H][nope + R], cache [num_blocks][B][L + R] and w_kv "
         "[H][nope + value][L] must be contiguous tensors of one type");
    const int64_t seqs = lens.size(0), value = out.size(2), lat = w.size(2), rope = cache.size(2) - lat;
    const int64_t nope = query.size(2) - rope;
    need(fn, w.size(1) == nope + value, "w_kv must be [H][nope + value][L]");
    check_tables(fn, tables, lens, seqs);
    need(fn, vector_of(starts, seqs + 1, at::kInt), "query_starts must be contiguous int32 [S + 1]");
    need(fn, ws == nullptr || ws->is_contiguous(), "workspace must be contiguous");
    check_status(fn, status);
    const OnDevice on(one_device(fn, query, &out, &cache, &w, &tables, &starts, &lens, ws, status),
                      whole(a[12]));
    return call_unlocked(
        g_latent_prefill, ptr(&out), ptr(&query), ptr(&cache), ptr(&w),
        static_cast<int32_t*>(ptr(&tables)), static_cast<int32_t*>(ptr(&starts)),
        static_cast<int32_t*>(ptr(&lens)), narrow(seqs), narrow(query.size(0)), narrow(query.size(1)),
        narrow(lat), narrow(rope), narrow(nope), narrow(value), narrow(cache.size(1)),
        narrow(tables.size(1)), cache.size(0), narrow(max_query), narrow(max_context),
        static_cast<float>(scale), ptr(ws), bytes(ws), type_code(type), static_cast<int32_t*>(ptr(status)),
        on.stream);
}

template <int (*call)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    try {
        if (n != N) throw Refused("wrong number of arguments");
        return PyLong_FromLong(call(args));
    } catch (const Refused& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// bind(rope_append, latent_append, latent_decode, latent_prefill): the
// addresses of the library's functions.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    try {
        if (n != 4) throw Refused("bind: four addresses");
        g_rope_append = reinterpret_cast<decltype(g_rope_append)>(whole(args[0]));
        g_latent_append = reinterpret_cast<decltype(g_latent_append)>(whole(args[1]));
        g_latent_decode = reinterpret_cast<decltype(g_latent_decode)>(whole(args[2]));
        g_latent_prefill = reinterpret_cast<decltype(g_latent_prefill)>(whole(args[3]));
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
        return nullptr;
    }
    Py_RETURN_NONE;
}

template <typename F>
PyCFunction as_method(F f)
{
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"bind", as_method(bind), METH_FASTCALL, "the library's functions"},
    {"rope_append", as_method(entry<rope_append, 19>), METH_FASTCALL, "pa_rope_append"},
    {"latent_append", as_method(entry<latent_append, 12>), METH_FASTCALL, "pa_latent_append"},
    {"latent_decode", as_method(entry<latent_decode, 10>), METH_FASTCALL, "pa_latent_decode"},
    {"latent_prefill", as_method(entry<latent_prefill, 13>), METH_FASTCALL, "pa_latent_prefill"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", "argument marshalling for libpa.so", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

// The file's name carries no version, so it says for itself what it was built
// for: the torch as an attribute, the Python here.
PyMODINIT_FUNC PyInit__marshal(void)
{
    const std::string built = std::to_string(PY_MAJOR_VERSION) + "." + std::to_string(PY_MINOR_VERSION) + ".";
    if (std::string(Py_GetVersion()).compare(0, built.size(), built) != 0) {
        PyErr_Format(PyExc_ImportError, "built for Python %sx", built.c_str());
        return nullptr;
    }
    PyObject* m = PyModule_Create(&module);
    if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", PA_TORCH_VERSION) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
