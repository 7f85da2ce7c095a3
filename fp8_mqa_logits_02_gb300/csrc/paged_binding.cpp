// The paged operators' Python binding: checks torch tensors, allocates results, and calls the C
// entry points of libfp8mqa.so (their addresses come from the Python side, which loads the library).
// A serving step makes these calls once per layer and token, and the same checks written in Python
// took longer than the kernels of a short request do.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>
#include <string>

#include "../../include/fp8_mqa_logits.h"

namespace {

struct Raised {};  // a Python error is set

struct Entries {
    decltype(&fp8_mqa_cache_write) cache_write = nullptr;
    decltype(&fp8_mqa_cache_read) cache_read = nullptr;
    decltype(&fp8_mqa_logits_paged) logits_paged = nullptr;
    decltype(&fp8_mqa_attention_paged_workspace_bytes) workspace_bytes = nullptr;
    decltype(&fp8_mqa_attention_paged) attention_paged = nullptr;
} g_entry;

PyObject* g_error = nullptr;  // Fp8MqaError

constexpr int64_t kHeads = 32, kDim = 128;

[[noreturn]] void bad(PyObject* type, const std::string& what)
{
    PyErr_SetString(type, what.c_str());
    throw Raised{};
}

std::string list(c10::IntArrayRef v)
{
    std::string s = "[";
    for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
    return s + "]";
}

std::string name_of(at::ScalarType t) { return std::string("torch.") + c10::toString(t); }

void done(int status, const char* name)
{
    if (status == FP8MQA_OK) return;
    PyObject* args = Py_BuildValue("(is)", status, name);
    if (args) PyErr_SetObject(g_error, args);
    Py_XDECREF(args);
    throw Raised{};
}

const at::Tensor& tensor(PyObject* o, const char* name)
{
    if (!THPVariable_Check(o)) bad(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}

// A CUDA tensor on `device`, or on any for the first one of a call.
const at::Tensor& cuda_tensor(PyObject* o, const char* name, const c10::Device* device = nullptr)
{
    const at::Tensor& t = tensor(o, name);
    if (!t.is_cuda())
        bad(PyExc_ValueError, std::string(name) + " must be a CUDA tensor (the library has no CPU path)");
    if (device && t.device() != *device)
        bad(PyExc_ValueError, std::string(name) + " is on " + t.device().str() + ", expected " + device->str());
    return t;
}

// An int32 tensor of d0 (negative: any size), or d0 x any, whose last dimension is contiguous.
const at::Tensor& ints(PyObject* o, const char* name, const c10::Device& device, int dims, int64_t d0)
{
    const at::Tensor& t = cuda_tensor(o, name, &device);
    if (t.scalar_type() != at::kInt)
        bad(PyExc_TypeError, std::string(name) + " must be int32, got " + name_of(t.scalar_type()));
    if (t.dim() != dims || (d0 >= 0 && t.size(0) != d0))
        bad(PyExc_ValueError, std::string(name) + " must be [" + (d0 < 0 ? "any" : std::to_string(d0)) +
                                  (dims == 2 ? ", any], got " : "], got ") + list(t.sizes()));
    if (t.size(dims - 1) > 1 && t.stride(dims - 1) != 1)
        bad(PyExc_ValueError, std::string(name) + " must be contiguous in its last dimension");
    // the C interface takes the columns as an int32
    if (dims == 2 && t.size(1) > INT32_MAX)
        bad(PyExc_ValueError, std::string(name) + " is too large: " + list(t.sizes()));
    return t;
}

// The type's number in the C interface, or -1.
int32_t type_of(at::ScalarType t)
{
    switch (t) {
        case at::kFloat8_e4m3fn: return FP8MQA_E4M3;
        case at::kBFloat16: return FP8MQA_BF16;
        case at::kHalf: return FP8MQA_F16;
        case at::kFloat: return FP8MQA_F32;
        default: return -1;
    }
}

// A cache of e4m3 data and its scales, or of the type `other` without.
fp8mqa_cache cache_of(PyObject* data_o, PyObject* scale_o, const char* name, const c10::Device& device,
                      at::ScalarType other = at::kFloat8_e4m3fn)
{
    const std::string what(name);
    const at::Tensor& data = cuda_tensor(data_o, (what + " data").c_str(), &device);
    const at::ScalarType dtype = data.scalar_type();
    if (data.dim() != 4)
        bad(PyExc_ValueError, what + " data must be [pages, page_size, heads, dim], got " + list(data.sizes()));
    if (data.stride(3) != 1) bad(PyExc_ValueError, what + " data must be contiguous in its last dimension");
    fp8mqa_cache c;
    c.data = data.data_ptr();
    c.scale = nullptr;
    c.pages = data.size(0);
    for (int i = 1; i < 4; ++i)
        if (data.size(i) > INT32_MAX) bad(PyExc_ValueError, what + " data is too large: " + list(data.sizes()));
    c.page_size = int32_t(data.size(1));
    c.heads = int32_t(data.size(2));
    c.dim = int32_t(data.size(3));
    c.type = type_of(dtype);
    c.page_stride = data.stride(0);
    c.row_stride = data.stride(1);
    c.head_stride = data.stride(2);
    c.scale_page_stride = c.scale_row_stride = c.scale_head_stride = 0;
    if (dtype == at::kFloat8_e4m3fn) {
        const at::Tensor& scale = cuda_tensor(scale_o, (what + " scale").c_str(), &device);
        if (scale.scalar_type() != at::kFloat || scale.dim() != 3 || scale.size(0) != data.size(0) ||
            scale.size(1) != data.size(1) || scale.size(2) != data.size(2))
            bad(PyExc_ValueError, what + " scale must be float32 " + list(data.sizes().slice(0, 3)));
        c.scale = static_cast<float*>(scale.data_ptr());
        c.scale_page_stride = scale.stride(0);
        c.scale_row_stride = scale.stride(1);
        c.scale_head_stride = scale.stride(2);
    } else {
        if (dtype != other)
            bad(PyExc_TypeError, what + " data must be " + name_of(at::kFloat8_e4m3fn) +
                                     (other == at::kFloat8_e4m3fn ? "" : " or " + name_of(other)) + ", got " +
                                     name_of(dtype));
        if (scale_o != Py_None) bad(PyExc_ValueError, what + " scale goes with float8_e4m3fn data only");
    }
    return c;
}

at::Tensor empty(c10::IntArrayRef sizes, at::ScalarType type, const c10::Device& device)
{
    return at::empty(sizes, at::TensorOptions().dtype(type).device(device));
}

void* current_stream(const c10::Device& device)
{
    return static_cast<void*>(c10::cuda::getCurrentCUDAStream(device.index()).stream());
}

// Runs a C entry without the interpreter's lock.
template <class F>
int unlocked(F f)
{
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = f();
    Py_END_ALLOW_THREADS
    return rc;
}

void expect(Py_ssize_t n, Py_ssize_t want)
{
    if (n != want) bad(PyExc_TypeError, "wrong number of arguments");
    if (!g_entry.attention_paged) bad(PyExc_RuntimeError, "the library's entry points are not bound");
}

// slots, k, k_data, k_scale, v, v_data, v_scale
PyObject* cache_write(PyObject* const* a, Py_ssize_t n)
{
    expect(n, 7);
    const c10::Device device = cuda_tensor(a[2], "k data").device();
    const fp8mqa_cache ck = cache_of(a[2], a[3], "k", device);
    const at::Tensor& slots = ints(a[0], "slots", device, 1, -1);
    const bool pair = a[4] != Py_None;
    if (pair != (a[5] != Py_None) || pair != (a[6] != Py_None))
        bad(PyExc_ValueError, "v, v_data and v_scale go together");
    auto rows = [&](PyObject* o, const char* name, const at::Tensor* like) -> const at::Tensor& {
        const at::Tensor& x = cuda_tensor(o, name, &device);
        const int32_t type = type_of(x.scalar_type());
        if (type < 0 || type == FP8MQA_E4M3 || (like && x.scalar_type() != like->scalar_type()))
            bad(PyExc_TypeError, std::string(name) + " must be bfloat16, float16 or float32" +
                                     (like ? " as k is" : "") + ", got " + name_of(x.scalar_type()));
        if (x.dim() != 3 || x.size(0) != slots.size(0) || x.size(1) != ck.heads || x.size(2) != ck.dim)
            bad(PyExc_ValueError, std::string(name) + " must be " + list({slots.size(0), ck.heads, ck.dim}) +
                                      ", got " + list(x.sizes()));
        if (x.stride(2) != 1)
            bad(PyExc_ValueError, std::string(name) + " must be contiguous in its last dimension");
        return x;
    };
    const at::Tensor& k = rows(a[1], "k", nullptr);
    fp8mqa_cache cv;
    const void* v_ptr = nullptr;
    int64_t v_row = 0, v_head = 0;
    if (pair) {
        cv = cache_of(a[5], a[6], "v", device);
        if (cv.page_size != ck.page_size || cv.heads != ck.heads || cv.dim != ck.dim)
            bad(PyExc_ValueError, "v data must be " + list({ck.page_size, ck.heads, ck.dim}) + " a page, as k data is");
        const at::Tensor& v = rows(a[4], "v", &k);
        v_ptr = v.data_ptr();
        v_row = v.stride(0);
        v_head = v.stride(1);
    }
    const c10::cuda::CUDAGuard guard(device);
    const auto* s = static_cast<const int32_t*>(slots.data_ptr());
    const int64_t T = slots.size(0), row = k.stride(0), head = k.stride(1);
    const void* k_ptr = k.data_ptr();
    const int32_t type = type_of(k.scalar_type());
    void* stream = current_stream(device);
    done(unlocked([&] {
             return g_entry.cache_write(s, T, type, k_ptr, row, head, &ck, v_ptr, v_row, v_head,
                                        pair ? &cv : nullptr, stream);
         }),
         "fp8_mqa_cache_write");
    Py_RETURN_NONE;
}

// data, scale, table, starts, total, dtype
PyObject* cache_read(PyObject* const* a, Py_ssize_t n)
{
    expect(n, 6);
    const c10::Device device = cuda_tensor(a[0], "data").device();
    const fp8mqa_cache c = cache_of(a[0], a[1], "cache", device);
    const at::Tensor& table = ints(a[2], "table", device, 2, -1);
    const at::Tensor& starts = ints(a[3], "starts", device, 1, table.size(0) + 1);
    const int32_t type = THPDtype_Check(a[5]) ? type_of(reinterpret_cast<THPDtype*>(a[5])->scalar_type) : -1;
    if (type < 0)
        bad(PyExc_TypeError, "dtype must be float8_e4m3fn, bfloat16, float16 or float32");
    const at::ScalarType dtype = reinterpret_cast<THPDtype*>(a[5])->scalar_type;
    const long long total = PyLong_AsLongLong(a[4]);
    if (total == -1 && PyErr_Occurred()) throw Raised{};
    if (total < 0) bad(PyExc_ValueError, "total must not be negative");
    const c10::cuda::CUDAGuard guard(device);
    at::Tensor out = empty({total, c.heads, c.dim}, dtype, device), scales;
    if (type == FP8MQA_E4M3) scales = empty({total, c.heads}, at::kFloat, device);
    const auto* ids = static_cast<const int32_t*>(table.data_ptr());
    const auto* from = static_cast<const int32_t*>(starts.data_ptr());
    const int64_t by = table.stride(0), B = table.size(0);
    const int32_t cols = int32_t(table.size(1));
    void* to = out.data_ptr();
    float* to_scale = scales.defined() ? static_cast<float*>(scales.data_ptr()) : nullptr;
    void* stream = current_stream(device);
    done(unlocked([&] { return g_entry.cache_read(&c, ids, by, cols, from, B, total, type, to, to_scale, stream); }),
         "fp8_mqa_cache_read");
    if (!scales.defined()) return THPVariable_Wrap(std::move(out));
    return Py_BuildValue("(NN)", THPVariable_Wrap(std::move(out)), THPVariable_Wrap(std::move(scales)));
}

// q, data, scale, w, table, lens, max_len, out, clean_logits
PyObject* logits_paged(PyObject* const* a, Py_ssize_t n)
{
    expect(n, 9);
    const at::Tensor& q = cuda_tensor(a[0], "q");
    const c10::Device device = q.device();
    if (q.scalar_type() != at::kFloat8_e4m3fn || q.dim() != 4 || q.size(2) != kHeads || q.size(3) != kDim ||
        !q.is_contiguous())
        bad(PyExc_ValueError, "q must be contiguous float8_e4m3fn [B, T, 32, 128]");
    const int64_t B = q.size(0), T = q.size(1);
    const at::Tensor& w = cuda_tensor(a[3], "w", &device);
    if (w.scalar_type() != at::kFloat || w.dim() != 3 || w.size(0) != B || w.size(1) != T ||
        w.size(2) != kHeads || !w.is_contiguous())
        bad(PyExc_ValueError, "w must be contiguous float32 " + list({B, T, kHeads}));
    const fp8mqa_cache c = cache_of(a[1], a[2], "key", device);
    if (c.heads != 1 || c.dim != kDim) bad(PyExc_ValueError, "key data must be [pages, page_size, 1, 128]");
    const at::Tensor& table = ints(a[4], "table", device, 2, B);
    const at::Tensor& lens = ints(a[5], "lens", device, 1, B);
    const int32_t cols = int32_t(table.size(1));
    long long N = int64_t(cols) * c.page_size;
    if (a[6] != Py_None) {
        N = PyLong_AsLongLong(a[6]);
        if (N == -1 && PyErr_Occurred()) throw Raised{};
        if (N < 0) bad(PyExc_ValueError, "max_len must not be negative");
    }
    const int clean = PyObject_IsTrue(a[8]);
    if (clean < 0) throw Raised{};
    const c10::cuda::CUDAGuard guard(device);
    at::Tensor out;
    int64_t ld = N;
    if (a[7] == Py_None) {
        out = empty({B * T, N}, at::kFloat, device);
    } else {
        out = cuda_tensor(a[7], "out", &device);
        if (out.scalar_type() != at::kFloat || out.dim() != 2 || out.size(0) != B * T || out.size(1) != N ||
            (N > 1 && out.stride(1) != 1))
            bad(PyExc_ValueError, "out must be float32 " + list({B * T, N}) + " with contiguous rows");
        if (B * T > 1) ld = out.stride(0);
    }
    const auto* q_ptr = static_cast<const uint8_t*>(q.data_ptr());
    const auto* w_ptr = static_cast<const float*>(w.data_ptr());
    const auto* ids = static_cast<const int32_t*>(table.data_ptr());
    const auto* len = static_cast<const int32_t*>(lens.data_ptr());
    const int64_t by = table.stride(0);
    auto* to = static_cast<float*>(out.data_ptr());
    void* stream = current_stream(device);
    if (T > INT32_MAX) bad(PyExc_ValueError, "q has too many tokens");
    done(unlocked([&] {
             return g_entry.logits_paged(q_ptr, w_ptr, B, int32_t(T), kHeads, kDim, &c, ids, by, cols, len, to, ld,
                                         N, clean, stream);
         }),
         "fp8_mqa_logits_paged");
    if (a[7] != Py_None) {
        Py_INCREF(a[7]);
        return a[7];
    }
    return THPVariable_Wrap(std::move(out));
}

// q, k_data, v_data, table, lens, sm_scale, k_scale, v_scale, indices, return_lse
PyObject* attention_paged(PyObject* const* a, Py_ssize_t n)
{
    expect(n, 10);
    const at::Tensor& q = cuda_tensor(a[0], "q");
    const c10::Device device = q.device();
    const at::ScalarType dtype = q.scalar_type();
    if (dtype != at::kBFloat16 && dtype != at::kHalf)
        bad(PyExc_TypeError, "q must be bfloat16 or float16, got " + name_of(dtype));
    if (q.dim() != 3 || q.stride(2) != 1)
        bad(PyExc_ValueError, "q must be [B, q_heads, dim], contiguous in its last dimension");
    const int64_t B = q.size(0), heads = q.size(1), dim = q.size(2);
    const fp8mqa_cache k = cache_of(a[1], a[6], "k", device, dtype), v = cache_of(a[2], a[7], "v", device, dtype);
    if (k.pages != v.pages || k.page_size != v.page_size || k.heads != v.heads || k.dim != v.dim || k.type != v.type)
        bad(PyExc_ValueError, "k data and v data must have one shape and type");
    if (k.dim != dim || heads == 0 || heads > INT32_MAX || k.heads == 0 || heads % k.heads != 0)
        bad(PyExc_ValueError, "q " + list(q.sizes()) + " does not go with a cache of " +
                                  list({k.pages, k.page_size, k.heads, k.dim}));
    const at::Tensor& table = ints(a[3], "table", device, 2, B);
    const at::Tensor& lens = ints(a[4], "lens", device, 1, B);
    const int32_t* indices = nullptr;
    int64_t indices_by = 0;
    int32_t n_indices = -1;
    if (a[8] != Py_None) {
        const at::Tensor& t = ints(a[8], "indices", device, 2, B);
        indices = static_cast<const int32_t*>(t.data_ptr());
        indices_by = t.stride(0);
        n_indices = int32_t(t.size(1));
    }
    double scale = 1.0 / std::sqrt(double(dim));
    if (a[5] != Py_None) {
        scale = PyFloat_AsDouble(a[5]);
        if (scale == -1.0 && PyErr_Occurred()) throw Raised{};
    }
    const int want_lse = PyObject_IsTrue(a[9]);
    if (want_lse < 0) throw Raised{};
    const c10::cuda::CUDAGuard guard(device);
    at::Tensor out = empty({B, heads, dim}, dtype, device), lse;
    if (want_lse) lse = empty({B, heads}, at::kFloat, device);
    const uint64_t bytes = g_entry.workspace_bytes(int32_t(heads), k.heads, k.dim);
    const at::Tensor space = empty({int64_t(bytes)}, at::kByte, device);
    const void* q_ptr = q.data_ptr();
    const int64_t q_row = q.stride(0), q_head = q.stride(1), by = table.stride(0);
    const auto* ids = static_cast<const int32_t*>(table.data_ptr());
    const auto* len = static_cast<const int32_t*>(lens.data_ptr());
    const int32_t cols = int32_t(table.size(1)), type = type_of(dtype);
    void *to = out.data_ptr(), *space_ptr = space.data_ptr(), *stream = current_stream(device);
    float* lse_ptr = lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr;
    done(unlocked([&] {
             return g_entry.attention_paged(q_ptr, type, B, int32_t(heads), q_row, q_head, &k, &v, ids, by, cols,
                                            len, indices, indices_by, n_indices, float(scale), to, lse_ptr,
                                            space_ptr, bytes, stream);
         }),
         "fp8_mqa_attention_paged");
    if (!lse.defined()) return THPVariable_Wrap(std::move(out));
    return Py_BuildValue("(NN)", THPVariable_Wrap(std::move(out)), THPVariable_Wrap(std::move(lse)));
}

// The entry points' addresses (cache_write, cache_read, logits_paged, workspace_bytes,
// attention_paged) and the error class.
PyObject* bind(PyObject* const* a, Py_ssize_t n)
{
    if (n != 6) bad(PyExc_TypeError, "wrong number of arguments");
    void* p[5];
    for (int i = 0; i < 5; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null entry point");
            throw Raised{};
        }
    }
    Py_INCREF(a[5]);
    Py_XDECREF(g_error);
    g_error = a[5];
    g_entry.cache_write = reinterpret_cast<decltype(g_entry.cache_write)>(p[0]);
    g_entry.cache_read = reinterpret_cast<decltype(g_entry.cache_read)>(p[1]);
    g_entry.logits_paged = reinterpret_cast<decltype(g_entry.logits_paged)>(p[2]);
    g_entry.workspace_bytes = reinterpret_cast<decltype(g_entry.workspace_bytes)>(p[3]);
    g_entry.attention_paged = reinterpret_cast<decltype(g_entry.attention_paged)>(p[4]);
    Py_RETURN_NONE;
}

// No C++ exception leaves a function of this module: torch's become its Python errors.
template <PyObject* (*kFunction)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    try {
        return kFunction(args, n);
    } catch (const Raised&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

template <PyObject* (*kFunction)(PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&guarded<kFunction>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<cache_write>("cache_write"), method<cache_read>("cache_read"),
                           method<logits_paged>("logits_paged"), method<attention_paged>("attention_paged"),
                           method<bind>("bind"), {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_paged_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_binding() { return PyModule_Create(&g_module); }
