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
#include "overlap.h"

namespace {

struct Raised {};  // a Python error is set

struct Entries {
    decltype(&fp8_mqa_cache_write) cache_write = nullptr;
    decltype(&fp8_mqa_cache_read) cache_read = nullptr;
    decltype(&fp8_mqa_logits_paged) logits_paged = nullptr;
    decltype(&fp8_mqa_attention_paged_workspace_bytes) workspace_bytes = nullptr;
    decltype(&fp8_mqa_attention_paged) attention_paged = nullptr;
    decltype(&fp8_mqa_pages_update) pages_update = nullptr;
    decltype(&fp8_mqa_norm_rotate) norm_rotate = nullptr;
} g_entry;

PyObject* g_error = nullptr;     // Fp8MqaError
PyTypeObject* g_step = nullptr;  // PagesStep, a tuple of five

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
        case at::ScalarType::Float4_e2m1fn_x2: return FP8MQA_E2M1;
        default: return -1;
    }
}

// A cache of e4m3 data and its scales, of e2m1 data (unless groups_o is NULL, where such caches are not taken) with
// its groups' scales too, or of the type `other` without.
fp8mqa_cache cache_of(PyObject* data_o, PyObject* scale_o, PyObject* groups_o, const char* name,
                      const c10::Device& device, at::ScalarType other = at::kFloat8_e4m3fn)
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
    c.type = type_of(dtype);
    const bool four = c.type == FP8MQA_E2M1 && groups_o;
    // two values an element
    if (four && data.size(3) > INT32_MAX / 2)
        bad(PyExc_ValueError, what + " data is too large: " + list(data.sizes()));
    c.dim = int32_t(data.size(3)) * (four ? 2 : 1);
    c.page_stride = data.stride(0);
    c.row_stride = data.stride(1);
    c.head_stride = data.stride(2);
    c.scale_page_stride = c.scale_row_stride = c.scale_head_stride = 0;
    c.groups = nullptr;
    c.group_page_stride = c.group_row_stride = c.group_head_stride = 0;
    if (!four && dtype != at::kFloat8_e4m3fn && dtype != other)
        bad(PyExc_TypeError, what + " data must be " + name_of(at::kFloat8_e4m3fn) +
                                 (groups_o ? ", torch.float4_e2m1fn_x2" : "") +
                                 (other == at::kFloat8_e4m3fn ? "" : " or " + name_of(other)) + ", got " + name_of(dtype));
    if (!four && groups_o && groups_o != Py_None)
        bad(PyExc_ValueError, what + " groups go with float4_e2m1fn_x2 data only");
    if (four) {
        const at::Tensor& groups = cuda_tensor(groups_o, (what + " groups").c_str(), &device);
        if (groups.scalar_type() != at::kFloat8_e4m3fn || groups.dim() != 4 || groups.size(0) != data.size(0) ||
            groups.size(1) != data.size(1) || groups.size(2) != data.size(2) || groups.size(3) != c.dim / 16)
            bad(PyExc_ValueError, what + " groups must be float8_e4m3fn " +
                                      list({data.size(0), data.size(1), data.size(2), c.dim / 16}));
        if (groups.size(3) > 1 && groups.stride(3) != 1)
            bad(PyExc_ValueError, what + " groups must be contiguous in their last dimension");
        c.groups = static_cast<uint8_t*>(groups.data_ptr());
        c.group_page_stride = groups.stride(0);
        c.group_row_stride = groups.stride(1);
        c.group_head_stride = groups.stride(2);
    }
    if (dtype == at::kFloat8_e4m3fn || four) {
        const at::Tensor& scale = cuda_tensor(scale_o, (what + " scale").c_str(), &device);
        if (scale.scalar_type() != at::kFloat || scale.dim() != 3 || scale.size(0) != data.size(0) ||
            scale.size(1) != data.size(1) || scale.size(2) != data.size(2))
            bad(PyExc_ValueError, what + " scale must be float32 " + list(data.sizes().slice(0, 3)));
        c.scale = static_cast<float*>(scale.data_ptr());
        c.scale_page_stride = scale.stride(0);
        c.scale_row_stride = scale.stride(1);
        c.scale_head_stride = scale.stride(2);
    } else {
        if (scale_o != Py_None) bad(PyExc_ValueError, what + " scale goes with float8_e4m3fn" +
                                                   std::string(groups_o ? " or float4_e2m1fn_x2" : "") + " data only");
    }
    return c;
}

at::Tensor empty(c10::IntArrayRef sizes, at::ScalarType type, const c10::Device& device)
{
    return at::empty(sizes, at::TensorOptions().dtype(type).device(device));
}

// n elements of a one-dimensional tensor, from `from` on.
at::Tensor part_of(const at::Tensor& base, int64_t from, int64_t n)
{
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::TensorImpl::VIEW, c10::Storage(base.storage()),
                                                            base.key_set(), base.dtype());
    t.unsafeGetTensorImpl()->set_storage_offset(from);
    t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
    return t;
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

// slots, k, k_data, k_scale, v, v_data, v_scale, k_groups, v_groups
PyObject* cache_write(PyObject* const* a, Py_ssize_t n)
{
    expect(n, 9);
    const c10::Device device = cuda_tensor(a[2], "k data").device();
    const fp8mqa_cache ck = cache_of(a[2], a[3], a[7], "k", device);
    const at::Tensor& slots = ints(a[0], "slots", device, 1, -1);
    const bool pair = a[4] != Py_None;
    if (pair != (a[5] != Py_None) || pair != (a[6] != Py_None) || (!pair && a[8] != Py_None))
        bad(PyExc_ValueError, "v, v_data and v_scale go together");
    auto rows = [&](PyObject* o, const char* name, const at::Tensor* like) -> const at::Tensor& {
        const at::Tensor& x = cuda_tensor(o, name, &device);
        const int32_t type = type_of(x.scalar_type());
        if (type < 0 || type == FP8MQA_E4M3 || type == FP8MQA_E2M1 || (like && x.scalar_type() != like->scalar_type()))
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
        cv = cache_of(a[5], a[6], a[8], "v", device);
        if (cv.type != ck.type) bad(PyExc_TypeError, "v data must be of k data's type");
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

// data, scale, table, starts, total, dtype, groups
PyObject* cache_read(PyObject* const* a, Py_ssize_t n)
{
    expect(n, 7);
    const c10::Device device = cuda_tensor(a[0], "data").device();
    const fp8mqa_cache c = cache_of(a[0], a[1], a[6], "cache", device);
    const at::Tensor& table = ints(a[2], "table", device, 2, -1);
    const at::Tensor& starts = ints(a[3], "starts", device, 1, table.size(0) + 1);
    const int32_t type = THPDtype_Check(a[5]) ? type_of(reinterpret_cast<THPDtype*>(a[5])->scalar_type) : -1;
    if (type < 0 || type == FP8MQA_E2M1 || (type == FP8MQA_E4M3 && c.type == FP8MQA_E2M1))
        bad(PyExc_TypeError, c.type == FP8MQA_E2M1
                                 ? "dtype must be bfloat16, float16 or float32 for a cache in 4 bits"
                                 : "dtype must be float8_e4m3fn, bfloat16, float16 or float32");
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
    const fp8mqa_cache c = cache_of(a[1], a[2], nullptr, "key", device);
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

// q, k_data, v_data, table, lens, sm_scale, k_scale, v_scale, indices, return_lse, k_groups, v_groups
PyObject* attention_paged(PyObject* const* a, Py_ssize_t n)
{
    expect(n, 12);
    const at::Tensor& q = cuda_tensor(a[0], "q");
    const c10::Device device = q.device();
    const at::ScalarType dtype = q.scalar_type();
    if (dtype != at::kBFloat16 && dtype != at::kHalf)
        bad(PyExc_TypeError, "q must be bfloat16 or float16, got " + name_of(dtype));
    if (q.dim() != 3 || q.stride(2) != 1)
        bad(PyExc_ValueError, "q must be [B, q_heads, dim], contiguous in its last dimension");
    const int64_t B = q.size(0), heads = q.size(1), dim = q.size(2);
    const fp8mqa_cache k = cache_of(a[1], a[6], a[10], "k", device, dtype),
                       v = cache_of(a[2], a[7], a[11], "v", device, dtype);
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

// table, lens, change, free, n_free, page_size, total
PyObject* pages_update(PyObject* const* a, Py_ssize_t n)
{
    expect(n, 7);
    const c10::Device device = cuda_tensor(a[0], "table").device();
    const at::Tensor& table = ints(a[0], "table", device, 2, -1);
    const int64_t B = table.size(0), cols = table.size(1);
    const at::Tensor& lens = ints(a[1], "lens", device, 1, B);
    const at::Tensor& change = ints(a[2], "change", device, 1, B);
    const at::Tensor& pool = ints(a[3], "free", device, 1, -1);
    const at::Tensor& n_free = ints(a[4], "n_free", device, 1, 1);
    const long long page = PyLong_AsLongLong(a[5]);
    if (page == -1 && PyErr_Occurred()) throw Raised{};
    const long long total = PyLong_AsLongLong(a[6]);
    if (total == -1 && PyErr_Occurred()) throw Raised{};
    if (page < 1 || page > INT32_MAX) bad(PyExc_ValueError, "page_size must be 1 or more");
    if (total < 0 || total > INT32_MAX) bad(PyExc_ValueError, "total must be 0 or more, and under 2^31");
    if (B > 1 && table.stride(0) < cols) bad(PyExc_ValueError, "the rows of table must not overlap: they are written");
    const c10::cuda::CUDAGuard guard(device);
    // one allocation for the five results, each on 16 bytes: five of them took half of the call
    const int64_t size[5] = {total, total, total, B + 1, B};
    int64_t at[6] = {0};
    for (int i = 0; i < 5; ++i) at[i + 1] = at[i] + (size[i] + 3) / 4 * 4;
    const at::Tensor base = empty({at[5]}, at::kInt, device);
    at::Tensor out[5];
    int32_t* to[5];
    for (int i = 0; i < 5; ++i) {
        out[i] = part_of(base, at[i], size[i]);
        to[i] = static_cast<int32_t*>(base.data_ptr()) + at[i];
    }
    auto *ids = static_cast<int32_t*>(table.data_ptr()), *len = static_cast<int32_t*>(lens.data_ptr());
    auto *stack = static_cast<int32_t*>(pool.data_ptr()), *height = static_cast<int32_t*>(n_free.data_ptr());
    const auto* by = static_cast<const int32_t*>(change.data_ptr());
    const int64_t pitch = table.stride(0), capacity = pool.size(0);
    void* stream = current_stream(device);
    done(unlocked([&] {
             return g_entry.pages_update(ids, pitch, int32_t(cols), int32_t(page), len, by, B, stack, capacity, height,
                                         total, to[0], to[1], to[2], to[3], to[4], stream);
         }),
         "fp8_mqa_pages_update");
    PyObject* const result = g_step->tp_alloc(g_step, 5);  // a kind of tuple
    if (!result) throw Raised{};
    for (int i = 0; i < 5; ++i) PyTuple_SET_ITEM(result, i, THPVariable_Wrap(std::move(out[i])));
    return result;
}

// The bytes of rows [T, heads, dim], and of a contiguous tensor.
fp8mqa::Places rows_of(const at::Tensor& t)
{
    const int64_t e = t.element_size();
    return {t.data_ptr(), t.size(0), t.stride(0) * e, t.size(1), t.stride(1) * e, t.size(2) * e};
}
fp8mqa::Places all_of(const at::Tensor& t) { return fp8mqa::bytes_at(t.data_ptr(), int64_t(t.nbytes())); }

// q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, dtype, q_out, k_out
PyObject* norm_rotate(PyObject* const* a, Py_ssize_t n)
{
    expect(n, 11);
    const at::Tensor& q = cuda_tensor(a[0], "q");
    const c10::Device device = q.device();
    const at::ScalarType type = q.scalar_type();
    if (type != at::kBFloat16 && type != at::kHalf && type != at::kFloat)
        bad(PyExc_TypeError, "q must be bfloat16, float16 or float32, got " + name_of(type));
    at::ScalarType to = type;
    if (a[8] != Py_None) {
        to = THPDtype_Check(a[8]) ? reinterpret_cast<THPDtype*>(a[8])->scalar_type : at::kByte;
        if (to != type && to != at::kFloat8_e4m3fn)
            bad(PyExc_TypeError, "dtype must be float8_e4m3fn or q's, " + name_of(type));
    }
    const bool e4m3 = to == at::kFloat8_e4m3fn;
    if (q.dim() != 3) bad(PyExc_ValueError, "q must be [T, heads, dim], got " + list(q.sizes()));
    const int64_t T = q.size(0), dim = q.size(2);
    if (dim != 64 && dim != 128) bad(PyExc_ValueError, "q must have heads of 64 or 128 values, got " + list(q.sizes()));
    const at::Tensor& positions = cuda_tensor(a[2], "positions", &device);
    if (positions.scalar_type() != at::kInt && positions.scalar_type() != at::kLong)
        bad(PyExc_TypeError, "positions must be int32 or int64, got " + name_of(positions.scalar_type()));
    if (positions.dim() != 1 || positions.size(0) != T || (T > 1 && positions.stride(0) != 1))
        bad(PyExc_ValueError, "positions must be contiguous " + list({T}) + ", got " + list(positions.sizes()));
    const at::Tensor& freq = cuda_tensor(a[3], "inv_freq", &device);
    if (freq.scalar_type() != at::kFloat) bad(PyExc_TypeError, "inv_freq must be float32, got " + name_of(freq.scalar_type()));
    if (freq.dim() != 1 || !freq.is_contiguous() || 2 * freq.size(0) > dim || freq.size(0) % 8 != 0)
        bad(PyExc_ValueError, "inv_freq must be contiguous, a multiple of 8 and at most dim / 2 frequencies, got " +
                                  list(freq.sizes()));
    const double eps = PyFloat_AsDouble(a[6]);
    if (eps == -1.0 && PyErr_Occurred()) throw Raised{};
    const int interleaved = PyObject_IsTrue(a[7]);
    if (interleaved < 0) throw Raised{};
    const c10::cuda::CUDAGuard guard(device);
    fp8mqa_heads heads[2] = {};
    at::Tensor out[2], scale[2];
    PyObject* given[2] = {nullptr, nullptr};
    for (int i = 0; i < 2; ++i) {
        const std::string name(i ? "k" : "q");
        if (i && a[1] == Py_None) {
            if (a[5] != Py_None || a[10] != Py_None) bad(PyExc_ValueError, "k_weight and k_out go with k");
            continue;
        }
        const at::Tensor& x = cuda_tensor(a[i], name.c_str(), &device);
        if (x.scalar_type() != type) bad(PyExc_TypeError, "k must be " + name_of(type) + " as q is, got " + name_of(x.scalar_type()));
        if (x.dim() != 3 || x.size(0) != T || x.size(2) != dim || x.size(1) > INT32_MAX)
            bad(PyExc_ValueError, name + " must be " + list({T, x.dim() == 3 ? x.size(1) : 1, dim}) + ", got " + list(x.sizes()));
        if (x.stride(2) != 1) bad(PyExc_ValueError, name + " must be contiguous in its last dimension");
        fp8mqa_heads& h = heads[i];
        h.x = x.data_ptr();
        h.row_stride = x.stride(0);
        h.head_stride = x.stride(1);
        h.heads = int32_t(x.size(1));
        h.weight_type = type_of(type);
        if (a[4 + i] != Py_None) {
            const at::Tensor& w = cuda_tensor(a[4 + i], (name + "_weight").c_str(), &device);
            if (w.scalar_type() != type && w.scalar_type() != at::kFloat)
                bad(PyExc_TypeError, name + "_weight must be " + name_of(type) + " or torch.float32, got " + name_of(w.scalar_type()));
            if (w.dim() != 1 || w.size(0) != dim || w.stride(0) != 1)
                bad(PyExc_ValueError, name + "_weight must be contiguous " + list({dim}) + ", got " + list(w.sizes()));
            h.weight = w.data_ptr();
            h.weight_type = type_of(w.scalar_type());
        }
        if (a[9 + i] != Py_None) {
            const at::Tensor& o = cuda_tensor(a[9 + i], (name + "_out").c_str(), &device);
            if (e4m3) bad(PyExc_ValueError, name + "_out does not go with float8_e4m3fn results");
            if (o.scalar_type() != type || o.dim() != 3 || o.size(0) != T || o.size(1) != x.size(1) || o.size(2) != dim ||
                o.stride(2) != 1)
                bad(PyExc_ValueError, name + "_out must be " + name_of(type) + " " + list(x.sizes()) +
                                          ", contiguous in its last dimension");
            // written: no two rows may overlap
            if (!fp8mqa::apart(rows_of(o))) bad(PyExc_ValueError, name + "_out must not overlap");
            given[i] = a[9 + i];
            h.out = o.data_ptr();
            h.out_row_stride = o.stride(0);
            h.out_head_stride = o.stride(1);
        } else {
            out[i] = empty({T, x.size(1), dim}, to, device);
            h.out = out[i].data_ptr();
            h.out_row_stride = out[i].stride(0);
            h.out_head_stride = out[i].stride(1);
            if (e4m3) {
                scale[i] = empty({T, x.size(1)}, at::kFloat, device);
                h.out_scale = static_cast<float*>(scale[i].data_ptr());
            }
        }
    }
    // written: a result may take the place of its own rows, and else overlaps nothing of the call
    for (int i = 0; i < 2; ++i) {
        if (!given[i]) continue;
        const fp8mqa::Places to = rows_of(THPVariable_Unpack(given[i]));
        auto with = [&](bool overlaps, const char* what) {
            if (overlaps) bad(PyExc_ValueError, std::string(i ? "k" : "q") + "_out must not overlap " + what);
        };
        for (int j = 0; j < 2; ++j) {
            if (j && a[1] == Py_None) continue;
            const fp8mqa::Places x = rows_of(THPVariable_Unpack(a[j]));
            with(!(i == j && fp8mqa::same_places(to, x)) && fp8mqa::meet(to, x),
                 i != j ? (j ? "k" : "q") : i ? "k unless it is k" : "q unless it is q");
            if (a[4 + j] != Py_None) with(fp8mqa::meet(to, all_of(THPVariable_Unpack(a[4 + j]))), j ? "k_weight" : "q_weight");
        }
        if (i && given[0]) with(fp8mqa::meet(to, rows_of(THPVariable_Unpack(given[0]))), "q_out");
        with(fp8mqa::meet(to, all_of(positions)), "positions");
        with(fp8mqa::meet(to, all_of(freq)), "inv_freq");
    }
    const void* pos = positions.data_ptr();
    const auto* f = static_cast<const float*>(freq.data_ptr());
    const int32_t wide = positions.scalar_type() == at::kLong ? 8 : 4, rotated = int32_t(2 * freq.size(0));
    void* stream = current_stream(device);
    done(unlocked([&] {
             return g_entry.norm_rotate(&heads[0], a[1] == Py_None ? nullptr : &heads[1], type_of(type), type_of(to), T,
                                        int32_t(dim), pos, wide, f, rotated, interleaved, float(eps), stream);
         }),
         "fp8_mqa_norm_rotate");
    PyObject* result[2];
    for (int i = 0; i < 2; ++i) {
        if (given[i]) {
            Py_INCREF(given[i]);
            result[i] = given[i];
        } else if (!out[i].defined()) {
            Py_INCREF(Py_None);
            result[i] = Py_None;
        } else {
            result[i] = THPVariable_Wrap(std::move(out[i]));
            if (e4m3) result[i] = Py_BuildValue("(NN)", result[i], THPVariable_Wrap(std::move(scale[i])));
        }
    }
    return Py_BuildValue("(NN)", result[0], result[1]);
}

// The entry points' addresses (cache_write, cache_read, logits_paged, workspace_bytes,
// attention_paged, pages_update, norm_rotate), the error class and the type of a step's result.
PyObject* bind(PyObject* const* a, Py_ssize_t n)
{
    if (n != 9) bad(PyExc_TypeError, "wrong number of arguments");
    void* p[7];
    for (int i = 0; i < 7; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null entry point");
            throw Raised{};
        }
    }
    Py_INCREF(a[7]);
    Py_XDECREF(g_error);
    g_error = a[7];
    if (!PyType_Check(a[8]) || !PyType_IsSubtype(reinterpret_cast<PyTypeObject*>(a[8]), &PyTuple_Type))
        bad(PyExc_TypeError, "the step's type must be a kind of tuple");
    Py_INCREF(a[8]);
    Py_XDECREF(reinterpret_cast<PyObject*>(g_step));
    g_step = reinterpret_cast<PyTypeObject*>(a[8]);
    g_entry.cache_write = reinterpret_cast<decltype(g_entry.cache_write)>(p[0]);
    g_entry.cache_read = reinterpret_cast<decltype(g_entry.cache_read)>(p[1]);
    g_entry.logits_paged = reinterpret_cast<decltype(g_entry.logits_paged)>(p[2]);
    g_entry.workspace_bytes = reinterpret_cast<decltype(g_entry.workspace_bytes)>(p[3]);
    g_entry.attention_paged = reinterpret_cast<decltype(g_entry.attention_paged)>(p[4]);
    g_entry.pages_update = reinterpret_cast<decltype(g_entry.pages_update)>(p[5]);
    g_entry.norm_rotate = reinterpret_cast<decltype(g_entry.norm_rotate)>(p[6]);
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
                           method<pages_update>("pages_update"), method<norm_rotate>("norm_rotate"),
                           method<bind>("bind"), {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_paged_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_binding() { return PyModule_Create(&g_module); }
