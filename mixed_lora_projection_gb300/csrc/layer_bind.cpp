// Python's side of the operators between the projections: reads tensors, allocates outputs and calls
// the C entry points of lora_layer.h, whose addresses layer.py hands over once.
//
// A step of decode calls these every few microseconds of GPU work, so the marshalling is native. Host time of a
// call with its outputs allocated, against the same checks in Python through ctypes (one core of Grace): norm of
// 48 rows 4.2 and 15.3 us, in 8 bits by groups 5.0 and 20.6, append of 48 rows 3.7 and 20.9, attention of one row
// 6.2 and 19.5.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <vector>

#include "lora_layer.h"

namespace {

decltype(&lora_linear_add_rms_norm) g_norm;
decltype(&lora_linear_kv_append) g_append;
decltype(&lora_linear_attn_forward) g_attend;
PyObject* g_check;                                     // (code, entry point) -> raises

constexpr auto kBf16 = at::kBFloat16;
constexpr auto kFp8 = at::kFloat8_e4m3fn;

const at::Tensor& tensor(PyObject* o, const char* name) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
    return THPVariable_Unpack(o);
}
const at::Tensor& cuda_tensor(PyObject* o, const char* name) {
    const at::Tensor& t = tensor(o, name);
    TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA tensor");
    return t;
}
void* pointer(const at::Tensor& t, at::ScalarType dtype, at::Device device, const char* name) {
    TORCH_CHECK_TYPE(t.scalar_type() == dtype, name, " must be ", dtype, ", got ", t.scalar_type());
    TORCH_CHECK_VALUE(t.device() == device, name, " must be on ", device, ", is on ", t.device());
    return t.data_ptr();
}
struct Rows {
    void* p = nullptr;
    int64_t stride = 0;
};
// [rows, width] with contiguous rows.
Rows rows_of(const at::Tensor& t, int64_t rows, int64_t width, at::ScalarType dtype, at::Device device, const char* name) {
    void* p = pointer(t, dtype, device, name);
    TORCH_CHECK_VALUE(t.dim() == 2 && t.size(0) == rows && t.size(1) == width, name, " must have shape [", rows, ", ", width, "], has ",
                      t.sizes());
    TORCH_CHECK_VALUE(t.stride(1) == 1 || width <= 1, name, "'s rows must be contiguous");
    return {p, rows > 1 ? t.stride(0) : width};
}
struct Heads {
    void* p = nullptr;
    int64_t stride = 0, head = 0;
};
// [rows, heads, dim] with contiguous features.
Heads heads_of(const at::Tensor& t, int64_t heads, int64_t dim, at::Device device, const char* name) {
    void* p = pointer(t, kBf16, device, name);
    TORCH_CHECK_VALUE(t.dim() == 3 && t.size(1) == heads && t.size(2) == dim, name, " must have shape [rows, ", heads, ", ", dim, "], has ",
                      t.sizes());
    TORCH_CHECK_VALUE(t.stride(2) == 1, name, "'s features must be contiguous");
    // an axis of one has no stride of its own
    return {p, t.size(0) > 1 ? t.stride(0) : std::max(t.stride(0), dim) / 8 * 8, heads > 1 ? t.stride(1) : dim};
}
// (through the dispatcher, at::empty, an output takes ~0.4 us more)
at::Tensor empty(at::IntArrayRef sizes, at::ScalarType dtype, at::Device device) {
    return at::Tensor(at::detail::empty_cuda(sizes, dtype, device, std::nullopt));
}
int to_int(PyObject* o, const char* name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    TORCH_CHECK_VALUE(v >= INT_MIN && v <= INT_MAX, name, " is out of range");
    return (int)v;
}
double to_double(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}
// The stream a call runs on: `o`, or the device's current one. A given stream is the current one while the call lasts,
// so that the outputs allocated in it come from that stream's memory: a block of another stream's may still be read by
// work queued there, and would go back to it when the output is dropped, whether or not this call has run.
struct OnStream {
    c10::cuda::OptionalCUDAStreamGuard guard;
    void* handle;
    OnStream(PyObject* o, at::Device device) {
        if (o == Py_None) {
            handle = c10::cuda::getCurrentCUDAStream(device.index()).stream();
            return;
        }
        static PyObject* const name = PyUnicode_InternFromString("cuda_stream");
        THPObjectPtr v(PyObject_GetAttr(o, name));
        if (!v) throw python_error();
        handle = PyLong_AsVoidPtr(v.get());
        if (!handle && PyErr_Occurred()) throw python_error();
        guard.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(handle), device.index()));
    }
};
template <class F>
int unlocked(F&& call) {                               // the call may wait for room in the stream's queue
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = call();
    Py_END_ALLOW_THREADS;
    return rc;
}
void check(int rc, const char* what) {
    if (rc == LORA_OK) return;
    THPObjectPtr r(PyObject_CallFunction(g_check, "is", rc, what));
    throw python_error();
}
void ready(Py_ssize_t n, Py_ssize_t want) {
    TORCH_CHECK(g_check, "not bound to the library");
    TORCH_CHECK_TYPE(n == want, "wrong number of arguments");
}
bool given(PyObject* o) { return o != Py_None; }
// A tensor of the caller's has been written: autograd's check of saved tensors goes by this count.
void wrote(const at::Tensor& t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
PyObject* same(PyObject* o) {
    Py_INCREF(o);
    return o;
}

// The caches [n_pages, page_size, n_kv_heads, head_dim] and the batch; q_offsets' values go to `offsets`.
lora_kv_cache cache_of(PyObject* k_cache, PyObject* v_cache, PyObject* q_offsets, PyObject* kv_lens, PyObject* block_table,
                       at::Device device, std::vector<int32_t>& offsets) {
    const at::Tensor &k = tensor(k_cache, "k_cache"), &v = tensor(v_cache, "v_cache");
    TORCH_CHECK_VALUE(k.dim() == 4 && v.sizes() == k.sizes(),
                      "k_cache and v_cache must both have shape [n_pages, page_size, n_kv_heads, head_dim]");
    lora_kv_cache c{};
    c.k = pointer(k, kBf16, device, "k_cache");
    c.v = pointer(v, kBf16, device, "v_cache");
    TORCH_CHECK_VALUE(k.stride(3) == 1 && v.stride(3) == 1, "the caches' features must be contiguous");
    for (int i = 0; i < 4; ++i) TORCH_CHECK_VALUE(k.size(i) <= INT_MAX, "the caches are too large");
    c.n_pages = (int)k.size(0);
    c.page_size = (int)k.size(1);
    c.n_kv_heads = (int)k.size(2);
    c.head_dim = (int)k.size(3);
    // an axis of one has no stride of its own
    c.k_page_stride = c.n_pages > 1 ? k.stride(0) : c.head_dim;
    c.v_page_stride = c.n_pages > 1 ? v.stride(0) : c.head_dim;
    c.k_token_stride = k.stride(1);
    c.v_token_stride = v.stride(1);
    c.k_head_stride = c.n_kv_heads > 1 ? k.stride(2) : c.head_dim;
    c.v_head_stride = c.n_kv_heads > 1 ? v.stride(2) : c.head_dim;
    const at::Tensor& table = tensor(block_table, "block_table");
    c.block_table = static_cast<const int32_t*>(pointer(table, at::kInt, device, "block_table"));
    TORCH_CHECK_VALUE(table.dim() == 2 && (table.stride(1) == 1 || table.size(1) <= 1) && table.size(0) <= INT_MAX && table.size(1) <= INT_MAX,
                      "block_table must have shape [n_seqs, pages_per_seq] with contiguous rows");
    c.n_seqs = (int)table.size(0);
    c.pages_per_seq = (int)table.size(1);
    c.table_stride = c.n_seqs > 1 ? table.stride(0) : c.pages_per_seq;
    const at::Tensor& lens = tensor(kv_lens, "kv_lens");
    c.kv_lens = static_cast<const int32_t*>(pointer(lens, at::kInt, device, "kv_lens"));
    TORCH_CHECK_VALUE(lens.dim() == 1 && lens.size(0) == c.n_seqs && (c.n_seqs <= 1 || lens.stride(0) == 1),
                      "kv_lens must be contiguous with shape (", c.n_seqs, ",)");
    THPObjectPtr seq(PySequence_Fast(q_offsets, "q_offsets must be a sequence of integers"));
    if (!seq) throw python_error();
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq.get());
    TORCH_CHECK_VALUE(n == c.n_seqs + 1, "q_offsets must hold one more entry than there are sequences");
    offsets.resize(n);
    for (Py_ssize_t i = 0; i < n; ++i) offsets[i] = to_int(PySequence_Fast_GET_ITEM(seq.get(), i), "q_offsets");
    c.q_offsets = offsets.data();
    return c;
}

void* address(PyObject* o) {
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw python_error();
    return p;
}

// bind(add_rms_norm, kv_append, attn_forward, check): addresses of the entry points, and what raises their errors
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    TORCH_CHECK_TYPE(n == 4, "wrong number of arguments");
    g_norm = reinterpret_cast<decltype(g_norm)>(address(a[0]));
    g_append = reinterpret_cast<decltype(g_append)>(address(a[1]));
    g_attend = reinterpret_cast<decltype(g_attend)>(address(a[2]));
    Py_XSETREF(g_check, same(a[3]));
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// norm(x, weight, residual, eps, weight_offset, out, h_out, scales, group, stream); group -1: bf16, (y, h);
// else 8 bits, (q, scales, h)
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    ready(n, 10);
    const at::Tensor& x = cuda_tensor(a[0], "x");
    const at::Device dev = x.device();
    const int group = to_int(a[8], "group");
    TORCH_CHECK_VALUE(x.dim() == 2, "x must have shape [rows, width]");
    const int64_t rows = x.size(0), width = x.size(1);
    TORCH_CHECK_VALUE(rows <= INT_MAX && width <= INT_MAX, "x is too large");
    const Rows xr = rows_of(x, rows, width, kBf16, dev, "x");
    const at::Tensor& weight = tensor(a[1], "weight");
    const void* const wp = pointer(weight, kBf16, dev, "weight");
    TORCH_CHECK_VALUE(weight.dim() == 1 && weight.size(0) == width && (weight.stride(0) == 1 || width <= 1),
                      "weight must be contiguous with shape (", width, ",)");
    Rows rr, hr, yr, qr;
    at::Tensor out, scales, h;
    const float eps = (float)to_double(a[3]), offset = (float)to_double(a[4]);
    if (given(a[2])) rr = rows_of(tensor(a[2], "residual"), rows, width, kBf16, dev, "residual");
    const c10::cuda::CUDAGuard guard(dev);
    const OnStream stream(a[9], dev);
    float* sp = nullptr;
    if (given(a[5])) out = tensor(a[5], "out");
    else out = empty({rows, width}, group < 0 ? kBf16 : kFp8, dev);
    if (group < 0) {
        yr = rows_of(out, rows, width, kBf16, dev, "out");
    } else {
        TORCH_CHECK_VALUE(group == 0 || group == 32 || group == 64 || group == 128 || group == 256, "group must be 0, 32, 64, 128 or 256");
        const int64_t per = group ? (width + group - 1) / group : 1;
        qr = rows_of(out, rows, width, kFp8, dev, "out");
        if (given(a[7])) {
            scales = tensor(a[7], "scales");
            TORCH_CHECK_VALUE(scales.dim() == 2 && scales.size(0) == rows && scales.size(1) == per && scales.is_contiguous(),
                              "scales must be contiguous with shape (", rows, ", ", per, ")");
        } else {
            scales = empty({rows, per}, at::kFloat, dev);
        }
        sp = static_cast<float*>(pointer(scales, at::kFloat, dev, "scales"));
    }
    if (given(a[6])) h = tensor(a[6], "h_out");
    else if (given(a[2]) || (yr.p == xr.p && rows)) h = empty({rows, width}, kBf16, dev);   // (y over x: h is x no more)
    if (h.defined()) hr = rows_of(h, rows, width, kBf16, dev, "h_out");
    check(unlocked([&] {
              return g_norm(xr.p, xr.stride, rr.p, rr.stride, wp, offset, eps, (int)rows, (int)width, hr.p, hr.stride, yr.p, yr.stride, qr.p,
                            qr.stride, sp, group < 0 ? 0 : group, stream.handle);
          }),
          "lora_linear_add_rms_norm");
    if (given(a[5])) wrote(out);
    if (given(a[6])) wrote(h);
    if (group >= 0 && given(a[7])) wrote(scales);
    THPObjectPtr o(given(a[5]) ? same(a[5]) : THPVariable_Wrap(out));
    THPObjectPtr hh(given(a[6]) ? same(a[6]) : h.defined() ? THPVariable_Wrap(h) : same(a[0]));
    if (group < 0) return PyTuple_Pack(2, o.get(), hh.get());
    THPObjectPtr s(given(a[7]) ? same(a[7]) : THPVariable_Wrap(scales));
    return PyTuple_Pack(3, o.get(), s.get(), hh.get());
    END_HANDLE_TH_ERRORS
}

// append(q, k, v, q_offsets, kv_lens, block_table, k_cache, v_cache, cos, sin, q_out, stream) -> q_out
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    ready(n, 12);
    TORCH_CHECK_VALUE(given(a[0]) || !given(a[10]), "q_out goes with q");
    const at::Tensor &k = cuda_tensor(a[1], "k"), &v = tensor(a[2], "v");
    const at::Device dev = k.device();
    std::vector<int32_t> offsets;
    const lora_kv_cache c = cache_of(a[6], a[7], a[3], a[4], a[5], dev, offsets);
    const int64_t T = offsets.back();
    int rot = 0, positions = 0;
    const float *cp = nullptr, *sp = nullptr;
    TORCH_CHECK_VALUE(given(a[8]) == given(a[9]), "cos and sin go together");
    if (given(a[8])) {
        const at::Tensor &cos = tensor(a[8], "cos"), &sin = tensor(a[9], "sin");
        TORCH_CHECK_VALUE(cos.dim() == 2 && cos.sizes() == sin.sizes() && cos.is_contiguous() && sin.is_contiguous() &&
                              cos.size(0) <= INT_MAX && cos.size(1) <= INT_MAX / 2,
                          "cos and sin must be contiguous and have one shape [n_positions, rot / 2]");
        positions = (int)cos.size(0);
        rot = 2 * (int)cos.size(1);
        cp = static_cast<const float*>(pointer(cos, at::kFloat, dev, "cos"));
        sp = static_cast<const float*>(pointer(sin, at::kFloat, dev, "sin"));
    }
    const Heads kr = heads_of(k, c.n_kv_heads, c.head_dim, dev, "k"), vr = heads_of(v, c.n_kv_heads, c.head_dim, dev, "v");
    TORCH_CHECK_VALUE(k.size(0) == T && v.size(0) == T && (!given(a[0]) || (tensor(a[0], "q").dim() == 3 && tensor(a[0], "q").size(0) == T)),
                      "q, k and v must have q_offsets[-1] rows");
    Heads qr, orr;
    int heads = 0;
    const c10::cuda::CUDAGuard guard(dev);
    const OnStream stream(a[11], dev);
    THPObjectPtr out(same(given(a[10]) ? a[10] : a[0]));
    if (given(a[0]) && (rot || given(a[10]))) {
        const at::Tensor& q = tensor(a[0], "q");
        heads = (int)q.size(1);
        qr = heads_of(q, heads, c.head_dim, dev, "q");
        if (!given(a[10])) out = THPVariable_Wrap(empty(q.sizes(), kBf16, dev));
        const at::Tensor& o = tensor(out.get(), "q_out");
        TORCH_CHECK_VALUE(o.sizes() == q.sizes(), "q_out must have q's shape");
        orr = heads_of(o, heads, c.head_dim, dev, "q_out");
    }
    check(unlocked([&] {
              return g_append(&c, qr.p, qr.stride, qr.head, orr.p, orr.stride, orr.head, heads, kr.p, kr.stride, kr.head, vr.p, vr.stride,
                              vr.head, cp, sp, rot, positions, stream.handle);
          }),
          "lora_linear_kv_append");
    wrote(tensor(a[6], "k_cache"));
    wrote(tensor(a[7], "v_cache"));
    if (given(a[10])) wrote(tensor(a[10], "q_out"));
    return out.release();
    END_HANDLE_TH_ERRORS
}

// attend(handle, n_heads, head_dim, device, q, k_cache, v_cache, q_offsets, kv_lens, block_table, scale, window, sinks,
// out, stream) -> out
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    ready(n, 15);
    lora_attn* const handle = static_cast<lora_attn*>(given(a[0]) ? address(a[0]) : nullptr);
    const int heads = to_int(a[1], "n_heads"), dim = to_int(a[2], "head_dim");
    const at::Device dev(at::kCUDA, (c10::DeviceIndex)to_int(a[3], "device"));
    const at::Tensor& q = tensor(a[4], "q");
    std::vector<int32_t> offsets;
    const lora_kv_cache c = cache_of(a[5], a[6], a[7], a[8], a[9], dev, offsets);
    TORCH_CHECK_VALUE(q.dim() == 3 && q.size(0) == offsets.back(), "q must have q_offsets[-1] rows");
    const Heads qr = heads_of(q, heads, dim, dev, "q");
    const float scale = given(a[10]) ? (float)to_double(a[10]) : (float)(1.0 / std::sqrt((double)dim));
    const int window = to_int(a[11], "window"), sinks = to_int(a[12], "sinks");
    const OnStream stream(a[14], dev);
    THPObjectPtr out(given(a[13]) ? same(a[13]) : THPVariable_Wrap(empty(q.sizes(), kBf16, dev)));
    const at::Tensor& o = tensor(out.get(), "out");
    TORCH_CHECK_VALUE(o.sizes() == q.sizes(), "out must have q's shape");
    const Heads orr = heads_of(o, heads, dim, dev, "out");
    check(unlocked([&] {
              return g_attend(handle, &c, qr.p, qr.stride, qr.head, orr.p, orr.stride, orr.head, scale, window, sinks, stream.handle);
          }),
          "lora_linear_attn_forward");
    if (given(a[13])) wrote(o);
    return out.release();
    END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(F));
}
PyMethodDef methods[] = {{"bind", fast<bind>(), METH_FASTCALL, nullptr},
                         {"norm", fast<norm>(), METH_FASTCALL, nullptr},
                         {"append", fast<append>(), METH_FASTCALL, nullptr},
                         {"attend", fast<attend>(), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layer_bind() {
    PyObject* const m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", LAYER_BIND_FOR) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
