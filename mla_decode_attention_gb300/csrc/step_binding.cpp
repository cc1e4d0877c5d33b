// Python module `_step`: argument checks and marshalling of the calls that a
// serving loop makes for every layer and step (mla_append_kv,
// mla_query_norm_rope, mla_window_decode).  They run for a few microseconds on
// the GPU, and the same checks written in Python took longer than that (9 to 12
// us a call in all on the Grace host, 3 so).  Each function returns the
// status of the C function of the same name; a wrong tensor raises ValueError
// before anything is launched.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>

#include "mla_decode.h"

namespace {

struct Refused {};  // a Python error is set

[[noreturn]] void refuse(const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(PyExc_ValueError, format, args);
  va_end(args);
  throw Refused();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse("%s must be a tensor", name);
  return THPVariable_Unpack(o);
}

int device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse("%s must be on a CUDA device", name);
  return t.get_device();
}

void on(const at::Tensor& t, int device, const char* name) {
  if (!t.is_cuda() || t.get_device() != device) refuse("%s must be on device %d", name, device);
}

// Data of a contiguous tensor of n values; None is NULL where it may be left out.
void* vector(PyObject* o, at::ScalarType type, int64_t n, const char* name, int device, bool optional = false) {
  if (o == Py_None && optional) return nullptr;
  const at::Tensor& t = tensor(o, name);
  on(t, device, name);
  if (t.scalar_type() != type || t.numel() != n || !t.is_contiguous())
    refuse("%s must be a contiguous %s tensor of %lld values", name, c10::toString(type), static_cast<long long>(n));
  return t.data_ptr();
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}
int narrow(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v != static_cast<int>(v)) refuse("%s does not fit 32 bits", name);
  return static_cast<int>(v);
}
// Sizes of a tensor as the C functions take them (they refuse what is too large).
int size(int64_t v) { return v > INT32_MAX ? INT32_MAX : static_cast<int>(v); }
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return static_cast<float>(v);
}

cudaStream_t stream_of(PyObject* o, int device) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(device).stream();
  PyObject* raw = PyObject_HasAttrString(o, "cuda_stream") ? PyObject_GetAttrString(o, "cuda_stream") : Py_NewRef(o);
  if (!raw) throw Refused();
  const long long v = PyLong_AsLongLong(raw);
  Py_DECREF(raw);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return reinterpret_cast<cudaStream_t>(v);
}

struct Table {
  const int32_t* data;
  int64_t stride, width;
};
Table block_table(PyObject* o, int64_t batch, int device) {
  const at::Tensor& t = tensor(o, "block_table");
  on(t, device, "block_table");
  if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != batch || (t.size(1) > 1 && t.stride(1) != 1))
    refuse("block_table must be an int32 tensor [%lld, max_pages] with unit column stride", static_cast<long long>(batch));
  return {static_cast<const int32_t*>(t.data_ptr()), t.stride(0), t.size(1)};
}

// Columns of queries and new rows that go with a cache of this format.
int64_t cache_columns(const at::Tensor& t, int format, int device) {
  const int64_t width = format == MLA_KV_BF16 ? 576 : format == MLA_KV_FP8_656 ? 656 : format == MLA_KV_FP8_528 ? 528 : 0;
  if (!width) refuse("unknown kv_format %d", format);
  on(t, device, "kv_cache");
  if (t.scalar_type() != (format == MLA_KV_BF16 ? at::kBFloat16 : at::kByte) || t.dim() != 3 || t.size(1) != 64 ||
      t.size(2) != width || !t.is_contiguous())
    refuse("kv_format %d needs a contiguous %s kv_cache [pages, 64, %d]", format,
           format == MLA_KV_BF16 ? "bfloat16" : "uint8", static_cast<int>(width));
  return format == MLA_KV_FP8_528 ? 512 : 576;
}

struct Rope {
  const float* table;
  int64_t rows;
};
Rope rope_table(PyObject* o, int device) {
  if (o == Py_None) return {nullptr, 0};
  const at::Tensor& t = tensor(o, "rope_table");
  on(t, device, "rope_table");
  if (t.scalar_type() != at::kFloat || t.dim() != 2 || t.size(1) != 64 || !t.is_contiguous())
    refuse("rope_table must be a contiguous float32 tensor [positions, 64]");
  return {static_cast<const float*>(t.data_ptr()), t.size(0)};
}

// Runs call() with `device` current.
template <class Call>
PyObject* launch(int device, const Call& call) {
  const int before = c10::cuda::current_device();
  if (before != device) c10::cuda::set_device(static_cast<c10::DeviceIndex>(device));
  const int status = call();
  if (before != device) c10::cuda::set_device(static_cast<c10::DeviceIndex>(before));
  return PyLong_FromLong(status);
}

template <class Body>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, const Body& body) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return nullptr;
  }
  try {
    return body();
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// kv_new, kv_cache, kv_format, block_table, cache_seqlens, rope_table, rope_style, norm_weight, norm_eps, new_lens, err, stream
PyObject* append_kv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&] {
    const at::Tensor& cache = tensor(a[1], "kv_cache");
    const int device = device_of(cache, "kv_cache"), format = narrow(a[2], "kv_format");
    const int64_t d = cache_columns(cache, format, device);
    const at::Tensor& x = tensor(a[0], "kv_new");
    on(x, device, "kv_new");
    if (x.scalar_type() != at::kBFloat16 || x.dim() != 3 || x.size(2) != d || x.stride(2) != 1)
      refuse("kv_new must be a bfloat16 tensor [batch, s_new, %d] with unit column stride", static_cast<int>(d));
    const int64_t b = x.size(0), s = x.size(1);
    int64_t token = x.stride(1);
    if (s == 1)
      token = b > 1 ? x.stride(0) : d;
    else if (b > 1 && x.stride(0) != s * token)
      refuse("kv_new's token slots must be evenly spaced over the batch");
    const auto* lens = static_cast<const int32_t*>(vector(a[4], at::kInt, b, "cache_seqlens", device));
    const auto* fresh = static_cast<const int32_t*>(vector(a[9], at::kInt, b, "new_lens", device, true));
    const auto* weight = static_cast<const float*>(vector(a[7], at::kFloat, 512, "norm_weight", device, true));
    auto* err = static_cast<uint32_t*>(vector(a[10], at::kInt, 1, "err", device, true));
    const Table bt = block_table(a[3], b, device);
    const Rope rope = rope_table(a[5], device);
    const int style = narrow(a[6], "rope_style");
    const float eps = real(a[8]);
    const cudaStream_t stream = stream_of(a[11], device);
    return launch(device, [&] {
      return mla_append_kv(x.data_ptr(), token, lens, fresh, size(b), size(s), rope.table, rope.rows, style, weight, eps,
                           cache.data_ptr(), format, cache.size(0), bt.data, bt.stride, bt.width, err, stream);
    });
  });
}

// Strides of a [b, s, h, d] tensor: from token slot to token slot over the whole
// batch, and from head to head.
void head_strides(const at::Tensor& t, const char* name, int64_t* token, int64_t* head) {
  if (t.scalar_type() != at::kBFloat16 || t.stride(3) != 1)
    refuse("%s must be a bfloat16 tensor with unit column stride", name);
  const int64_t b = t.size(0), s = t.size(1), h = t.size(2), d = t.size(3);
  *head = h == 1 ? d : t.stride(2);
  *token = t.stride(1);
  if (s == 1)
    *token = b > 1 ? t.stride(0) : h * *head;
  else if (b > 1 && t.stride(0) != s * *token)
    refuse("%s's token slots must be evenly spaced over the batch", name);
}

// q, out, cache_seqlens, rope_table, rope_style, norm_weight, norm_eps, new_lens, err, stream
PyObject* query_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&] {
    const at::Tensor &q = tensor(a[0], "q"), &out = tensor(a[1], "out");
    const int device = device_of(q, "q");
    on(out, device, "out");
    if (q.dim() != 4 || q.sizes() != out.sizes()) refuse("q and out must be [batch, s_q, h_q, d]");
    const int64_t b = q.size(0), s = q.size(1), h = q.size(2), d = q.size(3);
    int64_t q_token, q_head, out_token, out_head;
    head_strides(q, "q", &q_token, &q_head);
    head_strides(out, "out", &out_token, &out_head);
    const auto* lens = static_cast<const int32_t*>(vector(a[2], at::kInt, b, "cache_seqlens", device));
    const auto* fresh = static_cast<const int32_t*>(vector(a[7], at::kInt, b, "new_lens", device, true));
    const auto* weight = static_cast<const float*>(vector(a[5], at::kFloat, d, "norm_weight", device, true));
    auto* err = static_cast<uint32_t*>(vector(a[8], at::kInt, 1, "err", device, true));
    const Rope rope = rope_table(a[3], device);
    const int style = narrow(a[4], "rope_style");
    const float eps = real(a[6]);
    const cudaStream_t stream = stream_of(a[9], device);
    return launch(device, [&] {
      return mla_query_norm_rope(q.data_ptr(), q_token, q_head, lens, fresh, size(b), size(s), size(h), size(d), rope.table,
                                 rope.rows, style, weight, eps, out.data_ptr(), out_token, out_head, err, stream);
    });
  });
}

// q, kv_cache, kv_format, block_table, cache_seqlens, softmax_scale, window, sinks, num_sm_parts, workspace, out, lse,
// err, stream, attn_sink, new_lens
PyObject* window_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&] {
    const at::Tensor &q = tensor(a[0], "q"), &cache = tensor(a[1], "kv_cache");
    const int device = device_of(q, "q"), format = narrow(a[2], "kv_format");
    const int64_t d = cache_columns(cache, format, device);
    if (q.scalar_type() != at::kBFloat16 || q.dim() != 4 || q.size(3) != d || !q.is_contiguous())
      refuse("q must be a contiguous bfloat16 tensor [batch, s_q, h_q, %d]", static_cast<int>(d));
    const int64_t b = q.size(0), s = q.size(1), h = q.size(2);
    const at::Tensor& out = tensor(a[10], "out");
    on(out, device, "out");
    if (out.scalar_type() != at::kBFloat16 || out.dim() != 4 || out.size(0) != b || out.size(1) != s || out.size(2) != h ||
        out.size(3) != 512 || !out.is_contiguous())
      refuse("out must be a contiguous bfloat16 tensor [batch, s_q, h_q, 512]");
    auto* lse = static_cast<float*>(vector(a[11], at::kFloat, b * h * s, "lse", device));
    const auto* lens = static_cast<const int32_t*>(vector(a[4], at::kInt, b, "cache_seqlens", device));
    const auto* fresh = static_cast<const int32_t*>(vector(a[15], at::kInt, b, "new_lens", device, true));
    const auto* sink = static_cast<const float*>(vector(a[14], at::kFloat, h, "attn_sink", device, true));
    auto* err = static_cast<uint32_t*>(vector(a[12], at::kInt, 1, "err", device, true));
    const Table bt = block_table(a[3], b, device);
    void* ws = nullptr;
    size_t ws_bytes = 0;
    if (a[9] != Py_None) {
      const at::Tensor& w = tensor(a[9], "workspace");
      on(w, device, "workspace");
      if (!w.is_contiguous()) refuse("workspace must be contiguous");
      ws = w.data_ptr();
      ws_bytes = w.nbytes();
    }
    const float scale = real(a[5]);
    const int window = narrow(a[6], "window"), sinks = narrow(a[7], "sinks"), parts = narrow(a[8], "num_sm_parts");
    const cudaStream_t stream = stream_of(a[13], device);
    return launch(device, [&] {
      return mla_window_decode(q.data_ptr(), cache.data_ptr(), format, cache.size(0), bt.data, bt.stride, bt.width, lens,
                               fresh, size(b), size(s), size(h), window, sinks, scale, sink, parts, ws, ws_bytes,
                               out.data_ptr(), lse, err, stream);
    });
  });
}

PyMethodDef methods[] = {
    {"append_kv", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(append_kv)), METH_FASTCALL, nullptr},
    {"query_norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(query_norm_rope)), METH_FASTCALL, nullptr},
    {"window_decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(window_decode)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_step", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__step() { return PyModule_Create(&module); }
