// binding.cpp — the Python calls of the decoder-block operators.
//
// A decode step's calls take the GPU two to ten microseconds, less than their
// argument checks, output allocations and ctypes marshalling took in Python
// (15 µs for the norms of 8 rows).  Here the same checks and allocations are
// made in C++ on torch's tensors, and the library's C entry points are called
// through their addresses, which bind() receives from the loaded library.
// Every function launches on its tensors' device, on that device's current
// stream; tensors of several devices are refused.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cmath>
#include <cstdint>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "bitdelta_block.h"

namespace {

decltype(&bitdelta_add_norm) g_add_norm = nullptr;
decltype(&bitdelta_kv_append) g_kv_append = nullptr;
decltype(&bitdelta_attention) g_attention = nullptr;

struct Refused {};  // a Python error has been set

[[noreturn]] void refuse(const char* format, const char* name, const char* what = "") {
  PyErr_Format(PyExc_ValueError, format, name, what);
  throw Refused{};
}

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    default: return "another type";
  }
}

// A call's tensors, all on the device that it launches on.
struct Tensors {
  int64_t device;  // index; the first tensor's where it is negative

  const at::Tensor& get(PyObject* o, at::ScalarType type, const char* name) {
    if (!THPVariable_Check(o)) refuse("%s must be a tensor", name);
    const at::Tensor& t = THPVariable_Unpack(o);
    const c10::Device d = t.device();
    if (!d.is_cuda()) refuse("%s must be a CUDA tensor", name);
    if (device < 0) device = d.index();
    if (d.index() != device) refuse("%s is on another device than the call's other tensors", name);
    if (t.scalar_type() != type) refuse("%s must be %s", name, type_name(type));
    if (!t.is_contiguous()) refuse("%s must be contiguous", name);
    return t;
  }
  const at::Tensor& shaped(PyObject* o, at::ScalarType type, at::IntArrayRef shape,
                           const char* name) {
    const at::Tensor& t = get(o, type, name);
    if (t.sizes() != shape) refuse("%s does not have the shape that the call needs", name);
    return t;
  }
  const at::Tensor* maybe(PyObject* o, at::ScalarType type, const char* name) {
    return o == Py_None ? nullptr : &get(o, type, name);
  }
};
void* address(const at::Tensor* t) { return t == nullptr ? nullptr : t->data_ptr(); }
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return v;
}
void* pointer(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (p == nullptr && PyErr_Occurred()) throw Refused{};
  return p;
}
bd_stream_t stream_of(const at::Tensor& t) {
  return reinterpret_cast<bd_stream_t>(
      c10::cuda::getCurrentCUDAStream(t.device().index()).stream());
}
// (at::empty's work without its way through the dispatcher: the norms of 8 rows,
// two outputs, 7.1 -> 4.6 µs of host time a call)
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
  return at::Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}
PyObject* two(const at::Tensor& a, const at::Tensor& b) {
  PyObject* r = PyTuple_New(2);
  if (r == nullptr) throw Refused{};
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(a));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(b));
  return r;
}

template <typename F>
PyObject* guarded(Py_ssize_t have, Py_ssize_t want, F f) {
  if (have != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, have);
    return nullptr;
  }
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// bind(add_norm, kv_append, attention): the entry points' addresses.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject* {
    g_add_norm = reinterpret_cast<decltype(g_add_norm)>(pointer(a[0]));
    g_kv_append = reinterpret_cast<decltype(g_kv_append)>(pointer(a[1]));
    g_attention = reinterpret_cast<decltype(g_attention)>(pointer(a[2]));
    Py_RETURN_NONE;
  });
}

// Refuses a table of norm_table() whose weights are shorter than the rows: the
// kernel would read past them.
void check_width(PyObject* table, int64_t d, const char* name) {
  static PyObject* const attribute = PyUnicode_InternFromString("norm_width");
  PyObject* const width = PyObject_GetAttr(table, attribute);
  if (width == nullptr) {  // pointers that the caller made
    if (!PyErr_ExceptionMatches(PyExc_AttributeError)) throw Refused{};
    PyErr_Clear();
    return;
  }
  const int64_t have = PyLong_AsLongLong(width);
  Py_DECREF(width);
  if (have == -1 && PyErr_Occurred()) throw Refused{};
  if (have < d) refuse("%s's weights are shorter than y's rows", name);
}

// add_norm(y, residual, pre_table, post_table, gate, scale, eps, seg_offsets,
// seg_variant, residual_out, out) -> (h, x), or the status code of a refusal.
PyObject* add_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    Tensors in{-1};
    const at::Tensor& y = in.get(a[0], at::kBFloat16, "y");
    if (y.dim() < 1) refuse("%s must have at least one dimension", "y");
    const int64_t d = y.size(-1);
    at::ScalarType rtype = at::kBFloat16;
    const at::Tensor* residual = nullptr;
    if (a[1] != Py_None) {
      if (THPVariable_Check(a[1])) rtype = THPVariable_Unpack(a[1]).scalar_type();
      if (rtype != at::kBFloat16 && rtype != at::kFloat)
        refuse("%s must be bfloat16 or float32", "residual");
      residual = &in.shaped(a[1], rtype, y.sizes(), "residual");
    }
    if (a[2] == Py_None) refuse("%s is required", "pre_table");
    const at::Tensor& pre = in.get(a[2], at::kLong, "pre_table");
    check_width(a[2], d, "pre_table");
    const at::Tensor* post = in.maybe(a[3], at::kLong, "post_table");
    if (post != nullptr) check_width(a[3], d, "post_table");
    if (post != nullptr && post->numel() != pre.numel())
      refuse("pre_table and %s must have the same number of slots", "post_table");
    const at::Tensor* gate = in.maybe(a[4], at::kBFloat16, "gate");
    int64_t gate_stride = 0;
    if (gate != nullptr) {
      if (gate->dim() > 1 && gate->sizes() == y.sizes())
        gate_stride = d;
      else if (gate->dim() != 1 || gate->size(0) != d)
        refuse("%s must be [d] or have the shape of y", "gate");
    }
    const double scale = number(a[5]), eps = number(a[6]);
    if ((a[7] == Py_None) != (a[8] == Py_None))
      refuse("%s and seg_variant go together", "seg_offsets");
    const at::Tensor* offsets = in.maybe(a[7], at::kInt, "seg_offsets");
    const at::Tensor* variant = in.maybe(a[8], at::kInt, "seg_variant");
    const int64_t n_seg = variant != nullptr ? variant->numel() : 0;
    if (offsets != nullptr && offsets->numel() != n_seg + 1)
      refuse("%s must have one entry more than seg_variant", "seg_offsets");
    if (n_seg == 0) variant = offsets;  // no segments: an address that is not read
    const at::Tensor* h_out =
        a[9] != Py_None ? &in.shaped(a[9], rtype, y.sizes(), "residual_out") : nullptr;
    const at::Tensor* x_out =
        a[10] != Py_None ? &in.shaped(a[10], at::kBFloat16, y.sizes(), "out") : nullptr;
    const c10::cuda::CUDAGuard guard(y.device());
    const at::Tensor h = h_out != nullptr ? *h_out : fresh(y.sizes(), rtype, y);
    const at::Tensor x = x_out != nullptr ? *x_out : fresh(y.sizes(), at::kBFloat16, y);
    const bd_status st = g_add_norm(
        static_cast<const uint16_t*>(y.data_ptr()), d > 0 ? y.numel() / d : 0, d,
        address(residual), h.data_ptr(), rtype == at::kFloat ? BD_RESIDUAL_F32 : BD_RESIDUAL_BF16,
        static_cast<const uint16_t*>(address(gate)), gate_stride, static_cast<float>(scale),
        static_cast<float>(eps), static_cast<const uint16_t* const*>(pre.data_ptr()),
        static_cast<const uint16_t* const*>(address(post)), static_cast<int32_t>(pre.numel()),
        static_cast<const int32_t*>(address(offsets)),
        static_cast<const int32_t*>(address(variant)), static_cast<int32_t>(n_seg),
        static_cast<uint16_t*>(x.data_ptr()), stream_of(y));
    if (st != BD_OK) return PyLong_FromLong(st);
    return two(h, x);
  });
}

// A batch as the Python class holds it: the C struct, the device of its tables,
// plan and workspace, and the stream that last used them.
struct Batch {
  bd_attention_batch c;
  int64_t device;
  uint64_t stream;
};

// Tells the allocator that `stream` uses the batch's tensors too, so that their
// memory is not handed out while work there is in flight, even where the batch
// is dropped at once.  The caller cannot: plan and workspace are the batch's own.
bd_stream_t used_by_current_stream(Batch* b, PyObject* tensors) {
  const c10::cuda::CUDAStream s =
      c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(b->device));
  const uint64_t handle = reinterpret_cast<uint64_t>(s.stream());
  if (b->stream != handle) {
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(tensors); ++i)
      c10::cuda::CUDACachingAllocator::recordStream(
          THPVariable_Unpack(PyTuple_GET_ITEM(tensors, i)).storage().data_ptr(), s);
    b->stream = handle;
  }
  return reinterpret_cast<bd_stream_t>(s.stream());
}

// used_by_current_stream(batch, its tensors) -> the handle of that stream.
PyObject* used(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 2, [&]() -> PyObject* {
    return PyLong_FromVoidPtr(used_by_current_stream(static_cast<Batch*>(pointer(a[0])), a[1]));
  });
}

// A call's cache: its shape goes into the batch's struct.
struct Cache {
  uint16_t *k, *v;
};
Cache cache_of(Tensors& in, Batch* b, PyObject* k_pages, PyObject* v_pages) {
  const at::Tensor& kp = in.get(k_pages, at::kBFloat16, "k_pages");
  const at::Tensor& vp = in.get(v_pages, at::kBFloat16, "v_pages");
  if (kp.dim() != 4 || kp.sizes() != vp.sizes() || kp.size(1) != b->c.n_kv_heads ||
      kp.size(2) != b->c.page_size || kp.size(3) != b->c.head_dim)
    refuse("k_pages and %s must be [n_pages, n_kv_heads, page_size, head_dim]", "v_pages");
  b->c.n_pages = kp.size(0);
  return {static_cast<uint16_t*>(kp.data_ptr()), static_cast<uint16_t*>(vp.data_ptr())};
}

// kv_append(batch, its tensors, qkv, rope, k_pages, v_pages, interleaved, out) ->
// q, or a status code.
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    Batch* batch = static_cast<Batch*>(pointer(a[0]));
    const bd_attention_batch& b = batch->c;
    Tensors in{batch->device};
    const int64_t width = static_cast<int64_t>(b.n_q_heads + 2 * b.n_kv_heads) * b.head_dim;
    const at::Tensor& qkv = in.shaped(a[2], at::kBFloat16, {b.n_tokens, width}, "qkv");
    const at::Tensor* rope = in.maybe(a[3], at::kFloat, "rope");
    if (rope != nullptr && rope->dim() != 2) refuse("%s must be [positions, rot_dim]", "rope");
    const int64_t rows = rope != nullptr ? rope->size(0) : 0;
    const int64_t rot = rope != nullptr ? rope->size(1) : 0;
    const int pairs = PyObject_IsTrue(a[6]);
    if (pairs < 0) throw Refused{};
    const int64_t shape[3] = {b.n_tokens, b.n_q_heads, b.head_dim};
    const at::Tensor* out =
        a[7] != Py_None ? &in.shaped(a[7], at::kBFloat16, shape, "out") : nullptr;
    const Cache cache = cache_of(in, batch, a[4], a[5]);
    const c10::cuda::CUDAGuard guard(qkv.device());
    const at::Tensor q = out != nullptr ? *out : fresh(shape, at::kBFloat16, qkv);
    const bd_status st = g_kv_append(
        &b, static_cast<const uint16_t*>(qkv.data_ptr()), static_cast<const float*>(address(rope)),
        rows, static_cast<int32_t>(rot < INT32_MAX ? rot : INT32_MAX),
        pairs != 0 ? BD_ROPE_PAIRS : BD_ROPE_HALVES, cache.k, cache.v,
        static_cast<uint16_t*>(q.data_ptr()), used_by_current_stream(batch, a[1]));
    if (st != BD_OK) return PyLong_FromLong(st);
    return THPVariable_Wrap(q);
  });
}

// attention(batch, its tensors, plan, plan_bytes, workspace, workspace_bytes, q,
// k_pages, v_pages, scale, out, lse) -> (out, lse), or a status code.
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    Batch* batch = static_cast<Batch*>(pointer(a[0]));
    const bd_attention_batch& b = batch->c;
    Tensors in{batch->device};
    const int64_t shape[3] = {b.n_tokens, b.n_q_heads, b.head_dim};
    const at::IntArrayRef rows(shape, 2);
    const at::Tensor& q = in.shaped(a[6], at::kBFloat16, shape, "q");
    const double scale =
        a[9] == Py_None ? 1.0 / std::sqrt(static_cast<double>(b.head_dim)) : number(a[9]);
    const at::Tensor* o_out =
        a[10] != Py_None ? &in.shaped(a[10], at::kBFloat16, shape, "out") : nullptr;
    const at::Tensor* l_out =
        a[11] != Py_None ? &in.shaped(a[11], at::kFloat, rows, "lse") : nullptr;
    const Cache cache = cache_of(in, batch, a[7], a[8]);
    const c10::cuda::CUDAGuard guard(q.device());
    const at::Tensor out = o_out != nullptr ? *o_out : fresh(shape, at::kBFloat16, q);
    const at::Tensor lse = l_out != nullptr ? *l_out : fresh(rows, at::kFloat, q);
    const bd_status st = g_attention(
        &b, pointer(a[2]), PyLong_AsSize_t(a[3]), static_cast<const uint16_t*>(q.data_ptr()),
        cache.k, cache.v, static_cast<float>(scale), static_cast<uint16_t*>(out.data_ptr()),
        static_cast<float*>(lse.data_ptr()), pointer(a[4]), PyLong_AsSize_t(a[5]),
        used_by_current_stream(batch, a[1]));
    if (st != BD_OK) return PyLong_FromLong(st);
    return two(out, lse);
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
constexpr PyCFunction as_function() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef methods[] = {
    {"bind", as_function<bind>(), METH_FASTCALL, nullptr},
    {"add_norm", as_function<add_norm>(), METH_FASTCALL, nullptr},
    {"used_by_current_stream", as_function<used>(), METH_FASTCALL, nullptr},
    {"kv_append", as_function<kv_append>(), METH_FASTCALL, nullptr},
    {"attention", as_function<attention>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
