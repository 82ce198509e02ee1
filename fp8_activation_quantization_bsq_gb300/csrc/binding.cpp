// Python module _bsq_binding: the calls of layer.py from torch tensors to the C ABI (bsq.h).
//
// A call for a single token keeps the GPU busy for two to four microseconds; reading the tensors' attributes, allocating and
// converting the arguments from Python took the host 13.5 us for routing and 24 for the rows' order.  The checks, the allocation of missing outputs
// and the call are therefore compiled: 3.7 us a projection, 4.5 a rotation or routing, routing and rows 10.2 (through the dispatcher's allocation
// 4.3, 5.3 and 13.1).  Refused arguments raise ValueError, statuses BsqError; work goes to the given or current stream, and outputs are
// allocated under it.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <optional>

#include "bsq.h"

namespace {

PyObject* g_error = nullptr;  // BsqError(code, what)

struct Refused {};  // a Python exception is set

[[noreturn]] void refuse(const char* what) {
  PyErr_SetString(PyExc_ValueError, what);
  throw Refused();
}
[[noreturn]] void pending() { throw Refused(); }

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_ValueError, "%s must be a tensor", what);
    throw Refused();
  }
  return THPVariable_Unpack(o);
}
bool given(PyObject* o) { return o != Py_None; }

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) pending();
  return v;
}
int32_t integer32(PyObject* o) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse("an integer argument is out of range");
  return static_cast<int32_t>(v);
}
float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) pending();
  return static_cast<float>(v);
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) pending();
  return v != 0;
}

// bsq_dtype, or -1.
int dtype_of(at::ScalarType t) {
  return t == at::kBFloat16 ? BSQ_BF16 : t == at::kHalf ? BSQ_F16 : t == at::kFloat ? BSQ_F32 : -1;
}
bool on(const at::Tensor& t, int index) { return t.is_cuda() && t.get_device() == index; }
bool plain(const at::Tensor& t, at::ScalarType type, int index) { return t.scalar_type() == type && on(t, index) && t.is_contiguous(); }

// The device and stream of a call, current while it lasts.
struct Call {
  int index;
  std::optional<c10::cuda::CUDAStreamGuard> stream_guard;
  std::optional<c10::cuda::CUDAGuard> device_guard;
  cudaStream_t stream;
  Call(int device, PyObject* given_stream) : index(device) {
    if (given_stream != Py_None) {
      PyObject* id = PyObject_GetAttrString(given_stream, "stream_id");
      PyObject* at = id ? PyObject_GetAttrString(given_stream, "device_index") : nullptr;
      const long long i = id ? PyLong_AsLongLong(id) : 0, d = at ? PyLong_AsLongLong(at) : 0;
      Py_XDECREF(id);
      Py_XDECREF(at);
      if (PyErr_Occurred()) pending();
      if (d != device) refuse("the stream must be on the tensors' device");
      const c10::cuda::CUDAStream s(c10::Stream::unpack3(i, static_cast<c10::DeviceIndex>(d), c10::DeviceType::CUDA));
      stream_guard.emplace(s);
      stream = s.stream();
    } else {
      device_guard.emplace(static_cast<c10::DeviceIndex>(device));
      stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
    }
  }
  at::Tensor make(at::IntArrayRef shape, at::ScalarType type) const {
    return at::Tensor(at::detail::empty_cuda(shape, type, c10::Device(c10::DeviceType::CUDA, static_cast<c10::DeviceIndex>(index)), std::nullopt));
  }
  void check(int32_t rc, const char* name) const {
    if (rc == BSQ_OK) return;
    if (PyObject* e = PyObject_CallFunction(g_error, "is", static_cast<int>(rc), name)) {
      PyErr_SetObject(g_error, e);
      Py_DECREF(e);
    }
    throw Refused();
  }
};

// packed_linear(x, w, w_scales, fmt, w_sf, add, out_dtype, out, stream)
PyObject* packed_linear(PyObject* const* a) {
  const at::Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "w"), &scales = tensor(a[2], "w_scales");
  const int dt = dtype_of(x.scalar_type());
  if ((dt != BSQ_BF16 && dt != BSQ_F16) || x.dim() != 2 || !x.is_cuda() || (x.stride(1) != 1 && x.size(0) > 0))
    refuse("x must be a 2-D bfloat16 or float16 CUDA tensor with unit inner stride");
  const int64_t tokens = x.size(0), cols = x.size(1);
  const int index = x.get_device();
  const int32_t fmt = integer32(a[3]);
  if (!plain(w, at::kByte, index) || w.dim() != 2 || cols % 32 != 0 || w.size(1) != bsq_packed_row_bytes(fmt, cols))
    refuse("w must be a contiguous uint8 (rows, row bytes of cols) tensor on x's CUDA device, cols a multiple of 32");
  const int64_t rows = w.size(0);
  if (!plain(scales, at::kByte, index) || scales.numel() != bsq_scales5d_bytes(fmt, rows, cols))
    refuse("w_scales must be a contiguous uint8 tensor of the weights' 5D scales on x's device");
  const float* sf = nullptr;
  if (fmt == BSQ_NVFP4) {
    if (!given(a[4])) refuse("nvfp4 needs w_sf, a float32 tensor of one element on x's device");
    const at::Tensor& t = tensor(a[4], "w_sf");
    if (t.scalar_type() != at::kFloat || t.numel() != 1 || !on(t, index)) refuse("nvfp4 needs w_sf, a float32 tensor of one element on x's device");
    sf = static_cast<const float*>(t.data_ptr());
  }
  const Call call(index, a[8]);
  at::Tensor made;
  PyObject* result = a[7];
  at::ScalarType type = x.scalar_type();
  if (given(a[6])) {
    if (!THPDtype_Check(a[6])) refuse("out_dtype must be a torch dtype");
    type = reinterpret_cast<THPDtype*>(a[6])->scalar_type;
  } else if (given(result)) {
    type = tensor(result, "out").scalar_type();
  }
  const int od = dtype_of(type);
  if (od != dt && od != BSQ_F32) refuse("out_dtype must be x's type or float32");
  if (given(result)) {
    const at::Tensor& o = tensor(result, "out");
    if (o.scalar_type() != type || !on(o, index) || o.dim() != 2 || o.size(0) != tokens || o.size(1) != rows || (o.stride(1) != 1 && o.numel() > 0))
      refuse("out must be a (tokens, rows) tensor of out_dtype with unit inner stride on x's device");
  } else {
    made = call.make({tokens, rows}, type);
  }
  const at::Tensor& out = given(result) ? THPVariable_Unpack(result) : made;
  const void* add = nullptr;
  int64_t ld_add = 0;
  if (given(a[5])) {
    const at::Tensor& t = tensor(a[5], "add");
    const bool matrix = t.dim() == 2 && t.size(0) == tokens && t.size(1) == rows, bias = t.dim() == 1 && t.size(0) == rows;
    if (t.scalar_type() != type || !on(t, index) || (!matrix && !bias) || (t.stride(-1) != 1 && t.numel() > 0))
      refuse("add must be a (tokens, rows) or (rows) tensor of the output's type with unit inner stride on x's device");
    add = t.data_ptr();
    ld_add = matrix ? t.stride(0) : 0;
  }
  call.check(bsq_packed_linear(fmt, dt, x.data_ptr(), tokens, cols, tokens > 1 ? x.stride(0) : cols, w.data_ptr(), scales.data_ptr(), rows, sf,
                               add, ld_add, od, out.data_ptr(), tokens > 1 ? out.stride(0) : rows, call.stream),
             "bsq_packed_linear");
  return given(result) ? Py_NewRef(result) : THPVariable_Wrap(made);
}

// qk_norm_rope(q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, q_out, k_out, stream)
PyObject* qk_norm_rope(PyObject* const* a) {
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &pos = tensor(a[2], "positions"), &freq = tensor(a[3], "inv_freq");
  const int dt = dtype_of(q.scalar_type());
  if ((dt != BSQ_BF16 && dt != BSQ_F16) || q.dim() != 3 || !q.is_cuda() || (q.stride(2) != 1 && q.numel() > 0))
    refuse("q must be a (tokens, heads, dim) bfloat16 or float16 CUDA tensor with unit inner stride");
  const int64_t tokens = q.size(0), heads = q.size(1), dim = q.size(2);
  const int index = q.get_device();
  if (k.scalar_type() != q.scalar_type() || !on(k, index) || k.dim() != 3 || k.size(0) != tokens || k.size(2) != dim ||
      (k.stride(2) != 1 && k.numel() > 0))
    refuse("k must be a (tokens, kv_heads, dim) tensor of q's type and device with unit inner stride");
  if (!plain(pos, at::kInt, index) || pos.dim() != 1 || pos.size(0) != tokens || !plain(freq, at::kFloat, index) || freq.dim() != 1)
    refuse("positions must be an int32 (tokens) and inv_freq a float32 (pairs) contiguous tensor on q's device");
  const void* weight[2] = {nullptr, nullptr};
  int wd = -1;
  for (int i = 0; i < 2; ++i)
    if (given(a[4 + i])) {
      const at::Tensor& w = tensor(a[4 + i], "a weight");
      const int d = dtype_of(w.scalar_type());
      if ((d != dt && d != BSQ_F32) || !on(w, index) || w.dim() != 1 || w.size(0) != dim || !w.is_contiguous())
        refuse("q_weight and k_weight must be contiguous (dim) tensors of q's type or float32 on q's device");
      if (wd >= 0 && d != wd) refuse("q_weight and k_weight must have one type");
      wd = d;
      weight[i] = w.data_ptr();
    }
  const float eps = number(a[6]);
  const bool interleaved = truth(a[7]);
  for (int i = 0; i < 2; ++i)
    if (given(a[8 + i])) {
      const at::Tensor &o = tensor(a[8 + i], "an output"), &in = i ? k : q;
      if (o.scalar_type() != in.scalar_type() || !on(o, index) || o.sizes() != in.sizes() || (o.stride(2) != 1 && o.numel() > 0))
        refuse("q_out and k_out must have their inputs' shapes, types and device and unit inner strides");
    }
  if (heads > INT32_MAX || k.size(1) > INT32_MAX || dim > INT32_MAX || freq.size(0) > INT32_MAX) refuse("a size is out of range");
  const Call call(index, a[10]);
  at::Tensor made[2];
  for (int i = 0; i < 2; ++i)
    if (!given(a[8 + i])) made[i] = call.make({tokens, i ? k.size(1) : heads, dim}, q.scalar_type());
  const at::Tensor &qo = given(a[8]) ? THPVariable_Unpack(a[8]) : made[0], &ko = given(a[9]) ? THPVariable_Unpack(a[9]) : made[1];
  call.check(bsq_qk_norm_rope(dt, q.data_ptr(), q.stride(0), q.stride(1), k.data_ptr(), k.stride(0), k.stride(1), tokens,
                              static_cast<int32_t>(heads), static_cast<int32_t>(k.size(1)), static_cast<int32_t>(dim),
                              static_cast<const int32_t*>(pos.data_ptr()), static_cast<const float*>(freq.data_ptr()),
                              static_cast<int32_t>(freq.size(0)), interleaved, weight[0], weight[1], wd >= 0 ? wd : dt, eps, qo.data_ptr(),
                              qo.stride(0), qo.stride(1), ko.data_ptr(), ko.stride(0), ko.stride(1), call.stream),
             "bsq_qk_norm_rope");
  PyObject* out[2];
  for (int i = 0; i < 2; ++i) out[i] = given(a[8 + i]) ? Py_NewRef(a[8 + i]) : THPVariable_Wrap(made[i]);
  return Py_BuildValue("(NN)", out[0], out[1]);
}

// moe_route(logits, top_k, sigmoid, bias, groups, top_groups, group_top, renormalize, scale, ids, weights, stream)
PyObject* moe_route(PyObject* const* a) {
  const at::Tensor& z = tensor(a[0], "logits");
  const int dt = dtype_of(z.scalar_type());
  if (dt < 0 || z.dim() != 2 || !z.is_cuda() || (z.stride(1) != 1 && z.size(1) > 1 && z.size(0) > 0))
    refuse("logits must be a 2-D float32, bfloat16 or float16 CUDA tensor with unit inner stride");
  const int64_t tokens = z.size(0), experts = z.size(1);
  const int index = z.get_device();
  const int32_t top_k = integer32(a[1]);
  if (experts > INT32_MAX || top_k < 0) refuse("a size is out of range");
  const float* bias = nullptr;
  if (given(a[3])) {
    const at::Tensor& b = tensor(a[3], "bias");
    if (!plain(b, at::kFloat, index) || b.dim() != 1 || b.size(0) != experts)
      refuse("bias must be a contiguous float32 (experts) tensor on the logits' device");
    bias = static_cast<const float*>(b.data_ptr());
  }
  const bool sigmoid = truth(a[2]), renormalize = truth(a[7]);
  const int32_t groups = integer32(a[4]), top_groups = integer32(a[5]), group_top = integer32(a[6]);
  const float scale = number(a[8]);
  for (int i = 0; i < 2; ++i)
    if (given(a[9 + i])) {
      const at::Tensor& o = tensor(a[9 + i], "an output");
      if (!plain(o, i ? at::kFloat : at::kInt, index) || o.dim() != 2 || o.size(0) != tokens || o.size(1) != top_k)
        refuse(i ? "weights must be a contiguous float32 (tokens, top_k) tensor on the logits' device"
                 : "ids must be a contiguous int32 (tokens, top_k) tensor on the logits' device");
    }
  const Call call(index, a[11]);
  at::Tensor made[2];
  for (int i = 0; i < 2; ++i)
    if (!given(a[9 + i])) made[i] = call.make({tokens, top_k}, i ? at::kFloat : at::kInt);
  const at::Tensor &ids = given(a[9]) ? THPVariable_Unpack(a[9]) : made[0], &weights = given(a[10]) ? THPVariable_Unpack(a[10]) : made[1];
  call.check(bsq_moe_route(dt, z.data_ptr(), tokens > 1 ? z.stride(0) : experts, tokens, static_cast<int32_t>(experts), top_k, sigmoid, bias, groups,
                           top_groups, group_top, renormalize, scale, static_cast<int32_t*>(ids.data_ptr()),
                           static_cast<float*>(weights.data_ptr()), call.stream),
             "bsq_moe_route");
  PyObject* out[2];
  for (int i = 0; i < 2; ++i) out[i] = given(a[9 + i]) ? Py_NewRef(a[9 + i]) : THPVariable_Wrap(made[i]);
  return Py_BuildValue("(NN)", out[0], out[1]);
}

// moe_rows(ids, experts, stream)
PyObject* moe_rows(PyObject* const* a) {
  const at::Tensor& ids = tensor(a[0], "ids");
  if (ids.scalar_type() != at::kInt || ids.dim() != 2 || !ids.is_cuda() || !ids.is_contiguous())
    refuse("ids must be a contiguous int32 (tokens, top_k) CUDA tensor");
  const int64_t tokens = ids.size(0), top_k = ids.size(1);
  const int32_t experts = integer32(a[1]);
  if (top_k > INT32_MAX || experts < 0) refuse("a size is out of range");
  const Call call(ids.get_device(), a[2]);
  const at::Tensor out[4] = {call.make({int64_t(experts) + 1}, at::kInt), call.make({int64_t(experts) + 1}, at::kInt),
                             call.make({tokens * top_k}, at::kInt), call.make({tokens, top_k}, at::kInt)};
  call.check(bsq_moe_rows(static_cast<const int32_t*>(ids.data_ptr()), tokens, static_cast<int32_t>(top_k), experts,
                          static_cast<uint32_t*>(out[0].data_ptr()), static_cast<uint32_t*>(out[1].data_ptr()),
                          static_cast<int32_t*>(out[2].data_ptr()), static_cast<int32_t*>(out[3].data_ptr()), call.stream),
             "bsq_moe_rows");
  return Py_BuildValue("(NNNN)", THPVariable_Wrap(out[0]), THPVariable_Wrap(out[1]), THPVariable_Wrap(out[2]), THPVariable_Wrap(out[3]));
}

// One Python function of N positional arguments; nothing C++ throws passes it.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, %zd given", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

PyObject* set_error(PyObject*, PyObject* type) {
  Py_XSETREF(g_error, Py_NewRef(type));
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&entry<F, N>));
}

PyMethodDef methods[] = {{"packed_linear", fast<packed_linear, 9>(), METH_FASTCALL, nullptr},
                         {"qk_norm_rope", fast<qk_norm_rope, 11>(), METH_FASTCALL, nullptr},
                         {"moe_route", fast<moe_route, 12>(), METH_FASTCALL, nullptr},
                         {"moe_rows", fast<moe_rows, 3>(), METH_FASTCALL, nullptr},
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bsq_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bsq_binding() { return PyModule_Create(&module); }
