// mxcalls.cpp -- the host's part of the microscaled calls, natively.
//
// A decode step's kernels take two to five microseconds; reading a tensor's
// shape, type and address, checking them, allocating the result and handing
// fifteen arguments to the library takes longer in Python.  This module does
// the same for the calls that mx.py would let through unchanged -- tensors of
// the right kind on the current device -- and returns None for every other
// one, which mx.py then takes itself: it checks again, raises what there is to
// raise, changes the device.  So every rule and every message is mx.py's, and
// without this module everything works, later.
//
// Tensors are read and made through ATen: reading one through its Python
// attributes took 0.35 us, making one by a Python call of torch.empty 1.6 us.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stddef.h>
#include <stdint.h>
#include <structmember.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <new>
#include <optional>

#include "strata_moe.h"

namespace {

// ---------------------------------------------------------------- what setup() hands over
struct Library {
  decltype(&moe_mx_quantize) quantize;
  decltype(&moe_mx_dequantize) dequantize;
  decltype(&moe_add_rmsnorm) add_rmsnorm;
  decltype(&moe_mx_linear) linear;
  decltype(&moe_mx_pack_experts) pack;
  decltype(&moe_mx_unpack_experts) unpack;
  decltype(&strata_expert_bytes) expert_bytes;
} lib;
PyObject* torch_tensor;    // torch.Tensor
PyObject* torch_param;     // torch.nn.Parameter
PyTypeObject* matrix_type; // Matrix below
PyTypeObject* mx_type;     // mx.py's MXTensor, a subclass of it
PyTypeObject* norm_type;   // mx.py's AddNorm, a named tuple
PyObject *s_cuda_stream, *s_device_index;  // interned names

// ---------------------------------------------------------------- MXTensor's fields
struct Matrix {
  PyObject_HEAD
  int fmt, layout;
  Py_ssize_t rows, K;
  at::Tensor both;           // one allocation for both planes
  PyObject *codes, *scales;  // a plane's tensor, where it has one of its own or was asked for
};

PyObject* matrix_new(PyTypeObject* type, PyObject*, PyObject*) {
  PyObject* o = type->tp_alloc(type, 0);
  if (o) new (&reinterpret_cast<Matrix*>(o)->both) at::Tensor();
  return o;
}

int matrix_traverse(PyObject* o, visitproc visit, void* arg) {
  Matrix* m = reinterpret_cast<Matrix*>(o);
  Py_VISIT(Py_TYPE(o));
  Py_VISIT(m->codes);
  Py_VISIT(m->scales);
  return 0;
}
int matrix_clear(PyObject* o) {
  Matrix* m = reinterpret_cast<Matrix*>(o);
  Py_CLEAR(m->codes);
  Py_CLEAR(m->scales);
  return 0;
}
void matrix_dealloc(PyObject* o) {
  PyTypeObject* type = Py_TYPE(o);
  PyObject_GC_UnTrack(o);
  matrix_clear(o);
  reinterpret_cast<Matrix*>(o)->both.~Tensor();
  type->tp_free(o);
  Py_DECREF(type);
}
PyMemberDef matrix_members[] = {
    {"_fmt", T_INT, offsetof(Matrix, fmt), 0, nullptr},
    {"_layout", T_INT, offsetof(Matrix, layout), 0, nullptr},
    {"_rows", T_PYSSIZET, offsetof(Matrix, rows), 0, nullptr},
    {"_K", T_PYSSIZET, offsetof(Matrix, K), 0, nullptr},
    {"_codes", T_OBJECT, offsetof(Matrix, codes), 0, nullptr},
    {"_scales", T_OBJECT, offsetof(Matrix, scales), 0, nullptr},
    {nullptr, 0, 0, 0, nullptr}};
PyObject* get_both(PyObject* o, void*) {
  const at::Tensor& t = reinterpret_cast<Matrix*>(o)->both;
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
int set_both(PyObject* o, PyObject* v, void*) {
  if (v && v != Py_None && !THPVariable_Check(v)) {
    PyErr_SetString(PyExc_TypeError, "a tensor or None is wanted");
    return -1;
  }
  reinterpret_cast<Matrix*>(o)->both = v && v != Py_None ? THPVariable_Unpack(v) : at::Tensor();
  return 0;
}
PyGetSetDef matrix_getset[] = {{"_both", get_both, set_both, nullptr, nullptr},
                               {nullptr, nullptr, nullptr, nullptr, nullptr}};
PyType_Slot matrix_slots[] = {{Py_tp_new, (void*)matrix_new},
                              {Py_tp_getset, (void*)matrix_getset},
                              {Py_tp_traverse, (void*)matrix_traverse},
                              {Py_tp_clear, (void*)matrix_clear},
                              {Py_tp_dealloc, (void*)matrix_dealloc},
                              {Py_tp_members, (void*)matrix_members},
                              {Py_tp_doc, (void*)"Fields of a microscaled matrix."},
                              {0, nullptr}};
PyType_Spec matrix_spec = {"expert_ffn_execution_b200._mxcalls.Matrix", sizeof(Matrix), 0,
                           Py_TPFLAGS_DEFAULT | Py_TPFLAGS_BASETYPE | Py_TPFLAGS_HAVE_GC,
                           matrix_slots};

// ---------------------------------------------------------------- reading tensors
// A function that finds something it does not take returns false with no
// exception set; callers pass that on as None.
bool pass() {
  PyErr_Clear();
  return false;
}

int dtype_of(at::ScalarType t) {
  return t == at::kFloat ? STRATA_DTYPE_F32 : t == at::kHalf ? STRATA_DTYPE_F16 : t == at::kBFloat16 ? STRATA_DTYPE_BF16 : -1;
}
int dtype_of(PyObject* o) {
  return THPDtype_Check(o) ? dtype_of(reinterpret_cast<THPDtype*>(o)->scalar_type) : -1;
}
at::ScalarType scalar_type(int dt) {
  return dt == STRATA_DTYPE_F32 ? at::kFloat : dt == STRATA_DTYPE_F16 ? at::kHalf : at::kBFloat16;
}

struct Tensor {
  int dtype = -1;  // STRATA_DTYPE_*, 8: uint8, 32: int32
  int index = -1;
  void* ptr = nullptr;
  int dims = 0;
  int64_t size[3] = {0, 0, 0}, stride[3] = {0, 0, 0};
  bool rows_contiguous() const {
    return dims == 2 && (size[1] <= 1 || stride[1] == 1) &&
           (size[0] <= 1 || stride[0] == size[1] || size[1] == 0);
  }
};

// Reads a torch.Tensor (or Parameter; no other subclass) of one to three
// dimensions on a CUDA device.  Throws for one without memory of its own.
bool read(PyObject* o, Tensor* t) {
  PyObject* type = reinterpret_cast<PyObject*>(Py_TYPE(o));
  if (type != torch_tensor && type != torch_param) return false;
  const at::Tensor& v = THPVariable_Unpack(o);
  if (!v.is_cuda() || v.layout() != at::kStrided || v.is_neg()) return false;
  const at::ScalarType st = v.scalar_type();
  t->dtype = st == at::kByte ? 8 : st == at::kInt ? 32 : dtype_of(st);
  t->index = v.device().index();
  t->dims = (int)v.dim();
  if (t->dtype < 0 || t->index < 0 || t->index >= 64 || t->dims < 1 || t->dims > 3) return false;
  const at::IntArrayRef size = v.sizes(), stride = v.strides();
  for (int i = 0; i < t->dims; ++i) {
    t->size[i] = size[i];
    t->stride[i] = stride[i];
  }
  t->ptr = v.data_ptr();
  return true;
}

bool address(PyObject* o, void** p) {
  const unsigned long long v = PyLong_Check(o) ? PyLong_AsUnsignedLongLong(o) : 0;
  if (v == ~0ull && PyErr_Occurred()) return pass();
  *p = reinterpret_cast<void*>(v);
  return PyLong_Check(o);
}

// Where a call runs: on device `index`, which has to be the current one, on
// the current stream or, where the call names another, on that one, which is
// then the current one while the call allocates and launches (mx.py's _place()).
struct Target {
  void* handle = nullptr;
  std::optional<c10::cuda::CUDAStream> other;
};
bool target(int index, PyObject* stream, Target* to) {
  if (c10::impl::TorchDispatchModeTLS::any_modes_set() || c10::cuda::current_device() != index)
    return false;
  to->handle = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
  if (stream == Py_None) return true;
  void* handle = nullptr;
  if (PyLong_Check(stream)) {
    if (!address(stream, &handle)) return false;
  } else {
    PyObject* s = PyObject_GetAttr(stream, s_cuda_stream);
    PyObject* of = s ? PyObject_GetAttr(stream, s_device_index) : nullptr;
    const bool fits = of && PyLong_Check(of) && PyLong_AsLong(of) == index && address(s, &handle);
    Py_XDECREF(s);
    Py_XDECREF(of);
    if (!fits) return pass();
  }
  if (handle == to->handle) return true;
  if (reinterpret_cast<uintptr_t>(handle) < 4096) return false;  // a default stream's handle
  to->handle = handle;
  to->other = c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(handle), (c10::DeviceIndex)index);
  return true;
}

at::Tensor empty(at::IntArrayRef size, at::ScalarType type, int index) {
  return at::Tensor(at::detail::empty_cuda(size, type, at::Device(at::kCUDA, (c10::DeviceIndex)index),
                                           std::nullopt));
}

int64_t code_bytes(int64_t rows, int fmt, int64_t K) { return rows * (fmt == STRATA_MX_FP4 ? K / 2 : K); }
int64_t scale_bytes(int64_t rows, int64_t K, int layout) {
  return layout == STRATA_MX_TILES ? (rows + 127) / 128 * ((K + 127) / 128) * 512 : rows * (K / 32);
}
bool format(long fmt, int64_t rows, int64_t K, long layout) {
  return (fmt == STRATA_MX_FP4 || fmt == STRATA_MX_FP8) &&
         (layout == STRATA_MX_ROWS || layout == STRATA_MX_TILES) && rows >= 0 && rows < 1LL << 31 &&
         K >= 32 && K < 1LL << 31 && K % 32 == 0;
}

// Where the scales are in one allocation of both planes.
int64_t scales_at(int fmt, int64_t rows, int64_t K) {
  return (code_bytes(rows, fmt, K) + 255) & ~(int64_t)255;
}

// An MXTensor as it is now.  Its tensors may have been given other memory
// since the last call, so each call asks them, as mx.py's _planes().
struct Mx {
  int fmt, layout, index;
  int64_t rows, K;
  uint8_t *codes, *scales;
};
bool plane(const Tensor& t, int64_t bytes) {
  if (t.dtype != 8) return false;
  if (t.dims == 1) return t.size[0] == bytes && (bytes <= 1 || t.stride[0] == 1);
  return t.rows_contiguous() && t.size[0] * t.size[1] == bytes;
}
bool read_mx(PyObject* o, Mx* q) {
  if (Py_TYPE(o) != mx_type) return false;
  const Matrix& m = *reinterpret_cast<Matrix*>(o);
  if (!format(m.fmt, m.rows, m.K, m.layout)) return false;
  q->fmt = m.fmt;
  q->layout = m.layout;
  q->rows = m.rows;
  q->K = m.K;
  int index[2];
  PyObject* own[2] = {m.codes, m.scales};
  uint8_t** at[2] = {&q->codes, &q->scales};
  const int64_t bytes[2] = {code_bytes(m.rows, m.fmt, m.K), scale_bytes(m.rows, m.K, m.layout)};
  const int64_t offset[2] = {0, scales_at(m.fmt, m.rows, m.K)};
  for (int i = 0; i < 2; ++i) {
    if (own[i] && own[i] != Py_None) {
      Tensor t;
      if (!read(own[i], &t) || !plane(t, bytes[i])) return false;
      index[i] = t.index;
      *at[i] = static_cast<uint8_t*>(t.ptr);
    } else {
      if (!m.both.defined() || !m.both.is_cuda()) return false;
      index[i] = m.both.device().index();
      *at[i] = static_cast<uint8_t*>(m.both.data_ptr()) + offset[i];
    }
  }
  q->index = index[0];
  return index[0] == index[1];
}

// Memory for an MXTensor that a call writes, both planes in one allocation.
struct Planes {
  at::Tensor both;
  uint8_t *codes = nullptr, *scales = nullptr;
  Planes() = default;
  Planes(int fmt, int64_t rows, int64_t K, int layout, int index) {
    const int64_t at = scales_at(fmt, rows, K);
    both = empty({at + scale_bytes(rows, K, layout)}, at::kByte, index);
    codes = static_cast<uint8_t*>(both.data_ptr());
    scales = codes + at;
  }
};
PyObject* new_matrix(Planes&& p, int fmt, int64_t rows, int64_t K, int layout) {
  PyObject* o = matrix_new(mx_type, nullptr, nullptr);
  if (!o) return nullptr;
  Matrix* m = reinterpret_cast<Matrix*>(o);
  m->fmt = fmt;
  m->layout = layout;
  m->rows = rows;
  m->K = K;
  m->both = std::move(p.both);
  return o;
}

// Makes the outputs and calls the library without the interpreter's lock (a
// call may wait for the allocator or the device).  Anything but STRATA_OK, an
// exception among it, leaves the call to mx.py.
template <typename F>
int32_t launch(const Target& to, F f) {
  int32_t rc = STRATA_ECUDA;
  Py_BEGIN_ALLOW_THREADS
  try {
    c10::cuda::OptionalCUDAStreamGuard guard;
    if (to.other) guard.reset_stream(*to.other);
    rc = f();
  } catch (const std::exception&) {
  }
  Py_END_ALLOW_THREADS
  return rc;
}
// A call's own part: exceptions (a tensor without memory of its own) are None.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    return F(args, n);
  } catch (const std::exception&) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

bool small_int(PyObject* o, long* v) {
  if (!PyLong_Check(o)) return false;
  *v = PyLong_AsLong(o);
  return !(*v == -1 && PyErr_Occurred()) || pass();
}

#define NOT_TAKEN      \
  do {                 \
    Py_RETURN_NONE;    \
  } while (0)

// ---------------------------------------------------------------- the calls
// Each returns None for a call it does not take, and for one that the library
// refuses (nothing was enqueued then; mx.py's own call says why).

PyObject* quantize(PyObject* const* args, Py_ssize_t n) {  // x, fmt, layout, stream
  Tensor x;
  long fmt, layout;
  Target to;
  if (n != 4 || !small_int(args[1], &fmt) || !small_int(args[2], &layout) || !read(args[0], &x) ||
      x.dims != 2 || x.dtype > 2 || !format(fmt, x.size[0], x.size[1], layout) ||
      !target(x.index, args[3], &to))
    NOT_TAKEN;
  if (x.size[0] > 0 && x.stride[1] != 1) NOT_TAKEN;
  Planes p;
  const int32_t rc = launch(to, [&] {
    p = Planes((int)fmt, x.size[0], x.size[1], (int)layout, x.index);
    return lib.quantize(x.ptr, x.dtype, 1, (int32_t)x.size[0], (int32_t)x.size[1], x.stride[0], 0,
                        (int32_t)fmt, p.codes, 0, p.scales, (int32_t)layout, 0, to.handle);
  });
  if (rc != STRATA_OK) NOT_TAKEN;
  return new_matrix(std::move(p), (int)fmt, x.size[0], x.size[1], (int)layout);
}

// q, codes, scales, fmt, rows, K, layout: fills in q; True where it did.
PyObject* wrap(PyObject* const* args, Py_ssize_t n) {
  Tensor codes, scales;
  long fmt, rows, K, layout;
  if (n != 7 || Py_TYPE(args[0]) != mx_type || !small_int(args[3], &fmt) ||
      !small_int(args[4], &rows) || !small_int(args[5], &K) || !small_int(args[6], &layout) ||
      !format(fmt, rows, K, layout) || !read(args[1], &codes) || !read(args[2], &scales) ||
      codes.index != scales.index || !plane(codes, code_bytes(rows, (int)fmt, K)) ||
      !plane(scales, scale_bytes(rows, K, (int)layout)))
    NOT_TAKEN;
  Matrix* m = reinterpret_cast<Matrix*>(args[0]);
  m->fmt = (int)fmt;
  m->layout = (int)layout;
  m->rows = rows;
  m->K = K;
  m->both = at::Tensor();
  Py_XSETREF(m->codes, Py_NewRef(args[1]));
  Py_XSETREF(m->scales, Py_NewRef(args[2]));
  Py_RETURN_TRUE;
}

PyObject* dequantize(PyObject* const* args, Py_ssize_t n) {  // q, dtype, stream
  Target to;
  Mx q;
  if (n != 3 || !read_mx(args[0], &q)) NOT_TAKEN;
  const int dt = dtype_of(args[1]);
  if (dt < 0 || !target(q.index, args[2], &to)) NOT_TAKEN;
  at::Tensor out;
  const int32_t rc = launch(to, [&] {
    out = empty({q.rows, q.K}, scalar_type(dt), q.index);
    return lib.dequantize(q.codes, 0, q.scales, q.layout, 0, q.fmt, 1, (int32_t)q.rows, (int32_t)q.K,
                          out.data_ptr(), dt, q.K, 0, to.handle);
  });
  if (rc != STRATA_OK) NOT_TAKEN;
  return THPVariable_Wrap(std::move(out));
}

// x, delta, gain, eps, out_dtype, fmt, layout, residual_out, stream
PyObject* add_rmsnorm(PyObject* const* args, Py_ssize_t n) {
  Tensor x, delta, gain, res;
  long fmt, layout;
  Target to;
  if (n != 9 || !PyFloat_Check(args[3]) || !small_int(args[5], &fmt) || !small_int(args[6], &layout) ||
      !read(args[0], &x) || x.dtype > 2 || !x.rows_contiguous() || x.size[0] >= 1LL << 31 ||
      x.size[1] >= 1LL << 31)
    NOT_TAKEN;
  const bool has_delta = args[1] != Py_None, has_gain = args[2] != Py_None;
  const bool has_out = args[4] != Py_None, has_res = args[7] != Py_None;
  const int od = has_out ? dtype_of(args[4]) : 0;
  if (od < 0 || (!has_out && !fmt) || (fmt && !format(fmt, x.size[0], x.size[1], layout))) NOT_TAKEN;
  auto like_x = [&](const Tensor& t) {
    return t.dtype <= 2 && t.index == x.index && t.rows_contiguous() && t.size[0] == x.size[0] &&
           t.size[1] == x.size[1];
  };
  if (has_delta && (!read(args[1], &delta) || !like_x(delta))) NOT_TAKEN;
  if (has_res && (!read(args[7], &res) || !like_x(res) || res.dtype != x.dtype)) NOT_TAKEN;
  if (has_gain && (!read(args[2], &gain) || gain.dtype != 0 || gain.index != x.index ||
                   gain.dims != 1 || gain.size[0] != x.size[1] ||
                   (gain.size[0] > 1 && gain.stride[0] != 1)))
    NOT_TAKEN;
  if (!target(x.index, args[8], &to)) NOT_TAKEN;
  const float eps = (float)PyFloat_AS_DOUBLE(args[3]);
  at::Tensor r, out;
  Planes p;
  const int32_t rc = launch(to, [&] {
    if (has_delta && !has_res) {
      r = empty({x.size[0], x.size[1]}, scalar_type(x.dtype), x.index);
      res.ptr = r.data_ptr();
    }
    if (has_out) out = empty({x.size[0], x.size[1]}, scalar_type(od), x.index);
    if (fmt) p = Planes((int)fmt, x.size[0], x.size[1], (int)layout, x.index);
    return lib.add_rmsnorm(x.ptr, x.dtype, delta.ptr, has_delta ? delta.dtype : 0,
                           static_cast<const float*>(gain.ptr), (int32_t)x.size[0],
                           (int32_t)x.size[1], eps, res.ptr, has_out ? out.data_ptr() : nullptr, od,
                           (int32_t)fmt, p.codes, p.scales, (int32_t)layout, to.handle);
  });
  if (rc != STRATA_OK) NOT_TAKEN;
  // AddNorm((residual, out, mx)), by the tuple's constructor
  PyObject* parts = PyTuple_New(3);
  PyObject* one = parts ? PyTuple_Pack(1, parts) : nullptr;
  PyObject* result = nullptr;
  if (one) {
    PyObject* a = has_res ? Py_NewRef(args[7]) : has_delta ? THPVariable_Wrap(std::move(r)) : Py_NewRef(args[0]);
    PyObject* b = has_out ? THPVariable_Wrap(std::move(out)) : Py_NewRef(Py_None);
    PyObject* c = fmt ? new_matrix(std::move(p), (int)fmt, x.size[0], x.size[1], (int)layout)
                      : Py_NewRef(Py_None);
    PyTuple_SET_ITEM(parts, 0, a);
    PyTuple_SET_ITEM(parts, 1, b);
    PyTuple_SET_ITEM(parts, 2, c);
    if (a && b && c) result = PyTuple_Type.tp_new(norm_type, one, nullptr);
  }
  Py_XDECREF(one);
  Py_XDECREF(parts);
  return result;
}

// x, w, bias, out_dtype, out, dev_status, stream
PyObject* linear(PyObject* const* args, Py_ssize_t n) {
  Mx x, w;
  if (n != 7 || !read_mx(args[0], &x) || !read_mx(args[1], &w)) NOT_TAKEN;
  Tensor bias, out, status;
  Target to;
  if (x.K != w.K || x.layout != STRATA_MX_TILES || w.layout != STRATA_MX_TILES || x.index != w.index)
    NOT_TAKEN;
  const bool has_bias = args[2] != Py_None, has_out = args[4] != Py_None;
  if (has_bias && (!read(args[2], &bias) || bias.dtype != 0 || bias.index != x.index ||
                   bias.dims != 1 || bias.size[0] != w.rows || (bias.size[0] > 1 && bias.stride[0] != 1)))
    NOT_TAKEN;
  if (args[5] != Py_None && (!read(args[5], &status) || status.dtype != 32 ||
                             status.index != x.index || status.dims != 1 || status.size[0] < 1))
    NOT_TAKEN;
  int64_t ldy = w.rows;
  int dt = has_out ? -1 : dtype_of(args[3]);
  if (has_out) {
    if (!read(args[4], &out) || out.dtype > 2 || out.index != x.index || out.dims != 2 ||
        out.size[0] != x.rows || out.size[1] != w.rows || (w.rows > 1 && out.stride[1] != 1) ||
        (x.rows > 1 && out.stride[0] < w.rows))
      NOT_TAKEN;
    dt = out.dtype;
    if (x.rows > 1) ldy = out.stride[0];
  }
  if (dt < 0 || !target(x.index, args[6], &to)) NOT_TAKEN;
  at::Tensor y;
  const int32_t rc = launch(to, [&] {
    if (!has_out) {
      y = empty({x.rows, w.rows}, scalar_type(dt), x.index);
      out.ptr = y.data_ptr();
    }
    return lib.linear(x.codes, x.fmt, x.scales, (int32_t)x.rows, w.codes, w.fmt, w.scales,
                      (int32_t)w.rows, (int32_t)w.K, static_cast<const float*>(bias.ptr), out.ptr,
                      dt, ldy, static_cast<int32_t*>(status.ptr), to.handle);
  });
  if (rc != STRATA_OK) NOT_TAKEN;
  return has_out ? Py_NewRef(args[4]) : THPVariable_Wrap(std::move(y));
}

PyObject* pack(PyObject* const* args, Py_ssize_t n) {  // gate, up, down, stream: the blobs
  Tensor w[3];
  Target to;
  if (n != 4) NOT_TAKEN;
  int64_t rows[3], experts[3];
  for (int i = 0; i < 3; ++i) {
    if (!read(args[i], &w[i]) || w[i].dims != 3 || w[i].dtype > 2 || w[i].stride[2] != 1 ||
        w[i].dtype != w[0].dtype || w[i].index != w[0].index)
      NOT_TAKEN;
    rows[i] = w[i].stride[1];
    experts[i] = w[i].stride[0];
  }
  const int64_t E = w[0].size[0], I = w[0].size[1], H = w[0].size[2];
  if (E < 1 || I < 128 || H < 128 || E >> 31 || I >> 31 || H >> 31 || w[1].size[0] != E ||
      w[1].size[1] != I || w[1].size[2] != H || w[2].size[0] != E || w[2].size[1] != H ||
      w[2].size[2] != I || !target(w[0].index, args[3], &to))
    NOT_TAKEN;
  at::Tensor blobs;
  const int32_t rc = launch(to, [&] {
    const int64_t bytes = (int64_t)lib.expert_bytes(STRATA_FMT_MXFP4_32, (int32_t)H, (int32_t)I);
    if (!bytes) return (int32_t)STRATA_EINVAL;
    blobs = empty({E, bytes}, at::kByte, w[0].index);
    return lib.pack(w[0].ptr, w[1].ptr, w[2].ptr, w[0].dtype, rows, experts, (int32_t)E, (int32_t)H,
                    (int32_t)I, blobs.data_ptr(), (uint64_t)bytes, to.handle);
  });
  if (rc != STRATA_OK) NOT_TAKEN;
  return THPVariable_Wrap(std::move(blobs));
}

PyObject* unpack(PyObject* const* args, Py_ssize_t n) {  // blobs, H, I, dtype, stream
  Tensor b;
  long H, I;
  Target to;
  if (n != 5 || !read(args[0], &b) || b.dims != 2 || b.dtype != 8 || b.stride[1] != 1 ||
      b.size[0] >> 31 || !small_int(args[1], &H) || !small_int(args[2], &I) || H < 128 || I < 128 ||
      H >> 31 || I >> 31)
    NOT_TAKEN;
  const int dt = dtype_of(args[3]);
  if (dt < 0 || !target(b.index, args[4], &to)) NOT_TAKEN;
  at::Tensor w[3];
  const int32_t rc = launch(to, [&] {
    for (int i = 0; i < 3; ++i)
      w[i] = i < 2 ? empty({b.size[0], I, H}, scalar_type(dt), b.index)
                   : empty({b.size[0], H, I}, scalar_type(dt), b.index);
    return lib.unpack(b.ptr, (uint64_t)b.stride[0], (int32_t)b.size[0], (int32_t)H, (int32_t)I,
                      w[0].data_ptr(), w[1].data_ptr(), w[2].data_ptr(), dt, to.handle);
  });
  if (rc != STRATA_OK) NOT_TAKEN;
  PyObject* all = PyTuple_New(3);
  for (int i = 0; all && i < 3; ++i) {
    PyObject* o = THPVariable_Wrap(std::move(w[i]));
    if (!o) {
      Py_CLEAR(all);
      break;
    }
    PyTuple_SET_ITEM(all, i, o);
  }
  return all;
}

// setup(addresses, torch.Tensor, Parameter, MXTensor, AddNorm)
PyObject* setup(PyObject*, PyObject* args) {
  unsigned long long f[7];
  PyObject* o[4];
  if (!PyArg_ParseTuple(args, "(KKKKKKK)OOOO", &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &f[6], &o[0],
                        &o[1], &o[2], &o[3]))
    return nullptr;
  if (!PyType_Check(o[2]) || !PyType_IsSubtype((PyTypeObject*)o[2], matrix_type) ||
      !PyType_Check(o[3]) || !PyType_IsSubtype((PyTypeObject*)o[3], &PyTuple_Type)) {
    PyErr_SetString(PyExc_TypeError, "MXTensor must be a subclass of Matrix, AddNorm of tuple");
    return nullptr;
  }
  lib.quantize = reinterpret_cast<decltype(lib.quantize)>(f[0]);
  lib.dequantize = reinterpret_cast<decltype(lib.dequantize)>(f[1]);
  lib.add_rmsnorm = reinterpret_cast<decltype(lib.add_rmsnorm)>(f[2]);
  lib.linear = reinterpret_cast<decltype(lib.linear)>(f[3]);
  lib.pack = reinterpret_cast<decltype(lib.pack)>(f[4]);
  lib.unpack = reinterpret_cast<decltype(lib.unpack)>(f[5]);
  lib.expert_bytes = reinterpret_cast<decltype(lib.expert_bytes)>(f[6]);
  Py_XSETREF(torch_tensor, Py_NewRef(o[0]));
  Py_XSETREF(torch_param, Py_NewRef(o[1]));
  Py_XSETREF(mx_type, reinterpret_cast<PyTypeObject*>(Py_NewRef(o[2])));
  Py_XSETREF(norm_type, reinterpret_cast<PyTypeObject*>(Py_NewRef(o[3])));
  Py_RETURN_NONE;
}

#define CALL(f) {#f, (PyCFunction)(void*)call<f>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, "Hands over the library's functions and mx.py's types."},
    CALL(wrap),         // MXTensor's fields: True, or None
    CALL(quantize),     // what mx.py's function of the name returns, or None
    CALL(dequantize),
    CALL(add_rmsnorm),
    CALL(linear),
    CALL(pack),         // pack_experts' blobs, or None
    CALL(unpack),       // what unpack_experts returns, or None
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_mxcalls",
                          "The host's part of the microscaled calls.", -1, methods,
                          nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mxcalls(void) {
  s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  s_device_index = PyUnicode_InternFromString("device_index");
  PyObject* m = PyModule_Create(&module_def);
  PyObject* type = PyType_FromSpec(&matrix_spec);
  matrix_type = reinterpret_cast<PyTypeObject*>(type);
  if (!m || !type || !s_cuda_stream || !s_device_index || PyModule_AddObject(m, "Matrix", type) < 0 ||
      PyModule_AddStringConstant(m, "torch_version", STRATA_TORCH) < 0)
    return nullptr;
  return m;
}
