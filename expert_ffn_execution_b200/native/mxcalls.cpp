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
// Only the CPython interface is used: tensors are read through their Python
// attributes and made by torch.empty.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stddef.h>
#include <stdint.h>
#include <structmember.h>

#include "strata_moe.h"

namespace {

// ---------------------------------------------------------------- what setup() hands over
struct Library {
  decltype(&moe_mx_quantize) quantize;
  decltype(&moe_mx_dequantize) dequantize;
  decltype(&moe_add_rmsnorm) add_rmsnorm;
  decltype(&moe_mx_linear) linear;
} lib;
PyObject* torch_empty;     // torch.empty
PyObject* torch_tensor;    // torch.Tensor
PyObject* torch_param;     // torch.nn.Parameter
PyObject* current_device;  // () -> index
PyObject* current_stream;  // index -> handle
PyObject* dtypes[3];       // float32, float16, bfloat16, by STRATA_DTYPE_*
PyObject* uint8;
PyObject* int32;
PyTypeObject* matrix_type; // Matrix below
PyTypeObject* mx_type;     // mx.py's MXTensor, a subclass of it
PyObject* add_norm;        // mx.py's AddNorm
PyObject* devices[64];     // torch.device("cuda", i), as they are met
PyObject* torch_device;

// interned names
PyObject *s_shape, *s_stride, *s_dtype, *s_data_ptr, *s_get_device, *s_cuda_stream, *s_cuda;
PyObject *kw_empty;  // ("dtype", "device")

// ---------------------------------------------------------------- MXTensor's fields
struct Matrix {
  PyObject_HEAD
  int fmt, layout;
  Py_ssize_t rows, K;
  unsigned long long codes_ptr, scales_ptr;
  int index;  // of the CUDA device, -1: none
  PyObject* device;
  PyObject *both, *codes, *scales;  // one allocation, or the two planes' tensors
};

int matrix_traverse(PyObject* o, visitproc visit, void* arg) {
  Matrix* m = reinterpret_cast<Matrix*>(o);
  Py_VISIT(Py_TYPE(o));
  Py_VISIT(m->device);
  Py_VISIT(m->both);
  Py_VISIT(m->codes);
  Py_VISIT(m->scales);
  return 0;
}
int matrix_clear(PyObject* o) {
  Matrix* m = reinterpret_cast<Matrix*>(o);
  Py_CLEAR(m->device);
  Py_CLEAR(m->both);
  Py_CLEAR(m->codes);
  Py_CLEAR(m->scales);
  return 0;
}
void matrix_dealloc(PyObject* o) {
  PyTypeObject* type = Py_TYPE(o);
  PyObject_GC_UnTrack(o);
  matrix_clear(o);
  type->tp_free(o);
  Py_DECREF(type);
}
PyMemberDef matrix_members[] = {
    {"fmt", T_INT, offsetof(Matrix, fmt), 0, nullptr},
    {"layout", T_INT, offsetof(Matrix, layout), 0, nullptr},
    {"rows", T_PYSSIZET, offsetof(Matrix, rows), 0, nullptr},
    {"K", T_PYSSIZET, offsetof(Matrix, K), 0, nullptr},
    {"codes_ptr", T_ULONGLONG, offsetof(Matrix, codes_ptr), 0, nullptr},
    {"scales_ptr", T_ULONGLONG, offsetof(Matrix, scales_ptr), 0, nullptr},
    {"index", T_INT, offsetof(Matrix, index), 0, nullptr},
    {"device", T_OBJECT, offsetof(Matrix, device), 0, nullptr},
    {"_both", T_OBJECT, offsetof(Matrix, both), 0, nullptr},
    {"_codes", T_OBJECT, offsetof(Matrix, codes), 0, nullptr},
    {"_scales", T_OBJECT, offsetof(Matrix, scales), 0, nullptr},
    {nullptr, 0, 0, 0, nullptr}};
PyType_Slot matrix_slots[] = {{Py_tp_traverse, (void*)matrix_traverse},
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

struct Tensor {
  int dtype = -1;  // STRATA_DTYPE_*, 8: uint8, 32: int32
  int index = -1;
  uint64_t ptr = 0;
  int dims = 0;
  int64_t size[2] = {0, 0}, stride[2] = {0, 0};
  bool rows_contiguous() const {
    return dims == 2 && (size[1] <= 1 || stride[1] == 1) &&
           (size[0] <= 1 || stride[0] == size[1] || size[1] == 0);
  }
};

bool number(PyObject* o, int64_t* v) {  // steals o
  if (!o) return pass();
  *v = PyLong_AsLongLong(o);
  Py_DECREF(o);
  return !(*v == -1 && PyErr_Occurred()) || pass();
}

// Reads a torch.Tensor (or Parameter; no other subclass) of one or two dimensions.
bool read(PyObject* o, Tensor* t) {
  PyObject* type = reinterpret_cast<PyObject*>(Py_TYPE(o));
  if (type != torch_tensor && type != torch_param) return false;
  PyObject* d = PyObject_GetAttr(o, s_dtype);
  if (!d) return pass();
  t->dtype = d == dtypes[0] ? 0 : d == dtypes[1] ? 1 : d == dtypes[2] ? 2 : d == uint8 ? 8 : d == int32 ? 32 : -1;
  Py_DECREF(d);
  if (t->dtype < 0) return false;
  int64_t v;
  if (!number(PyObject_CallMethodNoArgs(o, s_get_device), &v) || v < 0 || v >= 64) return false;
  t->index = (int)v;
  if (!number(PyObject_CallMethodNoArgs(o, s_data_ptr), &v)) return false;
  t->ptr = (uint64_t)v;
  PyObject* shape = PyObject_GetAttr(o, s_shape);
  PyObject* stride = PyObject_CallMethodNoArgs(o, s_stride);
  bool ok = shape && stride && PyTuple_Check(shape) && PyTuple_Check(stride);
  if (ok) {
    t->dims = (int)PyTuple_GET_SIZE(shape);
    ok = (t->dims == 1 || t->dims == 2) && PyTuple_GET_SIZE(stride) == t->dims;
    for (int i = 0; ok && i < t->dims; ++i) {
      t->size[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i));
      t->stride[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(stride, i));
    }
  }
  Py_XDECREF(shape);
  Py_XDECREF(stride);
  return PyErr_Occurred() || !ok ? pass() : true;
}

bool is_mx(PyObject* o) { return Py_TYPE(o) == mx_type; }

int dtype_of(PyObject* o) { return o == dtypes[0] ? 0 : o == dtypes[1] ? 1 : o == dtypes[2] ? 2 : -1; }

// The stream's handle on device `index`, which has to be the current one.
bool target(int index, PyObject* stream, void** handle) {
  int64_t v;
  if (!number(PyObject_CallNoArgs(current_device), &v) || v != index) return false;
  PyObject* s;
  if (stream == Py_None) {
    PyObject* i = PyLong_FromLong(index);
    if (!i) return pass();
    s = PyObject_CallOneArg(current_stream, i);
    Py_DECREF(i);
  } else if (PyLong_Check(stream)) {
    s = Py_NewRef(stream);
  } else {
    s = PyObject_GetAttr(stream, s_cuda_stream);
  }
  if (!number(s, &v)) return false;
  *handle = reinterpret_cast<void*>(v);
  return true;
}

PyObject* device_object(int index) {  // borrowed
  if (!devices[index])
    devices[index] = PyObject_CallFunction(torch_device, "Oi", s_cuda, index);
  return devices[index];
}

// torch.empty(a[, b], dtype=dtype, device=device): a new reference, and its address.
PyObject* empty(int dims, int64_t a, int64_t b, PyObject* dtype, PyObject* device, uint64_t* ptr) {
  PyObject* args[5] = {nullptr, PyLong_FromLongLong(a), nullptr, nullptr, nullptr};
  int n = 1;
  if (dims == 2) args[1 + n++] = PyLong_FromLongLong(b);
  args[1 + n] = dtype;
  args[2 + n] = device;
  PyObject* t = nullptr;
  if (args[1] && args[n])
    t = PyObject_Vectorcall(torch_empty, args + 1, (size_t)n | PY_VECTORCALL_ARGUMENTS_OFFSET, kw_empty);
  Py_XDECREF(args[1]);
  if (dims == 2) Py_XDECREF(args[2]);
  if (!t) return nullptr;
  PyObject* p = PyObject_CallMethodNoArgs(t, s_data_ptr);
  *ptr = p ? PyLong_AsUnsignedLongLong(p) : 0;
  Py_XDECREF(p);
  if (PyErr_Occurred()) Py_CLEAR(t);
  return t;
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

// An MXTensor to be written by a call, both planes in one allocation.
Matrix* new_matrix(int fmt, int64_t rows, int64_t K, int layout, int index) {
  PyObject* dev = device_object(index);
  if (!dev) return nullptr;
  Matrix* m = reinterpret_cast<Matrix*>(mx_type->tp_alloc(mx_type, 0));
  if (!m) return nullptr;
  const int64_t at = (code_bytes(rows, fmt, K) + 255) & ~(int64_t)255;
  uint64_t ptr = 0;
  m->both = empty(1, at + scale_bytes(rows, K, layout), 0, uint8, dev, &ptr);
  if (!m->both) {
    Py_DECREF(m);
    return nullptr;
  }
  m->fmt = fmt;
  m->layout = layout;
  m->rows = rows;
  m->K = K;
  m->index = index;
  m->device = Py_NewRef(dev);
  m->codes = Py_NewRef(Py_None);
  m->scales = Py_NewRef(Py_None);
  m->codes_ptr = ptr;
  m->scales_ptr = ptr + at;
  return m;
}

template <typename F>
int32_t launch(F f) {
  int32_t rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f();
  Py_END_ALLOW_THREADS
  return rc;
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

PyObject* quantize(PyObject*, PyObject* const* args, Py_ssize_t n) {  // x, fmt, layout, stream
  Tensor x;
  long fmt, layout;
  void* stream;
  if (n != 4 || !small_int(args[1], &fmt) || !small_int(args[2], &layout) || !read(args[0], &x) ||
      x.dims != 2 || x.dtype > 2 || !format(fmt, x.size[0], x.size[1], layout) ||
      !target(x.index, args[3], &stream))
    NOT_TAKEN;
  if (x.size[0] > 0 && x.stride[1] != 1) NOT_TAKEN;
  Matrix* m = new_matrix((int)fmt, x.size[0], x.size[1], (int)layout, x.index);
  if (!m) return nullptr;
  const int32_t rc = launch([&] {
    return lib.quantize(reinterpret_cast<const void*>(x.ptr), x.dtype, 1, (int32_t)m->rows,
                        (int32_t)m->K, x.stride[0], 0, m->fmt, reinterpret_cast<void*>(m->codes_ptr), 0,
                        reinterpret_cast<void*>(m->scales_ptr), m->layout, 0, stream);
  });
  if (rc != STRATA_OK) {
    Py_DECREF(m);
    NOT_TAKEN;
  }
  return reinterpret_cast<PyObject*>(m);
}

// q, codes, scales, fmt, rows, K, layout: fills in q; True where it did.
PyObject* wrap(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Tensor codes, scales;
  long fmt, rows, K, layout;
  if (n != 7 || !is_mx(args[0]) || !read(args[1], &codes) || !read(args[2], &scales) ||
      !small_int(args[3], &fmt) || !small_int(args[4], &rows) || !small_int(args[5], &K) ||
      !small_int(args[6], &layout) || !format(fmt, rows, K, layout))
    Py_RETURN_FALSE;
  auto plane = [](const Tensor& t, int64_t bytes) {
    if (t.dims == 1) return t.size[0] == bytes && (bytes <= 1 || t.stride[0] == 1);
    return t.rows_contiguous() && t.size[0] * t.size[1] == bytes;
  };
  if (codes.dtype != 8 || scales.dtype != 8 || codes.index != scales.index ||
      !plane(codes, code_bytes(rows, (int)fmt, K)) || !plane(scales, scale_bytes(rows, K, (int)layout)))
    Py_RETURN_FALSE;
  PyObject* dev = device_object(codes.index);
  if (!dev) return nullptr;
  Matrix* m = reinterpret_cast<Matrix*>(args[0]);
  m->fmt = (int)fmt;
  m->layout = (int)layout;
  m->rows = rows;
  m->K = K;
  m->index = codes.index;
  m->codes_ptr = codes.ptr;
  m->scales_ptr = scales.ptr;
  Py_XSETREF(m->device, Py_NewRef(dev));
  Py_XSETREF(m->both, Py_NewRef(Py_None));
  Py_XSETREF(m->codes, Py_NewRef(args[1]));
  Py_XSETREF(m->scales, Py_NewRef(args[2]));
  Py_RETURN_TRUE;
}

PyObject* dequantize(PyObject*, PyObject* const* args, Py_ssize_t n) {  // q, dtype, stream
  void* stream;
  if (n != 3 || !is_mx(args[0])) NOT_TAKEN;
  Matrix* m = reinterpret_cast<Matrix*>(args[0]);
  const int dt = dtype_of(args[1]);
  if (dt < 0 || m->index < 0 || !target(m->index, args[2], &stream)) NOT_TAKEN;
  uint64_t ptr = 0;
  PyObject* out = empty(2, m->rows, m->K, args[1], m->device, &ptr);
  if (!out) return nullptr;
  const int32_t rc = launch([&] {
    return lib.dequantize(reinterpret_cast<const void*>(m->codes_ptr), 0,
                          reinterpret_cast<const void*>(m->scales_ptr), m->layout, 0, m->fmt, 1,
                          (int32_t)m->rows, (int32_t)m->K, reinterpret_cast<void*>(ptr), dt, m->K, 0,
                          stream);
  });
  if (rc != STRATA_OK) {
    Py_DECREF(out);
    NOT_TAKEN;
  }
  return out;
}

// x, delta, gain, eps, out_dtype, fmt, layout, residual_out, stream
PyObject* add_rmsnorm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Tensor x, delta, gain, res;
  long fmt, layout;
  void* stream;
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
  if (!target(x.index, args[8], &stream)) NOT_TAKEN;
  PyObject* dev = device_object(x.index);
  if (!dev) return nullptr;
  PyObject *r = nullptr, *out = nullptr, *result = nullptr;
  Matrix* m = nullptr;
  uint64_t r_ptr = 0, out_ptr = 0;
  int32_t rc = STRATA_OK;
  if (has_res) {
    r = Py_NewRef(args[7]);
    r_ptr = res.ptr;
  } else if (has_delta) {
    r = empty(2, x.size[0], x.size[1], dtypes[x.dtype], dev, &r_ptr);
    if (!r) goto end;
  } else {
    r = Py_NewRef(args[0]);
  }
  if (has_out) {
    out = empty(2, x.size[0], x.size[1], args[4], dev, &out_ptr);
    if (!out) goto end;
  } else {
    out = Py_NewRef(Py_None);
  }
  if (fmt && !(m = new_matrix((int)fmt, x.size[0], x.size[1], (int)layout, x.index))) goto end;
  rc = launch([&] {
    return lib.add_rmsnorm(
        reinterpret_cast<const void*>(x.ptr), x.dtype, reinterpret_cast<const void*>(delta.ptr),
        has_delta ? delta.dtype : 0, reinterpret_cast<const float*>(gain.ptr), (int32_t)x.size[0],
        (int32_t)x.size[1], (float)PyFloat_AS_DOUBLE(args[3]), reinterpret_cast<void*>(r_ptr),
        reinterpret_cast<void*>(out_ptr), od, (int32_t)fmt,
        reinterpret_cast<void*>(m ? m->codes_ptr : 0), reinterpret_cast<void*>(m ? m->scales_ptr : 0),
        (int32_t)layout, stream);
  });
  if (rc == STRATA_OK) {
    PyObject* parts[3] = {r, out, m ? reinterpret_cast<PyObject*>(m) : Py_None};
    result = PyObject_Vectorcall(add_norm, parts, 3, nullptr);
  } else {
    result = Py_NewRef(Py_None);
  }
end:
  Py_XDECREF(r);
  Py_XDECREF(out);
  Py_XDECREF(m);
  return result;
}

// x, w, bias, out_dtype, out, dev_status, stream
PyObject* linear(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 7 || !is_mx(args[0]) || !is_mx(args[1])) NOT_TAKEN;
  Matrix *x = reinterpret_cast<Matrix*>(args[0]), *w = reinterpret_cast<Matrix*>(args[1]);
  Tensor bias, out, status;
  void* stream;
  if (x->K != w->K || x->layout != STRATA_MX_TILES || w->layout != STRATA_MX_TILES || x->index < 0 ||
      x->index != w->index)
    NOT_TAKEN;
  const bool has_bias = args[2] != Py_None, has_out = args[4] != Py_None;
  if (has_bias && (!read(args[2], &bias) || bias.dtype != 0 || bias.index != x->index ||
                   bias.dims != 1 || bias.size[0] != w->rows || (bias.size[0] > 1 && bias.stride[0] != 1)))
    NOT_TAKEN;
  if (args[5] != Py_None && (!read(args[5], &status) || status.dtype != 32 ||
                             status.index != x->index || status.dims != 1 || status.size[0] < 1))
    NOT_TAKEN;
  int64_t ldy = w->rows;
  int dt = has_out ? -1 : dtype_of(args[3]);
  if (has_out) {
    if (!read(args[4], &out) || out.dtype > 2 || out.index != x->index || out.dims != 2 ||
        out.size[0] != x->rows || out.size[1] != w->rows || (w->rows > 1 && out.stride[1] != 1) ||
        (x->rows > 1 && out.stride[0] < w->rows))
      NOT_TAKEN;
    dt = out.dtype;
    if (x->rows > 1) ldy = out.stride[0];
  }
  if (dt < 0 || !target(x->index, args[6], &stream)) NOT_TAKEN;
  PyObject* y;
  if (has_out) {
    y = Py_NewRef(args[4]);
  } else {
    y = empty(2, x->rows, w->rows, args[3], x->device, &out.ptr);
    if (!y) return nullptr;
  }
  const int32_t rc = launch([&] {
    return lib.linear(reinterpret_cast<const void*>(x->codes_ptr), x->fmt,
                      reinterpret_cast<const void*>(x->scales_ptr), (int32_t)x->rows,
                      reinterpret_cast<const void*>(w->codes_ptr), w->fmt,
                      reinterpret_cast<const void*>(w->scales_ptr), (int32_t)w->rows, (int32_t)w->K,
                      reinterpret_cast<const float*>(bias.ptr), reinterpret_cast<void*>(out.ptr), dt,
                      ldy, reinterpret_cast<int32_t*>(status.ptr), stream);
  });
  if (rc != STRATA_OK) {
    Py_DECREF(y);
    NOT_TAKEN;
  }
  return y;
}

// setup(addresses, torch.empty, torch.Tensor, Parameter, torch.device, current_device, current_stream,
//       (float32, float16, bfloat16, uint8, int32), MXTensor, AddNorm)
PyObject* setup(PyObject*, PyObject* args) {
  unsigned long long f[4];
  PyObject* o[8];
  PyObject* t[5];
  if (!PyArg_ParseTuple(args, "(KKKK)OOOOOO(OOOOO)OO", &f[0], &f[1], &f[2], &f[3], &o[0], &o[1],
                        &o[2], &o[3], &o[4], &o[5], &t[0], &t[1], &t[2], &t[3], &t[4], &o[6], &o[7]))
    return nullptr;
  if (!PyType_Check(o[6]) || !PyType_IsSubtype((PyTypeObject*)o[6], matrix_type)) {
    PyErr_SetString(PyExc_TypeError, "MXTensor must be a subclass of Matrix");
    return nullptr;
  }
  lib.quantize = reinterpret_cast<decltype(lib.quantize)>(f[0]);
  lib.dequantize = reinterpret_cast<decltype(lib.dequantize)>(f[1]);
  lib.add_rmsnorm = reinterpret_cast<decltype(lib.add_rmsnorm)>(f[2]);
  lib.linear = reinterpret_cast<decltype(lib.linear)>(f[3]);
  PyObject** to[] = {&torch_empty,  &torch_tensor,   &torch_param,
                     &torch_device, &current_device, &current_stream};
  for (int i = 0; i < 6; ++i) Py_XSETREF(*to[i], Py_NewRef(o[i]));
  for (int i = 0; i < 3; ++i) Py_XSETREF(dtypes[i], Py_NewRef(t[i]));
  Py_XSETREF(uint8, Py_NewRef(t[3]));
  Py_XSETREF(int32, Py_NewRef(t[4]));
  Py_XSETREF(mx_type, reinterpret_cast<PyTypeObject*>(Py_NewRef(o[6])));
  Py_XSETREF(add_norm, Py_NewRef(o[7]));
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, "Hands over the library's functions and torch's."},
    {"wrap", (PyCFunction)(void*)wrap, METH_FASTCALL, "MXTensor's fields; False where it does not take them."},
    {"quantize", (PyCFunction)(void*)quantize, METH_FASTCALL, "mx_quantize, or None."},
    {"dequantize", (PyCFunction)(void*)dequantize, METH_FASTCALL, "MXTensor.dequantize, or None."},
    {"add_rmsnorm", (PyCFunction)(void*)add_rmsnorm, METH_FASTCALL, "add_rmsnorm, or None."},
    {"linear", (PyCFunction)(void*)linear, METH_FASTCALL, "mx_linear, or None."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_mxcalls",
                          "The host's part of the microscaled calls.", -1, methods,
                          nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mxcalls(void) {
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  s_dtype = PyUnicode_InternFromString("dtype");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  s_cuda = PyUnicode_InternFromString("cuda");
  kw_empty = Py_BuildValue("(ss)", "dtype", "device");
  PyObject* m = PyModule_Create(&module_def);
  PyObject* type = PyType_FromSpec(&matrix_spec);
  matrix_type = reinterpret_cast<PyTypeObject*>(type);
  if (!m || !type || !kw_empty || PyModule_AddObject(m, "Matrix", type) < 0) return nullptr;
  return m;
}
