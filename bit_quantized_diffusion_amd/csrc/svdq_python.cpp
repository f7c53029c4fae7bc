// Python side of the 16-bit and 8-bit block operators: argument checks, output and
// workspace tensors, the device and the stream of a call.
//
// The smallest calls take longer on the host than on the device.  With the
// same checks in Python and a ctypes call one of 77 tokens x 12 heads took 9.6
// us (attention), of 1 x 256 x 3072 8.9 (linear16) and of 1 x 768 8.1 (layer
// norm); so they take 6.8, 6.2 and 6.2, of which the launch is 3.6.  Tensors
// are seen through their Python methods (dtype, get_device, shape, stride,
// data_ptr, new_empty) alone.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/svdq.h"

namespace {

// set once by setup(): torch's Tensor, dtypes and functions
PyObject *g_tensor, *g_bf16, *g_f16, *g_f32, *g_u8, *g_i32, *g_stream, *g_current, *g_set_device, *g_check, *g_f8, *g_i8;
PyObject *s_dtype, *s_shape, *s_stride, *s_get_device, *s_data_ptr, *s_new_empty, *s_is_contiguous, *s_numel;
PyObject* s_kw_dtype;   // ("dtype",)

constexpr int64_t kMost = (int64_t(1) << 31) - (int64_t(1) << 16);   // rows that the library counts

class Ref {
 public:
  explicit Ref(PyObject* p = nullptr) : p_(p) {}
  ~Ref() { Py_XDECREF(p_); }
  Ref(const Ref&) = delete;
  Ref& operator=(const Ref&) = delete;
  void reset(PyObject* p) {
    Py_XDECREF(p_);
    p_ = p;
  }
  PyObject* get() const { return p_; }
  PyObject* release() {
    PyObject* p = p_;
    p_ = nullptr;
    return p;
  }
  explicit operator bool() const { return p_ != nullptr; }

 private:
  PyObject* p_;
};

constexpr int kDims = 5;

// What a call needs to know of a tensor.  More than kDims dimensions: dims
// alone is true.
struct Tensor {
  PyObject* dtype = nullptr;   // borrowed: torch's dtypes are never freed
  int64_t shape[kDims] = {}, stride[kDims] = {};
  int dims = 0;
  long device = -1;
  void* ptr = nullptr;

  bool dense() const { return dims == 0 || shape[dims - 1] <= 1 || stride[dims - 1] == 1; }
  // row stride of a matrix (a single row has none, and gets its length)
  int64_t ld() const { return shape[0] > 1 ? stride[0] : shape[1]; }
};

bool read(PyObject* t, Tensor& out) {
  if (!PyType_IsSubtype(Py_TYPE(t), reinterpret_cast<PyTypeObject*>(g_tensor))) {
    PyErr_SetString(PyExc_TypeError, "not a tensor");
    return false;
  }
  Ref dtype(PyObject_GetAttr(t, s_dtype));
  if (!dtype) return false;
  out.dtype = dtype.get();
  Ref device(PyObject_CallMethodNoArgs(t, s_get_device));
  if (!device) return false;
  out.device = PyLong_AsLong(device.get());
  Ref shape(PyObject_GetAttr(t, s_shape)), stride(PyObject_CallMethodNoArgs(t, s_stride));
  Ref ptr(PyObject_CallMethodNoArgs(t, s_data_ptr));
  if (!shape || !stride || !ptr) return false;
  out.ptr = PyLong_AsVoidPtr(ptr.get());
  if (!PyTuple_Check(shape.get()) || !PyTuple_Check(stride.get()) ||
      PyTuple_GET_SIZE(shape.get()) != PyTuple_GET_SIZE(stride.get())) {
    PyErr_SetString(PyExc_TypeError, "not a tensor");
    return false;
  }
  out.dims = static_cast<int>(PyTuple_GET_SIZE(shape.get()));
  for (int i = 0; i < out.dims && i < kDims; ++i) {
    out.shape[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(shape.get(), i));
    out.stride[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(stride.get(), i));
  }
  return !PyErr_Occurred();
}

// What is not a tensor on a device at all.
bool no_tensor(const char* name, const char* layout) {
  if (PyErr_Occurred()) {
    if (!PyErr_ExceptionMatches(PyExc_AttributeError) && !PyErr_ExceptionMatches(PyExc_RuntimeError) &&
        !PyErr_ExceptionMatches(PyExc_TypeError))
      return false;
    PyErr_Clear();
  }
  PyErr_Format(PyExc_TypeError, "%s: expected a device tensor%s%s", name, *layout ? " " : "", layout);
  return false;
}

bool not_dense(const char* name) {
  PyErr_Format(PyExc_ValueError, "%s: the last dimension must be contiguous", name);
  return false;
}

// A call's first operand.
bool operand(PyObject* o, int dims, const char* name, const char* layout, Tensor& t, int& code) {
  if (!read(o, t)) return no_tensor(name, layout);
  if (t.dtype != g_bf16 && t.dtype != g_f16) {
    PyErr_Format(PyExc_TypeError, "%s: expected a bfloat16 or float16 tensor, got %S", name, t.dtype);
    return false;
  }
  if (t.dims != dims || t.device < 0) return no_tensor(name, layout);
  if (!t.dense()) return not_dense(name);
  code = t.dtype == g_bf16 ? SVDQ_BF16 : SVDQ_F16;
  return true;
}

bool same_kind(PyObject* o, const Tensor& first, const char* name, Tensor& t) {
  if (!read(o, t)) return no_tensor(name, "");
  if (t.dtype == first.dtype && t.device == first.device) return true;
  PyErr_Format(PyExc_TypeError, "%s: expected %S on cuda:%ld, got %S on device %ld", name, first.dtype, first.device,
               t.dtype, t.device);
  return false;
}

// Tensor t, read from o, has this shape and a dense last dimension.
bool shaped(PyObject* o, const Tensor& t, int dims, int64_t a, int64_t b, int64_t c, const char* name) {
  const int64_t want[3] = {a, b, c};
  bool same = t.dims == dims;
  for (int i = 0; same && i < dims; ++i) same = t.shape[i] == want[i];
  if (!same) {
    Ref shape(PyObject_GetAttr(o, s_shape));
    Ref tuple(shape ? PySequence_Tuple(shape.get()) : nullptr);
    if (!tuple) return false;
    if (dims == 1)
      PyErr_Format(PyExc_ValueError, "%s: expected shape (%lld,), got %R", name, static_cast<long long>(a), tuple.get());
    else if (dims == 2)
      PyErr_Format(PyExc_ValueError, "%s: expected shape (%lld, %lld), got %R", name, static_cast<long long>(a),
                   static_cast<long long>(b), tuple.get());
    else
      PyErr_Format(PyExc_ValueError, "%s: expected shape (%lld, %lld, %lld), got %R", name, static_cast<long long>(a),
                   static_cast<long long>(b), static_cast<long long>(c), tuple.get());
    return false;
  }
  return t.dense() || not_dense(name);
}

// A tensor of the first operand's dtype and device, and of this shape.
bool like(PyObject* o, const Tensor& first, int dims, int64_t a, int64_t b, int64_t c, const char* name, Tensor& t) {
  return same_kind(o, first, name, t) && shaped(o, t, dims, a, b, c, name);
}

// A per-group matrix [groups][width] or one vector [width], checked against
// the rows it has to cover.
struct Grouped {
  void* ptr = nullptr;
  int64_t ld = 0, groups = 1, rows = 1;
};

bool integer(PyObject* o, int64_t& v) {
  v = PyLong_AsLongLong(o);
  return !(v == -1 && PyErr_Occurred());
}

bool grouped(PyObject* o, const Tensor& first, int64_t rows, int64_t width, PyObject* group_rows, const char* name,
             Grouped& g) {
  Tensor t;
  if (!same_kind(o, first, name, t)) return false;
  g.ptr = t.ptr;
  g.ld = width;
  if (t.dims == 1) {
    g.rows = rows > 1 ? rows : 1;
    return shaped(o, t, 1, width, 0, 0, name);
  }
  if (!shaped(o, t, 2, t.dims == 2 ? t.shape[0] : 0, width, 0, name)) return false;
  g.groups = t.shape[0];
  if (group_rows == Py_None) {
    if (!g.groups || rows % g.groups) {
      PyErr_Format(PyExc_ValueError, "%s: %lld rows do not divide into %lld groups; pass group_rows", name,
                   static_cast<long long>(rows), static_cast<long long>(g.groups));
      return false;
    }
    g.rows = rows / g.groups > 1 ? rows / g.groups : 1;
  } else if (!integer(group_rows, g.rows)) {
    return false;
  }
  if (g.rows < 1 || rows / g.rows + (rows % g.rows != 0) > g.groups) {
    PyErr_Format(PyExc_ValueError, "%s: %lld groups of %lld rows do not cover %lld rows", name,
                 static_cast<long long>(g.groups), static_cast<long long>(g.rows), static_cast<long long>(rows));
    return false;
  }
  if (g.rows > kMost) g.rows = kMost;   // one group either way
  if (g.groups > 1) g.ld = t.stride[0];
  return true;
}

bool countable(std::initializer_list<int64_t> sizes, const char* what) {
  for (int64_t s : sizes)
    if (s > kMost) {
      PyErr_Format(PyExc_ValueError, "%s: a dimension is longer than the library counts (2^31 - 2^16)", what);
      return false;
    }
  return true;
}

// x.new_empty(sizes...), of another dtype if given
PyObject* new_empty(PyObject* x, std::initializer_list<int64_t> sizes, PyObject* dtype = nullptr) {
  PyObject* args[kDims + 2] = {x};
  size_t n = 1;
  bool ok = true;
  for (int64_t s : sizes) ok = (args[n++] = PyLong_FromLongLong(s)) && ok;
  PyObject* r = nullptr;
  args[n] = dtype;
  if (ok) r = PyObject_VectorcallMethod(s_new_empty, args, n, dtype ? s_kw_dtype : nullptr);
  for (size_t i = 1; i < n; ++i) Py_XDECREF(args[i]);
  return r;
}

// The output: `given`, checked, or a new tensor.
PyObject* output(PyObject* given, PyObject* x, const Tensor& first, int dims, int64_t a, int64_t b, int64_t c, Tensor& t) {
  if (given != Py_None) {
    if (!like(given, first, dims, a, b, c, "out", t)) return nullptr;
    Py_INCREF(given);
    return given;
  }
  PyObject* o = dims == 2 ? new_empty(x, {a, b}) : new_empty(x, {a, b, c});
  if (!o) return nullptr;
  const int64_t shape[3] = {a, b, c};
  int64_t dense = 1;
  for (int i = dims - 1; i >= 0; --i) {
    t.shape[i] = shape[i];
    t.stride[i] = dense;
    dense *= shape[i];
  }
  t.dims = dims;
  Ref ptr(PyObject_CallMethodNoArgs(o, s_data_ptr));
  if (!ptr) {
    Py_DECREF(o);
    return nullptr;
  }
  t.ptr = PyLong_AsVoidPtr(ptr.get());
  return o;
}

// "auto" allocates on the call's stream, None gives none, a uint8 tensor is
// used as it is.  `keep` holds what was allocated until the call is made.
bool workspace_of(PyObject* given, PyObject* x, const Tensor& first, size_t bytes, void*& ptr, size_t& size, Ref& keep) {
  ptr = nullptr;
  size = 0;
  if (given == Py_None) return true;
  if (PyUnicode_Check(given)) {
    if (PyUnicode_CompareWithASCIIString(given, "auto")) {
      PyErr_SetString(PyExc_ValueError, "workspace must be 'auto', None or a uint8 device tensor");
      return false;
    }
    if (!bytes) return true;
    keep.reset(new_empty(x, {static_cast<int64_t>(bytes)}, g_u8));
    if (!keep) return false;
    given = keep.get();
  }
  Tensor t;
  if (!read(given, t)) return no_tensor("workspace", "");
  Ref contiguous(PyObject_CallMethodNoArgs(given, s_is_contiguous)), numel(PyObject_CallMethodNoArgs(given, s_numel));
  if (!contiguous || !numel) return false;
  if (t.dtype != g_u8 || t.device != first.device || contiguous.get() != Py_True) {
    PyErr_SetString(PyExc_TypeError, "workspace: expected a contiguous uint8 tensor on the call's device");
    return false;
  }
  int64_t n;
  if (!integer(numel.get(), n)) return false;
  ptr = t.ptr;
  size = static_cast<size_t>(n);
  return true;
}

bool fine(int status) {
  if (status == SVDQ_OK) return true;
  Ref r(PyObject_CallFunction(g_check, "i", status));   // raises
  if (r) PyErr_SetString(PyExc_RuntimeError, "svdq: unknown status");
  return false;
}

bool set_device(long device) {
  Ref r(PyObject_CallFunction(g_set_device, "l", device));
  return static_cast<bool>(r);
}

// Runs call(stream) with `device` current, on its current stream.
template <typename F>
bool run(long device, F call) {
  Ref current(PyObject_CallNoArgs(g_current));
  if (!current) return false;
  const long before = PyLong_AsLong(current.get());
  if (before == -1 && PyErr_Occurred()) return false;
  if (before != device && !set_device(device)) return false;
  Ref index(PyLong_FromLong(device));
  Ref stream(index ? PyObject_CallOneArg(g_stream, index.get()) : nullptr);
  void* s = stream ? PyLong_AsVoidPtr(stream.get()) : nullptr;
  bool ok = stream && !PyErr_Occurred();
  int status = SVDQ_OK;
  if (ok) {
    Py_BEGIN_ALLOW_THREADS
    status = call(s);
    Py_END_ALLOW_THREADS
  }
  if (before != device) {
    // back to the caller's device, an error of the call kept
    PyObject *type, *value, *trace;
    PyErr_Fetch(&type, &value, &trace);
    const bool back = set_device(before);
    if (type || back) {
      if (!back) PyErr_Clear();
      PyErr_Restore(type, value, trace);
    }
    ok = ok && back;
  }
  return ok && fine(status);
}

bool count_of(const char* fn, Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%s: expected %zd arguments, got %zd", fn, want, n);
  return false;
}

// Starts of packed sequences: an int32 tensor [batch + 1].
bool starts(PyObject* o, const Tensor& first, const char* name, void*& ptr, int64_t& batch) {
  Tensor t;
  if (!read(o, t)) return no_tensor(name, "[batch+1]");
  if (t.dtype != g_i32 || t.device != first.device || t.dims != 1 || !t.dense()) {
    PyErr_Format(PyExc_TypeError, "%s: expected a contiguous int32 tensor [batch+1] on cuda:%ld", name, first.device);
    return false;
  }
  if (t.shape[0] < 2) {
    PyErr_Format(PyExc_ValueError, "%s: expected batch + 1 >= 2 entries", name);
    return false;
  }
  ptr = t.ptr;
  batch = t.shape[0] - 1;
  return true;
}

// attention(q, k, v, cu_seqlens_q, cu_seqlens_k, causal, scale, out, return_lse, workspace)
PyObject* attention(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!count_of("attention", n, 10)) return nullptr;
  Tensor q, k, v, o;
  int code;
  if (!operand(args[0], 3, "q", "[tokens][heads][head_dim]", q, code) || !same_kind(args[1], q, "k", k)) return nullptr;
  if (k.dims != 3) {
    no_tensor("k", "[tokens][heads][head_dim]");
    return nullptr;
  }
  const int64_t total_q = q.shape[0], heads_q = q.shape[1], d = q.shape[2], total_k = k.shape[0], heads_k = k.shape[1];
  if (!shaped(args[1], k, 3, total_k, heads_k, d, "k") || !like(args[2], q, 3, total_k, heads_k, d, "v", v)) return nullptr;
  int64_t batch = 1, batch_k = 1;
  void *cu_q = nullptr, *cu_k = nullptr;
  if (args[3] == Py_None) {
    if (args[4] != Py_None) {
      PyErr_SetString(PyExc_ValueError, "cu_seqlens_k without cu_seqlens_q");
      return nullptr;
    }
  } else {
    if (!starts(args[3], q, "cu_seqlens_q", cu_q, batch)) return nullptr;
    cu_k = cu_q;
    if (args[4] == Py_None) {
      if (total_k != total_q) {
        PyErr_SetString(PyExc_ValueError, "cu_seqlens_k is needed where q and k have different numbers of tokens");
        return nullptr;
      }
    } else if (args[4] != args[3]) {
      if (!starts(args[4], q, "cu_seqlens_k", cu_k, batch_k)) return nullptr;
      if (batch_k != batch) {
        PyErr_SetString(PyExc_ValueError, "cu_seqlens_q and cu_seqlens_k must have the same number of entries");
        return nullptr;
      }
    }
  }
  if (!countable({total_q, heads_q, total_k, heads_k, d, batch}, "attention")) return nullptr;
  const int causal = PyObject_IsTrue(args[5]), with_lse = PyObject_IsTrue(args[8]);
  if (causal < 0 || with_lse < 0) return nullptr;
  double scale = d > 1 ? 1.0 / sqrt(static_cast<double>(d)) : 1.0;
  if (args[6] != Py_None) {
    scale = PyFloat_AsDouble(args[6]);
    if (scale == -1.0 && PyErr_Occurred()) return nullptr;
  }
  Ref out(output(args[7], args[0], q, 3, total_q, heads_q, d, o));
  if (!out) return nullptr;
  Ref lse;
  Tensor l;
  if (with_lse) {
    lse.reset(new_empty(args[0], {total_q, heads_q}, g_f32));
    if (!lse || !read(lse.get(), l)) return nullptr;
  }
  // dimensions of size 1 have no stride, and get that of a dense tensor
  int64_t strides[8];
  const Tensor* const all[4] = {&q, &k, &v, &o};
  for (int i = 0; i < 4; ++i) {
    strides[2 * i] = all[i]->shape[0] > 1 ? all[i]->stride[0] : all[i]->shape[1] * d;
    strides[2 * i + 1] = all[i]->shape[1] > 1 ? all[i]->stride[1] : d;
  }
  const int tq = static_cast<int>(total_q), tk = static_cast<int>(total_k), b = static_cast<int>(batch);
  const int hq = static_cast<int>(heads_q), hk = static_cast<int>(heads_k), hd = static_cast<int>(d);
  size_t bytes = 0, size;
  if (args[9] != Py_None && !fine(svdq_attention_workspace_size(tq, tk, b, hq, hk, hd, &bytes))) return nullptr;
  void* ws;
  Ref keep;
  if (!workspace_of(args[9], args[0], q, bytes, ws, size, keep)) return nullptr;
  if (!run(q.device, [&](void* stream) {
        return svdq_attention(q.ptr, k.ptr, v.ptr, o.ptr, static_cast<float*>(l.ptr), static_cast<int32_t*>(cu_q),
                              static_cast<int32_t*>(cu_k), b, tq, tk, hq, hk, hd, strides, static_cast<float>(scale),
                              causal, code, ws, size, stream);
      }))
    return nullptr;
  return with_lse ? PyTuple_Pack(2, out.get(), lse.get()) : out.release();
}

// linear16(x, w, bias, activation code, gate, residual, group_rows, out, workspace)
PyObject* linear16(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!count_of("linear16", n, 9)) return nullptr;
  Tensor x, w, bias, residual, y;
  int code;
  if (!operand(args[0], 2, "x", "[M][K]", x, code) || !same_kind(args[1], x, "w", w)) return nullptr;
  if (w.dims != 2) {
    no_tensor("w", "[N][K]");
    return nullptr;
  }
  const int64_t M = x.shape[0], K = x.shape[1], N = w.shape[0];
  if (!shaped(args[1], w, 2, N, K, 0, "w") || !countable({M, N, K}, "linear16")) return nullptr;
  const long act = PyLong_AsLong(args[3]);
  if (act == -1 && PyErr_Occurred()) return nullptr;
  if (args[2] != Py_None && !like(args[2], x, 1, N, 0, 0, "bias", bias)) return nullptr;
  Grouped gate;
  if (args[4] != Py_None && !grouped(args[4], x, M, N, args[6], "gate", gate)) return nullptr;
  if (args[5] != Py_None && !like(args[5], x, 2, M, N, 0, "residual", residual)) return nullptr;
  Ref out(output(args[7], args[0], x, 2, M, N, 0, y));
  if (!out) return nullptr;
  if (M == 0) return out.release();
  const int m = static_cast<int>(M), nn = static_cast<int>(N), k = static_cast<int>(K);
  size_t bytes = 0, size;
  if (args[8] != Py_None && !fine(svdq_linear16_workspace_size_for(x.ptr, x.ld(), w.ptr, w.ld(), m, nn, k, &bytes))) return nullptr;
  void* ws;
  Ref keep;
  if (!workspace_of(args[8], args[0], x, bytes, ws, size, keep)) return nullptr;
  if (!run(x.device, [&](void* stream) {
        return svdq_linear16(x.ptr, x.ld(), w.ptr, w.ld(), bias.ptr, gate.ptr, gate.ld, static_cast<int>(gate.rows),
                             residual.ptr, residual.ptr ? residual.ld() : 0, y.ptr, y.ld(), m, nn, k,
                             static_cast<int>(act), code, ws, size, stream);
      }))
    return nullptr;
  return out.release();
}

// layer_norm(x, weight, bias, scale, shift, group_rows, eps, out)
PyObject* layer_norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!count_of("layer_norm", n, 8)) return nullptr;
  Tensor x, weight, bias, y;
  int code;
  if (!operand(args[0], 2, "x", "[M][K]", x, code)) return nullptr;
  const int64_t M = x.shape[0], K = x.shape[1];
  if (!countable({M, K}, "layer_norm")) return nullptr;
  if (args[1] != Py_None && !like(args[1], x, 1, K, 0, 0, "weight", weight)) return nullptr;
  if (args[2] != Py_None && !like(args[2], x, 1, K, 0, 0, "bias", bias)) return nullptr;
  Grouped scale, shift;
  if (args[3] != Py_None && !grouped(args[3], x, M, K, args[5], "scale", scale)) return nullptr;
  if (args[4] != Py_None && !grouped(args[4], x, M, K, args[5], "shift", shift)) return nullptr;
  if (args[3] != Py_None && args[4] != Py_None &&
      (scale.rows != shift.rows || scale.groups != shift.groups || (scale.ld != shift.ld && scale.groups > 1))) {
    PyErr_SetString(PyExc_ValueError, "scale and shift must have the same groups and row stride");
    return nullptr;
  }
  const Grouped& g = args[3] != Py_None ? scale : shift;
  const double eps = PyFloat_AsDouble(args[6]);
  if (eps == -1.0 && PyErr_Occurred()) return nullptr;
  Ref out(output(args[7], args[0], x, 2, M, K, 0, y));
  if (!out) return nullptr;
  if (M == 0) return out.release();
  if (!run(x.device, [&](void* stream) {
        return svdq_layer_norm(x.ptr, x.ld(), weight.ptr, bias.ptr, scale.ptr, shift.ptr, g.ld, static_cast<int>(g.rows),
                               y.ptr, y.ld(), static_cast<int>(M), static_cast<int>(K), static_cast<float>(eps), code,
                               stream);
      }))
    return nullptr;
  return out.release();
}

// t, read from o, is a contiguous matrix of this dtype, shape and device.
bool exactly(PyObject* o, const Tensor& t, PyObject* dtype, long device, int64_t a, int64_t b, const char* name) {
  if (t.dtype != dtype || t.device != device || device < 0) {
    PyErr_Format(PyExc_TypeError, "%s: expected %S on cuda:%ld, got %S on device %ld", name, dtype, device, t.dtype, t.device);
    return false;
  }
  if (!shaped(o, t, 2, a, b, 0, name)) return false;
  int64_t dense = 1;
  for (int i = 1; i >= 0; --i) {
    if (t.shape[i] > 1 && t.stride[i] != dense) {
      PyErr_Format(PyExc_ValueError, "%s: must be contiguous", name);
      return false;
    }
    dense *= t.shape[i];
  }
  return true;
}

int64_t blocks_of(int64_t n) { return (n + SVDQ_FP8_BLOCK - 1) / SVDQ_FP8_BLOCK; }

void* pointer_of(PyObject* o) {
  Ref ptr(PyObject_CallMethodNoArgs(o, s_data_ptr));
  return ptr ? PyLong_AsVoidPtr(ptr.get()) : nullptr;
}

// Whether two matrices of 16-bit values, [rows][width] of at least 1 x 1 with
// row strides of `width` or more, share a value.
bool overlap(const Tensor& a, const Tensor& b) {
  const int64_t rows = a.shape[0], width = 2 * a.shape[1], la = 2 * a.ld(), lb = 2 * b.ld();   // bytes
  uintptr_t pa = reinterpret_cast<uintptr_t>(a.ptr), pb = reinterpret_cast<uintptr_t>(b.ptr);
  const uintptr_t end_a = pa + (rows - 1) * la + width, end_b = pb + (rows - 1) * lb + width;
  if (pa >= end_b || pb >= end_a) return false;
  if (la == lb) {
    // rows i of a and j of b meet if |pb - pa + (j - i) la| < width: the two j - i next to -(pb - pa) / la
    const uint64_t gap = pa < pb ? pb - pa : pa - pb, steps = gap / la, rest = gap % la;
    return (rest < static_cast<uint64_t>(width) && steps < static_cast<uint64_t>(rows)) ||
           (static_cast<uint64_t>(la) - rest < static_cast<uint64_t>(width) && steps + 1 < static_cast<uint64_t>(rows));
  }
  for (int64_t i = 0, j = 0; i < rows && j < rows;) {   // both in order
    const uintptr_t x = pa + i * la, y = pb + j * lb;
    if (x < y + width && y < x + width) return true;
    if (x < y)
      ++i;
    else
      ++j;
  }
  return false;
}

// rms_norm(x, weight, residual, eps, out, residual_out, codes) -> y or (codes, scales), and h with a residual
PyObject* rms_norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!count_of("rms_norm", n, 7)) return nullptr;
  Tensor x, weight, residual, sum, y;
  int code;
  if (!operand(args[0], 2, "x", "[M][K]", x, code)) return nullptr;
  const int64_t M = x.shape[0], K = x.shape[1];
  if (!countable({M, K}, "rms_norm")) return nullptr;
  const int codes = PyObject_IsTrue(args[6]);
  if (codes < 0) return nullptr;
  if (args[1] != Py_None && !like(args[1], x, 1, K, 0, 0, "weight", weight)) return nullptr;
  if (args[2] != Py_None && !like(args[2], x, 2, M, K, 0, "residual", residual)) return nullptr;
  const double eps = PyFloat_AsDouble(args[3]);
  if (eps == -1.0 && PyErr_Occurred()) return nullptr;
  if (args[5] != Py_None && args[2] == Py_None) {
    PyErr_SetString(PyExc_ValueError, "residual_out without residual");
    return nullptr;
  }
  Ref out, scales, h;
  void *yq = nullptr, *ys = nullptr;
  if (codes) {
    if (K % 16) {
      PyErr_Format(PyExc_ValueError, "x: rows of codes take multiples of 16 values, got %lld", static_cast<long long>(K));
      return nullptr;
    }
    out.reset(new_empty(args[0], {M, K}, g_f8));
    if (out) scales.reset(new_empty(args[0], {blocks_of(K), M}, g_f32));
    if (!out || !scales) return nullptr;
    yq = pointer_of(out.get());
    ys = pointer_of(scales.get());
  } else {
    out.reset(output(args[4], args[0], x, 2, M, K, 0, y));
    if (!out) return nullptr;
  }
  if (residual.ptr || args[2] != Py_None) {
    if (args[5] != Py_None) {
      if (!like(args[5], x, 2, M, K, 0, "residual_out", sum)) return nullptr;
      Py_INCREF(args[5]);
      h.reset(args[5]);
    } else {
      h.reset(output(Py_None, args[0], x, 2, M, K, 0, sum));
      if (!h) return nullptr;
    }
  }
  if (M && K && args[4] != Py_None && args[5] != Py_None && y.ld() >= K && sum.ld() >= K && overlap(y, sum)) {
    PyErr_SetString(PyExc_ValueError, "residual_out: shares memory with out");
    return nullptr;
  }
  if (M && !run(x.device, [&](void* stream) {
        return svdq_rms_norm(x.ptr, x.ld(), residual.ptr, residual.ptr ? residual.ld() : 0, weight.ptr, sum.ptr,
                             sum.ptr ? sum.ld() : 0, y.ptr, y.ptr ? y.ld() : 0, static_cast<uint8_t*>(yq),
                             static_cast<float*>(ys), static_cast<int>(M), static_cast<int>(K), static_cast<float>(eps), code,
                             stream);
      }))
    return nullptr;
  if (codes) return h ? PyTuple_Pack(3, out.get(), scales.get(), h.get()) : PyTuple_Pack(2, out.get(), scales.get());
  return h ? PyTuple_Pack(2, out.get(), h.get()) : out.release();
}

// quantize_fp8(x) -> (codes, scales)
PyObject* quantize_fp8(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!count_of("quantize_fp8", n, 1)) return nullptr;
  Tensor x;
  int code;
  if (!operand(args[0], 2, "x", "[M][K]", x, code)) return nullptr;
  const int64_t M = x.shape[0], K = x.shape[1];
  if (!countable({M, K}, "quantize_fp8")) return nullptr;
  Ref xq(new_empty(args[0], {M, K}, g_f8)), xs(new_empty(args[0], {blocks_of(K), M}, g_f32));
  if (!xq || !xs) return nullptr;
  void *q = pointer_of(xq.get()), *s = pointer_of(xs.get());
  if (M && !run(x.device, [&](void* stream) {
        return svdq_quantize_fp8(x.ptr, x.ld(), static_cast<uint8_t*>(q), static_cast<float*>(s), static_cast<int>(M),
                                 static_cast<int>(K), code, stream);
      }))
    return nullptr;
  return PyTuple_Pack(2, xq.get(), xs.get());
}

// gemm_fp8(xq, xs, wq, ws, bias, activation code, gate, residual, group_rows, dtype, out), and with xs None, xq
// being 16-bit activations: their codes are made first
PyObject* gemm_fp8(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!count_of("gemm_fp8", n, 11)) return nullptr;
  Tensor x, xs, wq, ws, bias, residual, y, like_y;
  int code;
  const bool whole = args[1] == Py_None;
  if (whole) {
    if (!operand(args[0], 2, "x", "[M][K]", x, code)) return nullptr;
  } else {
    if (args[9] != g_bf16 && args[9] != g_f16) {
      PyErr_SetString(PyExc_ValueError, "dtype: expected torch.bfloat16 or torch.float16");
      return nullptr;
    }
    code = args[9] == g_bf16 ? SVDQ_BF16 : SVDQ_F16;
    if (!read(args[0], x)) {
      no_tensor("xq", "[M][K]");
      return nullptr;
    }
    if (x.dims != 2 || x.device < 0) {
      no_tensor("xq", "[M][K]");
      return nullptr;
    }
  }
  const int64_t M = x.shape[0], K = x.shape[1];
  if (!read(args[2], wq) || wq.dims != 2) {
    no_tensor("wq", "[N][K]");
    return nullptr;
  }
  const int64_t N = wq.shape[0];
  if (!countable({M, N, K}, "gemm_fp8")) return nullptr;
  if ((!whole && !read(args[1], xs)) || !read(args[3], ws)) {
    no_tensor(whole || xs.dtype ? "ws" : "xs", "");
    return nullptr;
  }
  if (!whole && (!exactly(args[0], x, g_f8, x.device, M, K, "xq") || !exactly(args[1], xs, g_f32, x.device, blocks_of(K), M, "xs")))
    return nullptr;
  if (!exactly(args[2], wq, g_f8, x.device, N, K, "wq") ||
      !exactly(args[3], ws, g_f32, x.device, blocks_of(N), blocks_of(K), "ws"))
    return nullptr;
  like_y.dtype = code == SVDQ_BF16 ? g_bf16 : g_f16;
  like_y.device = x.device;
  const long act = PyLong_AsLong(args[5]);
  if (act == -1 && PyErr_Occurred()) return nullptr;
  if (args[4] != Py_None && !like(args[4], like_y, 1, N, 0, 0, "bias", bias)) return nullptr;
  Grouped gate;
  if (args[6] != Py_None && !grouped(args[6], like_y, M, N, args[8], "gate", gate)) return nullptr;
  if (args[7] != Py_None && !like(args[7], like_y, 2, M, N, 0, "residual", residual)) return nullptr;
  Ref out;
  if (args[10] != Py_None || whole) {
    out.reset(output(args[10], args[0], like_y, 2, M, N, 0, y));
  } else {
    out.reset(new_empty(args[0], {M, N}, like_y.dtype));
    if (out && !read(out.get(), y)) return nullptr;
  }
  if (!out) return nullptr;
  if (M == 0) return out.release();
  const int m = static_cast<int>(M), nn = static_cast<int>(N), k = static_cast<int>(K);
  Ref codes;
  uint8_t* q = static_cast<uint8_t*>(x.ptr);
  float* s = static_cast<float*>(xs.ptr);
  if (whole) {
    // codes and scales in one piece; K is a multiple of 16, or the first call refuses it
    codes.reset(new_empty(args[0], {(M * K + 15) / 16 * 16 + 4 * M * blocks_of(K)}, g_u8));
    if (!codes) return nullptr;
    q = static_cast<uint8_t*>(pointer_of(codes.get()));
    s = reinterpret_cast<float*>(q + (M * K + 15) / 16 * 16);
  }
  if (!run(x.device, [&](void* stream) {
        if (whole)
          if (const int st = svdq_quantize_fp8(x.ptr, x.ld(), q, s, m, k, code, stream)) return st;
        return svdq_gemm_fp8(q, s, static_cast<uint8_t*>(wq.ptr), static_cast<float*>(ws.ptr), bias.ptr, gate.ptr, gate.ld,
                             static_cast<int>(gate.rows), residual.ptr, residual.ptr ? residual.ld() : 0, y.ptr, y.ld(), m,
                             nn, k, static_cast<int>(act), code, stream);
      }))
    return nullptr;
  return out.release();
}

// The paged cache (codes of keys and values, exponents) and where the
// sequences of a call with `total` tokens stand in it.
struct Paged {
  Tensor k, v, exponents, table, lengths;
  void* cu = nullptr;
  int64_t batch = 0;

  // args: k codes, v codes, exponents, block_table, lengths, cu_seqlens
  bool init(PyObject* const* args, long device, int64_t total) {
    if (!read(args[0], k) || k.dims != 4) return no_tensor("cache.k", "[pages][heads][64][head_dim]");
    const int64_t pages = k.shape[0], heads = k.shape[1], D = k.shape[3];
    if (!whole(args[0], k, g_f8, device, {pages, heads, SVDQ_PAGE, D}, "cache.k") ||
        !read(args[1], v) || !whole(args[1], v, g_f8, device, {pages, heads, 4, D, 16}, "cache.v") ||
        !read(args[2], exponents) || !whole(args[2], exponents, g_i8, device, {pages, heads, 2}, "cache.exponents"))
      return named();
    if (!read(args[4], lengths) || lengths.dims != 1) return no_tensor("lengths", "[batch]");
    batch = lengths.shape[0];
    if (!whole(args[4], lengths, g_i32, device, {batch}, "lengths")) return false;
    if (!read(args[3], table) || table.dims != 2) return no_tensor("block_table", "[batch][width]");
    if (!whole(args[3], table, g_i32, device, {batch, table.shape[1]}, "block_table")) return false;
    if (args[5] == Py_None) {
      if (total != batch) {
        PyErr_Format(PyExc_ValueError, "without cu_seqlens each of the %lld sequences has one token, got %lld",
                     static_cast<long long>(batch), static_cast<long long>(total));
        return false;
      }
    } else {
      Tensor first;
      first.device = device;
      int64_t n;
      if (!starts(args[5], first, "cu_seqlens", cu, n)) return false;
      if (n != batch) {
        PyErr_SetString(PyExc_ValueError, "cu_seqlens: expected one entry more than lengths has");
        return false;
      }
    }
    return countable({pages, heads, D, batch, table.shape[1], total}, "cache");
  }

 private:
  // an error is set, if not by read()
  static bool named() { return PyErr_Occurred() ? false : no_tensor("cache", ""); }

  static bool whole(PyObject*, const Tensor& t, PyObject* dtype, long device, std::initializer_list<int64_t> shape,
                    const char* name) {
    if (t.dtype != dtype || t.device != device) {
      PyErr_Format(PyExc_TypeError, "%s: expected %S on cuda:%ld, got %S on device %ld", name, dtype, device, t.dtype, t.device);
      return false;
    }
    bool fits = t.dims == static_cast<int>(shape.size());
    int64_t dense = 1;
    for (int i = t.dims - 1; fits && i >= 0; --i) {
      fits = t.shape[i] == shape.begin()[i] && (t.shape[i] <= 1 || t.stride[i] == dense);
      dense *= t.shape[i];
    }
    if (!fits) PyErr_Format(PyExc_ValueError, "%s: wrong shape for this cache and batch, or not contiguous", name);
    return fits;
  }
};

// strides of a tensor [tokens][heads][head_dim]; a dimension of size 1 has that of a dense one
void strides_of(const Tensor& t, int64_t* to) {
  to[0] = t.shape[0] > 1 ? t.stride[0] : t.shape[1] * t.shape[2];
  to[1] = t.shape[1] > 1 ? t.stride[1] : t.shape[2];
}

// cache_append(k codes, v codes, exponents, block_table, lengths, cu_seqlens, k, v, q, rope, interleaved, q_out)
PyObject* cache_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!count_of("cache_append", n, 12)) return nullptr;
  Tensor k, v, q, out, rope;
  int code;
  if (!operand(args[6], 3, "k", "[tokens][heads][head_dim]", k, code)) return nullptr;
  const int64_t total = k.shape[0], heads_k = k.shape[1], D = k.shape[2];
  if (!like(args[7], k, 3, total, heads_k, D, "v", v)) return nullptr;
  Paged p;
  if (!p.init(args, k.device, total)) return nullptr;
  if (p.k.shape[1] != heads_k || p.k.shape[3] != D) {
    PyErr_Format(PyExc_ValueError, "k: the cache has %lld heads of %lld", static_cast<long long>(p.k.shape[1]),
                 static_cast<long long>(p.k.shape[3]));
    return nullptr;
  }
  int64_t rotary = 0, rope_rows = 0;
  if (args[9] != Py_None) {
    if (!read(args[9], rope) || rope.dims != 2) {
      no_tensor("rope", "[positions][rotary]");
      return nullptr;
    }
    rope_rows = rope.shape[0];
    rotary = rope.shape[1];
    if (!exactly(args[9], rope, g_f32, k.device, rope_rows, rotary, "rope")) return nullptr;
  }
  const int interleaved = PyObject_IsTrue(args[10]);
  if (interleaved < 0) return nullptr;
  Ref rotated;
  int64_t heads_q = heads_k, strides[8] = {};
  if (args[8] != Py_None) {
    if (!same_kind(args[8], k, "q", q)) return nullptr;
    heads_q = q.dims == 3 ? q.shape[1] : 0;
    if (!shaped(args[8], q, 3, total, heads_q, D, "q")) return nullptr;
    rotated.reset(output(args[11], args[8], k, 3, total, heads_q, D, out));
    if (!rotated) return nullptr;
    strides_of(q, strides);
    strides_of(out, strides + 6);
  } else if (args[11] != Py_None) {
    PyErr_SetString(PyExc_ValueError, "q_out without q");
    return nullptr;
  }
  if (!countable({heads_q, rope_rows, rotary}, "cache_append")) return nullptr;
  strides_of(k, strides + 2);
  strides_of(v, strides + 4);
  if (!run(k.device, [&](void* stream) {
        return svdq_cache_append(q.ptr, k.ptr, v.ptr, out.ptr, strides, static_cast<uint8_t*>(p.k.ptr),
                                 static_cast<uint8_t*>(p.v.ptr), static_cast<int8_t*>(p.exponents.ptr),
                                 static_cast<int>(p.k.shape[0]), static_cast<int32_t*>(p.table.ptr),
                                 static_cast<int>(p.table.shape[1]), static_cast<int32_t*>(p.lengths.ptr),
                                 static_cast<int32_t*>(p.cu), static_cast<int>(p.batch), static_cast<int>(total),
                                 static_cast<int>(heads_q), static_cast<int>(heads_k), static_cast<int>(D),
                                 static_cast<float*>(rope.ptr), static_cast<int>(rope_rows), static_cast<int>(rotary),
                                 interleaved, code, stream);
      }))
    return nullptr;
  if (rotated) return rotated.release();
  Py_RETURN_NONE;
}

// attention_paged(k codes, v codes, exponents, block_table, lengths, cu_seqlens, q, causal, scale, out, return_lse,
// workspace)
PyObject* attention_paged(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!count_of("attention_paged", n, 12)) return nullptr;
  Tensor q, o, l;
  int code;
  if (!operand(args[6], 3, "q", "[tokens][heads][head_dim]", q, code)) return nullptr;
  const int64_t total = q.shape[0], heads_q = q.shape[1], D = q.shape[2];
  Paged p;
  if (!p.init(args, q.device, total)) return nullptr;
  const int64_t heads_k = p.k.shape[1];
  if (p.k.shape[3] != D) {
    PyErr_Format(PyExc_ValueError, "q: the cache has heads of %lld", static_cast<long long>(p.k.shape[3]));
    return nullptr;
  }
  if (!countable({heads_q}, "attention_paged")) return nullptr;
  const int causal = PyObject_IsTrue(args[7]), with_lse = PyObject_IsTrue(args[10]);
  if (causal < 0 || with_lse < 0) return nullptr;
  double scale = D > 1 ? 1.0 / sqrt(static_cast<double>(D)) : 1.0;
  if (args[8] != Py_None) {
    scale = PyFloat_AsDouble(args[8]);
    if (scale == -1.0 && PyErr_Occurred()) return nullptr;
  }
  Ref out(output(args[9], args[6], q, 3, total, heads_q, D, o)), lse;
  if (!out) return nullptr;
  if (with_lse) {
    lse.reset(new_empty(args[6], {total, heads_q}, g_f32));
    if (!lse) return nullptr;
    l.ptr = pointer_of(lse.get());
  }
  int64_t strides[4];
  strides_of(q, strides);
  strides_of(o, strides + 2);
  const int t = static_cast<int>(total), b = static_cast<int>(p.batch), w = static_cast<int>(p.table.shape[1]);
  const int hq = static_cast<int>(heads_q), hk = static_cast<int>(heads_k), d = static_cast<int>(D);
  size_t bytes = 0, size;
  if (args[11] != Py_None && !fine(svdq_attention_paged_workspace_size(t, b, w, hq, hk, d, &bytes))) return nullptr;
  void* ws;
  Ref keep;
  if (!workspace_of(args[11], args[6], q, bytes, ws, size, keep)) return nullptr;
  if (!run(q.device, [&](void* stream) {
        return svdq_attention_paged(q.ptr, o.ptr, static_cast<float*>(l.ptr), strides, static_cast<uint8_t*>(p.k.ptr),
                                    static_cast<uint8_t*>(p.v.ptr), static_cast<int8_t*>(p.exponents.ptr),
                                    static_cast<int>(p.k.shape[0]), static_cast<int32_t*>(p.table.ptr), w,
                                    static_cast<int32_t*>(p.lengths.ptr), static_cast<int32_t*>(p.cu), b, t, hq, hk, d,
                                    static_cast<float>(scale), causal, code, ws, size, stream);
      }))
    return nullptr;
  return with_lse ? PyTuple_Pack(2, out.get(), lse.get()) : out.release();
}

// setup(Tensor, bfloat16, float16, float32, uint8, int32, current stream, current device, set device, check, e4m3, int8)
PyObject* setup(PyObject*, PyObject* const* args, Py_ssize_t n) {
  PyObject** const to[] = {&g_tensor, &g_bf16, &g_f16, &g_f32, &g_u8, &g_i32, &g_stream, &g_current, &g_set_device, &g_check, &g_f8, &g_i8};
  constexpr Py_ssize_t kCount = sizeof(to) / sizeof(to[0]);
  if (!count_of("setup", n, kCount)) return nullptr;
  if (!PyType_Check(args[0])) {
    PyErr_SetString(PyExc_TypeError, "setup: expected torch's Tensor type first");
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < kCount; ++i) {
    Py_INCREF(args[i]);
    Py_XSETREF(*to[i], args[i]);
  }
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* ready(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  if (!g_check) {
    PyErr_SetString(PyExc_RuntimeError, "setup() has not been called");
    return nullptr;
  }
  return F(self, args, n);
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction entry() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef g_methods[] = {
    {"attention", entry<ready<attention>>(), METH_FASTCALL, nullptr},
    {"linear16", entry<ready<linear16>>(), METH_FASTCALL, nullptr},
    {"layer_norm", entry<ready<layer_norm>>(), METH_FASTCALL, nullptr},
    {"rms_norm", entry<ready<rms_norm>>(), METH_FASTCALL, nullptr},
    {"quantize_fp8", entry<ready<quantize_fp8>>(), METH_FASTCALL, nullptr},
    {"gemm_fp8", entry<ready<gemm_fp8>>(), METH_FASTCALL, nullptr},
    {"cache_append", entry<ready<cache_append>>(), METH_FASTCALL, nullptr},
    {"attention_paged", entry<ready<attention_paged>>(), METH_FASTCALL, nullptr},
    {"setup", entry<setup>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_block_ops", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block_ops() {
  const struct {
    PyObject** to;
    const char* text;
  } names[] = {{&s_dtype, "dtype"},       {&s_shape, "shape"},         {&s_stride, "stride"},
               {&s_get_device, "get_device"}, {&s_data_ptr, "data_ptr"}, {&s_new_empty, "new_empty"},
               {&s_is_contiguous, "is_contiguous"}, {&s_numel, "numel"}};
  for (const auto& e : names)
    if (!*e.to && !(*e.to = PyUnicode_InternFromString(e.text))) return nullptr;
  if (!s_kw_dtype && !(s_kw_dtype = PyTuple_Pack(1, s_dtype))) return nullptr;
  return PyModule_Create(&g_module);
}
