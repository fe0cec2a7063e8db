// binding.cpp - the torch side of the residual block's calls (ops.py): checks
// of the tensor arguments, allocation of outputs and workspaces on the current
// stream, and the call of the C entry point. A Python module of its own,
// because the smallest of these calls take the GPU three microseconds and the
// same steps in Python took the host twenty.
//
// Wrong arguments raise ValueError before anything is launched; a status other
// than CONV2D_OK goes to abi.check (Conv2dError).
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "conv2d.h"

namespace {

constexpr int64_t kGroup = 32;

// The library's entry points, resolved by init().
#define ENTRIES(X)                                                                                                 \
  X(conv2d_q8_encode) X(conv2d_q8_decode) X(conv2d_rms_norm_fwd) X(conv2d_rms_norm_bwd)                            \
  X(conv2d_rms_norm_bwd_workspace_size) X(conv2d_dense_fwd) X(conv2d_dense_bwd) X(conv2d_dense_fwd_workspace_size) \
  X(conv2d_dense_bwd_workspace_size)
struct Lib {
#define X(f) decltype(&::f) f = nullptr;
  ENTRIES(X)
#undef X
} lib;

struct Refused {
  std::string why;
};
[[noreturn]] void refuse(const std::string& name, const std::string& why) { throw Refused{name + ": " + why}; }
struct Raised {};  // a Python error is set

enum : unsigned { kF32 = 1, kBF16 = 2, kF16 = 4, kE4M3 = 8, kHalf = kBF16 | kF16, kFloats = kF32 | kHalf };

unsigned type_bit(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return kF32;
    case at::kBFloat16: return kBF16;
    case at::kHalf: return kF16;
    case at::kFloat8_e4m3fn: return kE4M3;
    default: return 0;
  }
}
int32_t type_code(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return CONV2D_FP32;
    case at::kBFloat16: return CONV2D_BF16;
    case at::kHalf: return CONV2D_FP16;
    default: return CONV2D_E4M3;
  }
}
std::string type_name(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kHalf: return "torch.float16";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    default: return std::string("torch ") + c10::toString(t);
  }
}
std::string type_names(unsigned mask) {
  std::string s;
  for (at::ScalarType t : {at::kFloat, at::kBFloat16, at::kHalf, at::kFloat8_e4m3fn})
    if (type_bit(t) & mask) s += (s.empty() ? "" : ", ") + type_name(t);
  return s;
}
std::string shape_name(const at::Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}
std::string pair_name(int64_t a, int64_t b) { return "(" + std::to_string(a) + ", " + std::to_string(b) + ")"; }

bool given(PyObject* o) { return o != Py_None; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(name, std::string("expected a torch.Tensor, got ") + Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}
// A Q8 (a named tuple of q, scale, group).
bool is_q8(PyObject* o) { return PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 3; }
PyObject* q8_item(PyObject* o, int i) { return PyTuple_GET_ITEM(o, i); }
int64_t group_arg(PyObject* o) {
  const int64_t g = PyLong_Check(o) ? PyLong_AsLongLong(o) : -1;
  if (g != 0 && g != kGroup) throw Refused{"group: 0 (a whole row) or 32"};
  return g;
}
int64_t scale_columns(int64_t cols, int64_t group) { return group ? (cols + kGroup - 1) / kGroup : 1; }

struct Source {
  int64_t rows, cols;
  at::Device dev;
  at::ScalarType type;
};
// The argument that the others are checked against.
Source source(PyObject* o, const char* name, unsigned types) {
  if (!is_q8(o) && !THPVariable_Check(o))
    refuse(name, std::string("expected a torch.Tensor or Q8, got ") + Py_TYPE(o)->tp_name);
  const at::Tensor& t = tensor(is_q8(o) ? q8_item(o, 0) : o, name);
  if (t.dim() != 2 || t.size(1) < 1) refuse(name, "expected rows by at least one feature, got shape " + shape_name(t));
  if (!(type_bit(t.scalar_type()) & types))
    refuse(name, "dtype " + type_name(t.scalar_type()) + " is not one of " + type_names(types));
  return {t.size(0), t.size(1), t.device(), t.scalar_type()};
}

conv2d_mat mat_of(const at::Tensor& t, const char* name, int64_t rows, int64_t cols, unsigned types, at::Device dev) {
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
    refuse(name, "shape " + shape_name(t) + " does not match " + pair_name(rows, cols));
  if (!(type_bit(t.scalar_type()) & types))
    refuse(name, "dtype " + type_name(t.scalar_type()) + " is not one of " + type_names(types));
  if (t.device() != dev) refuse(name, "must be on " + dev.str() + " (got " + t.device().str() + ")");
  const int64_t ld = rows > 1 ? t.stride(0) : cols;
  if ((cols > 1 && t.stride(1) != 1) || ld < cols)
    refuse(name, "features must be contiguous and rows must not overlap (strides " +
                     pair_name(t.stride(0), t.stride(1)) + ")");
  void* p = t.data_ptr();
  if (reinterpret_cast<uintptr_t>(p) & 15) refuse(name, "must start on a 16-byte boundary");
  return {p, ld, type_code(t.scalar_type()), 0, nullptr};
}
// A matrix argument; types with kE4M3 take a Q8.
conv2d_mat mat(PyObject* o, const char* name, int64_t rows, int64_t cols, unsigned types, at::Device dev) {
  if (is_q8(o)) {
    if (!(types & kE4M3)) refuse(name, "an 8-bit matrix is not taken here");
    const int64_t group = group_arg(q8_item(o, 2));
    const at::Tensor& s = tensor(q8_item(o, 1), name);
    const int64_t sc = scale_columns(cols, group);
    if (s.scalar_type() != at::kByte || s.dim() != 2 || s.size(0) != rows || s.size(1) != sc)
      refuse(name, "scales are uint8 of shape " + pair_name(rows, sc));
    if (!s.is_contiguous() || s.device() != dev) refuse(name, "scales must be contiguous and on " + dev.str());
    conv2d_mat m = mat_of(tensor(q8_item(o, 0), name), name, rows, cols, kE4M3, dev);
    m.group = static_cast<int32_t>(group);
    m.scale = static_cast<uint8_t*>(s.data_ptr());
    return m;
  }
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() == at::kFloat8_e4m3fn) refuse(name, "8-bit values need their scales (Q8)");
  return mat_of(t, name, rows, cols, types & ~kE4M3, dev);
}
float* vec_of(const at::Tensor& t, const char* name, int64_t n, at::Device dev) {
  if (t.scalar_type() != at::kFloat || t.dim() != 1 || t.size(0) != n || !t.is_contiguous() || t.device() != dev)
    refuse(name, "expected a contiguous float32 tensor of shape (" + std::to_string(n) + ",) on " + dev.str() + ", got " +
                     type_name(t.scalar_type()) + " " + shape_name(t) + " on " + t.device().str());
  float* p = static_cast<float*>(t.data_ptr());
  if (reinterpret_cast<uintptr_t>(p) & 15) refuse(name, "must start on a 16-byte boundary");
  return p;
}
float* vec(PyObject* o, const char* name, int64_t n, at::Device dev) { return vec_of(tensor(o, name), name, n, dev); }

// Straight from the CUDA allocator's factory: the dispatcher's way costs a call half as much again.
at::Tensor make(at::IntArrayRef size, at::ScalarType t, at::Device dev) {
  if (dev.is_cuda()) return at::detail::empty_cuda(size, t, dev, std::nullopt);
  return at::empty(size, at::TensorOptions().dtype(t).device(dev));
}
conv2d_mat new_mat(at::Tensor& t, int64_t rows, int64_t cols, at::ScalarType type, at::Device dev) {
  t = make({rows, cols}, type, dev);
  return {t.data_ptr(), cols, type_code(type), 0, nullptr};
}
conv2d_mat new_q8(at::Tensor& q, at::Tensor& s, int64_t rows, int64_t cols, int64_t group, at::Device dev) {
  q = make({rows, cols}, at::kFloat8_e4m3fn, dev);
  s = make({rows, scale_columns(cols, group)}, at::kByte, dev);
  return {q.data_ptr(), cols, CONV2D_E4M3, static_cast<int32_t>(group), static_cast<uint8_t*>(s.data_ptr())};
}

void* stream_of(at::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }
int32_t small(int64_t v, const char* what) {
  if (v > INT32_MAX) refuse(what, "too large");
  return static_cast<int32_t>(v);
}
// Makes the call on the current stream of the tensors' device; raises what its status says.
template <typename F>
void run(at::Device dev, const char* name, F&& call) {
  if (!dev.is_cuda()) throw Refused{"the tensors must be in CUDA device memory (got " + dev.str() + ")"};
  const c10::DeviceGuard guard(dev);
  const int rc = call(stream_of(dev));
  if (rc == CONV2D_OK) return;
  PyObject* abi = PyImport_ImportModule("conv2d_layer_gb300.abi");
  PyObject* r = abi ? PyObject_CallMethod(abi, "check", "is", rc, name) : nullptr;
  Py_XDECREF(r);
  Py_XDECREF(abi);
  if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s: status %d", name, rc);
  throw Raised{};
}

PyObject* wrap(const at::Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
// A new reference to an argument that is handed back.
PyObject* same(PyObject* o) {
  Py_INCREF(o);
  return o;
}
template <size_t N>
PyObject* tuple(PyObject* const (&items)[N]) {
  PyObject* t = PyTuple_New(N);
  for (size_t i = 0; i < N; ++i) PyTuple_SET_ITEM(t, static_cast<Py_ssize_t>(i), items[i]);
  return t;
}

// ---------------------------------------------------------------- calls
// q8_encode(x, group, out) -> (q, scale) or None when out was handed in
PyObject* q8_encode(PyObject* const* a) {
  const Source s = source(a[0], "x", kFloats);
  at::Tensor q, sc;
  const conv2d_mat x = mat(a[0], "x", s.rows, s.cols, kFloats, s.dev);
  if (given(a[2]) && !is_q8(a[2])) refuse("out", "expected a Q8");
  const conv2d_mat o = given(a[2]) ? mat(a[2], "out", s.rows, s.cols, kE4M3, s.dev)
                                   : new_q8(q, sc, s.rows, s.cols, group_arg(a[1]), s.dev);
  const int32_t cols = small(s.cols, "x");
  run(s.dev, "conv2d_q8_encode", [&](void* st) { return lib.conv2d_q8_encode(s.rows, cols, &x, &o, st); });
  if (given(a[2])) Py_RETURN_NONE;
  return tuple({wrap(q), wrap(sc)});
}

// q8_decode(q8, dtype, out) -> out
PyObject* q8_decode(PyObject* const* a) {
  if (!is_q8(a[0])) refuse("q8", "expected a Q8");
  const Source s = source(a[0], "q8", kE4M3);
  const at::ScalarType t = THPDtype_Check(a[1]) ? reinterpret_cast<THPDtype*>(a[1])->scalar_type : at::kByte;
  if (!(type_bit(t) & kFloats)) refuse("dtype", "one of " + type_names(kFloats));
  const conv2d_mat q = mat(a[0], "q8", s.rows, s.cols, kE4M3, s.dev);
  at::Tensor out;
  const conv2d_mat o = given(a[2]) ? mat(a[2], "out", s.rows, s.cols, type_bit(t), s.dev) : new_mat(out, s.rows, s.cols, t, s.dev);
  const int32_t cols = small(s.cols, "q8");
  run(s.dev, "conv2d_q8_decode", [&](void* st) { return lib.conv2d_q8_decode(s.rows, cols, &q, &o, st); });
  return given(a[2]) ? same(a[2]) : wrap(out);
}

// rms_norm_fwd(x, gamma, eps, residual, y, group, h, q8, inv_rms) -> (h, y, q, scale, inv_rms); q and scale are
// None unless they were made here
PyObject* rms_norm_fwd(PyObject* const* a) {
  const Source s = source(a[0], "x", kFloats);
  const unsigned t = type_bit(s.type);
  const conv2d_mat x = mat(a[0], "x", s.rows, s.cols, t, s.dev);
  const float* gamma = vec(a[1], "gamma", s.cols, s.dev);
  const double eps = PyFloat_AsDouble(a[2]);
  if (eps == -1.0 && PyErr_Occurred()) throw Raised{};
  if (!given(a[3]) && given(a[6])) refuse("h", "an output of x + residual, but there is no residual");
  if (a[4] == Py_False && !given(a[5]) && !given(a[7]))
    throw Refused{"y or an 8-bit form of it (group, q8) must be asked for"};
  if (given(a[7]) && !is_q8(a[7])) refuse("q8", "expected a Q8");
  at::Tensor h, y, q, sc, inv;
  conv2d_mat mr, mh, my, mq;
  if (given(a[3])) {
    mr = mat(a[3], "residual", s.rows, s.cols, t, s.dev);
    mh = given(a[6]) ? mat(a[6], "h", s.rows, s.cols, t, s.dev) : new_mat(h, s.rows, s.cols, s.type, s.dev);
  }
  const bool has_y = a[4] != Py_False, has_q = given(a[5]) || given(a[7]);
  if (has_y) my = a[4] == Py_True ? new_mat(y, s.rows, s.cols, s.type, s.dev) : mat(a[4], "y", s.rows, s.cols, t, s.dev);
  if (given(a[7])) mq = mat(a[7], "q8", s.rows, s.cols, kE4M3, s.dev);
  else if (has_q) mq = new_q8(q, sc, s.rows, s.cols, group_arg(a[5]), s.dev);
  float* pi;
  if (given(a[8])) {
    pi = vec(a[8], "inv_rms", s.rows, s.dev);
  } else {
    inv = make({s.rows}, at::kFloat, s.dev);
    pi = static_cast<float*>(inv.data_ptr());
  }
  const int32_t cols = small(s.cols, "x");
  run(s.dev, "conv2d_rms_norm_fwd", [&](void* st) {
    return lib.conv2d_rms_norm_fwd(s.rows, cols, static_cast<float>(eps), &x, given(a[3]) ? &mr : nullptr, gamma,
                                   given(a[3]) ? &mh : nullptr, has_y ? &my : nullptr, has_q ? &mq : nullptr, pi, st);
  });
  return tuple({!given(a[3]) ? same(a[0]) : given(a[6]) ? same(a[6]) : wrap(h),
                !has_y ? same(Py_None) : a[4] == Py_True ? wrap(y) : same(a[4]), wrap(q), wrap(sc),
                given(a[8]) ? same(a[8]) : wrap(inv)});
}

// rms_norm_bwd(h, gamma, inv_rms, dy, dh, dx, dgamma, need_dx, need_dgamma) -> (dx, dgamma)
PyObject* rms_norm_bwd(PyObject* const* a) {
  const Source s = source(a[0], "h", kFloats);
  const unsigned t = type_bit(s.type);
  const bool need_dx = PyObject_IsTrue(a[7]) == 1, need_dg = PyObject_IsTrue(a[8]) == 1;
  if (!need_dx && !need_dg) throw Refused{"need_dx or need_dgamma"};
  const conv2d_mat h = mat(a[0], "h", s.rows, s.cols, t, s.dev);
  const float* gamma = vec(a[1], "gamma", s.cols, s.dev);
  const float* inv = vec(a[2], "inv_rms", s.rows, s.dev);
  const conv2d_mat dy = mat(a[3], "dy", s.rows, s.cols, t, s.dev);
  conv2d_mat dh, mx;
  if (given(a[4])) dh = mat(a[4], "dh", s.rows, s.cols, t, s.dev);
  at::Tensor dx, dg, ws;
  if (need_dx)
    mx = given(a[5]) ? mat(a[5], "dx", s.rows, s.cols, t, s.dev) : new_mat(dx, s.rows, s.cols, s.type, s.dev);
  const int32_t cols = small(s.cols, "h");
  float* pg = nullptr;
  if (need_dg) {
    if (given(a[6])) {
      pg = vec(a[6], "dgamma", s.cols, s.dev);
    } else {
      dg = make({s.cols}, at::kFloat, s.dev);
      pg = static_cast<float*>(dg.data_ptr());
    }
  }
  run(s.dev, "conv2d_rms_norm_bwd", [&](void* st) {
    const size_t n = need_dg ? lib.conv2d_rms_norm_bwd_workspace_size(s.rows, cols) : 0;  // of the current device
    if (n) ws = make({static_cast<int64_t>(n)}, at::kByte, s.dev);
    return lib.conv2d_rms_norm_bwd(s.rows, cols, &h, gamma, inv, &dy, given(a[4]) ? &dh : nullptr,
                                   need_dx ? &mx : nullptr, pg, need_dg && given(a[6]), n ? ws.data_ptr() : nullptr, n, st);
  });
  return tuple({!need_dx ? same(Py_None) : given(a[5]) ? same(a[5]) : wrap(dx),
                !need_dg ? same(Py_None) : given(a[6]) ? same(a[6]) : wrap(dg)});
}

// dense_fwd(x, w, bias, act, residual, save, dtype, y, pre_act) -> (y, z, scale); save: 0 none, 1 full, 2 q8; z and
// scale are None unless they were made here
PyObject* dense_fwd(PyObject* const* a) {
  const Source s = source(a[0], "x", kHalf | kE4M3), sw = source(a[1], "w", kHalf | kE4M3);
  if (sw.rows < 1) refuse("w", "expected at least one output feature");
  at::ScalarType t = THPDtype_Check(a[6]) ? reinterpret_cast<THPDtype*>(a[6])->scalar_type : at::ScalarType::Undefined;
  for (const Source* o : {&s, &sw}) {
    if (o->type == at::kFloat8_e4m3fn) continue;
    if (t != at::ScalarType::Undefined && t != o->type)
      throw Refused{"dtype " + type_name(t) + ", but an operand is " + type_name(o->type)};
    t = o->type;
  }
  if (!(type_bit(t) & kHalf)) throw Refused{"dtype: bfloat16 or float16 (needed where both operands are Q8)"};
  const unsigned bit = type_bit(t);
  const int64_t M = s.rows, K = s.cols, N = sw.rows;
  const conv2d_mat x = mat(a[0], "x", M, K, bit | kE4M3, s.dev), w = mat(a[1], "w", N, K, bit | kE4M3, s.dev);
  const float* bias = given(a[2]) ? vec(a[2], "bias", N, s.dev) : nullptr;
  conv2d_mat mr, my, mz;
  if (given(a[4])) mr = mat(a[4], "residual", M, N, bit, s.dev);
  const long save = PyLong_AsLong(a[5]);
  at::Tensor y, z, sc, ws;
  if (given(a[8])) {
    if (save == 0 || is_q8(a[8]) != (save == 2)) refuse("pre_act", "not an output for this save");
    mz = mat(a[8], "pre_act", M, N, bit | kE4M3, s.dev);
    if (save == 2 && mz.group != kGroup) refuse("pre_act", "groups of 32");
  }
  my = given(a[7]) ? mat(a[7], "y", M, N, bit, s.dev) : new_mat(y, M, N, t, s.dev);
  if (!given(a[8]) && save == 1) mz = new_mat(z, M, N, t, s.dev);
  if (!given(a[8]) && save == 2) mz = new_q8(z, sc, M, N, kGroup, s.dev);
  const conv2d_dense_desc d = {M, small(K, "x"), small(N, "w"), static_cast<int32_t>(PyLong_AsLong(a[3])), type_code(t), 0};
  run(s.dev, "conv2d_dense_fwd", [&](void* st) {
    const size_t n = lib.conv2d_dense_fwd_workspace_size(&d, &x, &w);
    if (n > 256) ws = make({static_cast<int64_t>(n)}, at::kByte, s.dev);  // 256: nothing is kept in it
    return lib.conv2d_dense_fwd(&d, &x, &w, bias, given(a[4]) ? &mr : nullptr, save ? &mz : nullptr, &my,
                                ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? n : 0, st);
  });
  return tuple({given(a[7]) ? same(a[7]) : wrap(y), wrap(z), wrap(sc)});
}

// dense_bwd(x, w, dy, pre_act, act, grad_dtype, dx, dw, dbias, need_dx, need_dw, need_dbias) -> (dx, dw, dbias)
PyObject* dense_bwd(PyObject* const* a) {
  const Source s = source(a[2], "dy", kHalf);
  const unsigned bit = type_bit(s.type);
  const bool need_dx = PyObject_IsTrue(a[9]) == 1, need_dw = PyObject_IsTrue(a[10]) == 1, need_db = PyObject_IsTrue(a[11]) == 1;
  if (!need_dx && !need_dw && !need_db) throw Refused{"need_dx, need_dw or need_dbias"};
  const int64_t M = s.rows, N = s.cols;
  const int64_t K = need_dw ? source(a[0], "x", kHalf | kE4M3).cols : need_dx ? source(a[1], "w", kHalf | kE4M3).cols : 1;
  const long act = PyLong_AsLong(a[4]);
  conv2d_mat x, w, z, mx, mw;
  const conv2d_mat dy = mat(a[2], "dy", M, N, bit, s.dev);
  if (need_dw) x = mat(a[0], "x", M, K, bit | kE4M3, s.dev);
  if (need_dx) w = mat(a[1], "w", N, K, bit | kE4M3, s.dev);
  if (act) {
    if (!given(a[3])) refuse("pre_act", "needed behind an activation");
    z = mat(a[3], "pre_act", M, N, bit | kE4M3, s.dev);
  }
  if (need_dw && need_db && given(a[7]) != given(a[8]))
    throw Refused{"dw and dbias: hand in both to accumulate, or neither"};
  const bool accumulate = (need_dw && given(a[7])) || (need_db && given(a[8]));
  at::Tensor dx, dw, db;
  if (need_dx) mx = given(a[6]) ? mat(a[6], "dx", M, K, bit, s.dev) : new_mat(dx, M, K, s.type, s.dev);
  if (need_dw) {
    if (given(a[7])) {
      mw = mat(a[7], "dw", N, K, bit | kF32, s.dev);
    } else {
      const at::ScalarType t = THPDtype_Check(a[5]) ? reinterpret_cast<THPDtype*>(a[5])->scalar_type : at::kByte;
      if (t != at::kFloat && t != s.type) refuse("grad_dtype", "torch.float32 or " + type_name(s.type));
      mw = new_mat(dw, N, K, t, s.dev);
    }
  }
  float* pb = nullptr;
  if (need_db) {
    if (given(a[8])) {
      pb = vec(a[8], "dbias", N, s.dev);
    } else {
      db = make({N}, at::kFloat, s.dev);
      pb = static_cast<float*>(db.data_ptr());
    }
  }
  const conv2d_dense_desc d = {M, small(K, "x"), small(N, "dy"), static_cast<int32_t>(act), type_code(s.type), accumulate};
  const conv2d_mat *qx = need_dw ? &x : nullptr, *qw = need_dx ? &w : nullptr, *qz = act ? &z : nullptr,
                   *gx = need_dx ? &mx : nullptr, *gw = need_dw ? &mw : nullptr;
  run(s.dev, "conv2d_dense_bwd", [&](void* st) {
    const size_t n = lib.conv2d_dense_bwd_workspace_size(&d, qx, qw, qz, &dy, gx, gw, pb);
    const at::Tensor ws = make({static_cast<int64_t>(n)}, at::kByte, s.dev);
    return lib.conv2d_dense_bwd(&d, qx, qw, qz, &dy, gx, gw, pb, ws.data_ptr(), n, st);
  });
  return tuple({!need_dx ? same(Py_None) : given(a[6]) ? same(a[6]) : wrap(dx),
                !need_dw ? same(Py_None) : given(a[7]) ? same(a[7]) : wrap(dw),
                !need_db ? same(Py_None) : given(a[8]) ? same(a[8]) : wrap(db)});
}

// ---------------------------------------------------------------- module
// No C++ exception leaves a call: what torch throws (out of memory, say) becomes a RuntimeError.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(a);
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.why.c_str());
  } catch (const Raised&) {
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    PyErr_SetString(type ? type : PyExc_RuntimeError, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyObject* init(PyObject*, PyObject* path) {
  const char* p = PyUnicode_AsUTF8(path);
  if (!p) return nullptr;
  void* h = dlopen(p, RTLD_NOW | RTLD_LOCAL);
  if (!h) return PyErr_Format(PyExc_ImportError, "%s", dlerror());
#define X(f)                                                                       \
  lib.f = reinterpret_cast<decltype(lib.f)>(dlsym(h, #f));                         \
  if (!lib.f) return PyErr_Format(PyExc_ImportError, "%s lacks %s", p, #f);
  ENTRIES(X)
#undef X
  Py_RETURN_NONE;
}

#define ENTRY(f, n) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"init", init, METH_O, "Resolves the library's entry points."},
                         ENTRY(q8_encode, 3),
                         ENTRY(q8_decode, 3),
                         ENTRY(rms_norm_fwd, 9),
                         ENTRY(rms_norm_bwd, 9),
                         ENTRY(dense_fwd, 9),
                         ENTRY(dense_bwd, 12),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
