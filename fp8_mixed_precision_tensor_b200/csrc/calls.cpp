// calls.cpp -- the block-scaled operators' arguments, read from tensors and
// handed to libfp8.so without the interpreter.
//
// The kernels behind these calls take a few microseconds, and so do the checks
// of their arguments in Python (two to four; a call through ctypes adds one):
// a 256 x 256 training step of six calls was bound by them, 47 us where the GPU
// needs 21.  Each function here takes its operator's arguments in order and
// returns True once the work is enqueued.  Whatever is not plainly a valid call
// on the current device and its current stream returns False and leaves nothing
// enqueued: the Python function then makes the call itself, or says what is
// wrong with it.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>

#include "../../include/fp8.h"

namespace {

struct {
  decltype(&fp8_block_cast) cast;
  decltype(&fp8_block_cast_square) cast_square;
  decltype(&fp8_block_linear_fwd) fwd;
  decltype(&fp8_block_linear_tokens) tokens;
  decltype(&fp8_block_linear_dgrad) dgrad;
  decltype(&fp8_block_linear_wgrad) wgrad;
  decltype(&fp8_act_fwd) act_fwd;
  decltype(&fp8_act_bwd) act_bwd;
} g_fp8;

// Thrown where the Python function has to decide.
struct NotPlain {};
void need(bool ok) {
  if (!ok) throw NotPlain();
}

const at::Tensor &tensor(PyObject *o) {
  need(THPVariable_Check(o));
  return THPVariable_Unpack(o);
}

int integer(PyObject *o) {
  need(PyLong_CheckExact(o));
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw NotPlain();
  }
  need(v >= INT_MIN && v <= INT_MAX);
  return (int)v;
}

bool given(PyObject *o) { return o != Py_None; }

int type_code(const at::Tensor &t) {
  switch (t.scalar_type()) {
    case at::kFloat: return FP8_DT_F32;
    case at::kBFloat16: return FP8_DT_BF16;
    case at::kHalf: return FP8_DT_F16;
    default: throw NotPlain();
  }
}

// A call's device (that of its first tensor) and stream.
struct Call {
  int device;
  void *stream;
  Call(const at::Tensor &first, PyObject *stream_arg) {
    need(first.is_cuda() && !given(stream_arg));
    device = first.get_device();
    need(device == c10::cuda::current_device());
    stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
  }
};

struct Shape {
  int rows, cols;
};
Shape shape_of(const at::Tensor &t) {
  need(t.dim() == 2 && t.size(0) <= INT_MAX && t.size(1) <= INT_MAX);
  return {(int)t.size(0), (int)t.size(1)};
}

// Row stride of a [rows, cols] matrix whose rows are contiguous and do not overlap.
size_t row_stride(const at::Tensor &t, Shape s, const Call &call) {
  need(t.is_cuda() && t.get_device() == call.device && t.dim() == 2 && t.size(0) == s.rows && t.size(1) == s.cols);
  need((t.stride(1) == 1 || s.cols <= 1) && (t.stride(0) >= s.cols || s.rows <= 1));
  return s.rows > 1 ? (size_t)t.stride(0) : (size_t)s.cols;
}

// Codes q of a matrix of this shape and the scales s of `outer` rows of `red` elements; absent where both are None.
struct Blocks {
  fp8_blocks b;
  bool present = false;
  Blocks(PyObject *q, PyObject *s, Shape shape, int outer, int red, const Call &call) {
    if (!given(q) && !given(s)) return;
    const at::Tensor &tq = tensor(q), &ts = tensor(s);
    need(tq.scalar_type() == at::kByte && ts.scalar_type() == at::kByte);
    const int64_t bytes = ((int64_t)outer + 127) / 128 * (((int64_t)red + 511) / 512) * 512;
    need(ts.is_cuda() && ts.get_device() == call.device && ts.is_contiguous() && ts.numel() >= bytes);
    const size_t ld = row_stride(tq, shape, call);
    b = {static_cast<uint8_t *>(tq.data_ptr()), static_cast<uint8_t *>(ts.data_ptr()),
         shape.rows > 1 ? ld : (ld + 15) / 16 * 16};
    present = true;
  }
  const fp8_blocks *get() const { return present ? &b : nullptr; }
};

// A high-precision matrix.
struct Matrix {
  void *p = nullptr;
  int type = 0;
  size_t ld = 0;
  Matrix() = default;
  Matrix(const at::Tensor &t, Shape s, const Call &call)
      : p(t.data_ptr()), type(type_code(t)), ld(row_stride(t, s, call)) {}
};

Matrix product_out(PyObject *o, Shape s, PyObject *rto, const Call &call) {
  Matrix m(tensor(o), s, call);
  need(rto == Py_True || rto == Py_False);
  if (rto == Py_True) {
    need(m.type == FP8_DT_BF16);
    m.type = FP8_DT_BF16_RTO;
  }
  return m;
}

struct Vector {
  const void *p = nullptr;
  int type = 0;
  Vector(PyObject *o, int n, const Call &call) {
    if (!given(o)) return;
    const at::Tensor &t = tensor(o);
    need(t.is_cuda() && t.get_device() == call.device && t.numel() == n && t.is_contiguous());
    p = t.data_ptr();
    type = type_code(t);
  }
};

// Runs f, which returns libfp8's status, on `n` arguments.  The interpreter is
// free meanwhile: a launch waits where the stream's queue is full.
template <typename F>
PyObject *run(Py_ssize_t have, Py_ssize_t n, F f) {
  bool ok = false;
  if (have == n) {
    try {
      auto launch = f();
      Py_BEGIN_ALLOW_THREADS;
      ok = launch() == FP8_OK;
      Py_END_ALLOW_THREADS;
    } catch (...) {  // NotPlain, or a tensor without storage
    }
  }
  return PyBool_FromLong(ok);
}

// x, fmt, margin, q_row, s_row, q_col, s_col, stream
PyObject *block_cast(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return run(n, 8, [&] {
    const at::Tensor &x = tensor(a[0]);
    const Call call(x, a[7]);
    const Shape s = shape_of(x);
    const Matrix m(x, s, call);
    const int fmt = integer(a[1]), margin = integer(a[2]);
    const Blocks row(a[3], a[4], s, s.rows, s.cols, call), col(a[5], a[6], s, s.cols, s.rows, call);
    return [=] {
      return g_fp8.cast(m.p, m.type, s.rows, s.cols, m.ld, fmt, margin, row.get(), col.get(), call.stream);
    };
  });
}

// x, fmt, margin, q, s_row, s_col, stream
PyObject *block_cast_square(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return run(n, 7, [&] {
    const at::Tensor &x = tensor(a[0]);
    const Call call(x, a[6]);
    const Shape s = shape_of(x);
    const Matrix m(x, s, call);
    const int fmt = integer(a[1]), margin = integer(a[2]);
    const Blocks row(a[3], a[4], s, s.rows, s.cols, call), col(a[3], a[5], s, s.cols, s.rows, call);
    need(row.present && col.present);
    return [=] {
      return g_fp8.cast_square(m.p, m.type, s.rows, s.cols, m.ld, fmt, margin, row.get(), col.b.s, call.stream);
    };
  });
}

// xq, xs, wq, ws, y, bias, stream, rto
PyObject *linear_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return run(n, 8, [&] {
    const at::Tensor &xq = tensor(a[0]);
    const Call call(xq, a[6]);
    const Shape x = shape_of(xq), w = shape_of(tensor(a[2]));
    const int M = x.rows, K = x.cols, N = w.rows;
    const Matrix y = product_out(a[4], {M, N}, a[7], call);
    const Vector bias(a[5], N, call);
    const Blocks bx(a[0], a[1], x, M, K, call), bw(a[2], a[3], {N, K}, N, K, call);
    need(bx.present && bw.present);
    return [=] {
      return g_fp8.fwd(bx.get(), bw.get(), bias.p, bias.type, y.p, y.type, y.ld, M, N, K, call.stream);
    };
  });
}

// x, wq, ws, y, bias, margin, stream, rto
PyObject *linear_tokens(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return run(n, 8, [&] {
    const at::Tensor &x = tensor(a[0]);
    const Call call(x, a[6]);
    const Shape s = shape_of(x);
    const int M = s.rows, K = s.cols, N = shape_of(tensor(a[1])).rows, margin = integer(a[5]);
    const Matrix m(x, s, call), y = product_out(a[3], {M, N}, a[7], call);
    const Vector bias(a[4], N, call);
    const Blocks bw(a[1], a[2], {N, K}, N, K, call);
    need(bw.present);
    return [=] {
      return g_fp8.tokens(m.p, m.type, m.ld, margin, bw.get(), bias.p, bias.type, y.p, y.type, y.ld, M, N, K,
                          call.stream);
    };
  });
}

// dyq, dys, dy_fmt, wq, ws_col, dx, stream, rto
PyObject *linear_dgrad(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return run(n, 8, [&] {
    const at::Tensor &dyq = tensor(a[0]);
    const Call call(dyq, a[6]);
    const Shape dy = shape_of(dyq);
    const int M = dy.rows, N = dy.cols, K = shape_of(tensor(a[3])).cols, fmt = integer(a[2]);
    const Matrix dx = product_out(a[5], {M, K}, a[7], call);
    const Blocks bd(a[0], a[1], dy, M, N, call), bw(a[3], a[4], {N, K}, K, N, call);
    need(bd.present && bw.present);
    return [=] {
      return g_fp8.dgrad(bd.get(), fmt, bw.get(), dx.p, dx.type, dx.ld, M, N, K, call.stream);
    };
  });
}

// dyq, dys_col, dy_fmt, xq, xs_col, dw, stream, rto
PyObject *linear_wgrad(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return run(n, 8, [&] {
    const at::Tensor &dyq = tensor(a[0]);
    const Call call(dyq, a[6]);
    const Shape dy = shape_of(dyq);
    const int M = dy.rows, N = dy.cols, K = shape_of(tensor(a[3])).cols, fmt = integer(a[2]);
    const Matrix dw = product_out(a[5], {N, K}, a[7], call);
    const Blocks bd(a[0], a[1], dy, N, M, call), bx(a[3], a[4], {M, K}, K, M, call);
    need(bd.present && bx.present);
    return [=] {
      return g_fp8.wgrad(bd.get(), fmt, bx.get(), dw.p, dw.type, dw.ld, M, N, K, call.stream);
    };
  });
}

// h, act, margin, ckpt_q, ckpt_s, a_q, a_s, a, stream
PyObject *act_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return run(n, 9, [&] {
    const at::Tensor &h = tensor(a[0]);
    const Call call(h, a[8]);
    const Shape s = shape_of(h);
    const Matrix m(h, s, call);
    const int act = integer(a[1]), margin = integer(a[2]);
    const Blocks ckpt(a[3], a[4], s, s.rows, s.cols, call), codes(a[5], a[6], s, s.rows, s.cols, call);
    const Matrix out = given(a[7]) ? Matrix(tensor(a[7]), s, call) : Matrix();
    need(ckpt.present && (!out.p || out.type == m.type));
    return [=] {
      return g_fp8.act_fwd(m.p, m.type, s.rows, s.cols, m.ld, act, margin, ckpt.get(), codes.get(), out.p, out.ld,
                           call.stream);
    };
  });
}

// ckpt_q, ckpt_s, da, act, fmt, margin, dh_q, dh_s, dh_q_col, dh_s_col, a_q_col, a_s_col, dh, stream
PyObject *act_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return run(n, 14, [&] {
    const at::Tensor &da = tensor(a[2]);
    const Call call(da, a[13]);
    const Shape s = shape_of(da);
    const Matrix m(da, s, call);
    const int act = integer(a[3]), fmt = integer(a[4]), margin = integer(a[5]);
    const Blocks ckpt(a[0], a[1], s, s.rows, s.cols, call), row(a[6], a[7], s, s.rows, s.cols, call);
    const Blocks col(a[8], a[9], s, s.cols, s.rows, call), acol(a[10], a[11], s, s.cols, s.rows, call);
    const Matrix out = given(a[12]) ? Matrix(tensor(a[12]), s, call) : Matrix();
    need(ckpt.present && (!out.p || out.type == m.type));
    return [=] {
      return g_fp8.act_bwd(ckpt.get(), m.p, m.type, s.rows, s.cols, m.ld, act, fmt, margin, row.get(), col.get(),
                           acol.get(), out.p, out.ld, call.stream);
    };
  });
}

// Addresses of libfp8.so's entry points, in g_fp8's order.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  void *p[sizeof(g_fp8) / sizeof(void *)];
  if (n != (Py_ssize_t)(sizeof(p) / sizeof(p[0]))) {
    PyErr_SetString(PyExc_TypeError, "one address per entry point");
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < n; i++) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return nullptr;
    }
  }
  static_assert(sizeof(p) == sizeof(g_fp8), "pointers only");
  memcpy(&g_fp8, p, sizeof(p));
  Py_RETURN_NONE;
}

#define ENTRY(name) {#name, (PyCFunction)(void *)name, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {ENTRY(bind),         ENTRY(block_cast),   ENTRY(block_cast_square), ENTRY(linear_fwd),
                           ENTRY(linear_tokens), ENTRY(linear_dgrad), ENTRY(linear_wgrad),      ENTRY(act_fwd),
                           ENTRY(act_bwd),       {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// The module, with the torch whose headers it was compiled with.
PyMODINIT_FUNC PyInit__calls() {
  PyObject *m = PyModule_Create(&g_module);
  if (m && PyModule_AddStringConstant(m, "torch_version", FP8_TORCH_VERSION) < 0) Py_CLEAR(m);
  return m;
}
