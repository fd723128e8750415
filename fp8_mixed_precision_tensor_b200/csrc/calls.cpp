// calls.cpp -- the arguments of the block-scaled operators and of the passes
// around them, read from tensors and handed to libfp8.so without the interpreter.
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

struct {
  decltype(&fp8_norm_fwd) norm_fwd;
  decltype(&fp8_norm_bwd) norm_bwd;
  decltype(&fp8_logprob_fwd) logprob_fwd;
  decltype(&fp8_logprob_bwd) logprob_bwd;
  decltype(&fp8_distill_fwd) distill_fwd;
  decltype(&fp8_distill_bwd) distill_bwd;
} g_passes;

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

float real(PyObject *o) {
  need(PyFloat_CheckExact(o));
  return (float)PyFloat_AS_DOUBLE(o);
}

// An optional [rows, cols] matrix of this type.
Matrix matrix_of(PyObject *o, Shape s, int type, const Call &call) {
  if (!given(o)) return Matrix();
  const Matrix m(tensor(o), s, call);
  need(m.type == type);
  return m;
}

// An optional contiguous tensor of rows, or rows x cols (cols < 0: rows), of a scalar type.
void *dense(PyObject *o, at::ScalarType type, int64_t rows, int64_t cols, const Call &call) {
  if (!given(o)) return nullptr;
  const at::Tensor &t = tensor(o);
  need(t.is_cuda() && t.get_device() == call.device && t.scalar_type() == type && t.is_contiguous());
  need(t.dim() == (cols < 0 ? 1 : 2) && t.size(0) == rows && (cols < 0 || t.size(1) == cols));
  return t.data_ptr();
}

// Optional int32 or int64 indices.
const void *indices(PyObject *o, int64_t rows, int64_t cols, const Call &call, int &bytes) {
  bytes = 0;
  if (!given(o)) return nullptr;
  const at::ScalarType type = tensor(o).scalar_type();
  need(type == at::kInt || type == at::kLong);
  bytes = type == at::kInt ? 4 : 8;
  return dense(o, type, rows, cols, call);
}

fp8_vector vector_of(PyObject *o, int n, const Call &call) {
  const Vector v(o, n, call);
  return {const_cast<void *>(v.p), v.type};
}

// A gate of [cols] or [gates, cols]: the vector, its rows and row stride.
fp8_vector gate_of(PyObject *o, Shape s, const Call &call, int &gate_rows, size_t &ld) {
  gate_rows = s.rows > 0 ? s.rows : 1;
  ld = (size_t)s.cols;
  if (!given(o)) return {nullptr, 0};
  const at::Tensor &t = tensor(o);
  if (t.dim() == 1) return vector_of(o, s.cols, call);
  const Shape g = shape_of(t);
  need(g.rows > 0 && s.rows % g.rows == 0);
  const Matrix m(t, {g.rows, s.cols}, call);
  if (s.rows > 0) gate_rows = s.rows / g.rows;
  ld = m.ld;
  return {m.p, m.type};
}

// h, r, r_out, stats, pre, post, w, b, post_w, post_b, gate, res_scale, eps, margin, x, x_q, x_s, x_q_col, x_s_col, stream
PyObject *norm_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return run(n, 20, [&] {
    const at::Tensor &rt = tensor(a[1]);
    const Call call(rt, a[19]);
    const Shape s = shape_of(rt);
    const Matrix r(rt, s, call);
    const int type = given(a[0]) ? type_code(tensor(a[0])) : given(a[14]) ? type_code(tensor(a[14])) : r.type;
    const Matrix h = matrix_of(a[0], s, type, call), ro = matrix_of(a[2], s, r.type, call), x = matrix_of(a[14], s, type, call);
    float *stats = static_cast<float *>(dense(a[3], at::kFloat, s.rows, 4, call));
    fp8_norm_params p = {};
    p.rows = s.rows, p.cols = s.cols, p.dtype = type, p.res_dtype = r.type;
    p.pre = integer(a[4]), p.post = integer(a[5]);
    p.w = vector_of(a[6], s.cols, call), p.b = vector_of(a[7], s.cols, call);
    p.post_w = vector_of(a[8], s.cols, call), p.post_b = vector_of(a[9], s.cols, call);
    p.gate = gate_of(a[10], s, call, p.gate_rows, p.ld_gate);
    p.res_scale = real(a[11]), p.eps = real(a[12]);
    const int margin = integer(a[13]);
    const Blocks row(a[15], a[16], s, s.rows, s.cols, call), col(a[17], a[18], s, s.cols, s.rows, call);
    return [=] {
      return g_passes.norm_fwd(&p, h.p, h.ld, r.p, r.ld, ro.p, ro.ld, stats, x.p, x.ld, margin, row.get(), col.get(),
                               call.stream);
    };
  });
}

// dx, dr_out, h, r_out, stats, pre, post, w, post_w, post_b, gate, res_scale, dh, dr, dw, db, dpost_w, dpost_b, dgate,
// workspace, stream
PyObject *norm_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return run(n, 21, [&] {
    need(given(a[0]) && given(a[3]));  // (a pass without a pre norm takes the long way)
    const at::Tensor &dxt = tensor(a[0]);
    const Call call(dxt, a[20]);
    const Shape s = shape_of(dxt);
    const Matrix dx(dxt, s, call), ro(tensor(a[3]), s, call);
    const Matrix dro = matrix_of(a[1], s, ro.type, call), h = matrix_of(a[2], s, dx.type, call);
    const Matrix dh = matrix_of(a[12], s, dx.type, call), dr = matrix_of(a[13], s, ro.type, call);
    const float *stats = static_cast<const float *>(dense(a[4], at::kFloat, s.rows, 4, call));
    fp8_norm_params p = {};
    p.rows = s.rows, p.cols = s.cols, p.dtype = dx.type, p.res_dtype = ro.type;
    p.pre = integer(a[5]), p.post = integer(a[6]);
    p.w = vector_of(a[7], s.cols, call), p.post_w = vector_of(a[8], s.cols, call), p.post_b = vector_of(a[9], s.cols, call);
    p.gate = gate_of(a[10], s, call, p.gate_rows, p.ld_gate);
    p.res_scale = real(a[11]);
    fp8_norm_grads g = {};
    g.w = vector_of(a[14], s.cols, call), g.b = vector_of(a[15], s.cols, call);
    g.post_w = vector_of(a[16], s.cols, call), g.post_b = vector_of(a[17], s.cols, call);
    int gate_rows;
    g.gate = gate_of(a[18], s, call, gate_rows, g.ld_gate);
    if (g.gate.p) g.gates = tensor(a[18]).dim() == 1 ? 1 : (int)tensor(a[18]).size(0);
    need(!g.gate.p || (p.gate.p && tensor(a[18]).sizes() == tensor(a[10]).sizes()));
    void *ws = nullptr;
    size_t bytes = 0;
    if (given(a[19])) {
      const at::Tensor &w = tensor(a[19]);
      need(w.is_cuda() && w.get_device() == call.device && w.is_contiguous());
      ws = w.data_ptr();
      bytes = w.numel() * w.element_size();
    }
    return [=] {
      return g_passes.norm_bwd(&p, dx.p, dx.ld, dro.p, dro.ld, h.p, h.ld, ro.p, ro.ld, stats, dh.p, dh.ld, dr.p, dr.ld, &g,
                               ws, bytes, call.stream);
    };
  });
}

// logits, tokens, logp, stats, inv_temp, entropy, top_logp, top_ids, stream
PyObject *logprob_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return run(n, 9, [&] {
    const at::Tensor &z = tensor(a[0]);
    const Call call(z, a[8]);
    const Shape s = shape_of(z);
    const Matrix m(z, s, call);
    int token_bytes;
    const void *tokens = indices(a[1], s.rows, -1, call, token_bytes);
    float *logp = static_cast<float *>(dense(a[2], at::kFloat, s.rows, -1, call));
    float *stats = static_cast<float *>(dense(a[3], at::kFloat, s.rows, 4, call));
    const float beta = real(a[4]);
    float *entropy = static_cast<float *>(dense(a[5], at::kFloat, s.rows, -1, call));
    const int top = given(a[6]) ? shape_of(tensor(a[6])).cols : 0;
    float *top_logp = static_cast<float *>(dense(a[6], at::kFloat, s.rows, top, call));
    int *top_ids = static_cast<int *>(dense(a[7], at::kInt, s.rows, top, call));
    return [=] {
      return g_passes.logprob_fwd(m.p, m.type, s.rows, s.cols, m.ld, beta, tokens, token_bytes, logp, entropy, top, top_logp,
                                  top_ids, stats, call.stream);
    };
  });
}

// logits, tokens, stats, dlogp, inv_temp, dentropy, fmt, margin, d_q, d_s, d_q_col, d_s_col, dlogits, stream
PyObject *logprob_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return run(n, 14, [&] {
    const at::Tensor &z = tensor(a[0]);
    const Call call(z, a[13]);
    const Shape s = shape_of(z);
    const Matrix m(z, s, call);
    int token_bytes;
    const void *tokens = indices(a[1], s.rows, -1, call, token_bytes);
    const float *stats = static_cast<const float *>(dense(a[2], at::kFloat, s.rows, 4, call));
    const float *g = static_cast<const float *>(dense(a[3], at::kFloat, s.rows, -1, call));
    const float beta = real(a[4]);
    const float *ge = static_cast<const float *>(dense(a[5], at::kFloat, s.rows, -1, call));
    const int fmt = integer(a[6]), margin = integer(a[7]);
    const Blocks row(a[8], a[9], s, s.rows, s.cols, call), col(a[10], a[11], s, s.cols, s.rows, call);
    const Matrix d = matrix_of(a[12], s, m.type, call);
    return [=] {
      return g_passes.logprob_bwd(m.p, m.type, s.rows, s.cols, m.ld, beta, tokens, token_bytes, stats, g, ge, fmt, margin,
                                  row.get(), col.get(), d.p, d.ld, call.stream);
    };
  });
}

// logits, ids, values, loss, stats, list_ids, list_q, form, inv_temp, stream
PyObject *distill_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return run(n, 10, [&] {
    const at::Tensor &z = tensor(a[0]);
    const Call call(z, a[9]);
    const Shape s = shape_of(z);
    const Matrix m(z, s, call);
    const at::Tensor &v = tensor(a[2]);
    const int top = shape_of(v).cols, value_type = type_code(v);
    int id_bytes;
    const void *ids = indices(a[1], s.rows, top, call, id_bytes);
    const void *values = dense(a[2], v.scalar_type(), s.rows, top, call);
    float *loss = static_cast<float *>(dense(a[3], at::kFloat, s.rows, -1, call));
    float *stats = static_cast<float *>(dense(a[4], at::kFloat, s.rows, 4, call));
    int *list_ids = static_cast<int *>(dense(a[5], at::kInt, s.rows, top, call));
    float *list_q = static_cast<float *>(dense(a[6], at::kFloat, s.rows, top, call));
    const int form = integer(a[7]);
    const float beta = real(a[8]);
    return [=] {
      return g_passes.distill_fwd(m.p, m.type, s.rows, s.cols, m.ld, beta, form, top, ids, id_bytes, values, value_type, loss,
                                  stats, list_ids, list_q, call.stream);
    };
  });
}

// logits, list_ids, list_q, stats, dloss, inv_temp, fmt, margin, d_q, d_s, d_q_col, d_s_col, dlogits, stream
PyObject *distill_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return run(n, 14, [&] {
    const at::Tensor &z = tensor(a[0]);
    const Call call(z, a[13]);
    const Shape s = shape_of(z);
    const Matrix m(z, s, call);
    const int top = shape_of(tensor(a[2])).cols;
    const int *list_ids = static_cast<const int *>(dense(a[1], at::kInt, s.rows, top, call));
    const float *list_q = static_cast<const float *>(dense(a[2], at::kFloat, s.rows, top, call));
    const float *stats = static_cast<const float *>(dense(a[3], at::kFloat, s.rows, 4, call));
    const float *g = static_cast<const float *>(dense(a[4], at::kFloat, s.rows, -1, call));
    const float beta = real(a[5]);
    const int fmt = integer(a[6]), margin = integer(a[7]);
    const Blocks row(a[8], a[9], s, s.rows, s.cols, call), col(a[10], a[11], s, s.cols, s.rows, call);
    const Matrix d = matrix_of(a[12], s, m.type, call);
    return [=] {
      return g_passes.distill_bwd(m.p, m.type, s.rows, s.cols, m.ld, beta, top, list_ids, list_q, stats, g, fmt, margin,
                                  row.get(), col.get(), d.p, d.ld, call.stream);
    };
  });
}

// Addresses of libfp8.so's entry points, in the order of g_fp8 (g_passes).
template <typename T>
PyObject *bind_to(T &to, PyObject *const *a, Py_ssize_t n) {
  void *p[sizeof(T) / sizeof(void *)];
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
  static_assert(sizeof(p) == sizeof(T), "pointers only");
  memcpy(&to, p, sizeof(p));
  Py_RETURN_NONE;
}
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) { return bind_to(g_fp8, a, n); }
PyObject *bind_passes(PyObject *, PyObject *const *a, Py_ssize_t n) { return bind_to(g_passes, a, n); }

#define ENTRY(name) {#name, (PyCFunction)(void *)name, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {ENTRY(bind),         ENTRY(block_cast),   ENTRY(block_cast_square), ENTRY(linear_fwd),
                           ENTRY(linear_tokens), ENTRY(linear_dgrad), ENTRY(linear_wgrad),      ENTRY(act_fwd),
                           ENTRY(act_bwd),       ENTRY(bind_passes), ENTRY(norm_fwd), ENTRY(norm_bwd),
                           ENTRY(logprob_fwd),   ENTRY(logprob_bwd), ENTRY(distill_fwd), ENTRY(distill_bwd), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// The module, with the torch whose headers it was compiled with.
PyMODINIT_FUNC PyInit__calls() {
  PyObject *m = PyModule_Create(&g_module);
  if (m && PyModule_AddStringConstant(m, "torch_version", FP8_TORCH_VERSION) < 0) Py_CLEAR(m);
  return m;
}
