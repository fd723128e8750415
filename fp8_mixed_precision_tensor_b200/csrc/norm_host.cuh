// norm_host.cuh -- argument checks and dispatch that the norms' two translation
// units share.
#pragma once

#include <math.h>

#include "host.cuh"
#include "norm.cuh"

namespace fp8lib {
namespace {

// A vector of parameters, or a matrix with cols elements a row: FP8_OK, or what is wrong with it.
int check_vector(const fp8_vector &v) {
  if (!v.p) return FP8_OK;
  if (!valid_dtype(v.dtype)) return FP8_ERR_INVALID_ARG;
  return reinterpret_cast<uintptr_t>(v.p) % dtype_bytes(v.dtype) ? FP8_ERR_UNALIGNED : FP8_OK;
}
norm::Vec vec_of(const fp8_vector &v) { return {v.p, v.dtype}; }

bool norm_kind(int k) { return k == FP8_NORM_NONE || k == FP8_NORM_RMS || k == FP8_NORM_LAYER; }

int check_norm(const fp8_norm_params *p, bool h) {
  if (!p || !valid_dtype(p->dtype) || (p->res_dtype != p->dtype && p->res_dtype != FP8_DT_F32) || p->rows < 0 ||
      p->cols < 0 || !norm_kind(p->pre) || !norm_kind(p->post) || !(p->eps >= 0.0f) || !isfinite(p->eps) ||
      !isfinite(p->res_scale) || (!h && p->rows && (p->post != FP8_NORM_NONE || p->gate.p)))
    return FP8_ERR_INVALID_ARG;
  int rc;
  for (const fp8_vector *v : {&p->w, &p->b, &p->post_w, &p->post_b, &p->gate})
    if ((rc = check_vector(*v))) return rc;
  if (p->gate.p && (p->gate_rows < 1 || p->ld_gate < (size_t)p->cols)) return FP8_ERR_INVALID_ARG;
  if (p->cols > FP8_NORM_COLS_MAX || too_long(p->rows, p->cols)) return FP8_ERR_UNSUPPORTED;
  return FP8_OK;
}

bool aligned_to(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Whether a matrix, where there is one, is read and written in whole groups of eight.
bool whole_groups(const void *p, int dtype, size_t ld, int cols) { return !p || (wide_rows(p, dtype, ld) && cols % 8 == 0); }

template <typename F>
void with_kind(int kind, F f) {
  if (kind == 1) f(std::integral_constant<int, 1>());
  else if (kind == 2) f(std::integral_constant<int, 2>());
  else if (kind == 3) f(std::integral_constant<int, 3>());
  else f(std::integral_constant<int, 4>());
}

template <typename F>
void with_norm_types(int dt, int rt, F f) {
  with_dtype(dt, [&](auto d) {
    constexpr int DT = decltype(d)::value;
    if (rt == dt) f(d, d);
    else if constexpr (DT != FP8_DT_F32) f(d, std::integral_constant<int, FP8_DT_F32>());
  });
}

int gate_rows_of(const fp8_norm_params *p) { return p->gate.p && p->gate_rows < p->rows ? p->gate_rows : p->rows; }

}  // namespace
}  // namespace fp8lib
