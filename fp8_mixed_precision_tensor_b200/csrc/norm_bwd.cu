// norm_bwd.cu -- the C ABI of the norms' backward pass (include/fp8.h).
//
// A translation unit of its own, for its many kernels: compiled beside the
// others.  What the shared headers define has names of its own here; nothing
// here raises a status.
#define fp8lib fp8lib_norm_bwd

#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "../../include/fp8.h"
#include "norm_host.cuh"

using namespace fp8lib;

extern "C" {

size_t fp8_norm_workspace_bytes(int rows, int cols, int gate_rows) {
  if (rows <= 0 || cols <= 0 || cols > FP8_NORM_COLS_MAX || gate_rows <= 0) return 0;
  const norm::Plan plan = norm::plan_of(rows, cols, gate_rows);
  return ((size_t)plan.ctas + (size_t)plan.units) * 2 * (size_t)norm::padded(cols) * sizeof(float);
}

int fp8_norm_bwd(const fp8_norm_params *p, const void *dx, size_t lddx, const void *dr_out, size_t lddr_out,
                 const void *h, size_t ldh, const void *r_out, size_t ldr_out, const float *stats, void *dh,
                 size_t lddh, void *dr, size_t lddr, const fp8_norm_grads *grads, void *workspace, size_t ws_bytes,
                 void *stream) {
  int rc = check_norm(p, h != nullptr);
  if (rc) return rc;
  const fp8_norm_grads none = {};
  const fp8_norm_grads &g = grads ? *grads : none;
  for (const fp8_vector *v : {&g.w, &g.b, &g.post_w, &g.post_b, &g.gate})
    if ((rc = check_vector(*v))) return rc;
  const int rows = p->rows, cols = p->cols;
  const bool pre = p->pre != FP8_NORM_NONE, post = p->post != FP8_NORM_NONE;
  const bool of_pre = g.w.p || g.b.p, of_post = g.post_w.p || g.post_b.p || g.gate.p;
  // (matrices without rows have no address)
  if ((rows && (pre != (dx != nullptr) || (!h && (dh || of_post)) || (!dh && !dr && !of_pre && !of_post))) ||
      (!pre && of_pre) || (!post && (g.post_w.p || g.post_b.p)) || (g.gate.p && !p->gate.p) ||
      (g.gate.p && (g.ld_gate < (size_t)cols || g.gates < 0)))
    return FP8_ERR_INVALID_ARG;
  if (cols == 0) return FP8_OK;
  if (rows && ((pre && ((rc = check_matrix(dx, p->dtype, cols, lddx)) || (rc = check_matrix(r_out, p->res_dtype, cols, ldr_out)))) ||
               (dr_out && (rc = check_matrix(dr_out, p->res_dtype, cols, lddr_out))) ||
               (h && (rc = check_matrix(h, p->dtype, cols, ldh))) || (dh && (rc = check_matrix(dh, p->dtype, cols, lddh))) ||
               (dr && (rc = check_matrix(dr, p->res_dtype, cols, lddr)))))
    return rc;
  if (rows && (pre || post) && !stats) return FP8_ERR_INVALID_ARG;
  if (!aligned16(stats) || !aligned16(workspace)) return FP8_ERR_UNALIGNED;
  const norm::Plan plan = norm::plan_of(rows, cols, gate_rows_of(p));
  const bool sums = of_pre || of_post;
  const bool bias = g.b.p || g.post_b.p || (g.gate.p && post && p->post_b.p);  // plain sums of dx or G
  if (sums && rows && (!workspace || ws_bytes < fp8_norm_workspace_bytes(rows, cols, gate_rows_of(p))))
    return FP8_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  norm::Bwd a = {};
  float *ws = static_cast<float *>(workspace);
  if (rows) {
    a.dx = dx, a.dro = dr_out, a.h = h, a.ro = r_out, a.stats = stats, a.dh = dh, a.dr = dr;
    a.lddx = lddx, a.lddro = lddr_out, a.ldh = ldh, a.ldro = ldr_out, a.lddh = lddh, a.lddr = lddr;
    a.rows = rows, a.cols = cols, a.pre = p->pre, a.post = p->post;
    a.w = vec_of(p->w), a.pw = vec_of(p->post_w), a.g = vec_of(p->gate);
    a.ldg = p->ld_gate;
    a.alpha = p->res_scale;
    const bool whole = whole_groups(dx, p->dtype, lddx, cols) && whole_groups(dr_out, p->res_dtype, lddr_out, cols) &&
                       whole_groups(h, p->dtype, ldh, cols) && whole_groups(pre ? r_out : nullptr, p->res_dtype, ldr_out, cols) &&
                       whole_groups(dh, p->dtype, lddh, cols) && whole_groups(dr, p->res_dtype, lddr, cols);
    a.ef = of_pre ? ws : nullptr;
    a.ac = of_post ? ws + (size_t)plan.ctas * 2 * norm::padded(cols) : nullptr;
    a.gate_rows = plan.gate_rows, a.unit_rows = plan.unit_rows, a.per_gate = plan.per_gate, a.units = plan.units;
    with_norm_types(p->dtype, p->res_dtype, [&](auto dt, auto rt) {
      constexpr int DT = decltype(dt)::value, RT = decltype(rt)::value;
      with_kind(plan.kind, [&](auto ck) {
        constexpr int CK = decltype(ck)::value;
        auto launch = [&](auto kernel, int mode) {
          const int columns = 8 * norm::eights(CK) * (CK == 4 ? plan.threads : norm::kCtaThreads<CK, norm::kStaged>);
          const int smem = norm::bwd_smem<DT, RT>(columns, h, dr_out, pre, h && (a.g.p || (post && a.pw.p)),
                                                  plan.groups > 1, mode, norm::held(CK, mode)).bytes;
          if (smem > kMostSmem) return FP8_ERR_UNSUPPORTED;
          if (int e = allow_smem(kernel)) return e;
          return launch_pdl(kernel, (unsigned)plan.ctas, dim3(plan.threads, plan.groups), smem, s, 1, a);
        };
        rc = FP8_ERR_UNSUPPORTED;
        if (whole && cols <= norm::kStagedCols) {
          if (pre && dr_out && h && dh && dr && (!post || a.pw.p))
            with_bool(post, [&](auto has_post) {
              with_bool(bias || CK >= 3, [&](auto has_bias) {
                constexpr bool kBias = decltype(has_bias)::value || CK >= 3;
                rc = launch(norm::k_norm_bwd<DT, RT, true, decltype(has_post)::value, kBias, CK, norm::kStaged>, norm::kStaged);
              });
            });
          else
            rc = launch(norm::k_norm_bwd<DT, RT, false, false, true, CK, norm::kStaged>, norm::kStaged);
        }
        if (rc == FP8_ERR_UNSUPPORTED)
          rc = launch(norm::k_norm_bwd<DT, RT, false, false, true, CK == 1 ? 1 : 4, norm::kDirect>, norm::kDirect);
      });
    });
    if (rc) return rc;
  }
  if (!sums) return FP8_OK;
  norm::Params q = {};
  q.ef = ws, q.ac = ws + (size_t)plan.ctas * 2 * norm::padded(cols);
  q.cols = cols, q.ctas = plan.ctas, q.per_gate = plan.per_gate;
  q.post = post, q.bias = bias;
  q.gates = rows ? (int)(plan.units / plan.per_gate) : g.gates > 1 ? g.gates : 1;  // (no rows: no partial sums, 0 each)
  q.pw = vec_of(p->post_w), q.pb = vec_of(p->post_b), q.g = vec_of(p->gate), q.ldg = p->ld_gate;
  q.dw = vec_of(g.w), q.db = vec_of(g.b), q.dpw = vec_of(g.post_w), q.dpb = vec_of(g.post_b), q.dg = vec_of(g.gate);
  q.lddg = g.ld_gate;
  q.col_blocks = (cols + 31) / 32;
  const long long jobs = 2 + (g.gate.p ? (long long)q.gates : 0);
  if (jobs * q.col_blocks > INT_MAX) return FP8_ERR_UNSUPPORTED;
  return launch_pdl(norm::k_norm_params, (unsigned)(jobs * q.col_blocks), dim3(32, norm::kParamLanes), 0, s, 1, q);
}

}  // extern "C"
