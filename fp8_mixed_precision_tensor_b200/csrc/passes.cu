// passes.cu -- the C ABI of include/fp8.h's passes between and behind the linear
// layers: norms with gate and residual (their backward pass: norm_bwd.cu), log
// probabilities, distillation.
//
// A translation unit of its own, compiled beside libfp8.cu.  Its copies of what
// the shared headers define (kernels, the device status word) have names of
// their own; fp8_get_status reads both status words.
#define fp8lib fp8lib_passes

#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <mutex>

#include "../../include/fp8.h"
#include "host.cuh"
#include "loss.cuh"
#include "norm.cuh"
#include "norm_host.cuh"

using namespace fp8lib;

namespace {

// SMs of the current device, looked up once.
int sm_count(int *out) {
  static std::mutex mu;
  static int sms[64] = {0};
  int dev;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return FP8_ERR_CUDA;
  std::lock_guard<std::mutex> lock(mu);
  if (!sms[dev] && cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return FP8_ERR_CUDA;
  *out = sms[dev];
  return FP8_OK;
}

struct LossArgs {
  const void *logits;
  int dtype, rows, cols;
  size_t ld;
  float inv_temp;
};
int check_loss(const LossArgs &a) {
  if (!valid_dtype(a.dtype) || a.rows < 0 || a.cols < 0 || !(a.inv_temp > 0.0f) || !isfinite(a.inv_temp * loss::kLog2e))
    return FP8_ERR_INVALID_ARG;
  if (a.rows == 0 || a.cols == 0) return FP8_OK;
  if (too_long(a.rows, a.cols)) return FP8_ERR_UNSUPPORTED;
  return check_matrix(a.logits, a.dtype, a.cols, a.ld);
}
bool index_bytes(int b) { return b == 4 || b == 8; }

// CTAs that share a row, and their threads.
struct LossGrid {
  unsigned ctas, threads;
  int vecs;  // 16-byte vectors of a CTA, at the most
};
LossGrid loss_grid(int rows, int cols, int dtype, int sms, unsigned least) {
  const int elems = dtype == FP8_DT_F32 ? 4 : 8, vecs = cols / elems;
  LossGrid g = {1, 0, 0};
  while (g.ctas < 8 && (long long)rows * g.ctas * 2 <= sms && vecs / (int)(2 * g.ctas) >= 512) g.ctas *= 2;
  g.vecs = (vecs + (int)g.ctas - 1) / (int)g.ctas;
  const long long all = (long long)rows * g.ctas;
  const unsigned most = all <= sms ? 1024u : all <= 2LL * sms ? 512u : all <= 4LL * sms ? 256u : 128u;  // (a CTA of 1024 threads fills an SM)
  g.threads = least;
  while (g.threads < most && (int)g.threads * 2 <= g.vecs) g.threads *= 2;
  return g;
}

template <int DT, int MODE, bool ENT>
int launch_loss_fwd(const loss::Fwd &p, const LossGrid &g, size_t smem, cudaStream_t s) {
  const auto kernel = loss::k_loss_fwd<DT, MODE, ENT>;
  if ((long long)p.rows * g.ctas > INT_MAX) return FP8_ERR_UNSUPPORTED;
  int rc;
  // (what a launch has unasked, 48 KB, holds the kernel's own shared memory too)
  if (smem > 48 * 1024 - kOwnSmem && (rc = allow_smem(kernel))) return rc;
  return launch_pdl(kernel, (unsigned)p.rows * g.ctas, g.threads, smem, s, g.ctas, p, g.ctas);
}

template <bool LIST>
int launch_loss_bwd(const loss::Bwd &p, int dtype, int fmt, cudaStream_t s) {
  int rc = FP8_OK;
  with_dtype(dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    if (p.out.q || p.out.qt) {
      with_fmt(fmt, [&](auto f) {
        constexpr int OUT = decltype(f)::value, KIND = LIST ? loss::kListed : loss::kToken;
        const auto kernel = !LIST && p.g_ent ? loss::k_loss_bwd_tiles<DT, loss::kTokenEntropy, OUT>
                                             : loss::k_loss_bwd_tiles<DT, KIND, OUT>;
        rc = launch_pdl(kernel, tile_grid(p.rows, p.cols), 512, 0, s, 1, p);
      });
      return;
    }
    constexpr int share = loss::kBwdThreads * loss::kBwdVecs;
    const long long vecs = p.cols / loss::kElems<DT>, chunks = vecs ? (vecs + share - 1) / share : 1;
    if (chunks * p.rows > INT_MAX) {
      rc = FP8_ERR_UNSUPPORTED;
      return;
    }
    rc = launch_pdl(loss::k_loss_bwd_rows<DT, LIST>, (unsigned)(chunks * p.rows), loss::kBwdThreads, 0, s, 1, p,
                    (unsigned)chunks);
  });
  return rc;
}

// The outputs of a gradient of the logits, and the factors that both have.
int loss_outputs(loss::Bwd &p, const LossArgs &a, const float *stats, int fmt, int margin, const fp8_blocks *row,
                 const fp8_blocks *col, void *d, size_t ldd) {
  if (!fp8_fmt(fmt) || margin < 0 || margin > 64) return FP8_ERR_INVALID_ARG;
  int rc = check_loss(a);
  if (rc || a.rows == 0 || a.cols == 0) return rc;
  if ((!row && !col && !d) || !stats) return FP8_ERR_INVALID_ARG;
  if ((row && (rc = check_blocks(row, a.cols))) || (col && (rc = check_blocks(col, a.cols))) ||
      (d && (rc = check_matrix(d, a.dtype, a.cols, ldd))))
    return rc;
  if (!aligned16(stats)) return FP8_ERR_UNALIGNED;
  const size_t e = dtype_bytes(a.dtype);
  p.z = static_cast<const uint8_t *>(a.logits);
  p.ld = a.ld * e;
  p.rows = a.rows;
  p.cols = a.cols;
  p.beta = a.inv_temp;
  p.stats = stats;
  p.d = static_cast<uint8_t *>(d);
  p.ldd = ldd * e;
  p.margin = margin;
  p.vec_z = wide_rows(a.logits, a.dtype, a.ld);
  p.vec_d = wide_rows(d, a.dtype, ldd);
  p.out = cast_out(row, col);
  return FP8_OK;
}

}  // namespace

extern "C" {

int fp8_norm_fwd(const fp8_norm_params *p, const void *h, size_t ldh, const void *r, size_t ldr, void *r_out,
                 size_t ldr_out, float *stats, void *x, size_t ldx, int margin, const fp8_blocks *x_row,
                 const fp8_blocks *x_col, void *stream) {
  int rc = check_norm(p, h != nullptr);
  if (rc) return rc;
  if (margin < 0 || margin > 64) return FP8_ERR_INVALID_ARG;
  const int rows = p->rows, cols = p->cols;
  if (rows == 0 || cols == 0) return FP8_OK;
  if ((p->pre == FP8_NORM_NONE && (x || x_row || x_col)) || (x_col && !stats) ||
      (!r_out && (h || p->res_scale != 1.0f)) || (!r_out && !x && !x_row && !x_col && !stats))
    return FP8_ERR_INVALID_ARG;
  if ((h && (rc = check_matrix(h, p->dtype, cols, ldh))) || (rc = check_matrix(r, p->res_dtype, cols, ldr)) ||
      (r_out && (rc = check_matrix(r_out, p->res_dtype, cols, ldr_out))) ||
      (x && (rc = check_matrix(x, p->dtype, cols, ldx))) || (x_row && (rc = check_blocks(x_row, cols))) ||
      (x_col && (rc = check_blocks(x_col, cols))))
    return rc;
  if (!aligned16(stats)) return FP8_ERR_UNALIGNED;
  norm::Fwd a = {};
  a.h = h, a.r = r, a.r_out = r_out, a.x = x, a.stats = stats;
  a.ldh = ldh, a.ldr = ldr, a.ldro = ldr_out, a.ldx = ldx;
  if (x_row) a.xq = x_row->q, a.xs = x_row->s, a.ldxq = x_row->ld;
  a.rows = rows, a.cols = cols, a.pre = p->pre, a.post = p->post;
  a.w = vec_of(p->w), a.b = vec_of(p->b), a.pw = vec_of(p->post_w), a.pb = vec_of(p->post_b), a.g = vec_of(p->gate);
  a.gate_rows = p->gate.p ? p->gate_rows : rows;
  a.ldg = p->ld_gate;
  a.alpha = p->res_scale, a.eps = p->eps, a.margin = margin;
  const bool whole = whole_groups(h, p->dtype, ldh, cols) && whole_groups(r, p->res_dtype, ldr, cols) &&
                     whole_groups(r_out, p->res_dtype, ldr_out, cols) && whole_groups(x, p->dtype, ldx, cols);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int sms;
  if ((rc = sm_count(&sms))) return rc;
  const norm::Plan plan = norm::plan_of(rows, cols, rows);
  const bool post = p->post != FP8_NORM_NONE;
  with_norm_types(p->dtype, p->res_dtype, [&](auto dt, auto rt) {
    constexpr int DT = decltype(dt)::value, RT = decltype(rt)::value;
    with_kind(plan.kind, [&](auto ck) {
      constexpr int CK = decltype(ck)::value;
      const int threads = plan.threads * plan.groups;
      auto launch = [&](auto kernel, int mode) {
        const int columns = 8 * norm::eights(CK) * (CK == 4 ? plan.threads : norm::kCtaThreads<CK, norm::kStaged>);
        const int smem = norm::fwd_smem<DT, RT>(columns, h, a.w.p, a.b.p, a.g.p || (post && a.pw.p), post && a.pb.p,
                                                mode, norm::held(CK, mode)).bytes;
        if (smem > kMostSmem) return FP8_ERR_UNSUPPORTED;
        if (int e = allow_smem(kernel)) return e;
        // as many CTAs as stay resident (80 registers a thread, 128 or 168 in the widest rows) share the rows out
        const int by_regs = 65536 / (threads * (CK == 4 ? 168 : CK == 3 ? 128 : 80)), by_smem = 232448 / (smem + 2048);
        const int resident = by_regs < by_smem ? by_regs : by_smem;
        const unsigned most = (unsigned)(sms * (resident > 1 ? resident : 1));
        const unsigned need = ((unsigned)rows + (unsigned)plan.groups - 1) / (unsigned)plan.groups;
        return launch_pdl(kernel, need < most ? need : most, dim3(plan.threads, plan.groups), smem, s, 1, a);
      };
      rc = FP8_ERR_UNSUPPORTED;
      if (whole && cols <= norm::kStagedCols) {
        const bool full = h && r_out && a.w.p && (!post || a.pw.p);
        with_bool(post, [&](auto has_post) {
          constexpr bool POST = decltype(has_post)::value;
          if (full && x && !x_row) rc = launch(norm::k_norm_fwd<DT, RT, 1, POST, CK, norm::kStaged>, norm::kStaged);
          else if (full && x_row && !x) rc = launch(norm::k_norm_fwd<DT, RT, 2, POST, CK, norm::kStaged>, norm::kStaged);
          else rc = launch(norm::k_norm_fwd<DT, RT, 0, false, CK, norm::kStaged>, norm::kStaged);
        });
      }
      if (rc == FP8_ERR_UNSUPPORTED)
        rc = launch(norm::k_norm_fwd<DT, RT, 0, false, CK == 1 ? 1 : 4, norm::kDirect>, norm::kDirect);
    });
    if (rc || !x_col) return;
    norm::Cols c = {};
    c.r = r_out ? r_out : r;
    c.ldr = r_out ? ldr_out : ldr;
    c.stats = stats;
    c.w = a.w, c.b = a.b;
    c.rows = rows, c.cols = cols, c.margin = margin, c.vec = wide_rows(c.r, p->res_dtype, c.ldr);
    c.qt = x_col->q, c.st = x_col->s, c.ldqt = x_col->ld;
    rc = launch_pdl(norm::k_norm_cols<RT>, tile_grid(rows, cols), 512, 0, s, 1, c);
  });
  return rc;
}

int fp8_logprob_fwd(const void *logits, int dtype, int rows, int cols, size_t ld, float inv_temp, const void *tokens,
                    int token_bytes, float *logp, float *entropy, int top, float *top_logp, int *top_ids,
                    float *stats, void *stream) {
  const LossArgs a = {logits, dtype, rows, cols, ld, inv_temp};
  int rc = check_loss(a);
  if (rc) return rc;
  if (top < 0 || top > FP8_TOP_MAX) return FP8_ERR_INVALID_ARG;
  if (rows == 0) return FP8_OK;  // (tensors without rows have no address)
  if ((logp != nullptr) != (tokens != nullptr) || (tokens && !index_bytes(token_bytes)) ||
      (top > 0) != (top_logp != nullptr) || (top > 0) != (top_ids != nullptr) || (!logp && !entropy && !top && !stats))
    return FP8_ERR_INVALID_ARG;
  if (cols == 0 || top > cols) return FP8_ERR_INVALID_ARG;
  if (!aligned16(stats) || (tokens && !aligned_to(tokens, token_bytes)) || !aligned_to(logp, 4) || !aligned_to(entropy, 4) ||
      !aligned_to(top_logp, 4) || !aligned_to(top_ids, 4))
    return FP8_ERR_UNALIGNED;
  int sms;
  if ((rc = sm_count(&sms))) return rc;
  loss::Fwd p = {};
  p.z = static_cast<const uint8_t *>(logits);
  p.ld = ld * dtype_bytes(dtype);
  p.rows = rows, p.cols = cols, p.beta = inv_temp;
  p.tokens = tokens, p.token_bytes = token_bytes, p.top = top;
  p.logp = logp, p.entropy = entropy, p.top_logp = top_logp, p.top_ids = top_ids, p.stats = stats;
  const LossGrid g = loss_grid(rows, cols, dtype, sms, 128);
  const size_t smem = top ? sizeof(loss::TopScratch) : 0;
  with_dtype(dtype, [&](auto dt) {
    with_bool(entropy != nullptr, [&](auto ent) {
      rc = launch_loss_fwd<decltype(dt)::value, loss::kLogprob, decltype(ent)::value>(p, g, smem,
                                                                                     static_cast<cudaStream_t>(stream));
    });
  });
  return rc;
}

int fp8_logprob_bwd(const void *logits, int dtype, int rows, int cols, size_t ld, float inv_temp, const void *tokens,
                    int token_bytes, const float *stats, const float *dlogp, const float *dentropy, int fmt, int margin,
                    const fp8_blocks *d_row, const fp8_blocks *d_col, void *dlogits, size_t ld_d, void *stream) {
  const LossArgs a = {logits, dtype, rows, cols, ld, inv_temp};
  if (rows > 0 && ((dlogp != nullptr) != (tokens != nullptr) || (!dlogp && !dentropy) || (tokens && !index_bytes(token_bytes))))
    return FP8_ERR_INVALID_ARG;
  loss::Bwd p = {};
  int rc = loss_outputs(p, a, stats, fmt, margin, d_row, d_col, dlogits, ld_d);
  if (rc || rows == 0 || cols == 0) return rc;
  if ((tokens && !aligned_to(tokens, token_bytes)) || !aligned_to(dlogp, 4) || !aligned_to(dentropy, 4))
    return FP8_ERR_UNALIGNED;
  p.tokens = tokens, p.token_bytes = token_bytes, p.g = dlogp, p.g_ent = dentropy;
  return launch_loss_bwd<false>(p, dtype, fmt, static_cast<cudaStream_t>(stream));
}

int fp8_distill_fwd(const void *logits, int dtype, int rows, int cols, size_t ld, float inv_temp, int form, int top,
                    const void *ids, int id_bytes, const void *values, int value_dtype, float *loss, float *stats,
                    int *list_ids, float *list_q, void *stream) {
  const LossArgs a = {logits, dtype, rows, cols, ld, inv_temp};
  int rc = check_loss(a);
  if (rc) return rc;
  if ((form != FP8_DISTILL_TOP && form != FP8_DISTILL_TAIL) || top < 1 || top > FP8_DISTILL_MAX || !index_bytes(id_bytes) ||
      !valid_dtype(value_dtype))
    return FP8_ERR_INVALID_ARG;
  if (rows == 0) return FP8_OK;
  if (cols == 0 || !ids || !values || !loss || !stats || !list_ids || !list_q) return FP8_ERR_INVALID_ARG;
  if (cols > FP8_DISTILL_COLS_MAX) return FP8_ERR_UNSUPPORTED;
  if (!aligned16(stats) || !aligned_to(ids, id_bytes) || !aligned_to(values, dtype_bytes(value_dtype)) ||
      !aligned_to(loss, 4) || !aligned_to(list_ids, 4) || !aligned_to(list_q, 4))
    return FP8_ERR_UNALIGNED;
  int sms;
  if ((rc = sm_count(&sms))) return rc;
  loss::Fwd p = {};
  p.z = static_cast<const uint8_t *>(logits);
  p.ld = ld * dtype_bytes(dtype);
  p.rows = rows, p.cols = cols, p.beta = inv_temp;
  p.top = top, p.ids = ids, p.id_bytes = id_bytes, p.values = values, p.value_dt = value_dtype;
  p.loss = loss, p.stats = stats, p.list_ids = list_ids, p.list_q = list_q;
  const LossGrid g = loss_grid(rows, cols, dtype, sms, top > 512 ? 256 : 128);
  const size_t marks = form != FP8_DISTILL_TAIL  ? 0
                       : dtype == FP8_DT_F32     ? loss::mark_bytes<FP8_DT_F32>(g.vecs, (int)g.threads)
                                                 : loss::mark_bytes<FP8_DT_BF16>(g.vecs, (int)g.threads);
  const size_t smem = sizeof(loss::ListScratch) + marks;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  with_dtype(dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    rc = form == FP8_DISTILL_TOP ? launch_loss_fwd<DT, loss::kListTop, false>(p, g, smem, s)
                                 : launch_loss_fwd<DT, loss::kListTail, false>(p, g, smem, s);
  });
  return rc;
}

int fp8_distill_bwd(const void *logits, int dtype, int rows, int cols, size_t ld, float inv_temp, int top,
                    const int *list_ids, const float *list_q, const float *stats, const float *dloss, int fmt,
                    int margin, const fp8_blocks *d_row, const fp8_blocks *d_col, void *dlogits, size_t ld_d,
                    void *stream) {
  const LossArgs a = {logits, dtype, rows, cols, ld, inv_temp};
  if (top < 1 || top > FP8_DISTILL_MAX || (rows > 0 && (!list_ids || !list_q || !dloss))) return FP8_ERR_INVALID_ARG;
  loss::Bwd p = {};
  int rc = loss_outputs(p, a, stats, fmt, margin, d_row, d_col, dlogits, ld_d);
  if (rc || rows == 0 || cols == 0) return rc;
  if (cols > FP8_DISTILL_COLS_MAX) return FP8_ERR_UNSUPPORTED;
  if (!aligned_to(list_ids, 4) || !aligned_to(list_q, 4) || !aligned_to(dloss, 4)) return FP8_ERR_UNALIGNED;
  p.g = dloss, p.K = top, p.list_ids = list_ids, p.list_q = list_q;
  return launch_loss_bwd<true>(p, dtype, fmt, static_cast<cudaStream_t>(stream));
}

// Reads and clears this unit's status word on the stream; the caller waits for it.
int passes_take_status(unsigned *host_out, cudaStream_t s) {
  k_take_status<<<1, 1, 0, s>>>();
  if (cudaGetLastError() != cudaSuccess) return FP8_ERR_CUDA;
  return cuda_rc(cudaMemcpyFromSymbolAsync(host_out, g_status_taken, sizeof(unsigned), 0, cudaMemcpyDeviceToHost, s));
}

}  // extern "C"
