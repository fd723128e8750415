// norm.cuh -- what stands between two sublayers: the norm of a sublayer's
// output, its gate, the scaled residual, and the norm before the next sublayer,
// with their backward pass.
//
//   u  = (h - mu1) rho1 w1 + b1  (or h)          rho = 1 / sqrt(mean((v - mu)^2) + eps)
//   r' = a r + g u,  rounded as it is stored      mu = mean, or 0 (RMS)
//   x  = n2 w2 + b2,  n2 = (r' - mu2) rho2
//
//   G   = dr' + rho2 (dx w2 - mean(dx w2) - n2 mean(dx w2 n2))     (the first mean: layer norms only)
//   dr  = a G
//   dh  = rho1 (q - mean(q) - n1 mean(q n1)),  q = G g w1           (g G without a post norm)
//   dw2 = sum dx n2,  db2 = sum dx
//   A   = sum G n1 (or G h), C = sum G over the rows of a gate row: dg = w1 A + b1 C,
//   dw1 = sum over the gate rows g A,  db1 = sum g C
//
// Each matrix is read and written once: the bytes of h, r, r', x forward, of dx,
// dr', r', h, dr, dh backward.
#pragma once

#include "block_scale.cuh"
#include "pipeline.cuh"

namespace fp8lib {
namespace norm {

using block::Raw8;

// A row belongs to a group of T threads (a multiple of 32) in each of C CTAs
// (a cluster); a thread holds NV vectors of eight neighbouring columns.
constexpr int kGroupThreads = 512;       // the most threads of a row in one CTA
constexpr int kFwdThreads = 256;         // a CTA takes several narrow rows, up to this many threads
constexpr int kBwdThreads = 512;
constexpr int kBwdCols = 8 * kBwdThreads;  // columns of a CTA in the backward pass

struct Vec {
  const void *p;
  int dt;
};

// Eight parameters at column c (a multiple of 8); `fill` where there are none.
__device__ __forceinline__ void load_param8(Vec v, size_t off, int c, int cols, float fill, float (&f)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j++) f[j] = fill;
  if (!v.p || c >= cols) return;
  if (v.dt == FP8_DT_F32) {
    const float *p = reinterpret_cast<const float *>(v.p) + off + c;
    if (c + 8 <= cols && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
      const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
      f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; j++)
      if (c + j < cols) f[j] = __ldg(p + j);
    return;
  }
  const uint16_t *p = reinterpret_cast<const uint16_t *>(v.p) + off + c;
  Raw8<FP8_DT_BF16> r;
  if (c + 8 <= cols && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p));
    r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
  } else {
    uint32_t e[8];
#pragma unroll
    for (int j = 0; j < 8; j++) e[j] = c + j < cols ? __ldg(p + j) : 0u;
#pragma unroll
    for (int j = 0; j < 4; j++) r.w[j] = e[2 * j] | (e[2 * j + 1] << 16);
  }
  if (v.dt == FP8_DT_BF16) {
    block::unpack8<FP8_DT_BF16>(r, f);
  } else {
    Raw8<FP8_DT_F16> h;
#pragma unroll
    for (int j = 0; j < 4; j++) h.w[j] = r.w[j];
    block::unpack8<FP8_DT_F16>(h, f);
  }
}

__device__ __forceinline__ float param_at(Vec v, size_t i, float fill) {
  if (!v.p) return fill;
  if (v.dt == FP8_DT_F32) return __ldg(reinterpret_cast<const float *>(v.p) + i);
  const uint16_t h = __ldg(reinterpret_cast<const uint16_t *>(v.p) + i);
  return v.dt == FP8_DT_BF16 ? __uint_as_float((uint32_t)h << 16) : __half2float(__ushort_as_half(h));
}

__device__ __forceinline__ void store_param(Vec v, size_t i, float x) {
  if (!v.p) return;
  if (v.dt == FP8_DT_F32) reinterpret_cast<float *>(const_cast<void *>(v.p))[i] = x;
  else if (v.dt == FP8_DT_BF16) reinterpret_cast<__nv_bfloat16 *>(const_cast<void *>(v.p))[i] = __float2bfloat16_rn(x);
  else reinterpret_cast<__half *>(const_cast<void *>(v.p))[i] = __float2half_rn(x);
}

// A row's eight elements at column c; 0 behind the row's end.
template <int DT>
__device__ __forceinline__ Raw8<DT> load_row8(const void *base, size_t ld, bool wide, int row, int rows, int c,
                                              int cols) {
  return wide ? block::load_raw8_wide<DT>(base, ld, row, c, rows, cols)
              : block::load_raw8_single<DT>(base, ld, row, c, rows, cols);
}

template <int DT>
__device__ __forceinline__ float as_stored(float x) {
  if constexpr (DT == FP8_DT_F32) return x;
  else if constexpr (DT == FP8_DT_BF16) return __bfloat162float(__float2bfloat16_rn(x));
  else return __half2float(__float2half_rn(x));
}

// Sums over the threads of a row.  Two buffers in turn: one barrier a sum.
struct RowSum {
  float (*slots)[2][128];  // shared memory: [2 buffers][2 sums][warps of the row's CTAs]
  int group, warps;        // this row's group in the CTA, its warps
  unsigned ctas, rank;     // CTAs of the row
  int buf;

  __device__ __forceinline__ void wait() const {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(warps * 32) : "memory");
  }

  template <int N>
  __device__ __forceinline__ void operator()(float (&v)[N]) {
    static_assert(N <= 2, "slots");
#pragma unroll
    for (int n = 0; n < N; n++)
#pragma unroll
      for (int b = 16; b > 0; b /= 2) v[n] += __shfl_xor_sync(0xffffffffu, v[n], b);
    if (warps == 1 && ctas == 1) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (ctas == 1) {
      const int at = group * warps;
      if (lane == 0) {
#pragma unroll
        for (int n = 0; n < N; n++) slots[buf][n][at + warp] = v[n];
      }
      wait();
#pragma unroll
      for (int n = 0; n < N; n++) v[n] = lane < warps ? slots[buf][n][at + lane] : 0.0f;
#pragma unroll
      for (int n = 0; n < N; n++)
#pragma unroll
        for (int b = 8; b > 0; b /= 2) v[n] += __shfl_xor_sync(0xffffffffu, v[n], b);
    } else {
      // every CTA of the cluster gets every warp's sum
      if ((unsigned)lane < ctas) {
#pragma unroll
        for (int n = 0; n < N; n++) {
          uint32_t there;
          asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                       : "=r"(there)
                       : "r"(smem_u32(&slots[buf][n][rank * warps + warp])), "r"(lane));
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(there), "f"(v[n]) : "memory");
        }
      }
      asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
#pragma unroll
      for (int n = 0; n < N; n++) {
        v[n] = 0.0f;
        for (int i = lane; i < (int)ctas * warps; i += 32) v[n] += slots[buf][n][i];
#pragma unroll
        for (int b = 16; b > 0; b /= 2) v[n] += __shfl_xor_sync(0xffffffffu, v[n], b);
      }
    }
#pragma unroll
    for (int n = 0; n < N; n++) v[n] = __shfl_sync(0xffffffffu, v[n], 0);
    buf ^= 1;
  }
};

__device__ __forceinline__ RowSum row_sum(float (*slots)[2][128], unsigned ctas) {
  RowSum s;
  s.slots = slots;
  s.group = threadIdx.y;
  s.warps = blockDim.x >> 5;
  s.ctas = ctas;
  s.rank = ctas > 1 ? blockIdx.x % ctas : 0;
  s.buf = 0;
  if (ctas > 1)  // the other CTAs' shared memory is there
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  return s;
}

// mean and rstd of a row whose NV x 8 elements a thread holds in v (n[i] of the
// eight are columns of the row).
template <int NV>
__device__ __forceinline__ float2 row_stats(const float (&v)[NV][8], const int (&n)[NV], int kind, int cols, float eps,
                                            RowSum &sum) {
  float mean = 0.0f;
  const float inv = 1.0f / (float)cols;
  if (kind == FP8_NORM_LAYER) {
    float t[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
      for (int j = 0; j < 8; j++) t[0] += j < n[i] ? v[i][j] : 0.0f;
    sum(t);
    mean = t[0] * inv;
  }
  float q[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NV; i++)
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const float d = j < n[i] ? v[i][j] - mean : 0.0f;
      q[0] = fmaf(d, d, q[0]);
    }
  sum(q);
  return make_float2(mean, rsqrtf(fmaf(q[0], inv, eps)));
}

// r' = a r + g u takes each product rounded: 0.9f is not 0.9, but 0.9f * 10
// rounds to 9, and sums of 16-bit numbers that lie halfway between two others
// (one in some thousand do) then go to the side that the scale as written gives.
struct Fwd {
  const void *h, *r;
  void *r_out, *x;
  float *stats;
  size_t ldh, ldr, ldro, ldx;
  uint8_t *xq, *xs;  // codes of 1x128 blocks, or null
  size_t ldxq;
  int rows, cols, pre, post;
  Vec w, b, pw, pb, g;
  int gate_rows;
  size_t ldg;
  float alpha, eps;
  int margin;
  int wide_h, wide_r, wide_ro, wide_x;
};

// The codes of a thread's eight elements of a row's 1x128 block (16 lanes hold
// one), its scale, and, with the last row, the padding of its scales.
__device__ __forceinline__ void store_block8(const Fwd &p, int row, int c, const float (&v)[8]) {
  float a = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; j += 2) a = block::absmax2(a, v[j], v[j + 1]);
  uint32_t m = __float_as_uint(a);
#pragma unroll
  for (int b = 8; b > 0; b /= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, b));
  const int k = block::block_exponent(m, kMaxE4M3, p.margin), l = threadIdx.x & 15;
  const int kblocks = (p.cols + 127) / 128, blk = c >> 7;
  if (blk < kblocks) {
    if (l == 0) block::put_scale(p.xs, row, blk, kblocks, k);
    if (row == p.rows - 1)
      for (int r = p.rows + l; r < (p.rows + 127) / 128 * 128; r += 16) block::put_scale(p.xs, r, blk, kblocks, 0);
  }
  float2 s[4];
  block::spread_scale(pow2f(k), s);
  const uint2 o = m >= 0x7f800000u ? block::enc8_any<FP8_E4M3>(v, s) : block::enc8<FP8_E4M3>(v, s);
  uint8_t *q = p.xq + (size_t)row * p.ldxq + c;
  if (c + 8 <= p.cols) {
    __stcs(reinterpret_cast<uint2 *>(q), o);
  } else if (c < p.cols) {
    for (int j = 0; j < p.cols - c; j++) q[j] = (uint8_t)((j < 4 ? o.x : o.y) >> (8 * (j & 3)));
  }
}

template <int DT, int RT, int NV>
__global__ void __launch_bounds__(kGroupThreads) k_norm_fwd(const Fwd p, unsigned ctas) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float slots[2][2][128];
  RowSum sum = row_sum(slots, ctas);
  const unsigned stride = gridDim.x / ctas * blockDim.y;
  int c[NV], n[NV];
#pragma unroll
  for (int i = 0; i < NV; i++) {
    c[i] = (int)((sum.rank * NV + i) * blockDim.x + threadIdx.x) * 8;
    n[i] = max(0, min(8, p.cols - c[i]));
  }
  for (unsigned at = blockIdx.x / ctas * blockDim.y + threadIdx.y; at < (unsigned)p.rows; at += stride) {
    const int row = (int)at;
    float v[NV][8], y[NV][8];
    if (p.h) {
#pragma unroll
      for (int i = 0; i < NV; i++) block::unpack8<DT>(load_row8<DT>(p.h, p.ldh, p.wide_h, row, p.rows, c[i], p.cols), v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < NV; i++)
#pragma unroll
        for (int j = 0; j < 8; j++) v[i][j] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < NV; i++) block::unpack8<RT>(load_row8<RT>(p.r, p.ldr, p.wide_r, row, p.rows, c[i], p.cols), y[i]);
    float2 s1 = make_float2(0.0f, 1.0f), s2 = make_float2(0.0f, 1.0f);
    if (p.post != FP8_NORM_NONE) {
      s1 = row_stats(v, n, p.post, p.cols, p.eps, sum);
#pragma unroll
      for (int i = 0; i < NV; i++) {
        float w[8], b[8];
        load_param8(p.pw, 0, c[i], p.cols, 1.0f, w);
        load_param8(p.pb, 0, c[i], p.cols, 0.0f, b);
#pragma unroll
        for (int j = 0; j < 8; j++) v[i][j] = fmaf((v[i][j] - s1.x) * s1.y, w[j], b[j]);
      }
    }
    const size_t gate_at = p.g.p ? (size_t)(row / p.gate_rows) * p.ldg : 0;
#pragma unroll
    for (int i = 0; i < NV; i++) {
      float g[8];
      load_param8(p.g, gate_at, c[i], p.cols, 1.0f, g);
#pragma unroll
      for (int j = 0; j < 8; j++)
        y[i][j] = j < n[i] ? as_stored<RT>(__fadd_rn(__fmul_rn(p.alpha, y[i][j]), __fmul_rn(g[j], v[i][j]))) : 0.0f;
      if (p.r_out) block::store8<RT>(p.wide_ro, p.r_out, p.ldro, row, c[i], p.rows, p.cols, y[i]);
    }
    if (p.pre != FP8_NORM_NONE) {
      s2 = row_stats(y, n, p.pre, p.cols, p.eps, sum);
      if (p.x || p.xq) {
#pragma unroll
        for (int i = 0; i < NV; i++) {
          float w[8], b[8];
          load_param8(p.w, 0, c[i], p.cols, 1.0f, w);
          load_param8(p.b, 0, c[i], p.cols, 0.0f, b);
#pragma unroll
          for (int j = 0; j < 8; j++) v[i][j] = j < n[i] ? fmaf((y[i][j] - s2.x) * s2.y, w[j], b[j]) : 0.0f;
          if (p.x) block::store8<DT>(p.wide_x, p.x, p.ldx, row, c[i], p.rows, p.cols, v[i]);
          if (p.xq) store_block8(p, row, c[i], v[i]);
        }
      }
    }
    if (p.stats && sum.rank == 0 && threadIdx.x == 0)
      reinterpret_cast<float4 *>(p.stats)[row] = make_float4(s1.x, s1.y, s2.x, s2.y);
  }
}

// x again from r' and its statistics, as codes of 128x1 blocks: tiles of
// block_scale.cuh.  2 B (or 4) read and 1 written per element.
struct Cols {
  const void *r;
  size_t ldr;
  const float *stats;
  Vec w, b;
  int rows, cols, margin, vec;
  uint8_t *qt, *st;
  size_t ldqt;
};

template <int RT>
__global__ void __launch_bounds__(512, 2) k_norm_cols(const Cols p) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int RP = 4;
  using G = block::Geo<RP>;
  __shared__ block::ColScratch<RP> sc;
  const int tiles_c = (p.cols + block::kTile - 1) / block::kTile;
  const auto [row0, col0] = block::tile_at(blockIdx.x, tiles_c);
  const int col = col0 + (threadIdx.x & 15) * 8;
  Raw8<RT> raw[RP];
  block::load_tile<RT>(p.r, p.ldr, p.vec, row0, col0, p.rows, p.cols, raw);
  float w[8], b[8], f[RP][8];
  load_param8(p.w, 0, col, p.cols, 1.0f, w);
  load_param8(p.b, 0, col, p.cols, 0.0f, b);
#pragma unroll
  for (int i = 0; i < RP; i++) {
    const int row = row0 + (threadIdx.x >> 4) + i * G::kStep;
    const float4 s = __ldg(reinterpret_cast<const float4 *>(p.stats) + min(row, p.rows - 1));
    block::unpack8<RT>(raw[i], f[i]);
#pragma unroll
    for (int j = 0; j < 8; j++)
      f[i][j] = row < p.rows && col + j < p.cols ? fmaf((f[i][j] - s.z) * s.w, w[j], b[j]) : 0.0f;
  }
  block::put_tile_maxima(f, sc);
  __syncthreads();
  bool bad = false;
  if (threadIdx.x < block::kTile)
    bad = block::finish_column(sc, threadIdx.x, p.st, row0, col0, p.rows, kMaxE4M3, p.margin);
  bad = __syncthreads_or(bad);
  block::store_tile_cols<FP8_E4M3>(f, sc, bad, p.qt, p.ldqt, row0, col0, p.rows, p.cols);
}

// ---------------------------------------------------------------- backward
// The rows are dealt out in units, each within one gate row; a cluster takes
// neighbouring units.  Its sums over rows stay in registers: dw2 and db2 until
// it ends, A and C until its unit does.
struct Plan {
  int ctas;                // per row
  int threads, groups;     // of a CTA
  int gate_rows, unit_rows, per_gate;  // rows of a gate row and of a unit, units per gate row
  long long units;
  int clusters;
};

constexpr int kMostClusters = 148;  // (a CTA of 512 threads on every SM of a B200)

inline Plan plan_of(int rows, int cols, int gate_rows) {
  Plan p = {};
  p.ctas = (cols + kBwdCols - 1) / kBwdCols;
  const int vecs = ((cols + 7) / 8 + p.ctas - 1) / p.ctas;
  p.threads = (vecs + 31) / 32 * 32;
  p.groups = p.ctas > 1 ? 1 : kBwdThreads / p.threads;
  p.gate_rows = gate_rows < rows ? gate_rows : rows;
  const int most = kMostClusters / p.ctas;
  p.unit_rows = rows / most + (rows % most != 0);
  if (p.unit_rows < p.groups) p.unit_rows = p.groups;
  if (rows == 0) return p;
  p.per_gate = p.gate_rows / p.unit_rows + (p.gate_rows % p.unit_rows != 0);
  p.units = ((long long)rows + p.gate_rows - 1) / p.gate_rows * p.per_gate;
  p.clusters = (int)(p.units < most ? p.units : most);
  return p;
}

struct Bwd {
  const void *dx, *dro, *h, *ro;
  const float *stats;
  void *dh, *dr;
  size_t lddx, lddro, ldh, ldro, lddh, lddr;
  int rows, cols, pre, post;
  Vec w, pw, g;
  size_t ldg;
  float alpha;
  int wide_dx, wide_dro, wide_h, wide_ro, wide_dh, wide_dr;
  float *ef, *ac;  // partial sums [cluster][2][cols] and [unit][2][cols], or null
  int gate_rows, unit_rows, per_gate;
  long long units;
};

// Adds up the groups of a CTA and writes one partial sum.
__device__ __forceinline__ void flush(float (&a)[8], float *comb, float *out, int c, int cols) {
  const int t = threadIdx.x, T = blockDim.x;
  if (blockDim.y > 1) {
    __syncthreads();
    float4 *at = reinterpret_cast<float4 *>(comb) + (threadIdx.y * T + t) * 2;
    at[0] = make_float4(a[0], a[1], a[2], a[3]);
    at[1] = make_float4(a[4], a[5], a[6], a[7]);
    __syncthreads();
    if (threadIdx.y == 0) {
      for (int y = 1; y < (int)blockDim.y; y++) {
        const float *q = comb + (y * T + t) * 8;
#pragma unroll
        for (int j = 0; j < 8; j++) a[j] += q[j];
      }
    }
  }
  if (threadIdx.y == 0) {
#pragma unroll
    for (int j = 0; j < 8; j++)
      if (c + j < cols) out[c + j] = a[j];
  }
#pragma unroll
  for (int j = 0; j < 8; j++) a[j] = 0.0f;
}

template <int DT, int RT>
__global__ void __launch_bounds__(kBwdThreads, 1) k_norm_bwd(const Bwd p, unsigned ctas) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float slots[2][2][128];
  __shared__ __align__(16) float comb[kBwdThreads * 8];
  RowSum sum = row_sum(slots, ctas);
  const int c = (int)(sum.rank * blockDim.x + threadIdx.x) * 8, n = max(0, min(8, p.cols - c));
  const float inv = 1.0f / (float)p.cols;
  const unsigned cluster = blockIdx.x / ctas, clusters = gridDim.x / ctas;
  const long long u0 = p.units * cluster / clusters, u1 = p.units * (cluster + 1) / clusters;
  float w2[8], E[8], F[8], A[8], C[8];
  load_param8(p.w, 0, c, p.cols, 1.0f, w2);
#pragma unroll
  for (int j = 0; j < 8; j++) E[j] = F[j] = A[j] = C[j] = 0.0f;
  for (long long u = u0; u < u1; u++) {
    const int gate = (int)(u / p.per_gate);
    const int first = gate * p.gate_rows, last = (int)min((long long)first + p.gate_rows, (long long)p.rows);
    const long long r0 = first + (u - (long long)gate * p.per_gate) * p.unit_rows;
    const int r1 = (int)min(r0 + p.unit_rows, (long long)last);
    float gw[8];
    load_param8(p.g, (size_t)gate * p.ldg, c, p.cols, 1.0f, gw);
    if (p.post != FP8_NORM_NONE) {
      float pw[8];
      load_param8(p.pw, 0, c, p.cols, 1.0f, pw);
#pragma unroll
      for (int j = 0; j < 8; j++) gw[j] *= pw[j];
    }
    for (long long row_ = r0 + threadIdx.y; row_ < r1; row_ += blockDim.y) {
      const int row = (int)row_;
      const float4 s = __ldg(reinterpret_cast<const float4 *>(p.stats) + row);
      float G[8], t[8], v[8];
      if (p.dro) {
        block::unpack8<RT>(load_row8<RT>(p.dro, p.lddro, p.wide_dro, row, p.rows, c, p.cols), G);
      } else {
#pragma unroll
        for (int j = 0; j < 8; j++) G[j] = 0.0f;
      }
      if (p.pre != FP8_NORM_NONE) {
        block::unpack8<DT>(load_row8<DT>(p.dx, p.lddx, p.wide_dx, row, p.rows, c, p.cols), t);
        block::unpack8<RT>(load_row8<RT>(p.ro, p.ldro, p.wide_ro, row, p.rows, c, p.cols), v);
        float m[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 8; j++) {
          v[j] = (v[j] - s.z) * s.w;  // n2
          E[j] = fmaf(t[j], v[j], E[j]);
          F[j] += t[j];
          t[j] *= w2[j];
          m[0] += t[j];
          m[1] = fmaf(t[j], v[j], m[1]);
        }
        sum(m);
        const float m0 = p.pre == FP8_NORM_LAYER ? m[0] * inv : 0.0f, m1 = m[1] * inv;
#pragma unroll
        for (int j = 0; j < 8; j++) G[j] = j < n ? fmaf(s.w, t[j] - m0 - v[j] * m1, G[j]) : 0.0f;
      }
      if (p.dr) {
#pragma unroll
        for (int j = 0; j < 8; j++) t[j] = p.alpha * G[j];
        block::store8<RT>(p.wide_dr, p.dr, p.lddr, row, c, p.rows, p.cols, t);
      }
      if (p.h) {
        block::unpack8<DT>(load_row8<DT>(p.h, p.ldh, p.wide_h, row, p.rows, c, p.cols), v);
        if (p.post != FP8_NORM_NONE) {
          float m[2] = {0.0f, 0.0f};
#pragma unroll
          for (int j = 0; j < 8; j++) {
            v[j] = (v[j] - s.x) * s.y;  // n1
            t[j] = G[j] * gw[j];
            m[0] += t[j];
            m[1] = fmaf(t[j], v[j], m[1]);
          }
          sum(m);
          const float m0 = p.post == FP8_NORM_LAYER ? m[0] * inv : 0.0f, m1 = m[1] * inv;
#pragma unroll
          for (int j = 0; j < 8; j++) t[j] = s.y * (t[j] - m0 - v[j] * m1);
        } else {
#pragma unroll
          for (int j = 0; j < 8; j++) t[j] = G[j] * gw[j];
        }
        if (p.dh) block::store8<DT>(p.wide_dh, p.dh, p.lddh, row, c, p.rows, p.cols, t);
#pragma unroll
        for (int j = 0; j < 8; j++) {
          A[j] = fmaf(G[j], v[j], A[j]);
          C[j] += G[j];
        }
      }
    }
    if (p.ac) {
      flush(A, comb, p.ac + (size_t)(2 * u) * p.cols, c, p.cols);
      flush(C, comb, p.ac + (size_t)(2 * u + 1) * p.cols, c, p.cols);
    }
  }
  if (p.ef) {
    flush(E, comb, p.ef + (size_t)(2 * cluster) * p.cols, c, p.cols);
    flush(F, comb, p.ef + (size_t)(2 * cluster + 1) * p.cols, c, p.cols);
  }
}

struct Params {
  const float *ef, *ac;
  int cols, clusters, gates, per_gate, post;
  Vec pw, pb, g;
  size_t ldg;
  Vec dw, db, dpw, dpb, dg;  // outputs
  size_t lddg;
};

constexpr int kParamLanes = 16;

// Adds up v over the lanes (threadIdx.y) of each column, in their order.
__device__ __forceinline__ float lane_sum(float v, float (&sh)[kParamLanes][33]) {
  __syncthreads();
  sh[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int y = 0; y < kParamLanes; y++) s += sh[y][threadIdx.x];
  return s;
}

// The parameters' gradients from the partial sums: 32 columns a CTA.
__global__ void __launch_bounds__(32 * kParamLanes) k_norm_params(const Params p) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float sh[kParamLanes][33];
  const int c = blockIdx.x * 32 + threadIdx.x, y = threadIdx.y;
  const bool in = c < p.cols;
  if (p.dw.p || p.db.p) {
    float e = 0.0f, f = 0.0f;
    if (in) {
      for (int i = y; i < p.clusters; i += kParamLanes) {
        e += p.ef[(size_t)(2 * i) * p.cols + c];
        f += p.ef[(size_t)(2 * i + 1) * p.cols + c];
      }
    }
    e = lane_sum(e, sh);
    f = lane_sum(f, sh);
    if (in && y == 0) {
      store_param(p.dw, c, e);
      store_param(p.db, c, f);
    }
  }
  if (!p.dg.p && !p.dpw.p && !p.dpb.p) return;
  const float pw = in && p.post != FP8_NORM_NONE ? param_at(p.pw, c, 1.0f) : 1.0f;
  const float pb = in && p.post != FP8_NORM_NONE ? param_at(p.pb, c, 0.0f) : 0.0f;
  // few gate rows: the lanes share each one's units; many: each lane takes whole gate rows
  const bool share = p.gates < kParamLanes;
  float wsum = 0.0f, bsum = 0.0f;
  for (int s = share ? 0 : y; s < p.gates; s += share ? 1 : kParamLanes) {
    float a = 0.0f, k = 0.0f;
    if (in) {
      for (long long i = share ? y : 0; i < p.per_gate; i += share ? kParamLanes : 1) {
        const size_t u = (size_t)s * p.per_gate + i;
        a += p.ac[2 * u * p.cols + c];
        k += p.ac[(2 * u + 1) * p.cols + c];
      }
    }
    if (share) {
      a = lane_sum(a, sh);
      k = lane_sum(k, sh);
    }
    if (in) {
      const float g = param_at(p.g, (size_t)s * p.ldg + c, 1.0f);
      wsum = fmaf(g, a, wsum);
      bsum = fmaf(g, k, bsum);
      if (!share || y == 0) store_param(p.dg, (size_t)s * p.lddg + c, fmaf(pw, a, pb * k));
    }
  }
  if (!share) {
    wsum = lane_sum(wsum, sh);
    bsum = lane_sum(bsum, sh);
  }
  if (in && y == 0) {
    store_param(p.dpw, c, wsum);
    store_param(p.dpb, c, bsum);
  }
}

}  // namespace norm
}  // namespace fp8lib
