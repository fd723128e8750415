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

// A row belongs to a group of T threads (a multiple of 32) of a CTA; a thread
// holds NV chunks of eight columns.  A CTA takes as many narrow rows at a time
// as it has threads for, and row after row while it lives.
constexpr int kThreads = 256;      // of a CTA, but for the widest rows
constexpr int kMostThreads = 512;
constexpr int kMostWarps = kMostThreads / 32;
constexpr int kStagedCols = 12288;  // the widest staged rows: 384 threads, 168 registers each
template <int NV, int MODE>
constexpr int kCtaThreads = NV < 4 ? kThreads : MODE == 0 ? kStagedCols / 32 : kMostThreads;

// How rows are read and written.
//   kStaged  eight neighbouring columns a chunk, in 16-byte pieces; the next
//            row's are copied into the thread's own part of shared memory while
//            it works on the present one (no barriers: nobody else reads them)
//   kDirect  rows that start anywhere: the lanes of a warp take neighbouring
//            columns, and element by element from memory, twice where two
//            passes need them
enum { kStaged = 0, kDirect = 1 };

// The chunk v of a thread, and whether it lies in the row (kStaged: all of it).
struct Place {
  int cols, t, T;
  template <int MODE>
  __device__ __forceinline__ int col(int v, int j) const {
    return MODE == kStaged ? (v * T + t) * 8 + j : (v * T + (t & ~31)) * 8 + 32 * j + (t & 31);
  }
  template <int MODE>
  __device__ __forceinline__ bool has(int v, int j) const {
    return col<MODE>(v, MODE == kStaged ? 0 : j) < cols;
  }
};

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


template <int MODE>
__device__ __forceinline__ void load_params(Vec v, size_t off, const Place &at, int chunk, float fill, float (&f)[8]) {
  if constexpr (MODE == kStaged) {
    load_param8(v, off, at.col<MODE>(chunk, 0), at.cols, fill, f);
  } else {
#pragma unroll
    for (int j = 0; j < 8; j++) f[j] = at.has<MODE>(chunk, j) ? param_at(v, off + at.col<MODE>(chunk, j), fill) : fill;
  }
}

template <int DT>
__device__ __forceinline__ float as_stored(float x) {
  if constexpr (DT == FP8_DT_F32) return x;
  else if constexpr (DT == FP8_DT_BF16) return __bfloat162float(__float2bfloat16_rn(x));
  else return __half2float(__float2half_rn(x));
}

template <int DT>
constexpr int kPieces = DT == FP8_DT_F32 ? 2 : 1;  // of 16 bytes in a chunk

// A matrix's chunks of one row.  `slot`: this matrix's part of the CTA's shared
// memory, [chunk][piece][thread] of 16 bytes.
template <int DT, int MODE>
struct Rows {
  const uint8_t *p;
  size_t ld;  // bytes
  uint8_t *slot;
  int threads, tid;

  __device__ __forceinline__ void fetch(const Place &at, int v, int row) const {
    if constexpr (MODE == kStaged) {
      if (!at.has<MODE>(v, 0)) return;
      const uint8_t *src = p + (size_t)row * ld + (size_t)at.col<MODE>(v, 0) * (DT == FP8_DT_F32 ? 4 : 2);
#pragma unroll
      for (int i = 0; i < kPieces<DT>; i++)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                         smem_u32(slot + (size_t)((v * kPieces<DT> + i) * threads + tid) * 16)),
                     "l"(src + 16 * i)
                     : "memory");
    }
  }
  __device__ __forceinline__ void get(const Place &at, int v, int row, float (&f)[8]) const {
    if constexpr (MODE == kStaged) {
      Raw8<DT> r;
#pragma unroll
      for (int i = 0; i < kPieces<DT>; i++) {
        const uint4 w = *reinterpret_cast<const uint4 *>(slot + (size_t)((v * kPieces<DT> + i) * threads + tid) * 16);
        r.w[4 * i] = w.x, r.w[4 * i + 1] = w.y, r.w[4 * i + 2] = w.z, r.w[4 * i + 3] = w.w;
      }
      block::unpack8<DT>(r, f);
    } else {
      const uint8_t *src = p + (size_t)row * ld;
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const int c = min(at.col<MODE>(v, j), at.cols - 1);
        if constexpr (DT == FP8_DT_F32) f[j] = reinterpret_cast<const float *>(src)[c];
        else if constexpr (DT == FP8_DT_BF16) f[j] = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(src)[c]);
        else f[j] = __half2float(reinterpret_cast<const __half *>(src)[c]);
      }
    }
  }
};

template <int DT, int MODE>
__device__ __forceinline__ void put_row(void *out, size_t ld, const Place &at, int v, int row, const float (&f)[8]) {
  if constexpr (MODE == kStaged) {
    if (!at.has<MODE>(v, 0)) return;
    constexpr int esz = DT == FP8_DT_F32 ? 4 : 2;
    uint4 w[DT == FP8_DT_F32 ? 2 : 1];
    block::pack8<DT>(f, w);
    uint4 *q = reinterpret_cast<uint4 *>(reinterpret_cast<uint8_t *>(out) + ((size_t)row * ld + at.col<MODE>(v, 0)) * esz);
    __stcs(q, w[0]);
    if constexpr (DT == FP8_DT_F32) __stcs(q + 1, w[1]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; j++)
      if (at.has<MODE>(v, j)) {
        const size_t i = (size_t)row * ld + at.col<MODE>(v, j);
        if constexpr (DT == FP8_DT_F32) reinterpret_cast<float *>(out)[i] = f[j];
        else if constexpr (DT == FP8_DT_BF16) reinterpret_cast<__nv_bfloat16 *>(out)[i] = __float2bfloat16_rn(f[j]);
        else reinterpret_cast<__half *>(out)[i] = __float2half_rn(f[j]);
      }
  }
}

// Zero outside the row.
template <int MODE>
__device__ __forceinline__ void mask(const Place &at, int v, float (&f)[8]) {
  if constexpr (MODE == kStaged) {
    if (!at.has<MODE>(v, 0)) {
#pragma unroll
      for (int j = 0; j < 8; j++) f[j] = 0.0f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; j++) f[j] = at.has<MODE>(v, j) ? f[j] : 0.0f;
  }
}

// Eight floats of a thread in shared memory, its own: [half][thread] of 16 bytes
// for each chunk.
__device__ __forceinline__ void put8(float *s, int threads, int tid, int v, const float (&f)[8]) {
  float4 *p = reinterpret_cast<float4 *>(s) + (size_t)v * 2 * threads + tid;
  p[0] = make_float4(f[0], f[1], f[2], f[3]);
  p[threads] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void get8(const float *s, int threads, int tid, int v, float (&f)[8]) {
  const float4 *p = reinterpret_cast<const float4 *>(s) + (size_t)v * 2 * threads + tid;
  const float4 a = p[0], b = p[threads];
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

// What the warps of a row's group tell one another: up to 8 numbers each, two
// buffers in turn, so that one barrier serves an exchange.
struct Exchange {
  float (*slots)[8][kMostWarps];  // shared memory [2][8][warps of the CTA]
  int group, warps, buf;

  __device__ __forceinline__ void put(int n, float x) { slots[buf][n][group * warps + (threadIdx.x >> 5)] = x; }
  __device__ __forceinline__ void wait() const {
    if (warps > 1) asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(warps * 32) : "memory");
    else __syncwarp();
  }
  __device__ __forceinline__ float get(int n, int w) const { return slots[buf][n][group * warps + w]; }
  __device__ __forceinline__ float sum(int n) const {
    float s = 0.0f;
    if ((warps & 3) == 0) {  // (rows of 1024 columns and more)
      for (int w = 0; w < warps; w += 4) {
        const float4 q = *reinterpret_cast<const float4 *>(&slots[buf][n][group * warps + w]);
        s += (q.x + q.y) + (q.z + q.w);
      }
    } else {
      for (int w = 0; w < warps; w++) s += get(n, w);
    }
    return s;
  }
  __device__ __forceinline__ void next() { buf ^= 1; }
};

// Sums over a warp of N numbers a thread, in halves: a step gives half of the
// numbers away and takes the other half's share, until each lane adds up one.
// Lane l then has the sum of number l / (32 / N).
template <int N>
__device__ __forceinline__ float warp_sums(float (&v)[N]) {
  static_assert(N == 1 || N == 2 || N == 4 || N == 8, "halved down to one");
  const int lane = threadIdx.x & 31;
  int bit = 16;
#pragma unroll
  for (int n = N / 2; n > 0; n /= 2, bit /= 2) {
#pragma unroll
    for (int i = 0; i < n; i++) {
      const float send = (lane & bit) ? v[i] : v[i + n], keep = (lane & bit) ? v[i + n] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
    }
  }
#pragma unroll
  for (; bit > 0; bit /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], bit);
  return v[0];
}

// The sums over a row of N numbers a thread, to every thread.
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], Exchange &x) {
  const float s = warp_sums(v);
  const int lane = threadIdx.x & 31;
  if (x.warps == 1) {
#pragma unroll
    for (int n = 0; n < N; n++) v[n] = __shfl_sync(0xffffffffu, s, n * (32 / N));
    return;
  }
  if (lane % (32 / N) == 0) x.put(lane / (32 / N), s);
  x.wait();
#pragma unroll
  for (int n = 0; n < N; n++) v[n] = x.sum(n);
  x.next();
}

// mean and rstd of a row of which a thread holds v, zero outside the row.  A
// layer norm's warps take the squares about their own mean, and those are joined
// about the row's (Chan, Golub, LeVeque), so that one exchange gives both and an
// offset costs no digits.
template <int MODE, int NV>
__device__ __forceinline__ float2 row_stats(const float (&v)[NV][8], const Place &at, int kind, float inv, float eps,
                                            Exchange &x) {
  if (kind == FP8_NORM_RMS) {
    float q[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
      for (int j = 0; j < 8; j++) q[0] = fmaf(v[i][j], v[i][j], q[0]);
    row_sums(q, x);
    return make_float2(0.0f, rsqrtf(fmaf(q[0], inv, eps)));
  }
  // columns of a warp: 256 a chunk
  auto count = [&](int w) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < NV; i++) n += max(0, min(256, at.cols - (i * at.T + w * 32) * 8));
    return n;
  };
  float s[1] = {0.0f}, q[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NV; i++)
#pragma unroll
    for (int j = 0; j < 8; j++) s[0] += v[i][j];
  const int own = count((int)threadIdx.x >> 5);
  const float total = warp_sums(s), mean_w = own ? total / (float)own : 0.0f;
#pragma unroll
  for (int i = 0; i < NV; i++)
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const float d = at.has<MODE>(i, j) ? v[i][j] - mean_w : 0.0f;
      q[0] = fmaf(d, d, q[0]);
    }
  const float sq = warp_sums(q);
  if (x.warps == 1) return make_float2(mean_w, rsqrtf(fmaf(sq, inv, eps)));
  if ((threadIdx.x & 31) == 0) {
    x.put(0, total);
    x.put(1, sq);
    x.put(2, mean_w);
  }
  x.wait();
  const float mean = x.sum(0) * inv;
  float m2 = 0.0f;
  for (int w = 0; w < x.warps; w++) {
    const float d = x.get(2, w) - mean;
    m2 += fmaf((float)count(w) * d, d, x.get(1, w));
  }
  x.next();
  return make_float2(mean, rsqrtf(fmaf(m2, inv, eps)));
}

__device__ __forceinline__ Exchange exchange(float (*slots)[8][kMostWarps]) {
  return {slots, (int)threadIdx.y, (int)(blockDim.x >> 5), 0};
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
};


// Scale bytes of rows behind the last one, up to a whole group of 128.
__device__ __forceinline__ void pad_scales(const Fwd &p, int blk, int kblocks, int l, int step) {
  for (int r = p.rows + l; r < (p.rows + 127) / 128 * 128; r += step) block::put_scale(p.xs, r, blk, kblocks, 0);
}

// The codes of a thread's chunk of a row's 1x128 blocks with their scales, and
// with the last row the padding of these.
template <int MODE>
__device__ __forceinline__ void put_codes(const Fwd &p, const Place &at, int v, int row, const float (&f)[8]) {
  const int lane = threadIdx.x & 31, kblocks = (p.cols + 127) / 128;
  uint8_t *q = p.xq + (size_t)row * p.ldxq;
  if constexpr (MODE == kStaged) {  // 16 lanes a block
    float a = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; j += 2) a = block::absmax2(a, f[j], f[j + 1]);
    uint32_t m = __float_as_uint(a);
#pragma unroll
    for (int b = 8; b > 0; b /= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, b));
    const int k = block::block_exponent(m, kMaxE4M3, p.margin), blk = at.col<MODE>(v, 0) >> 7, l = lane & 15;
    if (blk < kblocks) {
      if (l == 0) block::put_scale(p.xs, row, blk, kblocks, k);
      if (row == p.rows - 1) pad_scales(p, blk, kblocks, l, 16);
    }
    float2 s[4];
    block::spread_scale(pow2f(k), s);
    const uint2 o = m >= 0x7f800000u ? block::enc8_any<FP8_E4M3>(f, s) : block::enc8<FP8_E4M3>(f, s);
    if (at.has<MODE>(v, 0)) __stcs(reinterpret_cast<uint2 *>(q + at.col<MODE>(v, 0)), o);
  } else {  // a warp has two: elements 0 to 3 and 4 to 7 of its lanes
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const float a = block::absmax2(block::absmax2(0.0f, f[4 * h], f[4 * h + 1]), f[4 * h + 2], f[4 * h + 3]);
      const uint32_t m = warp_max_u32(__float_as_uint(a));
      const int k = block::block_exponent(m, kMaxE4M3, p.margin);
      const int blk = at.col<MODE>(v, 4 * h) >> 7;
      if (blk < kblocks) {
        if (lane == 0) block::put_scale(p.xs, row, blk, kblocks, k);
        if (row == p.rows - 1) pad_scales(p, blk, kblocks, lane, 32);
      }
      const float s = pow2f(k);
      const uint32_t o = enc4<FP8_E4M3>(f[4 * h] * s, f[4 * h + 1] * s, f[4 * h + 2] * s, f[4 * h + 3] * s);
#pragma unroll
      for (int j = 0; j < 4; j++)
        if (at.has<MODE>(v, 4 * h + j)) q[at.col<MODE>(v, 4 * h + j)] = (uint8_t)(o >> (8 * j));
    }
  }
}

// Shared memory of a CTA: the staged rows, then the parameters of each thread's
// columns as it needs them for every row.
struct FwdSmem {
  int stage, w, b, gw, gb, bytes;  // offsets; -1: absent.  gw, gb: the gate times the post norm's w and b
};
template <int DT, int RT>
__host__ __device__ inline FwdSmem fwd_smem(int chunks, bool h, bool w, bool b, bool gw, bool gb, int mode) {
  FwdSmem s;
  int at = mode == kStaged ? chunks * 16 * ((h ? kPieces<DT> : 0) + kPieces<RT>) : 0;
  auto take = [&](bool on) {
    const int o = on && mode == kStaged ? at : -1;
    at += o >= 0 ? chunks * 32 : 0;
    return o;
  };
  s.stage = 0;
  s.w = take(w), s.b = take(b), s.gw = take(gw), s.gb = take(gb);
  s.bytes = at;
  return s;
}

// POST: whether there is a post norm (kDirect goes by p.post).
template <int DT, int RT, bool POST, int NV, int MODE>
__global__ void __launch_bounds__(kCtaThreads<NV, MODE>, NV == 4 ? 1 : 4) k_norm_fwd(const Fwd p) {
  pdl_launch_dependents();
  pdl_wait();
  extern __shared__ __align__(16) uint8_t norm_smem[];
  __shared__ __align__(16) float slots[2][8][kMostWarps];
  Exchange ex = exchange(slots);
  const int threads = blockDim.x * blockDim.y, tid = threadIdx.y * blockDim.x + threadIdx.x;
  const Place at = {p.cols, (int)threadIdx.x, (int)blockDim.x};
  const bool post = MODE == kStaged ? POST : p.post != FP8_NORM_NONE;
  const bool scaled = p.g.p || (post && p.pw.p), shifted = post && p.pb.p;
  const FwdSmem lay = fwd_smem<DT, RT>(NV * threads, p.h, p.w.p, p.b.p, scaled, shifted, MODE);
  float *const w_s = reinterpret_cast<float *>(norm_smem + lay.w), *const b_s = reinterpret_cast<float *>(norm_smem + lay.b);
  float *const gw_s = reinterpret_cast<float *>(norm_smem + lay.gw), *const gb_s = reinterpret_cast<float *>(norm_smem + lay.gb);
  const Rows<RT, MODE> R = {static_cast<const uint8_t *>(p.r), p.ldr * (RT == FP8_DT_F32 ? 4 : 2), norm_smem, threads, tid};
  const Rows<DT, MODE> H = {static_cast<const uint8_t *>(p.h), p.ldh * (DT == FP8_DT_F32 ? 4 : 2),
                            norm_smem + NV * threads * 16 * kPieces<RT>, threads, tid};
  const unsigned stride = gridDim.x * blockDim.y;
  unsigned next = blockIdx.x * blockDim.y + threadIdx.y;
  auto fetch = [&](int v, unsigned row) {
    if (row >= (unsigned)p.rows) return;
    if (p.h) H.fetch(at, v, (int)row);
    R.fetch(at, v, (int)row);
  };
#pragma unroll
  for (int v = 0; v < NV; v++) fetch(v, next);
  asm volatile("cp.async.commit_group;" ::: "memory");
  if constexpr (MODE == kStaged) {
#pragma unroll
    for (int v = 0; v < NV; v++) {
      float f[8];
      if (p.w.p) load_params<MODE>(p.w, 0, at, v, 1.0f, f), put8(w_s, threads, tid, v, f);
      if (p.b.p) load_params<MODE>(p.b, 0, at, v, 0.0f, f), put8(b_s, threads, tid, v, f);
    }
  }
  // the gate's row times the post norm's w and b
  auto gate_params = [&](int v, int gate, float (&gw)[8], float (&gb)[8]) {
    load_params<MODE>(p.g, (size_t)gate * p.ldg, at, v, 1.0f, gw);
    if (shifted) {
      load_params<MODE>(p.pb, 0, at, v, 0.0f, gb);
#pragma unroll
      for (int j = 0; j < 8; j++) gb[j] *= gw[j];
    }
    if (post) {
      float f[8];
      load_params<MODE>(p.pw, 0, at, v, 1.0f, f);
#pragma unroll
      for (int j = 0; j < 8; j++) gw[j] *= f[j];
    }
  };
  const float inv = 1.0f / (float)p.cols;
  int gate = -1;
  for (; next < (unsigned)p.rows; next += stride) {
    const int row = (int)next;
    const int now = p.g.p ? row / p.gate_rows : 0;
    if (MODE == kStaged && (scaled || shifted) && now != gate) {  // (a thread's own part: nobody else waits for it)
      gate = now;
#pragma unroll
      for (int v = 0; v < NV; v++) {
        float gw[8], gb[8];
        gate_params(v, now, gw, gb);
        if (scaled) put8(gw_s, threads, tid, v, gw);
        if (shifted) put8(gb_s, threads, tid, v, gb);
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    float y[NV][8];
    float2 s1 = make_float2(0.0f, 1.0f), s2 = make_float2(0.0f, 1.0f);
    if (post) {
#pragma unroll
      for (int v = 0; v < NV; v++) {
        H.get(at, v, row, y[v]);
        mask<MODE>(at, v, y[v]);
      }
      s1 = row_stats<MODE, NV>(y, at, p.post, inv, p.eps, ex);
    }
#pragma unroll
    for (int v = 0; v < NV; v++) {
      float u[8], f[8];
      if (post) {
#pragma unroll
        for (int j = 0; j < 8; j++) u[j] = (y[v][j] - s1.x) * s1.y;
      } else if (p.h) {
        H.get(at, v, row, u);
      } else {
#pragma unroll
        for (int j = 0; j < 8; j++) u[j] = 0.0f;
      }
      float gb[8];
      if (MODE == kDirect) gate_params(v, now, f, gb);
      if (scaled) {
        if (MODE == kStaged) get8(gw_s, threads, tid, v, f);
#pragma unroll
        for (int j = 0; j < 8; j++) u[j] = __fmul_rn(u[j], f[j]);
      }
      if (shifted) {
        if (MODE == kStaged) get8(gb_s, threads, tid, v, gb);
#pragma unroll
        for (int j = 0; j < 8; j++) u[j] += gb[j];
      }
      R.get(at, v, row, f);
      fetch(v, next + stride);  // (what the chunk had has been read)
#pragma unroll
      for (int j = 0; j < 8; j++) y[v][j] = as_stored<RT>(__fadd_rn(__fmul_rn(p.alpha, f[j]), u[j]));
      mask<MODE>(at, v, y[v]);
      if (p.r_out) put_row<RT, MODE>(p.r_out, p.ldro, at, v, row, y[v]);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (p.pre != FP8_NORM_NONE) {
      s2 = row_stats<MODE, NV>(y, at, p.pre, inv, p.eps, ex);
      if (p.x || p.xq) {
#pragma unroll
        for (int v = 0; v < NV; v++) {
          float f[8];
#pragma unroll
          for (int j = 0; j < 8; j++) y[v][j] = (y[v][j] - s2.x) * s2.y;
          if (p.w.p) {
            if (MODE == kStaged) get8(w_s, threads, tid, v, f);
            else load_params<MODE>(p.w, 0, at, v, 1.0f, f);
#pragma unroll
            for (int j = 0; j < 8; j++) y[v][j] = __fmul_rn(y[v][j], f[j]);
          }
          if (p.b.p) {
            if (MODE == kStaged) get8(b_s, threads, tid, v, f);
            else load_params<MODE>(p.b, 0, at, v, 0.0f, f);
#pragma unroll
            for (int j = 0; j < 8; j++) y[v][j] = __fadd_rn(y[v][j], f[j]);
          }
          if (p.x) put_row<DT, MODE>(p.x, p.ldx, at, v, row, y[v]);
          if (p.xq) {
            mask<MODE>(at, v, y[v]);
            put_codes<MODE>(p, at, v, row, y[v]);
          }
        }
      }
    }
    if (p.stats && threadIdx.x == 0) reinterpret_cast<float4 *>(p.stats)[row] = make_float4(s1.x, s1.y, s2.x, s2.y);
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
      f[i][j] = row < p.rows && col + j < p.cols ? __fadd_rn(__fmul_rn((f[i][j] - s.z) * s.w, w[j]), b[j]) : 0.0f;
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
// The rows are dealt out in units, each within one gate row; a CTA takes
// neighbouring units.  Its sums over rows stay in registers: dw2 and db2 until
// it ends, A and C until its unit does.
//
// dh needs means of q = G g w1, and G needs means of dx w2: two exchanges, one
// waiting for the other.  But G is linear in its means: with H = dr' + rho2 dx w2,
//   q = gw H - gw rho2 (m0 + n2 m1)
//   mean(q)    = mean(gw H)    - rho2 (m0 mean(gw)    + m1 mean(gw n2))
//   mean(q n1) = mean(gw n1 H) - rho2 (m0 mean(gw n1) + m1 mean(gw n1 n2))
// so one pass over the row gives all of them in one exchange, and a second one
// (from shared memory) writes everything.
struct Plan {
  int chunks, threads, groups;         // NV; of a CTA: threads of a row, rows at a time
  int gate_rows, unit_rows, per_gate;  // rows of a gate row and of a unit, units per gate row
  long long units;
  int ctas;
};

constexpr int kSms = 148;

inline int padded(int cols) { return (cols + 7) / 8 * 8; }  // of a partial sum

inline Plan plan_of(int rows, int cols, int gate_rows) {
  Plan p = {};
  const int vecs = (cols + 7) / 8;
  p.chunks = vecs <= kThreads ? 1 : vecs <= 2 * kThreads ? 2 : 4;
  p.threads = (vecs + 32 * p.chunks - 1) / (32 * p.chunks) * 32;
  p.groups = p.threads < kThreads ? kThreads / p.threads : 1;
  p.gate_rows = gate_rows < rows ? gate_rows : rows;
  const int most = p.threads > kThreads ? kSms : 2 * kSms;
  p.unit_rows = rows / most + (rows % most != 0);
  if (p.unit_rows < p.groups) p.unit_rows = p.groups;
  if (rows == 0) return p;
  p.per_gate = p.gate_rows / p.unit_rows + (p.gate_rows % p.unit_rows != 0);
  p.units = ((long long)rows + p.gate_rows - 1) / p.gate_rows * p.per_gate;
  p.ctas = (int)(p.units < most ? p.units : most);
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
  float *ef, *ac;  // partial sums [CTA][2][padded cols] and [unit][2][padded cols], or null
  int gate_rows, unit_rows, per_gate;
  long long units;
};


struct BwdSmem {
  int w, gw, comb, bytes;
};
template <int DT, int RT>
__host__ __device__ inline BwdSmem bwd_smem(int chunks, bool h, bool dro, bool pre, bool scaled, bool groups, int mode) {
  BwdSmem s;
  int at = mode == kStaged ? chunks * 16 * ((h ? kPieces<DT> : 0) + (dro ? kPieces<RT> : 0) + (pre ? kPieces<DT> + kPieces<RT> : 0)) : 0;
  auto take = [&](bool on) {
    const int o = on && mode == kStaged ? at : -1;
    at += o >= 0 ? chunks * 32 : 0;
    return o;
  };
  s.w = take(pre), s.gw = take(scaled);
  s.comb = groups ? at : -1;
  at += groups ? kThreads * 32 : 0;
  s.bytes = at;
  return s;
}

// Adds up the groups of a CTA and writes one partial sum.
template <int MODE, int NV>
__device__ __forceinline__ void flush(float (&a)[8], float *comb, float *out, const Place &at, int v, int threads, int tid) {
  if (NV == 1 && blockDim.y > 1) {  // (rows of several chunks have a CTA to themselves)
    __syncthreads();
    put8(comb, threads, tid, 0, a);
    __syncthreads();
    if (threadIdx.y == 0) {
      for (int y = 1; y < (int)blockDim.y; y++) {
        float f[8];
        get8(comb, threads, y * blockDim.x + threadIdx.x, 0, f);
#pragma unroll
        for (int j = 0; j < 8; j++) a[j] += f[j];
      }
    }
  }
  if (threadIdx.y == 0) {
    if constexpr (MODE == kStaged) {
      if (at.has<MODE>(v, 0)) {
        float4 *o = reinterpret_cast<float4 *>(out + at.col<MODE>(v, 0));
        o[0] = make_float4(a[0], a[1], a[2], a[3]);
        o[1] = make_float4(a[4], a[5], a[6], a[7]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++)
        if (at.has<MODE>(v, j)) out[at.col<MODE>(v, j)] = a[j];
    }
  }
#pragma unroll
  for (int j = 0; j < 8; j++) a[j] = 0.0f;
}

// POST: whether there is a post norm; BIAS: whether sums of dx and of G are
// wanted (gradients of b, of post_b, and of a gate behind post_b).  kDirect goes
// by p.post, and takes the sums.
template <int DT, int RT, bool POST, bool BIAS, int NV, int MODE>
__global__ void __launch_bounds__(kCtaThreads<NV, MODE>, NV == 4 ? 1 : 2) k_norm_bwd(const Bwd p) {
  pdl_launch_dependents();
  pdl_wait();
  extern __shared__ __align__(16) uint8_t norm_smem[];
  __shared__ __align__(16) float slots[2][8][kMostWarps];
  Exchange ex = exchange(slots);
  const int threads = blockDim.x * blockDim.y, tid = threadIdx.y * blockDim.x + threadIdx.x;
  const Place at = {p.cols, (int)threadIdx.x, (int)blockDim.x};
  const bool post = MODE == kStaged ? POST : p.post != FP8_NORM_NONE;
  const bool pre = p.pre != FP8_NORM_NONE, scaled = p.h && (p.g.p || (post && p.pw.p));
  const BwdSmem lay = bwd_smem<DT, RT>(NV * threads, p.h, p.dro, pre, scaled, blockDim.y > 1, MODE);
  float *const w_s = reinterpret_cast<float *>(norm_smem + lay.w), *const gw_s = reinterpret_cast<float *>(norm_smem + lay.gw);
  float *const comb = reinterpret_cast<float *>(norm_smem + lay.comb);
  uint8_t *slot = norm_smem;
  auto take = [&](bool on, int pieces) {
    uint8_t *s = slot;
    slot += on ? NV * threads * 16 * pieces : 0;
    return s;
  };
  constexpr size_t de = DT == FP8_DT_F32 ? 4 : 2, re = RT == FP8_DT_F32 ? 4 : 2;
  const Rows<DT, MODE> DX = {static_cast<const uint8_t *>(p.dx), p.lddx * de, take(pre, kPieces<DT>), threads, tid};
  const Rows<RT, MODE> RO = {static_cast<const uint8_t *>(p.ro), p.ldro * re, take(pre, kPieces<RT>), threads, tid};
  const Rows<RT, MODE> DRO = {static_cast<const uint8_t *>(p.dro), p.lddro * re, take(p.dro, kPieces<RT>), threads, tid};
  const Rows<DT, MODE> H = {static_cast<const uint8_t *>(p.h), p.ldh * de, take(p.h, kPieces<DT>), threads, tid};
  auto fetch = [&](int v, int row) {
    if (pre) {
      DX.fetch(at, v, row);
      RO.fetch(at, v, row);
    }
    if (p.dro) DRO.fetch(at, v, row);
    if (p.h) H.fetch(at, v, row);
  };
  const float inv = 1.0f / (float)p.cols;
  const size_t ld_sum = (size_t)(p.cols + 7) / 8 * 8;
  const long long u0 = p.units * blockIdx.x / gridDim.x, u1 = p.units * (blockIdx.x + 1) / gridDim.x;
  float E[NV][8], F[NV][8], A[NV][8], C[NV][8];
#pragma unroll
  for (int v = 0; v < NV; v++)
#pragma unroll
    for (int j = 0; j < 8; j++) E[v][j] = F[v][j] = A[v][j] = C[v][j] = 0.0f;
  // the rows of unit u
  struct Span {
    long long first, last;
  };
  auto rows_of = [&](long long u) -> Span {
    const long long gate = u / p.per_gate, first = gate * p.gate_rows;
    const long long end = min(first + p.gate_rows, (long long)p.rows);
    const long long r0 = first + (u - gate * p.per_gate) * p.unit_rows;
    return {r0, min(r0 + p.unit_rows, end)};
  };
  float4 s_next = make_float4(0.0f, 1.0f, 0.0f, 1.0f);
  auto fetch_first = [&](long long u) {
    if (u >= u1) return;
    const Span s = rows_of(u);
    const long long row = s.first + threadIdx.y;
    if (row >= s.last) return;
#pragma unroll
    for (int v = 0; v < NV; v++) fetch(v, (int)row);
    if (p.stats) s_next = __ldg(reinterpret_cast<const float4 *>(p.stats) + row);
  };
  fetch_first(u0);
  asm volatile("cp.async.commit_group;" ::: "memory");
  if (MODE == kStaged && pre) {
#pragma unroll
    for (int v = 0; v < NV; v++) {
      float f[8];
      load_params<MODE>(p.w, 0, at, v, 1.0f, f);
      put8(w_s, threads, tid, v, f);
    }
  }
  auto weight = [&](int v, float (&f)[8]) {
    if (MODE == kStaged) get8(w_s, threads, tid, v, f);
    else load_params<MODE>(p.w, 0, at, v, 1.0f, f);
  };
  // the gate's row times the post norm's w
  auto gate_params = [&](int v, int gate, float (&g)[8]) {
    load_params<MODE>(p.g, (size_t)gate * p.ldg, at, v, 1.0f, g);
    if (post) {
      float f[8];
      load_params<MODE>(p.pw, 0, at, v, 1.0f, f);
#pragma unroll
      for (int j = 0; j < 8; j++) g[j] *= f[j];
    }
  };
  int gate_now = -1;
  for (long long u = u0; u < u1; u++) {
    const int gate = (int)(u / p.per_gate);
    const Span span = rows_of(u);
    if (MODE == kStaged && scaled && gate != gate_now) {
      gate_now = gate;
#pragma unroll
      for (int v = 0; v < NV; v++) {
        float g[8];
        gate_params(v, gate, g);
        put8(gw_s, threads, tid, v, g);
      }
    }
    auto gate_weight = [&](int v, float (&f)[8]) {
      if (MODE == kStaged) get8(gw_s, threads, tid, v, f);
      else gate_params(v, gate, f);
    };
    for (long long r = span.first + threadIdx.y; r < span.last; r += blockDim.y) {
      const int row = (int)r;
      const float4 s = s_next;
      const bool more = r + blockDim.y < span.last;
      if (more && p.stats) s_next = __ldg(reinterpret_cast<const float4 *>(p.stats) + row + blockDim.y);
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      float m0 = 0.0f, m1 = 0.0f, t0 = 0.0f, t1 = 0.0f;
      if (pre || post) {
        float k[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll(NV == 4 ? 1 : NV)
        for (int v = 0; v < NV; v++) {
          float t[8], n2[8];
          if (pre) {
            float w[8];
            DX.get(at, v, row, t);
            RO.get(at, v, row, n2);
            weight(v, w);
            mask<MODE>(at, v, t);
            mask<MODE>(at, v, n2);
#pragma unroll
            for (int j = 0; j < 8; j++) {
              n2[j] = (n2[j] - s.z) * s.w;
              t[j] *= w[j];
              k[0] = fmaf(t[j], n2[j], k[0]);
              k[1] += t[j];
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; j++) t[j] = n2[j] = 0.0f;
          }
          if (post) {
            float q[8], n1[8], h[8];
            if (p.dro) {
              DRO.get(at, v, row, h);
            } else {
#pragma unroll
              for (int j = 0; j < 8; j++) h[j] = 0.0f;
            }
            H.get(at, v, row, n1);
            if (scaled) {
              gate_weight(v, q);
            } else {
#pragma unroll
              for (int j = 0; j < 8; j++) q[j] = 1.0f;
            }
            mask<MODE>(at, v, q);
            mask<MODE>(at, v, h);
            mask<MODE>(at, v, n1);
#pragma unroll
            for (int j = 0; j < 8; j++) {
              n1[j] = (n1[j] - s.x) * s.y;
              const float qh = q[j] * fmaf(s.w, t[j], h[j]), qn = q[j] * n1[j];
              k[2] = fmaf(qh, n1[j], k[2]);
              k[3] = fmaf(qn, n2[j], k[3]);
              k[4] += qh;
              k[5] = fmaf(q[j], n2[j], k[5]);
              k[6] += qn;
              k[7] += q[j];
            }
          }
        }
        if (post) {
          if (p.pre == FP8_NORM_LAYER || p.post == FP8_NORM_LAYER) {
            row_sums(k, ex);
          } else {
            float few[4] = {k[0], k[1], k[2], k[3]};
            row_sums(few, ex);
            k[0] = few[0], k[2] = few[2], k[3] = few[3];
          }
        } else {
          float few[2] = {k[0], k[1]};
          row_sums(few, ex);
          k[0] = few[0], k[1] = few[1];
        }
        m1 = k[0] * inv;
        if (p.pre == FP8_NORM_LAYER) m0 = k[1] * inv;
        if (post) {
          t1 = (k[2] - s.w * fmaf(m0, k[6], m1 * k[3])) * inv;
          if (p.post == FP8_NORM_LAYER) t0 = (k[4] - s.w * fmaf(m0, k[7], m1 * k[5])) * inv;
        }
      }
#pragma unroll
      for (int v = 0; v < NV; v++) {
        float G[8], t[8], n[8];
        if (p.dro) {
          DRO.get(at, v, row, G);
        } else {
#pragma unroll
          for (int j = 0; j < 8; j++) G[j] = 0.0f;
        }
        if (pre) {
          float w[8];
          DX.get(at, v, row, t);
          RO.get(at, v, row, n);
          weight(v, w);
#pragma unroll
          for (int j = 0; j < 8; j++) {
            n[j] = (n[j] - s.z) * s.w;
            E[v][j] = fmaf(t[j], n[j], E[v][j]);
            if (BIAS) F[v][j] += t[j];
            G[j] = fmaf(s.w, fmaf(t[j], w[j], -m0) - n[j] * m1, G[j]);
          }
        }
        if (p.h) H.get(at, v, row, n);
        if (MODE == kStaged && more) fetch(v, row + (int)blockDim.y);  // (what the chunk had has been read)
        if (p.dr) {
#pragma unroll
          for (int j = 0; j < 8; j++) t[j] = p.alpha * G[j];
          put_row<RT, MODE>(p.dr, p.lddr, at, v, row, t);
        }
        if (p.h) {
          if (scaled) {
            gate_weight(v, t);
#pragma unroll
            for (int j = 0; j < 8; j++) t[j] *= G[j];
          } else {
#pragma unroll
            for (int j = 0; j < 8; j++) t[j] = G[j];
          }
          if (post) {
#pragma unroll
            for (int j = 0; j < 8; j++) {
              n[j] = (n[j] - s.x) * s.y;
              t[j] = s.y * (t[j] - t0 - n[j] * t1);
            }
          }
          if (p.dh) put_row<DT, MODE>(p.dh, p.lddh, at, v, row, t);
          if (p.ac) {
#pragma unroll
            for (int j = 0; j < 8; j++) {
              A[v][j] = fmaf(G[j], n[j], A[v][j]);
              if (BIAS) C[v][j] += G[j];
            }
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    fetch_first(u + 1);
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (p.ac) {
#pragma unroll
      for (int v = 0; v < NV; v++) {
        flush<MODE, NV>(A[v], comb, p.ac + (size_t)(2 * u) * ld_sum, at, v, threads, tid);
        if (BIAS) flush<MODE, NV>(C[v], comb, p.ac + (size_t)(2 * u + 1) * ld_sum, at, v, threads, tid);
      }
    }
  }
  if (p.ef) {
#pragma unroll
    for (int v = 0; v < NV; v++) {
      flush<MODE, NV>(E[v], comb, p.ef + (size_t)(2 * blockIdx.x) * ld_sum, at, v, threads, tid);
      if (BIAS) flush<MODE, NV>(F[v], comb, p.ef + (size_t)(2 * blockIdx.x + 1) * ld_sum, at, v, threads, tid);
    }
  }
}

struct Params {
  const float *ef, *ac;
  int cols, ctas, gates, per_gate;
  bool post, bias;
  Vec pw, pb, g;
  size_t ldg;
  Vec dw, db, dpw, dpb, dg;  // outputs
  size_t lddg;
  int col_blocks;
};

constexpr int kParamLanes = 32;

// The parameters' gradients from the partial sums: a CTA takes 32 columns of
// one job (the pre norm's, the post norm's, or one gate row's), its lanes
// (threadIdx.y) every 32nd partial sum.
__global__ void __launch_bounds__(32 * kParamLanes) k_norm_params(const Params p) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float sh[2][kParamLanes][33];
  const int job = (int)(blockIdx.x / p.col_blocks) - 2, c = (int)(blockIdx.x % p.col_blocks) * 32 + threadIdx.x;
  const int y = threadIdx.y;
  const size_t ld = (size_t)(p.cols + 7) / 8 * 8;
  const bool in = c < p.cols;
  float a = 0.0f, b = 0.0f;
  if (job == -2) {
    if (!p.dw.p && !p.db.p) return;
    if (in) {
#pragma unroll 4
      for (int i = y; i < p.ctas; i += kParamLanes) {
        a += p.ef[2 * i * ld + c];
        if (p.bias) b += p.ef[(2 * i + 1) * ld + c];
      }
    }
  } else if (job == -1) {
    if (!p.dpw.p && !p.dpb.p) return;
    const long long units = (long long)p.gates * p.per_gate;
    if (in) {
#pragma unroll 4
      for (long long i = y; i < units; i += kParamLanes) {
        const float g = param_at(p.g, (size_t)(i / p.per_gate) * p.ldg + c, 1.0f);
        a = fmaf(g, p.ac[2 * i * ld + c], a);
        if (p.bias) b = fmaf(g, p.ac[(2 * i + 1) * ld + c], b);
      }
    }
  } else {
    if (!p.dg.p) return;
    if (in) {
#pragma unroll 4
      for (int i = y; i < p.per_gate; i += kParamLanes) {
        const size_t u = (size_t)job * p.per_gate + i;
        a += p.ac[2 * u * ld + c];
        if (p.bias) b += p.ac[(2 * u + 1) * ld + c];
      }
    }
  }
  sh[0][y][threadIdx.x] = a;
  sh[1][y][threadIdx.x] = b;
  __syncthreads();
  if (y > 1) return;
  a = 0.0f;
#pragma unroll
  for (int i = 0; i < kParamLanes; i++) a += sh[y][i][threadIdx.x];  // in their order
  // the first lane has the sums with the normed value, the second the plain ones
  if (job < 0) {
    if (in) store_param(job == -2 ? (y == 0 ? p.dw : p.db) : (y == 0 ? p.dpw : p.dpb), c, a);
    return;
  }
  if (y == 1) {
    if (!p.post || !p.pb.p) return;
    // dg = w1 A + b1 C: C by way of shared memory, behind what the first lane reads
    sh[1][0][threadIdx.x] = a;
  }
  asm volatile("bar.sync 1, %0;" ::"r"(p.post && p.pb.p ? 64 : 32) : "memory");
  if (y == 0 && in) {
    if (p.post) a *= param_at(p.pw, c, 1.0f);
    if (p.post && p.pb.p) a = fmaf(param_at(p.pb, c, 0.0f), sh[1][0][threadIdx.x], a);
    store_param(p.dg, (size_t)job * p.lddg + c, a);
  }
}

}  // namespace norm
}  // namespace fp8lib
