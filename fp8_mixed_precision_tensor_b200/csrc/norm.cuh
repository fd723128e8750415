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

// A row belongs to a group of threads (a multiple of 32) of a CTA; a thread holds
// 8, 16 or 32 of its columns, as NV chunks of CW neighbouring ones: 8,
// or 4 where the residual is binary32, so that a warp reads and writes whole
// sectors of every matrix (chunks of 8 binary32 numbers in 16-byte pieces cost
// each sector twice: 46 instead of 40 us for 4096 x 4096 forward).  A CTA takes
// as many narrow rows at a time as it has threads for, and row after row while
// it lives.
constexpr int kThreads = 256;      // of a CTA, but for the widest rows
constexpr int kMostThreads = 512;
constexpr int kMostWarps = kMostThreads / 32;
// The widest staged rows: 384 threads, 168 registers each.  The parameters stand
// beside the staged row as 4 bytes a column each, and where both do not fit the
// row is read directly.  Of 16 bits: forward with both norms' biases from 11265
// columns on (10241 with a binary32 residual), backward with a binary32 residual
// and a gate or post norm from 11265; of binary32: forward with both biases from
// 9217, with one and a gate or post norm from 11265, backward from 11265 (9217
// with a gate or post norm).
constexpr int kStagedCols = 12288;
// How wide a row is: CK = 1 and 2, so many groups of eight columns a thread in
// CTAs of 256; 3, two of them in 512 threads (8192 columns; as four in 256
// threads, 8 warps an SM, 2048 rows took 51 and 150 us for 47 and 91); 4, four of
// them in up to 384 (or 512, kDirect).
__host__ __device__ constexpr int eights(int CK) { return CK == 3 ? 2 : CK; }
template <int CK, int MODE>
constexpr int kCtaThreads = CK < 3 ? kThreads : CK == 3 ? kMostThreads : MODE == 0 ? kStagedCols / 32 : kMostThreads;
// Whether the parameters are in shared memory (unaligned wide rows read them each time).
__host__ __device__ constexpr bool held(int CK, int mode) { return mode == 0 || CK == 1; }
template <int RT>
constexpr int kWidth = RT == FP8_DT_F32 ? 4 : 8;  // CW

// How rows are read and written.
//   kStaged  the next row's chunks are copied into the thread's own part of
//            shared memory while it works on the present one (no barriers:
//            nobody else reads them)
//   kDirect  rows that start anywhere: the lanes of a warp take neighbouring
//            columns, and element by element from memory, twice where two
//            passes need them
//            (and rows too wide to be staged).  No row is in flight while another
//            is worked on, and above 2048 columns a thread takes 32 of them, also
//            those behind the row's end: 4096 rows of 2051, 4099 and 8195
//            bfloat16, an RMS norm, 122, 212 and 372 us forward, 240, 486 and 749
//            backward; of 16384 447 and 895; of 12288 backward with a binary32
//            residual, both norms and a gate 1.7 ms, spilling 1.1 KB a thread.
enum { kStaged = 0, kDirect = 1 };

// The chunk v of a thread, and whether it lies in the row (kStaged: all of it).
// width: threads from one chunk's columns to the next one's; lanes: from one
// chunk's place in shared memory to the next one's (a constant, but for the
// widest rows: a CTA has 256 threads, in one row or several).
template <int CK, int CW, int MODE>
struct Place {
  int cols, t;
  __device__ __forceinline__ int width() const { return CK == 2 || CK == 3 ? kCtaThreads<CK, MODE> : (int)blockDim.x; }
  __device__ __forceinline__ int lanes() const { return CK == 4 ? (int)blockDim.x : kCtaThreads<CK, MODE>; }
  __device__ __forceinline__ int col(int v, int j) const {
    return MODE == kStaged ? (v * width() + t) * CW + j : (v * width() + (t & ~31)) * CW + 32 * j + (t & 31);
  }
  __device__ __forceinline__ bool has(int v, int j) const { return col(v, MODE == kStaged ? 0 : j) < cols; }
  // Whether the thread works on its chunk v.  Staged chunks outside the row are
  // skipped whole (by a branch that only a row's last warp splits at).
  __device__ __forceinline__ bool mine(int v) const { return MODE == kDirect || has(v, 0); }
};

// A chunk's elements as they are stored, 8 or 16 bytes.
template <int DT, int CW>
struct __align__(CW == 8 || DT == FP8_DT_F32 ? 16 : 8) Raw {
  static constexpr int kWords = DT == FP8_DT_F32 ? CW : CW / 2;
  static_assert(kWords <= 4, "one piece");
  uint32_t w[kWords];
};
template <int DT, int CW>
__device__ __forceinline__ void unpack(const Raw<DT, CW> &r, float (&f)[CW]) {
#pragma unroll
  for (int i = 0; i < Raw<DT, CW>::kWords; i++) {
    if constexpr (DT == FP8_DT_F32) {
      f[i] = __uint_as_float(r.w[i]);
    } else if constexpr (DT == FP8_DT_BF16) {
      f[2 * i] = __uint_as_float(r.w[i] << 16);
      f[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
    } else {
      const float2 h = h2f2(r.w[i]);
      f[2 * i] = h.x;
      f[2 * i + 1] = h.y;
    }
  }
}
template <int DT, int CW>
__device__ __forceinline__ Raw<DT, CW> pack(const float (&f)[CW]) {
  Raw<DT, CW> r;
#pragma unroll
  for (int i = 0; i < Raw<DT, CW>::kWords; i++) {
    if constexpr (DT == FP8_DT_F32) {
      r.w[i] = __float_as_uint(f[i]);
    } else if constexpr (DT == FP8_DT_BF16) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      r.w[i] = *reinterpret_cast<const uint32_t *>(&b);
    } else {
      r.w[i] = f16x2(f[2 * i], f[2 * i + 1]);
    }
  }
  return r;
}

struct Vec {
  const void *p;
  int dt;
};

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


// A chunk's parameters; `fill` where there are none.
template <int DT, int CW>
__device__ __forceinline__ bool load_vector(const void *p, size_t i, float (&f)[CW]) {
  using R = Raw<DT == FP8_DT_F32 ? FP8_DT_F32 : DT, DT == FP8_DT_F32 ? 4 : CW>;
  const uint8_t *q = reinterpret_cast<const uint8_t *>(p) + i * (DT == FP8_DT_F32 ? 4 : 2);
  if (reinterpret_cast<uintptr_t>(q) % alignof(R)) return false;
  if constexpr (DT == FP8_DT_F32) {
#pragma unroll
    for (int h = 0; h < CW / 4; h++) {
      const float4 v = __ldg(reinterpret_cast<const float4 *>(q) + h);
      f[4 * h] = v.x, f[4 * h + 1] = v.y, f[4 * h + 2] = v.z, f[4 * h + 3] = v.w;
    }
  } else {
    R r;
    if constexpr (CW == 8) *reinterpret_cast<uint4 *>(r.w) = __ldg(reinterpret_cast<const uint4 *>(q));
    else *reinterpret_cast<uint2 *>(r.w) = __ldg(reinterpret_cast<const uint2 *>(q));
    unpack<DT, CW>(r, f);
  }
  return true;
}
template <int CK, int CW, int MODE>
__device__ __forceinline__ void load_params(Vec v, size_t off, const Place<CK, CW, MODE> &at, int chunk, float fill,
                                            float (&f)[CW]) {
#pragma unroll
  for (int j = 0; j < CW; j++) f[j] = fill;
  if (!v.p) return;
  if constexpr (MODE == kStaged) {
    if (!at.has(chunk, 0)) return;
    const size_t i = off + at.col(chunk, 0);
    if (v.dt == FP8_DT_F32 ? load_vector<FP8_DT_F32, CW>(v.p, i, f)
                           : v.dt == FP8_DT_BF16 ? load_vector<FP8_DT_BF16, CW>(v.p, i, f) : load_vector<FP8_DT_F16, CW>(v.p, i, f))
      return;
  }
#pragma unroll
  for (int j = 0; j < CW; j++)
    if (at.has(chunk, j)) f[j] = param_at(v, off + at.col(chunk, j), fill);
}

// Eight parameters at column c.
__device__ __forceinline__ void load_eight(Vec v, int c, int cols, float fill, float (&f)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j++) f[j] = fill;
  if (!v.p || c >= cols) return;
  if (c + 8 <= cols && (v.dt == FP8_DT_F32 ? load_vector<FP8_DT_F32, 8>(v.p, c, f)
                                           : v.dt == FP8_DT_BF16 ? load_vector<FP8_DT_BF16, 8>(v.p, c, f)
                                                                 : load_vector<FP8_DT_F16, 8>(v.p, c, f)))
    return;
#pragma unroll
  for (int j = 0; j < 8; j++)
    if (c + j < cols) f[j] = param_at(v, c + j, fill);
}

template <int DT>
constexpr int kBytes = DT == FP8_DT_F32 ? 4 : 2;  // of an element

// Keeps a value in a register that the compiler would else fetch or work out
// again for every row.
template <typename V>
__device__ __forceinline__ void keep(V &v) {
  if constexpr (sizeof(V) == 8) asm volatile("" : "+l"(v));
  else asm volatile("" : "+r"(v));
}

// A matrix whose rows a thread reads, one after another.  kStaged: `p` is the
// thread's place in the row that is fetched next, and shared memory has
// [chunk][thread] of a chunk's bytes, `slot` the thread's place in the first;
// kDirect: the present row.
template <int DT, int CK, int CW, int MODE>
struct In {
  static constexpr int kChunk = sizeof(Raw<DT, CW>);
  const uint8_t *base;
  size_t ld;  // bytes
  uint8_t *slot;
  const uint8_t *p;
  long long step;

  __device__ __forceinline__ In(const void *m, size_t ld_elems, uint8_t *part, unsigned rows_apart)
      : base(static_cast<const uint8_t *>(m)), ld(ld_elems * kBytes<DT>),
        slot(part + (threadIdx.y * blockDim.x + threadIdx.x) * kChunk), p(nullptr), step((long long)ld * rows_apart) {
    keep(step);
  }
  __device__ __forceinline__ void seek(const Place<CK, CW, MODE> &at, long long row) {
    p = base + row * ld + (MODE == kStaged ? at.t * kChunk : 0);
  }
  __device__ __forceinline__ void advance() { p += step; }
  __device__ __forceinline__ void fetch(const Place<CK, CW, MODE> &at, int v) const {
    if constexpr (MODE == kStaged) {
      const uint32_t to = smem_u32(slot + v * at.lanes() * kChunk);
      const uint8_t *src = p + v * at.width() * kChunk;
      if constexpr (kChunk == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(src) : "memory");
      else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(src) : "memory");
    }
  }
  __device__ __forceinline__ void get(const Place<CK, CW, MODE> &at, int v, float (&f)[CW]) const {
    if constexpr (MODE == kStaged) {
      unpack<DT, CW>(*reinterpret_cast<const Raw<DT, CW> *>(slot + v * at.lanes() * kChunk), f);
    } else {
#pragma unroll
      for (int j = 0; j < CW; j++) {
        const int c = min(at.col(v, j), at.cols - 1);
        if constexpr (DT == FP8_DT_F32) f[j] = reinterpret_cast<const float *>(p)[c];
        else if constexpr (DT == FP8_DT_BF16) f[j] = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[c]);
        else f[j] = __half2float(reinterpret_cast<const __half *>(p)[c]);
      }
    }
  }
};

// A matrix whose rows a thread writes; put() leaves in f what was stored.
template <int DT, int CK, int CW, int MODE>
struct Out {
  static constexpr int kChunk = sizeof(Raw<DT, CW>);
  uint8_t *base;
  size_t ld;
  uint8_t *p;
  long long step;

  __device__ __forceinline__ Out(void *m, size_t ld_elems, unsigned rows_apart)
      : base(static_cast<uint8_t *>(m)), ld(ld_elems * kBytes<DT>), p(nullptr), step((long long)ld * rows_apart) {
    keep(step);
  }
  __device__ __forceinline__ void seek(const Place<CK, CW, MODE> &at, long long row) {
    p = base + row * ld + (MODE == kStaged ? at.t * kChunk : 0);
  }
  __device__ __forceinline__ void advance() { p += step; }
  __device__ __forceinline__ void put(const Place<CK, CW, MODE> &at, int v, float (&f)[CW], bool store = true) const {
    const Raw<DT, CW> r = pack<DT, CW>(f);
    if constexpr (DT != FP8_DT_F32) unpack<DT, CW>(r, f);
    if (!store) return;
    if constexpr (MODE == kStaged) {
      uint8_t *q = p + v * at.width() * kChunk;
      if constexpr (kChunk == 16) __stcs(reinterpret_cast<uint4 *>(q), *reinterpret_cast<const uint4 *>(r.w));
      else __stcs(reinterpret_cast<uint2 *>(q), *reinterpret_cast<const uint2 *>(r.w));
    } else {
#pragma unroll
      for (int j = 0; j < CW; j++)
        if (at.has(v, j)) {
          const int c = at.col(v, j);
          if constexpr (DT == FP8_DT_F32) reinterpret_cast<uint32_t *>(p)[c] = r.w[j];
          else reinterpret_cast<uint16_t *>(p)[c] = (uint16_t)(r.w[j >> 1] >> (16 * (j & 1)));
        }
    }
  }
};

template <int CW>
__device__ __forceinline__ void zero(float (&f)[CW]) {
#pragma unroll
  for (int j = 0; j < CW; j++) f[j] = 0.0f;
}
// Zero outside the row (kDirect).
template <int CK, int CW, int MODE>
__device__ __forceinline__ void mask(const Place<CK, CW, MODE> &at, int v, float (&f)[CW]) {
  if constexpr (MODE == kDirect) {
#pragma unroll
    for (int j = 0; j < CW; j++) f[j] = at.has(v, j) ? f[j] : 0.0f;
  }
}

// A chunk at a time on the packed binary32 instructions.
template <int CW>
__device__ __forceinline__ float2 pair(const float (&a)[CW], int j) {
  return make_float2(a[j], a[j + 1]);
}
template <int CW, typename F>
__device__ __forceinline__ void pairs(float (&o)[CW], F f) {
#pragma unroll
  for (int j = 0; j < CW; j += 2) {
    const float2 r = f(j);
    o[j] = r.x;
    o[j + 1] = r.y;
  }
}
template <int CW>
__device__ __forceinline__ void mul(float (&o)[CW], const float (&a)[CW], const float (&b)[CW]) {
  pairs(o, [&](int j) { return __fmul2_rn(pair(a, j), pair(b, j)); });
}
template <int CW>
__device__ __forceinline__ void mul(float (&o)[CW], const float (&a)[CW], float s) {
  pairs(o, [&](int j) { return __fmul2_rn(pair(a, j), both(s)); });
}
// o = s a + b with the product rounded: on single numbers, since packed products
// and sums are made one on the way, whatever rounding they ask for.
template <int CW>
__device__ __forceinline__ void scale_add(float (&o)[CW], float s, const float (&a)[CW], const float (&b)[CW]) {
#pragma unroll
  for (int j = 0; j < CW; j++) o[j] = __fadd_rn(__fmul_rn(s, a[j]), b[j]);
}
template <int CW>
__device__ __forceinline__ void add(float (&o)[CW], const float (&a)[CW], const float (&b)[CW]) {
  pairs(o, [&](int j) { return __fadd2_rn(pair(a, j), pair(b, j)); });
}
template <int CW>
__device__ __forceinline__ void add(float (&o)[CW], const float (&a)[CW], float s) {
  pairs(o, [&](int j) { return __fadd2_rn(pair(a, j), both(s)); });
}
// o = a b + c
template <int CW>
__device__ __forceinline__ void fma8(float (&o)[CW], const float (&a)[CW], const float (&b)[CW], const float (&c)[CW]) {
  pairs(o, [&](int j) { return __ffma2_rn(pair(a, j), pair(b, j), pair(c, j)); });
}
template <int CW>
__device__ __forceinline__ void fma8(float (&o)[CW], const float (&a)[CW], float s, const float (&c)[CW]) {
  pairs(o, [&](int j) { return __ffma2_rn(pair(a, j), both(s), pair(c, j)); });
}
template <int CW>
__device__ __forceinline__ void fma8(float (&o)[CW], const float (&a)[CW], const float (&b)[CW], float s) {
  pairs(o, [&](int j) { return __ffma2_rn(pair(a, j), pair(b, j), both(s)); });
}
// (v - mean) rstd: the difference first, so that a large mean costs no digits of it
template <int CW>
__device__ __forceinline__ void normed(float (&o)[CW], const float (&a)[CW], float mean, float rstd) {
  add(o, a, -mean);
  mul(o, o, rstd);
}
// s += sum of a b, in two halves
template <int CW>
__device__ __forceinline__ void dot(float2 &s, const float (&a)[CW], const float (&b)[CW]) {
#pragma unroll
  for (int j = 0; j < CW; j += 2) s = __ffma2_rn(pair(a, j), pair(b, j), s);
}
template <int CW>
__device__ __forceinline__ void plus(float2 &s, const float (&a)[CW]) {
#pragma unroll
  for (int j = 0; j < CW; j += 2) s = __fadd2_rn(s, pair(a, j));
}

// A chunk of floats of a thread in shared memory, its own: [16 bytes of the
// chunk][thread] for each chunk, s the thread's place in the first.
template <int CW>
__device__ __forceinline__ void put_own(uint8_t *s, int v, int width, const float (&f)[CW]) {
  float4 *p = reinterpret_cast<float4 *>(s) + v * (CW / 4) * width;
#pragma unroll
  for (int h = 0; h < CW / 4; h++) p[h * width] = make_float4(f[4 * h], f[4 * h + 1], f[4 * h + 2], f[4 * h + 3]);
}
template <int CW>
__device__ __forceinline__ void get_own(const uint8_t *s, int v, int width, float (&f)[CW]) {
  const float4 *p = reinterpret_cast<const float4 *>(s) + v * (CW / 4) * width;
#pragma unroll
  for (int h = 0; h < CW / 4; h++) {
    const float4 a = p[h * width];
    f[4 * h] = a.x, f[4 * h + 1] = a.y, f[4 * h + 2] = a.z, f[4 * h + 3] = a.w;
  }
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
    if (warps == 8) {  // (most rows: 256 threads)
      const float4 *q = reinterpret_cast<const float4 *>(slots[buf][n]);
      const float4 a = q[0], b = q[1];
      const float2 s = __fadd2_rn(__fadd2_rn(make_float2(a.x, a.y), make_float2(a.z, a.w)),
                                  __fadd2_rn(make_float2(b.x, b.y), make_float2(b.z, b.w)));
      return s.x + s.y;
    }
    float s = 0.0f;
    if ((warps & 3) == 0) {
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
template <int CK, int CW, int MODE, int NV>
__device__ __forceinline__ float2 row_stats(const float (&v)[NV][CW], const Place<CK, CW, MODE> &at, int kind, float inv, float eps,
                                            Exchange &x) {
  float2 s = both(0.0f);
  if (kind == FP8_NORM_RMS) {
#pragma unroll
    for (int i = 0; i < NV; i++) dot(s, v[i], v[i]);
    float q[1] = {s.x + s.y};
    row_sums(q, x);
    return make_float2(0.0f, rsqrtf(fmaf(q[0], inv, eps)));
  }
  // columns of a warp: 32 chunks each time
  auto count = [&](int w) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < NV; i++) n += max(0, min(32 * CW, at.cols - (i * at.width() + w * 32) * CW));
    return n;
  };
#pragma unroll
  for (int i = 0; i < NV; i++) plus(s, v[i]);
  float one[1] = {s.x + s.y};
  const int own = count((int)threadIdx.x >> 5);
  const float total = warp_sums(one), mean_w = own ? total / (float)own : 0.0f;
  s = both(0.0f);
#pragma unroll
  for (int i = 0; i < NV; i++) {
    if (at.mine(i)) {
      float d[CW];
      add(d, v[i], -mean_w);
      mask(at, i, d);
      dot(s, d, d);
    }
  }
  one[0] = s.x + s.y;
  const float sq = warp_sums(one);
  if (x.warps == 1) return make_float2(mean_w, rsqrtf(fmaf(sq, inv, eps)));
  if ((threadIdx.x & 31) == 0) {
    x.put(0, total);
    x.put(1, sq);
    x.put(2, mean_w);
  }
  x.wait();
  const float mean = x.sum(0) * inv;
  // lane w joins warp w
  const int lane = threadIdx.x & 31;
  float m2 = 0.0f;
  if (lane < x.warps) {
    const float d = x.get(2, lane) - mean;
    m2 = fmaf((float)count(lane) * d, d, x.get(1, lane));
  }
#pragma unroll
  for (int b = kMostWarps / 2; b > 0; b /= 2) m2 += __shfl_xor_sync(0xffffffffu, m2, b);
  m2 = __shfl_sync(0xffffffffu, m2, 0);
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
template <int CK, int CW, int MODE>
__device__ __forceinline__ void put_codes(const Fwd &p, const Place<CK, CW, MODE> &at, int v, int row, const float (&f)[CW]) {
  const int lane = threadIdx.x & 31, kblocks = (p.cols + 127) / 128;
  uint8_t *q = p.xq + (size_t)row * p.ldxq;
  // lanes l, l + 1 ... of `step` hold a block blk with this amax
  auto scale = [&](uint32_t m, int blk, int l, int step) {
    const int k = block::block_exponent(m, kMaxE4M3, p.margin);
    if (blk < kblocks) {
      if (l == 0) block::put_scale(p.xs, row, blk, kblocks, k);
      if (row == p.rows - 1) pad_scales(p, blk, kblocks, l, step);
    }
    return pow2f(k);
  };
  if constexpr (MODE == kStaged && CW == 8) {  // 16 lanes a block
    float a = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; j += 2) a = block::absmax2(a, f[j], f[j + 1]);
    uint32_t m = __float_as_uint(a);
#pragma unroll
    for (int b = 8; b > 0; b /= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, b));
    float2 s[4];
    block::spread_scale(scale(m, at.col(v, 0) >> 7, lane & 15, 16), s);
    const uint2 o = m >= 0x7f800000u ? block::enc8_any<FP8_E4M3>(f, s) : block::enc8<FP8_E4M3>(f, s);
    if (at.has(v, 0)) __stcs(reinterpret_cast<uint2 *>(q + at.col(v, 0)), o);
  } else {  // a warp a block: four elements of its lanes
#pragma unroll
    for (int h = 0; h < CW; h += 4) {
      const float a = block::absmax2(block::absmax2(0.0f, f[h], f[h + 1]), f[h + 2], f[h + 3]);
      const uint32_t m = warp_max_u32(__float_as_uint(a));
      const float s = scale(m, at.col(v, h) >> 7, lane, 32);
      const uint32_t o = enc4<FP8_E4M3>(f[h] * s, f[h + 1] * s, f[h + 2] * s, f[h + 3] * s);
      if constexpr (MODE == kStaged) {
        if (at.has(v, 0)) __stcs(reinterpret_cast<uint32_t *>(q + at.col(v, 0)), o);
      } else {
#pragma unroll
        for (int j = 0; j < 4; j++)
          if (at.has(v, h + j)) q[at.col(v, h + j)] = (uint8_t)(o >> (8 * j));
      }
    }
  }
}

// Shared memory of a CTA: the staged rows, then the parameters of each thread's
// columns as it needs them for every row.
struct FwdSmem {
  int stage, w, b, gw, gb, bytes;  // offsets; -1: absent.  gw, gb: the gate times the post norm's w and b
};
// of `columns` columns
template <int DT, int RT>
__host__ __device__ inline FwdSmem fwd_smem(int columns, bool h, bool w, bool b, bool gw, bool gb, int mode, bool held) {
  FwdSmem s;
  int at = mode == kStaged ? columns * ((h ? kBytes<DT> : 0) + kBytes<RT>) : 0;
  auto take = [&](bool on) {
    const int o = on && held ? at : -1;
    at += o >= 0 ? columns * 4 : 0;
    return o;
  };
  s.stage = 0;
  s.w = take(w), s.b = take(b), s.gw = take(gw), s.gb = take(gb);
  s.bytes = at;
  return s;
}

// One pass: h and r read, r' and x written.  A row's chunks stay in registers
// between its exchanges; the next row's are on their way into shared memory.
// 8192 x 12288 bfloat16, layer norm 129 us (6.2 TB/s; codes of the rows 189: one
// CTA of 12 warps hides a row's four rounds of shuffles and encoding alone);
// 4096 x 4096 bfloat16 22 (6.0), with a float32 residual, both norms and a gate
// 40 (5.0; codes 47), there bound by the latency of copies, shared memory and
// shuffles at 24 warps an SM (47 % of the issue slots busy); one token 3.1.
//
// FULL: h, r', both norms' w, and x in its type (1) or as codes of its rows (2),
// the common calls, with little left to ask for each chunk; POST: whether there
// is a post norm.  0: all asked for at run time.
template <int DT, int RT, int FULL, bool POST, int CK, int MODE>
__global__ void __launch_bounds__(kCtaThreads<CK, MODE>, CK >= 3 ? 1 : 3) k_norm_fwd(const Fwd p) {
  constexpr int CW = kWidth<RT>, NV = eights(CK) * 8 / CW;
  constexpr bool kHeld = held(CK, MODE);
  pdl_launch_dependents();
  pdl_wait();
  extern __shared__ __align__(16) uint8_t norm_smem[];
  __shared__ __align__(16) float slots[2][8][kMostWarps];
  Exchange ex = exchange(slots);
  const Place<CK, CW, MODE> at = {p.cols, (int)threadIdx.x};
  const int W = at.lanes();
  uint8_t *const own = norm_smem + (threadIdx.y * blockDim.x + threadIdx.x) * 16;
  const bool post = FULL ? POST : p.post != FP8_NORM_NONE;
  enum { kH = 1, kRout = 2, kX = 4, kXq = 8, kW = 16, kB = 32, kScaled = 64, kShifted = 128, kPre = 256 };
  int has = (p.h ? kH : 0) | (p.r_out ? kRout : 0) | (p.x ? kX : 0) | (p.xq ? kXq : 0) | (p.w.p ? kW : 0) | (p.b.p ? kB : 0) |
            (p.g.p || (post && p.pw.p) ? kScaled : 0) | (post && p.pb.p ? kShifted : 0) | (p.pre != FP8_NORM_NONE ? kPre : 0);
  constexpr int kKnown = FULL ? kH | kRout | kX | kXq | kW | kPre | (POST ? kScaled : kShifted) : 0;  // bits known here ...
  constexpr int kSet = FULL ? kH | kRout | (FULL == 1 ? kX : kXq) | kW | kPre | (POST ? kScaled : 0) : 0;  // ... and set
  auto on = [&](int bit) { return (kKnown & bit) ? (kSet & bit) != 0 : (has & bit) != 0; };
  const FwdSmem lay = fwd_smem<DT, RT>(8 * eights(CK) * W, on(kH), on(kW), on(kB), on(kScaled), on(kShifted), MODE, kHeld);
  uint8_t *const w_s = own + lay.w, *const b_s = own + lay.b, *const gw_s = own + lay.gw, *const gb_s = own + lay.gb;
  const unsigned stride = gridDim.x * blockDim.y;
  unsigned next = blockIdx.x * blockDim.y + threadIdx.y;
  In<RT, CK, CW, MODE> R(p.r, p.ldr, norm_smem, stride);
  In<DT, CK, CW, MODE> H(p.h, p.ldh, norm_smem + 8 * eights(CK) * W * kBytes<RT>, stride);
  Out<RT, CK, CW, MODE> Ro(p.r_out, p.ldro, stride);
  Out<DT, CK, CW, MODE> X(p.x, p.ldx, stride);
  R.seek(at, next), H.seek(at, next), Ro.seek(at, next), X.seek(at, next);
  if (next < (unsigned)p.rows) {
#pragma unroll
    for (int v = 0; v < NV; v++)
      if (at.mine(v)) {
        if (on(kH)) H.fetch(at, v);
        R.fetch(at, v);
      }
  }
  if (MODE == kStaged) R.advance(), H.advance();  // (the row behind)
  asm volatile("cp.async.commit_group;" ::: "memory");
  if constexpr (kHeld) {
#pragma unroll 1
    for (int v = 0; v < NV; v++) {  // (code that runs once: its fetch counts)
      float f[CW];
      if (on(kW)) load_params(p.w, 0, at, v, 1.0f, f), put_own(w_s, v, W, f);
      if (on(kB)) load_params(p.b, 0, at, v, 0.0f, f), put_own(b_s, v, W, f);
    }
  }
  keep(has);
  // the gate's row times the post norm's w and b
  auto gate_params = [&](int v, int gate, float (&gw)[CW], float (&gb)[CW]) {
    load_params(p.g, (size_t)gate * p.ldg, at, v, 1.0f, gw);
    if (on(kShifted)) {
      load_params(p.pb, 0, at, v, 0.0f, gb);
      mul(gb, gb, gw);
    }
    if (post) {
      float f[CW];
      load_params(p.pw, 0, at, v, 1.0f, f);
      mul(gw, gw, f);
    }
  };
  float inv = 1.0f / (float)p.cols, alpha = p.alpha, eps = p.eps;
  int inv_bits = __float_as_int(inv);
  keep(inv_bits);
  inv = __int_as_float(inv_bits);
  unsigned rows = (unsigned)p.rows;
  keep(rows);
  unsigned now = 0, gate_end = 0;  // the row's gate row, and the first row behind its rows
  for (; next < rows; next += stride) {
    const int row = (int)next;
    if ((on(kScaled) || on(kShifted)) && next >= gate_end) {
      now = next / (unsigned)p.gate_rows;
      gate_end = (now + 1) * (unsigned)p.gate_rows;
      if (gate_end < now) gate_end = 0xffffffffu;
      if constexpr (kHeld) {  // (a thread's own part: nobody else waits for it)
#pragma unroll 1
        for (int v = 0; v < NV; v++) {
          float gw[CW], gb[CW];
          gate_params(v, (int)now, gw, gb);
          if (on(kScaled)) put_own(gw_s, v, W, gw);
          if (on(kShifted)) put_own(gb_s, v, W, gb);
        }
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    float y[NV][CW];
    float2 s1 = make_float2(0.0f, 1.0f), s2 = make_float2(0.0f, 1.0f);
    if (post) {
#pragma unroll
      for (int v = 0; v < NV; v++) {
        if (at.mine(v)) {
          H.get(at, v, y[v]);
          mask(at, v, y[v]);
        } else {
          zero(y[v]);
        }
      }
      s1 = row_stats(y, at, p.post, inv, eps, ex);
    }
    const bool more = next + stride < rows && next + stride > next;
#pragma unroll
    for (int v = 0; v < NV; v++) {
      if (!at.mine(v)) {
        zero(y[v]);
        continue;
      }
      float f[CW], gb[CW];
      if (post) normed(y[v], y[v], s1.x, s1.y);
      else if (on(kH)) H.get(at, v, y[v]);
      else zero(y[v]);
      if (!kHeld) gate_params(v, (int)now, f, gb);
      if (on(kScaled)) {
        if (kHeld) get_own(gw_s, v, W, f);
        mul(y[v], y[v], f);
      }
      if (on(kShifted)) {
        if (kHeld) get_own(gb_s, v, W, gb);
        add(y[v], y[v], gb);
      }
      R.get(at, v, f);
      if (MODE == kStaged && more) {  // (what the chunk had has been read)
        if (on(kH)) H.fetch(at, v);
        R.fetch(at, v);
      }
      scale_add(y[v], alpha, f, y[v]);
      Ro.put(at, v, y[v], on(kRout));
      mask(at, v, y[v]);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    R.advance(), H.advance(), Ro.advance();
    if (on(kPre)) {
      s2 = row_stats(y, at, p.pre, inv, eps, ex);
      if (on(kX) || on(kXq)) {
#pragma unroll
        for (int v = 0; v < NV; v++) {
          if (at.mine(v)) {
            float f[CW];
            normed(y[v], y[v], s2.x, s2.y);
            if (on(kW)) {
              if (kHeld) get_own(w_s, v, W, f);
              else load_params(p.w, 0, at, v, 1.0f, f);
              mul(y[v], y[v], f);
            }
            if (on(kB)) {
              if (kHeld) get_own(b_s, v, W, f);
              else load_params(p.b, 0, at, v, 0.0f, f);
              add(y[v], y[v], f);
            }
            if (on(kX)) {
              float f2[CW];
#pragma unroll
              for (int j = 0; j < CW; j++) f2[j] = y[v][j];
              X.put(at, v, f2);
            }
          }
          if (on(kXq)) {
            mask(at, v, y[v]);
            put_codes(p, at, v, row, y[v]);
          }
        }
      }
    }
    X.advance();
    if (p.stats && threadIdx.x == 0) reinterpret_cast<float4 *>(p.stats)[row] = make_float4(s1.x, s1.y, s2.x, s2.y);
  }
}

// x again from r' and its statistics, as codes of 128x1 blocks: tiles of
// block_scale.cuh.  2 B (or 4) read and 1 written per element: 8192 x 12288
// bfloat16 85 us (3.5 TB/s), 4096 x 4096 16, with a float32 residual 22; as
// k_block_cast two barriers a tile, which two CTAs of 16 warps hide in part
// (63 % of the issue slots busy).
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
  block::Raw8<RT> raw[RP];
  block::load_tile<RT>(p.r, p.ldr, p.vec, row0, col0, p.rows, p.cols, raw);
  float w[8], b[8], f[RP][8];
  load_eight(p.w, col, p.cols, 1.0f, w);
  load_eight(p.b, col, p.cols, 0.0f, b);
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
  int kind, threads, groups;           // CK; of a CTA: threads of a row, rows at a time
  int gate_rows, unit_rows, per_gate;  // rows of a gate row and of a unit, units per gate row
  long long units;
  int ctas;
};

constexpr int kSms = 148;

inline int padded(int cols) { return (cols + 7) / 8 * 8; }  // of a partial sum

inline Plan plan_of(int rows, int cols, int gate_rows) {
  Plan p = {};
  const int vecs = (cols + 7) / 8;
  p.kind = vecs <= kThreads ? 1 : vecs <= 2 * kThreads ? 2 : vecs <= 2 * kMostThreads ? 3 : 4;
  p.threads = p.kind == 2 ? kThreads : p.kind == 3 ? kMostThreads : (vecs + 32 * p.kind - 1) / (32 * p.kind) * 32;
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
__host__ __device__ inline BwdSmem bwd_smem(int columns, bool h, bool dro, bool pre, bool scaled, bool groups, int mode, bool held) {
  BwdSmem s;
  int at = mode == kStaged ? columns * ((h ? kBytes<DT> : 0) + (dro ? kBytes<RT> : 0) + (pre ? kBytes<DT> + kBytes<RT> : 0)) : 0;
  auto take = [&](bool on) {
    const int o = on && held ? at : -1;
    at += o >= 0 ? columns * 4 : 0;
    return o;
  };
  s.w = take(pre), s.gw = take(scaled);
  s.comb = groups ? at : -1;
  at += groups ? kThreads * 32 : 0;
  s.bytes = at;
  return s;
}

// Adds up the groups of a CTA and writes one partial sum.
template <int CK, int CW, int MODE>
__device__ __forceinline__ void flush(float (&a)[CW], uint8_t *comb, float *out, const Place<CK, CW, MODE> &at, int v) {
  if (CK == 1 && blockDim.y > 1) {  // (rows of several chunks have a CTA to themselves)
    uint8_t *own = comb + (threadIdx.y * blockDim.x + threadIdx.x) * 16;
    __syncthreads();
    put_own(own, 0, kThreads, a);
    __syncthreads();
    if (threadIdx.y == 0) {
      for (int y = 1; y < (int)blockDim.y; y++) {
        float f[CW];
        get_own(own + y * blockDim.x * 16, 0, kThreads, f);
        add(a, a, f);
      }
    }
  }
  if (threadIdx.y == 0) {
    if constexpr (MODE == kStaged) {
      if (at.has(v, 0)) {
        float4 *o = reinterpret_cast<float4 *>(out + at.col(v, 0));
#pragma unroll
        for (int h = 0; h < CW / 4; h++) o[h] = make_float4(a[4 * h], a[4 * h + 1], a[4 * h + 2], a[4 * h + 3]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < CW; j++)
        if (at.has(v, j)) out[at.col(v, j)] = a[j];
    }
  }
#pragma unroll
  for (int j = 0; j < CW; j++) a[j] = 0.0f;
}

// dx, dr', r' and h read, dr and dh written: 8192 x 12288 bfloat16 278 us without
// the parameters' gradients (4.4 TB/s) and 286 to 292 with, 4096 x 4096 with a
// float32 residual and both norms 59 and 69 (5.1 TB/s), 2048 x 8192 91.  Bound by
// the copies of one row in flight beside 12 to 16 warps.  Registers: a thread
// holds all four sums of its columns whether they are wanted or not (A and C are
// asked for at run time, F is there at CK >= 3); of 12288 columns they take 128 of
// 168, and without a gate and a post norm 64 of these stay 0 while 248 bytes spill.
//
// BIAS: whether sums of dx and of G are wanted (gradients of b, of post_b, and
// of a gate behind post_b).  FULL: dx, dr', h, both outputs and the post norm's
// w, the common call; POST: whether there is a post norm.  Else asked for at run
// time.
template <int DT, int RT, bool FULL, bool POST, bool BIAS, int CK, int MODE>
__global__ void __launch_bounds__(kCtaThreads<CK, MODE>, CK >= 3 ? 1 : 2) k_norm_bwd(const Bwd p) {
  constexpr int CW = kWidth<RT>, NV = eights(CK) * 8 / CW;
  constexpr bool kHeld = held(CK, MODE);
  pdl_launch_dependents();
  pdl_wait();
  extern __shared__ __align__(16) uint8_t norm_smem[];
  __shared__ __align__(16) float slots[2][8][kMostWarps];
  Exchange ex = exchange(slots);
  const Place<CK, CW, MODE> at = {p.cols, (int)threadIdx.x};
  const int W = at.lanes();
  const bool post = FULL ? POST : p.post != FP8_NORM_NONE;
  enum { kH = 1, kDro = 2, kDr = 4, kDh = 8, kAc = 16, kScaled = 32, kPre = 64, kLayer = 128, kPreLayer = 256, kPostLayer = 512,
         kStats = 1024 };
  int has = (p.h ? kH : 0) | (p.dro ? kDro : 0) | (p.dr ? kDr : 0) | (p.dh ? kDh : 0) | (p.ac ? kAc : 0) |
            (p.h && (p.g.p || (post && p.pw.p)) ? kScaled : 0) | (p.pre != FP8_NORM_NONE ? kPre : 0) |
            (p.pre == FP8_NORM_LAYER ? kPreLayer | kLayer : 0) | (p.post == FP8_NORM_LAYER ? kPostLayer | kLayer : 0) |
            (p.stats ? kStats : 0);
  constexpr int kKnown = FULL ? kH | kDro | kDr | kDh | kPre | kStats | (POST ? kScaled : kPostLayer) : 0;  // bits known here ...
  constexpr int kSet = FULL ? kH | kDro | kDr | kDh | kPre | kStats | (POST ? kScaled : 0) : 0;             // ... and set
  auto on = [&](int bit) { return (kKnown & bit) ? (kSet & bit) != 0 : (has & bit) != 0; };
  const BwdSmem lay = bwd_smem<DT, RT>(8 * eights(CK) * W, on(kH), on(kDro), on(kPre), on(kScaled), blockDim.y > 1, MODE, kHeld);
  uint8_t *const own = norm_smem + (threadIdx.y * blockDim.x + threadIdx.x) * 16;
  uint8_t *const w_s = own + lay.w, *const gw_s = own + lay.gw, *const comb = norm_smem + lay.comb;
  uint8_t *part = norm_smem;
  auto take = [&](bool on, int bytes) {
    uint8_t *s = part;
    part += on ? 8 * eights(CK) * W * bytes : 0;
    return s;
  };
  const unsigned apart = blockDim.y;
  In<DT, CK, CW, MODE> DX(p.dx, p.lddx, take(on(kPre), kBytes<DT>), apart);
  In<RT, CK, CW, MODE> RO(p.ro, p.ldro, take(on(kPre), kBytes<RT>), apart);
  In<RT, CK, CW, MODE> DRO(p.dro, p.lddro, take(on(kDro), kBytes<RT>), apart);
  In<DT, CK, CW, MODE> H(p.h, p.ldh, take(on(kH), kBytes<DT>), apart);
  Out<RT, CK, CW, MODE> DR(p.dr, p.lddr, apart);
  Out<DT, CK, CW, MODE> DH(p.dh, p.lddh, apart);
  keep(has);
  auto fetch = [&](int v) {
    if (!at.mine(v)) return;
    if (on(kPre)) {
      DX.fetch(at, v);
      RO.fetch(at, v);
    }
    if (on(kDro)) DRO.fetch(at, v);
    if (on(kH)) H.fetch(at, v);
  };
  auto advance_in = [&] { DX.advance(), RO.advance(), DRO.advance(), H.advance(); };
  const float inv = 1.0f / (float)p.cols, alpha = p.alpha;
  const size_t ld_sum = (size_t)(p.cols + 7) / 8 * 8;
  const long long u0 = p.units * blockIdx.x / gridDim.x, u1 = p.units * (blockIdx.x + 1) / gridDim.x;
  float E[NV][CW], F[NV][CW], A[NV][CW], C[NV][CW];
#pragma unroll
  for (int v = 0; v < NV; v++)
#pragma unroll
    for (int j = 0; j < CW; j++) E[v][j] = F[v][j] = A[v][j] = C[v][j] = 0.0f;
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
  // the first row of unit u for this group: its loads, and the pointers behind it
  auto fetch_first = [&](long long u) {
    if (u >= u1) return;
    const Span s = rows_of(u);
    const long long row = s.first + threadIdx.y;
    DX.seek(at, row), RO.seek(at, row), DRO.seek(at, row), H.seek(at, row);
    if (row < s.last) {
#pragma unroll
      for (int v = 0; v < NV; v++) fetch(v);
      if (on(kStats)) s_next = __ldg(reinterpret_cast<const float4 *>(p.stats) + row);
    }
    if (MODE == kStaged) advance_in();
  };
  fetch_first(u0);
  asm volatile("cp.async.commit_group;" ::: "memory");
  if (kHeld && on(kPre)) {
#pragma unroll 1
    for (int v = 0; v < NV; v++) {
      float f[CW];
      load_params(p.w, 0, at, v, 1.0f, f);
      put_own(w_s, v, W, f);
    }
  }
  auto weight = [&](int v, float (&f)[CW]) {
    if (kHeld) get_own(w_s, v, W, f);
    else load_params(p.w, 0, at, v, 1.0f, f);
  };
  // the gate's row times the post norm's w
  auto gate_params = [&](int v, int gate, float (&g)[CW]) {
    load_params(p.g, (size_t)gate * p.ldg, at, v, 1.0f, g);
    if (post) {
      float f[CW];
      load_params(p.pw, 0, at, v, 1.0f, f);
#pragma unroll
      for (int j = 0; j < CW; j++) g[j] *= f[j];
    }
  };
  int gate_now = -1;
  for (long long u = u0; u < u1; u++) {
    const int gate = (int)(u / p.per_gate);
    const Span span = rows_of(u);
    if (kHeld && (on(kScaled)) && gate != gate_now) {
      gate_now = gate;
#pragma unroll 1
      for (int v = 0; v < NV; v++) {
        float g[CW];
        gate_params(v, gate, g);
        put_own(gw_s, v, W, g);
      }
    }
    auto gate_weight = [&](int v, float (&f)[CW]) {
      if (kHeld) get_own(gw_s, v, W, f);
      else gate_params(v, gate, f);
    };
    const long long row0 = span.first + threadIdx.y;
    DR.seek(at, row0), DH.seek(at, row0);
    for (int row = (int)row0, left = (int)(span.last - row0); left > 0; row += apart, left -= apart) {
      const float4 s = s_next;
      const bool more = left > (int)apart;
      if (more && (on(kStats))) s_next = __ldg(reinterpret_cast<const float4 *>(p.stats) + row + apart);
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      float m0 = 0.0f, m1 = 0.0f, t0 = 0.0f, t1 = 0.0f;
      const bool pre = on(kPre), layer = on(kLayer);
      if (pre || post) {
        float2 k[8];
#pragma unroll
        for (int i = 0; i < 8; i++) k[i] = both(0.0f);
#pragma unroll(CK == 4 ? 1 : NV)
        for (int v = 0; v < NV; v++) {
          if (!at.mine(v)) continue;
          float t[CW], n2[CW];
          if (pre) {
            float w[CW];
            DX.get(at, v, t);
            RO.get(at, v, n2);
            weight(v, w);
            mask(at, v, t);
            normed(n2, n2, s.z, s.w);
            mul(t, t, w);
            dot(k[0], t, n2);
            if (layer) plus(k[1], t);
          } else {
            zero(t);
            zero(n2);
          }
          if (post) {
            float q[CW], n1[CW], h[CW];
            if (on(kDro)) DRO.get(at, v, h);
            else zero(h);
            H.get(at, v, n1);
            fma8(h, t, s.w, h);
            normed(n1, n1, s.x, s.y);
            if (on(kScaled)) {
              gate_weight(v, q);
            } else {
#pragma unroll
              for (int j = 0; j < CW; j++) q[j] = 1.0f;
            }
            mask(at, v, q);
            mul(h, q, h);    // gw H
            dot(k[2], h, n1);
            if (layer) {
              plus(k[4], h);
              plus(k[7], q);
              dot(k[5], q, n2);
            }
            mul(q, q, n1);  // gw n1
            dot(k[3], q, n2);
            if (layer) plus(k[6], q);
          }
        }
        float c[8];
#pragma unroll
        for (int i = 0; i < 8; i++) c[i] = k[i].x + k[i].y;
        if (post && layer) {
          row_sums(c, ex);
        } else if (post) {
          float few[4] = {c[0], c[2], c[3], 0.0f};
          row_sums(few, ex);
          c[0] = few[0], c[2] = few[1], c[3] = few[2];
        } else if (layer) {
          float few[2] = {c[0], c[1]};
          row_sums(few, ex);
          c[0] = few[0], c[1] = few[1];
        } else {
          float one[1] = {c[0]};
          row_sums(one, ex);
          c[0] = one[0];
        }
        m1 = c[0] * inv;
        if (on(kPreLayer)) m0 = c[1] * inv;
        if (post) {
          t1 = (c[2] - s.w * fmaf(m0, c[6], m1 * c[3])) * inv;
          if (on(kPostLayer)) t0 = (c[4] - s.w * fmaf(m0, c[7], m1 * c[5])) * inv;
        }
      }
#pragma unroll
      for (int v = 0; v < NV; v++) {
        if (!at.mine(v)) continue;
        float G[CW], t[CW], n[CW];
        if (on(kDro)) DRO.get(at, v, G);
        else zero(G);
        if (pre) {
          float w[CW];
          DX.get(at, v, t);
          RO.get(at, v, n);
          weight(v, w);
          normed(n, n, s.z, s.w);
          fma8(E[v], t, n, E[v]);
          if (BIAS) add(F[v], F[v], t);
          fma8(t, t, w, -m0);
          fma8(t, n, -m1, t);
          fma8(G, t, s.w, G);
        }
        if (on(kH)) H.get(at, v, n);
        if (MODE == kStaged && more) fetch(v);  // (what the chunk had has been read)
        if (on(kDr)) {
          mul(t, G, alpha);
          DR.put(at, v, t);
        }
        if (on(kH)) {
          if (post) normed(n, n, s.x, s.y);
          if (on(kAc)) {
            fma8(A[v], G, n, A[v]);
            if (BIAS) add(C[v], C[v], G);
          }
          if (on(kScaled)) {
            gate_weight(v, t);
            mul(G, G, t);
          }
          if (post) {
            add(G, G, -t0);
            fma8(G, n, -t1, G);
            mul(G, G, s.y);
          }
          if (on(kDh)) DH.put(at, v, G);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      advance_in();
      DR.advance(), DH.advance();
    }
    fetch_first(u + 1);
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (p.ac) {
#pragma unroll
      for (int v = 0; v < NV; v++) {
        flush(A[v], comb, p.ac + (size_t)(2 * u) * ld_sum, at, v);
        if (BIAS) flush(C[v], comb, p.ac + (size_t)(2 * u + 1) * ld_sum, at, v);
      }
    }
  }
  if (p.ef) {
#pragma unroll
    for (int v = 0; v < NV; v++) {
      flush(E[v], comb, p.ef + (size_t)(2 * blockIdx.x) * ld_sum, at, v);
      if (BIAS) flush(F[v], comb, p.ef + (size_t)(2 * blockIdx.x + 1) * ld_sum, at, v);
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
// (threadIdx.y) every 32nd partial sum.  Two or three microseconds behind the
// kernel above, and 4 to 8 in all with the sums' stores and loads.
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
