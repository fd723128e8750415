// block_act.cuh -- activation functions whose input is kept for the backward
// pass as E4M3 codes with a scale per 1x128 block: one byte per element
// instead of a 16-bit tensor.
//
// forward   a = act(h);  c = blocks(h) (the checkpoint);  optionally blocks(a),
//           the next product's operand, and a itself
// backward  h' = dec(c);  dh = da * act'(h');  optionally blocks of dh along
//           either axis (the operands of the gradient products), blocks of
//           act(h') along the rows (the weight gradient's other operand), and
//           dh itself
// so neither a nor any 16-bit activation has to survive the forward pass.
// The blocks are those of block_scale.cuh ("Training and inference of large
// language models using 8-bit floating point", 제안 방법, per block).
#pragma once

#include "block_scale.cuh"

namespace fp8lib {
namespace block {

// All three functions have the form act(h) = h * g(h) with a gate g that goes
// from 0 to 1 and satisfies g(-h) = 1 - g(h):  SiLU g = s(h);  tanh GELU g =
// s(2 c (h + 0.044715 h^3)), c = sqrt(2/pi) (since (1 + tanh(u)) / 2 = s(2u));
// GELU g = Phi(h).  With y = |h| and p = g(-y) = 1 - g(y), the small one of the
// two, computed on its own so that it keeps its relative accuracy,
//   act(h)  = max(h, 0) - y p
//   act'(h) = (h >= 0 ? 1 : 0) + sign(h) r,   r = y g'(y) - p,
// and for the sigmoid gates g' = p (1 - p) u', so r = p (y (1 - p) u' - 1).
//
// For h > 0 act(h) lies below h, possibly by less than binary32 shows.
// Rounded to nearest it would become h itself, and h, a 16-bit number, sits
// exactly on an FP8 rounding border one time in sixteen: the tie would then go
// to the even code where the true value goes to the lower one.  So y p is
// subtracted rounding toward zero, and da act' = da + da r is rounded to the
// side of da on which it lies.  p never reaches 0 (the smallest subnormal is
// added to it, which shows in nothing else), and r is then positive.
//
// These kernels were bound by the ALU pipe (minima, selects, logic: half the
// rate of FMA), so the arithmetic is on the packed binary32 instructions and
// the rest as little as it can be: 43 -> 24 instructions per element forward,
// 63 -> 42 backward, a sixth of the time then.  The erf form calls erfcf for
// every element and takes twice as long (times beside the kernels).
// ex2.approx and rcp.approx are within 2 units in the last place, and the
// argument's rounding adds about |u| units to exp(-u); exp(-u) below 2^-126
// counts as 0.
constexpr float kLeast = 1.4012984643e-45f;  // 2^-149
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float2 exp2_approx(float2 x) {
  float2 r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(x.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(x.y));
  return r;
}
__device__ __forceinline__ float2 rcp_approx(float2 x) {
  float2 r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(x.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(x.y));
  return r;
}

// The gates of two elements: y = |h|, at most 110 (exp(-110) is 0 in binary32;
// a NaN stays), p and, with GRAD, r.
template <int ACT, bool GRAD>
__device__ __forceinline__ void gate2(float2 h, float2 &y, float2 &p, float2 &r) {
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y.x) : "f"(fabsf(h.x)), "f"(110.0f));
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y.y) : "f"(fabsf(h.y)), "f"(110.0f));
  if constexpr (ACT == FP8_ACT_GELU_ERF) {
    const float2 e = make_float2(erfcf(y.x * 0.70710678118654752f), erfcf(y.y * 0.70710678118654752f));
    p = __ffma2_rn(e, both(0.5f), both(kLeast));
    if constexpr (GRAD) {
      const float2 s = exp2_approx(__fmul2_rn(__fmul2_rn(y, y), both(-0.5f * kLog2e)));
      // (where both have underflowed: y 2^-149 - 2^-149 > 0)
      r = __ffma2_rn(y, __ffma2_rn(s, both(0.39894228040143268f), both(kLeast)), make_float2(-p.x, -p.y));
    }
  } else {
    constexpr float c = 1.5957691216057308f;  // 2 sqrt(2/pi)
    float2 a, du = both(1.0f);
    if constexpr (ACT == FP8_ACT_GELU_TANH) {
      const float2 y2 = __fmul2_rn(y, y);
      a = __fmul2_rn(y, __ffma2_rn(both(-0.044715f * c * kLog2e), y2, both(-c * kLog2e)));
      du = __ffma2_rn(both(3.0f * 0.044715f * c), y2, both(c));
    } else {
      a = __fmul2_rn(y, both(-kLog2e));
    }
    const float2 e = exp2_approx(a);
    const float2 big = rcp_approx(__fadd2_rn(e, both(1.0f)));
    p = __ffma2_rn(e, big, both(kLeast));
    if constexpr (GRAD) {
      const float2 yb = __fmul2_rn(y, big);
      const float2 w = ACT == FP8_ACT_GELU_TANH ? __ffma2_rn(yb, du, both(-1.0f)) : __fadd2_rn(yb, both(-1.0f));
      r = __fmul2_rn(p, w);
    }
  }
}

__device__ __forceinline__ float2 act_value2(float2 h, float2 y, float2 p) {
  return __ffma2_rz(make_float2(-y.x, -y.y), p, make_float2(fmaxf(h.x, 0.0f), fmaxf(h.y, 0.0f)));
}

__device__ __forceinline__ float2 act_grad2(float2 h, float2 r, float2 da) {
  // r with the sign of h; da or, for h < 0, 0
  const uint32_t sx = __float_as_uint(h.x) & 0x80000000u, sy = __float_as_uint(h.y) & 0x80000000u;
  r = make_float2(__uint_as_float(__float_as_uint(r.x) ^ sx), __uint_as_float(__float_as_uint(r.y) ^ sy));
  const float2 base = make_float2(sx ? 0.0f : da.x, sy ? 0.0f : da.y);
  const float2 up = __ffma2_ru(da, r, base), down = __ffma2_rd(da, r, base);
  // the side: the sign of da r, kept from underflowing
  const float2 side = __fmul2_rn(__fmul2_rn(r, both(1.2676506e30f)), da);
  return make_float2(side.x > 0.0f ? up.x : down.x, side.y > 0.0f ? up.y : down.y);
}

// Adds 0 times a word's elements: stays 0 (of either sign) unless one is an
// infinity or a NaN.  One FMA per word, on the pipe that is less used here.
template <int DT>
__device__ __forceinline__ void add_non_finite(uint32_t &t, uint32_t w) {
  if constexpr (DT == FP8_DT_F32) asm("fma.rn.f32 %0, %1, 0f00000000, %0;" : "+r"(t) : "r"(w));
  else if constexpr (DT == FP8_DT_BF16) asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(t) : "r"(w), "r"(0u));
  else asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(t) : "r"(w), "r"(0u));
}
template <int DT>
__device__ __forceinline__ bool was_non_finite(uint32_t t) {
  return (t & (DT == FP8_DT_F32 ? 0x7fffffffu : 0x7fff7fffu)) != 0;
}

constexpr int kActThreads = 512;            // k_act_bwd
constexpr int kActStep = kActThreads / 16;  // rows between a thread's rows

struct ActFwd {
  const void *h;
  int rows, cols;
  size_t ldh;
  int margin;
  uint8_t *cq, *cs;  // the checkpoint
  size_t ldc;
  uint8_t *aq, *as;  // blocks of a, or null
  size_t lda_q;
  void *a;           // a itself in h's type, or null
  size_t lda;
  int vec_h, vec_a;  // rows of h / a start on 16-byte boundaries
};

// h is read once (2 B at 16 bits), one or two code bytes and / or a are written;
// 4096 x 16384 bfloat16 with a itself 63 us (5.4 TB/s; SiLU 62, GELU by erf 145),
// with its codes 61 (59, 149), bound by the issue slots (66 and 73 % busy).  Four rows per thread: act(h) of a thread's 32
// elements waits in registers for its rows' amaxes (eight rows each needed
// 184 registers and ran at a third of the occupancy).
template <int DT, int ACT, int RP>
__global__ void __launch_bounds__(kPartThreads<RP>, 1024 / kPartThreads<RP>) k_act_fwd(const ActFwd p) {
  pdl_launch_dependents();
  pdl_wait();
  const auto [row0, col0] = part_at<RP>(blockIdx.x, (p.cols + kTile - 1) / kTile);
  Raw8<DT> raw[RP];
  load_tile<DT>(p.h, p.ldh, p.vec_h, row0, col0, p.rows, p.cols, raw);
  cast_raw_rows<DT, FP8_E4M3>(raw, p.cq, p.cs, p.ldc, row0, col0, p.rows, p.cols, kMaxE4M3, p.margin);
  if (!p.aq && !p.a) return;
  float f[RP][8];
#pragma unroll
  for (int i = 0; i < RP; i++) {
    unpack8<DT>(raw[i], f[i]);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float2 h = make_float2(f[i][j], f[i][j + 1]);
      float2 y, q, r;
      gate2<ACT, false>(h, y, q, r);
      const float2 a = act_value2(h, y, q);
      f[i][j] = a.x;
      f[i][j + 1] = a.y;
    }
  }
  if (p.a) store_tile<DT>(p.vec_a, p.a, p.lda, row0, col0, p.rows, p.cols, f);
  if (p.aq) cast_tile_rows<FP8_E4M3>(f, p.aq, p.as, p.lda_q, row0, col0, p.rows, p.cols, kMaxE4M3, p.margin);
}

struct ActBwd {
  const uint8_t *cq, *cs;
  size_t ldc;
  const void *da;
  int rows, cols;
  size_t ldda;
  int margin;
  CastOut dh;          // blocks of dh along the columns (q, s) and the rows (qt, st), or null
  uint8_t *aqt, *ast;  // blocks of act(h') along the rows, or null
  size_t ldaqt;
  void *dh_hp;         // dh itself in da's type, or null
  size_t lddh;
  int vec_da, vec_dh;  // rows of da / dh start on 16-byte boundaries
};

__device__ __forceinline__ void cp_async(uint32_t dst, const void *src, int bytes, bool in) {
  const int n = in ? bytes : 0;  // the rest of the destination is zeroed
  if (bytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

// An infinite da (a gradient that overflowed) at h' >= 0: act' is positive
// there, so dh is da, where act_grad2's da + da r is inf - inf for r < 0.  v is
// h' or act(h'), which has its sign.
__device__ __forceinline__ bool stays_infinite(float v, float da) {
  return fabsf(da) == INFINITY && __float_as_uint(v) <= 0x7f800000u;
}
// That for a thread's part of a tile, v its act(h'): a rare path of its own, in
// which da is read again (dh may take da's place, but not before the tile is
// stored).  With the search for infinities 2 to 3 % of the pass.
template <int DT, int RP>
__device__ __forceinline__ void keep_infinite(const ActBwd &p, int row0, int col0, const float (&v)[RP][8],
                                              float (&d)[RP][8]) {
  const int row = row0 + (threadIdx.x >> 4), col = col0 + (threadIdx.x & 15) * 8;
#pragma unroll
  for (int i = 0; i < RP; i++) {
    float da[8];
    unpack8<DT>(load_raw8_single<DT>(p.da, p.ldda, row + Geo<RP>::kStep * i, col, p.rows, p.cols), da);
#pragma unroll
    for (int j = 0; j < 8; j++)
      if (stays_infinite(v[i][j], da[j])) d[i][j] = da[j];
  }
}

// dh of a thread whose da is not all finite, row by row and straight to memory
// (each element is read before it is written: dh may take da's place).
template <int DT, int ACT, int RP>
__device__ __forceinline__ void act_bwd_non_finite(const ActBwd &p, int row0, int col0) {
  const int col = col0 + (threadIdx.x & 15) * 8, kg = ((p.cols + kTile - 1) / kTile + 3) / 4;
#pragma unroll 1
  for (int i = 0; i < RP; i++) {
    const int row = row0 + (threadIdx.x >> 4) + Geo<RP>::kStep * i;
    if (row >= p.rows) break;
    float a[8], d[8];
    unpack8<DT>(load_raw8_single<DT>(p.da, p.ldda, row, col, p.rows, p.cols), d);
    decode8<FP8_E4M3>(load_codes8(p.cq, p.ldc, row, col, p.rows, p.cols), a);
    const float s = descale_of(p.cs[scale_at(row, col0 / kTile, kg)]);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float2 h = __fmul2_rn(make_float2(a[j], a[j + 1]), both(s)), da = make_float2(d[j], d[j + 1]);
      float2 y, v, r;
      gate2<ACT, true>(h, y, v, r);
      const float2 g = act_grad2(h, r, da);
      d[j] = stays_infinite(h.x, da.x) ? da.x : g.x;
      d[j + 1] = stays_infinite(h.y, da.y) ? da.y : g.y;
    }
    store8<DT>(false, p.dh_hp, p.lddh, row, col, p.rows, p.cols, d);
  }
}

// dh alone: parts of tiles, as k_act_fwd.  float32 with two rows per thread and
// ten CTAs per SM, 16-bit types with four and eight: 4096 x 16384 float32 91 us
// (6.6 TB/s; four rows 101, a persistent CTA of 512 threads 139), bfloat16 73
// (4.6; SiLU 69, GELU by erf 156; two rows 76, persistent 72; without the search
// for infinities 72), 73 % of the issue slots busy.
template <int DT>
constexpr int kPlainRows = DT == FP8_DT_F32 ? 2 : 4;
template <int DT, int ACT, int RP>
__global__ void __launch_bounds__(kPartThreads<RP>, (RP == 2 ? 1280 : 1024) / kPartThreads<RP>)
    k_act_bwd_plain(const ActBwd p) {
  pdl_launch_dependents();
  pdl_wait();
  const int tiles_c = (p.cols + kTile - 1) / kTile, kg = (tiles_c + 3) / 4;
  const auto [row0, col0] = part_at<RP>(blockIdx.x, tiles_c);
  const int col = col0 + (threadIdx.x & 15) * 8, row = row0 + (threadIdx.x >> 4);
  Raw8<DT> raw[RP];
  uint2 q[RP];
  uint32_t sb[RP];
  if (row0 + kTile <= p.rows && col0 + kTile <= p.cols) {  // inside: nothing to clamp, all loads in flight at once
    const uint8_t *c = p.cq + (size_t)row * p.ldc + col;
#pragma unroll
    for (int i = 0; i < RP; i++, c += Geo<RP>::kStep * p.ldc) q[i] = __ldcs(reinterpret_cast<const uint2 *>(c));
  } else {
#pragma unroll
    for (int i = 0; i < RP; i++) q[i] = load_codes8(p.cq, p.ldc, row + Geo<RP>::kStep * i, col, p.rows, p.cols);
  }
#pragma unroll
  for (int i = 0; i < RP; i++) sb[i] = p.cs[scale_at(min(row + Geo<RP>::kStep * i, p.rows - 1), col0 / kTile, kg)];
  load_tile<DT>(p.da, p.ldda, p.vec_da, row0, col0, p.rows, p.cols, raw);
  uint32_t odd = 0;
  float d[RP][8];
#pragma unroll
  for (int i = 0; i < RP; i++) {
    float a[8];
#pragma unroll
    for (int j = 0; j < Raw8<DT>::kWords; j++) add_non_finite<DT>(odd, raw[i].w[j]);
    decode8<FP8_E4M3>(q[i], a);
    unpack8<DT>(raw[i], d[i]);
    const float s = descale_of(sb[i]);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float2 h = __fmul2_rn(make_float2(a[j], a[j + 1]), both(s));
      float2 y, v, r;
      gate2<ACT, true>(h, y, v, r);
      const float2 g = act_grad2(h, r, make_float2(d[i][j], d[i][j + 1]));
      d[i][j] = g.x;
      d[i][j + 1] = g.y;
    }
  }
  if (was_non_finite<DT>(odd)) act_bwd_non_finite<DT, ACT, RP>(p, row0, col0);
  else store_tile<DT>(p.vec_dh, p.dh_hp, p.lddh, row0, col0, p.rows, p.cols, d);
}

// Shared memory of k_act_bwd: two buffers of a tile's codes and da, each
// thread's own elements at its own places, so that a thread waits for its own
// copies only.
template <int DT>
struct ActBwdSmem {
  static constexpr int kCodeBytes = kTile * kTile;
  static constexpr int kBuffer = kCodeBytes * (DT == FP8_DT_F32 ? 5 : 3);
  static constexpr int kBytes = 2 * kBuffer;
};

// One pass over 128x128 tiles: 1 + 2 B read, up to 3 code bytes (and 2 B of dh)
// written.  dh and act(h') of a thread's 32 elements stay in registers between
// the amaxes and the encoding, which leaves room for one CTA of 16 warps per
// SM; the next tile's inputs are copied into shared memory meanwhile.  Bound by
// latency (one CTA, two barriers a tile) and instruction issue (62 % of the
// slots, 31 % of the DRAM cycles): 4096 x 16384 bfloat16 to the codes of all
// three 130 us, up to 158 in a long run (SiLU 126, GELU by erf 221; float32 176,
// 168, 262).
// OUT: the format of dh's codes.
template <int DT, int ACT, int OUT>
__global__ void __launch_bounds__(kActThreads, 1) k_act_bwd(const ActBwd p) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int RP = 4, kVecs = Raw8<DT>::kWords / 4;
  using Smem = ActBwdSmem<DT>;
  extern __shared__ __align__(16) uint8_t act_smem[];
  __shared__ ColScratch<RP> sc[2];
  const int tiles_c = (p.cols + kTile - 1) / kTile;
  const unsigned tiles = (unsigned)((p.rows + kTile - 1) / kTile) * (unsigned)tiles_c;
  const int kg = (tiles_c + 3) / 4;
  const float gmax = OUT == FP8_E4M3 ? kMaxE4M3 : kMaxE5M2;
  const int c8 = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  const uint32_t smem = smem_u32(act_smem);
  uint32_t sb[RP];  // scale bytes of the tile in the buffer
  // Starts the copies of tile t into buffer b (tiles with a ragged or unaligned row are read directly instead).
  auto prefetch = [&](TileAt at, int b) {
    const int row0 = at.row0, col0 = at.col0, col = col0 + c8 * 8;
    if (wide_tile(p.vec_da, col0, p.cols)) {
      const uint32_t base = smem + b * Smem::kBuffer;
      if (row0 + kTile <= p.rows && col0 + kTile <= p.cols) {  // inside: nothing to leave out
        const uint8_t *cq = p.cq + (size_t)(row0 + r0) * p.ldc + col;
        const size_t esz = DT == FP8_DT_F32 ? 4 : 2;
        const uint8_t *da = reinterpret_cast<const uint8_t *>(p.da) + ((size_t)(row0 + r0) * p.ldda + col) * esz;
        const size_t cstep = kActStep * p.ldc, dstep = kActStep * p.ldda * esz;
#pragma unroll
        for (int i = 0; i < RP; i++, cq += cstep, da += dstep) {
          cp_async(base + (i * kActThreads + threadIdx.x) * 8, cq, 8, true);
#pragma unroll
          for (int v = 0; v < kVecs; v++)
            cp_async(base + Smem::kCodeBytes + ((i * kVecs + v) * kActThreads + threadIdx.x) * 16, da + 16 * v, 16, true);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        return;
      }
#pragma unroll
      for (int i = 0; i < RP; i++) {
        const int row = row0 + r0 + kActStep * i;
        const bool in = row < p.rows && col < p.cols;
        const size_t r = in ? row : 0, c = in ? col : 0;
        cp_async(base + (i * kActThreads + threadIdx.x) * 8, p.cq + r * p.ldc + c, 8, in);
        const uint8_t *src = reinterpret_cast<const uint8_t *>(p.da) + (r * p.ldda + c) * (DT == FP8_DT_F32 ? 4 : 2);
#pragma unroll
        for (int v = 0; v < kVecs; v++)
          cp_async(base + Smem::kCodeBytes + ((i * kVecs + v) * kActThreads + threadIdx.x) * 16, src + 16 * v, 16, in);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  TileAt next = tile_at(blockIdx.x, tiles_c);  // (the grid has at most one CTA per tile)
  prefetch(next, 0);
  int buf = 0;
  for (unsigned t = blockIdx.x; t < tiles; t += gridDim.x, buf ^= 1) {
    const int row0 = next.row0, col0 = next.col0;
    const int col = col0 + c8 * 8;
#pragma unroll
    for (int i = 0; i < RP; i++)
      sb[i] = p.cs[scale_at(min(row0 + r0 + kActStep * i, p.rows - 1), col0 / kTile, kg)];
    if (t + gridDim.x < tiles) {
      next = tile_at(t + gridDim.x, tiles_c);
      prefetch(next, buf ^ 1);
    } else asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    float a[RP][8], d[RP][8];
    uint32_t odd = 0;
    if (wide_tile(p.vec_da, col0, p.cols)) {
      const uint8_t *base = act_smem + buf * Smem::kBuffer;
#pragma unroll
      for (int i = 0; i < RP; i++) {
        decode8<FP8_E4M3>(*reinterpret_cast<const uint2 *>(base + (i * kActThreads + threadIdx.x) * 8), a[i]);
        Raw8<DT> raw;
#pragma unroll
        for (int v = 0; v < kVecs; v++)
          *reinterpret_cast<uint4 *>(&raw.w[4 * v]) = *reinterpret_cast<const uint4 *>(
              base + Smem::kCodeBytes + ((i * kVecs + v) * kActThreads + threadIdx.x) * 16);
        unpack8<DT>(raw, d[i]);
#pragma unroll
        for (int j = 0; j < Raw8<DT>::kWords; j++) add_non_finite<DT>(odd, raw.w[j]);
      }
    } else {
      Raw8<DT> raw[RP];
      load_tile<DT>(p.da, p.ldda, p.vec_da, row0, col0, p.rows, p.cols, raw);
#pragma unroll
      for (int i = 0; i < RP; i++) {
        decode8<FP8_E4M3>(load_codes8(p.cq, p.ldc, row0 + r0 + kActStep * i, col, p.rows, p.cols), a[i]);
        unpack8<DT>(raw[i], d[i]);
#pragma unroll
        for (int j = 0; j < Raw8<DT>::kWords; j++) add_non_finite<DT>(odd, raw[i].w[j]);
      }
    }
#pragma unroll
    for (int i = 0; i < RP; i++) {
      const float s = descale_of(sb[i]);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const float2 h = __fmul2_rn(make_float2(a[i][j], a[i][j + 1]), both(s));
        float2 y, q, r;
        gate2<ACT, true>(h, y, q, r);
        const float2 g = act_grad2(h, r, make_float2(d[i][j], d[i][j + 1]));
        d[i][j] = g.x;
        d[i][j + 1] = g.y;
        const float2 v = act_value2(h, y, q);
        a[i][j] = v.x;
        a[i][j + 1] = v.y;
      }
    }
    if (was_non_finite<DT>(odd)) keep_infinite<DT>(p, row0, col0, a, d);
    if (p.dh_hp) store_tile<DT>(p.vec_dh, p.dh_hp, p.lddh, row0, col0, p.rows, p.cols, d);
    // the two column reductions share their barriers
    const bool dcols = p.dh.qt != nullptr, acols = p.aqt != nullptr;
    if (dcols) put_tile_maxima(d, sc[0]);
    if (acols) put_tile_maxima(a, sc[1]);
    if (p.dh.q) cast_tile_rows<OUT>(d, p.dh.q, p.dh.s, p.dh.ldq, row0, col0, p.rows, p.cols, gmax, p.margin);
    if (dcols || acols) {
      __syncthreads();
      bool bad = false;
      const int c = threadIdx.x & (kTile - 1);
      if (dcols && threadIdx.x < kTile) bad = finish_column(sc[0], c, p.dh.st, row0, col0, p.rows, gmax, p.margin);
      if (acols && threadIdx.x / kTile == 1)
        bad = finish_column(sc[1], c, p.ast, row0, col0, p.rows, kMaxE4M3, p.margin);
      bad = __syncthreads_or(bad);
      if (dcols) store_tile_cols<OUT>(d, sc[0], bad, p.dh.qt, p.dh.ldqt, row0, col0, p.rows, p.cols);
      if (acols) store_tile_cols<FP8_E4M3>(a, sc[1], bad, p.aqt, p.ldaqt, row0, col0, p.rows, p.cols);
    }
  }
}

}  // namespace block
}  // namespace fp8lib
