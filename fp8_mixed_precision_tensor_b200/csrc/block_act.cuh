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
// from 0 to 1:  SiLU g = s(h);  tanh GELU g = s(2 c (h + 0.044715 h^3)),
// c = sqrt(2/pi) (since (1 + tanh(u)) / 2 = s(2u));  GELU g = Phi(h).
// q = 1 - g is computed on its own (not by subtraction), so that the small
// one of the two keeps its relative accuracy, and dg = g'(h).  __expf: error
// at most 2 + 1.17 |x| units in the last place of a number that scales a
// value already far below 1.
struct Gate {
  float h;  // the argument, limited to +-110 (where exp(-|h|) is 0 in binary32)
  float g, q, dg;
};

template <int ACT>
__device__ __forceinline__ Gate gate_of(float h0) {
  Gate r;
  const float h = h0 > 110.0f ? 110.0f : (h0 < -110.0f ? -110.0f : h0);  // a NaN stays
  r.h = h;
  if constexpr (ACT == FP8_ACT_GELU_ERF) {
    const float z = fabsf(h) * 0.70710678118654752f;
    const float small = 0.5f * erfcf(z), big = 1.0f - small;
    r.g = h > 0.0f ? big : small;
    r.q = h > 0.0f ? small : big;
    r.dg = __expf(-z * z) * 0.39894228040143268f;
  } else {
    float u = h, du = 1.0f;
    if constexpr (ACT == FP8_ACT_GELU_TANH) {
      const float c = 1.5957691216057308f, h2 = h * h;  // 2 sqrt(2/pi)
      u = c * (h + 0.044715f * h2 * h);
      du = c + (3.0f * 0.044715f * c) * h2;
    }
    const float e = __expf(-fabsf(u));
    const float big = __fdividef(1.0f, 1.0f + e), small = e * big;
    r.g = h > 0.0f ? big : small;
    r.q = h > 0.0f ? small : big;
    r.dg = big * small * du;
  }
  return r;
}

// act(h).  For h > 0 the value h - h q lies below h, possibly by less than
// binary32 shows.  Rounded to nearest it would become h itself, and h, a
// 16-bit number, sits exactly on an FP8 rounding border one time in sixteen:
// the tie would then go to the even code where the true value goes to the
// lower one.  Rounding toward zero keeps it below; a q that has underflowed
// counts as the smallest normal number.
__device__ __forceinline__ float act_value(const Gate &t, float h) {
  constexpr float tiny = 1.17549435e-38f;
  if (h > 0.0f) return __fmaf_rz(-t.h, fmaxf(t.q, tiny), h);
  return t.h * t.g;
}

// da * act'(h), act' = g + h g' = 1 + r with r = h g' - q.  For h > 0 the
// product is da + da r, rounded to the side of da on which it lies, for the
// same reason (r is positive where both its terms have underflowed).
__device__ __forceinline__ float act_grad(const Gate &t, float h, float da) {
  constexpr float tiny = 1.17549435e-38f;
  if (h > 0.0f) {
    float r = __fmaf_rn(t.h, t.dg, -t.q);
    if (r == 0.0f) r = tiny;
    return (da > 0.0f) == (r > 0.0f) ? __fmaf_ru(da, r, da) : __fmaf_rd(da, r, da);
  }
  return da * __fmaf_rn(t.h, t.dg, t.g);
}

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
};

// HBM-bound: h is read once (2 B at 16 bits), one or two code bytes and / or
// a are written.  A row's 128-block is 16 neighbouring lanes, its amax four
// shuffles; nothing is shared between rows, so there is no barrier.
template <int DT, int ACT, bool VEC>
__global__ void __launch_bounds__(kCastThreads) k_act_fwd(const ActFwd p) {
  const int tiles_c = (p.cols + kTile - 1) / kTile;
  const long long tiles = (long long)((p.rows + kTile - 1) / kTile) * tiles_c;
  const int c8 = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  for (long long t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int row0 = (int)(t / tiles_c) * kTile, col0 = (int)(t % tiles_c) * kTile;
    const int col = col0 + c8 * 8;
#pragma unroll 2
    for (int i = 0; i < kRowsPer; i++) {
      const int row = row0 + r0 + 16 * i;
      float h[8], a[8];
      load8<DT, VEC>(p.h, p.ldh, row, col, p.rows, p.cols, h);
      uint32_t mh = 0, ma = 0;
#pragma unroll
      for (int j = 0; j < 8; j++) {
        a[j] = act_value(gate_of<ACT>(h[j]), h[j]);
        mh = max(mh, absbits_f32(h[j]));
        ma = max(ma, absbits_f32(a[j]));
      }
      mh = max16(mh);
      const int kh = block_exponent(mh, kMaxE4M3, p.margin);
      if (c8 == 0) put_scale(p.cs, row, col0 / kTile, tiles_c, kh);
      cast_row8<FP8_E4M3>(p.cq, p.ldc, row, col, p.rows, p.cols, h, pow2f(kh));
      if (p.aq) {
        ma = max16(ma);
        const int ka = block_exponent(ma, kMaxE4M3, p.margin);
        if (c8 == 0) put_scale(p.as, row, col0 / kTile, tiles_c, ka);
        cast_row8<FP8_E4M3>(p.aq, p.lda_q, row, col, p.rows, p.cols, a, pow2f(ka));
      }
      if (p.a) store8<DT, VEC>(p.a, p.lda, row, col, p.rows, p.cols, a);
    }
  }
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
};

// One pass over a 128x128 tile: 1 + 2 B read, up to 3 code bytes (or 2 B of
// dh) written.  dh and act(h') of the tile stay in registers between the
// amaxes and the encoding.  GFMT: format of dh's codes.
template <int DT, int ACT, int GFMT, bool VEC>
__global__ void __launch_bounds__(kCastThreads) k_act_bwd(const ActBwd p) {
  __shared__ ColScratch sc[2];
  const int tiles_c = (p.cols + kTile - 1) / kTile;
  const long long tiles = (long long)((p.rows + kTile - 1) / kTile) * tiles_c;
  const int kg = (tiles_c + 3) / 4;
  const float gmax = GFMT == FP8_E4M3 ? kMaxE4M3 : kMaxE5M2;
  const int c8 = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  for (long long t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int row0 = (int)(t / tiles_c) * kTile, col0 = (int)(t % tiles_c) * kTile;
    const int col = col0 + c8 * 8;
    float a[kRowsPer][8], d[kRowsPer][8];
#pragma unroll
    for (int i = 0; i < kRowsPer; i++) {
      const int row = row0 + r0 + 16 * i;
      load_codes8<FP8_E4M3>(p.cq, p.ldc, row, col, p.rows, p.cols, a[i]);
      load8<DT, VEC>(p.da, p.ldda, row, col, p.rows, p.cols, d[i]);
    }
#pragma unroll
    for (int i = 0; i < kRowsPer; i++) {
      const int row = row0 + r0 + 16 * i;
      const float s = row < p.rows ? descale_of(p.cs[scale_at(row, col0 / kTile, kg)]) : 1.0f;
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const float h = a[i][j] * s;
        const Gate t2 = gate_of<ACT>(h);
        a[i][j] = act_value(t2, h);
        d[i][j] = act_grad(t2, h, d[i][j]);
      }
      if (p.dh_hp) store8<DT, VEC>(p.dh_hp, p.lddh, row, col, p.rows, p.cols, d[i]);
    }
    if (p.dh.q) cast_tile_rows<GFMT>(d, p.dh.q, p.dh.s, p.dh.ldq, row0, col0, p.rows, p.cols, gmax, p.margin);
    if (p.dh.qt)
      cast_tile_cols<GFMT>(d, sc[0], p.dh.qt, p.dh.st, p.dh.ldqt, row0, col0, p.rows, p.cols, gmax, p.margin);
    if (p.aqt)
      cast_tile_cols<FP8_E4M3>(a, sc[1], p.aqt, p.ast, p.ldaqt, row0, col0, p.rows, p.cols, kMaxE4M3, p.margin);
  }
}

}  // namespace block
}  // namespace fp8lib
