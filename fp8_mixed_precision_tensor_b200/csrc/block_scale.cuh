// block_scale.cuh -- power-of-two scales for blocks of 128 elements: their
// storage order, and the kernels that cast to and decode from such blocks.
//
// The per-tensor rule of "Training and inference of large language models
// using 8-bit floating point", 제안 방법 (the largest power of two that keeps
// the amax in range), applied to each 1x128, 128x1 or 128x128 block, so that
// an outlier costs only its own block precision.  A scale is kept as one
// byte, the biased exponent of the DEscale: value = dec(code) * 2^(byte-127)
// (the unsigned 8-bit exponent format of the tensor core's block-scaled
// products, which apply it in hardware).
//
// Order of the scale bytes of an operand with R outer indices and a reduction
// axis of C elements in KB = ceil(C/128) blocks: groups of 128 outer indices
// x 4 blocks, 512 bytes each, group (rb, kg) at (rb * ceil(KB/4) + kg) * 512;
// inside it the byte of outer index r, block b is at
//     (r % 32) * 16 + (r % 128 / 32) * 4 + b % 4.
// This is the order in which the tensor core wants them in tensor memory (32
// lanes x 16 bytes), so a product copies 512 bytes per 128 rows and 512
// elements of the reduction as they are; one 32-bit word holds a row's scales
// of four consecutive blocks and each MMA picks its byte.  Bytes of padding
// (r >= R, b >= KB) are 127 (a scale of 1).
#pragma once

#include "amax_cast.cuh"
#include "common.cuh"
#include "gemm.cuh"

namespace fp8lib {
namespace block {

__host__ __device__ inline size_t scale_groups(int outer, int red) {
  const size_t rb = ((size_t)outer + 127) / 128, kb = ((size_t)red + 127) / 128;
  return rb * ((kb + 3) / 4);
}

// Address of the scale byte of outer index r, reduction block b; kgroups = ceil(KB/4).
__device__ __forceinline__ size_t scale_at(int r, int b, int kgroups) {
  return ((size_t)(r >> 7) * kgroups + (b >> 2)) * 512 + (r & 31) * 16 + ((r & 127) >> 5) * 4 + (b & 3);
}

// Exponent k of the scale 2^k of a block with this amax (bit pattern).  For a
// normal amax 1.f 2^e and fmt_max = 1.75 2^E the rule's floor is E - e, less
// one where 1.f > 1.75: adding 2^23 - 1 - 0.75 2^23 to the bits carries into
// the exponent exactly then.  The rest (zero, subnormal, not finite) is rare
// and goes to the general rule.
__device__ __noinline__ int block_exponent_rare(uint32_t amax_bits, float fmax, int margin) {
  int k;
  if (!scale_exponent(__uint_as_float(amax_bits), fmax, margin, 0, k)) atomicOr(&g_status, FP8_STATUS_NONFINITE);
  return k;
}
__device__ __forceinline__ int block_exponent(uint32_t amax_bits, float fmax, int margin) {
  if (amax_bits - 0x00800000u >= 0x7f000000u) return block_exponent_rare(amax_bits, fmax, margin);
  const int top = (fmax == kMaxE4M3 ? 8 : 15) + 127;
  return clamp_exp(top - (int)((amax_bits + 0x1fffffu) >> 23) - margin);
}

// A cast tile is 128 x 128 elements: 16 threads across (8 elements each), RP
// rows per thread (rows r0 + i * 128 / RP), 16 * 128 / RP threads.
constexpr int kTile = 128;
constexpr int kCastThreads = 256;  // the plain casts: RP = 8
template <int RP>
struct Geo {
  static constexpr int kThreads = 16 * kTile / RP;
  static constexpr int kStep = kTile / RP;  // rows between a thread's rows
  static constexpr int kWarps = kThreads / 32;
};

// First row and column of tile t (row-major over tiles_c tiles across).
struct TileAt {
  int row0, col0;
};
__device__ __forceinline__ TileAt tile_at(unsigned t, unsigned tiles_c) {
  const unsigned r = t / tiles_c;
  return {(int)(r * kTile), (int)((t - r * tiles_c) * kTile)};
}

// Eight consecutive elements of a high-precision row as they are stored.
template <int DT>
struct __align__(16) Raw8 {
  static constexpr int kWords = DT == FP8_DT_F32 ? 8 : 4;
  uint32_t w[kWords];
};

// Whether a tile is read with 16-byte loads: rows start on 16-byte
// boundaries, and no group of eight elements straddles the row's end.
__device__ __forceinline__ bool wide_tile(bool vec, int col0, int cols) {
  return vec && (col0 + kTile <= cols || (cols & 7) == 0);
}

// Load of the eight elements at (row, col); those outside [rows, cols) are 0.
// The address is clamped instead of the load being skipped: without a branch
// around it, all of a thread's loads are in flight before the first is used.
// (Skipping with branches, the two-way cast of 8192 x 12288 bfloat16 took 234 us
// for 139.)
template <int DT>
__device__ __forceinline__ Raw8<DT> load_raw8_wide(const void *base, size_t ld, int row, int col, int rows,
                                                   int cols) {
  Raw8<DT> r;
  const bool in = row < rows && col < cols;
  const size_t at = (size_t)min(row, rows - 1) * ld + (col < cols ? col : 0);
  constexpr int esz = DT == FP8_DT_F32 ? 4 : 2;
  const uint4 *p = reinterpret_cast<const uint4 *>(reinterpret_cast<const uint8_t *>(base) + at * esz);
#pragma unroll
  for (int h = 0; h < Raw8<DT>::kWords / 4; h++) {
    const uint4 v = __ldcs(p + h);
    r.w[4 * h] = in ? v.x : 0u;
    r.w[4 * h + 1] = in ? v.y : 0u;
    r.w[4 * h + 2] = in ? v.z : 0u;
    r.w[4 * h + 3] = in ? v.w : 0u;
  }
  return r;
}

template <int DT>
__device__ __forceinline__ Raw8<DT> load_raw8_single(const void *base, size_t ld, int row, int col, int rows,
                                                     int cols) {
  Raw8<DT> r;
  const size_t at = (size_t)min(row, rows - 1) * ld;
  uint32_t e[8];
#pragma unroll
  for (int j = 0; j < 8; j++) {
    const size_t i = at + min(col + j, cols - 1);
    const uint32_t v = DT == FP8_DT_F32 ? __ldcs(reinterpret_cast<const uint32_t *>(base) + i)
                                        : (uint32_t)__ldcs(reinterpret_cast<const uint16_t *>(base) + i);
    e[j] = row < rows && col + j < cols ? v : 0u;
  }
#pragma unroll
  for (int j = 0; j < Raw8<DT>::kWords; j++) r.w[j] = DT == FP8_DT_F32 ? e[j] : e[2 * j] | (e[2 * j + 1] << 16);
  return r;
}

template <int DT>
__device__ __forceinline__ void unpack8(const Raw8<DT> &r, float (&f)[8]) {
#pragma unroll
  for (int j = 0; j < Raw8<DT>::kWords; j++) {
    if constexpr (DT == FP8_DT_F32) {
      f[j] = __uint_as_float(r.w[j]);
    } else if constexpr (DT == FP8_DT_BF16) {
      f[2 * j] = __uint_as_float(r.w[j] << 16);
      f[2 * j + 1] = __uint_as_float(r.w[j] & 0xffff0000u);
    } else {
      const float2 v = h2f2(r.w[j]);
      f[2 * j] = v.x;
      f[2 * j + 1] = v.y;
    }
  }
}

// A thread's part of a tile.
template <int DT, int RP>
__device__ __forceinline__ void load_tile(const void *x, size_t ld, bool vec, int row0, int col0, int rows, int cols,
                                          Raw8<DT> (&raw)[RP]) {
  const int row = row0 + (threadIdx.x >> 4), col = col0 + (threadIdx.x & 15) * 8;
  if (vec && row0 + kTile <= rows && col0 + kTile <= cols) {  // inside: nothing to clamp
    constexpr int esz = DT == FP8_DT_F32 ? 4 : 2;
    const uint8_t *p = reinterpret_cast<const uint8_t *>(x) + ((size_t)row * ld + col) * esz;
    const size_t step = (size_t)Geo<RP>::kStep * ld * esz;
#pragma unroll
    for (int i = 0; i < RP; i++, p += step)
#pragma unroll
      for (int h = 0; h < Raw8<DT>::kWords / 4; h++)
        *reinterpret_cast<uint4 *>(&raw[i].w[4 * h]) = __ldcs(reinterpret_cast<const uint4 *>(p) + h);
  } else if (wide_tile(vec, col0, cols)) {
#pragma unroll
    for (int i = 0; i < RP; i++) raw[i] = load_raw8_wide<DT>(x, ld, row + Geo<RP>::kStep * i, col, rows, cols);
  } else {
#pragma unroll
    for (int i = 0; i < RP; i++) raw[i] = load_raw8_single<DT>(x, ld, row + Geo<RP>::kStep * i, col, rows, cols);
  }
}

// Running maxima of magnitudes on the stored words: two 16-bit magnitudes per
// word, or one of 32 bits.  A NaN anywhere stays one.
template <int DT>
__device__ __forceinline__ uint32_t max_words(uint32_t m, uint32_t w) {
  uint32_t r;
  if constexpr (DT == FP8_DT_F32) {
    asm("{\n\t.reg .f32 t0;\n\tabs.f32 t0, %2;\n\tmax.NaN.f32 %0, %1, t0;\n\t}" : "=r"(r) : "r"(m), "r"(w));
  } else if constexpr (DT == FP8_DT_BF16) {
    asm("{\n\t.reg .b32 t0;\n\tabs.bf16x2 t0, %2;\n\tmax.NaN.bf16x2 %0, %1, t0;\n\t}" : "=r"(r) : "r"(m), "r"(w));
  } else {
    asm("{\n\t.reg .b32 t0;\n\tabs.f16x2 t0, %2;\n\tmax.NaN.f16x2 %0, %1, t0;\n\t}" : "=r"(r) : "r"(m), "r"(w));
  }
  return r;
}

// The binary32 bit pattern of a 16-bit magnitude.
template <int DT>
__device__ __forceinline__ uint32_t widen_abs(uint32_t h) {
  return DT == FP8_DT_BF16 ? h << 16 : absbits_f32(__half2float(__ushort_as_half((unsigned short)h)));
}

// The larger of a word's magnitudes as a binary32 bit pattern.
template <int DT>
__device__ __forceinline__ uint32_t word_abs(uint32_t m) {
  if constexpr (DT == FP8_DT_F32) return m;
  return widen_abs<DT>(max(m & 0xffffu, m >> 16));
}

// Running maximum of magnitudes over two floats; a NaN anywhere stays one and orders above inf as bits.
__device__ __forceinline__ float absmax2(float acc, float x, float y) {
  float r;
  asm("{\n\t.reg .f32 t0, t1;\n\tabs.f32 t0, %2;\n\tabs.f32 t1, %3;\n\tmax.NaN.f32 %0, %1, t0, t1;\n\t}"
      : "=f"(r)
      : "f"(acc), "f"(x), "f"(y));
  return r;
}

// enc4 for values none of which is NaN (a block with a finite amax): the
// saturating conversion alone.
// (Written out, so that the second pair is converted into the upper half of
// the first one's register: through cuda_fp8.h's 16-bit result each pair cost
// three more logic instructions.)
template <int FMT>
__device__ __forceinline__ uint32_t enc4_no_nan(float a, float b, float c, float d) {
  uint32_t r;
  if constexpr (FMT == FP8_E4M3)
    asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
  else
    asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e5m2x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e5m2x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// Four codes as floats.
template <int FMT>
__device__ __forceinline__ void dec4(uint32_t w, float2 &a, float2 &b) {
  uint32_t x, y;
  if constexpr (FMT == FP8_E4M3)
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(x), "=r"(y)
        : "r"(w));
  else
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e5m2x2 %0, lo;\n\t"
        "cvt.rn.f16x2.e5m2x2 %1, hi;\n\t}"
        : "=r"(x), "=r"(y)
        : "r"(w));
  a = h2f2(x);
  b = h2f2(y);
}

// f * s as codes, none of them NaN / any value.
template <int FMT>
__device__ __forceinline__ uint2 enc8(const float (&f)[8], const float2 (&s)[4]) {
  float2 y[4];
#pragma unroll
  for (int j = 0; j < 4; j++) y[j] = __fmul2_rn(make_float2(f[2 * j], f[2 * j + 1]), s[j]);
  return make_uint2(enc4_no_nan<FMT>(y[0].x, y[0].y, y[1].x, y[1].y), enc4_no_nan<FMT>(y[2].x, y[2].y, y[3].x, y[3].y));
}
template <int FMT>
__device__ __forceinline__ uint2 enc8_any(const float (&f)[8], const float2 (&s)[4]) {
  float2 y[4];
#pragma unroll
  for (int j = 0; j < 4; j++) y[j] = __fmul2_rn(make_float2(f[2 * j], f[2 * j + 1]), s[j]);
  return make_uint2(enc4<FMT>(y[0].x, y[0].y, y[1].x, y[1].y), enc4<FMT>(y[2].x, y[2].y, y[3].x, y[3].y));
}

// A thread's RP groups of eight codes to q (rows of ldq bytes, a multiple of
// 16; col a multiple of 8, so an 8-byte store is aligned).  One predicate per
// row; the group that straddles the row's end is stored apart.
template <int RP>
__device__ __forceinline__ void store_codes(uint8_t *q, size_t ldq, int row0, int col, int rows, int cols,
                                            const uint2 (&o)[RP]) {
  const int row = row0 + (threadIdx.x >> 4);
  uint8_t *p = q + (size_t)row * ldq + col;
  const int left = col + 8 <= cols ? rows - row : 0;  // rows that take whole groups
  const size_t step = (size_t)Geo<RP>::kStep * ldq;
  uint8_t *w = p;
#pragma unroll
  for (int i = 0; i < RP; i++, w += step)
    if (i * Geo<RP>::kStep < left) __stcs(reinterpret_cast<uint2 *>(w), o[i]);
  if (col < cols && col + 8 > cols) {
#pragma unroll 1
    for (int j = 0; j < cols - col; j++)
#pragma unroll
      for (int i = 0; i < RP; i++)
        if (row + i * Geo<RP>::kStep < rows)
          p[i * step + j] = (uint8_t)((j < 4 ? o[i].x : o[i].y) >> (8 * (j & 3)));
  }
}

// Scale byte of (r, b) plus, behind the last block, the padding of its group of four.
__device__ __forceinline__ void put_scale(uint8_t *s, int r, int b, int kblocks, int k) {
  const int kg = (kblocks + 3) >> 2;
  uint8_t *p = s + scale_at(r, b, kg);
  *p = (uint8_t)(127 - k);
  if (b == kblocks - 1)
    for (int j = (b & 3) + 1; j < 4; j++) p[j - (b & 3)] = 127;
}

// Where a cast writes: 1x128 blocks (q, s), 128x1 blocks (qt, st).
struct CastOut {
  uint8_t *q, *s;
  uint8_t *qt, *st;
  size_t ldq, ldqt;
};

// Scratch of a column reduction: the warps' maxima, then the 128 scales.
template <int RP>
struct ColScratch {
  uint32_t part[Geo<RP>::kWarps][kTile];
  float scale[kTile];
};

// From the warps' maxima (binary32 bit patterns in sc.part) to the tile's 128
// column scales: written to st, and to sc.scale.  Called by 128 threads, c the
// column of each; returns whether its amax is not finite.
template <int RP>
__device__ __forceinline__ bool finish_column(ColScratch<RP> &sc, int c, uint8_t *st, int row0, int col0, int rows,
                                              float fmax, int margin) {
  uint32_t a = 0;
#pragma unroll
  for (int w = 0; w < Geo<RP>::kWarps; w++) a = max(a, sc.part[w][c]);
  const int k = block_exponent(a, fmax, margin);
  sc.scale[c] = pow2f(k);
  put_scale(st, col0 + c, row0 / kTile, (rows + kTile - 1) / kTile, k);
  return a >= 0x7f800000u;
}

// The thread's eight column scales.
template <int RP>
__device__ __forceinline__ void get_column_scales(const ColScratch<RP> &sc, float2 (&s)[4]) {
  const int c8 = threadIdx.x & 15;
  *reinterpret_cast<float4 *>(&s[0]) = *reinterpret_cast<const float4 *>(&sc.scale[c8 * 8]);
  *reinterpret_cast<float4 *>(&s[2]) = *reinterpret_cast<const float4 *>(&sc.scale[c8 * 8 + 4]);
}

// The same for one tile, by all threads: the thread's scales to s.
template <int RP>
__device__ __forceinline__ bool column_scales(ColScratch<RP> &sc, uint8_t *st, int row0, int col0, int rows, float fmax,
                                              int margin, float2 (&s)[4]) {
  __syncthreads();
  const bool bad = threadIdx.x < kTile && finish_column(sc, threadIdx.x, st, row0, col0, rows, fmax, margin);
  const bool any = __syncthreads_or(bad);
  get_column_scales(sc, s);
  return any;
}

// A warp's eight column maxima per thread (lanes l and l + 16 hold the same columns) to sc.part.
template <int RP>
__device__ __forceinline__ void put_column_maxima(ColScratch<RP> &sc, uint32_t (&m)[8]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c8 = threadIdx.x & 15;
#pragma unroll
  for (int j = 0; j < 8; j++) m[j] = max(m[j], __shfl_xor_sync(0xffffffffu, m[j], 16));
  if (lane < 16) {
    *reinterpret_cast<uint4 *>(&sc.part[warp][c8 * 8]) = make_uint4(m[0], m[1], m[2], m[3]);
    *reinterpret_cast<uint4 *>(&sc.part[warp][c8 * 8 + 4]) = make_uint4(m[4], m[5], m[6], m[7]);
  }
}

// The column side of a tile of floats held in registers (v[i] = row r0 + i *
// Geo<RP>::kStep, columns c8*8 .. +7 of the tile at (row0, col0)): the maxima,
// and, once the scales are there, the codes.
template <int RP>
__device__ __forceinline__ void put_tile_maxima(const float (&v)[RP][8], ColScratch<RP> &sc) {
  uint32_t m[8];
#pragma unroll
  for (int j = 0; j < 8; j++) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < RP; i += 2) a = absmax2(a, v[i][j], v[i + 1][j]);
    m[j] = __float_as_uint(a);
  }
  put_column_maxima(sc, m);
}
template <int FMT, int RP>
__device__ __forceinline__ void store_tile_cols(const float (&v)[RP][8], const ColScratch<RP> &sc, bool bad,
                                                uint8_t *qt, size_t ldq, int row0, int col0, int rows, int cols) {
  float2 s[4];
  get_column_scales(sc, s);
  uint2 o[RP];
#pragma unroll
  for (int i = 0; i < RP; i++) o[i] = enc8<FMT>(v[i], s);
  if (bad) {
#pragma unroll
    for (int i = 0; i < RP; i++) o[i] = enc8_any<FMT>(v[i], s);
  }
  store_codes(qt, ldq, row0, col0 + (threadIdx.x & 15) * 8, rows, cols, o);
}

// The scales of a thread's RP row blocks: m[i] is the thread's maximum of its
// i-th row (a binary32 bit pattern), a row's 16 lanes each hold one.  Halving
// exchanges leave each group of 16 / RP lanes with one finished row (lane l of
// the 16 with row l * RP / 16), which computes and writes that row's scale; RP
// broadcasts return all of them.  Half the shuffles of separate reductions,
// one scale computation per thread instead of RP, and nothing to branch over:
// the separate form took 139 instead of 95 us for 8192 x 12288 bf16 in both
// directions.  Returns whether the warp saw an amax that is not finite.
template <int RP>
__device__ __forceinline__ uint32_t reduce_rows(const uint32_t (&m)[RP], int l) {
  static_assert((RP & (RP - 1)) == 0 && RP <= 8, "halved down to one row");
  uint32_t v[RP];
#pragma unroll
  for (int i = 0; i < RP; i++) v[i] = m[i];
  int bit = 8;
#pragma unroll
  for (int n = RP / 2; n > 0; n /= 2, bit /= 2) {
#pragma unroll
    for (int i = 0; i < n; i++) {
      const uint32_t send = (l & bit) ? v[i] : v[i + n], keep = (l & bit) ? v[i + n] : v[i];
      v[i] = max(keep, __shfl_xor_sync(0xffffffffu, send, bit));
    }
  }
#pragma unroll
  for (; bit > 0; bit /= 2) v[0] = max(v[0], __shfl_xor_sync(0xffffffffu, v[0], bit));
  return v[0];
}

template <int RP>
__device__ __forceinline__ bool row_scales(const uint32_t (&m)[RP], uint8_t *s, int row0, int col0, int tiles_c,
                                           float fmax, int margin, float (&out)[RP]) {
  const int lane = threadIdx.x & 31, l = lane & 15, r0 = threadIdx.x >> 4;
  const uint32_t v = reduce_rows<RP>(m, l);
  const int k = block_exponent(v, fmax, margin);
  if (l % (16 / RP) == 0) put_scale(s, row0 + r0 + Geo<RP>::kStep * (l * RP / 16), col0 / kTile, tiles_c, k);
  const float own = pow2f(k);
#pragma unroll
  for (int i = 0; i < RP; i++) out[i] = __shfl_sync(0xffffffffu, own, (lane & 16) + i * (16 / RP));
  return __any_sync(0xffffffffu, v >= 0x7f800000u);
}

// One scale as the four pairs of a group.
__device__ __forceinline__ void spread_scale(float s, float2 (&o)[4]) {
#pragma unroll
  for (int j = 0; j < 4; j++) o[j] = both(s);
}

// The row side of the same tile of floats.
template <int FMT, int RP>
__device__ __forceinline__ void cast_tile_rows(const float (&v)[RP][8], uint8_t *q, uint8_t *s, size_t ldq,
                                               int row0, int col0, int rows, int cols, float fmax, int margin) {
  uint32_t m[RP];
#pragma unroll
  for (int i = 0; i < RP; i++) {
    float a = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; j += 2) a = absmax2(a, v[i][j], v[i][j + 1]);
    m[i] = __float_as_uint(a);
  }
  float sc[RP];
  const bool nan = row_scales(m, s, row0, col0, (cols + kTile - 1) / kTile, fmax, margin, sc);
  uint2 o[RP];
#pragma unroll
  for (int i = 0; i < RP; i++) {
    float2 s4[4];
    spread_scale(sc[i], s4);
    o[i] = enc8<FMT>(v[i], s4);
  }
  if (nan) {
#pragma unroll
    for (int i = 0; i < RP; i++) {
      float2 s4[4];
      spread_scale(sc[i], s4);
      o[i] = enc8_any<FMT>(v[i], s4);
    }
  }
  store_codes(q, ldq, row0, col0 + (threadIdx.x & 15) * 8, rows, cols, o);
}

// A tile of elements as stored, encoded with one scale per row (sc) or per column pair (s4).
template <int DT, int FMT, int RP>
__device__ __forceinline__ void store_raw_rows(const Raw8<DT> (&raw)[RP], const float (&sc)[RP], bool nan, uint8_t *q,
                                               size_t ldq, int row0, int col, int rows, int cols) {
  uint2 o[RP];
#pragma unroll
  for (int i = 0; i < RP; i++) {
    float f[8];
    float2 s4[4];
    unpack8<DT>(raw[i], f);
    spread_scale(sc[i], s4);
    o[i] = enc8<FMT>(f, s4);
  }
  if (nan) {
#pragma unroll
    for (int i = 0; i < RP; i++) {
      float f[8];
      float2 s4[4];
      unpack8<DT>(raw[i], f);
      spread_scale(sc[i], s4);
      o[i] = enc8_any<FMT>(f, s4);
    }
  }
  store_codes(q, ldq, row0, col, rows, cols, o);
}

// The row side of a tile of elements as stored.
template <int DT, int FMT, int RP>
__device__ __forceinline__ void cast_raw_rows(const Raw8<DT> (&raw)[RP], uint8_t *q, uint8_t *s, size_t ldq,
                                              int row0, int col0, int rows, int cols, float fmax, int margin) {
  uint32_t m[RP];
#pragma unroll
  for (int i = 0; i < RP; i++) {
    m[i] = 0;
#pragma unroll
    for (int j = 0; j < Raw8<DT>::kWords; j++) m[i] = max_words<DT>(m[i], raw[i].w[j]);
    m[i] = word_abs<DT>(m[i]);
  }
  float sc[RP];
  const bool nan = row_scales(m, s, row0, col0, (cols + kTile - 1) / kTile, fmax, margin, sc);
  store_raw_rows<DT, FMT>(raw, sc, nan, q, ldq, row0, col0 + (threadIdx.x & 15) * 8, rows, cols);
}

// The kernels without blocks along the rows need nothing of a tile but its
// rows.  Their CTAs take a part of one.  RP rows per thread, 4 or 2: 128 threads
// of the 128 * 16 / RP that a whole tile would have; CTAs this small leave and
// are replaced one by one (4096 x 16384 bfloat16: forward 70 and 62 us in CTAs
// of 512 and 128 threads, with codes 71 and 60).  RP = 1, 512 threads with a row
// each, where there are no more tiles than SMs: a CTA then runs its code once,
// and a quarter of it is fetched sooner (500 x 2056 float32: forward 7.0 and 2.9
// us, backward 7.1 and 3.3).
template <int RP>
constexpr int kPartThreads = RP == 1 ? 512 : 128;
template <int RP>
constexpr int kParts = RP == 2 ? 8 : 4;  // of a tile
template <int RP>
__device__ __forceinline__ TileAt part_at(unsigned t, unsigned tiles_c) {
  if constexpr (RP == 1) {
    const unsigned r = t / tiles_c;
    return {(int)(r * 32), (int)((t - r * tiles_c) * kTile)};
  }
  TileAt at = tile_at(t / kParts<RP>, tiles_c);
  at.row0 += (int)(t % kParts<RP>) * 8;
  return at;
}

// Cast of x [rows, cols] to 1x128 blocks, 2 B read and 1 written per 16-bit
// element: 8192 x 12288 bfloat16 52 us (5.8 TB/s), 4096 x 4096 7.8, 1003 x 4104 3.1
// (4.4 in CTAs of a whole tile), 256 x 256 1.7 (2.3).
template <int DT, int FMT, int RP>
__global__ void __launch_bounds__(kPartThreads<RP>, 1024 / kPartThreads<RP>)
    k_block_cast_rows(const void *__restrict__ x, int rows, int cols, size_t ldx, int vec, int margin,
                      const CastOut out) {
  pdl_launch_dependents();
  pdl_wait();
  const auto [row0, col0] = part_at<RP>(blockIdx.x, (cols + kTile - 1) / kTile);
  Raw8<DT> raw[RP];
  load_tile<DT>(x, ldx, vec, row0, col0, rows, cols, raw);
  cast_raw_rows<DT, FMT>(raw, out.q, out.s, out.ldq, row0, col0, rows, cols, FMT == FP8_E4M3 ? kMaxE4M3 : kMaxE5M2,
                         margin);
}

// Cast of x to 128x1 blocks and, if wanted, to 1x128 blocks, x read once.
// Each CTA takes one 128x128 tile: it sits in registers as stored (64
// elements per thread), a row's amax is reduced over its 16 lanes, a column's
// over the thread's 8 rows and then through shared memory.  2 B read and 1 B
// written per direction and 16-bit element; 8192 x 12288 bfloat16 both ways 71
// to 91 us (5.7 to 4.4 TB/s).  Half of the issue slots and half of
// the DRAM cycles are busy: three CTAs hide a tile's latencies only in part.
// RP = 2 (1024 threads) where there are no more tiles than SMs: a CTA then runs
// its code once, and a quarter of it is fetched sooner (both ways, 777 x 1305 bfloat16: 6.6 and
// 4.7 us; 1024 x 2048: 5.4 and 3.4).
template <int DT, int FMT, int RP>
__global__ void __launch_bounds__(Geo<RP>::kThreads, RP == 2 ? 1 : DT == FP8_DT_F32 ? 2 : 3)
    k_block_cast(const void *__restrict__ x, int rows, int cols, size_t ldx, int vec, int margin, const CastOut out) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ ColScratch<RP> sc;
  const float fmax = FMT == FP8_E4M3 ? kMaxE4M3 : kMaxE5M2;
  const auto [row0, col0] = tile_at(blockIdx.x, (cols + kTile - 1) / kTile);
  Raw8<DT> raw[RP];
  load_tile<DT>(x, ldx, vec, row0, col0, rows, cols, raw);
  // the column maxima go out first: their barriers overlap the row side
  uint32_t w[Raw8<DT>::kWords], m[8];
#pragma unroll
  for (int j = 0; j < Raw8<DT>::kWords; j++) {
    w[j] = 0;
#pragma unroll
    for (int i = 0; i < RP; i++) w[j] = max_words<DT>(w[j], raw[i].w[j]);
    if constexpr (DT == FP8_DT_F32) {
      m[j] = w[j];
    } else {
      m[2 * j] = widen_abs<DT>(w[j] & 0xffffu);
      m[2 * j + 1] = widen_abs<DT>(w[j] >> 16);
    }
  }
  put_column_maxima(sc, m);
  if (out.q) cast_raw_rows<DT, FMT>(raw, out.q, out.s, out.ldq, row0, col0, rows, cols, fmax, margin);
  float2 s[4];
  const bool bad = column_scales(sc, out.st, row0, col0, rows, fmax, margin, s);
  uint2 o[RP];
#pragma unroll
  for (int i = 0; i < RP; i++) {
    float f[8];
    unpack8<DT>(raw[i], f);
    o[i] = enc8<FMT>(f, s);
  }
  if (bad) {
#pragma unroll
    for (int i = 0; i < RP; i++) {
      float f[8];
      unpack8<DT>(raw[i], f);
      o[i] = enc8_any<FMT>(f, s);
    }
  }
  store_codes(out.qt, out.ldqt, row0, col0 + (threadIdx.x & 15) * 8, rows, cols, o);
}

// Cast of x to 128x128 blocks: one set of codes, the block's scale repeated
// for each of its rows (out.s) and each of its columns (out.st), so that the
// codes serve products that reduce along either axis.  HBM-bound: 12288 x 12288
// bfloat16 73 us (6.2 TB/s); at the three CTAs per SM of more registers 89.
template <int DT, int FMT, int RP>
__global__ void __launch_bounds__(Geo<RP>::kThreads, RP == 2 ? 1 : DT == FP8_DT_F32 ? 2 : 4)
    k_block_cast_square(const void *__restrict__ x, int rows, int cols, size_t ldx, int vec, int margin,
                        const CastOut out) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ uint32_t red[32];
  const float fmax = FMT == FP8_E4M3 ? kMaxE4M3 : kMaxE5M2;
  const int tiles_c = (cols + kTile - 1) / kTile, tiles_r = (rows + kTile - 1) / kTile;
  const auto [row0, col0] = tile_at(blockIdx.x, tiles_c);
  Raw8<DT> raw[RP];
  load_tile<DT>(x, ldx, vec, row0, col0, rows, cols, raw);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < RP; i++)
#pragma unroll
    for (int j = 0; j < Raw8<DT>::kWords; j++) w = max_words<DT>(w, raw[i].w[j]);
  const uint32_t m = block_max_u32(word_abs<DT>(w), red);
  const int k = block_exponent(m, fmax, margin);
  if (threadIdx.x < kTile) {
    const int r = row0 + threadIdx.x, c = col0 + threadIdx.x;
    put_scale(out.s, r, col0 / kTile, tiles_c, r < rows ? k : 0);
    put_scale(out.st, c, row0 / kTile, tiles_r, c < cols ? k : 0);
  }
  float sc[RP];
#pragma unroll
  for (int i = 0; i < RP; i++) sc[i] = pow2f(k);
  store_raw_rows<DT, FMT>(raw, sc, m >= 0x7f800000u, out.q, out.ldq, row0, col0 + (threadIdx.x & 15) * 8, rows, cols);
}

// Eight codes at (row, col), 0 outside [rows, cols).
__device__ __forceinline__ uint2 load_codes8(const uint8_t *q, size_t ldq, int row, int col, int rows, int cols) {
  const uint8_t *p = q + (size_t)min(row, rows - 1) * ldq;
  uint2 v;
  if (col + 8 <= cols || (col >= cols && cols >= 8)) {  // as load_raw8_wide: clamped, not skipped
    v = __ldcs(reinterpret_cast<const uint2 *>(p + (col < cols ? col : 0)));
    if (row >= rows || col >= cols) v = make_uint2(0u, 0u);
  } else {
    uint32_t w[2] = {0u, 0u};
    for (int j = 0; j < cols - col; j++) w[j >> 2] |= (uint32_t)p[col + j] << (8 * (j & 3));
    v = row < rows ? make_uint2(w[0], w[1]) : make_uint2(0u, 0u);
  }
  return v;
}

template <int FMT>
__device__ __forceinline__ void decode8(uint2 v, float (&f)[8]) {
  const uint32_t w[2] = {v.x, v.y};
#pragma unroll
  for (int h = 0; h < 2; h++) {
    float2 a, b;
    dec4<FMT>(w[h], a, b);
    f[4 * h] = a.x;
    f[4 * h + 1] = a.y;
    f[4 * h + 2] = b.x;
    f[4 * h + 3] = b.y;
  }
}

// 2^(byte - 127), byte 0 included (a binary32 subnormal).
__device__ __forceinline__ float descale_of(uint32_t byte) {
  return byte == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
}

// Eight floats rounded to DT and stored at out[row, col...].
template <int DT>
__device__ __forceinline__ void store8(bool vec, void *out, size_t ld, int row, int col, int rows, int cols,
                                       const float (&f)[8]) {
  if (row >= rows || col >= cols) return;
  const size_t at = (size_t)row * ld + col;
  if constexpr (DT == FP8_DT_F32) {
    float *p = reinterpret_cast<float *>(out) + at;
    if (vec && col + 8 <= cols) {
      __stcs(reinterpret_cast<float4 *>(p), make_float4(f[0], f[1], f[2], f[3]));
      __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; j++)
      if (col + j < cols) p[j] = f[j];
  } else {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
      if constexpr (DT == FP8_DT_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t *>(&h);
      } else if constexpr (DT == FP8_DT_BF16_RTO) {
        w[k] = gemm::bf16x2_rto(f[2 * k], f[2 * k + 1]);
      } else {
        w[k] = f16x2(f[2 * k], f[2 * k + 1]);
      }
    }
    uint16_t *p = reinterpret_cast<uint16_t *>(out) + at;
    if (vec && col + 8 <= cols) {
      __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; j++)
      if (col + j < cols) p[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
  }
}

// Eight floats rounded to DT as 16-byte words.
template <int DT>
__device__ __forceinline__ void pack8(const float (&f)[8], uint4 (&w)[DT == FP8_DT_F32 ? 2 : 1]) {
  if constexpr (DT == FP8_DT_F32) {
    w[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    w[1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
  } else {
    uint32_t h[4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
      if constexpr (DT == FP8_DT_BF16) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
        h[k] = *reinterpret_cast<const uint32_t *>(&b);
      } else {
        h[k] = f16x2(f[2 * k], f[2 * k + 1]);
      }
    }
    w[0] = make_uint4(h[0], h[1], h[2], h[3]);
  }
}

// A thread's part of a tile of floats, rounded to DT.
template <int DT, int RP>
__device__ __forceinline__ void store_tile(bool vec, void *out, size_t ld, int row0, int col0, int rows, int cols,
                                           const float (&f)[RP][8]) {
  const int row = row0 + (threadIdx.x >> 4), col = col0 + (threadIdx.x & 15) * 8;
  if (wide_tile(vec, col0, cols)) {
    constexpr int esz = DT == FP8_DT_F32 ? 4 : 2;
    uint8_t *p = reinterpret_cast<uint8_t *>(out) + ((size_t)row * ld + col) * esz;
    const int left = col < cols ? rows - row : 0;
#pragma unroll
    for (int i = 0; i < RP; i++) {
      uint4 w[DT == FP8_DT_F32 ? 2 : 1];
      pack8<DT>(f[i], w);
      if (i * Geo<RP>::kStep < left) {
        uint4 *q = reinterpret_cast<uint4 *>(p + (size_t)(i * Geo<RP>::kStep) * ld * esz);
        __stcs(q, w[0]);
        if constexpr (DT == FP8_DT_F32) __stcs(q + 1, w[1]);
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < RP; i++) store8<DT>(false, out, ld, row + i * Geo<RP>::kStep, col, rows, cols, f[i]);
}

// Decode of blocked codes: x = dec(q) * 2^(byte - 127).  COLS: 128x1 blocks
// (scales of the transposed order), else 1x128 (or square) blocks.  1 B read and
// 2 written: 8192 x 12288 to bfloat16 70 us (4.3 TB/s; two thirds of the issue
// slots busy, with a 64-bit division per eight elements), from 128x1 blocks 152,
// where each element has a scale byte of its own to fetch.  No product and no
// pass of a layer goes through it.
template <int DT, int FMT, bool COLS>
__global__ void __launch_bounds__(kCastThreads)
    k_block_decode(const uint8_t *__restrict__ q, const uint8_t *__restrict__ s, int rows, int cols, size_t ldq,
                   void *__restrict__ x, size_t ldx, int vec) {
  pdl_launch_dependents();
  pdl_wait();
  const long long groups_c = (cols + 7) / 8;
  const long long groups = (long long)rows * groups_c;
  const int kg = COLS ? ((rows + 127) / 128 + 3) / 4 : ((cols + 127) / 128 + 3) / 4;
  for (long long g = (long long)blockIdx.x * blockDim.x + threadIdx.x; g < groups;
       g += (long long)gridDim.x * blockDim.x) {
    const int row = (int)(g / groups_c), col = (int)(g % groups_c) * 8;
    float f[8];
    decode8<FMT>(load_codes8(q, ldq, row, col, rows, cols), f);
    if constexpr (COLS) {
#pragma unroll
      for (int j = 0; j < 8; j++)
        if (col + j < cols) f[j] *= descale_of(s[scale_at(col + j, row >> 7, kg)]);
    } else {
      const float d = descale_of(s[scale_at(row, col >> 7, kg)]);
#pragma unroll
      for (int j = 0; j < 8; j++) f[j] *= d;
    }
    store8<DT>(vec, x, ldx, row, col, rows, cols, f);
  }
}

}  // namespace block
}  // namespace fp8lib
