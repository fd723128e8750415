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

constexpr int kBlock = 128;

__host__ __device__ inline size_t scale_groups(int outer, int red) {
  const size_t rb = ((size_t)outer + 127) / 128, kb = ((size_t)red + 127) / 128;
  return rb * ((kb + 3) / 4);
}

// Address of the scale byte of outer index r, reduction block b; kgroups = ceil(KB/4).
__device__ __forceinline__ size_t scale_at(int r, int b, int kgroups) {
  return ((size_t)(r >> 7) * kgroups + (b >> 2)) * 512 + (r & 31) * 16 + ((r & 127) >> 5) * 4 + (b & 3);
}

// Exponent k of the scale 2^k of a block with this amax (bit pattern).
__device__ __forceinline__ int block_exponent(uint32_t amax_bits, float fmax, int margin) {
  int k;
  if (!scale_exponent(__uint_as_float(amax_bits), fmax, margin, 0, k)) atomicOr(&g_status, FP8_STATUS_NONFINITE);
  return k;
}

constexpr int kTile = 128;         // a cast tile is 128 x 128 elements
constexpr int kCastThreads = 256;  // 16 threads across (8 elements each) x 16 rows, 8 rows per thread
constexpr int kRowsPer = kTile / (kCastThreads / 16);

// Eight consecutive elements of row `row` from column `col` on as floats;
// elements outside [rows, cols) are 0.  VEC: rows start on 16-byte boundaries.
template <int DT, bool VEC>
__device__ __forceinline__ void load8(const void *base, size_t ld, int row, int col, int rows, int cols,
                                      float (&f)[8]) {
  if (row >= rows || col >= cols) {
#pragma unroll
    for (int j = 0; j < 8; j++) f[j] = 0.0f;
    return;
  }
  const size_t at = (size_t)row * ld + col;
  if (VEC && col + 8 <= cols) {
    if constexpr (DT == FP8_DT_F32) {
      const uint4 *p = reinterpret_cast<const uint4 *>(reinterpret_cast<const float *>(base) + at);
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const uint4 v = __ldcs(p + h);
        f[4 * h] = __uint_as_float(v.x);
        f[4 * h + 1] = __uint_as_float(v.y);
        f[4 * h + 2] = __uint_as_float(v.z);
        f[4 * h + 3] = __uint_as_float(v.w);
      }
    } else {
      const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(base) + at));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; k++) {
        if constexpr (DT == FP8_DT_BF16) {
          f[2 * k] = __uint_as_float(w[k] << 16);
          f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        } else {
          const float2 t = h2f2(w[k]);
          f[2 * k] = t.x;
          f[2 * k + 1] = t.y;
        }
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; j++) f[j] = col + j < cols ? load1<DT>(base, at + j) : 0.0f;
}

// Eight values as codes of FMT at scale s, to q[row, col...] (rows of ldq
// bytes, a multiple of 16; col a multiple of 8, so an 8-byte store is aligned).
template <int FMT>
__device__ __forceinline__ void store_codes8(uint8_t *q, size_t ldq, int row, int col, int rows, int cols,
                                             uint32_t lo, uint32_t hi) {
  if (row >= rows || col >= cols) return;
  uint8_t *p = q + (size_t)row * ldq + col;
  if (col + 8 <= cols) {
    __stcs(reinterpret_cast<uint2 *>(p), make_uint2(lo, hi));
    return;
  }
  const unsigned long long w = ((unsigned long long)hi << 32) | lo;
  for (int j = 0; j < cols - col; j++) p[j] = (uint8_t)(w >> (8 * j));
}

template <int FMT>
__device__ __forceinline__ void cast_row8(uint8_t *q, size_t ldq, int row, int col, int rows, int cols,
                                          const float (&f)[8], float s) {
  store_codes8<FMT>(q, ldq, row, col, rows, cols, enc4<FMT>(f[0] * s, f[1] * s, f[2] * s, f[3] * s),
                    enc4<FMT>(f[4] * s, f[5] * s, f[6] * s, f[7] * s));
}

template <int FMT>
__device__ __forceinline__ void cast_col8(uint8_t *q, size_t ldq, int row, int col, int rows, int cols,
                                          const float (&f)[8], const float (&s)[8]) {
  store_codes8<FMT>(q, ldq, row, col, rows, cols,
                    enc4<FMT>(f[0] * s[0], f[1] * s[1], f[2] * s[2], f[3] * s[3]),
                    enc4<FMT>(f[4] * s[4], f[5] * s[5], f[6] * s[6], f[7] * s[7]));
}

// Scale byte of (r, b) plus, behind the last block, the padding of its group of four.
__device__ __forceinline__ void put_scale(uint8_t *s, int r, int b, int kblocks, int k) {
  const int kg = (kblocks + 3) >> 2;
  uint8_t *p = s + scale_at(r, b, kg);
  *p = (uint8_t)(127 - k);
  if (b == kblocks - 1)
    for (int j = (b & 3) + 1; j < 4; j++) p[j - (b & 3)] = 127;
}

__device__ __forceinline__ uint32_t max16(uint32_t v) {  // over the 16 lanes of a row
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Where a cast writes: 1x128 blocks (q, s), 128x1 blocks (qt, st); either q may be null.
struct CastOut {
  uint8_t *q, *s;
  uint8_t *qt, *st;
  size_t ldq, ldqt;
};

// Scratch of the column reduction: 8 warps x 128 columns, then the 128 scales.
struct ColScratch {
  uint32_t part[kCastThreads / 32][kTile];
  float scale[kTile];
};

// The column side of a tile held in registers: v[i] = row r0 + 16 i, columns
// c8*8 .. +7 of the tile at (row0, col0).  Reduces |v| over the tile's rows,
// writes the 128 scale bytes, and encodes with them.
template <int FMT>
__device__ __forceinline__ void cast_tile_cols(const float (&v)[kRowsPer][8], ColScratch &sc, uint8_t *qt,
                                               uint8_t *st, size_t ldq, int row0, int col0, int rows, int cols,
                                               float fmax, int margin) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c8 = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  uint32_t m[8];
#pragma unroll
  for (int j = 0; j < 8; j++) {
    m[j] = 0;
#pragma unroll
    for (int i = 0; i < kRowsPer; i++) m[j] = max(m[j], absbits_f32(v[i][j]));
    m[j] = max(m[j], __shfl_xor_sync(0xffffffffu, m[j], 16));
  }
  if (lane < 16) {
    *reinterpret_cast<uint4 *>(&sc.part[warp][c8 * 8]) = make_uint4(m[0], m[1], m[2], m[3]);
    *reinterpret_cast<uint4 *>(&sc.part[warp][c8 * 8 + 4]) = make_uint4(m[4], m[5], m[6], m[7]);
  }
  __syncthreads();
  if (threadIdx.x < kTile) {
    uint32_t a = 0;
#pragma unroll
    for (int w = 0; w < kCastThreads / 32; w++) a = max(a, sc.part[w][threadIdx.x]);
    const int k = block_exponent(a, fmax, margin);
    sc.scale[threadIdx.x] = pow2f(k);
    put_scale(st, col0 + threadIdx.x, row0 / kTile, (rows + kTile - 1) / kTile, k);
  }
  __syncthreads();
  float s[8];
  *reinterpret_cast<float4 *>(&s[0]) = *reinterpret_cast<const float4 *>(&sc.scale[c8 * 8]);
  *reinterpret_cast<float4 *>(&s[4]) = *reinterpret_cast<const float4 *>(&sc.scale[c8 * 8 + 4]);
#pragma unroll
  for (int i = 0; i < kRowsPer; i++)
    cast_col8<FMT>(qt, ldq, row0 + r0 + 16 * i, col0 + c8 * 8, rows, cols, v[i], s);
}

// The row side of the same tile: one block per row, reduced over the row's 16 threads.
template <int FMT>
__device__ __forceinline__ void cast_tile_rows(const float (&v)[kRowsPer][8], uint8_t *q, uint8_t *s, size_t ldq,
                                               int row0, int col0, int rows, int cols, float fmax, int margin) {
  const int c8 = threadIdx.x & 15, r0 = threadIdx.x >> 4;
#pragma unroll
  for (int i = 0; i < kRowsPer; i++) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; j++) m = max(m, absbits_f32(v[i][j]));
    m = max16(m);
    const int k = block_exponent(m, fmax, margin);
    if (c8 == 0) put_scale(s, row0 + r0 + 16 * i, col0 / kTile, (cols + kTile - 1) / kTile, k);
    cast_row8<FMT>(q, ldq, row0 + r0 + 16 * i, col0 + c8 * 8, rows, cols, v[i], pow2f(k));
  }
}

// Cast of x [rows, cols] to 1x128 blocks and / or 128x1 blocks, x read once.
// Each CTA takes 128x128 tiles: the tile sits in registers (64 elements per
// thread), a row's amax is reduced over its 16 lanes, a column's over the
// thread's 8 rows and then through shared memory.  HBM-bound.
template <int DT, int FMT, bool VEC>
__global__ void __launch_bounds__(kCastThreads)
    k_block_cast(const void *__restrict__ x, int rows, int cols, size_t ldx, int margin, const CastOut out) {
  __shared__ ColScratch sc;
  const float fmax = FMT == FP8_E4M3 ? kMaxE4M3 : kMaxE5M2;
  const int tiles_c = (cols + kTile - 1) / kTile;
  const long long tiles = (long long)((rows + kTile - 1) / kTile) * tiles_c;
  const int c8 = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  for (long long t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int row0 = (int)(t / tiles_c) * kTile, col0 = (int)(t % tiles_c) * kTile;
    float v[kRowsPer][8];
#pragma unroll
    for (int i = 0; i < kRowsPer; i++)
      load8<DT, VEC>(x, ldx, row0 + r0 + 16 * i, col0 + c8 * 8, rows, cols, v[i]);
    if (out.q) cast_tile_rows<FMT>(v, out.q, out.s, out.ldq, row0, col0, rows, cols, fmax, margin);
    if (out.qt) cast_tile_cols<FMT>(v, sc, out.qt, out.st, out.ldqt, row0, col0, rows, cols, fmax, margin);
  }
}

// Cast of x to 128x128 blocks: one set of codes, the block's scale repeated
// for each of its rows (out.s) and each of its columns (out.st), so that the
// codes serve products that reduce along either axis.
template <int DT, int FMT, bool VEC>
__global__ void __launch_bounds__(kCastThreads)
    k_block_cast_square(const void *__restrict__ x, int rows, int cols, size_t ldx, int margin, const CastOut out) {
  __shared__ uint32_t red[32];
  const float fmax = FMT == FP8_E4M3 ? kMaxE4M3 : kMaxE5M2;
  const int tiles_c = (cols + kTile - 1) / kTile, tiles_r = (rows + kTile - 1) / kTile;
  const long long tiles = (long long)tiles_r * tiles_c;
  const int c8 = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  for (long long t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int row0 = (int)(t / tiles_c) * kTile, col0 = (int)(t % tiles_c) * kTile;
    float v[kRowsPer][8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kRowsPer; i++) {
      load8<DT, VEC>(x, ldx, row0 + r0 + 16 * i, col0 + c8 * 8, rows, cols, v[i]);
#pragma unroll
      for (int j = 0; j < 8; j++) m = max(m, absbits_f32(v[i][j]));
    }
    m = block_max_u32(m, red);
    const int k = block_exponent(m, fmax, margin);
    if (threadIdx.x < kTile) {
      const int r = row0 + threadIdx.x, c = col0 + threadIdx.x;
      put_scale(out.s, r, col0 / kTile, tiles_c, r < rows ? k : 0);
      put_scale(out.st, c, row0 / kTile, tiles_r, c < cols ? k : 0);
    }
    const float s = pow2f(k);
#pragma unroll
    for (int i = 0; i < kRowsPer; i++)
      cast_row8<FMT>(out.q, out.ldq, row0 + r0 + 16 * i, col0 + c8 * 8, rows, cols, v[i], s);
  }
}

// Eight codes as floats, descaled.
template <int FMT>
__device__ __forceinline__ void load_codes8(const uint8_t *q, size_t ldq, int row, int col, int rows, int cols,
                                            float (&f)[8]) {
  uint32_t w[2] = {0u, 0u};
  if (row < rows && col < cols) {
    const uint8_t *p = q + (size_t)row * ldq + col;
    if (col + 8 <= cols) {
      const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(p));
      w[0] = v.x;
      w[1] = v.y;
    } else {
      for (int j = 0; j < cols - col; j++) w[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
    }
  }
#pragma unroll
  for (int h = 0; h < 2; h++) {
    const float2 a = dec2<FMT>(w[h]), b = dec2<FMT>(w[h] >> 16);
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
template <int DT, bool VEC>
__device__ __forceinline__ void store8(void *out, size_t ld, int row, int col, int rows, int cols,
                                       const float (&f)[8]) {
  if (row >= rows || col >= cols) return;
  const size_t at = (size_t)row * ld + col;
  if constexpr (DT == FP8_DT_F32) {
    float *p = reinterpret_cast<float *>(out) + at;
    if (VEC && col + 8 <= cols) {
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
    if (VEC && col + 8 <= cols) {
      __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; j++)
      if (col + j < cols) p[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
  }
}

// Decode of blocked codes: x = dec(q) * 2^(byte - 127).  COLS: 128x1 blocks
// (scales of the transposed order), else 1x128 (or square) blocks.
template <int DT, int FMT, bool COLS, bool VEC>
__global__ void __launch_bounds__(kCastThreads)
    k_block_decode(const uint8_t *__restrict__ q, const uint8_t *__restrict__ s, int rows, int cols, size_t ldq,
                   void *__restrict__ x, size_t ldx) {
  const long long groups_c = (cols + 7) / 8;
  const long long groups = (long long)rows * groups_c;
  const int kg = COLS ? ((rows + 127) / 128 + 3) / 4 : ((cols + 127) / 128 + 3) / 4;
  for (long long g = (long long)blockIdx.x * blockDim.x + threadIdx.x; g < groups;
       g += (long long)gridDim.x * blockDim.x) {
    const int row = (int)(g / groups_c), col = (int)(g % groups_c) * 8;
    float f[8];
    load_codes8<FMT>(q, ldq, row, col, rows, cols, f);
    if constexpr (COLS) {
#pragma unroll
      for (int j = 0; j < 8; j++)
        if (col + j < cols) f[j] *= descale_of(s[scale_at(col + j, row >> 7, kg)]);
    } else {
      const float d = descale_of(s[scale_at(row, col >> 7, kg)]);
#pragma unroll
      for (int j = 0; j < 8; j++) f[j] *= d;
    }
    store8<DT, VEC>(x, ldx, row, col, rows, cols, f);
  }
}

}  // namespace block
}  // namespace fp8lib
