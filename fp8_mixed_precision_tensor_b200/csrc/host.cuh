// host.cuh -- argument checks, dispatch and launches shared by the library's
// translation units.
#pragma once

#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include <type_traits>

#include "block_scale.cuh"

namespace fp8lib {
namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int cuda_rc(cudaError_t e) { return e == cudaSuccess ? FP8_OK : FP8_ERR_CUDA; }

template <typename K>
int set_smem(K kernel, int bytes) {
  return cuda_rc(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
}

constexpr int kOwnSmem = 2048;                // of a pass's kernel beside what a launch gives it, at the most
constexpr int kMostSmem = 232448 - kOwnSmem;  // of a launch
// Lets a kernel's launches take up to kMostSmem.  The limit is the kernel's, not
// a launch's: set to what one call needs it would refuse another thread's call
// between that one's setting and its launch.
template <typename K>
int allow_smem(K kernel) {
  return set_smem(kernel, kMostSmem);
}

bool valid_dtype(int dt) { return dt == FP8_DT_F32 || dt == FP8_DT_BF16 || dt == FP8_DT_F16; }

size_t dtype_bytes(int dt) { return dt == FP8_DT_F32 ? 4 : 2; }
bool fp8_fmt(int f) { return f == FP8_E4M3 || f == FP8_E5M2; }
// Kernels and launches round sizes up to tiles and groups of blocks in 32 bits (by 512 at the most).
bool too_long(int a, int b, int c = 0) {
  constexpr int kMost = INT_MAX - 1023;
  return a > kMost || b > kMost || c > kMost;
}
// A high-precision matrix argument: FP8_OK, or what is wrong with it.
int check_matrix(const void *p, int dtype, int cols, size_t ld) {
  if (!p || ld < (size_t)cols) return FP8_ERR_INVALID_ARG;
  return reinterpret_cast<uintptr_t>(p) % dtype_bytes(dtype) ? FP8_ERR_UNALIGNED : FP8_OK;
}
// Whether its rows start on 16-byte boundaries.
bool wide_rows(const void *p, int dtype, size_t ld) { return aligned16(p) && ld * dtype_bytes(dtype) % 16 == 0; }

int check_blocks(const fp8_blocks *b, int cols) {
  if (!b || !b->q || !b->s || b->ld < (size_t)cols) return FP8_ERR_INVALID_ARG;
  return aligned16(b->q) && aligned16(b->s) && b->ld % 16 == 0 ? FP8_OK : FP8_ERR_UNALIGNED;
}

// f(std::integral_constant<int, dtype>) for a runtime element type.
template <typename F>
void with_dtype(int dt, F f) {
  if (dt == FP8_DT_F32) f(std::integral_constant<int, FP8_DT_F32>());
  else if (dt == FP8_DT_BF16) f(std::integral_constant<int, FP8_DT_BF16>());
  else f(std::integral_constant<int, FP8_DT_F16>());
}
template <typename F>
void with_fmt(int fmt, F f) {
  if (fmt == FP8_E4M3) f(std::integral_constant<int, FP8_E4M3>());
  else f(std::integral_constant<int, FP8_E5M2>());
}
template <typename F>
void with_bool(bool b, F f) {
  if (b) f(std::true_type());
  else f(std::false_type());
}
// Launch with programmatic dependence on the stream's previous kernel (see
// pdl_wait); cluster > 1: clusters of that many CTAs.
template <typename... P, typename... A>
int launch_pdl(void (*kernel)(P...), unsigned grid, dim3 block, size_t smem, cudaStream_t stream, unsigned cluster,
               A... args) {
  if (grid == 0) return FP8_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cuda_rc(cudaLaunchKernelEx(&cfg, kernel, P(args)...));
}

// One CTA per 128x128 tile; 0 for more tiles than a grid can have (codes of 32 TB).
unsigned tile_grid(int rows, int cols) {
  const unsigned long long t = (unsigned long long)((rows + 127LL) / 128) * (unsigned long long)((cols + 127LL) / 128);
  return t <= 0x7fffffffull ? (unsigned)t : 0u;
}

block::CastOut cast_out(const fp8_blocks *row, const fp8_blocks *col) {
  block::CastOut o = {};
  if (row) { o.q = row->q; o.s = row->s; o.ldq = row->ld; }
  if (col) { o.qt = col->q; o.st = col->s; o.ldqt = col->ld; }
  return o;
}

}  // namespace
}  // namespace fp8lib

// passes.cu: reads and clears its status word on the stream; the caller waits for it.
extern "C" __attribute__((visibility("hidden"))) int passes_take_status(unsigned *host_out, cudaStream_t s);
