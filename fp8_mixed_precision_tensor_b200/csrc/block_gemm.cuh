// block_gemm.cuh -- FP8 products whose operands carry one power-of-two scale
// per block of 128 along the reduction, on the 5th-generation tensor cores.
//
//   C[r, c] = sum_b 2^(sa[r,b] + sb[c,b] - 254) sum_{k in block b} A(r, k) B(c, k)   (+ bias)
//
// tcgen05.mma kind::mxf8f6f4 takes a scale byte per row and 32 elements of
// the reduction from tensor memory and applies it while it multiplies, at the
// rate of the unscaled FP8 product.  A block of 128 is four such groups with
// the same byte: the packed scale words (see block_scale.cuh) are copied to
// tensor memory once per four blocks, and the four MMAs of a block name the
// block's byte (the instruction descriptor's scale ids).  The accumulator
// therefore holds the finished product: no partial sums leave the tensor
// core, and the epilogue only rounds.  Operand layouts, TMA rings, bounded
// waits and the abort protocol are those of gemm.cuh.
//
// "Training and inference of large language models using 8-bit floating
// point", 제안 방법 (scale, cast, multiply, undo the scale), per block.
#pragma once

#include "block_scale.cuh"
#include "gemm.cuh"

namespace fp8lib {
namespace bgemm {

using namespace gemm;

struct BArgs {
  int rows, cols;              // output extent along A's and B's outer indices
  int num_m_blocks, num_n_blocks, num_tiles, num_k_blocks, group_m;
  int whole;                   // pair kernel: tiles from this one on are worked as two halves of 128 columns
  int bn;                      // token kernels: tokens of the tile (a multiple of 16)
  int stages;                  // token kernels: ring depth
  uint32_t stage_bytes, tmem_cols;
  uint32_t idesc, desc_hi;
  const void *bias;            // per output feature, or null
  int bias_dtype;
  void *out;                   // pair kernel: [rows, cols]; token kernels: [cols, rows] (A holds the features)
  int out_dtype;
  size_t ld_out;               // elements
  int vec_out;                 // rows of `out` start on 16-byte boundaries
  // tokens cast in the kernel: x [cols, x_cols]
  const void *x;
  size_t ldx;
  int x_cols, x_vec, margin;
};

// Shared-memory descriptors of the block-scaled MMAs are passed as two words:
// the low one (address and leading offset) advances by 32-bit adds that cannot
// carry, the high one (stride, version, swizzle) comes from the kernel's
// arguments.  With 64-bit descriptors of constant high part in unrolled
// cta_group::2 MMAs this compiler (ptxas 12.9.86) gave the instruction wrong
// descriptors, depending on the code around it: every row was multiplied with
// the first rows' data, at the right scales.
constexpr uint32_t kDescHi = 64u | (1u << 14) | (2u << 29);  // 8-row groups 1024 B apart, 128-byte swizzle

// A block-scaled MMA, one CTA: D[tmem] (+)= A B with scales at sfa, sfb.
__device__ __forceinline__ void tc_mma_bs(uint32_t d, uint32_t ad, uint32_t bd, uint32_t hi, uint32_t idesc,
                                          uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %7};\n\tmov.b64 db, {%2, %7};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], da, db, %3, [%5], [%6], p;\n\t}" ::"r"(d),
      "r"(ad), "r"(bd), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb), "r"(hi)
      : "memory");
}

// The MMA issuers' loops run in the whole warp with one elected lane issuing:
// their many operands then stay in uniform registers, where the MMAs take them
// from.  In a loop of one lane every operand is moved there for each MMA
// (4096^3 on the pair kernel: 50.9 us, 47.8 this way).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ bool warp_ready(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
  return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) ||
         __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
}

// 512 bytes of scales (32 rows x 16 bytes) to the four columns at `taddr` of
// every lane quarter.
__device__ __forceinline__ void tc_cp_scales(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

// Descriptor of such a group in shared memory: no swizzle, 8-row cores 128 B apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)1 << 16;
  d |= (uint64_t)(128 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  return d;
}

// Bring a box of a tensor map into L2.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap *map, int c0, int c1) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1)
               : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

// Scale ids of block kb: byte kb % 4 of the packed words of both operands.
__device__ __forceinline__ uint32_t with_scale_ids(uint32_t idesc, int kb) {
  const uint32_t id = (uint32_t)kb & 3u;
  return idesc | (id << 4) | (id << 29);
}

__device__ __forceinline__ void store_one(const BArgs &a, size_t at, float y) {
  if (a.out_dtype == FP8_DT_F32) reinterpret_cast<float *>(a.out)[at] = y;
  else if (a.out_dtype == FP8_DT_BF16) reinterpret_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(y);
  else if (a.out_dtype == FP8_DT_F16) reinterpret_cast<__half *>(a.out)[at] = __float2half_rn(y);
  else reinterpret_cast<uint16_t *>(a.out)[at] = (uint16_t)(bf16x2_rto(y, y) & 0xffffu);
}

// ---------------------------------------------------------------------------
// The kernel for few tiles: few tokens, or a long reduction behind a small
// output.  The operand whose rows are neighbours in the output's memory (the
// weights; in wgrad x) is the MMA's 128-row operand, the other (the tokens; in
// wgrad dy) its columns, up to 128 of them, so that a batch below that wastes
// no multiplication on absent tokens.  A cluster of S CTAs takes a tile, each
// its share of the k-blocks (S = 1: no cluster).  The CTAs then
// exchange their partial tiles through distributed shared memory (posted
// stores; reading the others' parts instead cost 12 us at 128 columns), and
// each adds the S parts of its own tokens in rank order and stores them: no
// workspace, no atomics, the same bits each time.  Bound by latencies: start 3
// us, exchange 3, a k-block of a CTA 0.3 (operands in L2: 33 x 12288 x 4096 9.6
// us, 300 x 520 x 2056 7.9, 256 x 256 x 16384 10; weights from HBM: 33 x 12288 x
// 4096 13.6).
//   warp 0 TMA producer, warp 1 TMEM allocation and MMA issue, warps 2-5 epilogue.
constexpr int kSfCols = 8;      // tensor-memory columns of one set of scales: 4 of A, 4 of B
constexpr int kSfSets = 3;
// A group of four blocks writes a set of A's scales once and the next two
// groups write others.  A set is rewritten at the earliest nine blocks after
// its last block was multiplied; a ring of at most nine stages has by then
// seen those MMAs complete (its slot was refilled), so the copy cannot
// overtake a reader.
constexpr int kMaxStages = 9;

// One value to an output element where `p`; OUT as out_dtype.  Predicated, not
// branched around: with a branch per element 128 tokens took twice as long.
template <int OUT>
__device__ __forceinline__ void store_as(void *at, float y, bool p) {
  if constexpr (OUT == FP8_DT_F32) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t@q st.global.f32 [%0], %1;\n\t}" ::"l"(at), "f"(y),
                 "r"((int)p)
                 : "memory");
  } else {
    const uint16_t h = (uint16_t)(OUT == FP8_DT_BF16_RTO ? bf16x2_rto(y, y)
                                  : OUT == FP8_DT_F16    ? (uint32_t)__half_as_ushort(__float2half_rn(y))
                                                         : (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(y)));
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t@q st.global.b16 [%0], %1;\n\t}" ::"l"(at), "h"(h),
                 "r"((int)p)
                 : "memory");
  }
}
template <typename F>
__device__ __forceinline__ void with_out(int dtype, F f) {
  if (dtype == FP8_DT_BF16) f(std::integral_constant<int, FP8_DT_BF16>());
  else if (dtype == FP8_DT_F16) f(std::integral_constant<int, FP8_DT_F16>());
  else if (dtype == FP8_DT_F32) f(std::integral_constant<int, FP8_DT_F32>());
  else f(std::integral_constant<int, FP8_DT_BF16_RTO>());
}

// 16 columns of this lane's accumulator row.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15},"
      " [%16];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// This lane's feature: the tile's accumulator to out[token, feature];
// neighbouring lanes write neighbouring features.
__device__ __forceinline__ void store_tokens(const BArgs &a, int row, int col0, uint32_t tmem) {
  const float bias = a.bias && row < a.rows ? load_bias(a.bias, a.bias_dtype, row) : 0.0f;
  const int cols = min(a.cols - col0, a.bn);
  with_out(a.out_dtype, [&](auto out) {
    constexpr int OUT = decltype(out)::value, esz = OUT == FP8_DT_F32 ? 4 : 2;
    const size_t step = a.ld_out * esz;
    char *at = static_cast<char *>(a.out) + col0 * step + (size_t)row * esz;
#pragma unroll 1
    for (int c = 0; c < cols; c += 16) {
      uint32_t r[16];
      tmem_ld16(tmem + c, r);
#pragma unroll
      for (int j = 0; j < 16; j++) {
        store_as<OUT>(at, __fadd_rn(__uint_as_float(r[j]), bias), row < a.rows && c + j < cols);
        at += step;
      }
    }
  });
}

// The exchange: tokens in units of four, unit u finished by CTA u % S as its
// unit u / S.  The part of CTA s arrives in the owner's ring (free by then),
// slot s, per unit 128 rows x 16 bytes.  All threads of the CTA call it.
__device__ __forceinline__ void exchange_tokens(const BArgs &a, int splits, int rank, int row0, int col0,
                                                uint32_t base, uint32_t tmem_base) {
  const int cols = min(a.cols - col0, a.bn);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = warp & 3, row = row0 + q * 32 + lane;
  const int units = (cols + 3) / 4, per = (units + splits - 1) / splits;
  const bool mine = warp >= 2 && warp < 6;
  const float bias = mine && a.bias && row < a.rows ? load_bias(a.bias, a.bias_dtype, row) : 0.0f;
  cluster_sync();  // every CTA's MMAs have read their ring
  if (mine) {
    tc_fence_after();
    uint32_t at = base + (rank * per * BM + q * 32 + lane) * 16;
    uint32_t tmem = tmem_base + ((uint32_t)(q * 32) << 16);
    int owner = 0;
#pragma unroll 1
    for (int c = 0; c < cols; c += 16) {
      uint32_t r[16];
      tmem_ld16(tmem + c, r);
#pragma unroll
      for (int g = 0; g < 4; g++) {
        if (c + 4 * g < cols)
          asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(map_to_rank(at, (uint32_t)owner)),
                       "r"(r[4 * g]), "r"(r[4 * g + 1]), "r"(r[4 * g + 2]), "r"(r[4 * g + 3])
                       : "memory");
        if (++owner == splits) {
          owner = 0;
          at += BM * 16;
        }
      }
    }
    tc_fence_before();
  }
  cluster_sync();  // all parts have arrived
  if (mine) {
    with_out(a.out_dtype, [&](auto out) {
      constexpr int OUT = decltype(out)::value, esz = OUT == FP8_DT_F32 ? 4 : 2;
      const size_t step = a.ld_out * esz;
      char *at = static_cast<char *>(a.out) + (col0 + rank * 4) * step + (size_t)row * esz;
      uint32_t first = base + (q * 32 + lane) * 16;
#pragma unroll 1
      for (int c = rank * 4; c < cols; c += splits * 4, at += splits * 4 * step, first += BM * 16) {
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        uint32_t src = first;
#pragma unroll 2
        for (int s = 0; s < splits; s++, src += per * BM * 16) {
          float x[4];
          asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3])
                       : "r"(src)
                       : "memory");
#pragma unroll
          for (int j = 0; j < 4; j++) v[j] = __fadd_rn(v[j], x[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; j++)
          store_as<OUT>(at + j * step, __fadd_rn(v[j], bias), row < a.rows && c + j < cols);
      }
    });
  }
}

__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols) : "memory");
}

// A_MN, B_MN: the operand's codes are read along their rows (the weights in
// dgrad, both in wgrad).  Ring stage: A 16 KB, B bn x 128 B; scales of both
// (1 KB) with every fourth block.
constexpr int kSfSlot = 1024;
// At most: two CTAs per SM, whose 256 columns of tensor memory each fit it.  The
// library's other kernels that allocate tensor memory need more shared memory
// than is left beside one (at least 89 KB are used), so that no CTA of a cluster
// waits for tensor memory while another holds some.
constexpr int kFewSmemBytes = 112 * 1024;

template <bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kThreads)
    k_bgemm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
            const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
            const __grid_constant__ BArgs args, const int splits) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *base_ptr = smem_raw + (base - raw);
  const int S = args.stages;
  const uint32_t sf0 = base + S * args.stage_bytes;
  const uint32_t bar0 = sf0 + S * kSfSlot;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
  const uint32_t tfull_bar = bar0 + 8u * (2 * kMaxStages);
  const uint32_t drain_bar = bar0 + 8u * (2 * kMaxStages + 1);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(base_ptr + (bar0 - base) + 8 * (2 * kMaxStages + 2));
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = splits > 1 ? (int)cluster_rank() : 0;
  const int tile = (int)(blockIdx.x / splits);
  const int row0 = tile / args.num_n_blocks * BM, col0 = tile % args.num_n_blocks * 128;
  // this CTA's k-blocks
  const int kb0 = (int)((long long)args.num_k_blocks * rank / splits);
  const int kb1 = (int)((long long)args.num_k_blocks * (rank + 1) / splits);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; s++) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(tfull_bar, 1);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmSA);
    tma_prefetch_desc(&tmSB);
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), args.tmem_cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // Not before the allocation: a dependent CTA that took tensor memory first
  // and then waited for this kernel would wait for good.
  pdl_launch_dependents();
  pdl_wait();

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued_mask = 0, issued_par = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; kb++) {
        if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag)) { ok = false; break; }
        const uint32_t sa = base + stage * args.stage_bytes, ss = sf0 + stage * kSfSlot;
        const bool scales = kb == kb0 || (kb & 3) == 0;
        mbar_arrive_expect_tx(full_bar(stage), args.stage_bytes + (scales ? kSfSlot : 0));
        if (scales) {
          tma_load_3d(ss, &tmSA, 0, kb >> 2, row0 >> 7, full_bar(stage));
          tma_load_3d(ss + 512, &tmSB, 0, kb >> 2, col0 >> 7, full_bar(stage));
        }
        if (A_MN) tma_load_2d(sa, &tmA, row0, kb * BK, full_bar(stage));
        else      tma_load_2d(sa, &tmA, kb * BK, row0, full_bar(stage));
        if (B_MN) tma_load_2d(sa + BM * BK, &tmB, col0, kb * BK, full_bar(stage));
        else      tma_load_2d(sa + BM * BK, &tmB, kb * BK, col0, full_bar(stage));
        issued_mask |= 1u << stage;
        issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
        if (++stage == S) { stage = 0; phase ^= 1u; }
      }
      if (!ok) {
        for (int s = 0; s < S; s++)
          if (issued_mask & (1u << s)) mbar_wait_drain(full_bar(s), (issued_par >> s) & 1u);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    const bool elected = elect_one();
    const uint32_t a_d0 = (uint32_t)operand_desc<A_MN>(base, 0), b_d0 = (uint32_t)operand_desc<B_MN>(base + BM * BK, 0);
    constexpr uint32_t a_ks = A_MN ? (UMMA_K * 128) >> 4 : UMMA_K >> 4, b_ks = B_MN ? (UMMA_K * 128) >> 4 : UMMA_K >> 4;
    const uint32_t st_d = args.stage_bytes >> 4, sf_tmem = tmem_base + args.bn;
    int stage = 0, set = kSfSets - 1;
    uint32_t phase = 0;
    bool ok = true, issued_any = false;
    for (int kb = kb0; kb < kb1; kb++) {
      if (!warp_ready(full_bar(stage), phase, abort_flag)) { ok = false; break; }
      if (kb == kb0 || (kb & 3) == 0) {
        set = set == kSfSets - 1 ? 0 : set + 1;
        if (elected) {
          tc_cp_scales(sf_tmem + set * kSfCols, scale_desc(sf0 + stage * kSfSlot));
          tc_cp_scales(sf_tmem + set * kSfCols + 4, scale_desc(sf0 + stage * kSfSlot + 512));
        }
      }
      const uint32_t sfa = sf_tmem + set * kSfCols, so = (uint32_t)stage * st_d;
      const uint32_t idesc = with_scale_ids(args.idesc, kb);
      if (elected) {
#pragma unroll
        for (int ks = 0; ks < BK / UMMA_K; ks++)
          tc_mma_bs(tmem_base, a_d0 + so + ks * a_ks, b_d0 + so + ks * b_ks, args.desc_hi, idesc, sfa, sfa + 4,
                    (kb != kb0 || ks != 0) ? 1u : 0u);
        tc_commit(empty_bar(stage));
      }
      issued_any = true;
      if (++stage == S) { stage = 0; phase ^= 1u; }
    }
    if (ok) {
      if (elected) tc_commit(tfull_bar);
    } else if (issued_any) {
      if (elected) tc_commit(drain_bar);
      mbar_wait_drain(drain_bar, 0);
    }
    __syncwarp();
  } else {
    const bool got = __all_sync(0xffffffffu, mbar_wait(tfull_bar, 0, abort_flag));
    tc_fence_after();
    if (got && splits == 1)
      store_tokens(args, row0 + (warp & 3) * 32 + lane, col0, tmem_base + ((uint32_t)((warp & 3) * 32) << 16));
    tc_fence_before();
    __syncwarp();
  }
  if (splits > 1) exchange_tokens(args, splits, rank, row0, col0, base, tmem_base);

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_free(tmem_base, args.tmem_cols);
  }
}

// ---------------------------------------------------------------------------
// Tokens that come as x itself (at most 32): the cast and the product in one
// launch.  Here the tokens are the MMA's rows and 256 weight rows its columns:
// an MMA takes some 128 cycles whether it has 16 columns or 256, so with the
// weights as rows a CTA could not multiply more than 32 bytes of them a cycle
// (12288 x 4096 at one token: 18 us).  The rows of absent tokens need not exist:
// the A descriptor's 16 KB window runs over whatever lies behind the tokens'
// codes in shared memory, and what it makes of that lands in accumulator rows
// that nothing reads.
//   warp 0 TMA producer: 256 x 128-byte tiles of the weights, a ring of 4 to 6
//   warp 1 TMEM allocation and MMA issue
//   warps 2-17 cast x, a block of eight tokens at a time: a chain of some 1300
//   cycles behind a round trip to L2, so it takes many warps to keep ahead.
//   The codes live in a second ring, four blocks (a group of scale bytes) a
//   slot.  (Casting into the weights' own ring held a CTA to 45 GB/s.)
//   warps 4, 8, 12, 16 (accumulator rows 0..31) then finish, 64 columns each.
// A cluster of S CTAs shares a tile's reduction: unit u of eight features is
// finished by CTA u % S.  The parts go to the owner as asynchronous stores that
// count their bytes on a barrier of the owner's, into memory kept for them, so
// that the end of the reduction needs no cluster-wide barrier (two of them and
// the exchange took 2.7 us).
// Bound by the weights' HBM traffic, and below about 30 MB by the latencies of
// start, cast and exchange.  Weights from HBM: 12288 x 4096 at one token 14.7 us
// (3.4 TB/s; 16 at 32 tokens; cast and k_bgemm in two launches 15), 12288 x 12288
// 28 to 30 (5 TB/s), 4096 x 4096 at 16 tokens 8.4.  In L2 12288 x 4096 takes 11.6.
constexpr int kTokMaxStages = 6;
constexpr int kTokBN = 256;    // weight rows per tile
constexpr int kTokBatch = 8;   // tokens that one cast takes
constexpr int kTokWarps = 16;
constexpr int kTokThreads = 64 + 32 * kTokWarps;
constexpr int kTokPrefetch = 8;  // weight blocks (32 KB) brought into L2 ahead of the dependency wait
constexpr int kTokStageBytes = kTokBN * BK;
// Slots of the code ring, by the number of batches of eight tokens.  A parity
// wait tells only one phase of a slot from the next, so a casting warp must
// not be able to skip a whole turn of the ring: its next unit is kTokWarps
// units on, 4 / batches groups (4, 2, 2, 1).
__host__ __device__ constexpr int tok_groups(int batches) { return batches == 1 ? 4 : 3; }
constexpr int kTokMaxGroups = 4;
// Parts of a CTA's units of eight features: S * ceil(32 / S) <= 36 of them, 32 bytes per token.
__host__ __device__ constexpr int tok_parts(int batches) { return 36 * 32 * 8 * batches; }
__host__ __device__ constexpr int tok_fixed(int batches) {
  return tok_groups(batches) * (4096 * batches + 512) + tok_parts(batches) + 512 + 1024;
}
// What is left of the SM's shared memory holds weights in flight: it is their
// latency that bounds a CTA.
__host__ __device__ constexpr int tok_stages(int batches) {
  const int n = (232448 - tok_fixed(batches)) / (kTokStageBytes + 1024);
  return n < kTokMaxStages ? n : kTokMaxStages;
}
constexpr int kTokSfA = kTokBN;       // tensor-memory columns: 4 x 4 of the tokens' scales,
constexpr int kTokSfB = kTokBN + 16;  // 3 x 8 of the weights'
constexpr uint32_t kTokTmem = 512;

// Eight tokens' parts of one block: x[t0 .. t0+7, k0 .. k0+127], 16 lanes per
// token, 8 elements each, four pairs of tokens.
template <int DT>
__device__ __forceinline__ void load_tokens(const BArgs &a, int t0, int k0, int lane, block::Raw8<DT> (&raw)[4]) {
  const int c8 = lane & 15, half = lane >> 4;
  if (block::wide_tile(a.x_vec, k0, a.x_cols)) {
#pragma unroll
    for (int i = 0; i < 4; i++)
      raw[i] = block::load_raw8_wide<DT>(a.x, a.ldx, t0 + 2 * i + half, k0 + c8 * 8, a.cols, a.x_cols);
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++)
      raw[i] = block::load_raw8_single<DT>(a.x, a.ldx, t0 + 2 * i + half, k0 + c8 * 8, a.cols, a.x_cols);
  }
}

// The same eight tokens as E4M3 codes in the K-major 128-byte-swizzled tile at
// `tile`, and their scale bytes at byte kb % 4 of the words at `sf`.
template <int DT>
__device__ __forceinline__ void cast_tokens(const BArgs &a, int t0, int kb, uint32_t tile, uint32_t sf, int lane,
                                            const block::Raw8<DT> (&raw)[4]) {
  const int c8 = lane & 15, half = lane >> 4;
  uint32_t m[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    m[i] = 0;
#pragma unroll
    for (int j = 0; j < block::Raw8<DT>::kWords; j++) m[i] = block::max_words<DT>(m[i], raw[i].w[j]);
    m[i] = block::word_abs<DT>(m[i]);
  }
  const uint32_t v = block::reduce_rows<4>(m, c8);  // lane c8 holds pair c8 / 4
  const int k = block::block_exponent(v, kMaxE4M3, a.margin);
  const float own = pow2f(k);
  const bool nan = __any_sync(0xffffffffu, v >= 0x7f800000u);
  if ((c8 & 3) == 0)
    asm volatile("st.shared.u8 [%0], %1;" ::"r"(sf + (t0 + 2 * (c8 >> 2) + half) * 16 + (kb & 3)),
                 "r"((uint32_t)(127 - k))
                 : "memory");
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int t = t0 + 2 * i + half;
    const float s = __shfl_sync(0xffffffffu, own, (lane & 16) + 4 * i);
    float f[8];
    float2 s4[4];
    block::unpack8<DT>(raw[i], f);
    block::spread_scale(s, s4);
    const uint2 c = block::enc8<FP8_E4M3>(f, s4);
    const uint32_t at = tile + t * 128 + (((c8 >> 1) ^ (t & 7)) << 4) + (c8 & 1) * 8;
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(c.x), "r"(c.y) : "memory");
  }
  if (nan) {  // behind the common code, which a CTA mostly runs once, from a cold instruction cache
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int t = t0 + 2 * i + half;
      const float s = __shfl_sync(0xffffffffu, own, (lane & 16) + 4 * i);
      float f[8];
      float2 s4[4];
      block::unpack8<DT>(raw[i], f);
      block::spread_scale(s, s4);
      const uint2 c = block::enc8_any<FP8_E4M3>(f, s4);
      const uint32_t at = tile + t * 128 + (((c8 >> 1) ^ (t & 7)) << 4) + (c8 & 1) * 8;
      asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(c.x), "r"(c.y) : "memory");
    }
  }
}

// Eight features of this lane's token (and, with n < 8, fewer) to out.
__device__ __forceinline__ void store_features(const BArgs &a, int token, int col, const float (&v)[8]) {
  if (a.out_dtype == FP8_DT_F32) block::store8<FP8_DT_F32>(a.vec_out, a.out, a.ld_out, token, col, a.cols, a.rows, v);
  else if (a.out_dtype == FP8_DT_BF16) block::store8<FP8_DT_BF16>(a.vec_out, a.out, a.ld_out, token, col, a.cols, a.rows, v);
  else if (a.out_dtype == FP8_DT_F16) block::store8<FP8_DT_F16>(a.vec_out, a.out, a.ld_out, token, col, a.cols, a.rows, v);
  else block::store8<FP8_DT_BF16_RTO>(a.vec_out, a.out, a.ld_out, token, col, a.cols, a.rows, v);
}

template <int DT>
__global__ void __launch_bounds__(kTokThreads, 1)
    k_btokens(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmSW,
              const __grid_constant__ BArgs args, const int splits) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *base_ptr = smem_raw + (base - raw);
  const int batches = (args.cols + kTokBatch - 1) / kTokBatch, G = tok_groups(batches), S = tok_stages(batches);
  const uint32_t tile_bytes = (uint32_t)batches * 1024, group_bytes = 4 * tile_bytes;  // codes of a block, of a group
  const uint32_t ring0 = base + G * group_bytes;
  const uint32_t sfw0 = ring0 + S * kTokStageBytes;  // weights' scales, per stage
  const uint32_t sfx0 = sfw0 + S * 1024;             // tokens' scales, per slot
  const uint32_t parts0 = sfx0 + G * 512;
  const uint32_t bar0 = parts0 + tok_parts(batches);
  const int lanes = kTokBatch * batches;             // lanes of a part
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (kTokMaxStages + s); };
  auto cfull_bar = [&](int g) { return bar0 + 8u * (2 * kTokMaxStages + g); };
  auto cempty_bar = [&](int g) { return bar0 + 8u * (2 * kTokMaxStages + kTokMaxGroups + g); };
  const uint32_t tfull_bar = bar0 + 8u * (2 * kTokMaxStages + 2 * kTokMaxGroups);
  const uint32_t drain_bar = tfull_bar + 8u, parts_bar = tfull_bar + 16u, loaded_bar = tfull_bar + 24u;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(base_ptr + (loaded_bar + 8u - base));
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = splits > 1 ? (int)cluster_rank() : 0;
  const int row0 = (int)(blockIdx.x / splits) * kTokBN;  // first weight row
  const int kb0 = (int)((long long)args.num_k_blocks * rank / splits);
  const int kb1 = (int)((long long)args.num_k_blocks * (rank + 1) / splits);
  const int g0 = kb0 >> 2, groups = ((kb1 + 3) >> 2) - g0;  // groups of four blocks, by their scale bytes
  const int units_x = groups * 4 * batches;                 // casts
  const int units = (min(kTokBN, args.rows - row0) + 7) / 8, per = (units + splits - 1) / splits;
  const int owned = (units - rank + splits - 1) / splits;   // of this CTA

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; s++) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int g = 0; g < G; g++) {
      mbar_init(cfull_bar(g), 4 * batches);
      mbar_init(cempty_bar(g), 1);
    }
    mbar_init(tfull_bar, 1);
    mbar_init(drain_bar, 1);
    mbar_init(parts_bar, 1);
    mbar_init(loaded_bar, min(kTokWarps, units_x));
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (splits > 1 && owned > 0) mbar_arrive_expect_tx(parts_bar, (uint32_t)(owned * splits * args.cols * 32));
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmSW);
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), kTokTmem);
  tc_fence_before();
  if (splits > 1) cluster_sync();  // no CTA sends a part before its owner's barrier is set up
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_launch_dependents();  // (not before the allocation: see k_bgemm)
  // x and the first weights come into L2 while the stream's previous kernel
  // ends.  (L2 is where its writes go too, so what it still writes is read as
  // written by the loads after the wait.)  x first: behind 25 MB of weights
  // its loads took 2.5 us.
  {
    const int esz = DT == FP8_DT_F32 ? 4 : 2;
    const int c0 = g0 * 512, c1 = min((g0 + groups) * 512, args.x_cols), lines = ((c1 - c0) * esz + 127) / 128;
    for (int i = threadIdx.x; i < lines * args.cols; i += kTokThreads) {
      const int r = i / lines, c = c0 + (i - r * lines) * (128 / esz);
      asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const uint8_t *>(args.x) +
                                                   ((size_t)r * args.ldx + c) * esz)
                   : "memory");
    }
  }
  __syncthreads();
  if (threadIdx.x == 0)
    for (int kb = kb0; kb < min(kb1, kb0 + kTokPrefetch); kb++) tma_prefetch_2d(&tmW, kb * BK, row0);
  pdl_wait();

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued_mask = 0, issued_par = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; kb++) {
        // the ring's first fill waits for x: its 128 KB in front of the first
        // loads of x delayed them, and the casts behind them, by over 1 us
        if (kb == kb0 + 1 && !mbar_wait(loaded_bar, 0, abort_flag)) { ok = false; break; }
        if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag)) { ok = false; break; }
        const bool scales = kb == kb0 || (kb & 3) == 0;
        mbar_arrive_expect_tx(full_bar(stage), kTokStageBytes + (scales ? 1024 : 0));
        if (scales) tma_load_3d(sfw0 + stage * 1024, &tmSW, 0, kb >> 2, row0 >> 7, full_bar(stage));
        tma_load_2d(ring0 + stage * kTokStageBytes, &tmW, kb * BK, row0, full_bar(stage));
        issued_mask |= 1u << stage;
        issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
        if (++stage == S) { stage = 0; phase ^= 1u; }
      }
      if (!ok) {
        for (int s = 0; s < S; s++)
          if (issued_mask & (1u << s)) mbar_wait_drain(full_bar(s), (issued_par >> s) & 1u);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    const bool elected = elect_one();
    const uint32_t a_d0 = (uint32_t)operand_desc<false>(base, 0), b_d0 = (uint32_t)operand_desc<false>(ring0, 0);
    constexpr uint32_t ks_d = UMMA_K >> 4, st_d = kTokStageBytes >> 4;
    const uint32_t grp_d = group_bytes >> 4, tile_d = tile_bytes >> 4;
    int stage = 0, set = kSfSets - 1, slot = 0;
    uint32_t phase = 0, cphase = 0;
    bool ok = true, issued_any = false;
    for (int kb = kb0; kb < kb1; kb++) {
      const uint32_t sfa = tmem_base + kTokSfA + slot * 4;
      if (!warp_ready(full_bar(stage), phase, abort_flag)) { ok = false; break; }
      if (kb == kb0 || (kb & 3) == 0) {
        if (!warp_ready(cfull_bar(slot), cphase, abort_flag)) { ok = false; break; }
        set = set == kSfSets - 1 ? 0 : set + 1;
        if (elected) {
          tc_cp_scales(sfa, scale_desc(sfx0 + slot * 512));
          tc_cp_scales(tmem_base + kTokSfB + set * 8, scale_desc(sfw0 + stage * 1024));
          tc_cp_scales(tmem_base + kTokSfB + set * 8 + 4, scale_desc(sfw0 + stage * 1024 + 512));
        }
      }
      const uint32_t sfb = tmem_base + kTokSfB + set * 8;
      const uint32_t idesc = with_scale_ids(args.idesc, kb);
      const uint32_t ad = a_d0 + slot * grp_d + (kb & 3) * tile_d, bd = b_d0 + stage * st_d;
      if (elected) {
#pragma unroll
        for (int ks = 0; ks < BK / UMMA_K; ks++)
          tc_mma_bs(tmem_base, ad + ks * ks_d, bd + ks * ks_d, args.desc_hi, idesc, sfa, sfb,
                    (kb != kb0 || ks != 0) ? 1u : 0u);
        tc_commit(empty_bar(stage));
        if ((kb & 3) == 3) tc_commit(cempty_bar(slot));
      }
      if ((kb & 3) == 3 && ++slot == G) {
        slot = 0;
        cphase ^= 1u;
      }
      issued_any = true;
      if (++stage == S) { stage = 0; phase ^= 1u; }
    }
    if (ok) {
      if (elected) tc_commit(tfull_bar);
    } else if (issued_any) {
      if (elected) tc_commit(drain_bar);
      mbar_wait_drain(drain_bar, 0);
    }
    __syncwarp();
  } else {
    // Unit u: tokens of batch u % batches, block u / batches (counted from the
    // first group's first block; blocks of a group that another CTA multiplies
    // are cast too, so that every group has the same number of units).
    // The first turn only loads; one load and one cast site keep the code short.
    block::Raw8<DT> x[4];
    const int step_i = kTokWarps / batches, step_b = kTokWarps - step_i * batches;
    int i = (warp - 2) / batches, b = (warp - 2) - i * batches;  // the unit to load: block, batch
    int ci = -1, cb = 0, cg = 0, slot = 0;                       // the one to cast; its group, slot and the slot's turn
    uint32_t turn = 1;
    const int blocks = groups * 4;
    while (i < blocks || ci >= 0) {
      block::Raw8<DT> next[4];
      const bool more = i < blocks;
      if (more) load_tokens<DT>(args, b * kTokBatch, (g0 * 4 + i) * BK, lane, next);
      if (ci < 0) {
        uint32_t seen = 0;
#pragma unroll
        for (int j = 0; j < 4; j++) seen |= next[j].w[0];
        uint32_t any;  // (0 or 1: makes the arrive wait for the loads)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\tvote.sync.any.pred p, p, 0xffffffff;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(any)
                     : "r"(seen));
        if (lane == 0 && any <= 1u) mbar_arrive(loaded_bar);
      } else {
        for (slot += (ci >> 2) - cg, cg = ci >> 2; slot >= G; slot -= G) turn ^= 1u;
        if (!__all_sync(0xffffffffu, mbar_wait(cempty_bar(slot), turn, abort_flag))) break;
        cast_tokens<DT>(args, cb * kTokBatch, ci & 3, base + slot * group_bytes + (ci & 3) * tile_bytes,
                        sfx0 + slot * 512, lane, x);
        fence_async_shared();  // the MMAs and the scale copy read through the async proxy
        __syncwarp();
        if (lane == 0) mbar_arrive(cfull_bar(slot));
      }
      ci = more ? i : -1;
      if (!more) break;
      cb = b;
      i += step_i;
      b += step_b;
      if (b >= batches) {
        b -= batches;
        i++;
      }
#pragma unroll
      for (int j = 0; j < 4; j++) x[j] = next[j];
    }
    __syncwarp();
  }

  // ------------------------------------------------------------ finish
  if (warp >= 4 && (warp & 3) == 0) {     // accumulator rows 0..31
    const int c0 = ((warp >> 2) - 1) * 64;  // of these 64 columns
    const bool got = __all_sync(0xffffffffu, mbar_wait(tfull_bar, 0, abort_flag));
    tc_fence_after();
    // (after a timeout the parts are sent all the same: their owners count on them)
    int owner = splits > 1 ? (c0 / 8) % splits : 0;
    uint32_t part = parts0 + (uint32_t)((rank * per + c0 / 8 / splits) * 2 * lanes + lane) * 16;
#pragma unroll 1
    for (int c = c0; c < c0 + 64 && c / 8 < units; c += 16) {
      uint32_t r[16];
      tmem_ld16(tmem_base + c, r);
      if (splits == 1) {
        const int bcol = row0 + c + lane;
        const float bias = args.bias && lane < 16 && bcol < args.rows ? load_bias(args.bias, args.bias_dtype, bcol) : 0.0f;
#pragma unroll
        for (int j = 0; j < 16; j++)
          r[j] = __float_as_uint(__fadd_rn(__uint_as_float(r[j]), __shfl_sync(0xffffffffu, bias, j)));
#pragma unroll
        for (int g = 0; g < 2; g++) {
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; j++) v[j] = __uint_as_float(r[8 * g + j]);
          if (got) store_features(args, lane, row0 + c + 8 * g, v);
        }
      } else {  // to part `rank` of the owner's unit, `lanes` x 16 bytes per half
#pragma unroll
        for (int g = 0; g < 2; g++) {
          if (c / 8 + g < units && lane < args.cols) {
            const uint32_t bar = map_to_rank(parts_bar, (uint32_t)owner), dst = map_to_rank(part, (uint32_t)owner);
#pragma unroll
            for (int h = 0; h < 2; h++)
              asm volatile(
                  "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                      dst + h * lanes * 16),
                  "r"(r[8 * g + 4 * h]), "r"(r[8 * g + 4 * h + 1]), "r"(r[8 * g + 4 * h + 2]), "r"(r[8 * g + 4 * h + 3]),
                  "r"(bar)
                  : "memory");
          }
          if (++owner == splits) {
            owner = 0;
            part += 2 * lanes * 16;
          }
        }
      }
    }
    tc_fence_before();
  }
  __syncwarp();
  // No CTA leaves before every other has sent its parts (normally long since).
  if (splits > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  if (splits > 1 && owned > 0 && warp >= 2) {
    const bool got = __all_sync(0xffffffffu, mbar_wait(parts_bar, 0, abort_flag));
    for (int i = warp - 2; got && i < owned; i += kTokWarps) {
      const int col = row0 + (i * splits + rank) * 8;
      float bias = 0.0f;
      if (args.bias && lane < 8 && col + lane < args.rows) bias = load_bias(args.bias, args.bias_dtype, col + lane);
      float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
      for (int s = 0; s < splits; s++) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
          float p[4];
          asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(p[0]), "=f"(p[1]), "=f"(p[2]), "=f"(p[3])
                       : "r"(parts0 + (((s * per + i) * 2 + h) * lanes + min(lane, lanes - 1)) * 16)
                       : "memory");
#pragma unroll
          for (int j = 0; j < 4; j++) v[4 * h + j] = __fadd_rn(v[4 * h + j], p[j]);
        }
      }
      if (args.bias) {
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = __fadd_rn(v[j], __shfl_sync(0xffffffffu, bias, j));
      }
      store_features(args, lane, col, v);
    }
    __syncwarp();
  }
  if (splits > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");

  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_free(tmem_base, kTokTmem);
  }
}

// out[r, c] = bias[c] or 0: a product with an empty reduction.
__global__ void k_bgemm_empty(const BArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const size_t n = (size_t)a.rows * a.cols, stride = (size_t)gridDim.x * blockDim.x;
  for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += stride) {
    const int r = (int)(i / a.cols), c = (int)(i % a.cols);
    store_one(a, (size_t)r * a.ld_out + c, a.bias ? load_bias(a.bias, a.bias_dtype, c) : 0.0f);
  }
}

// ---------------------------------------------------------------------------
// Pair kernel: a cluster of two CTAs on two SMs computes 256 x 256 tiles with
// tcgen05.mma.cta_group::2, persistent over the tiles.  Each CTA loads its
// 128 rows of A, its 128 columns of B (32 KB per stage, 5 stages) and, every
// fourth block, the scales of its rows and of all 256 columns (each tensor
// core multiplies 128 rows by all columns).
//
// Tensor memory: two 256-column accumulators and the scales do not fit side
// by side in 512 columns, so the accumulators overlap by 32: the first is
// columns 0..255, the second 224..479, the scales 480..511.  The epilogue
// reads the shared 32 columns first and then lets the next tile's MMAs start;
// by the time a warp says so for one tile it has read all of the tile before,
// so that one signal covers both accumulators.  The gap between two tiles is
// one barrier round trip and two TMEM loads.
// Whole tiles fill the clusters in waves.  Where the last wave would leave half
// of the clusters idle, its tiles are worked as two halves of 128 columns (N =
// 128, the CTAs loading from columns 64 apart), so that it lasts half as long.
// Bound by the operands' way from L2 into shared memory (a k-block of the pair's
// MMAs alone takes 0.28 us, with its loads 0.38).  4096^3 48 to 53 us (2.6 to 2.9
// PFLOP/s), 4096 x 16384 x 4096 206, 8192 x 12288 x 12288 844 to 986 (2.5 to 2.9,
// power-capped); eight epilogue warps with four stages took 231 us for 205 at
// K = 16384, six stages with one staging box 61 for 52 at 4096^3.
//   warp 0 TMA producer (both CTAs), warp 1 TMEM allocation and MMA issue
//   (leader), warps 2-5 epilogue (both CTAs).
constexpr int kP2Stages = 5;
constexpr int kP2SfSlot = 512 + 1024;
constexpr int kP2Acc1 = 224;    // first column of the second accumulator
constexpr int kP2Sf = 480;      // two sets of scales, 16 columns each
constexpr int kP2OutBoxes = 2;  // staging boxes per epilogue warp (stores pipelined)
constexpr int kP2SmemBytes =
    kP2Stages * (kPairStageBytes + kP2SfSlot) + 4 * kP2OutBoxes * kWideStageOutBytes + 256 + 4 * 1024 + 1024;

__device__ __forceinline__ void tc_mma_bs_pair(uint32_t d, uint32_t ad, uint32_t bd, uint32_t hi, uint32_t idesc,
                                               uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %7};\n\tmov.b64 db, {%2, %7};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], da, db, %3, [%5], [%6], p;\n\t}" ::"r"(d),
      "r"(ad), "r"(bd), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb), "r"(hi)
      : "memory");
}

// The copy of scales in both CTAs of the pair, each from its own shared memory.
__device__ __forceinline__ void tc_cp_scales_pair(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

__device__ __forceinline__ void tc_commit_leader(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2,
                                                 uint32_t cluster_bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(cluster_bar)
      : "memory");
}

// A row's 32 values of two neighbouring columns each -> 16 packed words.
template <int OUT>
__device__ __forceinline__ uint32_t pack_out(float a, float b) {
  if constexpr (OUT == FP8_DT_BF16_RTO) return bf16x2_rto(a, b);
  if constexpr (OUT == FP8_DT_F16) return f16x2(a, b);
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// A staged box (32 rows of 128 bytes, swizzled) to rows at any alignment:
// neighbouring lanes store neighbouring elements.
template <int OUT>
__device__ __forceinline__ void store_box_elements(const BArgs &a, uint32_t stg, int row0, int col0, int lane) {
  constexpr int esz = OUT == FP8_DT_F32 ? 4 : 2;
  const int rows = min(32, a.rows - row0);
  for (int r = 0; r < rows; r++) {
#pragma unroll
    for (int h = 0; h < 4 / esz; h++) {
      const int e = h * 32 + lane;
      const uint32_t src = stg + r * 128 + (((e * esz >> 4) ^ (r & 7)) << 4) + (e * esz & 15);
      const size_t at = (size_t)(row0 + r) * a.ld_out + col0 + e;
      if (col0 + e >= a.cols) continue;
      if constexpr (esz == 4) {
        uint32_t v;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(src) : "memory");
        reinterpret_cast<uint32_t *>(a.out)[at] = v;
      } else {
        uint16_t v;
        asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(src) : "memory");
        reinterpret_cast<uint16_t *>(a.out)[at] = v;
      }
    }
  }
  __syncwarp();
}

// A tile's bias in an epilogue warp's kilobyte at `dst`, and 32 of its values,
// every lane the same, added to a row's sums.  (Handed out by shuffles from a
// lane each, the bias took half of a short product's time: 4096 x 16384 x 256
// bfloat16 69 us for 42, and 30 without bias; x 4096 176 for 166.)
__device__ __forceinline__ void stage_bias(const BArgs &a, int col0, uint32_t dst) {
  const int lane = (int)(threadIdx.x & 31);
  uint32_t raw[8];  // all loads in flight before the first is used
  if (a.bias_dtype == FP8_DT_F32) {
#pragma unroll
    for (int j = 0; j < 8; j++) raw[j] = static_cast<const uint32_t *>(a.bias)[min(col0 + j * 32 + lane, a.cols - 1)];
  } else {
#pragma unroll
    for (int j = 0; j < 8; j++) raw[j] = static_cast<const uint16_t *>(a.bias)[min(col0 + j * 32 + lane, a.cols - 1)];
  }
  __syncwarp();  // the tile before has been read
#pragma unroll
  for (int j = 0; j < 8; j++) {
    float b = __uint_as_float(raw[j]);
    if (a.bias_dtype == FP8_DT_BF16) b = __uint_as_float(raw[j] << 16);
    else if (a.bias_dtype == FP8_DT_F16) b = __half2float(__ushort_as_half((unsigned short)raw[j]));
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(dst + (j * 32 + lane) * 4), "f"(b) : "memory");
  }
  __syncwarp();
}
__device__ __forceinline__ void add_bias(uint32_t src, uint32_t (&r)[32]) {
#pragma unroll
  for (int j = 0; j < 32; j += 4) {
    float b[4];
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(b[0]), "=f"(b[1]), "=f"(b[2]), "=f"(b[3])
                 : "r"(src + j * 4)
                 : "memory");
#pragma unroll
    for (int k = 0; k < 4; k++) r[j + k] = __float_as_uint(__fadd_rn(__uint_as_float(r[j + k]), b[k]));
  }
}

template <bool A_MN, bool B_MN, int OUT>
__global__ void __launch_bounds__(kThreads, 1)
    k_bgemm2(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
             const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
             const __grid_constant__ CUtensorMap tmOut, const __grid_constant__ BArgs args) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *base_ptr = smem_raw + (base - raw);
  const uint32_t out_stage0 = base + kP2Stages * kPairStageBytes;
  const uint32_t sf0 = out_stage0 + 4 * kP2OutBoxes * kWideStageOutBytes;
  const uint32_t bar0 = sf0 + kP2Stages * kP2SfSlot;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (kP2Stages + s); };
  auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * kP2Stages + b); };
  auto sffree_bar = [&](int b) { return bar0 + 8u * (2 * kP2Stages + 2 + b); };
  const uint32_t tempty_bar = bar0 + 8u * (2 * kP2Stages + 4);
  const uint32_t drain_bar = bar0 + 8u * (2 * kP2Stages + 5);
  const uint32_t alloc_bar = bar0 + 8u * (2 * kP2Stages + 6);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(base_ptr + (bar0 - base) + 8 * (2 * kP2Stages + 7));
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, num_pairs = gridDim.x >> 1;
  // Item t of the work: its tile, and the half (0, 1) of it or -1 for the whole.
  const int num_items = args.whole + 2 * (args.num_tiles - args.whole);
  auto coords = [&](int t, int &mb, int &nb) {
    int half = -1;
    if (t >= args.whole) {
      half = (t - args.whole) & 1;
      t = args.whole + ((t - args.whole) >> 1);
    }
    const int per_band = args.group_m * args.num_n_blocks;
    const int band = t / per_band, first = band * args.group_m;
    const int rows_in_band = min(args.num_m_blocks - first, args.group_m);
    const int r = t - band * per_band;
    mb = first + r % rows_in_band;
    nb = r / rows_in_band;
    return half;
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kP2Stages; s++) {
      mbar_init(full_bar(s), 1);   // leader: its producer's arrive + both CTAs' bytes
      mbar_init(empty_bar(s), 1);  // one multicast commit per phase
    }
    for (int b = 0; b < 2; b++) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(sffree_bar(b), 1);
    }
    mbar_init(tempty_bar, 8);  // leader: 4 epilogue warps x 2 CTAs
    mbar_init(drain_bar, 1);
    mbar_init(alloc_bar, 2);   // leader: the issuing warps of both CTAs
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmSA);
    tma_prefetch_desc(&tmSB);
    if (args.vec_out) tma_prefetch_desc(&tmOut);
  }
  cluster_sync();  // barriers of both CTAs initialised before any cross-CTA signal
  // Tensor memory is taken when the stream's previous kernel has ended (by warp
  // 1, beside the first loads), given back by both CTAs before either leaves,
  // and the right to allocate with it.  A pair that allocated while CTAs of the
  // previous kernels still came and went on its SMs, gave up the right at once
  // and left without waiting for each other, once in some 10^7 pairs stood still
  // for good: one CTA held its columns, the other waited for its own on an SM on
  // which nothing else ran.  (1024^3 6.3 us then, 6.6 now; 2048^3 10.8 both ways.)
  pdl_wait();
  constexpr uint32_t tmem_base = 0;  // where all 512 columns begin

  if (warp == 0) {
    // ------------------------------------------------------------ producers (both CTAs, one thread)
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true, issued = false;
      for (int tile = pair; tile < num_items && ok; tile += num_pairs) {
        int mb, nb;
        const int half = coords(tile, mb, nb);
        const int arow = mb * 256 + (int)rank * 128;
        const int bcol = nb * 256 + (half < 0 ? (int)rank * 128 : half * 128 + (int)rank * 64);
        for (int kb = 0; kb < args.num_k_blocks; kb++) {
          if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag)) { ok = false; break; }
          const uint32_t sa = base + stage * kPairStageBytes, sb = sa + kPairHalf * BK, ss = sf0 + stage * kP2SfSlot;
          const uint32_t fb = map_to_rank(full_bar(stage), 0);
          const bool scales = (kb & 3) == 0;
          if (leader) mbar_arrive_expect_tx(full_bar(stage), 2 * (kPairStageBytes + (scales ? kP2SfSlot : 0)));
          if (scales) {
            tma_load_3d_pair(ss, &tmSA, 0, kb >> 2, arow >> 7, fb);
            tma_load_3d_pair(ss + 512, &tmSB, 0, kb >> 2, nb * 2, fb);
          }
          if (A_MN) tma_load_2d_pair(sa, &tmA, arow, kb * BK, fb);
          else      tma_load_2d_pair(sa, &tmA, kb * BK, arow, fb);
          if (B_MN) tma_load_2d_pair(sb, &tmB, bcol, kb * BK, fb);
          else      tma_load_2d_pair(sb, &tmB, kb * BK, bcol, fb);
          issued = true;
          if (++stage == kP2Stages) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok && issued) sleep_ns_bounded(50000);  // let copies in flight land
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ tensor memory, MMA issuer (leader)
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(512u)
                 : "memory");
    // Not before the allocation: a dependent CTA that took tensor memory first
    // and then waited for this kernel would wait for good.
    pdl_launch_dependents();
    tc_fence_before();
    if (lane == 0) mbar_arrive_remote(map_to_rank(alloc_bar, 0));
    if (leader) {
      const bool elected = elect_one();
      const uint32_t a_d0 = (uint32_t)operand_desc<A_MN>(base, 0);
      const uint32_t b_d0 = (uint32_t)operand_desc<B_MN>(base + kPairHalf * BK, 0);
      constexpr uint32_t a_ks = A_MN ? (UMMA_K * 128) >> 4 : UMMA_K >> 4;
      constexpr uint32_t b_ks = B_MN ? (UMMA_K * 128) >> 4 : UMMA_K >> 4;
      constexpr uint32_t st_d = kPairStageBytes >> 4;
      int stage = 0, n = 0;
      uint32_t phase = 0, group = 0;
      bool ok = warp_ready(alloc_bar, 0, abort_flag), issued_any = false;
      tc_fence_after();
      for (int tile = pair; tile < num_items && ok; tile += num_pairs, n++) {
        if (n > 0 && !warp_ready(tempty_bar, (uint32_t)(n - 1) & 1u, abort_flag)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (n & 1) * kP2Acc1;
        const bool split = tile >= args.whole;
        const uint32_t shape = split ? args.idesc ^ ((256u >> 3) << 17) ^ ((128u >> 3) << 17) : args.idesc;
        const uint32_t sfb_off = split && ((tile - args.whole) & 1) ? 8u : 4u;
        for (int kb = 0; kb < args.num_k_blocks; kb++) {
          if (!warp_ready(full_bar(stage), phase, abort_flag)) { ok = false; break; }
          if ((kb & 3) == 0) {  // the set's last readers, two groups ago, have completed
            const uint32_t set = group & 1u;
            if (group >= 2 && !warp_ready(sffree_bar(set), ((group >> 1) - 1) & 1u, abort_flag)) {
              ok = false;
              break;
            }
            const uint32_t sf = tmem_base + kP2Sf + set * 16, ss = sf0 + stage * kP2SfSlot;
            if (elected) {
              tc_cp_scales_pair(sf, scale_desc(ss));
              tc_cp_scales_pair(sf + 4, scale_desc(ss + 512));
              tc_cp_scales_pair(sf + 8, scale_desc(ss + 1024));
            }
            group++;
          }
          const uint32_t sfa = tmem_base + kP2Sf + ((group - 1) & 1u) * 16;
          const uint32_t so = (uint32_t)stage * st_d;
          const uint32_t idesc = with_scale_ids(shape, kb);
          if (elected) {
#pragma unroll
            for (int ks = 0; ks < BK / UMMA_K; ks++)
              tc_mma_bs_pair(d_tmem, a_d0 + so + ks * a_ks, b_d0 + so + ks * b_ks, args.desc_hi, idesc, sfa, sfa + sfb_off,
                             (kb | ks) != 0 ? 1u : 0u);
            tc_commit_pair(empty_bar(stage));
            if ((kb & 3) == 3 || kb == args.num_k_blocks - 1) tc_commit_leader(sffree_bar((group - 1) & 1u));
          }
          issued_any = true;
          if (++stage == kP2Stages) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        if (elected) tc_commit_pair(tfull_bar(n & 1));
      }
      if (!ok && issued_any) {
        if (elected) tc_commit_leader(drain_bar);
        mbar_wait_drain(drain_bar, 0);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3;
    const uint32_t stg0 = out_stage0 + (warp - 2) * kP2OutBoxes * kWideStageOutBytes;
    const uint32_t bias_s = bar0 + 256 + (warp - 2) * 1024;
    constexpr int kBox = OUT == FP8_DT_F32 ? 32 : 64;  // columns of one 128-byte box
    constexpr int kNum = 256 / kBox;
    uint32_t box = 0;
    int n = 0;
    for (int tile = pair; tile < num_items; tile += num_pairs, n++) {
      int mb, nb;
      const int half = coords(tile, mb, nb);
      const int tile_col = nb * 256 + max(half, 0) * 128;
      if (args.bias) stage_bias(args, tile_col, bias_s);  // while the tile is multiplied
      const bool got = __all_sync(0xffffffffu, mbar_wait(tfull_bar(n & 1), (uint32_t)(n >> 1) & 1u, abort_flag));
      if (!got) break;
      tc_fence_after();
      const int row0 = mb * 256 + (int)rank * kPairHalf + q * 32;
      const uint32_t acc = tmem_base + ((uint32_t)(q * 32) << 16) + (n & 1) * kP2Acc1;
#pragma unroll 1
      for (int i = 0; i < (half < 0 ? kNum : kNum / 2); i++) {
        // the first accumulator's last columns, the second's first ones are shared: read them first
        // (a half tile in the first accumulator leaves the shared columns alone)
        const int c = ((n & 1) || half >= 0 ? i : (i + kNum - 1) % kNum) * kBox;
        const int col0 = tile_col + c;
        uint32_t w[32];
        uint32_t r[32];
        tmem_ld32(acc + c, r);
        if (args.bias) add_bias(bias_s + c * 4, r);
        if constexpr (OUT == FP8_DT_F32) {
#pragma unroll
          for (int j = 0; j < 32; j++) w[j] = r[j];
        } else {
#pragma unroll
          for (int j = 0; j < 16; j++) w[j] = pack_out<OUT>(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
          tmem_ld32(acc + c + 32, r);
          if (args.bias) add_bias(bias_s + (c + 32) * 4, r);
#pragma unroll
          for (int j = 0; j < 16; j++)
            w[16 + j] = pack_out<OUT>(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
        }
        if (i == 0) {  // the shared columns are read: the next tile may start
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(map_to_rank(tempty_bar, 0));
        }
        const uint32_t stg = stg0 + box * kWideStageOutBytes;
        box ^= 1u;
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        __syncwarp();
#pragma unroll
        for (int ch = 0; ch < 8; ch++) {  // 16-byte chunk ch of this row, 128B swizzle
          const uint32_t addr = stg + lane * 128 + ((ch ^ (lane & 7)) << 4);
          st_shared_v4(addr, w[4 * ch], w[4 * ch + 1], w[4 * ch + 2], w[4 * ch + 3]);
        }
        if (!args.vec_out) {
          // Rows that do not start on 16-byte boundaries: element stores, a warp
          // per row (a lane per row took five times as long, 32 sectors a store).
          __syncwarp();
          store_box_elements<OUT>(args, stg, row0, col0, lane);
          continue;
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
          if (row0 < args.rows && col0 < args.cols) tma_store_2d(&tmOut, stg, col0, row0);
          bulk_commit();
        }
      }
    }
    if (lane == 0) bulk_wait0();  // every store has landed before the CTA exits
    __syncwarp();
  }

  tc_fence_before();
  __syncwarp();
  cluster_sync();  // the leader's MMAs no longer read this CTA's smem / TMEM
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512u) : "memory");
  }
  __syncwarp();
  cluster_sync();  // neither CTA leaves before both have given their columns back
}

}  // namespace bgemm
}  // namespace fp8lib
