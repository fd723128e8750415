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
  int bn;                      // output columns per tile (a multiple of 32, at most 256)
  int stages, sf_atoms_b;      // ring depth; 512-byte scale groups loaded per tile for B
  uint32_t stage_bytes, tmem_cols;
  uint32_t idesc, desc_hi;
  const void *bias;            // per output feature, or null
  int bias_dtype;
  void *out;
  int out_dtype;
  size_t ld_out;               // elements
  int swap;                    // 0: out[r, c]; 1: out[c, r] (A holds the features, B the tokens)
  int vec_out;                 // rows of `out` start on 16-byte boundaries
  // tokens form: B is cast from x [cols, x_cols] inside the kernel
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

constexpr int kSfSlot = 2048;   // per stage: A's 512 bytes, then up to 3 x 512 of B
constexpr int kSfCols = 16;     // tensor-memory columns of one set of scales (4 + up to 12)
constexpr int kSfSets = 3;
// Sets of scale columns: a group of four blocks writes its set once and the
// next three groups write others.  A set is rewritten at the earliest nine
// blocks after its last block was multiplied; a ring of at most nine stages
// has by then seen those MMAs complete (its slot was refilled), so the copy
// cannot overtake a reader.
constexpr int kMaxStages = 9;
constexpr int kNoCast = -1;     // B comes as codes; otherwise the element type of x
constexpr int kTokens = 32;     // tokens form: columns of its tile

constexpr int kTokenBatch = 8;  // tokens that one warp casts at a time
constexpr int kTokenThreads = 64 + 8 * 32;
constexpr int kTokenPrefetch = 16;  // weight blocks (16 KB each) brought into L2 ahead
constexpr int kTokenStages = 5;  // the least ring depth of the tokens form (see its casting warps)

// Eight tokens' parts of one stage: x[t0 .. t0+7, k0 .. k0+127], 16 lanes per
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
    uint2 c = block::enc8<FP8_E4M3>(f, s4);
    if (nan) c = block::enc8_any<FP8_E4M3>(f, s4);
    const uint32_t at = tile + t * 128 + (((c8 >> 1) ^ (t & 7)) << 4) + (c8 & 1) * 8;
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(c.x), "r"(c.y) : "memory");
  }
}

__device__ __forceinline__ void store_one(const BArgs &a, size_t at, float y) {
  if (a.out_dtype == FP8_DT_F32) reinterpret_cast<float *>(a.out)[at] = y;
  else if (a.out_dtype == FP8_DT_BF16) reinterpret_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(y);
  else if (a.out_dtype == FP8_DT_F16) reinterpret_cast<__half *>(a.out)[at] = __float2half_rn(y);
  else reinterpret_cast<uint16_t *>(a.out)[at] = (uint16_t)(bf16x2_rto(y, y) & 0xffffu);
}

// Output chunk of 32 accumulator columns of one lane.  Not swapped: out[row,
// col0...]; swapped: out[col0 + j, row], so that the lanes of a warp write
// neighbouring features of a token.
// bias: of feature col0 + lane (not swapped) or of this row's feature (swapped), loaded by the caller.
__device__ __forceinline__ void store_out(const BArgs &a, float (&v)[32], int n, int row, int col0, float bias) {
  if (a.swap) {
    if (row >= a.rows) return;
#pragma unroll
    for (int j = 0; j < 32; j++)
      if (j < n && col0 + j < a.cols)
        store_one(a, (size_t)(col0 + j) * a.ld_out + row, a.bias ? __fadd_rn(v[j], bias) : v[j]);
    return;
  }
  if (a.bias) {
#pragma unroll
    for (int j = 0; j < 32; j++) v[j] = __fadd_rn(v[j], __shfl_sync(0xffffffffu, bias, j));
  }
  if (row >= a.rows) return;
#pragma unroll
  for (int c = 0; c < 32; c += 8) {
    if (c >= n || col0 + c >= a.cols) break;
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; j++) f[j] = v[c + j];
    const int cols = min(a.cols, col0 + n);
#define FP8_STORE(DT) block::store8<DT>(a.vec_out, a.out, a.ld_out, row, col0 + c, a.rows, cols, f)
    if (a.out_dtype == FP8_DT_F32) FP8_STORE(FP8_DT_F32);
    else if (a.out_dtype == FP8_DT_BF16) FP8_STORE(FP8_DT_BF16);
    else if (a.out_dtype == FP8_DT_F16) FP8_STORE(FP8_DT_F16);
    else FP8_STORE(FP8_DT_BF16_RTO);
#undef FP8_STORE
  }
}

__device__ __forceinline__ float chunk_bias(const BArgs &a, int row, int col0) {
  const int i = a.swap ? row : col0 + (int)(threadIdx.x & 31);
  return a.bias && i < (a.swap ? a.rows : a.cols) ? load_bias(a.bias, a.bias_dtype, i) : 0.0f;
}

// ---------------------------------------------------------------------------
// One-CTA kernel: a tile of 128 x bn outputs per cluster of S CTAs, each of
// which reduces its share of the k-blocks (S = 1: no cluster).  Each CTA then
// sends every other its part of the partial tile through distributed shared
// memory (posted stores; reading the others' parts instead cost 12 us at 128
// columns), adds the S partial sums of its own bn / S columns in rank order
// and stores them: no workspace, no atomics, the same bits each time.
//   warp 0 TMA producer, warp 1 TMEM allocation and MMA issue, warps 2-5 epilogue.
// XDT != kNoCast is the form for few tokens: A holds the weights, and eight
// warps (four of them the epilogue's, idle until the accumulator is complete)
// cast the tokens' activations into the ring, eight tokens of one stage at a
// time, the next ones' loads in flight meanwhile, so that one launch does what
// the cast and the product do.  Bound by the weights' HBM traffic.
template <bool A_MN, bool B_MN, int XDT>
__global__ void __launch_bounds__(XDT == kNoCast ? kThreads : kTokenThreads)
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
  const int tile = blockIdx.x / splits;
  // this CTA's k-blocks
  const int kb0 = (int)((long long)args.num_k_blocks * rank / splits);
  const int kb1 = (int)((long long)args.num_k_blocks * (rank + 1) / splits);
  int mb, nb;
  {
    const int per_band = args.group_m * args.num_n_blocks;
    const int band = tile / per_band, first = band * args.group_m;
    const int rows_in_band = min(args.num_m_blocks - first, args.group_m);
    const int r = tile - band * per_band;
    mb = first + r % rows_in_band;
    nb = r / rows_in_band;
  }
  const int row0 = mb * BM, col0 = nb * args.bn;

  constexpr bool CAST = XDT != kNoCast;
  constexpr int kNumThreads = CAST ? kTokenThreads : kThreads;
  const int batches = (args.cols + kTokenBatch - 1) / kTokenBatch;  // tokens form: casts per stage
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; s++) {
      mbar_init(full_bar(s), CAST ? 1 + batches : 1);  // the producer's arrive, and the casting warps'
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(tfull_bar, 1);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmSA);
    if (!CAST) {
      tma_prefetch_desc(&tmB);
      tma_prefetch_desc(&tmSB);
    }
  }
  if constexpr (CAST) {  // token rows the cast never writes are zero
    for (int i = threadIdx.x; i < S * (kTokens * BK + 512) / 16; i += kNumThreads) {
      const int s = i / ((kTokens * BK + 512) / 16), o = (i % ((kTokens * BK + 512) / 16)) * 16;
      const uint32_t at = o < kTokens * BK ? base + s * args.stage_bytes + BM * BK + o
                                           : sf0 + s * kSfSlot + 512 + (o - kTokens * BK);
      st_shared_v4(at, 0u, 0u, 0u, 0u);
    }
    fence_async_shared();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(args.tmem_cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // Not before the allocation: a dependent CTA that took tensor memory first
  // and then waited for this kernel would wait for good.
  pdl_launch_dependents();
  // Tokens form: the first weights come into L2 while the stream's previous
  // kernel ends.  (L2 is where its writes go too, so a weight that it still
  // writes is read as written by the loads after the wait.)
  if (CAST && threadIdx.x == 0)
    for (int kb = kb0; kb < min(kb1, kb0 + kTokenPrefetch); kb++) tma_prefetch_2d(&tmA, kb * BK, row0);
  pdl_wait();
  const uint32_t sf_bytes = 512u + 512u * args.sf_atoms_b;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued_mask = 0, issued_par = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; kb++) {
        if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag)) { ok = false; break; }
        const uint32_t sa = base + stage * args.stage_bytes, sb = sa + BM * BK, ss = sf0 + stage * kSfSlot;
        const bool scales = kb == kb0 || (kb & 3) == 0;
        mbar_arrive_expect_tx(full_bar(stage), (CAST ? (uint32_t)(BM * BK) : args.stage_bytes) +
                                                   (scales ? (CAST ? 512u : sf_bytes) : 0u));
        if (scales) {
          tma_load_3d(ss, &tmSA, 0, kb >> 2, row0 >> 7, full_bar(stage));
          if (!CAST) tma_load_3d(ss + 512, &tmSB, 0, kb >> 2, col0 >> 7, full_bar(stage));
        }
        if (A_MN) tma_load_2d(sa, &tmA, row0, kb * BK, full_bar(stage));
        else      tma_load_2d(sa, &tmA, kb * BK, row0, full_bar(stage));
        if (CAST) {
        } else if (B_MN) {
          for (int c = 0; c < args.bn; c += 128)
            tma_load_2d(sb + c * BK, &tmB, col0 + c, kb * BK, full_bar(stage));
        } else {
          tma_load_2d(sb, &tmB, kb * BK, col0, full_bar(stage));
        }
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
    if (lane == 0) {
      const uint32_t a_d0 = (uint32_t)operand_desc<A_MN>(base, 0), b_d0 = (uint32_t)operand_desc<B_MN>(base + BM * BK, 0);
      constexpr uint32_t a_ks = A_MN ? (UMMA_K * 128) >> 4 : UMMA_K >> 4;
      constexpr uint32_t b_ks = B_MN ? (UMMA_K * 128) >> 4 : UMMA_K >> 4;
      const uint32_t st_d = args.stage_bytes >> 4;
      // the scales of a tile that starts inside a 128-row group: skip whole 32-row columns
      const uint32_t sfb_skip = (uint32_t)(col0 & 127) >> 5;
      const uint32_t sf_tmem = tmem_base + args.bn;
      int stage = 0, set = kSfSets - 1;
      uint32_t phase = 0;
      bool ok = true, issued_any = false;
      for (int kb = kb0; kb < kb1; kb++) {
        if (!stage_ready(full_bar(stage), phase, abort_flag)) { ok = false; break; }
        if (kb == kb0 || (kb & 3) == 0) {
          set = set == kSfSets - 1 ? 0 : set + 1;
          const uint32_t t = sf_tmem + set * kSfCols, ss = sf0 + stage * kSfSlot;
          tc_cp_scales(t, scale_desc(ss));
          if (!CAST)
            for (int i = 0; i < args.sf_atoms_b; i++) tc_cp_scales(t + 4 + 4 * i, scale_desc(ss + 512 + 512 * i));
        }
        const uint32_t sfa = sf_tmem + set * kSfCols;
        uint32_t sfb = sfa + 4 + sfb_skip;
        if (CAST) {  // every stage brings its own token scales; their columns belong to the ring slot
          sfb = sf_tmem + kSfSets * kSfCols + 4 * stage;
          tc_cp_scales(sfb, scale_desc(sf0 + stage * kSfSlot + 512));
        }
        const uint32_t so = (uint32_t)stage * st_d;
        const uint32_t idesc = with_scale_ids(args.idesc, kb);
#pragma unroll
        for (int ks = 0; ks < BK / UMMA_K; ks++)
          tc_mma_bs(tmem_base, a_d0 + so + ks * a_ks, b_d0 + so + ks * b_ks, args.desc_hi, idesc, sfa, sfb,
                    (kb != kb0 || ks != 0) ? 1u : 0u);
        tc_commit(empty_bar(stage));
        issued_any = true;
        if (++stage == S) { stage = 0; phase ^= 1u; }
      }
      if (ok) {
        tc_commit(tfull_bar);
      } else if (issued_any) {
        tc_commit(drain_bar);
        mbar_wait_drain(drain_bar, 0);
      }
    }
    __syncwarp();
  } else {
    const int q = warp & 3;
    const int row = row0 + q * 32 + lane;
    if constexpr (CAST) {
      // Unit u: batch u % batches of block kb0 + u / batches; the casting warps
      // take them in turn.  At most 4 * batches warps do, so that a warp's next
      // unit is at most four blocks on: a parity wait tells only one phase of a
      // ring slot from the next, and a warp that skipped a whole turn of the
      // ring (five stages at the least) could take an older phase for its own.
      const int units = (kb1 - kb0) * batches, step = min(8, 4 * batches);
      block::Raw8<XDT> raw[4];
      int u = warp - 2 < step ? warp - 2 : units;
      if (u < units) load_tokens<XDT>(args, u % batches * kTokenBatch, (kb0 + u / batches) * BK, lane, raw);
      for (; u < units; u += step) {
        const int i = u / batches, stage = i % S, t0 = u % batches * kTokenBatch;
        block::Raw8<XDT> next[4];
        const int un = min(u + step, units - 1);
        load_tokens<XDT>(args, un % batches * kTokenBatch, (kb0 + un / batches) * BK, lane, next);
        if (!__all_sync(0xffffffffu, mbar_wait(empty_bar(stage), ((uint32_t)(i / S) & 1u) ^ 1u, abort_flag))) break;
        cast_tokens<XDT>(args, t0, kb0 + i, base + stage * args.stage_bytes + BM * BK, sf0 + stage * kSfSlot + 512,
                         lane, raw);
        fence_async_shared();  // the MMAs and the scale copy read through the async proxy
        __syncwarp();
        if (lane == 0) mbar_arrive(full_bar(stage));
#pragma unroll
        for (int j = 0; j < 4; j++) raw[j] = next[j];
      }
      __syncwarp();
    }
    if (warp < 6) {
      float bias = args.swap && splits == 1 ? chunk_bias(args, row, 0) : 0.0f;
      const bool got = __all_sync(0xffffffffu, mbar_wait(tfull_bar, 0, abort_flag));
      tc_fence_after();
      if (got && splits == 1) {
#pragma unroll 1
        for (int c = 0; c < args.bn && col0 + c < args.cols; c += 32) {
          if (!args.swap) bias = chunk_bias(args, row, col0 + c);
          uint32_t r[32];
          tmem_ld32(tmem_base + ((uint32_t)(q * 32) << 16) + c, r);
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; j++) v[j] = __uint_as_float(r[j]);
          store_out(args, v, 32, row, col0 + c, bias);
        }
      }
      tc_fence_before();
      __syncwarp();
    }
  }

  if (splits > 1) {
    // Columns in units of 8 (a vector store), or 4 where the columns are
    // tokens; unit u is finished by CTA u % S, as its unit u / S.  The partial
    // of CTA s arrives at slot s of the owner's ring: per unit, groups of 4
    // columns x 128 rows x 16 bytes.
    const int unit = args.swap ? 4 : 8, groups = unit / 4;
    const int cols = min(args.bn, args.cols - col0), units = (cols + unit - 1) / unit;
    const int per = (units + splits - 1) / splits;
    cluster_sync();  // every CTA's MMAs have read their ring
    const int q = warp & 3, row = row0 + q * 32 + lane;
    float bias = 0.0f;
    if (warp >= 2 && warp < 6) {
      if (args.swap) bias = chunk_bias(args, row, 0);
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < cols; c += 32) {
        uint32_t r[32];
        tmem_ld32(tmem_base + ((uint32_t)(q * 32) << 16) + c, r);
#pragma unroll
        for (int g = 0; g < 8; g++) {
          const int u = (c + 4 * g) / unit;
          if (c + 4 * g >= cols) break;
          const uint32_t dst = map_to_rank(base, (uint32_t)(u % splits)) +
                               (((rank * per + u / splits) * groups + (g & (groups - 1))) * BM + q * 32 + lane) * 16;
          asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(r[4 * g]),
                       "r"(r[4 * g + 1]), "r"(r[4 * g + 2]), "r"(r[4 * g + 3])
                       : "memory");
        }
      }
      tc_fence_before();
    }
    cluster_sync();  // all parts have arrived
    if (warp >= 2 && warp < 6) {
#pragma unroll 1
      for (int i = 0, u = rank; u < units; i++, u += splits) {
        if (!args.swap) bias = chunk_bias(args, row, col0 + u * unit);
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; j++) v[j] = 0.0f;
#pragma unroll 2
        for (int s = 0; s < splits; s++) {
#pragma unroll
          for (int h = 0; h < 2; h++) {
            if (h >= groups) break;
            float x[4];
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3])
                         : "r"(base + (((s * per + i) * groups + h) * BM + q * 32 + lane) * 16)
                         : "memory");
#pragma unroll
            for (int j = 0; j < 4; j++) v[4 * h + j] = __fadd_rn(v[4 * h + j], x[j]);
          }
        }
        store_out(args, v, unit, row, col0 + u * unit, bias);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(args.tmem_cols)
                 : "memory");
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
//   warp 0 TMA producer (both CTAs), warp 1 TMEM allocation and MMA issue
//   (leader), warps 2-5 epilogue (both CTAs).
constexpr int kP2Stages = 5;
constexpr int kP2SfSlot = 512 + 1024;
constexpr int kP2Acc1 = 224;    // first column of the second accumulator
constexpr int kP2Sf = 480;      // two sets of scales, 16 columns each
constexpr int kP2OutBoxes = 2;  // staging boxes per epilogue warp (stores pipelined)
constexpr int kP2SmemBytes =
    kP2Stages * (kPairStageBytes + kP2SfSlot) + 4 * kP2OutBoxes * kWideStageOutBytes + 256 + 1024;

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
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(base_ptr + (bar0 - base) + 8 * (2 * kP2Stages + 6));
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
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmSA);
    tma_prefetch_desc(&tmSB);
    if (args.vec_out) tma_prefetch_desc(&tmOut);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  cluster_sync();  // barriers of both CTAs initialised before any cross-CTA signal
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // Not before the allocation: a dependent CTA that took tensor memory first
  // and then waited for this kernel would wait for good.
  pdl_launch_dependents();
  pdl_wait();

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
    // ------------------------------------------------------------ MMA issuer (leader, one thread)
    if (leader && lane == 0) {
      const uint32_t a_d0 = (uint32_t)operand_desc<A_MN>(base, 0);
      const uint32_t b_d0 = (uint32_t)operand_desc<B_MN>(base + kPairHalf * BK, 0);
      constexpr uint32_t a_ks = A_MN ? (UMMA_K * 128) >> 4 : UMMA_K >> 4;
      constexpr uint32_t b_ks = B_MN ? (UMMA_K * 128) >> 4 : UMMA_K >> 4;
      constexpr uint32_t st_d = kPairStageBytes >> 4;
      int stage = 0, n = 0;
      uint32_t phase = 0, group = 0;
      bool ok = true, issued_any = false;
      for (int tile = pair; tile < num_items && ok; tile += num_pairs, n++) {
        if (n > 0 && !mbar_wait(tempty_bar, (uint32_t)(n - 1) & 1u, abort_flag)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (n & 1) * kP2Acc1;
        const bool split = tile >= args.whole;
        const uint32_t shape = split ? args.idesc ^ ((256u >> 3) << 17) ^ ((128u >> 3) << 17) : args.idesc;
        const uint32_t sfb_off = split && ((tile - args.whole) & 1) ? 8u : 4u;
        for (int kb = 0; kb < args.num_k_blocks; kb++) {
          if (!stage_ready(full_bar(stage), phase, abort_flag)) { ok = false; break; }
          if ((kb & 3) == 0) {  // the set's last readers, two groups ago, have completed
            const uint32_t set = group & 1u;
            if (group >= 2 && !stage_ready(sffree_bar(set), ((group >> 1) - 1) & 1u, abort_flag)) {
              ok = false;
              break;
            }
            const uint32_t sf = tmem_base + kP2Sf + set * 16, ss = sf0 + stage * kP2SfSlot;
            tc_cp_scales_pair(sf, scale_desc(ss));
            tc_cp_scales_pair(sf + 4, scale_desc(ss + 512));
            tc_cp_scales_pair(sf + 8, scale_desc(ss + 1024));
            group++;
          }
          const uint32_t sfa = tmem_base + kP2Sf + ((group - 1) & 1u) * 16;
          const uint32_t so = (uint32_t)stage * st_d;
          const uint32_t idesc = with_scale_ids(shape, kb);
#pragma unroll
          for (int ks = 0; ks < BK / UMMA_K; ks++)
            tc_mma_bs_pair(d_tmem, a_d0 + so + ks * a_ks, b_d0 + so + ks * b_ks, args.desc_hi, idesc, sfa, sfa + sfb_off,
                           (kb | ks) != 0 ? 1u : 0u);
          tc_commit_pair(empty_bar(stage));
          if ((kb & 3) == 3 || kb == args.num_k_blocks - 1) tc_commit_leader(sffree_bar((group - 1) & 1u));
          issued_any = true;
          if (++stage == kP2Stages) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        tc_commit_pair(tfull_bar(n & 1));
      }
      if (!ok && issued_any) {
        tc_commit_leader(drain_bar);
        mbar_wait_drain(drain_bar, 0);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3;
    const uint32_t stg0 = out_stage0 + (warp - 2) * kP2OutBoxes * kWideStageOutBytes;
    constexpr int kBox = OUT == FP8_DT_F32 ? 32 : 64;  // columns of one 128-byte box
    constexpr int kNum = 256 / kBox;
    uint32_t box = 0;
    int n = 0;
    for (int tile = pair; tile < num_items; tile += num_pairs, n++) {
      int mb, nb;
      const int half = coords(tile, mb, nb);
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
        const int col0 = nb * 256 + max(half, 0) * 128 + c;
        uint32_t w[32];
        const float bias0 = chunk_bias(args, 0, col0);
        const float bias1 = OUT == FP8_DT_F32 ? 0.0f : chunk_bias(args, 0, col0 + 32);
        uint32_t r[32];
        tmem_ld32(acc + c, r);
        if (args.bias) {
#pragma unroll
          for (int j = 0; j < 32; j++)
            r[j] = __float_as_uint(__fadd_rn(__uint_as_float(r[j]), __shfl_sync(0xffffffffu, bias0, j)));
        }
        if constexpr (OUT == FP8_DT_F32) {
#pragma unroll
          for (int j = 0; j < 32; j++) w[j] = r[j];
        } else {
#pragma unroll
          for (int j = 0; j < 16; j++) w[j] = pack_out<OUT>(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
          tmem_ld32(acc + c + 32, r);
          if (args.bias) {
#pragma unroll
            for (int j = 0; j < 32; j++)
              r[j] = __float_as_uint(__fadd_rn(__uint_as_float(r[j]), __shfl_sync(0xffffffffu, bias1, j)));
          }
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
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512u) : "memory");
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

}  // namespace bgemm
}  // namespace fp8lib
