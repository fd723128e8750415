// loss.cuh -- what stands behind the last linear layer: log probabilities of
// given tokens with the entropy and the largest alternatives, distillation from
// a teacher's top logits, and the gradients of the logits, also as codes of
// 1x128 and 128x1 blocks for the products that follow.
//
// For a row z of logits and s = beta z, with m the largest z:
//   S = sum e^(s - beta m),  W = sum (s - beta m) e^(s - beta m)
//   log p_j = s_j - beta m - log S,   entropy = log S - W / S
// in one pass: each thread keeps the m, S and W of what it has seen and scales
// S and W down when m grows; the threads' are joined at the end.
//
//   d logp_t   / d z_j = beta ([j = t] - p_j)
//   d entropy  / d z_j = -beta p_j (log p_j + entropy)
//   distillation:  beta (p_j factor - q_j)
#pragma once

#include "block_scale.cuh"
#include "pipeline.cuh"

namespace fp8lib {
namespace loss {

using block::Raw8;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNone = -3.402823466e38f;  // below every logit but -inf
constexpr int kTop = FP8_TOP_MAX;
constexpr int kCandidates = 2048;
constexpr int kAbsent = 0x7fffffff;

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Elements of a 16-byte vector.
template <int DT>
constexpr int kElems = DT == FP8_DT_F32 ? 4 : 8;
template <int DT>
constexpr int kSize = DT == FP8_DT_F32 ? 4 : 2;

template <int DT>
__device__ __forceinline__ void unpack(uint4 v, float (&f)[kElems<DT>]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    if constexpr (DT == FP8_DT_F32) {
      f[i] = __uint_as_float(w[i]);
    } else if constexpr (DT == FP8_DT_BF16) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      const float2 h = h2f2(w[i]);
      f[2 * i] = h.x;
      f[2 * i + 1] = h.y;
    }
  }
}

template <int DT>
__device__ __forceinline__ float load_one(const uint8_t *row, int i) {
  if constexpr (DT == FP8_DT_F32) return reinterpret_cast<const float *>(row)[i];
  const uint16_t h = reinterpret_cast<const uint16_t *>(row)[i];
  return DT == FP8_DT_BF16 ? __uint_as_float((uint32_t)h << 16) : __half2float(__ushort_as_half(h));
}

template <int DT>
__device__ __forceinline__ void store_one(uint8_t *row, int i, float x) {
  if constexpr (DT == FP8_DT_F32) reinterpret_cast<float *>(row)[i] = x;
  else if constexpr (DT == FP8_DT_BF16) reinterpret_cast<__nv_bfloat16 *>(row)[i] = __float2bfloat16_rn(x);
  else reinterpret_cast<__half *>(row)[i] = __float2half_rn(x);
}

// A row as 16-byte vectors: `head` elements before the first boundary, `vecs`
// vectors, and the rest, fewer than a vector's.
struct RowShape {
  int head, vecs, tail;
};
template <int DT>
__device__ __forceinline__ RowShape row_shape(const uint8_t *row, int cols) {
  RowShape s;
  s.head = min(cols, (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / kSize<DT>);
  s.vecs = (cols - s.head) / kElems<DT>;
  s.tail = cols - s.head - s.vecs * kElems<DT>;
  return s;
}

__device__ __forceinline__ long long index_at(const void *p, int bytes, size_t i) {
  return bytes == 8 ? reinterpret_cast<const long long *>(p)[i] : (long long)reinterpret_cast<const int *>(p)[i];
}

// A token that counts, or -1.
__device__ __forceinline__ int token_at(const void *tokens, int bytes, int row, int cols) {
  if (!tokens) return -1;
  const long long t = index_at(tokens, bytes, row);
  if (t >= cols) atomicOr(&g_status, FP8_STATUS_BAD_INDEX);
  return t >= 0 && t < cols ? (int)t : -1;
}

// Order of logits as unsigned integers: NaN above all, -0 as +0; 0 for none.
__device__ __forceinline__ uint32_t order_key(float z) {
  if (z != z) return 0xffffffffu;
  const uint32_t u = __float_as_uint(z == 0.0f ? 0.0f : z);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k == 0xffffffffu ? 0x7fffffffu : k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

struct Fwd {
  const uint8_t *z;
  size_t ld;  // bytes
  int rows, cols;
  float beta;
  // log probabilities
  const void *tokens;
  int token_bytes, top;
  float *logp, *entropy, *top_logp, *stats;
  int *top_ids;
  // distillation
  const void *ids;
  int id_bytes, value_dt;
  const void *values;
  float *loss, *list_q;
  int *list_ids;
};

enum { kLogprob = 0, kListTop = 1, kListTail = 2 };

struct Part {  // of a row: what one CTA has seen
  float m, S, W, rest;
};

// Sum over the CTA in a fixed order; every thread gets it.
__device__ __forceinline__ float block_sum(float v, float *red) {
#pragma unroll
  for (int b = 16; b > 0; b /= 2) v += __shfl_xor_sync(0xffffffffu, v, b);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (threadIdx.x & 31) < (blockDim.x >> 5) ? red[threadIdx.x & 31] : 0.0f;
#pragma unroll
  for (int b = 16; b > 0; b /= 2) v += __shfl_xor_sync(0xffffffffu, v, b);
  return __shfl_sync(0xffffffffu, v, 0);
}
__device__ __forceinline__ float block_max(float v, float *red) {
#pragma unroll
  for (int b = 16; b > 0; b /= 2) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, b));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (threadIdx.x & 31) < (blockDim.x >> 5) ? red[threadIdx.x & 31] : kNone;
#pragma unroll
  for (int b = 16; b > 0; b /= 2) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, b));
  return __shfl_sync(0xffffffffu, v, 0);
}

__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_at(uint32_t addr, unsigned rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

// What a CTA reads of its row: the vectors [v0, v1), and with the first CTA the
// head, with the last one the tail.
struct Range {
  const uint8_t *row, *body;
  RowShape s;
  int v0, v1, head, tail;
};

template <int DT>
__device__ __forceinline__ Range range_of(const uint8_t *row, int cols, unsigned rank, unsigned ctas) {
  Range r;
  r.row = row;
  r.s = row_shape<DT>(row, cols);
  r.body = row + (size_t)r.s.head * kSize<DT>;
  const int share = (int)((r.s.vecs + ctas - 1) / ctas);
  r.v0 = min(r.s.vecs, (int)rank * share);
  r.v1 = min(r.s.vecs, r.v0 + share);
  r.head = rank == 0 ? r.s.head : 0;
  r.tail = rank == ctas - 1 ? r.s.tail : 0;
  return r;
}

// Calls f(column, logit) for every element of the range that this thread owns.
template <int DT, typename F>
__device__ __forceinline__ void each_own(const Range &r, F f) {
  const int t = threadIdx.x;
  if (t < r.head) f(t, load_one<DT>(r.row, t));
  for (int v = r.v0 + t; v < r.v1; v += blockDim.x) {
    float x[kElems<DT>];
    unpack<DT>(__ldg(reinterpret_cast<const uint4 *>(r.body) + v), x);
#pragma unroll
    for (int j = 0; j < kElems<DT>; j++) f(r.s.head + v * kElems<DT> + j, x[j]);
  }
  const int c = r.s.head + r.s.vecs * kElems<DT> + t - r.head;
  if (t >= r.head && t < r.head + r.tail) f(c, load_one<DT>(r.row, c));
}

struct TopScratch {
  unsigned long long list[kCandidates];  // (key, ~column): larger is earlier
  uint32_t group[32];
  int above, equal, ties;
  uint32_t bound;
  unsigned long long best[kTop];
  int wsum[32];
};

__device__ __forceinline__ unsigned long long candidate(uint32_t key, int col) {
  return (unsigned long long)key << 32 | (uint32_t)~col;
}

// The `top` first candidates of a list of n, in order, to out (0: none).
__device__ __forceinline__ void rank_list(const unsigned long long *list, int n, int top, unsigned long long *out) {
  for (int i = threadIdx.x; i < top; i += blockDim.x) out[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const unsigned long long c = list[i];
    int before = 0;
    for (int j = 0; j < n && before < top; j++) before += list[j] > c;
    if (before < top && c) out[before] = c;
  }
  __syncthreads();
}

// The `top` largest logits of the CTA's range, in order, to sh.best.  `most` is
// the thread's own largest.  The top-th largest maximum of 32 groups of threads
// is a bound that at least `top` elements reach; few others do, and only threads
// that own one read their elements again.  Where many are equal to the bound (a
// masked vocabulary) those of the lowest columns are taken in order; where too
// many lie above it the bound is raised by bisection.
template <int DT>
__device__ void top_of_range(const Range &r, float most, bool any, int top, TopScratch &sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const uint32_t own = any ? order_key(most) : 0u;
  const int per = warps;  // threads of a group: blockDim.x / 32, a power of two
  uint32_t g = own;
  for (int b = per / 2; b > 0; b /= 2) g = max(g, __shfl_xor_sync(0xffffffffu, g, b));
  if (threadIdx.x % per == 0) sh.group[threadIdx.x / per] = g;
  if (threadIdx.x == 0) sh.above = sh.equal = 0;
  __syncthreads();
  if (warp == 0) {
    const uint32_t k = sh.group[lane];
    int before = 0;
    for (int j = 0; j < 32; j++) {
      const uint32_t o = __shfl_sync(0xffffffffu, k, j);
      before += o > k || (o == k && j < lane);
    }
    if (before == top - 1) sh.bound = k;
  }
  __syncthreads();
  uint32_t bound = sh.bound;
  // candidates above the bound from the front, equal ones from the back
  auto collect = [&] {
    if (own >= bound)
      each_own<DT>(r, [&](int c, float z) {
        const uint32_t k = order_key(z);
        if (k > bound) {
          const int i = atomicAdd(&sh.above, 1);
          if (i < kCandidates / 2) sh.list[i] = candidate(k, c);
        } else if (k == bound) {
          const int i = atomicAdd(&sh.equal, 1);
          if (i < kCandidates / 2) sh.list[kCandidates - 1 - i] = candidate(k, c);
        }
      });
    __syncthreads();
  };
  collect();
  if (sh.above > kCandidates / 2) {
    // the largest bound that `top` elements reach: fewer than `top` lie above it
    uint32_t lo = bound, hi = 0xffffffffu;  // reached by enough; hi's successor by none
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo) / 2 + 1;
      __syncthreads();
      if (threadIdx.x == 0) sh.ties = 0;
      __syncthreads();
      int count = 0;
      if (own >= mid) each_own<DT>(r, [&](int, float z) { count += order_key(z) >= mid; });
      if (count) atomicAdd(&sh.ties, count);
      __syncthreads();
      if (sh.ties >= top) lo = mid;
      else hi = mid - 1;
    }
    bound = lo;
    __syncthreads();
    if (threadIdx.x == 0) sh.above = sh.equal = 0;
    __syncthreads();
    collect();
  }
  const int above = sh.above, equal = sh.equal;
  int n = above;
  if (equal <= kCandidates / 2) {
    // close the gap between the two ends
    unsigned long long mine[kCandidates / 2 / 128];
    int k = 0;
    for (int i = threadIdx.x; i < equal; i += blockDim.x) mine[k++] = sh.list[kCandidates - 1 - i];
    __syncthreads();
    k = 0;
    for (int i = threadIdx.x; i < equal; i += blockDim.x) sh.list[above + i] = mine[k++];
    n += equal;
    __syncthreads();
  } else if (above < top) {
    // the first top - above elements that equal the bound, by column
    int have = 0;
    const int want = top - above;
    auto round = [&](int c0, int count, auto load) {  // elements c0 .. c0 + count: one of each thread's
      const int c = c0 + threadIdx.x;
      const bool hit = (int)threadIdx.x < count && order_key(load(c)) == bound;
      const unsigned votes = __ballot_sync(0xffffffffu, hit);
      if (lane == 0) sh.wsum[warp] = __popc(votes);
      __syncthreads();
      int before = have + __popc(votes & ((1u << lane) - 1)), total = 0;
      for (int w = 0; w < warps; w++) {
        before += w < warp ? sh.wsum[w] : 0;
        total += sh.wsum[w];
      }
      if (hit && before < want) sh.list[above + before] = candidate(bound, c);
      have += total;
      __syncthreads();
    };
    auto load = [&](int c) { return load_one<DT>(r.row, c); };
    const int c0 = r.head ? 0 : r.s.head + r.v0 * kElems<DT>;
    const int c1 = r.tail ? r.s.head + r.s.vecs * kElems<DT> + r.tail : r.s.head + r.v1 * kElems<DT>;
    for (int c = c0; c < c1 && have < want; c += blockDim.x) round(c, min((int)blockDim.x, c1 - c), load);
    n += min(have, want);
  }
  rank_list(sh.list, n, top, sh.best);
}

struct ListScratch {
  int id[FP8_DISTILL_MAX];
};

// Running softmax of a row's elements and, for kListTail, of the unlisted ones
// alone (`marks`: a bit for each element of the body, by its place there).
template <int DT, int MODE, bool ENT>
__device__ __forceinline__ Part stream_row(const Range &r, float c2, const uint8_t *marks, uint32_t edge_marks,
                                           float &most, bool &any) {
  float m = kNone, S = 0.0f, W = 0.0f, L = 0.0f;  // L: of the listed ones
  float largest = -INFINITY;
  bool got = false;
  // n elements; bits: which of them are listed
  auto add = [&](const float *x, int n, uint32_t bits) {
    float t = x[0];
#pragma unroll
    for (int j = 1; j < n; j++) t = max_nan(t, x[j]);
    if constexpr (MODE == kLogprob) largest = max_nan(largest, t);
    const float m1 = max_nan(m, t);
    float d = (m - m1) * c2;
    if constexpr (ENT) {
      d = max_nan(d, -1000.0f);
      W = fmaf(S, d, W);
    }
    const float down = ex2(d);
    S *= down;
    if constexpr (MODE == kListTail) L *= down;
    if constexpr (ENT) W *= down;
    m = m1;
#pragma unroll
    for (int j = 0; j < n; j++) {
      float a = (x[j] - m) * c2;
      if constexpr (ENT) a = max_nan(a, -1000.0f);
      const float e = ex2(a);
      if constexpr (MODE == kListTail) {
        if (bits >> j & 1) L += e;
        else S += e;
      } else {
        S += e;
      }
      if constexpr (ENT) W = fmaf(e, a, W);
    }
    got = true;
  };
  const int t = threadIdx.x;
  if (t < r.head + r.tail) {
    const float x[1] = {load_one<DT>(r.row, t < r.head ? t : r.s.head + r.s.vecs * kElems<DT> + t - r.head)};
    add(x, 1, edge_marks >> (t < r.head ? t : 16 + t - r.head) & 1);
  }
  for (int v = r.v0 + t; v < r.v1; v += blockDim.x) {
    float x[kElems<DT>];
    unpack<DT>(__ldg(reinterpret_cast<const uint4 *>(r.body) + v), x);
    uint32_t bits = 0;
    if constexpr (MODE == kListTail) {
      const int at = (v - r.v0) * kElems<DT>;
      bits = marks[at >> 3] >> (at & 7);
    }
    add(x, kElems<DT>, bits);
  }
  most = largest;
  any = got;
  // (a thread that has seen only -inf has m = kNone: its parts are 0)
  return {m, S, W, L};
}

// The parts of several threads or CTAs joined.  W is in units of log 2.
template <int MODE, bool ENT>
__device__ __forceinline__ Part join_block(Part p, float c2, float *red) {
  const float m = block_max(p.m, red);
  float d = (p.m - m) * c2;
  if constexpr (ENT) {
    d = max_nan(d, -1000.0f);
    p.W = fmaf(p.S, d, p.W);
  }
  const float down = ex2(d);
  Part o = {m, block_sum(p.S * down, red), 0.0f, 0.0f};
  if constexpr (ENT) o.W = block_sum(p.W * down, red);
  if constexpr (MODE == kListTail) o.rest = block_sum(p.rest * down, red);
  return o;
}

template <int DT, int MODE, bool ENT>
__global__ void __launch_bounds__(1024) k_loss_fwd(const Fwd p, unsigned ctas) {
  pdl_launch_dependents();
  pdl_wait();
  extern __shared__ __align__(16) uint8_t loss_smem[];
  __shared__ float red[32];
  __shared__ Part parts[8];
  __shared__ uint32_t edge_bits;
  const unsigned rank = ctas > 1 ? blockIdx.x % ctas : 0;
  const int row = (int)(blockIdx.x / ctas);
  const uint8_t *z = p.z + (size_t)row * p.ld;
  const Range r = range_of<DT>(z, p.cols, rank, ctas);
  const float c2 = p.beta * kLog2e;
  ListScratch &list = *reinterpret_cast<ListScratch *>(loss_smem);
  uint8_t *marks = loss_smem + sizeof(ListScratch);
  float q_sum = 0.0f, top_value = 0.0f, mine_v[4], mine_q[4];
  int mine_id[4], mine_at[4];
  if constexpr (MODE != kLogprob) {
    // the list by id: an entry's place is the number of entries that come before it
    const int K = p.top;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int k = threadIdx.x + i * blockDim.x;
      mine_id[i] = kAbsent;
      mine_v[i] = -INFINITY;
      mine_at[i] = 0;
      if (k < K) {
        const size_t at = (size_t)row * K + k;
        const long long id = index_at(p.ids, p.id_bytes, at);
        if (id >= p.cols) atomicOr(&g_status, FP8_STATUS_BAD_INDEX);
        if (p.value_dt == FP8_DT_F32) {
          mine_v[i] = reinterpret_cast<const float *>(p.values)[at];
        } else {
          const uint16_t h = reinterpret_cast<const uint16_t *>(p.values)[at];
          mine_v[i] = p.value_dt == FP8_DT_BF16 ? __uint_as_float((uint32_t)h << 16) : __half2float(__ushort_as_half(h));
        }
        if (id >= 0 && id < p.cols && mine_v[i] != -INFINITY) mine_id[i] = (int)id;
        list.id[k] = mine_id[i];
      }
    }
    if (MODE == kListTail) {
      const int bytes = ((r.v1 - r.v0) * kElems<DT> + 7) / 8;
      for (int i = threadIdx.x; i < (bytes + 3) / 4; i += blockDim.x) reinterpret_cast<uint32_t *>(marks)[i] = 0;
      if (threadIdx.x == 0) edge_bits = 0;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int k = threadIdx.x + i * blockDim.x;
      bool again = false;
      if (k < K && mine_id[i] != kAbsent)
        for (int j = 0; j < k; j++) again |= list.id[j] == mine_id[i];
      if (again) mine_id[i] = kAbsent;
    }
    __syncthreads();
    float v_max = kNone;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int k = threadIdx.x + i * blockDim.x;
      if (k < K) list.id[k] = mine_id[i];
      if (mine_id[i] == kAbsent) mine_v[i] = -INFINITY;
      v_max = max_nan(v_max, mine_v[i]);
      if (MODE == kListTail && mine_id[i] != kAbsent) {
        const int e = mine_id[i] - r.s.head, body = r.s.vecs * kElems<DT>;
        if (e >= 0 && e < body) {
          const int b = e - r.v0 * kElems<DT>;
          if (b >= 0 && e < r.v1 * kElems<DT>) atomicOr(reinterpret_cast<uint32_t *>(marks) + (b >> 5), 1u << (b & 31));
        } else {
          atomicOr(&edge_bits, 1u << (e < 0 ? mine_id[i] : 16 + e - body));
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int k = threadIdx.x + i * blockDim.x;
      if (k < K)
        for (int j = 0; j < K; j++) {
          const int o = list.id[j];
          mine_at[i] += o < mine_id[i] || (o == mine_id[i] && j < k);
        }
    }
    if (MODE == kListTop) top_value = block_max(v_max, red);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      mine_q[i] = expf(MODE == kListTop ? (mine_v[i] - top_value) * p.beta : mine_v[i]);
      q_sum += mine_q[i];
    }
    q_sum = block_sum(q_sum, red);  // (its barriers also publish the marks)
  }
  float most;
  bool any;
  Part own = stream_row<DT, MODE, ENT>(r, c2, marks, MODE == kListTail ? edge_bits : 0u, most, any);
  Part all = join_block<MODE, ENT>(own, c2, red);
  TopScratch &top = *reinterpret_cast<TopScratch *>(loss_smem);
  if (MODE == kLogprob && p.top) top_of_range<DT>(r, most, any, p.top, top);
  if (ctas > 1) {
    if (threadIdx.x == 0) parts[rank] = all;
    cluster_wait();
    // every CTA reads the others' parts; the first one goes on
    if (rank == 0 && threadIdx.x > 0 && threadIdx.x < ctas) {
      const uint32_t there = cluster_at(smem_u32(&parts[threadIdx.x]), threadIdx.x);
      Part o;
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(o.m), "=f"(o.S), "=f"(o.W), "=f"(o.rest)
                   : "r"(there)
                   : "memory");
      parts[threadIdx.x] = o;
    }
    if (MODE == kLogprob && p.top && rank == 0) {
      for (int i = threadIdx.x; i < (int)ctas * p.top; i += blockDim.x) {
        unsigned long long c;
        const uint32_t there = cluster_at(smem_u32(&top.best[i % p.top]), i / p.top);
        asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(c) : "r"(there) : "memory");
        top.list[i] = c;
      }
    }
    cluster_wait();  // the others' shared memory has been read
    if (rank != 0) return;
    __syncthreads();
    float m = kNone;
    for (unsigned i = 0; i < ctas; i++) m = max_nan(m, parts[i].m);
    all = {m, 0.0f, 0.0f, 0.0f};
    for (unsigned i = 0; i < ctas; i++) {
      Part o = parts[i];
      const float d = max_nan((o.m - m) * c2, -1000.0f), down = ex2(d);
      all.W += fmaf(o.S, d, o.W) * down;
      all.S += o.S * down;
      all.rest += o.rest * down;
    }
    if (MODE == kLogprob && p.top) rank_list(top.list, (int)ctas * p.top, p.top, top.best);
  }
  constexpr float kLn2 = 0.69314718055994531f;
  const float S = MODE == kListTail ? all.S + all.rest : all.S;  // (rest: of the listed ones here)
  const bool none = S == 0.0f;
  const float log_S = logf(S);  // -inf for none
  if constexpr (MODE == kLogprob) {
    const float ent = ENT && !none ? fmaf(-all.W / S, kLn2, log_S) : 0.0f;
    if (threadIdx.x == 0) {
      if (p.logp) {
        const int t = token_at(p.tokens, p.token_bytes, row, p.cols);
        p.logp[row] = t < 0 ? 0.0f : none ? -INFINITY : p.beta * (load_one<DT>(z, t) - all.m) - log_S;
      }
      if (ENT && p.entropy) p.entropy[row] = ent;
      if (p.stats)
        reinterpret_cast<float4 *>(p.stats)[row] = make_float4(all.m, none ? 0.0f : 1.0f / S, none ? 0.0f : log_S, ent);
    }
    for (int i = threadIdx.x; i < p.top; i += blockDim.x) {
      const unsigned long long c = top.best[i];
      p.top_ids[(size_t)row * p.top + i] = (int)~(uint32_t)c;
      p.top_logp[(size_t)row * p.top + i] = none ? -INFINITY : p.beta * (key_value((uint32_t)(c >> 32)) - all.m) - log_S;
    }
  } else {
    const int K = p.top;
    const float log_q_sum = logf(q_sum), q_scale = MODE == kListTop && q_sum > 0.0f ? 1.0f / q_sum : 1.0f;
    float l = 0.0f;
    if (rank == 0) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int k = threadIdx.x + i * blockDim.x;
        if (k >= K) break;
        const float q = mine_q[i] * q_scale;
        if (mine_id[i] != kAbsent && q != 0.0f) {
          const float lq = MODE == kListTop ? (mine_v[i] - top_value) * p.beta - log_q_sum : mine_v[i];
          const float lp = none ? -INFINITY : p.beta * (load_one<DT>(z, mine_id[i]) - all.m) - log_S;
          l = fmaf(q, lq - lp, l);
        }
        p.list_ids[(size_t)row * K + mine_at[i]] = mine_id[i];
        p.list_q[(size_t)row * K + mine_at[i]] = q;
      }
    }
    l = block_sum(l, red);
    float listed = q_sum > 0.0f ? 1.0f : 0.0f, unlisted = listed;
    if (q_sum != q_sum) listed = unlisted = q_sum;
    if (MODE == kListTail) {
      const float q_rest = fmaxf(0.0f, 1.0f - q_sum);
      const bool there = q_rest > 0.0f && all.S > 0.0f;
      listed = q_sum + (there ? q_rest : 0.0f);
      unlisted = listed - (there ? q_rest * (S / all.S) : 0.0f);
      if (there) l += q_rest * (logf(q_rest) - (logf(all.S) - log_S));
    }
    if (threadIdx.x == 0) {
      p.loss[row] = l;
      reinterpret_cast<float4 *>(p.stats)[row] = make_float4(all.m, none ? 0.0f : 1.0f / S, listed, unlisted);
    }
  }
}

// ---------------------------------------------------------------- backward
struct Bwd {
  const uint8_t *z;
  size_t ld;  // bytes
  int rows, cols;
  float beta;
  const float *stats;
  const void *tokens;
  int token_bytes;
  const float *g, *g_ent;  // of logp and entropy; of the loss
  int K;
  const int *list_ids;
  const float *list_q;
  uint8_t *d;
  size_t ldd;  // bytes
  int margin, vec_z, vec_d;
  block::CastOut out;
};

// A row's factors: with a = (z - m) c2 and e = 2^a, d = e (k0 + k1 a), plus gt
// at the token; of a listed outcome e kl - gt q.
struct RowTerms {
  float m, k0, k1, kl, gt;
  int token;
};

template <bool LIST>
__device__ __forceinline__ RowTerms row_terms(const Bwd &p, int row) {
  const float4 s = __ldg(reinterpret_cast<const float4 *>(p.stats) + row);
  RowTerms r;
  r.m = s.x;
  const bool none = s.y == 0.0f;  // no distribution: no gradient
  if constexpr (LIST) {
    const float g = none ? 0.0f : p.beta * __ldg(p.g + row);
    r.k0 = g * s.w * s.y;
    r.kl = g * s.z * s.y;
    r.k1 = 0.0f;
    r.gt = g;
    r.token = -1;
  } else {
    r.token = p.g ? token_at(p.tokens, p.token_bytes, row, p.cols) : -1;
    const float g = none || r.token < 0 ? 0.0f : p.beta * __ldg(p.g + row);
    const float ge = none || !p.g_ent ? 0.0f : p.beta * __ldg(p.g_ent + row);
    r.gt = g;
    r.k0 = -(g + ge * (s.w - s.z)) * s.y;
    r.k1 = -ge * 0.69314718055994531f * s.y;
    r.kl = 0.0f;
  }
  return r;
}

__device__ __forceinline__ float scaled(float z, float m, float c2) { return max_nan((z - m) * c2, -1000.0f); }

// d itself: one row's chunk a CTA, in 16-byte vectors wherever the row starts.
constexpr int kBwdThreads = 256;
constexpr int kBwdVecs = 4;  // vectors of a thread
template <int DT, bool LIST>
__global__ void __launch_bounds__(kBwdThreads) k_loss_bwd_rows(const Bwd p, unsigned chunks) {
  pdl_launch_dependents();
  pdl_wait();
  const int row = (int)(blockIdx.x / chunks), chunk = (int)(blockIdx.x % chunks), t = threadIdx.x;
  const uint8_t *z = p.z + (size_t)row * p.ld;
  uint8_t *d = p.d + (size_t)row * p.ldd;
  const RowShape s = row_shape<DT>(z, p.cols);
  const uint8_t *body = z + (size_t)s.head * kSize<DT>;
  uint8_t *dbody = d + (size_t)s.head * kSize<DT>;
  const bool wide = (reinterpret_cast<uintptr_t>(dbody) & 15) == 0;
  const float c2 = p.beta * kLog2e;
  const RowTerms r = row_terms<LIST>(p, row);
  constexpr int E = kElems<DT>;
  const int v0 = chunk * (kBwdThreads * kBwdVecs);
  uint4 raw[kBwdVecs];
#pragma unroll
  for (int i = 0; i < kBwdVecs; i++) {
    const int v = v0 + i * kBwdThreads + t;
    raw[i] = v < s.vecs ? __ldcs(reinterpret_cast<const uint4 *>(body) + v) : make_uint4(0u, 0u, 0u, 0u);
  }
  // the head and the tail belong to the first chunk
  float edge = 0.0f;
  const bool has_edge = chunk == 0 && t < s.head + s.tail;
  const int edge_at = t < s.head ? t : s.vecs * E + t;
  if (has_edge) edge = load_one<DT>(z, edge_at);
  // listed outcomes of this chunk: read before d may take the logits' place
  float listed[4];
  int listed_at[4];
  if constexpr (LIST) {
    const int c0 = chunk == 0 ? 0 : s.head + v0 * E;
    const int c1 = s.head + min(s.vecs, v0 + kBwdThreads * kBwdVecs) * E, last = s.head + s.vecs * E;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      listed_at[i] = -1;
      const int k = t + i * kBwdThreads;
      if (k < p.K) {
        const int c = __ldg(p.list_ids + (size_t)row * p.K + k);
        if (c < p.cols && ((c >= c0 && c < c1) || (chunk == 0 && c >= last))) {
          listed_at[i] = c;
          listed[i] = fmaf(ex2(scaled(load_one<DT>(z, c), r.m, c2)), r.kl, -r.gt * __ldg(p.list_q + (size_t)row * p.K + k));
        }
      }
    }
    __syncthreads();
  }
  auto grad = [&](float x, int c) {
    const float a = scaled(x, r.m, c2);
    float g = ex2(a) * fmaf(r.k1, a, r.k0);
    if (!LIST && c == r.token) g += r.gt;
    return g;
  };
  if (has_edge) store_one<DT>(d, edge_at, grad(edge, edge_at));
#pragma unroll
  for (int i = 0; i < kBwdVecs; i++) {
    const int v = v0 + i * kBwdThreads + t;
    if (v >= s.vecs) break;
    float x[E];
    unpack<DT>(raw[i], x);
    const int c = s.head + v * E;
#pragma unroll
    for (int j = 0; j < E; j++) x[j] = grad(x[j], c + j);
    if (wide) {
      uint4 o;
      if constexpr (DT == FP8_DT_F32) {
        o = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
      } else {
        uint4 w[1];
        block::pack8<DT>(x, w);
        o = w[0];
      }
      __stcs(reinterpret_cast<uint4 *>(dbody) + v, o);
    } else {
#pragma unroll
      for (int j = 0; j < E; j++) store_one<DT>(d, c + j, x[j]);
    }
  }
  if constexpr (LIST) {
    __syncthreads();  // what is stored above is overwritten
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (listed_at[i] >= 0) store_one<DT>(d, listed_at[i], listed[i]);
  }
}

// Codes of d, and d itself where wanted: tiles of block_scale.cuh.
template <int DT, bool LIST, int OUT>
__global__ void __launch_bounds__(512, 2) k_loss_bwd_tiles(const Bwd p) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int RP = 4;
  using G = block::Geo<RP>;
  __shared__ block::ColScratch<RP> sc;
  __shared__ __align__(16) uint32_t marks[LIST ? block::kTile : 1][4];
  __shared__ int places[LIST ? block::kTile : 1];
  constexpr int esz = kSize<DT>;
  const int tiles_c = (p.cols + block::kTile - 1) / block::kTile;
  const auto [row0, col0] = block::tile_at(blockIdx.x, tiles_c);
  const int c8 = threadIdx.x & 15, col = col0 + c8 * 8, r0 = threadIdx.x >> 4;
  Raw8<DT> raw[RP];
  block::load_tile<DT>(p.z, p.ld / esz, p.vec_z, row0, col0, p.rows, p.cols, raw);
  if constexpr (LIST) {
    // the list entries of each row in this tile: marked, and where the first one stands
    if (threadIdx.x < block::kTile) {
      const int row = row0 + threadIdx.x;
      uint32_t m[4] = {0, 0, 0, 0};
      int lo = 0;
      if (row < p.rows) {
        const int *ids = p.list_ids + (size_t)row * p.K;
        int hi = p.K;
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (__ldg(ids + mid) < col0) lo = mid + 1;
          else hi = mid;
        }
        for (int k = lo; k < p.K; k++) {
          const int b = __ldg(ids + k) - col0;
          if (b >= block::kTile) break;
#pragma unroll
          for (int w = 0; w < 4; w++)
            if (b >> 5 == w) m[w] |= 1u << (b & 31);
        }
      }
      *reinterpret_cast<uint4 *>(marks[threadIdx.x]) = make_uint4(m[0], m[1], m[2], m[3]);
      places[threadIdx.x] = lo;
    }
    __syncthreads();
  }
  const float c2 = p.beta * kLog2e;
  float f[RP][8];
#pragma unroll
  for (int i = 0; i < RP; i++) {
    const int row = row0 + r0 + i * G::kStep;
    block::unpack8<DT>(raw[i], f[i]);
    if (row >= p.rows) {
#pragma unroll
      for (int j = 0; j < 8; j++) f[i][j] = 0.0f;
      continue;
    }
    const RowTerms r = row_terms<LIST>(p, row);
    uint32_t bits = 0;
    if constexpr (LIST) bits = marks[row - row0][c8 >> 2] >> ((c8 & 3) * 8) & 0xffu;
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const float a = scaled(f[i][j], r.m, c2), e = ex2(a);
      float g = e * fmaf(r.k1, a, r.k0);
      if (!LIST && col + j == r.token) g += r.gt;
      if (LIST && (bits >> j & 1)) {
        int k = places[row - row0];
#pragma unroll
        for (int w = 0; w < 4; w++) {
          const uint32_t m = marks[row - row0][w];
          const int first = c8 * 8 + j - w * 32;  // bits of this word that come before
          k += first >= 32 ? __popc(m) : first > 0 ? __popc(m & ((1u << first) - 1)) : 0;
        }
        g = fmaf(e, r.kl, -r.gt * __ldg(p.list_q + (size_t)row * p.K + k));
      }
      f[i][j] = col + j < p.cols ? g : 0.0f;
    }
  }
  if (p.d) block::store_tile<DT>(p.vec_d, p.d, p.ldd / esz, row0, col0, p.rows, p.cols, f);
  const float fmax = OUT == FP8_E4M3 ? kMaxE4M3 : kMaxE5M2;
  if (p.out.qt) block::put_tile_maxima(f, sc);
  if (p.out.q) block::cast_tile_rows<OUT>(f, p.out.q, p.out.s, p.out.ldq, row0, col0, p.rows, p.cols, fmax, p.margin);
  if (p.out.qt) {
    __syncthreads();
    bool bad = false;
    if (threadIdx.x < block::kTile)
      bad = block::finish_column(sc, threadIdx.x, p.out.st, row0, col0, p.rows, fmax, p.margin);
    bad = __syncthreads_or(bad);
    block::store_tile_cols<OUT>(f, sc, bad, p.out.qt, p.out.ldqt, row0, col0, p.rows, p.cols);
  }
}

}  // namespace loss
}  // namespace fp8lib
