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
//   distillation:  beta (p Q - q) of listed outcomes, beta p (Q - q' / p') of the others
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
  float m, S;
  float W, L;  // kListTail: the listed ones' m and S
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

// The larger of a vector's elements; a NaN anywhere stays one.
template <int DT>
__device__ __forceinline__ uint32_t max_word(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (DT == FP8_DT_F32) asm("max.NaN.f32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else if constexpr (DT == FP8_DT_BF16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <int DT>
__device__ __forceinline__ float widest(uint32_t w) {
  if constexpr (DT == FP8_DT_F32) return __uint_as_float(w);
  else if constexpr (DT == FP8_DT_BF16) return max_nan(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  else {
    const float2 v = h2f2(w);
    return max_nan(v.x, v.y);
  }
}
template <int DT>
constexpr uint32_t kMinusInf = DT == FP8_DT_F32 ? 0xff800000u : DT == FP8_DT_BF16 ? 0xff80ff80u : 0xfc00fc00u;

// Calls f(column, logit) for the elements of the range that this thread owns and
// whose key reaches `least`.
template <int DT, typename F>
__device__ __forceinline__ void each_own(const Range &r, uint32_t least, F f) {
  const int t = threadIdx.x, T = blockDim.x;
  if (t < r.head + r.tail) {
    const int c = t < r.head ? t : r.s.head + r.s.vecs * kElems<DT> + t - r.head;
    const float x = load_one<DT>(r.row, c);
    if (order_key(x) >= least) f(c, x);
  }
#pragma unroll 1
  for (int v = r.v0 + t; v < r.v1; v += 4 * T) {
    uint4 w[4];
#pragma unroll
    for (int u = 0; u < 4; u++) w[u] = __ldcg(reinterpret_cast<const uint4 *>(r.body) + min(v + u * T, r.v1 - 1));
    uint32_t pass = 0;
#pragma unroll
    for (int u = 0; u < 4; u++) {
      const float x = widest<DT>(max_word<DT>(max_word<DT>(w[u].x, w[u].y), max_word<DT>(w[u].z, w[u].w)));
      if (v + u * T < r.v1 && order_key(x) >= least) pass |= 1u << u;
    }
    while (pass) {
      const int u = __ffs(pass) - 1, c = r.s.head + (v + u * T) * kElems<DT>;
      pass &= pass - 1;
      const uint4 q = u == 0 ? w[0] : u == 1 ? w[1] : u == 2 ? w[2] : w[3];
      float x[kElems<DT>];
      unpack<DT>(q, x);
#pragma unroll
      for (int j = 0; j < kElems<DT>; j++)
        if (order_key(x[j]) >= least) f(c + j, x[j]);
    }
  }
}

struct __align__(16) TopScratch {
  unsigned long long list[kCandidates];  // (key, ~column): larger is earlier
  uint32_t group[64];
  int above, equal, ties;
  uint32_t bound;
  unsigned long long best[kTop];
  int wsum[32];
};

__device__ __forceinline__ unsigned long long candidate(uint32_t key, int col) {
  return (unsigned long long)key << 32 | (uint32_t)~col;
}

// The `top` first candidates of a list of n, in order, to out (0: none).  Eight
// lanes count together how many come before a candidate.
__device__ __forceinline__ void rank_list(const unsigned long long *list, int n, int top, unsigned long long *out) {
  constexpr int G = 8;
  const int g = threadIdx.x % G, rows = blockDim.x / G;
  for (int i = threadIdx.x; i < top; i += blockDim.x) out[i] = 0;
  __syncthreads();
  for (int i0 = 0; i0 < n; i0 += rows) {
    const int i = i0 + threadIdx.x / G;
    const unsigned long long c = i < n ? list[i] : 0ull;
    int before = 0;
#pragma unroll 4
    for (int j = g; j < n; j += G) before += list[j] > c;
#pragma unroll
    for (int b = G / 2; b > 0; b /= 2) before += __shfl_xor_sync(0xffffffffu, before, b);
    if (g == 0 && before < top && c) out[before] = c;
  }
  __syncthreads();
}

// The `top` largest logits of the CTA's range, in order, to sh.best.  `most` is
// the thread's own largest.  The top-th largest maximum of 64 groups of
// threads is a bound that at least `top` elements reach; few others do, and only threads
// that own one read their elements again.  Where many are equal to the bound (a
// masked vocabulary) those of the lowest columns are taken in order; where too
// many lie above it the bound is raised by bisection.
template <int DT>
__device__ void top_of_range(const Range &r, float most, bool any, int top, TopScratch &sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const uint32_t own = any ? order_key(most) : 0u;
  constexpr int groups = 64;
  const int per = blockDim.x / groups;  // (128 threads or more: 2 to 16, powers of two)
  uint32_t g = own;
  for (int b = per / 2; b > 0; b /= 2) g = max(g, __shfl_xor_sync(0xffffffffu, g, b));
  if (threadIdx.x % per == 0) sh.group[threadIdx.x / per] = g;
  if (threadIdx.x == 0) sh.above = sh.equal = 0;
  __syncthreads();
  if (threadIdx.x < groups) {
    const uint32_t k = sh.group[threadIdx.x];
    int more = 0, same = 0;  // groups above this one's maximum, and at it
#pragma unroll 4
    for (int j = 0; j < groups; j += 4) {
      const uint4 o = *reinterpret_cast<const uint4 *>(&sh.group[j]);
      more += (o.x > k) + (o.y > k) + (o.z > k) + (o.w > k);
      same += (o.x == k) + (o.y == k) + (o.z == k) + (o.w == k);
    }
    if (more < top && more + same >= top) sh.bound = k;
  }
  __syncthreads();
  uint32_t bound = sh.bound;
  // candidates above the bound from the front, equal ones from the back
  auto collect = [&] {
    if (own >= bound)
      each_own<DT>(r, bound, [&](int c, float z) {
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
      if (own >= mid) each_own<DT>(r, mid, [&](int, float) { count++; });
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

struct __align__(16) ListScratch {
  int id[FP8_DISTILL_MAX];
  float v[FP8_DISTILL_MAX];
};

// What a thread has seen: S and W about m.  kListTail: of the unlisted ones; L
// of the listed ones, about a largest of their own, ml.  (About one m for both,
// the unlisted sum is 0 in binary32 where the listed ones lie 88 or more above,
// and its logarithm and its share of the gradient are lost.)
template <int MODE, bool ENT>
struct Running {
  float m = kNone, ml = kNone, L = 0.0f, largest = -INFINITY;
  float2 S = make_float2(0.0f, 0.0f), W2 = make_float2(0.0f, 0.0f);
  bool any = false;

  // m grows to include t
  __device__ __forceinline__ void raise(float t, float c2) {
    if constexpr (MODE == kLogprob) largest = max_nan(largest, t);
    any = true;
    const float m1 = max_nan(m, t);
    float d = (m - m1) * c2;
    if constexpr (ENT) {
      d = max_nan(d, -1000.0f);
      W2 = __ffma2_rn(S, both(d), W2);
    }
    const float down = ex2(d);
    S = __fmul2_rn(S, both(down));
    if constexpr (ENT) W2 = __fmul2_rn(W2, both(down));
    m = m1;
  }
  // n elements, none above m
  template <int N>
  __device__ __forceinline__ void add(const float (&x)[N], float c2) {
    if constexpr (N == 1) {
      float a = (x[0] - m) * c2;
      if constexpr (ENT) a = max_nan(a, -1000.0f);
      const float e = ex2(a);
      S.x += e;
      if constexpr (ENT) W2.x = fmaf(e, a, W2.x);
    } else {
#pragma unroll
      for (int j = 0; j < N; j += 2) {
        float2 a = __fmul2_rn(__fadd2_rn(make_float2(x[j], x[j + 1]), both(-m)), both(c2));
        if constexpr (ENT) a = make_float2(max_nan(a.x, -1000.0f), max_nan(a.y, -1000.0f));
        const float2 e = make_float2(ex2(a.x), ex2(a.y));
        S = __fadd2_rn(S, e);
        if constexpr (ENT) W2 = __ffma2_rn(e, a, W2);
      }
    }
  }
  // the thread's listed elements; -inf for none
  __device__ __forceinline__ void add_listed(const float (&x)[4], float c2) {
    ml = max_nan(max_nan(max_nan(max_nan(ml, x[0]), x[1]), x[2]), x[3]);
#pragma unroll
    for (int i = 0; i < 4; i++) L += ex2((x[i] - ml) * c2);
  }
};

// Where element e of a CTA's body has its bit: a thread's kRun vectors of one
// step stand side by side, so that it asks once for all of them.
constexpr int kRun = 4;
template <int DT>
__device__ __forceinline__ int mark_at(int e) {
  const int v = e / kElems<DT>, T = blockDim.x, step = v / (kRun * T), in = v - step * kRun * T;
  return (step * T + in % T) * (kRun * kElems<DT>) + in / T * kElems<DT> + e % kElems<DT>;
}
template <int DT>
__host__ __device__ inline size_t mark_bytes(int vecs, int threads) {
  return (size_t)((vecs + kRun * threads - 1) / (kRun * threads)) * threads * (kRun * kElems<DT> / 8);
}

// Running softmax of a row's elements, for kListTail of the unlisted ones alone
// (`marks`: a bit for each element, see mark_at).  Four
// vectors at a time: their loads are in flight together, and m is raised once.
// Per element of a 16-bit row: one exponential (16 a cycle and SM: 46 us for
// 4096 x 50304), some four other instructions.
template <int DT, int MODE, bool ENT>
__device__ __forceinline__ Running<MODE, ENT> stream_row(const Range &r, float c2, const uint8_t *marks, uint32_t edge_marks) {
  constexpr int E = kElems<DT>;
  Running<MODE, ENT> s;
  const int t = threadIdx.x, T = blockDim.x;
  if (t < r.head + r.tail) {
    const float x[1] = {load_one<DT>(r.row, t < r.head ? t : r.s.head + r.s.vecs * E + t - r.head)};
    if (!(MODE == kListTail && (edge_marks >> (t < r.head ? t : 16 + t - r.head) & 1))) {
      s.raise(x[0], c2);
      s.add(x, c2);
    }
  }
  const uint4 *body = reinterpret_cast<const uint4 *>(r.body);
  const uint32_t none = kMinusInf<DT>;
  int step = t;
  for (int v = r.v0 + t; v < r.v1; v += kRun * T, step += T) {
    uint4 w[kRun];
    bool skip = false;  // runs with listed elements are left to add_marked
    if constexpr (MODE == kListTail)
      skip = (E == 8 ? reinterpret_cast<const uint32_t *>(marks)[step] : (uint32_t)reinterpret_cast<const uint16_t *>(marks)[step]) != 0;
#pragma unroll
    for (int u = 0; u < kRun; u++) {
      w[u] = make_uint4(none, none, none, none);
      if (!skip && v + u * T < r.v1) w[u] = __ldcg(body + v + u * T);
    }
    uint32_t k = w[0].x;
#pragma unroll
    for (int u = 0; u < kRun; u++)
      k = max_word<DT>(max_word<DT>(max_word<DT>(max_word<DT>(k, w[u].x), w[u].y), w[u].z), w[u].w);
    s.raise(widest<DT>(k), c2);
#pragma unroll
    for (int u = 0; u < kRun; u++) {
      float x[E];
      unpack<DT>(w[u], x);
      s.add(x, c2);
    }
  }
  // (a thread that has seen only -inf has m = kNone, and its sums are 0)
  return s;
}

// The unlisted ones of the run of element e of the body, which is listed, if none
// before it in the run is: lane g of G takes every G-th of its vectors.  (Tested inside the
// stream, two of three steps of a warp took the slow way: 142 us for 4096 x
// 50304 with 64 entries a row.)
template <int DT, bool ENT>
__device__ __forceinline__ void add_marked(Running<kListTail, ENT> &s, const Range &r, float c2, const uint8_t *marks, int e,
                                           int g, int G) {
  constexpr int E = kElems<DT>, kBits = kRun * E;
  const int T = blockDim.x, b = mark_at<DT>(e), run = b / kBits;
  const uint32_t bits = E == 8 ? reinterpret_cast<const uint32_t *>(marks)[run]
                               : (uint32_t)reinterpret_cast<const uint16_t *>(marks)[run];
  if (bits & ((1u << (b % kBits)) - 1)) return;
#pragma unroll 1
  for (int u = g; u < kRun; u += G) {
    const int v = r.v0 + run / T * (kRun * T) + u * T + run % T;
    if (v >= r.v1) break;
    const uint4 w = __ldcg(reinterpret_cast<const uint4 *>(r.body) + v);
    float x[E], most = -INFINITY;
    unpack<DT>(w, x);
#pragma unroll
    for (int j = 0; j < E; j++) {
      if (bits >> (u * E + j) & 1) x[j] = -INFINITY;
      most = max_nan(most, x[j]);
    }
    s.raise(most, c2);
    s.add(x, c2);
  }
}

// Parts about their own m joined about the largest.  W is in units of log 2.
template <int MODE>
__device__ __forceinline__ Part about(Part p, float m, float ml, float c2) {
  const float d = max_nan((p.m - m) * c2, -1000.0f), down = ex2(d);
  if constexpr (MODE == kListTail) return {m, p.S * down, ml, p.L * ex2((p.W - ml) * c2)};
  return {m, p.S * down, fmaf(p.S, d, p.W) * down, 0.0f};
}

// Joins the lanes' parts.
template <int MODE, bool ENT>
__device__ __forceinline__ Part join_lanes(Part p, float c2) {
  float m = p.m, ml = p.W;
#pragma unroll
  for (int b = 16; b > 0; b /= 2) {
    m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, b));
    if constexpr (MODE == kListTail) ml = max_nan(ml, __shfl_xor_sync(0xffffffffu, ml, b));
  }
  p = about<MODE>(p, m, ml, c2);
#pragma unroll
  for (int b = 16; b > 0; b /= 2) {
    p.S += __shfl_xor_sync(0xffffffffu, p.S, b);
    if constexpr (ENT) p.W += __shfl_xor_sync(0xffffffffu, p.W, b);
    if constexpr (MODE == kListTail) p.L += __shfl_xor_sync(0xffffffffu, p.L, b);
  }
  return p;
}

// The CTA's part, to every thread: the warps by shuffles, then one exchange.
template <int MODE, bool ENT>
__device__ __forceinline__ Part join_block(const Running<MODE, ENT> &s, float c2, Part *warps) {
  Part p = join_lanes<MODE, ENT>({s.m, s.S.x + s.S.y, MODE == kListTail ? s.ml : s.W2.x + s.W2.y, s.L}, c2);
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = p;
  __syncthreads();
  // each warp joins all of them, a lane a part
  const int lane = threadIdx.x & 31;
  p = lane < (int)(blockDim.x >> 5) ? warps[lane] : Part{kNone, 0.0f, MODE == kListTail ? kNone : 0.0f, 0.0f};
  return join_lanes<MODE, ENT>(p, c2);
}

// One row a CTA (128 threads where there are many rows: 4096 x 50304 bfloat16 77
// us in CTAs of 256, 72 so, 5.7 TB/s; with the entropy 75, lists of 64: 84, in
// the tail form 94), or a cluster's where there are few (one row of 50304 4.7
// us, with 20 alternatives 10).  Neither HBM (59 % busy) nor the exponential unit
// (69 %) is full: warps wait for loads, four vectors each in flight, at 27 warps
// an SM.
template <int DT, int MODE, bool ENT>
__global__ void __launch_bounds__(1024) k_loss_fwd(const Fwd p, unsigned ctas) {
  pdl_launch_dependents();
  pdl_wait();
  extern __shared__ __align__(16) uint8_t loss_smem[];
  __shared__ float red[32];
  __shared__ __align__(16) Part parts[8], warp_parts[32];
  __shared__ uint32_t edge_bits;
  const unsigned rank = ctas > 1 ? blockIdx.x % ctas : 0;
  const int row = (int)(blockIdx.x / ctas);
  const uint8_t *z = p.z + (size_t)row * p.ld;
  const Range r = range_of<DT>(z, p.cols, rank, ctas);
  const float c2 = p.beta * kLog2e;
  ListScratch &list = *reinterpret_cast<ListScratch *>(loss_smem);
  uint8_t *marks = loss_smem + sizeof(ListScratch);
  // an entry belongs to the first of G lanes, which look at the list together; a thread has at most four
  const int K = MODE == kLogprob ? 0 : p.top, K4 = (K + 3) / 4;
  const int G = K * 4 <= (int)blockDim.x ? 4 : K * 2 <= (int)blockDim.x ? 2 : 1;
  const int lead = threadIdx.x % G == 0, first = threadIdx.x / G, apart = blockDim.x / G;
  float top_value = 0.0f, mine_v[4], mine_q[4];
  int mine_id[4], mine_at[4];
  if constexpr (MODE != kLogprob) {
    for (int k = threadIdx.x; k < K4 * 4; k += blockDim.x) {
      int id = kAbsent;
      float v = -INFINITY;
      if (k < K) {
        const size_t at = (size_t)row * K + k;
        const long long i = index_at(p.ids, p.id_bytes, at);
        if (i >= p.cols) atomicOr(&g_status, FP8_STATUS_BAD_INDEX);
        if (p.value_dt == FP8_DT_F32) {
          v = reinterpret_cast<const float *>(p.values)[at];
        } else {
          const uint16_t h = reinterpret_cast<const uint16_t *>(p.values)[at];
          v = p.value_dt == FP8_DT_BF16 ? __uint_as_float((uint32_t)h << 16) : __half2float(__ushort_as_half(h));
        }
        if (i >= 0 && i < p.cols && v != -INFINITY) id = (int)i;
        else v = -INFINITY;
      }
      list.id[k] = id;
      list.v[k] = v;
    }
    if (MODE == kListTail) {
      const int words = (int)mark_bytes<DT>(r.v1 - r.v0, blockDim.x) / 4;  // (128 threads or more: whole words)
      for (int i = threadIdx.x; i < words; i += blockDim.x) reinterpret_cast<uint32_t *>(marks)[i] = 0;
      if (threadIdx.x == 0) edge_bits = 0;
    }
    __syncthreads();
    // an entry's place by id is the number of entries that come before it; the same id earlier in the list: listed again
    float v_max = kNone, q_sum = 0.0f;
    int dropped = 0;  // whether one of the thread's entries is listed again
    auto larger = [&](int j) {
      const float4 v = reinterpret_cast<const float4 *>(list.v)[j];
      v_max = max_nan(max_nan(max_nan(max_nan(v_max, v.x), v.y), v.z), v.w);
    };
    auto to_group = [&] {
      for (int b = G / 2; b > 0; b /= 2) v_max = max_nan(v_max, __shfl_xor_sync(0xffffffffu, v_max, b));
    };
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int k = first + i * apart;
      mine_id[i] = kAbsent;
      mine_v[i] = -INFINITY;
      mine_at[i] = -1;
      if (i * apart >= K) continue;  // (the same for all lanes)
      const int id = k < K ? list.id[k] : kAbsent;
      int before = 0, again = 0;
      for (int j = threadIdx.x % G; j < K4; j += G) {
        const int4 o = reinterpret_cast<const int4 *>(list.id)[j];
        const int e[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int n = 0; n < 4; n++) {
          const int same = e[n] == id && 4 * j + n < k;
          again += same;
          before += (e[n] < id) + same;
        }
        if (MODE == kListTop && i == 0) larger(j);
      }
      for (int b = G / 2; b > 0; b /= 2) {
        before += __shfl_xor_sync(0xffffffffu, before, b);
        again += __shfl_xor_sync(0xffffffffu, again, b);
      }
      if (MODE == kListTop && i == 0) to_group();
      if (!lead || k >= K) continue;
      mine_at[i] = before;
      mine_id[i] = id;
      mine_q[i] = 0.0f;
      if (id == kAbsent) continue;
      if (again) {
        mine_q[i] = -1.0f;  // stands behind the first one and counts for nothing
        dropped = 1;
        continue;
      }
      mine_v[i] = list.v[k];
      if (MODE == kListTail) {
        mine_q[i] = expf(mine_v[i]);
        q_sum += mine_q[i];
      }
      if (MODE == kListTail) {
        const int e = id - r.s.head, body = r.s.vecs * kElems<DT>;
        if (e >= 0 && e < body) {
          if (e >= r.v0 * kElems<DT> && e < r.v1 * kElems<DT>) {
            const int b = mark_at<DT>(e - r.v0 * kElems<DT>);
            atomicOr(reinterpret_cast<uint32_t *>(marks) + (b >> 5), 1u << (b & 31));
          }
        } else {
          atomicOr(&edge_bits, 1u << (e < 0 ? id : 16 + e - body));
        }
      }
    }
    if constexpr (MODE == kListTop) {
      if (__syncthreads_or(dropped)) {  // rare: the largest value among those that count
#pragma unroll
        for (int i = 0; i < 4; i++)
          if (mine_id[i] != kAbsent && mine_q[i] < 0.0f) list.v[first + i * apart] = -INFINITY;
        __syncthreads();
        v_max = kNone;
        for (int j = threadIdx.x % G; j < K4; j += G) larger(j);
        to_group();
      }
      top_value = v_max;
#pragma unroll
      for (int i = 0; i < 4; i++) {
        if (mine_id[i] == kAbsent || mine_q[i] < 0.0f) continue;
        mine_q[i] = expf((mine_v[i] - top_value) * p.beta);
        q_sum += mine_q[i];
      }
    }
#pragma unroll
    for (int b = 16; b > 0; b /= 2) q_sum += __shfl_xor_sync(0xffffffffu, q_sum, b);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = q_sum;
    if (MODE == kListTail) __syncthreads();  // the marks (red is read behind the next exchange)
  }
  Running<MODE, ENT> own = stream_row<DT, MODE, ENT>(r, c2, marks, MODE == kListTail ? edge_bits : 0u);
  float mine_z[4];  // the listed logits
  if constexpr (MODE == kListTail) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      mine_z[i] = -INFINITY;
      if (mine_id[i] != kAbsent && !(mine_q[i] < 0.0f) && rank == 0) mine_z[i] = load_one<DT>(z, mine_id[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
      if (i * apart >= K) continue;
      const int lead_lane = (threadIdx.x & 31) / G * G;
      const bool counts = mine_at[i] >= 0 && mine_id[i] != kAbsent && !(mine_q[i] < 0.0f);
      const int id = __shfl_sync(0xffffffffu, counts ? mine_id[i] : kAbsent, lead_lane);
      const int e = id - r.s.head - r.v0 * kElems<DT>;
      if (id != kAbsent && e >= 0 && e < (r.v1 - r.v0) * kElems<DT>)
        add_marked<DT, ENT>(own, r, c2, marks, e, threadIdx.x % G, G);
    }
    own.add_listed(mine_z, c2);
  }
  Part all = join_block<MODE, ENT>(own, c2, warp_parts);
  float q_sum = 0.0f;
  if constexpr (MODE != kLogprob) {
    for (int w = 0; w < (int)(blockDim.x >> 5); w++) q_sum += red[w];
  }
  TopScratch &top = *reinterpret_cast<TopScratch *>(loss_smem);
  if (MODE == kLogprob && p.top) top_of_range<DT>(r, own.largest, own.any, p.top, top);
  if (ctas > 1) {
    if (threadIdx.x == 0) parts[rank] = all;
    cluster_wait();
    // every CTA reads the others' parts; the first one goes on
    if (rank == 0 && threadIdx.x > 0 && threadIdx.x < ctas) {
      const uint32_t there = cluster_at(smem_u32(&parts[threadIdx.x]), threadIdx.x);
      Part o;
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(o.m), "=f"(o.S), "=f"(o.W), "=f"(o.L)
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
    all = {m, 0.0f, MODE == kListTail ? parts[0].W : 0.0f, parts[0].L};  // (the first CTA has all listed ones)
    for (unsigned i = 0; i < ctas; i++) {
      const Part o = about<MODE>(parts[i], m, parts[i].W, c2);
      if (MODE != kListTail) all.W += o.W;
      all.S += o.S;
    }
    if (MODE == kLogprob && p.top) rank_list(top.list, (int)ctas * p.top, p.top, top.best);
  }
  constexpr float kLn2 = 0.69314718055994531f;
  // the row's m and S, and those of the unlisted ones, which are `down` of it about its m
  const float m_row = MODE == kListTail ? max_nan(all.m, all.W) : all.m;
  const float down = MODE == kListTail ? ex2((all.m - m_row) * c2) : 1.0f;
  const float S = MODE == kListTail ? fmaf(all.S, down, all.L * ex2((all.W - m_row) * c2)) : all.S;
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
        reinterpret_cast<float4 *>(p.stats)[row] = make_float4(all.m, none ? 0.0f : 1.0f / S, none ? 0.0f : log_S, ENT ? ent : NAN);  // (an entropy's gradient needs one)
    }
    for (int i = threadIdx.x; i < p.top; i += blockDim.x) {
      const unsigned long long c = top.best[i];
      p.top_ids[(size_t)row * p.top + i] = (int)~(uint32_t)c;
      p.top_logp[(size_t)row * p.top + i] = none ? -INFINITY : p.beta * (key_value((uint32_t)(c >> 32)) - all.m) - log_S;
    }
  } else {
    const float log_q_sum = logf(q_sum), q_scale = MODE == kListTop && q_sum > 0.0f ? 1.0f / q_sum : 1.0f;
    float l = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      if (mine_at[i] < 0) continue;
      const float q = mine_q[i] < 0.0f ? mine_q[i] : mine_q[i] * q_scale;
      if (mine_id[i] != kAbsent && !(mine_q[i] <= 0.0f)) {
        const float lq = MODE == kListTop ? (mine_v[i] - top_value) * p.beta - log_q_sum : mine_v[i];
        const float lp = none ? -INFINITY : p.beta * ((MODE == kListTail ? mine_z[i] : load_one<DT>(z, mine_id[i])) - m_row) - log_S;
        l = fmaf(q, lq - lp, l);
      }
      p.list_ids[(size_t)row * K + mine_at[i]] = mine_id[i];
      p.list_q[(size_t)row * K + mine_at[i]] = q;
    }
    l = block_sum(l, red);
    // factors of e^(s - s_m): of a listed outcome about the row's m, of an unlisted one about theirs
    float whole = q_sum > 0.0f ? 1.0f : 0.0f, rest = 0.0f;
    if (q_sum != q_sum) whole = q_sum;
    if (MODE == kListTail) {
      const float q_rest = fmaxf(0.0f, 1.0f - q_sum);
      whole = q_sum;
      if (q_rest > 0.0f && all.S > 0.0f) {
        whole += q_rest;
        rest = q_rest / all.S;  // (S >= 1: their largest one)
        // p' itself where binary32 holds it (the logarithms of S and of its part are rounded at their own size)
        const float p_rest = all.S * down / S;
        l = fmaf(q_rest, p_rest > 1e-30f ? logf(q_rest / p_rest) : logf(q_rest) - (fmaf(p.beta, all.m - m_row, logf(all.S)) - log_S), l);
      }
    }
    if (threadIdx.x == 0) {
      p.loss[row] = l;
      const float listed = none ? 0.0f : whole / S;
      reinterpret_cast<float4 *>(p.stats)[row] = make_float4(m_row, listed, all.m, none ? 0.0f : fmaf(listed, down, -rest));
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
// at the token; of a listed outcome, e about ml, e kl - gt q.
struct RowTerms {
  float m, k0, k1, ml, kl, gt;
  int token;
};

template <bool LIST>
__device__ __forceinline__ RowTerms row_terms(const Bwd &p, int row) {
  const float4 s = __ldg(reinterpret_cast<const float4 *>(p.stats) + row);
  RowTerms r;
  const bool none = s.y == 0.0f;  // no distribution (or nothing listed): no gradient
  if constexpr (LIST) {
    const float g = none ? 0.0f : p.beta * __ldg(p.g + row);
    r.m = s.z;
    r.k0 = g * s.w;
    r.ml = s.x;
    r.kl = g * s.y;
    r.k1 = 0.0f;
    r.gt = g;
    r.token = -1;
  } else {
    r.m = s.x;
    r.ml = 0.0f;
    r.token = p.g ? token_at(p.tokens, p.token_bytes, row, p.cols) : -1;
    const float g = none || r.token < 0 ? 0.0f : p.beta * __ldg(p.g + row);
    const float ge = none || !p.g_ent ? 0.0f : p.beta * __ldg(p.g_ent + row);
    r.gt = g;
    r.k0 = (0.0f - (p.g_ent && !none ? g + ge * (s.w - s.z) : g)) * s.y;  // (+0 where there is no gradient)
    r.k1 = -ge * 0.69314718055994531f * s.y;
    r.kl = 0.0f;
  }
  return r;
}

__device__ __forceinline__ float scaled(float z, float m, float c2) { return max_nan((z - m) * c2, -1000.0f); }

// d itself: one row's chunk a CTA, in 16-byte vectors wherever the row starts.
// HBM-bound: 4096 x 50304 bfloat16 121 us (rows of 50257 the same; with lists of
// 64 138 to 141, their entries written behind the rest).  That is 6.8 TB/s of
// logits and gradient, above the copy rate: a part of either is still in L2 from
// the call before, or stays there.
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
          const float q = __ldg(p.list_q + (size_t)row * p.K + k);
          if (!(q < 0.0f)) {  // (not listed again)
            listed_at[i] = c;
            listed[i] = fmaf(ex2(scaled(load_one<DT>(z, c), r.ml, c2)), r.kl, -r.gt * q);
          }
        }
      }
    }
    __syncthreads();
  }
  auto grad = [&](float x, int c) {
    const float a = scaled(x, r.m, c2);
    float g = ex2(a) * (LIST ? r.k0 : fmaf(r.k1, a, r.k0));
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

// Codes of d, and d itself where wanted: tiles of block_scale.cuh.  The 16 lanes
// of a tile's row share RP rows: lane i works out the i-th one's factors (and
// which of the tile's columns are listed) while the tile's loads are in flight,
// and passes them on by shuffles; no barrier before the column maxima.  4096 x
// 50304 bfloat16 211 us (3.9 TB/s of logits read and codes written), with lists
// 302 (each tile row searches its list anew), rows of 50257 294 and 385 (element
// loads), 2048 x 50304 float32 116 and 173.  65 % of the issue slots are busy, two
// CTAs of 16 warps an SM between two barriers.
enum { kToken = 0, kTokenEntropy = 1, kListed = 2 };

template <int DT, int KIND, int OUT>
__global__ void __launch_bounds__(512, 2) k_loss_bwd_tiles(const Bwd p) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int RP = 4;
  constexpr bool LIST = KIND == kListed;
  using G = block::Geo<RP>;
  __shared__ block::ColScratch<RP> sc;
  constexpr int esz = kSize<DT>;
  const int tiles_c = (p.cols + block::kTile - 1) / block::kTile;
  const auto [row0, col0] = block::tile_at(blockIdx.x, tiles_c);
  const int c8 = threadIdx.x & 15, col = col0 + c8 * 8, r0 = row0 + (threadIdx.x >> 4);
  Raw8<DT> raw[RP];
  block::load_tile<DT>(p.z, p.ld / esz, p.vec_z, row0, col0, p.rows, p.cols, raw);
  RowTerms own = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, -1};  // rows behind the last: 0
  uint32_t marks[4] = {0, 0, 0, 0};                    // listed columns of the tile
  {
    const int row = r0 + c8 * G::kStep;
    if (c8 < RP && row < p.rows) {
      own = row_terms<LIST>(p, row);
      if constexpr (LIST) {
        const int *ids = p.list_ids + (size_t)row * p.K;
        int lo = 0, hi = p.K;
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
            if (b >> 5 == w) marks[w] |= 1u << (b & 31);
        }
        own.token = lo;  // the first entry there
      } else if (own.token >= 0) {
        own.token -= col0;
      }
    }
  }
  const float c2 = p.beta * kLog2e;
  const int lane0 = threadIdx.x & 16;
  float f[RP][8];
#pragma unroll
  for (int i = 0; i < RP; i++) {
    const float m = __shfl_sync(0xffffffffu, own.m, lane0 + i), k0 = __shfl_sync(0xffffffffu, own.k0, lane0 + i);
    const float gt = __shfl_sync(0xffffffffu, own.gt, lane0 + i);
    const int token = __shfl_sync(0xffffffffu, own.token, lane0 + i);
    float k1 = 0.0f;
    if constexpr (KIND == kTokenEntropy) k1 = __shfl_sync(0xffffffffu, own.k1, lane0 + i);
    block::unpack8<DT>(raw[i], f[i]);
    float2 e[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
      float2 a = __fmul2_rn(__fadd2_rn(make_float2(f[i][2 * j], f[i][2 * j + 1]), both(-m)), both(c2));
      if constexpr (KIND == kTokenEntropy) a = make_float2(max_nan(a.x, -1000.0f), max_nan(a.y, -1000.0f));
      e[j] = make_float2(ex2(a.x), ex2(a.y));
      float2 g;
      if constexpr (KIND == kTokenEntropy) g = __fmul2_rn(e[j], __ffma2_rn(both(k1), a, both(k0)));
      else g = __fmul2_rn(e[j], both(k0));
      f[i][2 * j] = g.x;
      f[i][2 * j + 1] = g.y;
    }
    if constexpr (LIST) {
      const float kl = __shfl_sync(0xffffffffu, own.kl, lane0 + i);
      uint32_t bits = 0;
#pragma unroll
      for (int w = 0; w < 4; w++) {
        const uint32_t word = __shfl_sync(0xffffffffu, marks[w], lane0 + i);
        if (c8 >> 2 == w) bits = word >> ((c8 & 3) * 8) & 0xffu;
      }
      if (bits) {  // rare: the list's entries of these columns
        const int row = r0 + i * G::kStep;
        const size_t at = (size_t)row * p.K;
        const uint8_t *z = p.z + (size_t)row * p.ld;  // read again (d, which may take its place, is written below)
        const float ml = __ldg(p.stats + 4 * (size_t)row);
        int k = token;
#pragma unroll 1
        for (uint32_t left = bits; left; left &= left - 1) {
          const int j = __ffs(left) - 1;
          while (k < p.K && __ldg(p.list_ids + at + k) != col + j) k++;
          if (k == p.K) break;  // (in no list in order)
          const float v = fmaf(ex2(scaled(load_one<DT>(z, col + j), ml, c2)), kl, -gt * __ldg(p.list_q + at + k));
#pragma unroll
          for (int n = 0; n < 8; n++)
            if (n == j) f[i][n] = v;
        }
      }
    } else {
      const int at = token - c8 * 8;
      if (token >= 0 && (unsigned)at < 8u) {
#pragma unroll
        for (int j = 0; j < 8; j++)
          if (j == at) f[i][j] += gt;
      }
    }
    if (col + 8 > p.cols) {  // the row's end
#pragma unroll
      for (int j = 0; j < 8; j++)
        if (col + j >= p.cols) f[i][j] = 0.0f;
    }
    if (r0 + i * G::kStep >= p.rows) {  // NaN here would spoil a column's scale: the clamped load is of another row
#pragma unroll
      for (int j = 0; j < 8; j++) f[i][j] = 0.0f;
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
