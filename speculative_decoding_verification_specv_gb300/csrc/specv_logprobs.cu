// specv_logprobs.cu -- log probabilities of given tokens, with the entropy of
// their rows and the most likely alternatives; and the gradient.
//
// For a row z of V logits and its token x:
//   m = max_v z_v,  S = sum_v e^{z_v - m},  T = sum_v e^{z_v - m} (z_v - m)
//   log p_x = (z_x - m) - ln S            entropy = ln S - T / S
// and the top_n largest entries in the order (value falling, index rising),
// each with its own log probability.
//
// The forward kernel reads a row once.  S CTAs (a cluster where S > 1) share a
// row, each an equal run of its 16-byte vectors; thread t of a CTA takes every
// NT-th vector of the run: its strip.  The streaming loop keeps S and T about a
// reference that follows the strip's maximum only when that has risen by more
// than kLazy, and, of the alternatives, nothing but the maximum and the vector that
// first held it (two instructions per vector), for the whole strip or for each of its
// eight segments (long rows, several alternatives).  After the loop
//   1. the 32 largest strip maxima over groups of NT / 32 threads are sorted, and
//      the top_n-th, as the pair (value, vector), is the threshold: at least
//      top_n entries are no worse, one in each of as many strips;
//   2. the strips or segments that reach it, about top_n of them, are read again and
//      their entries that reach it are collected;
//   3. a warp sorts those and keeps the first top_n.
// An entry worse than the threshold has top_n better ones, so none is missed; the
// pair's order makes equal values, a constant row for instance, select top_n
// strips as well.  Rows that put more than kCand entries above the threshold take
// a repeated search instead, whose result is the same.
//
// What bounds it.  2304 rows of 128256 fp32 entries take 184 us (1.18 GB, 6.4 TB/s, 0.95
// of the copy peak) with one alternative, 175 with none, 199 with 20; in bf16 102 us
// with none (0.59 GB, 5.8 TB/s: nine instructions per entry), 110 with one, 124 with 20.
// Few rows are bound by latency: nine rows of 128256 bf16 entries 7.0 us, five
// alternatives.  Rows of some thousand entries are bound by what a row costs whatever its
// length, a batch of the streaming loop and the selection: 30000 of 2500 fp32 entries
// (0.3 GB) 129 us with no alternatives, 227 with five.
#include <algorithm>

#include <cooperative_groups.h>

#include "specv_internal.h"
#include "specv_rowstat.cuh"

namespace cg = cooperative_groups;

namespace specv {

namespace {

constexpr int kUnroll = 4;      // vectors in flight per thread, and as many being folded
constexpr int kCand = 512;      // entries collected above the threshold
constexpr int kSegTop = 5;          // strips are cut into segments from so many alternatives on ...
constexpr int kSegVectors = 12288;  // ... in rows of so many vectors
// Terms may exceed the reference by e^8: sums stay far from overflow (2^31 e^8 <
// 10^13), and a strip of ordinary logits moves its reference once or twice.
constexpr float kLazy = 8.0f;

template <int NT, bool CLUSTER, int SEGS>
struct LogprobShared {
  float red[NT / 32][3];
  uint64_t group[32];
  uint64_t tau;
  int n_strips, n_cand;
  uint64_t keys[SEGS > 1 ? SEGS : 1][SEGS > 1 ? NT : 1];  // of every segment
  uint16_t strips[NT * SEGS];                              // thread + NT * segment
  uint64_t cand[kCand];
  uint64_t best[NT / 32];
  float4 part[CLUSTER ? kMaxCluster : 1];
  uint64_t part_top[CLUSTER ? kMaxCluster : 1][kMaxTop];
};

// Running sums of a strip.
struct StripSums {
  float ref = -3.402823466e38f;  // the reference of s and t (finite, or +inf)
  uint64_t s = 0, t = 0;         // packed partial sums
  float top = -INFINITY;         // the segment's maximum ...
  int top_vec = 0;               // ... and the first vector that holds it
};

template <typename T, int U>
__device__ __forceinline__ void fold(StripSums &a, const uint4 (&v)[U], int k, int step) {
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const float m = vector_max<T>(v[u]);
    if (m > a.top) {
      a.top = m;
      a.top_vec = k + u * step;
    }
  }
  if (a.top > a.ref + kLazy) {
    const float d = fmaxf(a.ref - a.top, kFarBelow), f = ex2(d * kLog2e);
    const uint64_t f2 = pack2(f, f);
    a.t = mul2(f2, fma2(a.s, pack2(d, d), a.t));
    a.s = mul2(f2, a.s);
    a.ref = a.top;
  }
  const uint64_t neg = pack2(-a.ref, -a.ref), scale = pack2(kLog2e, kLog2e);
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < Elem<T>::kPerVec / 2; ++i) {
      const uint64_t d = add2(pair_of<T>(v[u], i), neg);
      float d0, d1, x0, x1;
      unpack2(d, d0, d1);
      unpack2(mul2(d, scale), x0, x1);
      const uint64_t e = pack2(ex2(x0), ex2(x1));
      a.s = add2(a.s, e);
      a.t = fma2(e, pack2(fmaxf(d0, kFarBelow), fmaxf(d1, kFarBelow)), a.t);
    }
}

// The CTA's top_n largest keys among the strips of vectors [lo, hi): lane i of warp
// 0 returns the i-th.  Every thread calls it.
template <typename T, int NT, bool CLUSTER, int SEGS>
__device__ __forceinline__ uint64_t select_top(LogprobShared<NT, CLUSTER, SEGS> &sh,
                                               const RowVectors<T> &row, int lo, int hi, int top_n,
                                               int segs, int seg_vecs, uint64_t strip_key) {
  constexpr int kGroup = NT / 32;
  constexpr int VW = Elem<T>::kPerVec;
  const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint64_t key = strip_key;
#pragma unroll
  for (int off = kGroup / 2; off > 0; off >>= 1) key = max_u64(key, shfl_xor_u64(key, off));
  if (tid % kGroup == 0) sh.group[tid / kGroup] = key;
  if (tid == 0) sh.n_strips = sh.n_cand = 0;
  __syncthreads();
  if (warp == 0) {
    const uint64_t sorted = warp_sort(sh.group[lane]);
    if (lane == top_n - 1) sh.tau = sorted;
  }
  __syncthreads();
  const uint64_t tau = sh.tau;  // 0: fewer than top_n groups hold an entry, all entries count
  if (strip_key != 0 && strip_key >= tau)
    for (int g = 0; g < segs; ++g) {
      const uint64_t k = SEGS > 1 ? sh.keys[g][tid] : strip_key;
      if (k != 0 && k >= tau) sh.strips[atomicAdd(&sh.n_strips, 1)] = (uint16_t)(tid + NT * g);
    }
  __syncthreads();
  const float t_value = tau == 0 ? -INFINITY : key_value(tau);
  const int t_vec = tau == 0 ? -1 : (int)key_index(tau);
  const int n_strips = sh.n_strips;
  for (int64_t i = tid; i < (int64_t)n_strips * seg_vecs; i += NT) {
    const int s = (int)(i / seg_vecs), at = sh.strips[s];
    const int64_t of = (int64_t)(at / NT) * seg_vecs + (i - (int64_t)s * seg_vecs);
    const int64_t k64 = lo + at % NT + of * NT;
    const int k = k64 < hi ? (int)k64 : hi;
    if (k >= hi) continue;
    const uint4 v = row.load(k);
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      const float z = Elem<T>::get(v, e);
      if (z > t_value || (z == t_value && k <= t_vec)) {
        const int at = atomicAdd(&sh.n_cand, 1);
        if (at < kCand) sh.cand[at] = order_key(z, (uint32_t)row.index(k, e));
      }
    }
  }
  __syncthreads();
  const int n_cand = sh.n_cand;
  uint64_t top = 0;
  if (n_cand <= kCand) {
    if (warp == 0)
      for (int c = 0; c < n_cand; c += 32) {
        const uint64_t next = warp_sort(c + lane < n_cand ? sh.cand[c + lane] : 0);
        top = c == 0 ? next : warp_merge(top, next);
      }
    return top;
  }
  // the repeated search: the largest key below the last one found
  uint64_t last = ~0ull;
  for (int i = 0; i < top_n; ++i) {
    uint64_t k = 0;
    for (int64_t j = lo + tid; j < hi; j += NT) {
      const uint4 v = row.load((int)j);
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        const float z = Elem<T>::get(v, e);
        const uint64_t c = z > -INFINITY ? order_key(z, (uint32_t)row.index((int)j, e)) : 0;
        if (c < last && c > k) k = c;
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) k = max_u64(k, shfl_xor_u64(k, off));
    if (lane == 0) sh.best[warp] = k;
    __syncthreads();
    for (int w = 0; w < NT / 32; ++w) k = max_u64(k, sh.best[w]);
    if (lane == i) top = k;
    last = k;
    __syncthreads();
  }
  return top;
}

template <typename T, int NT, bool CLUSTER, int SEGS>
__global__ void __launch_bounds__(NT, NT == 32 ? 24 : 1024 / NT)
    logprobs_kernel(LogprobArgs a, int S) {
  __shared__ LogprobShared<NT, CLUSTER, SEGS> sh;
  const int64_t r = CLUSTER ? (int64_t)blockIdx.x / S : (int64_t)blockIdx.x;
  const int rank = CLUSTER ? (int)cg::this_cluster().block_rank() : 0;
  const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int V = a.V, top_n = a.top_n;
  const int32_t x = a.tokens[r];
  if (CLUSTER) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  if (x < 0 || x >= V) {  // no token (-1): the row is not read; an invalid one: NaN
    if (CLUSTER) cluster_sit_out();
    if (rank != 0) return;
    const float fill = x == -1 ? 0.0f : quiet_nan();
    if (tid == 0) {
      a.logprob[r] = fill;
      a.entropy[r] = fill;
      a.stats[r] = make_float2(fill, fill);
    }
    for (int i = tid; i < top_n; i += NT) {
      a.top_tokens[r * top_n + i] = -1;
      a.top_logprobs[r * top_n + i] = x == -1 ? -INFINITY : quiet_nan();
    }
    return;
  }
  const T *first = static_cast<const T *>(a.logits) + row_offset(r, a.N, a.stride_b, a.stride_n);
  const RowVectors<T> row(first, V, Span{a.logits, a.logits_end});
  const int per = (row.count + S - 1) / S;
  const int lo = min(row.count, rank * per), hi = min(row.count, lo + per);
  const float zx = rank == 0 && tid == 0 ? Elem<T>::load(first + x) : 0.0f;

  // -------------------------------------------------- the strip's sums and maximum
  StripSums sums;
  constexpr int kBatch = NT * kUnroll;
  constexpr uint32_t none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
  const int plain_hi = min(hi, row.full_hi);
  auto load_batch = [&](int base, uint4 (&v)[kUnroll]) {
    if (base >= row.full_lo && base <= plain_hi - kBatch) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) v[u] = row.load_full(base + u * NT + tid);
    } else {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int k = base + u * NT + tid;
        v[u] = make_uint4(none, none, none, none);
        if (k < hi) v[u] = row.load(k);
      }
    }
  };
  const int batches = (hi - lo + kBatch - 1) / kBatch;
  const int seg_batches = max(1, (batches + SEGS - 1) / SEGS);
  int segs = 0;
  uint64_t strip_key = 0;  // the strip's maximum (0: it has none)
  uint4 cur[kUnroll], next[kUnroll];
  load_batch(lo, cur);
  for (int base = lo; base < hi;) {
    const int stop = SEGS > 1 && hi - base > seg_batches * kBatch ? base + seg_batches * kBatch : hi;
    for (; base < stop; base += kBatch) {
      const bool more = hi - base > kBatch;
      if (more) load_batch(base + kBatch, next);
      fold<T, kUnroll>(sums, cur, base + tid, NT);
      if (more) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) cur[u] = next[u];
      }
    }
    const uint64_t key = sums.top > -INFINITY ? order_key(sums.top, (uint32_t)sums.top_vec) : 0;
    if (SEGS > 1) {
      sh.keys[segs][tid] = key;
      sums.top = -INFINITY;
    } else {
      strip_key = key;
    }
    ++segs;
  }
  if (SEGS > 1)
    for (int g = 0; g < segs; ++g) strip_key = max_u64(strip_key, sh.keys[g][tid]);

  // ------------------------------------------------------------------ merge: the CTA
  float M = strip_key != 0 ? key_value(strip_key) : -INFINITY, s, t, s1, t1;
  unpack2(sums.s, s, s1);
  unpack2(sums.t, t, t1);
  s += s1;
  t += t1;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, off));
  recentre(sums.ref, M, s, t);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    s += __shfl_xor_sync(~0u, s, off);
    t += __shfl_xor_sync(~0u, t, off);
  }
  if (lane == 0) {
    sh.red[warp][0] = M;
    sh.red[warp][1] = s;
    sh.red[warp][2] = t;
  }
  uint64_t top = 0;  // lane i of warp 0: the i-th largest key
  if (top_n > 0)
    top = select_top<T>(sh, row, lo, hi, top_n, segs, seg_batches * kUnroll, strip_key);
  else
    __syncthreads();
  if (warp == 0) {
    constexpr int kNW = NT / 32;
    M = lane < kNW ? sh.red[lane][0] : -INFINITY;
    s = lane < kNW ? sh.red[lane][1] : 0.0f;
    t = lane < kNW ? sh.red[lane][2] : 0.0f;
    const float m = M;
#pragma unroll
    for (int off = kNW / 2; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, off));
    M = __shfl_sync(~0u, M, 0);
    recentre(m, M, s, t);
#pragma unroll
    for (int off = kNW / 2; off > 0; off >>= 1) {
      s += __shfl_xor_sync(~0u, s, off);
      t += __shfl_xor_sync(~0u, t, off);
    }
  }

  // -------------------------------------------------------------- merge: the cluster
  if (CLUSTER) {
    cg::cluster_group cluster = cg::this_cluster();
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // every CTA has begun
    if (warp == 0) {
      if (lane == 0) *cluster.map_shared_rank(&sh.part[rank], 0) = make_float4(M, s, t, 0.0f);
      if (lane < top_n) *cluster.map_shared_rank(&sh.part_top[rank][lane], 0) = top;
    }
    cluster.sync();
    if (rank != 0) return;
    if (warp == 0) {
      const float4 p = lane < S ? sh.part[lane] : make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
      M = p.x;
      s = p.y;
      t = p.z;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, off));
      recentre(p.x, M, s, t);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        s += __shfl_xor_sync(~0u, s, off);
        t += __shfl_xor_sync(~0u, t, off);
      }
      if (top_n > 0)
        for (int q = 1; q < S; ++q) top = warp_merge(top, lane < top_n ? sh.part_top[q][lane] : 0);
    }
  }
  if (warp != 0) return;
  s = __shfl_sync(~0u, s, 0);
  t = __shfl_sync(~0u, t, 0);
  const bool bad = !(s < INFINITY);  // a NaN or +inf entry
  const bool empty = !bad && M == -INFINITY;
  const float ln = logf(s);
  if (lane == 0) {
    a.logprob[r] = bad ? quiet_nan() : empty ? -INFINITY : (zx - M) - ln;
    a.entropy[r] = bad ? quiet_nan() : empty ? 0.0f : fmaxf(ln - t / s, 0.0f);
    a.stats[r] = bad ? make_float2(quiet_nan(), quiet_nan()) : make_float2(M, empty ? 0.0f : ln);
  }
  if (lane < top_n) {
    const bool some = !bad && top != 0;
    a.top_tokens[r * top_n + lane] = some ? (int32_t)key_index(top) : -1;
    a.top_logprobs[r * top_n + lane] =
        bad ? quiet_nan() : some ? (key_value(top) - M) - ln : -INFINITY;
  }
}

// ------------------------------------------------------------------ the gradient
//   dz_v = g (1[v = x] - p_v) - h p_v (ln p_v + H)
// from the statistics of the forward pass: each entry is read and its gradient
// written once, at the copy rate (2048 rows of 128256 bf16 entries, a tenth of them without
// a token, 147 us, 6.8 TB/s).  A warp takes some packs per lane of one row, on the grid of
// the output's row.
constexpr int kGradNT = 256;
// Packs per lane: 8 in flight for aligned rows; rows to be joined keep 4 (their
// registers).  The 2048 rows above: 147 us with 8, 146 with 4, 162 with 2; 2349 rows of
// 14957 bf16 entries in a padded buffer: 29 us with 4, 35 with 8.
template <bool SHIFTED>
constexpr int kGradUnroll = SHIFTED ? 4 : 8;
template <bool SHIFTED>
constexpr int kGradUnit = 32 * kGradUnroll<SHIFTED>;  // packs of a warp's share

template <typename T, bool SHIFTED>
__global__ void __launch_bounds__(kGradNT) logprobs_grad_kernel(LogprobGradArgs a, uint32_t units) {
  constexpr int VW = Elem<T>::kPerVec;
  constexpr int U = kGradUnroll<SHIFTED>, kUnit = kGradUnit<SHIFTED>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint64_t unit = (uint64_t)blockIdx.x * (kGradNT / 32) + warp;  // share `unit % units` of row
  const int64_t r = unit >> 32 == 0 ? (uint32_t)unit / units : unit / units;
  if (r >= a.R) return;
  const int k0 = (int)(unit - (uint64_t)r * units) * kUnit;
  const T *row = static_cast<const T *>(a.logits) + row_offset(r, a.N, a.stride_b, a.stride_n);
  T *out = static_cast<T *>(a.out) + r * (int64_t)a.V;
  const Grid<T> grid(out, a.V);
  const int32_t x = a.tokens[r];
  const float2 st = a.stats[r];
  const float g = a.grad_logprob[r], H = a.entropy[r];
  const float h = a.grad_entropy != nullptr ? a.grad_entropy[r] : 0.0f;
  const bool bad = x < -1 || x >= a.V;
  const bool zero = x == -1 || (!bad && st.x == -INFINITY);
  PackTile<T, SHIFTED, U> z;
  if (zero || bad) {
    const float fill = zero ? 0.0f : quiet_nan();
#pragma unroll
    for (int i = 0; i < z.kPairs; ++i) z.put(i, fill, fill);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int k = k0 + 32 * j + lane;
      if (k < grid.count) store_pack<T>(out, grid, k, z.v[j]);
    }
    return;
  }
  const GridRow<T, SHIFTED> from(row, grid, Span{a.logits, a.logits_end});
  z.load(from, grid, k0, grid.count);
  // the lane that holds the token's entry
  const int64_t kx = ((int64_t)x + grid.mis) / VW;
  const bool mine = kx >= k0 && kx < k0 + kUnit && ((int)(kx - k0) & 31) == lane;
  float zx = 0.0f;
  if (mine) zx = widen(*reinterpret_cast<const volatile T *>(row + x));
  z.join(from, grid, k0, grid.count);

  const uint64_t m2 = pack2(-st.x, -st.x), l2 = pack2(-st.y, -st.y), scale = pack2(kLog2e, kLog2e);
  const float c = -__fmaf_rn(h, H, g);  // out = p (c - h ln p)
  const uint64_t c2 = pack2(c, c), h2 = pack2(-h, -h);
#pragma unroll
  for (int i = 0; i < z.kPairs; ++i) {
    const uint64_t lp = add2(add2(z.pair(i), m2), l2);
    float l0, l1, e0, e1, d0, d1;
    unpack2(lp, l0, l1);
    unpack2(mul2(lp, scale), e0, e1);
    const uint64_t in = fma2(h2, pack2(fmaxf(l0, kFarBelow), fmaxf(l1, kFarBelow)), c2);
    unpack2(mul2(pack2(ex2(e0), ex2(e1)), in), d0, d1);
    z.put(i, d0, d1);
  }
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int k = k0 + 32 * j + lane;
    if (k < grid.count) store_pack<T>(out, grid, k, z.v[j]);
  }
  if (mine) {
    const float lp = (zx - st.x) - st.y;
    out[x] = narrow<T>(__fmaf_rn(ex2(lp * kLog2e), __fmaf_rn(-h, fmaxf(lp, kFarBelow), c), g));
  }
}

template <typename T, int NT, bool CLUSTER, int SEGS>
cudaError_t launch_forward(const LogprobArgs &a, int S, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.R * S), 1, 1);
  cfg.blockDim = dim3(NT, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)S;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CLUSTER ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<T, NT, CLUSTER, SEGS>, a, S);
}

template <typename T>
cudaError_t forward(const LogprobArgs &a, int sms, int S, cudaStream_t stream) {
  constexpr int kVW = Elem<T>::kPerVec;
  const int64_t vectors = (a.V + kVW - 1) / kVW;
  // Short rows: a warp per row, up to 8 vectors per lane.
  if (S == 0 && vectors <= 32 * 8) return launch_forward<T, 32, false, 1>(a, 1, stream);
  // CTAs per row: as many as one wave of 4 CTAs per SM allows, up to 8, each with 1200
  // vectors at least (a batch of the streaming loop is 1024).  Measured: 9 rows of
  // 16032 vectors 6.6 us with S = 8, 7.8 with 16, 12.3 with 1; 185 rows of 12501 15.9
  // with S = 2, 18.7 with 1, 21.1 with 4 (two waves); 77 rows of 1101 5.8 with S = 1,
  // 6.5 with 2; 2304 rows of 32064 188 with S = 1, 214 with 2.
  if (S == 0) {
    const int64_t most = std::min<int64_t>(4 * sms / a.R, vectors / 1200);
    S = (int)std::max<int64_t>(1, std::min<int64_t>(most, 8));
  }
  while (S > 1 && a.R * S > INT32_MAX) S /= 2;
  if (S > 1) return launch_forward<T, 256, true, 1>(a, S, stream);
  // Segments, for several alternatives of long rows: what is read again of a strip,
  // from DRAM in a batch whose rows overfill L2, is then an eighth.  2304 rows, us with
  // and without: of 32064 vectors fp32 20 alternatives 199 and 279, 5 188 and 199, 4 188
  // and 194, bf16 20 224 and 295, 5 212 and 217, 4 212 and 212; of 16032 fp32 20 110 and
  // 134, 5 105 and 106, bf16 20 124 and 147, 5 119 and 116; of 12288 fp32 20 86 and 98, 5
  // 82 and 79, bf16 20 97 and 108, 5 93 and 88; of 9000 fp32 20 70 and 75, 5 66 and 63.
  // Many alternatives gain from shorter rows on than five do: near the edge the rule
  // costs five alternatives up to 5 % and gives twenty 10 %.
  return a.top_n >= kSegTop && vectors >= kSegVectors
             ? launch_forward<T, 256, false, 8>(a, 1, stream)
             : launch_forward<T, 256, false, 1>(a, 1, stream);
}

}  // namespace

cudaError_t logprobs_prepare() {
  cudaError_t e = cudaFuncSetAttribute(logprobs_kernel<float, 256, true, 1>,
                                       cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(logprobs_kernel<uint16_t, 256, true, 1>,
                             cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  return e;
}

cudaError_t logprobs_launch(const LogprobArgs &a, int dtype_bf16, int sms, int S,
                            cudaStream_t stream) {
  return dtype_bf16 ? forward<uint16_t>(a, sms, S, stream) : forward<float>(a, sms, S, stream);
}

template <typename T, bool SHIFTED>
static cudaError_t launch_grad(const LogprobGradArgs &a, cudaStream_t stream) {
  constexpr int VW = Elem<T>::kPerVec;
  // shares of a row, wherever it begins
  const int64_t packs = ((int64_t)a.V + (SHIFTED ? 2 : 1) * (VW - 1)) / VW;
  const int64_t units = (packs + kGradUnit<SHIFTED> - 1) / kGradUnit<SHIFTED>;
  const int64_t ctas = (a.R * units + kGradNT / 32 - 1) / (kGradNT / 32);
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  logprobs_grad_kernel<T, SHIFTED><<<(unsigned)ctas, kGradNT, 0, stream>>>(a, (uint32_t)units);
  return cudaGetLastError();
}

cudaError_t logprobs_grad_launch(const LogprobGradArgs &a, int dtype_bf16, cudaStream_t stream) {
  // Every row of both arrays begins on a 16-byte boundary where their addresses, the
  // strides and V in bytes are multiples of 16.
  const uint64_t bits = reinterpret_cast<uint64_t>(a.logits) | reinterpret_cast<uint64_t>(a.out) |
                        (uint64_t)(a.stride_b | a.stride_n | a.V) * (dtype_bf16 ? 2 : 4);
  if (dtype_bf16)
    return bits % 16 == 0 ? launch_grad<uint16_t, false>(a, stream)
                          : launch_grad<uint16_t, true>(a, stream);
  return bits % 16 == 0 ? launch_grad<float, false>(a, stream) : launch_grad<float, true>(a, stream);
}

}  // namespace specv
