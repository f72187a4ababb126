// specv_distill.cu -- the divergence of the draft's rows from the target's, and
// its gradient with respect to the draft logits.
//
// With p = softmax(z_t), q = softmax(z_q) and a weight w per row pair:
//   forward  L = w sum_v p_v (ln p_v - ln q_v)   dL/dz_q = w (q - p)
//   reverse  L = w sum_v q_v (ln q_v - ln p_v)   dL/dz_q = w q (ln q - ln p - L/w)
// Pass 1 takes, about references r_t and r_q near the rows' maxima, the sums
//   S_t = sum e^{z_t - r_t},  S_q = sum e^{z_q - r_q},
//   T = sum e^{a} (a - c),  a = z - r of the leading row, c of the other one,
// so that L / w = T / S_a - ln S_a + ln S_c; pass 2 writes the gradient.
//
// S CTAs (a cluster) share a pair of rows, each the same run of both.  A thread
// keeps its entries of both rows in registers from the first pass to the second
// (a tile of kRegs registers per row and thread), so a pair that fits the
// cluster's registers is read once; of a longer one all but the last tile is read
// again, from L2.  One cluster barrier lies between the passes: every warp sends
// its partial sums to every CTA of the cluster, and each warp merges all of them.
#include <cooperative_groups.h>

#include "specv_block.cuh"
#include "specv_internal.h"
#include "specv_rowstat.cuh"

namespace cg = cooperative_groups;

namespace specv {

namespace {

constexpr int kRegs = 16;   // registers per thread that hold a row's entries
constexpr float kLazy = 8.0f;

// W consecutive entries of a row in registers, read and written as one access of
// W * sizeof(T) bytes; entry pairs are widened as they are used.
template <typename T, int W>
struct Pack;
template <typename T>
struct Pack<T, 16 / sizeof(T)> {
  static constexpr int kRegsEach = 4;
  uint4 v;
  __device__ __forceinline__ void none() {
    constexpr uint32_t n = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
    v = make_uint4(n, n, n, n);
  }
  __device__ __forceinline__ void load(const T *p) {
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
  }
  __device__ __forceinline__ uint64_t pair(int i) const { return pair_of<T>(v, i); }
  __device__ __forceinline__ float largest() const { return vector_max<T>(v); }
  // the same registers take the gradient's entries, pair by pair
  __device__ __forceinline__ void put(int i, float a, float b) {
    if constexpr (sizeof(T) == 2) {
      uint32_t &w = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
    } else if (i == 0) {
      v.x = __float_as_uint(a);
      v.y = __float_as_uint(b);
    } else {
      v.z = __float_as_uint(a);
      v.w = __float_as_uint(b);
    }
  }
  __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<uint4 *>(p) = v; }
};
template <>
struct Pack<uint16_t, 2> {
  static constexpr int kRegsEach = 1;
  uint32_t v;
  __device__ __forceinline__ void none() { v = 0xff80ff80u; }
  __device__ __forceinline__ void load(const uint16_t *p) {
    asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(v) : "l"(p));
  }
  __device__ __forceinline__ uint64_t pair(int) const {
    return pack2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  }
  __device__ __forceinline__ float largest() const {
    return fmaxf(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  }
  __device__ __forceinline__ void put(int, float a, float b) {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(b), "f"(a));
  }
  __device__ __forceinline__ void store(uint16_t *p) const { *reinterpret_cast<uint32_t *>(p) = v; }
};
// single entries, widened on load
template <typename T>
struct Single {
  float v;
  __device__ __forceinline__ void none() { v = -INFINITY; }
  __device__ __forceinline__ void load(const T *p) {
    if constexpr (sizeof(T) == 2) {
      uint16_t h;
      asm volatile("ld.global.L1::no_allocate.u16 %0, [%1];" : "=h"(h) : "l"(p));
      v = bf16_bits_to_float(h);
    } else {
      asm volatile("ld.global.L1::no_allocate.f32 %0, [%1];" : "=f"(v) : "l"(p));
    }
  }
  __device__ __forceinline__ void store(T *p) const { *p = narrow<T>(v); }
};

// A tile: a thread's entries of one row.  Access j covers entries
// ((j * NT) + tid) * W onwards of the tile; pairs(f) calls f(register-pair index)
// over packed pairs whatever W is.
template <typename T, int W, int NT>
struct Tile {
  static constexpr int kAccesses = kRegs / Pack<T, W>::kRegsEach;
  static constexpr int kPairsEach = W / 2;
  static constexpr int kPairs = kAccesses * kPairsEach;
  static constexpr int kEntries = kAccesses * W;  // per thread
  Pack<T, W> a[kAccesses];
  __device__ __forceinline__ void load(int j, const T *p) { a[j].load(p); }
  __device__ __forceinline__ void none(int j) { a[j].none(); }
  __device__ __forceinline__ void store(int j, T *p) const { a[j].store(p); }
  __device__ __forceinline__ uint64_t pair(int i) const {
    return a[i / kPairsEach].pair(i % kPairsEach);
  }
  __device__ __forceinline__ void put(int i, float x, float y) {
    a[i / kPairsEach].put(i % kPairsEach, x, y);
  }
  __device__ __forceinline__ float largest() const {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < kAccesses; ++j) m = fmaxf(m, a[j].largest());
    return m;
  }
};
template <typename T, int NT>
struct Tile<T, 1, NT> {
  static constexpr int kAccesses = kRegs;
  static constexpr int kPairs = kRegs / 2;
  static constexpr int kEntries = kRegs;
  Single<T> a[kAccesses];
  __device__ __forceinline__ void load(int j, const T *p) { a[j].load(p); }
  __device__ __forceinline__ void none(int j) { a[j].none(); }
  __device__ __forceinline__ void store(int j, T *p) const { a[j].store(p); }
  __device__ __forceinline__ uint64_t pair(int i) const { return pack2(a[2 * i].v, a[2 * i + 1].v); }
  __device__ __forceinline__ void put(int i, float x, float y) {
    a[2 * i].v = x;
    a[2 * i + 1].v = y;
  }
  __device__ __forceinline__ float largest() const {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < kAccesses; ++j) m = fmaxf(m, a[j].v);
    return m;
  }
};

// Partial sums of a row pair about the references (rt, rq).
struct PairSums {
  float rt = -3.402823466e38f, rq = -3.402823466e38f;
  float st = 0.0f, sq = 0.0f, t = 0.0f;
};

// The same sums about references (Mt, Mq), not below the old ones where a row has
// entries.  REVERSE: the draft row leads.
template <bool REVERSE>
__device__ __forceinline__ void move_to(PairSums &x, float Mt, float Mq) {
  const float dt = fmaxf(__fsub_rn(x.rt, Mt), kFarBelow), dq = fmaxf(__fsub_rn(x.rq, Mq), kFarBelow);
  const float ft = ex2(__fmul_rn(dt, kLog2e)), fq = ex2(__fmul_rn(dq, kLog2e));
  const float lead = REVERSE ? x.sq : x.st, f = REVERSE ? fq : ft;
  // (a sum that vanishes takes an infinite one of its terms with it)
  x.t = lead == 0.0f || f == 0.0f
            ? 0.0f
            : __fmul_rn(f, __fmaf_rn(lead, REVERSE ? dq - dt : dt - dq, x.t));
  x.st = x.st == 0.0f ? 0.0f : __fmul_rn(x.st, ft);
  x.sq = x.sq == 0.0f ? 0.0f : __fmul_rn(x.sq, fq);
  x.rt = Mt;
  x.rq = Mq;
}

template <int NT>
struct DistillShared {
  float4 a[kMaxCluster * (NT / 32)];  // (rt, st, rq, sq) of every warp of the cluster
  float t[kMaxCluster * (NT / 32)];
};

template <typename T, int W, int NT, bool REVERSE>
__global__ void __launch_bounds__(NT, 768 / NT) distill_kernel(DistillArgs a, int S) {
  using TileT = Tile<T, W, NT>;
  constexpr int kNW = NT / 32;
  __shared__ DistillShared<NT> sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = S > 1 ? (int)cluster.block_rank() : 0;
  const int64_t r = (int64_t)blockIdx.x / S;
  const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int V = a.V;
  const T *zt =
      static_cast<const T *>(a.target) + row_offset(r, a.K, a.target_stride_b, a.target_stride_k);
  const T *zq =
      static_cast<const T *>(a.draft) + row_offset(r, a.K, a.draft_stride_b, a.draft_stride_k);
  T *out = a.out_grad == nullptr ? nullptr : static_cast<T *>(a.out_grad) + r * (int64_t)V;
  // this CTA's accesses [lo, hi) of W entries, in tiles (V is a multiple of W)
  const int n = V / W, per = (n + S - 1) / S;
  const int lo = min(n, rank * per), hi = min(n, lo + per);
  constexpr int kTile = TileT::kAccesses * NT;
  const int tiles = (hi - lo + kTile - 1) / kTile;
  const float w = a.weight == nullptr ? 1.0f : a.weight[r];

  TileT xt, xq;
  auto zero_fill = [&]() {
    if (out == nullptr) return;
#pragma unroll
    for (int i = 0; i < TileT::kPairs; ++i) xq.put(i, 0.0f, 0.0f);
    for (int k = lo + tid; k < hi; k += NT) xq.store(0, out + (int64_t)k * W);
  };
  if (w == 0.0f) {
    if (rank == 0 && tid == 0) a.out_loss[r] = 0.0f;
    zero_fill();
    return;
  }
  if (S > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");

  auto load_tile = [&](int tile) {
    const int base = lo + tile * kTile + tid;
#pragma unroll
    for (int j = 0; j < TileT::kAccesses; ++j) {
      const int k = base + j * NT;
      if (k < hi) {
        xt.load(j, zt + (int64_t)k * W);
        xq.load(j, zq + (int64_t)k * W);
      } else {
        xt.none(j);
        xq.none(j);
      }
    }
  };

  // ------------------------------------------------------------- pass 1: the sums
  PairSums x;
  const uint64_t scale = pack2(kLog2e, kLog2e), minus = pack2(-1.0f, -1.0f);
  for (int tile = 0; tile < tiles; ++tile) {
    load_tile(tile);
    const float mt = xt.largest(), mq = xq.largest();
    if (mt > x.rt + kLazy || mq > x.rq + kLazy) move_to<REVERSE>(x, fmaxf(x.rt, mt), fmaxf(x.rq, mq));
    const uint64_t nt = pack2(-x.rt, -x.rt), nq = pack2(-x.rq, -x.rq);
    uint64_t st = 0, sq = 0;
    float t0 = 0.0f, t1 = 0.0f;
#pragma unroll
    for (int i = 0; i < TileT::kPairs; ++i) {
      const uint64_t dt = add2(xt.pair(i), nt), dq = add2(xq.pair(i), nq);
      float a0, a1, b0, b1, d0, d1;
      unpack2(mul2(dt, scale), a0, a1);
      unpack2(mul2(dq, scale), b0, b1);
      a0 = ex2(a0);
      a1 = ex2(a1);
      b0 = ex2(b0);
      b1 = ex2(b1);
      st = add2(st, pack2(a0, a1));
      sq = add2(sq, pack2(b0, b1));
      unpack2(REVERSE ? fma2(dt, minus, dq) : fma2(dq, minus, dt), d0, d1);
      // an entry without leading probability adds nothing (its difference may be
      // infinite or NaN); one with it against a masked entry adds +inf
      const float e0 = REVERSE ? b0 : a0, e1 = REVERSE ? b1 : a1;
      if (e0 > 0.0f) t0 = __fmaf_rn(e0, d0, t0);
      if (e1 > 0.0f) t1 = __fmaf_rn(e1, d1, t1);
    }
    float s0, s1;
    unpack2(st, s0, s1);
    x.st += s0 + s1;
    unpack2(sq, s0, s1);
    x.sq += s0 + s1;
    x.t += t0 + t1;
  }

  // --------------------------------- merge: the warp, then all warps of the cluster
  auto merge_lanes = [&](PairSums &y) {
    float Mt = y.rt, Mq = y.rq;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      Mt = fmaxf(Mt, __shfl_xor_sync(~0u, Mt, off));
      Mq = fmaxf(Mq, __shfl_xor_sync(~0u, Mq, off));
    }
    move_to<REVERSE>(y, Mt, Mq);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      y.st += __shfl_xor_sync(~0u, y.st, off);
      y.sq += __shfl_xor_sync(~0u, y.sq, off);
      y.t += __shfl_xor_sync(~0u, y.t, off);
    }
  };
  merge_lanes(x);
  const float4 mine = make_float4(x.rt, x.st, x.rq, x.sq);
  if (S > 1) {
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // every CTA has begun
    if (lane < S) {
      *cluster.map_shared_rank(&sh.a[rank * kNW + warp], lane) = mine;
      *cluster.map_shared_rank(&sh.t[rank * kNW + warp], lane) = x.t;
    }
    cluster.sync();
  } else {
    if (lane == 0) {
      sh.a[warp] = mine;
      sh.t[warp] = x.t;
    }
    __syncthreads();
  }
  const int parts = S * kNW;
  PairSums y;
  for (int i = lane; i < parts; i += 32) {
    const float4 p = sh.a[i];
    y.rt = fmaxf(y.rt, p.x);
    y.rq = fmaxf(y.rq, p.z);
  }
  for (int i = lane; i < parts; i += 32) {
    const float4 p = sh.a[i];
    PairSums z;
    z.rt = p.x;
    z.st = p.y;
    z.rq = p.z;
    z.sq = p.w;
    z.t = sh.t[i];
    move_to<REVERSE>(z, y.rt, y.rq);
    y.st += z.st;
    y.sq += z.sq;
    y.t += z.t;
  }
  merge_lanes(y);

  const bool bad = !(y.st < INFINITY) || !(y.sq < INFINITY);  // a NaN or +inf entry
  const bool empty = !bad && (y.st == 0.0f || y.sq == 0.0f);  // a row masks every entry
  const float lt = logf(y.st), lq = logf(y.sq);
  float kl = REVERSE ? y.t / y.sq - lq + lt : y.t / y.st - lt + lq;
  kl = bad ? quiet_nan() : kl < 0.0f ? 0.0f : kl;
  if (rank == 0 && tid == 0) a.out_loss[r] = empty ? 0.0f : w * kl;
  if (out == nullptr) return;
  if (empty) {
    zero_fill();
    return;
  }

  // --------------------------------------------------------- pass 2: the gradient
  const float wg = bad ? quiet_nan() : w;
  const float c = kl == INFINITY ? quiet_nan() : lt - lq - kl;
  const uint64_t mt2 = pack2(-y.rt, -y.rt), mq2 = pack2(-y.rq, -y.rq);
  const uint64_t lt2 = pack2(-lt * kLog2e, -lt * kLog2e), lq2 = pack2(-lq * kLog2e, -lq * kLog2e);
  const uint64_t w2 = pack2(wg, wg), c2 = pack2(c, c);
  for (int tile = tiles - 1; tile >= 0; --tile) {
    if (tile != tiles - 1) load_tile(tile);
#pragma unroll
    for (int i = 0; i < TileT::kPairs; ++i) {
      const uint64_t dt = add2(xt.pair(i), mt2), dq = add2(xq.pair(i), mq2);
      float q0, q1, g0, g1;
      unpack2(fma2(dq, scale, lq2), q0, q1);
      q0 = ex2(q0);
      q1 = ex2(q1);
      if (REVERSE) {
        const uint64_t wq = mul2(w2, pack2(q0, q1));
        unpack2(mul2(wq, add2(fma2(dt, minus, dq), c2)), g0, g1);
        if (q0 == 0.0f) g0 = 0.0f;
        if (q1 == 0.0f) g1 = 0.0f;
        if (bad) g0 = g1 = quiet_nan();
      } else {
        float p0, p1;
        unpack2(fma2(dt, scale, lt2), p0, p1);
        unpack2(mul2(w2, fma2(pack2(ex2(p0), ex2(p1)), minus, pack2(q0, q1))), g0, g1);
      }
      xq.put(i, g0, g1);
    }
    const int base = lo + tile * kTile + tid;
#pragma unroll
    for (int j = 0; j < TileT::kAccesses; ++j) {
      const int k = base + j * NT;
      if (k < hi) xq.store(j, out + (int64_t)k * W);
    }
  }
}

template <typename T, int W, int NT, bool REVERSE>
cudaError_t launch(const DistillArgs &a, int S, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.B * a.K * S), 1, 1);
  cfg.blockDim = dim3(NT, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)S;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = S > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, distill_kernel<T, W, NT, REVERSE>, a, S);
}

constexpr int kSmallNT = 64, kNT = 256;

template <typename T, int W, bool REVERSE>
cudaError_t plan(const DistillArgs &a, int S, cudaStream_t stream) {
  // Short rows: one tile of 64 threads.
  if (S == 0 && a.V <= Tile<T, W, kSmallNT>::kEntries * kSmallNT)
    return launch<T, W, kSmallNT, REVERSE>(a, 1, stream);
  // The fewest CTAs whose registers hold the pair of rows, 16 at most.
  if (S == 0) {
    constexpr int64_t kTile = (int64_t)Tile<T, W, kNT>::kEntries * kNT;
    const int64_t need = (a.V + kTile - 1) / kTile;
    S = need < kMaxCluster ? (int)need : kMaxCluster;
  }
  while (S > 1 && a.B * a.K * S > INT32_MAX) S /= 2;
  return launch<T, W, kNT, REVERSE>(a, S, stream);
}

template <typename T, int W>
cudaError_t plan(const DistillArgs &a, int reverse, int S, cudaStream_t stream) {
  return reverse ? plan<T, W, true>(a, S, stream) : plan<T, W, false>(a, S, stream);
}

template <typename T, int W>
cudaError_t prepare() {
  cudaError_t e = cudaFuncSetAttribute(distill_kernel<T, W, kNT, false>,
                                       cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(distill_kernel<T, W, kNT, true>,
                             cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  return e;
}

}  // namespace

cudaError_t distill_prepare() {
  cudaError_t e = prepare<float, 4>();
  if (e == cudaSuccess) e = prepare<float, 1>();
  if (e == cudaSuccess) e = prepare<uint16_t, 8>();
  if (e == cudaSuccess) e = prepare<uint16_t, 2>();
  if (e == cudaSuccess) e = prepare<uint16_t, 1>();
  return e;
}

cudaError_t distill_launch(const DistillArgs &a, int dtype_bf16, int reverse, int S,
                           cudaStream_t stream) {
  // The widest access that every row of all three arrays allows: their addresses,
  // the strides and V in bytes are multiples of it.
  const int elem = dtype_bf16 ? 2 : 4;
  const uint64_t bits =
      reinterpret_cast<uint64_t>(a.target) | reinterpret_cast<uint64_t>(a.draft) |
      reinterpret_cast<uint64_t>(a.out_grad) |
      (uint64_t)(a.target_stride_b | a.target_stride_k | a.draft_stride_b | a.draft_stride_k | a.V) *
          elem;
  if (dtype_bf16) {
    if (bits % 16 == 0) return plan<uint16_t, 8>(a, reverse, S, stream);
    return bits % 4 == 0 ? plan<uint16_t, 2>(a, reverse, S, stream)
                         : plan<uint16_t, 1>(a, reverse, S, stream);
  }
  return bits % 16 == 0 ? plan<float, 4>(a, reverse, S, stream)
                        : plan<float, 1>(a, reverse, S, stream);
}

}  // namespace specv
