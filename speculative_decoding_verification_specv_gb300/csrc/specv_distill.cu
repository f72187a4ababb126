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
// Long rows.  S CTAs (a cluster) share a pair, each the same run of both rows, cut
// into chunks of 4 KB per row.  An issuing warp brings the chunks into shared memory
// with bulk copies, six or four of them ahead of the 128 consuming threads; after pass
// 1 these last ones are still there for pass 2, the others are copied again, most of
// them from L2 (1.2 of the rows' bytes leave DRAM).  Between the passes every warp sends
// its partial sums to every CTA of the cluster, and each warp merges all of them: one
// cluster barrier.  Rows that lie off the 16-byte boundaries are joined from whole
// vectors as they are read from shared memory.
//
// What bounds it.  2048 pairs of 128256 fp32 entries take 545 us (3.15 GB, 5.8 TB/s,
// 0.85 of the copy peak), 1024 of bf16 155 us (0.79 GB, 5.1 TB/s); the loss alone, one
// pass, 298 us (7.1 TB/s) and 87 (6.0).  The warps issue 0.51
// (fp32) and 0.73 (bf16) of the time, at four exponentials and some thirty instructions
// per entry pair.  Of a CTA's time at 2048 fp32 pairs 13 % go by until its first chunk
// is there, 38 % in pass 1, 18 % in the cluster barrier, 28 % in pass 2 (clock stamps,
// four CTAs per SM), which the other CTAs of the SM cover only in part.  Tried and not
// kept: the pair in registers instead (715 us with S = 8), register double buffers (841),
// clusters that stay and copy ahead into their next pair (607), 16 KB chunks or more
// threads with fewer CTAs per SM (570 to 750), sums without a maximum search (574).
//
// Short rows: a warp holds a pair in registers.
#include <algorithm>

#include <cooperative_groups.h>

#include "specv_block.cuh"
#include "specv_internal.h"
#include "specv_rowstat.cuh"

namespace cg = cooperative_groups;

namespace specv {

namespace {

constexpr float kLazy = 8.0f;   // what a term may exceed its reference by, as a power of e

// Logits may lie as far apart as their type reaches (a mask of its lowest value in one
// row of a pair only), and T adds such a distance for every entry of the run with up to
// e^kLazy times it.  Distances are therefore held times kSmall where they go into T: a
// power of two, so that nothing else is rounded differently, and T stays below 2^128 with
// 2^31 entries.  Only distances below 2^-82 lose bits.
constexpr float kLarge = 17592186044416.0f;  // 2^44
constexpr float kSmall = 1.0f / kLarge;

// Partial sums of a row pair about the references (rt, rq).
struct PairSums {
  float rt = -3.402823466e38f, rq = -3.402823466e38f;
  float st = 0.0f, sq = 0.0f;
  float t = 0.0f;  // T times kSmall
};

// The same sums about references (Mt, Mq), not below the old ones where a row has
// entries.  REVERSE: the draft row leads.  The leading row's move scales T, both rows'
// moves enter it as they are: the other row's may be any distance.
template <bool REVERSE>
__device__ __forceinline__ void move_to(PairSums &x, float Mt, float Mq) {
  const float dt = __fmaf_rn(x.rt, kSmall, -Mt * kSmall), dq = __fmaf_rn(x.rq, kSmall, -Mq * kSmall);
  const float ft = ex2(__fmul_rn(dt, kLog2e * kLarge)), fq = ex2(__fmul_rn(dq, kLog2e * kLarge));
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

// ------------------------------------------------------------------ shared steps
struct Merged {
  float lt, lq;  // log2 S of the target's and the draft's row
  float rt, rq;  // their references
  float kl;      // the divergence: NaN for a row with a NaN or +inf
  bool empty;    // a row masks every entry
};

template <bool REVERSE>
__device__ __forceinline__ void merge_lanes(PairSums &y) {
  move_to<REVERSE>(y, warp_max(y.rt), warp_max(y.rq));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    y.st += __shfl_xor_sync(~0u, y.st, off);
    y.sq += __shfl_xor_sync(~0u, y.sq, off);
    y.t += __shfl_xor_sync(~0u, y.t, off);
  }
}

// log2 of a positive normal number: exactly the exponent, and the SFU's logarithm
// (absolute error near 2^-22 there) of a mantissa in [0.75, 1.5).
__device__ __forceinline__ float log2_of(float s) {
  const int bits = __float_as_int(s), e = (bits - 0x3f400000) >> 23;
  return lg2(__int_as_float(bits - (e << 23))) + (float)e;
}

// What follows from a pair's sums.
template <bool REVERSE>
__device__ __forceinline__ Merged merged(const PairSums &y) {
  Merged m;
  const bool bad = !(y.st < INFINITY) || !(y.sq < INFINITY);
  m.empty = !bad && (y.st == 0.0f || y.sq == 0.0f);
  m.lt = log2_of(y.st);
  m.lq = log2_of(y.sq);
  m.rt = y.rt;
  m.rq = y.rq;
  const float mean = __fmul_rn(__fdividef(y.t, REVERSE ? y.sq : y.st), kLarge);
  const float kl = __fmaf_rn(REVERSE ? m.lt - m.lq : m.lq - m.lt, kLn2, mean);
  m.kl = bad ? quiet_nan() : kl < 0.0f ? 0.0f : kl;
  return m;
}

// The partials of `parts` warps (a: rt, st, rq, sq), merged by a warp; every lane
// returns the same.
template <bool REVERSE>
__device__ __forceinline__ Merged merge_parts(const float4 *a, const float *t, int parts) {
  const int lane = threadIdx.x & 31;
  PairSums y;
  for (int i = lane; i < parts; i += 32) {
    y.rt = fmaxf(y.rt, a[i].x);
    y.rq = fmaxf(y.rq, a[i].z);
  }
  for (int i = lane; i < parts; i += 32) {
    PairSums z;
    z.rt = a[i].x;
    z.st = a[i].y;
    z.rq = a[i].z;
    z.sq = a[i].w;
    z.t = t[i];
    move_to<REVERSE>(z, y.rt, y.rq);
    y.st += z.st;
    y.sq += z.sq;
    y.t += z.t;
  }
  merge_lanes<REVERSE>(y);
  return merged<REVERSE>(y);
}

// t += e d where e > 0, else nothing, whatever d is.
__device__ __forceinline__ void fma_if_positive(float &t, float e, float d) {
  asm("{\n\t.reg .pred p;\n\tsetp.gt.f32 p, %1, 0f00000000;\n\t@p fma.rn.f32 %0, %1, %2, %0;\n\t}"
      : "+f"(t)
      : "f"(e), "f"(d));
}

// Adds the entries of two tiles to the sums.
template <typename T, bool REVERSE, typename TileT>
__device__ __forceinline__ void fold_pair(PairSums &x, const TileT &xt, const TileT &xq) {
  const float mt = xt.largest(), mq = xq.largest();
  if (mt > x.rt + kLazy || mq > x.rq + kLazy)
    move_to<REVERSE>(x, fmaxf(x.rt, mt), fmaxf(x.rq, mq));
  const float rt = -x.rt * kSmall, rq = -x.rq * kSmall;
  const uint64_t nt = pack2(rt, rt), nq = pack2(rq, rq);
  const uint64_t small = pack2(kSmall, kSmall), minus = pack2(-1.0f, -1.0f);
  const uint64_t scale = pack2(kLog2e * kLarge, kLog2e * kLarge);
  uint64_t st = 0, sq = 0;
  float t0 = 0.0f, t1 = 0.0f;
#pragma unroll
  for (int i = 0; i < TileT::kPairs; ++i) {
    const uint64_t dt = fma2(xt.pair(i), small, nt), dq = fma2(xq.pair(i), small, nq);
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
    fma_if_positive(t0, e0, d0);
    fma_if_positive(t1, e1, d1);
  }
  float s0, s1;
  unpack2(st, s0, s1);
  x.st += s0 + s1;
  unpack2(sq, s0, s1);
  x.sq += s0 + s1;
  x.t += t0 + t1;
}

// What the gradient needs of a row pair, in packed pairs.  The reverse gradient is a
// product of q and a distance: q is held times 2^kGradShift and distances divided by it, so
// that a q just below the smallest normal number times a large distance is not lost, and
// the distance of two entries anywhere in fp32's range is finite.  (16: the exponents of
// the entries that matter, -20 to 0, stay small numbers and lose no bits to the shift.)
constexpr int kGradShift = 16;
template <bool REVERSE>
struct GradTerms {
  // (reverse: distances in units of 2^kGradShift)
  static constexpr float kUnit = REVERSE ? 1.0f / (1 << kGradShift) : 1.0f;
  uint64_t rt, rq;  // -r
  uint64_t lt, lq;  // -log2 (kUnit S)
  uint64_t w, c;
  bool bad;
  __device__ __forceinline__ GradTerms(const Merged &m, float weight) {
    constexpr float unit = kUnit, log2_unit = REVERSE ? kGradShift : 0.0f;
    bad = m.kl != m.kl;
    const float wg = bad ? quiet_nan() : weight;
    const float cc = m.kl == INFINITY ? quiet_nan() : ((m.lt - m.lq) * kLn2 - m.kl) * unit;
    const float ft = -m.rt * unit, fq = -m.rq * unit;
    const float et = log2_unit - m.lt, eq = log2_unit - m.lq;
    rt = pack2(ft, ft);
    rq = pack2(fq, fq);
    lt = pack2(et, et);
    lq = pack2(eq, eq);
    w = pack2(wg, wg);
    c = pack2(cc, cc);
  }
};

// Puts the gradient of the entries of xt and xq into xq.
template <typename T, bool REVERSE, typename TileT>
__device__ __forceinline__ void gradient(const GradTerms<REVERSE> &g, const TileT &xt, TileT &xq) {
  constexpr float kUnit = GradTerms<REVERSE>::kUnit, kScale = kLog2e / kUnit;
  const uint64_t scale = pack2(kScale, kScale), minus = pack2(-1.0f, -1.0f);
  const uint64_t unit = pack2(kUnit, kUnit);
#pragma unroll
  for (int i = 0; i < TileT::kPairs; ++i) {
    const uint64_t dt = REVERSE ? fma2(xt.pair(i), unit, g.rt) : add2(xt.pair(i), g.rt);
    const uint64_t dq = REVERSE ? fma2(xq.pair(i), unit, g.rq) : add2(xq.pair(i), g.rq);
    float q0, q1, g0, g1;
    unpack2(fma2(dq, scale, g.lq), q0, q1);
    q0 = ex2(q0);
    q1 = ex2(q1);
    if (REVERSE) {
      unpack2(mul2(g.w, mul2(pack2(q0, q1), add2(fma2(dt, minus, dq), g.c))), g0, g1);
      if (q0 == 0.0f) g0 = 0.0f;
      if (q1 == 0.0f) g1 = 0.0f;
      if (g.bad) g0 = g1 = quiet_nan();
    } else {
      float p0, p1;
      unpack2(fma2(dt, scale, g.lt), p0, p1);
      unpack2(mul2(g.w, fma2(pack2(ex2(p0), ex2(p1)), minus, pack2(q0, q1))), g0, g1);
    }
    xq.put(i, g0, g1);
  }
}

// ------------------------------------------------------------------- short rows
// A warp per pair, which it holds in registers: U packs of each row per lane.
constexpr int kShortNT = 128;
constexpr int kShortPacks = 8;  // U at most: pairs of 2048 bf16 or 1024 fp32 entries

// (four CTAs per SM: 12495 pairs of 1513 bf16 entries, half of them left out, 39 us, with
// the registers it would take otherwise 42; with none left out 46 both)
template <typename T, bool SHIFTED, bool REVERSE, int U>
__global__ void __launch_bounds__(kShortNT, 4) distill_short_kernel(DistillArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t r = (int64_t)blockIdx.x * (kShortNT / 32) + (threadIdx.x >> 5);
  if (r >= a.B * a.K) return;
  const T *zt =
      static_cast<const T *>(a.target) + row_offset(r, a.K, a.target_stride_b, a.target_stride_k);
  const T *zq =
      static_cast<const T *>(a.draft) + row_offset(r, a.K, a.draft_stride_b, a.draft_stride_k);
  T *out = a.out_grad == nullptr ? nullptr : static_cast<T *>(a.out_grad) + r * (int64_t)a.V;
  const Grid<T> grid(out != nullptr ? static_cast<const void *>(out) : zq, a.V);
  const float w = a.weight == nullptr ? 1.0f : a.weight[r];
  PackTile<T, SHIFTED, U> xt, xq;
  auto store = [&]() {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int k = 32 * j + lane;
      if (k < grid.count) store_pack<T>(out, grid, k, xq.v[j]);
    }
  };
  auto zero = [&]() {
    if (lane == 0) a.out_loss[r] = 0.0f;
    if (out == nullptr) return;
#pragma unroll
    for (int i = 0; i < xq.kPairs; ++i) xq.put(i, 0.0f, 0.0f);
    store();
  };
  if (w == 0.0f) {
    zero();
    return;
  }
  const GridRow<T, SHIFTED> rt(zt, grid, Span{a.target, a.target_end}),
      rq(zq, grid, Span{a.draft, a.draft_end});
  xt.load(rt, grid, 0, grid.count);
  xq.load(rq, grid, 0, grid.count);
  xt.join(rt, grid, 0, grid.count);
  xq.join(rq, grid, 0, grid.count);
  PairSums x;
  fold_pair<T, REVERSE>(x, xt, xq);
  merge_lanes<REVERSE>(x);
  const Merged m = merged<REVERSE>(x);
  if (m.empty) {
    zero();
    return;
  }
  if (lane == 0) a.out_loss[r] = w * m.kl;
  if (out == nullptr) return;
  gradient<T, REVERSE>(GradTerms<REVERSE>(m, w), xt, xq);
  store();
}

// -------------------------------------------------------------------- long rows
constexpr int kNT = 128;     // consuming threads; one more warp issues the copies
constexpr int kUnroll = 2;   // packs per thread of a chunk
constexpr int kChunk = kNT * kUnroll;              // packs of a chunk
constexpr int kChunkBytes = (kChunk + 1) * 16;     // a shifted row's chunk needs one vector more

// BUFFERS: chunks of both rows held per CTA, MIN_CTAS: CTAs per SM that leaves room for.
template <int BUFFERS>
struct __align__(16) DistillShared {
  float4 a[kMaxCluster * (kNT / 32)];  // (rt, st, rq, sq) of every warp of the cluster
  float t[kMaxCluster * (kNT / 32)];
  uint64_t full[BUFFERS], empty[BUFFERS];
  int lost;  // set when a copy did not land in time
};

// A thread's packs of a chunk, read from shared memory.  `inner`: the chunk's packs are
// whole in every row, and it has no end; else entries outside the row become -inf.
template <typename T, bool SHIFTED>
struct ChunkTile {
  static constexpr int kPairs = kUnroll * Elem<T>::kPerVec / 2;
  uint4 v[kUnroll];
  __device__ __forceinline__ void load(const GridRow<T, SHIFTED> &r, const Grid<T> &grid,
                                       const uint4 *buf, int k0, int end, bool inner) {
    constexpr int VW = Elem<T>::kPerVec;
    const uint4 *p = buf + (int)threadIdx.x;
    if (inner) {
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) v[j] = p[j * kNT];
      if (SHIFTED && r.shift != 0) {
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) v[j] = shifted<T>(v[j], p[j * kNT + 1], r.shift);
      }
      return;
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const int k = k0 + j * kNT + (int)threadIdx.x;
      v[j] = PackTile<T, SHIFTED, 1>::none();
      if (k >= end) continue;
      if (k >= r.lo && k < r.hi) {
        v[j] = p[j * kNT];
        if (SHIFTED && r.shift != 0) v[j] = shifted<T>(v[j], p[j * kNT + 1], r.shift);
        if (SHIFTED && !grid.full(k)) mask_outside<T>(v[j], (int64_t)k * VW - grid.mis, grid.V);
      } else if (SHIFTED) {
        v[j] = load_entries<T>(r.row, (int64_t)k * VW - grid.mis, grid.V);
      }
    }
  }
  __device__ __forceinline__ uint64_t pair(int i) const {
    constexpr int kEach = Elem<T>::kPerVec / 2;
    return pair_of<T>(v[i / kEach], i % kEach);
  }
  __device__ __forceinline__ float largest() const {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) m = fmaxf(m, vector_max<T>(v[j]));
    return m;
  }
  __device__ __forceinline__ void put(int i, float a, float b) {
    constexpr int kEach = Elem<T>::kPerVec / 2;
    put_pair<T>(v[i / kEach], i % kEach, a, b);
  }
};

// Waits as mbar_wait does, for phase `parity` of `bar`, at most kWaitLimitNs; the
// thread is suspended meanwhile (kSuspendNs at a time) instead of polling: warps that
// poll take the issue slots of those at work.
constexpr uint32_t kSuspendNs = 1000 * 1000;
__device__ __forceinline__ bool wait_suspended(uint64_t *bar, uint32_t parity) {
  uint64_t t0 = 0;
  for (uint32_t it = 0; it < kSpinLimit; ++it) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(kSuspendNs)
        : "memory");
    if (ok) return true;
    if (it == 0) t0 = global_timer_ns();
    if (global_timer_ns() - t0 > kWaitLimitNs) break;
  }
  return mbar_try_wait(bar, parity);  // (the time may have passed while the GPU was lent out)
}

// tma_load_1d with an L2 eviction policy.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar,
                                          uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], "
      "%2, [%3], %4;" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

template <typename T, bool SHIFTED, bool REVERSE, int BUFFERS, int MIN_CTAS>
__global__ void __launch_bounds__(kNT + 32, MIN_CTAS) distill_kernel(DistillArgs a, int S) {
  constexpr int kNW = kNT / 32, kBuffers = BUFFERS;
  extern __shared__ __align__(16) unsigned char chunks[];  // [kBuffers][2][kChunkBytes]
  __shared__ DistillShared<BUFFERS> sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = S > 1 ? (int)cluster.block_rank() : 0;
  const int64_t r = (int64_t)blockIdx.x / S;
  const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T *zt =
      static_cast<const T *>(a.target) + row_offset(r, a.K, a.target_stride_b, a.target_stride_k);
  const T *zq =
      static_cast<const T *>(a.draft) + row_offset(r, a.K, a.draft_stride_b, a.draft_stride_k);
  T *out = a.out_grad == nullptr ? nullptr : static_cast<T *>(a.out_grad) + r * (int64_t)a.V;
  // the packs of the gradient's row (of the draft's where none is wanted)
  const Grid<T> grid(out != nullptr ? static_cast<const void *>(out) : zq, a.V);
  const int per = (grid.count + S - 1) / S;
  const int lo = min(grid.count, rank * per), hi = min(grid.count, lo + per);
  const int n = (hi - lo + kChunk - 1) / kChunk;  // chunks of this CTA
  const float w = a.weight == nullptr ? 1.0f : a.weight[r];

  auto zero_fill = [&]() {  // by the consuming threads
    if (out == nullptr || warp == kNW) return;
    for (int k = lo + tid; k < hi; k += kNT) store_pack<T>(out, grid, k, make_uint4(0, 0, 0, 0));
  };
  if (tid == 0) {
    sh.lost = 0;
    for (int b = 0; b < kBuffers; ++b) {
      mbar_init(&sh.full[b], 1);
      mbar_init(&sh.empty[b], kNW);
    }
    mbar_fence_init();
  }
  if (S > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  __syncthreads();
  if (w == 0.0f) {
    if (rank == 0 && tid == 0) a.out_loss[r] = 0.0f;
    zero_fill();
    if (S > 1) cluster_sit_out();
    return;
  }

  const GridRow<T, SHIFTED> rt(zt, grid, Span{a.target, a.target_end}),
      rq(zq, grid, Span{a.draft, a.draft_end});
  auto buffer = [&](int c, int which) {
    return reinterpret_cast<uint4 *>(chunks + ((c % kBuffers) * 2 + which) * kChunkBytes);
  };
  // Chunk c goes to buffer c mod kBuffers.  The copies run 0 .. n-1 for pass 1, then
  // n-kBuffers-1 .. 0 for pass 2, which begins with the chunks still held.  The m-th
  // copy into a buffer completes phase m of its `full` barrier and waits for phase
  // m-1 of its `empty` one; load_1 and load_2 are the m of a chunk in each pass.
  auto load_1 = [&](int c) { return c / kBuffers; };
  auto load_2 = [&](int c) {
    const int held = (n - 1 - c % kBuffers) / kBuffers;  // copies before the held chunk's
    return held + (held - c / kBuffers);
  };

  if (warp == kNW) {  // ------------------------------------------- the issuing warp
    bool fine = true;
    // what is read again is kept in L2 rather than what is not (2048 pairs of 128256
    // fp32 entries, six chunks held: 549 us, without 567)
    uint64_t keep, drop;
    asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(keep));
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(drop));
    auto issue = [&](int c, int m, uint64_t policy) {
      const int b = c % kBuffers, k0 = lo + c * kChunk, k1 = min(hi, k0 + kChunk);
      if (m > 0) fine = fine && wait_suspended(&sh.empty[b], (m - 1) & 1);
      if (!fine || *(volatile int *)&sh.lost) return;
      const int t0 = max(k0, rt.first), t1 = min(k1 + (rt.shift != 0), rt.last);
      const int q0 = max(k0, rq.first), q1 = min(k1 + (rq.shift != 0), rq.last);
      const uint32_t bt = t1 > t0 ? (t1 - t0) * 16 : 0, bq = q1 > q0 ? (q1 - q0) * 16 : 0;
      mbar_arrive_expect_tx(&sh.full[b], bt + bq);
      if (bt) bulk_load(buffer(c, 0) + (t0 - k0), rt.base + (int64_t)t0 * 16, bt, &sh.full[b], policy);
      if (bq) bulk_load(buffer(c, 1) + (q0 - k0), rq.base + (int64_t)q0 * 16, bq, &sh.full[b], policy);
    };
    if (lane == 0)
      for (int c = 0; c < n; ++c)
        issue(c, load_1(c), out != nullptr && c + kBuffers < n ? keep : drop);
    __syncwarp();
    if (S > 1) {
      asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
      cluster.sync();
    } else {
      __syncthreads();
    }
    if (out == nullptr || n <= kBuffers) return;
    const Merged m = merge_parts<REVERSE>(sh.a, sh.t, S * kNW);
    if (!m.empty && lane == 0)
      for (int c = n - kBuffers - 1; c >= 0; --c) issue(c, load_2(c), drop);
    return;
  }

  // --------------------------------------------------------------- pass 1: the sums
  ChunkTile<T, SHIFTED> xt, xq;
  PairSums x;
  // A copy that does not land in time (not expected) ends the copying and makes the
  // results NaN; the copies still in flight, kBuffers at most, are waited for as well.
  int lost = 0;
  // packs that are whole in all three rows
  const int in_lo = max(max(rt.lo, rq.lo), grid.full_lo);
  const int in_hi = min(min(rt.hi, rq.hi), min(grid.full_hi, hi));
  auto is_inner = [&](int c) {
    const int k0 = lo + c * kChunk;
    return k0 >= in_lo && k0 + kChunk <= in_hi;
  };
  auto take = [&](int c, int m, bool wait, bool inner) {
    if (wait && lost <= kBuffers && (!wait_suspended(&sh.full[c % kBuffers], m & 1) || lost > 0)) {
      ++lost;
      *(volatile int *)&sh.lost = 1;
    }
    const int k0 = lo + c * kChunk;
    xt.load(rt, grid, buffer(c, 0), k0, hi, inner);
    xq.load(rq, grid, buffer(c, 1), k0, hi, inner);
  };
  auto release = [&](int c) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.empty[c % kBuffers]);
  };
  for (int c = 0; c < n; ++c) {
    take(c, load_1(c), true, is_inner(c));
    fold_pair<T, REVERSE>(x, xt, xq);
    if (c + kBuffers < n) release(c);
  }
  if (lost > 0) x.st = quiet_nan();

  // --------------------------------- merge: the warp, then all warps of the cluster
  merge_lanes<REVERSE>(x);
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
  const Merged m = merge_parts<REVERSE>(sh.a, sh.t, S * kNW);
  if (rank == 0 && tid == 0) a.out_loss[r] = m.empty ? 0.0f : w * m.kl;
  if (out == nullptr) return;
  if (m.empty) {
    zero_fill();
    return;
  }

  // ----------------------------------------------------------- pass 2: the gradient
  GradTerms<REVERSE> g(m, w);
  for (int c = n - 1; c >= 0; --c) {
    const bool inner = is_inner(c);
    take(c, load_2(c), c < n - kBuffers, inner);
    if (c >= kBuffers) release(c);
    if (lost > 0) {
      g.w = pack2(quiet_nan(), quiet_nan());
      g.bad = true;
    }
    gradient<T, REVERSE>(g, xt, xq);
    const int k0 = lo + c * kChunk + tid;
    if (inner) {
      uint4 *to = reinterpret_cast<uint4 *>(out + ((int64_t)k0 * Elem<T>::kPerVec - grid.mis));
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) __stcs(to + j * kNT, xq.v[j]);
    } else {
#pragma unroll
      for (int j = 0; j < kUnroll; ++j)
        if (k0 + j * kNT < hi) store_pack<T>(out, grid, k0 + j * kNT, xq.v[j]);
    }
  }
}

template <typename T, bool SHIFTED, bool REVERSE, int BUFFERS, int MIN_CTAS>
cudaError_t launch_long(const DistillArgs &a, int S, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.B * a.K * S), 1, 1);
  cfg.blockDim = dim3(kNT + 32, 1, 1);
  cfg.dynamicSmemBytes = BUFFERS * 2 * kChunkBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)S;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = S > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, distill_kernel<T, SHIFTED, REVERSE, BUFFERS, MIN_CTAS>, a, S);
}

template <typename T, bool SHIFTED, bool REVERSE>
cudaError_t plan(const DistillArgs &a, int sms, int S, cudaStream_t stream) {
  constexpr int kVW = Elem<T>::kPerVec;
  // packs of a row, wherever it begins
  const int64_t packs = ((int64_t)a.V + (SHIFTED ? 2 : 1) * (kVW - 1)) / kVW;
  if (S == 0 && packs <= 32 * kShortPacks) {
    const int64_t ctas = (a.B * a.K + kShortNT / 32 - 1) / (kShortNT / 32);
    if (packs <= 32 * 2)
      distill_short_kernel<T, SHIFTED, REVERSE, 2><<<(unsigned)ctas, kShortNT, 0, stream>>>(a);
    else if (packs <= 32 * 4)
      distill_short_kernel<T, SHIFTED, REVERSE, 4><<<(unsigned)ctas, kShortNT, 0, stream>>>(a);
    else
      distill_short_kernel<T, SHIFTED, REVERSE, kShortPacks>
          <<<(unsigned)ctas, kShortNT, 0, stream>>>(a);
    return cudaGetLastError();
  }
  // CTAs per pair: so many that each takes 4096 packs of a row at most, more while one
  // wave of 4 CTAs per SM has room for them, 8 at most.  More CTAs hold more of the pair
  // but wait longer for one another.  Measured, us: 2048 pairs of 32064 packs S = 8 544,
  // 6 595, 4 663; 1024 of 16032 S = 4 155, 8 158, 2 178; 396 of 9760 S = 3 47, 1 46, 8 48;
  // 1776 of 3019 S = 1 48, 2 54; 34 of 14540 S = 8 9.0, 4 11.9, 2 20.7.
  if (S == 0) {
    const int64_t pairs = a.B * a.K;
    S = (int)std::min<int64_t>((packs + 4095) / 4096, 8);
    const int64_t room = std::min<int64_t>(4 * sms / pairs, packs / 512);
    if (S < room) S = (int)std::min<int64_t>(room, 8);
  }
  while (S > 1 && a.B * a.K * S > INT32_MAX) S /= 2;
  // Six chunks held and four CTAs per SM where that is one wave, else four and six: a
  // full GPU gains more from CTAs than from what they hold.  Us, six held and four: 1024
  // pairs of 16032 packs 159 and 155, 2048 of 32064 555 and 544, 880 of 3429 (joined)
  // 48.0 and 43.0, 9207 of 1140 96 and 88; 133 of 6251 (joined) 15.8 and 16.9, 24 of
  // 12545 8.1 and 8.7.
  if (a.B * a.K * S <= 4 * sms) return launch_long<T, SHIFTED, REVERSE, 6, 4>(a, S, stream);
  return launch_long<T, SHIFTED, REVERSE, 4, 6>(a, S, stream);
}

template <typename T, bool SHIFTED>
cudaError_t plan(const DistillArgs &a, int reverse, int sms, int S, cudaStream_t stream) {
  return reverse ? plan<T, SHIFTED, true>(a, sms, S, stream)
                 : plan<T, SHIFTED, false>(a, sms, S, stream);
}

template <typename T, bool SHIFTED, bool REVERSE, int BUFFERS, int MIN_CTAS>
cudaError_t prepare_one() {
  const auto kernel = distill_kernel<T, SHIFTED, REVERSE, BUFFERS, MIN_CTAS>;
  cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             BUFFERS * 2 * kChunkBytes);
  return e;
}
template <typename T, bool SHIFTED, bool REVERSE>
cudaError_t prepare_both() {
  const cudaError_t e = prepare_one<T, SHIFTED, REVERSE, 6, 4>();
  return e == cudaSuccess ? prepare_one<T, SHIFTED, REVERSE, 4, 6>() : e;
}
template <typename T>
cudaError_t prepare() {
  cudaError_t e = prepare_both<T, false, false>();
  if (e == cudaSuccess) e = prepare_both<T, false, true>();
  if (e == cudaSuccess) e = prepare_both<T, true, false>();
  if (e == cudaSuccess) e = prepare_both<T, true, true>();
  return e;
}

}  // namespace

cudaError_t distill_prepare() {
  const cudaError_t e = prepare<float>();
  return e == cudaSuccess ? prepare<uint16_t>() : e;
}

cudaError_t distill_launch(const DistillArgs &a, int dtype_bf16, int reverse, int sms, int S,
                           cudaStream_t stream) {
  // Every row of all three arrays begins on a 16-byte boundary where their
  // addresses, the strides and V in bytes are multiples of 16.
  const uint64_t bits =
      reinterpret_cast<uint64_t>(a.target) | reinterpret_cast<uint64_t>(a.draft) |
      reinterpret_cast<uint64_t>(a.out_grad) |
      (uint64_t)(a.target_stride_b | a.target_stride_k | a.draft_stride_b | a.draft_stride_k | a.V) *
          (dtype_bf16 ? 2 : 4);
  if (dtype_bf16)
    return bits % 16 == 0 ? plan<uint16_t, false>(a, reverse, sms, S, stream)
                          : plan<uint16_t, true>(a, reverse, sms, S, stream);
  return bits % 16 == 0 ? plan<float, false>(a, reverse, sms, S, stream)
                        : plan<float, true>(a, reverse, sms, S, stream);
}

}  // namespace specv
