// specv_rowstat.cuh -- what the log-probability and the distillation kernels
// share: rows as aligned vectors, packed fp32 arithmetic, ordered keys and their
// sorting across a warp.
//
// A row's softmax statistics are (m, S) = (max_v z_v, sum_v e^{z_v - m}); the
// entropy and the divergences need one more sum of the form
// T = sum_v e^{z_v - m} t_v, taken in the same pass.  All sums are fp32, formed
// per thread and merged in a fixed order, so equal inputs give equal outputs.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "specv_device.cuh"

namespace specv {

// Differences z - m are held above this where they are multiplied by e^{z - m}
// (which is 0 there): a masked entry then adds 0 * kFarBelow and not 0 * -inf.
constexpr float kFarBelow = -1e4f;

// Where row r = (b, n) of a [B][N][V] view with element strides (sb, sn, 1) begins
// (B * N < 2^31).
__device__ __forceinline__ int64_t row_offset(int64_t r, int N, int64_t sb, int64_t sn) {
  const uint32_t b = (uint32_t)r / (uint32_t)N, n = (uint32_t)r - b * (uint32_t)N;
  return b * sb + n * sn;
}

// Maximum over the warp; a NaN is passed over.
__device__ __forceinline__ float warp_max(float x) {
  float m;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
  return m;
}

__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fffffff); }

// fp32 -> the logits' type, rounded to nearest even.
template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ uint16_t narrow<uint16_t>(float x) {
  uint16_t h;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(x));
  return h;
}

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t x) { return bf16_bits_to_float(x); }

// A CTA that has nothing to do for its row stays until the cluster's last barrier all
// the same (it has arrived at the first one like the others): CTAs of one cluster that
// read different tokens or weights, because a caller writes them meanwhile, then
// produce one wrong row and not a store into a CTA that has ended.
__device__ __forceinline__ void cluster_sit_out() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// ------------------------------------------------------- packed pairs of fp32
// sm_103a adds, multiplies and fuses two fp32 values per instruction, each
// rounded as its scalar form.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t x, float &lo, float &hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// --------------------------------------------------------------- rows as vectors
// Replaces the entries of a vector that lie outside [0, V) by -inf; its first entry
// has index `first`.
template <typename T>
__device__ __forceinline__ void mask_outside(uint4 &v, int64_t first, int V) {
#pragma unroll
  for (int e = 0; e < Elem<T>::kPerVec; ++e)
    if (first + e < 0 || first + e >= V) Elem<T>::put_bits(v, e, Elem<T>::kNegInfBits);
}

// Entries [first, first + VW) of a row, one by one: what lies outside the row is -inf.
template <typename T>
__device__ __noinline__ uint4 load_entries(const T *row, int64_t first, int V) {
  constexpr uint32_t none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
  uint4 x = make_uint4(none, none, none, none);
#pragma unroll
  for (int e = 0; e < Elem<T>::kPerVec; ++e) {
    const int64_t c = first + e;
    if (c >= 0 && c < V) {
      uint32_t bits;
      if constexpr (sizeof(T) == 2) {
        uint16_t h;
        asm volatile("ld.global.u16 %0, [%1];" : "=h"(h) : "l"(row + c));
        bits = h;
      } else {
        asm volatile("ld.global.u32 %0, [%1];" : "=r"(bits) : "l"(row + c));
      }
      Elem<T>::put_bits(x, e, bits);
    }
  }
  return x;
}

// The memory that a view of rows spans, from its first entry to past its last.  Any
// whole 16-byte vector within it may be read: one that straddles a row's end brings
// entries of a neighbouring row or of the gap between rows, which are replaced by
// -inf.  Only the span's own ends are read entry by entry.
struct Span {
  const void *lo, *hi;
};

// A row seen as 16-byte vectors of the aligned memory that holds it: vector k covers
// entries [k VW - mis, (k + 1) VW - mis).  Vectors [full_lo, full_hi) lie within the
// row; vectors [lo, hi) within the span.
template <typename T>
struct RowVectors {
  const T *row;
  const char *base;  // 16-byte aligned, at or before the row's first entry
  int mis;           // entries between base and the row's first one
  int V;
  int count;         // vectors that hold entries of the row
  int full_lo, full_hi, lo, hi;

  __device__ __forceinline__ RowVectors(const T *row_, int V_, const Span &span) {
    constexpr int VW = Elem<T>::kPerVec;
    row = row_;
    const uint64_t at = reinterpret_cast<uint64_t>(row);
    mis = (int)(at % 16) / (int)sizeof(T);
    base = reinterpret_cast<const char *>(at - at % 16);
    V = V_;
    count = (int)(((int64_t)V + mis + VW - 1) / VW);
    full_lo = mis != 0 ? 1 : 0;
    full_hi = (int)(((int64_t)V + mis) / VW);
    lo = base >= span.lo ? 0 : 1;
    hi = base + (int64_t)count * 16 <= span.hi ? count : full_hi;
  }
  // the entry's index in the row (outside [0, V) for what an edge vector pads)
  __device__ __forceinline__ int64_t index(int k, int e) const {
    return (int64_t)k * Elem<T>::kPerVec + e - mis;
  }
  __device__ __forceinline__ uint4 load_full(int k) const {
    return ld_stream16(base + (int64_t)k * 16);
  }
  __device__ __forceinline__ uint4 load(int k) const {
    if (k < lo || k >= hi) return load_entries<T>(row, index(k, 0), V);
    uint4 v = load_full(k);
    if (k < full_lo || k >= full_hi) mask_outside<T>(v, index(k, 0), V);
    return v;
  }
};

// Entries 2 i and 2 i + 1 of a vector, widened to a packed pair.
template <typename T>
__device__ __forceinline__ uint64_t pair_of(const uint4 &v, int i) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t w = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
    return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  } else {
    return i == 0 ? pack2(__uint_as_float(v.x), __uint_as_float(v.y))
                  : pack2(__uint_as_float(v.z), __uint_as_float(v.w));
  }
}

// Largest entry of a vector; a NaN is passed over.
template <typename T>
__device__ __forceinline__ float vector_max(const uint4 &v) {
  if constexpr (sizeof(T) == 2) {
    uint32_t a, b;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(v.x), "r"(v.y));
    asm("max.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(v.z), "r"(v.w));
    asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
    return fmaxf(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
  } else {
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)),
                 fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
}

// A partial's sums (s, t) taken about m, moved to the reference M >= m.  An empty
// partial (s = 0) adds nothing.
__device__ __forceinline__ void recentre(float m, float M, float &s, float &t) {
  if (s == 0.0f) {
    t = 0.0f;
    return;
  }
  const float d = fmaxf(__fsub_rn(m, M), kFarBelow);
  const float f = ex2(__fmul_rn(d, kLog2e));
  t = __fmul_rn(f, __fmaf_rn(s, d, t));
  s = __fmul_rn(s, f);
}

// ------------------------------------------------------------------ ordered keys
// Values as whole numbers in the same order (-0 and +0 alike), over the
// complement of an index: the larger key is the larger value, and among equal
// values the lower index.  No entry has key 0.
__device__ __forceinline__ uint64_t order_key(float z, uint32_t index) {
  uint32_t b = __float_as_uint(__fadd_rn(z, 0.0f));
  b = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return ((uint64_t)b << 32) | (uint32_t)~index;
}
__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t b = (uint32_t)(key >> 32);
  return __uint_as_float((b & 0x80000000u) ? (b & 0x7fffffffu) : ~b);
}
__device__ __forceinline__ uint32_t key_index(uint64_t key) { return ~(uint32_t)key; }

__device__ __forceinline__ uint64_t shfl_xor_u64(uint64_t x, int off) {
  return __shfl_xor_sync(0xffffffffu, (unsigned long long)x, off);
}
__device__ __forceinline__ uint64_t max_u64(uint64_t a, uint64_t b) { return a > b ? a : b; }

// One compare-exchange of a bitonic network over the warp's lanes: the lower lane
// of each pair keeps the larger key where `falling`.
__device__ __forceinline__ uint64_t exchange(uint64_t key, int off, bool falling) {
  const uint64_t other = shfl_xor_u64(key, off);
  const bool lower = (threadIdx.x & off) == 0;
  return (key > other) == (lower == falling) ? key : other;
}
// The warp's keys in falling order (lane 0 the largest).
__device__ __forceinline__ uint64_t warp_sort(uint64_t key) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int off = size >> 1; off > 0; off >>= 1)
      key = exchange(key, off, size == 32 || (lane & size) == 0);
  return key;
}
// The 32 largest of two lists in falling order, in falling order.
__device__ __forceinline__ uint64_t warp_merge(uint64_t a, uint64_t b) {
  const uint64_t back = __shfl_sync(0xffffffffu, (unsigned long long)b, 31 - (threadIdx.x & 31));
  a = max_u64(a, back);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) a = exchange(a, off, true);
  return a;
}

// ------------------------------------------------------ rows on another row's grid
// A warp's share of a row, U 16-byte packs per lane, on the grid of a row that may
// sit differently against the 16-byte boundaries (the row of a contiguous output,
// say, whose width no vector divides): pack k of the grid covers entries
// [k VW - mis, (k + 1) VW - mis).  Lane l's j-th pack is k0 + 32 j + l.

template <typename T>
struct Grid {
  int mis;      // entries before the row in its first pack
  int V;
  int count;    // packs
  int full_lo, full_hi;  // packs wholly within the row

  __device__ __forceinline__ Grid(const void *row, int V_) {
    constexpr int VW = Elem<T>::kPerVec;
    mis = (int)(reinterpret_cast<uint64_t>(row) % 16) / (int)sizeof(T);
    V = V_;
    count = (int)(((int64_t)V + mis + VW - 1) / VW);
    full_lo = mis != 0 ? 1 : 0;
    full_hi = (int)(((int64_t)V + mis) / VW);
  }
  __device__ __forceinline__ bool full(int k) const { return k >= full_lo && k < full_hi; }
};

// A row to be read on a grid.  Where its entries sit `shift` entries into the
// aligned vectors of memory, a pack is joined from two of them, the second of
// which is the next lane's first: one load per pack and lane, and shuffles.
template <typename T, bool SHIFTED>
struct GridRow {
  const T *row;
  const char *base;   // the vector that holds the grid's pack 0 (or its start)
  int shift;          // 0..VW-1
  int first, last;    // the vectors of the row, counted from base, that may be read
  int lo, hi;         // packs whose vectors may be read

  __device__ __forceinline__ GridRow(const T *row_, const Grid<T> &grid, const Span &span) {
    constexpr int VW = Elem<T>::kPerVec;
    row = row_;
    const uint64_t at = reinterpret_cast<uint64_t>(row);
    if (!SHIFTED) {
      base = reinterpret_cast<const char *>(at);
      shift = 0;
      lo = first = 0;
      hi = last = grid.full_hi;
      return;
    }
    const int mis = (int)(at % 16) / (int)sizeof(T);
    const int d = mis - grid.mis;  // where the grid's pack 0 begins in the row's own vectors
    const int back = d < 0 ? 1 : 0;
    shift = d + back * VW;
    base = reinterpret_cast<const char *>(at - at % 16) - back * 16;
    // pack k is joined from vectors k and, with a shift, k + 1; of those up to the one
    // past the last pack, the ones within the span
    const int64_t before = static_cast<const char *>(span.lo) - base;
    const int64_t room = (static_cast<const char *>(span.hi) - base) / 16;
    first = before > 0 ? (int)((before + 15) / 16) : 0;
    last = room < grid.count + 1 ? (int)room : grid.count + 1;
    lo = first;
    hi = last - (shift != 0 ? 1 : 0);
  }
};

// VW entries from `shift` (1..VW-1) entries into vector a, continued in vector b.
template <typename T>
__device__ __forceinline__ uint4 shifted(const uint4 &a, const uint4 &b, int shift) {
  const int words = sizeof(T) == 2 ? shift >> 1 : shift;
  uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (words & 2) {
#pragma unroll
    for (int i = 0; i < 6; ++i) x[i] = x[i + 2];
  }
  if (words & 1) {
#pragma unroll
    for (int i = 0; i < 5; ++i) x[i] = x[i + 1];
  }
  if (sizeof(T) == 2 && (shift & 1)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __funnelshift_r(x[i], x[i + 1], 16);
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}

// Puts entries 2 i and 2 i + 1 of a vector, rounded to the logits' type.
template <typename T>
__device__ __forceinline__ void put_pair(uint4 &x, int i, float a, float b) {
  if constexpr (sizeof(T) == 2) {
    uint32_t &w = i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
  } else if (i == 0) {
    x.x = __float_as_uint(a);
    x.y = __float_as_uint(b);
  } else {
    x.z = __float_as_uint(a);
    x.w = __float_as_uint(b);
  }
}

template <typename T, bool SHIFTED, int U>
struct PackTile {
  static constexpr int kPairs = U * Elem<T>::kPerVec / 2;  // packed pairs of entries
  uint4 v[U + (SHIFTED ? 1 : 0)];

  __device__ __forceinline__ static uint4 load16(const char *p) {
    uint4 x;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                 : "l"(p));
    return x;
  }
  __device__ __forceinline__ static uint4 none() {
    constexpr uint32_t n = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
    return make_uint4(n, n, n, n);
  }
  // whether every pack of the share is whole, and its vectors may be read
  __device__ __forceinline__ static bool plain(const GridRow<T, SHIFTED> &r, const Grid<T> &grid,
                                               int k0, int end) {
    return k0 >= max(r.lo, grid.full_lo) && k0 + 32 * U <= min(min(r.hi, grid.full_hi), end);
  }

  // The vectors of packs k0 + 32 j + lane, on their way.
  __device__ __forceinline__ void load(const GridRow<T, SHIFTED> &r, const Grid<T> &grid, int k0,
                                       int end) {
    const int lane = threadIdx.x & 31;
    const char *p = r.base + ((int64_t)k0 + lane) * 16;
    if (plain(r, grid, k0, end)) {
#pragma unroll
      for (int j = 0; j < U; ++j) v[j] = load16(p + j * 512);
      // lane 31's second vector of the last pack, fetched by lane 0
      if (SHIFTED && r.shift != 0 && lane == 0) v[U] = load16(p + U * 512);
      return;
    }
#pragma unroll
    for (int j = 0; j < U + (SHIFTED ? 1 : 0); ++j) {
      const int k = k0 + 32 * j + lane;
      v[j] = none();
      if (k >= r.first && k < min(r.last, end + (SHIFTED ? 1 : 0)) && (j < U || lane == 0))
        v[j] = load16(p + j * 512);
    }
  }

  // Joins the packs from their vectors (every lane of the warp); what lies outside the
  // row or at `end` and after becomes -inf.
  __device__ __forceinline__ void join(const GridRow<T, SHIFTED> &r, const Grid<T> &grid, int k0,
                                       int end) {
    if constexpr (SHIFTED) {
      const int lane = threadIdx.x & 31;
      if (r.shift != 0) {
#pragma unroll
        for (int j = 0; j < U; ++j) {
          const uint4 &n = v[j + 1];
          uint4 next;  // the next lane's vector; lane 31's is the next pack's first
          next.x = __shfl_sync(0xffffffffu, lane == 0 ? n.x : v[j].x, (lane + 1) & 31);
          next.y = __shfl_sync(0xffffffffu, lane == 0 ? n.y : v[j].y, (lane + 1) & 31);
          next.z = __shfl_sync(0xffffffffu, lane == 0 ? n.z : v[j].z, (lane + 1) & 31);
          next.w = __shfl_sync(0xffffffffu, lane == 0 ? n.w : v[j].w, (lane + 1) & 31);
          v[j] = shifted<T>(v[j], next, r.shift);
        }
      }
      if (plain(r, grid, k0, end)) return;
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int k = k0 + 32 * j + lane;
        const int64_t c = (int64_t)k * Elem<T>::kPerVec - grid.mis;
        if (k >= end)
          v[j] = none();
        else if (k < r.lo || k >= r.hi)
          v[j] = load_entries<T>(r.row, c, grid.V);
        else if (!grid.full(k))
          mask_outside<T>(v[j], c, grid.V);
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
    for (int j = 0; j < U; ++j) m = fmaxf(m, vector_max<T>(v[j]));
    return m;
  }
  __device__ __forceinline__ void put(int i, float a, float b) {
    constexpr int kEach = Elem<T>::kPerVec / 2;
    put_pair<T>(v[i / kEach], i % kEach, a, b);
  }
};
// Writes a pack of a row on its own grid: a full one as one access, an edge one
// entry by entry.  Streaming stores: what is written is not read again here, and
// ordinary stores took the L2 from the rows still to be read (gradient of 2048 rows of
// 128256 bf16 entries: 157 us, streaming 147).
template <typename T>
__device__ __forceinline__ void store_pack(T *row, const Grid<T> &grid, int k, const uint4 &v) {
  constexpr int VW = Elem<T>::kPerVec;
  T *p = row + ((int64_t)k * VW - grid.mis);
  if (grid.full(k)) {
    __stcs(reinterpret_cast<uint4 *>(p), v);
  } else {
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      const int64_t c = (int64_t)k * VW - grid.mis + e;
      if (c >= 0 && c < grid.V) p[e] = narrow<T>(Elem<T>::get(v, e));
    }
  }
}

}  // namespace specv
