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

// Where row r = (b, n) of a [B][N][V] view with element strides (sb, sn, 1) begins.
__device__ __forceinline__ int64_t row_offset(int64_t r, int N, int64_t sb, int64_t sn) {
  const int64_t b = r / N;
  return b * sb + (r - b * N) * sn;
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
// A row seen as 16-byte vectors of the aligned memory that holds it: vector k
// covers entries [k VW - mis, (k + 1) VW - mis).  Vectors [full_lo, full_hi) lie
// within the row; the others (the first of a row off a 16-byte boundary, the last
// of a ragged one) are read entry by entry, and what is not the row's is -inf.
template <typename T>
struct RowVectors {
  const char *base;  // 16-byte aligned, at or before the row's first entry
  int mis;           // entries between base and the row's first one
  int V;
  int count;         // vectors that hold entries of the row
  int full_lo, full_hi;

  __device__ __forceinline__ RowVectors(const T *row, int V_) {
    constexpr int VW = Elem<T>::kPerVec;
    const uint64_t at = reinterpret_cast<uint64_t>(row);
    mis = (int)(at % 16) / (int)sizeof(T);
    base = reinterpret_cast<const char *>(at - at % 16);
    V = V_;
    count = (int)(((int64_t)V + mis + VW - 1) / VW);
    full_lo = mis != 0 ? 1 : 0;
    full_hi = (int)(((int64_t)V + mis) / VW);
  }
  __device__ __forceinline__ bool full(int k) const { return k >= full_lo && k < full_hi; }
  // the entry's index in the row (outside [0, V) for what an edge vector pads)
  __device__ __forceinline__ int64_t index(int k, int e) const {
    return (int64_t)k * Elem<T>::kPerVec + e - mis;
  }
  __device__ __forceinline__ uint4 load_full(int k) const {
    return ld_stream16(base + (int64_t)k * 16);
  }
  __device__ __noinline__ uint4 load_edge(int k) const {
    constexpr uint32_t none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
    uint4 v = make_uint4(none, none, none, none);
    const T *p = reinterpret_cast<const T *>(base + (int64_t)k * 16);
#pragma unroll
    for (int e = 0; e < Elem<T>::kPerVec; ++e) {
      const int64_t c = index(k, e);
      if (c >= 0 && c < V) Elem<T>::put_bits(v, e, Elem<T>::load_bits(p + e));
    }
    return v;
  }
  __device__ __forceinline__ uint4 load(int k) const { return full(k) ? load_full(k) : load_edge(k); }
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

}  // namespace specv
