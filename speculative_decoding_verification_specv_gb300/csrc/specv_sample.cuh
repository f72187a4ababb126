// specv_sample.cuh -- what the sampling kernels of long and of short rows share: the order of
// values, a row's parameters and weights, exact sums.
#pragma once

#include <cstdint>

#include "specv_internal.h"
#include "specv_rowstat.cuh"

namespace specv {

// 16 bytes through the ordinary path: the row may be overwritten by the same kernel
// (filtering in place), which the read-only path does not allow.
__device__ __forceinline__ uint4 load16(const char *p) {
  uint4 x;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "l"(p));
  return x;
}
template <typename T>
__device__ __forceinline__ uint4 load_vec(const RowVectors<T> &row, int k) {
  if (k < row.lo || k >= row.hi) return load_entries<T>(row.row, row.index(k, 0), row.V);
  uint4 v = load16(row.base + (int64_t)k * 16);
  if (k < row.full_lo || k >= row.full_hi) mask_outside<T>(v, row.index(k, 0), row.V);
  return v;
}

// max(a, b), NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

// The order of values as whole numbers (-0 and +0 alike): the upper half of order_key.
__device__ __forceinline__ uint32_t value_key(float z) {
  const uint32_t b = __float_as_uint(__fadd_rn(z, 0.0f));
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}

// What a row's draw depends on.
struct RowParams {
  float m, r;       // the largest entry, 1 / T
  float min_p;
  float scale;      // weights are counted in units of 1 / scale
  // the threshold: entries above tau, and those equal to it up to index `tie`
  float tau;
  int tie;

  __device__ __forceinline__ float weight(float z) const {
    return expf(__fmul_rn(__fsub_rn(z, m), r));
  }
  __device__ __forceinline__ bool in_order(float z, int i) const {
    return z > tau || (z == tau && i <= tie);
  }
  // whether a threshold leaves anything out
  __device__ __forceinline__ bool cut() const { return tau > -INFINITY; }
  __device__ __forceinline__ uint64_t units(float w) const {
    return __float2ull_rn(w * scale);  // (a power of two: exact)
  }
};

__device__ __forceinline__ uint64_t warp_sum_u64(uint64_t x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += shfl_xor_u64(x, off);
  return x;
}

// Sums of weights in whole units, each weight as RowParams::units counts it: every sum of the
// same weights is the same number, whatever its order.  t = fl(1 + w) holds w to 2^-23, and
// w - (t - 1) is exact; added to M = 1.5 2^23 units it is rounded to a unit.  The lower bits
// of t and of that sum are whole numbers, added up in 32 bits: up to 256 weights of at most 1.
// (Weights one by one as whole numbers, by the conversion instructions: 2048 rows of 128256
// fp32 entries that nothing filters 303 us, 235 this way.)
struct UnitSum {
  uint32_t hi, lo;
};
struct Units {
  static constexpr uint32_t kOne = 0x3f800000u;  // 1, in bits
  uint64_t magic;   // M twice
  uint32_t bits;    // of M
  uint32_t step;    // units in 2^-23
  __device__ __forceinline__ explicit Units(float scale) {
    const float m = __fmul_rn(12582912.0f, __frcp_rn(scale));  // (powers of two: exact)
    magic = pack2(m, m);
    bits = __float_as_uint(m);
    step = (uint32_t)(scale * 1.1920928955078125e-7f);
  }
  // An empty sum that n weights will be added to.
  __device__ __forceinline__ UnitSum begin(int n) const {
    return UnitSum{0u - (uint32_t)n * kOne, 0u - (uint32_t)n * bits};
  }
  // What each of two weights adds.
  __device__ __forceinline__ void split(float w0, float w1, UnitSum &a, UnitSum &b) const {
    const uint64_t w = pack2(w0, w1), t = add2(w, pack2(1.0f, 1.0f)), minus = pack2(-1.0f, -1.0f);
    const uint64_t rest = add2(fma2(add2(t, minus), minus, w), magic);
    float x, y;
    unpack2(t, x, y);
    a.hi = __float_as_uint(x), b.hi = __float_as_uint(y);
    unpack2(rest, x, y);
    a.lo = __float_as_uint(x), b.lo = __float_as_uint(y);
  }
  // What a weight of 0 adds.
  __device__ __forceinline__ UnitSum none() const { return UnitSum{kOne, bits}; }
  __device__ __forceinline__ static void add(UnitSum &s, const UnitSum &a, const UnitSum &b) {
    s.hi += a.hi + b.hi;
    s.lo += a.lo + b.lo;
  }
  __device__ __forceinline__ uint64_t total(const UnitSum &s) const {
    return (uint64_t)s.hi * step + (uint64_t)(int64_t)(int32_t)s.lo;
  }
  // The sum over the warp of 32 weights of each lane.
  __device__ __forceinline__ uint64_t warp_total(const UnitSum &s) const {
    const uint64_t hi = ((uint64_t)__reduce_add_sync(~0u, s.hi >> 16) << 16) +
                        __reduce_add_sync(~0u, s.hi & 0xffffu);
    return hi * step + (uint64_t)(int64_t)__reduce_add_sync(~0u, (int32_t)s.lo);
  }
};

// Largest entry of a vector; NaN if it holds one.
template <typename T>
__device__ __forceinline__ float vector_max_nan(const uint4 &v) {
  if constexpr (sizeof(T) == 2) {
    uint32_t a, b;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(v.x), "r"(v.y));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(v.z), "r"(v.w));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
    return max_nan(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
  } else {
    return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)),
                   max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
}

// floor(f x), or ceil(f x), of a share f in [0, 1] of a sum x < 2^62, in whole numbers: fp64
// instructions run at 1/64 of the fp32 rate, and every thread of a row takes this step.
__device__ __forceinline__ uint64_t part_of(float f, uint64_t x, bool up) {
  const uint32_t bits = __float_as_uint(f);
  if (bits < 0x00800000u) return up && bits != 0 && x != 0 ? 1 : 0;
  const uint64_t digits = (bits & 0x7fffffu) | 0x800000u;
  const int shift = 150 - (int)(bits >> 23);  // f = digits 2^-shift; at least 23
  const uint64_t lo = x * digits, hi = __umul64hi(x, digits);
  if (shift > 87) return up && x != 0 ? 1 : 0;
  uint64_t y, left;
  if (shift < 64) {
    y = (hi << (64 - shift)) | (lo >> shift);
    left = lo << (64 - shift);
  } else {
    y = hi >> (shift - 64);
    left = lo | (shift > 64 ? hi << (128 - shift) : 0);
  }
  return y + (up && left != 0 ? 1 : 0);
}
// ceil(share x) of a mass x, at least 1.
__device__ __forceinline__ uint64_t share_of(float share, uint64_t x) {
  const uint64_t n = part_of(share, x, true);
  return n < 1 ? 1 : n;
}
// floor(u x), below x.
__device__ __forceinline__ uint64_t point_of(float u, uint64_t x) {
  const uint64_t t = part_of(u, x, false);
  return t < x ? t : x - 1;
}

template <typename T>
__device__ __forceinline__ T param(const T *each, T all, int64_t r) {
  return each != nullptr ? each[r] : all;
}

// Held within the finite values of type T: a kept entry that overflowed at a small
// temperature would be masked, or spoil its row.
template <typename T>
__device__ __forceinline__ float finite(float x) {
  constexpr float most = sizeof(T) == 2 ? 3.3895313892515355e38f : 3.402823466385288598e38f;
  return fminf(fmaxf(x, -most), most);
}

// ln of a kept sum of `all` units, at least one weight of 1.
__device__ __forceinline__ float ln_units(uint64_t all, float one) {
  // (all - one is exact: close to a weight of 1 the logarithm keeps its digits)
  const float over = (float)(all - (uint64_t)one) / one;
  return over < 1.0f ? log1pf(over) : logf((float)all / one);
}

// A row's sampling parameters, as the call gives them.
struct Request {
  float r, top_p, min_p, u;  // r: 1 / T
  int top_k;
  bool greedy;               // T is 0, or so little that 1 / T overflows
  bool by_k, by_p, by_a;     // which filters can leave anything out
  bool bad;                  // a value outside its range

  __device__ __forceinline__ Request(const SampleArgs &a, int64_t row) {
    // (-0 + 0 is +0: of -0 the reciprocal would be -inf, and the bits no share)
    const float T = __fadd_rn(param(a.temperature, a.temperature_all, row), 0.0f);
    top_p = __fadd_rn(param(a.top_p, a.top_p_all, row), 0.0f);
    top_k = param(a.top_k, a.top_k_all, row);
    min_p = __fadd_rn(param(a.min_p, a.min_p_all, row), 0.0f);
    u = a.u != nullptr ? __fadd_rn(a.u[row], 0.0f) : 0.0f;
    greedy = __frcp_rn(T) > 3.402823466e38f;
    r = greedy ? 1.0f : __fdiv_rn(1.0f, T);
    if (greedy) top_k = 1;
    by_k = top_k > 0 && top_k < a.V;
    by_p = !greedy && top_p < 1.0f;
    by_a = !greedy && min_p > 0.0f;
    bad = !(T >= 0.0f && T < INFINITY) || !(top_p >= 0.0f) || !(min_p >= 0.0f && min_p <= 1.0f) ||
          !(u >= 0.0f && u <= 1.0f);
  }
};

}  // namespace specv
