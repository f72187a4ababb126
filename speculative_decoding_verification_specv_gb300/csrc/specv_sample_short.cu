// specv_sample_short.cu -- sampling and filtering of short rows: a warp per row, which holds
// it in registers, 32 entries per lane.
//
// The same definition as for long rows, by the same exact sums.  A threshold is the largest
// value c for which the count (or the mass) of the entries z >= c reaches the target: a
// binary search over the order of the values, a count or a sum over the lane's entries and
// one across the warp in each step.  For a count it ends where the count is the target, as it
// is after some ten steps; top-k below 33 begins at the k-th largest of the lanes' maxima.
// What equals c is cut at an index.  The draw takes running sums over the row's vectors in
// order, 32 at a time.
// Where top-k leaves 64 entries or fewer they are compared one with another instead.
// Bound by instructions, some thousands for each row, at 16 warps per SM (128 registers):
// 4096 rows of 1000 fp32 entries (16 MB, 2.4 us) 21 us with no filter, 33 with top-k 50, 38
// with top-p 0.9 on top, 56 with top-p alone; a CTA of 256 threads per row took 71, 66, 72
// and 89.
#include "specv_internal.h"
#include "specv_rowstat.cuh"
#include "specv_sample.cuh"

namespace specv {

namespace {

constexpr int kNT = 128;
constexpr int kFew = 64;  // entries that top-k leaves and that are looked at one by one

// The order of a type's values as whole numbers, and back.
template <typename T>
struct Order;
template <>
struct Order<float> {
  __device__ __forceinline__ static uint32_t key(float z) { return value_key(z); }
  __device__ __forceinline__ static float value(uint32_t k) { return value_of(k); }
};
template <>
struct Order<uint16_t> {
  __device__ __forceinline__ static uint32_t key(float z) { return value_key(z) >> 16; }
  __device__ __forceinline__ static float value(uint32_t k) {
    return value_of(k & 0x8000u ? k << 16 : (k << 16) | 0xffffu);
  }
};

template <typename T>
struct ShortRow {
  static constexpr int VW = Elem<T>::kPerVec, kEach = kShortEntries / 32, kVecs = kEach / VW;
  uint4 v[kVecs];
  float w[kEach];  // weights of the entries in order, 0 of the others

  __device__ __forceinline__ float z(int i) const { return Elem<T>::get(v[i / VW], i % VW); }

  __device__ __forceinline__ int count(float c) const {
    int n = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) n += z(i) >= c ? 1 : 0;
    return __reduce_add_sync(~0u, n);
  }
  __device__ __forceinline__ uint64_t mass(float c, float scale) const {
    const Units units(scale);
    UnitSum sum = units.begin(kEach), a, b;
#pragma unroll
    for (int i = 0; i < kEach; i += 2) {
      units.split(z(i) >= c ? w[i] : 0.0f, z(i + 1) >= c ? w[i + 1] : 0.0f, a, b);
      Units::add(sum, a, b);
    }
    return units.warp_total(sum);
  }
  // The index of the n-th entry (from 1) that equals c, in index order.
  __device__ __forceinline__ int nth_equal(const RowVectors<T> &row, float c, int n) const {
    const int lane = threadIdx.x & 31;
    int index = 0x7fffffff;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      int own = 0;
#pragma unroll
      for (int e = 0; e < VW; ++e) own += z(j * VW + e) == c ? 1 : 0;
      int upto = own;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(~0u, upto, off);
        if (lane >= off) upto += x;
      }
      const int all = __shfl_sync(~0u, upto, 31);
      int left = n - (upto - own);
      if (left >= 1 && left <= own) {
#pragma unroll
        for (int e = 0; e < VW; ++e)
          if (z(j * VW + e) == c && --left == 0) index = (int)row.index(j * 32 + lane, e);
      }
      n -= all;
    }
    return (int)__reduce_min_sync(~0u, (unsigned)index);
  }
};

// The largest key in [lo, hi] whose value's `reached` is at least target, where that of lo
// is; ends early where `reached` is the target and `exact`.
template <typename T, typename F>
__device__ __forceinline__ uint32_t search(uint32_t lo, uint32_t hi, uint64_t target, bool exact,
                                           F reached) {
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo) / 2 + ((hi - lo) & 1);
    const uint64_t x = reached(Order<T>::value(mid));
    if (x >= target) lo = mid;
    else hi = mid - 1;
    if (exact && x == target) break;
  }
  return lo;
}

template <typename T, typename TO>
__global__ void __launch_bounds__(kNT, 4) sample_short_kernel(const __grid_constant__ SampleArgs a) {
  using Row = ShortRow<T>;
  constexpr int VW = Row::VW, kEach = Row::kEach, kVecs = Row::kVecs;
  const int lane = threadIdx.x & 31;
  __shared__ uint64_t keys[kNT / 32][kFew], weights[kNT / 32][kFew];
  uint64_t *const key = keys[threadIdx.x >> 5], *const weight = weights[threadIdx.x >> 5];
  const int64_t r = (int64_t)blockIdx.x * (kNT / 32) + (threadIdx.x >> 5);
  if (r >= a.R) return;
  const T *first = static_cast<const T *>(a.logits) + row_offset(r, a.N, a.stride_b, a.stride_n);
  const RowVectors<T> row(first, a.V, Span{a.logits, a.logits_end});
  Row x;
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    constexpr uint32_t none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
    x.v[j] = make_uint4(none, none, none, none);
    if (j * 32 + lane < row.count) x.v[j] = load_vec<T>(row, j * 32 + lane);
  }
  const Request q(a, r);
  float own = -INFINITY;
#pragma unroll
  for (int j = 0; j < kVecs; ++j) own = max_nan(own, vector_max_nan<T>(x.v[j]));
  float m = own;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = max_nan(m, __shfl_xor_sync(~0u, m, off));
  const bool bad = q.bad || !(m < INFINITY);
  RowParams p;
  p.m = m;
  p.r = q.r;
  p.min_p = q.greedy ? 0.0f : q.min_p;
  p.scale = a.scale;
  p.tau = -INFINITY;
  p.tie = -1;
  const bool none = bad || m == -INFINITY;
  int few = -1;  // entries in key and weight, if they hold all that are kept
  if (!none) {
    constexpr float least = sizeof(T) == 2 ? -3.3895313892515355e38f : -3.402823466e38f;
    const uint32_t top = Order<T>::key(m), lowest = Order<T>::key(least);
    if (q.by_k && x.count(least) > q.top_k) {
      uint32_t lo = lowest;
      if (q.top_k <= 32) {
        const uint64_t sorted = warp_sort(own > -INFINITY ? order_key(own, lane) : 0);
        const uint64_t kth = __shfl_sync(~0u, (unsigned long long)sorted, q.top_k - 1);
        if (kth != 0) lo = Order<T>::key(key_value(kth));
      }
      const uint32_t c = search<T>(lo, top, (uint64_t)q.top_k, true,
                                   [&](float at) -> uint64_t { return (uint64_t)x.count(at); });
      p.tau = Order<T>::value(c);
      p.tie = 0x7fffffff;
      const int reached = x.count(p.tau);
      if (reached > q.top_k) {
        int equal = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) equal += x.z(i) == p.tau ? 1 : 0;
        equal = __reduce_add_sync(~0u, equal);
        p.tie = x.nth_equal(row, p.tau, q.top_k - (reached - equal));
      }
    }
    if (q.by_k && q.top_k <= kFew && p.cut()) {
      // the few entries that are left, each against all: what weighs before it in order
      few = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const float z = x.z(i);
        const int at = (int)row.index((i / VW) * 32 + lane, i % VW);
        const bool in = p.in_order(z, at);
        const uint32_t where = __ballot_sync(~0u, in);
        const int slot = few + __popc(where & ((1u << lane) - 1));
        if (in && slot < kFew) {
          key[slot] = order_key(z, (uint32_t)at);
          weight[slot] = p.units(p.weight(z));
        }
        few += __popc(where);
      }
      few = min(few, kFew);
      __syncwarp();
      if (q.by_p) {
        uint64_t before[2] = {0, 0}, all = 0;
        const uint64_t own[2] = {lane < few ? key[lane] : 0, lane + 32 < few ? key[lane + 32] : 0};
        for (int i = 0; i < few; ++i) {
          const uint64_t k = key[i], y = weight[i];
          all += y;
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (k > own[j]) before[j] += y;
        }
        const uint64_t target = share_of(q.top_p, all);
        uint64_t last = ~0ull;  // the last one kept
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (lane + 32 * j < few && before[j] < target) last = own[j] < last ? own[j] : last;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
          const uint64_t y = shfl_xor_u64(last, off);
          last = y < last ? y : last;
        }
        p.tau = key_value(last);
        p.tie = (int)key_index(last);
      }
    } else if (q.by_p) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const float z = x.z(i);
        const int at = (int)row.index((i / VW) * 32 + lane, i % VW);
        x.w[i] = p.in_order(z, at) ? p.weight(z) : 0.0f;
      }
      const uint64_t target = share_of(q.top_p, x.mass(-INFINITY, p.scale));
      const uint32_t c = search<T>(lowest, top, target, false,
                                   [&](float at) { return x.mass(at, p.scale); });
      const float tau = Order<T>::value(c);
      const uint64_t reached = x.mass(tau, p.scale), each = p.units(p.weight(tau));
      // the entries at tau that the target does not want, of those in order
      int equal = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int at = (int)row.index((i / VW) * 32 + lane, i % VW);
        equal += x.z(i) == tau && p.in_order(x.z(i), at) ? 1 : 0;
      }
      equal = __reduce_add_sync(~0u, equal);
      const uint64_t before = reached - (uint64_t)equal * each;
      const int64_t wanted = each != 0 && target > before ? (int64_t)((target - before + each - 1) / each) : equal;
      if (wanted < equal) {
        p.tie = x.nth_equal(row, tau, (int)wanted);
      } else if (tau > p.tau) {
        p.tie = 0x7fffffff;
      }
      p.tau = tau;
    }
  }
  TO *out = a.filtered != nullptr ? static_cast<TO *>(a.filtered) + r * (int64_t)a.V : nullptr;
  if (a.u != nullptr) {
    if (none) {
      if (lane == 0) {
        a.tokens[r] = -1;
        a.logprob[r] = bad ? quiet_nan() : 0.0f;
        a.lse[r] = bad ? quiet_nan() : -INFINITY;
      }
    } else if (few >= 0) {
      // the kept ones, each against all: what weighs before it by index
      uint64_t below[2] = {0, 0}, all = 0;
      const uint64_t own[2] = {lane < few ? key[lane] : 0, lane + 32 < few ? key[lane + 32] : 0};
      const uint64_t edge = order_key(p.tau, (uint32_t)p.tie);
      auto kept = [&](uint64_t k) { return k >= edge && p.weight(key_value(k)) >= p.min_p; };
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (lane + 32 * j < few && !kept(own[j])) weight[lane + 32 * j] = 0;
      __syncwarp();
      for (int i = 0; i < few; ++i) {
        const uint64_t k = key[i], y = weight[i];
        all += y;
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (key_index(k) < key_index(own[j])) below[j] += y;
      }
      uint64_t t = point_of(q.u, all);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (lane + 32 * j < few && t >= below[j] && t < below[j] + weight[lane + 32 * j]) {
          const float ln = ln_units(all, p.scale);
          a.tokens[r] = (int)key_index(own[j]);
          a.logprob[r] = __fmul_rn(__fsub_rn(key_value(own[j]), m), p.r) - ln;
          a.lse[r] = q.greedy ? 0.0f : finite<float>(__fmaf_rn(m, p.r, ln));
        }
    } else {
      uint64_t part[kVecs], all = 0;
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        part[j] = 0;
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          const float z = x.z(j * VW + e);
          const bool in = p.in_order(z, (int)row.index(j * 32 + lane, e));
          const float w = in ? p.weight(z) : 0.0f;
          x.w[j * VW + e] = w >= p.min_p ? w : 0.0f;
          part[j] += p.units(x.w[j * VW + e]);
        }
        all += part[j];
      }
      all = warp_sum_u64(all);
      uint64_t t = point_of(q.u, all);
      int token = -1;
      float zx = 0.0f;
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        uint64_t upto = part[j];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const uint64_t y = __shfl_up_sync(~0u, (unsigned long long)upto, off);
          if (lane >= off) upto += y;
        }
        const uint64_t whole = __shfl_sync(~0u, (unsigned long long)upto, 31);
        uint64_t sum = upto - part[j];
        if (t >= sum && t < upto) {  // one lane of one j
#pragma unroll
          for (int e = 0; e < VW; ++e) {
            const uint64_t y = p.units(x.w[j * VW + e]);
            if (t >= sum && t < sum + y) {
              token = (int)row.index(j * 32 + lane, e);
              zx = x.z(j * VW + e);
            }
            sum += y;
          }
        }
        t = t >= whole ? t - whole : ~0ull >> 1;  // (found: beyond every later sum)
      }
      if (token >= 0) {
        const float ln = ln_units(all, p.scale);
        a.tokens[r] = token;
        a.logprob[r] = __fmul_rn(__fsub_rn(zx, m), p.r) - ln;
        a.lse[r] = q.greedy ? 0.0f : finite<float>(__fmaf_rn(m, p.r, ln));
      }
    }
  }
  if (out == nullptr) return;
  const bool alike = sizeof(T) == sizeof(TO) &&
                     reinterpret_cast<uint64_t>(out) % 16 == reinterpret_cast<uint64_t>(row.row) % 16;
  auto value = [&](float z, int i) {
    if (none) return bad ? quiet_nan() : -INFINITY;
    const bool kept = p.in_order(z, i) && (p.min_p <= 0.0f || p.weight(z) >= p.min_p);
    return kept ? (q.greedy ? 0.0f : finite<TO>(__fmul_rn(z, p.r))) : -INFINITY;
  };
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    const int k = j * 32 + lane;
    if (k >= row.count) continue;
    if (sizeof(T) == sizeof(TO) && alike && k >= row.full_lo && k < row.full_hi) {
      const int i = (int)row.index(k, 0);
      uint4 y;
#pragma unroll
      for (int e = 0; e < VW / 2; ++e)
        put_pair<T>(y, e, value(x.z(j * VW + 2 * e), i + 2 * e),
                    value(x.z(j * VW + 2 * e + 1), i + 2 * e + 1));
      __stcs(reinterpret_cast<uint4 *>(out + i), y);
    } else {
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        const int64_t i = row.index(k, e);
        if (i >= 0 && i < row.V) out[i] = narrow<TO>(value(x.z(j * VW + e), (int)i));
      }
    }
  }
}

template <typename T, typename TO>
cudaError_t launch(const SampleArgs &a, cudaStream_t stream) {
  const unsigned ctas = (unsigned)((a.R + kNT / 32 - 1) / (kNT / 32));
  sample_short_kernel<T, TO><<<ctas, kNT, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t sample_short_launch(const SampleArgs &a, int dtype_bf16, int out_bf16,
                                cudaStream_t stream) {
  if (dtype_bf16)
    return out_bf16 ? launch<uint16_t, uint16_t>(a, stream) : launch<uint16_t, float>(a, stream);
  return launch<float, float>(a, stream);
}

}  // namespace specv
