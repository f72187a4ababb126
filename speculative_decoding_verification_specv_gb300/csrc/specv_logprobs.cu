// specv_logprobs.cu -- log probabilities of given tokens, with the entropy of
// their rows and the most likely alternatives; and the gradient.
//
// For a row z of V logits and its token x:
//   m = max_v z_v,  S = sum_v e^{z_v - m},  T = sum_v e^{z_v - m} (z_v - m)
//   log p_x = (z_x - m) - ln S            entropy = ln S - T / S
// and the top_n largest entries in the order (value falling, index rising),
// each with its own log probability.
#include "specv_internal.h"
#include "specv_rowstat.cuh"

namespace specv {

namespace {

constexpr int kNT = 256;

// Values as whole numbers in the same order (-0 and +0 alike), over the
// complement of the index: the larger key is the larger value, and among equal
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

template <typename T>
__global__ void __launch_bounds__(kNT) logprobs_kernel(LogprobArgs a) {
  __shared__ float red[kNT / 32][3];
  __shared__ uint64_t best[kNT / 32];
  const int64_t r = blockIdx.x;
  const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int V = a.V;
  const T *row = static_cast<const T *>(a.logits) + row_offset(r, a.N, a.stride_b, a.stride_n);
  const int32_t x = a.tokens[r];
  if (x < 0 || x >= V) {  // no token (-1): the row is not read; an invalid one: NaN
    const float fill = x == -1 ? 0.0f : quiet_nan();
    if (tid == 0) {
      a.logprob[r] = fill;
      a.entropy[r] = fill;
      a.stats[r] = make_float2(fill, fill);
    }
    for (int i = tid; i < a.top_n; i += kNT) {
      a.top_tokens[r * a.top_n + i] = -1;
      a.top_logprobs[r * a.top_n + i] = x == -1 ? -INFINITY : quiet_nan();
    }
    return;
  }
  float m = -INFINITY, s = 0.0f, t = 0.0f;
  for (int64_t v = tid; v < V; v += kNT) {
    const float z = Elem<T>::load(row + v);
    if (z > m) {
      const float d = fmaxf(m - z, kFarBelow), f = ex2(d * kLog2e);
      t = f * (t + s * d);
      s *= f;
      m = z;
    }
    const float d = z - (m == -INFINITY ? 0.0f : m), e = ex2(d * kLog2e);
    s += e;
    t = __fmaf_rn(e, fmaxf(d, kFarBelow), t);
  }
  // merge: the maximum first, then every partial recentred on it
  float M = m;
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, off));
  if (lane == 0) red[warp][0] = M;
  __syncthreads();
  for (int w = 0; w < kNT / 32; ++w) M = fmaxf(M, red[w][0]);
  if (s == 0.0f) {
    t = 0.0f;
  } else {
    const float d = fmaxf(m - M, kFarBelow), f = ex2(d * kLog2e);
    t = f * (t + s * d);
    s *= f;
  }
  for (int off = 16; off > 0; off >>= 1) {
    s += __shfl_xor_sync(~0u, s, off);
    t += __shfl_xor_sync(~0u, t, off);
  }
  if (lane == 0) {
    red[warp][1] = s;
    red[warp][2] = t;
  }
  __syncthreads();
  float S = 0.0f, Tw = 0.0f;
  for (int w = 0; w < kNT / 32; ++w) {
    S += red[w][1];
    Tw += red[w][2];
  }
  const bool bad = !(S < INFINITY);  // a NaN or +inf entry
  const bool none = !bad && M == -INFINITY;
  const float ln = logf(S);
  if (tid == 0) {
    const float z = Elem<T>::load(row + x);
    a.logprob[r] = bad ? quiet_nan() : none ? -INFINITY : (z - M) - ln;
    a.entropy[r] = bad ? quiet_nan() : none ? 0.0f : fmaxf(ln - Tw / S, 0.0f);
    a.stats[r] = bad ? make_float2(quiet_nan(), quiet_nan())
                     : make_float2(M, none ? 0.0f : ln);
  }
  // the alternatives: the largest key below the last one found
  uint64_t last = ~0ull;
  for (int i = 0; i < a.top_n; ++i) {
    uint64_t k = 0;
    for (int64_t v = tid; v < V; v += kNT) {
      const float z = Elem<T>::load(row + v);
      const uint64_t c = z > -INFINITY ? order_key(z, (uint32_t)v) : 0;
      if (c < last && c > k) k = c;
    }
    for (int off = 16; off > 0; off >>= 1) {
      const uint64_t o = shfl_xor_u64(k, off);
      k = o > k ? o : k;
    }
    __syncthreads();
    if (lane == 0) best[warp] = k;
    __syncthreads();
    for (int w = 0; w < kNT / 32; ++w) k = best[w] > k ? best[w] : k;
    if (tid == 0) {
      a.top_tokens[r * a.top_n + i] = bad || k == 0 ? -1 : (int32_t)key_index(k);
      a.top_logprobs[r * a.top_n + i] =
          bad ? quiet_nan() : k == 0 ? -INFINITY : (key_value(k) - M) - ln;
    }
    last = k;
  }
}

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

// dz_v = g (1[v = x] - p_v) - h p_v (ln p_v + H): one CTA per row.
template <typename T>
__global__ void __launch_bounds__(kNT) logprobs_grad_kernel(LogprobGradArgs a) {
  const int64_t r = blockIdx.x;
  const int V = a.V;
  const T *row = static_cast<const T *>(a.logits) + row_offset(r, a.N, a.stride_b, a.stride_n);
  T *out = static_cast<T *>(a.out) + r * (int64_t)V;
  const int32_t x = a.tokens[r];
  const float2 st = a.stats[r];
  const float H = a.entropy[r], g = a.grad_logprob[r];
  const float h = a.grad_entropy != nullptr ? a.grad_entropy[r] : 0.0f;
  const bool zero = x == -1 || st.x == -INFINITY;
  const bool bad = x < -1 || x >= V;
  for (int64_t v = threadIdx.x; v < V; v += kNT) {
    float d = 0.0f;
    if (bad) {
      d = quiet_nan();
    } else if (!zero) {
      const float lp = (Elem<T>::load(row + v) - st.x) - st.y;
      const float p = ex2(lp * kLog2e);
      d = (v == x ? g : 0.0f) - p * (g + h * (fmaxf(lp, kFarBelow) + H));
    }
    out[v] = narrow<T>(d);
  }
}

}  // namespace

cudaError_t logprobs_launch(const LogprobArgs &a, int dtype_bf16, cudaStream_t stream) {
  if (dtype_bf16)
    logprobs_kernel<uint16_t><<<(unsigned)a.R, kNT, 0, stream>>>(a);
  else
    logprobs_kernel<float><<<(unsigned)a.R, kNT, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t logprobs_grad_launch(const LogprobGradArgs &a, int dtype_bf16, cudaStream_t stream) {
  if (dtype_bf16)
    logprobs_grad_kernel<uint16_t><<<(unsigned)a.R, kNT, 0, stream>>>(a);
  else
    logprobs_grad_kernel<float><<<(unsigned)a.R, kNT, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace specv
