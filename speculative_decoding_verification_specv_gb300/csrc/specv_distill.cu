// specv_distill.cu -- the divergence of the draft's rows from the target's, and
// its gradient with respect to the draft logits.
//
// With p = softmax(z_t), q = softmax(z_q) and a weight w per row pair:
//   forward  L = w sum_v p_v (ln p_v - ln q_v)   dL/dz_q = w (q - p)
//   reverse  L = w sum_v q_v (ln q_v - ln p_v)   dL/dz_q = w q (ln q - ln p - L/w)
// Pass 1 takes (m, S) of both rows and the sum
//   T = sum_v e^{a_v} (a_v - c_v)
// of the leading row's a = z - m against the other's c, so that
//   L / w = T / S_a - ln S_a + ln S_c;
// pass 2 writes the gradient.
#include "specv_internal.h"
#include "specv_rowstat.cuh"

namespace specv {

namespace {

constexpr int kNT = 256;

template <typename T>
__device__ __forceinline__ float load_plain(const T *p) {
  if constexpr (sizeof(T) == 4)
    return *reinterpret_cast<const float *>(p);
  else
    return bf16_bits_to_float(*p);
}

__device__ __forceinline__ float block_max(float *red, float x) {
  for (int off = 16; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, off));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  for (int w = 0; w < kNT / 32; ++w) x = fmaxf(x, red[w]);
  return x;
}
__device__ __forceinline__ float block_add(float *red, float x) {
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(~0u, x, off);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0.0f;
  for (int w = 0; w < kNT / 32; ++w) x += red[w];
  return x;
}

template <typename T, bool REVERSE>
__global__ void __launch_bounds__(kNT) distill_kernel(DistillArgs a) {
  __shared__ float red[kNT / 32];
  const int64_t r = blockIdx.x;
  const int tid = (int)threadIdx.x, V = a.V;
  const T *zt = static_cast<const T *>(a.target) + row_offset(r, a.K, a.target_stride_b, a.target_stride_k);
  const T *zq = static_cast<const T *>(a.draft) + row_offset(r, a.K, a.draft_stride_b, a.draft_stride_k);
  T *out = a.out_grad == nullptr ? nullptr : static_cast<T *>(a.out_grad) + r * (int64_t)V;
  const float w = a.weight == nullptr ? 1.0f : a.weight[r];
  float mt = -INFINITY, mq = -INFINITY;
  if (w != 0.0f)
    for (int64_t v = tid; v < V; v += kNT) {
      mt = fmaxf(mt, load_plain(zt + v));
      mq = fmaxf(mq, load_plain(zq + v));
    }
  mt = block_max(red, mt);
  mq = block_max(red, mq);
  bool zero = w == 0.0f;
  float st = 0.0f, sq = 0.0f, t = 0.0f;
  if (!zero) {
    const float ct = mt == -INFINITY ? 0.0f : mt, cq = mq == -INFINITY ? 0.0f : mq;
    for (int64_t v = tid; v < V; v += kNT) {
      const float dt = load_plain(zt + v) - ct, dq = load_plain(zq + v) - cq;
      const float et = ex2(dt * kLog2e), eq = ex2(dq * kLog2e);
      st += et;
      sq += eq;
      if (REVERSE) {
        if (eq > 0.0f) t = __fmaf_rn(eq, dq - dt, t);
      } else {
        if (et > 0.0f) t = __fmaf_rn(et, dt - dq, t);
      }
    }
    st = block_add(red, st);
    sq = block_add(red, sq);
    t = block_add(red, t);
  }
  const bool bad = !(st < INFINITY) || !(sq < INFINITY);
  zero = zero || (!bad && (mt == -INFINITY || mq == -INFINITY));
  const float lt = logf(st), lq = logf(sq);
  float kl = REVERSE ? t / sq - lq + lt : t / st - lt + lq;
  kl = bad ? quiet_nan() : kl < 0.0f ? 0.0f : kl;
  if (tid == 0) a.out_loss[r] = zero ? 0.0f : w * kl;
  if (out == nullptr) return;
  const float nt = -lt * kLog2e, nq = -lq * kLog2e;
  const float c = kl == INFINITY ? quiet_nan() : lt - lq - kl;
  for (int64_t v = tid; v < V; v += kNT) {
    float g = 0.0f;
    if (!zero) {
      const float dt = load_plain(zt + v) - mt, dq = load_plain(zq + v) - mq;
      const float q = ex2(__fmaf_rn(dq, kLog2e, nq));
      if (REVERSE) {
        g = q > 0.0f ? w * q * (dq - dt + c) : 0.0f;
      } else {
        g = w * (q - ex2(__fmaf_rn(dt, kLog2e, nt)));
      }
      if (bad) g = quiet_nan();
    }
    out[v] = narrow<T>(g);
  }
}

template <typename T>
cudaError_t launch(const DistillArgs &a, int reverse, cudaStream_t stream) {
  const unsigned grid = (unsigned)(a.B * a.K);
  if (reverse)
    distill_kernel<T, true><<<grid, kNT, 0, stream>>>(a);
  else
    distill_kernel<T, false><<<grid, kNT, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t distill_launch(const DistillArgs &a, int dtype_bf16, int reverse, cudaStream_t stream) {
  return dtype_bf16 ? launch<uint16_t>(a, reverse, stream) : launch<float>(a, reverse, stream);
}

}  // namespace specv
