// specv_clip.cu -- the 2-norm over many gradients, and clipping to a largest
// norm.
//
//   norm = sqrt(sum_tensors sum_i x_i^2),  c = min(1, max_norm / (norm + eps)),
//   out_i = round(c x_i)
// Two launches.  The first sums squares: chunk k of kChunkBytes (whole tensors
// are cut into chunks, tensor by tensor) goes to CTA k mod grid, each thread
// adds at most kChunkBytes / (4 NT) squares in fp32 and then the chunk to a
// double.  The CTAs' sums are written out; every CTA of the second launch adds
// them in the same order, so all hold the same norm, and scales its chunks.
#include "specv_internal.h"
#include "specv_rowstat.cuh"

namespace specv {

namespace {

constexpr int kNT = 256;
constexpr int kChunk = 8192;  // elements

__device__ __forceinline__ int find_tensor(const ClipArgs &a, int64_t chunk) {
  int lo = 0, hi = a.n - 1;  // the last tensor that begins at or before the chunk
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.first[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ float load_any(const ClipArgs &a, int t, int64_t i) {
  return a.bf16[t] ? bf16_bits_to_float(static_cast<const uint16_t *>(a.in[t])[i])
                   : static_cast<const float *>(a.in[t])[i];
}

__device__ __forceinline__ double block_sum_d(double *red, double x) {
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(~0u, x, off);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0.0;
  for (int w = 0; w < kNT / 32; ++w) x += red[w];
  return x;
}

__global__ void __launch_bounds__(kNT) clip_norm_kernel(const __grid_constant__ ClipArgs a) {
  __shared__ double red[kNT / 32];
  double sum = 0.0;
  for (int64_t k = blockIdx.x; k < a.chunks; k += gridDim.x) {
    const int t = find_tensor(a, k);
    const int64_t lo = (k - a.first[t]) * kChunk, hi = min(a.count[t], lo + kChunk);
    float s = 0.0f;
    for (int64_t i = lo + threadIdx.x; i < hi; i += kNT) {
      const float x = load_any(a, t, i);
      s = __fmaf_rn(x, x, s);
    }
    sum += (double)s;
  }
  sum = block_sum_d(red, sum);
  if (threadIdx.x == 0) a.partial[a.partial_at + blockIdx.x] = sum;
}

__global__ void __launch_bounds__(kNT) clip_scale_kernel(const __grid_constant__ ClipArgs a) {
  __shared__ double red[kNT / 32];
  double sum = 0.0;
  for (int i = threadIdx.x; i < a.partials; i += kNT) sum += a.partial[i];
  const float norm = (float)sqrt(block_sum_d(red, sum));
  if (a.out_norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *a.out_norm = norm;
  // a norm that is not finite gives no factor: the values are left as they are
  const float c = norm < INFINITY ? fminf(1.0f, a.max_norm / (norm + kClipEps)) : 1.0f;
  for (int64_t k = blockIdx.x; k < a.chunks; k += gridDim.x) {
    const int t = find_tensor(a, k);
    if (c == 1.0f && a.out[t] == a.in[t]) continue;
    const int64_t lo = (k - a.first[t]) * kChunk, hi = min(a.count[t], lo + kChunk);
    for (int64_t i = lo + threadIdx.x; i < hi; i += kNT) {
      const float y = c * load_any(a, t, i);
      if (a.bf16[t]) {
        uint16_t h;
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(y));
        static_cast<uint16_t *>(a.out[t])[i] = h;
      } else {
        static_cast<float *>(a.out[t])[i] = y;
      }
    }
  }
}

}  // namespace

int64_t clip_chunks(const void *, int64_t count, int) { return (count + kChunk - 1) / kChunk; }

cudaError_t clip_norm_launch(const ClipArgs &a, int grid, cudaStream_t stream) {
  clip_norm_kernel<<<grid, kNT, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t clip_scale_launch(const ClipArgs &a, int grid, cudaStream_t stream) {
  clip_scale_kernel<<<grid, kNT, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace specv
