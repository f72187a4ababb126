// specv_clip.cu -- the 2-norm over many gradients, and clipping to a largest
// norm.
//
//   norm = sqrt(sum_tensors sum_i x_i^2),  c = min(1, max_norm / (norm + eps)),
//   out_i = round(c x_i)
// Two launches.  Each gradient is cut into chunks of kChunkBytes of the aligned
// memory that holds it (the first may begin before the gradient, off a 16-byte
// boundary, the last end after it; what is not the gradient's is not read), and
// the chunks of all gradients are dealt to the CTAs in turn.  The first launch sums
// squares, in fp32 within a thread's share of a chunk (two interleaved sums of up to 16
// terms) and without further rounding beyond; every CTA writes its sum.  Every CTA of
// the second launch adds those sums in the same order, so that all hold the same norm
// (no atomics, one result), and scales the chunks that the CTA of its number has
// summed, the last ones first: those the first launch has left in L2, which the
// results, stored as streaming data, do not push out (2.2 GB: 1040 us a call; with
// the chunks dealt from the end 1071, with ordinary stores 1120).  The second launch
// begins while the first drains (programmatic dependent launch).  The gradients of a
// call travel in the launches' parameters: nothing is copied to the device first.
// Bound by HBM for large sets (two reads and a write: 976 us for the 2.2 GB), by the
// two launches for small ones (16 MB: 6.0 to 6.4 us).
#include "specv_internal.h"
#include "specv_rowstat.cuh"

namespace specv {

namespace {

constexpr int kNT = 256;
constexpr int kVecs = 4;                              // 16-byte vectors per thread and chunk
constexpr int kChunkBytes = kNT * kVecs * 16;

// The gradient that chunk k belongs to.
template <typename Args>
__device__ __forceinline__ int find_tensor(const Args &a, int k) {
  int lo = 0, hi = a.n - 1;  // the last one that begins at or before the chunk
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.first[mid] <= k) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ uint4 load16(const char *p) {
  uint4 x;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "l"(p));
  return x;
}

// A chunk: its vectors lie at base + 16 (tid + u kNT); entry e of that vector is entry
// at + (tid + u kNT) VW + e of the gradient, which has `count` entries.
struct Chunk {
  const char *base;
  int64_t at, count;
  bool whole;  // every vector lies within the gradient
};
template <typename Args>
__device__ __forceinline__ Chunk chunk_of(const Args &a, int t, int k, int elem) {
  const uint64_t p = reinterpret_cast<uint64_t>(a.in[t]);
  const int mis = (int)(p % 16) / elem, per_vec = 16 / elem;
  Chunk c;
  const int64_t vec = (int64_t)(k - a.first[t]) * (kNT * kVecs);
  c.base = reinterpret_cast<const char *>(p - p % 16) + vec * 16;
  c.at = vec * per_vec - mis;
  c.count = a.count[t];
  c.whole = c.at >= 0 && c.at + (int64_t)kNT * kVecs * per_vec <= c.count;
  return c;
}

// Sum of the squares of a vector's entries, in two interleaved sums.
template <typename T>
__device__ __forceinline__ uint64_t add_squares(uint64_t s, const uint4 &v) {
#pragma unroll
  for (int i = 0; i < Elem<T>::kPerVec / 2; ++i) {
    const uint64_t x = pair_of<T>(v, i);
    s = fma2(x, x, s);
  }
  return s;
}

// A thread's vectors of a chunk; what is not the gradient's is 0.
template <typename T>
__device__ __forceinline__ void load_chunk(const Chunk &c, uint4 (&v)[kVecs]) {
  constexpr int VW = Elem<T>::kPerVec;
  const char *p = c.base + (int)threadIdx.x * 16;
  if (c.whole) {
#pragma unroll
    for (int u = 0; u < kVecs; ++u) v[u] = load16(p + u * (kNT * 16));
    return;
  }
#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
    const int64_t first = c.at + ((int64_t)threadIdx.x + u * kNT) * VW;
    v[u] = make_uint4(0, 0, 0, 0);
    if (first >= 0 && first + VW <= c.count) {
      v[u] = load16(p + u * (kNT * 16));
    } else if (first < c.count && first + VW > 0) {
      const T *q = reinterpret_cast<const T *>(p + u * (kNT * 16));
#pragma unroll
      for (int e = 0; e < VW; ++e)
        if (first + e >= 0 && first + e < c.count) {
          if constexpr (sizeof(T) == 2)
            Elem<T>::put_bits(v[u], e, q[e]);
          else
            Elem<T>::put_bits(v[u], e, __float_as_uint(q[e]));
        }
    }
  }
}

template <typename T>
__device__ __forceinline__ float chunk_squares(const Chunk &c) {
  uint4 v[kVecs];
  load_chunk<T>(c, v);
  uint64_t s = 0;
#pragma unroll
  for (int u = 0; u < kVecs; ++u) s = add_squares<T>(s, v[u]);
  float s0, s1;
  unpack2(s, s0, s1);
  return s0 + s1;
}

// A sum as a pair of fp32, lo holding what hi rounds away (about 48 bits together).
// fp64 additions run at 1/64 of the fp32 rate here: with them the CTAs' reductions
// took longer than the reading (a draft head of 16 MB: 13 us a call).
struct Sum {
  float hi = 0.0f, lo = 0.0f;
};
__device__ __forceinline__ Sum operator+(const Sum &a, const Sum &b) {
  Sum s;
  s.hi = __fadd_rn(a.hi, b.hi);
  const float part = __fsub_rn(s.hi, a.hi);
  const float off = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s.hi, part)), __fsub_rn(b.hi, part));
  // (an overflow leaves hi infinite; what it rounds away is then of no account)
  s.lo = s.hi < INFINITY ? __fadd_rn(off, __fadd_rn(a.lo, b.lo)) : 0.0f;
  return s;
}
// The CTA's sum in a fixed order, in every thread.
__device__ __forceinline__ Sum block_sum(Sum *red, Sum x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    Sum y;
    y.hi = __shfl_xor_sync(~0u, x.hi, off);
    y.lo = __shfl_xor_sync(~0u, x.lo, off);
    // (lanes take their pair in the same order: the sum is the same in both)
    x = (threadIdx.x & off) == 0 ? x + y : y + x;
  }
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  x = red[0];
#pragma unroll
  for (int w = 1; w < kNT / 32; ++w) x = x + red[w];
  return x;
}

template <int CAP>
__global__ void __launch_bounds__(kNT, kClipCtasPerSm)
    clip_norm_kernel(const __grid_constant__ ClipArgs<CAP> a) {
  __shared__ Sum red[kNT / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Sum sum;
  for (int64_t k = blockIdx.x; k < a.chunks; k += gridDim.x) {
    const int t = find_tensor(a, (int)k);
    Sum x;
    x.hi = a.bf16[t] ? chunk_squares<uint16_t>(chunk_of(a, t, (int)k, 2))
                     : chunk_squares<float>(chunk_of(a, t, (int)k, 4));
    sum = sum + x;
  }
  sum = block_sum(red, sum);
  if (threadIdx.x == 0) a.partial[a.partial_at + blockIdx.x] = make_float2(sum.hi, sum.lo);
}

// A vector's entries times c, rounded once.
template <typename T>
__device__ __forceinline__ uint4 scaled(const uint4 &v, uint64_t c) {
  uint4 y;
#pragma unroll
  for (int i = 0; i < Elem<T>::kPerVec / 2; ++i) {
    float a, b;
    unpack2(mul2(pair_of<T>(v, i), c), a, b);
    put_pair<T>(y, i, a, b);
  }
  return y;
}

template <typename T>
__device__ __forceinline__ void scale_chunk(const void *from, void *to, const Chunk &c,
                                            float factor) {
  constexpr int VW = Elem<T>::kPerVec;
  T *out = static_cast<T *>(to);
  const uint64_t f = pack2(factor, factor);
  // vectors where the output lies as the input against the 16-byte boundaries
  const bool alike = (reinterpret_cast<uint64_t>(from) - reinterpret_cast<uint64_t>(out)) % 16 == 0;
  uint4 v[kVecs];
  load_chunk<T>(c, v);
#pragma unroll
  for (int u = 0; u < kVecs; ++u) v[u] = scaled<T>(v[u], f);
  T *q = out + c.at + (int)threadIdx.x * VW;
  if (alike && c.whole) {
#pragma unroll
    for (int u = 0; u < kVecs; ++u) __stcs(reinterpret_cast<uint4 *>(q + u * (kNT * VW)), v[u]);
    return;
  }
#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
    const int64_t first = c.at + ((int64_t)threadIdx.x + u * kNT) * VW;
    if (alike && first >= 0 && first + VW <= c.count) {
      *reinterpret_cast<uint4 *>(q + u * (kNT * VW)) = v[u];
    } else {
#pragma unroll
      for (int e = 0; e < VW; ++e)
        if (first + e >= 0 && first + e < c.count) q[u * (kNT * VW) + e] = narrow<T>(Elem<T>::get(v[u], e));
    }
  }
}

template <int CAP>
__global__ void __launch_bounds__(kNT, kClipCtasPerSm)
    clip_scale_kernel(const __grid_constant__ ClipArgs<CAP> a) {
  __shared__ Sum red[kNT / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Sum sum;
  for (int i = threadIdx.x; i < a.partials; i += kNT) {
    Sum x;
    x.hi = a.partial[i].x;
    x.lo = a.partial[i].y;
    sum = sum + x;
  }
  sum = block_sum(red, sum);
  const float norm = sqrtf(__fadd_rn(sum.hi, sum.lo));
  if (a.out_norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *a.out_norm = norm;
  // a norm that is not finite gives no factor: the values are left as they are
  const float c = norm < INFINITY ? fminf(1.0f, a.max_norm / (norm + kClipEps)) : 1.0f;
  if (c == 1.0f && a.in_place) return;
  // the chunks that this CTA's number has summed, the last one first
  const int64_t mine = (a.chunks - 1 - blockIdx.x) / gridDim.x;
  for (int64_t j = blockIdx.x + mine * gridDim.x; j >= 0; j -= gridDim.x) {
    const int k = (int)j, t = find_tensor(a, k);
    if (c == 1.0f && a.out[t] == a.in[t]) continue;
    if (a.bf16[t])
      scale_chunk<uint16_t>(a.in[t], a.out[t], chunk_of(a, t, k, 2), c);
    else
      scale_chunk<float>(a.in[t], a.out[t], chunk_of(a, t, k, 4), c);
  }
}

}  // namespace

int64_t clip_chunks(const void *in, int64_t count, int bf16) {
  const int elem = bf16 ? 2 : 4;
  const int64_t mis = (int64_t)(reinterpret_cast<uint64_t>(in) % 16) / elem;
  return (mis + count + kChunkBytes / elem - 1) / (kChunkBytes / elem);
}

template <int CAP>
cudaError_t clip_norm_launch(const ClipArgs<CAP> &a, int grid, cudaStream_t stream) {
  clip_norm_kernel<CAP><<<grid, kNT, 0, stream>>>(a);
  return cudaGetLastError();
}

template <int CAP>
cudaError_t clip_scale_launch(const ClipArgs<CAP> &a, int grid, bool after_norm,
                              cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(kNT, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = after_norm ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, clip_scale_kernel<CAP>, a);
}

template cudaError_t clip_norm_launch(const ClipArgs<kClipFew> &, int, cudaStream_t);
template cudaError_t clip_norm_launch(const ClipArgs<kClipMany> &, int, cudaStream_t);
template cudaError_t clip_scale_launch(const ClipArgs<kClipFew> &, int, bool, cudaStream_t);
template cudaError_t clip_scale_launch(const ClipArgs<kClipMany> &, int, bool, cudaStream_t);

}  // namespace specv
