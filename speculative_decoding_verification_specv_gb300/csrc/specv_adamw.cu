// specv_adamw.cu -- an AdamW step over many tensors in one launch, with states in
// 32 bits or in 8.
//
//   g' = c g,  c = min(1, max_norm / (norm + eps_clip))        (c = 1 without a norm)
//   m' = b1 m + (1 - b1) g',   v' = b2 v + (1 - b2) g'^2
//   p' = p (1 - lr wd) - lr / (1 - b1^t) m' / (sqrt(v') / sqrt(1 - b2^t) + eps)
// in fp32, p' from the 32-bit master where a tensor has one, rounded once to the
// weight's type.  The products of the two averages are rounded one by one (no fused
// multiply-add), so that what is rounded to 8 bits afterwards does not depend on how a
// compiler contracts them.
//
// A warp takes blocks of 256 entries, eight per lane: entries 4 lane + 0..3 of either
// half, so that every type is read in whole coalesced vectors (16, 8 or 4 bytes a lane).
// An 8-bit state holds a block as one fp32 scale and 256 e4m3 values, for m and for
// sqrt(v); the root because its range is half that of v in binades: e4m3 reaches 2^-17.8
// below the block's largest root, 2^-35.6 below its largest v.  The block's largest
// entry maps to 448, so the scale follows the state itself.  Values are rounded up or
// down at random with the probability of the distance: an average that moves by one part
// in a thousand per step would never leave a value rounded to nearest 4 bits.  The bits
// are a hash of (seed, step, tensor, entry), 16 for each value: the entry's index added to a
// key of 32 bits, so tensors and steps take stretches of one sequence of 2^32 (stretches that
// overlap are shifted against the entries, and a value's rounding stays unbiased).  A root that
// is not 0 is never stored as 0: its weight would move by m / eps.
//
// 32-bit states are bound by HBM: 434 M weights, most bf16 with masters (12.1 GB), 1702 us, 7.1 TB/s,
// above the copy rate since more is read than written.  8-bit states by instructions, 58 for
// each entry (the hash, the codes and their decoding half of them): the same weights without
// masters (4.5 GB, 668 us at the copy rate) 908 us.
#include <type_traits>

#include "specv_internal.h"
#include "specv_rowstat.cuh"

namespace specv {

namespace {

constexpr int kNT = 256;
constexpr int kBlock = 256;                     // entries that share a scale
constexpr float kTiny = 7.888609052210118e-31f; // 2^-100

// The tensor that chunk k belongs to.
template <typename Args>
__device__ __forceinline__ int find_tensor(const Args &a, uint32_t k) {
  int lo = 0, hi = a.n - 1;  // the last one that begins at or before the chunk
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.first[mid] <= k) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// 32 bits from 32 bits: products with odd constants (the first bits of the fractions of
// sqrt 2, sqrt 3 and sqrt 7) and shifts.
constexpr uint32_t kMix0 = 0x6A09E667u, kMix1 = 0xBB67AE85u, kMix2 = 0xA54FF53Bu;
// After the first product, without the last step.
__host__ __device__ __forceinline__ uint32_t mix_rest(uint32_t x) {
  x ^= x >> 16;
  x *= kMix1;
  x ^= x >> 15;
  return x * kMix2;
}
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
  x = mix_rest(x * kMix0);
  return x ^ (x >> 16);
}

// b^t in fp64 for t >= 0.
__host__ __device__ __forceinline__ double power(double b, int64_t t) {
  double y = 1.0;
  for (; t > 0; t >>= 1, b *= b)
    if (t & 1) y *= b;
  return y;
}

// Entries 4 lane + 0..3 of both halves of a block that begins at p; `vec`: vectors may be
// used, `left`: entries from the block's start to the tensor's end.
template <typename T>
__device__ __forceinline__ void load8(const void *from, int64_t at, int left, bool vec,
                                      float (&x)[8]) {
  const int lane = threadIdx.x & 31;
  const T *p = static_cast<const T *>(from) + at + 4 * lane;
  if (vec) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (sizeof(T) == 4) {
        float4 v;
        asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                     : "l"(p + 128 * h));
        x[4 * h] = v.x, x[4 * h + 1] = v.y, x[4 * h + 2] = v.z, x[4 * h + 3] = v.w;
      } else {
        uint2 v;
        asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
                     : "=r"(v.x), "=r"(v.y)
                     : "l"(p + 128 * h));
        x[4 * h] = __uint_as_float(v.x << 16), x[4 * h + 1] = __uint_as_float(v.x & 0xffff0000u);
        x[4 * h + 2] = __uint_as_float(v.y << 16), x[4 * h + 3] = __uint_as_float(v.y & 0xffff0000u);
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int i = (j & 3) + (j >> 2) * 128;
    x[j] = i + 4 * lane < left ? widen(*(reinterpret_cast<const volatile T *>(p) + i)) : 0.0f;
  }
}

template <typename T>
__device__ __forceinline__ void store8(void *to, int64_t at, int left, bool vec,
                                       const float (&x)[8]) {
  const int lane = threadIdx.x & 31;
  T *p = static_cast<T *>(to) + at + 4 * lane;
  if (vec) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (sizeof(T) == 4) {
        __stcs(reinterpret_cast<float4 *>(p + 128 * h),
               make_float4(x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]));
      } else {
        uint2 v;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v.x) : "f"(x[4 * h + 1]), "f"(x[4 * h]));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v.y) : "f"(x[4 * h + 3]), "f"(x[4 * h + 2]));
        __stcs(reinterpret_cast<uint2 *>(p + 128 * h), v);
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int i = (j & 3) + (j >> 2) * 128;
    if (i + 4 * lane < left) p[i] = narrow<T>(x[j]);
  }
}

// The e4m3 values of a block, as four bytes for each half.
__device__ __forceinline__ uint2 load_codes(const void *from, int64_t at, int left, bool vec) {
  const int lane = threadIdx.x & 31;
  const uint8_t *p = static_cast<const uint8_t *>(from) + at + 4 * lane;
  uint2 v = make_uint2(0, 0);
  if (vec) {
    asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(v.x) : "l"(p));
    asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(v.y) : "l"(p + 128));
    return v;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int i = (j & 3) + (j >> 2) * 128;
    if (i + 4 * lane < left)
      (j < 4 ? v.x : v.y) |= (uint32_t)*(reinterpret_cast<const volatile uint8_t *>(p) + i)
                             << (8 * (j & 3));
  }
  return v;
}
__device__ __forceinline__ void store_codes(void *to, int64_t at, int left, bool vec, uint2 v) {
  const int lane = threadIdx.x & 31;
  uint8_t *p = static_cast<uint8_t *>(to) + at + 4 * lane;
  if (vec) {
    __stcs(reinterpret_cast<unsigned *>(p), v.x);
    __stcs(reinterpret_cast<unsigned *>(p + 128), v.y);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int i = (j & 3) + (j >> 2) * 128;
    if (i + 4 * lane < left) p[i] = (uint8_t)((j < 4 ? v.x : v.y) >> (8 * (j & 3)));
  }
}
__device__ __forceinline__ void decode(uint32_t four, float scale, float *x) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t halves;
    const uint16_t two = (uint16_t)(four >> (16 * h));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(halves) : "h"(two));
    float lo, hi;
    asm("{.reg .f16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}"
        : "=f"(lo), "=f"(hi)
        : "r"(halves));
    x[2 * h] = __fmul_rn(lo, scale);
    x[2 * h + 1] = __fmul_rn(hi, scale);
  }
}

// What maps a block x whose largest magnitude is `top` to e4m3 times 2^-120: (the scale, the
// factor).  Below 2^-100 the block is stored as zeros; a top that is not finite makes the
// scale NaN.  From 2^14 on the factor would leave fp32's normal numbers: x is made smaller,
// a ROOT that is not 0 not below 2^-100, so that it is still known from 0 (either way its code
// is the smallest one).
template <bool ROOT>
__device__ __forceinline__ float2 block_scale(float top, float (&x)[8]) {
  constexpr float kDown = 7.52316384526264e-37f;  // 2^-120
  if (top < kTiny) return make_float2(0.0f, 0.0f);
  if (!(top < INFINITY)) return make_float2(quiet_nan(), 0.0f);
  const float scale = __fmul_rn(top, 1.0f / 448.0f);
  if (top >= 16384.0f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float least = ROOT ? fminf(x[i], kTiny) : 0.0f;
      x[i] = __fmul_rn(x[i], 5.421010862427522e-20f);  // 2^-64
      if (ROOT) x[i] = fmaxf(x[i], least);
    }
    top = __fmul_rn(top, 5.421010862427522e-20f);
  }
  return make_float2(scale, __fmul_rn(__fmul_rn(448.0f, __frcp_rn(top)), kDown));
}
// Values in [0, 448] times 2^-120: e4m3's exponents, the subnormal one too, are then the lowest
// of fp32, and the bits from the 20th on are the code.  From bit 24 on here: y's bits 16 times
// over, and 16 random bits just below, with half of the last of them, that round it up with
// the probability of the remainder.  (The block's largest is 448 to an ulp or two: short of
// the next code for every random number.)
__device__ __forceinline__ uint32_t code_of(float y, uint32_t random) {
  return (__float_as_uint(y) << 4) + random;
}
// The upper bytes of four words.
__device__ __forceinline__ uint32_t upper_bytes(const uint32_t *x) {
  return __byte_perm(__byte_perm(x[0], x[1], 0x0073), __byte_perm(x[2], x[3], 0x0073), 0x5410);
}

// The approximate forms, off by an ulp or two: the root and the quotient go into a step of a
// weight (and a root into 4 bits).  With the rounded ones the kernel was bound by them (8
// bits, 434 M entries: 1612 us a call).  The root takes squares below fp32's normal numbers
// too (gradients below 2^-58: 916 us against 914 with those taken for 0); a denominator is a
// root of at least 2^-74.5, or eps, and never that small.
__device__ __forceinline__ float root_of(float x) {
  float y;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The larger of a and |b|; NaN if either is.
__device__ __forceinline__ float larger(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(fabsf(b)));
  return m;
}

// The largest of non-negative values over the warp; a NaN is the largest.
__device__ __forceinline__ float warp_top(float x) {
  return __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(x)));
}

struct Scalars {
  float clip, step_size, inv_root;  // c, lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  uint32_t step;
  float lr;                         // where the rate is on the device
};

// What a CTA needs to know of its tensor.
struct Tensor {
  void *p;
  const void *g;
  void *m, *v;
  float *scales, *master;
  bool p16, g16;
  uint32_t key;  // of the rounding
};
// The step's numbers, each twice; those that the launch knows stay in its parameters.
struct Factors {
  const uint64_t &b1, &not_b1, &b2, &not_b2, &eps;
  uint64_t clip, inv_root, minus_size, decay;
};
// Types that are common together, a whole block in vectors; or any.
enum Kind { kAny, kBf16, kF32, kBf16Master };

// A block of 256 entries from `at` on, `left` of them within the tensor.
template <bool STATE8, int KIND>
__device__ __forceinline__ void step_block(const Tensor &x, const Factors &f, int64_t at, int left,
                                           bool aligned) {
  const int lane = threadIdx.x & 31;
  const bool vec = KIND != kAny || (aligned && left == kBlock);
  const bool p16 = KIND == kAny ? x.p16 : KIND != kF32, g16 = KIND == kAny ? x.g16 : KIND != kF32;
  const bool master = KIND == kAny ? x.master != nullptr : KIND == kBf16Master;
  float g[8], m[8], v[8], w[8];
  if (g16) load8<uint16_t>(x.g, at, left, vec, g);
  else load8<float>(x.g, at, left, vec, g);
  if (master) load8<float>(x.master, at, left, vec, w);
  else if (p16) load8<uint16_t>(x.p, at, left, vec, w);
  else load8<float>(x.p, at, left, vec, w);
  float *scale = nullptr;
  if (STATE8) {
    const uint2 cm = load_codes(x.m, at, left, vec), cv = load_codes(x.v, at, left, vec);
    scale = x.scales + at / kBlock * 2;
    const float sm = scale[0], sv = scale[1];
    decode(cm.x, sm, m), decode(cm.y, sm, m + 4);
    decode(cv.x, sv, v), decode(cv.y, sv, v + 4);
  } else {
    load8<float>(x.m, at, left, vec, m);
    load8<float>(x.v, at, left, vec, v);
  }
  float top_m = 0.0f, top_v = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    uint64_t v2 = pack2(v[i], v[i + 1]);
    if (STATE8) v2 = mul2(v2, v2);
    const uint64_t g2 = mul2(pack2(g[i], g[i + 1]), f.clip);
    const uint64_t m2 = add2(mul2(pack2(m[i], m[i + 1]), f.b1), mul2(g2, f.not_b1));
    v2 = add2(mul2(v2, f.b2), mul2(mul2(g2, g2), f.not_b2));
    unpack2(m2, m[i], m[i + 1]);
    unpack2(v2, v[i], v[i + 1]);
    const float r0 = root_of(v[i]), r1 = root_of(v[i + 1]);
    float d0, d1;
    unpack2(fma2(pack2(r0, r1), f.inv_root, f.eps), d0, d1);
    const uint64_t step = mul2(mul2(m2, pack2(reciprocal(d0), reciprocal(d1))), f.minus_size);
    unpack2(fma2(pack2(w[i], w[i + 1]), f.decay, step), w[i], w[i + 1]);
    if (STATE8) {
      v[i] = r0, v[i + 1] = r1;
      top_m = larger(larger(top_m, m[i]), m[i + 1]);
      top_v = larger(larger(top_v, r0), r1);
    }
  }
  if (p16) store8<uint16_t>(x.p, at, left, vec, w);
  else store8<float>(x.p, at, left, vec, w);
  if (master) store8<float>(x.master, at, left, vec, w);
  if (!STATE8) {
    store8<float>(x.m, at, left, vec, m);
    store8<float>(x.v, at, left, vec, v);
    return;
  }
  top_m = warp_top(top_m);
  top_v = warp_top(top_v);
  const float2 fm = block_scale<false>(top_m, m), fv = block_scale<true>(top_v, v);
  // The hash of an entry is that of its index added to the tensor's key; its first product
  // is taken once for the block.  (A block begins at a multiple of 256: no carry into the
  // index's upper half.)
  const uint32_t base = ((uint32_t)at + (x.key ^ (uint32_t)(at >> 32)) + 4u * lane) * kMix0;
  uint32_t em[8], ev[8];  // a code in the upper byte of each
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t h = mix_rest(base + (uint32_t)((i & 3) + (i >> 2) * 128) * kMix0);
    // its upper half for m, the exclusive or of both halves for the root
    const uint32_t upper = ((h >> 8) & 0xffff00u) | 0x80u;
    const uint32_t lower = ((h << 8) ^ upper) & 0xffff80u;
    em[i] = code_of(__fmul_rn(fabsf(m[i]), fm.y), upper) | (__float_as_uint(m[i]) & 0x80000000u);
    // (a root that is not 0 is above 2^-101: at least the smallest code)
    ev[i] = max(code_of(__fmul_rn(v[i], fv.y), lower), min(__float_as_uint(v[i]), 1u << 24));
  }
  store_codes(x.m, at, left, vec, make_uint2(upper_bytes(em), upper_bytes(em + 4)));
  store_codes(x.v, at, left, vec, make_uint2(upper_bytes(ev), upper_bytes(ev + 4)));
  if (lane == 0) scale[0] = fm.x, scale[1] = fv.x;
}

template <bool STATE8, int CAP>
__global__ void __launch_bounds__(kNT, STATE8 ? 5 : 4) adamw_kernel(const __grid_constant__ AdamwArgs<CAP> a) {
  __shared__ Scalars sh;
  Scalars s{1.0f, a.step_size, a.inv_root, (uint32_t)a.step, 0.0f};
  if (a.step_device != nullptr || a.lr_device != nullptr) {
    if (threadIdx.x == 0) {
      const int64_t t = a.step_device != nullptr ? *a.step_device : a.step;
      s.lr = a.lr_device != nullptr ? *a.lr_device : 0.0f;
      s.step_size = (float)((a.lr_device != nullptr ? (double)s.lr : a.lr) /
                            (1.0 - power(a.beta1, t)));
      s.inv_root = (float)(1.0 / sqrt(1.0 - power(a.beta2, t)));
      s.step = (uint32_t)t;
      if (t < 1) s.clip = quiet_nan();  // no step has that number
      sh = s;
    }
    __syncthreads();
    s = sh;
    if (s.clip != s.clip) return;
  }
  if (a.norm != nullptr) {
    const float norm = *a.norm;
    if (!(norm < INFINITY)) return;  // the step is left out
    s.clip = fminf(1.0f, __fdiv_rn(a.max_norm, __fadd_rn(norm, kClipEps)));
  }
  const int t = find_tensor(a, blockIdx.x);
  const int64_t count = a.count[t];
  const uint8_t flags = a.flags[t];
  const bool aligned = flags & 4;
  const Tensor x{a.param[t], a.grad[t], a.exp_avg[t], a.exp_avg_sq[t], a.scales[t], a.master[t],
                 (flags & 1) != 0, (flags & 2) != 0,
                 STATE8 ? mix(mix(a.seed_key ^ s.step) ^ a.index[t]) : 0};
  const float decay = a.lr_device != nullptr
                          ? (float)(1.0 - (double)s.lr * (double)a.weight_decay[t])
                          : a.decay[t];
  auto twice = [](float y) { return pack2(y, y); };
  const Factors f{a.b1, a.not_b1, a.b2, a.not_b2, a.eps,
                  twice(s.clip), twice(s.inv_root), twice(-s.step_size), twice(decay)};
  const int warp = threadIdx.x >> 5;
  constexpr int kWarps = kNT / 32;
  int64_t at = (int64_t)(blockIdx.x - a.first[t]) * (a.blocks * kWarps * kBlock) + warp * kBlock;
  auto blocks = [&](auto kind) {
#pragma unroll 1
    for (int j = 0; j < a.blocks; ++j, at += kWarps * kBlock) {
      if (at >= count) return;
      const int left = (int)min(count - at, (int64_t)kBlock);
      if (left == kBlock)
        step_block<STATE8, decltype(kind)::value>(x, f, at, left, aligned);
      else
        step_block<STATE8, kAny>(x, f, at, left, aligned);
    }
  };
  if (aligned && x.p16 && x.g16 && x.master == nullptr)
    blocks(std::integral_constant<int, kBf16>());
  else if (aligned && x.p16 && x.g16)
    blocks(std::integral_constant<int, kBf16Master>());
  else if (aligned && !x.p16 && !x.g16 && x.master == nullptr)
    blocks(std::integral_constant<int, kF32>());
  else
    blocks(std::integral_constant<int, kAny>());
}

}  // namespace

int64_t adamw_chunks(int64_t count, int blocks) {
  const int64_t chunk = (int64_t)kNT / 32 * kBlock * blocks;
  return (count + chunk - 1) / chunk;
}

// Blocks that a warp takes one after the other.  With 32-bit states one: 434 M entries 1702 us,
// with two 1726.  With 8-bit states, which are bound by instructions, the CTA's start is
// shared by four where that leaves five waves of CTAs: 434 M entries 908 us with 4, 901 with
// 8, 1086 with 2; 0.8 M entries 8.3 us with 2, 9.9 with 4.
int adamw_blocks(int64_t entries, int state8, int sms) {
  if (!state8) return 1;
  const int64_t most = entries / ((int64_t)kNT / 32 * kBlock * 25 * sms);
  return most < 1 ? 1 : most > 4 ? 4 : (int)most;
}

double adamw_power(double b, int64_t t) { return power(b, t); }

uint32_t adamw_seed_key(uint64_t seed) { return mix(mix((uint32_t)seed) ^ (uint32_t)(seed >> 32)); }

template <int CAP>
cudaError_t adamw_launch(const AdamwArgs<CAP> &a, int state8, int grid, cudaStream_t stream) {
  if (state8)
    adamw_kernel<true, CAP><<<grid, kNT, 0, stream>>>(a);
  else
    adamw_kernel<false, CAP><<<grid, kNT, 0, stream>>>(a);
  return cudaGetLastError();
}

template cudaError_t adamw_launch(const AdamwArgs<kAdamwFew> &, int, int, cudaStream_t);
template cudaError_t adamw_launch(const AdamwArgs<kAdamwMany> &, int, int, cudaStream_t);

}  // namespace specv
