// specv_api_ops.cu -- the C ABI of the operators on the step's logits (declared
// in include/specv.h): log probabilities, distillation, gradient clipping.
//
// Host-side work only: argument validation, launch shapes, the launches.
#include <cstdint>
#include <mutex>

#include <nvtx3/nvToolsExt.h>

#include "specv.h"
#include "specv_internal.h"

namespace {

struct NvtxRange {
  explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange &) = delete;
  NvtxRange &operator=(const NvtxRange &) = delete;
};

specv_status status_of(cudaError_t e) {
  if (e == cudaSuccess) return SPECV_OK;
  specv::note_cuda_error(e);
  return SPECV_ERR_CUDA;
}

constexpr int64_t kLimit = (int64_t)1 << 62;
constexpr int64_t kClipElements = (int64_t)1 << 40;  // chunk numbers stay below 2^31

// Sizes and strides of a [B][N][V] view: every element offset stays below 2^62.
bool view_ok(int64_t B, int32_t N, int32_t V, int64_t sb, int64_t sn) {
  if (B < 1 || N < 1 || V < 1 || sb < 0 || sn < 0) return false;
  if (B > INT32_MAX / N) return false;
  return sb <= kLimit / 4 / B && sn <= kLimit / 4 / N;
}

// Past the last element of such a view.
const void *view_end(const void *p, int64_t B, int32_t N, int32_t V, int64_t sb, int64_t sn,
                     int64_t dtype) {
  return static_cast<const char *>(p) +
         ((B - 1) * sb + (N - 1) * sn + V) * (dtype == SPECV_BF16 ? 2 : 4);
}

bool dtype_ok(int64_t dtype) { return dtype == SPECV_F32 || dtype == SPECV_BF16; }

bool misaligned(const void *p, int64_t dtype) {
  return (uintptr_t)p % (dtype == SPECV_BF16 ? 2 : 4) != 0;
}
// 32-bit arrays (null ones pass)
template <typename... P>
bool words_misaligned(const P *...p) {
  return (... || ((uintptr_t)p % 4 != 0));
}

// The launches of specv_clip_grads: the norm's, then the scaling's, each for up to CAP
// gradients.
template <int CAP>
cudaError_t clip_launches(const specv_grad *grads, int64_t n, float max_norm, float *out_norm,
                          float2 *partial, int64_t groups, int per_launch, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  specv::ClipArgs<CAP> a;
  a.partial = partial;
  a.max_norm = max_norm;
  for (int scale = 0; scale < 2; ++scale) {
    int64_t at = 0;
    int partials = 0;
    for (int64_t g = 0; g < groups && e == cudaSuccess; ++g) {
      a.n = 0;
      a.chunks = 0;
      a.in_place = 1;
      for (; at < n && a.n < CAP; ++at) {
        if (grads[at].count == 0) continue;
        const int k = a.n++;
        a.in_place &= grads[at].out == grads[at].grad;
        a.in[k] = grads[at].grad;
        a.out[k] = grads[at].out;
        a.count[k] = grads[at].count;
        a.bf16[k] = grads[at].dtype == SPECV_BF16;
        a.first[k] = (int)a.chunks;
        a.chunks += specv::clip_chunks(a.in[k], a.count[k], a.bf16[k]);
      }
      int grid = a.chunks < per_launch ? (int)a.chunks : per_launch;
      if (grid < 1) grid = 1;
      a.out_norm = g == 0 ? out_norm : nullptr;
      if (scale == 0) {
        a.partial_at = partials;
        partials += grid;
        a.partials = partials;
        e = specv::clip_norm_launch(a, grid, st);
      } else {
        e = specv::clip_scale_launch(a, grid, g == 0, st);
      }
    }
  }
  return e;
}

}  // namespace

extern "C" {

specv_status specv_token_logprobs(const void *logits, const int32_t *tokens, int64_t B, int32_t N,
                                  int32_t V, int64_t stride_b, int64_t stride_n,
                                  specv_dtype dtype, int32_t top_n, float *out_logprob,
                                  float *out_entropy, float *out_stats, int32_t *out_top_tokens,
                                  float *out_top_logprobs, void *stream) {
  NvtxRange range("specv_token_logprobs");
  if (!logits || !tokens || !out_logprob || !out_entropy || !out_stats)
    return SPECV_ERR_INVALID_ARG;
  if (!view_ok(B, N, V, stride_b, stride_n) || !dtype_ok(dtype) || misaligned(logits, dtype))
    return SPECV_ERR_INVALID_ARG;
  if (top_n < 0 || top_n > specv::kMaxTop) return SPECV_ERR_INVALID_ARG;
  if (top_n > 0 && (!out_top_tokens || !out_top_logprobs)) return SPECV_ERR_INVALID_ARG;
  if (words_misaligned(tokens, out_logprob, out_entropy, out_top_tokens, out_top_logprobs) ||
      (uintptr_t)out_stats % sizeof(float2) != 0)  // written as pairs
    return SPECV_ERR_INVALID_ARG;
  int sms = 0;
  const int ready = specv::device_ready(&sms);
  if (ready != SPECV_OK) return (specv_status)ready;
  specv::LogprobArgs a;
  a.logits = logits;
  a.logits_end = view_end(logits, B, N, V, stride_b, stride_n, dtype);
  a.tokens = tokens;
  a.R = B * N;
  a.N = N;
  a.V = V;
  a.stride_b = stride_b;
  a.stride_n = stride_n;
  a.top_n = top_n;
  a.logprob = out_logprob;
  a.entropy = out_entropy;
  a.stats = reinterpret_cast<float2 *>(out_stats);
  a.top_tokens = out_top_tokens;
  a.top_logprobs = out_top_logprobs;
  return status_of(specv::logprobs_launch(a, dtype == SPECV_BF16, sms, specv::cluster_override(),
                                          static_cast<cudaStream_t>(stream)));
}

specv_status specv_token_logprobs_backward(const void *logits, const int32_t *tokens,
                                           const float *stats, const float *entropy,
                                           const float *grad_logprob, const float *grad_entropy,
                                           int64_t B, int32_t N, int32_t V, int64_t stride_b,
                                           int64_t stride_n, specv_dtype dtype, void *out_grad,
                                           void *stream) {
  NvtxRange range("specv_token_logprobs_backward");
  if (!logits || !tokens || !stats || !entropy || !grad_logprob || !out_grad)
    return SPECV_ERR_INVALID_ARG;
  if (!view_ok(B, N, V, stride_b, stride_n) || !dtype_ok(dtype) || misaligned(logits, dtype) ||
      misaligned(out_grad, dtype))
    return SPECV_ERR_INVALID_ARG;
  if (words_misaligned(tokens, entropy, grad_logprob, grad_entropy) ||
      (uintptr_t)stats % sizeof(float2) != 0)  // read as pairs
    return SPECV_ERR_INVALID_ARG;
  int sms = 0;
  const int ready = specv::device_ready(&sms);
  if (ready != SPECV_OK) return (specv_status)ready;
  specv::LogprobGradArgs a;
  a.logits = logits;
  a.logits_end = view_end(logits, B, N, V, stride_b, stride_n, dtype);
  a.tokens = tokens;
  a.stats = reinterpret_cast<const float2 *>(stats);
  a.entropy = entropy;
  a.grad_logprob = grad_logprob;
  a.grad_entropy = grad_entropy;
  a.R = B * N;
  a.N = N;
  a.V = V;
  a.stride_b = stride_b;
  a.stride_n = stride_n;
  a.out = out_grad;
  return status_of(
      specv::logprobs_grad_launch(a, dtype == SPECV_BF16, static_cast<cudaStream_t>(stream)));
}

specv_status specv_distill(const void *target_logits, const void *draft_logits,
                           const float *weight, int64_t B, int32_t K, int32_t V,
                           int64_t target_stride_b, int64_t target_stride_k,
                           int64_t draft_stride_b, int64_t draft_stride_k, specv_dtype dtype,
                           specv_divergence kind, float *out_loss, void *out_grad, void *stream) {
  NvtxRange range("specv_distill");
  if (!target_logits || !draft_logits || !out_loss) return SPECV_ERR_INVALID_ARG;
  if (!view_ok(B, K, V, target_stride_b, target_stride_k) ||
      !view_ok(B, K, V, draft_stride_b, draft_stride_k) || !dtype_ok(dtype))
    return SPECV_ERR_INVALID_ARG;
  if (kind != SPECV_FORWARD_KL && kind != SPECV_REVERSE_KL) return SPECV_ERR_INVALID_ARG;
  if (misaligned(target_logits, dtype) || misaligned(draft_logits, dtype) ||
      misaligned(out_grad, dtype) || words_misaligned(weight, out_loss))
    return SPECV_ERR_INVALID_ARG;
  int sms = 0;
  const int ready = specv::device_ready(&sms);
  if (ready != SPECV_OK) return (specv_status)ready;
  specv::DistillArgs a;
  a.target = target_logits;
  a.draft = draft_logits;
  a.target_end = view_end(target_logits, B, K, V, target_stride_b, target_stride_k, dtype);
  a.draft_end = view_end(draft_logits, B, K, V, draft_stride_b, draft_stride_k, dtype);
  a.weight = weight;
  a.B = B;
  a.K = K;
  a.V = V;
  a.target_stride_b = target_stride_b;
  a.target_stride_k = target_stride_k;
  a.draft_stride_b = draft_stride_b;
  a.draft_stride_k = draft_stride_k;
  a.out_loss = out_loss;
  a.out_grad = out_grad;
  return status_of(specv::distill_launch(a, dtype == SPECV_BF16, kind == SPECV_REVERSE_KL, sms,
                                         specv::cluster_override(), static_cast<cudaStream_t>(stream)));
}

specv_status specv_clip_grads(const specv_grad *grads, int64_t n, float max_norm, float *out_norm,
                              void *stream) {
  NvtxRange range("specv_clip_grads");
  if (n < 0 || (n > 0 && !grads) || !out_norm || !(max_norm >= 0.0f)) return SPECV_ERR_INVALID_ARG;
  if (words_misaligned(out_norm)) return SPECV_ERR_INVALID_ARG;
  int64_t live = 0, elements = 0;  // gradients with elements, and those
  for (int64_t i = 0; i < n; ++i) {
    const specv_grad &g = grads[i];
    if (g.count < 0 || g.count > kClipElements || !dtype_ok(g.dtype)) return SPECV_ERR_INVALID_ARG;
    if (g.count == 0) continue;
    if (!g.grad || !g.out || misaligned(g.grad, g.dtype) || misaligned(g.out, g.dtype))
      return SPECV_ERR_INVALID_ARG;
    ++live;
    elements += g.count;
    if (elements > kClipElements) return SPECV_ERR_INVALID_ARG;
  }
  int sms = 0;
  const int ready = specv::device_ready(&sms);
  if (ready != SPECV_OK) return (specv_status)ready;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // One launch of each kernel per kClipMany gradients; the sums of the norm's launches
  // lie one after the other.
  const int64_t groups = live > 0 ? (live + specv::kClipMany - 1) / specv::kClipMany : 1;
  int per_launch = specv::kClipCtasPerSm * sms;
  if (groups * per_launch > specv::kClipPartials) per_launch = (int)(specv::kClipPartials / groups);
  if (per_launch < 1) return SPECV_ERR_INVALID_ARG;  // millions of gradients
  void *scratch = nullptr;
  const size_t bytes = sizeof(float2) * specv::kClipPartials;
  bool cached = false;
  std::unique_lock<std::mutex> turn;  // the second launch reads what the first one leaves
  try {
    turn = specv::stream_turn(st);
    cached = specv::stream_scratch(st, bytes, &scratch);
  } catch (...) {
    return SPECV_ERR_NO_MEMORY;
  }
  cudaError_t e = cudaSuccess;
  if (!cached && (e = cudaMallocAsync(&scratch, bytes, st)) != cudaSuccess) {
    specv::note_cuda_error(e);
    (void)cudaGetLastError();
    return SPECV_ERR_NO_MEMORY;
  }
  float2 *partial = static_cast<float2 *>(scratch);
  if (e == cudaSuccess)
    e = live <= specv::kClipFew
            ? clip_launches<specv::kClipFew>(grads, n, max_norm, out_norm, partial, groups,
                                             per_launch, st)
            : clip_launches<specv::kClipMany>(grads, n, max_norm, out_norm, partial, groups,
                                              per_launch, st);
  if (!cached) {
    const cudaError_t ef = cudaFreeAsync(scratch, st);
    if (e == cudaSuccess) e = ef;
  }
  return status_of(e);
}

}  // extern "C"
