// Log probabilities of given tokens with entropy and top alternatives, and
// the gradient with respect to the logits.
//
// With z = scale x over a row of V logits, m = max z, S = sum exp(z - m) and
// W = sum exp(z - m) (z - m):
//   lse = m + log S,   logprob = z_target - lse,   entropy = log S - W / S,
//   grad_j = scale (gl 1[j = target] - p_j (gl + ge (log p_j + entropy))).
//
// One CTA per row.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <new>
#include <vector>

#include "../../include/muon.h"
#include "check.cuh"
#include "host.h"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTop = 32;

struct LogprobParams {
  const void* x;
  const int64_t* targets;
  float* logprobs;
  float* lse;
  float* entropy;
  float* top_logprobs;
  int64_t* top_ids;
  const float* gl;
  const float* ge;
  void* grad;
  long long stride, grad_stride;
  int vocab, top;
  float scale;
};

template <bool BF16>
__device__ __forceinline__ float at(const void* x, long long i) {
  if constexpr (BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(x)[i]);
  else return static_cast<const float*>(x)[i];
}

// A number's place in the order of alternatives: larger values first, then
// lower indices; NaN below every number.
__device__ __forceinline__ unsigned long long order_key(float x, int j) {
  x = isnan(x) ? -INFINITY : x + 0.0f;  // -0 equals 0
  const uint32_t u = __float_as_uint(x);
  const uint32_t k = u & 0x80000000u ? ~u : u | 0x80000000u;
  return static_cast<unsigned long long>(k) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(j));
}

template <typename T, typename F>
__device__ __forceinline__ T block_reduce(T v, F f, T* scratch) {
  for (int d = 16; d > 0; d /= 2) v = f(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  v = scratch[0];
  for (int w = 1; w < kThreads / 32; ++w) v = f(v, scratch[w]);
  return v;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) logprob_score(const __grid_constant__ LogprobParams P) {
  __shared__ float scratch[kThreads / 32];
  __shared__ unsigned long long key_scratch[kThreads / 32];
  const long long row = blockIdx.x, base = row * P.stride;
  const int64_t target = P.targets[row];
  const int t = threadIdx.x;
  if (target < 0) {
    if (t == 0) P.logprobs[row] = P.lse[row] = P.entropy[row] = 0.0f;
    if (t < P.top) P.top_logprobs[row * P.top + t] = 0.0f, P.top_ids[row * P.top + t] = -1;
    return;
  }
  auto add = [](float a, float b) { return a + b; };
  float m = -INFINITY;
  for (int j = t; j < P.vocab; j += kThreads) m = fmaxf(m, at<BF16>(P.x, base + j) * P.scale);
  m = block_reduce(m, [](float a, float b) { return fmaxf(a, b); }, scratch);
  const float ref = m == -INFINITY ? 0.0f : m;
  float s = 0.0f, w = 0.0f;
  for (int j = t; j < P.vocab; j += kThreads) {
    const float d = at<BF16>(P.x, base + j) * P.scale - ref;
    const float e = expf(d);
    s += e;
    if (e > 0.0f) w += e * d;
  }
  s = block_reduce(s, add, scratch);
  w = block_reduce(w, add, scratch);
  const float lse = m + logf(s);
  if (t == 0) {
    P.lse[row] = lse;
    P.entropy[row] = s == 0.0f ? 0.0f : logf(s) - w / s;
    P.logprobs[row] = target >= P.vocab ? NAN
                      : lse == -INFINITY ? -INFINITY : at<BF16>(P.x, base + target) * P.scale - lse;
  }
  unsigned long long last = ~0ull;
  for (int k = 0; k < P.top; ++k) {
    unsigned long long best = 0;
    for (int j = t; j < P.vocab; j += kThreads) {
      const unsigned long long q = order_key(at<BF16>(P.x, base + j), j);
      if (q < last && q > best) best = q;
    }
    best = block_reduce(best, [](unsigned long long a, unsigned long long b) { return a > b ? a : b; }, key_scratch);
    last = best;
    if (t == 0) {
      const int j = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(best));
      P.top_ids[row * P.top + k] = j;
      P.top_logprobs[row * P.top + k] = lse == -INFINITY ? -INFINITY : at<BF16>(P.x, base + j) * P.scale - lse;
    }
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) logprob_grad(const __grid_constant__ LogprobParams P) {
  const long long row = blockIdx.x, base = row * P.stride, out = row * P.grad_stride;
  const int64_t target = P.targets[row];
  const bool on = target >= 0;
  const float lse = on ? P.lse[row] : 0.0f;
  const float gl = !on ? 0.0f : target < P.vocab ? P.gl[row] : NAN;
  const float ge = on && P.ge ? P.ge[row] : 0.0f, h = on && P.ge ? P.entropy[row] : 0.0f;
  for (int j = threadIdx.x; j < P.vocab; j += kThreads) {
    float v = 0.0f;
    if (on) {
      const float d = at<BF16>(P.x, base + j) * P.scale - lse;
      const float p = lse == -INFINITY ? 0.0f : expf(d);
      v = p == 0.0f ? (isnan(gl) ? gl : 0.0f) : -p * (gl + ge * (d + h));
      if (j == target) v += gl;
    }
    if constexpr (BF16) static_cast<__nv_bfloat16*>(P.grad)[out + j] = __float2bfloat16_rn(v * P.scale);
    else static_cast<float*>(P.grad)[out + j] = v * P.scale;
  }
}

muon_status_t check_logits(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t stride,
                           const int64_t* targets, float scale) {
  if (dtype != MUON_BF16 && dtype != MUON_F32) return MUON_ERR_INVALID_ARG;
  if (rows < 0 || vocab < 1 || stride < vocab) return MUON_ERR_INVALID_ARG;
  if (!(scale > 0.0f && scale <= 1e6f)) return MUON_ERR_INVALID_ARG;
  if (rows == 0) return MUON_OK;
  if (!logits || !targets) return MUON_ERR_INVALID_ARG;
  if (vocab > (1LL << 30) || rows > INT32_MAX || stride > (1LL << 32)) return MUON_ERR_TOO_LARGE;
  if (!aligned_to(logits, dtype == MUON_F32 ? 4 : 2) || !aligned_to(targets, 8)) return MUON_ERR_MISALIGNED;
  return MUON_OK;
}

uint64_t matrix_bytes(int64_t rows, int64_t cols, int64_t stride, int dtype) {
  return (static_cast<uint64_t>(rows - 1) * stride + cols) * (dtype == MUON_F32 ? 4 : 2);
}

// What both directions check and launch; grad, gl: null for a score alone,
// lse and entropy are read (score = false) or written.
muon_status_t run(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                  const int64_t* targets, float scale, int top, bool score, float* logprobs, float* lse,
                  float* entropy, float* top_logprobs, int64_t* top_ids, bool backward, const float* gl,
                  const float* ge, void* grad, int64_t grad_stride, void* stream) {
  muon_status_t st = check_logits(logits, dtype, rows, vocab, row_stride, targets, scale);
  if (st != MUON_OK) return st;
  if (score && (top < 0 || top > kMaxTop || top > vocab)) return MUON_ERR_INVALID_ARG;
  if (backward && grad_stride < vocab) return MUON_ERR_INVALID_ARG;
  if (rows == 0) return MUON_OK;
  if (backward && grad_stride > (1LL << 32)) return MUON_ERR_TOO_LARGE;
  if (score && (!logprobs || !lse || !entropy || (top > 0 && (!top_logprobs || !top_ids)))) return MUON_ERR_INVALID_ARG;
  if (backward && (!gl || !grad || !lse || (ge && !entropy))) return MUON_ERR_INVALID_ARG;
  if (!aligned_to(logprobs, 4) || !aligned_to(lse, 4) || !aligned_to(entropy, 4) || !aligned_to(top_logprobs, 4) ||
      !aligned_to(top_ids, 8) || !aligned_to(gl, 4) || !aligned_to(ge, 4) ||
      !aligned_to(grad, dtype == MUON_F32 ? 4 : 2))
    return MUON_ERR_MISALIGNED;
  const uint64_t r = static_cast<uint64_t>(rows);
  try {
    std::vector<Span> v = {span_of(targets, r * 8, false)};
    if (score) {
      v.push_back(span_of(logprobs, r * 4, true));
      v.push_back(span_of(top_logprobs, r * top * 4, true));
      v.push_back(span_of(top_ids, r * top * 8, true));
    }
    v.push_back(span_of(lse, r * 4, score));
    if (entropy) v.push_back(span_of(entropy, r * 4, score));
    if (backward) {
      v.push_back(span_of(gl, r * 4, false));
      if (ge) v.push_back(span_of(ge, r * 4, false));
      v.push_back(span_of(grad, matrix_bytes(rows, vocab, grad_stride, dtype), true));
    }
    if (!backward || grad != logits || grad_stride != row_stride)
      v.push_back(span_of(logits, matrix_bytes(rows, vocab, row_stride, dtype), false));
    if (spans_conflict(v)) return MUON_ERR_ALIASING;
  } catch (const std::bad_alloc&) {
    return MUON_ERR_HOST_MEMORY;
  }
  int sms = 0;
  st = device_sms(sms);
  if (st != MUON_OK) return st;
  LogprobParams P{};
  P.x = logits;
  P.targets = targets;
  P.logprobs = logprobs;
  P.lse = lse;
  P.entropy = entropy;
  P.top_logprobs = top_logprobs;
  P.top_ids = top_ids;
  P.gl = gl;
  P.ge = ge;
  P.grad = grad;
  P.stride = row_stride;
  P.grad_stride = grad_stride;
  P.vocab = static_cast<int>(vocab);
  P.top = score ? top : 0;
  P.scale = scale;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>(rows);
  if (score) {
    if (dtype == MUON_BF16) logprob_score<true><<<grid, kThreads, 0, s>>>(P);
    else logprob_score<false><<<grid, kThreads, 0, s>>>(P);
    if (cudaGetLastError() != cudaSuccess) return MUON_ERR_CUDA;
  }
  if (backward) {
    if (dtype == MUON_BF16) logprob_grad<true><<<grid, kThreads, 0, s>>>(P);
    else logprob_grad<false><<<grid, kThreads, 0, s>>>(P);
    if (cudaGetLastError() != cudaSuccess) return MUON_ERR_CUDA;
  }
  return MUON_OK;
}

}  // namespace

MUON_CHECK_READER(check_failures_logprob)
}  // namespace muon

extern "C" muon_status_t token_logprobs(const void* logits, int dtype, int64_t rows, int64_t vocab,
                                        int64_t row_stride, const int64_t* targets, float scale, int top,
                                        float* logprobs, float* lse, float* entropy, float* top_logprobs,
                                        int64_t* top_ids, void* stream) {
  return muon::run(logits, dtype, rows, vocab, row_stride, targets, scale, top, true, logprobs, lse, entropy,
                   top_logprobs, top_ids, false, nullptr, nullptr, nullptr, 0, stream);
}

extern "C" muon_status_t token_logprobs_backward(const void* logits, int dtype, int64_t rows, int64_t vocab,
                                                 int64_t row_stride, const int64_t* targets, float scale,
                                                 const float* lse, const float* entropy, const float* grad_logprobs,
                                                 const float* grad_entropy, void* grad, int64_t grad_stride,
                                                 void* stream) {
  return muon::run(logits, dtype, rows, vocab, row_stride, targets, scale, 0, false, nullptr,
                   const_cast<float*>(lse), const_cast<float*>(entropy), nullptr, nullptr, true, grad_logprobs,
                   grad_entropy, grad, grad_stride, stream);
}

extern "C" muon_status_t token_logprobs_loss(const void* logits, int dtype, int64_t rows, int64_t vocab,
                                             int64_t row_stride, const int64_t* targets, float scale, int top,
                                             const float* grad_logprobs, const float* grad_entropy, float* logprobs,
                                             float* lse, float* entropy, float* top_logprobs, int64_t* top_ids,
                                             void* grad, int64_t grad_stride, void* stream) {
  return muon::run(logits, dtype, rows, vocab, row_stride, targets, scale, top, true, logprobs, lse, entropy,
                   top_logprobs, top_ids, true, grad_logprobs, grad_entropy, grad, grad_stride, stream);
}
