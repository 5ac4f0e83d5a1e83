// AdamW over many tensors at once, moments in 32 bits or in 8.
//
// Per element, t the step, in float32 (each operation rounded, none fused, so
// that codes do not depend on how the compiler contracts):
//   g' = grad_scale * g
//   m1 = b1 m + (1-b1) g';   v1 = b2 v + (1-b2) (g' g')
//   u  = m1 / (sqrt(v1) r2 + eps),           r2 = 1 / sqrt(1 - b2^t)
//   p1 = p - (u lr/(1-b1^t) + lr wd p mask), mask as in the cautious Adam step
// with the scalars formed in double on the host and rounded once.
//
// 8-bit moments.  A block of 256 consecutive elements of a tensor shares a
// power-of-two scale.  E = floor(log2 max |x|) (at least -100); the first
// moment is stored as E4M3 codes of x / 2^(E-7), the second as E5M2 codes of
// x / 2^(E-14), so the largest code is 256 or 2^15 and none overflows.  A
// power of two loses nothing with floating-point codes and makes value =
// code * scale exact.
// The codes are rounded stochastically: with beta2 = 0.999 the second moment
// moves by 0.1 % a step and E5M2's neighbours are 25 % apart, so rounding to
// nearest would freeze it, while rounding up with the probability of the
// remainder keeps the moving average unbiased.  The 16 random bits a moment
// takes come from a counter hash of (seed, step, tensor, element): the result
// does not depend on the launch.  bfloat16 parameters are rounded in the same
// way with 16 other bits, since updates are often below half their spacing.
// Codes are made in the integer representation: |x| 2^-E 2^(14-127) has in its
// exponent field the exponent field of the E4M3 code (subnormals included),
// so adding 20 random bits and dropping 20 rounds it; E5M2 likewise with 29
// and 21.
//
// Work: one warp per 256-element block, 8 elements a lane; eight warps share
// 32 blocks of one tensor.  One launch covers up to kMaxTensors tensors of
// the same types; the table is in the kernel's parameters.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <vector>

#include "../../include/muon.h"
#include "check.cuh"
#include "host.h"

namespace muon {
namespace {

constexpr int kQBlock = 256;       // elements that share a scale
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCtaBlocks = 32;     // 256-element blocks per CTA
constexpr int kMaxTensors = 400;   // per launch: the table fills the 32 KB of kernel parameters

struct AdamwTensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  long long numel;
  float step;     // lr / (1 - b1^t)
  float decay;    // lr * weight decay
  uint32_t key;   // of the random bits
  int first;      // first CTA of this tensor in the launch
  int vec;        // every array is aligned for the vector path
  int pad;
};

struct AdamwParams {
  AdamwTensor t[kMaxTensors];
  int n;
  int cautious;
  float b1, b2, omb1, omb2, r2, eps;
  const float* grad_scale;
};
static_assert(sizeof(AdamwParams) <= 32764, "kernel parameters are limited to 32764 bytes");

constexpr uint32_t kC0 = 0x9E3779B1u, kC1 = 0x6A09E667u, kC2 = 0xBB67AE85u;

__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
  x = (x ^ (x >> 16)) * kC1;
  x = (x ^ (x >> 15)) * kC2;
  return x ^ (x >> 16);
}

__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

template <bool BF16>
__device__ __forceinline__ void load8(const void* base, long long i, float (&x)[8]) {
  if constexpr (BF16) {
    const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + i);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[2 * k] = __uint_as_float(w[k] << 16);
      x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
  } else {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
    const float4 a = f[0], b = f[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
}

template <bool BF16>
__device__ __forceinline__ float load1(const void* base, long long i) {
  if constexpr (BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(base)[i]);
  else return static_cast<const float*>(base)[i];
}

__device__ __forceinline__ float e4m3(uint32_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(c), __NV_E4M3)));
}
__device__ __forceinline__ float e5m2(uint32_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(c), __NV_E5M2)));
}

// Rounds x down or up to bfloat16 with 16 random bits; NaN and infinity as they are.
__device__ __forceinline__ uint32_t bf16_stochastic(float x, uint32_t h) {
  const uint32_t u = __float_as_uint(x);
  const uint32_t r = (h * kC0) >> 16;
  const bool finite = (u & 0x7F800000u) != 0x7F800000u;
  const uint32_t nan = (u & 0x7FFFFFFFu) > 0x7F800000u ? 0x40u : 0u;
  return finite ? (u + r) >> 16 : (u >> 16) | nan;
}

// Largest |x| of the warp's block as the bits of a non-negative float; NaN is
// above infinity, so neither is lost.
__device__ __forceinline__ uint32_t block_max(const float (&x)[8]) {
  uint32_t a = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) a = max(a, __float_as_uint(x[k]) & 0x7FFFFFFFu);
  return __reduce_max_sync(0xFFFFFFFFu, a);
}

template <bool PB, bool GB, bool B8>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ AdamwParams P) {
  int lo = 0, hi = P.n - 1;  // the tensor: largest i with first <= blockIdx.x
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (P.t[mid].first <= static_cast<int>(blockIdx.x)) lo = mid; else hi = mid - 1;
  }
  const AdamwTensor& T = P.t[lo];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float gs = P.grad_scale ? *P.grad_scale : 1.0f;
  const long long b0 = static_cast<long long>(blockIdx.x - T.first) * kCtaBlocks;
  for (int j = warp; j < kCtaBlocks; j += kWarps) {
    const long long blk = b0 + j, i0 = blk * kQBlock;
    if (i0 >= T.numel) break;
    if (!MUON_CHECK(i0 >= 0)) break;
    const int left = static_cast<int>(min(static_cast<long long>(kQBlock), T.numel - i0));
    const bool vec = T.vec && left == kQBlock;
    float p[8], g[8], m[8], v[8];
    float sm = 1.0f, sv = 1.0f;
    if (B8) sm = T.ms[blk], sv = T.vs[blk];
    const int at0 = vec ? lane * 8 : lane, dat = vec ? 1 : 32;
    if (vec) {
      load8<PB>(T.p, i0 + at0, p);
      load8<GB>(T.g, i0 + at0, g);
      if constexpr (B8) {
        const uint2 cm = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(T.m) + i0 + at0);
        const uint2 cv = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(T.v) + i0 + at0);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          m[k] = e4m3(((k < 4 ? cm.x : cm.y) >> (8 * (k & 3))) & 0xFF);
          v[k] = e5m2(((k < 4 ? cv.x : cv.y) >> (8 * (k & 3))) & 0xFF);
        }
      } else {
        load8<false>(T.m, i0 + at0, m);
        load8<false>(T.v, i0 + at0, v);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int at = lane + 32 * k;
        p[k] = g[k] = m[k] = v[k] = 0.0f;
        if (at >= left) continue;
        p[k] = load1<PB>(T.p, i0 + at);
        g[k] = load1<GB>(T.g, i0 + at);
        if constexpr (B8) {
          m[k] = e4m3(static_cast<const uint8_t*>(T.m)[i0 + at]);
          v[k] = e5m2(static_cast<const uint8_t*>(T.v)[i0 + at]);
        } else {
          m[k] = static_cast<const float*>(T.m)[i0 + at];
          v[k] = static_cast<const float*>(T.v)[i0 + at];
        }
      }
    }
    const uint32_t key = T.key + static_cast<uint32_t>(static_cast<unsigned long long>(i0) >> 32) * kC1;
    uint32_t h[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (B8) {
        m[k] = __fmul_rn(m[k], sm);
        v[k] = __fmul_rn(v[k], sv);
      }
      const float gk = __fmul_rn(g[k], gs);
      m[k] = __fadd_rn(__fmul_rn(m[k], P.b1), __fmul_rn(gk, P.omb1));
      v[k] = __fadd_rn(__fmul_rn(v[k], P.b2), __fmul_rn(__fmul_rn(gk, gk), P.omb2));
      const float u = __fdiv_rn(m[k], __fadd_rn(__fmul_rn(__fsqrt_rn(v[k]), P.r2), P.eps));
      const bool on = !P.cautious || (u > 0.0f && p[k] > 0.0f) || (u < 0.0f && p[k] < 0.0f);
      const float dec = on ? __fmul_rn(p[k], T.decay) : 0.0f;
      p[k] = __fsub_rn(p[k], __fadd_rn(__fmul_rn(u, T.step), dec));
      if (B8 || PB) h[k] = mix(static_cast<uint32_t>(i0 + at0 + k * dat) * kC0 + key);
    }
    uint32_t cm[8], cv[8];
    if constexpr (B8) {
      const uint32_t am = block_max(m), av = block_max(v);
      const int em = min(max(static_cast<int>(am >> 23) - 127, -100), 126);
      const int ev = min(max(static_cast<int>(av >> 23) - 127, -100), 126);
      const float im = pow2i(-em), iv = pow2i(-ev);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float ym = __fmul_rn(__fmul_rn(fabsf(m[k]), im), 0x1p-113f);
        const float yv = __fmul_rn(__fmul_rn(fabsf(v[k]), iv), 0x1p-98f);
        cm[k] = ((__float_as_uint(ym) + ((h[k] & 0xFFFFu) << 4 | 8u)) >> 20 & 0x7Fu) | (__float_as_uint(m[k]) >> 24 & 0x80u);
        cv[k] = (__float_as_uint(yv) + ((h[k] >> 16) << 5 | 16u)) >> 21 & 0x7Fu;
      }
      if (lane == 0) {  // a block with a value that is not finite (or 2^127 and more) becomes NaN
        T.ms[blk] = am < 0x7F000000u ? pow2i(em - 7) : __uint_as_float(0x7FC00000u);
        T.vs[blk] = av < 0x7F000000u ? pow2i(ev - 14) : __uint_as_float(0x7FC00000u);
      }
    }
    if (vec) {
      if constexpr (PB) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w[k] = bf16_stochastic(p[2 * k], h[2 * k]) | bf16_stochastic(p[2 * k + 1], h[2 * k + 1]) << 16;
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(T.p) + i0 + at0) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        float4* f = reinterpret_cast<float4*>(static_cast<float*>(T.p) + i0 + at0);
        f[0] = make_float4(p[0], p[1], p[2], p[3]);
        f[1] = make_float4(p[4], p[5], p[6], p[7]);
      }
      if constexpr (B8) {
        auto four = [](const uint32_t* c) { return c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24; };
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(T.m) + i0 + at0) = make_uint2(four(cm), four(cm + 4));
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(T.v) + i0 + at0) = make_uint2(four(cv), four(cv + 4));
      } else {
        float4* a = reinterpret_cast<float4*>(static_cast<float*>(T.m) + i0 + at0);
        float4* b = reinterpret_cast<float4*>(static_cast<float*>(T.v) + i0 + at0);
        a[0] = make_float4(m[0], m[1], m[2], m[3]);
        a[1] = make_float4(m[4], m[5], m[6], m[7]);
        b[0] = make_float4(v[0], v[1], v[2], v[3]);
        b[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int at = lane + 32 * k;
        if (at >= left) continue;
        if constexpr (PB) static_cast<uint16_t*>(T.p)[i0 + at] = static_cast<uint16_t>(bf16_stochastic(p[k], h[k]));
        else static_cast<float*>(T.p)[i0 + at] = p[k];
        if constexpr (B8) {
          static_cast<uint8_t*>(T.m)[i0 + at] = static_cast<uint8_t>(cm[k]);
          static_cast<uint8_t*>(T.v)[i0 + at] = static_cast<uint8_t>(cv[k]);
        } else {
          static_cast<float*>(T.m)[i0 + at] = m[k];
          static_cast<float*>(T.v)[i0 + at] = v[k];
        }
      }
    }
  }
}

using KernelPtr = void (*)(AdamwParams);

// Index: bfloat16 parameters | bfloat16 gradients << 1 | 8-bit moments << 2.
const KernelPtr kKernels[8] = {
    adamw_kernel<false, false, false>, adamw_kernel<true, false, false>, adamw_kernel<false, true, false>,
    adamw_kernel<true, true, false>,   adamw_kernel<false, false, true>, adamw_kernel<true, false, true>,
    adamw_kernel<false, true, true>,   adamw_kernel<true, true, true>,
};

bool vector_aligned(const adamw_tensor_desc& d) {
  return aligned_to(d.param, 16) && aligned_to(d.grad, 16) && aligned_to(d.exp_avg, d.state_bits == 8 ? 8 : 16) &&
         aligned_to(d.exp_avg_sq, d.state_bits == 8 ? 8 : 16);
}

muon_status_t check_tensors(const adamw_tensor_desc* t, int n, bool need_grads) {
  if (n < 0 || (n > 0 && !t)) return MUON_ERR_INVALID_ARG;
  std::vector<Span> spans;
  spans.reserve(static_cast<size_t>(n) * 6);
  for (int i = 0; i < n; ++i) {
    const adamw_tensor_desc& d = t[i];
    if (d.numel < 0 || d.reserved != 0) return MUON_ERR_INVALID_ARG;
    if (d.param_dtype != MUON_BF16 && d.param_dtype != MUON_F32) return MUON_ERR_INVALID_ARG;
    if (d.grad_dtype != MUON_BF16 && d.grad_dtype != MUON_F32) return MUON_ERR_INVALID_ARG;
    if (d.state_bits != 8 && d.state_bits != 32) return MUON_ERR_INVALID_ARG;
    if (!std::isfinite(d.lr) || !std::isfinite(d.weight_decay)) return MUON_ERR_INVALID_ARG;
    if (d.numel == 0) continue;
    const bool small = d.state_bits == 8;
    if (!d.param || (need_grads && !d.grad) || !d.exp_avg || !d.exp_avg_sq) return MUON_ERR_INVALID_ARG;
    if (small != (d.exp_avg_scale != nullptr) || small != (d.exp_avg_sq_scale != nullptr)) return MUON_ERR_INVALID_ARG;
    if (d.numel > (1LL << 40)) return MUON_ERR_TOO_LARGE;
    const uint64_t np = d.param_dtype == MUON_F32 ? 4 : 2, ng = d.grad_dtype == MUON_F32 ? 4 : 2, ns = small ? 1 : 4;
    if (!aligned_to(d.param, np) || (d.grad && !aligned_to(d.grad, ng)) || !aligned_to(d.exp_avg, ns) ||
        !aligned_to(d.exp_avg_sq, ns) || !aligned_to(d.exp_avg_scale, 4) || !aligned_to(d.exp_avg_sq_scale, 4))
      return MUON_ERR_MISALIGNED;
    const uint64_t n64 = static_cast<uint64_t>(d.numel), nb = (n64 + kQBlock - 1) / kQBlock;
    spans.push_back(span_of(d.param, n64 * np, true));
    if (d.grad) spans.push_back(span_of(d.grad, n64 * ng, false));
    spans.push_back(span_of(d.exp_avg, n64 * ns, true));
    spans.push_back(span_of(d.exp_avg_sq, n64 * ns, true));
    if (small) {
      spans.push_back(span_of(d.exp_avg_scale, nb * 4, true));
      spans.push_back(span_of(d.exp_avg_sq_scale, nb * 4, true));
    }
  }
  return spans_conflict(spans) ? MUON_ERR_ALIASING : MUON_OK;
}

}  // namespace
}  // namespace muon

// One launch's tensors, in the order of the caller's list.
struct adamw_plan {
  struct Launch {
    int kind;                 // index into kKernels
    long long ctas;
    std::vector<muon::AdamwTensor> t;
    std::vector<int> index;   // position in the caller's list
  };
  std::vector<adamw_tensor_desc> desc;
  std::vector<Launch> launches;

  muon_status_t build();
};

muon_status_t adamw_plan::build() {
  using namespace muon;
  launches.clear();
  int open[8];
  for (int& o : open) o = -1;
  for (size_t i = 0; i < desc.size(); ++i) {
    const adamw_tensor_desc& d = desc[i];
    if (d.numel == 0) continue;
    const int kind = (d.param_dtype == MUON_BF16) | (d.grad_dtype == MUON_BF16) << 1 | (d.state_bits == 8) << 2;
    if (open[kind] < 0 || launches[open[kind]].t.size() == static_cast<size_t>(kMaxTensors)) {
      open[kind] = static_cast<int>(launches.size());
      launches.push_back({kind, 0, {}, {}});
    }
    Launch& l = launches[open[kind]];
    AdamwTensor a{};
    a.p = d.param;
    a.g = d.grad;
    a.m = d.exp_avg;
    a.v = d.exp_avg_sq;
    a.ms = d.exp_avg_scale;
    a.vs = d.exp_avg_sq_scale;
    a.numel = d.numel;
    a.first = static_cast<int>(l.ctas);
    a.vec = vector_aligned(d);
    l.ctas += (d.numel + kQBlock * kCtaBlocks - 1) / (kQBlock * kCtaBlocks);
    if (l.ctas > 0x7FFFFFFFLL) return MUON_ERR_TOO_LARGE;
    l.t.push_back(a);
    l.index.push_back(static_cast<int>(i));
  }
  return MUON_OK;
}

namespace muon {
namespace {

muon_status_t run_plan(const adamw_plan& plan, double beta1, double beta2, double eps, int cautious, int64_t step,
                       uint64_t seed, const float* grad_scale, cudaStream_t s) {
  if (step < 1 || !(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0) ||
      !std::isfinite(eps))
    return MUON_ERR_INVALID_ARG;
  if (!aligned_to(grad_scale, 4)) return MUON_ERR_MISALIGNED;
  const double bc1 = 1.0 - std::pow(beta1, static_cast<double>(step));
  const double bc2 = 1.0 - std::pow(beta2, static_cast<double>(step));
  if (!(bc1 > 0.0) || !(bc2 > 0.0)) return MUON_ERR_INVALID_ARG;
  for (const auto& l : plan.launches)
    for (const AdamwTensor& t : l.t)
      if (!t.g) return MUON_ERR_INVALID_ARG;
  if (plan.launches.empty()) return MUON_OK;
  int sms = 0;
  const muon_status_t st = device_sms(sms);
  if (st != MUON_OK) return st;
  const uint32_t k = mix(mix(static_cast<uint32_t>(seed) + kC0 * static_cast<uint32_t>(step)) ^ static_cast<uint32_t>(seed >> 32));
  for (const auto& l : plan.launches) {
    AdamwParams P;
    P.n = static_cast<int>(l.t.size());
    std::memcpy(P.t, l.t.data(), l.t.size() * sizeof(AdamwTensor));
    for (int i = 0; i < P.n; ++i) {
      const adamw_tensor_desc& d = plan.desc[l.index[i]];
      P.t[i].step = static_cast<float>(d.lr / bc1);
      P.t[i].decay = static_cast<float>(d.lr * d.weight_decay);
      P.t[i].key = mix(k + kC0 * static_cast<uint32_t>(l.index[i]));
    }
    P.cautious = cautious ? 1 : 0;
    P.b1 = static_cast<float>(beta1);
    P.b2 = static_cast<float>(beta2);
    P.omb1 = static_cast<float>(1.0 - beta1);
    P.omb2 = static_cast<float>(1.0 - beta2);
    P.r2 = static_cast<float>(1.0 / std::sqrt(bc2));
    P.eps = static_cast<float>(eps);
    P.grad_scale = grad_scale;
    kKernels[l.kind]<<<static_cast<unsigned>(l.ctas), kThreads, 0, s>>>(P);
    if (cudaGetLastError() != cudaSuccess) return MUON_ERR_CUDA;
  }
  return MUON_OK;
}

}  // namespace

MUON_CHECK_READER(check_failures_adamw)
}  // namespace muon

extern "C" {

muon_status_t adamw_plan_create(const adamw_tensor_desc* tensors, int n_tensors, adamw_plan** plan) {
  if (!plan) return MUON_ERR_INVALID_ARG;
  *plan = nullptr;
  try {
    muon_status_t st = muon::check_tensors(tensors, n_tensors, false);
    if (st != MUON_OK) return st;
    adamw_plan* p = new adamw_plan;
    p->desc.assign(tensors, tensors + n_tensors);
    st = p->build();
    if (st != MUON_OK) {
      delete p;
      return st;
    }
    *plan = p;
    return MUON_OK;
  } catch (const std::bad_alloc&) {
    return MUON_ERR_HOST_MEMORY;
  }
}

muon_status_t adamw_plan_set_grads(adamw_plan* plan, const void* const* grads, const int32_t* grad_dtypes) {
  if (!plan || (!plan->desc.empty() && (!grads || !grad_dtypes))) return MUON_ERR_INVALID_ARG;
  try {
    adamw_plan next;
    next.desc = plan->desc;
    for (size_t i = 0; i < next.desc.size(); ++i) {
      next.desc[i].grad = grads[i];
      next.desc[i].grad_dtype = grad_dtypes[i];
    }
    muon_status_t st = muon::check_tensors(next.desc.data(), static_cast<int>(next.desc.size()), true);
    if (st == MUON_OK) st = next.build();
    if (st != MUON_OK) return st;
    std::swap(*plan, next);
    return MUON_OK;
  } catch (const std::bad_alloc&) {
    return MUON_ERR_HOST_MEMORY;
  }
}

muon_status_t adamw_plan_set_rates(adamw_plan* plan, const double* lr, const double* weight_decay) {
  if (!plan || (!plan->desc.empty() && (!lr || !weight_decay))) return MUON_ERR_INVALID_ARG;
  for (size_t i = 0; i < plan->desc.size(); ++i)
    if (!std::isfinite(lr[i]) || !std::isfinite(weight_decay[i])) return MUON_ERR_INVALID_ARG;
  for (size_t i = 0; i < plan->desc.size(); ++i) {
    plan->desc[i].lr = lr[i];
    plan->desc[i].weight_decay = weight_decay[i];
  }
  return MUON_OK;
}

muon_status_t adamw_plan_step(const adamw_plan* plan, double beta1, double beta2, double eps, int cautious,
                              int64_t step, uint64_t seed, const float* grad_scale, void* stream) {
  if (!plan) return MUON_ERR_INVALID_ARG;
  return muon::run_plan(*plan, beta1, beta2, eps, cautious, step, seed, grad_scale, static_cast<cudaStream_t>(stream));
}

void adamw_plan_destroy(adamw_plan* plan) { delete plan; }

muon_status_t adamw_step(const adamw_tensor_desc* tensors, int n_tensors, double beta1, double beta2, double eps,
                         int cautious, int64_t step, uint64_t seed, const float* grad_scale, void* stream) {
  try {
    muon_status_t st = muon::check_tensors(tensors, n_tensors, true);
    if (st != MUON_OK) return st;
    adamw_plan p;
    p.desc.assign(tensors, tensors + n_tensors);
    st = p.build();
    if (st != MUON_OK) return st;
    return muon::run_plan(p, beta1, beta2, eps, cautious, step, seed, grad_scale, static_cast<cudaStream_t>(stream));
  } catch (const std::bad_alloc&) {
    return MUON_ERR_HOST_MEMORY;
  }
}

}  // extern "C"
