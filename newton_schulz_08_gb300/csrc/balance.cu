// Balance loss of a router with its per-expert counts, and its gradient.
//
// Per token p = softmax(logits).  Over the kept tokens of a group g: counts
// c_e of the expert ids, f = c / sum c, P = mean of p, and
//   balance = mean_g E sum_e f_e P_e,     z = mean over tokens of lse^2,
//   d/dx_e  = p_e (a_e - sum_j a_j p_j) + gz 2 lse / N p_e,
//   a_e     = gb / G' (E f_e - 1) / N_g
// (the gradient does not change when a constant is added to a; taking 1 off
// E f, whose mean is 1, keeps the difference a_e - sum_j a_j p_j exact where
// the load is nearly balanced).
//
// A row has at most 1024 entries, so it lives in registers: L lanes (a power
// of two) share a row, 8 entries a lane and chunk of 8 L, and 32 / L rows go
// through a warp at a time.  HBM-bound: a row is read once forward, read and
// written once backward.
//
// Forward, two launches.  balance_rows: each CTA takes consecutive rows of
// one group and leaves partial sums of p and lse^2, counts and token numbers
// in the workspace.  balance_finish: one CTA per group adds the partials in
// their order, and the last CTA to arrive adds the groups in theirs, so equal
// calls give equal bits; only whole numbers are added with atomics.
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
constexpr int kWarps = kThreads / 32;
constexpr int kFinishThreads = 512;
constexpr int kMaxExperts = 1024;
constexpr int kTargetCtas = 608;  // four per SM
constexpr float kLog2e = 1.4426950408889634f;

struct BalanceParams {
  const void* x;
  const int64_t* ids;
  const uint8_t* mask;
  void* grad;
  long long stride, grad_stride;
  long long group_rows;  // rows of a group
  long long cta_rows;    // rows of a CTA
  long long groups;
  int parts;             // CTAs per group
  int experts, top, lanes;
  int vec;
  // partial results of CTA i: sums[i][experts], counts[i][experts], tokens[i], squares[i]
  float* sums;
  int* part_counts;
  int* part_tokens;
  float* squares;
  float* group_loss;
  unsigned* arrived;
  // results
  float* stats;
  int* counts;
  int* tokens;
  float* mean;
  float* weights;
  const float* grad_balance;
  const float* grad_z;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Position of a lane's entry k of chunk c: neighbours in the vector layout,
// L apart where rows are not aligned.
__device__ __forceinline__ int entry(const BalanceParams& P, int c, int k, int sub) {
  return P.vec ? (c * P.lanes + sub) * 8 + k : c * P.lanes * 8 + k * P.lanes + sub;
}

template <bool BF16, int NC>
__device__ __forceinline__ void load_row(const BalanceParams& P, long long row, int sub, bool on, float (&x)[NC][8]) {
  const long long base = row * P.stride;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[c][k] = -INFINITY;
    if (!on) continue;
    const int e0 = entry(P, c, 0, sub);
    if (P.vec) {
      if (e0 >= P.experts) continue;
      if constexpr (BF16) {
        const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(P.x) + base + e0);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[c][2 * k] = __uint_as_float(w[k] << 16);
          x[c][2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        }
      } else {
        const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(P.x) + base + e0);
        const float4 a = f[0], b = f[1];
        x[c][0] = a.x; x[c][1] = a.y; x[c][2] = a.z; x[c][3] = a.w;
        x[c][4] = b.x; x[c][5] = b.y; x[c][6] = b.z; x[c][7] = b.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int e = entry(P, c, k, sub);
        if (e >= P.experts) continue;
        if constexpr (BF16) x[c][k] = __bfloat162float(static_cast<const __nv_bfloat16*>(P.x)[base + e]);
        else x[c][k] = static_cast<const float*>(P.x)[base + e];
      }
    }
  }
}

// x becomes the row's probabilities (0 where the row is off); returns lse.
template <int NC>
__device__ __forceinline__ float softmax_row(int lanes, bool on, float (&x)[NC][8]) {
  float m = -INFINITY;
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int k = 0; k < 8; ++k) m = fmaxf(m, x[c][k]);
  for (int d = lanes / 2; d > 0; d /= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
  float s = 0.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[c][k] = ex2((x[c][k] - m) * kLog2e);
      s += x[c][k];
    }
  for (int d = lanes / 2; d > 0; d /= 2) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
  const float inv = on ? 1.0f / s : 0.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int k = 0; k < 8; ++k) x[c][k] = on ? x[c][k] * inv : 0.0f;
  return m + logf(s);
}

template <bool BF16, int NC>
__global__ void __launch_bounds__(kThreads) balance_rows(const __grid_constant__ BalanceParams P) {
  extern __shared__ float smem[];
  float* sp = smem;                                               // kWarps x experts
  int* sc = reinterpret_cast<int*>(smem + kWarps * P.experts);    // experts
  __shared__ int s_tokens[kWarps];
  __shared__ float s_sq[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane & (P.lanes - 1), rows_warp = 32 / P.lanes, mine = lane / P.lanes;
  const long long g = blockIdx.x / P.parts;
  const long long r0 = static_cast<long long>(blockIdx.x % P.parts) * P.cta_rows;
  const long long r1 = min(P.group_rows, r0 + P.cta_rows);
  const long long first = g * P.group_rows;
  if (blockIdx.x == 0 && threadIdx.x == 0) *P.arrived = 0;
  for (int e = threadIdx.x; e < P.experts; e += kThreads) sc[e] = 0;
  __syncthreads();

  float acc[NC][8], sq = 0.0f;
  int tokens = 0;
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[c][k] = 0.0f;
  for (long long r = r0 + warp * rows_warp; r < r1; r += kWarps * rows_warp) {
    const long long row = first + r + mine;
    const bool on = r + mine < r1 && (!P.mask || P.mask[row]);
    float x[NC][8];
    load_row<BF16, NC>(P, row, sub, on, x);
    const float lse = softmax_row<NC>(P.lanes, on, x);
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[c][k] += x[c][k];
    if (on && sub == 0) {
      sq += lse * lse;
      ++tokens;
    }
  }
  // the assignments of this CTA's rows
  const long long i1 = (first + r1) * P.top;
  for (long long i = (first + r0) * P.top + threadIdx.x; i < i1; i += kThreads) {
    if (P.mask && !P.mask[i / P.top]) continue;
    const int64_t e = P.ids[i];
    if (e >= 0 && e < P.experts) atomicAdd(&sc[e], 1);
  }
  // rows of a warp, then warps, in order
  for (int d = P.lanes; d < 32; d *= 2) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[c][k] += __shfl_xor_sync(0xFFFFFFFFu, acc[c][k], d);
  }
  if (mine == 0) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int e = entry(P, c, k, sub);
        if (e < P.experts) sp[warp * P.experts + e] = acc[c][k];
      }
  }
  for (int d = 16; d > 0; d /= 2) {
    sq += __shfl_xor_sync(0xFFFFFFFFu, sq, d);
    tokens += __shfl_xor_sync(0xFFFFFFFFu, tokens, d);
  }
  if (lane == 0) s_sq[warp] = sq, s_tokens[warp] = tokens;
  __syncthreads();
  const long long out = static_cast<long long>(blockIdx.x) * P.experts;
  for (int e = threadIdx.x; e < P.experts; e += kThreads) {
    float s = 0.0f;
    for (int w = 0; w < kWarps; ++w) s += sp[w * P.experts + e];
    P.sums[out + e] = s;
    P.part_counts[out + e] = sc[e];
  }
  if (threadIdx.x == 0) {
    float s = 0.0f;
    int n = 0;
    for (int w = 0; w < kWarps; ++w) s += s_sq[w], n += s_tokens[w];
    P.squares[blockIdx.x] = s;
    P.part_tokens[blockIdx.x] = n;
  }
}

// Sum over the CTA's threads in a fixed order; every thread gets it.
template <typename T>
__device__ __forceinline__ T block_sum(T v, T* scratch) {
  for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  T s = 0;
  for (int w = 0; w < kFinishThreads / 32; ++w) s += scratch[w];
  return s;
}

__global__ void __launch_bounds__(kFinishThreads) balance_finish(const __grid_constant__ BalanceParams P) {
  __shared__ float s_sum[kFinishThreads];
  __shared__ int s_cnt[kFinishThreads];
  __shared__ float s_mean[kMaxExperts];
  __shared__ int s_total[kMaxExperts];
  __shared__ float f_scratch[kFinishThreads / 32];
  __shared__ int i_scratch[kFinishThreads / 32];
  __shared__ unsigned s_last;
  const long long g = blockIdx.x, base = g * P.parts;
  int n = 0;
  for (int i = threadIdx.x; i < P.parts; i += kFinishThreads) n += P.part_tokens[base + i];
  n = block_sum(n, i_scratch);
  const float inv_n = n > 0 ? 1.0f / static_cast<float>(n) : 0.0f;
  // `width` experts at a time, the partials dealt over the threads left
  int width = 32;
  while (width < P.experts && width < kFinishThreads) width *= 2;
  const int deals = kFinishThreads / width, deal = threadIdx.x / width;
  for (int e0 = 0; e0 < P.experts; e0 += width) {
    const int e = e0 + (threadIdx.x & (width - 1));
    float s = 0.0f;
    int c = 0;
    if (e < P.experts) {
#pragma unroll 8
      for (int i = deal; i < P.parts; i += deals) {
        s += P.sums[(base + i) * P.experts + e];
        c += P.part_counts[(base + i) * P.experts + e];
      }
    }
    __syncthreads();
    s_sum[threadIdx.x] = s;
    s_cnt[threadIdx.x] = c;
    __syncthreads();
    if (deal == 0 && e < P.experts) {
      for (int k = 1; k < deals; ++k) s += s_sum[k * width + threadIdx.x], c += s_cnt[k * width + threadIdx.x];
      s_mean[e] = s * inv_n;
      s_total[e] = c;
    }
  }
  __syncthreads();
  int assigned = 0;
  for (int e = threadIdx.x; e < P.experts; e += kFinishThreads) assigned += s_total[e];
  assigned = block_sum(assigned, i_scratch);
  const float share = assigned > 0 ? static_cast<float>(P.experts) / static_cast<float>(assigned) : 0.0f;
  float loss = 0.0f;
  for (int e = threadIdx.x; e < P.experts; e += kFinishThreads) {
    const float f = share * static_cast<float>(s_total[e]);  // experts * f_e
    loss += f * s_mean[e];
    P.counts[g * P.experts + e] = s_total[e];
    P.mean[g * P.experts + e] = s_mean[e];
    P.weights[g * P.experts + e] = assigned > 0 ? (f - 1.0f) * inv_n : 0.0f;
  }
  loss = block_sum(loss, f_scratch);
  if (threadIdx.x == 0) {
    P.group_loss[g] = loss;
    P.tokens[g] = n;
    __threadfence();
    s_last = atomicAdd(P.arrived, 1u) + 1u == gridDim.x;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  float balance = 0.0f, squares = 0.0f;
  float kept = 0.0f;
  int some = 0;
  for (long long i = threadIdx.x; i < P.groups; i += kFinishThreads) {
    balance += __ldcg(P.group_loss + i);
    const int t = __ldcg(P.tokens + i);
    kept += static_cast<float>(t);
    some += t > 0;
  }
  for (long long i = threadIdx.x; i < P.groups * P.parts; i += kFinishThreads) squares += P.squares[i];
  balance = block_sum(balance, f_scratch);
  squares = block_sum(squares, f_scratch);
  kept = block_sum(kept, f_scratch);
  some = block_sum(some, i_scratch);
  if (threadIdx.x == 0) {
    P.stats[0] = some > 0 ? balance / static_cast<float>(some) : 0.0f;
    P.stats[1] = some > 0 ? squares / kept : 0.0f;
    P.stats[2] = some > 0 ? 1.0f / static_cast<float>(some) : 0.0f;
    P.stats[3] = some > 0 ? 2.0f / kept : 0.0f;
  }
}

template <bool BF16, int NC>
__global__ void __launch_bounds__(kThreads) balance_grad(const __grid_constant__ BalanceParams P) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane & (P.lanes - 1), rows_warp = 32 / P.lanes, mine = lane / P.lanes;
  const long long g = blockIdx.x / P.parts;
  const long long r0 = static_cast<long long>(blockIdx.x % P.parts) * P.cta_rows;
  const long long r1 = min(P.group_rows, r0 + P.cta_rows);
  const long long first = g * P.group_rows;
  const float gb = *P.grad_balance * P.stats[2], gz = *P.grad_z * P.stats[3];
  float a[NC][8];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int e = entry(P, c, k, sub);
      a[c][k] = e < P.experts ? gb * P.weights[g * P.experts + e] : 0.0f;
    }
  for (long long r = r0 + warp * rows_warp; r < r1; r += kWarps * rows_warp) {
    const long long row = first + r + mine;
    const bool in = r + mine < r1, on = in && (!P.mask || P.mask[row]);
    float x[NC][8];
    load_row<BF16, NC>(P, row, sub, on, x);
    const float lse = softmax_row<NC>(P.lanes, on, x);
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) s = fmaf(a[c][k], x[c][k], s);
    for (int d = P.lanes / 2; d > 0; d /= 2) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    const float shift = on ? gz * lse - s : 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) x[c][k] = on ? x[c][k] * (a[c][k] + shift) : 0.0f;
    if (!in) continue;
    const long long base = row * P.grad_stride;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int e0 = entry(P, c, 0, sub);
      if (P.vec) {
        if (e0 >= P.experts) continue;
        if constexpr (BF16) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(x[c][2 * k], x[c][2 * k + 1]);
            w[k] = *reinterpret_cast<const uint32_t*>(&b);
          }
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(P.grad) + base + e0) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
          float4* f = reinterpret_cast<float4*>(static_cast<float*>(P.grad) + base + e0);
          f[0] = make_float4(x[c][0], x[c][1], x[c][2], x[c][3]);
          f[1] = make_float4(x[c][4], x[c][5], x[c][6], x[c][7]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int e = entry(P, c, k, sub);
          if (e >= P.experts) continue;
          if constexpr (BF16) static_cast<__nv_bfloat16*>(P.grad)[base + e] = __float2bfloat16_rn(x[c][k]);
          else static_cast<float*>(P.grad)[base + e] = x[c][k];
        }
      }
    }
  }
}

using KernelPtr = void (*)(BalanceParams);

// Index: 0, 1, 2 for up to 256, 512, 1024 experts; + 3 for bfloat16.
const KernelPtr kRows[6] = {balance_rows<false, 1>, balance_rows<false, 2>, balance_rows<false, 4>,
                            balance_rows<true, 1>,  balance_rows<true, 2>,  balance_rows<true, 4>};
const KernelPtr kGrad[6] = {balance_grad<false, 1>, balance_grad<false, 2>, balance_grad<false, 4>,
                            balance_grad<true, 1>,  balance_grad<true, 2>,  balance_grad<true, 4>};

// The split of the rows: lanes per row, CTAs per group, rows per CTA.
struct Split {
  int lanes, kernel, parts;
  long long group_rows, cta_rows;
};

Split split_of(int64_t tokens, int experts, int64_t groups) {
  Split s;
  s.lanes = 1;
  while (s.lanes < 32 && s.lanes * 8 < experts) s.lanes *= 2;
  s.kernel = experts <= 256 ? 0 : experts <= 512 ? 1 : 2;
  s.group_rows = tokens / groups;
  const long long pass = static_cast<long long>(kWarps) * (32 / s.lanes);  // rows of a CTA at a time
  const long long most = (s.group_rows + pass - 1) / pass;
  long long parts = (kTargetCtas + groups - 1) / groups;
  if (parts > most) parts = most;
  if (parts < 1) parts = 1;
  s.cta_rows = (s.group_rows + parts - 1) / parts;
  s.cta_rows = (s.cta_rows + pass - 1) / pass * pass;
  if (s.cta_rows < 1) s.cta_rows = 1;
  s.parts = static_cast<int>((s.group_rows + s.cta_rows - 1) / s.cta_rows);
  if (s.parts < 1) s.parts = 1;
  return s;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

struct Layout {
  size_t arrived, sums, counts, tokens, squares, loss, total;
};

Layout layout_of(const Split& s, int experts, int64_t groups) {
  const size_t n = static_cast<size_t>(groups) * s.parts;
  Layout l;
  l.arrived = 0;
  l.sums = 256;
  l.counts = l.sums + up256(n * experts * 4);
  l.tokens = l.counts + up256(n * experts * 4);
  l.squares = l.tokens + up256(n * 4);
  l.loss = l.squares + up256(n * 4);
  l.total = l.loss + up256(static_cast<size_t>(groups) * 4);
  return l;
}

muon_status_t check_shape(int dtype, int64_t tokens, int experts, int64_t stride, int64_t groups) {
  if (dtype != MUON_BF16 && dtype != MUON_F32) return MUON_ERR_INVALID_ARG;
  if (tokens < 0 || experts < 1 || experts > kMaxExperts || groups < 1 || stride < experts) return MUON_ERR_INVALID_ARG;
  if (tokens % groups != 0) return MUON_ERR_INVALID_ARG;
  if (tokens > INT32_MAX || groups > INT32_MAX || stride > (1LL << 32)) return MUON_ERR_TOO_LARGE;
  if (split_of(tokens, experts, groups).parts * groups > INT32_MAX) return MUON_ERR_TOO_LARGE;
  return MUON_OK;
}

uint64_t matrix_bytes(int64_t rows, int cols, int64_t stride, int size) {
  return rows > 0 ? (static_cast<uint64_t>(rows - 1) * stride + cols) * size : 0;
}

}  // namespace

MUON_CHECK_READER(check_failures_balance)
}  // namespace muon

extern "C" size_t balance_loss_workspace_size(int64_t tokens, int experts, int64_t groups) {
  using namespace muon;
  if (check_shape(MUON_F32, tokens, experts, experts, groups) != MUON_OK) return 0;
  return layout_of(split_of(tokens, experts, groups), experts, groups).total;
}

extern "C" muon_status_t balance_loss(const void* logits, int dtype, int64_t tokens, int experts, int64_t row_stride,
                                      const int64_t* ids, int top, const uint8_t* mask, int64_t groups, float* stats,
                                      int32_t* counts, int32_t* n_tokens, float* mean_probs, float* weights,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  using namespace muon;
  muon_status_t st = check_shape(dtype, tokens, experts, row_stride, groups);
  if (st != MUON_OK) return st;
  if (top < 1 || top > experts) return MUON_ERR_INVALID_ARG;
  if (tokens * top > INT32_MAX) return MUON_ERR_TOO_LARGE;
  if (!stats || !counts || !n_tokens || !mean_probs || !weights || !workspace || (tokens > 0 && (!logits || !ids)))
    return MUON_ERR_INVALID_ARG;
  const int size = dtype == MUON_F32 ? 4 : 2;
  if (!aligned_to(logits, size) || !aligned_to(ids, 8) || !aligned_to(stats, 4) || !aligned_to(counts, 4) ||
      !aligned_to(n_tokens, 4) || !aligned_to(mean_probs, 4) || !aligned_to(weights, 4) || !aligned_to(workspace, 256))
    return MUON_ERR_MISALIGNED;
  const Split s = split_of(tokens, experts, groups);
  const Layout l = layout_of(s, experts, groups);
  if (workspace_bytes < l.total) return MUON_ERR_WORKSPACE_TOO_SMALL;
  try {
    const uint64_t ge = static_cast<uint64_t>(groups) * experts * 4;
    std::vector<Span> v = {span_of(logits, matrix_bytes(tokens, experts, row_stride, size), false),
                           span_of(ids, static_cast<uint64_t>(tokens) * top * 8, false),
                           span_of(mask, mask ? tokens : 0, false),
                           span_of(stats, 16, true), span_of(counts, ge, true),
                           span_of(n_tokens, static_cast<uint64_t>(groups) * 4, true), span_of(mean_probs, ge, true),
                           span_of(weights, ge, true), span_of(workspace, l.total, true)};
    if (spans_conflict(v)) return MUON_ERR_ALIASING;
  } catch (const std::bad_alloc&) {
    return MUON_ERR_HOST_MEMORY;
  }
  int sms = 0;
  st = device_sms(sms);
  if (st != MUON_OK) return st;
  char* ws = static_cast<char*>(workspace);
  BalanceParams P{};
  P.x = logits;
  P.ids = ids;
  P.mask = mask;
  P.stride = row_stride;
  P.group_rows = s.group_rows;
  P.cta_rows = s.cta_rows;
  P.groups = groups;
  P.parts = s.parts;
  P.experts = experts;
  P.top = top;
  P.lanes = s.lanes;
  P.vec = experts % 8 == 0 && row_stride * size % 16 == 0 && aligned_to(logits, 16);
  P.arrived = reinterpret_cast<unsigned*>(ws + l.arrived);
  P.sums = reinterpret_cast<float*>(ws + l.sums);
  P.part_counts = reinterpret_cast<int*>(ws + l.counts);
  P.part_tokens = reinterpret_cast<int*>(ws + l.tokens);
  P.squares = reinterpret_cast<float*>(ws + l.squares);
  P.group_loss = reinterpret_cast<float*>(ws + l.loss);
  P.stats = stats;
  P.counts = counts;
  P.tokens = n_tokens;
  P.mean = mean_probs;
  P.weights = weights;
  cudaStream_t str = static_cast<cudaStream_t>(stream);
  const size_t smem = static_cast<size_t>(kWarps + 1) * experts * 4;
  kRows[s.kernel + (dtype == MUON_BF16 ? 3 : 0)]<<<static_cast<unsigned>(s.parts * groups), kThreads, smem, str>>>(P);
  if (cudaGetLastError() != cudaSuccess) return MUON_ERR_CUDA;
  balance_finish<<<static_cast<unsigned>(groups), kFinishThreads, 0, str>>>(P);
  return cudaGetLastError() == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

extern "C" muon_status_t balance_loss_backward(const void* logits, int dtype, int64_t tokens, int experts,
                                               int64_t row_stride, const uint8_t* mask, int64_t groups,
                                               const float* stats, const float* weights, const float* grad_balance,
                                               const float* grad_z, void* grad, int64_t grad_stride, void* stream) {
  using namespace muon;
  muon_status_t st = check_shape(dtype, tokens, experts, row_stride, groups);
  if (st != MUON_OK) return st;
  if (grad_stride < experts) return MUON_ERR_INVALID_ARG;
  if (grad_stride > (1LL << 32)) return MUON_ERR_TOO_LARGE;
  if (tokens == 0) return MUON_OK;
  if (!logits || !stats || !weights || !grad_balance || !grad_z || !grad) return MUON_ERR_INVALID_ARG;
  const int size = dtype == MUON_F32 ? 4 : 2;
  if (!aligned_to(logits, size) || !aligned_to(grad, size) || !aligned_to(stats, 4) || !aligned_to(weights, 4) ||
      !aligned_to(grad_balance, 4) || !aligned_to(grad_z, 4))
    return MUON_ERR_MISALIGNED;
  try {
    std::vector<Span> v = {span_of(mask, mask ? tokens : 0, false),
                           span_of(stats, 16, false), span_of(weights, static_cast<uint64_t>(groups) * experts * 4, false),
                           span_of(grad_balance, 4, false), span_of(grad_z, 4, false),
                           span_of(grad, matrix_bytes(tokens, experts, grad_stride, size), true)};
    if (grad != logits || grad_stride != row_stride)
      v.push_back(span_of(logits, matrix_bytes(tokens, experts, row_stride, size), false));
    if (spans_conflict(v)) return MUON_ERR_ALIASING;
  } catch (const std::bad_alloc&) {
    return MUON_ERR_HOST_MEMORY;
  }
  int sms = 0;
  st = device_sms(sms);
  if (st != MUON_OK) return st;
  const Split s = split_of(tokens, experts, groups);
  BalanceParams P{};
  P.x = logits;
  P.mask = mask;
  P.grad = grad;
  P.stride = row_stride;
  P.grad_stride = grad_stride;
  P.group_rows = s.group_rows;
  P.cta_rows = s.cta_rows;
  P.groups = groups;
  P.parts = s.parts;
  P.experts = experts;
  P.lanes = s.lanes;
  P.vec = experts % 8 == 0 && row_stride * size % 16 == 0 && grad_stride * size % 16 == 0 && aligned_to(logits, 16) &&
          aligned_to(grad, 16);
  P.stats = const_cast<float*>(stats);
  P.weights = const_cast<float*>(weights);
  P.grad_balance = grad_balance;
  P.grad_z = grad_z;
  kGrad[s.kernel + (dtype == MUON_BF16 ? 3 : 0)]<<<static_cast<unsigned>(s.parts * groups), kThreads, 0,
                                                   static_cast<cudaStream_t>(stream)>>>(P);
  return cudaGetLastError() == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
