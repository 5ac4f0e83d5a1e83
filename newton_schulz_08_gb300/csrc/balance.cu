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
// of two) share a row, 8 entries a lane and chunk of 8 L.  A warp takes
// 32 / L rows side by side and, up to 512 experts, two such sets at a time:
// the reductions of a row are a chain of ten shuffles, and two chains overlap.
// HBM-bound: a row is read once forward, read and written once backward.
// 131072 x 256 float32: forward 31 us of 21 that its bytes take, backward 42 of
// 40 (one set: 44 and 56; four leave room for fewer warps: 43 and 55; scalar
// arithmetic in place of pairs: 36 and 48).
// Rows off the 16-byte boundaries (a number of experts that is no multiple of 8) come
// through shared memory in tiles instead, copied as one run: there a few
// threads, without a shuffle each, take a row's sums, and then a thread an
// expert's (65536 x 161 bfloat16: forward 28 -> 20 us, backward 42 -> 23,
// against entry by entry from global memory; the bytes take 4 and 6).
//
// Forward, two launches.  balance_rows: each CTA takes consecutive rows of
// one group and leaves partial sums of p and lse^2, counts and the numbers of
// tokens and assignments in the workspace.  balance_finish: each CTA adds the
// partials of some experts of a group in their order, and the last CTA to
// arrive adds the losses in theirs, so equal calls give equal bits; only whole
// numbers are added with atomics.
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
constexpr int kTileBytes = 42 * 1024;  // of a tile: four CTAs per SM
constexpr int kTargetCtas = 608;  // four per SM
constexpr float kLog2e = 1.4426950408889634f;
// Up to here one fused operation x log2(e) - m log2(e) does for an exponent: the
// product of m is rounded, which multiplies every power of the row by at most
// 1 +- 2^-14.  Probabilities do not see a common factor; lse is off by less than its
// own spacing.  Beyond it the factor would leave float32's range in the end.
constexpr float kFar = 1024.0f;

struct BalanceParams {
  const void* x;
  const int64_t* ids;
  const uint8_t* mask;
  void* grad;
  long long stride, grad_stride;
  long long tokens_all;  // rows of all groups
  long long group_rows;  // rows of a group
  long long cta_rows;    // rows of a CTA
  long long groups;
  int parts;             // CTAs per group
  int experts, top, lanes;
  int tile_rows;         // rows of a tile, a power of two up to kThreads
  int width, slices;     // balance_finish: experts of a CTA (a power of two), CTAs per group
  // partial results of CTA i: sums[i][experts], counts[i][experts], numbers[i] (tokens, assignments), squares[i]
  float* sums;
  int* part_counts;
  int2* numbers;
  float* squares;
  float* group_loss;     // of balance_finish's CTAs
  float* group_squares;
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

// First entry of a lane's chunk c.
__device__ __forceinline__ int entry(const BalanceParams& P, int c, int sub) { return (c * P.lanes + sub) * 8; }

template <bool BF16, int NC>
__device__ __forceinline__ void load_row(const BalanceParams& P, long long row, int sub, bool on, float (&x)[NC][8]) {
  const long long base = row * P.stride;
  if (!MUON_CHECK(!on || (row >= 0 && row < P.tokens_all))) on = false;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[c][k] = -INFINITY;
    const int e0 = entry(P, c, sub);
    if (!on || e0 >= P.experts) continue;
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
  }
}

template <bool BF16, int NC>
__device__ __forceinline__ void store_row(const BalanceParams& P, long long row, int sub, const float (&x)[NC][8]) {
  const long long base = row * P.grad_stride;
  if (!MUON_CHECK(row >= 0 && row < P.tokens_all)) return;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int e0 = entry(P, c, sub);
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
  }
}

// x becomes exp(x - largest) of its row, which times inv is the probability;
// both are 0 where a row is off.  U rows of a lane at a time, entries in pairs.
template <int NC, int U>
__device__ __forceinline__ void softmax_rows(int lanes, const bool (&on)[U], float (&x)[U][NC][8], float (&inv)[U], float (&lse)[U]) {
  float m[U], s[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    m[u] = -INFINITY;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) m[u] = fmaxf(m[u], x[u][c][k]);
  }
  for (int d = lanes / 2; d > 0; d /= 2)
#pragma unroll
    for (int u = 0; u < U; ++u) m[u] = fmaxf(m[u], __shfl_xor_sync(0xFFFFFFFFu, m[u], d));
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float shift = on[u] ? -m[u] * kLog2e : 0.0f;
    if (on[u] && fabsf(m[u]) > kFar) {  // a row far from zero, or masked as a whole: the difference first
      shift = 0.0f;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k) x[u][c][k] -= m[u];
    }
    float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const float2 t = __ffma2_rn(make_float2(x[u][c][k], x[u][c][k + 1]), make_float2(kLog2e, kLog2e), make_float2(shift, shift));
        const float2 e = make_float2(ex2(t.x), ex2(t.y));
        sum = __fadd2_rn(sum, e);
        x[u][c][k] = e.x;
        x[u][c][k + 1] = e.y;
      }
    s[u] = sum.x + sum.y;
  }
  for (int d = lanes / 2; d > 0; d /= 2)
#pragma unroll
    for (int u = 0; u < U; ++u) s[u] += __shfl_xor_sync(0xFFFFFFFFu, s[u], d);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    inv[u] = on[u] ? __fdividef(1.0f, s[u]) : 0.0f;
    // s lies between 1 and 1024, but for the rounding of the shift.  The fast
    // logarithm is off by 2^-21 near 1, else by 3 units in the last place, which
    // is of the size of what its terms' powers (2 units) leave in s
    lse[u] = m[u] + __logf(s[u]);
  }
}

template <typename T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

// Sets of rows that a warp works on at a time.
template <int NC>
constexpr int kSets = NC <= 2 ? 2 : 1;

template <bool BF16, int NC>
__global__ void __launch_bounds__(kThreads, 4) balance_rows(const __grid_constant__ BalanceParams P) {
  extern __shared__ float smem[];
  float* sp = smem;                                               // kWarps x experts
  int* sc = reinterpret_cast<int*>(smem + kWarps * P.experts);    // experts
  __shared__ int2 s_numbers[kWarps];
  __shared__ float s_sq[kWarps];
  constexpr int kU = kSets<NC>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane & (P.lanes - 1), rows_warp = 32 / P.lanes, mine = lane / P.lanes;
  const long long g = blockIdx.x / P.parts;
  const long long r0 = static_cast<long long>(blockIdx.x % P.parts) * P.cta_rows;
  const long long r1 = min(P.group_rows, r0 + P.cta_rows);
  const long long first = g * P.group_rows;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // balance_finish waits for this grid's end
  if (blockIdx.x == 0 && threadIdx.x == 0) *P.arrived = 0;
  for (int e = threadIdx.x; e < P.experts; e += kThreads) sc[e] = 0;
  __syncthreads();
  // the assignments of this CTA's rows
  int assigned = 0;
  const long long i1 = (first + r1) * P.top;
#pragma unroll 8
  for (long long i = (first + r0) * P.top + threadIdx.x; i < i1; i += kThreads) {
    const int64_t e = P.ids[i];
    if (e < 0 || e >= P.experts || (P.mask && !P.mask[static_cast<unsigned>(i) / static_cast<unsigned>(P.top)])) continue;
    atomicAdd(&sc[e], 1);
    ++assigned;
  }

  float acc[NC][8], sq = 0.0f;
  int tokens = 0;
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[c][k] = 0.0f;
  for (long long r = r0 + warp * rows_warp; r < r1; r += kU * kWarps * rows_warp) {
    float x[kU][NC][8];
    bool on[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const long long at = r + u * kWarps * rows_warp + mine;
      on[u] = at < r1 && (!P.mask || P.mask[first + at]);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) load_row<BF16, NC>(P, first + r + u * kWarps * rows_warp + mine, sub, on[u], x[u]);
    float inv[kU], lse[kU];
    softmax_rows<NC, kU>(P.lanes, on, x, inv, lse);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          const float2 p = __ffma2_rn(make_float2(x[u][c][k], x[u][c][k + 1]), make_float2(inv[u], inv[u]),
                                      make_float2(acc[c][k], acc[c][k + 1]));
          acc[c][k] = p.x;
          acc[c][k + 1] = p.y;
        }
      if (on[u] && sub == 0) {
        sq += lse[u] * lse[u];
        ++tokens;
      }
    }
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
        const int e = entry(P, c, sub) + k;
        if (e < P.experts) sp[warp * P.experts + e] = acc[c][k];
      }
  }
  sq = warp_sum(sq);
  tokens = warp_sum(tokens);
  assigned = warp_sum(assigned);
  if (lane == 0) s_sq[warp] = sq, s_numbers[warp] = make_int2(tokens, assigned);
  __syncthreads();
  const long long out = static_cast<long long>(blockIdx.x) * P.experts;
  for (int e = threadIdx.x; e < P.experts; e += kThreads) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += sp[w * P.experts + e];
    P.sums[out + e] = s;
    P.part_counts[out + e] = sc[e];
  }
  if (threadIdx.x == 0) {
    float s = 0.0f;
    int2 n = make_int2(0, 0);
    for (int w = 0; w < kWarps; ++w) s += s_sq[w], n.x += s_numbers[w].x, n.y += s_numbers[w].y;
    P.squares[blockIdx.x] = s;
    P.numbers[blockIdx.x] = n;
  }
}

// A CTA takes `width` experts of a group, their partials dealt over its threads.
__global__ void __launch_bounds__(kFinishThreads) balance_finish(const __grid_constant__ BalanceParams P) {
  constexpr int kFinishWarps = kFinishThreads / 32;
  __shared__ float s_sum[kFinishThreads];
  __shared__ int s_cnt[kFinishThreads];
  __shared__ float3 s_all[kFinishWarps];
  __shared__ int2 s_numbers[kFinishWarps];
  __shared__ float s_loss[kFinishWarps];
  __shared__ unsigned s_last;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int slice = blockIdx.x % P.slices, deals = kFinishThreads / P.width, deal = t / P.width;
  const long long g = blockIdx.x / P.slices, base = g * P.parts;
  const int e = slice * P.width + (t & (P.width - 1));
  int2 n = make_int2(0, 0);  // tokens, assignments
  float squares = 0.0f;
  for (int i = t; i < P.parts; i += kFinishThreads) {
    const int2 m = P.numbers[base + i];
    squares += P.squares[base + i];
    n.x += m.x;
    n.y += m.y;
  }
  float s = 0.0f;
  int c = 0;
  if (e < P.experts) {
#pragma unroll 8
    for (int i = deal; i < P.parts; i += deals) {
      s += P.sums[(base + i) * P.experts + e];
      c += P.part_counts[(base + i) * P.experts + e];
    }
  }
  n.x = warp_sum(n.x);
  n.y = warp_sum(n.y);
  squares = warp_sum(squares);
  if (lane == 0) s_numbers[warp] = n, s_loss[warp] = squares;
  s_sum[t] = s;
  s_cnt[t] = c;
  __syncthreads();
  n = make_int2(0, 0);
  squares = 0.0f;
#pragma unroll
  for (int w = 0; w < kFinishWarps; ++w) n.x += s_numbers[w].x, n.y += s_numbers[w].y, squares += s_loss[w];
  const float inv_n = n.x > 0 ? 1.0f / static_cast<float>(n.x) : 0.0f;
  const float share = n.y > 0 ? static_cast<float>(P.experts) / static_cast<float>(n.y) : 0.0f;
  float loss = 0.0f;
  if (deal == 0 && e < P.experts) {
    for (int k = 1; k < deals; ++k) s += s_sum[k * P.width + t], c += s_cnt[k * P.width + t];
    const float mean = s * inv_n, f = share * static_cast<float>(c);  // experts * f_e
    loss = f * mean;
    P.counts[g * P.experts + e] = c;
    P.mean[g * P.experts + e] = mean;
    P.weights[g * P.experts + e] = n.y > 0 ? (f - 1.0f) * inv_n : 0.0f;
  }
  loss = warp_sum(loss);
  __syncthreads();
  if (lane == 0) s_loss[warp] = loss;
  __syncthreads();
  if (t == 0) {
    loss = 0.0f;
    for (int w = 0; w < kFinishWarps; ++w) loss += s_loss[w];
    P.group_loss[blockIdx.x] = loss;
    if (slice == 0) P.tokens[g] = n.x, P.group_squares[g] = squares;
    __threadfence();
    s_last = gridDim.x == 1 || atomicAdd(P.arrived, 1u) + 1u == gridDim.x;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  float3 all = make_float3(0.0f, 0.0f, 0.0f);  // losses, squares, tokens
  int some = 0;
  for (long long i = t; i < P.groups * P.slices; i += kFinishThreads) {
    all.x += __ldcg(P.group_loss + i);
    if (i >= P.groups) continue;
    const int k = __ldcg(P.tokens + i);
    all.y += __ldcg(P.group_squares + i);
    all.z += static_cast<float>(k);
    some += k > 0;
  }
  all = make_float3(warp_sum(all.x), warp_sum(all.y), warp_sum(all.z));
  some = warp_sum(some);
  if (lane == 0) s_all[warp] = all, s_cnt[warp] = some;
  __syncthreads();
  if (t == 0) {
    all = make_float3(0.0f, 0.0f, 0.0f);
    some = 0;
    for (int w = 0; w < kFinishWarps; ++w) {
      all.x += s_all[w].x, all.y += s_all[w].y, all.z += s_all[w].z;
      some += s_cnt[w];
    }
    P.stats[0] = some > 0 ? all.x / static_cast<float>(some) : 0.0f;
    P.stats[1] = some > 0 ? all.y / all.z : 0.0f;
    P.stats[2] = some > 0 ? 1.0f / static_cast<float>(some) : 0.0f;
    P.stats[3] = some > 0 ? 2.0f / all.z : 0.0f;
  }
}

template <bool BF16, int NC>
__global__ void __launch_bounds__(kThreads, 4) balance_grad(const __grid_constant__ BalanceParams P) {
  constexpr int kU = kSets<NC>;
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
      const int e = entry(P, c, sub) + k;
      a[c][k] = e < P.experts ? gb * P.weights[g * P.experts + e] : 0.0f;
    }
  for (long long r = r0 + warp * rows_warp; r < r1; r += kU * kWarps * rows_warp) {
    float x[kU][NC][8], inv[kU], lse[kU], s[kU];
    bool in[kU], on[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const long long at = r + u * kWarps * rows_warp + mine;
      in[u] = at < r1;
      on[u] = in[u] && (!P.mask || P.mask[first + at]);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) load_row<BF16, NC>(P, first + r + u * kWarps * rows_warp + mine, sub, on[u], x[u]);
    softmax_rows<NC, kU>(P.lanes, on, x, inv, lse);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int k = 0; k < 8; k += 2)
          sum = __ffma2_rn(make_float2(a[c][k], a[c][k + 1]), make_float2(x[u][c][k], x[u][c][k + 1]), sum);
      s[u] = sum.x + sum.y;
    }
    for (int d = P.lanes / 2; d > 0; d /= 2)
#pragma unroll
      for (int u = 0; u < kU; ++u) s[u] += __shfl_xor_sync(0xFFFFFFFFu, s[u], d);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (!in[u]) continue;
      // e inv (a + shift), with the sum of a p in the shift
      const float shift = on[u] ? (gz * lse[u] - s[u] * inv[u]) * inv[u] : 0.0f;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          const float2 w = __ffma2_rn(make_float2(a[c][k], a[c][k + 1]), make_float2(inv[u], inv[u]), make_float2(shift, shift));
          const float2 v = __fmul2_rn(make_float2(x[u][c][k], x[u][c][k + 1]), w);
          x[u][c][k] = on[u] ? v.x : 0.0f;
          x[u][c][k + 1] = on[u] ? v.y : 0.0f;
        }
      store_row<BF16, NC>(P, first + r + u * kWarps * rows_warp + mine, sub, x[u]);
    }
  }
}

// ------------------------------------------------ tiles (rows off the vectors)

// `rows` rows from row `row` on, into `tile` with their own pitch of `experts`
// entries; returns where the first one begins.  A run without gaps is copied
// in 16-byte vectors, its ends entry by entry.  No barrier.
template <typename T>
__device__ __forceinline__ T* load_tile(const BalanceParams& P, long long row, int rows, unsigned char* tile) {
  const T* x = static_cast<const T*>(P.x) + row * P.stride;
  if (!MUON_CHECK(row >= 0 && row + rows <= P.tokens_all && rows <= P.tile_rows)) rows = 0;
  const int n = rows * P.experts, t = threadIdx.x;
  if (P.stride != P.experts) {
    T* const to = reinterpret_cast<T*>(tile);
    for (int r = t >> 5; r < rows; r += kWarps)
      for (int e = t & 31; e < P.experts; e += 32) to[r * P.experts + e] = x[r * P.stride + e];
    return to;
  }
  constexpr int kN = 16 / sizeof(T);
  const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(x) & 15u) / static_cast<int>(sizeof(T));
  T* const to = reinterpret_cast<T*>(tile) + shift;  // 16-byte boundaries fall together
  const int head = min(n, (kN - shift) % kN), vecs = (n - head) / kN;
  const unsigned dst = static_cast<unsigned>(__cvta_generic_to_shared(to + head));
  for (int i = t; i < vecs; i += kThreads)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 16 * i), "l"(x + head + i * kN) : "memory");
  if (t < head) to[t] = x[t];
  const int rest = head + vecs * kN;
  if (t < n - rest) to[rest + t] = x[rest + t];
  asm volatile("cp.async.wait_all;" ::: "memory");
  return to;
}

__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }

// Largest entry and sum of a row that `q` neighbouring lanes share, and with A
// the sum weighted by a.
template <typename T, bool A>
__device__ __forceinline__ void row_sums(const T* x, int experts, int q, int part, const float* a, float& m, float& s, float& sa) {
  m = -INFINITY;
#pragma unroll 4
  for (int e = part; e < experts; e += q) m = fmaxf(m, value(x[e]));
  for (int d = q / 2; d > 0; d /= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
  s = sa = 0.0f;
#pragma unroll 4
  for (int e = part; e < experts; e += q) {
    const float p = ex2((value(x[e]) - m) * kLog2e);
    s += p;
    if (A) sa = fmaf(a[e], p, sa);
  }
  for (int d = q / 2; d > 0; d /= 2) {
    s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    if (A) sa += __shfl_xor_sync(0xFFFFFFFFu, sa, d);
  }
}

// NE: experts of a thread, 256 apart.
template <typename T, int NE>
__global__ void __launch_bounds__(kThreads) balance_rows_tile(const __grid_constant__ BalanceParams P) {
  extern __shared__ __align__(16) unsigned char dynamic[];
  __shared__ float2 s_row[kThreads];  // largest entry, 1 / sum (0: left out)
  __shared__ int s_count[NE * kThreads];
  __shared__ float s_acc[kThreads];
  __shared__ int2 s_numbers[kWarps];
  __shared__ float s_sq[kWarps];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int q = kThreads / P.tile_rows, part = t & (q - 1), mine = t / q;
  const long long g = blockIdx.x / P.parts;
  const long long r0 = static_cast<long long>(blockIdx.x % P.parts) * P.cta_rows;
  const long long r1 = min(P.group_rows, r0 + P.cta_rows);
  const long long first = g * P.group_rows;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // balance_finish waits for this grid's end
  if (blockIdx.x == 0 && t == 0) *P.arrived = 0;
  for (int e = t; e < P.experts; e += kThreads) s_count[e] = 0;
  __syncthreads();
  int assigned = 0, tokens = 0;
  const long long i1 = (first + r1) * P.top;
#pragma unroll 8
  for (long long i = (first + r0) * P.top + t; i < i1; i += kThreads) {
    const int64_t e = P.ids[i];
    if (e < 0 || e >= P.experts || (P.mask && !P.mask[static_cast<unsigned>(i) / static_cast<unsigned>(P.top)])) continue;
    atomicAdd(&s_count[e], 1);
    ++assigned;
  }
  // an expert's sum: `width` threads for the experts, the rows dealt over the others
  int width = 32;
  while (width < P.experts && width < kThreads) width *= 2;
  const int e = t & (width - 1), deal = t / width, deals = kThreads / width;
  float acc[NE] = {}, sq = 0.0f;
  for (long long r = r0; r < r1; r += P.tile_rows) {
    const int rows = static_cast<int>(min(static_cast<long long>(P.tile_rows), r1 - r));
    const T* x = load_tile<T>(P, first + r, rows, dynamic);
    __syncthreads();
    const bool in = mine < rows, on = in && (!P.mask || P.mask[first + r + mine]);
    float m, s, unused;
    row_sums<T, false>(x + (in ? mine : 0) * P.experts, P.experts, q, part, nullptr, m, s, unused);
    if (part == 0) {
      s_row[mine] = make_float2(m, on ? 1.0f / s : 0.0f);
      if (on) {
        const float lse = m + logf(s);
        sq += lse * lse;
        ++tokens;
      }
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < NE; ++c) {
      if (e + c * kThreads >= P.experts) continue;
      const T* const from = x + e + c * kThreads;
#pragma unroll 4
      for (int k = deal; k < rows; k += deals) {
        const float2 row = s_row[k];
        const float p = ex2((value(from[k * P.experts]) - row.x) * kLog2e) * row.y;
        acc[c] += row.y != 0.0f ? p : 0.0f;
      }
    }
    __syncthreads();
  }
  s_acc[t] = acc[0];
  sq = warp_sum(sq);
  tokens = warp_sum(tokens);
  assigned = warp_sum(assigned);
  if (lane == 0) s_sq[warp] = sq, s_numbers[warp] = make_int2(tokens, assigned);
  __syncthreads();
  const long long out = static_cast<long long>(blockIdx.x) * P.experts;
#pragma unroll
  for (int c = 0; c < NE; ++c) {
    const int at = t + c * kThreads;
    if (at >= P.experts) continue;
    if (c == 0)  // deals = 1 where there are more experts than threads
      for (int k = 1; k < deals; ++k) acc[0] += s_acc[k * width + t];
    P.sums[out + at] = acc[c];
    P.part_counts[out + at] = s_count[at];
  }
  if (t == 0) {
    float s = 0.0f;
    int2 n = make_int2(0, 0);
    for (int w = 0; w < kWarps; ++w) s += s_sq[w], n.x += s_numbers[w].x, n.y += s_numbers[w].y;
    P.squares[blockIdx.x] = s;
    P.numbers[blockIdx.x] = n;
  }
}

template <typename T, int NE>
__global__ void __launch_bounds__(kThreads) balance_grad_tile(const __grid_constant__ BalanceParams P) {
  extern __shared__ __align__(16) unsigned char dynamic[];
  __shared__ float3 s_row[kThreads];  // largest entry, 1 / sum (0: left out), shift
  __shared__ float s_a[NE * kThreads];
  constexpr int kPerLane = kThreads / 32;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int q = kThreads / P.tile_rows, part = t & (q - 1), mine = t / q;
  const long long g = blockIdx.x / P.parts;
  const long long r0 = static_cast<long long>(blockIdx.x % P.parts) * P.cta_rows;
  const long long r1 = min(P.group_rows, r0 + P.cta_rows);
  const long long first = g * P.group_rows;
  const float gb = *P.grad_balance * P.stats[2], gz = *P.grad_z * P.stats[3];
  for (int e = t; e < P.experts; e += kThreads) s_a[e] = gb * P.weights[g * P.experts + e];
  __syncthreads();
  float a[kPerLane];  // NE = 1
#pragma unroll
  for (int k = 0; k < kPerLane; ++k) a[k] = lane + 32 * k < P.experts ? s_a[lane + 32 * k] : 0.0f;
  for (long long r = r0; r < r1; r += P.tile_rows) {
    const int rows = static_cast<int>(min(static_cast<long long>(P.tile_rows), r1 - r));
    const T* x = load_tile<T>(P, first + r, rows, dynamic);
    __syncthreads();
    const bool in = mine < rows, on = in && (!P.mask || P.mask[first + r + mine]);
    float m, s, sa;
    row_sums<T, true>(x + (in ? mine : 0) * P.experts, P.experts, q, part, s_a, m, s, sa);
    const float inv = 1.0f / s;
    if (part == 0) s_row[mine] = make_float3(m, on ? inv : 0.0f, gz * (m + logf(s)) - sa * inv);
    __syncthreads();
    for (int k = warp; k < rows; k += kWarps) {
      const float3 row = s_row[k];
      T* const o = static_cast<T*>(P.grad) + (first + r + k) * P.grad_stride + lane;
      const T* const from = x + k * P.experts + lane;
      auto entry_ = [&](int c, float weight) {
        const float p = ex2((value(from[32 * c]) - row.x) * kLog2e) * row.y;
        const float v = row.y != 0.0f ? p * (weight + row.z) : 0.0f;
        if constexpr (sizeof(T) == 2) o[32 * c] = __float2bfloat16_rn(v);
        else o[32 * c] = v;
      };
      if constexpr (NE == 1) {
#pragma unroll
        for (int c = 0; c < kPerLane; ++c)
          if (lane + 32 * c < P.experts) entry_(c, a[c]);
      } else {
#pragma unroll 4
        for (int c = 0; lane + 32 * c < P.experts; ++c) entry_(c, s_a[lane + 32 * c]);
      }
    }
    __syncthreads();
  }
}

using KernelPtr = void (*)(BalanceParams);

#define KERNELS(F) F<false, 1>, F<false, 2>, F<false, 4>, F<true, 1>, F<true, 2>, F<true, 4>
// Index: 0, 1, 2 for up to 256, 512, 1024 experts; + 3 for bfloat16.
const KernelPtr kRows[6] = {KERNELS(balance_rows)};
const KernelPtr kGrad[6] = {KERNELS(balance_grad)};
#undef KERNELS
// Index: more than kThreads experts; + 2 for bfloat16.
const KernelPtr kRowsTile[4] = {balance_rows_tile<float, 1>, balance_rows_tile<float, 4>, balance_rows_tile<__nv_bfloat16, 1>,
                                balance_rows_tile<__nv_bfloat16, 4>};
const KernelPtr kGradTile[4] = {balance_grad_tile<float, 1>, balance_grad_tile<float, 4>, balance_grad_tile<__nv_bfloat16, 1>,
                                balance_grad_tile<__nv_bfloat16, 4>};

// The split of the rows: lanes per row, CTAs per group, rows per CTA; and of
// balance_finish: experts of a CTA, CTAs per group.
struct Split {
  int lanes, kernel, parts, width, slices;
  long long group_rows, cta_rows;
};

Split split_of(int64_t tokens, int experts, int64_t groups) {
  Split s;
  s.lanes = 1;
  while (s.lanes < 32 && s.lanes * 8 < experts) s.lanes *= 2;
  s.kernel = experts <= 256 ? 0 : experts <= 512 ? 1 : 2;
  s.group_rows = tokens / groups;
  const int sets = s.kernel < 2 ? 2 : 1;
  const long long pass = static_cast<long long>(kWarps) * (32 / s.lanes);  // rows of a CTA in one set
  const long long most = (s.group_rows + pass - 1) / pass;
  long long parts = (kTargetCtas + groups - 1) / groups;
  if (parts > most) parts = most;
  if (parts < 1) parts = 1;
  s.cta_rows = (s.group_rows + parts - 1) / parts;
  // whole rounds of all sets, unless that leaves SMs without rows
  const long long round = s.cta_rows >= pass * sets ? pass * sets : pass;
  s.cta_rows = (s.cta_rows + round - 1) / round * round;
  if (s.cta_rows < 1) s.cta_rows = 1;
  s.parts = static_cast<int>((s.group_rows + s.cta_rows - 1) / s.cta_rows);
  if (s.parts < 1) s.parts = 1;
  // at least one partial a thread, 32 experts a warp: 131072 x 256 in one group
  // leaves 608 partials an expert: the call takes 60 us over eight CTAs, 86 in
  // one (65536 x 160: 36 and 60; 16384 x 520: 42 and 116)
  s.width = 32;
  while (s.width < kFinishThreads && s.width < experts && kFinishThreads / s.width > s.parts) s.width *= 2;
  s.slices = (experts + s.width - 1) / s.width;
  return s;
}

// Rows of a tile: a power of two, at least 8 (1024 float32 experts: 32 KB).
// Returns the tile's bytes, with room for its shift against 16 bytes.
size_t use_tiles(BalanceParams& P, int size) {
  // the kernels for more experts hold 3 KB more of their own; all stay below 48 KB
  const long long most = kTileBytes - (P.experts > kThreads ? 3 * 1024 : 0);
  P.tile_rows = kThreads;
  while (P.tile_rows > 8 && static_cast<long long>(P.tile_rows) * P.experts * size > most) P.tile_rows /= 2;
  return static_cast<size_t>(P.tile_rows) * P.experts * size + 16;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

struct Layout {
  size_t arrived, sums, counts, tokens, squares, loss, group_squares, total;
};

Layout layout_of(const Split& s, int experts, int64_t groups) {
  const size_t n = static_cast<size_t>(groups) * s.parts;
  Layout l;
  l.arrived = 0;
  l.sums = 256;
  l.counts = l.sums + up256(n * experts * 4);
  l.tokens = l.counts + up256(n * experts * 4);
  l.squares = l.tokens + up256(n * 8);
  l.loss = l.squares + up256(n * 4);
  l.group_squares = l.loss + up256(static_cast<size_t>(groups) * s.slices * 4);
  l.total = l.group_squares + up256(static_cast<size_t>(groups) * 4);
  return l;
}

muon_status_t check_shape(int dtype, int64_t tokens, int experts, int64_t stride, int64_t groups) {
  if (dtype != MUON_BF16 && dtype != MUON_F32) return MUON_ERR_INVALID_ARG;
  if (tokens < 0 || experts < 1 || experts > kMaxExperts || groups < 1 || stride < experts) return MUON_ERR_INVALID_ARG;
  if (tokens % groups != 0) return MUON_ERR_INVALID_ARG;
  if (tokens > INT32_MAX || groups > INT32_MAX || stride > (1LL << 32)) return MUON_ERR_TOO_LARGE;
  const Split s = split_of(tokens, experts, groups);
  if (s.parts * groups > INT32_MAX || s.slices * groups > INT32_MAX) return MUON_ERR_TOO_LARGE;
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
  P.tokens_all = tokens;
  P.group_rows = s.group_rows;
  P.cta_rows = s.cta_rows;
  P.groups = groups;
  P.parts = s.parts;
  P.experts = experts;
  P.top = top;
  P.lanes = s.lanes;
  P.width = s.width;
  P.slices = s.slices;
  const bool vec = experts % 8 == 0 && row_stride * size % 16 == 0 && aligned_to(logits, 16);
  P.arrived = reinterpret_cast<unsigned*>(ws + l.arrived);
  P.sums = reinterpret_cast<float*>(ws + l.sums);
  P.part_counts = reinterpret_cast<int*>(ws + l.counts);
  P.numbers = reinterpret_cast<int2*>(ws + l.tokens);
  P.squares = reinterpret_cast<float*>(ws + l.squares);
  P.group_loss = reinterpret_cast<float*>(ws + l.loss);
  P.group_squares = reinterpret_cast<float*>(ws + l.group_squares);
  P.stats = stats;
  P.counts = counts;
  P.tokens = n_tokens;
  P.mean = mean_probs;
  P.weights = weights;
  cudaStream_t str = static_cast<cudaStream_t>(stream);
  const bool bf16 = dtype == MUON_BF16;
  size_t smem = static_cast<size_t>(kWarps + 1) * experts * 4;
  KernelPtr rows = kRows[s.kernel + (bf16 ? 3 : 0)];
  if (!vec) {
    smem = use_tiles(P, size);
    rows = kRowsTile[(experts > kThreads ? 1 : 0) + (bf16 ? 2 : 0)];
  }
  rows<<<static_cast<unsigned>(s.parts * groups), kThreads, smem, str>>>(P);
  if (cudaGetLastError() != cudaSuccess) return MUON_ERR_CUDA;
  // launched while balance_rows still runs; it waits for that grid's end
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(s.slices * groups));
  cfg.blockDim = dim3(kFinishThreads);
  cfg.stream = str;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, balance_finish, P) == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
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
  P.tokens_all = tokens;
  P.group_rows = s.group_rows;
  P.cta_rows = s.cta_rows;
  P.groups = groups;
  P.parts = s.parts;
  P.experts = experts;
  P.lanes = s.lanes;
  const bool vec = experts % 8 == 0 && row_stride * size % 16 == 0 && grad_stride * size % 16 == 0 && aligned_to(logits, 16) &&
          aligned_to(grad, 16);
  P.stats = const_cast<float*>(stats);
  P.weights = const_cast<float*>(weights);
  P.grad_balance = grad_balance;
  P.grad_z = grad_z;
  const bool bf16 = dtype == MUON_BF16;
  size_t smem = 0;
  KernelPtr rows = kGrad[s.kernel + (bf16 ? 3 : 0)];
  if (!vec) {
    smem = use_tiles(P, size);
    rows = kGradTile[(experts > kThreads ? 1 : 0) + (bf16 ? 2 : 0)];
  }
  rows<<<static_cast<unsigned>(s.parts * groups), kThreads, smem, static_cast<cudaStream_t>(stream)>>>(P);
  return cudaGetLastError() == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
