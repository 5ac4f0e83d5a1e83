// Layer norm over rows with its backward pass.
//
//   s = x + residual (rounded to x's type, where there is a residual),
//   y = (s - mean) rstd w + b,   rstd = 1 / sqrt(mean((s - mean)^2) + eps);
//   with gw = g w and xhat = (s - mean) rstd,
//   grad_x = rstd (gw - mean(gw) - xhat mean(gw xhat)) (+ grad_sum),
//   grad_w = sum over rows of g xhat,   grad_b = sum over rows of g.
//
// A row lives in the registers of W warps, V groups of 8 entries a thread, so
// that it is read once and the variance is taken of differences with the
// mean.  Backward, a thread keeps the same columns for every row of its CTA and
// adds their gradients of weight and bias in registers; each CTA leaves one row
// of partial sums, which norm_columns adds in their order: equal calls give
// equal bits.  Rows wider than the registers hold are read again
// (norm_forward_wide, norm_rows_wide + norm_columns_wide).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "../../include/muon.h"
#include "check.cuh"
#include "host.h"

namespace muon {
namespace {

struct RowParams {
  const void* x;
  const void* residual;   // or null
  const void* grad;
  const void* grad_sum;   // or null
  const void* weight;     // or null (1)
  const void* bias;       // or null (0)
  void* y;                // forward: y; backward: grad_x
  void* sum;              // forward: s, or null
  float* mean;
  float* rstd;
  float* partial;         // backward: parts x 2 x cols
  float* grad_weight;     // or null
  float* grad_bias;       // or null
  float2* rows2;          // wide backward: mean(gw), mean(gw xhat) of each row
  long long sx, sr, sg, sgs, sy, ssum;  // row pitches
  long long rows;
  int cols, parts;
  int weight_f32;
  int vec;                // every row of every array may be read in vectors
  float eps;
};

template <bool BF16>
struct Raw {
  uint4 q[BF16 ? 1 : 2];
};

__device__ __forceinline__ float weight_at(const void* w, int f32, int c) {
  return f32 ? static_cast<const float*>(w)[c] : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[c]);
}

// Column of entry e of a thread's group v: 8 neighbours where rows are read in
// vectors, else neighbours in neighbouring threads.
template <bool VEC, int T>
__device__ __forceinline__ int column(int v, int e, int t) { return VEC ? (v * T + t) * 8 + e : (v * 8 + e) * T + t; }

template <bool BF16, bool VEC, int T>
__device__ __forceinline__ void load(const void* base, long long at, int cols, int v, int t, float (&x)[8]) {
  if constexpr (VEC) {
    const int c = (v * T + t) * 8;
    if (c + 8 <= cols) {
      if constexpr (BF16) {
        const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + at + c);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[2 * k] = __uint_as_float(w[k] << 16);
          x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        }
      } else {
        const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at + c);
        const float4 a = f[0], b = f[1];
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
      }
      return;
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int c = column<VEC, T>(v, e, t);
    x[e] = 0.0f;
    if (c < cols) {
      if constexpr (BF16)
        x[e] = __bfloat162float(static_cast<const __nv_bfloat16*>(base)[at + c]);
      else
        x[e] = static_cast<const float*>(base)[at + c];
    }
  }
}

template <bool BF16, bool VEC, int T>
__device__ __forceinline__ void store(void* base, long long at, int cols, int v, int t, const float (&x)[8]) {
  if constexpr (VEC) {
    const int c = (v * T + t) * 8;
    if (c + 8 <= cols) {
      if constexpr (BF16) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
          w[k] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + at + c) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        float4* f = reinterpret_cast<float4*>(static_cast<float*>(base) + at + c);
        f[0] = make_float4(x[0], x[1], x[2], x[3]);
        f[1] = make_float4(x[4], x[5], x[6], x[7]);
      }
      return;
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int c = column<VEC, T>(v, e, t);
    if (c < cols) {
      if constexpr (BF16)
        static_cast<__nv_bfloat16*>(base)[at + c] = __float2bfloat16_rn(x[e]);
      else
        static_cast<float*>(base)[at + c] = x[e];
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

__device__ __forceinline__ float rounded_sum(float a, float b, bool bf16) {
  const float s = a + b;
  return bf16 ? __bfloat162float(__float2bfloat16_rn(s)) : s;
}

// Sum over the W warps of a row group; `slot`: W floats of shared memory per
// use.  Every use of a row has slots of its own, and a barrier of the group.
template <int W>
__device__ __forceinline__ float row_sum(float v, float* slot, int group, int warp_in) {
  v = warp_sum(v);
  if constexpr (W > 1) {
    if ((threadIdx.x & 31) == 0) slot[warp_in] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(W * 32) : "memory");
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += slot[w];
  }
  return v;
}

template <int W>
__device__ __forceinline__ float2 row_sum2(float a, float b, float2* slot, int group, int warp_in) {
  a = warp_sum(a);
  b = warp_sum(b);
  if constexpr (W > 1) {
    if ((threadIdx.x & 31) == 0) slot[warp_in] = make_float2(a, b);
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(W * 32) : "memory");
    a = b = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float2 s = slot[w];
      a += s.x;
      b += s.y;
    }
  }
  return make_float2(a, b);
}

__host__ __device__ constexpr int threads_of(int w) { return w >= 4 ? 32 * w : 128; }

// Forward: a row group of W warps takes rows one after another.
template <bool BF16, bool VEC, int W, int V>
__global__ void __launch_bounds__(threads_of(W)) norm_forward(const __grid_constant__ RowParams P) {
  constexpr int T = 32 * W, kGroups = threads_of(W) / T;
  __shared__ float slots[kGroups][2][2][W];  // by parity of the row, use
  const int group = threadIdx.x / T, t = threadIdx.x % T, warp_in = t >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const float inv = 1.0f / static_cast<float>(P.cols);
  int parity = 0;
  for (long long r = static_cast<long long>(blockIdx.x) * kGroups + group; r < P.rows;
       r += static_cast<long long>(gridDim.x) * kGroups, parity ^= 1) {
    float x[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) load<BF16, VEC, T>(P.x, r * P.sx, P.cols, v, t, x[v]);
    if (P.residual) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float a[8];
        load<BF16, VEC, T>(P.residual, r * P.sr, P.cols, v, t, a);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[v][e] = rounded_sum(x[v][e], a[e], BF16);
        store<BF16, VEC, T>(P.sum, r * P.ssum, P.cols, v, t, x[v]);
      }
    }
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += x[v][e];  // (zeros past the row's end)
    const float mean = row_sum<W>(s, slots[group][parity][0], group, warp_in) * inv;
    s = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = column<VEC, T>(v, e, t) < P.cols ? x[v][e] - mean : 0.0f;
        s = fmaf(d, d, s);
      }
    const float var = row_sum<W>(s, slots[group][parity][1], group, warp_in) * inv;
    const float rstd = 1.0f / sqrtf(var + P.eps);
    if (t == 0) {
      P.mean[r] = mean;
      P.rstd[r] = rstd;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = column<VEC, T>(v, e, t);
        float w = 1.0f, b = 0.0f;
        if (c < P.cols) {
          if (P.weight) w = weight_at(P.weight, P.weight_f32, c);
          if (P.bias) b = weight_at(P.bias, P.weight_f32, c);
        }
        y[e] = fmaf((x[v][e] - mean) * rstd, w, b);
      }
      store<BF16, VEC, T>(P.y, r * P.sy, P.cols, v, t, y);
    }
  }
}

// Backward: as norm_forward; a CTA leaves one row of partial sums.
template <bool BF16, bool VEC, int W, int V>
__global__ void __launch_bounds__(threads_of(W)) norm_backward(const __grid_constant__ RowParams P) {
  constexpr int T = 32 * W, kGroups = threads_of(W) / T;
  __shared__ float2 slots[kGroups][2][W];
  extern __shared__ float sums[];  // kGroups > 1: [2][V * 8 * T]
  const int group = threadIdx.x / T, t = threadIdx.x % T, warp_in = t >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const float inv = 1.0f / static_cast<float>(P.cols);
  float dw[V][8], db[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[v][e] = db[v][e] = 0.0f;
  int parity = 0;
  for (long long r = static_cast<long long>(blockIdx.x) * kGroups + group; r < P.rows;
       r += static_cast<long long>(gridDim.x) * kGroups, parity ^= 1) {
    const float mean = P.mean[r], rstd = P.rstd[r];
    float g[V][8], h[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      load<BF16, VEC, T>(P.grad, r * P.sg, P.cols, v, t, g[v]);
      load<BF16, VEC, T>(P.x, r * P.sx, P.cols, v, t, h[v]);
    }
    float a = 0.0f, b = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = column<VEC, T>(v, e, t);
        if (c < P.cols) {
          const float xhat = (h[v][e] - mean) * rstd;
          dw[v][e] = fmaf(g[v][e], xhat, dw[v][e]);
          db[v][e] += g[v][e];
          if (P.weight) g[v][e] *= weight_at(P.weight, P.weight_f32, c);
          h[v][e] = xhat;
          a += g[v][e];
          b = fmaf(g[v][e], xhat, b);
        }
      }
    const float2 s = row_sum2<W>(a, b, slots[group][parity], group, warp_in);
    const float c1 = s.x * inv, c2 = s.y * inv;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float o[8];
      if (P.grad_sum) {
        load<BF16, VEC, T>(P.grad_sum, r * P.sgs, P.cols, v, t, o);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = 0.0f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = fmaf(rstd, g[v][e] - c1 - h[v][e] * c2, o[e]);
      store<BF16, VEC, T>(P.y, r * P.sy, P.cols, v, t, o);
    }
  }
  if (!P.partial) return;
  float* out = P.partial + static_cast<long long>(blockIdx.x) * 2 * P.cols;
  if constexpr (kGroups > 1) {
    // the groups' sums, one group after another
    for (int k = 0; k < kGroups; ++k) {
      if (group == k) {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int i = (v * 8 + e) * T + t;
            sums[i] = k ? sums[i] + dw[v][e] : dw[v][e];
            sums[V * 8 * T + i] = k ? sums[V * 8 * T + i] + db[v][e] : db[v][e];
          }
      }
      __syncthreads();
    }
    if (group != 0) return;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dw[v][e] = sums[(v * 8 + e) * T + t];
        db[v][e] = sums[V * 8 * T + (v * 8 + e) * T + t];
      }
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = column<VEC, T>(v, e, t);
      if (c < P.cols && MUON_CHECK(static_cast<int>(blockIdx.x) < P.parts)) {
        out[c] = dw[v][e];
        out[P.cols + c] = db[v][e];
      }
    }
}

// Adds the partial sums: 32 columns a CTA, its 8 warps take parts in turn.
__global__ void __launch_bounds__(256) norm_columns(const __grid_constant__ RowParams P) {
  __shared__ float2 part[8][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = static_cast<int>(blockIdx.x) * 32 + lane;
  float a = 0.0f, b = 0.0f;
  if (c < P.cols) {
#pragma unroll 4
    for (int p = w; p < P.parts; p += 8) {
      const float* row = P.partial + static_cast<long long>(p) * 2 * P.cols;
      a += row[c];
      b += row[P.cols + c];
    }
  }
  part[w][lane] = make_float2(a, b);
  __syncthreads();
  if (w == 0 && c < P.cols) {
    a = b = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      a += part[k][lane].x;
      b += part[k][lane].y;
    }
    if (P.grad_weight) P.grad_weight[c] = a;
    if (P.grad_bias) P.grad_bias[c] = b;
  }
}

// ------------------------------------------------ rows wider than registers
constexpr int kWide = 1024;

__device__ __forceinline__ float block_sum(float v, float* slots) {
  v = warp_sum(v);
  __syncthreads();  // the last use has been read
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(slots[threadIdx.x & 31]);
}

template <bool BF16>
__device__ __forceinline__ float entry(const void* base, long long at) {
  if constexpr (BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(base)[at]);
  return static_cast<const float*>(base)[at];
}

template <bool BF16>
__device__ __forceinline__ void put(void* base, long long at, float v) {
  if constexpr (BF16)
    static_cast<__nv_bfloat16*>(base)[at] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(base)[at] = v;
}

template <bool BF16>
__global__ void __launch_bounds__(kWide) norm_forward_wide(const __grid_constant__ RowParams P) {
  __shared__ float slots[32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const float inv = 1.0f / static_cast<float>(P.cols);
  for (long long r = blockIdx.x; r < P.rows; r += gridDim.x) {
    auto value = [&](int c) {
      const float x = entry<BF16>(P.x, r * P.sx + c);
      return P.residual ? rounded_sum(x, entry<BF16>(P.residual, r * P.sr + c), BF16) : x;
    };
    float s = 0.0f;
    for (int c = threadIdx.x; c < P.cols; c += kWide) {
      const float x = value(c);
      if (P.residual) put<BF16>(P.sum, r * P.ssum + c, x);
      s += x;
    }
    const float mean = block_sum(s, slots) * inv;
    s = 0.0f;
    for (int c = threadIdx.x; c < P.cols; c += kWide) {
      const float d = value(c) - mean;
      s = fmaf(d, d, s);
    }
    const float rstd = 1.0f / sqrtf(block_sum(s, slots) * inv + P.eps);
    if (threadIdx.x == 0) {
      P.mean[r] = mean;
      P.rstd[r] = rstd;
    }
    for (int c = threadIdx.x; c < P.cols; c += kWide) {
      const float w = P.weight ? weight_at(P.weight, P.weight_f32, c) : 1.0f;
      const float b = P.bias ? weight_at(P.bias, P.weight_f32, c) : 0.0f;
      put<BF16>(P.y, r * P.sy + c, fmaf((value(c) - mean) * rstd, w, b));
    }
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kWide) norm_rows_wide(const __grid_constant__ RowParams P) {
  __shared__ float slots[32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const float inv = 1.0f / static_cast<float>(P.cols);
  for (long long r = blockIdx.x; r < P.rows; r += gridDim.x) {
    const float mean = P.mean[r], rstd = P.rstd[r];
    float a = 0.0f, b = 0.0f;
    for (int c = threadIdx.x; c < P.cols; c += kWide) {
      const float w = P.weight ? weight_at(P.weight, P.weight_f32, c) : 1.0f;
      const float g = entry<BF16>(P.grad, r * P.sg + c) * w;
      a += g;
      b = fmaf(g, (entry<BF16>(P.x, r * P.sx + c) - mean) * rstd, b);
    }
    a = block_sum(a, slots);
    b = block_sum(b, slots);
    if (threadIdx.x == 0) P.rows2[r] = make_float2(a * inv, b * inv);
  }
}

// 256 columns a CTA, a share of the rows: gradients of x and partial sums.
template <bool BF16>
__global__ void __launch_bounds__(256) norm_columns_wide(const __grid_constant__ RowParams P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int c = static_cast<int>(blockIdx.x) * 256 + static_cast<int>(threadIdx.x);
  if (c >= P.cols) return;
  const float w = P.weight ? weight_at(P.weight, P.weight_f32, c) : 1.0f;
  const long long per = (P.rows + P.parts - 1) / P.parts;
  const long long r0 = blockIdx.y * per, r1 = min(P.rows, r0 + per);
  float dw = 0.0f, db = 0.0f;
#pragma unroll 4
  for (long long r = r0; r < r1; ++r) {
    const float rstd = P.rstd[r], xhat = (entry<BF16>(P.x, r * P.sx + c) - P.mean[r]) * rstd;
    const float g = entry<BF16>(P.grad, r * P.sg + c);
    const float2 s = P.rows2[r];
    dw = fmaf(g, xhat, dw);
    db += g;
    const float add = P.grad_sum ? entry<BF16>(P.grad_sum, r * P.sgs + c) : 0.0f;
    put<BF16>(P.y, r * P.sy + c, fmaf(rstd, g * w - s.x - xhat * s.y, add));
  }
  if (!P.partial) return;
  float* out = P.partial + static_cast<long long>(blockIdx.y) * 2 * P.cols;
  out[c] = dw;
  out[P.cols + c] = db;
}

// ---------------------------------------------------------------- launches
using KernelPtr = void (*)(RowParams);

struct Choice {
  KernelPtr fn;
  int threads, rows_per_cta, capacity, smem;
};

template <bool BACKWARD, bool BF16, bool VEC, int W, int V>
Choice choice() {
  Choice c;
  if constexpr (BACKWARD)
    c.fn = norm_backward<BF16, VEC, W, V>;
  else
    c.fn = norm_forward<BF16, VEC, W, V>;
  c.threads = threads_of(W);
  c.rows_per_cta = c.threads / (32 * W);
  c.capacity = 32 * W * V * 8;
  c.smem = BACKWARD && c.rows_per_cta > 1 ? 2 * V * 8 * 32 * W * 4 : 0;
  return c;
}

// The narrowest form that holds a row; false: none does.
template <bool BACKWARD, bool BF16, bool VEC>
bool choose(int64_t cols, Choice& out) {
  const Choice all[] = {choice<BACKWARD, BF16, VEC, 1, 1>(), choice<BACKWARD, BF16, VEC, 1, 2>(),
                        choice<BACKWARD, BF16, VEC, 1, 3>(), choice<BACKWARD, BF16, VEC, 1, 4>(),
                        choice<BACKWARD, BF16, VEC, 4, 2>(), choice<BACKWARD, BF16, VEC, 8, 2>(),
                        choice<BACKWARD, BF16, VEC, 16, 2>(), choice<BACKWARD, BF16, VEC, 16, 4>()};
  for (const Choice& c : all)
    if (cols <= c.capacity) {
      out = c;
      return true;
    }
  return false;
}

template <bool BACKWARD>
bool choose(bool bf16, bool vec, int64_t cols, Choice& c) {
  if (bf16) return vec ? choose<BACKWARD, true, true>(cols, c) : choose<BACKWARD, true, false>(cols, c);
  return vec ? choose<BACKWARD, false, true>(cols, c) : choose<BACKWARD, false, false>(cols, c);
}

constexpr int kMaxParts = 608;  // rows of partial sums: four CTAs per SM
constexpr int kWideParts = 64;

cudaError_t launch(const void* fn, dim3 grid, int threads, int smem, const RowParams& P, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[] = {const_cast<RowParams*>(&P)};
  return cudaLaunchKernelExC(&cfg, fn, args);
}

uint64_t matrix_bytes(int64_t rows, int64_t cols, int64_t stride, int size) {
  return rows && cols ? (static_cast<uint64_t>(rows - 1) * stride + cols) * size : 0;
}

bool finite_eps(double eps) { return std::isfinite(eps) && eps >= 0; }

constexpr int64_t kMaxCols = 1 << 24;

muon_status_t check_sizes(int dtype, int weight_dtype, int64_t rows, int64_t cols) {
  if ((dtype != MUON_BF16 && dtype != MUON_F32) || (weight_dtype != MUON_BF16 && weight_dtype != MUON_F32) || rows < 0 ||
      cols < 1)
    return MUON_ERR_INVALID_ARG;
  if (cols > kMaxCols || rows > 0x7FFFFFFF) return MUON_ERR_TOO_LARGE;
  return MUON_OK;
}

}  // namespace

MUON_CHECK_READER(check_failures_layernorm)

}  // namespace muon

using namespace muon;

extern "C" muon_status_t layer_norm(const void* x, int dtype, int64_t rows, int64_t cols, int64_t row_stride,
                                    const void* residual, int64_t residual_stride, const void* weight, const void* bias,
                                    int weight_dtype, float eps, void* y, int64_t y_stride, void* sum,
                                    int64_t sum_stride, float* mean, float* rstd, void* stream) {
  muon_status_t st = check_sizes(dtype, weight_dtype, rows, cols);
  if (st != MUON_OK) return st;
  if (row_stride < cols || y_stride < cols || !finite_eps(eps) || (residual != nullptr) != (sum != nullptr) ||
      (residual && (residual_stride < cols || sum_stride < cols)))
    return MUON_ERR_INVALID_ARG;
  if (std::max({row_stride, y_stride, residual ? residual_stride : 0, residual ? sum_stride : 0}) > (1LL << 32))
    return MUON_ERR_TOO_LARGE;
  if (rows == 0) return MUON_OK;
  if (!x || !y || !mean || !rstd) return MUON_ERR_INVALID_ARG;
  const int size = dtype == MUON_F32 ? 4 : 2, wsize = weight_dtype == MUON_F32 ? 4 : 2;
  if (!aligned_to(x, size) || !aligned_to(y, size) || !aligned_to(residual, size) || !aligned_to(sum, size) ||
      !aligned_to(weight, wsize) || !aligned_to(bias, wsize) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return MUON_ERR_MISALIGNED;
  try {
    // a row is read before it is written: y may be x, sum may be x or residual
    const bool x_written = (!residual && x == y && row_stride == y_stride) || (sum == x && sum_stride == row_stride);
    const bool residual_written = sum == residual && sum_stride == residual_stride;
    std::vector<Span> v = {span_of(x, x_written ? 0 : matrix_bytes(rows, cols, row_stride, size), false),
                           span_of(residual, residual && !residual_written ? matrix_bytes(rows, cols, residual_stride, size) : 0, false),
                           span_of(weight, weight ? cols * wsize : 0, false), span_of(bias, bias ? cols * wsize : 0, false),
                           span_of(y, matrix_bytes(rows, cols, y_stride, size), true),
                           span_of(sum, sum ? matrix_bytes(rows, cols, sum_stride, size) : 0, true),
                           span_of(mean, rows * 4, true), span_of(rstd, rows * 4, true)};
    if (spans_conflict(v)) return MUON_ERR_ALIASING;
  } catch (const std::bad_alloc&) {
    return MUON_ERR_HOST_MEMORY;
  }
  int sms = 0;
  st = device_sms(sms);
  if (st != MUON_OK) return st;
  RowParams P{};
  P.x = x, P.residual = residual, P.weight = weight, P.bias = bias, P.y = y, P.sum = sum, P.mean = mean, P.rstd = rstd;
  P.sx = row_stride, P.sr = residual_stride, P.sy = y_stride, P.ssum = sum_stride;
  P.rows = rows;
  P.cols = static_cast<int>(cols);
  P.weight_f32 = weight_dtype == MUON_F32;
  P.eps = eps;
  auto rows_aligned = [&](const void* p, int64_t stride) { return !p || (aligned_to(p, 16) && stride * size % 16 == 0); };
  const bool vec = rows_aligned(x, row_stride) && rows_aligned(residual, residual_stride) && rows_aligned(y, y_stride) &&
                   rows_aligned(sum, sum_stride);
  cudaStream_t str = static_cast<cudaStream_t>(stream);
  const bool bf16 = dtype == MUON_BF16;
  Choice c;
  cudaError_t e;
  if (choose<false>(bf16, vec, cols, c)) {
    const int64_t ctas = std::min<int64_t>((rows + c.rows_per_cta - 1) / c.rows_per_cta, static_cast<int64_t>(sms) * 64);
    e = launch(reinterpret_cast<const void*>(c.fn), dim3(static_cast<unsigned>(ctas)), c.threads, c.smem, P, str);
  } else {
    e = launch(bf16 ? reinterpret_cast<const void*>(&norm_forward_wide<true>) : reinterpret_cast<const void*>(&norm_forward_wide<false>),
               dim3(static_cast<unsigned>(std::min<int64_t>(rows, sms * 2))), kWide, 0, P, str);
  }
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

extern "C" size_t layer_norm_backward_workspace_size(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 1 || cols > kMaxCols || rows > 0x7FFFFFFF) return 0;
  Choice c;
  const bool wide = !choose<true>(true, true, cols, c);
  return static_cast<size_t>(wide ? kWideParts : kMaxParts) * 2 * cols * 4 + (wide ? static_cast<size_t>(rows) * 8 : 0);
}

extern "C" muon_status_t layer_norm_backward(const void* grad, int64_t grad_stride, const void* x, int64_t row_stride,
                                             int dtype, int64_t rows, int64_t cols, const float* mean, const float* rstd,
                                             const void* weight, int weight_dtype, const void* grad_sum,
                                             int64_t grad_sum_stride, void* grad_x, int64_t grad_x_stride,
                                             float* grad_weight, float* grad_bias, void* workspace,
                                             size_t workspace_bytes, void* stream) {
  muon_status_t st = check_sizes(dtype, weight_dtype, rows, cols);
  if (st != MUON_OK) return st;
  if (row_stride < cols || grad_stride < cols || grad_x_stride < cols || (grad_sum && grad_sum_stride < cols))
    return MUON_ERR_INVALID_ARG;
  if (std::max({row_stride, grad_stride, grad_x_stride, grad_sum ? grad_sum_stride : 0}) > (1LL << 32))
    return MUON_ERR_TOO_LARGE;
  const bool columns = grad_weight || grad_bias;
  Choice c;
  const bool wide = !choose<true>(true, true, cols, c);
  const size_t need = layer_norm_backward_workspace_size(rows, cols);
  if (rows > 0) {
    if (!grad || !x || !mean || !rstd || !grad_x) return MUON_ERR_INVALID_ARG;
    if (columns || wide) {
      if (!workspace) return MUON_ERR_INVALID_ARG;
      if (!aligned_to(workspace, 256)) return MUON_ERR_MISALIGNED;
      if (workspace_bytes < need) return MUON_ERR_WORKSPACE_TOO_SMALL;
    }
  }
  const int size = dtype == MUON_F32 ? 4 : 2, wsize = weight_dtype == MUON_F32 ? 4 : 2;
  if (!aligned_to(grad, size) || !aligned_to(x, size) || !aligned_to(grad_sum, size) || !aligned_to(grad_x, size) ||
      !aligned_to(weight, wsize) || !aligned_to(mean, 4) || !aligned_to(rstd, 4) || !aligned_to(grad_weight, 4) ||
      !aligned_to(grad_bias, 4))
    return MUON_ERR_MISALIGNED;
  try {
    std::vector<Span> v = {span_of(x, matrix_bytes(rows, cols, row_stride, size), false),
                           span_of(mean, rows * 4, false), span_of(rstd, rows * 4, false),
                           span_of(weight, weight ? cols * wsize : 0, false),
                           span_of(grad_x, matrix_bytes(rows, cols, grad_x_stride, size), true),
                           span_of(grad_weight, grad_weight ? cols * 4 : 0, true),
                           span_of(grad_bias, grad_bias ? cols * 4 : 0, true),
                           span_of(workspace, rows > 0 && (columns || wide) ? need : 0, true)};
    // grad_x may be grad, or grad_sum, itself: a row is read before it is written
    if (grad != grad_x || grad_stride != grad_x_stride)
      v.push_back(span_of(grad, matrix_bytes(rows, cols, grad_stride, size), false));
    if (grad_sum && (grad_sum != grad_x || grad_sum_stride != grad_x_stride))
      v.push_back(span_of(grad_sum, matrix_bytes(rows, cols, grad_sum_stride, size), false));
    if (spans_conflict(v)) return MUON_ERR_ALIASING;
  } catch (const std::bad_alloc&) {
    return MUON_ERR_HOST_MEMORY;
  }
  int sms = 0;
  st = device_sms(sms);
  if (st != MUON_OK) return st;
  cudaStream_t str = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if ((grad_weight && cudaMemsetAsync(grad_weight, 0, cols * 4, str) != cudaSuccess) ||
        (grad_bias && cudaMemsetAsync(grad_bias, 0, cols * 4, str) != cudaSuccess))
      return MUON_ERR_CUDA;
    return MUON_OK;
  }
  RowParams P{};
  P.grad = grad, P.x = x, P.grad_sum = grad_sum, P.weight = weight, P.y = grad_x;
  P.mean = const_cast<float*>(mean), P.rstd = const_cast<float*>(rstd);
  P.sg = grad_stride, P.sx = row_stride, P.sgs = grad_sum_stride, P.sy = grad_x_stride;
  P.rows = rows;
  P.cols = static_cast<int>(cols);
  P.weight_f32 = weight_dtype == MUON_F32;
  P.grad_weight = grad_weight, P.grad_bias = grad_bias;
  P.partial = columns ? static_cast<float*>(workspace) : nullptr;
  const bool bf16 = dtype == MUON_BF16;
  cudaError_t e;
  if (!wide) {
    auto rows_aligned = [&](const void* p, int64_t stride) { return !p || (aligned_to(p, 16) && stride * size % 16 == 0); };
    const bool vec = rows_aligned(x, row_stride) && rows_aligned(grad, grad_stride) &&
                     rows_aligned(grad_sum, grad_sum_stride) && rows_aligned(grad_x, grad_x_stride);
    choose<true>(bf16, vec, cols, c);
    P.parts = static_cast<int>(std::min<int64_t>({(rows + c.rows_per_cta - 1) / c.rows_per_cta, sms * 4, kMaxParts}));
    e = launch(reinterpret_cast<const void*>(c.fn), dim3(static_cast<unsigned>(P.parts)), c.threads, c.smem, P, str);
  } else {
    P.rows2 = reinterpret_cast<float2*>(static_cast<char*>(workspace) + static_cast<size_t>(kWideParts) * 2 * cols * 4);
    P.parts = static_cast<int>(std::min<int64_t>(rows, kWideParts));
    e = launch(bf16 ? reinterpret_cast<const void*>(&norm_rows_wide<true>) : reinterpret_cast<const void*>(&norm_rows_wide<false>),
               dim3(static_cast<unsigned>(std::min<int64_t>(rows, sms * 2))), kWide, 0, P, str);
    if (e == cudaSuccess)
      e = launch(bf16 ? reinterpret_cast<const void*>(&norm_columns_wide<true>) : reinterpret_cast<const void*>(&norm_columns_wide<false>),
                 dim3(static_cast<unsigned>((cols + 255) / 256), static_cast<unsigned>(P.parts)), 256, 0, P, str);
  }
  if (e == cudaSuccess && columns)
    e = launch(reinterpret_cast<const void*>(&norm_columns), dim3(static_cast<unsigned>((cols + 31) / 32)), 256, 0, P, str);
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
