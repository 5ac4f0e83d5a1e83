// Layer norm over rows with its backward pass.
//
//   s = x + residual (rounded to x's type, where there is a residual),
//   y = (s - mean) rstd w + b,   rstd = 1 / sqrt(mean((s - mean)^2) + eps);
//   with gw = g w and xhat = (s - mean) rstd,
//   grad_x = rstd (gw - mean(gw) - xhat mean(gw xhat)) (+ grad_sum),
//   grad_w = sum over rows of g xhat,   grad_b = sum over rows of g.
//
// Bound by memory: a row is read once and its results are written once.  What
// stands in the way is latency (two dependent sums over the row) and, at 2
// bytes an entry, the number of instructions.  So
//   - rows are copied to shared memory with cp.async, the next one while this
//     one is worked on (norm_forward, norm_backward), or several rows a CTA at
//     a time (norm_forward_long): no registers are held for what is in flight;
//   - arithmetic is on two numbers at a time (rows.cuh), the weights lie in
//     shared memory as float32, and the variance is taken of differences with the mean;
//   - a row belongs to 4 to 32 lanes of a warp, or 2 to 32 warps, by its length;
//   - rows off 16 bytes at one offset in all arrays (odd lengths, contiguous)
//     are taken in units of memory, the row's entries turned within them; at
//     different offsets, entries move between neighbouring lanes (long rows
//     forward) or between two units in shared memory (rows.cuh).
// Backward, a thread has the same columns in every row and adds their
// gradients of weight and bias in registers; it makes two passes over the row
// in shared memory (its two means, then grad_x).  Each CTA leaves one row of
// partial sums, which norm_columns adds in their order: equal calls give equal
// bits.  Rows that fit into neither are read again: forward past 220 KB (with its
// residual's), and past 16384 entries where the residual begins at another offset
// than x, which norm_forward_long does not turn (3500 x 20000 bfloat16 with a
// residual 154 us at one offset, 250 so; 2000 x 20000 float32 142 and 169); backward past 16384 entries.
//
// Measured, of the measured copy bandwidth: forward 32768 x 1600 bfloat16 with a residual 72 us
// (0.87), 20000 x 2048 float32 59 (0.83), 6000 x 12800 bfloat16 93 (0.50),
// 3001 x 12289 bfloat16 58 (0.38), 40000 x 1601 with a residual 117 (0.66);
// backward 32768 x 1600 with grad_sum 107 (0.59), 20000 x 2048 float32 91 (0.81),
// 3001 x 12289 78 (0.43), 40000 x 1601 with grad_sum 143 (0.54), 3500 x 20000 372 (0.17).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <exception>
#include <iterator>
#include <map>
#include <mutex>
#include <new>
#include <tuple>
#include <vector>

#include "../../include/muon.h"
#include "check.cuh"
#include "host.h"
#include "rows.cuh"

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
  int weight_vec;         // weight and bias begin on 16 bytes
  int units_lane;         // 16-byte units of a row that a lane has (norm_forward_long: of a row)
  int warps;              // norm_forward_long: of a row
  int stages;             // 2: a row is copied while the one before it is worked on
  int weights_shared;     // weight (and bias) are held in shared memory
  float eps;
};

__device__ __forceinline__ float weight_at(const void* w, int f32, int c) {
  return f32 ? static_cast<const float*>(w)[c] : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[c]);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

using rows::Pair;

__device__ __forceinline__ float rounded_sum(float a, float b, bool bf16) {
  const float s = a + b;
  return bf16 ? __bfloat162float(__float2bfloat16_rn(s)) : s;
}

// A row's place in a CTA: L lanes of a warp (several rows a warp), or W whole
// warps, each with a piece of it.  A lane has up to V units of 16 bytes (N entries).
template <bool BF16, int L, int W, int N>
struct Shape {
  static constexpr int kE = rows::Unit<BF16>::n, kV = N / kE;
  static constexpr int kThreads = W > 8 ? 32 * W : 256, kWarps = kThreads / 32;
  static constexpr int kResident = kThreads > 256 ? 1 : 2;  // CTAs per SM that registers are kept for
  static constexpr int kGroups = kWarps / W;       // row groups of W warps
  static constexpr int kRows = 32 / L;             // rows of a warp at a time
  static constexpr int kCapacity = L * W * kV * kE;
};

template <int L>
__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Sums over a row; `slot`: W entries of shared memory.  Every use within a row
// has slots of its own, and so have neighbouring rows.
template <int L, int W>
__device__ __forceinline__ float row_sum(float v, float* slot, int group, int warp_in) {
  v = lane_sum<L>(v);
  if constexpr (W > 1) {
    if ((threadIdx.x & 31) == 0) slot[warp_in] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(W * 32) : "memory");
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += slot[w];
  }
  return v;
}

template <int L, int W>
__device__ __forceinline__ float2 row_sum2(float a, float b, float2* slot, int group, int warp_in) {
  a = lane_sum<L>(a);
  b = lane_sum<L>(b);
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

// Whether a row's spread is so small beside its mean (2^-10) that the mean's own
// rounding shows: the row's sum and 1 / cols are rounded, which leaves the mean
// up to some hundred of its spacings off, and a constant row would seem to have a spread.  Then the
// mean of the differences d with it is added to it, and the squares of the new
// differences are summed: an error of (e mean) becomes one of (e^2 mean), so a
// constant row's mean is the constant.  (Adding up d in every row beside d^2 instead:
// 32768 x 1600 bfloat16 with a residual 75 us in place of 71.)
__device__ __forceinline__ bool hardly_spread(float mean, float var) {
  return isfinite(mean) && mean != 0.0f && var <= mean * mean * 0x1p-20f;
}

template <bool BF16>
__device__ __forceinline__ char* row_of(const void* base, long long r, long long pitch, int c0) {
  return const_cast<char*>(static_cast<const char*>(base)) + (r * pitch + c0) * (BF16 ? 2 : 4);
}

// Weights in shared memory, float32: four-entry parts of a unit apart, so that a
// warp reads whole lines.  `units` of a row, of whose first one `before` entries are in front of it.
template <bool BF16>
__device__ __forceinline__ void stage_weights(uint32_t at, const void* w, int f32, float none, int cols, int units, int thread,
                                              int threads, int before = 0) {
  constexpr int E = rows::Unit<BF16>::n;
  for (int i = thread; i < units * E; i += threads) {
    const int u = i / E, e = i - u * E;
    const float v = w && i >= before && i - before < cols ? weight_at(w, f32, i - before) : none;
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + ((e >> 2) * units + u) * 16 + (e & 3) * 4), "f"(v) : "memory");
  }
}

// VECTORS: not held ones may be read by the vector (norm_forward_long; beside the other kernels' unrolled loops the code
// for it costs more than it gives: gradients of 9000 x 8192 103 us, 152 with it).
template <bool BF16, bool VECTORS = false, bool COMMON = false>
__device__ __forceinline__ void weights(const RowParams& P, uint32_t at, const void* w, float none, int unit, int units,
                                        Pair (&x)[rows::Unit<BF16>::n / 2], int before = 0) {
  constexpr int E = rows::Unit<BF16>::n;
  if (P.weights_shared) {
#pragma unroll
    for (int p = 0; p < E / 4; ++p) {
      const uint4 q = rows::shared_load(at + (p * units + unit) * 16);
      x[2 * p] = rows::pair(__uint_as_float(q.x), __uint_as_float(q.y));
      x[2 * p + 1] = rows::pair(__uint_as_float(q.z), __uint_as_float(q.w));
    }
  } else if (VECTORS && w && P.weight_vec && (unit + 1) * E <= P.cols) {
    if (P.weight_f32) {
#pragma unroll
      for (int p = 0; p < E / 4; ++p) {
        const float4 q = __ldg(static_cast<const float4*>(w) + unit * (E / 4) + p);
        x[2 * p] = rows::pair(q.x, q.y);
        x[2 * p + 1] = rows::pair(q.z, q.w);
      }
    } else {
#pragma unroll
      for (int p = 0; p < E / 4; ++p) {
        const uint2 q = __ldg(static_cast<const uint2*>(w) + unit * (E / 4) + p);
        x[2 * p] = rows::pair(__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xFFFF0000u));
        x[2 * p + 1] = rows::pair(__uint_as_float(q.y << 16), __uint_as_float(q.y & 0xFFFF0000u));
      }
    }
  } else {
    auto at_column = [&](int c) { return w && (!COMMON || c >= 0) && c < P.cols ? weight_at(w, P.weight_f32, c) : none; };
    const int c0 = unit * E - (COMMON ? before : 0);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) x[i] = rows::pair(at_column(c0 + 2 * i), at_column(c0 + 2 * i + 1));
  }
}

// Where rows begin off 16 bytes alike, weights lie by their entry of a unit,
// which turns with the row's offset: lanes read neighbouring words at any offset.
__host__ __device__ constexpr int turned_pitch(int units) { return (units + 31) / 32 * 32 + 4; }

template <bool BF16>
__device__ __forceinline__ void stage_turned(const RowParams& P, uint32_t wa, uint32_t ba, int units) {
  constexpr int E = rows::Unit<BF16>::n;
  const int pitch = turned_pitch(units);
#pragma unroll 4
  for (int i = threadIdx.x; i < units * E; i += blockDim.x) {
    const uint32_t to = ((i % E) * pitch + i / E) * 4;
    const float w = P.weight && i < P.cols ? weight_at(P.weight, P.weight_f32, i) : 1.0f;
    const float b = P.bias && i < P.cols ? weight_at(P.bias, P.weight_f32, i) : 0.0f;
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(wa + to), "f"(w) : "memory");
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(ba + to), "f"(b) : "memory");
  }
}

// Weights and biases of a unit of memory, whose first `before` entries belong to the
// unit in front (any number where that is not the row's).
template <bool BF16>
__device__ __forceinline__ void turned_weights(const RowParams& P, uint32_t wa, uint32_t ba, int unit, int pitch, int before,
                                               Pair (&w)[rows::Unit<BF16>::n / 2], Pair (&b)[rows::Unit<BF16>::n / 2]) {
  constexpr int E = rows::Unit<BF16>::n;
  if (P.weights_shared) {
    float v[2][E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const uint32_t from = (((e - before) & (E - 1)) * pitch + unit - (e < before)) * 4;
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[0][e]) : "r"(wa + from) : "memory");
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[1][e]) : "r"(ba + from) : "memory");
    }
#pragma unroll
    for (int i = 0; i < E / 2; ++i) w[i] = rows::pair(v[0][2 * i], v[0][2 * i + 1]), b[i] = rows::pair(v[1][2 * i], v[1][2 * i + 1]);
  } else {
    auto at_column = [&](const void* p, float none, int e) {
      const int c = unit * E + e - before;
      return p && c >= 0 && c < P.cols ? weight_at(p, P.weight_f32, c) : none;
    };
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      w[i] = rows::pair(at_column(P.weight, 1.0f, 2 * i), at_column(P.weight, 1.0f, 2 * i + 1));
      b[i] = rows::pair(at_column(P.bias, 0.0f, 2 * i), at_column(P.bias, 0.0f, 2 * i + 1));
    }
  }
}

// Where rows begin: anywhere, on 16 bytes, or off them at the same offset in all arrays.
enum Begin : int { kAny, kAligned, kAlike };

// Forward: the row groups of all CTAs take rows in turn.  A lane has its entries of the row in registers from the
// slot on: of three passes over the slot instead, 32768 x 1600 with a residual took 79 us in place of 71.
template <bool BF16, bool ALIGNED, int L, int W, int N>
__global__ void __launch_bounds__(Shape<BF16, L, W, N>::kThreads, Shape<BF16, L, W, N>::kResident) norm_forward(const __grid_constant__ RowParams P) {
  using S = Shape<BF16, L, W, N>;
  constexpr int V = S::kV, E = S::kE, H = E / 2;
  extern __shared__ uint4 dynamic[];
  __shared__ float slots[S::kGroups][2][2][W];  // by parity of the row, use
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / W, warp_in = warp % W, sub = lane % L;
  const int units = P.units_lane * L * W;
  const int unit0 = warp_in * P.units_lane * L, c0 = unit0 * E;  // this warp's piece of a row
  const int piece = P.cols - c0;                                  // entries from there on
  const int n = min(P.units_lane, max(0, (piece + L * E - 1) / (L * E)));
  uint32_t at = rows::shared_address(dynamic);
  const uint32_t wa = at, ba = at + units * E * 4;
  if (P.weights_shared) at += 2 * units * E * 4;
  // slots: [stage][array][warp][row of the warp]
  const uint32_t slot_bytes = (P.units_lane * L + 1) * 16, array_bytes = slot_bytes * S::kRows * S::kWarps;
  const uint32_t stage_bytes = (P.residual ? 2 : 1) * array_bytes;
  at += slot_bytes * (warp * S::kRows + lane / L);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const float inv = 1.0f / static_cast<float>(P.cols);
  const long long step = static_cast<long long>(gridDim.x) * S::kGroups * S::kRows;
  long long r0 = (static_cast<long long>(blockIdx.x) * S::kGroups + group) * S::kRows;
  // this lane's row, here and (`next`) where rows are fetched
  long long r = r0 + lane / L, next = r;
  const char *nx = row_of<BF16>(P.x, next, P.sx, c0), *nr = row_of<BF16>(P.residual, next, P.sr, c0);
  char *py = row_of<BF16>(P.y, r, P.sy, c0), *ps = row_of<BF16>(P.sum, r, P.ssum, c0);
  uint32_t shift_x = rows::shift_of(nx), shift_r = rows::shift_of(nr);
  auto fetch = [&](int stage) {
    if (next - lane / L < P.rows && MUON_CHECK(next >= 0)) {
      const uint32_t to = at + stage * stage_bytes;
      const bool none = L < 32 && next >= P.rows;  // a warp's rows past the last one are zeros
      rows::fetch<BF16, ALIGNED, L, V>(to, none ? row_of<BF16>(P.x, 0, 0, 0) : nx, piece, sub, n, none);
      if (P.residual) rows::fetch<BF16, ALIGNED, L, V>(to + array_bytes, none ? row_of<BF16>(P.residual, 0, 0, 0) : nr, piece, sub, n, none);
    }
    rows::copies_commit();
    next += step;
    nx += step * P.sx * (16 / E);
    nr += step * P.sr * (16 / E);
  };
  const bool ahead = P.stages == 2;
  if (ahead) fetch(0);
  if (P.weights_shared) {
    stage_weights<BF16>(wa, P.weight, P.weight_f32, 1.0f, P.cols, units, threadIdx.x, S::kThreads);
    stage_weights<BF16>(ba, P.bias, P.weight_f32, 0.0f, P.cols, units, threadIdx.x, S::kThreads);
    __syncthreads();
  }
  for (int it = 0; r0 < P.rows; r0 += step, ++it) {
    const int stage = ahead ? it & 1 : 0;
    fetch(ahead ? stage ^ 1 : 0);
    rows::copies_wait(ahead);
    if (!ALIGNED) __syncwarp();
    const bool inside = L == 32 || r < P.rows;
    const int left = inside ? piece : 0;
    const uint32_t slot = at + stage * stage_bytes;
    Pair x[V][H], s = rows::pair(0.0f);
    const uint32_t shift = ALIGNED ? 0u : shift_x;
    if (P.residual) {
      uint4 q[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (v >= n) break;
        const int k = v * L + sub;
        Pair a[H];
        rows::numbers<BF16>(rows::unit<ALIGNED>(slot, shift, k), x[v]);
        rows::numbers<BF16>(rows::unit<ALIGNED>(slot + array_bytes, ALIGNED ? 0u : shift_r, k), a);
#pragma unroll
        for (int i = 0; i < H; ++i) x[v][i] = rows::add(x[v][i], a[i]);
        q[v] = rows::pack<BF16>(x[v]);
        rows::numbers<BF16>(q[v], x[v]);
        if (ALIGNED) rows::store_unit<BF16>(ps, k, left, q[v], inside && v + 1 < n);
      }
      if (!ALIGNED) {
        __syncwarp();  // every lane has read its neighbours' units
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (v < n) rows::shared_store(slot + 16 * (v * L + sub), q[v]);
        __syncwarp();
        rows::store_shifted<BF16, L, V>(slot, ps, left, sub, n);
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (v >= n) break;
        rows::numbers<BF16>(rows::unit<ALIGNED>(slot, shift, v * L + sub), x[v]);
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (v >= n) break;
#pragma unroll
      for (int i = 0; i < H; ++i) s = rows::add(s, x[v][i]);  // (zeros past the row's end)
    }
    float mean = row_sum<L, W>(rows::total(s), slots[group][it & 1][0], group, warp_in) * inv;
    s = rows::pair(0.0f);
    const Pair minus = rows::pair(-mean);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (v >= n) break;
      if ((v + 1) * L * E > piece) {  // (the same in every lane)
#pragma unroll
        for (int i = 0; i < H; ++i) {
          const int c = (v * L + sub) * E + 2 * i;
          float a, b;
          rows::split(x[v][i], a, b);
          x[v][i] = rows::pair(c < piece ? a : mean, c + 1 < piece ? b : mean);
        }
      }
#pragma unroll
      for (int i = 0; i < H; ++i) {
        x[v][i] = rows::add(x[v][i], minus);
        s = rows::fma(x[v][i], x[v][i], s);
      }
    }
    float var = row_sum<L, W>(rows::total(s), slots[group][it & 1][1], group, warp_in) * inv;
    const bool again = hardly_spread(mean, var);  // (the same in all lanes of the row)
    if (L < 32 ? __any_sync(0xFFFFFFFFu, again) : again) {
      s = rows::pair(0.0f);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (v >= n) break;
#pragma unroll
        for (int i = 0; i < H; ++i) s = rows::add(s, x[v][i]);
      }
      // (slots: every warp of the row is past its last sum but one)
      const float off = row_sum<L, W>(rows::total(s), slots[group][it & 1][0], group, warp_in) * inv;
      const float moved = again ? mean + off - mean : 0.0f;
      s = rows::pair(0.0f);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (v >= n) break;
#pragma unroll
        for (int i = 0; i < H; ++i) {
          const int c = (v * L + sub) * E + 2 * i;
          float a, b;
          rows::split(x[v][i], a, b);
          x[v][i] = rows::pair(c < piece ? a - moved : 0.0f, c + 1 < piece ? b - moved : 0.0f);
          s = rows::fma(x[v][i], x[v][i], s);
        }
      }
      const float squares = row_sum<L, W>(rows::total(s), slots[group][it & 1][1], group, warp_in) * inv;
      if (again) mean += off, var = squares;
    }
    const float rstd = 1.0f / sqrtf(var + P.eps);
    if (sub == 0 && warp_in == 0 && r < P.rows) {
      P.mean[r] = mean;
      P.rstd[r] = rstd;
    }
    const Pair scale = rows::pair(rstd);
    if (!ALIGNED) __syncwarp();
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (v >= n) break;
      const int k = v * L + sub;
      Pair w[H], b[H];
      weights<BF16>(P, wa, P.weight, 1.0f, unit0 + k, units, w);
      weights<BF16>(P, ba, P.bias, 0.0f, unit0 + k, units, b);
#pragma unroll
      for (int i = 0; i < H; ++i) x[v][i] = rows::fma(rows::mul(x[v][i], scale), w[i], b[i]);
      if (ALIGNED)
        rows::store_unit<BF16>(py, k, left, rows::pack<BF16>(x[v]), inside && v + 1 < n);
      else
        rows::shared_store(slot + 16 * k, rows::pack<BF16>(x[v]));
    }
    if (!ALIGNED) {
      __syncwarp();
      rows::store_shifted<BF16, L, V>(slot, py, left, sub, n);
      __syncwarp();  // before the slot is filled again
      shift_x = (shift_x + static_cast<uint32_t>(step * P.sx) * (16 / E)) & 15;
      shift_r = (shift_r + static_cast<uint32_t>(step * P.sr) * (16 / E)) & 15;
    }
    r += step;
    py += step * P.sy * (16 / E);
    ps += step * P.ssum * (16 / E);
  }
  rows::copies_wait(0);
}

// Forward for long rows, and for rows off 16 bytes in the same way in all arrays
// (COMMON).  A row stays in shared memory for three passes: W warps a row, one
// row at a time each, and as many rows a CTA as fit, whose copies and barriers
// hide behind one another (two slots a row and half the rows: 3001 x 12289
// bfloat16 66 us, 58 so).  Units are those of memory: nothing moves between
// lanes, a thread reads what it has copied, and entries beside the row are left
// out of its first and last unit.  MOVED: results begin at other offsets than what is read;
// a unit of theirs comes from two neighbouring lanes.
template <bool BF16, bool COMMON, bool MOVED>
__global__ void __launch_bounds__(1024) norm_forward_long(const __grid_constant__ RowParams P) {
  constexpr int E = rows::Unit<BF16>::n, H = E / 2, kSize = 16 / E;
  extern __shared__ uint4 dynamic[];
  __shared__ float slots[2][2][32];  // by parity of the row, use
  const int W = P.warps, T = 32 * W, group = static_cast<int>(threadIdx.x) / T, t = static_cast<int>(threadIdx.x) - group * T;
  const int units = P.units_lane;  // of a row
  uint32_t at = rows::shared_address(dynamic);
  const int pitch = COMMON ? turned_pitch(units) : units;
  const uint32_t wa = at, ba = at + E * pitch * 4;
  if (P.weights_shared) at += 2 * E * pitch * 4;
  const uint32_t array_bytes = units * 16, slot = at + group * (P.residual ? 2 : 1) * array_bytes;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const float inv = 1.0f / static_cast<float>(P.cols);
  const long long step = static_cast<long long>(gridDim.x) * (blockDim.x / T);
  long long r = static_cast<long long>(blockIdx.x) * (blockDim.x / T) + group;
  const int row_bytes = P.cols * kSize;
  auto copy = [&](uint32_t to, const void* base, long long p) {
    const char* from = row_of<BF16>(base, r, p, 0);
    const int shift = COMMON ? static_cast<int>(rows::shift_of(from)) : 0, bytes = row_bytes + shift;
    from -= shift;
#pragma unroll 4
    for (int k = 16 * t; k < bytes; k += 16 * T) rows::copy_ahead(to + k, from + k, min(bytes - k, 16));
  };
  auto fetch = [&] {
    if (r < P.rows && MUON_CHECK(r >= 0)) {
      copy(slot, P.x, P.sx);
      if (P.residual) copy(slot + array_bytes, P.residual, P.sr);
    }
    rows::copies_commit();
  };
  fetch();
  if (P.weights_shared) {
    if constexpr (COMMON) {
      stage_turned<BF16>(P, wa, ba, units);
    } else {
      stage_weights<BF16>(wa, P.weight, P.weight_f32, 1.0f, P.cols, units, threadIdx.x, blockDim.x);
      stage_weights<BF16>(ba, P.bias, P.weight_f32, 0.0f, P.cols, units, threadIdx.x, blockDim.x);
    }
    __syncthreads();
  }
  auto sum_of_row = [&](float v, float* slot) {
    v = warp_sum(v);
    if (W > 1) {
      slot += group * W;
      if ((t & 31) == 0) slot[t >> 5] = v;
      asm volatile("bar.sync %0, %1;" ::"r"(group), "r"(T) : "memory");
      v = 0.0f;
#pragma unroll 4
      for (int w = 0; w < W; ++w) v += slot[w];
    }
    return v;
  };
  for (int it = 0; r < P.rows; ++it) {
    rows::copies_wait(0);
    const int shift = COMMON ? static_cast<int>(rows::shift_of(row_of<BF16>(P.x, r, P.sx, 0))) : 0, before = shift / kSize;
    char* y = row_of<BF16>(P.y, r, P.sy, 0) - shift;
    const int n = before + P.cols, last = (n - 1) / E;  // entries up to the row's end; its last unit
    // entries [from, to) of unit k are the row's
    auto first = [&](int k) { return COMMON && k == 0 ? before : 0; };
    auto end = [&](int k) { return min(n - k * E, E); };
    auto edge = [&](int k) { return k == last || (COMMON && k == 0); };
    auto only = [&](Pair (&x)[H], int k) {
#pragma unroll
      for (int i = 0; i < H; ++i) {
        float a, b;
        rows::split(x[i], a, b);
        x[i] = rows::pair(2 * i >= first(k) && 2 * i < end(k) ? a : 0.0f, 2 * i + 1 >= first(k) && 2 * i + 1 < end(k) ? b : 0.0f);
      }
    };
    auto store = [&](char* p, int k, const uint4& q) {
      if constexpr (MOVED) {
        const int lane = threadIdx.x & 31;
        const uint32_t rel = rows::shift_of(p);
        if (rel != 0) {  // (the same in every lane)
          const uint4 front = make_uint4(__shfl_up_sync(0xFFFFFFFFu, q.x, 1), __shfl_up_sync(0xFFFFFFFFu, q.y, 1),
                                         __shfl_up_sync(0xFFFFFFFFu, q.z, 1), __shfl_up_sync(0xFFFFFFFFu, q.w, 1));
          if (k > last) return;
          const int moved = static_cast<int>(rel) / kSize, left = n + moved - k * E;
          char* unit = p - rel + 16 * k;
          const int from = max(lane == 0 ? moved : 0, before + moved - k * E), to = min(left, E);
          if (from <= 0 && to == E)
            *reinterpret_cast<uint4*>(unit) = rows::funnel(front, q, 16 - rel);
          else
            rows::store_some<BF16>(unit, rows::funnel(front, q, 16 - rel), from, to);
          if (lane == 31 || k == last)
            rows::store_some<BF16>(unit + 16, rows::funnel(q, q, 16 - rel), max(0, before + moved - (k + 1) * E), min(left - E, moved));
          return;
        }
        if (k > last) return;
      }
      if (!edge(k) || (first(k) == 0 && end(k) == E))
        *reinterpret_cast<uint4*>(p + 16 * k) = q;
      else
        rows::store_some<BF16>(p + 16 * k, q, first(k), end(k));
    };
    // (with stores from two lanes a warp goes on together, lanes past the row's end with any numbers)
    auto goes_on = [&](int k) { return MOVED ? k - static_cast<int>(threadIdx.x & 31) <= last : k <= last; };
    Pair s = rows::pair(0.0f);
#pragma unroll 2
    for (int k = t; P.residual ? goes_on(k) : k <= last; k += T) {
      const uint32_t unit = 16 * (MOVED ? min(k, last) : k);
      Pair x[H];
      rows::numbers<BF16>(rows::shared_load(slot + unit), x);
      if (P.residual) {
        Pair a[H];
        rows::numbers<BF16>(rows::shared_load(slot + array_bytes + unit), a);
#pragma unroll
        for (int i = 0; i < H; ++i) x[i] = rows::add(x[i], a[i]);
        const uint4 q = rows::pack<BF16>(x);
        if (!MOVED || k <= last) rows::shared_store(slot + 16 * k, q);
        store(row_of<BF16>(P.sum, r, P.ssum, 0) - shift, k, q);
        if (MOVED && k > last) break;
        rows::numbers<BF16>(q, x);
      }
      if (COMMON && k == 0) only(x, k);
#pragma unroll
      for (int i = 0; i < H; ++i) s = rows::add(s, x[i]);
    }
    float mean = sum_of_row(rows::total(s), slots[it & 1][0]) * inv;
    Pair minus = rows::pair(-mean);
    s = rows::pair(0.0f);
#pragma unroll 2
    for (int k = t; k <= last; k += T) {
      Pair x[H];
      rows::numbers<BF16>(rows::shared_load(slot + 16 * k), x);
#pragma unroll
      for (int i = 0; i < H; ++i) x[i] = rows::add(x[i], minus);
      if (edge(k)) only(x, k);
#pragma unroll
      for (int i = 0; i < H; ++i) s = rows::fma(x[i], x[i], s);
    }
    float var = sum_of_row(rows::total(s), slots[it & 1][1]) * inv;
    if (hardly_spread(mean, var)) {  // (the same in all threads of the row)
#pragma unroll 1
      for (int pass = 0; pass < 2; ++pass) {
        s = rows::pair(0.0f);
#pragma unroll 1
        for (int k = t; k <= last; k += T) {
          Pair x[H];
          rows::numbers<BF16>(rows::shared_load(slot + 16 * k), x);
#pragma unroll
          for (int i = 0; i < H; ++i) x[i] = rows::add(x[i], minus);
          if (edge(k)) only(x, k);
#pragma unroll
          for (int i = 0; i < H; ++i) s = pass ? rows::fma(x[i], x[i], s) : rows::add(s, x[i]);
        }
        // (slots: every warp of the row is past its last sum but one)
        const float q = sum_of_row(rows::total(s), slots[it & 1][pass]) * inv;
        if (pass)
          var = q;
        else
          mean += q, minus = rows::pair(-mean);
      }
    }
    const float rstd = 1.0f / sqrtf(var + P.eps);
    if (t == 0) {
      P.mean[r] = mean;
      P.rstd[r] = rstd;
    }
    const Pair scale = rows::pair(rstd);
#pragma unroll 2
    for (int k = t; goes_on(k); k += T) {
      const int unit = MOVED ? min(k, last) : k;
      Pair x[H], w[H], b[H];
      rows::numbers<BF16>(rows::shared_load(slot + 16 * unit), x);
      if constexpr (COMMON) {
        turned_weights<BF16>(P, wa, ba, unit, pitch, before, w, b);
      } else {
        weights<BF16, true>(P, wa, P.weight, 1.0f, unit, units, w);
        weights<BF16, true>(P, ba, P.bias, 0.0f, unit, units, b);
      }
#pragma unroll
      for (int i = 0; i < H; ++i) x[i] = rows::fma(rows::mul(rows::add(x[i], minus), scale), w[i], b[i]);
      store(y, k, rows::pack<BF16>(x));
    }
    r += step;
    fetch();
  }
}

// Backward: as norm_forward.  The two means are taken in one pass over the row
// in shared memory and the gradient in a second one, so that registers hold the
// columns' sums; a CTA leaves one row of partial sums.
template <bool BF16, int ROWS, int L, int W, int N>
__global__ void __launch_bounds__(Shape<BF16, L, W, N>::kThreads, Shape<BF16, L, W, N>::kResident) norm_backward(const __grid_constant__ RowParams P) {
  using S = Shape<BF16, L, W, N>;
  constexpr int V = S::kV, E = S::kE, H = E / 2;
  constexpr bool COMMON = ROWS == kAlike, ALIGNED = ROWS != kAny;  // (alike: units of memory, as if aligned)
  static_assert(!COMMON || L == 32, "the rows of a warp begin at one offset");
  extern __shared__ uint4 dynamic[];
  __shared__ float2 slots[S::kGroups][2][W];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / W, warp_in = warp % W, sub = lane % L;
  const int units = P.units_lane * L * W;
  const long long step = static_cast<long long>(gridDim.x) * S::kGroups * S::kRows;
  const long long r0_first = (static_cast<long long>(blockIdx.x) * S::kGroups + group) * S::kRows;
  // entries that the row's first unit holds of others: the same in every row of this group
  const int before = COMMON ? static_cast<int>(rows::shift_of(row_of<BF16>(P.x, r0_first, P.sx, 0))) / (16 / E) : 0;
  const int unit0 = warp_in * P.units_lane * L, c0 = unit0 * E - before;
  const int piece = P.cols - c0;
  const int n = min(P.units_lane, max(0, (piece + L * E - 1) / (L * E)));
  uint32_t at = rows::shared_address(dynamic);
  // (alike: a group has weights of its own, moved by what its rows begin with)
  const uint32_t wa = at + (COMMON ? group * units * E * 4 : 0);
  if (P.weights_shared) at += (COMMON ? S::kGroups : 1) * units * E * 4;
  const uint32_t slot_bytes = (P.units_lane * L + 1) * 16, array_bytes = slot_bytes * S::kRows * S::kWarps;
  const uint32_t stage_bytes = (P.grad_sum ? 3 : 2) * array_bytes;
  at += slot_bytes * (warp * S::kRows + lane / L);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const float inv = 1.0f / static_cast<float>(P.cols);
  long long r0 = r0_first;
  float mean = 0.0f, rstd = 0.0f;  // of the row that is fetched
  long long r = r0 + lane / L, next = r;
  const char *nx = row_of<BF16>(P.x, next, P.sx, c0), *ng = row_of<BF16>(P.grad, next, P.sg, c0);
  const char* ns = row_of<BF16>(P.grad_sum, next, P.sgs, c0);
  char* out = row_of<BF16>(P.y, r, P.sy, c0);
  uint32_t shift_x = rows::shift_of(nx), shift_g = rows::shift_of(ng), shift_s = rows::shift_of(ns);
  auto fetch = [&](int stage) {
    if (next - lane / L < P.rows && MUON_CHECK(next >= 0)) {
      const uint32_t to = at + stage * stage_bytes;
      const bool none = L < 32 && next >= P.rows;
      rows::fetch<BF16, ALIGNED, L, V>(to, none ? row_of<BF16>(P.x, 0, 0, 0) : nx, piece, sub, n, none);
      rows::fetch<BF16, ALIGNED, L, V>(to + array_bytes, none ? row_of<BF16>(P.grad, 0, 0, 0) : ng, piece, sub, n, none);
      if (P.grad_sum) rows::fetch<BF16, ALIGNED, L, V>(to + 2 * array_bytes, none ? row_of<BF16>(P.grad_sum, 0, 0, 0) : ns, piece, sub, n, none);
      if (L < 32) mean = rstd = 0.0f;  // (a warp's rows past the last one: xhat is 0)
      if (L == 32 || next < P.rows) {
        mean = P.mean[next];
        rstd = P.rstd[next];
      }
    }
    rows::copies_commit();
    next += step;
    nx += step * P.sx * (16 / E);
    ng += step * P.sg * (16 / E);
    ns += step * P.sgs * (16 / E);
  };
  const bool ahead = P.stages == 2;
  if (ahead) fetch(0);
  if (P.weights_shared) {
    stage_weights<BF16>(wa, P.weight, P.weight_f32, 1.0f, P.cols, units, static_cast<int>(threadIdx.x) - (COMMON ? group * W * 32 : 0),
                        COMMON ? W * 32 : S::kThreads, before);
    __syncthreads();
  }
  // zeros for entries in front of the row
  auto only = [&](int unit, Pair (&x)[H]) {
    if (unit != 0) return;
#pragma unroll
    for (int i = 0; i < H; ++i) {
      float a, b;
      rows::split(x[i], a, b);
      x[i] = rows::pair(2 * i >= before ? a : 0.0f, 2 * i + 1 >= before ? b : 0.0f);
    }
  };
  Pair dw[V][H], db[V][H];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < H; ++i) dw[v][i] = db[v][i] = rows::pair(0.0f);
  for (int it = 0; r0 < P.rows; r0 += step, ++it) {
    const int stage = ahead ? it & 1 : 0;
    if (!ahead) fetch(0);
    // (gradients past the row's end are zeros, and with them all that is added up; so are those of
    // a warp's rows past the last one)
    const Pair minus = rows::pair(-mean), scale = rows::pair(rstd);
    if (ahead) fetch(stage ^ 1);
    rows::copies_wait(ahead);
    if (!ALIGNED) __syncwarp();
    const bool inside = L == 32 || r < P.rows;
    const int left = inside ? piece : 0;
    const uint32_t slot = at + stage * stage_bytes;
    Pair a = rows::pair(0.0f), b = rows::pair(0.0f);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (v >= n) break;
      const int k = v * L + sub;
      Pair x[H], g[H], w[H];
      rows::numbers<BF16>(rows::unit<ALIGNED>(slot, ALIGNED ? 0u : shift_x, k), x);
      rows::numbers<BF16>(rows::unit<ALIGNED>(slot + array_bytes, ALIGNED ? 0u : shift_g, k), g);
      weights<BF16, false, COMMON>(P, wa, P.weight, 1.0f, unit0 + k, units, w, before);
      if (COMMON && v == 0) {
        only(unit0 + k, x);
        only(unit0 + k, g);
      }
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const Pair xhat = rows::mul(rows::add(x[i], minus), scale);
        dw[v][i] = rows::fma(g[i], xhat, dw[v][i]);
        db[v][i] = rows::add(db[v][i], g[i]);
        const Pair gw = rows::mul(g[i], w[i]);
        a = rows::add(a, gw);
        b = rows::fma(gw, xhat, b);
      }
    }
    float2 s = row_sum2<L, W>(rows::total(a), rows::total(b), slots[group][it & 1], group, warp_in);
    // Where mean rstd leaves float32's range the row is constant (else a difference is 2^-25 of the mean at least, and rstd
    // at most sqrt(cols) over it): xhat is 0, but infinite in the zeros beside the row, and times their gradient, 0, NaN.
    // (A select at the row's beginning, for every row: 9000 x 8192 bfloat16 145 us in place of 104.)
    if (isnan(s.y)) {
      float m, q, unused;
      rows::split(minus, m, unused);
      rows::split(scale, q, unused);
      if (isinf(m * q) && !isinf(q)) s.y = 0.0f;
    }
    const Pair c1 = rows::pair(-s.x * inv), c2 = rows::pair(-s.y * inv);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (v >= n) break;
      const int k = v * L + sub;
      Pair x[H], g[H], w[H], o[H];
      rows::numbers<BF16>(rows::unit<ALIGNED>(slot, ALIGNED ? 0u : shift_x, k), x);
      rows::numbers<BF16>(rows::unit<ALIGNED>(slot + array_bytes, ALIGNED ? 0u : shift_g, k), g);
      weights<BF16, false, COMMON>(P, wa, P.weight, 1.0f, unit0 + k, units, w, before);
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const Pair xhat = rows::mul(rows::add(x[i], minus), scale);
        o[i] = rows::fma(xhat, c2, rows::fma(g[i], w[i], c1));
      }
      if (P.grad_sum) {
        rows::numbers<BF16>(rows::unit<ALIGNED>(slot + 2 * array_bytes, ALIGNED ? 0u : shift_s, k), x);
#pragma unroll
        for (int i = 0; i < H; ++i) o[i] = rows::fma(scale, o[i], x[i]);
      } else {
#pragma unroll
        for (int i = 0; i < H; ++i) o[i] = rows::mul(scale, o[i]);
      }
      if (ALIGNED) {
        if (COMMON && v == 0 && before != 0 && unit0 + k == 0)
          rows::store_some<BF16>(out + 16 * k, rows::pack<BF16>(o), before, min(left, E));
        else
          rows::store_unit<BF16>(out, k, left, rows::pack<BF16>(o), inside && v + 1 < n);
      } else {
        __syncwarp();  // the neighbours have read this unit of x
        rows::shared_store(slot + 16 * k, rows::pack<BF16>(o));
      }
    }
    if (!ALIGNED) {
      __syncwarp();
      rows::store_shifted<BF16, L, V>(slot, out, left, sub, n);
      __syncwarp();
      shift_x = (shift_x + static_cast<uint32_t>(step * P.sx) * (16 / E)) & 15;
      shift_g = (shift_g + static_cast<uint32_t>(step * P.sg) * (16 / E)) & 15;
      shift_s = (shift_s + static_cast<uint32_t>(step * P.sgs) * (16 / E)) & 15;
    }
    r += step;
    out += step * P.sy * (16 / E);
  }
  rows::copies_wait(0);
  if (!P.partial) return;
  // the rows of a warp, then the groups one after another in shared memory
  if constexpr (L < 32) {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < H; ++i)
#pragma unroll
        for (int o = L; o < 32; o <<= 1) {
          dw[v][i] = rows::add(dw[v][i], __shfl_xor_sync(0xFFFFFFFFu, dw[v][i], o));
          db[v][i] = rows::add(db[v][i], __shfl_xor_sync(0xFFFFFFFFu, db[v][i], o));
        }
  }
  Pair* sums = reinterpret_cast<Pair*>(dynamic);  // [2][units * H]
  __syncthreads();                                // (every slot and weight has been read)
  for (int q = 0; q < S::kGroups; ++q) {
    if (group == q && lane < L) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (v >= n) break;
        const int c = (unit0 + v * L + sub) * H;
        if constexpr (COMMON) {
          float* column = reinterpret_cast<float*>(dynamic);
#pragma unroll
          for (int i = 0; i < E; ++i) {
            const int at_column = 2 * c + i - before;
            if (at_column < 0 || at_column >= P.cols) continue;
            float w0, w1, b0, b1;
            rows::split(dw[v][i / 2], w0, w1);
            rows::split(db[v][i / 2], b0, b1);
            column[at_column] = (q ? column[at_column] : 0.0f) + (i & 1 ? w1 : w0);
            column[units * E + at_column] = (q ? column[units * E + at_column] : 0.0f) + (i & 1 ? b1 : b0);
          }
          continue;
        }
#pragma unroll
        for (int i = 0; i < H; ++i) {
          sums[c + i] = q ? rows::add(sums[c + i], dw[v][i]) : dw[v][i];
          sums[units * H + c + i] = q ? rows::add(sums[units * H + c + i], db[v][i]) : db[v][i];
        }
      }
    }
    __syncthreads();
  }
  if (!MUON_CHECK(static_cast<int>(blockIdx.x) < P.parts)) return;
  float* to = P.partial + static_cast<long long>(blockIdx.x) * 2 * P.cols;
  const float* all = reinterpret_cast<const float*>(dynamic);
  for (int i = threadIdx.x; i < 2 * P.cols; i += S::kThreads) to[i] = all[i < P.cols ? i : units * E + i - P.cols];
}

// Adds the partial sums: 32 columns a CTA, its warps take parts in turn.
constexpr int kColumnWarps = 32;

__global__ void __launch_bounds__(32 * kColumnWarps) norm_columns(const __grid_constant__ RowParams P) {
  __shared__ float2 part[kColumnWarps][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = static_cast<int>(blockIdx.x) * 32 + lane;
  float a = 0.0f, b = 0.0f;
  if (c < P.cols) {
#pragma unroll 8
    for (int p = w; p < P.parts; p += kColumnWarps) {
      const float* row = P.partial + static_cast<long long>(p) * 2 * P.cols;
      a += row[c];
      b += row[P.cols + c];
    }
  }
  part[w][lane] = make_float2(a, b);
  __syncthreads();
  // a warp a column: its 32 parts
  const float2 q = part[lane][w];
  a = warp_sum(q.x);
  b = warp_sum(q.y);
  const int col = static_cast<int>(blockIdx.x) * 32 + w;
  if (lane == 0 && col < P.cols) {
    if (P.grad_weight) P.grad_weight[col] = a;
    if (P.grad_bias) P.grad_bias[col] = b;
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
    // (a thread reads its own sums again, not x, which they may have taken the place of)
    auto value = [&](int c) { return P.residual ? entry<BF16>(P.sum, r * P.ssum + c) : entry<BF16>(P.x, r * P.sx + c); };
    // The mean over the row; a thread adds up its entries 64 at a time, so that no chain of additions is long.
    auto mean_of = [&](auto number) {
      float s = 0.0f;
      for (int c0 = threadIdx.x; c0 < P.cols; c0 += 64 * kWide) {
        float part = 0.0f;
        for (int c = c0; c < min(P.cols, c0 + 64 * kWide); c += kWide) part += number(c);
        s += part;
      }
      return block_sum(s, slots) * inv;
    };
    auto square = [](float d) { return d * d; };
    float mean = mean_of([&](int c) {
      float x = entry<BF16>(P.x, r * P.sx + c);
      if (P.residual) {
        x = rounded_sum(x, entry<BF16>(P.residual, r * P.sr + c), BF16);
        put<BF16>(P.sum, r * P.ssum + c, x);
      }
      return x;
    });
    float var = mean_of([&](int c) { return square(value(c) - mean); });
    if (hardly_spread(mean, var)) {  // (the same in all threads)
      mean += mean_of([&](int c) { return value(c) - mean; });
      var = mean_of([&](int c) { return square(value(c) - mean); });
    }
    const float rstd = 1.0f / sqrtf(var + P.eps);
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
constexpr int kSmemLimit = 220 * 1024;

struct Form {
  KernelPtr fn;
  int threads, rows_per_cta, capacity;  // capacity: entries of a row
  int lanes, warps, entries;            // lanes of a warp and warps per row, entries of a unit
  bool alike;                           // for rows that begin off 16 bytes alike
};

template <bool BACKWARD, bool BF16, int ROWS, int L, int W, int N = 32>
Form form() {
  using S = Shape<BF16, L, W, N>;
  KernelPtr fn;
  if constexpr (BACKWARD)
    fn = norm_backward<BF16, ROWS, L, W, N>;
  else
    fn = norm_forward<BF16, ROWS == kAligned, L, W, N>;
  // A row that begins off 16 bytes takes up to E - 1 entries more.  One warp has such rows up to 768 entries, as
  // its groups' weights do not fit beside more (30000 x 1001 float32 with grad_sum 179 us, 108 with four warps; 30000 x 515 60 and 76).
  constexpr int kLess = ROWS != kAlike ? 0 : W == 1 ? S::kCapacity / 4 : S::kE - 1;
  return {fn, S::kThreads, S::kGroups * S::kRows, S::kCapacity - kLess, L, W, S::kE, ROWS == kAlike};
}

// The narrowest form that holds a row: 4 lanes up to 128 entries, doubled up to a
// warp (1024), then whole warps (up to 16384).  Null: none does.  Where rows are
// few, a form with one unit a lane, for their latency.  Backward, rows of whole warps
// have 16 entries a lane up to 8192, as the sums of 32 columns leave too few registers
// beside them (32 and 16 a lane: 20000 x 2048 float32 121 and 92 us, 9000 x 8192
// bfloat16 121 and 103, 32768 x 1600 113 and 108, 16384 x 4096 110 and 118).  Forward, 32
// are better throughout (16384 x 4096 68 us, 85 with 16; 64: 104 us in place of 71 for
// 32768 x 1600, as the code outgrows the instruction cache).
template <bool BACKWARD, bool BF16, int ROWS>
const Form* choose(int64_t cols, bool few) {
  constexpr int kHalf = BACKWARD ? 2 : 1, kEntries = 32 / kHalf;
  // (rows that begin alike: one row a warp at least)
  static const Form all[] = {form<BACKWARD, BF16, ROWS == kAlike ? kAny : ROWS, 4, 1>(),
                             form<BACKWARD, BF16, ROWS == kAlike ? kAny : ROWS, 8, 1>(),
                             form<BACKWARD, BF16, ROWS == kAlike ? kAny : ROWS, 16, 1>(),
                             form<BACKWARD, BF16, ROWS, 32, 1>(),
                             form<BACKWARD, BF16, ROWS, 32, 2 * kHalf, kEntries>(),
                             form<BACKWARD, BF16, ROWS, 32, 4 * kHalf, kEntries>(),
                             form<BACKWARD, BF16, ROWS, 32, 8 * kHalf, kEntries>(),
                             form<BACKWARD, BF16, ROWS, 32, 16>()};
  const Form& last = all[std::size(all) - 1];
  const int64_t want = few ? cols * Shape<BF16, 32, 1, 32>::kV : cols;
  for (const Form& f : all)
    if (want <= f.capacity) return &f;
  return cols <= last.capacity ? &last : nullptr;
}

template <bool BACKWARD>
const Form* choose(bool bf16, Begin rows, int64_t cols, bool few) {
  if constexpr (BACKWARD) {
    if (rows == kAlike) return bf16 ? choose<true, true, kAlike>(cols, few) : choose<true, false, kAlike>(cols, few);
  }
  if (bf16) return rows == kAligned ? choose<BACKWARD, true, kAligned>(cols, few) : choose<BACKWARD, true, kAny>(cols, few);
  return rows == kAligned ? choose<BACKWARD, false, kAligned>(cols, few) : choose<BACKWARD, false, kAny>(cols, few);
}

// CTAs of a kernel that an SM holds with so much shared memory; the first
// query on a device raises the kernel's limit there.  0: an error.
int resident(const Form& f, int smem) try {
  static std::mutex mu;
  static std::map<std::tuple<int, KernelPtr, int>, int> known;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> lk(mu);
  int& n = known[{dev, f.fn, smem}];
  if (n == 0) {
    const void* fn = reinterpret_cast<const void*>(f.fn);
    int q = 0;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&q, fn, f.threads, smem) != cudaSuccess)
      return 0;
    n = std::max(q, 1);
  }
  return n;
} catch (const std::exception&) {  // (none crosses a C entry)
  return 0;
}

// How a CTA's shared memory is used for rows of `cols` entries: `arrays` of them
// are copied ahead, `vectors` weights held.  Two stages where they fit; weights
// where they fit beside those.
int layout(RowParams& P, const Form& f, int arrays, int vectors, bool alike) {
  const int lane_entries = f.lanes * f.warps * f.entries;
  P.units_lane = static_cast<int>((P.cols + (alike ? f.entries - 1 : 0) + lane_entries - 1) / lane_entries);
  const int units = P.units_lane * f.lanes * f.warps;
  const int stage = arrays * (P.units_lane * f.lanes + 1) * 16 * (f.threads / f.lanes);
  const int held = vectors * (alike ? f.threads / (32 * f.warps) : 1) * units * f.entries * 4;
  P.stages = 2 * stage <= kSmemLimit ? 2 : 1;
  P.weights_shared = held + P.stages * stage <= kSmemLimit;
  return P.stages * stage + (P.weights_shared ? held : 0);
}

struct Long {
  int threads, groups, smem;
};

// How norm_forward_long takes rows of P.cols entries (`per` a unit).  False: a row does not fit.
// Weights are held where three rows fit beside them (6000 x 12800 bfloat16 93 us,
// 100 read from L2; with a residual, two rows beside them: 161 and 134), or their
// loads would be by the entry (COMMON).  Warps: 32 a CTA, with five units a lane or more (10000 x 4099 with a
// residual 79 us with 2 warps a row, 95 with 4), but more of them where rows are few.
bool long_shape(RowParams& P, int arrays, bool common, int per, int64_t rows, int sms, Long& shape) {
  P.units_lane = static_cast<int>((P.cols + static_cast<int64_t>(common ? per - 1 : 0) + per - 1) / per);
  const int64_t row = static_cast<int64_t>(arrays) * P.units_lane * 16;
  const int64_t held = 2LL * per * (common ? turned_pitch(P.units_lane) : P.units_lane) * 4;
  if (row > kSmemLimit) return false;
  P.weights_shared = held + (common ? 1 : 3) * row <= kSmemLimit;
  const int64_t room = kSmemLimit - (P.weights_shared ? held : 0), fit = std::min<int64_t>(room / row, 32);
  P.warps = 1;
  while (P.warps * fit < 32 && 2 * P.warps * 160 <= P.units_lane) P.warps *= 2;
  while (P.warps < 32 && 2 * P.warps * rows <= 32 * sms && 2 * P.warps * 8 <= P.units_lane) P.warps *= 2;
  const int groups = static_cast<int>(std::min<int64_t>({32 / P.warps, fit, rows}));
  shape = {32 * P.warps * groups, groups, static_cast<int>((P.weights_shared ? held : 0) + groups * row)};
  return true;
}

constexpr int kMaxParts = 608;  // rows of partial sums: four CTAs per SM at most
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
  P.weight_vec = aligned_to(weight, 16) && aligned_to(bias, 16);
  auto rows_aligned = [&](const void* p, int64_t stride) { return !p || (aligned_to(p, 16) && stride * size % 16 == 0); };
  const bool vec = rows_aligned(x, row_stride) && rows_aligned(residual, residual_stride) && rows_aligned(y, y_stride) &&
                   rows_aligned(sum, sum_stride);
  cudaStream_t str = static_cast<cudaStream_t>(stream);
  const bool bf16 = dtype == MUON_BF16;
  cudaError_t e;
  const uint32_t low = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(x)) & 15;
  auto alike = [&](const void* p, int64_t stride) {
    return !p || ((static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15) == low && (stride - row_stride) * size % 16 == 0);
  };
  const bool together = alike(residual, residual_stride), common = !rows_aligned(x, row_stride);
  const bool moved = !alike(y, y_stride) || !alike(sum, sum_stride);
  // Long rows, and rows that begin off 16 bytes alike, if they are not short: 40000 x 1601 bfloat16 with a residual
  // 157 us in the registers, 116 so; 30000 x 515 float32 48 and 39; 100000 x 255 bfloat16 66 and 134.  Results at other
  // offsets (from rows a multiple of 16 bytes apart): 3001 x 12289 78 us and 71, 40000 x 1601 with a residual 157 and 169.
  Long shape{};
  if (together && (vec || moved ? cols > 8192 : cols * size >= 1536) && long_shape(P, residual ? 2 : 1, common, 16 / size, rows, sms, shape)) {
    const KernelPtr fns[2][2][2] = {{{norm_forward_long<false, false, false>, norm_forward_long<false, false, true>},
                                     {norm_forward_long<false, true, false>, norm_forward_long<false, true, true>}},
                                    {{norm_forward_long<true, false, false>, norm_forward_long<true, false, true>},
                                     {norm_forward_long<true, true, false>, norm_forward_long<true, true, true>}}};
    const KernelPtr fn = fns[bf16][common][moved];
    const Form f{fn, shape.threads, shape.groups, 0, 32, P.warps, 16 / size, common};
    const int per_sm = resident(f, shape.smem);
    if (per_sm == 0) return MUON_ERR_CUDA;
    const int64_t ctas = std::min<int64_t>((rows + shape.groups - 1) / shape.groups, static_cast<int64_t>(sms) * per_sm);
    e = launch(reinterpret_cast<const void*>(fn), dim3(static_cast<unsigned>(ctas)), shape.threads, shape.smem, P, str);
  } else if (const Form* f = choose<false>(bf16, vec ? kAligned : kAny, cols, rows <= 2 * sms)) {
    const int smem = layout(P, *f, residual ? 2 : 1, 2, false), per_sm = resident(*f, smem);
    if (per_sm == 0) return MUON_ERR_CUDA;
    const int64_t ctas = std::min<int64_t>((rows + f->rows_per_cta - 1) / f->rows_per_cta, static_cast<int64_t>(sms) * per_sm);
    e = launch(reinterpret_cast<const void*>(f->fn), dim3(static_cast<unsigned>(ctas)), f->threads, smem, P, str);
  } else {
    e = launch(bf16 ? reinterpret_cast<const void*>(&norm_forward_wide<true>) : reinterpret_cast<const void*>(&norm_forward_wide<false>),
               dim3(static_cast<unsigned>(std::min<int64_t>(rows, sms * 2))), kWide, 0, P, str);
  }
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

extern "C" size_t layer_norm_backward_workspace_size(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 1 || cols > kMaxCols || rows > 0x7FFFFFFF) return 0;
  const bool wide = !choose<true>(true, kAny, cols, false);
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
  const bool wide = !choose<true>(true, kAny, cols, false);
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
    const uint32_t low = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(x)) & 15;
    auto alike = [&](const void* p, int64_t stride) {
      return !p || ((static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15) == low && (stride - row_stride) * size % 16 == 0);
    };
    const Begin begin = vec ? kAligned : alike(grad, grad_stride) && alike(grad_sum, grad_sum_stride) && alike(grad_x, grad_x_stride) ? kAlike : kAny;
    const Form* f = choose<true>(bf16, begin, cols, rows <= 2 * sms);
    if (!f) f = choose<true>(bf16, kAny, cols, rows <= 2 * sms);
    const bool turned = begin == kAlike && f->alike;
    const int smem = layout(P, *f, grad_sum ? 3 : 2, 1, turned), per_sm = resident(*f, smem);
    if (per_sm == 0) return MUON_ERR_CUDA;
    int64_t parts = std::min<int64_t>({(rows + f->rows_per_cta - 1) / f->rows_per_cta, static_cast<int64_t>(sms) * per_sm, kMaxParts});
    // a group's rows begin at one offset where a multiple of 8 (float32: 4) rows lies between them
    if (turned) parts = (parts + 7) / 8 * 8;
    P.parts = static_cast<int>(std::min<int64_t>(parts, kMaxParts));
    e = launch(reinterpret_cast<const void*>(f->fn), dim3(static_cast<unsigned>(P.parts)), f->threads, smem, P, str);
  } else {
    P.rows2 = reinterpret_cast<float2*>(static_cast<char*>(workspace) + static_cast<size_t>(kWideParts) * 2 * P.cols * 4);
    P.parts = static_cast<int>(std::min<int64_t>(rows, kWideParts));
    e = launch(bf16 ? reinterpret_cast<const void*>(&norm_rows_wide<true>) : reinterpret_cast<const void*>(&norm_rows_wide<false>),
               dim3(static_cast<unsigned>(std::min<int64_t>(rows, sms * 2))), kWide, 0, P, str);
    if (e == cudaSuccess)
      e = launch(bf16 ? reinterpret_cast<const void*>(&norm_columns_wide<true>) : reinterpret_cast<const void*>(&norm_columns_wide<false>),
                 dim3(static_cast<unsigned>((cols + 255) / 256), static_cast<unsigned>(P.parts)), 256, 0, P, str);
  }
  if (e == cudaSuccess && columns)
    e = launch(reinterpret_cast<const void*>(&norm_columns), dim3(static_cast<unsigned>((cols + 31) / 32)), 32 * kColumnWarps, 0, P, str);
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
