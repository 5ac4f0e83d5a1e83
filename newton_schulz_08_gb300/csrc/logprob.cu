// Log probabilities of given tokens with entropy and top alternatives, and
// the gradient with respect to the logits.
//
// With z = scale x over a row of V logits, m = max z, S = sum exp(z - m) and
// W = sum exp(z - m) (z - m):
//   lse = m + log S,   logprob = z_target - lse,   entropy = log S - W / S,
//   grad_j = scale (gl 1[j = target] - p_j (gl + ge (log p_j + entropy))).
//
// HBM-bound: 2 or 4 bytes read per entry, and as many written for a
// gradient; about five instructions an entry.  The logits of a row are read
// once for whatever a call computes from them:
//   - up to 8 KB (logprob_warp): the row stays in the registers of up to 32
//     lanes, and no warp waits for another;
//   - a score of longer rows streams through registers (logprob_score), over a
//     cluster where rows are few;
//   - the loss keeps longer rows in shared memory (logprob_loss), up to 104 KB a
//     CTA so that two CTAs of an SM overlap one's loads with the other's
//     arithmetic, over a cluster of two where they are longer (or more where
//     rows are few); the CTAs exchange their sums through distributed shared
//     memory.  Rows beyond 208 KB are scored and then read again.
// The backward pass alone knows the sums and is elementwise (logprob_grad).
// Long rows are added up in parts of 16 to 52 entries a lane, and then the parts;
// and where sums show entries far above their reference, a larger one is taken and
// a score's batch, or the loss's row in shared memory, added up again.  2^t t of an
// entry with t far above 0 carries a rounding of that size into the entropy, and
// small shares are lost beside a large one in a long chain: entropies of 130000
// logits with few large shares were 5e-6 off so (rms; the largest 5e-5), and are
// 9e-8 (8e-7).
// Entries of -inf: exponents are held above -1000, where 2^t is 0 and 0 * t
// stays 0.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <vector>

#include "../../include/muon.h"
#include "check.cuh"
#include "host.h"

namespace cg = cooperative_groups;

namespace muon {
namespace {

constexpr int kMaxTop = 32;
constexpr int kMaxCluster = 8;
constexpr int kHeldRanks = 2;             // CTAs that a row's loss is spread over for its length
constexpr int kWarpVecs = 512;            // longest row of logprob_warp in 16-byte vectors
constexpr int kWarpThreads = 256;
constexpr int kWarpCandidates = 256;
constexpr int kWarpFew = 96;              // more than that may be ties
constexpr int kSegmentBytes = 104 * 1024; // of a row in one CTA's shared memory
constexpr int kGradThreads = 256;
constexpr int kGradVecs = 4;              // 16-byte vectors per thread of logprob_grad
constexpr int kCandidates = 256;
constexpr int kHits = 256;
constexpr int kScoreChunks = 16;
constexpr int kTopGroups = 64;
constexpr int kLossStatic = 12 * 1024;    // shared memory of a logprob_loss CTA beside its part of the row, at most
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kFloor = -1000.0f;        // least exponent
constexpr float kLost = 4096.0f;          // an lse beyond it may be off by 2^-12 and more
constexpr float kAbove = 6.0f;            // mean exponent that asks for a larger reference
constexpr float kAboveSum = 64.0f;        // and the sum of a batch: an entry of exponent 6, or many
constexpr float kNear = 65536.0f;         // largest exponent of a reference in the short form for bfloat16
constexpr float kMasked = -1e30f;         // its floor for logits in sums
constexpr float kNearScale = 1e-24f;      // and least scale: the floor's exponent is -10^6

enum Mode { kScore = 0, kLoss = 1, kBackward = 2 };

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
  long long rows, stride, grad_stride;
  int vocab, top;
  float scale;
  int lanes;        // logprob_warp: lanes per row
  int log_ranks;    // logprob_score, logprob_loss: CTAs per row, as a power of two
  int segment;      // logprob_loss: vectors that a CTA has room for
  int group;        // and of them in each of its four groups of copies, a multiple of the threads
  int chunks;       // logprob_grad: CTAs per row
  float near;       // largest exponent of a reference in the short form for bfloat16 (0: none does)
  uint32_t floor2;  // two bfloat16 numbers whose exponent is -2 kNear, for the short form of gradients
};

template <bool BF16>
__device__ __forceinline__ float at(const void* x, long long i) {
  if constexpr (BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(x)[i]);
  else return static_cast<const float*>(x)[i];
}

template <bool BF16>
__device__ __forceinline__ void put(void* x, long long i, float v) {
  if constexpr (BF16) static_cast<__nv_bfloat16*>(x)[i] = __float2bfloat16_rn(v);
  else static_cast<float*>(x)[i] = v;
}

// A 16-byte vector holds 8 or 4 entries.
template <bool BF16>
constexpr int kPer = BF16 ? 8 : 4;

template <bool BF16>
__device__ __forceinline__ void unpack(uint4 q, float (&x)[kPer<BF16>]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (BF16) {
      x[2 * k] = __uint_as_float(w[k] << 16);
      x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    } else {
      x[k] = __uint_as_float(w[k]);
    }
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack(const float (&x)[kPer<BF16>]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (BF16) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
      w[k] = *reinterpret_cast<const uint32_t*>(&b);
    } else {
      w[k] = __float_as_uint(x[k]);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Read once: it goes past L1.
__device__ __forceinline__ uint4 load_once(const uint4* p) {
  uint4 v;
  asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

template <bool BF16>
__device__ __forceinline__ uint4 masked_vector() {
  const uint32_t w = BF16 ? 0xFF80FF80u : 0xFF800000u;  // -inf
  return make_uint4(w, w, w, w);
}

// Largest entry of vectors (NaN left out); bfloat16 in pairs until value().
template <bool BF16>
struct VecMax {
  uint32_t m = BF16 ? 0xFF80FF80u : 0xFF800000u;
  __device__ __forceinline__ void add(uint4 q) {
    if constexpr (BF16) {
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
      __nv_bfloat162 b[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) b[k] = *reinterpret_cast<const __nv_bfloat162*>(&w[k]);
      const __nv_bfloat162 r = __hmax2(__hmax2(*reinterpret_cast<const __nv_bfloat162*>(&m), b[0]),
                                       __hmax2(__hmax2(b[1], b[2]), b[3]));
      m = *reinterpret_cast<const uint32_t*>(&r);
    } else {
      m = __float_as_uint(fmaxf(fmaxf(fmaxf(__uint_as_float(m), __uint_as_float(q.x)), __uint_as_float(q.y)),
                                fmaxf(__uint_as_float(q.z), __uint_as_float(q.w))));
    }
  }
  __device__ __forceinline__ float value() const {
    if constexpr (BF16) return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
    else return __uint_as_float(m);
  }
};

template <bool BF16>
__device__ __forceinline__ float vec_max(uint4 q) {
  VecMax<BF16> m;
  m.add(q);
  return m.value();
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// A number's place in the order of alternatives: larger values first, then
// lower indices; NaN below every number.  0 is below every place.
__device__ __forceinline__ uint32_t ordered(float x) {
  x = isnan(x) ? -INFINITY : x + 0.0f;  // -0 equals 0
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ unsigned long long place(float x, int j) {
  return static_cast<unsigned long long>(ordered(x)) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(j));
}
__device__ __forceinline__ int place_index(unsigned long long p) { return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(p)); }
__device__ __forceinline__ float place_value(unsigned long long p) {
  const uint32_t k = static_cast<uint32_t>(p >> 32);
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// Sums of a row or of a part of it: s = sum 2^t, w = sum 2^t t with
// t = (x - m) scale log2(e).
struct Sums {
  float m, s, w;
};

__device__ __forceinline__ float reference(float m) { return m == -INFINITY ? 0.0f : m; }

// Adds N entries, two at a time (paired float32 instructions).
template <int N>
__device__ __forceinline__ void accumulate(float2& s, float2& w, const float (&x)[N], float ref, float c2) {
  const float2 minus = make_float2(-ref, -ref), scale = make_float2(c2, c2);
#pragma unroll
  for (int k = 0; k < N; k += 2) {
    float2 t = __fmul2_rn(__fadd2_rn(make_float2(x[k], x[k + 1]), minus), scale);
    t = make_float2(max_nan(t.x, kFloor), max_nan(t.y, kFloor));
    const float2 e = make_float2(ex2(t.x), ex2(t.y));
    s = __fadd2_rn(s, e);
    w = __ffma2_rn(e, t, w);
  }
}

// The short form for bfloat16, where the exponent of the reference, ref c2, is
// below kNear: entries are held above a floor in pairs before they are widened
// (whatever the reference, its exponent is one of a power of 0), and the exponent
// is one fused operation of K = -ref c2 (44 instructions a vector against 52).
// K is rounded, by up to 2^-9; that goes into every exponent alike and is taken
// out of the sums (settle) and of the gradient's factors (near_of).
template <bool BF16>
__device__ __forceinline__ bool near_fits(const LogprobParams& P, float ref, float c2) {
  return !BF16 || fabsf(__fmul_rn(-ref, c2)) < P.near;
}

// 2^d for |d| <= 2^-8.
__device__ __forceinline__ float ex2_small(float d) {
  const float x = d * kLn2;
  return fmaf(x, fmaf(x, 0.5f, 1.0f), 1.0f);
}

// Adds a vector.
template <bool BF16>
__device__ __forceinline__ void accumulate_near(float2& s, float2& w, uint4 q, float ref, float c2) {
  if constexpr (BF16) {
    const __nv_bfloat162 floor2 = __floats2bfloat162_rn(kMasked, kMasked);
    uint32_t v[4] = {q.x, q.y, q.z, q.w};
    const float k = __fmul_rn(-ref, c2);
    const float2 scale = make_float2(c2, c2), K = make_float2(k, k);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 b = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&v[k]), floor2);
      v[k] = *reinterpret_cast<const uint32_t*>(&b);
      const float2 t = __ffma2_rn(make_float2(__uint_as_float(v[k] << 16), __uint_as_float(v[k] & 0xFFFF0000u)), scale, K);
      const float2 e = make_float2(ex2(t.x), ex2(t.y));
      s = __fadd2_rn(s, e);
      w = __ffma2_rn(e, t, w);
    }
  } else {
    float x[4];
    unpack<false>(q, x);
    accumulate(s, w, x, ref, c2);
  }
}

// What the exponents of accumulate_near were short of, -(ref c2 + K): one fused
// operation gives it exactly.
template <bool BF16>
__device__ __forceinline__ float near_residue(float ref, float c2) {
  return BF16 ? -fmaf(ref, c2, __fmul_rn(-ref, c2)) : 0.0f;
}

// Sums of accumulate_near against a.m become what they stand for.
template <bool BF16>
__device__ __forceinline__ void settle(Sums& a, float c2) {
  if constexpr (BF16) {
    const float d = near_residue<BF16>(reference(a.m), c2), f = ex2_small(d);
    a.w = fmaf(d, a.s, a.w) * f;
    a.s *= f;
  }
}

__device__ __forceinline__ Sums merge(const Sums& a, const Sums& b, float c2) {
  Sums r;
  r.m = fmaxf(a.m, b.m);
  const float ref = reference(r.m);
  const float ta = max_nan((a.m - ref) * c2, kFloor), tb = max_nan((b.m - ref) * c2, kFloor);
  const float fa = ex2(ta), fb = ex2(tb);
  r.s = a.s * fa + b.s * fb;
  r.w = fmaf(a.s, ta, a.w) * fa + fmaf(b.s, tb, b.w) * fb;
  return r;
}

// Sums that accumulate_near has taken against `from` become those against `to`.
template <bool BF16>
__device__ __forceinline__ void move_reference(float2& s, float2& w, float from, float to, float c2) {
  const float t = max_nan((from - to) * c2 + (near_residue<BF16>(from, c2) - near_residue<BF16>(to, c2)), kFloor), f = ex2(t);
  w = __fmul2_rn(__ffma2_rn(s, make_float2(t, t), w), make_float2(f, f));
  s = __fmul2_rn(s, make_float2(f, f));
}

// What follows from a row's sums.
struct RowStats {
  float m, log_s, entropy, lse;
  bool empty;  // every entry -inf
};

// d: of sums that are not settled.  It multiplies S and moves W / S alike.
__device__ __forceinline__ RowStats stats_of(const Sums& a, float scale, float d = 0.0f) {
  RowStats r;
  r.empty = a.s == 0.0f;
  r.m = reference(a.m);
  r.log_s = r.empty ? 0.0f : logf(a.s);
  r.entropy = r.empty ? 0.0f : r.log_s - kLn2 * (a.w / a.s);
  r.log_s = fmaf(d, kLn2, r.log_s);
  r.lse = r.empty ? -INFINITY : fmaf(r.m, scale, r.log_s);
  return r;
}

__device__ __forceinline__ float logprob_of(const RowStats& r, float x, float scale) {
  const float v = r.empty ? -INFINITY : (x - r.m) * scale - r.log_s;
  return v > 0.0f ? 0.0f : v;  // rounding alone takes the logarithm of a share above 0
}

// The gradient of a row: with d = log p_j = (x_j - m) scale - log_s,
// grad_j = exp(d) (a d + b) [+ at_target at the target].
struct RowGrad {
  float m, log_s, a, b, at_target;
};

__device__ __forceinline__ RowGrad grad_of(const LogprobParams& P, const RowStats& r, float gl, float ge, int64_t target) {
  RowGrad g;
  if (target >= P.vocab) gl = NAN;
  g.m = r.m;
  g.log_s = r.log_s;
  g.a = r.empty ? 0.0f : -P.scale * ge;
  g.b = r.empty ? 0.0f : -P.scale * (gl + ge * r.entropy);
  if (isnan(r.log_s) || target >= P.vocab) g.b = NAN;
  g.at_target = r.empty ? 0.0f : P.scale * gl;
  return g;
}

// What the backward pass knows of a row.
__device__ __forceinline__ RowStats stats_from_lse(const LogprobParams& P, long long row) {
  RowStats r;
  r.lse = P.lse[row];
  r.empty = r.lse == -INFINITY;
  r.m = 0.0f;
  r.log_s = r.empty ? 0.0f : r.lse;
  r.entropy = P.ge ? P.entropy[row] : 0.0f;
  return r;
}

// Whether lse is so large beside log S (a row far from zero, masked as a whole,
// or at a low temperature) that probabilities taken from it would be off by its
// rounding: up to kLost by 2^-13 of themselves at most (a thirty-second of what
// rounding to bfloat16 may do), beyond by more, in the end altogether.
// An infinite lse is that of an empty row or a product beyond float32's range.
__device__ __forceinline__ bool log_s_is_lost(const RowStats& r) { return fabsf(r.lse) > kLost; }

// x[k], entries j .. j+N-1 of the row, become their gradients.
template <int N>
__device__ __forceinline__ void grad_entries(const RowGrad& g, float scale, int64_t target, int j, float (&x)[N]) {
  const float2 minus = make_float2(-g.m, -g.m), z = make_float2(scale, scale), log_s = make_float2(-g.log_s, -g.log_s);
  const float2 a = make_float2(g.a, g.a), b = make_float2(g.b, g.b), log2e = make_float2(kLog2e, kLog2e);
#pragma unroll
  for (int k = 0; k < N; k += 2) {
    float2 d = __ffma2_rn(__fadd2_rn(make_float2(x[k], x[k + 1]), minus), z, log_s);
    d = make_float2(max_nan(d.x, kFloor), max_nan(d.y, kFloor));
    const float2 t = __fmul2_rn(d, log2e);
    const float2 v = __fmul2_rn(make_float2(ex2(t.x), ex2(t.y)), __ffma2_rn(a, d, b));
    x[k] = v.x;
    x[k + 1] = v.y;
  }
  const unsigned long long at = static_cast<unsigned long long>(target - j);
  if (at < N) {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (at == k) x[k] += g.at_target;
  }
}

// The same for a vector.  bfloat16 in the short form, t = log2 p_j in one fused operation;
// the floor follows the scale, so that a2 t stays finite (0 times it is 0).
struct NearGrad {
  float c2, K, a2, b;  // t = x c2 + K, grad = 2^t (a2 t + b)
  bool fits;
};

template <bool BF16>
__device__ __forceinline__ NearGrad near_of(const LogprobParams& P, const RowGrad& g) {
  NearGrad h;
  const float l = g.log_s * kLog2e;
  h.c2 = P.scale * kLog2e;
  h.K = -fmaf(g.m, h.c2, l);
  h.fits = !BF16 || fabsf(h.K) < P.near;
  // log2 p_j is t + d, as K is rounded; the difference from m c2 is exact but for a rounding of the size of l
  const float d = -(fmaf(g.m, h.c2, h.K) + l), f = ex2_small(d), a2 = g.a * kLn2;
  h.a2 = a2 * f;
  h.b = fmaf(a2, d, g.b) * f;
  return h;
}

template <bool BF16>
__device__ __forceinline__ uint4 grad_near(const LogprobParams& P, const RowGrad& g, const NearGrad& h, int64_t target, int j, uint4 q) {
  float x[kPer<BF16>];
  if constexpr (BF16) {
    uint32_t v[4] = {q.x, q.y, q.z, q.w};
    const float2 c2 = make_float2(h.c2, h.c2), K = make_float2(h.K, h.K), a2 = make_float2(h.a2, h.a2), b = make_float2(h.b, h.b);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 f = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&v[k]), *reinterpret_cast<const __nv_bfloat162*>(&P.floor2));
      v[k] = *reinterpret_cast<const uint32_t*>(&f);
      const float2 t = __ffma2_rn(make_float2(__uint_as_float(v[k] << 16), __uint_as_float(v[k] & 0xFFFF0000u)), c2, K);
      const float2 e = __fmul2_rn(make_float2(ex2(t.x), ex2(t.y)), __ffma2_rn(a2, t, b));
      x[2 * k] = e.x;
      x[2 * k + 1] = e.y;
    }
    const unsigned long long at = static_cast<unsigned long long>(target - j);
    if (at < 8) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (at == k) x[k] += g.at_target;
    }
  } else {
    unpack<false>(q, x);
    grad_entries(g, P.scale, target, j, x);
  }
  return pack<BF16>(x);
}

__device__ __forceinline__ float grad_entry(const RowGrad& g, float scale, int64_t target, int j, float x) {
  const float d = max_nan(fmaf(x - g.m, scale, -g.log_s), kFloor);
  return ex2(d * kLog2e) * fmaf(g.a, d, g.b) + (j == target ? g.at_target : 0.0f);
}

// The 16-byte vectors of a row, counted from the 16-byte boundary at or below
// its first entry; `shift` entries of the first vector lie before the row.
template <bool BF16>
struct RowVectors {
  const unsigned char* base;
  int shift, count, vocab;
  __device__ __forceinline__ RowVectors(const void* x, long long offset, int vocab_) : vocab(vocab_) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(x) + static_cast<uintptr_t>(offset) * (BF16 ? 2 : 4);
    base = reinterpret_cast<const unsigned char*>(a & ~static_cast<uintptr_t>(15));
    shift = static_cast<int>(a & 15) / (BF16 ? 2 : 4);
    count = static_cast<unsigned>(shift + vocab + kPer<BF16> - 1) / kPer<BF16>;
  }
  __device__ __forceinline__ int first(int v) const { return v * kPer<BF16> - shift; }  // index of the vector's first entry
  __device__ __forceinline__ bool whole(int v) const { return first(v) >= 0 && first(v) + kPer<BF16> <= vocab; }
  // A vector at an end of the row from its entries; what lies outside counts as masked.
  __device__ __noinline__ uint4 end(int v) const {
    float x[kPer<BF16>];
#pragma unroll
    for (int k = 0; k < kPer<BF16>; ++k) {
      const int j = first(v) + k;
      x[k] = j >= 0 && j < vocab ? at<BF16>(base, v * static_cast<long long>(kPer<BF16>) + k) : -INFINITY;
    }
    return pack<BF16>(x);
  }
  // The same from what the vector holds.
  __device__ __noinline__ uint4 mask(int v, uint4 q) const {
    float x[kPer<BF16>];
    unpack<BF16>(q, x);
#pragma unroll
    for (int k = 0; k < kPer<BF16>; ++k) {
      const int j = first(v) + k;
      if (j < 0 || j >= vocab) x[k] = -INFINITY;
    }
    return pack<BF16>(x);
  }
};

// A vector of entries that begin anywhere (rows of logits and gradient that
// fall differently: the gradient is stored in vectors, the logits are read in
// words).  An odd place of bfloat16 reads the entry before and the one after.
// Backward of 2398 x 114679 bfloat16: 208 us so, 167 where rows fall alike; of
// 4096 x 32001 float32 160 (entry by entry 166).
template <bool BF16>
__device__ __forceinline__ uint4 unaligned(const void* x, long long i) {
  if constexpr (BF16) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(static_cast<const __nv_bfloat16*>(x) + i);
    const uint32_t* w = reinterpret_cast<const uint32_t*>(a & ~static_cast<uintptr_t>(3));
    uint4 q = make_uint4(w[0], w[1], w[2], w[3]);
    if (a & 2) q = make_uint4(__byte_perm(q.x, q.y, 0x5432), __byte_perm(q.y, q.z, 0x5432), __byte_perm(q.z, q.w, 0x5432),
                              __byte_perm(q.w, w[4], 0x5432));
    return q;
  } else {
    const uint32_t* w = static_cast<const uint32_t*>(x) + i;
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// --------------------------------------------------- rows in registers (warps)

// Has what is computed from q computed again rather than kept in registers.
__device__ __forceinline__ void anew(uint4& q) { asm volatile("" : "+r"(q.x), "+r"(q.y), "+r"(q.z), "+r"(q.w)); }

// The entries of a vector that lie inside the row, one by one.
template <bool BF16>
__device__ __noinline__ void store_entries(void* grad, long long out, int j, int vocab, uint4 y) {
  float x[kPer<BF16>];
  unpack<BF16>(y, x);
#pragma unroll
  for (int k = 0; k < kPer<BF16>; ++k)
    if (j + k >= 0 && j + k < vocab) put<BF16>(grad, out + j + k, x[k]);
}

// Collected places of one warp, and of its first entries in order.
struct WarpTop {
  unsigned long long candidate[kWarpCandidates];
  unsigned long long top[kMaxTop];
};

// The `top` first places of a row that a whole warp holds, into S.top, found
// as described at TopScratch with the halves of a lane's entries as groups;
// false where more entries reach the bound than there is room for, ties apart.
template <bool BF16, int NV>
__device__ __forceinline__ bool warp_top(const LogprobParams& P, const RowVectors<BF16>& R, uint4 (&q)[NV], int lane, WarpTop& S) {
  constexpr int kN = kPer<BF16>;
  const unsigned before = (1u << lane) - 1;
  float half[2] = {-INFINITY, -INFINITY};
  if constexpr (NV == 1) {
    constexpr uint32_t kNone = BF16 ? 0xFF80FF80u : 0xFF800000u;
    half[0] = vec_max<BF16>(make_uint4(q[0].x, q[0].y, kNone, kNone));
    half[1] = vec_max<BF16>(make_uint4(q[0].z, q[0].w, kNone, kNone));
  } else {
#pragma unroll
    for (int u = 0; u < NV; ++u) half[u & 1] = fmaxf(half[u & 1], vec_max<BF16>(q[u]));
  }
  uint32_t bound = 0, left[2] = {ordered(half[0]), ordered(half[1])};
  for (int k = 0; k < P.top; ++k) {  // one maximum after the other (32 of them take less than ranking all 64 by counting)
    const uint32_t own = max(left[0], left[1]);
    bound = __reduce_max_sync(0xFFFFFFFFu, own);
    if (lane == __ffs(__ballot_sync(0xFFFFFFFFu, own == bound)) - 1) (left[0] == bound ? left[0] : left[1]) = 0;
  }
  int n = 0;  // the same in every lane
  auto add = [&](bool on, float x, int j) {
    const unsigned m = __ballot_sync(0xFFFFFFFFu, on);
    const int i = n + __popc(m & before);
    if (on && i < kWarpCandidates) S.candidate[i] = place(x, j);
    n += __popc(m);
  };
  int pass = 0;
#pragma unroll 1
  for (;; ++pass) {
    const float least = place_value(static_cast<unsigned long long>(bound) << 32);
    n = 0;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      anew(q[u]);  // what depends on it is not kept for the other pass
      unsigned hits = __ballot_sync(0xFFFFFFFFu, vec_max<BF16>(q[u]) >= least);
      if (__popc(hits) > 16) {  // an entry of every lane at a time
        float x[kN];
        unpack<BF16>(q[u], x);
#pragma unroll
        for (int k = 0; k < kN; ++k) {
          const int j = R.first(lane + 32 * u) + k;
          add(j >= 0 && j < P.vocab && ordered(x[k]) >= bound, x[k], j);
        }
        continue;
      }
      for (; hits != 0; hits &= hits - 1) {  // one vector after the other, an entry a lane
        const int from = __ffs(hits) - 1;
        const uint32_t w[4] = {__shfl_sync(0xFFFFFFFFu, q[u].x, from), __shfl_sync(0xFFFFFFFFu, q[u].y, from),
                               __shfl_sync(0xFFFFFFFFu, q[u].z, from), __shfl_sync(0xFFFFFFFFu, q[u].w, from)};
        const int word = BF16 ? lane >> 1 & 3 : lane & 3;
        const uint32_t both = word < 2 ? (word == 0 ? w[0] : w[1]) : (word == 2 ? w[2] : w[3]);
        const float x = __uint_as_float(!BF16 ? both : lane & 1 ? both & 0xFFFF0000u : both << 16);
        const int j = R.first(from + 32 * u) + lane;
        add(lane < kN && j >= 0 && j < P.vocab && ordered(x) >= bound, x, j);
      }
    }
    if (n <= kWarpFew || pass == 1) break;
    ++bound;  // what is above it, then the first of the equal entries
  }
  if (n > kWarpCandidates) return false;
  if (pass == 1) {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      if (n >= P.top) continue;  // the same in every lane
      float x[kN];
      unpack<BF16>(q[u], x);
      unsigned ties = 0;
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        const int j = R.first(lane + 32 * u) + k;
        ties |= static_cast<unsigned>(j >= 0 && j < P.vocab && ordered(x[k]) == bound - 1) << k;
      }
      int upto = __popc(ties);
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
        if (lane >= d) upto += o;
      }
      int i = n + upto - __popc(ties);
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        if (!(ties >> k & 1)) continue;
        if (i < P.top) S.candidate[i] = place(x[k], R.first(lane + 32 * u) + k);
        ++i;
      }
      n += __shfl_sync(0xFFFFFFFFu, upto, 31);
      if (n > P.top) n = P.top;
    }
  }
  __syncwarp();
  for (int i = lane; i < n; i += 32) {
    const unsigned long long mine = S.candidate[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += S.candidate[j] > mine;
    if (rank < P.top) S.top[rank] = mine;
  }
  __syncwarp();
  return true;
}

template <bool BF16, int NV, int MODE>
__global__ void __launch_bounds__(kWarpThreads, NV == 16 ? 2 : NV == 8 ? 3 : 4) logprob_warp(const __grid_constant__ LogprobParams P) {
  constexpr int kN = kPer<BF16>;
  __shared__ WarpTop S[MODE == kBackward ? 1 : kWarpThreads / 32];
  const int lane = threadIdx.x & 31, sub = lane & (P.lanes - 1), rows_warp = 32 / P.lanes;
  const long long row = (static_cast<long long>(blockIdx.x) * (kWarpThreads / 32) + (threadIdx.x >> 5)) * rows_warp + lane / P.lanes;
  const bool in = row < P.rows;
  // every load is issued before the first one is waited for, the logits of
  // rows that are left out among them
  const int64_t target = in ? P.targets[row] : -1;
  float gl = 0.0f, ge = 0.0f;
  if (MODE != kScore && in) gl = P.gl[row], ge = P.ge ? P.ge[row] : 0.0f;
  const bool on = target >= 0;
  const RowVectors<BF16> R(P.x, in ? row * P.stride : 0, P.vocab);
  const int lo = R.shift > 0 ? 1 : 0;  // the vectors inside the row: lo .. lo+wholes-1
  const int wholes = max(0, static_cast<int>(static_cast<unsigned>(R.shift + P.vocab) / kN) - lo);
  // A vector at an end of the row is read whole where what it holds of other
  // rows or of the gap between rows lies inside the matrix (what another warp
  // may be writing there is masked): all loads of the row are in flight at once
  const unsigned char* const x0 = static_cast<const unsigned char*>(P.x);
  const unsigned char* const x1 = x0 + ((P.rows - 1) * P.stride + P.vocab) * (BF16 ? 2 : 4);
  const int from = R.base < x0 ? 1 : 0;
  const unsigned safe = in ? max(0, R.count - from - (R.base + R.count * 16LL > x1 ? 1 : 0)) : 0;
  uint4 q[NV];
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int v = sub + P.lanes * u;
    q[u] = masked_vector<BF16>();
    if (static_cast<unsigned>(v - from) < safe) q[u] = *reinterpret_cast<const uint4*>(R.base + v * 16LL);
    else if (in && v < R.count) q[u] = R.end(v);
  }
  float x_target = 0.0f;
  if (MODE != kBackward && on && target < P.vocab) x_target = at<BF16>(P.x, row * P.stride + target);
  if (wholes < R.count) {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int v = sub + P.lanes * u;
      if (static_cast<unsigned>(v - lo) >= static_cast<unsigned>(wholes) && v < R.count) q[u] = R.mask(v, q[u]);
    }
  }
  RowStats r{};
  if (MODE == kBackward && on) r = stats_from_lse(P, row);
  if (MODE != kBackward || __any_sync(0xFFFFFFFFu, on && log_s_is_lost(r))) {
    Sums a{-INFINITY, 0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < NV; ++u) a.m = fmaxf(a.m, vec_max<BF16>(q[u]));
    for (int d = P.lanes / 2; d > 0; d /= 2) a.m = fmaxf(a.m, __shfl_xor_sync(0xFFFFFFFFu, a.m, d));
    const float c2 = P.scale * kLog2e;
    auto add_up = [&](Sums& a, auto add) {
      float2 s{}, w{};
#pragma unroll
      for (int u = 0; u < NV; ++u) add(s, w, q[u]);
      a.s = s.x + s.y;
      a.w = w.x + w.y;
      for (int d = P.lanes / 2; d > 0; d /= 2) {
        a.s += __shfl_xor_sync(0xFFFFFFFFu, a.s, d);
        a.w += __shfl_xor_sync(0xFFFFFFFFu, a.w, d);
      }
    };
    const bool near = near_fits<BF16>(P, reference(a.m), c2);
    float d = near_residue<BF16>(reference(a.m), c2);
    add_up(a, [&](float2& s, float2& w, uint4 v) { accumulate_near<BF16>(s, w, v, reference(a.m), c2); });
    if (BF16 && __any_sync(0xFFFFFFFFu, !near && on)) {
      Sums far = a;
      add_up(far, [&](float2& s, float2& w, uint4 v) {
        float x[kN];
        unpack<BF16>(v, x);
        accumulate(s, w, x, reference(a.m), c2);
      });
      if (!near) a = far, d = 0.0f;
    }
    if (MODE != kBackward) {
      r = stats_of(a, P.scale, d);
    } else if (log_s_is_lost(r)) {
      const float entropy = r.entropy;
      r = stats_of(a, P.scale, d);
      r.entropy = entropy;
    }
  }
  if constexpr (MODE != kBackward) {
    if (in && sub == 0) {
      P.lse[row] = on ? r.lse : 0.0f;
      P.entropy[row] = on ? r.entropy : 0.0f;
      P.logprobs[row] = !on ? 0.0f : target >= P.vocab ? NAN : logprob_of(r, x_target, P.scale);
    }
    if (P.top > 0) {
      WarpTop& T = S[threadIdx.x >> 5];
      if (!__any_sync(0xFFFFFFFFu, on)) {
        if (in)
          for (int k = sub; k < P.top; k += P.lanes) P.top_ids[row * P.top + k] = -1, P.top_logprobs[row * P.top + k] = 0.0f;
      } else if (P.lanes == 32 && warp_top<BF16, NV>(P, R, q, lane, T)) {
        if (in && lane < P.top) {
          P.top_ids[row * P.top + lane] = place_index(T.top[lane]);
          P.top_logprobs[row * P.top + lane] = logprob_of(r, place_value(T.top[lane]), P.scale);
        }
      } else {  // a few entries a lane, or a row of ties: one maximum after the other
        unsigned long long last = ~0ull;
        for (int k = 0; k < P.top; ++k) {
          unsigned long long best = 0;
#pragma unroll 1
          for (int u = 0; u < NV; ++u) {
            uint4 qu = q[0];
#pragma unroll
            for (int i = 1; i < NV; ++i) qu = i == u ? q[i] : qu;
            float x[kN];
            unpack<BF16>(qu, x);
#pragma unroll
            for (int i = 0; i < kN; ++i) {
              const int j = R.first(sub + P.lanes * u) + i;
              const unsigned long long v = j >= 0 && j < P.vocab ? place(x[i], j) : 0;
              if (v < last && v > best) best = v;
            }
          }
          for (int d = P.lanes / 2; d > 0; d /= 2) {
            const unsigned long long o = __shfl_xor_sync(0xFFFFFFFFu, best, d);
            best = o > best ? o : best;
          }
          last = best;
          if (in && sub == 0) {
            P.top_ids[row * P.top + k] = on ? place_index(best) : -1;
            P.top_logprobs[row * P.top + k] = on ? logprob_of(r, place_value(best), P.scale) : 0.0f;
          }
        }
      }
    }
  }
  if constexpr (MODE != kScore) {
    __syncwarp();  // in place: the target's logit has been read
    if (!in) return;
    RowGrad g{};
    if (on) g = grad_of(P, r, gl, ge, target);
    const NearGrad near = near_of<BF16>(P, g);
    const long long out = row * P.grad_stride;
    const RowVectors<BF16> O(P.grad, out, P.vocab);
    uint4* const o = reinterpret_cast<uint4*>(const_cast<unsigned char*>(O.base));
    const bool same = O.shift == R.shift;
    // the logits are widened anew: kept from the sums they would take the
    // registers of twice as many warps
#pragma unroll
    for (int u = 0; u < NV; ++u) anew(q[u]);
    if (!on || near.fits) {
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        const int v = sub + P.lanes * u;
        if (v >= R.count) continue;
        uint4 y = make_uint4(0, 0, 0, 0);
        if (on) y = grad_near<BF16>(P, g, near, target, R.first(v), q[u]);
        if (same && static_cast<unsigned>(v - lo) < static_cast<unsigned>(wholes)) o[v] = y;
        else store_entries<BF16>(P.grad, out, R.first(v), P.vocab, y);
      }
    } else {  // a row far from zero
#pragma unroll 1
      for (int u = 0; u < NV; ++u) {
        uint4 qu = q[0];
#pragma unroll
        for (int i = 1; i < NV; ++i) qu = i == u ? q[i] : qu;
        const int v = sub + P.lanes * u;
        if (v >= R.count) continue;
        float x[kN];
        unpack<BF16>(qu, x);
        grad_entries(g, P.scale, target, R.first(v), x);
        store_entries<BF16>(P.grad, out, R.first(v), P.vocab, pack<BF16>(x));
      }
    }
  }
}

// ------------------------------------------------ rows in shared memory (CTAs)

template <int THREADS, typename F>
__device__ __forceinline__ float cta_reduce(float v, F f, float* scratch) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v = f(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  v = scratch[0];
#pragma unroll
  for (int w = 1; w < THREADS / 32; ++w) v = f(v, scratch[w]);
  return v;
}

template <int THREADS>
__device__ __forceinline__ float2 cta_sum2(float2 v, float2* scratch) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) {
    v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, d);
    v.y += __shfl_xor_sync(0xFFFFFFFFu, v.y, d);
  }
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  v = scratch[0];
#pragma unroll
  for (int w = 1; w < THREADS / 32; ++w) v = __fadd2_rn(v, scratch[w]);
  return v;
}

// The alternatives of the row at hand, or of a CTA's part of it.  Collected
// are the entries that reach a bound; `top` at least of the row's entries do.
template <int THREADS, int CHUNKS>
struct TopScratch {
  uint32_t group_max[kTopGroups];
  uint32_t bound;
  int n, hits;
  uint16_t hit[kHits];                // chunk * THREADS + thread
  float chunk_max[CHUNKS][THREADS];   // largest entry of each chunk of a thread's vectors
  unsigned long long candidate[kCandidates];
  unsigned long long best[THREADS / 32];
  unsigned long long top[kMaxTop];
};

// The bound: the top-th largest of the maxima of kTopGroups groups of
// neighbouring threads, `own` being a thread's largest entry.  A group's
// threads share its comparison with the others.  Two barriers; the first one
// also shows what was written to shared memory before.
template <int THREADS, int CHUNKS>
__device__ __forceinline__ void top_bound(int top, float own, TopScratch<THREADS, CHUNKS>& S) {
  constexpr int kGroup = THREADS / kTopGroups, kEach = kTopGroups / kGroup;
  const int t = threadIdx.x, group = t / kGroup, part = t % kGroup;
  uint32_t mine = ordered(own);
#pragma unroll
  for (int d = 1; d < kGroup; d *= 2) mine = max(mine, __shfl_xor_sync(0xFFFFFFFFu, mine, d));
  if (part == 0) S.group_max[group] = mine;
  if (t == 0) S.n = S.hits = 0;
  if (t < kMaxTop) S.top[t] = 0;
  __syncthreads();
  int rank = 0;  // equal ones by their number
#pragma unroll
  for (int j = 0; j < kEach; j += 4) {
    const int at = part * kEach + j;
    const uint4 o = *reinterpret_cast<const uint4*>(&S.group_max[at]);
    rank += (o.x > mine || (o.x == mine && at < group)) + (o.y > mine || (o.y == mine && at + 1 < group)) +
            (o.z > mine || (o.z == mine && at + 2 < group)) + (o.w > mine || (o.w == mine && at + 3 < group));
  }
#pragma unroll
  for (int d = 1; d < kGroup; d *= 2) rank += __shfl_xor_sync(0xFFFFFFFFu, rank, d);
  if (part == 0 && rank == top - 1) S.bound = mine;
  __syncthreads();
}

// Collects from one vector, whose first entry is j0.
template <bool BF16, int THREADS, int CHUNKS>
__device__ __forceinline__ void collect(uint4 v, int j0, int vocab, TopScratch<THREADS, CHUNKS>& S) {
  const uint32_t bound = S.bound;
  if (ordered(vec_max<BF16>(v)) < bound) return;
  float x[kPer<BF16>];
  unpack<BF16>(v, x);
#pragma unroll
  for (int k = 0; k < kPer<BF16>; ++k) {
    const int j = j0 + k;
    if (ordered(x[k]) < bound || j < 0 || j >= vocab) continue;
    const int at = atomicAdd(&S.n, 1);
    if (at < kCandidates) S.candidate[at] = place(x[k], j);
  }
}

// Collects from the chunks whose largest entry reaches the bound, spread over
// all threads.  vector(i) is vector i of the CTA's part, n in all, entry
// `first` beginning vector 0; thread t has seen t, t + THREADS, ..., `each` of
// them to a chunk, and `own` is its largest entry.  Two barriers.
template <bool BF16, int THREADS, int CHUNKS, typename V>
__device__ __forceinline__ void collect_seen(float own, int chunks, int each, int n, int first, int vocab, V vector,
                                             TopScratch<THREADS, CHUNKS>& S) {
  const uint32_t bound = S.bound;
  const float least = place_value(static_cast<unsigned long long>(bound) << 32);
  if (ordered(own) >= bound) {
    for (int c = 0; c < chunks; ++c) {
      if (S.chunk_max[c][threadIdx.x] < least) continue;
      const int h = atomicAdd(&S.hits, 1);
      if (h < kHits) S.hit[h] = static_cast<uint16_t>(c * THREADS + threadIdx.x);
    }
  }
  __syncthreads();
  if (S.hits > kHits) {  // as if there were too many candidates
    if (threadIdx.x == 0) S.n = kCandidates + 1;
  } else {
    const unsigned pairs = S.hits * each;
    for (unsigned q = threadIdx.x; q < pairs; q += THREADS) {
      const unsigned h = q / static_cast<unsigned>(each);
      const int c = S.hit[h] / THREADS, thread = S.hit[h] % THREADS;
      const int i = thread + (c * each + static_cast<int>(q - h * each)) * THREADS;
      if (i >= n) continue;
      collect<BF16>(vector(i), first + i * kPer<BF16>, vocab, S);
    }
  }
  __syncthreads();
}

// gather() collects what reaches the bound.  Where that is more than there is
// room for, many entries equal the bound (a mask that leaves fewer than `top`
// entries, logits that a coarse type makes equal): then it collects what is
// above the bound, and of the entries first .. last-1 of the row in global
// memory the first ones that equal it are added, as many as `top` takes.
template <bool BF16, int THREADS, int CHUNKS, typename G>
__device__ __forceinline__ void gather_top(int top, const void* x, long long base, int first, int last, TopScratch<THREADS, CHUNKS>& S,
                                           G gather) {
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  int pass = 0;
#pragma unroll 1
  for (;; ++pass) {
    gather();
    if (pass == 1 || S.n <= kCandidates) break;
    __syncthreads();
    if (t == 0) S.n = S.hits = 0, ++S.bound;
    __syncthreads();
  }
  if (pass == 0 || S.n > kCandidates) return;
  const uint32_t equal = S.bound - 1;
  int n = S.n;
  for (int from = first; n < top && from < last; from += THREADS) {
    const int j = from + t;
    const float v = j < last ? at<BF16>(x, base + j) : 0.0f;
    const bool tie = j < last && ordered(v) == equal;
    const unsigned ties = __ballot_sync(0xFFFFFFFFu, tie);
    __syncthreads();  // S.best has been read
    if (lane == 0) S.best[warp] = __popc(ties);
    __syncthreads();
    int place_ = n + __popc(ties & ((1u << lane) - 1));
    for (int w = 0; w < THREADS / 32; ++w) {
      const int count = static_cast<int>(S.best[w]);
      if (w < warp) place_ += count;
      n += count;
    }
    if (tie && place_ < top) S.candidate[place_] = place(v, j);
  }
  __syncthreads();
  if (t == 0) S.n = max(S.n, min(n, top));
  __syncthreads();
}

// Ranks what was collected by counting, into S.top (0 where there are fewer).
// Where more was collected than there is room for it takes one maximum after
// the other of `x`, the entries first .. last-1 of a row in global memory.
template <bool BF16, int THREADS, int CHUNKS>
__device__ __forceinline__ void top_rank(int top, const void* x, long long base, int first, int last, TopScratch<THREADS, CHUNKS>& S) {
  const int t = threadIdx.x, n = S.n;
  if (n <= kCandidates) {
    for (int i = t; i < n; i += THREADS) {
      const unsigned long long mine = S.candidate[i];
      int rank = 0;
#pragma unroll 4
      for (int j = 0; j < n; ++j) rank += S.candidate[j] > mine;
      if (rank < top) S.top[rank] = mine;
    }
  } else {
    unsigned long long before = ~0ull;
    for (int k = 0; k < top; ++k) {
      unsigned long long best = 0;
#pragma unroll 4
      for (int j = first + t; j < last; j += THREADS) {
        const unsigned long long v = place(at<BF16>(x, base + j), j);
        if (v < before && v > best) best = v;
      }
#pragma unroll
      for (int d = 16; d > 0; d /= 2) {
        const unsigned long long o = __shfl_xor_sync(0xFFFFFFFFu, best, d);
        best = o > best ? o : best;
      }
      if ((t & 31) == 0) S.best[t >> 5] = best;
      __syncthreads();
      for (int w = 0; w < THREADS / 32; ++w) best = S.best[w] > best ? S.best[w] : best;
      if (t == 0) S.top[k] = best;
      before = best;
      __syncthreads();
    }
  }
  __syncthreads();
}

// Sums of the entries first .. last-1 of a row in global memory against their
// largest: where a nearer reference was too far off.
template <bool BF16, int THREADS>
__device__ __noinline__ Sums sums_again(const void* x, long long base, int first, int last, float c2, float* scratch, float2* pair_scratch) {
  float m = -INFINITY;
#pragma unroll 4
  for (int j = first + static_cast<int>(threadIdx.x); j < last; j += THREADS) m = fmaxf(m, at<BF16>(x, base + j));
  Sums a{};
  a.m = cta_reduce<THREADS>(m, [](float p, float q) { return fmaxf(p, q); }, scratch);
  float2 s{}, w{};
  constexpr int kPass = 16 * 2 * THREADS;
  for (int j0 = first + static_cast<int>(threadIdx.x); j0 < last; j0 += kPass) {
    float2 sp{}, wp{};
#pragma unroll 2
    for (int j = j0; j < min(last, j0 + kPass); j += 2 * THREADS) {
      const float v[2] = {at<BF16>(x, base + j), j + THREADS < last ? at<BF16>(x, base + j + THREADS) : -INFINITY};
      accumulate(sp, wp, v, reference(a.m), c2);
    }
    s = __fadd2_rn(s, sp);
    w = __fadd2_rn(w, wp);
  }
  const float2 sums = cta_sum2<THREADS>(make_float2(s.x + s.y, w.x + w.y), pair_scratch);
  a.s = sums.x;
  a.w = sums.y;
  return a;
}

// What the CTAs of a cluster tell one another.  Sums of one row are read while
// the next row's are written; the row after that may only write once the next
// row's exchange has kept every CTA.
struct Exchange {
  Sums sums[2][kMaxCluster];
  unsigned long long top[kMaxCluster][kMaxTop];
};

// One CTA's part of a row: vectors v0 .. v0+n-1.
template <bool BF16>
struct RowPart {
  const unsigned char* src;  // vector v0
  int shift, v0, n;
  int lo, wholes;            // the row's whole vectors: lo .. lo+wholes-1
  __device__ __forceinline__ int first(int i) const { return (v0 + i) * kPer<BF16> - shift; }
  __device__ __forceinline__ bool whole(int i) const { return static_cast<unsigned>(v0 + i - lo) < static_cast<unsigned>(wholes); }
};

template <bool BF16>
__device__ __forceinline__ RowPart<BF16> part_of(const LogprobParams& P, long long row, int rank) {
  const RowVectors<BF16> R(P.x, row * P.stride, P.vocab);
  RowPart<BF16> p;
  // at most 2^28 + 1 vectors and eight CTAs, a power of two of them: no division
  p.v0 = static_cast<int>(static_cast<unsigned>(R.count) * rank >> P.log_ranks);
  p.n = static_cast<int>(static_cast<unsigned>(R.count) * (rank + 1) >> P.log_ranks) - p.v0;
  if (!MUON_CHECK(row >= 0 && row < P.rows && p.v0 + p.n <= R.count)) p.n = 0;
  if (!MUON_CHECK(P.segment == 0 || (p.n <= P.segment && p.n <= 4 * P.group))) p.n = min(P.segment, 4 * P.group);
  p.src = R.base + p.v0 * 16LL;
  p.shift = R.shift;
  p.lo = R.shift > 0 ? 1 : 0;
  p.wholes = static_cast<unsigned>(R.shift + P.vocab) / kPer<BF16> - p.lo;
  return p;
}

// Sums of a CTA's part of a row in shared memory against its largest entry.
template <bool BF16, int THREADS>
__device__ __noinline__ Sums segment_again(const uint4* q, int n, float c2, float* scratch, float2* pair_scratch) {
  VecMax<BF16> largest;
  for (int i = threadIdx.x; i < n; i += THREADS) largest.add(q[i]);
  Sums a{};
  a.m = cta_reduce<THREADS>(largest.value(), [](float x, float y) { return fmaxf(x, y); }, scratch);
  float2 s{}, w{};
#pragma unroll 1
  for (int i0 = threadIdx.x; i0 < n; i0 += 8 * THREADS) {
    float2 sp{}, wp{};
#pragma unroll 2
    for (int i = i0; i < min(n, i0 + 8 * THREADS); i += THREADS) {
      float x[kPer<BF16>];
      unpack<BF16>(q[i], x);
      accumulate(sp, wp, x, reference(a.m), c2);
    }
    s = __fadd2_rn(s, sp);
    w = __fadd2_rn(w, wp);
  }
  const float2 sums = cta_sum2<THREADS>(make_float2(s.x + s.y, w.x + w.y), pair_scratch);
  a.s = sums.x;
  a.w = sums.y;
  return a;
}

// A cluster takes one row after the other (persistent).  A CTA's part of a
// row lies in its shared memory as vectors in four groups; a thread's vectors
// are the ones it copies, so it works on a group without waiting for other
// threads, and copies the next row's group as soon as it is done with one:
// the loads go on while sums are exchanged and alternatives ranked.  Groups are
// the same vectors of every row, however many the row's place makes of it: what
// is copied for the next row then lies where this row is done with.
template <bool BF16, int THREADS, bool TOP>
__global__ void __launch_bounds__(THREADS, THREADS == 128 ? 8 : 3) logprob_loss(const __grid_constant__ LogprobParams P) {
  extern __shared__ __align__(16) unsigned char segment[];
  __shared__ float scratch[2][THREADS / 32];
  __shared__ float2 pair_scratch[2][THREADS / 32];
  __shared__ Exchange X;
  __shared__ __align__(16) TopScratch<TOP ? THREADS : 32, TOP ? 4 : 1> S;
  constexpr int kN = kPer<BF16>;
  constexpr bool kParts = THREADS == 256;  // 128 threads have at most 16 vectors each
  const cg::cluster_group cluster = cg::this_cluster();
  const int ranks = 1 << P.log_ranks, rank = blockIdx.x & (ranks - 1);
  const int t = threadIdx.x;
  const long long clusters = gridDim.x >> P.log_ranks;
  uint4* const q = reinterpret_cast<uint4*>(segment);
  const float c2 = P.scale * kLog2e;
  auto largest = [](float x, float y) { return fmaxf(x, y); };

  // one group of copies, empty past the last row and for rows that are left out
  auto copy = [&](const RowPart<BF16>& p, bool on, int group) {
    if (on) {
      const int end = min(p.n, (group + 1) * P.group);
      int i = group * P.group + t;
      const unsigned char* src = p.src + i * 16LL;
      unsigned dst = static_cast<unsigned>(__cvta_generic_to_shared(q + i));
      for (; i < end; i += THREADS, src += THREADS * 16, dst += THREADS * 16) {
        if (p.whole(i)) {
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
        } else {  // an end of the row; what lies outside counts as masked
          float x[kN];
#pragma unroll
          for (int k = 0; k < kN; ++k) {
            const int j = p.first(i) + k;
            x[k] = j >= 0 && j < P.vocab ? at<BF16>(src, k) : -INFINITY;
          }
          q[i] = pack<BF16>(x);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  long long row = blockIdx.x >> P.log_ranks;
  int64_t target = P.targets[row];
  RowPart<BF16> p = part_of<BF16>(P, row, rank);
  // a CTA's shared memory is written by others only once it has begun
  if (ranks > 1) cg::cluster_group::barrier_arrive();
#pragma unroll 1
  for (int g = 0; g < 4; ++g) copy(p, target >= 0, g);
  if (ranks > 1) cg::cluster_group::barrier_wait();

  // `turn` flips with every row that is exchanged, not with rows that are left
  // out: between two writes of a slot of X.sums there is then the exchange of
  // the other slot, which a CTA passes only after it has read the first
  for (int turn = 0; row < P.rows;) {
    const long long next = row + clusters;
    const int64_t next_target = next < P.rows ? P.targets[next] : -1;
    const bool next_on = next_target >= 0;
    const RowPart<BF16> np = part_of<BF16>(P, next_on ? next : row, rank);
    const long long base = row * P.stride, out = row * P.grad_stride;
    const int j0 = max(0, p.first(0)), j1 = min(P.vocab, p.first(p.n));  // this CTA's entries
    // the gradient's vectors begin where the row's do
    const RowVectors<BF16> O(P.grad, out, P.vocab);
    const bool same = O.shift == p.shift;
    uint4* const o = reinterpret_cast<uint4*>(const_cast<unsigned char*>(O.base)) + p.v0;

    if (target < 0) {
      if (rank == 0 && t == 0) P.logprobs[row] = P.lse[row] = P.entropy[row] = 0.0f;
      if (TOP && rank == 0 && t < P.top) P.top_logprobs[row * P.top + t] = 0.0f, P.top_ids[row * P.top + t] = -1;
      if (same) {
        for (int i = t; i < p.n; i += THREADS) {
          if (p.whole(i)) {
            o[i] = make_uint4(0, 0, 0, 0);
          } else {
            for (int k = 0; k < kN; ++k) {
              const int j = p.first(i) + k;
              if (j >= 0 && j < P.vocab) put<BF16>(P.grad, out + j, 0.0f);
            }
          }
        }
      } else {
        for (int j = j0 + t; j < j1; j += THREADS) put<BF16>(P.grad, out + j, 0.0f);
      }
#pragma unroll 1
      for (int g = 0; g < 4; ++g) copy(np, next_on, g);
      row = next;
      target = next_target;
      p = np;
      continue;
    }

    float x_target = 0.0f;
    if (t == 0 && rank == 0 && target < P.vocab) x_target = at<BF16>(P.x, base + target);

    // Sums against the largest of the first vectors, which is near enough to
    // the row's largest entry unless S or W says otherwise.
    float2 s{}, w{};
    Sums a{};
    float own = -INFINITY;
    asm volatile("cp.async.wait_group 3;" ::: "memory");
    a.m = reference(cta_reduce<THREADS>(t < p.n ? vec_max<BF16>(q[t]) : -INFINITY, largest, scratch[turn]));
    // three newer groups at any time: this row's, then empty ones
#pragma unroll 1
    for (int group = 0; group < 4; ++group) {
      asm volatile("cp.async.wait_group 3;" ::: "memory");
      const int end = min(p.n, (group + 1) * P.group);
      VecMax<BF16> chunk;
      float2 sg{}, wg{};
#pragma unroll 2
      for (int i = group * P.group + t; i < end; i += THREADS) {
        const uint4 v = q[i];
        if (TOP) chunk.add(v);
        accumulate_near<BF16>(kParts ? sg : s, kParts ? wg : w, v, a.m, c2);
      }
      if constexpr (kParts) {
        s = __fadd2_rn(s, sg);
        w = __fadd2_rn(w, wg);
      }
      if constexpr (TOP) {
        S.chunk_max[group][t] = chunk.value();
        own = fmaxf(own, chunk.value());
      }
      copy(np, false, group);
    }
    const float2 sums = cta_sum2<THREADS>(make_float2(s.x + s.y, w.x + w.y), pair_scratch[turn]);
    a.s = sums.x;
    a.w = sums.y;
    settle<BF16>(a, c2);
    if (!(near_fits<BF16>(P, a.m, c2) && a.s >= 0.5f && a.s < 0x1p60f && a.w <= kAbove * a.s)) {
      __syncthreads();  // the scratch arrays have been read
      a = segment_again<BF16, THREADS>(q, p.n, c2, scratch[turn], pair_scratch[turn]);
    }
    if (ranks > 1) {
      if (t < ranks) cluster.map_shared_rank(&X, t)->sums[turn][rank] = a;
      cluster.sync();
    }
    if (ranks > 1) {
      a = X.sums[turn][0];
      for (int k = 1; k < ranks; ++k) a = merge(a, X.sums[turn][k], c2);
    }
    const RowStats r = stats_of(a, P.scale);
    if (rank == 0 && t == 0) {
      P.lse[row] = r.lse;
      P.entropy[row] = r.entropy;
      P.logprobs[row] = target < P.vocab ? logprob_of(r, x_target, P.scale) : NAN;
    }
    if constexpr (TOP) {
      top_bound(P.top, own, S);
      gather_top<BF16>(P.top, P.x, base, j0, j1, S, [&] {
        collect_seen<BF16>(own, 4, P.group / THREADS, p.n, p.first(0), P.vocab, [&](int i) { return q[i]; }, S);
      });
      top_rank<BF16>(P.top, P.x, base, j0, j1, S);
      if (ranks > 1) {
        if (t < P.top) cluster.map_shared_rank(&X, 0)->top[rank][t] = S.top[t];
        cluster.sync();
        if (rank == 0) {
          const int all = ranks * P.top;
          for (int i = t; i < all; i += THREADS) {
            const unsigned long long mine = X.top[i / P.top][i % P.top];
            int place_ = 0;
            for (int j = 0; j < all; ++j) place_ += X.top[j / P.top][j % P.top] > mine;
            if (mine != 0 && place_ < P.top) S.top[place_] = mine;
          }
          __syncthreads();
        }
      }
      if (rank == 0 && t < P.top) {
        P.top_ids[row * P.top + t] = place_index(S.top[t]);
        P.top_logprobs[row * P.top + t] = logprob_of(r, place_value(S.top[t]), P.scale);
      }
      __syncthreads();  // S is free for the next row
    }

    const RowGrad g = grad_of(P, r, P.gl[row], P.ge ? P.ge[row] : 0.0f, target);
    const NearGrad near = near_of<BF16>(P, g);
    if (same && near.fits) {
#pragma unroll 1
      for (int group = 0; group < 4; ++group) {
        const int end = min(p.n, (group + 1) * P.group);
#pragma unroll 2
        for (int i = group * P.group + t; i < end; i += THREADS) {
          const int j = p.first(i);
          const uint4 v = grad_near<BF16>(P, g, near, target, j, q[i]);
          if (p.whole(i)) {
            o[i] = v;
          } else {
            float x[kN];
            unpack<BF16>(v, x);
            for (int k = 0; k < kN; ++k)
              if (j + k >= 0 && j + k < P.vocab) put<BF16>(P.grad, out + j + k, x[k]);
          }
        }
        copy(np, next_on, group);
      }
    } else {  // the gradient's whole vectors and its ends, whichever thread copied the logits
      const int from = p.first(0), v0 = (j0 + O.shift + kN - 1) / kN, v1 = max(v0, (j1 + O.shift) / kN);
      uint4* const whole = reinterpret_cast<uint4*>(const_cast<unsigned char*>(O.base));
#pragma unroll 2
      for (int v = v0 + t; v < v1; v += THREADS) {
        float x[kN];
        unpack<BF16>(unaligned<BF16>(segment, O.first(v) - from), x);
        grad_entries(g, P.scale, target, O.first(v), x);
        whole[v] = pack<BF16>(x);
      }
      const int head = min(j1, O.first(v0)) - j0, tail = O.first(v1);
      const int j = t < head ? j0 + t : tail + t - head;
      if (t < head || j < j1)
        put<BF16>(P.grad, out + j, grad_entry(g, P.scale, target, j, at<BF16>(segment, j - from)));
      __syncthreads();
#pragma unroll 1
      for (int group = 0; group < 4; ++group) copy(np, next_on, group);
    }
    turn ^= 1;
    row = next;
    target = next_target;
    p = np;
  }
  // others may still write this CTA's sums or alternatives
  if (ranks > 1) cluster.sync();
}

// ------------------------------------------------- scores of long rows (CTAs)

// A warp's sums of a row up to a batch, and of the batch, against m.
struct BatchSums {
  float2 s, w, sb, wb;
  float m;
};

// The batch, vectors first, first + THREADS, ... before `end`, held entries far
// above m: a new reference, and the batch again.
template <bool BF16, int THREADS>
__device__ __forceinline__ BatchSums batch_again(BatchSums g, const uint4* src, int first, int end, float c2) {
  VecMax<BF16> largest;
  for (int i = first; i < end; i += THREADS) largest.add(src[i]);
  float m = fmaxf(g.m, largest.value());
#pragma unroll
  for (int d = 16; d > 0; d /= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
  if (!(m > g.m)) return g;
  move_reference<BF16>(g.s, g.w, reference(g.m), m, c2);
  g.m = m;
  g.sb = g.wb = make_float2(0.0f, 0.0f);
  for (int i = first; i < end; i += THREADS) accumulate_near<BF16>(g.sb, g.wb, src[i], m, c2);
  return g;
}

// As a call it leaves the kernels with alternatives their registers (16384 x 50304
// bfloat16 with 5: 282 us, 292 in line); the others are faster with it in line (239 and 257).
template <bool BF16, int THREADS>
__device__ __noinline__ BatchSums batch_again_called(BatchSums g, const uint4* src, int first, int end, float c2) {
  return batch_again<BF16, THREADS>(g, src, first, end, c2);
}

// One row per CTA, or per cluster where rows are few.  The logits pass through
// registers, two batches of four vectors a thread.  Each warp adds up against
// the largest entry of its own first batch, or of a later one that stands far
// above it.
template <bool BF16, int THREADS, bool TOP>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) logprob_score(const __grid_constant__ LogprobParams P) {
  constexpr int kWarps = THREADS / 32, kU = 4, kBatch = kU * THREADS;
  __shared__ Sums warp_sums[kWarps];
  __shared__ float scratch[kWarps];
  __shared__ float2 pair_scratch[kWarps];
  __shared__ Exchange X;
  __shared__ __align__(16) TopScratch<TOP ? THREADS : 32, TOP ? kScoreChunks : 1> S;
  const cg::cluster_group cluster = cg::this_cluster();
  const int ranks = 1 << P.log_ranks, rank = blockIdx.x & (ranks - 1);
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const long long row = blockIdx.x >> P.log_ranks, base = row * P.stride;
  const int64_t target = P.targets[row];
  if (target < 0) {  // every CTA of the cluster returns
    if (rank == 0 && t == 0) P.logprobs[row] = P.lse[row] = P.entropy[row] = 0.0f;
    if (TOP && rank == 0 && t < P.top) P.top_logprobs[row * P.top + t] = 0.0f, P.top_ids[row * P.top + t] = -1;
    return;
  }
  // a CTA's shared memory is written by others only once it has begun
  if (ranks > 1) cg::cluster_group::barrier_arrive();
  const RowPart<BF16> p = part_of<BF16>(P, row, rank);
  // the part's whole vectors src[0 .. n-1]; the row's other two (its ends) are
  // put together from their entries by one thread each
  const bool head = p.v0 < p.lo, tail = p.v0 + p.n > p.lo + p.wholes;
  const uint4* const src = reinterpret_cast<const uint4*>(p.src) + head;
  const int n = p.n - head - tail;
  const float c2 = P.scale * kLog2e;
  uint4 a[kU], b[kU], end = masked_vector<BF16>();
  if (t == 0 && head) end = RowVectors<BF16>(P.x, base, P.vocab).end(p.v0);
  if (t == 32 && tail) end = RowVectors<BF16>(P.x, base, P.vocab).end(p.v0 + p.n - 1);
#pragma unroll
  for (int u = 0; u < kU; ++u) a[u] = t + u * THREADS < n ? load_once(src + t + u * THREADS) : masked_vector<BF16>();
  float x_target = 0.0f;
  if (t == 0 && rank == 0 && target < P.vocab) x_target = at<BF16>(P.x, base + target);
  Sums sums{};
  VecMax<BF16> near;
  near.add(end);
#pragma unroll
  for (int u = 0; u < kU; ++u) near.add(a[u]);
  sums.m = near.value();
#pragma unroll
  for (int d = 16; d > 0; d /= 2) sums.m = fmaxf(sums.m, __shfl_xor_sync(0xFFFFFFFFu, sums.m, d));
  float2 s{}, w{};
  bool found = sums.m != -INFINITY;
  if (warp < 2) accumulate_near<BF16>(s, w, end, reference(sums.m), c2);
  // a chunk: batches of a thread that share a largest entry, a power of two of them
  const int batches = (n + kBatch - 1) / kBatch;
  int log_chunk = 0;
  while (TOP && batches > kScoreChunks << log_chunk) ++log_chunk;
  for (int k = 0; k < batches; ++k) {
    const int i = k * kBatch + t;
    if (!found) {  // masked entries alone so far
#pragma unroll
      for (int u = 0; u < kU; ++u) sums.m = i + u * THREADS < n ? fmaxf(sums.m, vec_max<BF16>(a[u])) : sums.m;
#pragma unroll
      for (int d = 16; d > 0; d /= 2) sums.m = fmaxf(sums.m, __shfl_xor_sync(0xFFFFFFFFu, sums.m, d));
      found = sums.m != -INFINITY;
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (i + kBatch + u * THREADS < n) b[u] = load_once(src + i + kBatch + u * THREADS);
    VecMax<BF16> largest;
    float2 sb{}, wb{};
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (i + u * THREADS < n) {
        if (TOP) largest.add(a[u]);
        accumulate_near<BF16>(sb, wb, a[u], reference(sums.m), c2);
      }
      a[u] = b[u];
    }
    if (__any_sync(0xFFFFFFFFu, fmaxf(sb.x, sb.y) > kAboveSum)) {
      constexpr auto again = TOP ? batch_again_called<BF16, THREADS> : batch_again<BF16, THREADS>;
      const BatchSums g = again({s, w, sb, wb, sums.m}, src, i, min(n, (k + 1) * kBatch), c2);
      s = g.s, w = g.w, sb = g.sb, wb = g.wb, sums.m = g.m;
    }
    s = __fadd2_rn(s, sb);
    w = __fadd2_rn(w, wb);
    if constexpr (TOP) {
      float* const chunk = &S.chunk_max[k >> log_chunk][t];
      *chunk = (k & ((1 << log_chunk) - 1)) == 0 ? largest.value() : fmaxf(*chunk, largest.value());
    }
  }
  sums.s = s.x + s.y;
  sums.w = w.x + w.y;
#pragma unroll
  for (int d = 16; d > 0; d /= 2) {
    sums.s += __shfl_xor_sync(0xFFFFFFFFu, sums.s, d);
    sums.w += __shfl_xor_sync(0xFFFFFFFFu, sums.w, d);
  }
  settle<BF16>(sums, c2);
  if (!near_fits<BF16>(P, reference(sums.m), c2)) sums.s = NAN;
  // A warp that saw masked entries alone has m = -inf and no sum; any other sum
  // out of range means that its reference was too far off, or too large.
  if (lane == 0) warp_sums[warp] = sums;
  const int chunks = (batches + (1 << log_chunk) - 1) >> log_chunk;
  float own = vec_max<BF16>(end);
  if constexpr (TOP) {
    for (int c = 0; c < chunks; ++c) own = fmaxf(own, S.chunk_max[c][t]);
    top_bound(P.top, own, S);
  } else {
    __syncthreads();
  }
  bool far = false;
#pragma unroll
  for (int k = 0; k < kWarps; ++k)
    far |= !(warp_sums[k].s >= 0.5f && warp_sums[k].s < 0x1p60f) && !(warp_sums[k].s == 0.0f && warp_sums[k].m == -INFINITY);
  if (far) {
    sums = sums_again<BF16, THREADS>(P.x, base, max(0, p.first(0)), min(P.vocab, p.first(p.n)), c2, scratch, pair_scratch);
  } else if (warp == 0) {
    sums = warp_sums[0];
#pragma unroll
    for (int k = 1; k < kWarps; ++k) sums = merge(sums, warp_sums[k], c2);
  }
  if constexpr (TOP) {
    const int j0 = max(0, p.first(0)), j1 = min(P.vocab, p.first(p.n));
    gather_top<BF16>(P.top, P.x, base, j0, j1, S, [&] {
      if (warp < 2) collect<BF16>(end, p.first(t == 0 ? 0 : p.n - 1), P.vocab, S);
      collect_seen<BF16>(own, chunks, kU << log_chunk, n, p.first(head), P.vocab, [&](int i) { return load_once(src + i); }, S);
    });
    top_rank<BF16>(P.top, P.x, base, j0, j1, S);
  }
  if (ranks > 1) {
    cg::cluster_group::barrier_wait();
    if (t == 0) cluster.map_shared_rank(&X, 0)->sums[0][rank] = sums;
    if (TOP && t < P.top) cluster.map_shared_rank(&X, 0)->top[rank][t] = S.top[t];
    cluster.sync();
    if (rank != 0) return;
    if (warp == 0) {
      sums = X.sums[0][0];
      for (int k = 1; k < ranks; ++k) sums = merge(sums, X.sums[0][k], c2);
    }
    if constexpr (TOP) {
      const int all = ranks * P.top;
      for (int i = t; i < all; i += THREADS) {
        const unsigned long long mine = X.top[i / P.top][i % P.top];
        int place_ = 0;
        for (int j = 0; j < all; ++j) place_ += X.top[j / P.top][j % P.top] > mine;
        if (mine != 0 && place_ < P.top) S.top[place_] = mine;
      }
      __syncthreads();
    }
  }
  if (warp != 0) return;
  const RowStats r = stats_of(sums, P.scale);
  if (t == 0) {
    P.lse[row] = r.lse;
    P.entropy[row] = r.entropy;
    P.logprobs[row] = target < P.vocab ? logprob_of(r, x_target, P.scale) : NAN;
  }
  if (TOP && t < P.top) {
    P.top_ids[row * P.top + t] = place_index(S.top[t]);
    P.top_logprobs[row * P.top + t] = logprob_of(r, place_value(S.top[t]), P.scale);
  }
}

// ---------------------------------------------------- backward, elementwise

template <bool BF16>
__global__ void __launch_bounds__(kGradThreads) logprob_grad(const __grid_constant__ LogprobParams P) {
  __shared__ float scratch[kGradThreads / 32];
  __shared__ float2 pair_scratch[kGradThreads / 32];
  constexpr int kN = kPer<BF16>;
  const long long row = blockIdx.x / P.chunks;
  const int chunk = blockIdx.x % P.chunks, t = threadIdx.x;
  const int64_t target = P.targets[row];
  const bool on = target >= 0;
  const long long base = row * P.stride, out = row * P.grad_stride;
  const RowVectors<BF16> R(P.x, base, P.vocab), O(P.grad, out, P.vocab);
  const int v0 = chunk * kGradThreads * kGradVecs, v1 = min(R.count, v0 + kGradThreads * kGradVecs);
  const bool same = R.shift == O.shift;
  uint4 q[kGradVecs];
  if (on && same) {
#pragma unroll
    for (int u = 0; u < kGradVecs; ++u) {
      const int v = v0 + u * kGradThreads + t;
      if (v < v1 && R.whole(v)) q[u] = *reinterpret_cast<const uint4*>(R.base + static_cast<long long>(v) * 16);
    }
  }
  RowStats r{};
  if (on) r = stats_from_lse(P, row);
  if (on && log_s_is_lost(r)) {  // the row's first CTA takes all of it, with its own sums
    if (chunk != 0) return;
    const Sums a = sums_again<BF16, kGradThreads>(P.x, base, 0, P.vocab, P.scale * kLog2e, scratch, pair_scratch);
    const float entropy = r.entropy;
    r = stats_of(a, P.scale);
    r.entropy = entropy;
    const RowGrad g = grad_of(P, r, P.gl[row], P.ge ? P.ge[row] : 0.0f, target);
    constexpr int kU = 8;  // loads before the first store: the gradient may be written over the logits
    for (int j0 = t; j0 < P.vocab; j0 += kU * kGradThreads) {
      float x[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int j = j0 + u * kGradThreads;
        x[u] = j < P.vocab ? at<BF16>(P.x, base + j) : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int j = j0 + u * kGradThreads;
        if (j < P.vocab) put<BF16>(P.grad, out + j, grad_entry(g, P.scale, target, j, x[u]));
      }
    }
    return;
  }
  RowGrad g{};
  if (on) g = grad_of(P, r, P.gl[row], P.ge ? P.ge[row] : 0.0f, target);
  if (same) {
    uint4* const o = reinterpret_cast<uint4*>(const_cast<unsigned char*>(O.base));
#pragma unroll
    for (int u = 0; u < kGradVecs; ++u) {
      const int v = v0 + u * kGradThreads + t;
      if (v >= v1) continue;
      const int j = R.first(v);
      if (R.whole(v)) {
        float x[kN] = {};
        if (on) {
          unpack<BF16>(q[u], x);
          grad_entries(g, P.scale, target, j, x);
        }
        o[v] = pack<BF16>(x);
      } else {
        for (int k = 0; k < kN; ++k)
          if (j + k >= 0 && j + k < P.vocab) put<BF16>(P.grad, out + j + k, on ? grad_entry(g, P.scale, target, j + k, at<BF16>(P.x, base + j + k)) : 0.0f);
      }
    }
  } else {  // the gradient's vectors
    uint4* const o = reinterpret_cast<uint4*>(const_cast<unsigned char*>(O.base));
    const int end = min(O.count, v0 + kGradThreads * kGradVecs);
    auto inside = [&](int v) { return O.first(v) > 0 && O.first(v) + kN < P.vocab; };
#pragma unroll
    for (int u = 0; u < kGradVecs; ++u) {
      const int v = v0 + u * kGradThreads + t;
      q[u] = make_uint4(0, 0, 0, 0);
      if (on && v < end && inside(v)) q[u] = unaligned<BF16>(P.x, base + O.first(v));
    }
#pragma unroll
    for (int u = 0; u < kGradVecs; ++u) {
      const int v = v0 + u * kGradThreads + t;
      if (v >= end) continue;
      const int j = O.first(v);
      if (inside(v)) {
        float x[kN] = {};
        if (on) {
          unpack<BF16>(q[u], x);
          grad_entries(g, P.scale, target, j, x);
        }
        o[v] = pack<BF16>(x);
      } else {
        for (int k = 0; k < kN; ++k)
          if (j + k >= 0 && j + k < P.vocab) put<BF16>(P.grad, out + j + k, on ? grad_entry(g, P.scale, target, j + k, at<BF16>(P.x, base + j + k)) : 0.0f);
      }
    }
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

using KernelPtr = void (*)(LogprobParams);

#define WARPS(BF16, MODE)                                                                                  \
  logprob_warp<BF16, 1, MODE>, logprob_warp<BF16, 2, MODE>, logprob_warp<BF16, 4, MODE>, logprob_warp<BF16, 8, MODE>, \
      logprob_warp<BF16, 16, MODE>
// Index: 0 .. 4 for 1, 2, 4, 8, 16 vectors a lane; + 5 mode; + 15 for bfloat16.
const KernelPtr kWarpKernels[30] = {WARPS(false, kScore), WARPS(false, kLoss), WARPS(false, kBackward),
                                    WARPS(true, kScore),  WARPS(true, kLoss),  WARPS(true, kBackward)};
#undef WARPS

// Index: 256 threads | alternatives << 1 | bfloat16 << 2.
const KernelPtr kLossKernels[8] = {
    logprob_loss<false, 128, false>, logprob_loss<false, 256, false>, logprob_loss<false, 128, true>,
    logprob_loss<false, 256, true>,  logprob_loss<true, 128, false>,  logprob_loss<true, 256, false>,
    logprob_loss<true, 128, true>,   logprob_loss<true, 256, true>,
};

// Index: 256 threads | alternatives << 1 | bfloat16 << 2.
const KernelPtr kScoreKernels[8] = {
    logprob_score<false, 128, false>, logprob_score<false, 256, false>, logprob_score<false, 128, true>,
    logprob_score<false, 256, true>, logprob_score<true, 128, false>,   logprob_score<true, 256, false>,
    logprob_score<true, 128, true>,   logprob_score<true, 256, true>,
};

cudaError_t launch_clusters(KernelPtr f, const LogprobParams& P, long long clusters, int threads, size_t smem, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters << P.log_ranks));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1u << P.log_ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, f, P);
}

// CTAs per row: at least `ranks`; where rows are few more, while every one
// keeps 4 KB of the row and the GPU has room for them.
int spread(int ranks, long long rows, long long bytes, int sms) {
  while (ranks < kMaxCluster && rows * ranks * 2 <= 2LL * sms && bytes / (ranks * 2) >= 4096) ranks *= 2;
  return ranks;
}

cudaError_t launch_score(LogprobParams P, bool bf16, long long bytes, int sms, cudaStream_t stream) {
  const int ranks = spread(1, P.rows, bytes, sms);
  while (1 << P.log_ranks < ranks) ++P.log_ranks;
  // 128 threads a row: eight rows of an SM overlap one's loads with another's
  // reductions (4096 x 50257 bfloat16 with 5 alternatives 100 us, 32768 x 6000
  // without 100; 256 threads: 110 and 157; 64: 109 for the latter).  A row that is
  // spread wants its CTAs' loads in flight at once.
  const bool wide = ranks > 1;
  return launch_clusters(kScoreKernels[(wide ? 1 : 0) | (P.top > 0 ? 2 : 0) | (bf16 ? 4 : 0)], P, P.rows, wide ? 256 : 128, 0, stream);
}

// vecs: the most vectors that a row of `bytes` with its ends can have here.
cudaError_t launch_loss(LogprobParams P, bool bf16, long long bytes, long long vecs, int sms, cudaStream_t stream) {
  int ranks = 1;
  while (bytes > static_cast<long long>(ranks) * kSegmentBytes) ranks *= 2;
  ranks = spread(ranks, P.rows, bytes, sms);
  while (1 << P.log_ranks < ranks) ++P.log_ranks;
  const long long part = (bytes + 15) / 16 / ranks + 1;  // vectors
  const bool wide = part > 2048;                         // 32 KB: 256 threads take eight vectors each
  const KernelPtr f = kLossKernels[(wide ? 1 : 0) | (P.top > 0 ? 2 : 0) | (bf16 ? 4 : 0)];
  const int threads = wide ? 256 : 128;
  P.segment = static_cast<int>(part);
  P.group = static_cast<int>(((vecs + ranks - 1) / ranks + 4 * threads - 1) / (4 * threads)) * threads;
  const size_t smem = static_cast<size_t>(part) * 16;
  const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(f), cudaFuncAttributeMaxDynamicSharedMemorySize, kSegmentBytes + 64);
  if (e != cudaSuccess) return e;
  // as many clusters as are resident at a time (more would only wait)
  const long long per_sm = std::min<long long>(wide ? 3 : 8, (228 * 1024) / (smem + kLossStatic));
  const long long resident = std::max<long long>(1, per_sm * sms / ranks);
  return launch_clusters(f, P, std::min<long long>(P.rows, resident), threads, smem, stream);
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
  const int size = dtype == MUON_F32 ? 4 : 2;
  const int64_t bytes = vocab * size + 32;  // of a row, with both ends' partial vectors
  // longer rows are read twice: 4096 x 128256 bfloat16 take 515 us so, 603 over clusters of four
  const bool held = bytes <= static_cast<int64_t>(kHeldRanks) * kSegmentBytes;
  const int64_t per_cta = 16 * kGradThreads * kGradVecs, chunks = (bytes + per_cta - 1) / per_cta;
  // a row's vectors: all rows begin on a 16-byte boundary, or anywhere
  const bool even = aligned_to(logits, 16) && row_stride * size % 16 == 0;
  const int64_t vecs = even ? (vocab * size + 15) / 16 : (bytes - 2) / 16;
  if (vecs > kWarpVecs && rows > INT32_MAX / chunks) return MUON_ERR_TOO_LARGE;
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
  P.rows = rows;
  P.stride = row_stride;
  P.grad_stride = grad_stride;
  P.vocab = static_cast<int>(vocab);
  P.top = score ? top : 0;
  P.scale = scale;
  P.near = scale * kLog2e >= kNearScale ? kNear : 0.0f;
  const float floor = -2.0f * kNear / (scale * kLog2e);  // rounded to bfloat16 towards 0
  uint32_t bits = 0;
  std::memcpy(&bits, &floor, 4);
  P.floor2 = (bits >> 16) | (bits & 0xFFFF0000u);
  const cudaStream_t str = static_cast<cudaStream_t>(stream);
  const bool bf16 = dtype == MUON_BF16;
  cudaError_t err = cudaSuccess;
  if (vecs <= kWarpVecs) {
    // A lane takes one vector before the row takes more lanes; eight where there
    // are rows for every warp, as a warp's instructions then serve several rows
    // (65536 x 300 bfloat16: score 25 us, 42 with one; loss 37 and 61; backward
    // 29 and 44).  One for alternatives, which a whole warp finds faster
    // (65536 x 300 with five: 82 us, 190 with eight).
    const int each = P.top > 0 || rows < 32LL * sms ? 1 : 8;
    P.lanes = 1;
    while (P.lanes < 32 && P.lanes * each < vecs) P.lanes *= 2;
    int k = 0;
    while (P.lanes << k < vecs) ++k;
    const long long per = static_cast<long long>(kWarpThreads / 32) * (32 / P.lanes);
    const unsigned grid = static_cast<unsigned>((rows + per - 1) / per);
    const int mode = !backward ? kScore : score ? kLoss : kBackward;
    kWarpKernels[k + 5 * mode + (bf16 ? 15 : 0)]<<<grid, kWarpThreads, 0, str>>>(P);
    err = cudaGetLastError();
  } else {
    if (score && backward && held) err = launch_loss(P, bf16, bytes, vecs, sms, str);
    else if (score) err = launch_score(P, bf16, bytes, sms, str);
    if (err == cudaSuccess && backward && !(score && held)) {
      P.chunks = static_cast<int>(chunks);
      (bf16 ? logprob_grad<true> : logprob_grad<false>)<<<static_cast<unsigned>(rows * P.chunks), kGradThreads, 0, str>>>(P);
      err = cudaGetLastError();
    }
  }
  return err == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
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
