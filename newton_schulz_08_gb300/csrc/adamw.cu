// AdamW over many tensors at once, moments in 32 bits or in 8.
//
// Per element, t the step, in float32:
//   g' = grad_scale * g
//   m1 = b1 m + (1-b1) g';   v1 = b2 v + (1-b2) (g' g')
//   u  = m1 / (sqrt(v1) r2 + eps),           r2 = 1 / sqrt(1 - b2^t)
//   p1 = p - (u lr/(1-b1^t) + lr wd p mask), mask as in the cautious Adam step
// with the scalars formed in double on the host and rounded once.  In the
// moments every operation is rounded and none fused, so that codes do not
// depend on how the compiler contracts; u takes the approximate root and
// reciprocal (a few units in the last place of a change that is small beside p),
// which take subnormals for zeros.  A second moment below 2^-126 has a root below
// 2^-63: where eps does not cover that (eps < 2^-41 r2), u takes a root and a
// quotient of the whole range, in kernels of their own (as a branch in the others
// it cost the 8-bit steps 3 to 8 %: 386 us for 373, 231 for 213).
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
// A block's range is that of the codes: gradients that differ by more than 2^12
// within it leave small second moments at 0 beside first ones that are not, and
// u grows far beyond 1 (its root mean square against the exact one's, eps 1e-12:
// 1.03 at 2^12, 24 at 2^14, 390 at 2^16; the largest is bounded by eps alone).
// Codes are made in the integer representation: |x| 2^-E 2^(14-127) has in its
// exponent field the exponent field of the E4M3 code (subnormals included),
// so adding 20 random bits and dropping 20 rounds it; E5M2 likewise with 29
// and 21.
//
// Work: one warp per 256-element block, 8 elements a lane; eight warps share
// eight blocks of one tensor.  One launch covers up to kMaxTensors tensors of
// the same types; the table is in the kernel's parameters.
// Bound: 32-bit moments by HBM (float32 parameters, bfloat16 gradients: 26
// bytes an element, 154.5 M of them 565 us, 7.1 TB/s); 8-bit ones by HBM and
// instruction issue alike (14 bytes, about 54 instructions: 373 us, 5.8 TB/s);
// bfloat16 parameters by issue (10 bytes; 62 instructions, off a 16-byte
// boundary 76: 213 us for 82.3 M, 3.9 TB/s).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <memory>
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
constexpr int kMaxTensors = 400;   // per launch: the table fills the 32 KB of kernel parameters
constexpr int kFewTensors = 44;    // 4 KB: a call of one tensor takes 8.3 us, 9.7 with the large table

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
  int even;       // and its bfloat16 ones begin on 16-byte boundaries
};

struct AdamwParams {
  int n;
  int cautious;
  float b1, b2, omb1, omb2, r2, eps;
  const float* grad_scale;
};
template <int N>
struct AdamwTable : AdamwParams {
  AdamwTensor t[N];
};
static_assert(sizeof(AdamwTable<kMaxTensors>) <= 32764, "kernel parameters are limited to 32764 bytes");

constexpr uint32_t kC0 = 0x9E3779B1u, kC1 = 0x6A09E667u, kC2 = 0xBB67AE85u;

__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
  x = (x ^ (x >> 16)) * kC1;
  x = (x ^ (x >> 15)) * kC2;
  return x ^ (x >> 16);
}

__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

__device__ __forceinline__ float sqrt_approx(float x) {  // below 2^-126: 0
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float sqrt_whole(float x) {
  float y;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float div_whole(float x, float y) {
  float z;
  asm("div.full.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
  return z;
}
__device__ __forceinline__ float max3_abs_nan(float a, float b, float c) {
  float y;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ float warp_max_nan(float a) {
  float y;
  asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(a));
  return y;
}

// Paired product and sum.  The compiler makes one fused operation of a paired
// product and a paired sum that takes it, whatever their rounding modifiers:
// where both have to be rounded the sum is two scalar ones.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add_apart(float2 a, float2 b) { return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y)); }

// A lane's eight entries as four pairs.
struct Eight {
  float2 v[4];
};

__device__ __forceinline__ Eight widen(uint4 q) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  Eight x;
#pragma unroll
  for (int k = 0; k < 4; ++k) x.v[k] = make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
  return x;
}

// A block of a bfloat16 array that begins `off` bytes past a 16-byte boundary
// passes as the 16-byte vectors it touches; shuffles move entries between
// neighbouring lanes (through shared memory the step of 82.3 M bfloat16
// parameters took 226 us in place of 213).  The vectors at its two ends reach into
// the neighbouring blocks: they are read whole (what is not the block's own is
// not used, and another warp may be writing it) and written entry by entry.
__device__ __forceinline__ unsigned offset_of(const void* at) { return static_cast<unsigned>(reinterpret_cast<uintptr_t>(at)) & 15u; }

// Bytes `by` (even, 2 to 14) and on of the eight words a, b.
__device__ __forceinline__ uint4 cut(uint4 a, uint4 b, unsigned by) {
  uint32_t w[7] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z};
  if (by & 8u) w[0] = a.z, w[1] = a.w, w[2] = b.x, w[3] = b.y, w[4] = b.z, w[5] = b.w;
  if (by & 4u) {
#pragma unroll
    for (int k = 0; k < 5; ++k) w[k] = w[k + 1];
  }
  const uint32_t pick = by & 2u ? 0x5432u : 0x3210u;
  return make_uint4(__byte_perm(w[0], w[1], pick), __byte_perm(w[1], w[2], pick), __byte_perm(w[2], w[3], pick),
                    __byte_perm(w[3], w[4], pick));
}

__device__ __forceinline__ uint4 shuffle(uint4 q, int from) {
  return make_uint4(__shfl_sync(0xFFFFFFFFu, q.x, from), __shfl_sync(0xFFFFFFFFu, q.y, from), __shfl_sync(0xFFFFFFFFu, q.z, from),
                    __shfl_sync(0xFFFFFFFFu, q.w, from));
}

// What a lane reads of the warp's 256 entries of an array from `i` on.
struct Raw {
  uint4 a, b;  // float32: eight entries; bfloat16: a, and lane 0 the vector past lane 31's
};

template <bool BF16>
__device__ __forceinline__ Raw fetch(const void* base, long long i, int lane) {
  Raw r{};
  if constexpr (BF16) {
    const __nv_bfloat16* at = static_cast<const __nv_bfloat16*>(base) + i;
    const unsigned off = offset_of(at);
    const uint4* v = reinterpret_cast<const uint4*>(reinterpret_cast<const unsigned char*>(at) - off) + lane;
    r.a = *v;
    if (off != 0 && lane == 0) r.b = v[32];
  } else {
    const uint4* f = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + i + 8 * lane);
    r.a = f[0];
    r.b = f[1];
  }
  return r;
}

// A lane's eight entries from what the warp has read.
template <bool BF16>
__device__ __forceinline__ Eight align(const Raw& r, const void* base, int lane) {
  if constexpr (BF16) {
    const unsigned off = offset_of(base);  // a block is a multiple of 16 bytes
    if (off == 0) return widen(r.a);
    return widen(cut(r.a, shuffle(lane == 0 ? r.b : r.a, (lane + 1) & 31), off));
  } else {
    auto f = [](uint32_t x, uint32_t y) { return make_float2(__uint_as_float(x), __uint_as_float(y)); };
    return {{f(r.a.x, r.a.y), f(r.a.z, r.a.w), f(r.b.x, r.b.y), f(r.b.z, r.b.w)}};
  }
}

__device__ __forceinline__ void store_bf16(__nv_bfloat16* at, int lane, uint4 q) {
  const unsigned off = offset_of(at);
  uint4* v = reinterpret_cast<uint4*>(reinterpret_cast<unsigned char*>(at) - off) + lane;
  if (off == 0) {
    *v = q;
    return;
  }
  const uint4 own = cut(shuffle(q, (lane - 1) & 31), q, 16 - off);
  if (lane > 0) *v = own;
  // the first entries, before the first boundary, and the last ones
  const bool head = lane < static_cast<int>(16 - off) / 2;
  const uint4 end = shuffle(q, head ? 0 : 31);
  const uint32_t word = lane & 4 ? (lane & 2 ? end.w : end.z) : (lane & 2 ? end.y : end.x);
  if (lane < 8) reinterpret_cast<uint16_t*>(at)[head ? lane : 248 + lane] = static_cast<uint16_t>(lane & 1 ? word >> 16 : word);
}

__device__ __forceinline__ void store_f32(float* at, int lane, const Eight& x) {
  float4* f = reinterpret_cast<float4*>(at + 8 * lane);
  f[0] = make_float4(x.v[0].x, x.v[0].y, x.v[1].x, x.v[1].y);
  f[1] = make_float4(x.v[2].x, x.v[2].y, x.v[3].x, x.v[3].y);
}

// Entry `k` of the strided layout: lane + 32 k of the block, 0 past its end.
template <bool BF16>
__device__ __forceinline__ Eight load_strided(const void* base, long long i, int lane, int left) {
  Eight x;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int at = lane + 32 * k;
    float y = 0.0f;
    if (at < left) {
      if constexpr (BF16) y = __bfloat162float(static_cast<const __nv_bfloat16*>(base)[i + at]);
      else y = static_cast<const float*>(base)[i + at];
    }
    (k & 1 ? x.v[k / 2].y : x.v[k / 2].x) = y;
  }
  return x;
}

__device__ __forceinline__ uint2 load_codes_strided(const void* base, long long i, int lane, int left) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int at = lane + 32 * k;
    if (at < left) w[k / 4] |= static_cast<uint32_t>(static_cast<const uint8_t*>(base)[i + at]) << (8 * (k & 3));
  }
  return make_uint2(w[0], w[1]);
}

// Values of eight codes, times the block's scale.
template <bool E4M3>
__device__ __forceinline__ Eight decode(uint2 c, float scale) {
  Eight x;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t w = (k < 2 ? c.x : c.y) >> (16 * (k & 1));
    float2 f;
    if constexpr (E4M3) {
      f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w), __NV_E4M3)));
    } else {  // the upper byte of a half
      const uint32_t h = __byte_perm(w, 0, 0x1404);
      f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    }
    x.v[k] = mul2(f, make_float2(scale, scale));
  }
  return x;
}

// Eight codes of x with 16 random bits each; unit = 2^-E of the block.  The
// integer is shifted so that the code fills its top byte: what the random bits
// are added to lies below, and the sign (E4M3) is put back from x.
template <bool E4M3>
__device__ __forceinline__ uint2 encode(const Eight& x, float unit, const uint32_t (&h)[8]) {
  constexpr float kField = E4M3 ? 0x1p-113f : 0x1p-98f;
  constexpr int kShift = E4M3 ? 4 : 3;
  uint32_t w[2];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t u[4], c[4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float2 y = mul2(mul2(x.v[2 * half + k], make_float2(unit, unit)), make_float2(kField, kField));
      u[2 * k] = __float_as_uint(y.x);
      u[2 * k + 1] = __float_as_uint(y.y);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)  // 0x80, then the low (E4M3) or high 16 random bits
      c[k] = (u[k] << kShift) + __byte_perm(h[4 * half + k], 0x80u, E4M3 ? 0x5104 : 0x5324);
    w[half] = __byte_perm(__byte_perm(c[0], c[1], 0x0073), __byte_perm(c[2], c[3], 0x0073), 0x5410);
    if constexpr (E4M3)
      w[half] = (w[half] & 0x7F7F7F7Fu) |
                (__byte_perm(__byte_perm(u[0], u[1], 0x0073), __byte_perm(u[2], u[3], 0x0073), 0x5410) & 0x80808080u);
    else
      w[half] &= 0x7F7F7F7Fu;
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ float block_max(const Eight& x) {
  float a = max3_abs_nan(x.v[0].x, x.v[0].y, x.v[1].x);
  a = max3_abs_nan(a, x.v[1].y, x.v[2].x);
  a = max3_abs_nan(a, x.v[2].y, x.v[3].x);
  return warp_max_nan(max3_abs_nan(a, x.v[3].y, x.v[3].y));
}

// The step of eight elements: m, v and p in, out.
template <bool WHOLE>
__device__ __forceinline__ void update(const AdamwParams& P, float step, float decay, float gs, const Eight& g, Eight& p, Eight& m,
                                       Eight& v) {
  auto both = [](float a) { return make_float2(a, a); };
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 gk = mul2(g.v[k], both(gs));
    m.v[k] = add_apart(mul2(m.v[k], both(P.b1)), mul2(gk, both(P.omb1)));
    v.v[k] = add_apart(mul2(v.v[k], both(P.b2)), mul2(mul2(gk, gk), both(P.omb2)));
    float2 u;
    if constexpr (WHOLE) {
      const float2 den = __ffma2_rn(make_float2(sqrt_whole(v.v[k].x), sqrt_whole(v.v[k].y)), both(P.r2), both(P.eps));
      u = make_float2(div_whole(m.v[k].x, den.x), div_whole(m.v[k].y, den.y));
    } else {
      const float2 den = __ffma2_rn(make_float2(sqrt_approx(v.v[k].x), sqrt_approx(v.v[k].y)), both(P.r2), both(P.eps));
      u = mul2(m.v[k], make_float2(rcp_approx(den.x), rcp_approx(den.y)));
    }
    float2 dec = mul2(p.v[k], both(decay));
    if (P.cautious) {
      auto agree = [](float a, float b) { return (a > 0.0f && b > 0.0f) || (a < 0.0f && b < 0.0f); };
      if (!agree(u.x, p.v[k].x)) dec.x = 0.0f;
      if (!agree(u.y, p.v[k].y)) dec.y = 0.0f;
    }
    const float2 move = __ffma2_rn(u, both(step), dec);
    p.v[k] = __fadd2_rn(p.v[k], make_float2(-move.x, -move.y));
  }
}

// Rounds p to bfloat16 with the random bits (NaN and infinity as they are).
__device__ __forceinline__ uint4 narrow(const Eight& p, const uint32_t (&h)[8]) {
  float2 bad = make_float2(0.0f, 0.0f);  // 0 times what is not finite is not 0
#pragma unroll
  for (int k = 0; k < 4; ++k) bad = __ffma2_rn(p.v[k], make_float2(0.0f, 0.0f), bad);
  const bool finite = bad.x + bad.y == 0.0f;
  uint32_t u[8], w[4];
#pragma unroll
  for (int k = 0; k < 8; ++k) u[k] = __float_as_uint(k & 1 ? p.v[k / 2].y : p.v[k / 2].x);
  if (finite) {
#pragma unroll
    for (int k = 0; k < 8; ++k) u[k] += h[k] * kC0 >> 16;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if ((u[k] & 0x7F800000u) != 0x7F800000u) u[k] += h[k] * kC0 >> 16;
      else if (u[k] & 0x7FFFFFu) u[k] |= 0x400000u;
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = __byte_perm(u[2 * k], u[2 * k + 1], 0x7632);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// What a lane reads of a whole block in the vector layout.
struct Fetched {
  Raw p, g, m, v;  // float32 moments; codes: a.x and a.y
  float sm, sv;
};

template <bool PB, bool GB, bool B8>
__device__ __forceinline__ Fetched fetch_block(const AdamwTensor& T, long long blk, int lane) {
  const long long i0 = blk * kQBlock;
  Fetched f{};
  f.p = fetch<PB>(T.p, i0, lane);
  f.g = fetch<GB>(T.g, i0, lane);
  if constexpr (B8) {
    const uint2 cm = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(T.m) + i0 + 8 * lane);
    const uint2 cv = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(T.v) + i0 + 8 * lane);
    f.m.a = make_uint4(cm.x, cm.y, 0, 0);
    f.v.a = make_uint4(cv.x, cv.y, 0, 0);
    f.sm = T.ms[blk];
    f.sv = T.vs[blk];
  } else {
    f.m = fetch<false>(T.m, i0, lane);
    f.v = fetch<false>(T.v, i0, lane);
  }
  return f;
}

// One block from what has been read of it; `left` entries in the strided
// layout, all of them (VEC) in the vector layout.
template <bool PB, bool GB, bool B8, bool VEC, bool WHOLE>
__device__ __forceinline__ void step_block(const AdamwParams& P, const AdamwTensor& T, long long blk, int lane, int left, float gs,
                                           Eight& p, const Eight& g, Eight& m, Eight& v) {
  const long long i0 = blk * kQBlock;
  update<WHOLE>(P, T.step, T.decay, gs, g, p, m, v);
  uint32_t h[8];
  if constexpr (B8 || PB) {
    const uint32_t key = T.key + static_cast<uint32_t>(static_cast<unsigned long long>(i0) >> 32) * kC1;
    const uint32_t x0 = static_cast<uint32_t>(i0 + (VEC ? 8 * lane : lane)) * kC0 + key;
#pragma unroll
    for (int k = 0; k < 8; ++k) h[k] = mix(x0 + k * (VEC ? kC0 : 32u * kC0));
  }
  uint2 cm, cv;
  if constexpr (B8) {
    const uint32_t am = __float_as_uint(block_max(m)), av = __float_as_uint(block_max(v));
    const int em = min(max(static_cast<int>(am >> 23) - 127, -100), 126);
    const int ev = min(max(static_cast<int>(av >> 23) - 127, -100), 126);
    cm = encode<true>(m, pow2i(-em), h);
    cv = encode<false>(v, pow2i(-ev), h);
    if (lane == 0) {  // a block with a value that is not finite (or 2^127 and more) becomes NaN
      T.ms[blk] = am < 0x7F000000u ? pow2i(em - 7) : __uint_as_float(0x7FC00000u);
      T.vs[blk] = av < 0x7F000000u ? pow2i(ev - 14) : __uint_as_float(0x7FC00000u);
    }
  }
  if constexpr (VEC) {
    if constexpr (PB) store_bf16(static_cast<__nv_bfloat16*>(T.p) + i0, lane, narrow(p, h));
    else store_f32(static_cast<float*>(T.p) + i0, lane, p);
    if constexpr (B8) {
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(T.m) + i0 + 8 * lane) = cm;
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(T.v) + i0 + 8 * lane) = cv;
    } else {
      store_f32(static_cast<float*>(T.m) + i0, lane, m);
      store_f32(static_cast<float*>(T.v) + i0, lane, v);
    }
  } else {
    uint4 np = make_uint4(0, 0, 0, 0);
    if constexpr (PB) np = narrow(p, h);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int at = lane + 32 * k;
      if (at >= left) continue;
      auto entry = [k](const Eight& x) { return k & 1 ? x.v[k / 2].y : x.v[k / 2].x; };
      if constexpr (PB) {
        const uint32_t w[4] = {np.x, np.y, np.z, np.w};
        static_cast<uint16_t*>(T.p)[i0 + at] = static_cast<uint16_t>(w[k / 2] >> (16 * (k & 1)));
      } else {
        static_cast<float*>(T.p)[i0 + at] = entry(p);
      }
      if constexpr (B8) {
        static_cast<uint8_t*>(T.m)[i0 + at] = static_cast<uint8_t>((k < 4 ? cm.x : cm.y) >> (8 * (k & 3)));
        static_cast<uint8_t*>(T.v)[i0 + at] = static_cast<uint8_t>((k < 4 ? cv.x : cv.y) >> (8 * (k & 3)));
      } else {
        static_cast<float*>(T.m)[i0 + at] = entry(m);
        static_cast<float*>(T.v)[i0 + at] = entry(v);
      }
    }
  }
}

// One block a warp: the CTAs at work then cover one stretch of every array.
// With eight blocks a warp, CTAs 16,384 elements apart, the 8-bit step of
// 100.7 M float32 parameters took 358 us in place of 250.
template <bool PB, bool GB, bool B8, int N, bool WHOLE>
__global__ void __launch_bounds__(kThreads, 4) adamw_kernel(const __grid_constant__ AdamwTable<N> P) {
  int lo = 0, hi = P.n - 1;  // the tensor: largest i with first <= blockIdx.x
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (P.t[mid].first <= static_cast<int>(blockIdx.x)) lo = mid; else hi = mid - 1;
  }
  const AdamwTensor& T = P.t[lo];
  const int lane = threadIdx.x & 31;
  const float gs = P.grad_scale ? *P.grad_scale : 1.0f;
  const long long blk = static_cast<long long>(blockIdx.x - T.first) * kWarps + (threadIdx.x >> 5), i0 = blk * kQBlock;
  if (i0 >= T.numel) return;
  if (!MUON_CHECK(i0 >= 0)) return;
  const int left = static_cast<int>(min(static_cast<long long>(kQBlock), T.numel - i0));
  Eight m, v;
  const bool inner = blk > 0 && i0 + kQBlock + 8 <= T.numel;  // with room for the vectors at both ends
  if (T.vec && left == kQBlock && (T.even || inner)) {
    const Fetched f = fetch_block<PB, GB, B8>(T, blk, lane);
    Eight p = align<PB>(f.p, T.p, lane);
    const Eight g = align<GB>(f.g, T.g, lane);
    if constexpr (B8) {
      m = decode<true>(make_uint2(f.m.a.x, f.m.a.y), f.sm);
      v = decode<false>(make_uint2(f.v.a.x, f.v.a.y), f.sv);
    } else {
      m = align<false>(f.m, T.m, lane);
      v = align<false>(f.v, T.v, lane);
    }
    step_block<PB, GB, B8, true, WHOLE>(P, T, blk, lane, kQBlock, gs, p, g, m, v);
  } else {  // a tensor's last block (and first), and arrays off the vectors' boundaries
    Eight p = load_strided<PB>(T.p, i0, lane, left);
    const Eight g = load_strided<GB>(T.g, i0, lane, left);
    if constexpr (B8) {
      m = decode<true>(load_codes_strided(T.m, i0, lane, left), T.ms[blk]);
      v = decode<false>(load_codes_strided(T.v, i0, lane, left), T.vs[blk]);
    } else {
      m = load_strided<false>(T.m, i0, lane, left);
      v = load_strided<false>(T.v, i0, lane, left);
    }
    step_block<PB, GB, B8, false, WHOLE>(P, T, blk, lane, left, gs, p, g, m, v);
  }
}

template <int N>
using KernelPtr = void (*)(AdamwTable<N>);

// Index: bfloat16 parameters | bfloat16 gradients << 1 | 8-bit moments << 2.
template <int N, bool WHOLE>
const KernelPtr<N> kKernels[8] = {
    adamw_kernel<false, false, false, N, WHOLE>, adamw_kernel<true, false, false, N, WHOLE>,
    adamw_kernel<false, true, false, N, WHOLE>,  adamw_kernel<true, true, false, N, WHOLE>,
    adamw_kernel<false, false, true, N, WHOLE>,  adamw_kernel<true, false, true, N, WHOLE>,
    adamw_kernel<false, true, true, N, WHOLE>,   adamw_kernel<true, true, true, N, WHOLE>,
};

// Whether a lane may take eight neighbouring elements: 16-byte float32 arrays,
// 8-byte codes; bfloat16 arrays may begin anywhere.
bool vector_aligned(const adamw_tensor_desc& d) {
  const uintptr_t state = d.state_bits == 8 ? 8 : 16;
  return (d.param_dtype == MUON_BF16 || aligned_to(d.param, 16)) && (d.grad_dtype == MUON_BF16 || aligned_to(d.grad, 16)) &&
         aligned_to(d.exp_avg, state) && aligned_to(d.exp_avg_sq, state);
}

// The written ranges of a checked list, by address.
void written_ranges(const adamw_tensor_desc* t, int n, std::vector<Span>& spans) {
  spans.clear();
  spans.reserve(static_cast<size_t>(n) * 5);
  for (int i = 0; i < n; ++i) {
    const adamw_tensor_desc& d = t[i];
    if (d.numel == 0) continue;
    const uint64_t n64 = static_cast<uint64_t>(d.numel), nb = (n64 + kQBlock - 1) / kQBlock, ns = d.state_bits == 8 ? 1 : 4;
    spans.push_back(span_of(d.param, n64 * (d.param_dtype == MUON_F32 ? 4 : 2), true));
    spans.push_back(span_of(d.exp_avg, n64 * ns, true));
    spans.push_back(span_of(d.exp_avg_sq, n64 * ns, true));
    if (d.state_bits != 8) continue;
    spans.push_back(span_of(d.exp_avg_scale, nb * 4, true));
    spans.push_back(span_of(d.exp_avg_sq_scale, nb * 4, true));
  }
  std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
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
  std::vector<muon::Span> written;  // no two of them overlap; left empty where no grad_scale comes

  muon_status_t build();
  bool writes(const void* p, uint64_t bytes) const;  // any of these bytes
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
    a.even = aligned_to(d.param, 16) && aligned_to(d.grad, 16);
    l.ctas += (d.numel + kQBlock * kWarps - 1) / (kQBlock * kWarps);
    if (l.ctas > 0x7FFFFFFFLL) return MUON_ERR_TOO_LARGE;
    l.t.push_back(a);
    l.index.push_back(static_cast<int>(i));
  }
  return MUON_OK;
}

bool adamw_plan::writes(const void* p, uint64_t bytes) const {
  const muon::Span s = muon::span_of(p, bytes, false);
  auto next = std::upper_bound(written.begin(), written.end(), s.lo, [](uintptr_t at, const muon::Span& w) { return at < w.lo; });
  return (next != written.begin() && (next - 1)->hi > s.lo) || (next != written.end() && next->lo < s.hi);
}

namespace muon {
namespace {

template <int N, bool WHOLE>
cudaError_t launch(const adamw_plan& plan, const adamw_plan::Launch& l, const AdamwParams& scalars, double bc1, uint32_t key,
                   cudaStream_t s) {
  AdamwTable<N> P;
  static_cast<AdamwParams&>(P) = scalars;
  P.n = static_cast<int>(l.t.size());
  std::memcpy(P.t, l.t.data(), l.t.size() * sizeof(AdamwTensor));
  for (int i = 0; i < P.n; ++i) {
    const adamw_tensor_desc& d = plan.desc[l.index[i]];
    P.t[i].step = static_cast<float>(d.lr / bc1);
    P.t[i].decay = static_cast<float>(d.lr * d.weight_decay);
    P.t[i].key = mix(key + kC0 * static_cast<uint32_t>(l.index[i]));
  }
  kKernels<N, WHOLE>[l.kind]<<<static_cast<unsigned>(l.ctas), kThreads, 0, s>>>(P);
  return cudaGetLastError();
}

muon_status_t run_plan(const adamw_plan& plan, double beta1, double beta2, double eps, int cautious, int64_t step,
                       uint64_t seed, const float* grad_scale, cudaStream_t s) {
  if (step < 1 || !(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0) ||
      !std::isfinite(eps))
    return MUON_ERR_INVALID_ARG;
  if (!aligned_to(grad_scale, 4)) return MUON_ERR_MISALIGNED;
  if (grad_scale && plan.writes(grad_scale, 4)) return MUON_ERR_ALIASING;
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
  AdamwParams P;
  P.cautious = cautious ? 1 : 0;
  P.b1 = static_cast<float>(beta1);
  P.b2 = static_cast<float>(beta2);
  P.omb1 = static_cast<float>(1.0 - beta1);
  P.omb2 = static_cast<float>(1.0 - beta2);
  P.r2 = static_cast<float>(1.0 / std::sqrt(bc2));
  P.eps = static_cast<float>(eps);
  P.grad_scale = grad_scale;
  const bool whole = P.eps < 0x1p-41f * P.r2;
  for (const auto& l : plan.launches) {
    const bool few = l.t.size() <= static_cast<size_t>(kFewTensors);
    const cudaError_t e = whole ? launch<kMaxTensors, true>(plan, l, P, bc1, k, s)
                          : few ? launch<kFewTensors, false>(plan, l, P, bc1, k, s)
                                : launch<kMaxTensors, false>(plan, l, P, bc1, k, s);
    if (e != cudaSuccess) return MUON_ERR_CUDA;
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
    std::unique_ptr<adamw_plan> p(new adamw_plan);
    p->desc.assign(tensors, tensors + n_tensors);
    st = p->build();
    if (st != MUON_OK) return st;
    muon::written_ranges(tensors, n_tensors, p->written);
    *plan = p.release();
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
    next.written.swap(plan->written);  // the same arrays
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
    if (grad_scale) muon::written_ranges(tensors, n_tensors, p.written);
    return muon::run_plan(p, beta1, beta2, eps, cautious, step, seed, grad_scale, static_cast<cudaStream_t>(stream));
  } catch (const std::bad_alloc&) {
    return MUON_ERR_HOST_MEMORY;
  }
}

}  // extern "C"
