// Quantisation to 4-bit floating point with block scales, and its inverse.
//
// A code is E2M1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign.  `block` consecutive
// entries along the axis that a product contracts share a scale:
//   block 32: 2^e, the least with max |x| <= 6 2^e, as E8M0;
//   block 16: 2^k s, s = E4M3(max |x| / 6 / 2^k), 2^k the tensor's, the least
//     with max |x| <= 6 448 2^k (fp4_amax_kernel finds the maximum).
// Power-of-two factors are exact, so the quotient x / scale is rounded at most
// once, and nothing depends on the launch.  Quotients by s and by 6 are products
// with the divisor's reciprocal, corrected by their remainder (Markstein 1990): the
// result is the correctly rounded quotient where the reciprocal is the nearest number to 1 / s, the
// product within a spacing of the quotient, and the remainder no subnormal number.
//
// One pass writes the codes along the rows, those across them (the operand of
// the transposed product), or both: a CTA takes 128 x 128 entries, so that
// either way its scales are whole 512-byte tiles of the layout that the
// product copies to TMEM, and each row of codes is 64 bytes.  The tile is
// copied to shared memory with cp.async (at any alignment of the rows); codes
// along a row are made 32 bytes a lane, those across two bfloat16 columns or
// one float32 column by 32 rows a thread, and leave through shared memory in 16-byte pieces.
//
// Bound by memory while rounding to nearest with blocks of 32 (maxima are taken of
// packed halves, quotients by multiplication), by instructions with
// stochastic rounding (a hash per two entries, an addition and a shift each:
// arithmetic pipes 86 % busy); blocks of 16 read x once more for the tensor's
// maximum.  Measured, 16384 x 6400 bfloat16: along 44 us (0.90 of the
// measured copy bandwidth), across 45, both 60 (0.80), both stochastic 130;
// blocks of 16: along 83, both 126, both stochastic 219.  fp4_values of
// 50304 x 768 to bfloat16: 20 us (0.71).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <exception>
#include <mutex>
#include <new>
#include <set>
#include <utility>
#include <vector>

#include "../../include/muon.h"
#include "check.cuh"
#include "fp4.h"
#include "host.h"
#include "rows.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = kFp4Tile;

struct Target {
  uint8_t* codes;     // null: not written
  uint8_t* scales;
  long long pitch;    // bytes of a row of codes
  long long ktiles;   // scale tiles along a row
  long long row_tiles;
  uint32_t key;       // of the random bits
};

struct QuantParams {
  const void* x;
  long long stride;
  int rows, cols;
  int vec;            // rows may be read in 16-byte vectors
  int tiles_x;        // CTAs along a row
  Target along, across;
  float* scale;       // block 16: the tensor's 2^k, its max |x|, and that of each of the `parts` of fp4_amax_kernel
  int parts;
};

constexpr int kMaxParts = FP4_SCALE_FLOATS - 2;
constexpr int kAmaxThreads = 1024;

constexpr uint32_t kC0 = 0x9E3779B1u, kC1 = 0x6A09E667u, kC2 = 0xBB67AE85u;

__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
  x = (x ^ x >> 16) * kC1;
  x = (x ^ x >> 15) * kC2;
  return x ^ x >> 16;
}

// Random bits of entries 2 (j + k) and 2 (j + k) + 1 of the operand (low and high
// half), counted through its rows; j is a multiple of 4 or k is 0 .. 3 of
// one row, so that only j may carry into the upper half.
__device__ __forceinline__ uint32_t random32(uint64_t j, int k, uint32_t key) {
  const uint64_t i = j + static_cast<uint64_t>(k);
  return mix(static_cast<uint32_t>(i) * kC0 + key + static_cast<uint32_t>(i >> 32) * kC1);
}

using rows::Pair;

// 2^e, e in -127 .. 127.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(e < -126 ? 1u << 22 : static_cast<uint32_t>(e + 127) << 23); }

// Exponent of the tensor's power of two from the bits of its largest finite magnitude.
__device__ __forceinline__ int tensor_exponent(uint32_t amax) {
  return max(static_cast<int>((amax + (0x7FFFFFu - 0x280000u)) >> 23) - 138, -127);  // 2688 = 1.3125 * 2^11
}

// A block's scale: its code, and what its entries are divided by.
struct Scale {
  uint32_t code;  // 0xFF / 0x7F: NaN
  float up;       // block 32: entries times this are in units of the scale; block 16: times 2^-k
  float s, r;     // block 16: then divided by s, r = 1 / s rounded (0 for 0)
};

template <int BLOCK>
__host__ __device__ constexpr uint32_t nan_code() { return BLOCK == 32 ? 0xFFu : 0x7Fu; }

template <int BLOCK, bool SR>
__device__ __forceinline__ Scale block_scale(uint32_t amax, float up_tensor) {
  Scale q;
  const bool bad = amax >= 0x7F800000u;  // infinite or NaN
  if constexpr (BLOCK == 32) {
    const int e = max(static_cast<int>((amax + 0x3FFFFFu) >> 23) - 129, -127);  // 6 = 1.5 * 2^2
    q.code = bad ? nan_code<32>() : static_cast<uint32_t>(e + 127);
    q.up = bad ? 0.0f : __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    q.s = q.r = 1.0f;
  } else {
    // max / 6 to nearest: Markstein's correction; by a division where the remainder may be a subnormal number
    const float top = __uint_as_float(amax), t = top * (1.0f / 6.0f);
    float sixth = fmaf(fmaf(t, -6.0f, top), 1.0f / 6.0f, t);
    if (amax < (27u << 23) || bad) sixth = __fdiv_rn(top, 6.0f);  // below 2^-100
    const float want = sixth * up_tensor;
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(0.0f), "f"(bad ? 0.0f : want));
    auto value = [](uint32_t code) {
      const float normal = __uint_as_float((code << 20) + (120u << 23));
      return code < 8 ? static_cast<float>(code) * 0.001953125f : normal;
    };
    uint32_t code = c & 0x7Fu;
    // upwards: nothing is cut off, so that rounding stays right in the mean (`want` may have left float32's range)
    if (SR && !bad && (code == 0 ? sixth > 0.0f : value(code) < want)) ++code;
    q.s = value(code);
    q.code = bad ? nan_code<16>() : code;
    q.up = bad ? 0.0f : up_tensor;
    // 1 / s to nearest: a Newton-Raphson step from the hardware's reciprocal, which is within a spacing (the step rounds to
    // nearest for any significand but one of all ones; s has four significant bits)
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(q.s));
    q.r = code == 0 ? 0.0f : fmaf(r, fmaf(-q.s, r, 1.0f), r);
  }
  return q;
}

// Eight numbers by their scale, rounded to nearest.  Blocks of 16: x / s by
// Markstein's correction; its remainder is a subnormal number only where the
// quotient is far below the least code either way.  Signs are chosen so that a zero keeps its own.
template <int BLOCK>
__device__ __forceinline__ void in_units(Pair (&x)[4], const Scale& q) {
  if constexpr (BLOCK == 32) {
    const Pair up = rows::pair(q.up);
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = rows::mul(x[k], up);
  } else {
    const Pair up = rows::pair(-q.up), r = rows::pair(-q.r), s = rows::pair(q.s);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const Pair y = rows::mul(x[k], up), t = rows::mul(y, r);
      x[k] = rows::fma(rows::fma(t, s, y), r, t);
    }
  }
}

// Eight codes, the first in the low bits, of numbers in units of their scale.
__device__ __forceinline__ uint32_t codes_nearest(const Pair (&y)[4]) {
  float v[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) rows::split(y[k], v[2 * k], v[2 * k + 1]);
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return w;
}

// The same with random numbers: a random number below the last kept bit of the
// significand is added and the rest dropped.  Times 2^-126, rounded towards zero
// (which decides as the exact number does), magnitudes below 1 are float32's
// subnormal numbers, whose spacing is that of the codes 0 and 0.5: then the
// exponent and the highest bit of the significand are the code.  `bits`: one word per two numbers.
template <int BLOCK>
__device__ __forceinline__ uint32_t codes_random(const Pair (&y)[4], const uint32_t (&bits)[4]) {
  const Pair least = rows::pair(__uint_as_float(1u << 23));  // 2^-126
  uint32_t w = 0;
#pragma unroll
  for (int k = 3; k >= 0; --k) {
    Pair t;
    asm("mul.rz.f32x2 %0, %1, %2;" : "=l"(t) : "l"(y[k]), "l"(least));
    float v[2];
    rows::split(t, v[0], v[1]);
#pragma unroll
    for (int h = 1; h >= 0; --h) {
      const uint32_t b = __float_as_uint(v[h]);
      // (the largest code may be passed by the quotient's rounding: blocks of 16)
      uint32_t m = b << 6;
      if (BLOCK == 16) m = min(m, 7u << 28);
      const uint32_t r = ((h ? bits[k] >> 4 : bits[k] << 12) & 0x0FFFF000u) | 0x800u;
      w = __funnelshift_l((m + r) | (b & 0x80000000u), w, 4);
    }
  }
  return w;
}

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {  // of unsigned halves
  uint32_t m;
  asm("max.u16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
  return m;
}

// A row of the tile in shared memory: 128 entries, and where rows do not begin on
// 16 bytes one unit more, as they lie in memory.
template <bool BF16>
struct Tile {
  static constexpr int size = BF16 ? 2 : 4;
  // a lane's entries of a row: two units of 16 bytes (float32 with 16 entries a lane, whose units lie 64 bytes
  // apart: 144 us for 16384 x 6400 both ways, 121 with 8; bfloat16 with 8: 68, 60 with 16)
  static constexpr int units = 2, entries = 32 / size, lanes = kTile / entries, rows = kThreads / lanes;
  static constexpr int pitch = kTile * size + 16;       // bytes of a row
  static constexpr int bytes = kTile * pitch;
};

constexpr int kStagePitch = kTile + 4;            // words: codes of 8 rows, by row and column
constexpr int kStageBytes = 16 * kStagePitch * 4;

template <bool BF16, bool ACROSS>
__host__ __device__ constexpr int tile_smem() { return Tile<BF16>::bytes + (ACROSS ? kStageBytes : 0); }

template <bool BF16>
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return BF16 ? max2(a, b) : max(a, b); }

// Eight numbers of a lane's: bfloat16, the first (h = 0) or second half.
template <bool BF16>
__device__ __forceinline__ void numbers8(const uint4 (&q)[2], int h, Pair (&x)[4]) {
  if constexpr (BF16) {
    rows::numbers<true>(q[h], x);
  } else {
    x[0] = rows::pair(__uint_as_float(q[0].x), __uint_as_float(q[0].y));
    x[1] = rows::pair(__uint_as_float(q[0].z), __uint_as_float(q[0].w));
    x[2] = rows::pair(__uint_as_float(q[1].x), __uint_as_float(q[1].y));
    x[3] = rows::pair(__uint_as_float(q[1].z), __uint_as_float(q[1].w));
  }
}

// The codes of eight numbers with this scale; `j`: of their first pair.
template <int BLOCK, bool SR>
__device__ __forceinline__ uint32_t codes8(Pair (&x)[4], const Scale& q, uint64_t j, uint32_t key) {
  in_units<BLOCK>(x, q);
  uint32_t w;
  if constexpr (SR) {
    uint32_t bits[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) bits[k] = random32(j, k, key);
    w = codes_random<BLOCK>(x, bits);
  } else {
    w = codes_nearest(x);
  }
  return q.code == nan_code<BLOCK>() ? 0u : w;  // (0 times what is not finite)
}

template <bool BF16, int BLOCK, bool SR, bool ALONG, bool ACROSS>
__global__ void __launch_bounds__(kThreads, BF16 ? 5 : 3) fp4_quantize_kernel(const __grid_constant__ QuantParams P) {
  using T = Tile<BF16>;
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kTiles = 32 / BLOCK;  // scale tiles of 128 entries of K
  __shared__ __align__(16) uint8_t sf_along[kTiles * 512], sf_across[kTiles * 512];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x;
  const int by = static_cast<int>(blockIdx.x) / P.tiles_x, bx = static_cast<int>(blockIdx.x) - by * P.tiles_x;
  const int r0 = by * kTile, c0 = bx * kTile;
  const uint32_t tile = rows::shared_address(smem);
  // T::lanes lanes a row, T::rows rows at a time
  const int g = tid % T::lanes, row = tid / T::lanes, col = c0 + T::entries * g;
  {
    const char* p = static_cast<const char*>(P.x) + ((r0 + row) * P.stride + c0) * T::size;
    uint32_t to = tile + row * T::pitch + g * (16 * T::units);
#pragma unroll
    for (int i = 0; i < kTile / T::rows; ++i) {
      const uint32_t shift = P.vec ? 0u : rows::shift_of(p);
      const char* from = p - shift;
      // bytes from the row's first unit here on that belong to it
      const int bytes = r0 + row + T::rows * i < P.rows ? min(P.cols - c0, kTile + 8) * T::size + static_cast<int>(shift) : 0;
#pragma unroll
      for (int u = 0; u < T::units + 1; ++u) {
        const int at = (g * T::units + u) * 16, have = min(max(bytes - at, 0), 16);
        if (u < T::units || (g == T::lanes - 1 && shift != 0)) rows::copy_ahead(to + 16 * u, have ? from + at : static_cast<const char*>(P.x) - rows::shift_of(P.x), have);
      }
      p += T::rows * P.stride * T::size;
      to += T::rows * T::pitch;
    }
    rows::copies_commit();
  }
  float up = 1.0f;
  if constexpr (BLOCK == 16) {
    uint32_t top = 0;
    for (int i = tid & 31; i < P.parts; i += 32) top = max(top, __float_as_uint(P.scale[2 + i]));
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    const int k = tensor_exponent(top);
    up = pow2(-k);
    if (blockIdx.x == 0 && tid == 0) {
      P.scale[0] = pow2(k);
      P.scale[1] = __uint_as_float(top);
    }
  }
  rows::copies_wait(0);
  __syncwarp();
  if (ALONG || !P.vec) {
    uint32_t at = tile + row * T::pitch + g * (16 * T::units);
    uint8_t* out = P.along.codes + (r0 + row) * P.along.pitch + col / 2;
    uint64_t j = static_cast<uint64_t>(r0 + row) * ((P.cols + 1) / 2) + col / 2;
    const char* p = static_cast<const char*>(P.x) + ((r0 + row) * P.stride + c0) * T::size;
#pragma unroll 1
    for (int i = 0; i < kTile / T::rows; ++i) {
      const int r = row + T::rows * i;
      uint4 q[T::units];
#pragma unroll
      for (int u = 0; u < T::units; ++u) q[u] = rows::shared_load(at + 16 * u);
      if (!P.vec) {  // to the lane's own place, for those who read columns
        const uint32_t shift = rows::shift_of(p);
        const uint4 next = rows::shared_load(at + 16 * T::units);
        if (shift) {
#pragma unroll
          for (int u = 0; u < T::units; ++u) q[u] = rows::funnel(q[u], u + 1 < T::units ? q[u + 1] : next, shift);
        }
        __syncwarp();
        if constexpr (ACROSS) {
#pragma unroll
          for (int u = 0; u < T::units; ++u) rows::shared_store(at + 16 * u, q[u]);
        }
        p += T::rows * P.stride * T::size;
      }
      if constexpr (ALONG) {
        uint32_t m = 0;
#pragma unroll
        for (int u = 0; u < T::units; ++u) {
          constexpr uint32_t k = BF16 ? 0x7FFF7FFFu : 0x7FFFFFFFu;
          m = larger<BF16>(m, larger<BF16>(larger<BF16>(q[u].x & k, q[u].y & k), larger<BF16>(q[u].z & k, q[u].w & k)));
        }
        constexpr int kShare = BLOCK / T::entries;  // lanes of a block
        if constexpr (kShare > 1) m = larger<BF16>(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        if constexpr (kShare > 2) m = larger<BF16>(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        if constexpr (BF16) m = max(m << 16, m & 0xFFFF0000u);
        const Scale sc = block_scale<BLOCK, SR>(m, up);
        uint32_t word[2];
#pragma unroll
        for (int h = 0; h < T::entries / 8; ++h) {
          Pair x[4];
          numbers8<BF16>(q, h, x);
          word[h] = codes8<BLOCK, SR>(x, sc, j + 4 * h, P.along.key);
        }
        const bool inside = r0 + r < P.rows;
        if (inside && col / 2 < P.along.pitch && MUON_CHECK(col >= 0 && col / 2 + T::entries / 2 <= P.along.pitch)) {
          if constexpr (BF16)
            *reinterpret_cast<uint2*>(out) = make_uint2(word[0], word[1]);
          else
            *reinterpret_cast<uint32_t*>(out) = word[0];
        }
        const int b = g / kShare;
        if (g % kShare == 0) sf_along[(b >> 2) * 512 + (r & 31) * 16 + (r >> 5) * 4 + (b & 3)] = inside ? sc.code : 0;
        out += T::rows * P.along.pitch;
        j += static_cast<uint64_t>(T::rows) * ((P.cols + 1) / 2);
      }
      at += T::rows * T::pitch;
    }
  }
  __syncthreads();
  if constexpr (ALONG) {
    const long long kt = static_cast<long long>(bx) * kTiles + (tid >> 5);
    if (tid < 32 * kTiles && by < P.along.row_tiles && kt < P.along.ktiles)
      reinterpret_cast<uint4*>(P.along.scales + (by * P.along.ktiles + kt) * 512)[tid & 31] =
          reinterpret_cast<const uint4*>(sf_along)[tid];
  }
  if constexpr (ACROSS) {
    // 32 rows of a column at a time: bfloat16, two columns a thread; float32, one, twice
    constexpr int kColumns = BF16 ? 2 : 1;
    uint32_t* stage = reinterpret_cast<uint32_t*>(smem + T::bytes);
#pragma unroll 1
    for (int pass = 0; pass < 2 / kColumns; ++pass) {
      const int item = pass * kThreads + tid;
      const int cp = BF16 ? item & 63 : item & 127, rb = BF16 ? item >> 6 : item >> 7;
      const uint32_t from = tile + rb * 32 * T::pitch + cp * 4;
      auto word_at = [&](int i) {
        uint32_t w;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(from + i * T::pitch) : "memory");
        return w;
      };
#pragma unroll 1
      for (int b = 0; b < 32 / BLOCK; ++b) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < BLOCK; ++i) top = larger<BF16>(top, word_at(b * BLOCK + i) & (BF16 ? 0x7FFF7FFFu : 0x7FFFFFFFu));
        Scale sc[kColumns];
#pragma unroll
        for (int h = 0; h < kColumns; ++h) {
          const int c = kColumns * cp + h, blk = rb * (32 / BLOCK) + b;  // blk: along K within the tile
          sc[h] = block_scale<BLOCK, SR>(BF16 ? (h ? top & 0xFFFF0000u : top << 16) : top, up);
          sf_across[(blk >> 2) * 512 + (c & 31) * 16 + (c >> 5) * 4 + (blk & 3)] = c0 + c < P.cols ? sc[h].code : 0;
        }
#pragma unroll 1
        for (int o = b * (BLOCK / 8); o < (b + 1) * (BLOCK / 8); ++o) {
          uint32_t v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = word_at(8 * o + i);
#pragma unroll
          for (int h = 0; h < kColumns; ++h) {
            const int c = kColumns * cp + h;
            Pair x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t lo = v[2 * k], hi = v[2 * k + 1];
              if constexpr (BF16)
                x[k] = h ? rows::pair(__uint_as_float(lo & 0xFFFF0000u), __uint_as_float(hi & 0xFFFF0000u))
                         : rows::pair(__uint_as_float(lo << 16), __uint_as_float(hi << 16));
              else
                x[k] = rows::pair(__uint_as_float(lo), __uint_as_float(hi));
            }
            const uint64_t j = SR ? static_cast<uint64_t>(c0 + c) * ((P.rows + 1) / 2) + (r0 + rb * 32 + 8 * o) / 2 : 0;
            stage[(rb * 4 + o) * kStagePitch + c] = codes8<BLOCK, SR>(x, sc[h], j, P.across.key);
          }
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int piece = i * kThreads + tid, c = piece >> 2, w = (piece & 3) * 4;
      const long long byte = r0 / 2 + w * 4;
      if (c0 + c < P.cols && byte < P.across.pitch && MUON_CHECK(byte + 16 <= P.across.pitch))
        *reinterpret_cast<uint4*>(P.across.codes + (c0 + c) * P.across.pitch + byte) =
            make_uint4(stage[w * kStagePitch + c], stage[(w + 1) * kStagePitch + c], stage[(w + 2) * kStagePitch + c],
                       stage[(w + 3) * kStagePitch + c]);
    }
    const long long kt = static_cast<long long>(by) * kTiles + (tid >> 5);
    if (tid < 32 * kTiles && bx < P.across.row_tiles && kt < P.across.ktiles)
      reinterpret_cast<uint4*>(P.across.scales + (bx * P.across.ktiles + kt) * 512)[tid & 31] =
          reinterpret_cast<const uint4*>(sf_across)[tid];
  }
}

// Largest finite magnitude of a matrix: each CTA leaves that of its part in
// out[blockIdx.x] (one atomic maximum would have to be cleared first: 3001 x 1217
// float32 both ways 31 us in a graph with that, 19 so).  A warp takes 128 units
// of 16 bytes of a row.  Units are those of memory; entries beside the row are
// left out of the first and the last one.  Contiguous rows are read as rows of
// any other length (the last one shorter).
template <bool BF16>
__global__ void __launch_bounds__(kAmaxThreads) fp4_amax_kernel(const char* x, long long stride, int cols, long long total, int pieces,
                                                            long long items, float* out) {
  constexpr int size = BF16 ? 2 : 4, per = 16 / size;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  uint32_t top = 0;
  constexpr int kWarps = kAmaxThreads / 32;
  const long long step = static_cast<long long>(gridDim.x) * kWarps;
  for (long long item = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); item < items; item += step) {
    const long long r = items <= 0x7FFFFFFF ? static_cast<long long>(static_cast<uint32_t>(item) / static_cast<uint32_t>(pieces)) : item / pieces;
    const int k0 = static_cast<int>(item - r * pieces) * 128 + lane;
    const char* p = x + r * stride * size;
    const int before = static_cast<int>(rows::shift_of(p)) / size;
    const int n = static_cast<int>(min(static_cast<long long>(cols), total - r * stride));
    p -= before * size;
    uint4 q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = k0 + 32 * i;
      q[i] = k * per < before + n ? __ldg(reinterpret_cast<const uint4*>(p) + k) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      constexpr uint32_t mask = BF16 ? 0x7FFF7FFFu : 0x7FFFFFFFu;
      const uint4 a = make_uint4(q[i].x & mask, q[i].y & mask, q[i].z & mask, q[i].w & mask);
      uint32_t m = larger<BF16>(larger<BF16>(a.x, a.y), larger<BF16>(a.z, a.w));
      if constexpr (BF16) m = max(m << 16, m & 0xFFFF0000u);
      const int e0 = (k0 + 32 * i) * per - before;  // entry of the row that the unit begins with
      if (m >= 0x7F800000u || e0 < 0 || e0 + per > n) {  // some are not finite or not the row's: one by one
        m = 0;
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int k = 0; k < per; ++k) {
          const uint32_t v = BF16 ? (k & 1 ? w[k >> 1] & 0xFFFF0000u : w[k >> 1] << 16) : w[k & 3];
          if (v < 0x7F800000u && e0 + k >= 0 && e0 + k < n) m = max(m, v);
        }
      }
      top = max(top, m);
    }
  }
  __shared__ uint32_t part[kWarps];
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if (lane == 0) part[threadIdx.x >> 5] = top;
  __syncthreads();
  if (threadIdx.x < 32) {
    top = __reduce_max_sync(0xFFFFFFFFu, part[lane]);
    if (lane == 0) out[blockIdx.x] = __uint_as_float(top);
  }
}

// The numbers that codes stand for: 128 rows x 256 columns a CTA, whose scales are
// whole tiles; a warp takes 16 rows, a lane 8 codes (4 bytes) of each.  E2M1 numbers
// as bfloat16 come byte-wise from two tables of 8 that fit in registers.
template <bool BF16, int BLOCK>
__global__ void __launch_bounds__(kThreads) fp4_values_kernel(const uint8_t* codes, const uint8_t* scales, const float* scale,
                                                              int rows, int cols, int tiles_x, long long pitch,
                                                              long long ktiles, void* out, long long stride, int vec) {
  constexpr int kTiles = 64 / BLOCK, kRows = kTile / (kThreads / 32), kBatch = 8;
  __shared__ __align__(16) uint8_t sf[kTiles * 512];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int by = static_cast<int>(blockIdx.x) / tiles_x, bx = static_cast<int>(blockIdx.x) - by * tiles_x;
  const int c = bx * 256 + lane * 8, r0 = warp * kRows;  // r0: within the tile
  // A factor past 2^118, whose product with a block's scale may leave float32's range though 0 times it, or half of it,
  // does not, is taken as 2^16 times less and the codes' numbers as that much more (never so with fp4_quantize's factors).
  float tensor = BLOCK == 16 ? *scale : 1.0f;
  const bool far = BLOCK == 16 && fabsf(tensor) > 0x1p118f && !isinf(tensor);
  if (far) tensor *= 0x1p-16f;
  const uint32_t below2 = far ? 0x47474700u : 0x3F3F3F00u, from2 = far ? 0x48484848u : 0x40404040u;
  if (threadIdx.x < 32 * kTiles)
    reinterpret_cast<uint4*>(sf)[threadIdx.x] = __ldg(reinterpret_cast<const uint4*>(scales + (by * ktiles + bx * kTiles) * 512) + threadIdx.x);
  const uint8_t* from = codes + (static_cast<long long>(by) * kTile + r0) * pitch + c / 2;
  const long long at = (static_cast<long long>(by) * kTile + r0) * stride + c;
  const int n = c < cols ? min(kRows, rows - by * kTile - r0) : 0;
  __syncthreads();
#pragma unroll 1
  for (int base = 0; base < kRows; base += kBatch) {
    uint32_t word[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      word[i] = base + i < n ? __ldg(reinterpret_cast<const uint32_t*>(from + (base + i) * pitch)) : 0u;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (base + i >= n) continue;
      const int r = r0 + base + i, b = lane * 8 / BLOCK;
      const uint32_t code = sf[(b >> 2) * 512 + (r & 31) * 16 + (r >> 5) * 4 + (b & 3)];
      float s;
      if constexpr (BLOCK == 32) {
        s = code == 255 ? NAN : pow2(static_cast<int>(code) - 127);
      } else {
        s = code == 0x7F ? NAN : code < 8 ? code * 0.001953125f : __uint_as_float((code << 20) + (120u << 23));
        s *= tensor;
      }
      Pair v[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t four = word[i] >> (16 * h), select = four & 0x7777u;
        const uint32_t hi = __byte_perm(below2, from2, select), lo = __byte_perm(0xC0800000u, 0xC0804000u, select);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t x = __byte_perm(lo, hi, k ? 0x62 : 0x40) << 16, y = __byte_perm(lo, hi, k ? 0x73 : 0x51) << 16;
          const uint32_t sx = four << (28 - 8 * k) & 0x80000000u, sy = four << (24 - 8 * k) & 0x80000000u;
          v[2 * h + k] = rows::mul(rows::pair(__uint_as_float(x | sx), __uint_as_float(y | sy)), rows::pair(s));
        }
      }
      char* o = static_cast<char*>(out) + (at + (base + i) * stride) * (BF16 ? 2 : 4);
      if constexpr (BF16) {
        const uint4 q = rows::pack<true>(v);
        if (vec && c + 8 <= cols)
          *reinterpret_cast<uint4*>(o) = q;
        else
          rows::store_some<true>(o, q, 0, cols - c);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const Pair two[2] = {v[2 * h], v[2 * h + 1]};
          const uint4 q = rows::pack<false>(two);
          if (vec && c + 8 <= cols)
            reinterpret_cast<uint4*>(o)[h] = q;
          else
            rows::store_some<false>(o + 16 * h, q, 0, cols - c - 4 * h);
        }
      }
    }
  }
}

cudaError_t launch(const void* fn, dim3 grid, int smem, void** args, cudaStream_t stream, int threads = kThreads) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, fn, args);
}

template <bool BF16, int BLOCK, bool SR>
const void* quantize_fn(bool along, bool across) {
  if (along && across) return reinterpret_cast<const void*>(&fp4_quantize_kernel<BF16, BLOCK, SR, true, true>);
  if (along) return reinterpret_cast<const void*>(&fp4_quantize_kernel<BF16, BLOCK, SR, true, false>);
  return reinterpret_cast<const void*>(&fp4_quantize_kernel<BF16, BLOCK, SR, false, true>);
}

template <bool BF16>
const void* quantize_fn(int block, bool random, bool along, bool across) {
  if (block == 32)
    return random ? quantize_fn<BF16, 32, true>(along, across) : quantize_fn<BF16, 32, false>(along, across);
  return random ? quantize_fn<BF16, 16, true>(along, across) : quantize_fn<BF16, 16, false>(along, across);
}

// Raises a kernel's limit of shared memory at its first use on the current device.
bool raise_limit(const void* fn, int smem) try {
  static std::mutex mu;
  static std::set<std::pair<int, const void*>> done;
  int dev = 0;
  if (smem <= 40 * 1024) return true;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  std::lock_guard<std::mutex> lk(mu);
  if (done.count({dev, fn})) return true;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return false;
  done.insert({dev, fn});
  return true;
} catch (const std::exception&) {  // (none crosses a C entry)
  return false;
}

uint64_t matrix_bytes(int64_t rows, int64_t cols, int64_t stride, int size) {
  return rows && cols ? (static_cast<uint64_t>(rows - 1) * stride + cols) * size : 0;
}

}  // namespace

MUON_CHECK_READER(check_failures_fp4)

}  // namespace muon

using namespace muon;

extern "C" size_t fp4_codes_size(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || rows > kFp4MaxDim || cols > kFp4MaxDim) return 0;
  return static_cast<size_t>(rows) * fp4_pitch(cols);
}

extern "C" size_t fp4_scales_size(int64_t rows, int64_t cols, int block) {
  if (rows < 0 || cols < 0 || rows > kFp4MaxDim || cols > kFp4MaxDim || (block != 16 && block != 32)) return 0;
  return static_cast<size_t>(fp4_row_tiles(rows)) * fp4_ktiles(cols, block) * 512;
}

extern "C" muon_status_t fp4_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int64_t row_stride,
                                      const fp4_matrix* along, const fp4_matrix* across, int stochastic,
                                      uint64_t seed, void* stream) {
  if ((dtype != MUON_BF16 && dtype != MUON_F32) || rows < 0 || cols < 0 || row_stride < cols || (!along && !across))
    return MUON_ERR_INVALID_ARG;
  if (rows > kFp4MaxDim || cols > kFp4MaxDim || row_stride > (1LL << 32)) return MUON_ERR_TOO_LARGE;
  for (const fp4_matrix* m : {along, across}) {
    if (!m) continue;
    const muon_status_t st = fp4_check(m);
    if (st != MUON_OK) return st;
  }
  if (along && (along->rows != rows || along->cols != cols)) return MUON_ERR_INVALID_ARG;
  if (across && (across->rows != cols || across->cols != rows)) return MUON_ERR_INVALID_ARG;
  if (along && across && (along->block != across->block || along->scale != across->scale)) return MUON_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return MUON_OK;
  if (!x) return MUON_ERR_INVALID_ARG;
  const int size = dtype == MUON_F32 ? 4 : 2;
  if (!aligned_to(x, size)) return MUON_ERR_MISALIGNED;
  const fp4_matrix& first = along ? *along : *across;
  const int block = first.block;
  // CTAs of 128 x 128 entries, with the padding of either target's scales
  const int64_t gx = std::max(along ? (cols + 255) / 256 * 2 : 0, (cols + 127) / 128);
  const int64_t gy = std::max(across ? (rows + 255) / 256 * 2 : 0, (rows + 127) / 128);
  if (gx * gy > 0x7FFFFFFF) return MUON_ERR_TOO_LARGE;
  try {
    std::vector<Span> v = {span_of(x, matrix_bytes(rows, cols, row_stride, size), false)};
    if (along) fp4_spans(v, *along, true);
    if (across) {
      fp4_matrix m = *across;
      if (along) m.scale = nullptr;  // the same one
      fp4_spans(v, m, true);
    }
    if (spans_conflict(v)) return MUON_ERR_ALIASING;
  } catch (const std::bad_alloc&) {
    return MUON_ERR_HOST_MEMORY;
  }
  int sms = 0;
  const muon_status_t dev = device_sms(sms);
  if (dev != MUON_OK) return dev;
  QuantParams P{};
  P.x = x;
  P.stride = row_stride;
  P.rows = static_cast<int>(rows);
  P.cols = static_cast<int>(cols);
  P.vec = aligned_to(x, 16) && row_stride * size % 16 == 0;
  P.tiles_x = static_cast<int>(gx);
  P.scale = first.scale;
  auto target = [&](const fp4_matrix* m, uint32_t axis) {
    Target t{};
    if (!m) return t;
    t.codes = static_cast<uint8_t*>(m->codes);
    t.scales = static_cast<uint8_t*>(m->scales);
    t.pitch = fp4_pitch(m->cols);
    t.ktiles = fp4_ktiles(m->cols, block);
    t.row_tiles = fp4_row_tiles(m->rows);
    t.key = mix(mix(static_cast<uint32_t>(seed) + kC0 * axis) ^ static_cast<uint32_t>(seed >> 32));
    return t;
  };
  P.along = target(along, 1);
  P.across = target(across, 0);
  cudaStream_t str = static_cast<cudaStream_t>(stream);
  const bool bf16 = dtype == MUON_BF16;
  const void* fn = bf16 ? quantize_fn<true>(block, stochastic != 0, along != nullptr, across != nullptr)
                        : quantize_fn<false>(block, stochastic != 0, along != nullptr, across != nullptr);
  const int smem = across ? (bf16 ? tile_smem<true, true>() : tile_smem<false, true>())
                          : (bf16 ? tile_smem<true, false>() : tile_smem<false, false>());
  if (!raise_limit(fn, smem)) return MUON_ERR_CUDA;
  if (block == 16) {
    const int per = 16 / size;
    const char* p = static_cast<const char*>(x);
    // contiguous rows as rows of 128 units of memory
    const bool begin = aligned_to(x, 16), flat = row_stride == cols && rows * cols > 128 * per;
    const int run = (begin ? 128 : 127) * per;
    long long stride = flat ? run : row_stride, total = flat ? rows * cols : INT64_MAX;
    int length = static_cast<int>(flat ? run : cols);
    int pieces = static_cast<int>(((length + per - 1LL) / per + (begin && stride % per == 0 ? 0 : 1) + 127) / 128);
    long long items = (flat ? (total + stride - 1) / stride : rows) * pieces;
    float* parts = P.scale + 2;
    P.parts = static_cast<int>(std::min<int64_t>((items + kAmaxThreads / 32 - 1) / (kAmaxThreads / 32), std::min(sms, kMaxParts)));
    void* args[] = {&p, &stride, &length, &total, &pieces, &items, &parts};
    if (launch(bf16 ? reinterpret_cast<const void*>(&fp4_amax_kernel<true>) : reinterpret_cast<const void*>(&fp4_amax_kernel<false>),
               dim3(static_cast<unsigned>(P.parts)), 0, args, str, kAmaxThreads) != cudaSuccess)
      return MUON_ERR_CUDA;
  }
  void* args[] = {&P};
  if (launch(fn, dim3(static_cast<unsigned>(gx * gy)), smem, args, str) != cudaSuccess)
    return MUON_ERR_CUDA;
  return MUON_OK;
}

extern "C" muon_status_t fp4_values(const fp4_matrix* q, void* out, int dtype, int64_t out_stride, void* stream) {
  const muon_status_t st = fp4_check(q);
  if (st != MUON_OK) return st;
  if ((dtype != MUON_BF16 && dtype != MUON_F32) || out_stride < q->cols) return MUON_ERR_INVALID_ARG;
  if (out_stride > (1LL << 32)) return MUON_ERR_TOO_LARGE;
  if (q->rows == 0 || q->cols == 0) return MUON_OK;
  if (!out) return MUON_ERR_INVALID_ARG;
  const int size = dtype == MUON_F32 ? 4 : 2;
  if (!aligned_to(out, size)) return MUON_ERR_MISALIGNED;
  try {
    std::vector<Span> v = {span_of(out, matrix_bytes(q->rows, q->cols, out_stride, size), true)};
    fp4_spans(v, *q, false);
    if (spans_conflict(v)) return MUON_ERR_ALIASING;
  } catch (const std::bad_alloc&) {
    return MUON_ERR_HOST_MEMORY;
  }
  int sms = 0;
  const muon_status_t dev = device_sms(sms);
  if (dev != MUON_OK) return dev;
  const uint8_t* codes = static_cast<const uint8_t*>(q->codes);
  const uint8_t* scales = static_cast<const uint8_t*>(q->scales);
  const float* scale = q->scale;
  const int64_t tiles = (q->cols + 255) / 256;
  if (tiles * fp4_row_tiles(q->rows) > 0x7FFFFFFF) return MUON_ERR_TOO_LARGE;
  int rows = static_cast<int>(q->rows), cols = static_cast<int>(q->cols), tiles_x = static_cast<int>(tiles);
  long long pitch = fp4_pitch(q->cols), ktiles = fp4_ktiles(q->cols, q->block), stride = out_stride;
  int vec = aligned_to(out, 16) && out_stride * size % 16 == 0;
  void* args[] = {&codes, &scales, &scale, &rows, &cols, &tiles_x, &pitch, &ktiles, &out, &stride, &vec};
  const void* fn = q->block == 32 ? (dtype == MUON_BF16 ? reinterpret_cast<const void*>(&fp4_values_kernel<true, 32>)
                                                        : reinterpret_cast<const void*>(&fp4_values_kernel<false, 32>))
                                  : (dtype == MUON_BF16 ? reinterpret_cast<const void*>(&fp4_values_kernel<true, 16>)
                                                        : reinterpret_cast<const void*>(&fp4_values_kernel<false, 16>));
  if (launch(fn, dim3(static_cast<unsigned>(tiles * fp4_row_tiles(q->rows))), 0, args, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return MUON_ERR_CUDA;
  return MUON_OK;
}
