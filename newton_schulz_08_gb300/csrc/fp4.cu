// Quantisation to 4-bit floating point with block scales, and its inverse.
//
// A code is E2M1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign.  `block` consecutive
// entries along the axis that a product contracts share a scale:
//   block 32: 2^e, the least with max |x| <= 6 2^e, as E8M0;
//   block 16: 2^k s, s = E4M3(max |x| / 6 / 2^k), 2^k the tensor's, the least
//     with max |x| <= 6 448 2^k (fp4_amax_kernel finds the maximum).
// Power-of-two factors are exact, so the quotient x / scale is rounded at most
// once (a division by s, whose reciprocal is corrected by its remainder),
// and nothing depends on the launch.
//
// One pass writes the codes along the rows, those across them (the operand of
// the transposed product), or both: a CTA takes 128 x 128 entries, so that
// either way its scales are whole 512-byte tiles of the layout that the
// product copies to TMEM, and each row of codes is 64 bytes.  Codes along a row
// come from the registers of the loads (8 entries a thread, the maximum over
// 2 or 4 neighbouring lanes); those across from the same entries in shared
// memory, two columns by 32 rows a thread.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <new>
#include <vector>

#include "../../include/muon.h"
#include "check.cuh"
#include "fp4.h"
#include "host.h"

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
  float* scale;       // block 16: the tensor's 2^k and max |x|
};

constexpr uint32_t kC0 = 0x9E3779B1u, kC1 = 0x6A09E667u, kC2 = 0xBB67AE85u;

__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
  x = (x ^ x >> 16) * kC1;
  x = (x ^ x >> 15) * kC2;
  return x ^ x >> 16;
}

// Random bits of entries 2 j and 2 j + 1 of a row of the operand (low and
// high half), j counted through the operand.
__device__ __forceinline__ uint32_t random32(uint64_t j, uint32_t key) {
  return mix(static_cast<uint32_t>(j) * kC0 + key + static_cast<uint32_t>(j >> 32) * kC1);
}

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// 2^e, e in -127 .. 127.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(e < -126 ? 1u << 22 : static_cast<uint32_t>(e + 127) << 23); }

// Exponent of the tensor's power of two from the bits of its largest finite magnitude.
__device__ __forceinline__ int tensor_exponent(uint32_t amax) {
  return max(static_cast<int>((amax + (0x7FFFFFu - 0x280000u)) >> 23) - 138, -127);  // 2688 = 1.3125 * 2^11
}

// A block's scale: its code, and what its entries are divided by.
struct Scale {
  uint32_t code;
  float up;     // block 32: entries times this are in units of the scale; block 16: times 2^-k
  float s, r;   // block 16: then divided by s, r = 1 / s rounded
};

template <int BLOCK, bool SR>
__device__ __forceinline__ Scale block_scale(uint32_t amax, float up_tensor) {
  Scale q;
  const bool bad = amax >= 0x7F800000u;  // infinite or NaN
  if constexpr (BLOCK == 32) {
    const int e = max(static_cast<int>((amax + 0x3FFFFFu) >> 23) - 129, -127);  // 6 = 1.5 * 2^2
    q.code = bad ? 0xFFu : static_cast<uint32_t>(e + 127);
    q.up = bad ? 0.0f : pow2(-e);
    q.s = q.r = 1.0f;
  } else {
    const float sixth = __fdiv_rn(__uint_as_float(amax), 6.0f), want = sixth * up_tensor;
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
    q.code = bad ? 0x7Fu : code;
    q.up = bad ? 0.0f : up_tensor;
    q.r = code == 0 ? 0.0f : __frcp_rn(q.s);
  }
  return q;
}

template <int BLOCK>
__device__ __forceinline__ float in_units(float x, const Scale& q) {
  float y = x * q.up;
  if constexpr (BLOCK == 16) {
    // y / s to nearest: the product with the rounded reciprocal, corrected by its remainder
    // (which would turn -0 into 0)
    const float t = y * q.r;
    y = copysignf(fmaf(fmaf(-t, q.s, y), q.r, t), x);
  }
  return y;
}

// Two codes, `lo` in the low half of a byte.
__device__ __forceinline__ uint32_t codes_nearest(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\tcvt.u32.u8 %0, b;\n\t}" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// One code: the significand's kept bits after a random number below the last
// of them is added.  Magnitudes below 1 are moved up by 1, where the spacing
// 0.5 of the codes is that of the kept bits; the sum is rounded towards zero,
// which decides as the exact one does.
__device__ __forceinline__ uint32_t code_random(float y, uint32_t r16) {
  const float a = fminf(fabsf(y), 6.0f);
  const bool small = a < 1.0f;
  const float t = small ? __fadd_rz(a, 1.0f) : a;
  const uint32_t c = ((__float_as_uint(t) + (r16 << 6) + 32u) >> 22) - (small ? 254u : 252u);
  return c | (__float_as_uint(y) >> 28 & 8u);
}

template <bool SR>
__device__ __forceinline__ uint32_t code_pair(float lo, float hi, uint32_t bits) {
  if constexpr (SR) return code_random(lo, bits & 0xFFFFu) | code_random(hi, bits >> 16) << 4;
  return codes_nearest(lo, hi);
}

// Eight entries of a row from column c0 on, zeros past its end.
template <bool BF16>
__device__ __forceinline__ void load8(const QuantParams& P, long long row, int c0, float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = 0.0f;
  if (row >= P.rows || c0 >= P.cols) return;
  const long long at = row * P.stride + c0;
  if (P.vec && c0 + 8 <= P.cols) {
    if constexpr (BF16) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(P.x) + at));
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] = __uint_as_float(w[k] << 16);
        v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
      }
    } else {
      const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(P.x) + at);
      const float4 a = __ldg(f), b = __ldg(f + 1);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (c0 + k >= P.cols) continue;
    if constexpr (BF16)
      v[k] = __bfloat162float(static_cast<const __nv_bfloat16*>(P.x)[at + k]);
    else
      v[k] = static_cast<const float*>(P.x)[at + k];
  }
}

constexpr int kStagePitch = 80;  // bytes of a staged row of codes across: 64 and a gap

template <bool BF16>
__host__ __device__ constexpr int tile_bytes() { return kTile * kTile * (BF16 ? 2 : 4); }

template <bool BF16, int BLOCK, bool SR, bool ALONG, bool ACROSS>
__global__ void __launch_bounds__(kThreads) fp4_quantize_kernel(const __grid_constant__ QuantParams P) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kTiles = 32 / BLOCK;  // scale tiles of 128 entries of K
  __shared__ __align__(16) uint8_t sf_along[kTiles * 512], sf_across[kTiles * 512];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x;
  const int by = static_cast<int>(blockIdx.x) / P.tiles_x, bx = static_cast<int>(blockIdx.x) - by * P.tiles_x;
  const int r0 = by * kTile, c0 = bx * kTile;
  float up = 1.0f;
  if constexpr (BLOCK == 16) {
    const int k = tensor_exponent(__float_as_uint(P.scale[1]));
    up = pow2(-k);
    if (blockIdx.x == 0 && tid == 0) P.scale[0] = pow2(k);
  }
  uint8_t* tile = smem;
  uint8_t* stage = smem + tile_bytes<BF16>();
  {
    const int g = tid & 15;  // 8 columns
    const int col = c0 + 8 * g;
    constexpr int kBatch = 4;
#pragma unroll
    for (int half = 0; half < 8 / kBatch; ++half) {
      float v[kBatch][8];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) load8<BF16>(P, r0 + (half * kBatch + i) * 16 + (tid >> 4), col, v[i]);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int r = (half * kBatch + i) * 16 + (tid >> 4);
        if constexpr (ACROSS) {
          if constexpr (BF16) {
            uint4 w;
            w.x = __byte_perm(__float_as_uint(v[i][0]), __float_as_uint(v[i][1]), 0x7632);
            w.y = __byte_perm(__float_as_uint(v[i][2]), __float_as_uint(v[i][3]), 0x7632);
            w.z = __byte_perm(__float_as_uint(v[i][4]), __float_as_uint(v[i][5]), 0x7632);
            w.w = __byte_perm(__float_as_uint(v[i][6]), __float_as_uint(v[i][7]), 0x7632);
            *reinterpret_cast<uint4*>(tile + r * (kTile * 2) + g * 16) = w;
          } else {
            float4* t = reinterpret_cast<float4*>(tile + r * (kTile * 4) + g * 32);
            t[0] = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
            t[1] = make_float4(v[i][4], v[i][5], v[i][6], v[i][7]);
          }
        }
        if constexpr (ALONG) {
          uint32_t m = 0;
#pragma unroll
          for (int k = 0; k < 8; ++k) m = max(m, magnitude(v[i][k]));
          m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
          if constexpr (BLOCK == 32) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
          const Scale q = block_scale<BLOCK, SR>(m, up);
          uint32_t word = 0;
          const uint64_t j = static_cast<uint64_t>(r0 + r) * ((P.cols + 1) / 2) + col / 2;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t bits = SR ? random32(j + k, P.along.key) : 0u;
            float lo = in_units<BLOCK>(v[i][2 * k], q), hi = in_units<BLOCK>(v[i][2 * k + 1], q);
            if (q.up == 0.0f) lo = hi = 0.0f;  // 0 times what is not finite
            word |= code_pair<SR>(lo, hi, bits) << (8 * k);
          }
          if (r0 + r < P.rows && col / 2 < P.along.pitch &&
              MUON_CHECK(col >= 0 && col / 2 + 4 <= P.along.pitch))
            *reinterpret_cast<uint32_t*>(P.along.codes + (r0 + r) * P.along.pitch + col / 2) = word;
          const int b = BLOCK == 32 ? g >> 2 : g >> 1;
          if ((g & (BLOCK / 8 - 1)) == 0)
            sf_along[(b >> 2) * 512 + (r & 31) * 16 + (r >> 5) * 4 + (b & 3)] = r0 + r < P.rows ? q.code : 0;
        }
      }
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
    // two columns by 32 rows a thread
    const int cp = tid & 63, rb = tid >> 6;
    float v[2][32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const int r = rb * 32 + i;
      if constexpr (BF16) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(tile + r * (kTile * 2) + cp * 4);
        v[0][i] = __uint_as_float(w << 16);
        v[1][i] = __uint_as_float(w & 0xFFFF0000u);
      } else {
        const float2 f = *reinterpret_cast<const float2*>(tile + r * (kTile * 4) + cp * 8);
        v[0][i] = f.x;
        v[1][i] = f.y;
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = 2 * cp + h;
      uint32_t word[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int b = 0; b < 32 / BLOCK; ++b) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < BLOCK; ++i) m = max(m, magnitude(v[h][b * BLOCK + i]));
        const Scale q = block_scale<BLOCK, SR>(m, up);
        const uint64_t j = static_cast<uint64_t>(c0 + c) * ((P.rows + 1) / 2) + (r0 + rb * 32 + b * BLOCK) / 2;
#pragma unroll
        for (int k = 0; k < BLOCK / 2; ++k) {
          const uint32_t bits = SR ? random32(j + k, P.across.key) : 0u;
          float lo = in_units<BLOCK>(v[h][b * BLOCK + 2 * k], q), hi = in_units<BLOCK>(v[h][b * BLOCK + 2 * k + 1], q);
          if (q.up == 0.0f) lo = hi = 0.0f;
          const int byte = b * BLOCK / 2 + k;
          word[byte >> 2] |= code_pair<SR>(lo, hi, bits) << (8 * (byte & 3));
        }
        const int blk = rb * (32 / BLOCK) + b;  // along K within the tile
        sf_across[(blk >> 2) * 512 + (c & 31) * 16 + (c >> 5) * 4 + (blk & 3)] = c0 + c < P.cols ? q.code : 0;
      }
      *reinterpret_cast<uint4*>(stage + c * kStagePitch + rb * 16) = make_uint4(word[0], word[1], word[2], word[3]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int piece = i * kThreads + tid, c = piece >> 2, at = (piece & 3) * 16;
      const long long byte = r0 / 2 + at;
      if (c0 + c < P.cols && byte < P.across.pitch && MUON_CHECK(byte + 16 <= P.across.pitch))
        *reinterpret_cast<uint4*>(P.across.codes + (c0 + c) * P.across.pitch + byte) =
            *reinterpret_cast<const uint4*>(stage + c * kStagePitch + at);
    }
    const long long kt = static_cast<long long>(by) * kTiles + (tid >> 5);
    if (tid < 32 * kTiles && bx < P.across.row_tiles && kt < P.across.ktiles)
      reinterpret_cast<uint4*>(P.across.scales + (bx * P.across.ktiles + kt) * 512)[tid & 31] =
          reinterpret_cast<const uint4*>(sf_across)[tid];
  }
}

// Largest finite magnitude of a matrix, as the bits of a float, into *out (0 before).
template <bool BF16>
__global__ void __launch_bounds__(kThreads) fp4_amax_kernel(const __grid_constant__ QuantParams P, uint32_t* out) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint32_t m = 0;
  const int groups = (P.cols + 7) / 8;
  // 16 rows x 128 columns a step: 16 threads a row
  const long long steps_c = (groups + 15) / 16, steps = steps_c * ((P.rows + 15) / 16);
  for (long long s = blockIdx.x; s < steps; s += gridDim.x) {
    float v[8];
    const long long sr = s / steps_c;
    load8<BF16>(P, sr * 16 + (threadIdx.x >> 4), static_cast<int>(s - sr * steps_c) * 128 + (threadIdx.x & 15) * 8, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t a = magnitude(v[k]);
      if (a < 0x7F800000u) m = max(m, a);
    }
  }
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if ((threadIdx.x & 31) == 0 && m) atomicMax(out, m);
}

// The numbers that codes stand for: 8 codes a thread.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) fp4_values_kernel(const uint8_t* codes, const uint8_t* scales, const float* scale,
                                                              int rows, int cols, int block, long long pitch,
                                                              long long ktiles, void* out, long long stride, int vec) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int groups = (cols + 7) / 8;
  const float tensor = block == 16 ? *scale : 1.0f;
  const long long total = static_cast<long long>(rows) * groups;
  for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * kThreads) {
    const long long r = i / groups;
    const int c = static_cast<int>(i - r * groups) * 8;
    const uint32_t word = *reinterpret_cast<const uint32_t*>(codes + r * pitch + c / 2);
    const long long b = c / block;
    const uint32_t code = scales[((r >> 7) * ktiles + (b >> 2)) * 512 + (r & 31) * 16 + ((r & 127) >> 5) * 4 + (b & 3)];
    float s;
    if (block == 32) {
      s = code == 255 ? NAN : pow2(static_cast<int>(code) - 127);
    } else {
      s = code == 0x7F ? NAN : code < 8 ? code * 0.001953125f : __uint_as_float((code << 20) + (120u << 23));
      s *= tensor;
    }
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t q = word >> (4 * k) & 15u, e = q >> 1 & 3u, m = q & 1u;
      const float a = e == 0 ? 0.5f * m : __uint_as_float((126u + e) << 23 | m << 22);
      v[k] = (q & 8u ? -a : a) * s;
    }
    if constexpr (BF16) {
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out) + r * stride + c;
      if (vec && c + 8 <= cols) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
          w[k] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(o) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (c + k < cols) o[k] = __float2bfloat16_rn(v[k]);
      }
    } else {
      float* o = static_cast<float*>(out) + r * stride + c;
      if (vec && c + 8 <= cols) {
        reinterpret_cast<float4*>(o)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(o)[1] = make_float4(v[4], v[5], v[6], v[7]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (c + k < cols) o[k] = v[k];
      }
    }
  }
}

cudaError_t launch(const void* fn, dim3 grid, int smem, void** args, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
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
  const int smem = across ? (bf16 ? tile_bytes<true>() : tile_bytes<false>()) + kTile * kStagePitch : 0;
  if (smem > 40 * 1024 && cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return MUON_ERR_CUDA;
  if (block == 16) {
    if (cudaMemsetAsync(P.scale + 1, 0, 4, str) != cudaSuccess) return MUON_ERR_CUDA;
    uint32_t* bits = reinterpret_cast<uint32_t*>(P.scale + 1);
    const int64_t steps = (rows + 15) / 16 * ((cols + 127) / 128);
    void* args[] = {&P, &bits};
    if (launch(bf16 ? reinterpret_cast<const void*>(&fp4_amax_kernel<true>) : reinterpret_cast<const void*>(&fp4_amax_kernel<false>),
               dim3(static_cast<unsigned>(std::min<int64_t>(steps, sms * 8))), 0, args, str) != cudaSuccess)
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
  int rows = static_cast<int>(q->rows), cols = static_cast<int>(q->cols), block = q->block;
  long long pitch = fp4_pitch(q->cols), ktiles = fp4_ktiles(q->cols, block), stride = out_stride;
  int vec = aligned_to(out, 16) && out_stride * size % 16 == 0;
  const int64_t groups = q->rows * ((q->cols + 7) / 8);
  void* args[] = {&codes, &scales, &scale, &rows, &cols, &block, &pitch, &ktiles, &out, &stride, &vec};
  if (launch(dtype == MUON_BF16 ? reinterpret_cast<const void*>(&fp4_values_kernel<true>)
                                : reinterpret_cast<const void*>(&fp4_values_kernel<false>),
             dim3(static_cast<unsigned>(std::min<int64_t>((groups + kThreads - 1) / kThreads, sms * 32))), 0, args,
             static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return MUON_ERR_CUDA;
  return MUON_OK;
}
