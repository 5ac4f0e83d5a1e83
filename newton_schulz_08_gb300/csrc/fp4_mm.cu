// Product of two matrices in 4-bit codes with block scales, C = A B^T, on the
// sm_103a tensor cores (tcgen05.mma with block scales, K = 64 per instruction,
// fp32 accumulators in TMEM).
//
//   out[i][j] = sum over blocks b of  sa[i][b] sb[j][b] sum_k a[i][k] b[j][k]
//
// (times the tensors' factors for blocks of 16).  Codes arrive in shared
// memory by TMA, 256 entries of K (128 bytes, 128-byte swizzle) a stage; their
// scales arrive as whole 512-byte tiles and one instruction copies such a tile
// to the 4 TMEM columns where the MMAs read it.
//
// Two kernels share the roles (a TMA producer, an MMA issuer, epilogue warps;
// every wait is bounded, see ns_gemm.cu):
//   fp4_pair_kernel   many tiles: persistent pairs of CTAs, 256 x 256 tiles
//     with cta_group::2.  Two accumulators of 256 columns and 48 columns of
//     scales do not fit into 512: the accumulators overlap by 48 columns.  The
//     epilogue reads the half of its columns that holds the overlap first, and
//     the next tile's MMAs start then.
//   fp4_tile_kernel   few tiles: a CTA computes 128 x BN (BN 32, 64, 128; the
//     larger matrix gives the 128 rows, so a few tokens are the narrow side), and
//     a cluster of up to 8 CTAs splits K: each sends every CTA its partial sums
//     of that one's rows of the tile, and each adds them in the order of the
//     CTAs, so equal calls give equal bits.
// Large products are bound by the tensor cores and, with short K, by the
// epilogue's writes; small ones by latency (a few stages of K, the sums over
// the cluster).  What it took:
//   - the MMA warp stays converged and one elected lane issues, so that
//     descriptors stay in uniform registers: 8192^3 257 -> 167 us;
//   - an accumulator is given back without waiting for the epilogue's stores
//     (a relaxed arrival; the reads of TMEM are complete by then): 167 -> 156;
//   - scales by tcgen05.cp: put into TMEM by warps (tcgen05.st) 8192^3 took 397 us.
// Measured (blocks of 32, bfloat16 out, m x n x k): 8192^3 155 us, 7.1 PFLOP/s (3.65 times the
// measured bf16 rate), blocks of 16 160; 16384 x 6400 x 1600 75 (0.58 of four times
// that rate, 0.46 of the bandwidth), 6400 x 1600 x 16384 66; 512 x 6400 x 1600
// 8.0, 3 x 6400 x 1600 5.4, 64 x 8192 x 8192 11.6 (weights in the L2; 16 from memory, 0.35 of the bandwidth).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstring>
#include <mutex>
#include <new>
#include <vector>

#include "../../include/muon.h"
#include "check.cuh"
#include "fp4.h"
#include "host.h"
#include "plan.h"
#include "ptx.cuh"
#include "rows.cuh"

namespace muon {
namespace {

constexpr int kDepthBytes = kFp4Depth / 2;  // of a row of codes per stage

struct MmParams {
  CUtensorMap codes_a, codes_b;    // bytes, box 128 x 128 (narrow side: BN rows), 128-byte swizzle
  CUtensorMap scales_a, scales_b;  // 512-byte tiles as rows, box: the tiles of a stage
  const float* scale_a;            // factors of the tensors, or null
  const float* scale_b;
  void* out;
  long long stride;
  int m, n, k;                     // rows of a, rows of b, entries of a row
  int tiles_m, tiles_n;
  int ktiles;                      // scale tiles along a row of either matrix
  int f32;                         // out: float32, else bfloat16
  int vec;                         // rows of out in 16-byte vectors
  int swapped;                     // tile kernel: a holds out's columns, b its rows
  int* status;
  long long wait_budget;
  int inject_stall;
};

__device__ __forceinline__ void raise_timeout(const MmParams& P, volatile int* abort) {
  *abort = 1;
  atomicOr(P.status, kStatusTimeout);
}

// The product of the tensors' factors as two factors: what an accumulator is
// multiplied with, one after the other.  Where the product is a normal number it is the first one, rounded
// once (exact for powers of two, which fp4_quantize writes), and the second is 1.  Where
// it is below those, the first is the product times 2^126, so that the sum is rounded at the last step;
// where it is above float32's range, the two are as they are.
struct Factors {
  float a, b;
};
__device__ __forceinline__ Factors tensor_factors(const MmParams& P) {
  if (!P.scale_a) return {1.0f, 1.0f};
  const float x = *P.scale_a, y = *P.scale_b, p = x * y;
  if (isinf(p)) return {x, y};
  if (fabsf(p) < 0x1p-126f) {  // (then the smaller one is below 2^-63)
    const bool less = fabsf(x) < fabsf(y);
    return {(less ? x : y) * 0x1p126f * (less ? y : x), 0x1p-126f};
  }
  return {p, 1.0f};
}

// The tensors' factors, on 32 accumulators.
__device__ __forceinline__ void scale32(const MmParams& P, const Factors& f, uint32_t (&r)[32]) {
  if (!P.scale_a) return;
#pragma unroll
  for (int k = 0; k < 32; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * f.a);
  if (f.b != 1.0f) {
#pragma unroll
    for (int k = 0; k < 32; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * f.b);
  }
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Scale tiles of a stage (4 scales each): 2 for blocks of 32, 4 for blocks of 16.
template <int BLOCK>
constexpr int kGroups = kFp4Depth / (4 * BLOCK);

// Writes 32 rows x 64 columns of accumulators, a row per lane, through the
// warp's 4 KB of shared memory in whole 128-byte lines: rows row0 .. and
// columns col0 .. of out.
__device__ __forceinline__ void store_rows(const MmParams& P, uint32_t stage, int lane, int row0, int col0,
                                           uint32_t (&lo)[32], uint32_t (&hi)[32], const Factors& f) {
  const int size = P.f32 ? 4 : 2, width = 128 / size;
  scale32(P, f, lo);
  scale32(P, f, hi);
  // this lane's 16 bytes of every fourth row
  const int j = lane & 7, r0 = lane >> 3, left = P.m - row0 - r0;
  const long long step = 4 * P.stride * size;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c0 = col0 + h * width;
    if ((h && !P.f32) || c0 >= P.n) break;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (P.f32) {
          w[e] = h ? hi[4 * k + e] : lo[4 * k + e];
        } else {
          const uint32_t(&half)[32] = k < 4 ? lo : hi;
          w[e] = pack_bf16x2(__uint_as_float(half[8 * (k & 3) + 2 * e]), __uint_as_float(half[8 * (k & 3) + 2 * e + 1]));
        }
      }
      ptx::sts128(stage + lane * 128 + ((k ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
    }
    __syncwarp();
    char* at = static_cast<char*>(P.out) + ((row0 + r0) * P.stride + c0) * size;
    if (P.vec && c0 + width <= P.n) {
      at += j * 16;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        uint32_t a, b, c, d;
        ptx::lds128(stage + (4 * k + r0) * 128 + ((j ^ ((4 * k + r0) & 7)) << 4), a, b, c, d);
        if (4 * k < left && MUON_CHECK(c0 + (j + 1) * 16 / size <= P.n)) *reinterpret_cast<uint4*>(at) = make_uint4(a, b, c, d);
        at += step;
      }
    } else {
      // rows off the 16-byte boundaries, or ending here: each lane composes an
      // aligned unit of two neighbouring pieces; units with entries of others are stored by the entry
      const int per = 16 / size, have = min(width, P.n - c0);
#pragma unroll 1
      for (int k = 0; 4 * k < min(left, 32 - r0); ++k, at += step) {
        const int r = 4 * k + r0;
        auto piece = [&](int p) {
          uint4 q;
          ptx::lds128(stage + r * 128 + ((p ^ (r & 7)) << 4), q.x, q.y, q.z, q.w);
          return q;
        };
        const uint32_t shift = rows::shift_of(at);
        const int before = static_cast<int>(shift) / size;
        const uint4 last = piece(j);
        uint4 q = last;
        if (shift) q = rows::funnel(piece(j ? j - 1 : 0), q, 16 - shift);
        const int first = j ? 0 : before, room = min(per, have + before - j * per);
        char* to = at + 16 * j - static_cast<int>(shift);
        if (first == 0 && room == per)
          *reinterpret_cast<uint4*>(to) = q;
        else if (P.f32)
          rows::store_some<false>(to, q, first, room);
        else
          rows::store_some<true>(to, q, first, room);
        if (j == 7 && shift) {
          q = rows::funnel(last, last, 16 - shift);
          const int end = min(before, have + before - 8 * per);
          if (P.f32)
            rows::store_some<false>(to + 16, q, 0, end);
          else
            rows::store_some<true>(to + 16, q, 0, end);
        }
      }
    }
  }
  __syncwarp();
}

// ------------------------------------------------------------------- pairs
constexpr int kPairStages = 5;
constexpr int kPairEpiWarps = 8;
constexpr int kPairThreads = 64 + 32 * kPairEpiWarps;
constexpr int kPairCodes = 128 * kDepthBytes;                       // of either operand per CTA and stage
constexpr int kPairScalesA = 4 * 512, kPairScalesB = 2 * 4 * 512;   // room for blocks of 16
constexpr int kPairStage = 2 * kPairCodes + kPairScalesA + kPairScalesB;
constexpr int kPairSmem = kPairStages * kPairStage + kPairEpiWarps * 4096 + 1024 + 256;
constexpr int kAccStep = 208;                                        // columns from one accumulator to the other
constexpr int kScaleCol = 464;                                       // scales: 16 columns of A, 32 of B

template <int BLOCK>
__global__ void __launch_bounds__(kPairThreads, 1) fp4_pair_kernel(const __grid_constant__ MmParams P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int kG = kGroups<BLOCK>;
  constexpr uint32_t kBytes = 2 * kPairCodes + 3 * kG * 512;  // of a CTA per stage
  uint8_t* staging = smem + kPairStages * kPairStage;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + kPairEpiWarps * 4096);
  uint64_t* full = bars;                    // leader: both CTAs' stage landed
  uint64_t* empty = bars + kPairStages;     // stage free in this CTA
  uint64_t* tfull = bars + 2 * kPairStages; // [2] accumulator ready
  uint64_t* tempty = tfull + 2;             // leader: what the next tile overwrites has been read
  uint64_t* drain = tempty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* never = reinterpret_cast<volatile int*>(tmem_slot + 2);  // stays 0

  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  const int pair = static_cast<int>(ptx::cluster_id_x()), npairs = static_cast<int>(ptx::nclusters_x());
  const int total = P.tiles_m * P.tiles_n;
  const int kblocks = (P.k + kFp4Depth - 1) / kFp4Depth;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      ptx::mbar_init(ptx::smem_addr(&full[s]), 1);
      ptx::mbar_init(ptx::smem_addr(&empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) ptx::mbar_init(ptx::smem_addr(&tfull[a]), 1);
    ptx::mbar_init(ptx::smem_addr(tempty), 2 * kPairEpiWarps);
    ptx::mbar_init(ptx::smem_addr(drain), 1);
    *abort = 0;
    *never = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(ptx::smem_addr(tmem_slot), 512);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  __syncwarp();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  if (threadIdx.x == 0) {
    ptx::prefetch_tmap(&P.codes_a);
    ptx::prefetch_tmap(&P.codes_b);
    ptx::prefetch_tmap(&P.scales_a);
    ptx::prefetch_tmap(&P.scales_b);
  }
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  if (blockIdx.x == 0 && threadIdx.x == 0) *P.status = 0;
  const uint32_t tmem = *tmem_slot;
  const long long budget = P.wait_budget;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------------------- producer
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = pair; ok && t < total; t += npairs) {
        const int I = t % P.tiles_m, J = t / P.tiles_m;
        const int ra = 2 * I + static_cast<int>(rank);  // 128-row tile of A
        for (int kb = 0; kb < kblocks; ++kb) {
          if (!ptx::mbar_wait(ptx::smem_addr(&empty[stage]), phase ^ 1, budget, abort)) {
            raise_timeout(P, abort);
            ok = false;
            break;
          }
          const uint32_t fb = ptx::map_to_rank(ptx::smem_addr(&full[stage]), 0);
          const uint32_t sa = ptx::smem_addr(smem + stage * kPairStage), sb = sa + kPairCodes;
          const uint32_t fa = sb + kPairCodes, fbs = fa + kPairScalesA;
          if (rank == 0) ptx::mbar_arrive_expect_tx(ptx::smem_addr(&full[stage]), 2 * kBytes);
          ptx::tma_load_2d_pair(sa, &P.codes_a, fb, kb * kDepthBytes, ra * 128);
          ptx::tma_load_2d_pair(sb, &P.codes_b, fb, kb * kDepthBytes, J * 256 + static_cast<int>(rank) * 128);
          ptx::tma_load_2d_pair(fa, &P.scales_a, fb, 0, ra * P.ktiles + kb * kG);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            ptx::tma_load_2d_pair(fbs + j * kG * 512, &P.scales_b, fb, 0, (2 * J + j) * P.ktiles + kb * kG);
          if (++stage == kPairStages) stage = 0, phase ^= 1;
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && !P.inject_stall) {
      // -------------------------------------------------------- MMA issuer
      // The whole warp runs the loop and one lane issues: what the instructions
      // take is the same in every lane and stays in uniform registers.
      int stage = 0, it = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = pair; ok && t < total; t += npairs, ++it) {
        const int acc = it & 1;
        // the epilogue has read what this tile's accumulator shares with the last one's
        ok = it == 0 || ptx::mbar_wait_cluster(ptx::smem_addr(tempty), (it - 1) & 1, budget, abort);
        if (!ok) raise_timeout(P, abort);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t d = tmem + acc * kAccStep;
        for (int kb = 0; kb < kblocks; ++kb) {
          const uint32_t sa = ptx::smem_addr(smem + stage * kPairStage), sb = sa + kPairCodes;
          const uint32_t fa = sb + kPairCodes, fb = fa + kPairScalesA;
          const uint64_t a0 = ptx::sdesc_sw128(sa, 16, 1024), b0 = ptx::sdesc_sw128(sb, 16, 1024);
          const uint64_t fa0 = ptx::sdesc_plain(fa, 128), fb0 = ptx::sdesc_plain(fb, 128);  // (512 bytes on: + 32)
          const int steps = min(4, (P.k - kb * kFp4Depth + 63) / 64);
          ok = ptx::mbar_wait(ptx::smem_addr(&full[stage]), phase, budget, abort);
          if (!ok) raise_timeout(P, abort);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
#pragma unroll
            for (int g = 0; g < kG; ++g) {
              ptx::tmem_copy_scales<true>(tmem + kScaleCol + 4 * g, fa0 + 32 * g);
#pragma unroll
              for (int j = 0; j < 2; ++j)
                ptx::tmem_copy_scales<true>(tmem + kScaleCol + 16 + 8 * g + 4 * j, fb0 + 32 * (j * kG + g));
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (k >= steps) break;
              const int g = BLOCK == 32 ? k >> 1 : k;
              const uint32_t idesc = ptx::idesc_fp4(256, 256, BLOCK, BLOCK == 32 ? 2 * (k & 1) : 0);
              ptx::mma_fp4<BLOCK, true>(d, a0 + 2 * k, b0 + 2 * k, idesc, tmem + kScaleCol + 4 * g,
                                        tmem + kScaleCol + 16 + 8 * g, (kb | k) != 0 ? 1u : 0u);
            }
            ptx::mma_commit_pair_mc(ptx::smem_addr(&empty[stage]), 0x3);
          }
          __syncwarp();
          if (++stage == kPairStages) stage = 0, phase ^= 1;
        }
        if (!ok) break;
        if (ptx::elect_one()) ptx::mma_commit_pair_mc(ptx::smem_addr(&tfull[acc]), 0x3);
        __syncwarp();
      }
      if (ptx::elect_one()) ptx::mma_commit_pair(ptx::smem_addr(drain));
      __syncwarp();
      ptx::mbar_wait(ptx::smem_addr(drain), 0, budget, never);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    // Two warps per TMEM lane quarter, a half of the columns each, 64 columns at
    // a time: first those that the next tile's accumulator overlaps (the last
    // 48 of the first accumulator, the first 48 of the second).
    const int q = warp & 3, half = (warp - 2) >> 2;
    const uint32_t stage = ptx::smem_addr(staging + (warp - 2) * 4096);
    const uint32_t tempty_leader = ptx::map_to_rank(ptx::smem_addr(tempty), 0);
    const Factors f = tensor_factors(P);
    int it = 0;
    for (int t = pair; t < total; t += npairs, ++it) {
      const int I = t % P.tiles_m, J = t / P.tiles_m;
      const int acc = it & 1;
      const bool ok = ptx::mbar_wait(ptx::smem_addr(&tfull[acc]), (it >> 1) & 1, budget, abort);
      if (!ok) raise_timeout(P, abort);
      if (__any_sync(0xFFFFFFFFu, !ok || *abort)) break;
      ptx::tc_fence_after();
      const uint32_t tb = tmem + (static_cast<uint32_t>(q * 32) << 16) + acc * kAccStep + half * 128;
      const int row0 = I * 256 + static_cast<int>(rank) * 128 + q * 32;
#pragma unroll 1
      for (int p = 0; p < 2; ++p) {
        const int c = ((acc == 0) ^ p) ? 64 : 0;
        uint32_t lo[32], hi[32];
        __syncwarp();
        ptx::tmem_ld32(tb + c, lo);
        ptx::tmem_ld32(tb + c + 32, hi);
        ptx::tmem_ld_wait(lo);
        ptx::tmem_ld_wait(hi);
        if (p == 0) {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive_cluster_relaxed(tempty_leader);
        }
        const int col0 = J * 256 + half * 128 + c;
        if (row0 < P.m && col0 < P.n) store_rows(P, stage, lane, row0, col0, lo, hi, f);
      }
    }
  }

  ptx::tc_fence_before();
  if (*abort) {
    // give copies this CTA issued before giving up time to land
    const long long t0 = clock64();
    while (clock64() - t0 < 200000) {
    }
  }
  __syncwarp();
  ptx::cluster_sync();
  if (warp == 1) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, 512);
  }
}

// ------------------------------------------------------------------- tiles
constexpr int kTileThreads = 192;
constexpr int kTileScales = 4 * 512;  // of either operand, room for blocks of 16

template <int BN>
struct TileShape {
  static constexpr int stages = BN == 128 ? 3 : 4;
  static constexpr int stage = 128 * kDepthBytes + BN * kDepthBytes + 2 * kTileScales;
  static constexpr int smem = stages * stage + 1024 + 256;
  static_assert(stages * stage >= BN * (128 + 4 * 8) * 4 && stages * stage >= 4 * 4096, "the ring is reused");
  static_assert(stage % 1024 == 0, "swizzled tiles begin on 1 KB");
};

template <int BLOCK, int BN>
__global__ void __launch_bounds__(kTileThreads) fp4_tile_kernel(const __grid_constant__ MmParams P) {
  using Shape = TileShape<BN>;
  constexpr int kSt = Shape::stages, kG = kGroups<BLOCK>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kSt * Shape::stage);
  uint64_t* empty = full + kSt;
  uint64_t* tfull = empty + kSt;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tfull + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* never = reinterpret_cast<volatile int*>(tmem_slot + 2);

  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
  const int rank = static_cast<int>(ptx::cluster_ctarank());
  const int tile = static_cast<int>(ptx::cluster_id_x());
  const int splits = static_cast<int>(gridDim.x / ptx::nclusters_x());
  const int I = tile % P.tiles_m, J = tile / P.tiles_m;
  const int kblocks = (P.k + kFp4Depth - 1) / kFp4Depth, per = (kblocks + splits - 1) / splits;
  const int kb0 = rank * per, kb1 = min(kblocks, kb0 + per);
  const int n0 = J * BN;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kSt; ++s) {
      ptx::mbar_init(ptx::smem_addr(&full[s]), 1);
      ptx::mbar_init(ptx::smem_addr(&empty[s]), 1);
    }
    ptx::mbar_init(ptx::smem_addr(tfull), 1);
    *abort = 0;
    *never = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_addr(tmem_slot), 256);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (threadIdx.x == 0) {
    ptx::prefetch_tmap(&P.codes_a);
    ptx::prefetch_tmap(&P.codes_b);
    ptx::prefetch_tmap(&P.scales_a);
    ptx::prefetch_tmap(&P.scales_b);
  }
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  if (blockIdx.x == 0 && threadIdx.x == 0) *P.status = 0;
  const uint32_t tmem = *tmem_slot;
  const uint32_t tsa = tmem + 128, tsb = tmem + 160;  // scales
  const long long budget = P.wait_budget;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!ptx::mbar_wait(ptx::smem_addr(&empty[stage]), phase ^ 1, budget, abort)) {
          raise_timeout(P, abort);
          break;
        }
        const uint32_t bar = ptx::smem_addr(&full[stage]);
        const uint32_t sa = ptx::smem_addr(smem + stage * Shape::stage), sb = sa + 128 * kDepthBytes;
        const uint32_t fa = sb + BN * kDepthBytes, fb = fa + kTileScales;
        ptx::mbar_arrive_expect_tx(bar, (128 + BN) * kDepthBytes + 2 * kG * 512);
        ptx::tma_load_2d(sa, &P.codes_a, bar, kb * kDepthBytes, I * 128);
        ptx::tma_load_2d(sb, &P.codes_b, bar, kb * kDepthBytes, n0);
        ptx::tma_load_2d(fa, &P.scales_a, bar, 0, I * P.ktiles + kb * kG);
        ptx::tma_load_2d(fb, &P.scales_b, bar, 0, (n0 >> 7) * P.ktiles + kb * kG);
        if (++stage == kSt) stage = 0, phase ^= 1;
      }
    }
  } else if (warp == 1) {
    if (!P.inject_stall && kb0 < kb1) {  // (uniform, as in the pair kernel)
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      const int word = (n0 & 127) >> 5;  // 32-row group of the scale tile that the narrow side begins at
      for (int kb = kb0; kb < kb1; ++kb) {
        const uint32_t sa = ptx::smem_addr(smem + stage * Shape::stage), sb = sa + 128 * kDepthBytes;
        const uint32_t fa = sb + BN * kDepthBytes, fb = fa + kTileScales;
        const uint64_t a0 = ptx::sdesc_sw128(sa, 16, 1024), b0 = ptx::sdesc_sw128(sb, 16, 1024);
        const uint64_t fa0 = ptx::sdesc_plain(fa, 128), fb0 = ptx::sdesc_plain(fb, 128);
        const int steps = min(4, (P.k - kb * kFp4Depth + 63) / 64);
        ok = ptx::mbar_wait(ptx::smem_addr(&full[stage]), phase, budget, abort);
        if (!ok) raise_timeout(P, abort);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
#pragma unroll
          for (int g = 0; g < kG; ++g) {
            ptx::tmem_copy_scales<false>(tsa + 4 * g, fa0 + 32 * g);
            ptx::tmem_copy_scales<false>(tsb + 4 * g, fb0 + 32 * g);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k >= steps) break;
            const int g = BLOCK == 32 ? k >> 1 : k;
            const uint32_t idesc = ptx::idesc_fp4(128, BN, BLOCK, BLOCK == 32 ? 2 * (k & 1) : 0);
            ptx::mma_fp4<BLOCK, false>(tmem, a0 + 2 * k, b0 + 2 * k, idesc, tsa + 4 * g, tsb + 4 * g + word,
                                       kb > kb0 || k > 0 ? 1u : 0u);
          }
          ptx::mma_commit(ptx::smem_addr(&empty[stage]));
        }
        __syncwarp();
        if (++stage == kSt) stage = 0, phase ^= 1;
      }
      // (also after a timeout: what was issued completes before the CTA goes on)
      if (ptx::elect_one()) ptx::mma_commit(ptx::smem_addr(tfull));
      __syncwarp();
      if (!ok) ptx::mbar_wait(ptx::smem_addr(tfull), 0, budget, never);
    }
  }
  const int q = warp & 3;
  bool ok = warp < 2;
  if (warp >= 2) {
    ok = kb0 >= kb1 || ptx::mbar_wait(ptx::smem_addr(tfull), 0, budget, abort);
    if (!ok) raise_timeout(P, abort);
    ok = __all_sync(0xFFFFFFFFu, ok && !*abort);
    ptx::tc_fence_after();
  }
  const Factors f = tensor_factors(P);
  const int slice = 128 / splits;  // rows of the tile that a CTA of the cluster adds up
  // partial sums: [CTA they are of][column][row of the slice], 4 floats of padding a column: lanes
  // next to one another along either side read their 16 bytes from different banks
  const uint32_t partial = ptx::smem_addr(smem);
  if (splits > 1) {
    __syncwarp();
    ptx::cluster_sync();  // no CTA of the cluster still reads its operands
  }
  if (warp >= 2 && ok) {
    const uint32_t tb = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const int row = q * 32 + lane;
    if (splits > 1) {
      uint32_t to = ptx::map_to_rank(partial + (rank * BN * (slice + 4) + (row & (slice - 1))) * 4, row / slice);
#pragma unroll 1
      for (int c = 0; c < BN; c += 32) {
        uint32_t r[32];
        __syncwarp();
        ptx::tmem_ld32(tb + c, r);
        ptx::tmem_ld_wait(r);
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          ptx::st_cluster_b32(to, kb0 < kb1 ? r[k] : 0u);
          to += (slice + 4) * 4;
        }
      }
    } else if (P.swapped) {
      // a lane is a column of out, an accumulator column a row of it
      const int col = I * 128 + row, size = P.f32 ? 4 : 2;
      char* at = static_cast<char*>(P.out) + (n0 * P.stride + col) * size;
      const long long step = P.stride * size;
#pragma unroll 1
      for (int c = 0; c < BN; c += 32) {
        const int have = P.n - n0 - c;  // rows of out from here on
        if (have <= 0) break;
        uint32_t r[32];
        __syncwarp();
        ptx::tmem_ld32(tb + c, r);
        ptx::tmem_ld_wait(r);
        scale32(P, f, r);
        if (col < P.m) {
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            if (k < have) {
              if (P.f32)
                *reinterpret_cast<uint32_t*>(at) = r[k];
              else
                *reinterpret_cast<__nv_bfloat16*>(at) = __float2bfloat16_rn(__uint_as_float(r[k]));
            }
            at += step;
          }
        }
      }
    } else {
      const uint32_t stage = ptx::smem_addr(smem + q * 4096);
      const int row0 = I * 128 + q * 32;
#pragma unroll 1
      for (int c = 0; c < BN; c += 64) {
        uint32_t lo[32], hi[32];
        __syncwarp();
        ptx::tmem_ld32(tb + c, lo);
        if (BN > 32) ptx::tmem_ld32(tb + c + 32, hi);
        ptx::tmem_ld_wait(lo);
        if (BN > 32) {
          ptx::tmem_ld_wait(hi);
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) hi[k] = 0u;
        }
        if (row0 < P.m && n0 + c < P.n) store_rows(P, stage, lane, row0, n0 + c, lo, hi, f);
      }
    }
  }
  ptx::tc_fence_before();
  if (*abort) {
    const long long t0 = clock64();
    while (clock64() - t0 < 200000) {
    }
  }
  if (splits > 1) {
    __syncwarp();
    ptx::cluster_sync();  // every CTA's partial sums are there
    // this CTA's rows of the tile, 4 of a column a thread, lanes along out's rows
    // (slice and BN are powers of two)
    const int quads = slice / 4, bits = P.swapped ? 31 - __clz(quads) : 31 - __clz(BN), m0 = I * 128 + rank * slice;
#pragma unroll 2
    for (int i = static_cast<int>(threadIdx.x); i < quads * BN; i += kTileThreads) {
      const int in = i & ((1 << bits) - 1), over = i >> bits;
      const int r = 4 * (P.swapped ? in : over), c = P.swapped ? over : in;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
      for (int s = 0; s < splits; ++s) {
        float4 p;
        ptx::lds128f(partial + ((s * BN + c) * (slice + 4) + r) * 4, p);
        v.x += p.x, v.y += p.y, v.z += p.z, v.w += p.w;
      }
      const float x[4] = {v.x * f.a * f.b, v.y * f.a * f.b, v.z * f.a * f.b, v.w * f.a * f.b};
      const int gm = m0 + r, gn = n0 + c;
      if (gm >= P.m || gn >= P.n) continue;
      const long long o = P.swapped ? gn * P.stride + gm : gm * P.stride + gn;
      if (P.swapped && P.vec && gm + 4 <= P.m) {
        if (P.f32)
          *reinterpret_cast<float4*>(static_cast<float*>(P.out) + o) = make_float4(x[0], x[1], x[2], x[3]);
        else
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(P.out) + o) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
        continue;
      }
      const long long next = P.swapped ? 1 : P.stride;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (gm + k >= P.m) break;
        if (P.f32)
          static_cast<float*>(P.out)[o + k * next] = x[k];
        else
          static_cast<__nv_bfloat16*>(P.out)[o + k * next] = __float2bfloat16_rn(x[k]);
      }
    }
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 256);
  }
}

// ---------------------------------------------------------------- launches
struct Kernel {
  const void* fn;
  int smem, threads;
};

template <int BLOCK>
Kernel kernel_of(int bn) {
  switch (bn) {
    case 32: return {reinterpret_cast<const void*>(&fp4_tile_kernel<BLOCK, 32>), TileShape<32>::smem, kTileThreads};
    case 64: return {reinterpret_cast<const void*>(&fp4_tile_kernel<BLOCK, 64>), TileShape<64>::smem, kTileThreads};
    case 128: return {reinterpret_cast<const void*>(&fp4_tile_kernel<BLOCK, 128>), TileShape<128>::smem, kTileThreads};
    default: return {reinterpret_cast<const void*>(&fp4_pair_kernel<BLOCK>), kPairSmem, kPairThreads};
  }
}

void config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute (&attr)[2], const Kernel& k, int cluster, cudaStream_t stream) {
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg = {};
  cfg.blockDim = dim3(static_cast<unsigned>(k.threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(k.smem);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
}

constexpr int kMaxDevices = 64;
std::mutex g_mu;
int g_pairs[kMaxDevices][8] = {};  // by device and kernel: 0 unknown, else what can be resident (tile kernels: 1)

// Raises the kernel's shared-memory limit on the current device at its first
// use there; *pairs: CTA pairs of the pair kernel that can be resident.
cudaError_t prepare(const Kernel& k, int slot, bool pair, int sms, int* pairs) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(g_mu);
  int& n = g_pairs[dev][slot];
  if (n <= 0) {
    e = cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
    if (e != cudaSuccess) return e;
    int q = 1;
    if (pair) {
      cudaLaunchConfig_t cfg;
      cudaLaunchAttribute attr[2];
      config(cfg, attr, k, 2, nullptr);
      cfg.gridDim = dim3(static_cast<unsigned>(sms));
      e = cudaOccupancyMaxActiveClusters(&q, k.fn, &cfg);
      if (e != cudaSuccess) return e;
    }
    n = q > 0 ? q : 1;
  }
  *pairs = std::min(n, sms / 2);
  return cudaSuccess;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// CTAs that share a tile's K blocks.  A block takes a CTA 0.25 us; sending and
// adding partial sums costs as much as `cost` blocks, more between two CTAs, who add half a
// tile each, than among more.  us with 1, 2, 4 and 8 CTAs: 13 tiles of 32 columns, 7 blocks
// 5.1, 6.0, 4.4, 4.5, 64 blocks 19.8, 13.4, 9.0, 7.4; 32 tiles of 128 columns, 7 blocks 7.1, 10.5, 7.4, 7.5, 64
// blocks 21.3, 18.2, 13.2, 15.8; 76 tiles of 128, 25 blocks 11.6, 13.6, 20.1.  They have an SM each, but two
// narrow ones may share one (64 tiles of 32 columns, 64 blocks 20.1, 14.1, 11.0, 16.6; 50 of them, 7 blocks 5.5, 6.0, 6.0).
int tile_splits(int64_t tiles, int64_t kblocks, int bn, int sms) {
  for (int s = 8; s > 1; s /= 2) {
    const bool shared = s == 4 && bn == 32 && kblocks >= 16;
    const int64_t cost = s == 2 ? 2 + bn / 8 : 2 + bn / 32;
    if (s <= kblocks && tiles * s <= (shared ? 2 : 1) * sms && kblocks - kblocks / s >= cost) return s;
  }
  return 1;
}

}  // namespace

MUON_CHECK_READER(check_failures_fp4_mm)

}  // namespace muon

using namespace muon;

extern "C" muon_status_t fp4_mm(const fp4_matrix* a, const fp4_matrix* b, void* out, int dtype, int64_t out_stride,
                                void* workspace, size_t workspace_bytes, void* stream) {
  for (const fp4_matrix* m : {a, b}) {
    const muon_status_t st = fp4_check(m);
    if (st != MUON_OK) return st;
  }
  if (a->block != b->block || a->cols != b->cols || (dtype != MUON_BF16 && dtype != MUON_F32) || out_stride < b->rows)
    return MUON_ERR_INVALID_ARG;
  if (out_stride > (1LL << 32)) return MUON_ERR_TOO_LARGE;
  if (a->rows == 0 || b->rows == 0) return MUON_OK;
  if (!out || !workspace) return MUON_ERR_INVALID_ARG;
  const int size = dtype == MUON_F32 ? 4 : 2;
  if (!aligned_to(out, size) || !aligned_to(workspace, 256)) return MUON_ERR_MISALIGNED;
  if (workspace_bytes < 256) return MUON_ERR_WORKSPACE_TOO_SMALL;
  const int64_t m = a->rows, n = b->rows, k = a->cols;
  try {
    std::vector<Span> v = {span_of(out, (static_cast<uint64_t>(m - 1) * out_stride + n) * size, true),
                           span_of(workspace, 256, true)};
    fp4_spans(v, *a, false);
    fp4_spans(v, *b, false);
    if (spans_conflict(v)) return MUON_ERR_ALIASING;
  } catch (const std::bad_alloc&) {
    return MUON_ERR_HOST_MEMORY;
  }
  int sms = 0;
  muon_status_t st = device_sms(sms);
  if (st != MUON_OK) return st;
  cudaStream_t str = static_cast<cudaStream_t>(stream);
  if (k == 0) {  // empty sums
    if (cudaMemsetAsync(workspace, 0, 256, str) != cudaSuccess ||
        cudaMemset2DAsync(out, out_stride * size, 0, n * size, m, str) != cudaSuccess)
      return MUON_ERR_CUDA;
    return MUON_OK;
  }
  MmParams P;
  std::memset(&P, 0, sizeof(P));
  // The tile kernel's 128 rows are the larger matrix's.  Pairs take over where its
  // tiles are more than the SMs (m x n x k, bfloat16 out, us, tiles and pairs: 1024 x 2048 x 6400
  // 12.2 and 13.1; 1600 x 1600 x 1600 8.0 and 7.7, x 16384 28.9 and 25.3; 64 x 50304 x 1600
  // 15.7 and 13.6), but not for up to 32 rows, whose 256 would be mostly empty (8 x 50304 x 1600 11.6 and 18.2).
  const int64_t pair_tiles = ceil_div(m, 256) * ceil_div(n, 256);
  const int64_t narrow = std::min(m, n);
  const int width = narrow <= 32 ? 32 : narrow <= 64 ? 64 : 128;
  const bool pair = width > 32 && ceil_div(std::max(m, n), 128) * ceil_div(narrow, width) > sms;
  const bool swapped = !pair && n > m;
  const fp4_matrix& big = swapped ? *b : *a;
  const fp4_matrix& small = swapped ? *a : *b;
  const int bn = pair ? 0 : width;
  const int rows_b = pair ? 128 : bn;
  P.tiles_m = static_cast<int>(ceil_div(big.rows, pair ? 256 : 128));
  P.tiles_n = static_cast<int>(ceil_div(small.rows, pair ? 256 : bn));
  if (static_cast<int64_t>(P.tiles_m) * P.tiles_n > (1 << 27)) return MUON_ERR_TOO_LARGE;
  P.ktiles = static_cast<int>(fp4_ktiles(k, a->block));
  const int groups = kFp4Depth / (4 * a->block);
  auto maps = [&](const fp4_matrix& x, CUtensorMap* codes, CUtensorMap* scales, int box_rows) {
    const int64_t tiles = fp4_row_tiles(x.rows) * P.ktiles;
    return encode_map_2d(codes, x.codes, 1, fp4_pitch(k), x.rows, fp4_pitch(k), kDepthBytes, box_rows, true) &&
           encode_map_2d(scales, x.scales, 4, 128, tiles, 512, 128, groups, false);
  };
  if (!maps(big, &P.codes_a, &P.scales_a, 128) || !maps(small, &P.codes_b, &P.scales_b, rows_b)) return MUON_ERR_CUDA;
  P.scale_a = big.scale;
  P.scale_b = small.scale;
  P.out = out;
  P.stride = out_stride;
  P.m = static_cast<int>(big.rows);
  P.n = static_cast<int>(small.rows);
  P.k = static_cast<int>(k);
  P.f32 = dtype == MUON_F32;
  P.vec = aligned_to(out, 16) && out_stride * size % 16 == 0;
  P.swapped = swapped;
  P.status = static_cast<int*>(workspace);
  P.wait_budget = wait_budget();
  P.inject_stall = inject_stall();
  const Kernel kern = a->block == 32 ? kernel_of<32>(bn) : kernel_of<16>(bn);
  const int slot = (a->block == 32 ? 4 : 0) + (bn == 0 ? 0 : bn == 32 ? 1 : bn == 64 ? 2 : 3);
  int pairs = 0;
  if (prepare(kern, slot, pair, sms, &pairs) != cudaSuccess) return MUON_ERR_CUDA;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  if (pair) {
    config(cfg, attr, kern, 2, str);
    cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min<int64_t>(pairs, pair_tiles)));
  } else {
    const int64_t tiles = static_cast<int64_t>(P.tiles_m) * P.tiles_n, kblocks = ceil_div(k, kFp4Depth);
    const int splits = tile_splits(tiles, kblocks, bn, sms);
    config(cfg, attr, kern, splits, str);
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * splits));
  }
  cfg.numAttrs = 2;
  void* args[] = {&P};
  if (cudaLaunchKernelExC(&cfg, kern.fn, args) != cudaSuccess) return MUON_ERR_CUDA;
  return MUON_OK;
}
