// Layout of a matrix in 4-bit codes (include/muon.h, fp4_matrix), shared by
// the quantise passes (fp4.cu) and the product (fp4_mm.cu).
#pragma once

#include <cstdint>

#include "../../include/muon.h"
#include "host.h"

namespace muon {

constexpr int kFp4Tile = 128;   // rows of a scale tile
constexpr int kFp4Depth = 256;  // entries along K that scales are padded to: a K block of the product
constexpr int64_t kFp4MaxDim = 0x7FFFFF00;

// Bytes of a row of codes: two per byte, rows padded to 32 entries (16 bytes).
inline int64_t fp4_pitch(int64_t cols) { return (cols + 31) / 32 * 16; }
// Scale tiles (128 rows x 4 scales, 512 bytes) along K.
inline int64_t fp4_ktiles(int64_t cols, int block) { return (cols + kFp4Depth - 1) / kFp4Depth * (kFp4Depth / (4 * block)); }
inline int64_t fp4_row_tiles(int64_t rows) { return (rows + kFp4Tile - 1) / kFp4Tile; }

// Status of a matrix as an operand: sizes, pointers, alignment.
inline muon_status_t fp4_check(const fp4_matrix* m) {
  if (!m || m->rows < 0 || m->cols < 0 || (m->block != 16 && m->block != 32) || m->reserved != 0)
    return MUON_ERR_INVALID_ARG;
  if (m->rows > kFp4MaxDim || m->cols > kFp4MaxDim) return MUON_ERR_TOO_LARGE;
  if ((m->block == 16) != (m->scale != nullptr)) return MUON_ERR_INVALID_ARG;
  if (m->rows > 0 && m->cols > 0) {
    if (!m->codes || !m->scales) return MUON_ERR_INVALID_ARG;
    if (fp4_row_tiles(m->rows) * fp4_ktiles(m->cols, m->block) > 0x7FFFFFFF) return MUON_ERR_TOO_LARGE;
  }
  if (!aligned_to(m->codes, 16) || !aligned_to(m->scales, 16) || !aligned_to(m->scale, 4)) return MUON_ERR_MISALIGNED;
  return MUON_OK;
}

inline uint64_t fp4_code_bytes(const fp4_matrix& m) { return static_cast<uint64_t>(m.rows) * fp4_pitch(m.cols); }
inline uint64_t fp4_scale_bytes(const fp4_matrix& m) {
  return static_cast<uint64_t>(fp4_row_tiles(m.rows)) * fp4_ktiles(m.cols, m.block) * 512;
}

inline void fp4_spans(std::vector<Span>& v, const fp4_matrix& m, bool write) {
  v.push_back(span_of(m.codes, fp4_code_bytes(m), write));
  v.push_back(span_of(m.scales, fp4_scale_bytes(m), write));
  v.push_back(span_of(m.scale, m.scale ? (write ? FP4_SCALE_FLOATS : 2) * 4 : 0, write));
}

}  // namespace muon
