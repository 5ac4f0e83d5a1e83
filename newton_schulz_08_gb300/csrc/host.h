// Host-side helpers shared by the entry points: the current device, and the
// overlap check of a call's byte ranges.
#pragma once

#include <cuda.h>

#include <algorithm>
#include <cstdint>
#include <vector>

#include "../../include/muon.h"

namespace muon {

// MUON_OK and the SM count when the current device is compute capability
// 10.3, else the error to return (muon_capi.cu).
muon_status_t device_sms(int& sms);

// The knobs of muon_set_debug that other units' kernels follow (muon_capi.cu).
long long wait_budget();
int inject_stall();

// 2-D tensor map of rows x cols elements of 1 or 4 bytes (row pitch in bytes),
// with or without 128-byte swizzle; false on failure (muon_capi.cu).
bool encode_map_2d(CUtensorMap* map, const void* base, int size, uint64_t cols, uint64_t rows, uint64_t pitch,
                   uint32_t box_cols, uint32_t box_rows, bool swizzle);

struct Span {
  uintptr_t lo, hi;  // [lo, hi)
  bool write;
};

inline Span span_of(const void* p, uint64_t bytes, bool write) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return {a, a + static_cast<uintptr_t>(bytes), write};
}

// Whether a written range overlaps another range (read ranges may overlap
// one another).  Sorts `s`: n log n, as a call may bring thousands of ranges.
inline bool spans_conflict(std::vector<Span>& s) {
  std::sort(s.begin(), s.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
  uintptr_t end = 0, end_written = 0;
  for (const Span& r : s) {
    if (r.hi == r.lo) continue;
    if (r.lo < end_written || (r.write && r.lo < end)) return true;
    end = std::max(end, r.hi);
    if (r.write) end_written = std::max(end_written, r.hi);
  }
  return false;
}

inline bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace muon
