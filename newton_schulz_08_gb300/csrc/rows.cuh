// Rows of bfloat16 or float32 entries at any alignment of the element, moved
// between global and shared memory in 16-byte units by the lanes that use them.
//
// A lane's unit k of a row (8 or 4 entries) is copied ahead with cp.async to
// the same place of a slot in shared memory, so that a row is in flight while
// the one before it is worked on and takes no registers.  Where a row does not
// begin on 16 bytes, the slot holds the aligned units that contain it, one
// more than the row has, and a lane takes its entries from two neighbouring
// ones; results go back the same way.  Only units that hold an entry of the
// row are read.  A slot is used by one warp.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace muon {
namespace rows {

template <bool BF16>
struct Unit {
  static constexpr int size = BF16 ? 2 : 4;
  static constexpr int n = 16 / size;  // entries
};

__device__ __forceinline__ uint32_t shared_address(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ uint4 shared_load(uint32_t at) {
  uint4 q;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(at) : "memory");
  return q;
}

__device__ __forceinline__ void shared_store(uint32_t at, const uint4& q) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(q.x), "r"(q.y), "r"(q.z), "r"(q.w) : "memory");
}

// 16 bytes: the first `bytes` (0 .. 16) from memory, zeros behind them.
__device__ __forceinline__ void copy_ahead(uint32_t at, const void* from, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(from), "r"(bytes) : "memory");
}

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copies_wait(int left) {  // all but the last `left` (0 or 1) groups
  if (left)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// 16 bytes from byte `shift` (0 .. 15, even) of a and b together.
__device__ __forceinline__ uint4 funnel(const uint4& a, const uint4& b, uint32_t shift) {
  uint32_t w0 = a.x, w1 = a.y, w2 = a.z, w3 = a.w, w4 = b.x, w5 = b.y, w6 = b.z, w7 = b.w;
  if (shift & 8) w0 = w2, w1 = w3, w2 = w4, w3 = w5, w4 = w6, w5 = w7;
  if (shift & 4) w0 = w1, w1 = w2, w2 = w3, w3 = w4, w4 = w5;
  const uint32_t sel = shift & 2 ? 0x5432 : 0x3210;
  return make_uint4(__byte_perm(w0, w1, sel), __byte_perm(w1, w2, sel), __byte_perm(w2, w3, sel), __byte_perm(w3, w4, sel));
}

__device__ __forceinline__ uint32_t shift_of(const void* p) { return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15); }

__device__ __forceinline__ void copy_ahead(uint32_t at, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
}

// Starts the copies of units k = sub, sub + L, ... (n of them) of a piece of a
// row that begins at `p` and has `left` entries, more than (n - 1) L units of
// them: only the last one may reach past them, and has zeros there.  The last
// lane also copies the unit behind the piece's last one.  `none`: zeros throughout.
template <bool BF16, bool ALIGNED, int L, int V>
__device__ __forceinline__ void fetch(uint32_t slot, const char* p, int left, int sub, int n, bool none) {
  using U = Unit<BF16>;
  const uint32_t shift = ALIGNED ? 0u : shift_of(p);
  const char* from = p - shift + 16 * sub;
  const uint32_t to = slot + 16 * sub;
  // bytes of the last unit, and of the one behind the piece
  const int have = min(left, n * L * U::n + U::n) * U::size + static_cast<int>(shift) - 16 * (n - 1) * L;
  const int last = none ? 0 : min(max(have - 16 * sub, 0), 16);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (v + 1 < n) {
      if (none)
        copy_ahead(to + 16 * L * v, from, 0);
      else
        copy_ahead(to + 16 * L * v, from + 16 * L * v);
    } else if (v + 1 == n) {
      // (nothing is read where there are 0 bytes, so the address does not matter then)
      copy_ahead(to + 16 * L * v, last ? from + 16 * L * v : p - shift, last);
    }
  }
  if constexpr (!ALIGNED) {
    if (sub == L - 1 && n > 0) {
      const int behind = none ? 0 : min(max(have - 16 * L, 0), 16);
      copy_ahead(slot + 16 * n * L, behind ? p - shift + 16 * n * L : p - shift, behind);
    }
  }
}

// Arithmetic on two float32 numbers at a time.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair(float a, float b) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(a), "f"(b));
  return p;
}
__device__ __forceinline__ Pair pair(float a) { return pair(a, a); }
__device__ __forceinline__ void split(Pair p, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p)); }
__device__ __forceinline__ float total(Pair p) {
  float a, b;
  split(p, a, b);
  return a + b;
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  Pair p;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(a), "l"(b));
  return p;
}
__device__ __forceinline__ Pair mul(Pair a, Pair b) {
  Pair p;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(a), "l"(b));
  return p;
}
__device__ __forceinline__ Pair fma(Pair a, Pair b, Pair c) {
  Pair p;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p) : "l"(a), "l"(b), "l"(c));
  return p;
}

// A unit's entries as numbers, and back (rounded to nearest).
template <bool BF16>
__device__ __forceinline__ void numbers(const uint4& q, Pair (&x)[Unit<BF16>::n / 2]) {
  if constexpr (BF16) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  } else {
    x[0] = pair(__uint_as_float(q.x), __uint_as_float(q.y));
    x[1] = pair(__uint_as_float(q.z), __uint_as_float(q.w));
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack(const Pair (&x)[Unit<BF16>::n / 2]) {
  uint32_t w[4];
  if constexpr (BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      split(x[i], a, b);
      const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float a, b;
      split(x[i], a, b);
      w[2 * i] = __float_as_uint(a);
      w[2 * i + 1] = __float_as_uint(b);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Unit k of a piece that was fetched to `slot` (zeros past the row's end).
template <bool ALIGNED>
__device__ __forceinline__ uint4 unit(uint32_t slot, uint32_t shift, int k) {
  uint4 q = shared_load(slot + 16 * k);
  if constexpr (!ALIGNED) {
    if (shift) q = funnel(q, shared_load(slot + 16 * k + 16), shift);
  }
  return q;
}

// Entries [from, to) of a unit.
template <bool BF16>
__device__ __forceinline__ void store_some(char* p, const uint4& q, int from, int to) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int k = 0; k < Unit<BF16>::n; ++k) {
    if (k < from || k >= to) continue;
    if constexpr (BF16)
      reinterpret_cast<uint16_t*>(p)[k] = static_cast<uint16_t>(w[k >> 1] >> (16 * (k & 1)));
    else
      reinterpret_cast<uint32_t*>(p)[k] = w[k];
  }
}

// Unit k of a piece that begins on 16 bytes; `whole`: it lies within the piece.
template <bool BF16>
__device__ __forceinline__ void store_unit(char* p, int k, int left, const uint4& q, bool whole) {
  using U = Unit<BF16>;
  const int room = left - k * U::n;
  if (whole || room >= U::n)
    *reinterpret_cast<uint4*>(p + 16 * k) = q;
  else if (room > 0)
    store_some<BF16>(p + 16 * k, q, 0, room);
}

// The piece at `p` from the units that the warp has put into the slot.
template <bool BF16, int L, int V>
__device__ __forceinline__ void store_shifted(uint32_t slot, char* p, int left, int sub, int n) {
  using U = Unit<BF16>;
  const uint32_t shift = shift_of(p);
  const int before = static_cast<int>(shift) / U::size;  // entries of the first aligned unit in front of the piece
#pragma unroll
  for (int v = 0; v <= V; ++v) {
    if (v > n || (v == n && (sub != 0 || shift == 0))) break;
    const int k = v * L + sub, room = left + before - k * U::n;
    if (room <= 0) break;
    uint4 q = v < n ? shared_load(slot + 16 * k) : make_uint4(0, 0, 0, 0);
    if (shift) q = funnel(k ? shared_load(slot + 16 * k - 16) : q, q, 16 - shift);
    // (the last aligned unit holds only what is left of the piece)
    const int to = min(room, v == n ? before : U::n), first = k == 0 ? before : 0;
    char* at = p - shift + 16 * k;
    if (first == 0 && to == U::n)
      *reinterpret_cast<uint4*>(at) = q;
    else
      store_some<BF16>(at, q, first, to);
  }
}

}  // namespace rows
}  // namespace muon
