// Device helpers of the row operators (RMS norm, microscaled 4-bit codes,
// dequantisers): 16-byte pieces of rows at any alignment, bf16 pairs, and
// reductions inside a 16-lane row of a wave.
//
// A lane owns pieces of eight consecutive columns, and 4, 8 or 16 neighbouring
// lanes own a group of 32, 64 or 128.  Rows of a width that is not a multiple
// of 8 start off 16 bytes: the pieces are then loaded and stored with the same
// 16-byte instructions at 2-byte alignment (gfx950 takes them; the vector
// types below say so to the compiler).  A row's last, partial piece is loaded
// from where it ends and shifted, so that no lane leaves the others' way; it is
// stored element by element.
#ifndef SILUQUANT_ROWS_H
#define SILUQUANT_ROWS_H

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace rows {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Two fp32 values -> two bf16 (nearest, ties to even), a in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

// Eight bf16 values, two to a word, the first in the low half of w[0].
struct Piece {
  uint32_t w[4];
};
__device__ __forceinline__ Piece zero_piece() { return {{0, 0, 0, 0}}; }

// What a piece may be, by the row's width: whole (kFull); whole or none of the
// row's (kWhole, widths of a multiple of 8); partial (kRagged), in rows of at
// least eight elements, or shorter ones (kTiny).  n: how many of its eight
// elements the row has, 0 and below for none; looked at as far as the kind asks.
enum Kind { kFull = 0, kWhole = 1, kRagged = 2, kTiny = 3 };

__device__ __forceinline__ Piece piece_of(const u32x4& v) { return {{v.x, v.y, v.z, v.w}}; }

// The elements d and on of a piece, in its first places, zeros behind them.
__device__ __forceinline__ Piece shifted(Piece v, int d) {
  if (d & 4) v = {{v.w[2], v.w[3], 0, 0}};
  if (d & 2) v = {{v.w[1], v.w[2], v.w[3], 0}};
  if (d & 1)
    v = {{__builtin_amdgcn_alignbit(v.w[1], v.w[0], 16), __builtin_amdgcn_alignbit(v.w[2], v.w[1], 16),
          __builtin_amdgcn_alignbit(v.w[3], v.w[2], 16), v.w[3] >> 16}};
  if (d >= 8) v = zero_piece();
  return v;
}

// kNt: streamed, for what nobody reads soon.
template <Kind kKind, bool kNt>
__device__ __forceinline__ Piece load_bf16(const uint16_t* p, int n) {
  auto at = [](const uint16_t* q) {
    const u32x4_a2* from = reinterpret_cast<const u32x4_a2*>(q);
    u32x4 v;
    if (kNt)
      v = __builtin_nontemporal_load(from);
    else
      v = *from;
    return piece_of(v);
  };
  if (kKind == kFull) return at(p);
  if (kKind == kWhole) return n > 0 ? at(p) : zero_piece();
  if (kKind == kRagged) {
    const int d = n < 8 ? 8 - n : 0;  // past the row's end: its last eight elements, all shifted out
    return shifted(at(p - d), d);
  }
  Piece r = zero_piece();
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) r.w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
  return r;
}

template <Kind kKind>
__device__ __forceinline__ void load_f32(float (&v)[8], const float* p, int n) {
  if (kKind == kTiny) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.0f;
    return;
  }
  const int d = kKind == kRagged && n < 8 ? 8 - n : 0;
  u32x4 a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
  if (kKind != kWhole || n > 0) {
    a = *reinterpret_cast<const u32x4_a4*>(p - d);
    b = *reinterpret_cast<const u32x4_a4*>(p - d + 4);
  }
  if (kKind == kRagged) {
    const u32x4 zero = {0, 0, 0, 0};
    if (d & 4) a = b, b = zero;
    if (d & 2) a = (u32x4){a.z, a.w, b.x, b.y}, b = (u32x4){b.z, b.w, 0, 0};
    if (d & 1) a = (u32x4){a.y, a.z, a.w, b.x}, b = (u32x4){b.y, b.z, b.w, 0};
    if (d >= 8) a = zero, b = zero;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(a[i]), v[4 + i] = __uint_as_float(b[i]);
}

template <Kind kKind, bool kNt>
__device__ __forceinline__ void store_bf16(uint16_t* p, const Piece& v, int n) {
  if (kKind == kFull || (kKind == kWhole ? n > 0 : n >= 8)) {
    const u32x4 x = {v.w[0], v.w[1], v.w[2], v.w[3]};
    u32x4_a2* q = reinterpret_cast<u32x4_a2*>(p);
    if (kNt)
      __builtin_nontemporal_store(x, q);
    else
      *q = x;
  } else if (kKind >= kRagged) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) p[i] = (uint16_t)(v.w[i >> 1] >> (16 * (i & 1)));
  }
}

// Eight one-byte codes.
template <Kind kKind>
__device__ __forceinline__ void store_codes(uint8_t* p, uint32_t lo, uint32_t hi, int n) {
  if (kKind == kFull || (kKind == kWhole ? n > 0 : n >= 8)) {
    __builtin_nontemporal_store((u32x2){lo, hi}, reinterpret_cast<u32x2_a1*>(p));
  } else if (kKind >= kRagged) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) p[i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
  }
}

__device__ __forceinline__ void unpack(float (&v)[8], const Piece& p) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(p.w[i]), v[2 * i + 1] = bf16_hi(p.w[i]);
}

// ---- reductions ----
// Lane exchanges inside a 16-lane row (DPP: no LDS): over 4 lanes the two quad
// permutations, over 8 the mirror of the half row, over 16 the mirror of the row.
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xf, 0xf, false);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;

__device__ __forceinline__ uint32_t max_u16(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

// The largest magnitude of a group of 8 * lanes (32, 64 or 128) values as bf16
// bits, in every lane of the group.  Magnitudes of bf16 numbers order as their
// bits do; a NaN is larger than everything, so that it shows in the scale.
template <bool kWide>
__device__ __forceinline__ uint32_t group_amax_bits(const Piece& p, int lanes) {
  uint32_t m = max_u16(max_u16(p.w[0] & 0x7fff7fffu, p.w[1] & 0x7fff7fffu),
                       max_u16(p.w[2] & 0x7fff7fffu, p.w[3] & 0x7fff7fffu));
  m = max_u16(m, dpp<kXor1>(m));
  m = max_u16(m, dpp<kXor2>(m));
  if (kWide) {
    if (lanes > 4) m = max_u16(m, dpp<kHalfMirror>(m));
    if (lanes > 8) m = max_u16(m, dpp<kMirror>(m));
  }
  return max(m & 0xffffu, m >> 16);
}

// Sums over 16 lanes, and over the 64 of a wave, in every lane, always added in
// the same order.
__device__ __forceinline__ float sum16(float v) {
  v += __uint_as_float(dpp<kXor1>(__float_as_uint(v)));
  v += __uint_as_float(dpp<kXor2>(__float_as_uint(v)));
  v += __uint_as_float(dpp<kHalfMirror>(__float_as_uint(v)));
  v += __uint_as_float(dpp<kMirror>(__float_as_uint(v)));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
  v = sum16(v);
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  return v;
}

// ---- host ----
struct Span {
  const void* p;
  int64_t bytes;
};
inline bool overlap(const Span& a, const Span& b) {
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && a.bytes > 0 && b.bytes > 0 && pa < pb + (uintptr_t)b.bytes && pb < pa + (uintptr_t)a.bytes;
}
inline bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

}  // namespace rows

#endif
