// What the norms share: the group quantiser of a row's pieces, sums over the waves
// of a workgroup, and how a row of any width is divided into pieces.
#ifndef SILUQUANT_NORM_ROWS_H
#define SILUQUANT_NORM_ROWS_H

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "rows.h"

namespace rows {

constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to an integer, ties to even

// Eight codes of the bf16 values in p.  int8: p * inv is one fp32 product, and
// adding kMagic leaves its nearest integer in the low byte.  E4M3: the hardware
// conversion (nearest, ties to even).  kSafe serves an inverse that overflowed:
// products clamp to the largest code, zeros stay zeros.
template <bool kE4M3, bool kSafe>
__device__ __forceinline__ u32x2 codes8(const Piece& p, float inv) {
  constexpr float kTop = kE4M3 ? 448.0f : 127.0f;
  float v[8];
  unpack(v, p);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = v[i] * inv;
    v[i] = !kSafe ? t : v[i] == 0.0f ? v[i] : __builtin_amdgcn_fmed3f(t, -kTop, kTop);
  }
  u32x2 out;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float* q = v + 4 * k;
    if (kE4M3) {
      int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
      out[k] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
    } else {
      uint32_t b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(q[i] + kMagic);
      const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u);
      const uint32_t hi = __builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400u);
      out[k] = lo | (hi << 16);
    }
  }
  return out;
}

// Scale of a group from its largest bf16 magnitude, and the scale's inverse.
template <bool kE4M3>
__device__ __forceinline__ float group_scale(uint32_t amax_bits) {
  const float amax = __uint_as_float(amax_bits << 16);
  return amax == 0.0f ? 1.0f : amax / (kE4M3 ? 448.0f : 127.0f);
}

// Codes and scale of one piece's group; every lane of the wave calls it.  Args has q
// [rows, D], s [rows, groups] and lg_lanes, the log2 of the lanes per group.
template <bool kE4M3, Kind kKind, class Args>
__device__ __forceinline__ void quantise(const Args& a, const Piece& y, int64_t row, int col, int n) {
  const uint32_t amax = group_amax_bits<true>(y, 1 << a.lg_lanes);
  const float scale = group_scale<kE4M3>(amax);
  const float inv = 1.0f / scale;
  u32x2 c = codes8<kE4M3, false>(y, inv);
  if (__any(inv == __builtin_huge_valf())) c = codes8<kE4M3, true>(y, inv);
  if (n > 0) {
    store_codes<kKind>(a.q + row * a.D + col, c.x, c.y, n);
    if ((threadIdx.x & ((1 << a.lg_lanes) - 1)) == 0) a.s[row * a.groups + (col >> (3 + a.lg_lanes))] = scale;
  }
}

// The sum over a workgroup's waves (16 at most) of their own sums, in wave order.
__device__ __forceinline__ float group_sum(float v, float (&s)[16], int wave, int waves) {
  const int lane = threadIdx.x & 63;
  v = wave_sum(v);
  if (lane == 0) s[wave] = v;
  __syncthreads();
  v = sum16((lane & 15) < waves ? s[lane & 15] : 0.0f);
  __syncthreads();  // before the next row's sums
  return v;
}

// f(kind, c) for the pieces of a lane.  Only the last can reach past the row:
// there are as many waves as the row fills with all pieces but it (D > 512 of
// one wave, D > 1024 (waves - 1) >= 512 waves of more).  Shifts and short stores
// for both pieces measured slower (16384 x 4100 forward 113 us, so 109; backward
// 151 and 142).  What rows off 16 bytes still cost (16384 x 4104: 85 and 98 us)
// is their unaligned loads and stores.
template <Kind kKind, int kPieces, class F>
__device__ __forceinline__ void each_piece(F&& f) {
  static_assert(kPieces == 1 || kPieces == 2, "one or two");
  if constexpr (kPieces == 2) f(std::integral_constant<Kind, kFull>{}, 0);
  f(std::integral_constant<Kind, kKind>{}, kPieces - 1);
}

// Eight gradients as fp32.
template <bool kF32, Kind kKind>
__device__ __forceinline__ void load_grad(float (&v)[8], const void* p, int64_t at, int n) {
  if constexpr (kF32)
    load_f32<kKind>(v, static_cast<const float*>(p) + at, n);
  else
    unpack(v, load_bf16<kKind, true>(static_cast<const uint16_t*>(p) + at, n));
}

// ---- host ----
// Calls f with the kind of the pieces of a row of D columns, where the lanes'
// pieces cover `covered`, as a type.  Two pieces per lane start at 513 columns.
template <int kPieces, class F>
void with_kind(int64_t D, int64_t covered, F&& f) {
  if (D == covered) return f(std::integral_constant<Kind, kFull>{});
  if (D % 8 == 0) return f(std::integral_constant<Kind, kWhole>{});
  if constexpr (kPieces == 1)
    if (D < 8) return f(std::integral_constant<Kind, kTiny>{});
  f(std::integral_constant<Kind, kRagged>{});
}

}  // namespace rows

#endif
