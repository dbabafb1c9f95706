// RMS norm with the residual's addition and the group quantiser of the library
// behind it, and its backward pass, for gfx950.
//
//   forward   h = bf16(x + residual);  rstd = 1 / sqrt(sum(h^2) / D + eps)
//             y = bf16((h * rstd) * w);  codes and scales of y by group
//   backward  n = h * rstd;  g = dy * w;  c = sum(g * n) / D
//             dx = bf16(rstd * (g - n * c) + d_h);  dw = sum over rows of dy * n
//
// Both read and write every element once and compute some ten operations on
// it: they are bound by memory.  A row stays in registers between its sum and
// its use, so nothing is read twice.  The sums are fp32; h is rounded to bf16
// before the statistics because that is the stream the next layer and the
// backward pass read, and y is rounded to bf16 before quantising as everywhere
// in this library, so that codes made here are those of the bf16 y.
//
// Layout: a lane owns two pieces of 8 columns.  Rows of up to 1024 columns go to
// a wave each, which needs no barrier; longer ones, up to 16384 columns, to a
// workgroup of as many waves as they fill.  More pieces per lane and fewer
// waves, which saves the barrier, measured slower (16384 x 4096: four waves of
// two pieces 80 us, one of eight 89 us): the loads of more waves are in flight
// while others compute.  At 16384 x 4096 the forward pass moves 470 MB in 80 us
// (5.9 TB/s), the backward pass 537 MB in 92 us (5.8 TB/s) and sums dw in 5 more;
// a plain 2 GiB copy reaches 4.8 TB/s here.  With x in fp32 102 us (5.9 TB/s),
// with y in bf16 in place of codes 93 us (5.8 TB/s), with dy in fp32 119 us (5.7
// TB/s, dw's sum included).  Rows past 16384 columns are walked twice: 2048 x
// 32768 takes 117 us forward (4.0 TB/s) and 149 us backward (3.6 TB/s), the same
// number of elements in rows of 16384 92 and 110 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "code_objects.h"
#include "rows.h"
#include "siluquant.h"

namespace {

using namespace rows;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));

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

struct NormArgs {
  const void* x;
  const uint16_t* residual;  // may be null, may be h itself
  const uint16_t* weight;
  uint8_t* q;  // null: no codes
  float* s;
  uint16_t* y;  // null: no bf16 y
  uint16_t* h;  // null: no h
  float* rstd;  // null: no statistics
  int64_t T;
  int D, lg_lanes, groups;  // lg_lanes: log2 of the lanes per group (4, 8, 16)
  float eps;
};

// h of one piece: x + residual in fp32, rounded once.
template <bool kXF32>
struct XPiece;
template <>
struct XPiece<false> {
  Piece v;
  template <Kind kKind>
  __device__ __forceinline__ void load(const void* x, int64_t at, int n) {
    v = load_bf16<kKind, false>(static_cast<const uint16_t*>(x) + at, n);
  }
  __device__ __forceinline__ Piece plus(const Piece& r) const {
    Piece o;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o.w[i] = pack_bf16(bf16_lo(v.w[i]) + bf16_lo(r.w[i]), bf16_hi(v.w[i]) + bf16_hi(r.w[i]));
    return o;
  }
  __device__ __forceinline__ Piece alone() const { return v; }
};
template <>
struct XPiece<true> {
  float v[8];
  template <Kind kKind>
  __device__ __forceinline__ void load(const void* x, int64_t at, int n) {
    load_f32<kKind>(v, static_cast<const float*>(x) + at, n);
  }
  __device__ __forceinline__ Piece plus(const Piece& r) const {
    Piece o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.w[i] = pack_bf16(v[2 * i] + bf16_lo(r.w[i]), v[2 * i + 1] + bf16_hi(r.w[i]));
    return o;
  }
  __device__ __forceinline__ Piece alone() const {
    Piece o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    return o;
  }
};

__device__ __forceinline__ float sum_squares(float acc, const Piece& p) {
  float v[8];
  unpack(v, p);
#pragma unroll
  for (int i = 0; i < 8; ++i) acc = __builtin_fmaf(v[i], v[i], acc);
  return acc;
}

__device__ __forceinline__ float inverse_rms(float sum, int D, float eps) { return 1.0f / sqrtf(sum / (float)D + eps); }

// y of one piece: (h * rstd) * w, rounded to bf16.
__device__ __forceinline__ Piece scaled(const Piece& h, const Piece& w, float rstd) {
  Piece o;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o.w[i] = pack_bf16((bf16_lo(h.w[i]) * rstd) * bf16_lo(w.w[i]), (bf16_hi(h.w[i]) * rstd) * bf16_hi(w.w[i]));
  return o;
}

// Codes and scale of one piece's group; every lane of the wave calls it.
template <bool kE4M3, Kind kKind>
__device__ __forceinline__ void quantise(const NormArgs& a, const Piece& y, int64_t row, int col, int n) {
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

// kOneWave: each wave of the workgroup takes rows of its own; otherwise the
// workgroup shares a row.  Piece c of a lane starts kPieces' width of the lanes
// further.
template <bool kOneWave, int kPieces, bool kXF32, Kind kKind, bool kE4M3>
__global__ __launch_bounds__(kOneWave ? 256 : 1024) void rms_norm_quant_kernel(const NormArgs a) {
  __shared__ float s_sum[16];
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int first = 8 * (kOneWave ? lane : (int)threadIdx.x), step = 8 * (kOneWave ? 64 : (int)blockDim.x);
  const int64_t rows_at_once = kOneWave ? waves : 1;
  for (int64_t row = blockIdx.x * rows_at_once + (kOneWave ? wave : 0); row < a.T; row += gridDim.x * rows_at_once) {
    const int64_t at = row * a.D + first;
    const int n0 = a.D - first;
    XPiece<kXF32> x[kPieces];
    Piece h[kPieces], w[kPieces];
    each_piece<kKind, kPieces>([&](auto kind, int c) { x[c].template load<decltype(kind)::value>(a.x, at + c * step, n0 - c * step); });
    if (a.residual) {
      Piece r[kPieces];
      each_piece<kKind, kPieces>([&](auto kind, int c) {
        r[c] = load_bf16<decltype(kind)::value, false>(a.residual + at + c * step, n0 - c * step);
      });
#pragma unroll
      for (int c = 0; c < kPieces; ++c) h[c] = x[c].plus(r[c]);
    } else {
#pragma unroll
      for (int c = 0; c < kPieces; ++c) h[c] = x[c].alone();
    }
    each_piece<kKind, kPieces>([&](auto kind, int c) {
      w[c] = load_bf16<decltype(kind)::value, false>(a.weight + first + c * step, n0 - c * step);
    });
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < kPieces; ++c) sum = sum_squares(sum, h[c]);
    sum = kOneWave ? wave_sum(sum) : group_sum(sum, s_sum, wave, waves);
    const float rstd = inverse_rms(sum, a.D, a.eps);
    if (a.rstd && first == 0) a.rstd[row] = rstd;
    each_piece<kKind, kPieces>([&](auto kind, int c) {
      constexpr Kind k = decltype(kind)::value;
      const int n = n0 - c * step;
      if (a.h) store_bf16<k, true>(a.h + at + c * step, h[c], n);
      const Piece y = scaled(h[c], w[c], rstd);
      if (a.y) store_bf16<k, true>(a.y + at + c * step, y, n);
      if (a.q) quantise<kE4M3, k>(a, y, row, first + c * step, n);
    });
  }
}

// Rows past 16384 columns: a workgroup of 1024 walks the row twice, the second
// time from h where it is kept (a lane reads back what it wrote itself).
constexpr int kWideThreads = 1024;
template <bool kXF32, bool kE4M3>
__global__ __launch_bounds__(kWideThreads) void rms_norm_quant_wide_kernel(const NormArgs a) {
  __shared__ float s_sum[16];
  const int tid = threadIdx.x;
  const int steps = (a.D + 8 * kWideThreads - 1) / (8 * kWideThreads);
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    const int64_t at = row * a.D;
    auto h_piece = [&](int col) {
      const int n = a.D - col;
      XPiece<kXF32> x;
      x.template load<kRagged>(a.x, at + col, n);
      return a.residual ? x.plus(load_bf16<kRagged, false>(a.residual + at + col, n)) : x.alone();
    };
    float sum = 0.0f;
    for (int i = 0; i < steps; ++i) {
      const int col = 8 * (i * kWideThreads + tid);
      const Piece h = h_piece(col);
      if (a.h) store_bf16<kRagged, true>(a.h + at + col, h, a.D - col);
      sum = sum_squares(sum, h);
    }
    sum = group_sum(sum, s_sum, tid >> 6, kWideThreads / 64);
    const float rstd = inverse_rms(sum, a.D, a.eps);
    if (a.rstd && tid == 0) a.rstd[row] = rstd;
    for (int i = 0; i < steps; ++i) {
      const int col = 8 * (i * kWideThreads + tid), n = a.D - col;
      const Piece h = a.h ? load_bf16<kRagged, false>(a.h + at + col, n) : h_piece(col);
      const Piece y = scaled(h, load_bf16<kRagged, false>(a.weight + col, n), rstd);
      if (a.y) store_bf16<kRagged, true>(a.y + at + col, y, n);
      if (a.q) quantise<kE4M3, kRagged>(a, y, row, col, n);
    }
  }
}

// ---- backward ----

struct BwdArgs {
  const void* dy;
  const uint16_t* h;
  const uint16_t* weight;
  const float* rstd;
  const uint16_t* d_h;  // may be null, may be dx itself
  uint16_t* dx;
  float* part;  // [gridDim.x, D] partial sums of dw (dw itself when there is one workgroup); null: no dw
  int64_t T;
  int D;
};

template <bool kF32, Kind kKind>
__device__ __forceinline__ void load_grad(float (&v)[8], const void* p, int64_t at, int n) {
  if constexpr (kF32)
    load_f32<kKind>(v, static_cast<const float*>(p) + at, n);
  else
    unpack(v, load_bf16<kKind, true>(static_cast<const uint16_t*>(p) + at, n));
}

// The same division of rows as in the forward pass.  A lane keeps the dw sums of
// its columns in registers over all its rows; where waves have rows of their
// own, their sums are added in LDS at the end, in wave order, so that the
// result does not depend on timing.
template <bool kOneWave, int kPieces, bool kDyF32, Kind kKind>
__global__ __launch_bounds__(kOneWave ? 512 : 1024) void rms_norm_bwd_kernel(const BwdArgs a) {
  __shared__ float s_dw[kOneWave ? 512 * kPieces : 1];
  __shared__ float s_sum[16];
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int first = 8 * (kOneWave ? lane : (int)threadIdx.x), step = 8 * (kOneWave ? 64 : (int)blockDim.x);
  const int n0 = a.D - first;
  Piece w[kPieces];
  float dw[kPieces][8];
  each_piece<kKind, kPieces>([&](auto kind, int c) {
    w[c] = load_bf16<decltype(kind)::value, false>(a.weight + first + c * step, n0 - c * step);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[c][i] = 0.0f;
  });
  const int64_t rows_at_once = kOneWave ? waves : 1;
  for (int64_t row = blockIdx.x * rows_at_once + (kOneWave ? wave : 0); row < a.T; row += gridDim.x * rows_at_once) {
    const int64_t at = row * a.D + first;
    const float rstd = a.rstd[row];
    float dy[kPieces][8];
    Piece h[kPieces], d[kPieces];
    each_piece<kKind, kPieces>([&](auto kind, int c) {
      load_grad<kDyF32, decltype(kind)::value>(dy[c], a.dy, at + c * step, n0 - c * step);
      h[c] = load_bf16<decltype(kind)::value, true>(a.h + at + c * step, n0 - c * step);
    });
    if (a.d_h) {
      each_piece<kKind, kPieces>([&](auto kind, int c) {
        d[c] = load_bf16<decltype(kind)::value, true>(a.d_h + at + c * step, n0 - c * step);
      });
    } else {
#pragma unroll
      for (int c = 0; c < kPieces; ++c) d[c] = zero_piece();
    }
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
      float hv[8], wv[8];
      unpack(hv, h[c]);
      unpack(wv, w[c]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = hv[i] * rstd;
        dw[c][i] = __builtin_fmaf(dy[c][i], n, dw[c][i]);
        sum = __builtin_fmaf(dy[c][i] * wv[i], n, sum);
      }
    }
    sum = kOneWave ? wave_sum(sum) : group_sum(sum, s_sum, wave, waves);
    const float mean = sum / (float)a.D;
    each_piece<kKind, kPieces>([&](auto kind, int c) {
      float hv[8], wv[8], dv[8], o[8];
      unpack(hv, h[c]);
      unpack(wv, w[c]);
      unpack(dv, d[c]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = hv[i] * rstd, g = dy[c][i] * wv[i];
        o[i] = __builtin_fmaf(rstd, __builtin_fmaf(-n, mean, g), dv[i]);
      }
      const Piece out = {{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7])}};
      store_bf16<decltype(kind)::value, false>(a.dx + at + c * step, out, n0 - c * step);
    });
  }
  if (!a.part) return;
  if (kOneWave) {
    // wave by wave into LDS; a lane only ever touches the places of its own columns
    for (int turn = 0; turn < waves; ++turn) {
      if (wave == turn) {
#pragma unroll
        for (int c = 0; c < kPieces; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float* p = &s_dw[(c * 8 + i) * 64 + lane];
            if (turn > 0) dw[c][i] += *p;
            *p = dw[c][i];
          }
      }
      __syncthreads();
    }
    if (wave != waves - 1) return;
  }
  float* out = a.part + (int64_t)blockIdx.x * a.D + first;
  each_piece<kKind, kPieces>([&](auto kind, int c) {
    const int n = n0 - c * step;
    if (decltype(kind)::value == kFull || n >= 8) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        *reinterpret_cast<f32x4_a4*>(out + c * step + 4 * k) =
            (f32x4){dw[c][4 * k], dw[c][4 * k + 1], dw[c][4 * k + 2], dw[c][4 * k + 3]};
    } else {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (i < n) out[c * step + i] = dw[c][i];
    }
  });
}

// dw[d] = the sum of the partial rows: 16 columns per workgroup, 64 strips of
// rows (every 64th), each in row order, and then the strips in pairs, halving
// their number, always the same ones.
constexpr int kSumStrips = 64, kSumCols = 16;
__global__ __launch_bounds__(kSumCols * kSumStrips) void rms_norm_dw_kernel(const float* part, float* dw, int parts, int D) {
  __shared__ float s[kSumStrips][kSumCols];
  const int c = threadIdx.x & (kSumCols - 1), strip = threadIdx.x / kSumCols;
  const int col = blockIdx.x * kSumCols + c;
  float sum = 0.0f;
  if (col < D) {
#pragma unroll 8
    for (int p = strip; p < parts; p += kSumStrips) sum += part[(int64_t)p * D + col];
  }
  s[strip][c] = sum;
  __syncthreads();
  for (int half = kSumStrips / 2; half > 0; half >>= 1) {
    if (strip < half) s[strip][c] += s[strip + half][c];
    __syncthreads();
  }
  if (strip == 0 && col < D) dw[col] = s[0][c];
}

// Rows past 16384 columns, in two launches: a workgroup per row for the mean,
// then tiles of columns over strips of rows.
template <bool kDyF32>
__global__ __launch_bounds__(kWideThreads) void rms_norm_bwd_mean_kernel(const BwdArgs a, float* mean) {
  __shared__ float s_sum[kWideThreads / 64];
  const int tid = threadIdx.x;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    const float rstd = a.rstd[row];
    float sum = 0.0f;
    for (int col = 8 * tid; col < a.D; col += 8 * kWideThreads) {
      float dy[8], hv[8], wv[8];
      load_grad<kDyF32, kRagged>(dy, a.dy, row * a.D + col, a.D - col);
      unpack(hv, load_bf16<kRagged, false>(a.h + row * a.D + col, a.D - col));
      unpack(wv, load_bf16<kRagged, false>(a.weight + col, a.D - col));
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(dy[i] * wv[i], hv[i] * rstd, sum);
    }
    sum = wave_sum(sum);
    if ((tid & 63) == 0) s_sum[tid >> 6] = sum;
    __syncthreads();
    if (tid == 0) {
      for (int i = 1; i < kWideThreads / 64; ++i) sum += s_sum[i];
      mean[row] = sum / (float)a.D;
    }
    __syncthreads();
  }
}
constexpr int kTileThreads = 256;
template <bool kDyF32>
__global__ __launch_bounds__(kTileThreads) void rms_norm_bwd_tile_kernel(const BwdArgs a, const float* mean) {
  const int col = 8 * ((int)blockIdx.x * kTileThreads + (int)threadIdx.x), n = a.D - col;
  if (n <= 0) return;
  float wv[8], dw[8] = {};
  unpack(wv, load_bf16<kRagged, false>(a.weight + col, n));
  for (int64_t row = blockIdx.y; row < a.T; row += gridDim.y) {
    const float rstd = a.rstd[row], m = mean[row];
    float dy[8], hv[8], dv[8], o[8];
    load_grad<kDyF32, kRagged>(dy, a.dy, row * a.D + col, n);
    unpack(hv, load_bf16<kRagged, false>(a.h + row * a.D + col, n));
    unpack(dv, a.d_h ? load_bf16<kRagged, false>(a.d_h + row * a.D + col, n) : zero_piece());
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = hv[i] * rstd;
      dw[i] = __builtin_fmaf(dy[i], t, dw[i]);
      o[i] = __builtin_fmaf(rstd, __builtin_fmaf(-t, m, dy[i] * wv[i]), dv[i]);
    }
    const Piece out = {{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7])}};
    store_bf16<kRagged, true>(a.dx + row * a.D + col, out, n);
  }
  if (a.part) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) a.part[(int64_t)blockIdx.y * a.D + col + i] = dw[i];
  }
}

constexpr int64_t kMaxD = int64_t(1) << 22, kMaxT = int64_t(1) << 31;
constexpr int kRegisterD = 16384;  // rows up to here stay in registers
constexpr int kMaxGrid = 1 << 20;  // workgroups of the forward kernels; further rows are walked

// Workgroups of the backward pass, each with a partial dw row: eight waves per
// CU (16384 x 4096, four waves each: 256 workgroups 104 us, 512 90 us, 1024 103
// us), and one workgroup per CU at the least.
int bwd_parts(int64_t T, int64_t D) {
  const int64_t waves = D <= 1024 ? 8 : D <= kRegisterD ? (D + 1023) / 1024 : 8;
  return (int)std::min<int64_t>(T, std::max<int64_t>(256, 2048 / waves));
}

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

template <bool kOneWave, int kPieces>
void launch_norm(const NormArgs& a, bool f32, bool e4m3, int waves, hipStream_t stream) {
  const int64_t groups = kOneWave ? (a.T + waves - 1) / waves : a.T;
  const dim3 grid((unsigned)std::min<int64_t>(groups, kMaxGrid)), block(64 * waves);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, a); };
  with_kind<kPieces>(a.D, 512 * kPieces * (kOneWave ? 1 : waves), [&](auto kind) {
    constexpr Kind k = decltype(kind)::value;
    if (f32)
      e4m3 ? go(rms_norm_quant_kernel<kOneWave, kPieces, true, k, true>) : go(rms_norm_quant_kernel<kOneWave, kPieces, true, k, false>);
    else
      e4m3 ? go(rms_norm_quant_kernel<kOneWave, kPieces, false, k, true>) : go(rms_norm_quant_kernel<kOneWave, kPieces, false, k, false>);
  });
}

template <bool kOneWave, int kPieces>
void launch_bwd(const BwdArgs& a, bool f32, int grid, int waves, hipStream_t stream) {
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(grid), dim3(64 * waves), 0, stream, a); };
  with_kind<kPieces>(a.D, 512 * kPieces * (kOneWave ? 1 : waves), [&](auto kind) {
    constexpr Kind k = decltype(kind)::value;
    f32 ? go(rms_norm_bwd_kernel<kOneWave, kPieces, true, k>) : go(rms_norm_bwd_kernel<kOneWave, kPieces, false, k>);
  });
}

}  // namespace

hipError_t code_objects::load_rmsnorm() { return load(rms_norm_dw_kernel); }

extern "C" {

__attribute__((visibility("default"))) int rms_norm_quant(const void* x, int x_dtype, const void* residual,
                                                          const void* weight, void* y_q, float* y_s, void* y_bf16,
                                                          void* h, float* rstd, int64_t T, int64_t D, int64_t group,
                                                          int code_format, float eps, hipStream_t stream) {
  if (group != 32 && group != 64 && group != 128) return SILUQUANT_ERR_BAD_GROUP;
  if (T < 0 || D < 0 || T > kMaxT || D > kMaxD || !(eps >= 0.0f) || eps == __builtin_huge_valf() ||
      (x_dtype != SILUQUANT_F32 && x_dtype != SILUQUANT_BF16) ||
      (code_format != SILUQUANT_CODE_INT8 && code_format != SILUQUANT_CODE_E4M3))
    return SILUQUANT_ERR_BAD_SHAPE;
  if (T == 0 || D == 0) return SILUQUANT_OK;
  if (!x || !weight || (!y_q && !y_bf16) || (y_q == nullptr) != (y_s == nullptr)) return SILUQUANT_ERR_NULL_PTR;
  if (misaligned(x, 16) || misaligned(residual, 16) || misaligned(weight, 16) || misaligned(y_q, 16) ||
      misaligned(y_bf16, 16) || misaligned(h, 16) || misaligned(y_s, 4) || misaligned(rstd, 4))
    return SILUQUANT_ERR_MISALIGNED;
  const bool f32 = x_dtype == SILUQUANT_F32;
  const int64_t groups = (D + group - 1) / group;
  const Span in[3] = {{x, T * D * (f32 ? 4 : 2)}, {residual, 2 * T * D}, {weight, 2 * D}};
  const Span out[5] = {{y_q, T * D}, {y_s, 4 * T * groups}, {y_bf16, 2 * T * D}, {h, 2 * T * D}, {rstd, 4 * T}};
  for (int o = 0; o < 5; ++o) {
    for (int i = 0; i < 3; ++i)
      if (overlap(out[o], in[i]) && !(o == 3 && i == 1 && h == residual)) return SILUQUANT_ERR_OVERLAP;
    for (int i = 0; i < o; ++i)
      if (overlap(out[o], out[i])) return SILUQUANT_ERR_OVERLAP;
  }
  const bool e4m3 = code_format == SILUQUANT_CODE_E4M3;
  const NormArgs a = {x, static_cast<const uint16_t*>(residual), static_cast<const uint16_t*>(weight),
                      static_cast<uint8_t*>(y_q), y_s, static_cast<uint16_t*>(y_bf16), static_cast<uint16_t*>(h),
                      rstd, T, (int)D, group == 32 ? 2 : group == 64 ? 3 : 4, (int)groups, eps};
  if (D > kRegisterD) {
    const dim3 grid((unsigned)std::min<int64_t>(T, kMaxGrid)), block(kWideThreads);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, a); };
    if (f32)
      e4m3 ? go(rms_norm_quant_wide_kernel<true, true>) : go(rms_norm_quant_wide_kernel<true, false>);
    else
      e4m3 ? go(rms_norm_quant_wide_kernel<false, true>) : go(rms_norm_quant_wide_kernel<false, false>);
  } else {
    if (D <= 512) launch_norm<true, 1>(a, f32, e4m3, 4, stream);
    else if (D <= 1024) launch_norm<true, 2>(a, f32, e4m3, 4, stream);
    else launch_norm<false, 2>(a, f32, e4m3, (int)((D + 1023) / 1024), stream);
  }
  return hipGetLastError() == hipSuccess ? SILUQUANT_OK : SILUQUANT_ERR_LAUNCH_FAILED;
}

__attribute__((visibility("default"))) int64_t rms_norm_bwd_workspace_bytes(int64_t T, int64_t D) {
  if (T < 0 || D < 0 || T > kMaxT || D > kMaxD) return -1;
  if (T == 0 || D == 0) return 0;
  return 4 * bwd_parts(T, D) * D + (D > kRegisterD ? 4 * T : 0);
}

__attribute__((visibility("default"))) int rms_norm_bwd(const void* dy, int dy_dtype, const void* h, const void* weight,
                                                        const float* rstd, const void* d_h, void* dx, float* dw,
                                                        void* workspace, int64_t workspace_bytes, int64_t T, int64_t D,
                                                        hipStream_t stream) {
  if (T < 0 || D < 0 || T > kMaxT || D > kMaxD || (dy_dtype != SILUQUANT_F32 && dy_dtype != SILUQUANT_BF16))
    return SILUQUANT_ERR_BAD_SHAPE;
  if (D == 0) return SILUQUANT_OK;
  const int64_t need = rms_norm_bwd_workspace_bytes(T, D);
  if (T == 0) {  // no rows: no gradient for the weight
    if (!dw) return SILUQUANT_OK;
    if (misaligned(dw, 4)) return SILUQUANT_ERR_MISALIGNED;
    hipLaunchKernelGGL(rms_norm_dw_kernel, dim3((unsigned)((D + kSumCols - 1) / kSumCols)), dim3(kSumCols * kSumStrips), 0, stream,
                       (const float*)nullptr, dw, 0, (int)D);
    return hipGetLastError() == hipSuccess ? SILUQUANT_OK : SILUQUANT_ERR_LAUNCH_FAILED;
  }
  const bool wide = D > kRegisterD;
  if (!dw && !wide) workspace = nullptr, workspace_bytes = need;  // not looked at
  if (!dy || !h || !weight || !rstd || !dx || ((dw || wide) && !workspace)) return SILUQUANT_ERR_NULL_PTR;
  if (workspace_bytes < need) return SILUQUANT_ERR_BAD_SHAPE;
  if (misaligned(dy, 16) || misaligned(h, 16) || misaligned(weight, 16) || misaligned(d_h, 16) || misaligned(dx, 16) ||
      misaligned(rstd, 4) || misaligned(dw, 4) || misaligned(workspace, 16))
    return SILUQUANT_ERR_MISALIGNED;
  const bool f32 = dy_dtype == SILUQUANT_F32;
  const Span in[5] = {{dy, T * D * (f32 ? 4 : 2)}, {h, 2 * T * D}, {weight, 2 * D}, {rstd, 4 * T}, {d_h, 2 * T * D}};
  const Span out[3] = {{dx, 2 * T * D}, {dw, 4 * D}, {workspace, workspace_bytes}};
  for (int o = 0; o < 3; ++o) {
    for (int i = 0; i < 5; ++i)
      if (overlap(out[o], in[i]) && !(o == 0 && i == 4 && dx == d_h)) return SILUQUANT_ERR_OVERLAP;
    for (int i = 0; i < o; ++i)
      if (overlap(out[o], out[i])) return SILUQUANT_ERR_OVERLAP;
  }
  const int parts = bwd_parts(T, D);
  float* ws = static_cast<float*>(workspace);
  float* part = !dw ? nullptr : parts == 1 ? dw : ws;
  const BwdArgs a = {dy, static_cast<const uint16_t*>(h), static_cast<const uint16_t*>(weight), rstd,
                     static_cast<const uint16_t*>(d_h), static_cast<uint16_t*>(dx), part, T, (int)D};
  if (wide) {
    float* mean = ws + (int64_t)parts * D;
    const dim3 rows_grid((unsigned)std::min<int64_t>(T, kMaxGrid));
    const dim3 tiles((unsigned)((D + 8 * kTileThreads - 1) / (8 * kTileThreads)), (unsigned)parts);
    if (f32) {
      hipLaunchKernelGGL((rms_norm_bwd_mean_kernel<true>), rows_grid, dim3(kWideThreads), 0, stream, a, mean);
      hipLaunchKernelGGL((rms_norm_bwd_tile_kernel<true>), tiles, dim3(kTileThreads), 0, stream, a, mean);
    } else {
      hipLaunchKernelGGL((rms_norm_bwd_mean_kernel<false>), rows_grid, dim3(kWideThreads), 0, stream, a, mean);
      hipLaunchKernelGGL((rms_norm_bwd_tile_kernel<false>), tiles, dim3(kTileThreads), 0, stream, a, mean);
    }
  } else {
    const int waves = (int)std::min<int64_t>((T + parts - 1) / parts, 8);
    if (D <= 512) launch_bwd<true, 1>(a, f32, parts, waves, stream);
    else if (D <= 1024) launch_bwd<true, 2>(a, f32, parts, waves, stream);
    else launch_bwd<false, 2>(a, f32, parts, (int)((D + 1023) / 1024), stream);
  }
  if (dw && parts > 1)
    hipLaunchKernelGGL(rms_norm_dw_kernel, dim3((unsigned)((D + kSumCols - 1) / kSumCols)), dim3(kSumCols * kSumStrips), 0, stream, part, dw,
                       parts, (int)D);
  return hipGetLastError() == hipSuccess ? SILUQUANT_OK : SILUQUANT_ERR_LAUNCH_FAILED;
}

}  // extern "C"
