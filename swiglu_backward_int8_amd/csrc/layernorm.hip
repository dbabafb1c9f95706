// Layer norm with a dropout and the residual's addition in front of it and the
// group quantiser of the library behind it, its backward pass, and the dropout
// alone, for gfx950.
//
//   forward   h = bf16(residual + dropout(x));  mean = sum(h) / D
//             rstd = 1 / sqrt(sum((h - mean)^2) / D + eps)
//             y = bf16(((h - mean) * rstd) * w + b);  codes and scales of y by group
//   backward  n = (h - mean) * rstd;  g = dy * w
//             dx = rstd * (g - sum(g) / D - n * sum(g * n) / D) + d_h
//             dx_drop = dropout'(dx);  dw = sum over rows of dy * n;  db = of dy
//
// All read and write every element once but for rows past 16384 columns, which are read
// twice.  Up to there a row stays in registers between its sums and its use.  The sum
// of squares is that of the differences from the mean, so that an offset of the row
// costs no bits: a wave takes its own columns' mean, then their squares around it, and
// the waves of a row exchange both at once (one barrier a row): with n_w columns, sum
// s_w and squares q_w of wave w,
//   mean = sum(s_w) / D;  sum((h - mean)^2) = sum(q_w + n_w (s_w / n_w - mean)^2).
// The sums are fp32; h is rounded to bf16 before the statistics because that is
// the stream the next layer and the backward pass read, and y is rounded to
// bf16 before quantising as everywhere in this library.
//
// Layout as in the RMS norm: a lane owns one or two pieces of 8 columns, rows of up
// to 1024 columns go to a wave each, longer ones, up to 16384, to a workgroup.
//
// Memory bounds the large ones (a large copy moves 5.1 TB/s): of 16384 x 4096 in bf16
// the forward pass with dropout and residual (x, residual, h and y, 537 MB) takes 94 us,
// 5.7 TB/s, without dropout 93, to int8 84; the backward pass with the stream's gradient
// and dropout (dy, h, d_h, dx and dx_drop, 671 MB) 125 us, 5.35 TB/s.  The smallest are
// a launch and one row's latency.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "code_objects.h"
#include "dropout.h"
#include "norm_rows.h"
#include "siluquant.h"

namespace {

using namespace rows;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));

struct LnArgs {
  const void* x;
  const uint16_t* residual;  // may be null, may be h itself
  const uint16_t* weight;
  const uint16_t* bias;  // may be null
  uint8_t* q;            // null: no codes
  float* s;
  uint16_t* y;  // null: no bf16 y
  uint16_t* h;  // null: no h
  float* mean;  // null: no statistics
  float* rstd;
  int64_t T;
  int D, lg_lanes, groups;  // lg_lanes: log2 of the lanes per group (4, 8, 16)
  bool e4m3;
  float eps;
  Dropout drop;
};

template <bool kF32, Kind kKind>
__device__ __forceinline__ void load_x(float (&v)[8], const void* p, int64_t at, int n) {
  if constexpr (kF32)
    load_f32<kKind>(v, static_cast<const float*>(p) + at, n);
  else
    unpack(v, load_bf16<kKind, false>(static_cast<const uint16_t*>(p) + at, n));
}

// Pieces are loaded as they lie in memory and settled where they are used: what is
// partial is loaded from where it ends, and shifting it at once would wait for it
// with the other loads of the row not yet asked for (16384 x 4100: forward 125 us, so
// 109; backward 221 and 178).
template <Kind kKind, bool kNt>
__device__ __forceinline__ Piece load_raw(const uint16_t* p, int n) {
  if constexpr (kKind == kRagged)
    return load_bf16<kFull, kNt>(p - (n < 8 ? 8 - n : 0), 8);
  else
    return load_bf16<kKind, kNt>(p, n);
}
template <Kind kKind>
__device__ __forceinline__ void settle(Piece& p, int n) {
  if constexpr (kKind == kRagged) p = shifted(p, n < 8 ? 8 - n : 0);
}

// Eight values as they were loaded: bf16 ones take half the registers.
template <bool kF32, bool kNt>
struct Loaded;
template <bool kNt>
struct Loaded<false, kNt> {
  Piece p;
  template <Kind kKind>
  __device__ __forceinline__ void load(const void* from, int64_t at, uint32_t col, int n) {
    p = load_raw<kKind, kNt>(static_cast<const uint16_t*>(from) + at + col, n);
  }
  template <Kind kKind>
  __device__ __forceinline__ void settled(int n) { settle<kKind>(p, n); }
  __device__ __forceinline__ void get(float (&v)[8]) const { unpack(v, p); }
};
template <bool kNt>
struct Loaded<true, kNt> {
  float p[8];
  template <Kind kKind>
  __device__ __forceinline__ void load(const void* from, int64_t at, uint32_t col, int n) {
    const float* q = static_cast<const float*>(from) + at + col;
    if constexpr (kKind == kRagged)
      load_f32<kFull>(p, q - (n < 8 ? 8 - n : 0), 8);
    else
      load_f32<kKind>(p, q, n);
  }
  template <Kind kKind>
  __device__ __forceinline__ void settled(int n) {
    if constexpr (kKind == kRagged) {
      const int d = n < 8 ? 8 - n : 0;
#pragma unroll
      for (int k = 4; k >= 1; k >>= 1)
        if (d & k) {
#pragma unroll
          for (int i = 0; i < 8; ++i) p[i] = i + k < 8 ? p[i + k] : 0.0f;
        }
      if (d >= 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = 0.0f;
      }
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p[i];
  }
};

// Makes the compiler unpack a piece again where it is used next: kept unpacked over
// a reduction, a row takes twice the registers.
__device__ __forceinline__ void fold(Piece& p) {
#pragma unroll
  for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(p.w[i]));
}

__device__ __forceinline__ Piece pack8(const float (&v)[8]) {
  return {{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])}};
}

// residual + v, eight fp32 additions.
__device__ __forceinline__ void add(float (&v)[8], const Piece& r) {
  float f[8];
  unpack(f, r);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = f[i] + v[i];
}

__device__ __forceinline__ float sum8(const Piece& p) {
  float v[8];
  unpack(v, p);
  return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
}

// acc + the squares of the differences from mean of a piece's first n elements.
template <Kind kKind>
__device__ __forceinline__ float squares(float acc, const Piece& p, float mean, int n) {
  if (kKind == kWhole && n <= 0) return acc;
  float v[8];
  unpack(v, p);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float d = kKind < kRagged || i < n ? v[i] - mean : 0.0f;
    acc = __builtin_fmaf(d, d, acc);
  }
  return acc;
}

__device__ __forceinline__ float inverse_std(float squares, int D, float eps) {
  return 1.0f / sqrtf(squares / (float)D + eps);
}

// y of one piece: ((h - mean) * rstd) * w + b, rounded to bf16.
__device__ __forceinline__ Piece normed(const Piece& h, const Piece& w, const Piece& b, float mean, float rstd) {
  float v[8], wv[8], bv[8];
  unpack(v, h);
  unpack(wv, w);
  unpack(bv, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __builtin_fmaf((v[i] - mean) * rstd, wv[i], bv[i]);
  return pack8(v);
}

// Zeros in a partial piece's places past the row, for its group's scale: what a row
// makes of the zeros there is (0 - mean) * rstd * 0, NaN where the first product overflows.
__device__ __forceinline__ Piece cut(Piece v, int n) {
  if (n < 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v.w[i] = n > 2 * i + 1 ? v.w[i] : n > 2 * i ? v.w[i] & 0xffffu : 0;
  }
  return v;
}

// kOneWave: each wave of the workgroup takes rows of its own; otherwise the
// workgroup shares a row.  Piece c of a lane starts kPieces' width of the lanes
// further.
template <bool kOneWave, int kPieces, bool kXF32, Kind kKind, bool kDrop>
__global__ __launch_bounds__(kOneWave ? 256 : 1024) void layer_norm_quant_kernel(const LnArgs a) {
  __shared__ float s_stat[2][2][16];  // [row's turn][sum, squares][wave]
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int first = 8 * (kOneWave ? lane : (int)threadIdx.x), step = 8 * (kOneWave ? 64 : (int)blockDim.x);
  const int64_t rows_at_once = kOneWave ? waves : 1;
  DropKey key = {};
  if (kDrop) key = drop_key(a.drop);
  int turn = 0;
  for (int64_t row = blockIdx.x * rows_at_once + (kOneWave ? wave : 0); row < a.T; row += gridDim.x * rows_at_once) {
    const int64_t at = row * a.D;  // the same in every lane: addresses are a scalar and a 32-bit offset
    const int n0 = a.D - first;
    auto col = [&](int c) { return (uint32_t)(first + c * step); };
    Loaded<kXF32, false> x[kPieces];
    Piece h[kPieces], w[kPieces];
    each_piece<kKind, kPieces>([&](auto kind, int c) { x[c].template load<decltype(kind)::value>(a.x, at, col(c), n0 - c * step); });
    if (a.residual) {
      each_piece<kKind, kPieces>([&](auto kind, int c) {
        h[c] = load_raw<decltype(kind)::value, false>(a.residual + at + col(c), n0 - c * step);
      });
    } else {
#pragma unroll
      for (int c = 0; c < kPieces; ++c) h[c] = zero_piece();
    }
    each_piece<kKind, kPieces>([&](auto kind, int c) {
      w[c] = load_raw<decltype(kind)::value, false>(a.weight + col(c), n0 - c * step);
    });
    each_piece<kKind, kPieces>([&](auto kind, int c) {
      constexpr Kind k = decltype(kind)::value;
      const int n = n0 - c * step;
      x[c].template settled<k>(n), settle<k>(h[c], n), settle<k>(w[c], n);
    });
    float sum = 0.0f, sq = 0.0f, mean, rstd;
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
      float v[8];
      x[c].get(v);
      if (kDrop) drop8(v, a.drop, key, row, first + c * step);
      if (a.residual) add(v, h[c]);
      h[c] = pack8(v);
      sum += sum8(h[c]);
      fold(h[c]);
      if (kDrop) __builtin_amdgcn_sched_barrier(0);  // one piece's generator at a time
    }
    sum = wave_sum(sum);
    // the columns of wave v of the workgroup
    auto columns = [&](int v) {
      int n = 0;
#pragma unroll
      for (int c = 0; c < kPieces; ++c) n += min(max(a.D - 512 * v - c * step, 0), 512);
      return (float)n;
    };
    mean = sum / (kOneWave ? (float)a.D : columns(wave));
    each_piece<kKind, kPieces>([&](auto kind, int c) { sq = squares<decltype(kind)::value>(sq, h[c], mean, n0 - c * step); });
    sq = wave_sum(sq);
    if (!kOneWave) {
      if (lane == 0) s_stat[turn][0][wave] = sum, s_stat[turn][1][wave] = sq;
      __syncthreads();
      const int v = lane & 15;
      const float s = v < waves ? s_stat[turn][0][v] : 0.0f, q = v < waves ? s_stat[turn][1][v] : 0.0f;
      turn ^= 1;  // the next row's go elsewhere: every wave has read these before that row's barrier lets any past it
      mean = sum16(s) / (float)a.D;
      const float n = columns(v), d = v < waves ? s / n - mean : 0.0f;
      sq = sum16(__builtin_fmaf(n * d, d, q));
    }
    rstd = inverse_std(sq, a.D, a.eps);
    if (first == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    each_piece<kKind, kPieces>([&](auto kind, int c) {
      constexpr Kind k = decltype(kind)::value;
      const int n = n0 - c * step;
      const Piece b = a.bias ? load_bf16<k, false>(a.bias + col(c), n) : zero_piece();
      fold(h[c]);
      if (a.h) store_bf16<k, true>(a.h + at + col(c), h[c], n);
      // an empty piece's y is zero, whatever the row's offset
      Piece y = normed(h[c], w[c], b, k == kWhole && n <= 0 ? 0.0f : mean, rstd);
      if (a.y) store_bf16<k, true>(a.y + at + col(c), y, n);
      if (a.q) {
        if (k >= kRagged) y = cut(y, n);
        a.e4m3 ? quantise<true, k>(a, y, row, first + c * step, n) : quantise<false, k>(a, y, row, first + c * step, n);
      }
    });
  }
}

// Rows past 16384 columns: a workgroup of 1024 walks the row twice, the second
// time from h where it is kept (a lane reads back what it wrote itself).  The
// first time every lane joins its pieces' means and squares one by one.  4096 x 20000
// takes 188 us, 3.5 TB/s of what has to be read and written once, 4096 x 20001 211.
constexpr int kWideThreads = 1024;
template <bool kXF32>
__global__ __launch_bounds__(kWideThreads) void layer_norm_quant_wide_kernel(const LnArgs a) {
  __shared__ float s_sum[16];
  const int tid = threadIdx.x, wave = tid >> 6, waves = kWideThreads / 64;
  const int steps = (a.D + 8 * kWideThreads - 1) / (8 * kWideThreads);
  DropKey key = {};
  if (a.drop.rng) key = drop_key(a.drop);
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    const int64_t at = row * a.D;
    auto h_piece = [&](int col) {
      const int n = a.D - col;
      float x[8];
      load_x<kXF32, kRagged>(x, a.x, at + col, n);
      if (a.drop.rng) drop8(x, a.drop, key, row, col);
      if (a.residual) add(x, load_bf16<kRagged, false>(a.residual + at + col, n));
      return pack8(x);
    };
    float count = 0.0f, mean = 0.0f, sq = 0.0f;
    for (int i = 0; i < steps; ++i) {
      const int col = 8 * (i * kWideThreads + tid), n = min(a.D - col, 8);
      const Piece h = h_piece(col);
      if (a.h) store_bf16<kRagged, true>(a.h + at + col, h, n);
      if (n > 0) {
        const float k = (float)n, m = sum8(h) / k, d = m - mean, part = k / (count + k);
        sq = squares<kRagged>(sq, h, m, n) + (count > 0.0f ? d * d * (count * part) : 0.0f);  // at first d is all of m
        mean = __builtin_fmaf(d, part, mean);
        count += k;
      }
    }
    const float own = mean;
    mean = group_sum(count * own, s_sum, wave, waves) / (float)a.D;
    sq = group_sum(__builtin_fmaf(count * (own - mean), own - mean, sq), s_sum, wave, waves);
    const float rstd = inverse_std(sq, a.D, a.eps);
    if (tid == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    for (int i = 0; i < steps; ++i) {
      const int col = 8 * (i * kWideThreads + tid), n = a.D - col;
      const Piece h = a.h ? load_bf16<kRagged, false>(a.h + at + col, n) : h_piece(col);
      const Piece b = a.bias ? load_bf16<kRagged, false>(a.bias + col, n) : zero_piece();
      Piece y = normed(h, load_bf16<kRagged, false>(a.weight + col, n), b, n > 0 ? mean : 0.0f, rstd);
      if (a.y) store_bf16<kRagged, true>(a.y + at + col, y, n);
      if (a.q) {
        if (a.D & 7) y = cut(y, n);
        a.e4m3 ? quantise<true, kRagged>(a, y, row, col, n) : quantise<false, kRagged>(a, y, row, col, n);
      }
    }
  }
}

// ---- backward ----

struct LnBwdArgs {
  const void* dy;
  const uint16_t* h;
  const uint16_t* weight;
  const float* mean;
  const float* rstd;
  const uint16_t* d_h;  // may be null, may be dx itself
  uint16_t* dx;
  uint16_t* dx_drop;  // null: nothing was dropped, or the gradient is not wanted
  float* part_dw;     // [gridDim.x, D] partial sums (the sums themselves when there is one workgroup); null: not wanted
  float* part_db;
  int64_t T;
  int D;
  Dropout drop;
};

// dx of one piece in fp32.  c1, c2: the row's sum(g) / D and sum(g * n) / D.
__device__ __forceinline__ void grad8(float (&o)[8], const float (&dy)[8], const Piece& h, const Piece& w, const Piece& d,
                                      float mean, float rstd, float c1, float c2) {
  float hv[8], wv[8], dv[8];
  unpack(hv, h);
  unpack(wv, w);
  unpack(dv, d);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float n = (hv[i] - mean) * rstd, g = __builtin_fmaf(dy[i], wv[i], -c1);
    o[i] = __builtin_fmaf(rstd, __builtin_fmaf(-n, c2, g), dv[i]);
  }
}

// The same division of rows as in the forward pass.  A lane keeps the dw and db
// sums of its columns in registers over all its rows; where waves have rows of
// their own, their sums are added in LDS at the end, in wave order, so that the
// result does not depend on timing.  Workgroups of more than eight waves have 128
// registers a lane: they read weight and d_h where they use them, and with dropout or
// rows off 16 bytes most keep up to 30 registers in scratch memory all the same (4096 x
// 12288 83 us, 4.85 TB/s, with dropout 101; 4096 x 11008, whose last pieces are partly
// empty, 80.5 and 122; 4096 x 9001 87 and 158).
//
// A row's loads go out while the one before is computed: without that the row's
// reductions and the memory take turns (16384 x 4096 with dropout 130 us for 125, ragged
// rows of 4100 289 us for 205).  The gradients are written past the caches, which
// nobody reads them from (130 us, so 125).
template <bool kOneWave, int kPieces, int kThreads, bool kDyF32, Kind kKind, bool kDrop>
__global__ __launch_bounds__(kThreads) void layer_norm_bwd_kernel(const LnBwdArgs a) {
  constexpr bool kLate = kThreads > 512;
  __shared__ float s_part[kOneWave ? 2 * 512 * kPieces : 1];
  __shared__ float s_stat[2][2][16];
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int first = 8 * (kOneWave ? lane : (int)threadIdx.x), step = 8 * (kOneWave ? 64 : (int)blockDim.x);
  const int n0 = a.D - first;
  auto col = [&](int c) { return (uint32_t)(first + c * step); };
  DropKey key = {};
  if (kDrop) key = drop_key(a.drop);
  Piece w[kPieces];
  float dw[kPieces][8], db[kPieces][8];
  auto load_weight = [&](auto kind, int c) {
    w[c] = load_bf16<decltype(kind)::value, false>(a.weight + col(c), n0 - c * step);
  };
  auto load_dh = [&](int64_t at, Piece (&d)[kPieces]) {
    if (a.d_h) {
      each_piece<kKind, kPieces>([&](auto kind, int c) {
        d[c] = load_raw<decltype(kind)::value, true>(a.d_h + at + col(c), n0 - c * step);
      });
    } else {
#pragma unroll
      for (int c = 0; c < kPieces; ++c) d[c] = zero_piece();
    }
  };
#pragma unroll
  for (int c = 0; c < kPieces; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[c][i] = db[c][i] = 0.0f;
  if (!kLate) each_piece<kKind, kPieces>(load_weight);
  // A row's loads, but with kLate, go out while the row before it is computed.
  struct Row {
    Loaded<kDyF32, true> dy[kPieces];
    Piece h[kPieces], d[kPieces];
    float mean, rstd;
  };
  auto load_row = [&](int64_t row, Row& r) {
    const int64_t at = row * a.D;
    r.mean = a.mean[row], r.rstd = a.rstd[row];
    each_piece<kKind, kPieces>([&](auto kind, int c) {
      r.dy[c].template load<decltype(kind)::value>(a.dy, at, col(c), n0 - c * step);
      r.h[c] = load_raw<decltype(kind)::value, true>(a.h + at + col(c), n0 - c * step);
    });
    if (!kLate) load_dh(at, r.d);
  };
  const int64_t stride = gridDim.x * (int64_t)(kOneWave ? waves : 1);
  int64_t row = blockIdx.x * (int64_t)(kOneWave ? waves : 1) + (kOneWave ? wave : 0);
  int turn = 0;
  Row next;
  if (!kLate && row < a.T) load_row(row, next);
  for (; row < a.T; row += stride) {
    const int64_t at = row * a.D;
    Row r;
    if (kLate) {
      load_row(row, r);
      each_piece<kKind, kPieces>(load_weight);
    } else {
      r = next;
      if (row + stride < a.T) load_row(row + stride, next);
    }
    const float mean = r.mean, rstd = r.rstd;
    each_piece<kKind, kPieces>([&](auto kind, int c) {
      constexpr Kind k = decltype(kind)::value;
      const int n = n0 - c * step;
      r.dy[c].template settled<k>(n), settle<k>(r.h[c], n);
      if (!kLate) settle<k>(r.d[c], n);
    });
    float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
      float hv[8], wv[8], dv[8];
      unpack(hv, r.h[c]);
      unpack(wv, w[c]);
      r.dy[c].get(dv);
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // places past the row have dy = 0, and n = 0 (-mean * rstd may overflow)
        const int left = n0 - c * step;
        const bool in = c < kPieces - 1 || kKind == kFull || (kKind == kWhole ? left > 0 : i < left);
        const float n = in ? (hv[i] - mean) * rstd : 0.0f, g = dv[i] * wv[i];
        dw[c][i] = __builtin_fmaf(dv[i], n, dw[c][i]);
        db[c][i] += dv[i];
        c1 += g;
        c2 = __builtin_fmaf(g, n, c2);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    c1 = wave_sum(c1), c2 = wave_sum(c2);
    if (!kOneWave) {
      if (lane == 0) s_stat[turn][0][wave] = c1, s_stat[turn][1][wave] = c2;
      __syncthreads();
      const int v = lane & 15;
      c1 = sum16(v < waves ? s_stat[turn][0][v] : 0.0f), c2 = sum16(v < waves ? s_stat[turn][1][v] : 0.0f);
      turn ^= 1;
    }
    c1 = c1 / (float)a.D, c2 = c2 / (float)a.D;
    if (kLate) {
      each_piece<kKind, kPieces>(load_weight);
      load_dh(at, r.d);
      each_piece<kKind, kPieces>([&](auto kind, int c) { settle<decltype(kind)::value>(r.d[c], n0 - c * step); });
    }
    each_piece<kKind, kPieces>([&](auto kind, int c) {
      constexpr Kind k = decltype(kind)::value;
      float dv[8], o[8];
      r.dy[c].get(dv);
      grad8(o, dv, r.h[c], w[c], r.d[c], mean, rstd, c1, c2);
      store_bf16<k, true>(a.dx + at + col(c), pack8(o), n0 - c * step);
      if (kDrop) {
        drop8(o, a.drop, key, row, first + c * step);
        store_bf16<k, true>(a.dx_drop + at + col(c), pack8(o), n0 - c * step);
        __builtin_amdgcn_sched_barrier(0);  // one piece's generator at a time
      }
    });
  }
  if (!a.part_dw && !a.part_db) return;
  if (kOneWave) {
    // wave by wave into LDS; a lane only ever touches the places of its own columns
    for (int turn = 0; turn < waves; ++turn) {
      if (wave == turn) {
#pragma unroll
        for (int c = 0; c < kPieces; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float* p = &s_part[2 * (c * 8 + i) * 64 + lane];
            if (turn > 0) dw[c][i] += p[0], db[c][i] += p[64];
            p[0] = dw[c][i], p[64] = db[c][i];
          }
      }
      __syncthreads();
    }
    if (wave != waves - 1) return;
  }
  auto write = [&](float* part, const float (&v)[kPieces][8]) {
    float* out = part + (int64_t)blockIdx.x * a.D + first;
    each_piece<kKind, kPieces>([&](auto kind, int c) {
      const int n = n0 - c * step;
      if (decltype(kind)::value == kFull || n >= 8) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
          *reinterpret_cast<f32x4_a4*>(out + c * step + 4 * k) =
              (f32x4){v[c][4 * k], v[c][4 * k + 1], v[c][4 * k + 2], v[c][4 * k + 3]};
      } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
          if (i < n) out[c * step + i] = v[c][i];
      }
    });
  };
  if (a.part_dw) write(a.part_dw, dw);
  if (a.part_db) write(a.part_db, db);
}

// dw[d] and db[d]: the sums of the partial rows (dw's by the workgroups with
// blockIdx.y 0, db's with 1): 32 columns per workgroup, 32 strips of rows (every
// 32nd), each in row order, and then the strips in pairs, halving their number,
// always the same ones.
constexpr int kSumStrips = 32, kSumCols = 32;  // lines of 128 bytes (16 columns, 64 strips: 16384 x 4096 128 us in place of 125)
struct SumArgs {
  const float* part[2];
  float* out[2];  // null: not wanted
  int parts, D;
};
__global__ __launch_bounds__(kSumCols * kSumStrips) void layer_norm_sum_kernel(const SumArgs a) {
  __shared__ float s[kSumStrips][kSumCols];
  const float* part = a.part[blockIdx.y];
  float* out = a.out[blockIdx.y];
  if (!out) return;
  const int c = threadIdx.x & (kSumCols - 1), strip = threadIdx.x / kSumCols;
  const int col = blockIdx.x * kSumCols + c;
  float sum = 0.0f;
  if (col < a.D) {
#pragma unroll 8
    for (int p = strip; p < a.parts; p += kSumStrips) sum += part[(int64_t)p * a.D + col];
  }
  s[strip][c] = sum;
  __syncthreads();
  for (int half = kSumStrips / 2; half > 0; half >>= 1) {
    if (strip < half) s[strip][c] += s[strip + half][c];
    __syncthreads();
  }
  if (strip == 0 && col < a.D) out[col] = s[0][c];
}

// Rows past 16384 columns, in two launches: a workgroup per row for the two
// sums, then tiles of columns over strips of rows.  4096 x 20000 takes 187 us, 3.5 TB/s
// of what has to be read and written once, with dropout 223; 4096 x 20001 239 and 278.
template <bool kDyF32>
__global__ __launch_bounds__(kWideThreads) void layer_norm_bwd_sums_kernel(const LnBwdArgs a, float* c1c2) {
  __shared__ float s_sum[16];
  const int tid = threadIdx.x, wave = tid >> 6, waves = kWideThreads / 64;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    const float mean = a.mean[row], rstd = a.rstd[row];
    float c1 = 0.0f, c2 = 0.0f;
    for (int col = 8 * tid; col < a.D; col += 8 * kWideThreads) {
      float dy[8], hv[8], wv[8];
      load_grad<kDyF32, kRagged>(dy, a.dy, row * a.D + col, a.D - col);
      unpack(hv, load_bf16<kRagged, false>(a.h + row * a.D + col, a.D - col));
      unpack(wv, load_bf16<kRagged, false>(a.weight + col, a.D - col));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float g = dy[i] * wv[i];
        c1 += g;
        c2 = __builtin_fmaf(g, i < a.D - col ? (hv[i] - mean) * rstd : 0.0f, c2);  // past the row -mean * rstd may overflow
      }
    }
    c1 = group_sum(c1, s_sum, wave, waves), c2 = group_sum(c2, s_sum, wave, waves);
    if (tid == 0) c1c2[2 * row] = c1 / (float)a.D, c1c2[2 * row + 1] = c2 / (float)a.D;
  }
}
constexpr int kTileThreads = 256;
template <bool kDyF32>
__global__ __launch_bounds__(kTileThreads) void layer_norm_bwd_tile_kernel(const LnBwdArgs a, const float* c1c2) {
  const int col = 8 * ((int)blockIdx.x * kTileThreads + (int)threadIdx.x), n = a.D - col;
  if (n <= 0) return;
  DropKey key = {};
  if (a.dx_drop) key = drop_key(a.drop);
  const Piece w = load_bf16<kRagged, false>(a.weight + col, n);
  float dw[8] = {}, db[8] = {};
  for (int64_t row = blockIdx.y; row < a.T; row += gridDim.y) {
    const float mean = a.mean[row], rstd = a.rstd[row];
    float dy[8], hv[8], o[8];
    load_grad<kDyF32, kRagged>(dy, a.dy, row * a.D + col, n);
    const Piece h = load_bf16<kRagged, false>(a.h + row * a.D + col, n);
    const Piece d = a.d_h ? load_bf16<kRagged, false>(a.d_h + row * a.D + col, n) : zero_piece();
    unpack(hv, h);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dw[i] = __builtin_fmaf(dy[i], (hv[i] - mean) * rstd, dw[i]);
      db[i] += dy[i];
    }
    grad8(o, dy, h, w, d, mean, rstd, c1c2[2 * row], c1c2[2 * row + 1]);
    store_bf16<kRagged, true>(a.dx + row * a.D + col, pack8(o), n);
    if (a.dx_drop) {
      drop8(o, a.drop, key, row, col);
      store_bf16<kRagged, true>(a.dx_drop + row * a.D + col, pack8(o), n);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i >= n) continue;
    if (a.part_dw) a.part_dw[(int64_t)blockIdx.y * a.D + col + i] = dw[i];
    if (a.part_db) a.part_db[(int64_t)blockIdx.y * a.D + col + i] = db[i];
  }
}

// ---- the dropout alone ----

struct DropArgs {
  const void* x;
  const uint16_t* residual;  // may be null
  uint16_t* out;             // may be x (bf16) or residual
  int64_t T, first;          // first: the launch's first piece
  int D, pieces;             // pieces: per row
  Dropout drop;
};
// Sixteen values a lane, four counters' words: 16384 x 4096 in 48 us, 5.6 TB/s (with a
// residual 70 us, 5.75); the generator's ten rounds of 32-bit products hide behind the
// memory only since their two exclusive ors are one instruction (52.8 us before).
constexpr int kDropThreads = 256, kDropPieces = 2;  // pieces per lane

template <bool kXF32, Kind kKind>
__global__ __launch_bounds__(kDropThreads) void dropout_add_kernel(const DropArgs a) {
  DropKey key = {};
  if (a.drop.rng) key = drop_key(a.drop);
  // the workgroup's first piece, and from there on in 32 bits
  const int64_t start = a.first + (int64_t)blockIdx.x * (kDropThreads * kDropPieces);
  const int64_t row0 = start / a.pieces;
  const uint32_t piece0 = (uint32_t)(start - row0 * a.pieces);
  int64_t row[kDropPieces], at[kDropPieces];
  int col[kDropPieces];
  float x[kDropPieces][8];
  Piece r[kDropPieces];
#pragma unroll
  for (int c = 0; c < kDropPieces; ++c) {
    const uint32_t p = piece0 + c * kDropThreads + threadIdx.x, down = p / (uint32_t)a.pieces;
    row[c] = row0 + down;
    col[c] = 8 * (int)(p - down * (uint32_t)a.pieces);
    at[c] = row[c] * a.D + col[c];
    if (row[c] < a.T) {
      load_x<kXF32, kKind>(x[c], a.x, at[c], a.D - col[c]);
      if (a.residual) r[c] = load_bf16<kKind, false>(a.residual + at[c], a.D - col[c]);
    }
  }
#pragma unroll
  for (int c = 0; c < kDropPieces; ++c) {
    if (row[c] >= a.T) continue;
    if (a.drop.rng) drop8(x[c], a.drop, key, row[c], col[c]);
    if (a.residual) add(x[c], r[c]);
    store_bf16<kKind, true>(a.out + at[c], pack8(x[c]), a.D - col[c]);
  }
}

constexpr int64_t kMaxD = int64_t(1) << 22, kMaxT = int64_t(1) << 31;
constexpr int64_t kMaxDropped = int64_t(1) << 40;  // elements of dropout_add
constexpr int kRegisterD = 16384;  // rows up to here stay in registers
constexpr int kMaxGrid = 1 << 20;  // workgroups of a launch: the forward kernels walk further rows, the dropout launches again

// Workgroups of the backward pass, each with a partial dw and db row: eight waves
// per CU, and one workgroup per CU at the least.
int bwd_parts(int64_t T, int64_t D) {
  const int64_t waves = D <= 1024 ? 8 : D <= kRegisterD ? (D + 1023) / 1024 : 8;
  return (int)std::min<int64_t>(T, std::max<int64_t>(256, 2048 / waves));
}

template <bool kOneWave, int kPieces>
void launch_norm(const LnArgs& a, bool f32, int waves, hipStream_t stream) {
  const int64_t groups = kOneWave ? (a.T + waves - 1) / waves : a.T;
  const dim3 grid((unsigned)std::min<int64_t>(groups, kMaxGrid)), block(64 * waves);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, a); };
  with_kind<kPieces>(a.D, 512 * kPieces * (kOneWave ? 1 : waves), [&](auto kind) {
    constexpr Kind k = decltype(kind)::value;
    if (f32)
      a.drop.rng ? go(layer_norm_quant_kernel<kOneWave, kPieces, true, k, true>) : go(layer_norm_quant_kernel<kOneWave, kPieces, true, k, false>);
    else
      a.drop.rng ? go(layer_norm_quant_kernel<kOneWave, kPieces, false, k, true>) : go(layer_norm_quant_kernel<kOneWave, kPieces, false, k, false>);
  });
}

template <bool kOneWave, int kPieces, int kThreads>
void launch_bwd(const LnBwdArgs& a, bool f32, int grid, int waves, hipStream_t stream) {
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(grid), dim3(64 * waves), 0, stream, a); };
  with_kind<kPieces>(a.D, 512 * kPieces * (kOneWave ? 1 : waves), [&](auto kind) {
    constexpr Kind k = decltype(kind)::value;
    if (f32)
      a.dx_drop ? go(layer_norm_bwd_kernel<kOneWave, kPieces, kThreads, true, k, true>) : go(layer_norm_bwd_kernel<kOneWave, kPieces, kThreads, true, k, false>);
    else
      a.dx_drop ? go(layer_norm_bwd_kernel<kOneWave, kPieces, kThreads, false, k, true>) : go(layer_norm_bwd_kernel<kOneWave, kPieces, kThreads, false, k, false>);
  });
}

void launch_sum(const SumArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(layer_norm_sum_kernel, dim3((unsigned)((a.D + kSumCols - 1) / kSumCols), 2), dim3(kSumCols * kSumStrips),
                     0, stream, a);
}

int launched() { return hipGetLastError() == hipSuccess ? SILUQUANT_OK : SILUQUANT_ERR_LAUNCH_FAILED; }

}  // namespace

hipError_t code_objects::load_layernorm() { return load(layer_norm_sum_kernel); }

extern "C" {

__attribute__((visibility("default"))) int layer_norm_quant(const void* x, int x_dtype, const void* residual,
                                                            const void* weight, const void* bias, void* y_q, float* y_s,
                                                            void* y_bf16, void* h, float* mean, float* rstd, int64_t T,
                                                            int64_t D, int64_t group, int code_format, float eps, float p,
                                                            const int64_t* rng, int64_t offset, hipStream_t stream) {
  if (group != 32 && group != 64 && group != 128) return SILUQUANT_ERR_BAD_GROUP;
  if (T < 0 || D < 0 || T > kMaxT || D > kMaxD || !(eps >= 0.0f) || eps == __builtin_huge_valf() || !probability(p) ||
      (x_dtype != SILUQUANT_F32 && x_dtype != SILUQUANT_BF16) ||
      (code_format != SILUQUANT_CODE_INT8 && code_format != SILUQUANT_CODE_E4M3))
    return SILUQUANT_ERR_BAD_SHAPE;
  if (T == 0 || D == 0) return SILUQUANT_OK;
  if (p == 0.0f) rng = nullptr;  // not looked at
  if (!x || !weight || (!y_q && !y_bf16) || (y_q == nullptr) != (y_s == nullptr) || (p > 0.0f && !rng))
    return SILUQUANT_ERR_NULL_PTR;
  if (misaligned(x, 16) || misaligned(residual, 16) || misaligned(weight, 16) || misaligned(bias, 16) ||
      misaligned(y_q, 16) || misaligned(y_bf16, 16) || misaligned(h, 16) || misaligned(y_s, 4) || misaligned(mean, 4) ||
      misaligned(rstd, 4) || misaligned(rng, 8))
    return SILUQUANT_ERR_MISALIGNED;
  const bool f32 = x_dtype == SILUQUANT_F32;
  const int64_t groups = (D + group - 1) / group;
  const Span in[5] = {{x, T * D * (f32 ? 4 : 2)}, {residual, 2 * T * D}, {weight, 2 * D}, {bias, 2 * D}, {rng, 16}};
  const Span out[6] = {{y_q, T * D}, {y_s, 4 * T * groups}, {y_bf16, 2 * T * D}, {h, 2 * T * D}, {mean, 4 * T}, {rstd, 4 * T}};
  for (int o = 0; o < 6; ++o) {
    for (int i = 0; i < 5; ++i)
      if (overlap(out[o], in[i]) && !(o == 3 && i == 1 && h == residual)) return SILUQUANT_ERR_OVERLAP;
    for (int i = 0; i < o; ++i)
      if (overlap(out[o], out[i])) return SILUQUANT_ERR_OVERLAP;
  }
  const LnArgs a = {x, static_cast<const uint16_t*>(residual), static_cast<const uint16_t*>(weight),
                    static_cast<const uint16_t*>(bias), static_cast<uint8_t*>(y_q), y_s, static_cast<uint16_t*>(y_bf16),
                    static_cast<uint16_t*>(h), mean, rstd, T, (int)D, group == 32 ? 2 : group == 64 ? 3 : 4, (int)groups,
                    code_format == SILUQUANT_CODE_E4M3, eps, make_dropout(p, rng, offset)};
  if (D > kRegisterD) {
    const dim3 grid((unsigned)std::min<int64_t>(T, kMaxGrid)), block(kWideThreads);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, a); };
    f32 ? go(layer_norm_quant_wide_kernel<true>) : go(layer_norm_quant_wide_kernel<false>);
  } else {
    if (D <= 512) launch_norm<true, 1>(a, f32, 4, stream);
    else if (D <= 1024) launch_norm<true, 2>(a, f32, 4, stream);
    else launch_norm<false, 2>(a, f32, (int)((D + 1023) / 1024), stream);
  }
  return launched();
}

__attribute__((visibility("default"))) int64_t layer_norm_bwd_workspace_bytes(int64_t T, int64_t D) {
  if (T < 0 || D < 0 || T > kMaxT || D > kMaxD) return -1;
  if (T == 0 || D == 0) return 0;
  return 8 * bwd_parts(T, D) * D + (D > kRegisterD ? 8 * T : 0);
}

__attribute__((visibility("default"))) int layer_norm_bwd(const void* dy, int dy_dtype, const void* h, const void* weight,
                                                          const float* mean, const float* rstd, const void* d_h, void* dx,
                                                          void* dx_drop, float* dw, float* db, void* workspace,
                                                          int64_t workspace_bytes, int64_t T, int64_t D, float p,
                                                          const int64_t* rng, int64_t offset, hipStream_t stream) {
  if (T < 0 || D < 0 || T > kMaxT || D > kMaxD || !probability(p) || (dx_drop && p == 0.0f) ||
      (dy_dtype != SILUQUANT_F32 && dy_dtype != SILUQUANT_BF16))
    return SILUQUANT_ERR_BAD_SHAPE;
  if (D == 0) return SILUQUANT_OK;
  const int64_t need = layer_norm_bwd_workspace_bytes(T, D);
  if (T == 0) {  // no rows: no gradient for the weight and the bias
    if (!dw && !db) return SILUQUANT_OK;
    if (misaligned(dw, 4) || misaligned(db, 4)) return SILUQUANT_ERR_MISALIGNED;
    if (overlap({dw, 4 * D}, {db, 4 * D})) return SILUQUANT_ERR_OVERLAP;
    launch_sum({{nullptr, nullptr}, {dw, db}, 0, (int)D}, stream);
    return launched();
  }
  const bool wide = D > kRegisterD, sums = dw || db;
  if (!sums && !wide) workspace = nullptr, workspace_bytes = need;  // not looked at
  if (!dx_drop) rng = nullptr;                                      // neither
  if (!dy || !h || !weight || !mean || !rstd || !dx || ((sums || wide) && !workspace) || (dx_drop && !rng))
    return SILUQUANT_ERR_NULL_PTR;
  if (workspace_bytes < need) return SILUQUANT_ERR_BAD_SHAPE;
  if (misaligned(dy, 16) || misaligned(h, 16) || misaligned(weight, 16) || misaligned(d_h, 16) || misaligned(dx, 16) ||
      misaligned(dx_drop, 16) || misaligned(mean, 4) || misaligned(rstd, 4) || misaligned(dw, 4) || misaligned(db, 4) ||
      misaligned(workspace, 16) || misaligned(rng, 8))
    return SILUQUANT_ERR_MISALIGNED;
  const bool f32 = dy_dtype == SILUQUANT_F32;
  const Span in[7] = {{dy, T * D * (f32 ? 4 : 2)}, {h, 2 * T * D}, {weight, 2 * D}, {mean, 4 * T}, {rstd, 4 * T},
                      {d_h, 2 * T * D}, {rng, 16}};
  const Span out[5] = {{dx, 2 * T * D}, {dx_drop, 2 * T * D}, {dw, 4 * D}, {db, 4 * D}, {workspace, workspace_bytes}};
  for (int o = 0; o < 5; ++o) {
    for (int i = 0; i < 7; ++i)
      if (overlap(out[o], in[i]) && !(o == 0 && i == 5 && dx == d_h)) return SILUQUANT_ERR_OVERLAP;
    for (int i = 0; i < o; ++i)
      if (overlap(out[o], out[i])) return SILUQUANT_ERR_OVERLAP;
  }
  const int parts = bwd_parts(T, D);
  float* ws = static_cast<float*>(workspace);
  float* part_dw = !dw ? nullptr : parts == 1 ? dw : ws;
  float* part_db = !db ? nullptr : parts == 1 ? db : ws + (int64_t)parts * D;
  const LnBwdArgs a = {dy, static_cast<const uint16_t*>(h), static_cast<const uint16_t*>(weight), mean, rstd,
                       static_cast<const uint16_t*>(d_h), static_cast<uint16_t*>(dx), static_cast<uint16_t*>(dx_drop),
                       part_dw, part_db, T, (int)D, make_dropout(p, rng, offset)};
  if (wide) {
    float* c1c2 = ws + 2 * (int64_t)parts * D;
    const dim3 rows_grid((unsigned)std::min<int64_t>(T, kMaxGrid));
    const dim3 tiles((unsigned)((D + 8 * kTileThreads - 1) / (8 * kTileThreads)), (unsigned)parts);
    if (f32) {
      hipLaunchKernelGGL((layer_norm_bwd_sums_kernel<true>), rows_grid, dim3(kWideThreads), 0, stream, a, c1c2);
      hipLaunchKernelGGL((layer_norm_bwd_tile_kernel<true>), tiles, dim3(kTileThreads), 0, stream, a, c1c2);
    } else {
      hipLaunchKernelGGL((layer_norm_bwd_sums_kernel<false>), rows_grid, dim3(kWideThreads), 0, stream, a, c1c2);
      hipLaunchKernelGGL((layer_norm_bwd_tile_kernel<false>), tiles, dim3(kTileThreads), 0, stream, a, c1c2);
    }
  } else {
    const int waves = (int)std::min<int64_t>((T + parts - 1) / parts, 8);
    if (D <= 512) launch_bwd<true, 1, 512>(a, f32, parts, waves, stream);
    else if (D <= 1024) launch_bwd<true, 2, 512>(a, f32, parts, waves, stream);
    else if (D <= 8192) launch_bwd<false, 2, 512>(a, f32, parts, (int)((D + 1023) / 1024), stream);
    else launch_bwd<false, 2, 1024>(a, f32, parts, (int)((D + 1023) / 1024), stream);
  }
  if (sums && parts > 1) launch_sum({{part_dw, part_db}, {dw, db}, parts, (int)D}, stream);
  return launched();
}

__attribute__((visibility("default"))) int dropout_add(const void* x, int x_dtype, const void* residual, void* out,
                                                       int64_t T, int64_t D, float p, const int64_t* rng, int64_t offset,
                                                       hipStream_t stream) {
  if (T < 0 || D < 0 || T > kMaxT || D > kMaxD || T * D > kMaxDropped || !probability(p) ||
      (x_dtype != SILUQUANT_F32 && x_dtype != SILUQUANT_BF16))
    return SILUQUANT_ERR_BAD_SHAPE;
  if (T == 0 || D == 0) return SILUQUANT_OK;
  if (p == 0.0f) rng = nullptr;  // not looked at
  if (!x || !out || (p > 0.0f && !rng)) return SILUQUANT_ERR_NULL_PTR;
  if (misaligned(x, 16) || misaligned(residual, 16) || misaligned(out, 16) || misaligned(rng, 8)) return SILUQUANT_ERR_MISALIGNED;
  const bool f32 = x_dtype == SILUQUANT_F32;
  const Span o = {out, 2 * T * D};
  if ((overlap(o, {x, T * D * (f32 ? 4 : 2)}) && (f32 || x != out)) || (overlap(o, {residual, 2 * T * D}) && residual != out) ||
      overlap(o, {rng, 16}))
    return SILUQUANT_ERR_OVERLAP;
  const int64_t pieces = (D + 7) / 8;
  DropArgs a = {x, static_cast<const uint16_t*>(residual), static_cast<uint16_t*>(out), T, 0, (int)D, (int)pieces,
                make_dropout(p, rng, offset)};
  // A launch has fewer than 2^32 threads.  More of them, each of whole workgroups, cost nothing at that size; a loop
  // over the pieces in the kernel made the ordinary sizes slower (16384 x 11008 125 us, so 121).
  auto go = [&](auto kernel) {
    constexpr int64_t kAtOnce = kDropThreads * kDropPieces;
    for (const int64_t groups = (T * pieces + kAtOnce - 1) / kAtOnce; a.first < T * pieces; a.first += kMaxGrid * kAtOnce) {
      const dim3 grid((unsigned)std::min<int64_t>(groups - a.first / kAtOnce, kMaxGrid));
      hipLaunchKernelGGL(kernel, grid, dim3(kDropThreads), 0, stream, a);
    }
  };
  if (D % 8 == 0)
    f32 ? go(dropout_add_kernel<true, kFull>) : go(dropout_add_kernel<false, kFull>);
  else if (D >= 8)
    f32 ? go(dropout_add_kernel<true, kRagged>) : go(dropout_add_kernel<false, kRagged>);
  else
    f32 ? go(dropout_add_kernel<true, kTiny>) : go(dropout_add_kernel<false, kTiny>);
  return launched();
}

}  // extern "C"
