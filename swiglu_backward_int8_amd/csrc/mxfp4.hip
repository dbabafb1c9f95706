// Microscaled 4-bit codes (OCP MX, MXFP4) of bf16 rows, and the dequantisers
// of every code format of the library, for gfx950.
//
// A block is 32 consecutive values: codes E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and
// their negatives; two to a byte, the first in the low half) and one E8M0
// exponent byte b, the values' common factor 2^(b - 127):
//   b = max(floor(log2(amax)) - 2, -127) + 127   (127 for a block of zeros,
//       255, NaN, for a block that holds an infinity or a NaN)
//   code = E2M1(v * 2^(127 - b)), nearest, ties to the even code, at most 6
// amax is a bf16 number, so floor(log2(amax)) is its exponent field, and the
// hardware's scaled conversions do the rest exactly.
//
// All of it is bound by memory: every element is read once and written once.
// Rows-only quantising and dequantising walk the tensor in pieces of eight
// values per lane (16 bytes of bf16), four independent pieces in flight per
// lane.  Quantising both axes reads x once: a lane holds 32 rows of eight
// columns in registers, so that a column's block lies inside the lane (no
// transpose through LDS) and a row's block inside four neighbouring lanes.
// Measured, over as many sets of tensors as leave the cache nothing of use: rows
// of 16384 x 11008 74 us (6.2 TB/s), dequantised 22016 x 4096 38 us (6.0 TB/s);
// both axes of 8192 x 4096 20 us (5.1 TB/s), of 16384 x 11008 130 us (4.3 TB/s;
// one set over and over, part of which stays in the Infinity Cache, 106), columns
// alone 16 and 92 us.  Of the 20 us reading and computing alone take 15: with all
// of a tile's rows in registers a wave's loads and stores do not overlap.  Rows
// that are not whole lines cost more (8192 x 4104: 29 us), in x and in the codes.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "code_objects.h"
#include "rows.h"
#include "siluquant.h"

namespace {

using namespace rows;

constexpr int kThreads = 256;

// E8M0 byte of a block from its largest magnitude (bf16 bits).
__device__ __forceinline__ uint32_t block_exponent(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 7;
  return e == 255u ? 255u : amax_bits == 0u ? 127u : e > 2u ? e - 2u : 0u;
}
// 2^(b - 127) as fp32 (2^-127 is a subnormal number).
__device__ __forceinline__ float exponent_value(uint32_t b) {
  return __uint_as_float(b == 0u ? 0x00400000u : b << 23);
}

// Eight bf16 values -> eight codes, the first in the low half of the low byte.
__device__ __forceinline__ uint32_t mx_codes8(const Piece& p, float scale) {
  uint32_t q = 0;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, p.w[0]), scale, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, p.w[1]), scale, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, p.w[2]), scale, 2);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, p.w[3]), scale, 3);
  return q;
}
__device__ __forceinline__ Piece mx_values8(uint32_t q, uint32_t b) {
  const float scale = exponent_value(b);
  Piece p;
  p.w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 0));
  p.w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 1));
  p.w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 2));
  p.w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 3));
  if (b == 255u) p = {{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u}};
  return p;
}

// ---- walking rows in pieces of eight columns ----
//
// A flat walk takes the tensor as one run of pieces (rows that are whole
// groups); otherwise 2^lg lanes share a row (as many as it has pieces, 256 at
// most) and a workgroup takes 256 >> lg rows at a time.
struct Where {
  int64_t row, col;
  int n;  // columns of the piece that the row has; 0 and below: a piece of padding
  bool live;
};
struct Walk {
  int64_t rows, pieces;  // per row, padding of the last group included
  int cols, lg;
  int64_t units, col_units;
};

template <class Op, Kind kKind, int kUnroll>
__global__ __launch_bounds__(kThreads) void piece_kernel(const Op op, const Walk k) {
  for (int64_t t = blockIdx.x; t * kUnroll < k.units; t += gridDim.x) {
    Where at[kUnroll];
    typename Op::In in[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t unit = t * kUnroll + u;
      if (kKind == kFull) {
        const int64_t p = unit * kThreads + threadIdx.x;
        at[u] = {0, 8 * p, 8, p < k.pieces};
      } else {
        const int64_t rg = unit / k.col_units;
        const int64_t p = ((unit - rg * k.col_units) << k.lg) + (threadIdx.x & ((1 << k.lg) - 1));
        const int64_t row = rg * (kThreads >> k.lg) + (threadIdx.x >> k.lg);
        at[u] = {row, 8 * p, (int)(k.cols - 8 * p), unit < k.units && row < k.rows && p < k.pieces};
      }
      in[u] = op.template load<kKind>(at[u]);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) op.template finish<kKind>(at[u], in[u]);
  }
}

template <class Op>
void launch_walk(const Op& op, int64_t R, int64_t C, int64_t group, hipStream_t stream) {
  Walk k = {};
  const bool flat = C % group == 0;
  if (flat) {
    k.rows = 1;
    k.pieces = R * C / 8;
    k.units = (k.pieces + kThreads - 1) / kThreads;
  } else {
    k.rows = R;
    k.cols = (int)C;
    k.pieces = (C + group - 1) / group * (group / 8);
    while (k.lg < 8 && (int64_t(1) << k.lg) < k.pieces) ++k.lg;
    k.col_units = (k.pieces + (1 << k.lg) - 1) >> k.lg;
    const int64_t per = kThreads >> k.lg;
    k.units = (R + per - 1) / per * k.col_units;
  }
  const bool many = k.units >= 4096;  // enough for four per thread and still a few workgroups per CU
  const int64_t groups = many ? (k.units + 3) / 4 : k.units;
  const dim3 grid((unsigned)std::min<int64_t>(groups, 1 << 22)), block(kThreads);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, op, k); };
  if (flat)
    many ? go(piece_kernel<Op, kFull, 4>) : go(piece_kernel<Op, kFull, 1>);
  else if (C >= 8)
    many ? go(piece_kernel<Op, kRagged, 4>) : go(piece_kernel<Op, kRagged, 1>);
  else
    many ? go(piece_kernel<Op, kTiny, 4>) : go(piece_kernel<Op, kTiny, 1>);
}

struct MxQuantRows {
  const uint16_t* x;
  uint8_t *q, *s;
  int64_t cols, blocks;  // per row
  using In = Piece;
  template <Kind kKind>
  __device__ __forceinline__ In load(const Where& a) const {
    return a.live ? load_bf16<kKind, true>(x + a.row * cols + a.col, a.n) : zero_piece();
  }
  template <Kind kKind>
  __device__ __forceinline__ void finish(const Where& a, const In& p) const {
    const uint32_t b = block_exponent(group_amax_bits<false>(p, 4));
    const uint32_t c = mx_codes8(p, exponent_value(b));
    if (a.live) {
      const int64_t piece = a.row * blocks * 4 + (a.col >> 3);
      __builtin_nontemporal_store(c, reinterpret_cast<uint32_t*>(q) + piece);
      if ((threadIdx.x & 3) == 0) s[piece >> 2] = (uint8_t)b;
    }
  }
};

struct MxDequantRows {
  const uint8_t *q, *s;
  uint16_t* out;
  int64_t cols, blocks;
  struct In {
    uint32_t c, b;
  };
  template <Kind kKind>
  __device__ __forceinline__ In load(const Where& a) const {
    In in = {0, 127};
    if (a.live) {
      const int64_t piece = a.row * blocks * 4 + (a.col >> 3);
      in.c = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(q) + piece);
      in.b = s[piece >> 2];
    }
    return in;
  }
  template <Kind kKind>
  __device__ __forceinline__ void finish(const Where& a, const In& in) const {
    if (a.live) store_bf16<kKind, true>(out + a.row * cols + a.col, mx_values8(in.c, in.b), a.n);
  }
};

template <bool kE4M3>
struct GroupDequant {
  const uint8_t* q;
  const float* s;
  uint16_t* out;
  int64_t cols, groups;
  int lg_group;  // log2 of the group's pieces
  struct In {
    uint32_t c[2];
    float s;
  };
  template <Kind kKind>
  __device__ __forceinline__ In load(const Where& a) const {
    In in = {{0, 0}, 0.0f};
    if (a.live && (kKind == kFull || a.n > 0)) {
      const uint8_t* p = q + a.row * cols + a.col;
      if (kKind == kFull || a.n >= 8) {
        const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x2_a1*>(p));
        in.c[0] = v.x, in.c[1] = v.y;
      } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
          if (i < a.n) in.c[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
      }
      in.s = s[a.row * groups + (a.col >> (3 + lg_group))];
    }
    return in;
  }
  template <Kind kKind>
  __device__ __forceinline__ void finish(const Where& a, const In& in) const {
    float v[8];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t c = in.c[k];
      if (kE4M3) {
        v[4 * k] = __builtin_amdgcn_cvt_f32_fp8(c, 0), v[4 * k + 1] = __builtin_amdgcn_cvt_f32_fp8(c, 1);
        v[4 * k + 2] = __builtin_amdgcn_cvt_f32_fp8(c, 2), v[4 * k + 3] = __builtin_amdgcn_cvt_f32_fp8(c, 3);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * k + i] = (float)(int8_t)(c >> (8 * i));
      }
    }
    Piece p;
#pragma unroll
    for (int i = 0; i < 4; ++i) p.w[i] = pack_bf16(v[2 * i] * in.s, v[2 * i + 1] * in.s);
    if (a.live) store_bf16<kKind, true>(out + a.row * cols + a.col, p, a.n);
  }
};

// ---- both axes in one read ----

typedef uint32_t u32_a1 __attribute__((aligned(1)));

struct BothArgs {
  const uint16_t* x;
  uint8_t *q, *s, *q_t, *s_t;  // q and s may be null together: columns only
  int64_t R;
  int K, blocks_k;
  int64_t blocks_r;
};

// A wave takes 128 rows x 128 columns, a workgroup kSide x kSide of those: lane
// (b, p) = (lane / 16, lane % 16) holds rows 32 b .. + 31 of columns 8 p .. + 7,
// so that a load covers 256 bytes of four rows and four neighbouring column
// blocks leave as 64 contiguous bytes.  Two waves side by side and two below
// each other write whole 128-byte lines of both kinds of codes (16384 x 11008,
// one set over and over: 103 us; four below each other 109, side by side 112).  The exponents meet in
// LDS, from where a thread stores all that a tile has of a column or of a row
// (stored from the lanes, a byte each, the columns' cost a fifth of the time and
// the rows' another 5 us).  Each XCD takes whole bands of rows, so that the lines
// that two neighbouring workgroups share are put together in its L2.
//
// Tiles inside the tensor need no care for its edges; kEdge is the kind of those
// that reach past its rows or columns (kFull: there are none).
template <Kind kEdge, int kSide>
__global__ __launch_bounds__(64 * kSide * kSide) void mx_quant_both_kernel(const BothArgs a, int64_t tiles,
                                                                           int64_t per_xcd, int tiles_k) {
  constexpr int kThreads = 64 * kSide * kSide, kRows = 128 * kSide, kCols = 128 * kSide, kBlocks = 4 * kSide;
  // exponents of a tile: a column's and a row's
  using Exps = std::conditional_t<kSide == 2, u32x2_a1, u32_a1>;
  static_assert(sizeof(Exps) == kBlocks, "one store");
  __shared__ __attribute__((aligned(16))) uint8_t s_col[kCols][kBlocks], s_row[kRows][kBlocks];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int blk = 4 * (wave / kSide) + (lane >> 4), col_in = 128 * (wave % kSide) + 8 * (lane & 15);

  // the wave's part of the tile at (row0, col0)
  auto part = [&](auto kind, int64_t row0, int col0) {
    constexpr Kind kKind = decltype(kind)::value;
    // streamed where rows are whole pieces of 16 bytes; others share pieces,
    // which have to stay in L2 (3000 x 4100: 21 us streamed, 16 cached; 8192 x
    // 4096: 20 us and 25).  Widths of a multiple of 8 but not of 64 share lines,
    // not pieces, and are streamed too (8192 x 4104: 29 us; not timed cached).
    constexpr bool kNt = kEdge <= kWhole;
    const int col = col0 + col_in, n = a.K - col;
    const bool in_block = col < 32 * a.blocks_k;  // the same for four neighbouring lanes
    const int64_t r0 = row0 + 32 * blk;
    const int rows_here = (int)(a.R - r0 < 32 ? (a.R - r0 > 0 ? a.R - r0 : 0) : 32);
    Piece x[32];
    const uint16_t* from = a.x + r0 * a.K + col;
    if (kKind == kFull) {
#pragma unroll
      for (int r = 0; r < 32; ++r) x[r] = load_bf16<kFull, kNt>(from + r * (int64_t)a.K, 8);
    } else if (kKind == kTiny) {
#pragma unroll
      for (int r = 0; r < 32; ++r) x[r] = r < rows_here ? load_bf16<kTiny, kNt>(from + r * (int64_t)a.K, n) : zero_piece();
    } else {
      // Whole pieces everywhere, and what is not the tensor's is taken out of
      // them: a branch for each row would load them one by one.  A piece past
      // the row's columns is read as the row's last one, one that the row's end
      // cuts runs on into the next row, and a row that has no next one, or is
      // past the last, is read as the one before it.
      const int d = n < 8 ? 8 - n : 0;
      const bool ends = kKind == kRagged && d > 0 && a.R - r0 <= 32;  // in the last row
      int last = rows_here - 1 - (ends && n > 0);
      const uint16_t* at = from;
      if (n <= 0 || last < 0) at -= d;
      if (rows_here <= 0) at = a.x;
#pragma unroll
      for (int r = 0; r < 32; ++r) {
        x[r] = load_bf16<kFull, kNt>(at, 8);
        if (r < last) at += a.K;
      }
      if (kKind == kRagged && row0 + kRows >= a.R) {
        const int last_row = (int)((a.R - 1) & 31);  // the tensor's last row, in its block
        Piece end = zero_piece();
        if (ends && rows_here > 0) end = load_bf16<kRagged, kNt>(from + last_row * (int64_t)a.K, n);
#pragma unroll
        for (int r = 0; r < 32; ++r)
          if (r == last_row && ends) x[r] = end;
      }
      if (row0 + kRows > a.R) {
#pragma unroll
        for (int r = 0; r < 32; ++r)
          if (r >= rows_here) x[r] = zero_piece();
      }
      if (col0 + kCols > a.K) {
        uint32_t keep[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) keep[k] = n > 2 * k + 1 ? ~0u : n == 2 * k + 1 ? 0xffffu : 0u;
#pragma unroll
        for (int r = 0; r < 32; ++r)
#pragma unroll
          for (int k = 0; k < 4; ++k) x[r].w[k] &= keep[k];
      }
    }
    // Rows past the last lie past the record count, and lanes past the blocks too.
    // All of the offset is the vector register's: the check need not count a scalar's.
    const int row_bytes = 16 * a.blocks_k;
    const auto to_q = __builtin_amdgcn_make_buffer_rsrc(a.q + row0 * row_bytes, 0, (int)(std::min<int64_t>(a.R - row0, kRows) * row_bytes), 0x20000);
    const uint32_t at_q = (uint32_t)(32 * blk * row_bytes + (col >> 1)) | (in_block ? 0 : 0x80000000u);
    if (a.q) {
#pragma unroll
      for (int r4 = 0; r4 < 8; ++r4) {
        uint32_t keep = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = 4 * r4 + j;
          const uint32_t b = block_exponent(group_amax_bits<false>(x[r], 4));
          const uint32_t c = mx_codes8(x[r], exponent_value(b));
          if (kKind == kFull)
            reinterpret_cast<uint32_t*>(a.q)[(r0 + r) * (4 * (int64_t)a.blocks_k) + (col >> 3)] = c;
          else
            __builtin_amdgcn_raw_buffer_store_b32(c, to_q, at_q + (uint32_t)(r * row_bytes), 0, 0);
          keep = (lane & 3) == j ? b : keep;
        }
        s_row[32 * blk + 4 * r4 + (lane & 3)][col_in >> 5] = (uint8_t)keep;
      }
    }
    // without this the magnitudes that the rows' maxima took would be kept for
    // the columns', in as many registers as x has (a wave per SIMD instead of two or three)
#pragma unroll
    for (int r = 0; r < 32; ++r) asm volatile("" : "+v"(x[r].w[0]), "+v"(x[r].w[1]), "+v"(x[r].w[2]), "+v"(x[r].w[3]));
#pragma unroll
    for (int h = 0; h < 4; ++h) {  // columns 2h and 2h + 1 of the lane
      uint32_t m = x[0].w[h] & 0x7fff7fffu;
#pragma unroll
      for (int r = 1; r < 32; ++r) m = max_u16(m, x[r].w[h] & 0x7fff7fffu);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t b = block_exponent(half ? m >> 16 : m & 0xffffu);
        const float scale = exponent_value(b);
        u32x4 codes;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          Piece p;
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const int r = 8 * k + 2 * t;
            p.w[t] = __builtin_amdgcn_perm(x[r + 1].w[h], x[r].w[h], half ? 0x07060302u : 0x05040100u);
          }
          codes[k] = mx_codes8(p, scale);
        }
        const int c = 2 * h + half;
        if (kKind == kFull || (c < n && rows_here > 0))
          *reinterpret_cast<u32x4*>(a.q_t + ((int64_t)(col + c) * a.blocks_r + (row0 >> 5) + blk) * 16) = codes;
        s_col[col_in + c][blk] = (uint8_t)b;
      }
    }
  };

  for (int64_t i = blockIdx.x >> 3; i < per_xcd; i += gridDim.x >> 3) {
    const int64_t tile = (blockIdx.x & 7) * per_xcd + i;
    if (tile >= tiles) break;
    const int64_t band = tile / tiles_k, row0 = band * kRows, rows = a.R - row0;
    const int col0 = (int)(tile - band * tiles_k) * kCols, cols = a.K - col0;
    const bool inside = kEdge == kFull || (kEdge != kTiny && rows >= kRows && cols >= kCols);
    if (inside) {
      if constexpr (kEdge != kTiny) part(std::integral_constant<Kind, kFull>{}, row0, col0);
    } else if constexpr (kEdge != kFull) {
      if (32 * (blk & ~3) < rows && 128 * (wave % kSide) < cols) part(std::integral_constant<Kind, kEdge>{}, row0, col0);
    }
    __syncthreads();
    auto store = [&](uint8_t* to, const uint8_t* from, int64_t n) {
      if (inside || n >= kBlocks) {
        *reinterpret_cast<Exps*>(to) = *reinterpret_cast<const Exps*>(from);
      } else {
        for (int k = 0; k < (int)n; ++k) to[k] = from[k];
      }
    };
#pragma unroll
    for (int c = threadIdx.x; c < kCols; c += kThreads)
      if (inside || c < cols)
        store(a.s_t + (int64_t)(col0 + c) * a.blocks_r + (row0 >> 5), s_col[c], a.blocks_r - (row0 >> 5));
    if (a.q) {
#pragma unroll
      for (int r = threadIdx.x; r < kRows; r += kThreads)
        if (inside || r < rows) store(a.s + (row0 + r) * a.blocks_k + (col0 >> 5), s_row[r], a.blocks_k - (col0 >> 5));
    }
    __syncthreads();
  }
}

constexpr int64_t kMaxCols = int64_t(1) << 22, kMaxRows = int64_t(1) << 31;

}  // namespace

hipError_t code_objects::load_mxfp4() { return load(piece_kernel<MxQuantRows, kFull, 1>); }

extern "C" {

__attribute__((visibility("default"))) int mxfp4_quant(const void* x, void* q, void* s, void* q_t, void* s_t, int64_t R,
                                                       int64_t K, hipStream_t stream) {
  if (R < 0 || K < 0 || R > kMaxRows || K > kMaxCols) return SILUQUANT_ERR_BAD_SHAPE;
  if (R == 0 || K == 0) return SILUQUANT_OK;
  if (!x || (!q && !q_t) || (q == nullptr) != (s == nullptr) || (q_t == nullptr) != (s_t == nullptr))
    return SILUQUANT_ERR_NULL_PTR;
  if (misaligned(x, 16) || misaligned(q, 16) || misaligned(q_t, 16)) return SILUQUANT_ERR_MISALIGNED;
  const int64_t bk = (K + 31) / 32, br = (R + 31) / 32;
  const Span all[5] = {{x, 2 * R * K}, {q, 16 * R * bk}, {s, R * bk}, {q_t, 16 * K * br}, {s_t, K * br}};
  for (int i = 1; i < 5; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(all[i], all[j])) return SILUQUANT_ERR_OVERLAP;
  const uint16_t* xb = static_cast<const uint16_t*>(x);
  uint8_t *qb = static_cast<uint8_t*>(q), *sb = static_cast<uint8_t*>(s);
  if (!q_t) {
    launch_walk(MxQuantRows{xb, qb, sb, K, bk}, R, K, 32, stream);
  } else {
    const BothArgs a = {xb, qb, sb, static_cast<uint8_t*>(q_t), static_cast<uint8_t*>(s_t), R, (int)K, (int)bk, br};
    auto launch = [&](auto side) {
      constexpr int kSide = decltype(side)::value, kTile = 128 * kSide;
      const int64_t tiles_k = (K + kTile - 1) / kTile;
      const int64_t tiles = (R + kTile - 1) / kTile * tiles_k, per_xcd = (tiles + 7) / 8;
      const dim3 grid((unsigned)(8 * std::min<int64_t>(per_xcd, 1 << 19)));
      auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(64 * kSide * kSide), 0, stream, a, tiles, per_xcd, (int)tiles_k);
      };
      if (K % kTile == 0 && R % kTile == 0)
        go(mx_quant_both_kernel<kFull, kSide>);
      else if (K % 8 == 0)
        go(mx_quant_both_kernel<kWhole, kSide>);
      else
        K > 8 ? go(mx_quant_both_kernel<kRagged, kSide>) : go(mx_quant_both_kernel<kTiny, kSide>);
    };
    // tiles of 256 x 256 where they give three CUs of four one (3000 x 4096: 13.4
    // us, of 128 x 128 13.5; 8192 x 4096: 20.1 and 22.1), of 128 x 128 otherwise
    // (1024 x 4096: 7.9 us, of 256 x 256 9.3)
    if ((R + 255) / 256 * ((K + 255) / 256) >= 192)
      launch(std::integral_constant<int, 2>{});
    else
      launch(std::integral_constant<int, 1>{});
  }
  return hipGetLastError() == hipSuccess ? SILUQUANT_OK : SILUQUANT_ERR_LAUNCH_FAILED;
}

__attribute__((visibility("default"))) int mxfp4_dequant(const void* q, const void* s, void* out, int64_t R, int64_t K,
                                                         hipStream_t stream) {
  if (R < 0 || K < 0 || R > kMaxRows || K > kMaxCols) return SILUQUANT_ERR_BAD_SHAPE;
  if (R == 0 || K == 0) return SILUQUANT_OK;
  if (!q || !s || !out) return SILUQUANT_ERR_NULL_PTR;
  if (misaligned(q, 16) || misaligned(out, 16)) return SILUQUANT_ERR_MISALIGNED;
  const int64_t bk = (K + 31) / 32;
  const Span o = {out, 2 * R * K};
  if (overlap(o, {q, 16 * R * bk}) || overlap(o, {s, R * bk})) return SILUQUANT_ERR_OVERLAP;
  launch_walk(MxDequantRows{static_cast<const uint8_t*>(q), static_cast<const uint8_t*>(s), static_cast<uint16_t*>(out), K, bk},
              R, K, 32, stream);
  return hipGetLastError() == hipSuccess ? SILUQUANT_OK : SILUQUANT_ERR_LAUNCH_FAILED;
}

__attribute__((visibility("default"))) int group_dequant(const void* q, const float* s, void* out, int64_t R, int64_t K,
                                                         int64_t group, int code_format, hipStream_t stream) {
  if (group != 32 && group != 64 && group != 128) return SILUQUANT_ERR_BAD_GROUP;
  if (R < 0 || K < 0 || R > kMaxRows || K > (int64_t(1) << 23) ||
      (code_format != SILUQUANT_CODE_INT8 && code_format != SILUQUANT_CODE_E4M3))
    return SILUQUANT_ERR_BAD_SHAPE;
  if (R == 0 || K == 0) return SILUQUANT_OK;
  if (!q || !s || !out) return SILUQUANT_ERR_NULL_PTR;
  if (misaligned(q, 16) || misaligned(s, 4) || misaligned(out, 16)) return SILUQUANT_ERR_MISALIGNED;
  const int64_t groups = (K + group - 1) / group;
  const Span o = {out, 2 * R * K};
  if (overlap(o, {q, R * K}) || overlap(o, {s, 4 * R * groups})) return SILUQUANT_ERR_OVERLAP;
  const int lg = group == 32 ? 2 : group == 64 ? 3 : 4;
  const uint8_t* qb = static_cast<const uint8_t*>(q);
  uint16_t* ob = static_cast<uint16_t*>(out);
  if (code_format == SILUQUANT_CODE_E4M3)
    launch_walk(GroupDequant<true>{qb, s, ob, K, groups, lg}, R, K, group, stream);
  else
    launch_walk(GroupDequant<false>{qb, s, ob, K, groups, lg}, R, K, group, stream);
  return hipGetLastError() == hipSuccess ? SILUQUANT_OK : SILUQUANT_ERR_LAUNCH_FAILED;
}

}  // extern "C"
