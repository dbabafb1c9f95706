// Product of two microscaled 4-bit operands on the CDNA4 matrix cores (gfx950):
//
//   C[m, n] = sum over blocks k of 2^(sA[m, k] - 127) * 2^(sB[n, k] - 127) *
//             (A[m, block k] . B[n, block k])
//
// A [M, K/2] and B [N, K/2] hold E2M1 codes row-major (C = A . B^T), sA and sB
// an E8M0 byte per 32 of them.  The scaled matrix instructions take both
// directly: a lane's operand is 32 codes (16 bytes) of one row, that is one
// block, and its exponent byte one of the four in a register, chosen by the
// instruction.  Sums are fp32; the products of two codes and their exponents
// are exact.
//
// The order of the blocks within a sum is free, as long as A and B agree.  So
// a lane takes four neighbouring blocks of its row for four successive
// instructions: its codes are 64 contiguous bytes and its four exponents one
// 32-bit word.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "code_objects.h"
#include "rows.h"
#include "siluquant.h"

namespace {

using namespace rows;

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
typedef uint32_t u32_a1 __attribute__((aligned(1)));

constexpr int kFp4 = 4;  // the operand format field of the scaled matrix instructions

template <int kByte>
__device__ __forceinline__ f32x4 mfma16(const u32x4& a, uint32_t sa, const u32x4& b, uint32_t sb, const f32x4& c) {
  const i32x8 wa = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8 wb = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wa, wb, c, kFp4, kFp4, kByte, (int)sa, kByte, (int)sb);
}

struct GemmArgs {
  const uint8_t *A, *sA, *B, *sB;
  void* C;
  int64_t M, N;
  int blocks;  // K / 32
  int tiles_m, tiles_n;
};

// Whether every row's exponents start on 4 bytes, in both operands.
bool words(const GemmArgs& a) { return a.blocks % 4 == 0 && !misaligned(a.sA, 4) && !misaligned(a.sB, 4); }

// Four consecutive columns of a row of C; `left` of them exist.
template <bool kBf16Out>
__device__ __forceinline__ void store4(void* C, int64_t at, const f32x4& v, int64_t left) {
  if constexpr (kBf16Out) {
    uint16_t* p = static_cast<uint16_t*>(C) + at;
    const u32x2 w = {pack_bf16(v.x, v.y), pack_bf16(v.z, v.w)};
    if (left >= 4) {
      *reinterpret_cast<u32x2_a2*>(p) = w;
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < left) p[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
  } else {
    float* p = static_cast<float*>(C) + at;
    if (left >= 4) {
      *reinterpret_cast<f32x4_a4*>(p) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < left) p[i] = v[i];
    }
  }
}

// A 16-byte chunk of a row of C, `left` columns of which exist at the least.
template <bool kBf16Out>
__device__ __forceinline__ void store_chunk(void* C, int64_t at, const u32x4& v, int64_t left) {
  if constexpr (kBf16Out) {
    uint16_t* p = static_cast<uint16_t*>(C) + at;
    if (left >= 8) {
      *reinterpret_cast<u32x4_a2*>(p) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (i < left) p[i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
    }
  } else {
    uint32_t* p = static_cast<uint32_t*>(C) + at;
    if (left >= 4) {
      *reinterpret_cast<u32x4_a4*>(p) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < left) p[i] = v[i];
    }
  }
}

// ---- few rows: operands straight from memory into registers ----
//
// A workgroup owns 16 kM rows of A by 16 kN rows of B; its kW waves split K in
// chunks of 16 blocks (512 values) and their sums meet in LDS.  Nothing is
// shared between waves, so nothing waits: the weight streams through once.
// Rows past M or N are read as the last row and not stored.  Bound by memory: 1 x
// 22016 x 4096 takes 11 us for 48 MB (4.4 TB/s, the launch included).
constexpr int kChunkBlocks = 16;

struct Frag {
  u32x4 c[4];
  uint32_t s;
};
// Lane (row, kb = lane / 16) of a chunk: blocks 4 kb .. 4 kb + 3 of it.
__device__ __forceinline__ Frag load_frag(const uint8_t* codes, const uint8_t* scales, int64_t row, int blocks,
                                          int chunk, int kb) {
  const int b = chunk * kChunkBlocks + 4 * kb;
  const uint8_t* p = codes + (row * blocks + b) * 16;
  const uint8_t* q = scales + row * blocks + b;
  Frag f;
  if (chunk * kChunkBlocks + kChunkBlocks <= blocks) {
#pragma unroll
    for (int j = 0; j < 4; ++j) f.c[j] = *reinterpret_cast<const u32x4*>(p + 16 * j);
    f.s = *reinterpret_cast<const u32_a1*>(q);
  } else {  // the chunk in which K ends: blocks past it are zeros
    f.s = 0x7f7f7f7fu;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f.c[j] = (u32x4){0, 0, 0, 0};
      if (b + j < blocks) {
        f.c[j] = *reinterpret_cast<const u32x4*>(p + 16 * j);
        f.s = (f.s & ~(0xffu << (8 * j))) | (uint32_t)q[j] << (8 * j);
      }
    }
  }
  return f;
}

template <int kM, int kN, int kW, bool kBf16Out>
__global__ __launch_bounds__(64 * kW) void mx_gemm_stream_kernel(const GemmArgs a) {
  __shared__ f32x4 s_sum[kW > 1 ? kW - 1 : 1][kM * kN][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, kb = lane >> 4;
  for (int64_t tile = blockIdx.x; tile < (int64_t)a.tiles_m * a.tiles_n; tile += gridDim.x) {
    const int tm = (int)(tile / a.tiles_n), tn = (int)(tile - (int64_t)tm * a.tiles_n);
    int64_t row_a[kM], row_b[kN];
#pragma unroll
    for (int i = 0; i < kM; ++i) {
      const int64_t m = ((int64_t)tm * kM + i) * 16 + r;
      row_a[i] = m < a.M ? m : a.M - 1;
    }
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const int64_t n = ((int64_t)tn * kN + j) * 16 + r;
      row_b[j] = n < a.N ? n : a.N - 1;
    }
    // The B rows come first in the instruction, so that a lane holds four
    // consecutive columns of C: D[row 4 kb + i][column r] = C[m = r][n = 4 kb + i].
    f32x4 acc[kM][kN];
#pragma unroll
    for (int i = 0; i < kM; ++i)
#pragma unroll
      for (int j = 0; j < kN; ++j) acc[i][j] = (f32x4){0, 0, 0, 0};
    const int chunks = (a.blocks + kChunkBlocks - 1) / kChunkBlocks;
    for (int c = wave; c < chunks; c += kW) {
      Frag fa[kM], fb[kN];
#pragma unroll
      for (int j = 0; j < kN; ++j) fb[j] = load_frag(a.B, a.sB, row_b[j], a.blocks, c, kb);
#pragma unroll
      for (int i = 0; i < kM; ++i) fa[i] = load_frag(a.A, a.sA, row_a[i], a.blocks, c, kb);
#pragma unroll
      for (int i = 0; i < kM; ++i)
#pragma unroll
        for (int j = 0; j < kN; ++j) {
          acc[i][j] = mfma16<0>(fb[j].c[0], fb[j].s, fa[i].c[0], fa[i].s, acc[i][j]);
          acc[i][j] = mfma16<1>(fb[j].c[1], fb[j].s, fa[i].c[1], fa[i].s, acc[i][j]);
          acc[i][j] = mfma16<2>(fb[j].c[2], fb[j].s, fa[i].c[2], fa[i].s, acc[i][j]);
          acc[i][j] = mfma16<3>(fb[j].c[3], fb[j].s, fa[i].c[3], fa[i].s, acc[i][j]);
        }
    }
    if (kW > 1 && wave > 0) {
#pragma unroll
      for (int i = 0; i < kM; ++i)
#pragma unroll
        for (int j = 0; j < kN; ++j) s_sum[wave - 1][i * kN + j][lane] = acc[i][j];
    }
    __syncthreads();
    if (wave == 0) {
#pragma unroll
      for (int i = 0; i < kM; ++i) {
        const int64_t m = ((int64_t)tm * kM + i) * 16 + r;
#pragma unroll
        for (int j = 0; j < kN; ++j) {
          for (int w = 0; w < kW - 1; ++w) acc[i][j] += s_sum[w][i * kN + j][lane];
          const int64_t n = ((int64_t)tn * kN + j) * 16 + 4 * kb;
          if (m < a.M && n < a.N) store4<kBf16Out>(a.C, m * a.N + n, acc[i][j], a.N - n);
        }
      }
    }
    __syncthreads();
  }
}

// ---- many rows: tiles through LDS ----
//
// A workgroup owns a tile of kTileA x kTileB results, its waves (2 x kWavesB)
// kFA x kFB blocks of 32 x 32 each.  A stage is 256 values (8 blocks, 128
// bytes) of every row of the tile: the codes go from memory straight into LDS
// (buffer loads with the lds flag), double buffered.  Rows of 128 bytes lie in
// LDS as eight 16-byte chunks, chunk c of row r at c ^ swz(r), so that the 16
// lanes that read a chunk of consecutive rows fall on distinct banks.
//
// Bound by the matrix cores' power: multiplying random codes from registers
// alone, nothing else running, they reach 6.6 PFLOP/s at a lowered clock (9.4
// with zeros).  256 x 256 tiles of 128 x 128 per wave, the most that fits the
// registers, read LDS for half of the cycles and L2 for a third.  16384 x 4096 x
// 11008: 311 to 330 us, 4.5 to 4.75 PFLOP/s; 16384 x 22016 x 4096: 690 to 710 us, 4.2 to 4.3.
// A stage of 2048 matrix cycles takes 2900; a tile's end (results out through
// LDS, next tile's start) as long as three stages, half of it the stores' way to
// memory (without any stores 640 us).  Loads not spread over two steps, larger
// or smaller rasters, eight waves of 128 x 64, patches outside the buffers, so
// that the second stage's loads need not follow the stores, and workgroups
// started out of step all measured slower or the same.
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kStageBlocks = 8;                 // per row and stage
constexpr int kRowBytes = 16 * kStageBlocks;    // 128
constexpr int kRasterRows = 4;                  // tile rows that are walked column by column together

__device__ __forceinline__ int swz(int r) { return (r ^ (r >> 3)) & 7; }

// Buffer resource words: base, 32-bit record count (loads at or past it read
// as zeros), raw addressing.
__device__ __forceinline__ i32x4 rsrc_words(const void* base, int bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  return (i32x4){__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
                 __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32) & 0xFFFF),
                 __builtin_amdgcn_readfirstlane(bytes), 0x00020000};
}

// Each lane reads 16 bytes at voff + soff (voff is checked against the record
// count, each 4 bytes for themselves); the wave writes them, lane by lane, to
// consecutive LDS bytes from address lds (M0) on.  Written as asm so that the
// compiler does not wait for them before every LDS read; the kernel waits
// itself.  The leading s_nop gives the wait states that the compiler cannot,
// since it does not look inside: one between the write of M0 and its use; and,
// with kSlow, five between a vector instruction's write of a scalar register
// (a scalar that was spilled to lanes comes back that way) and a load that
// reads it.  In the main loop the scalars stay in their registers, which the
// instruction checks of the tests hold it to, and 20 cycles a load would show.
template <bool kSlow>
__device__ __forceinline__ void lds_load16(i32x4 rs, uint32_t lds, uint32_t voff, uint32_t soff) {
  if (kSlow)
    asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
                 :
                 : "v"(voff), "s"(rs), "s"(__builtin_amdgcn_readfirstlane(soff)),
                   "{m0}"(__builtin_amdgcn_readfirstlane(lds))
                 : "memory");
  else
    asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
                 :
                 : "v"(voff), "s"(rs), "s"(__builtin_amdgcn_readfirstlane(soff)),
                   "{m0}"(__builtin_amdgcn_readfirstlane(lds))
                 : "memory");
}

__device__ __forceinline__ void lds_load4(i32x4 rs, uint32_t lds, uint32_t voff) {
  asm volatile("s_nop 4\n\tbuffer_load_dword %0, %1, 0 offen lds"
               :
               : "v"(voff), "s"(rs), "{m0}"(__builtin_amdgcn_readfirstlane(lds))
               : "memory");
}

template <int kByte>
__device__ __forceinline__ f32x16 mfma32(const u32x4& a, uint32_t sa, const u32x4& b, uint32_t sb, const f32x16& c) {
  const i32x8 wa = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8 wb = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wa, wb, c, kFp4, kFp4, kByte, (int)sa, kByte, (int)sb);
}

// kWords: rows of exponents start on 4 bytes (K is a multiple of 128, in aligned buffers).  They
// then go into LDS too, 32 blocks of every row at a time, a quarter of the next
// 32 with each stage: read from memory by every wave in every stage, 4 bytes a
// row, they doubled the requests to L2 and cost a quarter of the time.  Exponents
// of any other K, or off 4 bytes, are still read that way: 16384 x 22016 x 4064
// takes 932 us (4096: 690; 4096 off 4 bytes: 868), 4096 x 4096 x 4064 46 us (36).
//
// Workgroups are persistent (one per CU for 256 x 256, two for 128 x 128, or one
// with four buffers, whose loads are three stages ahead): the
// next tile's first stage is asked for before the present one's results are
// stored, and the stores drain behind its first stage.
template <int kFA, int kFB, int kWavesB, int kBufs>
struct TileShape {
  static constexpr int kWaves = 2 * kWavesB, kThreads = 64 * kWaves;
  static constexpr int kTileA = 64 * kFA, kTileB = 32 * kWavesB * kFB;  // rows of A and of B
  static constexpr int kPerCu = kFA * kFB * kWavesB * kBufs > 16 ? 1 : 2;  // workgroups that fit a CU's LDS
};
template <int kFA, int kFB, int kWavesB, int kBufs, bool kWords, bool kBf16Out>
__global__ __launch_bounds__(128 * kWavesB, (kFA * kFB * kWavesB * kBufs > 16 ? 1 : 2) * kWavesB / 2) void
mx_gemm_tile_kernel(const GemmArgs a, int per_xcd) {
  static_assert(kBufs == 2 || (kBufs == 4 && kWords), "exponents in registers are waited for with everything else");
  using Shape = TileShape<kFA, kFB, kWavesB, kBufs>;
  constexpr int kWaves = Shape::kWaves, kTileA = Shape::kTileA, kTileB = Shape::kTileB;
  constexpr int kStage = (kTileA + kTileB) * kRowBytes;     // A's rows, then B's
  constexpr int kLoadsA = kTileA / 8 / kWaves, kLoadsB = kTileB / 8 / kWaves;  // wave-wide loads per stage: 8 rows each
  constexpr int kLoads = kLoadsA + kLoadsB;
  constexpr int kSpanBytes = 32;                            // exponents of a row that are loaded together: four stages
  constexpr int kSpan = (kTileA + kTileB) * kSpanBytes;
  constexpr int kSpanLoads = (kTileA + kTileB) / 32;        // 32 rows each
  constexpr int kSpanPerWave = kSpanLoads / kWaves;         // of a span, one a stage
  // spans are loaded one span ahead into the other of two buffers; with more
  // stages on their way than the waits ask for, two ahead into four
  constexpr int kSpanBufs = kBufs, kSpansAhead = kBufs / 2;
  __shared__ __attribute__((aligned(16))) char s_tile[kBufs * kStage + (kWords ? kSpanBufs * kSpan : 0)];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = (wave / kWavesB) * 32 * kFA, wn = (wave % kWavesB) * 32 * kFB;
  const int lrow = lane & 31, half = lane >> 5;
  const int stages = (a.blocks + kStageBlocks - 1) / kStageBlocks;
  const int64_t row_bytes = (int64_t)a.blocks * 16;

  // Each XCD takes a contiguous range of tiles, in groups of kRasterRows tile
  // rows walked column by column, so that the tiles resident on one XCD share
  // their operands in its L2.  Rows past M or N read as zeros: the record
  // count ends at the last row.
  struct Tile {
    int64_t m0, n0;
    i32x4 a, b, ea, eb;  // buffer resources of its rows' codes and exponents
    int rows_a, rows_b;
  };
  auto tile_at = [&](int group, int in_group) {
    const int first_m = group * kRasterRows;
    const int gsz = min(a.tiles_m - first_m, kRasterRows);
    const int tn = gsz == 4 ? in_group >> 2 : gsz == 2 ? in_group >> 1 : gsz == 1 ? in_group : in_group / 3;
    Tile o;
    o.m0 = (int64_t)(first_m + in_group - tn * gsz) * kTileA, o.n0 = (int64_t)tn * kTileB;
    o.rows_a = a.M - o.m0 < kTileA ? (int)(a.M - o.m0) : kTileA;
    o.rows_b = a.N - o.n0 < kTileB ? (int)(a.N - o.n0) : kTileB;
    o.a = rsrc_words(a.A + o.m0 * row_bytes, (int)(o.rows_a * row_bytes));
    o.b = rsrc_words(a.B + o.n0 * row_bytes, (int)(o.rows_b * row_bytes));
    o.ea = rsrc_words(a.sA + o.m0 * a.blocks, o.rows_a * a.blocks);
    o.eb = rsrc_words(a.sB + o.n0 * a.blocks, o.rows_b * a.blocks);
    return o;
  };
  static_assert(kRasterRows == 4, "tile_at divides by 1 to 4");
  const int slots = gridDim.x >> 3, first_tile = (blockIdx.x & 7) * per_xcd;
  const int end_tile = min(first_tile + per_xcd, a.tiles_m * a.tiles_n);
  int at_tile = first_tile + (blockIdx.x >> 3);
  if (at_tile >= end_tile) return;
  const int per_group = kRasterRows * a.tiles_n;
  int group = at_tile / per_group, in_group = at_tile - group * per_group;
  Tile tile = tile_at(group, in_group);

  // Load i of this wave covers rows 8 (kLoads w + i) .. + 7 of an operand: lane
  // L writes row L / 8, physical chunk L % 8, and so reads chunk (L % 8) ^ swz.
  constexpr int kMostLoads = kLoadsA > kLoadsB ? kLoadsA : kLoadsB;
  static_assert(kLoadsA == kLoadsB, "A's and B's loads share their offsets");
  uint32_t voff[kMostLoads], past_k = 0;
#pragma unroll
  for (int i = 0; i < kMostLoads; ++i) {
    const int r = 8 * (kMostLoads * wave + i) + (lane >> 3);
    const int c = (lane & 7) ^ swz(r);
    voff[i] = (uint32_t)(r * row_bytes + 16 * c);
    past_k |= (uint32_t)((stages - 1) * kStageBlocks + c >= a.blocks) << i;  // in the last stage
  }
  const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>(&s_tile[0]);
  // Load l of stage s (even: of A, odd: of B).  Bit i of `past` sends load i of
  // either past the record count, where zeros are read: chunks past K, and all
  // of a stage past the last one (its zeros land in a buffer that nobody reads;
  // the loop below has no branches but its own, or the compiler would gather
  // the multiplications in one of its blocks).
  auto past = [&](int s) { return s < stages - 1 ? 0u : s == stages - 1 ? past_k : ~0u; };
  auto issue = [&](auto slow, int s, uint32_t past, int l) {
    const bool of_b = l & 1;
    const int i = l >> 1;
    const uint32_t at = lds0 + (s & (kBufs - 1)) * kStage + (of_b ? kTileA * kRowBytes : 0) + 8 * (kMostLoads * wave + i) * kRowBytes;
    lds_load16<decltype(slow)::value>(of_b ? tile.b : tile.a, at, voff[i] | ((past << (31 - i)) & 0x80000000u),
                                      (uint32_t)(s * kRowBytes));
  };

  // Exponents: lane (row, half) multiplies blocks 4 half .. 4 half + 3 of a
  // stage, four bytes of its row.  In the stage in which K ends the word may
  // reach past the row: what is not the row's is replaced by 127, and the codes
  // there are zeros.
  uint32_t keep_last = 0;  // which of the last stage's bytes are the row's
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if ((stages - 1) * kStageBlocks + 4 * half + j < a.blocks) keep_last |= 0xffu << (8 * j);
  uint32_t sa[kFA], sb[kFB], sa_next[kFA], sb_next[kFB];
  // Load p (one of kSpanPerWave) of this wave of exponent span c: 32 rows, two
  // lanes to a row, which change places in every other eight rows, so that the
  // words read below fall on twice as many banks; spans past K are not read.
  auto issue_span = [&](auto slow, int c, int p) {
    const int r = 32 * (kWaves * p + wave);  // of A's and B's rows in turn
    const bool of_b = r >= kTileA;
    const uint32_t at = (uint32_t)((r - (of_b ? kTileA : 0) + (lane >> 1)) * a.blocks + kSpanBytes * c + 16 * ((lane ^ (lane >> 4)) & 1));
    const uint32_t none = 4 * c < stages ? 0u : 0x80000000u;
    i32x4 rs;
#pragma unroll
    for (int w = 0; w < 4; ++w) rs[w] = of_b ? tile.eb[w] : tile.ea[w];
    lds_load16<decltype(slow)::value>(rs, lds0 + kBufs * kStage + (c & (kSpanBufs - 1)) * kSpan + r * kSpanBytes, at | none, 0);
  };
  // The exponents of stage s: from LDS, or (rows that start anywhere) asked for
  // in memory one stage ahead; a word that would pass the last row's end is
  // read earlier and shifted (both operands have at least four exponents).
  auto word_at = [&](int s, int row, int rows) { return min(row, rows - 1) * a.blocks + 4 * half + s * kStageBlocks; };
  auto word = [&](const uint8_t* e, int s, int row, int rows) {
    return *reinterpret_cast<const u32_a1*>(e + min(word_at(s, row, rows), rows * a.blocks - 4));
  };
  auto exponents_of = [&](const uint8_t* e, int64_t row) { return e + row * a.blocks; };
  auto exponents = [&](int s, uint32_t (&xa)[kFA], uint32_t (&xb)[kFB]) {
    const char* t = s_tile + kBufs * kStage + ((s >> 2) & (kSpanBufs - 1)) * kSpan + ((8 * (s & 3)) ^ (2 * (lrow & 8))) + 4 * half;
#pragma unroll
    for (int i = 0; i < kFA; ++i)
      xa[i] = kWords ? *reinterpret_cast<const uint32_t*>(t + (wm + 32 * i + lrow) * kSpanBytes)
                     : word(exponents_of(a.sA, tile.m0), s, wm + 32 * i + lrow, tile.rows_a);
#pragma unroll
    for (int i = 0; i < kFB; ++i)
      xb[i] = kWords ? *reinterpret_cast<const uint32_t*>(t + (kTileA + wn + 32 * i + lrow) * kSpanBytes)
                     : word(exponents_of(a.sB, tile.n0), s, wn + 32 * i + lrow, tile.rows_b);
  };
  auto finish_exponents = [&](int s, uint32_t (&xa)[kFA], uint32_t (&xb)[kFB]) {
    const uint32_t keep = s == stages - 1 ? keep_last : ~0u;
    auto finish = [&](uint32_t& x, int row, int rows) {
      if (!kWords) x >>= 8 * (max(word_at(s, row, rows) - (rows * a.blocks - 4), 0) & 3);
      x = (x & keep) | (0x7f7f7f7fu & ~keep);
    };
#pragma unroll
    for (int i = 0; i < kFA; ++i) finish(xa[i], wm + 32 * i + lrow, tile.rows_a);
#pragma unroll
    for (int i = 0; i < kFB; ++i) finish(xb[i], wn + 32 * i + lrow, tile.rows_b);
  };

  // Step j of a stage reads chunk 4 half + j of the wave's rows; block i's row
  // is 32 i further, which flips bit 2 of the chunk for odd i.
  const int base_a = (wm + lrow) * kRowBytes + 16 * ((4 * half) ^ swz(wm + lrow));
  const int base_b = kTileA * kRowBytes + (wn + lrow) * kRowBytes + 16 * ((4 * half) ^ swz(wn + lrow));
  u32x4 fa[2][kFA], fb[2][kFB];
  // Read n of a step's operands, in the order in which they are needed.
  constexpr int kReads = kFA + kFB;
  auto read = [&](int s, int j, int n) {
    const char* t = s_tile + (s & (kBufs - 1)) * kStage;
    const bool of_b = n != 1 && n <= kFB;
    const int i = n == 0 || n == 1 ? 0 : of_b ? n - 1 : n - kFB;
    u32x4& to = of_b ? fb[j & 1][i] : fa[j & 1][i];
    to = *reinterpret_cast<const u32x4*>(t + ((of_b ? base_b : base_a) ^ (16 * j) ^ (64 * (i & 1))) + 32 * kRowBytes * i);
  };

  f32x16 acc[kFA][kFB];

  // Step j of a stage: its multiplications, and after each of them (32 cycles of
  // the matrix core, 8 issues of the one wave that feeds it) a little of
  // everything else, in the order written: reads of the next step's operands,
  // loads of a later stage.
  constexpr int kSlots = kFA * kFB;
  auto step = [&](auto which, auto&& between) {
    constexpr int j = decltype(which)::value;
#pragma unroll
    for (int t = 0; t < kSlots; ++t) {
      const int i = t / kFB, k = t % kFB;
      acc[i][k] = mfma32<j>(fb[j & 1][k], sb[k], fa[j & 1][i], sa[i], acc[i][k]);
      between(t);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // Part n of `of`, spread over a step's slots from slot `from` on: f(n) at its slot.
  auto spread = [&](int t, int of, int from, auto&& f) {
#pragma unroll
    for (int n = 0; n < of; ++n)
      if (t == std::min(kSlots - 1, n * kSlots / of + from)) f(n);
  };
  using std::integral_constant;

  // A tile's first loads: all stages but one of the buffers, and the first spans
  // of exponents.
  constexpr int kFirstStages = (kBufs - 1) * kLoads;
  constexpr int kFirst = kFirstStages + (kWords ? kSpansAhead * kSpanPerWave : 0);
  auto start = [&](int l) {
    if (l < kFirstStages)
      issue(std::true_type{}, l / kLoads, past(l / kLoads), l % kLoads);
    else
      issue_span(std::true_type{}, (l - kFirstStages) / kSpanPerWave, (l - kFirstStages) % kSpanPerWave);
  };

  // The results of a wave leave through a patch of LDS (in the last buffer's
  // place), 32 rows of 128 bytes at a time, two blocks in turn: 16-byte chunk c
  // of row r at c ^ swz(r), the halves of a chunk swapped for rows with bit 4.
  constexpr int kPer = kBf16Out ? 8 : 4;               // columns per chunk
  constexpr int kPartsB = 32 * kFB / (8 * kPer);       // runs of columns
  constexpr int kPieces = kPartsB * kFA;               // of 32 rows x 128 bytes
  static_assert(kStage / kWaves >= 2 * 32 * 128, "two pieces fit");
  char* patch = s_tile + (kBufs - 1) * kStage + wave * (kStage / kWaves);
  // the next tile's first loads that go out with each piece
  constexpr int kPerPiece = std::max(8, (kFirst + kPieces - 1) / kPieces);
  // A whole tile's stores, four with each piece from two later on, that are
  // issued after the last of those loads: they need not have ended when the next
  // tile begins (16384 x 22016 x 4096: 686 us, 696 if all are waited for).
  constexpr int kStoresAfter = std::min(63, 4 * (kPieces + 2 - std::max(2, (kFirst - 1) / kPerPiece)));
  bool stored_whole = false;

#pragma unroll
  for (int l = 0; l < kFirst; ++l) start(l);
  static_assert(kLoads % 2 == 0 && kSpanLoads % kWaves == 0 && (kSpanPerWave == 4 || kSpanPerWave == 2), "every load has its place");
  for (;;) {
#pragma unroll
    for (int i = 0; i < kFA; ++i)
#pragma unroll
      for (int k = 0; k < kFB; ++k) acc[i][k] = (f32x16){};
    if (!kWords && stages > 0) exponents(0, sa, sb);
    // A wave that had nothing of a partial tile to store has read nothing back of what it
    // wrote to its patch; the compiler's barrier does not wait for that on its own, and the
    // others' loads go there from here on.
    asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
    if (kWords && stored_whole)
      asm volatile("s_waitcnt vmcnt(%0)" : : "i"(kStoresAfter) : "memory");
    else
      asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
    if (!kWords && stages > 0) finish_exponents(0, sa, sb);
    __syncthreads();
    // Before the last step of a stage every wave has read all of it: there the
    // next stage's loads are waited for, and after the barrier the loads of the
    // stage after it go into the buffer that has just been read, spread over
    // that last step and the first one of the next stage.
    if (stages > 0) {
      if (kWords) {
        exponents(0, sa, sb);
        finish_exponents(0, sa, sb);
      }
#pragma unroll
      for (int l = 0; l < kLoads / 2; ++l) issue(std::true_type{}, kBufs - 1, past(kBufs - 1), l);
#pragma unroll
      for (int n = 0; n < kReads; ++n) read(0, 0, n);
#pragma unroll 1
      for (int s = 0; s < stages; ++s) {
        if (!kWords) exponents(s + 1, sa_next, sb_next);
        __builtin_amdgcn_sched_barrier(0);
        const uint32_t past1 = past(s + kBufs - 1), past2 = past(s + kBufs);
        step(integral_constant<int, 0>{}, [&](int t) {
          spread(t, kReads, 0, [&](int n) { read(s, 1, n); });
          spread(t, kLoads / 2, 1, [&](int l) { issue(std::false_type{}, s + kBufs - 1, past1, kLoads / 2 + l); });
        });
        step(integral_constant<int, 1>{}, [&](int t) {
          spread(t, kReads, 0, [&](int n) { read(s, 2, n); });
          if (kWords && t == kSlots / 2)  // with fewer than four a span, some are loaded twice
            issue_span(std::false_type{}, (s >> 2) + kSpansAhead, s & (kSpanPerWave - 1));
        });
        step(integral_constant<int, 2>{}, [&](int t) { spread(t, kReads, 0, [&](int n) { read(s, 3, n); }); });
        // with four buffers the loads of two later stages, and the exponents
        // loaded meanwhile, may be on their way
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "i"(kBufs == 2 ? 0 : (kBufs - 2) * kLoads + kBufs - 1) : "memory");
        if (!kWords) {
          // the exponents are used here, so that the compiler's own wait for
          // them comes before the next loads and not after
          finish_exponents(s + 1, sa_next, sb_next);
#pragma unroll
          for (int i = 0; i < kFA; ++i) asm volatile("" : "+v"(sa_next[i]));
#pragma unroll
          for (int i = 0; i < kFB; ++i) asm volatile("" : "+v"(sb_next[i]));
        }
        __syncthreads();
        if (kWords) exponents(s + 1, sa_next, sb_next);
        __builtin_amdgcn_sched_barrier(0);
        step(integral_constant<int, 3>{}, [&](int t) {
          spread(t, kReads, 0, [&](int n) { read(s + 1, 0, n); });
          spread(t, kLoads / 2, 1, [&](int l) { issue(std::false_type{}, s + kBufs, past2, l); });
        });
        if (kWords) finish_exponents(s + 1, sa_next, sb_next);
#pragma unroll
        for (int i = 0; i < kFA; ++i) sa[i] = sa_next[i];
#pragma unroll
        for (int i = 0; i < kFB; ++i) sb[i] = sb_next[i];
      }
      // the loads past the last stage write LDS: they end before it is used again
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" : : : "memory");
    }
    __syncthreads();
    const int64_t m0 = tile.m0 + wm, n0 = tile.n0 + wn;
    const bool whole = tile.rows_a == kTileA && tile.rows_b == kTileB;
    at_tile += slots;
    const bool more = at_tile < end_tile;
    if (more) {
      in_group += slots;
      while (in_group >= per_group) in_group -= per_group, ++group;
      tile = tile_at(group, in_group);
    } else {
      tile.a.z = tile.b.z = tile.ea.z = tile.eb.z = 0;  // the first loads of no tile read nothing
    }

    // The B rows come first in the instruction, so that a lane holds four
    // consecutive columns: D[row 8 q + 4 half + e][column lrow], q = r / 4, e =
    // r % 4.  Stored from there, a store would touch 32 rows with 16 bytes each
    // (10 us for a tile of 256 x 256); out of the patch it is 8 rows of 128.
    // A wave's LDS operations are carried out in their order and its patch is
    // its own, so nothing waits but the stores for what they store.
    auto put = [&](int turn, int i, int part) {
      char* to = patch + (turn & 1) * 32 * 128 + lrow * 128;
#pragma unroll
      for (int k = 0; k < kPer / 4; ++k)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x16& d = acc[i][part * (kPer / 4) + k];
          if constexpr (kBf16Out)
            *reinterpret_cast<u32x2*>(to + 16 * ((4 * k + q) ^ swz(lrow)) + 8 * (half ^ (lrow >> 4))) =
                (u32x2){pack_bf16(d[4 * q], d[4 * q + 1]), pack_bf16(d[4 * q + 2], d[4 * q + 3])};
          else
            *reinterpret_cast<f32x4*>(to + 16 * ((2 * q + half) ^ swz(lrow))) =
                (f32x4){d[4 * q], d[4 * q + 1], d[4 * q + 2], d[4 * q + 3]};
        }
    };
    const int r = lane >> 3;
    u32x4 out[2][4];
    auto get = [&](int turn) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int row = 8 * x + r;
        const u32x4 v = *reinterpret_cast<const u32x4*>(patch + (turn & 1) * 32 * 128 + row * 128 + 16 * ((lane & 7) ^ swz(row)));
        out[turn & 1][x] = kBf16Out && x >= 2 ? (u32x4){v.z, v.w, v.x, v.y} : v;
      }
    };
    char* const to0 = static_cast<char*>(a.C) + ((m0 + r) * a.N + n0 + kPer * (lane & 7)) * (16 / kPer);
    auto loads = [&](int t) {
#pragma unroll
      for (int l = kPerPiece * t; l < kPerPiece * (t + 1); ++l)
        if (l < kFirst) start(l);
    };
    // Whole lines are streamed: left in L2, a round's results (4 MB an XCD) drive
    // out the operands (16384 x 22016 x 4096: 785 us, streamed 692).  Rows that
    // start inside lines are not: their lines have to meet in L2 (10308 x 10558 x
    // 384, fp32: streamed 384 us, else 221), and soon, so that a row's pieces
    // follow each other (146 us; rows of whole lines 94).  Whole lines go column
    // of pieces by column (16384 x 8192 x 4096, fp32: 286 us, by rows 301).
    auto store_whole = [&](auto streamed) {
      constexpr bool kStreamed = decltype(streamed)::value;
      auto row_of = [](int n) { return kStreamed ? n % kFA : n / kPartsB; };
      auto part_of = [](int n) { return kStreamed ? n / kFA : n % kPartsB; };
#pragma unroll
      for (int t = 0; t < kPieces + 2; ++t) {
        loads(t);
        if (t < kPieces) put(t, row_of(t), part_of(t));
        if (t >= 2) {
          auto at = [&](int x) {
            return reinterpret_cast<u32x4_a2*>(to0 + (32 * row_of(t - 2) + 8 * x) * a.N * (16 / kPer) + 128 * part_of(t - 2));
          };
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            if (kStreamed)
              __builtin_nontemporal_store(out[t & 1][x], at(x));
            else
              *at(x) = out[t & 1][x];
          }
        }
        if (t >= 1 && t <= kPieces) get(t - 1);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (kStreamed) asm volatile("; streamed");  // keeps the last stores from being merged with the others' last
    };
    if (whole && ((reinterpret_cast<uintptr_t>(a.C) | (uintptr_t)(a.N * (16 / kPer))) & 63) == 0) {
      store_whole(std::true_type{});
    } else if (whole) {
      store_whole(std::false_type{});
    } else {
#pragma unroll
      for (int t = 0; t < kPieces; ++t) {
        loads(t);
        put(t, t / kPartsB, t % kPartsB);
        get(t);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int64_t m = m0 + 32 * (t / kPartsB) + 8 * x + r, n = n0 + 8 * kPer * (t % kPartsB) + kPer * (lane & 7);
          if (m < a.M && n < a.N) store_chunk<kBf16Out>(a.C, m * a.N + n, out[t & 1][x], a.N - n);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (!more) break;
    stored_whole = whole;
  }
  asm volatile("s_waitcnt vmcnt(0)" : : : "memory");  // nothing writes LDS after the workgroup's end
}

template <int kFA, int kFB, int kWavesB, int kBufs>
void launch_tile(GemmArgs a, bool bf16, int cus, hipStream_t stream) {
  using Shape = TileShape<kFA, kFB, kWavesB, kBufs>;
  a.tiles_m = (int)((a.M + Shape::kTileA - 1) / Shape::kTileA);
  a.tiles_n = (int)((a.N + Shape::kTileB - 1) / Shape::kTileB);
  const int per_xcd = (int)(((int64_t)a.tiles_m * a.tiles_n + 7) / 8);
  const dim3 grid(8 * std::min(per_xcd, std::max(1, cus / 8) * Shape::kPerCu)), block(Shape::kThreads);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, a, per_xcd); };
  if (words(a)) {
    bf16 ? go(mx_gemm_tile_kernel<kFA, kFB, kWavesB, kBufs, true, true>)
         : go(mx_gemm_tile_kernel<kFA, kFB, kWavesB, kBufs, true, false>);
  } else if constexpr (kBufs == 2) {
    bf16 ? go(mx_gemm_tile_kernel<kFA, kFB, kWavesB, kBufs, false, true>)
         : go(mx_gemm_tile_kernel<kFA, kFB, kWavesB, kBufs, false, false>);
  }
}

// ---- few tiles: every wave its own slice of K ----
//
// With fewer tiles than CUs, or few rows, the time is that of memory's latency
// and of the weight's way through the chip.  A workgroup owns a tile of 32 kFA x
// 32 kFB results; its four waves take its stages (256 values, as above) in turn,
// each through a ring of kDepth stages of LDS that is its own: a wave waits for
// nothing but its own oldest loads, and 100 KB or more are on their way to
// every CU.  The four sums meet in LDS at the end.  64 x 4096 x 11008: 9.2 us for
// 25 MB, of which the launch and the two ends of the pipeline are about half.
constexpr int kSliceWaves = 4;

template <int kFA, int kFB, int kDepth, bool kBf16Out>
__global__ __launch_bounds__(64 * kSliceWaves, 1) void mx_gemm_slice_kernel(const GemmArgs a, int per_xcd) {
  constexpr int kTileA = 32 * kFA, kTileB = 32 * kFB;
  constexpr int kLoadsA = 4 * kFA, kLoadsB = 4 * kFB;         // 8 rows of 128 bytes each
  constexpr int kExps = kFA + kFB;                            // 32 rows of 8 exponents each
  constexpr int kPerStage = kLoadsA + kLoadsB + kExps;        // loads of a wave per stage
  constexpr int kCodes = (kTileA + kTileB) * kRowBytes, kStage = kCodes + kExps * 256;
  constexpr int kBlocks = kFA * kFB;
  constexpr int kRing = kSliceWaves * kDepth * kStage, kSums = (kSliceWaves - 1) * kBlocks * 64 * 64;
  static_assert(kPerStage * (kDepth - 1) <= 63, "the waits count to 63");
  __shared__ __attribute__((aligned(16))) char s_lds[kRing > kSums ? kRing : kSums];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lrow = lane & 31, half = lane >> 5;
  // XCDs take contiguous ranges of tiles, down the columns: the tiles that
  // share a piece of B are near each other
  const int tile = (blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
  if (tile >= a.tiles_m * a.tiles_n) return;
  const int tn = tile / a.tiles_m;
  const int64_t m0 = (int64_t)(tile - tn * a.tiles_m) * kTileA, n0 = (int64_t)tn * kTileB;
  const int rows_a = a.M - m0 < kTileA ? (int)(a.M - m0) : kTileA, rows_b = a.N - n0 < kTileB ? (int)(a.N - n0) : kTileB;
  const int64_t row_bytes = (int64_t)a.blocks * 16;
  const i32x4 ra = rsrc_words(a.A + m0 * row_bytes, (int)(rows_a * row_bytes));
  const i32x4 rb = rsrc_words(a.B + n0 * row_bytes, (int)(rows_b * row_bytes));
  const i32x4 rea = rsrc_words(a.sA + m0 * a.blocks, rows_a * a.blocks);
  const i32x4 reb = rsrc_words(a.sB + n0 * a.blocks, rows_b * a.blocks);
  const int stages = (a.blocks + kStageBlocks - 1) / kStageBlocks;
  const int mine = (stages - wave + kSliceWaves - 1) / kSliceWaves;  // stages wave, wave + 4, ...

  // Load l covers rows 8 l .. + 7, lane L row L / 8, physical chunk L % 8.
  constexpr int kMost = kLoadsA > kLoadsB ? kLoadsA : kLoadsB;
  uint32_t voff[kMost], past_k = 0;
#pragma unroll
  for (int l = 0; l < kMost; ++l) {
    const int r = 8 * l + (lane >> 3), c = (lane & 7) ^ swz(r);
    voff[l] = (uint32_t)(r * row_bytes + 16 * c);
    past_k |= (uint32_t)((stages - 1) * kStageBlocks + c >= a.blocks) << l;
  }
  const uint32_t voff_e = (uint32_t)((lane >> 1) * a.blocks + 4 * (lane & 1));
  const bool past_k_e = (stages - 1) * kStageBlocks + 4 * (lane & 1) >= a.blocks;
  const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>(&s_lds[0]) + wave * kDepth * kStage;
  // This wave's stage i into slot i mod kDepth; past its last, zeros that nobody reads.
  auto issue = [&](int i, int slot) {
    const int s = wave + kSliceWaves * i;
    const uint32_t past = s < stages - 1 ? 0u : s == stages - 1 ? past_k : ~0u;
    const uint32_t none = s < stages - 1 ? 0u : (s > stages - 1 || past_k_e) ? 0x80000000u : 0u;
    const uint32_t at = lds0 + slot * kStage;
#pragma unroll
    for (int l = 0; l < kMost; ++l) {
      const uint32_t v = voff[l] | ((past << (31 - l)) & 0x80000000u);
      if (l < kLoadsA) lds_load16<true>(ra, at + 1024 * l, v, (uint32_t)(s * kRowBytes));
      if (l < kLoadsB) lds_load16<true>(rb, at + kTileA * kRowBytes + 1024 * l, v, (uint32_t)(s * kRowBytes));
    }
#pragma unroll
    for (int e = 0; e < kExps; ++e) {
      const int block = e < kFA ? e : e - kFA;
      lds_load4(e < kFA ? rea : reb, at + kCodes + 256 * e,
                (voff_e + (uint32_t)(32 * block * a.blocks + s * kStageBlocks)) | none);
    }
  };

  f32x16 acc[kFA][kFB];
#pragma unroll
  for (int i = 0; i < kFA; ++i)
#pragma unroll
    for (int j = 0; j < kFB; ++j) acc[i][j] = (f32x16){};
  const int base_a = lrow * kRowBytes + 16 * ((4 * half) ^ swz(lrow)), base_b = kTileA * kRowBytes + base_a;
  auto compute = [&](int i, int slot) {
    const char* t = s_lds + (wave * kDepth + slot) * kStage;
    uint32_t sa[kFA], sb[kFB];
    // in the stage in which K ends, exponents past it: 127
    uint32_t keep = ~0u;
    if (wave + kSliceWaves * i == stages - 1) {
      keep = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if ((stages - 1) * kStageBlocks + 4 * half + j < a.blocks) keep |= 0xffu << (8 * j);
    }
#pragma unroll
    for (int x = 0; x < kFA; ++x)
      sa[x] = (*reinterpret_cast<const uint32_t*>(t + kCodes + 256 * x + 8 * lrow + 4 * half) & keep) | (0x7f7f7f7fu & ~keep);
#pragma unroll
    for (int x = 0; x < kFB; ++x)
      sb[x] = (*reinterpret_cast<const uint32_t*>(t + kCodes + 256 * (kFA + x) + 8 * lrow + 4 * half) & keep) |
              (0x7f7f7f7fu & ~keep);
    u32x4 fa[4][kFA], fb[4][kFB];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int x = 0; x < kFA; ++x)
        fa[j][x] = *reinterpret_cast<const u32x4*>(t + (base_a ^ (16 * j) ^ (64 * (x & 1))) + 32 * kRowBytes * x);
#pragma unroll
      for (int x = 0; x < kFB; ++x)
        fb[j][x] = *reinterpret_cast<const u32x4*>(t + (base_b ^ (16 * j) ^ (64 * (x & 1))) + 32 * kRowBytes * x);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");  // the slot may be written again from here on
    auto multiply = [&](auto step) {
      constexpr int j = decltype(step)::value;
#pragma unroll
      for (int x = 0; x < kFA; ++x)
#pragma unroll
        for (int y = 0; y < kFB; ++y) acc[x][y] = mfma32<j>(fb[j][y], sb[y], fa[j][x], sa[x], acc[x][y]);
    };
    multiply(std::integral_constant<int, 0>{});
    multiply(std::integral_constant<int, 1>{});
    multiply(std::integral_constant<int, 2>{});
    multiply(std::integral_constant<int, 3>{});
  };

#pragma unroll
  for (int i = 0; i < kDepth; ++i) issue(i, i);
  int slot = 0;
#pragma unroll 1
  for (int i = 0; i < mine; ++i) {
    asm volatile("s_waitcnt vmcnt(%0)" : : "i"(kPerStage * (kDepth - 1)) : "memory");
    compute(i, slot);
    issue(i + kDepth, slot);
    slot = slot + 1 == kDepth ? 0 : slot + 1;
  }
  asm volatile("s_waitcnt vmcnt(0)" : : : "memory");  // nothing writes LDS from here on
  __syncthreads();

  // Block b of the tile is summed and stored by wave b mod 4; the others leave
  // theirs in LDS, the sums are added in wave order.
  f32x4* sums = reinterpret_cast<f32x4*>(s_lds);  // [block][3 others][4][lane]
#pragma unroll
  for (int b = 0; b < kBlocks; ++b) {
    const int owner = b % kSliceWaves;
    if (wave == owner) continue;
    const int place = wave - (wave > owner ? 1 : 0);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const f32x16& d = acc[b / kFB][b % kFB];
      sums[((b * (kSliceWaves - 1) + place) * 4 + q) * 64 + lane] = (f32x4){d[4 * q], d[4 * q + 1], d[4 * q + 2], d[4 * q + 3]};
    }
  }
  __syncthreads();
#pragma unroll
  for (int b = 0; b < kBlocks; ++b) {
    if (wave != b % kSliceWaves) continue;
    const int64_t m = m0 + 32 * (b / kFB) + lrow;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const f32x16& d = acc[b / kFB][b % kFB];
      const f32x4 own = {d[4 * q], d[4 * q + 1], d[4 * q + 2], d[4 * q + 3]};
      f32x4 v = (f32x4){0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < kSliceWaves; ++w)
        v += w == b % kSliceWaves ? own : sums[((b * (kSliceWaves - 1) + w - (w > b % kSliceWaves ? 1 : 0)) * 4 + q) * 64 + lane];
      const int64_t n = n0 + 32 * (b % kFB) + 8 * q + 4 * half;
      if (m < a.M && n < a.N) store4<kBf16Out>(a.C, m * a.N + n, v, a.N - n);
    }
  }
}

template <int kFA, int kFB, int kDepth>
void launch_slice(GemmArgs a, bool bf16, hipStream_t stream) {
  a.tiles_m = (int)((a.M + 32 * kFA - 1) / (32 * kFA));
  a.tiles_n = (int)((a.N + 32 * kFB - 1) / (32 * kFB));
  const int per_xcd = (int)(((int64_t)a.tiles_m * a.tiles_n + 7) / 8);
  const dim3 grid(8 * per_xcd), block(64 * kSliceWaves);
  if (bf16)
    hipLaunchKernelGGL((mx_gemm_slice_kernel<kFA, kFB, kDepth, true>), grid, block, 0, stream, a, per_xcd);
  else
    hipLaunchKernelGGL((mx_gemm_slice_kernel<kFA, kFB, kDepth, false>), grid, block, 0, stream, a, per_xcd);
}

template <int kM, int kN, int kW>
void launch_stream(GemmArgs a, bool bf16, hipStream_t stream) {
  a.tiles_m = (int)((a.M + 16 * kM - 1) / (16 * kM));
  a.tiles_n = (int)((a.N + 16 * kN - 1) / (16 * kN));
  const dim3 grid((unsigned)std::min<int64_t>((int64_t)a.tiles_m * a.tiles_n, 1 << 20)), block(64 * kW);
  if (bf16)
    hipLaunchKernelGGL((mx_gemm_stream_kernel<kM, kN, kW, true>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((mx_gemm_stream_kernel<kM, kN, kW, false>), grid, block, 0, stream, a);
}

// Which kernel takes a product.  Measured at K = 4096 and N = 4096 or 22016
// unless noted; "words" are exponents in aligned words (K a multiple of 128).
//   * up to 16 rows: the stream, 16 columns per workgroup (1 x 4096 x 11008: 6.4
//     us, 32 columns 9.4), 32 from about two workgroups per CU on (16 x 22016:
//     16.6 and 13.5 us);
//   * few tiles: the smallest slices that need no second round of workgroups (64
//     x 4096 x 11008: 32 x 32 slices 9.4 us, 64 x 64 16.0, tiles of 128 33; 128 x
//     4096: 64 x 32 slices 7.4 us, 32 x 32 10.6; 256 x 4096: 64 x 64 slices 8.7
//     us, tiles of 128 15.1); up to 32 rows of more columns than that, the
//     stream (32 x 22016: 17.5 us, slices 18.5);
//   * tiles of 128 or of 256 by their rounds: one of 256 x 256 tiles takes 27 us,
//     one of 128 x 128 24 us, or 15 us when no CU has two of them (512 x 22016:
//     35 us and 47 us, 2048 x 4096: 27 us and 23 us), and then with four buffers
//     (1024 x 4096: 14.5 us, with two 16.5; 512 x 4096 x 11008: 27 and 35 us);
//   * without words, the stream in place of the slices (256 x 4096 x 1376: 7.3
//     us, tiles of 128 9.1; 512 x 4096 x 1376: 12.7 and 9.4 us).
// The tiles' rounds were measured at K = 4096 and decide at every K.  Tiles of 256
// and of 128, in us, the rule's choice first: 16384 x 22016 x 128 160 and 152, x
// 256 157 and 154, x 1024 262 and 301, x 11008 1718 and 2412; 8192 x 8192 x 128 34
// and 37, x 512 45 and 42, x 1024 66 and 62, x 11008 329 and 471; 4096 x 4096 x 128
// 11.4 and 10.0, x 1024 17.4 and 18.0, x 4064 46 and 69; 2048 x 4096 (128 first) x
// 256 7.0 and 8.5, x 11008 58 and 60.  It is never more than a seventh off there, and at
// short K the time is that of the results' way to memory (16384 x 22016 x 32: 158
// us, 4.6 TB/s).
void pick_and_launch(const GemmArgs& a, bool bf16, int cus, hipStream_t stream) {
  auto tiles = [&](int64_t tm, int64_t tn) { return ((a.M + tm - 1) / tm) * ((a.N + tn - 1) / tn); };
  if (a.M <= 32) {
    if (a.M <= 16)
      return tiles(16, 16) <= 2 * cus ? launch_stream<1, 1, 8>(a, bf16, stream) : launch_stream<1, 2, 8>(a, bf16, stream);
    if (tiles(32, 64) > cus) return launch_stream<2, 2, 4>(a, bf16, stream);
  }
  if (words(a)) {
    if (tiles(32, 32) <= cus) return launch_slice<1, 1, 4>(a, bf16, stream);
    if (a.M <= 32 && tiles(32, 64) <= cus) return launch_slice<1, 2, 3>(a, bf16, stream);
    if (tiles(64, 32) <= cus) return launch_slice<2, 1, 3>(a, bf16, stream);
    if (tiles(64, 64) <= cus) return launch_slice<2, 2, 2>(a, bf16, stream);
  } else {
    // (the tiles' reads of exponents need four of them in either operand)
    if (tiles(32, 32) <= 4 * cus || std::min(a.M, a.N) * a.blocks < 4) return launch_stream<2, 2, 4>(a, bf16, stream);
  }
  const int64_t small = tiles(128, 128), large = tiles(256, 256);
  const int64_t cost_small = small <= cus ? 15 : 24 * ((small + 2 * cus - 1) / (2 * cus));
  if (27 * ((large + cus - 1) / cus) <= cost_small)
    launch_tile<4, 4, 2, 2>(a, bf16, cus, stream);
  else if (small <= cus && words(a))
    launch_tile<2, 2, 2, 4>(a, bf16, cus, stream);
  else
    launch_tile<2, 2, 2, 2>(a, bf16, cus, stream);
}

}  // namespace

hipError_t code_objects::load_mxfp4gemm() { return load(mx_gemm_stream_kernel<1, 1, 8, true>); }

extern "C" {

__attribute__((visibility("default"))) int mxfp4_gemm(const void* A, const void* sA, const void* B, const void* sB,
                                                      void* C, int64_t M, int64_t N, int64_t K, int c_dtype,
                                                      hipStream_t stream) {
  if (M < 0 || N < 0 || K < 0 || K % 32 != 0 || K > (int64_t(1) << 22) || M > (int64_t(1) << 31) ||
      N > (int64_t(1) << 31) || (c_dtype != SILUQUANT_F32 && c_dtype != SILUQUANT_BF16))
    return SILUQUANT_ERR_BAD_SHAPE;
  if (M == 0 || N == 0) return SILUQUANT_OK;
  // tiles are counted in 32 bits, at 128 x 128 results each at the least
  if (((M + 127) / 128) * ((N + 127) / 128) > (int64_t(1) << 30)) return SILUQUANT_ERR_BAD_SHAPE;
  const bool bf16 = c_dtype == SILUQUANT_BF16;
  if (!C || (K > 0 && (!A || !sA || !B || !sB))) return SILUQUANT_ERR_NULL_PTR;
  if (misaligned(A, 16) || misaligned(B, 16) || misaligned(C, bf16 ? 2 : 4)) return SILUQUANT_ERR_MISALIGNED;
  const Span c = {C, M * N * (bf16 ? 2 : 4)};
  if (overlap(c, {A, M * K / 2}) || overlap(c, {sA, M * K / 32}) || overlap(c, {B, N * K / 2}) ||
      overlap(c, {sB, N * K / 32}))
    return SILUQUANT_ERR_OVERLAP;
  const GemmArgs a = {static_cast<const uint8_t*>(A), static_cast<const uint8_t*>(sA), static_cast<const uint8_t*>(B),
                      static_cast<const uint8_t*>(sB), C, M, N, (int)(K / 32), 0, 0};
  int dev = 0, cus = 0;  // asked on every call (the runtime answers from its cached properties): no state is kept
  if (hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0)
    return SILUQUANT_ERR_DEVICE;
  pick_and_launch(a, bf16, cus, stream);
  return hipGetLastError() == hipSuccess ? SILUQUANT_OK : SILUQUANT_ERR_LAUNCH_FAILED;
}

}  // extern "C"
