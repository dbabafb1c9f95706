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
// Rows past M or N are read as the last row and not stored.
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
  const int tn = blockIdx.x % a.tiles_n, tm = blockIdx.x / a.tiles_n;
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
  if (kW > 1) {
    if (wave > 0) {
#pragma unroll
      for (int i = 0; i < kM; ++i)
#pragma unroll
        for (int j = 0; j < kN; ++j) s_sum[wave - 1][i * kN + j][lane] = acc[i][j];
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int i = 0; i < kM; ++i)
#pragma unroll
      for (int j = 0; j < kN; ++j)
        for (int w = 0; w < kW - 1; ++w) acc[i][j] += s_sum[w][i * kN + j][lane];
  }
#pragma unroll
  for (int i = 0; i < kM; ++i) {
    const int64_t m = ((int64_t)tm * kM + i) * 16 + r;
    if (m >= a.M) continue;
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const int64_t n = ((int64_t)tn * kN + j) * 16 + 4 * kb;
      if (n < a.N) store4<kBf16Out>(a.C, m * a.N + n, acc[i][j], a.N - n);
    }
  }
}

// ---- many rows: tiles through LDS ----
//
// 256 threads, four waves in a 2 x 2 grid, a tile of 64 kF x 64 kF results; a
// wave owns kF x kF blocks of 32 x 32.  A stage is 256 values (8 blocks, 128
// bytes) of every row of the tile: the codes go from memory straight into LDS
// (buffer loads with the lds flag), double buffered, the exponents into
// registers.  Rows of 128 bytes lie in LDS as eight 16-byte chunks, chunk c of
// row r at c ^ swz(r), so that the 16 lanes that read a chunk of consecutive
// rows fall on distinct banks.
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kStageBlocks = 8;                 // per row and stage
constexpr int kRowBytes = 16 * kStageBlocks;    // 128
constexpr int kTileThreads = 256;
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

// Each lane reads 16 (or 4) bytes at voff + soff (voff is checked against the
// record count); the wave writes them, lane by lane, to consecutive LDS bytes
// from address lds (M0) on.  Written as asm so that
// the compiler does not wait for them before every LDS read; the kernel waits
// itself.  The leading s_nop is the wait state between the compiler's write of
// M0 and its use.
__device__ __forceinline__ void lds_load16(i32x4 rs, uint32_t lds, uint32_t voff, uint32_t soff) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
               :
               : "v"(voff), "s"(rs), "s"(__builtin_amdgcn_readfirstlane(soff)),
                 "{m0}"(__builtin_amdgcn_readfirstlane(lds))
               : "memory");
}

__device__ __forceinline__ void lds_load4(i32x4 rs, uint32_t lds, uint32_t voff) {
  asm volatile("s_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds"
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

// kWords: rows of exponents start on 4 bytes (K is a multiple of 128).  They
// then go into LDS too, 32 blocks of every row at a time, a quarter of the next
// 32 with each stage: read from memory by every wave in every stage, 4 bytes a
// row, they doubled the requests to L2 and cost a quarter of the time.
//
// Workgroups are persistent (one per CU for 256 x 256, two for 128 x 128): the
// next tile's first stage is asked for before the present one's results are
// stored, and the stores drain behind its first stage.
template <int kF, bool kWords, bool kBf16Out>
__global__ __launch_bounds__(kTileThreads, kF == 4 ? 1 : 2) void mx_gemm_tile_kernel(const GemmArgs a, int per_xcd) {
  constexpr int kT = 64 * kF;                        // rows of A, and of B, per tile
  constexpr int kOpBytes = kT * kRowBytes;           // one operand's stage
  constexpr int kLoads = kT / 8 / 4;                 // wave-wide loads per operand and stage: 8 rows each
  constexpr int kSpanBytes = 32;                     // exponents of a row that are loaded together: four stages
  constexpr int kSpan = 2 * kT * kSpanBytes;         // of all rows, A's and then B's
  __shared__ __attribute__((aligned(16))) char s_tile[4 * kOpBytes + (kWords ? 2 * kSpan : 0)];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = (wave >> 1) * 32 * kF, wn = (wave & 1) * 32 * kF;
  const int lrow = lane & 31, half = lane >> 5;
  const int stages = (a.blocks + kStageBlocks - 1) / kStageBlocks;
  const int64_t row_bytes = (int64_t)a.blocks * 16;

  // Each XCD takes a contiguous range of tiles, in groups of kRasterRows tile
  // rows walked column by column, so that the tiles resident on one XCD share
  // their operands in its L2.  Rows past M or N read as zeros: the record
  // count ends at the last row.
  struct Tile {
    int64_t m0, n0;
    const uint8_t *a, *b, *ea, *eb;
    int rows_a, rows_b;
  };
  auto tile_at = [&](int t) {
    const int per_group = kRasterRows * a.tiles_n;
    const int first_m = (t / per_group) * kRasterRows;
    const int in_group = t % per_group;
    const int gsz = min(a.tiles_m - first_m, kRasterRows);
    Tile o;
    o.m0 = (int64_t)(first_m + in_group % gsz) * kT, o.n0 = (int64_t)(in_group / gsz) * kT;
    o.rows_a = a.M - o.m0 < kT ? (int)(a.M - o.m0) : kT, o.rows_b = a.N - o.n0 < kT ? (int)(a.N - o.n0) : kT;
    o.a = a.A + o.m0 * row_bytes, o.b = a.B + o.n0 * row_bytes;
    o.ea = a.sA + o.m0 * a.blocks, o.eb = a.sB + o.n0 * a.blocks;
    return o;
  };
  const int slots = gridDim.x >> 3, first_tile = (blockIdx.x & 7) * per_xcd;
  const int end_tile = min(first_tile + per_xcd, a.tiles_m * a.tiles_n);
  int at_tile = first_tile + (blockIdx.x >> 3);
  if (at_tile >= end_tile) return;
  Tile tile = tile_at(at_tile);

  // Load i of this wave covers rows 8 (kLoads w + i) .. + 7 of an operand: lane
  // L writes row L / 8, physical chunk L % 8, and so reads chunk (L % 8) ^ swz.
  uint32_t voff[kLoads], voff_last[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = 8 * (kLoads * wave + i) + (lane >> 3);
    const int c = (lane & 7) ^ swz(r);
    voff[i] = (uint32_t)(r * row_bytes + 16 * c);
    voff_last[i] = (stages - 1) * kStageBlocks + c < a.blocks ? voff[i] : 0x80000000u;  // past K: zeros
  }
  const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>(&s_tile[0]);
  // Load i of stage s, A's and B's; past the last stage nothing is read (a
  // record count of 0) and zeros land in a buffer that nobody reads.  The loop
  // below has no branches but its own, or the compiler would gather the
  // multiplications in one of its blocks.
  auto issue = [&](int s, int i) {
    const uint32_t at = lds0 + (s & 1) * 2 * kOpBytes + 8 * (kLoads * wave + i) * kRowBytes;
    const uint32_t v = s == stages - 1 ? voff_last[i] : voff[i];
    const int live = (s - stages) >> 31;  // all ones before the end
    lds_load16(rsrc_words(tile.a, (int)(tile.rows_a * row_bytes) & live), at, v, (uint32_t)(s * kRowBytes));
    lds_load16(rsrc_words(tile.b, (int)(tile.rows_b * row_bytes) & live), at + kOpBytes, v, (uint32_t)(s * kRowBytes));
  };

  // Exponents: lane (row, half) multiplies blocks 4 half .. 4 half + 3 of a
  // stage, four bytes of its row.  In the stage in which K ends the word may
  // reach past the row: what is not the row's is replaced by 127, and the codes
  // there are zeros.
  uint32_t keep_last = 0;  // which of the last stage's bytes are the row's
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if ((stages - 1) * kStageBlocks + 4 * half + j < a.blocks) keep_last |= 0xffu << (8 * j);
  uint32_t sa[kF], sb[kF], sa_next[kF], sb_next[kF];
  // Piece p (one of 4 kF) of exponent span c: eight rows, eight lanes to a row.
  auto issue_span = [&](int c, int p) {
    const int r = 8 * (4 * p + wave);  // of A's and B's rows in turn
    const bool of_b = r >= kT;
    const int live = (4 * c - stages) >> 31;
    const int bytes = (of_b ? tile.rows_b : tile.rows_a) * a.blocks;
    lds_load4(rsrc_words(of_b ? tile.eb : tile.ea, bytes & live),
              lds0 + 4 * kOpBytes + (c & 1) * kSpan + r * kSpanBytes,
              (uint32_t)((r - (of_b ? kT : 0) + (lane >> 3)) * a.blocks + kSpanBytes * c + 4 * (lane & 7)));
  };
  // The exponents of stage s: from LDS, or (rows that start anywhere) asked for
  // in memory one stage ahead; a word that would pass the last row's end is
  // read earlier and shifted (both operands have at least four exponents).
  auto exponents = [&](int s, uint32_t (&xa)[kF], uint32_t (&xb)[kF]) {
#pragma unroll
    for (int i = 0; i < kF; ++i) {
      if (kWords) {
        const char* t = s_tile + 4 * kOpBytes + ((s >> 2) & 1) * kSpan + (s & 3) * kStageBlocks + 4 * half;
        xa[i] = *reinterpret_cast<const uint32_t*>(t + (wm + 32 * i + lrow) * kSpanBytes);
        xb[i] = *reinterpret_cast<const uint32_t*>(t + (kT + wn + 32 * i + lrow) * kSpanBytes);
      } else {
        const int oa = min(wm + 32 * i + lrow, tile.rows_a - 1) * a.blocks + 4 * half + s * kStageBlocks;
        const int ob = min(wn + 32 * i + lrow, tile.rows_b - 1) * a.blocks + 4 * half + s * kStageBlocks;
        xa[i] = *reinterpret_cast<const u32_a1*>(tile.ea + min(oa, tile.rows_a * a.blocks - 4));
        xb[i] = *reinterpret_cast<const u32_a1*>(tile.eb + min(ob, tile.rows_b * a.blocks - 4));
      }
    }
  };
  auto finish_exponents = [&](int s, uint32_t (&xa)[kF], uint32_t (&xb)[kF]) {
    const uint32_t keep = s == stages - 1 ? keep_last : ~0u;
#pragma unroll
    for (int i = 0; i < kF; ++i) {
      if (!kWords) {
        const int oa = min(wm + 32 * i + lrow, tile.rows_a - 1) * a.blocks + 4 * half + s * kStageBlocks;
        const int ob = min(wn + 32 * i + lrow, tile.rows_b - 1) * a.blocks + 4 * half + s * kStageBlocks;
        xa[i] >>= 8 * (max(oa - (tile.rows_a * a.blocks - 4), 0) & 3);
        xb[i] >>= 8 * (max(ob - (tile.rows_b * a.blocks - 4), 0) & 3);
      }
      xa[i] = (xa[i] & keep) | (0x7f7f7f7fu & ~keep);
      xb[i] = (xb[i] & keep) | (0x7f7f7f7fu & ~keep);
    }
  };

  // Step j of a stage reads chunk 4 half + j of the wave's rows; block i's row
  // is 32 i further, which flips bit 2 of the chunk for odd i.
  const int base_a = (wm + lrow) * kRowBytes + 16 * ((4 * half) ^ swz(wm + lrow));
  const int base_b = kOpBytes + (wn + lrow) * kRowBytes + 16 * ((4 * half) ^ swz(wn + lrow));
  u32x4 fa[2][kF], fb[2][kF];
  auto read = [&](int s, int j, int i) {
    const char* t = s_tile + (s & 1) * 2 * kOpBytes;
    fa[j & 1][i] = *reinterpret_cast<const u32x4*>(t + (base_a ^ (16 * j) ^ (64 * (i & 1))) + 32 * kRowBytes * i);
    fb[j & 1][i] = *reinterpret_cast<const u32x4*>(t + (base_b ^ (16 * j) ^ (64 * (i & 1))) + 32 * kRowBytes * i);
  };

  f32x16 acc[kF][kF];

  // Step j of a stage: row by row of its blocks, kF multiplications and then
  // the reads of the next step's operands (and loads of a later stage), in the
  // order written, so that the matrix cores never wait for an issue.
  auto step = [&](auto which, auto&& between) {
    constexpr int j = decltype(which)::value;
#pragma unroll
    for (int i = 0; i < kF; ++i) {
#pragma unroll
      for (int k = 0; k < kF; ++k) acc[i][k] = mfma32<j>(fb[j & 1][k], sb[k], fa[j & 1][i], sa[i], acc[i][k]);
      between(i);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  using std::integral_constant;

  auto start = [&] {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) issue(0, i);
    if (kWords) {
#pragma unroll
      for (int p = 0; p < 4 * kF; ++p) issue_span(0, p);
    }
  };

  // The results of a wave leave through a patch of LDS (the second stage's),
  // 128 bytes of each of its rows at a time: 16-byte chunk c of row r at c ^ r
  // (mod 8), the halves of a chunk swapped for rows with bit 4.
  constexpr int kPer = kBf16Out ? 8 : 4;             // columns per chunk
  constexpr int kParts = 32 * kF / (8 * kPer);
  constexpr int kStores = kParts * 4 * kF;           // a wave's stores of a whole tile
  char* patch = s_tile + 2 * kOpBytes + wave * 32 * kF * 128;

  start();
  bool whole_before = false;  // the stores of a whole tile are on their way behind this one's loads
  constexpr int kPerRow = kLoads / kF / 2;  // loads after each row of blocks of the two steps
  for (;;) {
#pragma unroll
    for (int i = 0; i < kF; ++i)
#pragma unroll
      for (int j = 0; j < kF; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    if (!kWords && stages > 0) exponents(0, sa, sb);
    // memory operations of a wave end in the order of their issue: the loads are
    // done when only the stores are left
    if (whole_before)
      asm volatile("s_waitcnt vmcnt(%0)" : : "i"(kStores < 63 ? kStores : 63) : "memory");
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
      for (int i = 0; i < kLoads / 2; ++i) issue(1, i);
#pragma unroll
      for (int i = 0; i < kF; ++i) read(0, 0, i);
#pragma unroll 1
      for (int s = 0; s < stages; ++s) {
        if (!kWords) exponents(s + 1, sa_next, sb_next);
        __builtin_amdgcn_sched_barrier(0);
        step(integral_constant<int, 0>{}, [&](int i) {
          read(s, 1, i);
#pragma unroll
          for (int l = 0; l < kPerRow; ++l) issue(s + 1, kLoads / 2 + kPerRow * i + l);
        });
        step(integral_constant<int, 1>{}, [&](int i) {
          read(s, 2, i);
          if (kWords) issue_span((s >> 2) + 1, kF * (s & 3) + i);
        });
        step(integral_constant<int, 2>{}, [&](int i) { read(s, 3, i); });
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" : : : "memory");
        if (!kWords) {
          // the exponents are used here, so that the compiler's own wait for
          // them comes before the next loads and not after
          finish_exponents(s + 1, sa_next, sb_next);
#pragma unroll
          for (int i = 0; i < kF; ++i) asm volatile("" : "+v"(sa_next[i]), "+v"(sb_next[i]));
        }
        __syncthreads();
        if (kWords) exponents(s + 1, sa_next, sb_next);
        __builtin_amdgcn_sched_barrier(0);
        step(integral_constant<int, 3>{}, [&](int i) {
          read(s + 1, 0, i);
#pragma unroll
          for (int l = 0; l < kPerRow; ++l) issue(s + 2, kPerRow * i + l);
        });
        if (kWords) finish_exponents(s + 1, sa_next, sb_next);
#pragma unroll
        for (int i = 0; i < kF; ++i) sa[i] = sa_next[i], sb[i] = sb_next[i];
      }
      // the loads past the last stage write LDS: they end before it is used again
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" : : : "memory");
    }
    __syncthreads();
    const int64_t m0 = tile.m0 + wm, n0 = tile.n0 + wn;
    const bool whole = tile.rows_a == kT && tile.rows_b == kT;
    at_tile += slots;
    const bool more = at_tile < end_tile;
    if (more) {
      tile = tile_at(at_tile);
      start();
    }

    // The B rows come first in the instruction, so that a lane holds four
    // consecutive columns: D[row 8 q + 4 half + e][column lrow], q = r / 4, e =
    // r % 4.  Stored from there, a store would touch 32 rows with 16 bytes each
    // (10 us for a tile of 256 x 256); out of the patch it is 8 rows of 128.
#pragma unroll
    for (int part = 0; part < kParts; ++part) {
#pragma unroll
      for (int i = 0; i < kF; ++i)
#pragma unroll
        for (int k = 0; k < kPer / 4; ++k)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x16& d = acc[i][part * (kPer / 4) + k];
            const int row = 32 * i + lrow;
            char* to = patch + row * 128;
            if constexpr (kBf16Out)
              *reinterpret_cast<u32x2*>(to + 16 * (((4 * k + q) ^ row) & 7) + 8 * (half ^ ((row >> 4) & 1))) =
                  (u32x2){pack_bf16(d[4 * q], d[4 * q + 1]), pack_bf16(d[4 * q + 2], d[4 * q + 3])};
            else
              *reinterpret_cast<f32x4*>(to + 16 * (((2 * q + half) ^ row) & 7)) =
                  (f32x4){d[4 * q], d[4 * q + 1], d[4 * q + 2], d[4 * q + 3]};
          }
      asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");  // the wave's own writes: no other wave touches its patch
      const int64_t n = n0 + 8 * kPer * part + kPer * (lane & 7);
#pragma unroll
      for (int r0 = 0; r0 < 32 * kF; r0 += 8) {
        const int row = r0 + (lane >> 3);
        u32x4 v = *reinterpret_cast<const u32x4*>(patch + row * 128 + 16 * ((lane ^ row) & 7));
        if (kBf16Out && (r0 & 16)) v = (u32x4){v.z, v.w, v.x, v.y};
        const int64_t m = m0 + row;
        if (whole)
          store_chunk<kBf16Out>(a.C, m * a.N + n, v, kPer);
        else if (m < a.M && n < a.N)
          store_chunk<kBf16Out>(a.C, m * a.N + n, v, a.N - n);
      }
      asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
    }
    if (!more) break;
    whole_before = whole;
  }
}

template <int kF>
void launch_tile(GemmArgs a, bool bf16, int cus, hipStream_t stream) {
  a.tiles_m = (int)((a.M + 64 * kF - 1) / (64 * kF));
  a.tiles_n = (int)((a.N + 64 * kF - 1) / (64 * kF));
  const int per_xcd = (int)(((int64_t)a.tiles_m * a.tiles_n + 7) / 8);
  const dim3 grid(8 * std::min(per_xcd, std::max(1, cus / 8) * (kF == 4 ? 1 : 2))), block(kTileThreads);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, a, per_xcd); };
  if (a.blocks % 4 == 0)
    bf16 ? go(mx_gemm_tile_kernel<kF, true, true>) : go(mx_gemm_tile_kernel<kF, true, false>);
  else
    bf16 ? go(mx_gemm_tile_kernel<kF, false, true>) : go(mx_gemm_tile_kernel<kF, false, false>);
}

template <int kM, int kN, int kW>
void launch_stream(GemmArgs a, bool bf16, hipStream_t stream) {
  a.tiles_m = (int)((a.M + 16 * kM - 1) / (16 * kM));
  a.tiles_n = (int)((a.N + 16 * kN - 1) / (16 * kN));
  const dim3 grid((unsigned)((int64_t)a.tiles_m * a.tiles_n)), block(64 * kW);
  if (bf16)
    hipLaunchKernelGGL((mx_gemm_stream_kernel<kM, kN, kW, true>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((mx_gemm_stream_kernel<kM, kN, kW, false>), grid, block, 0, stream, a);
}

}  // namespace

extern "C" {

__attribute__((visibility("default"))) int mxfp4_gemm(const void* A, const void* sA, const void* B, const void* sB,
                                                      void* C, int64_t M, int64_t N, int64_t K, int c_dtype,
                                                      hipStream_t stream) {
  if (M < 0 || N < 0 || K < 0 || K % 32 != 0 || K > (int64_t(1) << 22) || M > (int64_t(1) << 31) ||
      N > (int64_t(1) << 31) || (c_dtype != SILUQUANT_F32 && c_dtype != SILUQUANT_BF16))
    return SILUQUANT_ERR_BAD_SHAPE;
  if (M == 0 || N == 0) return SILUQUANT_OK;
  // workgroups are counted in 32 bits, at 16 x 16 results each at the least
  if (((M + 15) / 16) * ((N + 15) / 16) > (int64_t(1) << 30)) return SILUQUANT_ERR_BAD_SHAPE;
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
  if (M <= 16)
    launch_stream<1, 1, 8>(a, bf16, stream);
  else if (M <= 64)
    launch_stream<2, 2, 8>(a, bf16, stream);
  else if (N * (K / 32) < 4)
    launch_stream<2, 2, 8>(a, bf16, stream);
  else if (((M + 255) / 256) * ((N + 255) / 256) >= 128)
    launch_tile<4>(a, bf16, cus, stream);
  else
    launch_tile<2>(a, bf16, cus, stream);
  return hipGetLastError() == hipSuccess ? SILUQUANT_OK : SILUQUANT_ERR_LAUNCH_FAILED;
}

}  // extern "C"
