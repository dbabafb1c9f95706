// The gated projection in bf16 and its backward pass, on the CDNA4 matrix cores
// (gfx950):
//
//   forward   [gate | up] = x . W^T,  y = silu(gate) * up       x [T, D], W [2H, D]
//   backward  d_gu = [dy * up * s * (1 + gate * (1 - s)) | dy * gate * s],  s = sigmoid(gate)
//             dx = d_gu . W,  dW = d_gu^T . x                    (d_gu rounded to bf16)
//
// Products of bf16 numbers are exact in fp32 and summed there.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "code_objects.h"
#include "rows.h"
#include "siluquant.h"
#include "swiglu_plan.h"

namespace {

using namespace rows;
using namespace swiglu;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// silu(g) * u = g * s * u with the sigmoid s = 1 / (1 + exp(-g)) in parts that neither
// overflow nor lose small values: with h = exp(-|g| / 2) and r = 1 / (1 + h^2), s is r for
// g >= 0 and h^2 r below, where one h comes before u and one behind it (silu alone is a
// denormal number from g = -87 on, and 0 from -104).  Within 4 (|g| + 4) 2^-24 of itself:
// the exponent is rounded relative to itself, and h carries that twice (3e-7 in all for g
// in (-2, 0), 1e-6 at -20, 4e-6 at -80); for what is rounded to bf16 behind it.
__device__ __forceinline__ float silu_times(float g, float u) {
  const float h = __builtin_amdgcn_exp2f(-0.72134752044f * __builtin_fabsf(g));  // log2(e) / 2
  const float r = __builtin_amdgcn_rcpf(__builtin_fmaf(h, h, 1.0f)), part = g < 0.0f ? h : 1.0f;
  return (((g * part) * r) * u) * part;
}

// ---- d_gu ----
//
// In fp64 but for what is small: d_gu is an operand of two products, and arithmetic in
// fp32 rounds one value in a hundred thousand to its other neighbour in bf16 (13 in a
// million; this one 0.1).  fp64's range also holds every product and every sigmoid on
// the way.  Reads dy, gate and up once and writes d_gu: 16384 x 11008, 1.8 GB, in 309 us
// before the products, 5.8 TB/s (a large copy: 5.1), its arithmetic and memory about even;
// in fp32 296.

// exp(-a) for a >= 0, good to 1.1e-8 for every bf16 a up to 700: a = k ln 2 - r, |r| <=
// ln 2 / 2, where k times the first 13 bits of ln 2 and its distance from a (of 8 bits, up
// to 800) are exact in fp32; 1 + r in fp64 and the rest of the series, 0.07 at most, in
// fp32.  Past 800 it is 0 in fp64 too; a NaN is the caller's to keep.
__device__ __forceinline__ double exp_minus(float a) {
  constexpr float kHi = 0.693115234375f, kLo = (float)(0.69314718055994530942 - 0.693115234375);
  a = __builtin_fminf(a, 800.0f);
  const float k = __builtin_rintf(a * 1.44269504f), r = __builtin_fmaf(k, kHi, -a), left = k * kLo, q = r + left;
  float p = 1.0f / 40320;
  p = __builtin_fmaf(p, q, 1.0f / 5040);
  p = __builtin_fmaf(p, q, 1.0f / 720);
  p = __builtin_fmaf(p, q, 1.0f / 120);
  p = __builtin_fmaf(p, q, 1.0f / 24);
  p = __builtin_fmaf(p, q, 1.0f / 6);
  p = __builtin_fmaf(p, q, 0.5f);
  return __builtin_amdgcn_ldexp(1.0 + ((double)r + (double)__builtin_fmaf(p * q, q, left)), -(int)k);
}

struct GateArgs {
  const uint16_t* dy;  // [T, H]
  const uint16_t* gu;  // [T, 2H], may be d_gu
  uint16_t* d_gu;      // [T, 2H]
  int64_t T;
  int H;
};
__global__ __launch_bounds__(256) void swiglu_gate_bwd_kernel(const GateArgs a) {
  const int pieces = a.H / 8;
  const int64_t all = a.T * pieces;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < all; i += gridDim.x * 256ll) {
    const int64_t t = i / pieces;
    const int col = 8 * (int)(i - t * pieces);
    const uint16_t* from = a.gu + 2 * t * a.H + col;
    float d[8], g[8], u[8], dg[8], du[8];
    unpack(d, load_bf16<kFull, true>(a.dy + t * a.H + col, 8));
    unpack(g, load_bf16<kFull, true>(from, 8));
    unpack(u, load_bf16<kFull, true>(from + a.H, 8));
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      // s * (1 + gate * (1 - s)) as s + gate * w: w = s * (1 - s) is the same for -gate
      const double e = exp_minus(__builtin_fabsf(g[k])), m = 1.0 + e;
      double r = __builtin_amdgcn_rcpf((float)m);  // and a step of Newton's
      r = __builtin_fma(__builtin_fma(-m, r, 1.0), r, r);
      const double er = e * r, s = g[k] < 0.0f ? er : r, w = er * r;
      dg[k] = (float)(((double)d[k] * u[k]) * __builtin_fma((double)g[k], w, s));
      du[k] = (float)((double)d[k] * (s * g[k]));
    }
    auto pack8 = [](const float (&v)[8]) {
      return Piece{{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])}};
    };
    store_bf16<kFull, false>(a.d_gu + 2 * t * a.H + col, pack8(dg), 8);
    store_bf16<kFull, false>(a.d_gu + 2 * t * a.H + a.H + col, pack8(du), 8);
  }
}

// ---- products ----
//
// C [M, N] = sum over k of A[m, k] * B[n, k].  An operand is stored by rows, [rows,
// K], or by k, [K, rows]; the three products of this file are
//   kGated  A = x by rows,    B = the rows of Wg and Wu, whose results meet in a lane
//   kDx     A = d_gu by rows, B = W by k
//   kDw     A = d_gu by k,    B = x by k
enum Product { kGated = 0, kDx = 1, kDw = 2 };

struct GemmArgs {
  const uint16_t *A, *B;
  void* C;
  uint16_t* gu;    // kGated: [M, 2N], may be null
  int64_t M, N, K;  // kGated: N = H, half the rows of B
  int lda, ldb;    // elements from one stored row to the next
  int tiles_m, tiles_n;
  int64_t split_k;  // values of K per slice, K for one slice; slice blockIdx.y writes its own C [M, N] behind the others'
};

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// ---- tiles through LDS ----
//
// A workgroup owns a tile of kTileA x kTileB results, its waves (2 x kWavesB) kFA x
// kFB blocks of 32 x 32 each.  A stage is 64 values of k of every row of the tile: it
// goes from memory straight into LDS (buffer loads with the lds flag), one to three
// stages ahead of its use.  Workgroups stay and take tile after tile; the next tile's
// first stages are loaded while the results of the one before leave.
//
// Of the largest products (16384 x 11008 x 4096: gate and up 2.95 TFLOP) the forward
// pass takes 2360 us with gate and up kept (1250 TFLOP/s) and 2270 without (1300), dx
// 2110 (1400), dW 2270 (1300).  The chip's power bounds most of that: with zeros for
// operands, which cost it little, the same instructions take 1660 us (1780 TFLOP/s; dx
// 1880), and multiplying random numbers out of registers alone, with nothing loaded,
// reaches 1840.  The forward pass is further from that than dx (matrix cores busy 71% and
// 80%): the way out of its tiles, with gate and up through LDS in fp32 and one turn of
// pieces, is about 7 us, and each workgroup takes 22 of them.  Tiles of 256 x 256 by four waves read each operand from LDS least
// often: a wave's 128 x 128 results take 256 accumulators a lane.  Two buffers of A and
// three of B fill the 160 KB: loads are answered at some 25 bytes a cycle and CU when
// all ask, and what is on its way has to cover that (two buffers of each, zeros: 1390
// TFLOP/s for 1780).  Measured and not taken: the instruction of 16 x 16 x 32 (dx
// 2050 us for 2110, but the forward pass 2450 for 2360 and 777 x 1376 x 2048 25 for
// 19.6: twice as many instructions to issue beside the loads'), all of a stage's
// loads in one step, eight rows of tiles a group, non-temporal stores (as fast).
//
// An operand stored by rows lies in LDS as rows of 128 bytes, eight 16-byte chunks,
// chunk c of row r at c ^ swz(r): the 16 lanes that read a chunk of consecutive rows
// fall on distinct banks.  One stored by k lies there as 64 rows of its tile's width;
// the transposing LDS reads hand a lane four k of its column, 16 lanes reading 32
// bytes of each of four rows, and runs of 64 bytes of row r are exchanged by r & 3, so
// that the 32 lanes that are served together fall on all banks.
//
// The order of k within a sum is free as long as A and B agree: lane half h takes
// k = 8 (4 h + j) .. + 7 of a stage in step j, which is chunk 4 h + j of a row.
constexpr int kRowBytes = 2 * kStageK;
constexpr int kRasterRows = 4;  // tile rows that are walked column by column together

__device__ __forceinline__ int swz(int r) { return (r ^ (r >> 3)) & 7; }

// Buffer resource words: base, 32-bit record count (loads at or past it read as
// zeros), raw addressing.
__device__ __forceinline__ i32x4 rsrc_words(uint64_t base, int bytes) {
  return (i32x4){__builtin_amdgcn_readfirstlane((int)(uint32_t)base), __builtin_amdgcn_readfirstlane((int)(uint32_t)(base >> 32) & 0xFFFF),
                 __builtin_amdgcn_readfirstlane(bytes), 0x00020000};
}

// Each lane reads 16 bytes at voff + soff (voff is checked against the record
// count, each 4 bytes for themselves); the wave writes them, lane by lane, to
// consecutive LDS bytes from address lds (M0) on.  Written as asm so that the
// compiler does not wait for them before every LDS read; the kernel waits itself.
// The leading s_nop gives the wait states that the compiler cannot, since it does
// not look inside: one between the write of M0 and its use; and, with kSlow, five
// between a vector instruction's write of a scalar register and a load that reads it.
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

// Four k of a lane's column; p: the lane's 8 bytes of the 32 that 4 lanes read of a row.
__device__ __forceinline__ u32x2 read_transposed(const char* p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                       (__attribute__((address_space(3))) s16x4*)p));
}

__device__ __forceinline__ f32x16 mfma(const u32x4& a, const u32x4& b, const f32x16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

template <int kFA, int kFB, int kWavesB, int kBufs, bool kGatedTile>
struct TileShape {
  static constexpr int kWaves = 2 * kWavesB, kThreads = 64 * kWaves;
  static constexpr int kTileA = 64 * kFA, kTileB = 32 * kWavesB * kFB;  // rows of A and of B
  static constexpr int kStage = (kTileA + kTileB) * kRowBytes;
  // The results' way out: per wave, one or two pieces of 32 rows x 128 bytes (gated: of
  // gate and of up), in the last buffer's place or in one of their own.
  static constexpr int kPiece = 32 * 128 * (kGatedTile ? 2 : 1);
  static constexpr bool kUneven = kBufs == 3;  // two buffers of A's, three of B's
  static constexpr int kPatch = kUneven ? kTileB * kRowBytes : kStage;  // bytes in that place
  static constexpr int kTurns = kPatch >= 2 * kWaves * kPiece || kFA == 1 ? 2 : 1;
  static constexpr bool kOwnPatch = kPatch < kTurns * kWaves * kPiece;
  static constexpr int kBuffers = kUneven ? 2 * kTileA * kRowBytes + 3 * kTileB * kRowBytes : kBufs * kStage;
  static constexpr int kLds = kBuffers + (kOwnPatch ? kTurns * kWaves * kPiece : 0);
  static constexpr int kPerCu = 2 * kLds <= 160 * 1024 ? 2 : 1;  // workgroups that fit a CU's LDS
  static constexpr int kPerSimd = kPerCu * kWaves < 4 ? 1 : kPerCu * kWaves / 4;         // waves
};

// Where an operand's stage comes from.  By rows: the resource stays, k advances with
// the scalar offset.  By k: the base advances, and the record count ends at K.
template <bool kByK>
struct Source {
  i32x4 rs;
  uint32_t soff;
  // by k:
  uint64_t base;
  uint32_t step;         // bytes from one stage to the next
  int left;              // stages, this one among them
  int all, last;         // record counts: of a stage, and of the one in which K ends
  __device__ __forceinline__ void by_rows(const uint16_t* p, int64_t row, int rows, int64_t row_bytes) {
    rs = rsrc_words(reinterpret_cast<uint64_t>(p) + row * row_bytes, (int)(rows * row_bytes));
    soff = 0;
  }
  __device__ __forceinline__ void count() { rs = rsrc_words(base, left > 1 ? all : left == 1 ? last : 0); }
  __device__ __forceinline__ void by_k(const uint16_t* p, int64_t column, int64_t K, int row_bytes) {
    const int from = (int)(2 * column);  // into a row
    base = reinterpret_cast<uint64_t>(p) + from;
    step = (uint32_t)(kStageK * row_bytes);
    left = (int)((K + kStageK - 1) / kStageK);
    all = kStageK * row_bytes - from, last = (int)(K - (int64_t)(left - 1) * kStageK) * row_bytes - from;
    soff = 0;
    count();
  }
  __device__ __forceinline__ void advance() {
    if constexpr (kByK) {
      base += step, --left;
      count();
    } else {
      soff += kRowBytes;
    }
  }
  __device__ __forceinline__ void none() { rs.z = 0, left = 0; }  // reads zeros from here on
};

template <int kFA, int kFB, int kWavesB, int kBufs, Product kProduct, bool kKeep, bool kF32>
__global__ __launch_bounds__(128 * kWavesB, (TileShape<kFA, kFB, kWavesB, kBufs, kProduct == kGated>::kPerSimd)) void
swiglu_tile_kernel(const GemmArgs all, int per_xcd) {
  using Shape = TileShape<kFA, kFB, kWavesB, kBufs, kProduct == kGated>;
  constexpr int kWaves = Shape::kWaves, kTileA = Shape::kTileA, kTileB = Shape::kTileB;
  constexpr bool kAByK = kProduct == kDw, kBByK = kProduct != kGated;
  constexpr bool kUneven = Shape::kUneven;
  constexpr int kStage = Shape::kStage;                     // A's bytes, then B's
  constexpr int kLoadsA = kTileA / 8 / kWaves, kLoadsB = kTileB / 8 / kWaves;  // wave-wide loads of 1 KB per stage
  constexpr int kLoads = kLoadsA + kLoadsB;
  constexpr int kTileN = kProduct == kGated ? kTileB / 2 : kTileB;             // columns of C
  __shared__ __attribute__((aligned(16))) char s_tile[Shape::kLds];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = (wave / kWavesB) * 32 * kFA, wn = (wave % kWavesB) * 32 * kFB;
  const int lrow = lane & 31, half = lane >> 5;
  GemmArgs a = all;
  if (kProduct != kGated && kF32 && blockIdx.y > 0) {
    const int64_t k0 = blockIdx.y * a.split_k;
    a.A += kAByK ? k0 * a.lda : k0;
    a.B += k0 * a.ldb;
    a.C = static_cast<float*>(a.C) + blockIdx.y * a.M * a.N;
    a.K -= k0;
  }
  if (kProduct != kGated && kF32 && a.K > a.split_k) a.K = a.split_k;
  const int stages = (int)((a.K + kStageK - 1) / kStageK);

  // Each XCD takes a contiguous range of tiles, in groups of kRasterRows tile rows
  // walked column by column, so that the tiles resident on one XCD share their
  // operands in its L2.
  int64_t m0, n0;
  int rows_a, rows_n;
  Source<kAByK> sa;
  Source<kBByK> sb;
  Source<false> sb2;  // the up projection's rows
  auto tile_at = [&](int group, int in_group) {
    const int first_m = group * kRasterRows;
    const int gsz = min(a.tiles_m - first_m, kRasterRows);
    const int tn = gsz == 4 ? in_group >> 2 : gsz == 2 ? in_group >> 1 : gsz == 1 ? in_group : in_group / 3;
    m0 = (int64_t)(first_m + in_group - tn * gsz) * kTileA, n0 = (int64_t)tn * kTileN;
    rows_a = a.M - m0 < kTileA ? (int)(a.M - m0) : kTileA;
    rows_n = a.N - n0 < kTileN ? (int)(a.N - n0) : kTileN;
    if constexpr (kAByK)
      sa.by_k(a.A, m0, a.K, 2 * a.lda);
    else
      sa.by_rows(a.A, m0, rows_a, 2ll * a.lda);
    if constexpr (kBByK) {
      sb.by_k(a.B, n0, a.K, 2 * a.ldb);
    } else {
      sb.by_rows(a.B, n0, rows_n, 2ll * a.ldb);
      sb2.by_rows(a.B, a.N + n0, rows_n, 2ll * a.ldb);
    }
  };
  static_assert(!kAByK || kFA > 1, "runs are exchanged among four");
  static_assert(kRasterRows == 4, "tile_at divides by 1 to 4");
  const int slots = gridDim.x >> 3, first_tile = (blockIdx.x & 7) * per_xcd;
  const int end_tile = min(first_tile + per_xcd, a.tiles_m * a.tiles_n);
  int at_tile = first_tile + (blockIdx.x >> 3);
  if (at_tile >= end_tile) return;
  const int per_group = kRasterRows * a.tiles_n;
  int group = at_tile / per_group, in_group = at_tile - group * per_group;
  tile_at(group, in_group);

  // A wave's load i of an operand fills 1 KB of LDS, lane L its bytes 16 L and on.
  // By rows: eight rows; lane L writes row L / 8, physical chunk L % 8, and so reads
  // chunk (L % 8) ^ swz.  By k: the rows that 1 KB holds, runs of four chunks exchanged
  // by the row.  Where gate and up rows share a tile, the loads take them in turn, and
  // the rows lie so that a wave's 32 kFB rows are its gate columns and then the same
  // up columns.
  auto row_of_b = [&](int i) {  // LDS row of B's load i
    if constexpr (kProduct == kGated) {
      const int col = 8 * ((i >> 1) + kLoadsB / 2 * wave);
      return (col / (16 * kFB)) * 32 * kFB + (i & 1) * 16 * kFB + col % (16 * kFB);
    } else {
      return 8 * (kLoadsB * wave + i);
    }
  };
  uint32_t voff_a[kLoadsA], voff_b[kLoadsB], past_a = 0, past_b = 0;
  auto place = [&](bool by_k, int lds_row, int global_row, int width, int ld, uint32_t& voff, uint32_t& past, int i) {
    if (by_k) {
      const int byte = 128 * lds_row + 16 * lane, k = byte / width, c = (byte % width / 16) ^ (4 * (k & 3));
      voff = (uint32_t)(2 * k * ld + 16 * c);
    } else {
      const int c = (lane & 7) ^ swz(lds_row + (lane >> 3));
      voff = (uint32_t)((global_row + (lane >> 3)) * 2 * ld + 16 * c);
      past |= (uint32_t)((stages - 1) * kStageK + 8 * c >= a.K) << i;  // in the last stage
    }
  };
#pragma unroll
  for (int i = 0; i < kLoadsA; ++i) {
    const int r = 8 * (kLoadsA * wave + i);
    place(kAByK, r, r, 2 * kTileA, a.lda, voff_a[i], past_a, i);
  }
#pragma unroll
  for (int i = 0; i < kLoadsB; ++i)
    place(kBByK, row_of_b(i), 8 * ((i >> 1) + kLoadsB / 2 * wave), 2 * kTileB, a.ldb, voff_b[i], past_b, i);
  const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>(&s_tile[0]);
  // Load l of stage s, for which the sources stand.  Bit i of `past` sends load i of an
  // operand stored by rows past the record count, where zeros are read: chunks past K,
  // and all of a stage past the last one (its zeros land in a buffer that nobody
  // reads; the loop below has no branches but its own).
  auto past_of = [&](int s, uint32_t last) { return s < stages - 1 ? 0u : s == stages - 1 ? last : ~0u; };
  auto issue_a = [&](auto slow, int s, uint32_t at, int i) {
    const uint32_t off = kAByK ? voff_a[i] : voff_a[i] | ((past_of(s, past_a) << (31 - i)) & 0x80000000u);
    lds_load16<decltype(slow)::value>(sa.rs, at + 8 * (kLoadsA * wave + i) * kRowBytes, off, sa.soff);
  };
  auto issue_b = [&](auto slow, int s, uint32_t at, int i) {
    const uint32_t off = kBByK ? voff_b[i] : voff_b[i] | ((past_of(s, past_b) << (31 - i)) & 0x80000000u);
    const uint32_t to = at + row_of_b(i) * kRowBytes;
    if (kProduct == kGated && (i & 1))
      lds_load16<decltype(slow)::value>(sb2.rs, to, off, sb.soff);
    else
      lds_load16<decltype(slow)::value>(sb.rs, to, off, sb.soff);
  };
  // Where stage s of an operand lies in LDS.  Three buffers are told by turn_b, the
  // present stage's (0, 1, 2 in turn).
  constexpr int kABytes = kTileA * kRowBytes, kBBytes = kTileB * kRowBytes;
  uint32_t turn_b = 0;
  auto a_at = [&](int s) { return (uint32_t)(kUneven ? (s & 1) * kABytes : (s & (kBufs - 1)) * kStage); };
  auto b_at = [&](int s) { return (uint32_t)((s & (kBufs - 1)) * kStage + kABytes); };
  auto b_turn = [&](uint32_t ahead) {  // of the stage `ahead` (0 to 2) behind the present one
    const uint32_t t = turn_b + ahead;
    return 2 * kABytes + (t >= 3 ? t - 3 : t) * kBBytes;
  };
  auto issue = [&](auto slow, int s, int l) {
    // A's and B's loads in turn as long as there are both
    constexpr int kPairs = kLoadsA < kLoadsB ? kLoadsA : kLoadsB;
    const bool of_b = l < 2 * kPairs ? l & 1 : kLoadsB > kLoadsA;
    const int i = l < 2 * kPairs ? l >> 1 : l - kPairs;
    of_b ? issue_b(slow, s, lds0 + b_at(s), i) : issue_a(slow, s, lds0 + a_at(s), i);
  };
  auto advance = [&] { sa.advance(), sb.advance(); };

  // Step j of a stage reads k = 8 (4 half + j) .. + 7 of the wave's rows.  By rows:
  // chunk 4 half + j; block i's row is 32 i further, which flips bit 2 of the chunk for
  // odd i.  By k: rows 32 half + 8 j and on, in two reads of four; block i is 64 i bytes
  // further, exchanged like the runs.
  auto base_of = [&](bool by_k, int w0, int width) {
    if (by_k) {
      const int r = (lane >> 2) & 3;
      return (32 * half + r) * width + 64 * ((w0 / 32) ^ r) + 32 * ((lane >> 4) & 1) + 8 * (lane & 3);
    }
    return (w0 + lrow) * kRowBytes + 16 * ((4 * half) ^ swz(w0 + lrow));
  };
  const int base_a = base_of(kAByK, wm, 2 * kTileA), base_b = base_of(kBByK, wn, 2 * kTileB);
  u32x4 fa[2][kFA], fb[2][kFB];
  constexpr int kReads = kFA + kFB;
  // Read n of a step's operands, in the order in which they are needed.
  // at_a, at_b: where the stage's operands lie.
  auto read = [&](uint32_t at_a, uint32_t at_b, int j, int n) {
    const bool of_b = n != 1 && n <= kFB;
    const int i = n == 0 || n == 1 ? 0 : of_b ? n - 1 : n - kFB;
    u32x4& to = of_b ? fb[j & 1][i] : fa[j & 1][i];
    const int base = of_b ? base_b : base_a;
    const char* t = s_tile + (of_b ? at_b : at_a);
    if (of_b ? kBByK : kAByK) {
      const int width = 2 * (of_b ? kTileB : kTileA);
      const u32x2 lo = read_transposed(t + (base ^ (64 * i)) + 8 * j * width), hi = read_transposed(t + (base ^ (64 * i)) + (8 * j + 4) * width);
      to = (u32x4){lo.x, lo.y, hi.x, hi.y};
    } else {
      to = *reinterpret_cast<const u32x4*>(t + (base ^ (16 * j) ^ (64 * (i & 1))) + 32 * kRowBytes * i);
    }
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
      acc[i][k] = mfma(fb[j & 1][k], fa[j & 1][i], acc[i][k]);
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

  // A tile's first loads: all buffers but the last (uneven: B's last).
  constexpr int kFirst = kUneven ? 2 * kLoads : (kBufs - 1) * kLoads;
  auto start = [&](int l) {
    if (l > 0 && l % kLoads == 0) advance();
    const int s = l / kLoads;
    if constexpr (kUneven) {
      const int i = l % kLoads;
      if (i < kLoadsA)
        issue_a(std::true_type{}, s, lds0 + a_at(s), i);
      else
        issue_b(std::true_type{}, s, lds0 + 2 * kABytes + s * kBBytes, i - kLoadsA);
    } else {
      issue(std::true_type{}, s, l % kLoads);
    }
  };

  // The results of a wave leave through a patch of LDS (in the last buffer's
  // place), 32 rows of 128 bytes at a time, two pieces in turn: 16-byte chunk c
  // of row r at c ^ swz(r), the halves of a chunk swapped for rows with bit 4.
  constexpr int kPer = kF32 ? 4 : 8;                        // columns per chunk
  constexpr int kPartsB = kProduct == kGated ? kFB / 2 : 32 * kFB / (8 * kPer);  // runs of columns
  constexpr int kPieces = kPartsB * kFA;                    // of 32 rows x 128 bytes (gated: two such, of gate and up in fp32)
  constexpr int kTurns = Shape::kTurns, kPieceBytes = Shape::kPiece;
  static_assert(kTurns == 2 || kProduct == kGated, "the others alternate");
  char* patch = s_tile + (Shape::kOwnPatch ? Shape::kBuffers + wave * kTurns * kPieceBytes
                                           : Shape::kBuffers - Shape::kPatch + wave * (Shape::kPatch / kWaves));
  // The next tile's first loads go out with the first half of the pieces.  What is
  // stored after the last of them, if the tile is whole, need not have ended when the
  // next tile begins.
  constexpr int kPerPiece = std::max(8, (kFirst + kPieces - 1) / kPieces);
  constexpr int kPerStore = kProduct == kGated ? (kKeep ? 6 : 2) : 4;  // stores of a piece, kBehind pieces later on
  constexpr int kBehind = kProduct == kGated ? 1 : 2;
  constexpr int kStoresAfter = std::min(63, kPerStore * (kPieces + kBehind - std::max(kBehind, (kFirst - 1) / kPerPiece + 1)));
  bool stored_whole = false;

#pragma unroll
  for (int l = 0; l < kFirst; ++l) start(l);
  for (;;) {
#pragma unroll
    for (int i = 0; i < kFA; ++i)
#pragma unroll
      for (int k = 0; k < kFB; ++k) acc[i][k] = (f32x16){};
    // A wave that had nothing of a partial tile to store has read nothing back of what it
    // wrote to its patch; the compiler's barrier does not wait for that on its own, and the
    // others' loads go there from here on.
    asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
    if (stored_whole)
      asm volatile("s_waitcnt vmcnt(%0)" : : "i"(kStoresAfter) : "memory");
    else
      asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
    __syncthreads();
    // Before the last step of a stage every wave has read all of it: there the
    // next stage's loads are waited for, and after the barrier the loads of the
    // stage after it go into the buffer that has just been read, spread over
    // that last step and the first one of the next stage.
    if constexpr (kUneven) {
      // A's loads of two stages on are in a stage's last step, when its buffer has been
      // read; B's in the first two steps, one buffer further.
      sb.advance();
      turn_b = 0;
#pragma unroll
      for (int n = 0; n < kReads; ++n) read(0, b_turn(0), 0, n);
#pragma unroll 1
      for (int s = 0; s < stages; ++s) {
        const uint32_t now_a = a_at(s), now_b = b_turn(0), next_b = b_turn(1), load_b = lds0 + b_turn(2);
        __builtin_amdgcn_sched_barrier(0);
        step(integral_constant<int, 0>{}, [&](int t) {
          spread(t, kReads, 0, [&](int n) { read(now_a, now_b, 1, n); });
          spread(t, kLoadsB / 2, 1, [&](int i) { issue_b(std::false_type{}, s + 2, load_b, i); });
        });
        step(integral_constant<int, 1>{}, [&](int t) {
          spread(t, kReads, 0, [&](int n) { read(now_a, now_b, 2, n); });
          spread(t, kLoadsB / 2, 1, [&](int i) { issue_b(std::false_type{}, s + 2, load_b, kLoadsB / 2 + i); });
        });
        step(integral_constant<int, 2>{}, [&](int t) { spread(t, kReads, 0, [&](int n) { read(now_a, now_b, 3, n); }); });
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "i"(kLoadsB) : "memory");
        __syncthreads();
        advance();
        turn_b = turn_b == 2 ? 0 : turn_b + 1;
        __builtin_amdgcn_sched_barrier(0);
        step(integral_constant<int, 3>{}, [&](int t) {
          spread(t, kReads, 0, [&](int n) { read(a_at(s + 1), next_b, 0, n); });
          spread(t, kLoadsA, 1, [&](int i) { issue_a(std::false_type{}, s + 2, lds0 + now_a, i); });
        });
      }
    } else {
      advance();
#pragma unroll
      for (int l = 0; l < kLoads / 2; ++l) issue(std::true_type{}, kBufs - 1, l);
#pragma unroll
      for (int n = 0; n < kReads; ++n) read(a_at(0), b_at(0), 0, n);
#pragma unroll 1
      for (int s = 0; s < stages; ++s) {
        __builtin_amdgcn_sched_barrier(0);
        step(integral_constant<int, 0>{}, [&](int t) {
          spread(t, kReads, 0, [&](int n) { read(a_at(s), b_at(s), 1, n); });
          spread(t, kLoads / 2, 1, [&](int l) { issue(std::false_type{}, s + kBufs - 1, kLoads / 2 + l); });
        });
        step(integral_constant<int, 1>{}, [&](int t) { spread(t, kReads, 0, [&](int n) { read(a_at(s), b_at(s), 2, n); }); });
        step(integral_constant<int, 2>{}, [&](int t) { spread(t, kReads, 0, [&](int n) { read(a_at(s), b_at(s), 3, n); }); });
        // with four buffers the loads of two later stages may be on their way
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "i"((kBufs - 2) * kLoads) : "memory");
        __syncthreads();
        advance();
        __builtin_amdgcn_sched_barrier(0);
        step(integral_constant<int, 3>{}, [&](int t) {
          spread(t, kReads, 0, [&](int n) { read(a_at(s + 1), b_at(s + 1), 0, n); });
          spread(t, kLoads / 2, 1, [&](int l) { issue(std::false_type{}, s + kBufs, l); });
        });
      }
    }
    // the loads past the last stage write LDS: they end before it is used again
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" : : : "memory");
    __syncthreads();
    const int64_t row0 = m0 + wm, col0 = n0 + (kProduct == kGated ? wn / 2 : wn), rows = a.M - row0, columns = a.N - col0;
    const bool whole = rows_a == kTileA && rows_n == kTileN;
    at_tile += slots;
    const bool more = at_tile < end_tile;
    if (more) {
      in_group += slots;
      while (in_group >= per_group) in_group -= per_group, ++group;
      tile_at(group, in_group);
    } else {
      sa.none(), sb.none(), sb2.none();  // the first loads of no tile read nothing
    }

    // The B rows come first in the instruction, so that a lane holds four
    // consecutive columns: D[row 8 q + 4 half + e][column lrow], q = r / 4, e =
    // r % 4.  A wave's LDS operations are carried out in their order and its patch is
    // its own, so nothing waits but the stores for what they store.
    // The lane's number comes anew for every tile: else the compiler computes all
    // addresses below before the first tile and has no registers left for them.
    int l = lane;
    asm volatile("" : "+v"(l));
    auto put = [&, lrow = l & 31, half = l >> 5](int turn, int i, int part) {
      char* to = patch + (turn & 1) * 32 * 128 + lrow * 128;
#pragma unroll
      for (int k = 0; k < kPer / 4; ++k)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x16& d = acc[i][part * (kPer / 4) + k];
          if constexpr (kF32)
            *reinterpret_cast<f32x4*>(to + 16 * ((2 * q + half) ^ swz(lrow))) =
                (f32x4){d[4 * q], d[4 * q + 1], d[4 * q + 2], d[4 * q + 3]};
          else
            *reinterpret_cast<u32x2*>(to + 16 * ((4 * k + q) ^ swz(lrow)) + 8 * (half ^ (lrow >> 4))) =
                (u32x2){pack_bf16(d[4 * q], d[4 * q + 1]), pack_bf16(d[4 * q + 2], d[4 * q + 3])};
        }
    };
    const int r = l >> 3;
    u32x4 out[2][4] = {};  // set, or else it is kept from tile to tile
    auto get = [&](int turn) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int row = 8 * x + r;
        const u32x4 v = *reinterpret_cast<const u32x4*>(patch + (turn & 1) * 32 * 128 + row * 128 + 16 * ((l & 7) ^ swz(row)));
        out[turn & 1][x] = !kF32 && x >= 2 ? (u32x4){v.z, v.w, v.x, v.y} : v;
      }
    };
    auto loads = [&](int t) {
#pragma unroll
      for (int n = kPerPiece * t; n < kPerPiece * (t + 1); ++n)
        if (n < kFirst) start(n);
    };
    auto store = [](char* to, const u32x4& v) { *reinterpret_cast<u32x4*>(to) = v; };
    if constexpr (kProduct == kGated) {
      // Gate and up go through LDS as they are; four lanes read a row of 32 columns of
      // both, eight columns a lane, and store y and what is kept of gate and up.
      auto put_pair = [&, lrow = l & 31, half = l >> 5](int t) {
        char* to = patch + (t & (kTurns - 1)) * kPieceBytes + lrow * 128;
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x16& d = acc[t / kPartsB][t % kPartsB + p * kPartsB];
            *reinterpret_cast<f32x4*>(to + p * 32 * 128 + 16 * ((2 * q + half) ^ swz(lrow))) =
                (f32x4){d[4 * q], d[4 * q + 1], d[4 * q + 2], d[4 * q + 3]};
          }
      };
      auto finish = [&](int t, auto whole) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int row = 16 * x + (l >> 2), down = 32 * (t / kPartsB) + row, column = 32 * (t % kPartsB) + 8 * (l & 3);
          const char* from = patch + (t & (kTurns - 1)) * kPieceBytes + row * 128;
          float g[8], u[8], y[8];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int at = 16 * ((2 * (l & 3) + c) ^ swz(row));
            const f32x4 gv = *reinterpret_cast<const f32x4*>(from + at), uv = *reinterpret_cast<const f32x4*>(from + 32 * 128 + at);
#pragma unroll
            for (int e = 0; e < 4; ++e) g[4 * c + e] = gv[e], u[4 * c + e] = uv[e];
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = silu_times(g[e], u[e]);
          auto pack8 = [](const float (&v)[8]) {
            return (u32x4){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
          };
          if (decltype(whole)::value || (down < rows && column < columns)) {  // H is a multiple of 8: whole chunks
            store(static_cast<char*>(a.C) + ((row0 + down) * a.N + col0 + column) * 2, pack8(y));
            if (kKeep) {
              char* const to = reinterpret_cast<char*>(a.gu) + ((row0 + down) * 2 * a.N + col0 + column) * 2;
              store(to, pack8(g));
              store(to + 2 * a.N, pack8(u));
            }
          }
        }
      };
      auto all_pieces = [&](auto whole) {
#pragma unroll
        for (int t = 0; t <= kPieces; ++t) {
          if (t < kPieces) loads(t);
          if (t < kPieces && kTurns == 2) put_pair(t);
          if (t > 0) finish(t - 1, whole);
          if (t < kPieces && kTurns == 1) put_pair(t);
          __builtin_amdgcn_sched_barrier(0);
        }
      };
      if (whole)
        all_pieces(std::true_type{});
      else
        all_pieces(std::false_type{});
    } else {
      // where a lane's chunk of row 0 goes
      char* const to0 = static_cast<char*>(a.C) + ((row0 + r) * a.N + col0 + kPer * (l & 7)) * (16 / kPer);
      auto place = [&](int block, int part, int x) { return to0 + (32 * block + 8 * x) * a.N * (16 / kPer) + 128 * part; };
      if (whole) {
#pragma unroll
        for (int t = 0; t < kPieces + 2; ++t) {
          loads(t);
          if (t < kPieces) put(t, t / kPartsB, t % kPartsB);
          if (t >= 2) {
#pragma unroll
            for (int x = 0; x < 4; ++x) store(place((t - 2) / kPartsB, (t - 2) % kPartsB, x), out[t & 1][x]);
          }
          if (t >= 1 && t <= kPieces) get(t - 1);
          __builtin_amdgcn_sched_barrier(0);
        }
      } else {
#pragma unroll
        for (int t = 0; t < kPieces; ++t) {
          loads(t);
          put(t, t / kPartsB, t % kPartsB);
          get(t);
          const int part = t % kPartsB, first = 32 * (t / kPartsB) + r;
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (first + 8 * x < rows && 8 * kPer * part + kPer * (l & 7) < columns)  // N is a multiple of 8: whole chunks
              store(place(t / kPartsB, part, x), out[t & 1][x]);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    if (!more) break;
    stored_whole = whole;
  }
  asm volatile("s_waitcnt vmcnt(0)" : : : "memory");  // nothing writes LDS after the workgroup's end
}

template <int kFA, int kFB, int kWavesB, int kBufs, Product kProduct, bool kKeep, bool kF32>
void launch_tile(GemmArgs a, int cus, hipStream_t stream) {
  using Shape = TileShape<kFA, kFB, kWavesB, kBufs, kProduct == kGated>;
  a.tiles_m = (int)((a.M + Shape::kTileA - 1) / Shape::kTileA);
  const int tile_n = kProduct == kGated ? Shape::kTileB / 2 : Shape::kTileB;
  a.tiles_n = (int)((a.N + tile_n - 1) / tile_n);
  const int per_xcd = (int)(((int64_t)a.tiles_m * a.tiles_n + 7) / 8);
  const dim3 grid(8 * std::min(per_xcd, std::max(1, cus / 8) * Shape::kPerCu), (unsigned)((a.K + a.split_k - 1) / a.split_k)), block(Shape::kThreads);
  hipLaunchKernelGGL((swiglu_tile_kernel<kFA, kFB, kWavesB, kBufs, kProduct, kKeep, kF32>), grid, block, 0, stream, a, per_xcd);
}

// ---- few rows: operands straight from memory into registers ----
//
// The gated product of up to 64 rows of x.  A workgroup owns 16 rows of Wg and the same
// of Wu; its waves take K 128 values at a time in turn, and their sums meet in LDS.
// Nothing is shared between waves, so nothing waits: the weight streams through
// once, 64 bytes of a row with each load, a line with two.  Rows past M or N are read
// as the last row and not stored.  Reading the weight bounds it: one row of 11008 x 4096
// (180 MB) takes 36.6 us, 4.9 TB/s, where a large copy moves 5.1.  Sixteen rows of Wg a
// workgroup make 688 workgroups of it; with 32 they were 344, and took half as long again.
constexpr int kStreamK = 128, kStreamWaves = 8;
template <int kBlocks, bool kKeep>  // kBlocks: 16 rows of x each
__global__ __launch_bounds__(64 * kStreamWaves) void swiglu_stream_kernel(const GemmArgs a) {
  static_assert(kBlocks <= kStreamWaves, "a wave stores a block");
  __shared__ f32x4 s_sum[kStreamWaves][kBlocks][2][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, kb = lane >> 4;
  const int64_t n0 = 16ll * blockIdx.x, row = n0 + r < a.N ? n0 + r : a.N - 1;
  const uint16_t* const from_g = a.B + row * a.ldb + 8 * kb;
  const uint16_t* const from_u = a.B + (a.N + row) * a.ldb + 8 * kb;
  const uint16_t* from_x[kBlocks];
#pragma unroll
  for (int b = 0; b < kBlocks; ++b) from_x[b] = a.A + std::min<int64_t>(16 * b + r, a.M - 1) * a.lda + 8 * kb;
  f32x4 gate[kBlocks] = {}, up[kBlocks] = {};
  auto chunk = [&](int64_t k0, auto whole) {
    u32x4 fg[4], fu[4], fx[kBlocks][4];
    auto load = [&](const uint16_t* p, int j) {
      if (decltype(whole)::value || k0 + 32 * j + 8 * kb < a.K) return *reinterpret_cast<const u32x4*>(p + k0 + 32 * j);  // K is a multiple of 8
      return (u32x4){0, 0, 0, 0};
    };
#pragma unroll
    for (int j = 0; j < 4; ++j) fg[j] = load(from_g, j), fu[j] = load(from_u, j);
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int j = 0; j < 4; ++j) fx[b][j] = load(from_x[b], j);
    // The weight's rows come first in the instruction: a lane holds four columns of C.
    auto mfma16 = [](const u32x4& a, const u32x4& b, const f32x4& c) {
      return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    };
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) gate[b] = mfma16(fg[j], fx[b][j], gate[b]), up[b] = mfma16(fu[j], fx[b][j], up[b]);
  };
  const int64_t whole = a.K / kStreamK;
  for (int64_t c = wave; c < whole; c += kStreamWaves) chunk(c * kStreamK, std::true_type{});
  if (a.K % kStreamK != 0 && whole % kStreamWaves == wave) chunk(whole * kStreamK, std::false_type{});
#pragma unroll
  for (int b = 0; b < kBlocks; ++b) s_sum[wave][b][0][lane] = gate[b], s_sum[wave][b][1][lane] = up[b];
  __syncthreads();
  if (wave >= kBlocks) return;
  f32x4 g = s_sum[0][wave][0][lane], u = s_sum[0][wave][1][lane];
#pragma unroll
  for (int v = 1; v < kStreamWaves; ++v) g += s_sum[v][wave][0][lane], u += s_sum[v][wave][1][lane];
  const int64_t m = 16 * wave + r, n = n0 + 4 * kb;
  if (m >= a.M || n >= a.N) return;
  f32x4 y;
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = silu_times(g[e], u[e]);
  auto pack4 = [](const f32x4& v) { return (u32x2){pack_bf16(v.x, v.y), pack_bf16(v.z, v.w)}; };
  *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.C) + m * a.N + n) = pack4(y);
  if (kKeep) {
    *reinterpret_cast<u32x2*>(a.gu + m * 2 * a.N + n) = pack4(g);
    *reinterpret_cast<u32x2*>(a.gu + m * 2 * a.N + a.N + n) = pack4(u);
  }
}

// ---- slices of K joined ----

// out = the sum of the slices' fp32 results, in their order (always the same: the
// results do not depend on timing); n values, a multiple of 8.
template <bool kF32>
__global__ __launch_bounds__(256) void swiglu_join_kernel(const float* part, void* out, int slices, int64_t n) {
  for (int64_t i = 4 * (blockIdx.x * 256ll + threadIdx.x); i < n; i += 4 * gridDim.x * 256ll) {
    f32x4 sum = *reinterpret_cast<const f32x4*>(part + i);
    for (int s = 1; s < slices; ++s) sum += *reinterpret_cast<const f32x4*>(part + s * n + i);
    if (kF32)
      *reinterpret_cast<f32x4*>(static_cast<float*>(out) + i) = sum;
    else
      *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(out) + i) = (u32x2){pack_bf16(sum.x, sum.y), pack_bf16(sum.z, sum.w)};
  }
}

// Zeros, where there is nothing to sum.
__global__ __launch_bounds__(256) void swiglu_zero_kernel(u32x4* p, int64_t n) {
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) p[i] = (u32x4){0, 0, 0, 0};
}
void launch_zero(void* p, int64_t bytes, hipStream_t stream) {  // a multiple of 16
  if (p && bytes > 0)
    hipLaunchKernelGGL(swiglu_zero_kernel, dim3((unsigned)std::min<int64_t>((bytes / 16 + 255) / 256, 1 << 16)), dim3(256), 0, stream,
                       static_cast<u32x4*>(p), bytes / 16);
}

template <Product kProduct, bool kKeep, bool kF32>
void launch_tiles(const GemmArgs& a, Plan::Tiles tiles, int cus, hipStream_t stream) {
  if (tiles == Plan::k256) return launch_tile<4, 4, 2, 3, kProduct, kKeep, kF32>(a, cus, stream);
  if constexpr (kProduct != kDw) {
    if (tiles == Plan::k64) return launch_tile<1, 2, 2, 4, kProduct, kKeep, kF32>(a, cus, stream);
  }
  if (tiles == Plan::k128Two) return launch_tile<2, 2, 2, 2, kProduct, kKeep, kF32>(a, cus, stream);
  launch_tile<2, 2, 2, 4, kProduct, kKeep, kF32>(a, cus, stream);
}

template <bool kKeep>
void launch_gated(const GemmArgs& a, int cus, hipStream_t stream) {
  if (a.K == 0) {
    launch_zero(a.C, 2 * a.M * a.N, stream);
    launch_zero(a.gu, 4 * a.M * a.N, stream);
    return;
  }
  if (const int blocks = streamed(a.M, a.N, a.K)) {
    const dim3 grid((unsigned)((a.N + 15) / 16)), block(64 * kStreamWaves);
    if (blocks == 1)
      hipLaunchKernelGGL((swiglu_stream_kernel<1, kKeep>), grid, block, 0, stream, a);
    else if (blocks == 2)
      hipLaunchKernelGGL((swiglu_stream_kernel<2, kKeep>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((swiglu_stream_kernel<4, kKeep>), grid, block, 0, stream, a);
    return;
  }
  launch_tiles<kGated, kKeep, false>(a, plan(a.M, 2 * a.N, a.K, false, false).tiles, cus, stream);
}

template <Product kProduct>
Plan plan_of(int64_t M, int64_t N, int64_t K) {
  return plan(M, N, K, kProduct == kDw, true);
}
int64_t slice_bytes(const Plan& p, int64_t M, int64_t N) { return p.slices > 1 ? 4 * p.slices * M * N : 0; }

template <Product kProduct>
void launch_product(GemmArgs a, bool f32, void* workspace, int cus, hipStream_t stream) {
  if (a.K == 0) return launch_zero(a.C, a.M * a.N * (f32 ? 4 : 2), stream);
  const Plan p = plan_of<kProduct>(a.M, a.N, a.K);
  if (p.slices == 1) {
    a.split_k = a.K;
    f32 ? launch_tiles<kProduct, false, true>(a, p.tiles, cus, stream) : launch_tiles<kProduct, false, false>(a, p.tiles, cus, stream);
    return;
  }
  void* const C = a.C;
  const int64_t n = a.M * a.N, stages = (a.K + kStageK - 1) / kStageK;
  a.C = workspace;
  a.split_k = (stages + p.slices - 1) / p.slices * kStageK;
  launch_tiles<kProduct, false, true>(a, p.tiles, cus, stream);
  const int slices = (int)((a.K + a.split_k - 1) / a.split_k);
  const dim3 grid((unsigned)std::min<int64_t>((n / 4 + 255) / 256, 1 << 16));
  if (f32)
    hipLaunchKernelGGL((swiglu_join_kernel<true>), grid, dim3(256), 0, stream, static_cast<const float*>(workspace), C, slices, n);
  else
    hipLaunchKernelGGL((swiglu_join_kernel<false>), grid, dim3(256), 0, stream, static_cast<const float*>(workspace), C, slices, n);
}

bool device_cus(int* cus) {
  int dev = 0;
  return hipGetDevice(&dev) == hipSuccess &&
         hipDeviceGetAttribute(cus, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess && *cus > 0;
}

constexpr int64_t kMaxT = int64_t(1) << 31, kMaxD = int64_t(1) << 20, kMaxH = int64_t(1) << 20;

bool sizes(int64_t T, int64_t H, int64_t D) {
  if (T < 0 || H < 0 || D < 0 || T > kMaxT || H > kMaxH || D > kMaxD || H % 8 != 0 || D % 8 != 0) return false;
  auto tiles = [](int64_t a, int64_t b) { return ((a + 63) / 64) * ((b + 63) / 64); };  // counted in 32 bits
  return tiles(T, 2 * H) <= int64_t(1) << 30 && tiles(T, D) <= int64_t(1) << 30 && tiles(2 * H, D) <= int64_t(1) << 30;
}

int launched() { return hipGetLastError() == hipSuccess ? SILUQUANT_OK : SILUQUANT_ERR_LAUNCH_FAILED; }

}  // namespace

hipError_t code_objects::load_swiglugemm() { return load(swiglu_gate_bwd_kernel); }

extern "C" {

__attribute__((visibility("default"))) int swiglu_gemm(const void* x, const void* w, void* y, void* gu, int64_t T,
                                                       int64_t H, int64_t D, hipStream_t stream) {
  if (!sizes(T, H, D)) return SILUQUANT_ERR_BAD_SHAPE;
  if (T == 0 || H == 0) return SILUQUANT_OK;
  if (!y || (D > 0 && (!x || !w))) return SILUQUANT_ERR_NULL_PTR;
  if (misaligned(x, 16) || misaligned(w, 16) || misaligned(y, 16) || misaligned(gu, 16)) return SILUQUANT_ERR_MISALIGNED;
  const Span in[2] = {{x, 2 * T * D}, {w, 4 * H * D}}, out[2] = {{y, 2 * T * H}, {gu, 4 * T * H}};
  for (const Span& o : out)
    for (const Span& i : in)
      if (overlap(o, i)) return SILUQUANT_ERR_OVERLAP;
  if (overlap(out[0], out[1])) return SILUQUANT_ERR_OVERLAP;
  int cus = 0;
  if (!device_cus(&cus)) return SILUQUANT_ERR_DEVICE;
  const GemmArgs a = {static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(w), y, static_cast<uint16_t*>(gu), T, H, D,
                      (int)D, (int)D, 0, 0, D};
  gu ? launch_gated<true>(a, cus, stream) : launch_gated<false>(a, cus, stream);
  return launched();
}

__attribute__((visibility("default"))) int64_t swiglu_gemm_bwd_workspace_bytes(int64_t T, int64_t H, int64_t D) {
  if (!sizes(T, H, D)) return -1;
  if (T == 0 || H == 0 || D == 0) return 0;
  return std::max(slice_bytes(plan_of<kDx>(T, D, 2 * H), T, D), slice_bytes(plan_of<kDw>(2 * H, D, T), 2 * H, D));
}

__attribute__((visibility("default"))) int swiglu_gemm_bwd(const void* dy, const void* gu, const void* x, const void* w,
                                                           void* d_gu, void* dx, int dx_dtype, void* dw, int dw_dtype,
                                                           void* workspace, int64_t workspace_bytes, int64_t T, int64_t H,
                                                           int64_t D, hipStream_t stream) {
  if (!sizes(T, H, D) || (dx_dtype != SILUQUANT_F32 && dx_dtype != SILUQUANT_BF16) ||
      (dw_dtype != SILUQUANT_F32 && dw_dtype != SILUQUANT_BF16))
    return SILUQUANT_ERR_BAD_SHAPE;
  const bool dx32 = dx_dtype == SILUQUANT_F32, dw32 = dw_dtype == SILUQUANT_F32;
  const bool some = T > 0 && H > 0;
  if (T == 0 || D == 0) dx = nullptr;
  if (H == 0 || D == 0) dw = nullptr;
  if (!some && !dx && !dw) return SILUQUANT_OK;
  const int64_t need = dx || dw ? swiglu_gemm_bwd_workspace_bytes(T, H, D) : 0;
  // what is not needed is not looked at
  if (!dx) w = nullptr;
  if (!dw) x = nullptr;
  if (need == 0) workspace = nullptr, workspace_bytes = 0;
  if ((some && (!dy || !gu || !d_gu)) || (dw && T > 0 && !x) || (dx && H > 0 && !w) || (need > 0 && !workspace))
    return SILUQUANT_ERR_NULL_PTR;
  if (workspace_bytes < need) return SILUQUANT_ERR_BAD_SHAPE;
  if (misaligned(dy, 16) || misaligned(gu, 16) || misaligned(x, 16) || misaligned(w, 16) || misaligned(d_gu, 16) ||
      misaligned(dx, 16) || misaligned(dw, 16) || misaligned(workspace, 16))
    return SILUQUANT_ERR_MISALIGNED;
  const Span in[4] = {{dy, 2 * T * H}, {gu, 4 * T * H}, {x, 2 * T * D}, {w, 4 * H * D}};
  const Span out[4] = {{d_gu, 4 * T * H}, {dx, T * D * (dx32 ? 4 : 2)}, {dw, 2 * H * D * (dw32 ? 4 : 2)}, {workspace, need}};
  for (int o = 0; o < 4; ++o) {
    for (int i = 0; i < 4; ++i)
      if (overlap(out[o], in[i]) && !(o == 0 && i == 1 && d_gu == gu)) return SILUQUANT_ERR_OVERLAP;
    for (int i = 0; i < o; ++i)
      if (overlap(out[o], out[i])) return SILUQUANT_ERR_OVERLAP;
  }
  int cus = 0;
  if (!device_cus(&cus)) return SILUQUANT_ERR_DEVICE;
  uint16_t* d = static_cast<uint16_t*>(d_gu);
  if (some) {
    const GateArgs a = {static_cast<const uint16_t*>(dy), static_cast<const uint16_t*>(gu), d, T, (int)H};
    const int64_t groups = (T * (H / 8) + 255) / 256;
    hipLaunchKernelGGL(swiglu_gate_bwd_kernel, dim3((unsigned)std::min<int64_t>(groups, 1 << 20)), dim3(256), 0, stream, a);
  }
  if (dx)
    launch_product<kDx>({d, static_cast<const uint16_t*>(w), dx, nullptr, T, D, 2 * H, (int)(2 * H), (int)D, 0, 0, 0}, dx32, workspace,
                        cus, stream);
  if (dw)
    launch_product<kDw>({d, static_cast<const uint16_t*>(x), dw, nullptr, 2 * H, D, T, (int)(2 * H), (int)D, 0, 0, 0}, dw32, workspace,
                        cus, stream);
  return launched();
}

}  // extern "C"
