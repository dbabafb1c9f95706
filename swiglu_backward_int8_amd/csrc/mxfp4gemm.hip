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
      for (int i = 0; i < left; ++i) p[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
  } else {
    float* p = static_cast<float*>(C) + at;
    if (left >= 4) {
      *reinterpret_cast<f32x4_a4*>(p) = v;
    } else {
      for (int i = 0; i < left; ++i) p[i] = v[i];
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
  if (M <= 16)
    launch_stream<1, 1, 8>(a, bf16, stream);
  else if (M <= 64)
    launch_stream<2, 2, 8>(a, bf16, stream);
  else
    launch_stream<4, 4, 4>(a, bf16, stream);
  return hipGetLastError() == hipSuccess ? SILUQUANT_OK : SILUQUANT_ERR_LAUNCH_FAILED;
}

}  // extern "C"
