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

namespace {

using namespace rows;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// The sigmoid s = 1 / (1 + exp(-g)) in parts that neither overflow nor lose small
// values: with h = exp(-|g| / 2) and r = 1 / (1 + h^2), s is r for g >= 0 and h^2 r
// below, and 1 - s the other way round; what a value is multiplied by h^2 for goes
// through h twice (h^2 alone is 0 from g = -104 on, and has few bits before).  Off
// by some 1e-7 of itself: for what is rounded to bf16 once, behind it.
struct Sigmoid {
  float h, r;
  bool below;
  __device__ __forceinline__ explicit Sigmoid(float g) {
    h = __builtin_amdgcn_exp2f(-0.72134752044f * __builtin_fabsf(g));  // log2(e) / 2
    r = __builtin_amdgcn_rcpf(__builtin_fmaf(h, h, 1.0f));
    below = g < 0.0f;
  }
  __device__ __forceinline__ float times(float v) const { return (below ? (v * h) * h : v) * r; }  // v * s
  __device__ __forceinline__ float rest() const { return (below ? 1.0f : h * h) * r; }             // 1 - s
};

// The same to the last bit or so, for |g| up to 80: the exponent's argument in two
// parts, the reciprocal corrected once.  d_gu is an operand of two products, and an
// error of 1e-7 rounds one value in ten thousand to its other neighbour in bf16.
struct NearSigmoid {
  float e, r;
  bool below;
  static constexpr float kMost = 80.0f;
  __device__ __forceinline__ explicit NearSigmoid(float g) {
    constexpr float kHi = -1.44269504088896341f, kLo = (float)(-1.44269504088896341 - (double)kHi), kLn2 = 0.69314718056f;
    const float a = __builtin_fabsf(g), t = a * kHi;
    const float rest = __builtin_fmaf(a, kLo, __builtin_fmaf(a, kHi, -t));
    e = __builtin_amdgcn_exp2f(t);
    e = __builtin_fmaf(e, rest * kLn2, e);
    const float d = 1.0f + e;
    r = __builtin_amdgcn_rcpf(d);
    r = __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
    below = g < 0.0f;
  }
  __device__ __forceinline__ float times(float v) const { return v * (below ? e * r : r); }
  __device__ __forceinline__ float rest() const { return below ? r : e * r; }
};

// ---- d_gu ----

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
    auto grads = [&](auto sigmoid) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const decltype(sigmoid) s(g[k]);
        dg[k] = s.times(d[k] * u[k]) * __builtin_fmaf(g[k], s.rest(), 1.0f);
        du[k] = d[k] * s.times(g[k]);
      }
    };
    float top = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = __builtin_fmaxf(top, __builtin_fabsf(g[k]));
    if (__any(top > NearSigmoid::kMost))
      grads(Sigmoid(0.0f));
    else
      grads(NearSigmoid(0.0f));
    auto pack8 = [](const float (&v)[8]) {
      return Piece{{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])}};
    };
    store_bf16<kFull, false>(a.d_gu + 2 * t * a.H + col, pack8(dg), 8);
    store_bf16<kFull, false>(a.d_gu + 2 * t * a.H + a.H + col, pack8(du), 8);
  }
}

// ---- products ----

// C [M, N] = sum over k of A[m, k] * B[n, k].  A k-major operand is stored as [K,
// rows]; the others as [rows, K].  ld: elements from one stored row to the next.
struct GemmArgs {
  const uint16_t *A, *B, *B2;  // B2: the up projection's rows (forward)
  void* C;
  uint16_t* gu;  // forward: [M, 2N], may be null
  int64_t M, N, K;
  int64_t lda, ldb;
};

constexpr int kStep = 32, kPitch = kStep + 8;  // values of K per step; a row in LDS

template <bool kKMajor>
__device__ __forceinline__ void stage(uint16_t* to, const uint16_t* from, int64_t ld, int64_t row0, int64_t rows, int64_t k0,
                                      int64_t K) {
  for (int i = threadIdx.x; i < 64 * kStep; i += 256) {
    const int r = kKMajor ? i & 63 : i / kStep, k = kKMajor ? i >> 6 : i % kStep;
    uint16_t v = 0;
    if (row0 + r < rows && k0 + k < K) v = kKMajor ? from[(k0 + k) * ld + row0 + r] : from[(row0 + r) * ld + k0 + k];
    to[r * kPitch + k] = v;
  }
}

template <bool kAk, bool kBk, bool kGated, bool kF32>
__global__ __launch_bounds__(256) void swiglu_simple_kernel(const GemmArgs a) {
  __shared__ __attribute__((aligned(16))) uint16_t s_a[64 * kPitch], s_b[(kGated ? 2 : 1) * 64 * kPitch];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32, lrow = lane & 31, half = lane >> 5;
  const int64_t tiles_n = (a.N + 63) / 64;
  const int64_t m0 = blockIdx.x / tiles_n * 64, n0 = blockIdx.x % tiles_n * 64;
  f32x16 acc = {}, up = {};
  for (int64_t k0 = 0; k0 < a.K; k0 += kStep) {
    stage<kAk>(s_a, a.A, a.lda, m0, a.M, k0, a.K);
    stage<kBk>(s_b, a.B, a.ldb, n0, a.N, k0, a.K);
    if (kGated) stage<kBk>(s_b + 64 * kPitch, a.B2, a.ldb, n0, a.N, k0, a.K);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kStep; j += 16) {
      const bf16x8 fa = *reinterpret_cast<const bf16x8*>(s_a + (wm + lrow) * kPitch + j + 8 * half);
      const bf16x8 fb = *reinterpret_cast<const bf16x8*>(s_b + (wn + lrow) * kPitch + j + 8 * half);
      acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb, fa, acc, 0, 0, 0);
      if (kGated) {
        const bf16x8 fu = *reinterpret_cast<const bf16x8*>(s_b + (64 + wn + lrow) * kPitch + j + 8 * half);
        up = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fu, fa, up, 0, 0, 0);
      }
    }
    __syncthreads();
  }
  const int64_t m = m0 + wm + lrow;
  auto one = [](float v) { return (uint16_t)pack_bf16(v, 0.0f); };
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int64_t n = n0 + wn + 8 * (r / 4) + 4 * half + r % 4;
    if (m >= a.M || n >= a.N) continue;
    if (kGated) {
      static_cast<uint16_t*>(a.C)[m * a.N + n] = one(Sigmoid(acc[r]).times(acc[r]) * up[r]);
      if (a.gu) a.gu[m * 2 * a.N + n] = one(acc[r]), a.gu[m * 2 * a.N + a.N + n] = one(up[r]);
    } else if (kF32) {
      static_cast<float*>(a.C)[m * a.N + n] = acc[r];
    } else {
      static_cast<uint16_t*>(a.C)[m * a.N + n] = one(acc[r]);
    }
  }
}

template <bool kAk, bool kBk, bool kGated>
void launch_product(const GemmArgs& a, bool f32, hipStream_t stream) {
  const dim3 grid((unsigned)(((a.M + 63) / 64) * ((a.N + 63) / 64))), block(256);
  if (f32)
    hipLaunchKernelGGL((swiglu_simple_kernel<kAk, kBk, kGated, true>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((swiglu_simple_kernel<kAk, kBk, kGated, false>), grid, block, 0, stream, a);
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
  const uint16_t* wg = static_cast<const uint16_t*>(w);
  launch_product<false, false, true>({static_cast<const uint16_t*>(x), wg, wg + H * D, y, static_cast<uint16_t*>(gu), T, H, D, D, D},
                                     false, stream);
  return launched();
}

__attribute__((visibility("default"))) int64_t swiglu_gemm_bwd_workspace_bytes(int64_t T, int64_t H, int64_t D) {
  return sizes(T, H, D) ? 0 : -1;
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
  const int64_t need = swiglu_gemm_bwd_workspace_bytes(T, H, D);
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
  uint16_t* d = static_cast<uint16_t*>(d_gu);
  if (some) {
    const GateArgs a = {static_cast<const uint16_t*>(dy), static_cast<const uint16_t*>(gu), d, T, (int)H};
    const int64_t groups = (T * (H / 8) + 255) / 256;
    hipLaunchKernelGGL(swiglu_gate_bwd_kernel, dim3((unsigned)std::min<int64_t>(groups, 1 << 20)), dim3(256), 0, stream, a);
  }
  if (dx)
    launch_product<false, true, false>({d, static_cast<const uint16_t*>(w), nullptr, dx, nullptr, T, D, 2 * H, 2 * H, D}, dx32, stream);
  if (dw)
    launch_product<true, true, false>({d, static_cast<const uint16_t*>(x), nullptr, dw, nullptr, 2 * H, D, T, 2 * H, D}, dw32, stream);
  return launched();
}

}  // extern "C"
