/*
 * libsiluquant -- fused SwiGLU forward recompute, SwiGLU backward and
 * two-axis int8 quantisation for AMD Instinct MI355X (gfx950).
 *
 * The operation is the one the page "kernelgen-challenge-9-task3-silu-quant"
 * (githubhelp.com) defines: its entry-point listing gives the name and the
 * argument order, its two output bullets give the outputs, and its list of
 * design constraints gives the 128 x 128 tiling, the bf16 round trip before
 * quantising and the multiplication by a precomputed inverse scale.
 *
 * Plain C ABI: pointers and sizes only.  Device pointers are HIP device (or
 * managed) memory on the current HIP device; `stream` is a hipStream_t (NULL =
 * the null stream).  The library allocates nothing, keeps no state between
 * calls and never waits on a stream: every call checks its arguments, asks
 * the runtime for the current device's compute-unit count, enqueues its
 * kernels and returns, so a call may be captured into a HIP graph, the first
 * call of a process included.
 */
#ifndef SILUQUANT_H
#define SILUQUANT_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* The HIP runtime's stream handle, declared as the runtime declares it so
 * that this header needs no HIP header (repeating the typedef is allowed). */
typedef struct ihipStream_t* hipStream_t;

/* Status codes.  Every argument check runs on the host before any HIP call,
 * so a call that returns one of the first five codes has touched neither the
 * device nor any buffer. */
enum siluquant_status {
  SILUQUANT_OK = 0,
  SILUQUANT_ERR_NULL_PTR = 1,      /* a buffer pointer is NULL while T*H > 0 */
  SILUQUANT_ERR_BAD_SHAPE = 2,     /* T < 0, H < 0, too large, H not a multiple of 32 (q8_1 blocks)
                                      or K not a multiple of the group (GEMM) */
  SILUQUANT_ERR_BAD_GROUP = 3,     /* a group size the entry point does not take */
  SILUQUANT_ERR_MISALIGNED = 4,    /* x, grad_y, grad_input_q, y_q_t not 16-byte aligned,
                                      or a scale buffer not 4-byte aligned */
  SILUQUANT_ERR_OVERLAP = 5,       /* two buffers share bytes */
  SILUQUANT_ERR_DEVICE = 6,        /* a HIP runtime call failed (no current device, or the
                                      device query failed) */
  SILUQUANT_ERR_LAUNCH_FAILED = 7, /* the kernel launch reported an error */
};

/*
 * silu_dot_fwd_bwd_quant_fuse -- one fused pass.
 *
 * Inputs (read only):
 *   x       bf16 [T, 2H] row-major; columns [0, H) are gate, [H, 2H) are up.
 *   grad_y  bf16 [T, H]  row-major; the gradient of y = silu(gate) * up.
 * Outputs (fully overwritten; every element written):
 *   grad_input_q  int8 [T, 2H]       [d_gate | d_up] quantised per row, in groups of
 *                                    128 consecutive positions of the 2H-long row
 *                                    (the last group of a row has the 2H % 128
 *                                    positions that remain);
 *   grad_input_s  fp32 [T, ceil(2H/128)]  one scale per such group;
 *   y_q_t         int8 [H, T]        y transposed, quantised in groups of 128
 *                                    consecutive tokens along each row (the last
 *                                    group of a T that is not a multiple of 128
 *                                    has the T % 128 tokens that remain);
 *   y_s_t         fp32 [H, ceil(T/128)]  one scale per such group.
 * Arithmetic: fp32 throughout, no fused multiply-add.  s = 1 / (1 + exp(-g)) with
 * exp(-g) correctly rounded to fp32; y = (g*s)*u;
 * d_gate = ((d*u)*s) * (1 + g*(1 - s)); d_up = d*(g*s); each rounded to bf16
 * (nearest, ties to even) before quantising.  Per group: amax over the bf16
 * values, scale = amax/127 (1.0 when amax == 0), inv = 1/scale (fp32),
 * p = v*inv (one fp32 multiplication), q = clamp(rne(p), -127, 127) (nearest
 * integer, ties to even), with q = 0 for v == 0.
 *   -128 is never produced.  Inputs must be finite and keep y, d_gate and d_up
 *   finite.
 * Group size: `group` is 128 (the page's default), 64 or 32; the scale tensors
 *   are then grad_input_s fp32 [T, ceil(2H/group)] and y_s_t fp32
 *   [H, ceil(T/group)].  When H is not a multiple of `group`, the group at
 *   row position group * floor(H/group) holds the last H % group channels of
 *   d_gate and the first channels of d_up.  Any other group returns
 *   SILUQUANT_ERR_BAD_GROUP.
 * Sizes: any T >= 0 and H >= 0 (T == 0 or H == 0 is a no-op that returns
 *   SILUQUANT_OK), T <= 2^23, H <= 2^22.  y_q_t is written with 16-byte
 *   stores when T % 16 == 0; other T work, with narrower stores.  The results
 *   do not depend on the kernel that runs: H a multiple of `group` takes the
 *   tiled kernel; other multiples of 8 above 128 a tiled kernel that walks
 *   runs of channel blocks and hands each block's d_up to the shifted d_up
 *   groups (below 128, two work items per tile); H not a multiple of 8 (rows
 *   then start off 16 bytes) a tiled kernel over 128-position tiles of the
 *   2H-long row [d_gate | d_up] that loads aligned 16-byte pieces and shifts
 *   them across lanes (slower: d_up is computed in tiles of its own).
 * Ownership: the caller allocates and owns every buffer; the library keeps no
 *   pointer after the call returns.  Buffers must not overlap.
 * Asynchrony: the work is enqueued on `stream` and the call returns without
 *   waiting; outputs are valid once the stream reaches this point.  The
 *   kernels' 31 KB sigmoid table is constant data of the library's code
 *   object, so no call builds, allocates or waits for anything.
 * Returns a siluquant_status code.
 */
int silu_dot_fwd_bwd_quant_fuse(const void* x, const void* grad_y, int8_t* grad_input_q, float* grad_input_s,
                                int8_t* y_q_t, float* y_s_t, int64_t T, int64_t H, int64_t group,
                                hipStream_t stream);

/*
 * silu_dot_fwd_bwd_quant_fuse_fp8 -- the same pass with FP8 codes.
 *
 * The pages name an fp8 quantise kernel among the benchmarked ops (the AstrAI
 * commit page, csrc/bench, its list of added benchmarks) without fixing its
 * format; the format here is OCP FP8 E4M3 (the OCP 8-bit floating point
 * specification: bias 7, no infinities, largest finite 448, subnormals
 * k * 2^-9), which gfx950 converts to in hardware.
 *
 * Arguments, layouts, sizes, ownership, asynchrony and status codes are those
 * of silu_dot_fwd_bwd_quant_fuse; the recomputation of y and of the gradients
 * and the bf16 round trip are identical.  Only the code format differs:
 *   grad_input_q  uint8 [T, 2H] E4M3 bit patterns, per-row 128-channel groups;
 *   y_q_t         uint8 [H, T]  E4M3 bit patterns, 128-token groups;
 *   scale = amax/448 (fp32 division; 1.0 when amax == 0), inv = 1/scale (fp32);
 *   code = E4M3(v * inv) where v * inv is the fp32 product and the conversion
 *   rounds to nearest, ties to even; magnitudes above 448 (only reachable when
 *   inv overflows to infinity for a group of subnormal scale) saturate to
 *   +-448 (0x7E / 0xFE); a zero v gives the zero of its own sign (0x00 / 0x80).
 *   NaN codes (0x7F, 0xFF) are never produced.
 */
int silu_dot_fwd_bwd_quant_fuse_fp8(const void* x, const void* grad_y, void* grad_input_q, float* grad_input_s,
                                    void* y_q_t, float* y_s_t, int64_t T, int64_t H, int64_t group, hipStream_t stream);

/*
 * silu_fwd_quant -- forward SwiGLU with row-wise int8 group quantisation.
 *
 * The fused launch shape of kquant_swiglu_q8_1_rows on the page "kquant_mmq.rs"
 * (docs.atlascybernetics.ai): y = bf16((silu(gate) * up) * w[t]) rounded once to
 * bf16 (nearest, ties to even), then quantised per row in groups of `group`
 * (128, 64 or 32) contiguous channels exactly as above (scale = amax/127, 1.0 for an all-zero
 * group; q = clamp(rne(v * inv)), v == 0 -> 0).  With no row weight, y is the
 * same bf16 value the backward pass recomputes.  The page's `limit` argument
 * has no stated meaning and is not provided.
 *
 *   x           bf16 [T, 2H] as above (read only; 16-byte aligned)
 *   row_weight  fp32 [T], or NULL for weight 1 (4-byte aligned)
 *   y_q         int8 [T, H]       codes (16-byte aligned)
 *   y_s         fp32 [T, ceil(H/group)] one scale per group (4-byte aligned)
 *   y_bf16      bf16 [T, H] the rounded y, or NULL (16-byte aligned)
 * Sizes: any T >= 0 (T <= 2^31), any H >= 0 (H <= 2^22); the last group of a
 *   row has the H % group channels that remain when H is not a multiple of
 *   the group.  H not a multiple of 8 (rows off 16 bytes) loads aligned
 *   pieces and shifts them across lanes, and is slower; long rows of that
 *   kind go a token row x 512 channels per wave.
 * Same ownership, asynchrony and error conventions as above.
 */
int silu_fwd_quant(const void* x, const float* row_weight, int8_t* y_q, float* y_s, void* y_bf16, int64_t T,
                   int64_t H, int64_t group, hipStream_t stream);

/*
 * silu_fwd_quant_q8_1 -- the forward quantiser in the page's q8_1 block layout.
 *
 * The page "kquant_mmq.rs" (docs.atlascybernetics.ai) writes the fused
 * swiglu rows as block_q8_1: per 32 channels, 32 int8 codes and a half2
 * (d, sum), 36 bytes.  y is computed and quantised exactly as silu_fwd_quant
 * with group 32; the block holds, in this order (the page gives the content
 * and size, not the order):
 *   bytes 0-1   d    the group's fp32 scale (amax/127, 1.0 for an all-zero
 *                    group) rounded to IEEE binary16 (nearest, ties to even)
 *   bytes 2-3   sum  fl32(scale * sum of the 32 codes) rounded to binary16:
 *                    the block's values as its codes give them
 *   bytes 4-35  the 32 codes, channel order
 * both halves little-endian.  d overflows to infinity for scales past 65504
 * (|y| above about 8.3e6) and is 0 below 2^-25: the format's range.
 *
 *   x           bf16 [T, 2H] as above (read only; 16-byte aligned)
 *   row_weight  fp32 [T], or NULL for weight 1 (4-byte aligned)
 *   y_q8        uint8 [T, (H/32) * 36] the blocks (4-byte aligned)
 * Sizes: any T >= 0 (T <= 2^28), H a multiple of 32 (H <= 2^22).
 * Same ownership, asynchrony and error conventions as above.
 */
int silu_fwd_quant_q8_1(const void* x, const float* row_weight, void* y_q8, int64_t T, int64_t H, hipStream_t stream);

/*
 * kquant_swiglu_q8_1_rows -- the same forward quantiser in the argument shape
 * of the page's fused launch.
 *
 * The page "kquant_mmq.rs" (docs.atlascybernetics.ai) documents
 * kquant_swiglu_q8_1_rows: separate gate and up inputs, an optional weight
 * per row, and two outputs, h = bf16(swiglu(gate, up) * w[row]) and the
 * block_q8_1 blocks of h, byte-identical to the swiglu launch followed by the
 * q8_1 launch.  Here h and the blocks are exactly those of silu_fwd_quant_q8_1
 * (with y_bf16) on x = [gate | up]:
 *   gate, up  bf16 [rows, inter] row-major (read only; 16-byte aligned; they
 *             may share memory with each other)
 *   w         fp32 [rows], or NULL for weight 1 (4-byte aligned)
 *   h_bf16    bf16 [rows, inter] the rounded h, or NULL (16-byte aligned)
 *   out_q8    uint8 [rows, (inter/32) * 36] the blocks (4-byte aligned)
 * Sizes: any rows >= 0 (rows <= 2^28), inter a multiple of 32 (the page's
 *   check), inter <= 2^22.  The page's `limit` argument has no stated meaning
 *   and is not provided.  Outputs must not overlap any other buffer.
 * Same ownership, asynchrony and error conventions as above.
 */
int kquant_swiglu_q8_1_rows(const void* gate, const void* up, const float* w, void* h_bf16, void* out_q8,
                            int64_t rows, int64_t inter, hipStream_t stream);

/*
 * i8_gemm_group_scaled -- the consumer of the two quantised layouts.
 *
 * The fusion bullet of the page "kernelgen-challenge-9-task3-silu-quant"
 * names the K-group and M-group quantisations: groups of 128 along the
 * contraction axis of the GEMM that reads each product.  This is that GEMM, on
 * the matrix cores (v_mfma_i32_32x32x32_i8):
 *   C[m, n] = sum_g sA[m, g] * sB[n / Bb, g] * sum_{k in group g} A[m, k] * B[n, k]
 *   A  int8 [M, K] row-major (16-byte aligned), sA fp32 [M, K/group];
 *   B  int8 [N, K] row-major (16-byte aligned), sB fp32 [ceil(N/Bb), K/group];
 *   Bb = b_rows_per_scale: 1 (a scale per row of B and group, as y_s_t) or 128
 *        (one per 128 x 128 block of B, a pre-quantised weight);
 *   C  [M, N] row-major, fp32 (c_dtype SILUQUANT_GEMM_OUT_F32, 4-byte aligned)
 *      or bf16 (SILUQUANT_GEMM_OUT_BF16, 2-byte aligned), fully overwritten.
 * Uses: dgrad dX[T, D] = grad_input_q[T, 2H] . Wt[D, 2H]^T (sA = grad_input_s,
 *   Wt the gate/up weight transposed and quantised in 128 x 128 blocks, Bb =
 *   128); wgrad dW[D, H] = go_q_t[D, T] . y_q_t[H, T]^T (sB = y_s_t, Bb = 1).
 * Arithmetic: each group's integer dot is exact (int32); the groups are
 *   accumulated in ascending order as acc = fma(float(dot), sA * sB, acc) in
 *   fp32; bf16 output rounds that once (nearest, ties to even).
 * Group: `group` is 128, 64 or 32 (the pass's group sizes); sA is then
 *   [M, K/group] and sB [ceil(N/Bb), K/group].
 * Sizes: any M, N >= 0 (M == 0 or N == 0 is a no-op), K >= 0 a multiple of
 *   the group (K == 0 writes zeros), K <= 2^22.  Same ownership, asynchrony and status conventions
 *   as above; C must not overlap an input.
 */
enum siluquant_gemm_out { SILUQUANT_GEMM_OUT_F32 = 0, SILUQUANT_GEMM_OUT_BF16 = 1 };
int i8_gemm_group_scaled(const int8_t* A, const float* sA, const int8_t* B, const float* sB, void* C, int64_t M,
                         int64_t N, int64_t K, int64_t group, int64_t b_rows_per_scale, int c_dtype, hipStream_t stream);

/* ---- the norm before the products, and the microscaled 4-bit format ----
 *
 * The operators below follow the conventions above: row-major contiguous
 * tensors, buffers owned by the caller, nothing allocated, no state, every
 * check on the host before any launch, work enqueued on `stream`. */

/* Element types and code formats. */
enum siluquant_dtype { SILUQUANT_F32 = 0, SILUQUANT_BF16 = 1 };
enum siluquant_code_format { SILUQUANT_CODE_INT8 = 0, SILUQUANT_CODE_E4M3 = 1 };

/*
 * rms_norm_quant -- root-mean-square norm with the residual's addition, its
 * output quantised by row groups: in int8 the operand of i8_gemm_group_scaled;
 * E4M3 codes are for a product of the caller's (the library has none) or for
 * group_dequant.
 *
 *   h[t, d]  = bf16(x[t, d] + residual[t, d])        (one fp32 addition)
 *   rstd[t]  = 1 / sqrt(sum_d h[t, d]^2 / D + eps)   (fp32)
 *   y[t, d]  = bf16((h[t, d] * rstd[t]) * weight[d])
 *   codes and scales of y by groups of `group` channels of a row, as
 *   silu_fwd_quant (int8) or silu_dot_fwd_bwd_quant_fuse_fp8 (E4M3) quantises.
 *
 *   x         bf16 or fp32 [T, D] by x_dtype (SILUQUANT_BF16 / _F32: both
 *             output types of the products)
 *   residual  bf16 [T, D], or NULL for none
 *   weight    bf16 [D]
 *   y_q       int8 or E4M3 codes [T, D] by code_format, or NULL for none
 *   y_s       fp32 [T, ceil(D/group)], NULL together with y_q
 *   y_bf16    bf16 [T, D] the y that is quantised, or NULL (y_q and y_bf16 may
 *             not both be NULL)
 *   h         bf16 [T, D] the new residual stream, or NULL; may be `residual`
 *             itself (updated in place), no other overlap is taken
 *   rstd      fp32 [T], or NULL: what rms_norm_bwd needs
 *   All but y_s and rstd (4 bytes) are 16-byte aligned.
 * Sizes: T <= 2^31, D <= 2^22, any D (the last group of a row may be short);
 *   T == 0 or D == 0 is a no-op.  group: 128, 64 or 32.  eps: finite, >= 0 (a
 *   row of zeros with eps == 0 gives NaN).
 * y that is not finite shows in its group's scale: NaN where the group's y holds
 * a NaN, +infinity where it holds an infinity and no NaN (a weight that is, or a
 * product past bf16's range); the group's codes then mean nothing.  A NaN in a
 * row of h makes all of the row's y NaN, an infinity its own place alone (rstd
 * is 0 and the rest of the row too).  Other groups, and other rows, are not
 * affected.
 */
int rms_norm_quant(const void* x, int x_dtype, const void* residual, const void* weight, void* y_q, float* y_s,
                   void* y_bf16, void* h, float* rstd, int64_t T, int64_t D, int64_t group, int code_format, float eps,
                   hipStream_t stream);

/*
 * rms_norm_bwd -- the gradients of that norm (quantising passes the gradient
 * through unchanged).  With n = h * rstd and g = dy * weight:
 *
 *   dx[t, d] = bf16(rstd[t] * (g[t, d] - n[t, d] * sum_d(g * n) / D) + d_h[t, d])
 *   dw[d]    = sum_t dy[t, d] * n[t, d]
 *
 * dx is the gradient for x and for residual alike.
 *   dy      bf16 or fp32 [T, D] by dy_dtype (the dgrad product's two outputs)
 *   h, rstd, weight   as rms_norm_quant wrote and read them
 *   d_h     bf16 [T, D] the gradient that reaches h by other ways (the residual
 *           stream), or NULL; dx may be d_h itself
 *   dx      bf16 [T, D];  dw  fp32 [D], or NULL where the weight is not trained
 *   workspace  rms_norm_bwd_workspace_bytes(T, D) bytes, 16-byte aligned; only
 *           looked at when dw is wanted or D > 16384.  Its contents before and
 *           after a call mean nothing.  The sums do not depend on timing.
 * Sizes as above; T == 0 writes zeros to dw.  A workspace that is too small
 * returns SILUQUANT_ERR_BAD_SHAPE.
 */
int64_t rms_norm_bwd_workspace_bytes(int64_t T, int64_t D);
int rms_norm_bwd(const void* dy, int dy_dtype, const void* h, const void* weight, const float* rstd, const void* d_h,
                 void* dx, float* dw, void* workspace, int64_t workspace_bytes, int64_t T, int64_t D,
                 hipStream_t stream);

/*
 * mxfp4_quant -- bf16 rows as microscaled 4-bit codes (OCP MX, MXFP4).
 *
 * A block is 32 consecutive values of a row: E2M1 codes (magnitudes 0, 0.5, 1,
 * 1.5, 2, 3, 4, 6; bit 3 the sign) and one E8M0 byte b, their common factor
 * 2^(b - 127):
 *   b    = max(floor(log2(amax)) - 2, -127) + 127; 127 for a block of zeros;
 *          255 (NaN) for a block that holds an infinity or a NaN, whose codes
 *          then mean nothing
 *   code = E2M1(v * 2^(127 - b)), nearest, ties to the even code, at most 6 in
 *          magnitude; a zero keeps its sign
 * The last block of a row is filled up with zero codes, so any K will do.
 *   x    bf16 [R, K]
 *   q    uint8 [R, 16 * ceil(K/32)], two codes to a byte, the even column in
 *        the low half;  s  uint8 [R, ceil(K/32)]
 *   q_t  uint8 [K, 16 * ceil(R/32)], s_t  uint8 [K, ceil(R/32)]: the same of
 *        x's transpose, for the products that contract over rows
 * Either pair may be NULL; x is read once for both.  x, q, q_t 16-byte
 * aligned.  R <= 2^31, K <= 2^22; R == 0 or K == 0 is a no-op.
 */
int mxfp4_quant(const void* x, void* q, void* s, void* q_t, void* s_t, int64_t R, int64_t K, hipStream_t stream);

/*
 * mxfp4_gemm -- the product of two such operands on the matrix cores:
 *   C[m, n] = sum over blocks k of 2^(sA[m, k] - 127) * 2^(sB[n, k] - 127) *
 *             (A[m, block k] . B[n, block k])
 *   A uint8 [M, K/2], sA uint8 [M, K/32]; B uint8 [N, K/2], sB uint8 [N, K/32]
 *   (16-byte aligned codes); C fp32 (4-byte aligned) or bf16 (2-byte aligned)
 *   [M, N] by c_dtype, fully overwritten.
 * K counts whole blocks: a multiple of 32 (mxfp4_quant's rows are filled up).
 * Sums are fp32; bf16 output rounds them once (nearest, ties to even).  An
 * exponent byte of 255 makes the row or column of C it belongs to NaN.
 * Sizes: 0 <= M, N <= 2^31 (M == 0 or N == 0 is a no-op) with ceil(M/128) *
 * ceil(N/128) <= 2^30, K <= 2^22 (K == 0 writes zeros).  From single rows (the
 * weight streams through once) to large tiles.
 */
int mxfp4_gemm(const void* A, const void* sA, const void* B, const void* sB, void* C, int64_t M, int64_t N, int64_t K,
               int c_dtype, hipStream_t stream);

/*
 * The values that codes stand for, in bf16 (nearest, ties to even):
 *   mxfp4_dequant  out[r, k] = code * 2^(s - 127); NaN for an exponent byte of
 *                  255.  q, s as mxfp4_quant writes them, out bf16 [R, K].
 *   group_dequant  out[r, k] = bf16(fl32(code * s[r, k / group])), q int8 or
 *                  E4M3 [R, K] by code_format, s fp32 [R, ceil(K/group)]: the
 *                  row layouts of the quantisers above (y_q_t of the backward
 *                  pass included, with R = H, K = T).
 * q and out 16-byte aligned; R <= 2^31, K <= 2^22 (group_dequant: 2^23).
 */
int mxfp4_dequant(const void* q, const void* s, void* out, int64_t R, int64_t K, hipStream_t stream);
int group_dequant(const void* q, const float* s, void* out, int64_t R, int64_t K, int64_t group, int code_format,
                  hipStream_t stream);

/* ---- the same block in bf16: layer norm, dropout, gated projection ---- */

/*
 * A dropout's mask is made where it is used and never stored.  Element (t, d) of
 * a [T, D] tensor is dropped where word d % 4 of
 *   Philox4x32-10(key = rng[0], counter = (d / 4, t, rng[1] + offset))
 * is below p * 2^32 (nearest).  That is the generator of Salmon, Moraes, Dror and
 * Shaw ("Parallel random numbers: as easy as 1, 2, 3", SC 2011); the key's and the
 * counter's last two words are the 64-bit numbers' low and high halves.  What is
 * kept is multiplied by 1 / (1 - p), one fp32 number; what is dropped is 0,
 * whatever it was.  So the backward pass, given the same p, rng and offset, has
 * the forward pass's mask.
 *   p       0 <= p < 1 as fp32; 0: nothing is dropped, rng is not looked at
 *   rng     int64 [2] in device memory (8-byte aligned): a seed, and a number that
 *           the program changes from step to step.  Read when the kernels run: a
 *           captured call draws a new mask at a replay if they have changed.
 *   offset  added to rng[1] (modulo 2^64): tells the dropouts of a step apart.
 * Calls with the same seed and the same sum rng[1] + offset draw the same words, so
 * the sums of all steps and dropouts of a run have to differ: with the step's number
 * (below 2^32) in rng[1], the i-th dropout of a step takes offset i << 32.  Offset i
 * itself would be the mask that offset 0 draws i steps later.
 *
 * dropout_add -- out = bf16(residual + dropout(x)), one fp32 product and one fp32
 * sum.  On the gradient of out, without a residual, the backward pass for x.
 *   x         bf16 or fp32 [T, D] by x_dtype
 *   residual  bf16 [T, D], or NULL for none
 *   out       bf16 [T, D]; may be residual itself, or x itself if that is bf16
 * 16-byte aligned.  T <= 2^31, D <= 2^22, T * D <= 2^40; T == 0 or D == 0 is a
 * no-op.
 */
int dropout_add(const void* x, int x_dtype, const void* residual, void* out, int64_t T, int64_t D, float p,
                const int64_t* rng, int64_t offset, hipStream_t stream);

/*
 * layer_norm_quant -- layer norm with a dropout and the residual's addition in
 * front of it, its output in bf16, or quantised by row groups as rms_norm_quant's.
 *
 *   h[t, d]  = bf16(residual[t, d] + dropout(x)[t, d])     (as dropout_add)
 *   mean[t]  = sum_d h[t, d] / D
 *   rstd[t]  = 1 / sqrt(sum_d (h[t, d] - mean[t])^2 / D + eps)
 *   y[t, d]  = bf16(((h[t, d] - mean[t]) * rstd[t]) * weight[d] + bias[d])
 *   codes and scales of y by groups of `group` channels, as rms_norm_quant.
 *
 *   weight, bias  bf16 [D]; bias may be NULL for none
 *   mean, rstd    fp32 [T], or NULL: what layer_norm_bwd needs
 *   p, rng, offset  the dropout, as above
 *   The other arguments, alignments, sizes and the place of h (it may be `residual`
 *   itself) as rms_norm_quant.
 * A NaN or an infinity in a row of h makes all of the row's y NaN, which shows in
 * its scales as there; other rows are not affected.  A row of one value has a
 * variance of zero, up to the rounding of its mean: with eps == 0 its y means
 * nothing.
 * The statistics are fp32 and hold what that does: a row whose squared differences
 * from its mean sum to more than 3.4e38 has rstd 0 and the bias for y, one whose
 * values do y NaN; and where eps does not outweigh them, squares below 1e-38 lose bits.
 */
int layer_norm_quant(const void* x, int x_dtype, const void* residual, const void* weight, const void* bias, void* y_q,
                     float* y_s, void* y_bf16, void* h, float* mean, float* rstd, int64_t T, int64_t D, int64_t group,
                     int code_format, float eps, float p, const int64_t* rng, int64_t offset, hipStream_t stream);

/*
 * layer_norm_bwd -- the gradients of that norm.  With n = (h - mean) * rstd and
 * g = dy * weight:
 *
 *   dx[t, d]  = rstd[t] * (g[t, d] - sum_d(g) / D - n[t, d] * sum_d(g * n) / D) + d_h[t, d]
 *   dw[d]     = sum_t dy[t, d] * n[t, d];   db[d] = sum_t dy[t, d]
 *
 * dx, rounded to bf16, is the gradient of h: for the residual, and for x where
 * nothing was dropped.  dx_drop is the gradient for x through the dropout: the
 * same numbers before they are rounded, masked and multiplied as above.
 *   dy       bf16 or fp32 [T, D] by dy_dtype
 *   h, weight, mean, rstd   as layer_norm_quant wrote and read them
 *   d_h      bf16 [T, D], or NULL; dx may be d_h itself
 *   dx       bf16 [T, D];  dx_drop  bf16 [T, D], or NULL (it needs p > 0: with
 *            p == 0 it returns SILUQUANT_ERR_BAD_SHAPE); without it rng is not
 *            looked at
 *   dw, db   fp32 [D], either NULL where it is not wanted
 *   workspace  layer_norm_bwd_workspace_bytes(T, D) bytes, 16-byte aligned; only
 *            looked at when dw or db is wanted or D > 16384.  Its contents before
 *            and after a call mean nothing.  The sums do not depend on timing.
 * Sizes as layer_norm_quant; T == 0 writes zeros to dw and db.  A workspace that is
 * too small returns SILUQUANT_ERR_BAD_SHAPE.
 */
int64_t layer_norm_bwd_workspace_bytes(int64_t T, int64_t D);
int layer_norm_bwd(const void* dy, int dy_dtype, const void* h, const void* weight, const float* mean, const float* rstd,
                   const void* d_h, void* dx, void* dx_drop, float* dw, float* db, void* workspace,
                   int64_t workspace_bytes, int64_t T, int64_t D, float p, const int64_t* rng, int64_t offset,
                   hipStream_t stream);

/*
 * swiglu_gemm -- the gate and up projections, the activation and the product of a
 * gated feed-forward block in one kernel, on the matrix cores:
 *
 *   gate = x . Wg^T,  up = x . Wu^T  (fp32 sums of exact products)
 *   y[t, h] = bf16(gate[t, h] / (1 + exp(-gate[t, h])) * up[t, h])
 *
 *   x   bf16 [T, D]
 *   w   bf16 [2H, D]: Wg's H rows, then Wu's
 *   y   bf16 [T, H], from the sums as they are
 *   gu  bf16 [T, 2H]: [gate | up], rounded; or NULL.  What swiglu_gemm_bwd needs,
 *       and the x of silu_dot_fwd_bwd_quant_fuse and of silu_fwd_quant (whose y is
 *       that of the rounded gate and up).
 * All 16-byte aligned.  Sizes: any T <= 2^31, H and D multiples of 8 up to 2^20
 *   (rows of whole 16-byte pieces); T == 0 or H == 0 is a no-op, D == 0 gives
 *   zeros.  ceil(T/64) * ceil(2H/64), ceil(T/64) * ceil(D/64) and ceil(2H/64) *
 *   ceil(D/64) are at most 2^30.
 * An infinity or a NaN in a row of x or of w makes of the rows or columns it meets
 * what the formulas do: gate = -infinity gives NaN (0 times infinity).
 */
int swiglu_gemm(const void* x, const void* w, void* y, void* gu, int64_t T, int64_t H, int64_t D, hipStream_t stream);

/*
 * swiglu_gemm_bwd -- the gradients of that.  With s = 1 / (1 + exp(-gate)):
 *
 *   d_gu[t] = bf16([dy * up * s * (1 + gate * (1 - s)) | dy * (gate * s)])
 *   dx = d_gu . W;   dw = d_gu^T . x      (fp32 sums)
 *
 *   dy    bf16 [T, H];  gu, x, w as swiglu_gemm wrote and read them
 *   d_gu  bf16 [T, 2H]; may be gu itself.  Rounded to bf16, as the matrix cores
 *         take it; dx and dw are those of the rounded numbers.
 *   dx    bf16 or fp32 [T, D] by dx_dtype, or NULL where it is not wanted (w is
 *         then not looked at)
 *   dw    bf16 or fp32 [2H, D] by dw_dtype, or NULL (x is then not looked at)
 *   workspace  swiglu_gemm_bwd_workspace_bytes(T, H, D) bytes, which may be 0,
 *         16-byte aligned; only looked at when that is not 0 and dx or dw is
 *         wanted.  Its contents before and after a call mean nothing.  The sums do
 *         not depend on timing.
 * All 16-byte aligned; sizes as swiglu_gemm.  T == 0 writes zeros to dw, H == 0 to
 * dx.  A workspace that is too small returns SILUQUANT_ERR_BAD_SHAPE.
 */
int64_t swiglu_gemm_bwd_workspace_bytes(int64_t T, int64_t H, int64_t D);
int swiglu_gemm_bwd(const void* dy, const void* gu, const void* x, const void* w, void* d_gu, void* dx, int dx_dtype,
                    void* dw, int dw_dtype, void* workspace, int64_t workspace_bytes, int64_t T, int64_t H, int64_t D,
                    hipStream_t stream);

/* Optional: makes the HIP runtime load the library's kernels on the current
 * device now, which it otherwise does at the first launch.  No entry point
 * needs it first.  Enqueues nothing, allocates nothing itself; safe to call
 * repeatedly and from several threads.  SILUQUANT_ERR_DEVICE if there is no
 * usable current device. */
int siluquant_prepare(void);

/* Static text for a status code (never NULL). */
const char* siluquant_strerror(int status);

/* Bytes the pass must move per call: reads 6*T*H (x, grad_y), writes 3*T*H
 * int8 codes plus 4*(T*ceil(2H/group) + H*ceil(T/group)) bytes of scales.
 * Host-only arithmetic; returns -1 for negative sizes or a group other than
 * 32, 64 or 128. */
int64_t siluquant_algorithmic_bytes(int64_t T, int64_t H, int64_t group);

/* Diagnostics.  They run the fused kernel's own device helpers on their own so
 * that tests can compare intermediate values bit for bit; the pass itself
 * never needs them.
 *
 * siluquant_eval_sigmoid: s[i] = sigmoid of the bf16 gate gate[i] exactly as the
 *   fused kernel evaluates it.  gate: bf16 [n] (2-byte aligned), s: fp32 [n]
 *   (4-byte aligned), both device memory.  Enqueued on `stream`.
 * siluquant_eval_intermediates: the bf16 values the fused kernel quantises:
 *   y_bf16 [T, H] = bf16(y) and dgdu_bf16 [T, 2H] = [bf16(d_gate) | bf16(d_up)],
 *   from x [T, 2H] and grad_y [T, H] as above; any T, H >= 0; 2-byte aligned
 *   device buffers that must not overlap.  Enqueued on `stream`.
 * Both return siluquant_status codes with the same meanings as above. */
int siluquant_eval_sigmoid(const void* gate, float* s, int64_t n, hipStream_t stream);
int siluquant_eval_intermediates(const void* x, const void* grad_y, void* y_bf16, void* dgdu_bf16, int64_t T,
                                 int64_t H, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SILUQUANT_H */
