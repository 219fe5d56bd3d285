/*
 * kda_dense.h -- C ABI of what a hybrid decoder's layers need around the
 * recurrence and the cached attention: the residual's addition with its norm,
 * the projections in 8 bits, and rotary positions.  (Page "Kimi K3：架构、训练与百万
 * Token Agentic RL 技术解读" §3.2 names the projections W x that kda_decode_layer_step
 * takes as inputs; it says nothing of their storage.)
 *
 * The conventions of kda.h hold: device pointers owned by the caller, nothing
 * allocated, asynchronous on `stream`, argument errors found on the host before
 * anything is launched.  None of these calls needs scratch memory.  Each may start while
 * the kernel before it on its stream ends: its blocks then wait on the SMs, and what they
 * hold (threads, registers, shared and tensor memory) other streams do without meanwhile.
 *
 * 8-bit matrices: codes uint8 [rows][C], an E4M3 value each (sign, 4 exponent
 * bits of bias 7, 3 mantissa bits, no infinities, 0x7f and 0xff NaN, largest
 * 448), and scales uint8 [ceil(rows / R)][ceil(C / 128)], dense: the value of
 * an element is its code times 2^(byte - 127), the byte of its block of R rows
 * and 128 columns (the last blocks may be cut); byte 255 stands for NaN.  R is 1
 * for activations and 128 for weights.  What the library writes has the smallest
 * power of two, 2^-126 at least, that leaves no value of the block above 448,
 * codes rounded to nearest, ties to the even code; a block with an inf or NaN
 * among its values is stored as byte 255 and codes 0, which reads back as NaN.
 */
#ifndef KDA_GB300_KDA_DENSE_H
#define KDA_GB300_KDA_DENSE_H

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * x [T][C] dtype dt (row stride in elements, at least C) to 8 bits: codes [T][C] dense, scales
 * [ceil(T / block_rows)][ceil(C / 128)], block_rows 1 or 128.  Any T, C up to 2^31 - 512; rows that
 * begin on 16-byte boundaries (8 bytes for codes) take wide loads and stores.
 */
KDA_API kda_status kda_fp8_quant(const void* x, int64_t x_stride, int64_t T, int64_t C, int32_t block_rows,
                                 kda_dtype dt, uint8_t* codes, uint8_t* scales, cudaStream_t stream);

/*
 * The values that codes [T][C] (dense) and scales stand for, y [T][C] dtype dt, dense.  They are exact in
 * either type but below 2^-126 and above its largest value.
 */
KDA_API kda_status kda_fp8_values(const uint8_t* codes, const uint8_t* scales, int64_t T, int64_t C,
                                  int32_t block_rows, kda_dtype dt, void* y, cudaStream_t stream);

/*
 * The residual's addition and a root-mean-square norm of each row, C values:
 *   s = x + residual,   h = s in dt,   y = s / sqrt(sum s^2 / C + eps) * weight
 *
 *  x, residual  [T][C] dtype dt, row strides in elements; residual may be NULL (s = x, h not written)
 *  weight       fp32 [C], 4-byte aligned, or NULL (ones)
 *  h            [T][C] dtype dt, dense, NULL when residual is NULL; may be residual or x itself when that is dense
 *  y            [T][C] dtype dt, dense; may be x itself when that is dense (and h another array); or NULL, and then
 *  codes, scales  the same values in 8 bits, scales [T][ceil(C / 128)] (y NULL exactly when these are given)
 * s is summed and normed in fp32, y rounds once; h is s rounded.  A row whose squares leave
 * fp32's range is normed all the same; an infinite s makes its element NaN and the others 0,
 * as the formula does.  eps >= 0 and finite.
 * KDA_ERR_UNSUPPORTED: C beyond 32768.
 */
KDA_API kda_status kda_add_rmsnorm(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                                   const float* weight, float eps, int64_t T, int64_t C, kda_dtype dt, void* h, void* y,
                                   uint8_t* codes, uint8_t* scales, cudaStream_t stream);

/*
 * out[m][n] = sum_k A[m][k] W[n][k] over 8-bit matrices.
 *  a, a_scales  codes [M][K], row stride a_stride in bytes; scales [M][ceil(K / 128)] (R = 1)
 *  w, w_scales  codes [N][K], row stride w_stride in bytes; scales [ceil(N / 128)][ceil(K / 128)] (R = 128)
 *  out          [M][N] dtype dt, row stride out_stride in elements, at least N
 * K (at least 16) and the row strides of a and w are multiples of 16, a and w 16-byte aligned, out aligned to
 * its type.  Products are exact, sums fp32 in an order that depends on M, N, K and the number of the device's SMs
 * alone: the same call gives the same bits, and a bf16 output is the fp32 output rounded.  Their error's rms stays below
 * K 2^-28 of a row's (normally distributed values: 5e-7 of it for K = 12,288, 4e-6 for 2,048 rows of 16,384).  A NaN
 * code of a row of A reaches that row of out, one of W that column; a scale byte 255 its row, or its 128 columns.
 * KDA_ERR_UNSUPPORTED: K not a multiple of 16 or beyond 2^27; M or N beyond 2^31 - 512.
 */
KDA_API kda_status kda_fp8_matmul(const uint8_t* a, int64_t a_stride, const uint8_t* a_scales, const uint8_t* w,
                                  int64_t w_stride, const uint8_t* w_scales, int64_t M, int64_t N, int64_t K,
                                  kda_dtype dt, void* out, int64_t out_stride, cudaStream_t stream);

/* Flags of kda_rotary. */
enum { KDA_ROTARY_INTERLEAVED = 1, KDA_ROTARY_INVERSE = 2 };

/*
 * Rotary positions: of each head's D channels the first `rot` are turned in pairs,
 *   (a, b) -> amplitude (a cos t - b sin t, a sin t + b cos t),   t = positions[token] freqs[i],
 * pair i being channels (i, i + rot / 2), or (2 i, 2 i + 1) with KDA_ROTARY_INTERLEAVED; the others
 * stay.  KDA_ROTARY_INVERSE turns by -t (with amplitude 1 it undoes the rotation; it is the
 * rotation's gradient too).
 *
 *  q [T][Hq][D], k [T][Hk][D] dtype dt, and q_out, k_out of the same shapes: strides from token to
 *             token and head to head in elements, channels contiguous.  A part with no heads (0) may be
 *             NULL.  An output is its input (the same pointer and strides: in place), or none of its values is
 *             one of an input's; its heads and tokens do not lie over one another, or over the other output's.
 *             Inputs and outputs may lie between one another's tokens (with the same token stride) or heads
 *             (with the same head stride, a divisor of the token stride), as parts of one projection do;
 *             other ones lie apart from first to last byte.
 *  positions  int32[T] (kda_page_map's); a token with a negative one is not turned
 *  freqs      fp64[rot / 2]: radians per position, finite
 * Angles are reduced to a fraction of a turn in 64 bits of fixed point: at any position they are
 * right to 2^-24 of a turn, and sines and cosines to fp32's rounding.  rot is even, at most D.
 * 16-byte steps throughout (and rot a multiple of 16) take wide loads and stores.
 * KDA_ERR_UNSUPPORTED: D beyond 1024, or Hq + Hk.
 */
KDA_API kda_status kda_rotary(const void* q, int64_t q_token_stride, int64_t q_head_stride, int32_t Hq, const void* k,
                              int64_t k_token_stride, int64_t k_head_stride, int32_t Hk, const int32_t* positions,
                              int64_t T, int32_t D, int32_t rot, const double* freqs, float amplitude, int32_t flags,
                              kda_dtype dt, void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                              void* k_out, int64_t k_out_token_stride, int64_t k_out_head_stride, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_GB300_KDA_DENSE_H */
