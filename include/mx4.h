/*
 * mx4.h -- C ABI of the MX4 calls of libw12.so: 4-bit floating point under a
 * shared scale (the OCP Microscaling format MXFP4), the small and large
 * products with weights stored that way, and an expert layer on them, for AMD
 * MI355X (gfx950).  Beside the lossless W12 containers of w12.h this is the
 * lossy format: 4.25 bits a value.
 *
 * The format.
 *   block    = 32 consecutive values along K of one row (K % 32 == 0);
 *   scale    = one byte e a block, standing for 2^(e - 127); 255 is NaN;
 *   code     = sign << 3 | i, standing for +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}[i];
 *   value    = code * scale;
 *   encoding = e = max(0, E - 2) with E the largest biased fp32 exponent of the
 *              block (that is, floor(log2(largest magnitude)) - 2, at least
 *              -127; a block of zeros and fp32 subnormals has e = 0), each code
 *              the nearest one to value / 2^(e - 127), ties to the even i,
 *              magnitudes above 6 to 6; the sign of a zero is kept.  A block
 *              that holds an infinity or a NaN has e = 255 and codes 0: all of
 *              it reads back as NaN.
 *   layout   = a container holds B matrices of [R, K]; rows are padded to
 *              Rp = R rounded up to 16 a matrix, K to whole groups of 128
 *              (G = K / 128 rounded up).  Codes: 1 KB a (16-row tile T, group
 *              g), ordered by (T, g), T = b * Rp/16 + r/16; in it the 16-byte
 *              piece L = 16*q + r%16 holds k = 128*g + 32*q + 0..31, two codes
 *              a byte, the even k in the low half.  Scales: 256 bytes a (T,
 *              four groups), ordered; byte 4*L + g%4 is the scale of piece L of
 *              group g.  Padding has codes 0 and scales 127.
 * A piece is what one lane of a 64-wide wave feeds the matrix cores with, and a
 * scale's dword serves four groups of its lane.
 *
 * Conventions: those of w12.h (device pointers owned by the caller, work
 * enqueued on `stream`, arguments checked on the host before any launch, the
 * w12_status_t values returned, nothing allocated or kept, no
 * synchronisation).  Calls on different streams are independent; a workspace
 * needs no initial contents, must be 256-byte aligned, and calls that may run
 * at the same time need separate ones.  Results depend on no scheduling: the
 * same call on the same data returns the same bits.  Counts of zero rows
 * (R, M or T = 0) are valid and launch nothing.
 */
#ifndef MX4_H
#define MX4_H

#include <stddef.h>
#include <stdint.h>

#include "w12.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MX4_BLOCK 32
#define MX4_MAX_T 128        /* tokens of one mx4_moe call */
#define MX4_MAX_E 1024       /* its experts */
#define MX4_MAX_TOP_K 32     /* its experts a token */

/* Element types of mx4_quantize's input and of every output: the values of
 * w12_out_t. */

/* Static, never-NULL description of a status code, in the terms of the calls
 * below. */
const char *mx4_status_string(int status);

/* Bytes of the codes and of the scales of a container of B matrices [R, K]:
 * B*Rp/16*G*1024 and B*Rp/16*ceil(G/4)*256 (0 on a bad shape: B < 1, R < 0,
 * K < 32, K % 32 != 0, K >= 2^24, or 2^40 values and more). */
size_t mx4_codes_bytes(int64_t B, int64_t R, int64_t K);
size_t mx4_scales_bytes(int64_t B, int64_t R, int64_t K);

/*
 * mx4_quantize -- x [B, R, K] -> container.
 *   x      : device, BF16 bits or fp32 as x_type says (w12_out_t), rows of K
 *            contiguous values, row stride ldx and matrix stride ldb elements
 *            (ldx >= K; ldb is read only when B > 1), 16-byte aligned, both
 *            strides multiples of 16 bytes.
 *   codes, scales : device outputs, mx4_codes_bytes / mx4_scales_bytes, 16-byte
 *            aligned; padding included.
 * Errors: W12_ERR_NULL, W12_ERR_SHAPE, W12_ERR_DTYPE, W12_ERR_ALIGN,
 *         W12_ERR_HIP.
 */
int mx4_quantize(const void *x, int x_type, int64_t B, int64_t R, int64_t K,
                 int64_t ldx, int64_t ldb, void *codes, void *scales, void *stream);

/*
 * mx4_dequantize -- container -> y [B, R, K], the values it stands for: exact
 * in fp32 and in BF16 for every scale that mx4_quantize writes.
 *   y : device output, BF16 bits or fp32 as y_type says; strides and alignment
 *       as mx4_quantize's x.  Its matrices share no value: they lie one behind
 *       the other (ldb >= (R - 1) * ldy + K) or between each other's rows
 *       (ldb >= K, ldy >= (B - 1) * ldb + K).
 * Errors as mx4_quantize.
 */
int mx4_dequantize(const void *codes, const void *scales, int64_t B, int64_t R, int64_t K,
                   void *y, int y_type, int64_t ldy, int64_t ldb, void *stream);

/*
 * mx4_gemm -- y[m, n] = sum_k x[m, k] * W[n, k], W a container of one [N, K],
 * x BF16; any M.  The weights are expanded to BF16 (exactly) in registers, the
 * sums are fp32.
 *   x  : device BF16 [M, K], row stride ldx elements (ldx >= K, ldx % 8 == 0),
 *        16-byte aligned.  With ldx >= 2^23 and many rows the weights are
 *        read once for every 16 of them (copy such rows together first).
 *   y  : device output [M, N], row stride ldy >= N, BF16 bits (2-byte aligned)
 *        or fp32 (4-byte aligned) as y_type says.
 *   workspace : mx4_gemm_workspace_bytes(M, N, K, 0) bytes; NULL if that is 0.
 * Errors: W12_ERR_NULL, W12_ERR_SHAPE (N < 1, N > 2^27, M < 0, M > 2^24,
 *         M*N > 2^37 or ldx >= 2^23 with M > 16 * 65535, beside those of the
 *         sizes), W12_ERR_ALIGN, W12_ERR_DTYPE, W12_ERR_WORKSPACE,
 *         W12_ERR_HIP.
 */
int mx4_gemm(const uint16_t *x, int64_t M, int64_t ldx, const void *w_codes,
             const void *w_scales, int64_t N, int64_t K, void *y, int64_t ldy, int y_type,
             void *workspace, size_t workspace_bytes, void *stream);

/*
 * mx4_gemm_mx4 -- the same product with x a container of one [M, K]: both sides
 * go to the matrix cores as 4-bit codes with their scales, the sums are fp32.
 *   workspace : mx4_gemm_workspace_bytes(M, N, K, 1) bytes; NULL if that is 0.
 * Errors as mx4_gemm.
 */
int mx4_gemm_mx4(const void *x_codes, const void *x_scales, int64_t M, const void *w_codes,
                 const void *w_scales, int64_t N, int64_t K, void *y, int64_t ldy, int y_type,
                 void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes of mx4_gemm (x_mx4 = 0) or mx4_gemm_mx4 (x_mx4 = 1): partial
 * sums where K is split over workgroups, else 0.  Returns W12_OK, W12_ERR_NULL
 * or W12_ERR_SHAPE. */
int mx4_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int x_mx4, size_t *bytes);

/*
 * mx4_moe -- a mixture-of-experts layer for up to MX4_MAX_T tokens:
 *   S(t)    = the top_k experts of token t with the largest logits[t, e], ties to
 *             the lowest e;
 *   p(t, e) = exp(logits[t, e]) / sum over S(t) (renormalize != 0) or over all
 *             experts (renormalize = 0) of exp(logits[t, .]);
 *   h       = silu(G_e x_t) * (U_e x_t),  silu(a) = a / (1 + exp(-a));
 *   y[t]    = sum over e in S(t) of p(t, e) * D_e h.
 * An expert with logit -inf is never chosen, so such a token has fewer experts
 * (all of them -inf: y[t] = 0); a NaN logit makes its token's y NaN.  The
 * hidden values h are carried between the two products with all 24 bits of
 * their mantissa, the sums are fp32.
 *   x      : device BF16 [T, H], as mx4_gemm's.
 *   logits : device fp32 [T, E], row stride ldl >= E elements, 4-byte aligned.
 *   w13_*  : a container of E matrices [2*I, H], rows 0..I-1 of each G_e, rows
 *            I..2*I-1 U_e.
 *   w2_*   : a container of E matrices [H, I], D_e.
 *   y      : device output [T, H], as mx4_gemm's.
 *   workspace : mx4_moe_workspace_bytes(T, H, I, E, top_k, y_type) bytes.
 * H % 32 == 0, I % 32 == 0, 1 <= top_k <= min(E, MX4_MAX_TOP_K),
 * E <= MX4_MAX_E; (min(E, T*top_k) + T*top_k/16) times H/16 and times I/16 at
 * most 2^24.
 * Errors: W12_ERR_NULL, W12_ERR_SHAPE, W12_ERR_ALIGN, W12_ERR_DTYPE,
 *         W12_ERR_UNSUPPORTED (T, E or top_k over its limit),
 *         W12_ERR_WORKSPACE, W12_ERR_HIP.
 */
int mx4_moe(const uint16_t *x, int64_t T, int64_t ldx, const float *logits, int64_t ldl,
            const void *w13_codes, const void *w13_scales, const void *w2_codes,
            const void *w2_scales, int64_t H, int64_t I, int64_t E, int64_t top_k,
            int renormalize, void *y, int64_t ldy, int y_type, void *workspace,
            size_t workspace_bytes, void *stream);
int mx4_moe_workspace_bytes(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top_k,
                            int y_type, size_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* MX4_H */
