/*
 * qlora_block.h - what a transformer block needs next to its projections: the
 * root-mean-square norm in front of them with its backward, rows held in 8
 * bits with one scale each, and the 8-bit integer product that serves a layer
 * whose adapter has been merged.  Same conventions as qlora.h (dense row-major
 * 16-byte aligned device pointers, bf16 as uint16_t bits, work enqueued on
 * `stream`, arguments checked on the host before anything is launched, nothing
 * allocated).  Sizes need not be multiples of anything.  The _f16 entry points
 * take IEEE fp16 in place of bf16.
 */
#ifndef QLORA_BLOCK_MI355X_H
#define QLORA_BLOCK_MI355X_H

#include "qlora_act.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Longest row of rows8_quantize and of the 8-bit product (whose int32 sums then
 * stay below 2^31), longest row of the norm, and most rows (a grid of one
 * 1024-thread workgroup a row stays below 2^32 threads). */
#define QLORA_ROWS8_MAX 65536
#define QLORA_NORM_MAX 32768
#define QLORA_ROWS_MAX 2097152
/* Bytes from one row of codes to the next: K rounded up to a multiple of 128. */
#define QLORA_ROWS8_PITCH(K) (((int64_t)(K) + 127) / 128 * 128)

/*
 * rows8_quantize / rows8_dequantize - a matrix [R, K] in 8 bits, one scale per
 *   row: tokens of an activation, or output channels of a weight [N, K].
 *   With c = max|x| of a row:
 *     d = fl32(c / 127),  q = fl32(x fl32(127 / c)) rounded to an integer, ties to even,
 *   and the row stands for q d: x_out = RNE_16(fl32(q d)).  A row with c < 2^-120
 *   is stored as zeros; one that holds an inf or NaN has d = NaN and reads back as
 *   NaN.
 *   x      [R, K] 16-bit (device), read; R 1 .. QLORA_ROWS_MAX, K 1 .. QLORA_ROWS8_MAX, any value.
 *   codes  [R, QLORA_ROWS8_PITCH(K)] int8 (device), written by quantize: zeros past K.
 *   scale  [R] float (device), written by quantize.
 *   Errors: NULL, SHAPE, ALIGN, DEVICE.
 */
int rows8_quantize(const uint16_t* x, int64_t R, int64_t K, int8_t* codes, float* scale, void* stream);
int rows8_quantize_f16(const uint16_t* x, int64_t R, int64_t K, int8_t* codes, float* scale, void* stream);
int rows8_dequantize(const int8_t* codes, const float* scale, int64_t R, int64_t K, uint16_t* x_out, void* stream);
int rows8_dequantize_f16(const int8_t* codes, const float* scale, int64_t R, int64_t K, uint16_t* x_out,
                         void* stream);

/*
 * rmsnorm_fwd - root-mean-square norm of each row, with the residual's addition.
 *     h = RNE_16(x + residual)             (x without a residual)
 *     y = h (mean(h^2) + eps)^(-1/2) w     (w = 1 without a weight)
 *   in fp32, the sum of squares over a whole row included (rows whose squares
 *   leave fp32 at either end are summed scaled), with one rounding at each output.  The
 *   norm is that of the 16-bit h, so that the backward below, which reads h,
 *   differentiates what was computed.  A row that holds an inf or NaN gives
 *   what the formula gives: NaN at an inf and 0 beside it, NaN in all of a row
 *   with a NaN.
 *   x, residual  [T, D] 16-bit, read (residual may be NULL); T 1 .. QLORA_ROWS_MAX,
 *                D 1 .. QLORA_NORM_MAX.
 *   weight       [D] 16-bit, or float with weight_f32 = 1; or NULL.
 *   eps          > 0 and finite.
 *   h            [T, D] 16-bit, written when not NULL; may be x or residual.
 *   y            [T, D] 16-bit, written when not NULL.
 *   y_codes, y_scale  the fp32 y as rows8_quantize's rows [T, QLORA_ROWS8_PITCH(D)]
 *                and [T] (no rounding to 16 bits in between), written when not
 *                NULL (both or neither).  At least one of y and y_codes.
 *   Outputs overlap nothing else.
 *   Errors: NULL, SHAPE, ALIGN, VALUE (eps, weight_f32), DEVICE.
 */
int rmsnorm_fwd(const uint16_t* x, const uint16_t* residual, int64_t T, int64_t D, const void* weight,
                int weight_f32, float eps, uint16_t* h, uint16_t* y, int8_t* y_codes, float* y_scale, void* stream);
int rmsnorm_fwd_f16(const uint16_t* x, const uint16_t* residual, int64_t T, int64_t D, const void* weight,
                    int weight_f32, float eps, uint16_t* h, uint16_t* y, int8_t* y_codes, float* y_scale,
                    void* stream);

/*
 * rmsnorm_bwd - gradients of rmsnorm_fwd's y.  With r = (mean(h^2) + eps)^(-1/2),
 *   n = h r and g = dY w:
 *     dx = r (g - n mean(g n)) + dx_add
 *     dw = sum over rows of dY n
 *   in fp32 (g, dx and dw have to lie in its range; the squares and g h need
 *   not), the same bits on every run.  dx is the gradient of x and of the
 *   residual alike; dx_add is what reaches h on the residual path.
 *   dy, h     [T, D] 16-bit, read (h: the forward's, or its x without a residual).
 *   weight    as in the forward.
 *   dx_add    [T, D] 16-bit or NULL.
 *   dx        [T, D] 16-bit, written; may be dy or dx_add.
 *   d_weight  [D] of the weight's type, written when not NULL (needs a weight).
 *   workspace at least rmsnorm_workspace_bytes_bwd(T, D) bytes when d_weight is
 *             asked for.
 *   Errors: NULL, SHAPE, ALIGN, VALUE, WORKSPACE, DEVICE.
 */
int rmsnorm_bwd(const uint16_t* dy, const uint16_t* h, int64_t T, int64_t D, const void* weight, int weight_f32,
                float eps, const uint16_t* dx_add, uint16_t* dx, void* d_weight, void* workspace,
                size_t workspace_bytes, void* stream);
int rmsnorm_bwd_f16(const uint16_t* dy, const uint16_t* h, int64_t T, int64_t D, const void* weight, int weight_f32,
                    float eps, const uint16_t* dx_add, uint16_t* dx, void* d_weight, void* workspace,
                    size_t workspace_bytes, void* stream);
size_t rmsnorm_workspace_bytes_bwd(int64_t T, int64_t D);

/*
 * int8_linear_fwd - the product of two matrices held as 8-bit rows, with the
 *   epilogue of qlora_linear_act_fwd.
 *     Z = (sum_k xq[t, k] wq[n, k]) dx[t] dw[n] + bias
 *     Y = act(Z) * mul + residual
 *   The sum is exact (int32); everything after it is fp32, operation by
 *   operation as written (the smaller scale first), with one rounding at Y: the
 *   bits of an output depend neither on T and N nor on how the work is split.  A
 *   NaN scale makes its row of Y (its column, for a channel of W) NaN.
 *   x_codes [T, QLORA_ROWS8_PITCH(K)], x_scale [T]; w_codes [N, same pitch],
 *   w_scale [N]: as rows8_quantize or rmsnorm_fwd writes them (zeros past K).
 *   T 1 .. QLORA_ROWS_MAX, N 1 .. 2^20, K 1 .. QLORA_ROWS8_MAX, T N and T K at most 2^30.
 *   epilogue: bias [N], mul and residual [T, N] of Y's type or NULL, act; its
 *   z, z_codes and z_scale must be NULL.  y [T, N], written; may be the buffer of
 *   mul or of residual; no other overlap.
 *   workspace: at least int8_linear_workspace_bytes(T, K, N) bytes (may be 0,
 *   then NULL is allowed).
 *   Errors: NULL (epilogue itself too), SHAPE, ALIGN, VALUE (unknown act, a Z
 *   output), WORKSPACE, DEVICE.
 */
int int8_linear_fwd(const int8_t* x_codes, const float* x_scale, int64_t T, int64_t K, int64_t N,
                    const int8_t* w_codes, const float* w_scale, const qlora_epilogue* epilogue, uint16_t* y,
                    void* workspace, size_t workspace_bytes, void* stream);
int int8_linear_fwd_f16(const int8_t* x_codes, const float* x_scale, int64_t T, int64_t K, int64_t N,
                        const int8_t* w_codes, const float* w_scale, const qlora_epilogue* epilogue, uint16_t* y,
                        void* workspace, size_t workspace_bytes, void* stream);
size_t int8_linear_workspace_bytes(int64_t T, int64_t K, int64_t N);

#ifdef __cplusplus
}
#endif

#endif /* QLORA_BLOCK_MI355X_H */
