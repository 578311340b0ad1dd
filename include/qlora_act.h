/*
 * qlora_act.h - what surrounds the frozen-base linear layer in a transformer
 * block: the layer's forward with bias, activation, gating product and
 * residual in its epilogue, activation checkpoints in 8 bits, and the backward
 * that reads them.  Same conventions as qlora.h (dense row-major 16-byte
 * aligned device pointers, bf16 as uint16_t bits, work enqueued on `stream`,
 * arguments checked on the host before anything is launched, nothing
 * allocated); the layer, its storage and size limits are those of
 * qlora_linear_fwd.  The _f16 entry points take IEEE fp16 in place of bf16;
 * the _sq ones the single-quantization storage (bf16).
 */
#ifndef QLORA_ACT_MI355X_H
#define QLORA_ACT_MI355X_H

#include "qlora.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations.  gelu is z Phi(z) with the normal distribution function,
 * gelu_tanh its tanh form 0.5 z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))).
 * relu's slope at 0 is 0; a NaN gives NaN in every activation and slope. */
#define QLORA_ACT_NONE 0
#define QLORA_ACT_RELU 1
#define QLORA_ACT_SILU 2
#define QLORA_ACT_GELU 3
#define QLORA_ACT_GELU_TANH 4

/*
 * act8_quantize / act8_dequantize - an activation held in 8 bits.
 *   Blocks are 64 consecutive values (row-major; the last may be shorter).
 *   With c = max|x| of a block:
 *     d = fl32(c / 127),  q = fl32(x fl32(127 / c)) rounded to an integer, ties to even,
 *   and the block stands for q d: x_out = RNE_16(fl32(q d)).  |x_out - x| is at
 *   most d / 2 and the final roundings.  A block with c < 2^-120 is stored as
 *   zeros; one that holds an inf or NaN has d = NaN and reads back as NaN.
 *   x      [numel] 16-bit (device), read; numel 1 .. 2^43, any value.
 *   codes  [numel] int8 (device), written by quantize.
 *   scale  [ceil(numel/64)] float (device), written by quantize.
 *   Errors: NULL, SHAPE, ALIGN, DEVICE.
 */
int act8_quantize(const uint16_t* x, int64_t numel, int8_t* codes, float* scale, void* stream);
int act8_quantize_f16(const uint16_t* x, int64_t numel, int8_t* codes, float* scale, void* stream);
int act8_dequantize(const int8_t* codes, const float* scale, int64_t numel, uint16_t* x_out, void* stream);
int act8_dequantize_f16(const int8_t* codes, const float* scale, int64_t numel, uint16_t* x_out, void* stream);

/*
 * qlora_linear_act_fwd - the layer's forward with an epilogue.
 *     Z = X W'^T + scaling (X A) B + bias
 *     Y = act(Z) * mul + residual
 *   in fp32 from the products' sums on, with one rounding at each output; a
 *   NULL bias, mul or residual is left out.
 *   bias [N], mul [T, N], residual [T, N] 16-bit, read;  y [T, N], written.  y
 *   may be the buffer of mul or of residual (in place); no other overlap.
 *   z [T, N] 16-bit: Z, written when not NULL.
 *   z_codes [T*N] int8 and z_scale [T*N/64] float: act8_quantize's checkpoint
 *   of that 16-bit Z, written when not NULL (both or neither), whether or not
 *   z itself is.  (The backward below reads Z in either form.)
 *   Other arguments, sizes, workspace (qlora_workspace_bytes) and kernels by
 *   size as for qlora_linear_fwd; the workspace is left as that call leaves
 *   it.  With an empty epilogue Y is the same bits as qlora_linear_fwd's.
 *   Errors: NULL (epilogue itself, one of z_codes / z_scale alone), SHAPE,
 *   ALIGN, VALUE (scaling, unknown act), WORKSPACE, DEVICE.
 */
typedef struct qlora_epilogue {
    int act;                    /* QLORA_ACT_*                                    */
    const uint16_t* bias;       /* [N] or NULL                                    */
    const uint16_t* mul;        /* [T, N] or NULL                                 */
    const uint16_t* residual;   /* [T, N] or NULL                                 */
    uint16_t* z;                /* [T, N] or NULL, written                        */
    int8_t* z_codes;            /* [T*N] or NULL, written                         */
    float* z_scale;             /* [T*N/64], with z_codes                         */
} qlora_epilogue;
int qlora_linear_act_fwd(const uint16_t* x, int64_t T, int64_t K, int64_t N,
                         const uint8_t* codes, const uint8_t* absmax_fp8, const float* superscale,
                         const uint16_t* lora_a, const uint16_t* lora_b, int64_t r, float scaling,
                         const qlora_epilogue* epilogue, uint16_t* y,
                         void* workspace, size_t workspace_bytes, void* stream);
int qlora_linear_act_fwd_sq(const uint16_t* x, int64_t T, int64_t K, int64_t N,
                            const uint8_t* codes, const float* absmax,
                            const uint16_t* lora_a, const uint16_t* lora_b, int64_t r, float scaling,
                            const qlora_epilogue* epilogue, uint16_t* y,
                            void* workspace, size_t workspace_bytes, void* stream);
int qlora_linear_act_fwd_f16(const uint16_t* x, int64_t T, int64_t K, int64_t N,
                             const uint8_t* codes, const uint8_t* absmax_fp8, const float* superscale,
                             const uint16_t* lora_a, const uint16_t* lora_b, int64_t r, float scaling,
                             const qlora_epilogue* epilogue, uint16_t* y,
                             void* workspace, size_t workspace_bytes, void* stream);

/*
 * qlora_linear_act_bwd - backward of qlora_linear_act_fwd from saved
 *   activations, each of them 16-bit values or an 8-bit checkpoint.
 *     dZ    = dY * mul * act'(Z)         rounded to 16 bits for the products
 *     dX    = dZ W' + scaling (dZ B^T) A^T + dx_add
 *     dA    = scaling X^T (dZ B^T)       (only if d_lora_a != NULL)
 *     dB    = scaling (X A)^T dZ         (only if d_lora_b != NULL)
 *     dbias = sum over tokens of dZ      (only if d_bias != NULL; before its rounding)
 *     dmul  = dY * act(Z)                (only if d_mul != NULL)
 *   fp32 accumulation, 16-bit outputs, the same bits on every run.  The
 *   residual's gradient is dY itself.  A checkpointed X enters the products
 *   as act8_dequantize's 16-bit values, a checkpointed Z or mul as fl32(q d).
 *   x [T, K] is required iff d_lora_a or d_lora_b is; z [T, N] iff act is not
 *   QLORA_ACT_NONE or d_mul is asked for; mul [T, N] iff the forward had one.
 *   dx_add [T, K] 16-bit or NULL: added to dX before its rounding (the sum of
 *   the gradients of several layers on one input); may be dx itself.  dx is
 *   written; outputs overlap nothing else.
 *   workspace: at least qlora_act_workspace_bytes_bwd(T, K, N, r) bytes.
 *   Errors: NULL (a required activation or one of codes / scale missing),
 *   SHAPE, ALIGN, VALUE (scaling, unknown act, a saved activation in both
 *   forms), WORKSPACE, DEVICE.
 */
typedef struct qlora_saved {
    const uint16_t* values;     /* 16-bit values, or NULL                         */
    const int8_t* codes;        /* or the checkpoint's codes ...                  */
    const float* scale;         /* ... and scales                                 */
} qlora_saved;
typedef struct qlora_act_grad {
    int act;                    /* QLORA_ACT_*                                    */
    qlora_saved x, z, mul;      /* all NULL = absent                              */
    const uint16_t* dx_add;     /* [T, K] or NULL                                 */
    uint16_t* dx;               /* [T, K], written                                */
    uint16_t* d_lora_a;         /* [K, r] or NULL, written                        */
    uint16_t* d_lora_b;         /* [r, N] or NULL, written                        */
    uint16_t* d_bias;           /* [N] or NULL, written                           */
    uint16_t* d_mul;            /* [T, N] or NULL, written                        */
} qlora_act_grad;
int qlora_linear_act_bwd(const uint16_t* dy, int64_t T, int64_t K, int64_t N,
                         const uint8_t* codes, const uint8_t* absmax_fp8, const float* superscale,
                         const uint16_t* lora_a, const uint16_t* lora_b, int64_t r, float scaling,
                         const qlora_act_grad* grad, void* workspace, size_t workspace_bytes, void* stream);
int qlora_linear_act_bwd_sq(const uint16_t* dy, int64_t T, int64_t K, int64_t N,
                            const uint8_t* codes, const float* absmax,
                            const uint16_t* lora_a, const uint16_t* lora_b, int64_t r, float scaling,
                            const qlora_act_grad* grad, void* workspace, size_t workspace_bytes, void* stream);
int qlora_linear_act_bwd_f16(const uint16_t* dy, int64_t T, int64_t K, int64_t N,
                             const uint8_t* codes, const uint8_t* absmax_fp8, const float* superscale,
                             const uint16_t* lora_a, const uint16_t* lora_b, int64_t r, float scaling,
                             const qlora_act_grad* grad, void* workspace, size_t workspace_bytes, void* stream);

/* Device workspace (bytes) of qlora_linear_act_bwd for these sizes (at least
 * the forward's, so that both can use the same one); 0 for sizes the entry
 * points would reject. */
size_t qlora_act_workspace_bytes_bwd(int64_t T, int64_t K, int64_t N, int64_t r);

#ifdef __cplusplus
}
#endif

#endif /* QLORA_ACT_MI355X_H */
