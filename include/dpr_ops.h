/*
 * dpr_ops.h -- the operators of a backward pass that make the gradients the
 * buckets of dpr.h hold: layer norm (forward, and backward with the
 * reduction of the parameter gradients), activation checkpoints in 8 bits,
 * and a linear layer's weight gradient read from such a checkpoint.  They
 * are part of libdpr and share the conventions of dpr.h: device buffers
 * owned by the caller, asynchronous work on the caller's stream (every
 * kernel a programmatic dependent launch off the legacy default stream),
 * arguments checked on the host before anything is launched, a status as the
 * result.  Nothing is allocated: calls that need scratch memory take it as
 * `workspace`, whose size the matching *_workspace call gives.
 *
 * Activations are matrices of `rows` tokens by `width` channels, row by row:
 * element (r, c) is at data[r * stride + c], the stride in elements, at
 * least `width` where the call writes and at least 0 (one row for all) where
 * it only reads.  Any stride and any element-aligned address is accepted;
 * rows whose start is 32-byte aligned take the widest accesses.  A matrix
 * occupies everything from its first to its last element: an output may not
 * overlap that range of another buffer, beyond the in-place forms that a call
 * names.  Every sum and statistic is held in fp32, and results do not change
 * from run to run.
 */
#ifndef DPR_OPS_H
#define DPR_OPS_H

#include "dpr.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum dpr_dtype { DPR_BF16 = 0, DPR_FP32 = 1 } dpr_dtype;

#define DPR_MAX_ROWS (((int64_t)1) << 30)  /* tokens per call */
#define DPR_MAX_WIDTH (((int64_t)1) << 20) /* channels */
#define DPR_MAX_GRAD_ROWS (((int64_t)1) << 22) /* tokens of one weight gradient */
#define DPR_CHECKPOINT_BLOCK 32            /* channels that share one step */

/*
 * An activation held in 8 bits.  Block b of a row is channels 32b .. 32b+31
 * (the last one may be shorter); it has one step byte and its channels one
 * signed code each, and value = code * step, where the step is the fp32
 * number whose exponent field is the byte (2^(byte - 127); 0 for byte 0).
 * dpr_checkpoint_save chooses the smallest power of two with
 * max|x| / step < 127.5 (at least 2^-126; at most 2^121, where codes
 * saturate at 127) and rounds x / step to the nearest integer, ties to even.
 * An all-zero block has byte 0.  A block that holds an infinity or a NaN has
 * byte 255 and codes 0, and every value of it is restored as NaN, so that a
 * diverged step still shows in its gradients.  Steps are powers of two, so
 * code * step is exact in fp32 and in bf16: saving rounds once, restoring
 * never.
 *
 *   codes  element (r, c) at codes[r * code_stride + c], code_stride >= width
 *   steps  block (r, b) at steps[r * step_stride + b],
 *          step_stride >= ceil(width / 32)
 * Strides and addresses that are multiples of 16 take the widest accesses.
 */
typedef struct dpr_checkpoint {
    int8_t* codes;
    int64_t code_stride;
    uint8_t* steps;
    int64_t step_stride;
} dpr_checkpoint;

/*
 * Layer norm (Ba, Kiros and Hinton, "Layer Normalization", 2016), row by row:
 *   mean = sum_c x_c / width
 *   rstd = 1 / sqrt(sum_c (x_c - mean)^2 / width + eps)
 *   y_c  = (x_c - mean) * rstd * weight_c + bias_c
 * `dtype` is the type of x and y, `param_dtype` that of weight and bias.
 * weight == NULL stands for ones, bias == NULL for zeros.  mean and rstd
 * ([rows] fp32) may be NULL when no backward pass follows.  y may be x
 * itself (same address and stride).  x_ckpt and y_ckpt may be NULL; else the
 * call also saves x, or y as rounded to `dtype`, exactly as
 * dpr_checkpoint_save would.
 */
dpr_status dpr_layernorm_forward(const void* x, int64_t x_stride, int64_t rows, int64_t width,
                                 int dtype, const void* weight, const void* bias, int param_dtype,
                                 float eps, void* y, int64_t y_stride, float* mean, float* rstd,
                                 const dpr_checkpoint* x_ckpt, const dpr_checkpoint* y_ckpt,
                                 void* stream);

/*
 * The backward pass, with the forward's mean and rstd:
 *   xhat = (x - mean) * rstd,  g = dy * weight
 *   dx      = rstd * (g - avg_c(g) - xhat * avg_c(g * xhat))
 *   dweight = sum_rows dy * xhat,  dbias = sum_rows dy
 * x is read from `x`, or from its checkpoint when x_ckpt is not NULL (x is
 * then ignored; dy and dx keep `dtype`).  dx may be dy or x itself (same
 * address and stride).  dweight and dbias ([width], `grad_dtype`) may each
 * be NULL; with accumulate != 0 they are added to.  rows == 0 gives zero
 * gradients.  The workspace is 16-byte aligned and may be reused by the next
 * call on the same stream.
 */
dpr_status dpr_layernorm_backward_workspace(int64_t rows, int64_t width, int64_t* bytes);
dpr_status dpr_layernorm_backward(const void* dy, int64_t dy_stride, const void* x,
                                  int64_t x_stride, const dpr_checkpoint* x_ckpt, int64_t rows,
                                  int64_t width, int dtype, const void* weight, int param_dtype,
                                  const float* mean, const float* rstd, void* dx,
                                  int64_t dx_stride, void* dweight, void* dbias, int grad_dtype,
                                  int accumulate, void* workspace, int64_t workspace_bytes,
                                  void* stream);

/* Saves x ([rows, width], `dtype`) in 8 bits, and restores it. */
dpr_status dpr_checkpoint_save(const void* x, int64_t x_stride, int64_t rows, int64_t width,
                               int dtype, const dpr_checkpoint* ckpt, void* stream);
dpr_status dpr_checkpoint_load(const dpr_checkpoint* ckpt, int64_t rows, int64_t width, void* out,
                               int64_t out_stride, int dtype, void* stream);

/*
 * The weight gradient of y = x W^T with W [out_features, in_features], from
 * the checkpoint of x:
 *   dweight[o][i] = sum_t dy[t][o] * x~[t][i]
 * with x~ the restored checkpoint ([rows, in_features]) and dy bf16
 * ([rows, out_features]).  Products are exact and summed in fp32; dweight
 * (bf16 or fp32, `dtype`) is rounded once, after adding the old value when
 * accumulate != 0.  rows == 0 gives zeros.  The workspace is 16-byte aligned
 * and may be reused by the next call on the same stream; its size depends on
 * the sizes and, because inputs whose rows are not 16-byte aligned are first
 * copied into it, on the addresses and strides.
 */
dpr_status dpr_linear_weight_grad_workspace(const void* dy, int64_t dy_stride,
                                            const dpr_checkpoint* x_ckpt, int64_t rows,
                                            int64_t out_features, int64_t in_features,
                                            int64_t* bytes);
dpr_status dpr_linear_weight_grad(const void* dy, int64_t dy_stride, const dpr_checkpoint* x_ckpt,
                                  int64_t rows, int64_t out_features, int64_t in_features,
                                  void* dweight, int64_t dweight_stride, int dtype, int accumulate,
                                  void* workspace, int64_t workspace_bytes, void* stream);

/*
 * How often a wait inside these operators' kernels has run out on the current
 * device since the library was loaded (each wait is bounded; 0 unless the
 * hardware or the library is broken): at least once for every block in which
 * one did, whose call's result is incomplete.  Waits for all of the device's
 * work, on every stream.
 */
dpr_status dpr_device_wait_failures(uint32_t* count);

#ifdef __cplusplus
}
#endif

#endif /* DPR_OPS_H */
