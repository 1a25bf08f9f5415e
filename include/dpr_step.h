/*
 * dpr_step.h -- the operators of a training step around the ones of dpr_ops.h:
 * the RMS norm with the residual's addition, the linear layers of experts
 * (products grouped by expert, with their gradients), and the global norm and
 * clipping of the reduced gradients.  They are part of libdpr and share the
 * conventions of dpr.h and dpr_ops.h: activations are matrices of `rows` tokens
 * by `width` channels with any stride at any element-aligned address, scratch
 * memory is the caller's `workspace`, work is asynchronous on the caller's
 * stream, sums are held in fp32 or more, and results do not change from run to
 * run.
 */
#ifndef DPR_STEP_H
#define DPR_STEP_H

#include "dpr_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Root-mean-square norm (Zhang and Sennrich, "Root Mean Square Layer
 * Normalization", 2019) of the sum of an activation and the residual stream:
 *   h_c  = x_c + residual_c, rounded to `dtype` (h = x when residual is NULL)
 *   rstd = 1 / sqrt(sum_c h_c^2 / width + eps)
 *   y_c  = h_c * rstd * weight_c
 * `dtype` is the type of x, residual, h and y, `param_dtype` that of weight
 * (NULL stands for ones).  h is stored where the residual stream goes on
 * (NULL: not stored; needs a residual) and may be x or the residual itself; y
 * may be x or the residual, whichever h is not (same address and stride).
 * rstd ([rows] fp32) may be NULL when no backward pass follows.  h_ckpt and
 * y_ckpt may be NULL; else the call also saves h, or y as rounded to `dtype`,
 * exactly as dpr_checkpoint_save would; with y_ckpt y may be NULL: the output
 * in 8 bits alone.
 *
 * The squares are summed in fp32: a row whose sum of squares is beyond it has
 * rstd 0, and where eps is none, one whose squares are below 1e-38 loses digits.  The
 * order of a row's sum goes by the width, the layouts and the number of rows, so
 * that a token by itself and the same token among 1024 may differ in the last bit.
 */
dpr_status dpr_rmsnorm_forward(const void* x, int64_t x_stride, const void* residual,
                               int64_t residual_stride, int64_t rows, int64_t width, int dtype,
                               const void* weight, int param_dtype, float eps, void* h,
                               int64_t h_stride, void* y, int64_t y_stride, float* rstd,
                               const dpr_checkpoint* h_ckpt, const dpr_checkpoint* y_ckpt,
                               void* stream);

/*
 * The backward pass, with the forward's rstd:
 *   hhat = h * rstd,  g = dy * weight
 *   dx      = dh + rstd * (g - hhat * avg_c(g * hhat))
 *   dweight = sum_rows dy * hhat
 * dx is the gradient of x and of the residual alike; dh, the gradient that
 * reaches h past the norm (along the residual stream), may be NULL.  h is
 * read from `h`, or from its checkpoint when h_ckpt is not NULL (h is then
 * ignored).  dx may be dy, dh or h itself (same address and stride).  dweight
 * ([width], `grad_dtype`) may be NULL; with accumulate != 0 it is added to.
 * rows == 0 gives a zero gradient.  The workspace is 16-byte aligned and may
 * be reused by the next call on the same stream.
 */
dpr_status dpr_rmsnorm_backward_workspace(int64_t rows, int64_t width, int64_t* bytes);
dpr_status dpr_rmsnorm_backward(const void* dy, int64_t dy_stride, const void* dh,
                                int64_t dh_stride, const void* h, int64_t h_stride,
                                const dpr_checkpoint* h_ckpt, int64_t rows, int64_t width,
                                int dtype, const void* weight, int param_dtype, const float* rstd,
                                void* dx, int64_t dx_stride, void* dweight, int grad_dtype,
                                int accumulate, void* workspace, int64_t workspace_bytes,
                                void* stream);

/*
 * Linear layers of experts, over tokens sorted by expert: expert e's tokens
 * are the rows offsets[e] .. offsets[e + 1] - 1 of the activations, and its
 * weight is the matrix W_e [out_features, in_features].
 *   dpr_grouped_linear              y_t  = W_e x_t
 *   dpr_grouped_linear_input_grad   dx_t = W_e^T dy_t
 *   dpr_grouped_linear_weight_grad  dW_e = sum over e's tokens of dy_t x_t^T
 * offsets ([experts + 1] int32) is read on the device, as a router leaves it;
 * every value is taken as limited to 0 .. rows and as no less than those before
 * it, so that no row has two experts whatever the values are.  An expert may have no
 * tokens (its weight is not read; its weight gradient is zero).  Rows that
 * belong to no expert are not written, and what they hold has no effect (they
 * may be read).  At most DPR_MAX_GRAD_ROWS rows.
 *
 * x, dy and weight are bf16; weight e starts at weight + e * expert_stride,
 * its rows `weight_stride` apart.  Products are exact and summed in fp32; y,
 * dx and dweight (bf16 or fp32, `dtype`) are rounded once.  The weight
 * gradients read x, or its checkpoint when x_ckpt is not NULL (x is then
 * ignored); with accumulate != 0 they are added to.  The workspace is 16-byte
 * aligned and may be reused by the next call on the same stream; its size
 * depends on the sizes (long sums of few tiles are split over the GPU, their
 * parts joined in order) and, because inputs whose rows are not 16-byte aligned
 * may first be copied into it, on the strides and on the addresses modulo 16.
 */
#define DPR_MAX_EXPERTS 1024

dpr_status dpr_grouped_linear_workspace(const void* x, int64_t x_stride, int64_t rows,
                                        int64_t experts, const void* weight,
                                        int64_t weight_stride, int64_t expert_stride,
                                        int64_t out_features, int64_t in_features, int64_t* bytes);
dpr_status dpr_grouped_linear(const void* x, int64_t x_stride, int64_t rows,
                              const int32_t* offsets, int64_t experts, const void* weight,
                              int64_t weight_stride, int64_t expert_stride, int64_t out_features,
                              int64_t in_features, void* y, int64_t y_stride, int dtype,
                              void* workspace, int64_t workspace_bytes, void* stream);

dpr_status dpr_grouped_linear_input_grad_workspace(const void* dy, int64_t dy_stride, int64_t rows,
                                                   int64_t experts, const void* weight,
                                                   int64_t weight_stride, int64_t expert_stride,
                                                   int64_t out_features, int64_t in_features,
                                                   int64_t* bytes);
dpr_status dpr_grouped_linear_input_grad(const void* dy, int64_t dy_stride, int64_t rows,
                                         const int32_t* offsets, int64_t experts,
                                         const void* weight, int64_t weight_stride,
                                         int64_t expert_stride, int64_t out_features,
                                         int64_t in_features, void* dx, int64_t dx_stride,
                                         int dtype, void* workspace, int64_t workspace_bytes,
                                         void* stream);

dpr_status dpr_grouped_linear_weight_grad_workspace(const void* dy, int64_t dy_stride,
                                                    const void* x, int64_t x_stride,
                                                    const dpr_checkpoint* x_ckpt, int64_t rows,
                                                    int64_t experts, int64_t out_features,
                                                    int64_t in_features, int64_t* bytes);
dpr_status dpr_grouped_linear_weight_grad(const void* dy, int64_t dy_stride, const void* x,
                                          int64_t x_stride, const dpr_checkpoint* x_ckpt,
                                          int64_t rows, const int32_t* offsets, int64_t experts,
                                          int64_t out_features, int64_t in_features, void* dweight,
                                          int64_t dweight_stride, int64_t expert_stride, int dtype,
                                          int accumulate, void* workspace, int64_t workspace_bytes,
                                          void* stream);

/*
 * The global norm of a list of gradients, and their clipping: what stands
 * between the reduced partitions and the optimizer step.
 *   norm    = scale * sqrt(sum over all elements of all tensors of g^2)
 *   factor  = scale * (norm <= max_norm ? 1 : max_norm / norm)
 *   out     = g * factor
 * `scale` (positive, finite) undoes a loss scale or averages; `norm` is one
 * fp32 number on the device.  The sum neither overflows nor underflows,
 * whatever the elements' magnitudes (a norm beyond fp32 is infinite).  An
 * infinite norm clips to zero (and the infinities to NaN), a NaN makes every
 * gradient NaN: a diverged step shows.
 *
 * The list is recorded once: n tensors of numel[i] elements (0 allowed, at most
 * DPR_MAX_ELEMS, 2^38 in all) at src[i], written to dst[i], each bf16 or fp32
 * (src_dtype[i], dst_dtype[i]).
 * dst == NULL, or dst[i] == src[i] with the same type, is in place; otherwise
 * outputs overlap neither one another nor any input.  Any element-aligned
 * addresses are accepted; where both rows of a tensor can be 32-byte aligned
 * together, the widest accesses are taken.  The plan may be used on any stream
 * of the device it was made on, and by several calls of dpr_grad_norm at once if
 * their norms and workspaces differ.  It must outlive the work enqueued with it
 * and the graphs captured with it.  Making and destroying a plan allocate and
 * free device memory, which may wait for all of the device's work: once before
 * the steps and once behind them, and not while a stream is captured.
 *
 *   dpr_grad_norm        the norm
 *   dpr_grad_clip        the clipping by a norm that the device holds already
 *                        (of several devices' gradients, say)
 *   dpr_grad_norm_clip   both in one call
 * In place and with a factor of exactly 1 no gradient is written (they may be
 * read).  dpr_grad_norm and dpr_grad_norm_clip take dpr_grad_norm_workspace
 * bytes, 16-byte aligned, which the next call on the same stream may reuse.
 */
typedef struct dpr_grad_plan dpr_grad_plan;
#define DPR_MAX_GRADS (1 << 20)

dpr_status dpr_grad_plan_create(dpr_grad_plan** plan, int n, const void* const* src,
                                const int* src_dtype, void* const* dst, const int* dst_dtype,
                                const int64_t* numel, void* stream);
dpr_status dpr_grad_plan_destroy(dpr_grad_plan* plan);
dpr_status dpr_grad_norm_workspace(const dpr_grad_plan* plan, int64_t* bytes);
dpr_status dpr_grad_norm(const dpr_grad_plan* plan, float scale, float* norm, void* workspace,
                         int64_t workspace_bytes, void* stream);
dpr_status dpr_grad_clip(const dpr_grad_plan* plan, float scale, float max_norm, const float* norm,
                         void* stream);
dpr_status dpr_grad_norm_clip(const dpr_grad_plan* plan, float scale, float max_norm, float* norm,
                              void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DPR_STEP_H */
