/*
 * gbfuse_block -- the block-scaled 8-bit path: E4M3 codes whose scales are found
 * from the data, one float32 for every 128 columns of an activation's row and
 * for every 128 x 128 block of a weight, and the Linear on them.  Where one
 * static scale has to cover a tensor's largest outlier (gbf_add_rmsnorm_fp8,
 * gbf_linear_fp8_act), here an outlier costs its own 128 columns alone, and no
 * calibration is needed.  Part of libgbfuse.so; C ABI, GB300 (sm_103a).
 *
 * The conventions are gbfuse.h's: caller-owned dense buffers, work enqueued on
 * `stream` without synchronising, gbf_status return values with gbf_last_error()
 * for the message.  No call keeps state between calls or needs a workspace;
 * every call may be captured into a CUDA graph, allows programmatic dependent
 * launch, and gives the same bits whenever it is given the same inputs (on one GPU:
 * how the Linear cuts K goes by how many clusters a GPU holds at once).
 *
 * A block's scale and codes, in binary32:
 *   scale = max(RN(amax * RN(1 / 448)), 2^-100)      amax = the block's largest |y|
 *   code  = e4m3(RN(y * RN(1 / scale)))              to nearest even, saturated to +-448
 * and code * scale is the value.  Columns d - d % 128 ... d - 1 of a width d that
 * is no multiple of 128 are a block of their own.  A block that holds a NaN gets
 * scale NaN and NaN codes; one that holds an infinity (and no NaN) gets scale
 * infinity, NaN codes at the infinities and zeros elsewhere.
 *
 * Scales are dense row-major float32: [rows, ceil(d / 128)] of an activation,
 * [ceil(rows / 128), ceil(d / 128)] of a weight, 4-byte aligned.
 */
#ifndef GBFUSE_BLOCK_H
#define GBFUSE_BLOCK_H

#include "gbfuse.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * gbfb_add_rmsnorm_fp8 -- gbf_add_rmsnorm_fp8 with block scales found from the
 * row in place of the static fp8_scale: res_out = bf16(x + res_in) (or
 * res_in + gate * x), y = its RMSNorm / _noweight / AdaRMSNorm in float32, then
 * the codes and scales of y.  FlashRT §2.1 and §3 name the chain; the arguments
 * up to q_out, their layouts and aliasing are gbf_add_rmsnorm_fp8's.
 *
 * q_out: device uint8 [rows, hidden]; scales: device float32
 * [rows, ceil(hidden / 128)].  Requires hidden % 16 == 0 (the Linear's rule for
 * its rows), hidden <= 32768, 16-byte aligned tensors (scales: 4-byte).
 * rows == 0 enqueues nothing.
 */
GBF_API int gbfb_add_rmsnorm_fp8(const void* x, const void* res_in, void* res_out, const void* gate, int mode,
                                 const void* weight, const void* ada_scale, const void* ada_shift, uint8_t* q_out,
                                 float* scales, int64_t rows, int64_t hidden, float eps, void* stream);

/*
 * gbfb_gated_act_fp8 -- the codes and scales of y = act(gate) * up, which
 * gbf_gated_act writes as bf16: x is device bf16 [rows, 2d], gate then up; act is
 * GBF_ACT_SILU, GBF_ACT_GELU_TANH or GBF_ACT_GELU_ERF.  y is float32 (an
 * act(gate) below float32's normal range may count as zero), off by at most
 * (10 + 4 |z|) 2^-23 of itself (z the argument of the logistic function that SiLU
 * and the tanh GELU multiply by) or (10 + gate^2) 2^-23 (erf GELU), and never reaches
 * memory.  q_out: device uint8 [rows, d]; scales: device float32
 * [rows, ceil(d / 128)].  Requires d % 16 == 0 and 16-byte aligned x, q_out.
 */
GBF_API int gbfb_gated_act_fp8(const void* x, uint8_t* q_out, float* scales, int64_t rows, int64_t d, int act,
                               void* stream);

/*
 * gbfb_quantize_fp8 -- the codes and scales of x itself, device bf16 [rows, d]:
 * an attention's output in front of its projection (block_rows 1: a scale for
 * every 128 columns of a row), or a Linear's weight at load time (block_rows
 * 128: a scale for every 128 x 128 block; blocks at the edges are cut short).
 * Bit-reproducible: the two formulas above, one rounding a step.  q_out: device
 * uint8 [rows, d]; scales: device float32 [ceil(rows / block_rows), ceil(d / 128)].
 * Requires d % 16 == 0 and 16-byte aligned x, q_out.
 */
GBF_API int gbfb_quantize_fp8(const void* x, uint8_t* q_out, float* scales, int64_t rows, int64_t d, int block_rows,
                              void* stream);

/*
 * gbfb_linear_fp8 -- Y = act(X W^T + bias) on block-scaled codes, on the tcgen05
 * tensor cores (kind::f8f6f4, E4M3 x E4M3):
 *   y[m, n] = act(sum_b (sx[m, b] * sw[n / 128, b]) * sum_{k in block b} x[m, k] w[n, k] + bias[n])
 * The sum over a block of 128 k is the tensor core's, in float32; the product of
 * the two scales, its product with the block's sum and the sum over blocks are
 * float32, in registers; one bf16 rounding.  Scales may be any numbers.
 *
 * act is gbf_linear_bias_gelu's, evaluated as there, by forms for an epilogue whose
 * errors, in front of the rounding, are below
 *   GELU_TANH  |a| 2^-11.9 (the hardware's tanh, relative error 2^-10.9)
 *   GELU_ERF   |a| 2^-21   (an erf with an absolute error of 1.5e-7)
 *   SILU       |act(a)| (8 + 2 |a|) 2^-23
 * so a GELU's value at a strongly negative a, small beside |a|, is right to these
 * bounds only and not to a bf16 rounding of itself.  Over all bf16 a, what was seen
 * beyond one bf16 rounding is below |a| 2^-20 and |a| 2^-26: at a = -3 both are
 * within a rounding, at a = -5 the tanh GELU gives 0 for -2.3e-7.
 *
 * Xq: device uint8 E4M3 codes [M, K]; x_scales: device float32 [M, ceil(K / 128)];
 * Wq: device uint8 E4M3 codes [N, K] (nn.Linear [out, in] layout); w_scales:
 * device float32 [ceil(N / 128), ceil(K / 128)]; bias: device bf16 [N] or NULL;
 * Y: device bf16 [M, N]; act as gbf_linear_bias_gelu.  Requires K % 16 == 0,
 * N % 8 == 0, 16-byte aligned Xq, Wq, Y, bias (scales: 4-byte), M, N, K below 2^31
 * and fewer than 2^31 tiles of 64 x 128 of Y; Y may not overlap an input.  M == 0
 * enqueues nothing.  Waits are bounded as in gbf_linear_bias_gelu.
 */
GBF_API int gbfb_linear_fp8(const uint8_t* Xq, const float* x_scales, const uint8_t* Wq, const float* w_scales,
                            const void* bias, void* Y, int64_t M, int64_t N, int64_t K, int act, void* stream);

/*
 * gbfb_linear_fp8_plan -- what a gbfb_linear_fp8 call of these sizes launches on the
 * current device: *tile_rows 16, 32, 64 or 128 (single CTAs, that many rows of X a
 * tile) or 256 (CTA pairs), *split CTAs (pairs) of a cluster that cut K; both 0 for
 * M == 0.  For tests and tuning; enqueues nothing.
 */
GBF_API int gbfb_linear_fp8_plan(int64_t M, int64_t N, int64_t K, int* tile_rows, int* split);

#ifdef __cplusplus
}
#endif

#endif /* GBFUSE_BLOCK_H */
