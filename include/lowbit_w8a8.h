/*
 * lowbit_w8a8.h -- the part of liblowbit's C ABI that multiplies in 8-bit
 * integers: 8-bit weights with a scale for each output channel, 8-bit
 * activations with a scale for each token (BladeLLM model quantization,
 * "Quantization modes": act_and_weight_quant, dynamic activations).  It is the
 * mode for prompts and for training, where the product is bound by the matrix
 * cores; lowbit.h holds the weight-only mode, the quantizers and the status
 * codes.
 *
 * Weights are the 8-bit codes of lowbit_quantize_rtn, lowbit_quantize_rtn_sym
 * or lowbit_quantize_gptq[_sym] with bits = 8 and group_size = 0, unchanged:
 *    packed  uint32 [N][K/4]   code k of a row is its byte k
 *    scales  fp16   [N]        s
 *    zeros   int32  [N]        z;   deq = (code - z) * s
 *
 * Exact arithmetic contract:
 *  - activations (lowbit_quantize_act, and inside the products when they are
 *    given as fp16 or bf16): per token, amax = max_k |x| (exact),
 *    S = fl32(amax / 127), replaced by 1 when it is zero;
 *    a = clamp(rint(fl32(x / S)), -127, 127), both divisions IEEE fp32, rint
 *    half to even.  A token that holds an infinity or a NaN has S = NaN and
 *    codes 0, so everything computed from it is NaN;
 *  - the integer sum  d = sum_k a (code - z)  is exact;
 *    linear: y = (S * s) * d, in fp32, rounded once to the output type;
 *  - gated:  g and u are the linear products with the gate and up weights, in
 *    fp32 (not rounded); h = act(g) * u in fp32, rounded once.  act is
 *    LOWBIT_ACT_SILU  g / (1 + e^-g), or LOWBIT_ACT_GELU_TANH
 *    g / (1 + e^-2p), p = sqrt(2/pi) (g + 0.044715 g^3);
 *  - gradients go through the rounding of the activations unchanged and the
 *    weights are constants:  dx = sum_n (dy s_n) (code - z_n).  The factor
 *    dy s_n is rounded to 11 significant bits (fp16, after a power of two
 *    chosen for each token that makes the token's largest factor lie in
 *    [2^14, 2^15); a factor below 2^-29 of the largest loses bits; factors below
 *    fp32's normal range lose no others), the sums are fp32, dx is rounded once.
 *    For the gated block  du = dh act(g),  dg = dh u act'(g)  in fp32 from the
 *    given 16-bit g and u.  A token whose
 *    dy (dg, du) holds an infinity or a NaN, or whose factors dy s_n leave
 *    fp32's range, has an all-NaN dx.
 *    Sums over n may be split; their order is fixed by the sizes alone, so
 *    results repeat bit for bit.
 *
 * Layouts, ownership, alignment (16 bytes), streams and errors as in lowbit.h:
 * dense row-major device buffers owned by the caller, checks on the host
 * before anything is enqueued, no allocation, work enqueued on hip_stream of
 * the current device.
 *    x, dx   dtype [T][K]      y, dy, h, dh, gate, up   dtype [T][N]
 *
 * Shape rules (violations return LOWBIT_ERR_SHAPE): K > 0, K % 32 == 0,
 * K <= LOWBIT_W8A8_MAX_K (the sums are 32-bit); T, N <= LOWBIT_W8A8_MAX_TN,
 * T * N and T * K <= 2^36.  Any N, odd ones too.  T == 0 is an empty problem;
 * N == 0 leaves a product empty and a gradient zero.  A workspace smaller than
 * the *_workspace_bytes value, or not 256-byte aligned, returns LOWBIT_ERR_ARG;
 * calls on one workspace must not overlap.  Workspace sizes of zero allow a
 * null workspace; sizes are those of the current device, on which the call has
 * to be made too.  A size holds for its T, N and K only: it does not grow with
 * T throughout, since work that would leave compute units idle is shared out
 * with room for the shares (linear, 4096 x 4096: 17.0 MiB for 256 tokens, 3.9
 * for 1000).  A workspace for many T is one of the largest of their sizes; a
 * query takes less than a microsecond.
 */
#ifndef LOWBIT_W8A8_H
#define LOWBIT_W8A8_H

#include "lowbit.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LOWBIT_W8A8_MAX_K 131072
#define LOWBIT_W8A8_MAX_TN 1048576

/* Element types (others return LOWBIT_ERR_UNSUPPORTED). */
#define LOWBIT_F16 0
#define LOWBIT_BF16 1
#define LOWBIT_I8 2 /* x of the products only: codes of lowbit_quantize_act */

/* Activations of the gated block (others return LOWBIT_ERR_UNSUPPORTED). */
#define LOWBIT_ACT_SILU 0
#define LOWBIT_ACT_GELU_TANH 1

/*
 * Quantize activations x[T][K] (LOWBIT_F16 or LOWBIT_BF16) token by token:
 * codes int8 [T][K], scales fp32 [T] and sums int32 [T], the sum of a token's
 * codes (what a weight grid's zero point multiplies).
 */
LOWBIT_API int lowbit_quantize_act(const void* x, int dtype, int64_t T, int64_t K, int8_t* codes,
                                   float* scales, int32_t* sums, void* hip_stream);

/*
 * y[T][N] = x[T][K] * deq(packed)^T in 8-bit integers.  x is either fp16 or
 * bf16 (quantized on the way; x_scales and x_sums NULL) or LOWBIT_I8: codes of
 * lowbit_quantize_act with their scales and sums.  out_dtype is LOWBIT_F16 or
 * LOWBIT_BF16.  The workspace size depends on T, N, K and dtype (see above).
 */
LOWBIT_API int64_t lowbit_linear_w8a8_workspace_bytes(int64_t T, int64_t N, int64_t K, int dtype);
LOWBIT_API int lowbit_linear_w8a8(const void* x, int dtype, const float* x_scales,
                                  const int32_t* x_sums, int64_t T, const uint32_t* packed,
                                  const uint16_t* scales_f16, const int32_t* zeros, int64_t N,
                                  int64_t K, void* y, int out_dtype, void* workspace,
                                  int64_t workspace_bytes, void* hip_stream);

/*
 * h[T][N] = act(x * deq(gate)^T) * (x * deq(up)^T): both projections, the
 * activation and the product in one kernel.  gate_or_null and up_or_null (both
 * or neither) receive the two projections, rounded to out_dtype, for
 * lowbit_gated_w8a8_grad.
 */
LOWBIT_API int64_t lowbit_gated_w8a8_workspace_bytes(int64_t T, int64_t N, int64_t K, int dtype);
LOWBIT_API int lowbit_gated_w8a8(const void* x, int dtype, const float* x_scales,
                                 const int32_t* x_sums, int64_t T, const uint32_t* packed_gate,
                                 const uint16_t* scales_gate, const int32_t* zeros_gate,
                                 const uint32_t* packed_up, const uint16_t* scales_up,
                                 const int32_t* zeros_up, int64_t N, int64_t K, int act, void* h,
                                 void* gate_or_null, void* up_or_null, int out_dtype,
                                 void* workspace, int64_t workspace_bytes, void* hip_stream);

/*
 * dx[T][K] = dy[T][N] * deq(packed): the gradient of lowbit_linear_w8a8 with
 * respect to x, from the packed words as they lie (no transposed copy).
 */
LOWBIT_API int64_t lowbit_linear_w8a8_grad_workspace_bytes(int64_t T, int64_t N, int64_t K);
LOWBIT_API int lowbit_linear_w8a8_grad(const void* dy, int dtype, int64_t T,
                                       const uint32_t* packed, const uint16_t* scales_f16,
                                       const int32_t* zeros, int64_t N, int64_t K, void* dx,
                                       void* workspace, int64_t workspace_bytes,
                                       void* hip_stream);

/*
 * The gradient of lowbit_gated_w8a8 with respect to x, from dh and the gate
 * and up projections that the forward call kept (all dtype).  dgate_or_null
 * and dup_or_null (both or neither) receive dg and du rounded to dtype, from
 * which gradients of adapters beside the two projections follow.
 */
LOWBIT_API int64_t lowbit_gated_w8a8_grad_workspace_bytes(int64_t T, int64_t N, int64_t K);
LOWBIT_API int lowbit_gated_w8a8_grad(const void* dh, const void* gate, const void* up, int dtype,
                                      int64_t T, const uint32_t* packed_gate,
                                      const uint16_t* scales_gate, const int32_t* zeros_gate,
                                      const uint32_t* packed_up, const uint16_t* scales_up,
                                      const int32_t* zeros_up, int64_t N, int64_t K, int act,
                                      void* dx, void* dgate_or_null, void* dup_or_null,
                                      void* workspace, int64_t workspace_bytes, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* LOWBIT_W8A8_H */
