/*
 * lowbit_lora.h -- the part of liblowbit's C ABI for low-rank adapters beside
 * the shared projections of lowbit.h and lowbit_w8a8.h: the adapters of many
 * requests at once, and their gradients.  lowbit_adamw.h updates what these
 * gradients are of.
 *
 * Adapters lie in pools, one rank R and scale s for each of L adapters:
 *    a   dtype [L][R][K]      b   dtype [L][N][R]      scales  fp32 [L]
 * (a shorter adapter is padded with zero rows of a and zero columns of b).
 * Each of T tokens goes through one adapter or none, by a plan that holds for
 * every layer that the batch passes:
 *    order   int32 [T]     the tokens sorted by adapter, the earlier first
 *                          within one, those without an adapter last
 *    starts  int32 [L+1]   starts[l]: where adapter l's tokens begin in order;
 *                          starts[L]: where the tokens without one begin
 *
 * Exact arithmetic contract, with l the token's adapter:
 *  - v_t = a_l x_t: products of 16-bit values are exact, sums are fp32;
 *  - out_t = y_t + s_l (b_l v_t) in fp32, rounded once to dtype.  For the matrix
 *    cores s_l v_t, an fp32 value, is split into two 16-bit parts: 16 bits of
 *    each value for LOWBIT_BF16; for LOWBIT_F16 22 bits, after a power of two
 *    chosen for each token that makes its largest value lie in [2^14, 2^15) (a value below
 *    2^-17 of the largest loses bits, as fp16 subnormals do);
 *  - u_t = b_l^T dy_t in fp32;  dx_t = base_t + s_l (a_l^T u_t), in the same two parts;
 *  - da_l = s_l sum_t u_t x_t^T and db_l = s_l sum_t dy_t v_t^T over the adapter's
 *    tokens, fp32.  u and v enter in 24 bits, three parts, for LOWBIT_BF16.  For
 *    LOWBIT_F16 they enter in two parts after a power of two that follows the largest
 *    finite value so far, of up to 64 ranks together and of the tokens of one chunk of the
 *    adapter's, which can be thousands and all that it has.  A value of u or v is then
 *    off by 2^-22 of itself or by 2^-39 of that largest one, whichever is more: one 2^-30
 *    below it keeps about 9 bits, and one 2^-39 below it none;
 *  - a token without an adapter: out_t = y_t, v_t = 0, dx_t = base_t, and it
 *    adds nothing to da and db.  An adapter without tokens has zero gradients.
 *    Nothing of such a token's x and dy, nor of an adapter without tokens, reaches
 *    any result, infinities and NaN included.  An infinity elsewhere makes the results
 *    that it enters infinities or NaN (its products with the parts of one value may have
 *    different signs);
 *  - the order of the sums is fixed by the sizes and the plan alone, so results
 *    repeat bit for bit.
 *
 * Layouts, ownership, alignment (16 bytes), streams and errors as in lowbit.h:
 * dense row-major device buffers owned by the caller, checks on the host before
 * anything is enqueued, no allocation, work enqueued on hip_stream of the
 * current device.
 *    x, dx   dtype [T][K]     y, out, dy   dtype [T][N]     v   fp32 [T][R]
 * dtype is LOWBIT_F16 or LOWBIT_BF16 (lowbit_w8a8.h), one for all of a call.
 *
 * Shape rules (violations return LOWBIT_ERR_SHAPE): K > 0, K % 32 == 0,
 * K <= LOWBIT_W8A8_MAX_K; R > 0, R % 8 == 0, R <= LOWBIT_LORA_MAX_R;
 * 1 <= L <= LOWBIT_LORA_MAX_L; N >= LOWBIT_LORA_MIN_N; T, N <= LOWBIT_W8A8_MAX_TN;
 * T * N, T * K, L * R * K and L * R * N <= 2^36.  Odd N too.  T == 0 is an empty
 * problem (da and db of it are zero).
 * An order that is not a permutation or starts that do not rise give unspecified
 * results, but no access outside the buffers.
 * A workspace smaller than the *_workspace_bytes value, or not 256-byte aligned,
 * returns LOWBIT_ERR_ARG; calls on one workspace must not overlap.  A size holds
 * for its own T, N, K, R and L only.
 */
#ifndef LOWBIT_LORA_H
#define LOWBIT_LORA_H

#include "lowbit_w8a8.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LOWBIT_LORA_MAX_R 128
#define LOWBIT_LORA_MAX_L 1024
#define LOWBIT_LORA_MIN_N 8

/*
 * The plan of a batch: order and starts from ids[T], each token's adapter.  An id
 * outside [0, L) is none.
 */
LOWBIT_API int lowbit_lora_plan(const int32_t* ids, int64_t T, int64_t L, int32_t* order,
                                int32_t* starts, void* hip_stream);

/*
 * out[T][N] = y[T][N] + the adapters' part (y_or_null NULL: that part alone).  out
 * may be y itself; otherwise it shares memory with no input.  v_or_null receives
 * v, which lowbit_lora_grad takes.
 */
LOWBIT_API int64_t lowbit_lora_workspace_bytes(int64_t T, int64_t N, int64_t K, int64_t R,
                                               int64_t L);
LOWBIT_API int lowbit_lora(const void* x, int dtype, int64_t T, const int32_t* order,
                           const int32_t* starts, const void* a, const void* b,
                           const float* scales, int64_t L, int64_t R, int64_t N, int64_t K,
                           const void* y_or_null, void* out, float* v_or_null, void* workspace,
                           int64_t workspace_bytes, void* hip_stream);

/*
 * The gradients of lowbit_lora with respect to x, a and b, from dy, x and v.
 * dx[T][K] is base + the adapters' part, base being the gradient through the
 * shared projection (base_or_null NULL: the adapters' part alone); dx may be
 * base itself.  da fp32 [L][R][K] and db fp32 [L][N][R] are written whole.
 */
LOWBIT_API int64_t lowbit_lora_grad_workspace_bytes(int64_t T, int64_t N, int64_t K, int64_t R,
                                                    int64_t L);
LOWBIT_API int lowbit_lora_grad(const void* dy, const void* x, const float* v, int dtype, int64_t T,
                                const int32_t* order, const int32_t* starts, const void* a,
                                const void* b, const float* scales, int64_t L, int64_t R,
                                int64_t N, int64_t K, const void* base_or_null, void* dx,
                                float* da, float* db, void* workspace, int64_t workspace_bytes,
                                void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* LOWBIT_LORA_H */
