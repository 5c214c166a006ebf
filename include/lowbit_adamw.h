/*
 * lowbit_adamw.h -- the part of liblowbit's C ABI that updates parameters: one
 * AdamW step over many tensors at once (adapters, norms, or whole matrices
 * before they are quantized), with moments in 8 bits or in 32.
 *
 * The moments of all tensors lie in one buffer each, in blocks of
 * LOWBIT_ADAMW_BLOCK values: tensor i begins at the block after tensor i-1's
 * last one, and what its last block has beyond its values is zero.
 *    32 bits:  m, v       fp32  [blocks][256]
 *     8 bits:  m, v       uint8 [blocks][256]
 *              m_max, v_max  fp32 [blocks]   the largest |value| of a block
 *    master    fp32 [blocks][256]  the parameters in fp32 (or NULL: a step starts
 *              from the parameters themselves)
 *
 * What an 8-bit code stands for is code's number times its block's maximum:
 *    m   bit 7 is the sign; the number of a code c in 1..127 is the fp32 number of
 *        bits (c + 889) << 20: three bits of mantissa, 127 is 1, 1 is 1.25 * 2^-16
 *    v   the number of a code c in 1..255 is the fp32 number of bits
 *        (c + 761) << 20: three bits of mantissa, 255 is 1, 1 is 1.25 * 2^-32
 *    and code 0 is 0.  A block's largest value is held in 32 bits, so that what
 *    all values of a block have in common is not lost to the codes' steps.
 *
 * Exact arithmetic contract; b1 = fl32(beta1), c1 = fl32(1 - beta1) and so on, the
 * differences and powers in fp64, every operation on m and v one rounded fp32
 * operation:
 *    g  = grad * grad_scale        (grad alone without one)
 *    m' = b1 m + c1 g,   v' = b2 v + c2 (g g)
 *    p' = p * fl32(1 - lr * weight_decay)
 *         - fl32(lr / (1 - beta1^step)) * m' / (sqrt(v') * fl32((1 - beta2^step)^-1/2) + fl32(eps))
 *    in fp32, p' within some 2^-24 of itself and 2^-21 of the step taken, rounded to the
 *    parameters' type; master receives p' unrounded.  Where there is nothing to divide by (an
 *    eps of 0, and a v' that is 0 in fp32) no step is taken.
 * 8-bit moments are stored from m' and v':  max is the block's largest |value|,
 * or 0 where that is below 2^-126; q = |value| * fl32(1 / max), and with bits == 8 the code
 * is the one whose number is nearest to q, the upper of two at the same distance (for m,
 * q below 1.1875 * 2^-16 becomes 0; for v, a q that is not zero becomes 1 at least,
 * so that no second moment is lost that a first one may still be divided by).
 *    What that loses: codes lie 6% to 12% apart, and a step of beta2 = 0.999 changes v
 * by a thousandth of itself and of g^2, so a value's ratio to its block's largest moves only
 * when g^2 is some 30 to 60 times v, and it never falls.  Where all gradients of a block grow or
 * shrink together nothing is lost; where some change against the rest, their v stays
 * behind: after 7000 steps in which half of a block's gradients were a tenth of
 * before, their v was 72 times too large, and where half were four times as large, the
 * other half's was 7.7 times.
 *    bits == (8 | LOWBIT_ADAMW_RANDOM) has none of that: the code is that of one
 * of the two numbers next to q, the upper one where the fp32 bits of q plus r pass a
 * multiple of 2^20.  r = 16 h + 8, h the upper (m) or lower (v) 16 bits of
 * mix(p ^ mix(mix(step) + P)), p and P the lower and upper 32 bits of the value's place
 * in the moments, step its lower 32 bits, mix(x): x ^= x >> 16, x *= 0x6A09E667,
 * x ^= x >> 15, x *= 0xBB67AE85, x ^= x >> 16.  So v follows its definition in the mean
 * (within 0.67 to 1.45 of it for nine in ten values) and results still repeat bit for bit.  m with
 * q below 1.125 * 2^-16 becomes 0, v is never 0 for a q that is not.  The format is the
 * same, and the two can take turns on one state.
 * A block that holds an infinity or a NaN has a NaN maximum and codes 0: everything
 * computed from it is NaN.
 * A grad_scale that is an infinity or a NaN leaves everything as it was: a step of
 * scaled gradients that overflowed is skipped without asking the GPU.
 *
 * Layouts, ownership, alignment (16 bytes), streams and errors as in lowbit.h.
 * Results repeat bit for bit.
 */
#ifndef LOWBIT_ADAMW_H
#define LOWBIT_ADAMW_H

#include "lowbit_w8a8.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LOWBIT_ADAMW_BLOCK 256
#define LOWBIT_ADAMW_RANDOM 256 /* bits == (8 | LOWBIT_ADAMW_RANDOM): codes rounded up or down */
#define LOWBIT_F32 3 /* beside LOWBIT_F16 and LOWBIT_BF16: type of parameters and gradients */

/* One tensor of a step: device pointers (16-byte aligned), and how many values. */
typedef struct {
  void* param;
  const void* grad;
  int64_t n;
} lowbit_adamw_tensor;

/* The moments of the step's tensors, device pointers as laid out above (m_max and
 * v_max NULL with bits == 32; master NULL without a copy). */
typedef struct {
  void* m;
  void* v;
  float* m_max;
  float* v_max;
  float* master;
} lowbit_adamw_state;

/* lr_or_null and step_or_null: device values that take the place of lr and step,
 * read when the step runs (a captured step that is replayed with new ones);
 * grad_scale_or_null: a device factor of the gradients.  4-byte aligned. */
typedef struct {
  double lr, beta1, beta2, eps, weight_decay;
  int64_t step;
  const float* lr_or_null;
  const int32_t* step_or_null;
  const float* grad_scale_or_null;
} lowbit_adamw_options;

/*
 * One step over `count` tensors of one parameter type and one gradient type
 * (LOWBIT_F32, LOWBIT_F16, LOWBIT_BF16).  tensors, state and options are host
 * memory, read during the call.  bits is 8, 8 | LOWBIT_ADAMW_RANDOM or 32.
 *   LOWBIT_ERR_ARG: a null or misaligned pointer, n < 0, count < 0, step < 1, a beta
 *     outside [0, 1), or lr, eps or weight_decay negative or not finite; or memory that the
 *     step writes (a param, m, v, m_max, v_max, master) that shares a byte with another such
 *     piece, a gradient or a device scalar (gradients may share memory with one another);
 *   LOWBIT_ERR_SHAPE: more than 2^36 values in all;
 *   LOWBIT_ERR_UNSUPPORTED: another type, or other bits.
 *   LOWBIT_ERR_HIP: a launch failed, or the host has no memory to compare more than 59 tensors.
 * Tensors of no values take no block; count == 0 is an empty problem.
 */
LOWBIT_API int lowbit_adamw(const lowbit_adamw_tensor* tensors, int64_t count, int param_dtype,
                            int grad_dtype, int bits, const lowbit_adamw_state* state,
                            const lowbit_adamw_options* options, void* hip_stream);

/*
 * What 8-bit moments stand for: m and v fp32 [blocks][256].
 */
LOWBIT_API int lowbit_adamw_moments(const uint8_t* m, const uint8_t* v, const float* m_max,
                                    const float* v_max, int64_t blocks, float* m_out,
                                    float* v_out, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* LOWBIT_ADAMW_H */
