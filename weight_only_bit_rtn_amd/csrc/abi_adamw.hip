// abi_adamw.hip -- the exported entry points of the AdamW step: argument checks,
// then launches.  Every check runs on the host before anything is enqueued.
#include <stdint.h>

#include "../../include/lowbit_adamw.h"
#include "adamw.h"

static_assert(LOWBIT_ADAMW_BLOCK == lowbit::kAdamBlock && LOWBIT_F32 == lowbit::kAdamF32,
              "the header's constants are the library's");

namespace {

bool bad(const void* p) { return !p || (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool bad_or_null(const void* p, uintptr_t align) {
  return p && (reinterpret_cast<uintptr_t>(p) & (align - 1)) != 0;
}
bool is_type(int t) { return t == LOWBIT_F16 || t == LOWBIT_BF16 || t == LOWBIT_F32; }
// false for a NaN too
bool within(double v, double lo, double below) { return v >= lo && v < below; }
bool finite_positive(double v) { return within(v, 0.0, 1e300); }
int hip_status(hipError_t e) { return e == hipSuccess ? LOWBIT_OK : LOWBIT_ERR_HIP; }

constexpr int64_t kMostValues = (int64_t)1 << 36;

}  // namespace

extern "C" {

int lowbit_adamw(const lowbit_adamw_tensor* tensors, int64_t count, int param_dtype,
                 int grad_dtype, int bits, const lowbit_adamw_state* state,
                 const lowbit_adamw_options* options, void* hip_stream) {
  if (!is_type(param_dtype) || !is_type(grad_dtype) || (bits != 8 && bits != 32))
    return LOWBIT_ERR_UNSUPPORTED;
  if (count < 0 || !options) return LOWBIT_ERR_ARG;
  const lowbit_adamw_options& o = *options;
  if (!finite_positive(o.lr) || !finite_positive(o.eps) || !finite_positive(o.weight_decay) ||
      !within(o.beta1, 0.0, 1.0) || !within(o.beta2, 0.0, 1.0) || o.step < 1 ||
      bad_or_null(o.lr_or_null, 4) || bad_or_null(o.step_or_null, 4) ||
      bad_or_null(o.grad_scale_or_null, 4))
    return LOWBIT_ERR_ARG;
  if (count == 0) return LOWBIT_OK;
  if (!tensors || !state) return LOWBIT_ERR_ARG;
  int64_t values = 0;
  for (int64_t i = 0; i < count; i++) {
    const int64_t n = tensors[i].n;
    if (n < 0) return LOWBIT_ERR_ARG;
    if (n > kMostValues || (values += n) > kMostValues) return LOWBIT_ERR_SHAPE;
    if (n > 0 && (bad(tensors[i].param) || bad(tensors[i].grad))) return LOWBIT_ERR_ARG;
  }
  if (values == 0) return LOWBIT_OK;
  if (bad(state->m) || bad(state->v) || bad_or_null(state->master, 16)) return LOWBIT_ERR_ARG;
  if (bits == 8 ? bad(state->m_max) || bad(state->v_max) : state->m_max || state->v_max)
    return LOWBIT_ERR_ARG;
  static_assert(sizeof(lowbit_adamw_tensor) == sizeof(lowbit::AdamTensor), "one layout");
  return hip_status(lowbit::launch_adamw(
      reinterpret_cast<const lowbit::AdamTensor*>(tensors), count, param_dtype, grad_dtype, bits,
      {state->m, state->v, state->m_max, state->v_max, state->master},
      {o.lr, o.beta1, o.beta2, o.eps, o.weight_decay, o.step, o.lr_or_null, o.step_or_null,
       o.grad_scale_or_null},
      static_cast<hipStream_t>(hip_stream)));
}

int lowbit_adamw_moments(const uint8_t* m, const uint8_t* v, const float* m_max,
                         const float* v_max, int64_t blocks, float* m_out, float* v_out,
                         void* hip_stream) {
  if (blocks < 0) return LOWBIT_ERR_ARG;
  if (blocks > kMostValues / LOWBIT_ADAMW_BLOCK) return LOWBIT_ERR_SHAPE;
  if (blocks == 0) return LOWBIT_OK;
  if (bad(m) || bad(v) || bad(m_max) || bad(v_max) || bad(m_out) || bad(v_out))
    return LOWBIT_ERR_ARG;
  return hip_status(lowbit::launch_adamw_moments(m, v, m_max, v_max, blocks, m_out, v_out,
                                                 static_cast<hipStream_t>(hip_stream)));
}

}  // extern "C"
