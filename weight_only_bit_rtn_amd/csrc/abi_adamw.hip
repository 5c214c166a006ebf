// abi_adamw.hip -- the exported entry points of the AdamW step: argument checks,
// then launches.  Every check runs on the host before anything is enqueued.
#include <stdint.h>

#include <algorithm>
#include <memory>
#include <new>

#include "../../include/lowbit_adamw.h"
#include "adamw.h"

static_assert(LOWBIT_ADAMW_BLOCK == lowbit::kAdamBlock && LOWBIT_F32 == lowbit::kAdamF32 &&
                  LOWBIT_ADAMW_RANDOM == lowbit::kAdamRandom,
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

// What a step writes (tensors, moments, their maxima, the copy), in order of addresses: no
// piece may meet another, nor anything that the step reads (gradients, its scalars).  448
// tensors take 19 us of the host, 25 in a random order of addresses; a pair less than 1.
struct Piece {
  uintptr_t at, end;
};
class Written {
 public:
  explicit Written(int64_t most)
      : heap_(most > kFew ? new (std::nothrow) Piece[most] : nullptr), p_(most > kFew ? heap_.get() : few_) {}
  bool has_room() const { return p_ != nullptr; }
  void add(const void* at, int64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(at);
    if (at && bytes > 0) p_[n_++] = {a, a + bytes};
  }
  // Whether no piece meets the next; before the first question about others.
  bool apart() {
    const auto lower = [](const Piece& x, const Piece& y) { return x.at < y.at; };
    if (!std::is_sorted(p_, p_ + n_, lower)) std::sort(p_, p_ + n_, lower);
    for (int64_t i = 1; i < n_; i++)
      if (p_[i - 1].end > p_[i].at) return false;
    return true;
  }
  bool meets(const void* at, int64_t bytes) const {
    const uintptr_t a = reinterpret_cast<uintptr_t>(at);
    if (!at || bytes <= 0) return false;
    const Piece* next = std::upper_bound(p_, p_ + n_, a, [](uintptr_t x, const Piece& y) { return x < y.at; });
    return (next != p_ + n_ && next->at < a + bytes) || (next != p_ && next[-1].end > a);
  }

 private:
  static constexpr int64_t kFew = 64;
  Piece few_[kFew];
  std::unique_ptr<Piece[]> heap_;
  Piece* p_;
  int64_t n_ = 0;
};

}  // namespace

extern "C" {

int lowbit_adamw(const lowbit_adamw_tensor* tensors, int64_t count, int param_dtype,
                 int grad_dtype, int bits, const lowbit_adamw_state* state,
                 const lowbit_adamw_options* options, void* hip_stream) {
  if (!is_type(param_dtype) || !is_type(grad_dtype) ||
      (bits != 8 && bits != (8 | LOWBIT_ADAMW_RANDOM) && bits != 32))
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
  if (bits != 32 ? bad(state->m_max) || bad(state->v_max) : state->m_max || state->v_max)
    return LOWBIT_ERR_ARG;
  Written written(count + 5);
  if (!written.has_room()) return LOWBIT_ERR_HIP;  // no host memory
  const int64_t pw = param_dtype == LOWBIT_F32 ? 4 : 2, gw = grad_dtype == LOWBIT_F32 ? 4 : 2;
  const int64_t mw = bits == 32 ? 4 : 1;
  int64_t blocks = 0;
  for (int64_t i = 0; i < count; i++) {
    written.add(tensors[i].param, tensors[i].n * pw);
    blocks += (tensors[i].n + LOWBIT_ADAMW_BLOCK - 1) / LOWBIT_ADAMW_BLOCK;
  }
  written.add(state->m, blocks * LOWBIT_ADAMW_BLOCK * mw);
  written.add(state->v, blocks * LOWBIT_ADAMW_BLOCK * mw);
  written.add(state->m_max, blocks * 4);
  written.add(state->v_max, blocks * 4);
  written.add(state->master, blocks * LOWBIT_ADAMW_BLOCK * 4);
  if (!written.apart() || written.meets(o.lr_or_null, 4) || written.meets(o.step_or_null, 4) ||
      written.meets(o.grad_scale_or_null, 4))
    return LOWBIT_ERR_ARG;
  for (int64_t i = 0; i < count; i++)
    if (written.meets(tensors[i].grad, tensors[i].n * gw)) return LOWBIT_ERR_ARG;
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
