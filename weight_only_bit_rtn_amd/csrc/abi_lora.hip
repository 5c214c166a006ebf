// abi_lora.hip -- the exported entry points of the adapters: argument checks, then
// launches.  Every check runs on the host before anything is enqueued.
#include <stdint.h>

#include "../../include/lowbit_lora.h"
#include "lora.h"

namespace {

bool bad(const void* p) { return !p || (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool bad_or_null(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

constexpr int64_t kMost = (int64_t)1 << 36;

int check_plan(int64_t T, int64_t L) {
  if (T < 0 || L < 0) return LOWBIT_ERR_ARG;
  return T > LOWBIT_W8A8_MAX_TN || L == 0 || L > LOWBIT_LORA_MAX_L ? LOWBIT_ERR_SHAPE : LOWBIT_OK;
}
int check_sizes(int64_t T, int64_t N, int64_t K, int64_t R, int64_t L) {
  const int rc = check_plan(T, L);
  if (rc != LOWBIT_OK) return rc;
  if (N < 0 || K < 0 || R < 0) return LOWBIT_ERR_ARG;
  if (N < LOWBIT_LORA_MIN_N || N > LOWBIT_W8A8_MAX_TN || K == 0 || K % 32 != 0 || K > LOWBIT_W8A8_MAX_K) return LOWBIT_ERR_SHAPE;
  if (R == 0 || R % 8 != 0 || R > LOWBIT_LORA_MAX_R) return LOWBIT_ERR_SHAPE;
  if (T * N > kMost || T * K > kMost || L * R * K > kMost || L * R * N > kMost) return LOWBIT_ERR_SHAPE;
  return LOWBIT_OK;
}
bool is_float(int dtype) { return dtype == LOWBIT_F16 || dtype == LOWBIT_BF16; }
int check_workspace(const void* ws, int64_t bytes, int64_t need) {
  if (need == 0) return LOWBIT_OK;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || bytes < need) return LOWBIT_ERR_ARG;
  return LOWBIT_OK;
}
int hip_status(hipError_t e) { return e == hipSuccess ? LOWBIT_OK : LOWBIT_ERR_HIP; }

lowbit::LoraArgs args(int64_t T, const int32_t* order, const int32_t* starts, const void* a,
                      const void* b, const float* scales, int64_t L, int64_t R, int64_t N,
                      int64_t K) {
  return {order,  starts, static_cast<const uint16_t*>(a), static_cast<const uint16_t*>(b),
          scales, (int)L, (int)R, (int)N, (int)K, T};
}

}  // namespace

extern "C" {

int lowbit_lora_plan(const int32_t* ids, int64_t T, int64_t L, int32_t* order, int32_t* starts,
                     void* hip_stream) {
  const int rc = check_plan(T, L);
  if (rc != LOWBIT_OK) return rc;
  if (bad(starts) || (T > 0 && (bad(ids) || bad(order)))) return LOWBIT_ERR_ARG;
  return hip_status(lowbit::launch_lora_plan(ids, T, L, order, starts,
                                             static_cast<hipStream_t>(hip_stream)));
}

int64_t lowbit_lora_workspace_bytes(int64_t T, int64_t N, int64_t K, int64_t R, int64_t L) {
  const int rc = check_sizes(T, N, K, R, L);
  return rc != LOWBIT_OK ? rc : (int64_t)lowbit::lora_workspace_bytes({T, N, K, R, L});
}

int lowbit_lora(const void* x, int dtype, int64_t T, const int32_t* order, const int32_t* starts,
                const void* a, const void* b, const float* scales, int64_t L, int64_t R, int64_t N,
                int64_t K, const void* y_or_null, void* out, float* v_or_null, void* workspace,
                int64_t workspace_bytes, void* hip_stream) {
  const int64_t need = lowbit_lora_workspace_bytes(T, N, K, R, L);
  if (need < 0) return (int)need;
  if (!is_float(dtype)) return LOWBIT_ERR_UNSUPPORTED;
  if (T == 0) return LOWBIT_OK;
  if (bad(x) || bad(order) || bad(starts) || bad(a) || bad(b) || bad(scales) ||
      bad_or_null(y_or_null) || bad(out) || bad_or_null(v_or_null))
    return LOWBIT_ERR_ARG;
  const int rc = check_workspace(workspace, workspace_bytes, need);
  if (rc != LOWBIT_OK) return rc;
  return hip_status(lowbit::launch_lora(x, dtype, args(T, order, starts, a, b, scales, L, R, N, K),
                                        y_or_null, out, v_or_null, workspace,
                                        static_cast<hipStream_t>(hip_stream)));
}

int64_t lowbit_lora_grad_workspace_bytes(int64_t T, int64_t N, int64_t K, int64_t R, int64_t L) {
  const int rc = check_sizes(T, N, K, R, L);
  return rc != LOWBIT_OK ? rc : (int64_t)lowbit::lora_grad_workspace_bytes({T, N, K, R, L});
}

int lowbit_lora_grad(const void* dy, const void* x, const float* v, int dtype, int64_t T,
                     const int32_t* order, const int32_t* starts, const void* a, const void* b,
                     const float* scales, int64_t L, int64_t R, int64_t N, int64_t K,
                     const void* base_or_null, void* dx, float* da, float* db, void* workspace,
                     int64_t workspace_bytes, void* hip_stream) {
  const int64_t need = lowbit_lora_grad_workspace_bytes(T, N, K, R, L);
  if (need < 0) return (int)need;
  if (!is_float(dtype)) return LOWBIT_ERR_UNSUPPORTED;
  if (bad(da) || bad(db)) return LOWBIT_ERR_ARG;
  if (T > 0 && (bad(dy) || bad(x) || bad(v) || bad(order) || bad(starts) || bad(a) || bad(b) ||
                bad(scales) || bad_or_null(base_or_null) || bad(dx)))
    return LOWBIT_ERR_ARG;
  const int rc = check_workspace(workspace, workspace_bytes, need);
  if (rc != LOWBIT_OK) return rc;
  return hip_status(lowbit::launch_lora_grad(dy, x, v, dtype,
                                             args(T, order, starts, a, b, scales, L, R, N, K),
                                             base_or_null, dx, da, db, workspace,
                                             static_cast<hipStream_t>(hip_stream)));
}

}  // extern "C"
