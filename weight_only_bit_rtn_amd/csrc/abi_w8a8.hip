// abi_w8a8.hip -- the exported entry points of the 8-bit activation products:
// argument checks, then launches.  Every check runs on the host before
// anything is enqueued.
#include <stdint.h>

#include "../../include/lowbit_w8a8.h"
#include "w8a8.h"

static_assert(LOWBIT_F16 == lowbit::kF16 && LOWBIT_BF16 == lowbit::kBF16 &&
                  LOWBIT_I8 == lowbit::kI8 && LOWBIT_ACT_SILU == lowbit::kSilu &&
                  LOWBIT_ACT_GELU_TANH == lowbit::kGeluTanh,
              "the header's type and activation codes are the library's");

namespace {

bool bad(const void* p) { return !p || (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool bad_or_null(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// keeps every grid within 2^32 threads
constexpr int64_t kMostOutputs = (int64_t)1 << 36;

int check_sizes(int64_t T, int64_t N, int64_t K) {
  if (T < 0 || N < 0 || K < 0) return LOWBIT_ERR_ARG;
  if (T > LOWBIT_W8A8_MAX_TN || N > LOWBIT_W8A8_MAX_TN) return LOWBIT_ERR_SHAPE;
  if (K == 0 || K % 32 != 0 || K > LOWBIT_W8A8_MAX_K) return LOWBIT_ERR_SHAPE;
  if (T * N > kMostOutputs || T * K > kMostOutputs) return LOWBIT_ERR_SHAPE;
  return LOWBIT_OK;
}
bool is_float(int dtype) { return dtype == LOWBIT_F16 || dtype == LOWBIT_BF16; }
int check_act(int act) {
  return act == LOWBIT_ACT_SILU || act == LOWBIT_ACT_GELU_TANH ? LOWBIT_OK
                                                               : LOWBIT_ERR_UNSUPPORTED;
}
bool bad_weights(const uint32_t* packed, const uint16_t* scales, const int32_t* zeros) {
  return bad(packed) || bad(scales) || bad(zeros);
}
int check_workspace(const void* ws, int64_t bytes, int64_t need) {
  if (need == 0) return LOWBIT_OK;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || bytes < need) return LOWBIT_ERR_ARG;
  return LOWBIT_OK;
}
// fp16 and bf16 activations come alone, codes with their scales and sums.
int check_activations(const void* x, int dtype, const float* xs, const int32_t* sums) {
  if (bad(x)) return LOWBIT_ERR_ARG;
  if (dtype == LOWBIT_I8) return bad(xs) || bad(sums) ? LOWBIT_ERR_ARG : LOWBIT_OK;
  return xs || sums ? LOWBIT_ERR_ARG : LOWBIT_OK;
}
lowbit::W8 w8(const uint32_t* packed, const uint16_t* scales, const int32_t* zeros) {
  return {reinterpret_cast<const uint8_t*>(packed), scales, zeros};
}
int hip_status(hipError_t e) { return e == hipSuccess ? LOWBIT_OK : LOWBIT_ERR_HIP; }

int64_t product_workspace(int64_t T, int64_t N, int64_t K, int dtype, bool gated) {
  if (!is_float(dtype) && dtype != LOWBIT_I8) return LOWBIT_ERR_UNSUPPORTED;
  const int rc = check_sizes(T, N, K);
  return rc != LOWBIT_OK ? rc : (int64_t)lowbit::w8a8_workspace_bytes(T, N, K, dtype, gated);
}
int64_t grad_workspace(int64_t T, int64_t N, int64_t K, bool gated) {
  const int rc = check_sizes(T, N, K);
  return rc != LOWBIT_OK ? rc : (int64_t)lowbit::w8a8_grad_workspace_bytes(T, N, K, gated);
}

}  // namespace

extern "C" {

int lowbit_quantize_act(const void* x, int dtype, int64_t T, int64_t K, int8_t* codes,
                        float* scales, int32_t* sums, void* hip_stream) {
  if (!is_float(dtype)) return LOWBIT_ERR_UNSUPPORTED;
  const int rc = check_sizes(T, 0, K);
  if (rc != LOWBIT_OK || T == 0) return rc;
  if (bad(x) || bad(codes) || bad(scales) || bad(sums)) return LOWBIT_ERR_ARG;
  return hip_status(lowbit::launch_quantize_act(x, dtype, T, K, codes, scales, sums,
                                                static_cast<hipStream_t>(hip_stream)));
}

int64_t lowbit_linear_w8a8_workspace_bytes(int64_t T, int64_t N, int64_t K, int dtype) {
  return product_workspace(T, N, K, dtype, false);
}

int lowbit_linear_w8a8(const void* x, int dtype, const float* x_scales, const int32_t* x_sums,
                       int64_t T, const uint32_t* packed, const uint16_t* scales_f16,
                       const int32_t* zeros, int64_t N, int64_t K, void* y, int out_dtype,
                       void* workspace, int64_t workspace_bytes, void* hip_stream) {
  const int64_t need = product_workspace(T, N, K, dtype, false);
  if (need < 0) return (int)need;
  if (!is_float(out_dtype)) return LOWBIT_ERR_UNSUPPORTED;
  if (T == 0 || N == 0) return LOWBIT_OK;
  int rc = check_activations(x, dtype, x_scales, x_sums);
  if (rc != LOWBIT_OK) return rc;
  if (bad_weights(packed, scales_f16, zeros) || bad(y)) return LOWBIT_ERR_ARG;
  rc = check_workspace(workspace, workspace_bytes, need);
  if (rc != LOWBIT_OK) return rc;
  return hip_status(lowbit::launch_linear_w8a8(
      {x, dtype, x_scales, x_sums}, T, w8(packed, scales_f16, zeros), N, K, y, out_dtype,
      workspace, static_cast<hipStream_t>(hip_stream)));
}

int64_t lowbit_gated_w8a8_workspace_bytes(int64_t T, int64_t N, int64_t K, int dtype) {
  return product_workspace(T, N, K, dtype, true);
}

int lowbit_gated_w8a8(const void* x, int dtype, const float* x_scales, const int32_t* x_sums,
                      int64_t T, const uint32_t* packed_gate, const uint16_t* scales_gate,
                      const int32_t* zeros_gate, const uint32_t* packed_up,
                      const uint16_t* scales_up, const int32_t* zeros_up, int64_t N, int64_t K,
                      int act, void* h, void* gate_or_null, void* up_or_null, int out_dtype,
                      void* workspace, int64_t workspace_bytes, void* hip_stream) {
  const int64_t need = product_workspace(T, N, K, dtype, true);
  if (need < 0) return (int)need;
  if (!is_float(out_dtype)) return LOWBIT_ERR_UNSUPPORTED;
  int rc = check_act(act);
  if (rc != LOWBIT_OK) return rc;
  if (T == 0 || N == 0) return LOWBIT_OK;
  rc = check_activations(x, dtype, x_scales, x_sums);
  if (rc != LOWBIT_OK) return rc;
  if (bad_weights(packed_gate, scales_gate, zeros_gate) ||
      bad_weights(packed_up, scales_up, zeros_up) || bad(h) || bad_or_null(gate_or_null) ||
      bad_or_null(up_or_null) || !gate_or_null != !up_or_null)
    return LOWBIT_ERR_ARG;
  rc = check_workspace(workspace, workspace_bytes, need);
  if (rc != LOWBIT_OK) return rc;
  return hip_status(lowbit::launch_gated_w8a8(
      {x, dtype, x_scales, x_sums}, T, w8(packed_gate, scales_gate, zeros_gate),
      w8(packed_up, scales_up, zeros_up), N, K, act, h, gate_or_null, up_or_null, out_dtype,
      workspace, static_cast<hipStream_t>(hip_stream)));
}

int64_t lowbit_linear_w8a8_grad_workspace_bytes(int64_t T, int64_t N, int64_t K) {
  return grad_workspace(T, N, K, false);
}

int lowbit_linear_w8a8_grad(const void* dy, int dtype, int64_t T, const uint32_t* packed,
                            const uint16_t* scales_f16, const int32_t* zeros, int64_t N,
                            int64_t K, void* dx, void* workspace, int64_t workspace_bytes,
                            void* hip_stream) {
  const int64_t need = grad_workspace(T, N, K, false);
  if (need < 0) return (int)need;
  if (!is_float(dtype)) return LOWBIT_ERR_UNSUPPORTED;
  if (T == 0) return LOWBIT_OK;
  if (bad(dx)) return LOWBIT_ERR_ARG;
  if (N > 0 && (bad(dy) || bad_weights(packed, scales_f16, zeros))) return LOWBIT_ERR_ARG;
  const int rc = check_workspace(workspace, workspace_bytes, need);
  if (rc != LOWBIT_OK) return rc;
  const lowbit::W8 w = w8(packed, scales_f16, zeros);
  return hip_status(lowbit::launch_w8a8_grad(dy, nullptr, nullptr, dtype, T, w, w, false, N, K, 0,
                                             dx, nullptr, nullptr, workspace,
                                             static_cast<hipStream_t>(hip_stream)));
}

int64_t lowbit_gated_w8a8_grad_workspace_bytes(int64_t T, int64_t N, int64_t K) {
  return grad_workspace(T, N, K, true);
}

int lowbit_gated_w8a8_grad(const void* dh, const void* gate, const void* up, int dtype, int64_t T,
                           const uint32_t* packed_gate, const uint16_t* scales_gate,
                           const int32_t* zeros_gate, const uint32_t* packed_up,
                           const uint16_t* scales_up, const int32_t* zeros_up, int64_t N,
                           int64_t K, int act, void* dx, void* dgate_or_null, void* dup_or_null,
                           void* workspace, int64_t workspace_bytes, void* hip_stream) {
  const int64_t need = grad_workspace(T, N, K, true);
  if (need < 0) return (int)need;
  if (!is_float(dtype)) return LOWBIT_ERR_UNSUPPORTED;
  int rc = check_act(act);
  if (rc != LOWBIT_OK) return rc;
  if (T == 0) return LOWBIT_OK;
  if (bad(dx)) return LOWBIT_ERR_ARG;
  if (N > 0 && (bad(dh) || bad(gate) || bad(up) ||
                bad_weights(packed_gate, scales_gate, zeros_gate) ||
                bad_weights(packed_up, scales_up, zeros_up) || bad_or_null(dgate_or_null) ||
                bad_or_null(dup_or_null) || !dgate_or_null != !dup_or_null))
    return LOWBIT_ERR_ARG;
  rc = check_workspace(workspace, workspace_bytes, need);
  if (rc != LOWBIT_OK) return rc;
  return hip_status(lowbit::launch_w8a8_grad(
      dh, gate, up, dtype, T, w8(packed_gate, scales_gate, zeros_gate),
      w8(packed_up, scales_up, zeros_up), true, N, K, act, dx, dgate_or_null, dup_or_null,
      workspace, static_cast<hipStream_t>(hip_stream)));
}

}  // extern "C"
