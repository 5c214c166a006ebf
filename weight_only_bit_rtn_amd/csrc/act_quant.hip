// act_quant.hip -- per-token int8 quantization of activations.
//
// Per token t: amax = max_k |x|, S = fl32(amax / 127) (1 when that is zero),
// a = clamp(rint(fl32(x / S)), -127, 127), and the sum of the codes.  One
// workgroup per token holds its row in registers between the maximum and the
// codes, so x is read once: 2 bytes read and 1 written for each value, bound
// by HBM.
#include "w8a8.h"

namespace lowbit {
namespace {

// NC chunks of 8 values per thread, blockDim.x threads; chunk c of the row
// belongs to thread c mod blockDim.x.
template <int NC>
__global__ __launch_bounds__(1024) void quantize_act_kernel(const uint16_t* __restrict__ x,
                                                            int bf16, int K,
                                                            int8_t* __restrict__ codes,
                                                            float* __restrict__ scales,
                                                            int32_t* __restrict__ sums) {
  __shared__ int red[2][16];
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 63, wave = tid >> 6;
  const int waves = nt >> 6, chunks = K / 8;
  const int64_t row = blockIdx.x;
  const us8_t* xr = reinterpret_cast<const us8_t*>(x + row * K);
  us8_t v[NC];
  int top = 0;  // largest |x| as bits: the order of the absolute values
#pragma unroll
  for (int i = 0; i < NC; i++) {
    const int c = tid + i * nt;
    v[i] = us8_t{};
    if (c < chunks) v[i] = xr[c];
  }
#pragma unroll
  for (int i = 0; i < NC; i++)
#pragma unroll
    for (int j = 0; j < 8; j++) top = max(top, (int)(v[i][j] & 0x7fff));
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) top = max(top, __shfl_xor(top, off, kWave));
  if (lane == 0) red[0][wave] = top;
  __syncthreads();
  for (int w = 0; w < waves; w++) top = max(top, red[0][w]);
  const bool finite = top < (bf16 ? 0x7f80 : 0x7c00);
  const float amax = elem_to_f32((uint16_t)top, bf16);
  float s = amax / 127.0f;
  if (s == 0.0f) s = 1.0f;
  const float r = 1.0f / s;
  int sum = 0;
  uint2* cr = reinterpret_cast<uint2*>(codes + row * K);
#pragma unroll
  for (int i = 0; i < NC; i++) {
    const int c = tid + i * nt;
    if (c >= chunks) continue;
    uint32_t w[2] = {0, 0};
    if (finite) {
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const int a = act_code(elem_to_f32(v[i][j], bf16), s, r);
        sum += a;
        w[j / 4] |= (uint32_t)(a & 255) << (8 * (j % 4));
      }
    }
    cr[c] = make_uint2(w[0], w[1]);
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, kWave);
  if (lane == 0) red[1][wave] = sum;
  __syncthreads();
  if (tid == 0) {
    sum = 0;
    for (int w = 0; w < waves; w++) sum += red[1][w];
    scales[row] = finite ? s : __builtin_nanf("");
    sums[row] = sum;
  }
}

}  // namespace

hipError_t launch_quantize_act(const void* x, int dtype, int64_t T, int64_t K, int8_t* codes,
                               float* scales, int32_t* sums, hipStream_t stream) {
  const int chunks = (int)(K / 8);
  // Chunks per thread (us for 1 / 2 / 4): few tokens want many waves for each,
  // 1x4096 3.6 / 3.9 / 4.5; long rows fewer and fuller ones, 4096x11008
  // 39.4 / 39.8 / 33.0 (4.1 TB/s); 4096x4096 16.4 / 13.9 / 14.9.
  int nc = T <= 64 ? 1 : chunks > 1024 ? 4 : 2;
  while ((chunks + nc - 1) / nc > 1024) nc *= 2;
  const int nt = ((chunks + nc - 1) / nc + 63) / 64 * 64;
  const auto* xp = static_cast<const uint16_t*>(x);
  const dim3 grid((unsigned)T), block(nt);
  const int bf = dtype == kBF16, k = (int)K;
  if (nc <= 2)
    quantize_act_kernel<2><<<grid, block, 0, stream>>>(xp, bf, k, codes, scales, sums);
  else if (nc <= 4)
    quantize_act_kernel<4><<<grid, block, 0, stream>>>(xp, bf, k, codes, scales, sums);
  else if (nc <= 8)
    quantize_act_kernel<8><<<grid, block, 0, stream>>>(xp, bf, k, codes, scales, sums);
  else
    quantize_act_kernel<16><<<grid, block, 0, stream>>>(xp, bf, k, codes, scales, sums);
  return hipGetLastError();
}

}  // namespace lowbit
