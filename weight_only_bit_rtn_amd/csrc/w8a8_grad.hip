// w8a8_grad.hip -- input gradients through frozen 8-bit weights: of the
// linear layer and of the gated block.
//
//   dx[t][k] = sum_n d[t][n] s_n (code[n][k] - z_n)
//
// The rows' scales belong to the summed index, so they go into the gradient:
// a = d s, and with c' = code - 128, an exact fp16 integer,
//   dx[t][k] = 2^-e_t (sum_n a'[t][n] c'[n][k] + r_t),
//   a' = fp16(2^e_t a),  r_t = sum_n a'[t][n] (128 - z_n).
// e_t makes a token's largest |a'| lie in [2^14, 2^15): gradients of any size
// keep their 11 significant bits.  Rounding a to fp16 is the one rounding
// between the inputs and the output: the matrix cores take 16-bit operands at
// the rate measured here, and bf16 would keep 8 bits.
//
// Two kernels: one makes a', e and r (and, for the gated block, the gradients
// of both projections on the way), one multiplies.  The gated block's two
// products are one sum over the gate rows and then the up rows.
#include "w8a8.h"

namespace lowbit {
namespace {

constexpr int kStepN = 64;  // weight rows per pipeline step

struct PrepArgs {
  const uint16_t* d;
  const uint16_t* gate;
  const uint16_t* up;
  W8 w[2];
  uint16_t* a;  // [T][pitch]: gate part, then (from half) up part, zero padded
  float* r;
  int32_t* e;
  uint16_t* dgate;
  uint16_t* dup;
  int N, pitch, half, act, bf16;
};

__device__ __forceinline__ float block_sum(float v, float* red, int tid) {
  v = wave_sum_dpp(v);
  __syncthreads();
  if ((tid & 63) == 0) red[tid >> 6] = v;
  __syncthreads();
  v = 0;
  for (int w = 0; w < (int)blockDim.x / 64; w++) v += red[w];
  return v;
}
__device__ __forceinline__ float block_max(float v, float* red, int tid) {
  v = wave_max(v);
  __syncthreads();
  if ((tid & 63) == 0) red[tid >> 6] = v;
  __syncthreads();
  v = 0;
  for (int w = 0; w < (int)blockDim.x / 64; w++) v = fmaxf(v, red[w]);
  return v;
}

// One workgroup per token.
template <bool GATED>
__global__ __launch_bounds__(1024) void grad_prep_kernel(const PrepArgs p) {
  __shared__ float red[16];
  const int tid = threadIdx.x, nt = blockDim.x;
  const int64_t row = blockIdx.x;
  const bool bf = p.bf16;
  const uint16_t* d = p.d + row * p.N;
  // the (one or two) gradients of position n, before the weight scales
  auto grads = [&](int n, float& d0, float& d1) {
    d0 = elem_to_f32(d[n], bf);
    if constexpr (GATED) {
      float f, df;
      act_value_slope(elem_to_f32(p.gate[row * p.N + n], bf), p.act, f, df);
      const float u = elem_to_f32(p.up[row * p.N + n], bf);
      d1 = d0 * f;
      d0 = d0 * u * df;
    }
  };
  float top = 0;
  bool finite = true;
  for (int n = tid; n < p.N; n += nt) {
    float d0, d1 = 0;
    grads(n, d0, d1);
    finite = finite && fabsf(d0) < INFINITY && fabsf(d1) < INFINITY;
    top = fmaxf(top, fabsf(d0 * h_bits_to_f32(p.w[0].scales[n])));
    if constexpr (GATED) {
      top = fmaxf(top, fabsf(d1 * h_bits_to_f32(p.w[1].scales[n])));
      if (p.dgate) {
        p.dgate[row * p.N + n] = f32_to_elem(d0, bf);
        p.dup[row * p.N + n] = f32_to_elem(d1, bf);
      }
    }
  }
  top = block_max(finite ? top : INFINITY, red, tid);
  const bool ok = top < INFINITY;
  const int e = ok && top > 0 ? 15 - __builtin_amdgcn_frexp_expf(top) : 0;
  float r = 0;
  uint16_t* a = p.a + row * p.pitch;
  for (int n = tid; n < p.half; n += nt) {
    uint16_t a0 = 0, a1 = 0;
    if (n < p.N && ok) {
      float d0, d1 = 0;
      grads(n, d0, d1);
      a0 = f32_to_h_bits(__builtin_amdgcn_ldexpf(d0 * h_bits_to_f32(p.w[0].scales[n]), e));
      r += h_bits_to_f32(a0) * (float)(128 - p.w[0].zeros[n]);
      if constexpr (GATED) {
        a1 = f32_to_h_bits(__builtin_amdgcn_ldexpf(d1 * h_bits_to_f32(p.w[1].scales[n]), e));
        r += h_bits_to_f32(a1) * (float)(128 - p.w[1].zeros[n]);
      }
    }
    a[n] = a0;
    if constexpr (GATED) a[p.half + n] = a1;
  }
  r = block_sum(r, red, tid);
  if (tid == 0) {
    p.r[row] = ok ? r : __builtin_nanf("");
    p.e[row] = e;
  }
}

struct GradArgs {
  const uint16_t* a;
  const float* r;
  const int32_t* e;
  W8 w[2];
  void* dx;
  int T, N, K, pitch, half_steps, steps, bf16, tiles_m, tiles_n;
};

// Four code bytes to the exact fp16 integers code - 128: one byte permute
// drops two codes under the exponent bytes of 1024, one packed subtraction.
__device__ __forceinline__ void codes_to_f16(uint32_t w, h2_t& lo, h2_t& hi) {
  const h2_t off = {(_Float16)1152.0f, (_Float16)1152.0f};
  lo = as_h2(__builtin_amdgcn_perm(0x64646464u, w, 0x04010400u)) - off;
  hi = as_h2(__builtin_amdgcn_perm(0x64646464u, w, 0x04030402u)) - off;
}

// One workgroup of WM x WN waves: MT tokens by KT columns of dx, steps of 64
// weight rows through LDS in two buffers, one barrier per step.  The weight
// tile lies as it does in memory, rows of KT code bytes; the matrix cores
// need eight rows of one column per lane, which the transposing LDS read
// delivers (16 lanes read 8 rows of 16 bytes and get a column each).  Chunk c
// (16 bytes) of a row lies at c ^ (row & 7) in both tiles, so that neither
// kind of read meets one bank twice.
template <int MT, int KT, int WM, int WN>
__global__ __launch_bounds__(WM* WN * 64) void grad_kernel(const GradArgs p) {
  constexpr int kWaves = WM * WN;
  constexpr int MW = MT / WM, KW = KT / WN;
  constexpr int FM = MW / 16, FK = KW / 16;
  constexpr int kA = MT * kStepN * 2, kW = kStepN * KT, kBuf = kA + kW;
  constexpr int LA = kA / 1024 / kWaves, LW = kW / 1024 / kWaves;
  constexpr int kRows = 1024 / KT;  // weight rows per load
  static_assert(LA * 1024 * kWaves == kA && LW * 1024 * kWaves == kW, "whole loads");
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WM, wn = wave / WM;
  const int i16 = lane & 15, h = lane >> 4;
  int tm, tn;
  tile_of(blockIdx.x, gridDim.x, p.tiles_m, p.tiles_n, tm, tn);
  const int t0 = tm * MT, k0 = tn * KT;
  const uint32_t K = (uint32_t)p.K;

  const uint32_t pitch = (uint32_t)p.pitch * 2;
  const auto ra = buffer_of(p.a + (int64_t)t0 * p.pitch, (uint32_t)min(MT, p.T - t0) * pitch);
  uint32_t oa[LA], ow[LW];
  int la[LA], lw[LW], rw[LW];
#pragma unroll
  for (int i = 0; i < LA; i++) {
    const int row = (wave + i * kWaves) * 8;
    oa[i] = (uint32_t)(row + (lane >> 3)) * pitch + ((lane & 7) ^ (lane >> 3)) * 16;
    la[i] = row * kStepN * 2;
  }
  constexpr int kLanes = KT / 16;  // lanes per weight row
#pragma unroll
  for (int i = 0; i < LW; i++) {
    rw[i] = (wave + i * kWaves) * kRows + lane / kLanes;
    const int c = (lane % kLanes) ^ (rw[i] & 7);
    // columns past the end: not stored, so not loaded either
    ow[i] = k0 + c * 16 < p.K ? (uint32_t)rw[i] * K + k0 + c * 16 : 0x80000000u;
    lw[i] = kA + (wave + i * kWaves) * 1024;
  }
  auto stage = [&](uint32_t buf, int s) {
#pragma unroll
    for (int i = 0; i < LA; i++) load_to_lds(ra, buf + la[i], oa[i] + (uint32_t)s * (kStepN * 2));
    const int m = s >= p.half_steps;
    const int n = (s - m * p.half_steps) * kStepN;
    const auto rs = buffer_of(p.w[m].codes + (int64_t)n * K,
                              (uint32_t)max(0, min(kStepN, p.N - n)) * K);
#pragma unroll
    for (int i = 0; i < LW; i++) load_to_lds(rs, buf + lw[i], ow[i]);
  };

  f4_t acc[FK][FM];
#pragma unroll
  for (int i = 0; i < FK; i++)
#pragma unroll
    for (int j = 0; j < FM; j++) acc[i][j] = f4_t{0, 0, 0, 0};

  const uint32_t base = lds_address(lds);
  if (p.steps > 0) stage(base, 0);
  for (int s = 0; s < p.steps; s++) {
    uint8_t* buf = lds + (s & 1) * kBuf;
    lds_loads_left<0>();  // this step's loads of this wave have landed
    __syncthreads();   // and everyone's; the other buffer is free
    if (s + 1 < p.steps) stage(base + ((s + 1) & 1) * kBuf, s + 1);
    const uint8_t* ba = buf + (wm * MW + i16) * (kStepN * 2);
    const uint8_t* bw = buf + kA;
#pragma unroll
    for (int ks = 0; ks < 2; ks++) {
      h8_t fa[FM], fw[FK];
      // lanes 2r and 2r + 1 of 16 read the two halves of row r's 16 bytes
      const int n = ks * 32 + h * 8 + (i16 >> 1);
#pragma unroll
      for (int i = 0; i < FK; i++) {
        const int c = (wn * KW / 16 + i) ^ (n & 7);
        const i2_t w = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            (__attribute__((address_space(3))) i2_t*)(bw + n * KT + c * 16 + (i16 & 1) * 8));
        h2_t q[4];
        codes_to_f16((uint32_t)w[0], q[0], q[1]);
        codes_to_f16((uint32_t)w[1], q[2], q[3]);
        fw[i] = h8_t{q[0][0], q[0][1], q[1][0], q[1][1], q[2][0], q[2][1], q[3][0], q[3][1]};
      }
      const int at = ((ks * 4 + h) ^ (i16 & 7)) * 16;
#pragma unroll
      for (int j = 0; j < FM; j++)
        fa[j] = *reinterpret_cast<const h8_t*>(ba + j * 16 * (kStepN * 2) + at);
#pragma unroll
      for (int i = 0; i < FK; i++)
#pragma unroll
        for (int j = 0; j < FM; j++)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fw[i], fa[j], acc[i][j], 0, 0, 0);
    }
  }

  const bool bf = p.bf16;
#pragma unroll
  for (int j = 0; j < FM; j++) {
    const int t = t0 + wm * MW + j * 16 + i16;
    if (t >= p.T) continue;
    const float r = p.r[t];
    const int e = -p.e[t];
#pragma unroll
    for (int i = 0; i < FK; i++) {
      const int k = k0 + wn * KW + i * 16 + h * 4;
      if (k >= p.K) continue;
      us4_t out;
#pragma unroll
      for (int q = 0; q < 4; q++)
        out[q] = f32_to_elem(__builtin_amdgcn_ldexpf(acc[i][j][q] + r, e), bf);
      *reinterpret_cast<us4_t*>(static_cast<uint16_t*>(p.dx) + (int64_t)t * p.K + k) = out;
    }
  }
}

template <int MT, int KT, int WM, int WN>
hipError_t launch_tile(GradArgs p, hipStream_t stream) {
  constexpr int bytes = 2 * (MT * kStepN * 2 + kStepN * KT);
  auto kernel = grad_kernel<MT, KT, WM, WN>;
  hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(kernel), bytes);
  if (e != hipSuccess) return e;
  p.tiles_m = (p.T + MT - 1) / MT;
  p.tiles_n = (p.K + KT - 1) / KT;
  const int64_t total = (int64_t)p.tiles_m * p.tiles_n;
  if (total > INT32_MAX) return hipErrorInvalidValue;
  kernel<<<dim3((unsigned)total), dim3(WM * WN * 64), bytes, stream>>>(p);
  return hipGetLastError();
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }
int64_t padded(int64_t N) { return (N + kStepN - 1) / kStepN * kStepN; }

}  // namespace

size_t w8a8_grad_workspace_bytes(int64_t T, int64_t N, int64_t K, bool gated) {
  if (T == 0) return 0;
  return up256((size_t)T * padded(N) * (gated ? 4 : 2)) + 2 * up256((size_t)T * 4);
}

hipError_t launch_w8a8_grad(const void* dh, const void* gate, const void* up, int dtype, int64_t T,
                            const W8& wg, const W8& wu, bool gated, int64_t N, int64_t K, int act,
                            void* dx, void* dgate, void* dup, void* workspace,
                            hipStream_t stream) {
  const int64_t half = padded(N), pitch = gated ? 2 * half : half;
  auto* ws = static_cast<uint8_t*>(workspace);
  PrepArgs q{};
  q.d = static_cast<const uint16_t*>(dh);
  q.gate = static_cast<const uint16_t*>(gate);
  q.up = static_cast<const uint16_t*>(up);
  q.w[0] = wg;
  q.w[1] = wu;
  q.a = reinterpret_cast<uint16_t*>(ws);
  q.r = reinterpret_cast<float*>(ws + up256((size_t)T * pitch * 2));
  q.e = reinterpret_cast<int32_t*>(ws + up256((size_t)T * pitch * 2) + up256((size_t)T * 4));
  q.dgate = static_cast<uint16_t*>(dgate);
  q.dup = static_cast<uint16_t*>(dup);
  q.N = (int)N;
  q.pitch = (int)pitch;
  q.half = (int)half;
  q.act = act;
  q.bf16 = dtype == kBF16;
  int nt = 64;
  while (nt < 1024 && nt * 8 < N) nt *= 2;
  if (gated)
    grad_prep_kernel<true><<<dim3((unsigned)T), dim3(nt), 0, stream>>>(q);
  else
    grad_prep_kernel<false><<<dim3((unsigned)T), dim3(nt), 0, stream>>>(q);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  GradArgs p{};
  p.a = q.a;
  p.r = q.r;
  p.e = q.e;
  p.w[0] = wg;
  p.w[1] = wu;
  p.dx = dx;
  p.T = (int)T;
  p.N = (int)N;
  p.K = (int)K;
  p.pitch = (int)pitch;
  p.half_steps = (int)(half / kStepN);
  p.steps = (int)(pitch / kStepN);
  p.bf16 = q.bf16;
  if (T <= 64) return launch_tile<64, 128, 2, 2>(p, stream);
  if (T <= 512) return launch_tile<128, 128, 2, 2>(p, stream);
  return launch_tile<256, 256, 2, 4>(p, stream);
}

}  // namespace lowbit
