// w8a8_few.hip -- the 8-bit products for one to four tokens: a decoding step.
//
// Reading the weights is all that takes time (one byte each, used once per
// token), so each wave reads whole rows as they lie, 1 KiB per instruction,
// and multiplies with v_dot4_i32_i8; the matrix cores would want 16 rows per
// instruction, 64 bytes of each, and reading in such pieces ran at 5.0-5.6
// TB/s where whole rows run at 5.9.
//
// One workgroup of 16 waves per CU keeps the tokens' codes in LDS: it
// quantizes x itself when that is little (T K <= kFusedMost), while its
// first weights are on their way, and copies codes otherwise.  Wave w of
// workgroup b takes rows w G + b, then 16 G further (G workgroups), so few
// rows still spread over all CUs.  Two loads per lane are in flight, running
// ahead into the wave's next rows: 16 waves cover the latency, and loads past
// the last row only cost time (2 / 4 / 8 per lane, kernel alone, on weights rotated
// over 1 GiB: 1x256x256 4.6 / 5.1 / 6.3 us, 1x4096x4096 7.2 / 7.4 / 8.4, gated
// 1x28672x8192 79 / 81 / 80, 1x49152x12288 103 / 101 / 101).
#include "w8a8.h"

namespace lowbit {
namespace {

constexpr int kWaves = 16;
constexpr int kChunk = kFewChunk;  // bytes of a row per load
constexpr int kInFlight = 2;   // loads per lane

// Sum over the 64 lanes, in lane 63.
__device__ __forceinline__ int wave_sum_last(int v) {
#define LOWBIT_ADD(ctrl, rows) v += __builtin_amdgcn_update_dpp(0, v, ctrl, rows, 0xf, false)
  LOWBIT_ADD(0xb1, 0xf);   // quad_perm [1,0,3,2]
  LOWBIT_ADD(0x4e, 0xf);   // quad_perm [2,3,0,1]
  LOWBIT_ADD(0x141, 0xf);  // row_half_mirror
  LOWBIT_ADD(0x140, 0xf);  // row_mirror
  LOWBIT_ADD(0x142, 0xa);  // row_bcast:15 into rows 1 and 3
  LOWBIT_ADD(0x143, 0xc);  // row_bcast:31 into rows 2 and 3
#undef LOWBIT_ADD
  return v;
}

// Codes of all tokens into LDS (rows of few_pitch), scales and sums into meta
// (token t: meta[t] and meta[8 + t]).  Tokens share the waves out: 16 / TT
// waves each, the token's values held in registers between its maximum and
// its codes.  Ends with a barrier.
template <int TT>
__device__ __forceinline__ void quantize_here(const GemmArgs& p, int8_t* codes, int* meta,
                                              int* red) {
  constexpr int W = kWaves / TT;  // waves per token
  // Chunks of 8 values per lane: T K <= kFusedMost, and TT is the smallest power of
  // two that holds T, so T is TT / 2 + 1 at least and a row with its padding at most
  // few_pitch(kFusedMost / T) long.
  constexpr int NC = TT <= 2 ? 2 : 3;
  static_assert(few_pitch(kFusedMost / (TT / 2 + 1)) <= NC * 64 * W * 8, "whole rows");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int t = wave / W, part = wave % W;
  const bool mine = t < p.T;
  const int chunks = p.K / 8, all = few_pitch(p.K) / 8;
  us8_t v[NC];
  int top = 0;
  const us8_t* xr = reinterpret_cast<const us8_t*>(p.x + (int64_t)(mine ? t : 0) * p.K);
#pragma unroll
  for (int i = 0; i < NC; i++) {
    const int c = part * 64 + lane + i * (64 * W);
    v[i] = us8_t{};
    if (c < chunks) v[i] = xr[c];
  }
#pragma unroll
  for (int i = 0; i < NC; i++)
#pragma unroll
    for (int j = 0; j < 8; j++) top = max(top, (int)(v[i][j] & 0x7fff));
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) top = max(top, __shfl_xor(top, off, kWave));
  if (lane == 0) red[wave] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < W; w++) top = max(top, red[t * W + w]);
  const bool finite = top < (p.x_bf16 ? 0x7f80 : 0x7c00);
  float s = elem_to_f32((uint16_t)top, p.x_bf16) / 127.0f;
  if (s == 0.0f) s = 1.0f;
  const float r = 1.0f / s;
  int sum = 0;
#pragma unroll
  for (int i = 0; i < NC; i++) {
    const int c = part * 64 + lane + i * (64 * W);
    uint32_t w[2] = {0, 0};
    if (c < chunks && finite) {
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const int a = act_code(elem_to_f32(v[i][j], p.x_bf16), s, r);
        sum += a;
        w[j / 4] |= (uint32_t)(a & 255) << (8 * (j % 4));
      }
    }
    if (mine && c < all)
      *reinterpret_cast<uint2*>(codes + t * few_pitch(p.K) + c * 8) = make_uint2(w[0], w[1]);
  }
  sum = wave_sum_last(sum);
  if (lane == 63) red[kWaves + wave] = sum;
  __syncthreads();
  if (tid < p.T) {
    sum = 0;
#pragma unroll
    for (int w = 0; w < W; w++) sum += red[kWaves + tid * W + w];
    meta[8 + tid] = sum;
  }
  if (lane == 0 && part == 0 && mine)
    meta[t] = __builtin_bit_cast(int, finite ? s : __builtin_nanf(""));
  __syncthreads();
}

// TT tokens (those past T repeat the last).  An item is one output column: one
// weight row, or (gated) the same row of both matrices.
template <int TT, bool GATED, bool FUSED>
__global__ __launch_bounds__(kWaves * 64) void few_kernel(const GemmArgs p) {
  constexpr int M = GATED ? 2 : 1;
  constexpr int D = kInFlight / M;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  int* meta = reinterpret_cast<int*>(lds);  // scales, sums, scratch: 64 words
  int8_t* codes = reinterpret_cast<int8_t*>(lds + 256);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t K = (uint32_t)p.K;
  const int steps = (p.K + kChunk - 1) / kChunk, pitch = few_pitch(p.K);
  const int stride = gridDim.x * kWaves;
  const int first = wave * gridDim.x + blockIdx.x;

  i4_t w[D][M];
  int li = first, ls = 0;  // item and step of the next load
  // positions past a row's end and rows past the last come as zeros
  auto load = [&](i4_t(&wd)[M]) {
    const uint32_t k = (uint32_t)ls * kChunk + lane * 16;
    const uint32_t at = k < K ? k : 0x80000000u;
#pragma unroll
    for (int m = 0; m < M; m++)
      wd[m] = load16(checked_buffer(p.w[m].codes + (int64_t)li * K, li < p.N ? K : 0), at);
    if (++ls == steps) {
      ls = 0;
      li += stride;
    }
  };
  // lane t finishes token t's output of an item; it has the row's scale and zero
  // point loaded by then
  float sc[M];
  int z[M];
  auto load_params = [&](int item) {
    const int n = min(item, p.N - 1);
#pragma unroll
    for (int m = 0; m < M; m++) {
      sc[m] = h_bits_to_f32(p.w[m].scales[n]);
      z[m] = p.w[m].zeros[n];
    }
  };
  load_params(first);
#pragma unroll
  for (int d = 0; d < D; d++) load(w[d]);
  if constexpr (FUSED) {
    quantize_here<TT>(p, codes, meta, meta + 16);
  } else {
    for (int c = threadIdx.x; c < p.T * (pitch / 16); c += kWaves * 64) {
      const int t = c / (pitch / 16), k = c % (pitch / 16) * 16;
      i4_t v = {0, 0, 0, 0};
      if (k < p.K) v = *reinterpret_cast<const i4_t*>(p.a + (int64_t)t * K + k);
      *reinterpret_cast<i4_t*>(codes + c * 16) = v;
    }
    if (threadIdx.x < (unsigned)p.T) {
      meta[threadIdx.x] = __builtin_bit_cast(int, p.xs[threadIdx.x]);
      meta[8 + threadIdx.x] = p.xsum[threadIdx.x];
    }
    __syncthreads();
  }

  const float xs = __builtin_bit_cast(float, meta[min(lane, p.T - 1)]);
  const int total = meta[8 + min(lane, p.T - 1)];
  int acc[M][TT];
  for (int item = first, step = 0; item < p.N;) {
#pragma unroll
    for (int d = 0; d < D; d++) {
      if (step == 0) {
#pragma unroll
        for (int m = 0; m < M; m++)
#pragma unroll
          for (int t = 0; t < TT; t++) acc[m][t] = 0;
      }
      i4_t wx[M];
#pragma unroll
      for (int m = 0; m < M; m++) wx[m] = w[d][m] ^ (int)0x80808080;
#pragma unroll
      for (int t = 0; t < TT; t++) {
        const i4_t a = *reinterpret_cast<const i4_t*>(codes + min(t, p.T - 1) * pitch +
                                                      step * kChunk + lane * 16);
#pragma unroll
        for (int m = 0; m < M; m++)
#pragma unroll
          for (int q = 0; q < 4; q++)
            acc[m][t] = __builtin_amdgcn_sdot4(wx[m][q], a[q], acc[m][t], false);
      }
      load(w[d]);
      __builtin_amdgcn_sched_barrier(0);  // keeps the other loads in flight
      if (++step == steps) {
        if (item < p.N) {
          int mine[M] = {};
#pragma unroll
          for (int m = 0; m < M; m++)
#pragma unroll
            for (int t = 0; t < TT; t++) {
              const int v = __builtin_amdgcn_readlane(wave_sum_last(acc[m][t]), 63);
              if (lane == t) mine[m] = v;
            }
          if (lane < p.T) {
            float v[M];
#pragma unroll
            for (int m = 0; m < M; m++)
              v[m] = exact_sum(mine[m], 128 - z[m], total,
                               p.K <= 65536 && (uint32_t)z[m] < 256u) * (xs * sc[m]);
            const int64_t at = (int64_t)lane * p.N + item;
            auto put = [&](void* base, float f) {
              static_cast<uint16_t*>(base)[at] = f32_to_elem(f, p.bf16);
            };
            if constexpr (GATED) {
              put(p.y, act_value(v[0], p.act) * v[1]);
              if (p.g) {
                put(p.g, v[0]);
                put(p.u, v[1]);
              }
            } else {
              put(p.y, v[0]);
            }
          }
        }
        step = 0;
        item += stride;
        load_params(item);
      }
    }
  }
}

template <int TT, bool GATED, bool FUSED>
hipError_t launch_one(const GemmArgs& p, hipStream_t stream) {
  constexpr int most = 256 + kFewMostCodes;
  const int bytes = 256 + p.T * few_pitch(p.K);
  auto kernel = few_kernel<TT, GATED, FUSED>;
  hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(kernel), most);
  if (e != hipSuccess) return e;
  const int groups = p.N < device_cu_count() ? p.N : device_cu_count();
  kernel<<<dim3((unsigned)groups), dim3(kWaves * 64), bytes, stream>>>(p);
  return hipGetLastError();
}

template <int TT, bool GATED>
hipError_t launch_x(const GemmArgs& p, hipStream_t stream) {
  return p.a ? launch_one<TT, GATED, false>(p, stream)
             : launch_one<TT, GATED, true>(p, stream);
}

}  // namespace

hipError_t launch_few(const GemmArgs& p, bool gated, hipStream_t stream) {
  if (gated) {
    if (p.T <= 1) return launch_x<1, true>(p, stream);
    if (p.T <= 2) return launch_x<2, true>(p, stream);
    return launch_x<4, true>(p, stream);
  }
  if (p.T <= 1) return launch_x<1, false>(p, stream);
  return launch_x<2, false>(p, stream);
}

}  // namespace lowbit
