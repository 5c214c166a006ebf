// adamw.hip -- one AdamW step over many tensors, moments in 8 bits or in 32.
//
//   m' = b1 m + c1 g,  v' = b2 v + c2 g^2,
//   p' = p (1 - lr wd) - lr / (1 - beta1^t) m' / (sqrt(v') / sqrt(1 - beta2^t) + eps)
//
// Elementwise, so bound by HBM: fp32 parameters and gradients with 8-bit moments
// move 16 bytes a value, with 32-bit ones 28.  448 tensors of 112 thousand values take
// 172 us in four launches (4.7 TB/s), 100 million bf16 values with an fp32 copy 305 us
// (5.3 TB/s).  The tensors' addresses travel as kernel arguments, kMostTensors to a launch, so
// a step needs no table in device memory and can be captured.  A wave holds one block of
// 256 values, four to a lane: 16-byte loads of fp32, and the block's maximum stays within
// the wave.
//
// Every operation on the moments is rounded by itself (no contraction): their
// 8-bit codes are then the same wherever they are computed, also next to a border
// between two codes.
#include "adamw.h"

#include <cmath>

#include "w8a8.h"

#pragma clang fp contract(off)

namespace lowbit {
namespace {

constexpr int kMostTensors = 128;     // of a launch: with the rest below 4 KB of kernel arguments
constexpr int kWaves = 4;
// Blocks of a wave (us of 1 / 2 / 4, kernels alone: 448 fp32 tensors of 112 thousand values 172 /
// 182 / 212; 100 million bf16 values with an fp32 copy 306 / 300 / 310; two of 65536 3.6 / 4.0 / 5.3)
constexpr int kWaveBlocks = 1;
constexpr int kChunk = kWaves * kWaveBlocks * kAdamBlock;  // values of a workgroup

struct Entry {
  void* param;
  const void* grad;
  uint32_t n;            // a larger tensor is several entries, or launches
  uint32_t first_block;  // of its moments, after the launch's first one
};
struct Scalars {
  float b1, c1, b2, c2, eps;
  float decay;  // 1 - lr wd
  float alpha;  // lr / (1 - beta1^t)
  float rsq;    // (1 - beta2^t)^-1/2
};
struct Args {
  Entry t[kMostTensors];
  int32_t first_chunk[kMostTensors + 1];  // workgroups before a tensor's
  int32_t count;
  int64_t first_block;
  AdamState s;
  Scalars k;
  const float* grad_scale_at;
  const float* lr_at;
  const int32_t* step_at;
  double lr, beta1, beta2, decay;
  int64_t step;
};
static_assert(sizeof(Args) <= 4096, "kernel arguments");

// beta^t by squaring: 2^-53 t of relative error, far below what 1 - beta^t is rounded to.
__host__ __device__ inline double power(double beta, int64_t t) {
  double r = 1.0;
  for (; t > 0; t >>= 1, beta *= beta)
    if (t & 1) r *= beta;
  return r;
}
__host__ __device__ inline void scalars_of(double lr, double beta1, double beta2, double decay,
                                           int64_t step, Scalars& k) {
  k.decay = (float)(1.0 - lr * decay);
  k.alpha = (float)(lr / (1.0 - power(beta1, step)));
  k.rsq = (float)(1.0 / sqrt(1.0 - power(beta2, step)));
}

template <int TYPE>
struct Elem {
  typedef uint16_t raw;
  static __device__ __forceinline__ float get(raw b) { return elem_to_f32(b, TYPE == kBF16); }
  static __device__ __forceinline__ raw put(float v) { return f32_to_elem(v, TYPE == kBF16); }
};
template <>
struct Elem<kAdamF32> {
  typedef float raw;
  static __device__ __forceinline__ float get(raw v) { return v; }
  static __device__ __forceinline__ raw put(float v) { return v; }
};

// Four values from `at` on, `left` of them inside the tensor.
template <int TYPE>
__device__ __forceinline__ void load4(const void* from, int64_t at, int64_t left, float (&f)[4]) {
  typedef typename Elem<TYPE>::raw raw;
  typedef raw raw4 __attribute__((ext_vector_type(4)));
  const raw* p = static_cast<const raw*>(from) + at;
  raw4 v = {};
  if (left >= 4) {
    v = *reinterpret_cast<const raw4*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < 3; i++)
      if (i < left) v[i] = p[i];
  }
#pragma unroll
  for (int i = 0; i < 4; i++) f[i] = Elem<TYPE>::get(v[i]);
}
template <int TYPE>
__device__ __forceinline__ void store4(void* to, int64_t at, int64_t left, const float (&f)[4]) {
  typedef typename Elem<TYPE>::raw raw;
  typedef raw raw4 __attribute__((ext_vector_type(4)));
  raw* p = static_cast<raw*>(to) + at;
  raw4 v;
#pragma unroll
  for (int i = 0; i < 4; i++) v[i] = Elem<TYPE>::put(f[i]);
  if (left >= 4) {
    *reinterpret_cast<raw4*>(p) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 3; i++)
      if (i < left) p[i] = v[i];
  }
}

// The largest of the wave's values.
__device__ __forceinline__ uint32_t wave_top(uint32_t v) {
#define LOWBIT_DPP_TOP(ctrl, rmask) \
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rmask, 0xf, false))
  LOWBIT_DPP_TOP(0xb1, 0xf);   // quad_perm [1,0,3,2]
  LOWBIT_DPP_TOP(0x4e, 0xf);   // quad_perm [2,3,0,1]
  LOWBIT_DPP_TOP(0x141, 0xf);  // row_half_mirror
  LOWBIT_DPP_TOP(0x140, 0xf);  // row_mirror
  LOWBIT_DPP_TOP(0x142, 0xa);  // row_bcast:15
  LOWBIT_DPP_TOP(0x143, 0xc);  // row_bcast:31
#undef LOWBIT_DPP_TOP
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Numbers of codes: the upper bits of fp32, counted down from 1's.
constexpr uint32_t kDownM = 0x3F8 - 127, kDownV = 0x3F8 - 255;
template <uint32_t DOWN>
__device__ __forceinline__ float number(uint32_t code) {
  const float f = __builtin_bit_cast(float, (code << 20) + (DOWN << 20));
  return code ? f : 0.0f;
}
// The nearest code to q in [0, 1 + 2^-23]: the last one stands for 1, and no clamp is needed.
template <uint32_t DOWN>
__device__ __forceinline__ uint32_t nearest(float q) {
  return __builtin_elementwise_sub_sat((__builtin_bit_cast(uint32_t, q) + 0x80000u) >> 20, DOWN);
}

// One of the two codes next to q, each by its nearness: r / 2^20 of the way between their numbers
// and more goes up, 8 <= r < 2^20.  (From 1 + 2^-23 no r reaches past the last code.)
template <uint32_t DOWN>
__device__ __forceinline__ uint32_t either(float q, uint32_t r) {
  return __builtin_elementwise_sub_sat((__builtin_bit_cast(uint32_t, q) + r) >> 20, DOWN);
}
// 32 bits that depend on all of x's in no visible way; the factors are the first 32 binary
// digits behind the points of the square roots of 2 and 3.
__host__ __device__ inline uint32_t mixed(uint32_t x) {
  x = (x ^ x >> 16) * 0x6A09E667u;
  x = (x ^ x >> 15) * 0xBB67AE85u;
  return x ^ x >> 16;
}

__device__ __forceinline__ void unpack4(uint32_t cm, uint32_t cv, float m_max, float v_max,
                                        float (&m)[4], float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const float f = number<kDownM>((cm >> (8 * i)) & 127);
    const uint32_t sign = (cm << (24 - 8 * i)) & 0x80000000u;
    m[i] = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, f) | sign) * m_max;
    v[i] = number<kDownV>((cv >> (8 * i)) & 255) * v_max;
  }
}

// m / (sqrt(v) rsq + eps) where v or eps may be subnormal or 0: the operands of the hardware's
// square root and reciprocal are 2^64 times as large.  0 where there is nothing to divide by.
__device__ __forceinline__ float small_step(float m, float v, const Scalars& k) {
  const bool low = v < 0x1p-126f;
  float root = __builtin_amdgcn_sqrtf(low ? v * 0x1p64f : v);
  root = low ? root * 0x1p-32f : root;
  const float under = __builtin_fmaf(root, k.rsq, k.eps);
  if (under == 0.0f) return m * 0.0f;  // a NaN for an m that is no number
  const float up = under < 0x1p-126f ? 0x1p64f : 1.0f;
  return m * __builtin_amdgcn_rcpf(under * up) * up;
}

constexpr int kRandom8 = 8 | kAdamRandom;

template <int PT, int GT, int BITS, bool MASTER>
__global__ __launch_bounds__(kWaves * 64) void adamw_kernel(const Args a) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  // the tensor of this workgroup: the last that begins at or before it
  static_assert(kMostTensors <= 128, "two lookups of 64 lanes");
  const int at0 = a.first_chunk[min(lane, a.count)], at1 = a.first_chunk[min(lane + 64, a.count)];
  const int chunk = (int)blockIdx.x;
  const int t = __builtin_amdgcn_readfirstlane(
      __popcll(__ballot(lane < a.count && at0 <= chunk)) +
      __popcll(__ballot(lane + 64 < a.count && at1 <= chunk)) - 1);
  float scale = 1.0f;
  if (a.grad_scale_at) {
    scale = *a.grad_scale_at;
    if (!(fabsf(scale) < __builtin_inff())) return;
  }
  Scalars k = a.k;
  if (a.lr_at || a.step_at)
    scalars_of(a.lr_at ? (double)*a.lr_at : a.lr, a.beta1, a.beta2, a.decay,
               a.step_at ? (int64_t)max(*a.step_at, 1) : a.step, k);
  void* const param = a.t[t].param;
  const void* const grad = a.t[t].grad;
  const int64_t n = a.t[t].n, first = a.first_block + a.t[t].first_block;
  const int64_t e0 = ((int64_t)(chunk - a.first_chunk[t]) * kWaves + wave) *
                     (kWaveBlocks * kAdamBlock);
  float p[kWaveBlocks][4], g[kWaveBlocks][4], m[kWaveBlocks][4], v[kWaveBlocks][4];
#pragma unroll
  for (int j = 0; j < kWaveBlocks; j++) {
    const int64_t b = e0 + j * kAdamBlock;  // of the tensor
    if (b >= n) continue;
    const int64_t e = b + lane * 4, left = n - e;
    const int64_t s = first * kAdamBlock + e;  // of the moments
    load4<GT>(grad, e, left, g[j]);
    if (MASTER)
      load4<kAdamF32>(a.s.master, s, 4, p[j]);
    else
      load4<PT>(param, e, left, p[j]);
    if (BITS == 32) {
      load4<kAdamF32>(a.s.m, s, 4, m[j]);
      load4<kAdamF32>(a.s.v, s, 4, v[j]);
    } else {
      const int64_t block = first + b / kAdamBlock;
      unpack4(static_cast<const uint32_t*>(a.s.m)[s / 4], static_cast<const uint32_t*>(a.s.v)[s / 4],
              a.s.m_max[block], a.s.v_max[block], m[j], v[j]);
    }
  }
  // lane j and lane 4 + j: the maxima of block j's m and v, as bits
  uint32_t tops = 0;
#pragma unroll
  for (int j = 0; j < kWaveBlocks; j++) {
    const int64_t b = e0 + j * kAdamBlock;
    if (b >= n) continue;
    const int64_t e = b + lane * 4, left = n - e;
    const int64_t s = first * kAdamBlock + e;
    uint32_t top_m = 0, top_v = 0, least_v = ~0u;  // least_v: bits of the least v but 0, less 1
    float taken[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      float x = g[j][i];
      if (a.grad_scale_at) x = x * scale;
      m[j][i] = k.b1 * m[j][i] + k.c1 * x;
      v[j][i] = k.b2 * v[j][i] + k.c2 * (x * x);
    }
    if (left < 4) {
#pragma unroll
      for (int i = 0; i < 4; i++)
        if (i >= left) p[j][i] = m[j][i] = v[j][i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
      top_m = max(top_m, __builtin_bit_cast(uint32_t, m[j][i]) & 0x7fffffffu);
      top_v = max(top_v, __builtin_bit_cast(uint32_t, v[j][i]) & 0x7fffffffu);
      least_v = min(least_v, __builtin_bit_cast(uint32_t, v[j][i]) - 1);
      // The hardware's square root and reciprocal are off by 2^-23 of the step taken (with
      // their IEEE forms the 100 million values took 330 us).
      taken[i] = m[j][i] * __builtin_amdgcn_rcpf(
                               __builtin_fmaf(__builtin_amdgcn_sqrtf(v[j][i]), k.rsq, k.eps));
    }
    // both take a subnormal number for 0: a second moment below 2^-126, or an eps with no second moment
    if (least_v < 0x7fffffu || k.eps < 0x1p-126f)
#pragma unroll
      for (int i = 0; i < 4; i++) taken[i] = small_step(m[j][i], v[j][i], k);
#pragma unroll
    for (int i = 0; i < 4; i++) p[j][i] = __builtin_fmaf(-k.alpha, taken[i], p[j][i] * k.decay);
    if (MASTER) store4<kAdamF32>(a.s.master, s, 4, p[j]);
    store4<PT>(param, e, left, p[j]);
    if (BITS == 32) {
      store4<kAdamF32>(a.s.m, s, 4, m[j]);
      store4<kAdamF32>(a.s.v, s, 4, v[j]);
    } else {
      const uint32_t all_m = wave_top(top_m), all_v = wave_top(top_v);
      tops = lane == j ? all_m : lane == kWaveBlocks + j ? all_v : tops;
    }
  }
  if (BITS == 32) return;
  // Every lane its maximum: as it is stored, and its reciprocal.  A block that is not finite has
  // a NaN and codes 0, as a block of zeros has codes 0.
  const bool small = tops < 0x00800000u, finite = tops < 0x7f800000u;
  const float top = finite ? (small ? 0.0f : __builtin_bit_cast(float, tops)) : __builtin_nanf("");
  const float inverse = finite && !small ? 1.0f / top : 0.0f;
  const int64_t block = first + e0 / kAdamBlock;
  if (lane < 2 * kWaveBlocks && e0 + lane % kWaveBlocks * kAdamBlock < n)
    (lane < kWaveBlocks ? a.s.m_max : a.s.v_max)[block + lane % kWaveBlocks] = top;
  const uint64_t numbers = __ballot(finite);
#pragma unroll
  for (int j = 0; j < kWaveBlocks; j++) {
    const int64_t b = e0 + j * kAdamBlock;
    if (b >= n) continue;
    const int64_t s = first * kAdamBlock + b + lane * 4;
    const int lane_v = kWaveBlocks + j;
    const float inv_m = __builtin_bit_cast(
        float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, inverse), j));
    const float inv_v = __builtin_bit_cast(
        float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, inverse), lane_v));
    uint32_t cm = 0, cv = 0;
    // for each place a number of its own in every step, 16 bits for m and 16 for v
    uint32_t random[4];
    if (BITS == kRandom8) {
      const int64_t t = a.step_at ? (int64_t)max(*a.step_at, 1) : a.step;
      const uint32_t key = mixed(mixed((uint32_t)t) + (uint32_t)(s >> 32));
#pragma unroll
      for (int i = 0; i < 4; i++) random[i] = mixed(((uint32_t)s + i) ^ key);
    }
    if (numbers >> j & 1)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const float q = fabsf(m[j][i]) * inv_m;
        const uint32_t c = BITS == kRandom8 ? either<kDownM>(q, random[i] >> 16 << 4 | 8)
                                            : nearest<kDownM>(q);
        const uint32_t sign = __builtin_bit_cast(uint32_t, m[j][i]) >> 31 << 7;
        cm |= (c ? c | sign : 0u) << (8 * i);
      }
    if (numbers >> lane_v & 1)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const float q = v[j][i] * inv_v;
        const uint32_t c = BITS == kRandom8 ? either<kDownV>(q, (random[i] & 0xffff) << 4 | 8)
                                            : nearest<kDownV>(q);
        // one at least where q is not 0
        cv |= max(c, min(__builtin_bit_cast(uint32_t, q), 1u)) << (8 * i);
      }
    static_cast<uint32_t*>(a.s.m)[s / 4] = cm;
    static_cast<uint32_t*>(a.s.v)[s / 4] = cv;
  }
}

// One wave a block.
__global__ __launch_bounds__(256) void moments_kernel(const uint8_t* __restrict__ m,
                                                      const uint8_t* __restrict__ v,
                                                      const float* __restrict__ m_max,
                                                      const float* __restrict__ v_max,
                                                      int64_t blocks, float* __restrict__ m_out,
                                                      float* __restrict__ v_out) {
  const int64_t word = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t block = word / (kAdamBlock / 4);
  if (block >= blocks) return;
  float fm[4], fv[4];
  unpack4(reinterpret_cast<const uint32_t*>(m)[word], reinterpret_cast<const uint32_t*>(v)[word],
          m_max[block], v_max[block], fm, fv);
  store4<kAdamF32>(m_out, word * 4, 4, fm);
  store4<kAdamF32>(v_out, word * 4, 4, fv);
}

template <int PT, int GT, int BITS>
void launch(bool master, unsigned grid, const Args& a, hipStream_t stream) {
  if (master)
    adamw_kernel<PT, GT, BITS, true><<<grid, kWaves * 64, 0, stream>>>(a);
  else
    adamw_kernel<PT, GT, BITS, false><<<grid, kWaves * 64, 0, stream>>>(a);
}
template <int PT, int GT>
void launch(int bits, bool master, unsigned grid, const Args& a, hipStream_t stream) {
  if (bits == 8)
    launch<PT, GT, 8>(master, grid, a, stream);
  else if (bits == kRandom8)
    launch<PT, GT, kRandom8>(master, grid, a, stream);
  else
    launch<PT, GT, 32>(master, grid, a, stream);
}
template <int PT>
void launch(int gt, int bits, bool master, unsigned grid, const Args& a, hipStream_t stream) {
  if (gt == kF16)
    launch<PT, kF16>(bits, master, grid, a, stream);
  else if (gt == kBF16)
    launch<PT, kBF16>(bits, master, grid, a, stream);
  else
    launch<PT, kAdamF32>(bits, master, grid, a, stream);
}

}  // namespace

hipError_t launch_adamw(const AdamTensor* tensors, int64_t count, int param_type, int grad_type,
                        int bits, const AdamState& state, const AdamOptions& o,
                        hipStream_t stream) {
  Args a;
  a.s = state;
  a.k.b1 = (float)o.beta1;
  a.k.c1 = (float)(1.0 - o.beta1);
  a.k.b2 = (float)o.beta2;
  a.k.c2 = (float)(1.0 - o.beta2);
  a.k.eps = (float)o.eps;
  scalars_of(o.lr, o.beta1, o.beta2, o.decay, o.step, a.k);
  a.grad_scale_at = o.grad_scale_at;
  a.lr_at = o.lr_at;
  a.step_at = o.step_at;
  a.lr = o.lr;
  a.beta1 = o.beta1;
  a.beta2 = o.beta2;
  a.decay = o.decay;
  a.step = o.step;
  // 2^20 workgroups a launch at most: a larger tensor goes on in the next one
  constexpr int64_t kMostChunks = 1 << 20;
  int64_t i = 0, done = 0, block = 0;  // tensor, its values that earlier launches take, its first block
  while (i < count) {
    a.count = 0;
    int64_t chunks = 0;
    while (i < count && a.count < kMostTensors && chunks < kMostChunks) {
      const int64_t n = tensors[i].n - done;
      const int64_t take = n < (kMostChunks - chunks) * kChunk ? n : (kMostChunks - chunks) * kChunk;
      if (a.count == 0) a.first_block = block + done / kAdamBlock;
      if (take > 0) {
        const int64_t pw = param_type == kAdamF32 ? 4 : 2, gw = grad_type == kAdamF32 ? 4 : 2;
        a.t[a.count] = {static_cast<char*>(tensors[i].param) + done * pw,
                        static_cast<const char*>(tensors[i].grad) + done * gw, (uint32_t)take,
                        (uint32_t)(block + done / kAdamBlock - a.first_block)};
        a.first_chunk[a.count++] = (int32_t)chunks;
        chunks += (take + kChunk - 1) / kChunk;
      }
      if (take == n) {
        block += (tensors[i].n + kAdamBlock - 1) / kAdamBlock;
        i++;
        done = 0;
      } else {
        done += take;
      }
    }
    a.first_chunk[a.count] = (int32_t)chunks;
    if (chunks == 0) continue;
    const unsigned grid = (unsigned)chunks;
    const bool master = state.master != nullptr;
    if (param_type == kF16)
      launch<kF16>(grad_type, bits, master, grid, a, stream);
    else if (param_type == kBF16)
      launch<kBF16>(grad_type, bits, master, grid, a, stream);
    else
      launch<kAdamF32>(grad_type, bits, master, grid, a, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_adamw_moments(const uint8_t* m, const uint8_t* v, const float* m_max,
                                const float* v_max, int64_t blocks, float* m_out, float* v_out,
                                hipStream_t stream) {
  // grids are kept within 2^32 threads
  constexpr int64_t kMost = (int64_t)1 << 24;
  for (int64_t b = 0; b < blocks; b += kMost) {
    const int64_t take = blocks - b < kMost ? blocks - b : kMost;
    moments_kernel<<<(unsigned)((take + 3) / 4), 256, 0, stream>>>(
        m + b * kAdamBlock, v + b * kAdamBlock, m_max + b, v_max + b, take,
        m_out + b * kAdamBlock, v_out + b * kAdamBlock);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace lowbit
