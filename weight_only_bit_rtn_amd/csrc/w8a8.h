// w8a8.h -- what the 8-bit activation kernels share: element types, the
// activations of the gated block, LDS-direct tile loads, and the launchers
// behind the C ABI (not exported).
#pragma once

#include "common.h"
#include "w8a8_plan.h"

namespace lowbit {

enum ElemType { kF16 = 0, kBF16 = 1, kI8 = 2 };
enum ActKind { kSilu = 0, kGeluTanh = 1 };

typedef int i4_t __attribute__((ext_vector_type(4)));
typedef int i2_t __attribute__((ext_vector_type(2)));
typedef uint16_t us4_t __attribute__((ext_vector_type(4)));
typedef uint16_t us8_t __attribute__((ext_vector_type(8)));

// One weight matrix as the quantizers leave it (8 bits, one group per row).
struct W8 {
  const uint8_t* codes;  // [N][K] code bytes
  const uint16_t* scales;
  const int32_t* zeros;
};

__device__ __forceinline__ float elem_to_f32(uint16_t bits, bool bf16) {
  return bf16 ? __builtin_bit_cast(float, (uint32_t)bits << 16) : h_bits_to_f32(bits);
}
// Rounds an fp32 value to nearest even to the output type.  The value is one, in
// every kernel: left alone the compiler joins some kernels' last product with the
// conversion (v_fma_mixlo_f16), which rounds the exact product, and the same
// output would differ from kernel to kernel in the last bit.
__device__ __forceinline__ uint16_t f32_to_elem(float v, bool bf16) {
  asm volatile("" : "+v"(v));
  return bf16 ? __builtin_bit_cast(uint16_t, (__bf16)v) : f32_to_h_bits(v);
}

// sigma = 1 / (1 + e^-2q) with 2q = v (SiLU) or 2p (GELU, tanh form): both
// activations are v * sigma.  e^-2q overflows to infinity for very negative
// arguments and sigma is then 0, the limit.  GELU's cube is taken of v within
// [-16, 16]: beyond, sigma is 0 or 1 in fp32 already and its slope 0.  The
// hardware's exp2 and reciprocal are off by some 2^-24 of sigma each, and by 2^-24 for
// each unit of 2q, far below the 16-bit outputs' steps; the library's expf and a
// division took 420 -> 483 us on gated 4096x28672x1024, 47.8 -> 50.3 on 333x11008x4096.
__device__ __forceinline__ float act_sigma(float v, int act) {
  float e;
  if (act == kSilu) {
    e = v;
  } else {
    const float c = fminf(fmaxf(v, -16.0f), 16.0f);
    e = 1.5957691216057308f * (c + 0.044715f * c * c * c);
  }
  return __builtin_amdgcn_rcpf(1.0f + __expf(-e));
}
__device__ __forceinline__ float act_value(float v, int act) { return v * act_sigma(v, act); }
// The activation's value and slope: sigma + v sigma (1 - sigma) (2q)'.
__device__ __forceinline__ void act_value_slope(float v, int act, float& f, float& df) {
  const float s = act_sigma(v, act);
  f = v * s;
  float w = v;  // v (2q)'
  if (act != kSilu) {
    const float c = fminf(fmaxf(v, -16.0f), 16.0f);
    w = 1.5957691216057308f * c * (1.0f + 0.134145f * c * c);
  }
  df = s + s * (1.0f - s) * w;
}

// Buffer descriptor (raw, range-checked) of `bytes` bytes at a wave-uniform
// address.  A memory instruction may read a scalar register five wait states
// after a vector instruction (readfirstlane) wrote it; the compiler does not
// see to that for the assembly of load_to_lds(), so it is waited for here, once
// a descriptor (in each load it cost 4% at 4096 x 12288 x 12288).
__device__ __forceinline__ i4_t buffer_of(const void* base, uint32_t bytes) {
  const uint64_t at = reinterpret_cast<uint64_t>(base);
  i4_t rs{__builtin_amdgcn_readfirstlane((int)(uint32_t)at),
          __builtin_amdgcn_readfirstlane((int)((uint32_t)(at >> 32) & 0xffffu)),
          __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
  asm volatile("s_nop 4" : "+s"(rs));
  return rs;
}

// The LDS address of a pointer into shared memory.
__device__ __forceinline__ uint32_t lds_address(void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)p;
}

// 16 bytes per lane from a range-checked buffer straight into LDS: lane l's
// land at address at + 16 l (wave-uniform); an offset outside the buffer
// brings zeros.  Written in assembly, where it has no register result: behind
// the builtin the compiler waits for every such load in flight before a
// transposing LDS read (large gradient 4.1 -> 3.1 ms without those waits).
// The caller waits with lds_loads_left() before the barrier that publishes
// them, and for all of them before its wave ends.  A kernel that keeps
// descriptors in spilled scalar registers has SPILLED: they come back through a
// vector instruction, perhaps right before the load (see buffer_of()).
template <bool SPILLED = false>
__device__ __forceinline__ void load_to_lds(i4_t rs, uint32_t at, uint32_t offset) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop %3\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(at), "v"(offset), "s"(rs), "n"(SPILLED ? 3 : 0)
               : "memory", "m0");
}
// Waits until at most N of the wave's loads are on their way (they land in order).
template <int N>
__device__ __forceinline__ void lds_loads_left() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

// 16 bytes per lane from a range-checked buffer into registers; zeros from
// outside it.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t checked_buffer(const void* base, uint32_t bytes) {
  const uint64_t at = reinterpret_cast<uint64_t>(base);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)at);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(at >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((uint64_t)hi << 32 | lo),
                                           (short)0, __builtin_amdgcn_readfirstlane((int)bytes),
                                           0x00020000);
}
__device__ __forceinline__ i4_t load16(__amdgpu_buffer_rsrc_t rs, uint32_t offset) {
  return __builtin_bit_cast(i4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, (int)offset, 0, 0));
}

// Workgroup id -> tile: ids go round the 8 chiplets one by one, so give each
// chiplet (its own L2) a contiguous run of tiles, and walk the runs in bands
// of 8 token tiles by all weight tiles, so that the tiles in flight on one
// chiplet share few rows of both operands.  Ids from `total` on are tiles as they come.
__device__ __forceinline__ void tile_of(int id, int total, int tiles_m, int tiles_n, int& tm,
                                        int& tn) {
  const int q = total / 8, r = total % 8, xcd = id % 8, at = id / 8;
  const int t = id < total ? xcd * q + min(xcd, r) + at : id;
  constexpr int kBand = 8;
  const int band = t / (kBand * tiles_n), in = t % (kBand * tiles_n);
  const int rows = min(kBand, tiles_m - band * kBand);
  tm = band * kBand + in % rows;
  tn = in / rows;
}

// Code of one activation value: rint(fl32(x / s)) within [-127, 127], s the
// token's scale and r = fl32(1 / s).  x * r differs from x / s by less than
// 2^-15 for |x / s| < 128, so rint of the two can differ only when x * r lies
// within that of a half; there (and where r or the product overflows) the
// division is done.
__device__ __forceinline__ int act_code(float x, float s, float r) {
  const float q = x * r;
  float n = rintf(q);
  if (!(fabsf(q - n) <= 0.4999f)) n = rintf(x / s);
  return (int)fminf(fmaxf(n, -127.0f), 127.0f);
}

// Integer sum of one output to fp32: acc = sum a (code - 128), zc = 128 -
// zero point, total = sum a.  `small` (K <= 65536 and a zero point in
// [0, 255]): |total| < 2^23 and the sum of a (code - z) fits 32 bits;
// otherwise it is formed in fp64, where it is exact too (below 2^43).
__device__ __forceinline__ float exact_sum(int acc, int zc, int total, bool small) {
  if (small) return (float)(acc + __mul24(zc, total));
  return (float)((double)acc + (double)zc * (double)total);
}

struct GemmArgs {
  const int8_t* a;  // codes of the activations, or null: x is quantized in the kernel
  const uint16_t* x;
  const float* xs;
  const int32_t* xsum;
  W8 w[2];
  void* y;
  void* g;
  void* u;
  int T, N, K, act, bf16, x_bf16;
};

// Scales and 128 - zero points of four output columns n..n + 3.
template <bool GATED>
struct Columns {
  float sc[GATED ? 2 : 1][4];
  int zc[GATED ? 2 : 1][4];
  bool small;
  __device__ __forceinline__ Columns(const GemmArgs& p, int n) : small(p.K <= 65536) {
#pragma unroll
    for (int m = 0; m < (GATED ? 2 : 1); m++)
#pragma unroll
      for (int r = 0; r < 4; r++) {
        const int nn = min(n + r, p.N - 1);
        sc[m][r] = h_bits_to_f32(p.w[m].scales[nn]);
        const int z = p.w[m].zeros[nn];
        zc[m][r] = 128 - z;
        small = small && (uint32_t)z < 256u;
      }
  }
};

// The outputs of token t at columns n..n + 3 (n % 4 == 0) from their integer
// sums a0 (gated: the gate's, and a1 the up's); xs and total are the token's
// scale and the sum of its codes.
template <bool GATED>
__device__ __forceinline__ void store4(const GemmArgs& p, const Columns<GATED>& c, i4_t a0, i4_t a1,
                                       int n, int t, float xs, int total) {
  us4_t out, og, ou;
#pragma unroll
  for (int r = 0; r < 4; r++) {
    const float v = exact_sum(a0[r], c.zc[0][r], total, c.small) * (xs * c.sc[0][r]);
    if constexpr (GATED) {
      const float u = exact_sum(a1[r], c.zc[1][r], total, c.small) * (xs * c.sc[1][r]);
      out[r] = f32_to_elem(act_value(v, p.act) * u, p.bf16);
      og[r] = f32_to_elem(v, p.bf16);
      ou[r] = f32_to_elem(u, p.bf16);
    } else {
      out[r] = f32_to_elem(v, p.bf16);
    }
  }
  const int64_t at = (int64_t)t * p.N + n;
  auto put = [&](void* base, us4_t v) {
    uint16_t* d = static_cast<uint16_t*>(base) + at;
    if (p.N % 4 == 0) {
      *reinterpret_cast<us4_t*>(d) = v;
    } else {
#pragma unroll
      for (int r = 0; r < 4; r++)
        if (n + r < p.N) d[r] = v[r];
    }
  };
  put(p.y, out);
  if (GATED && p.g) {
    put(p.g, og);
    put(p.u, ou);
  }
}

// Products of one or two tokens (gated: up to four) whose codes fit LDS
// (w8a8_few.hip).  Without p.a the kernel quantizes p.x itself.
hipError_t launch_few(const GemmArgs& p, bool gated, hipStream_t stream);

// Products of at most kSkinnyMostT tokens (w8a8_skinny.hip).
hipError_t launch_skinny(const GemmArgs& p, bool gated, hipStream_t stream);

hipError_t launch_quantize_act(const void* x, int dtype, int64_t T, int64_t K, int8_t* codes,
                               float* scales, int32_t* sums, hipStream_t stream);

// The activations of a product: codes with their scales and sums, or fp16 /
// bf16 values that the launcher quantizes (into the workspace).
struct Activations {
  const void* x;
  int dtype;
  const float* scales;
  const int32_t* sums;
};

size_t w8a8_workspace_bytes(int64_t T, int64_t N, int64_t K, int dtype, bool gated);
hipError_t launch_linear_w8a8(const Activations& x, int64_t T, const W8& w, int64_t N, int64_t K,
                              void* y, int out_dtype, void* workspace, hipStream_t stream);
hipError_t launch_gated_w8a8(const Activations& x, int64_t T, const W8& gate, const W8& up,
                             int64_t N, int64_t K, int act, void* h, void* g, void* u,
                             int out_dtype, void* workspace, hipStream_t stream);

size_t w8a8_grad_workspace_bytes(int64_t T, int64_t N, int64_t K, bool gated);
hipError_t launch_w8a8_grad(const void* dh, const void* gate, const void* up, int dtype, int64_t T,
                            const W8& wg, const W8& wu, bool gated, int64_t N, int64_t K, int act,
                            void* dx, void* dgate, void* dup, void* workspace,
                            hipStream_t stream);

}  // namespace lowbit
