// lora.h -- what the adapter kernels share: element types and their matrix
// products, the tiles of a plan, and the launchers behind the C ABI (not exported).
#pragma once

#include "w8a8.h"

namespace lowbit {

typedef __bf16 bf8_t __attribute__((ext_vector_type(8)));

// Host arithmetic of the launches.  Every bound on a number of tiles counts one for
// each adapter that has tokens, whose last tile may be a part, and one for the tokens
// without an adapter.
struct LoraSizes {
  int64_t T, N, K, R, L;
};
inline int64_t lora_tiles(int64_t T, int64_t L, int tile) {
  const int64_t most = (T + tile - 1) / tile + L;
  return most < T ? most : T;
}
size_t lora_workspace_bytes(const LoraSizes& s);
size_t lora_grad_workspace_bytes(const LoraSizes& s);

struct LoraArgs {
  const int32_t *order, *starts;
  const uint16_t *a, *b;
  const float* scales;
  int L, R, N, K;
  int64_t T;
};

hipError_t launch_lora_plan(const int32_t* ids, int64_t T, int64_t L, int32_t* order,
                            int32_t* starts, hipStream_t stream);
hipError_t launch_lora(const void* x, int dtype, const LoraArgs& p, const void* y, void* out,
                       float* v, void* workspace, hipStream_t stream);
hipError_t launch_lora_grad(const void* dy, const void* x, const float* v, int dtype,
                            const LoraArgs& p, const void* base, void* dx, float* da, float* db,
                            void* workspace, hipStream_t stream);

#ifdef __HIPCC__

// 16-bit elements: eight to an operand of a 16x16x32 product, whose first operand has
// 16 rows and second 16 columns: a lane holds, of row (column) lane % 16, the eight
// terms from 8 (lane / 16) on; of the result, column lane % 16 and the four rows
// from 4 (lane / 16) on.
template <bool BF>
struct Half16;
template <>
struct Half16<false> {
  static __device__ __forceinline__ f4_t mma(us8_t a, us8_t b, f4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8_t, a),
                                                  __builtin_bit_cast(h8_t, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint16_t from(float v) {
    return __builtin_bit_cast(uint16_t, (_Float16)v);
  }
  static __device__ __forceinline__ float to(uint16_t v) { return h_bits_to_f32(v); }
};
template <>
struct Half16<true> {
  static __device__ __forceinline__ f4_t mma(us8_t a, us8_t b, f4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8_t, a),
                                                   __builtin_bit_cast(bf8_t, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint16_t from(float v) {
    return __builtin_bit_cast(uint16_t, (__bf16)v);
  }
  static __device__ __forceinline__ float to(uint16_t v) {
    return __builtin_bit_cast(float, (uint32_t)v << 16);
  }
};

// An fp32 value as a sum of PARTS 16-bit ones, each what the ones before leave over.
// An infinity (or a value that rounds to one) stays in the first part alone.
template <bool BF, int PARTS>
__device__ __forceinline__ void split_parts(float v, uint16_t (&part)[PARTS]) {
#pragma unroll
  for (int i = 0; i < PARTS; i++) {
    part[i] = Half16<BF>::from(v);
    const float had = Half16<BF>::to(part[i]);
    v = fabsf(had) < __builtin_inff() ? v - had : 0.0f;
  }
}
// The power of two that brings a largest |value| (its fp32 bits) into [2^14, 2^15);
// 0 for zero, an infinity or a NaN.
__device__ __forceinline__ int fp16_exponent(int top_bits) {
  if (top_bits == 0 || top_bits >= 0x7f800000) return 0;
  return 14 - (max(top_bits >> 23, 1) - 127);
}
__device__ __forceinline__ float times_power(float v, int e) { return __builtin_amdgcn_ldexpf(v, e); }

// Eight elements at a 2-byte address (rows of an odd length), as one load.
struct __attribute__((packed, aligned(2))) Packed8 {
  us8_t v;
};
__device__ __forceinline__ us8_t load8(const uint16_t* p) {
  return reinterpret_cast<const Packed8*>(p)->v;
}
__device__ __forceinline__ void store8(uint16_t* p, us8_t v) {
  reinterpret_cast<Packed8*>(p)->v = v;
}
// The same near a row's end: `left` of them lie inside (none where it is not positive).
__device__ __forceinline__ us8_t load8(const uint16_t* p, int64_t left) {
  if (left >= 8) return load8(p);
  us8_t v = {};
#pragma unroll
  for (int i = 0; i < 7; i++)
    if (i < left) v[i] = p[i];
  return v;
}
__device__ __forceinline__ void store8(uint16_t* p, us8_t v, int64_t left) {
  if (left >= 8) {
    store8(p, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 7; i++)
    if (i < left) p[i] = v[i];
}

// One tile of a plan: up to `size` tokens, order[begin ..), of one adapter, or (l == L)
// of the tokens without one; first and tiles: where the adapter's tokens begin, and how
// many tiles it has.
struct LoraTile {
  int l, begin, count, first, tiles;
};
// Tile `index` of the plan, found by every wave for itself: 64 adapters' tile counts
// at a time are summed along the lanes.  False beyond the last one.  starts is kept
// within [0, T], so that no plan leads outside the buffers.
__device__ __forceinline__ bool find_tile(const int32_t* __restrict__ starts, int L, int T,
                                          int size, int index, LoraTile& tile) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int base = 0; base <= L; base += 64) {
    const int l = base + lane;
    int s0 = T, s1 = T;
    if (l <= L) {
      s0 = min(max(starts[l], 0), T);
      s1 = l < L ? min(max(starts[l + 1], s0), T) : T;
    }
    const int tiles = (s1 - s0 + size - 1) / size;
    int sum = tiles;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int other = __shfl_up(sum, off, kWave);
      if (lane >= off) sum += other;
    }
    const uint64_t past = __ballot(index < before + sum);
    if (past) {
      const int at = __ffsll((unsigned long long)past) - 1;
      const int skip = (index - __shfl(before + sum - tiles, at, kWave)) * size;
      tile.l = __builtin_amdgcn_readfirstlane(base + at);
      tile.first = __builtin_amdgcn_readfirstlane(__shfl(s0, at, kWave));
      tile.tiles = __builtin_amdgcn_readfirstlane(__shfl(tiles, at, kWave));
      tile.begin = __builtin_amdgcn_readfirstlane(tile.first + skip);
      tile.count = __builtin_amdgcn_readfirstlane(min(size, __shfl(s1, at, kWave) - tile.begin));
      return true;
    }
    before += __shfl(sum, 63, kWave);
  }
  return false;
}
// The token at a place of order, kept within [0, T).
__device__ __forceinline__ int64_t token_at(const int32_t* __restrict__ order, int64_t T, int at) {
  const uint32_t t = (uint32_t)order[at];
  return t < (uint64_t)T ? (int64_t)t : 0;
}

#endif  // __HIPCC__

}  // namespace lowbit
