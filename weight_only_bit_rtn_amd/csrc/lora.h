// lora.h -- what the adapter kernels share: element types and their matrix
// products, the tiles of a plan, and the launchers behind the C ABI (not exported).
#pragma once

#include "lora_division.h"
#include "w8a8.h"

namespace lowbit {

typedef __bf16 bf8_t __attribute__((ext_vector_type(8)));

size_t lora_workspace_bytes(const LoraSizes& s);
size_t lora_grad_workspace_bytes(const LoraSizes& s);

struct LoraArgs {
  const int32_t *order, *starts;
  const uint16_t *a, *b;
  const float* scales;
  int L, R, N, K;
  int64_t T;
};

// A kernel launch with `lds` bytes of dynamic LDS.
template <typename... P, typename... A>
hipError_t launch_lds(void (*kernel)(P...), dim3 grid, int threads, int lds, hipStream_t stream,
                      A... args) {
  if (lds > 64 * 1024) {
    const hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(kernel), lds);
    if (e != hipSuccess) return e;
  }
  kernel<<<grid, threads, lds, stream>>>(args...);
  return hipGetLastError();
}

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
// Tile `index` of the plan, found by every wave for itself: 256 adapters' tile counts
// at a time, four to a lane, are summed along the lanes.  False beyond the last one.
// starts is kept within [0, T], so that no plan leads outside the buffers.
__device__ __forceinline__ bool find_tile(const int32_t* __restrict__ starts, int L, int T,
                                          int size, int index, LoraTile& tile) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int base = 0; base <= L; base += 256) {
    int s[5], tiles[4], all = 0;
#pragma unroll
    for (int j = 0; j < 5; j++) s[j] = starts[min(base + lane * 4 + j, L)];
#pragma unroll
    for (int j = 0; j < 5; j++) {
      s[j] = base + lane * 4 + j <= L ? min(max(s[j], 0), T) : T;
      if (j > 0) {
        s[j] = max(s[j], s[j - 1]);
        tiles[j - 1] = (s[j] - s[j - 1] + size - 1) / size;
        all += tiles[j - 1];
      }
    }
    int sum = all;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int other = __shfl_up(sum, off, kWave);
      if (lane >= off) sum += other;
    }
    const uint64_t past = __ballot(index < before + sum);
    if (past) {
      // the adapter among this lane's four, for the lane that has it
      int rest = index - (before + sum - all), l = 0;
      int first = s[0], end = s[1], n = tiles[0];
#pragma unroll
      for (int j = 1; j < 4; j++)
        if (l == j - 1 && rest >= n) {
          rest -= n;
          l = j;
          first = s[j];
          end = s[j + 1];
          n = tiles[j];
        }
      const int at = __ffsll((unsigned long long)past) - 1;
      tile.l = base + at * 4 + __builtin_amdgcn_readlane(l, at);
      tile.first = __builtin_amdgcn_readlane(first, at);
      tile.tiles = __builtin_amdgcn_readlane(n, at);
      tile.begin = tile.first + __builtin_amdgcn_readlane(rest, at) * size;
      tile.count = min(size, __builtin_amdgcn_readlane(end, at) - tile.begin);
      return true;
    }
    before += __builtin_amdgcn_readlane(sum, 63);
  }
  return false;
}
// The token at a place of order, kept within [0, T).
__device__ __forceinline__ int64_t token_at(const int32_t* __restrict__ order, int64_t T, int at) {
  const uint32_t t = (uint32_t)order[at];
  return t < (uint64_t)T ? (int64_t)t : 0;
}

// The wave's number within its workgroup, as a scalar: branches on it are uniform.
__device__ __forceinline__ int wave_of_group() {
  return __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
}

// Keeps the loads of one step together and in order.  The counter of loads under way is
// waited on in order, and where two paths meet for the worst of both: loads of two steps that
// are mixed before a loop make every round of it wait for the second one's too.
__device__ __forceinline__ void loads_stay() { __builtin_amdgcn_sched_barrier(0); }

// Matrices on their way to the matrix cores pass through an LDS region of the wave's own.
// An operand wants row lane % 16 in every lane, but the vector cache serves four
// consecutive lanes at once only where they lie within 64 bytes: loads in the operands'
// order took 64 of its cycles for 1 KB instead of 16, and x was read at 3 TB/s however
// many loads were under way.  So eight lanes load the 128 bytes of one row, and the operands
// are read from LDS.  LDS serves a wave's accesses in order, so a region of its own needs no
// wait but for the compiler's order:
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}
// Rows of 64 elements, 16-byte chunk c of a row in slot c ^ (row / 2) % 8: the 16 rows of an
// operand's read, and the eight of a lane group's write, take all banks.
__device__ __forceinline__ int row_slot(int row, int chunk) {
  return row * 64 + ((chunk ^ ((row >> 1) & 7)) << 3);
}
// ROWS rows as they were loaded, row 8 q + lane / 8 chunk lane % 8 in v[q].
template <int ROWS>
__device__ __forceinline__ void put_rows(uint16_t* to, const us8_t (&v)[ROWS / 8]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int q = 0; q < ROWS / 8; q++)
    *reinterpret_cast<us8_t*>(to + row_slot(q * 8 + (lane >> 3), lane & 7)) = v[q];
}
// The operand of rows 16 block.. and terms 32 half..
__device__ __forceinline__ us8_t get_operand(const uint16_t* from, int block, int half) {
  const int lane = threadIdx.x & 63;
  return *reinterpret_cast<const us8_t*>(
      from + row_slot(block * 16 + (lane & 15), half * 4 + (lane >> 4)));
}

// Adds up the waves' sums of a tile, RB x TB products each, into wave 0's, half of the
// waves into the other half again and again; two blocks of ranks at a time pass through
// `lds`, reduce_bytes() of it.
template <int RB, int TB, int W>
constexpr int reduce_bytes() {
  return W / 2 * TB * 16 * ((RB < 2 ? 1 : 2) * 16 + 4) * 4;
}
template <int RB, int TB, int W>
__device__ __forceinline__ void reduce_waves(f4_t (&acc)[RB][TB], int wave, char* lds) {
  constexpr int G = RB < 2 ? 1 : 2, PITCH = G * 16 + 4;
  float(*red)[TB * 16][PITCH] = reinterpret_cast<float(*)[TB * 16][PITCH]>(lds);
  const int lane = threadIdx.x & 63, i16 = lane & 15, h = lane >> 4;
#pragma unroll
  for (int g = 0; g < RB; g += G)
#pragma unroll
    for (int left = W / 2; left > 0; left >>= 1) {
      __syncthreads();
      if (wave >= left && wave < 2 * left)
#pragma unroll
        for (int i = 0; i < G; i++)
#pragma unroll
          for (int j = 0; j < TB; j++)
            *reinterpret_cast<f4_t*>(&red[wave - left][j * 16 + i16][i * 16 + h * 4]) =
                acc[g + i][j];
      __syncthreads();
      if (wave < left)
#pragma unroll
        for (int i = 0; i < G; i++)
#pragma unroll
          for (int j = 0; j < TB; j++)
            acc[g + i][j] +=
                *reinterpret_cast<const f4_t*>(&red[wave][j * 16 + i16][i * 16 + h * 4]);
    }
}
// Wave 0's sums of a tile as rows of ranks: out[token][R], `count` tokens, `ranks` ranks.
template <int RB, int TB>
__device__ __forceinline__ void store_shares(const f4_t (&acc)[RB][TB], float* out, int R,
                                             int count, int ranks) {
  const int lane = threadIdx.x & 63, i16 = lane & 15, h = lane >> 4;
#pragma unroll
  for (int i = 0; i < RB; i++)
#pragma unroll
    for (int j = 0; j < TB; j++)
      if (j * 16 + i16 < count && i * 16 + h * 4 < ranks)
        *reinterpret_cast<f4_t*>(out + (j * 16 + i16) * R + i * 16 + h * 4) = acc[i][j];
}

// Four ranks' values of one token: the sum of `splits` shares that lie `next` apart.
__device__ __forceinline__ f4_t add_shares(const float* at, int64_t next, int splits) {
  f4_t sum = *reinterpret_cast<const f4_t*>(at);
  int w = 1;
  for (; w + 3 <= splits; w += 3) {
    const f4_t s0 = *reinterpret_cast<const f4_t*>(at + w * next);
    const f4_t s1 = *reinterpret_cast<const f4_t*>(at + (w + 1) * next);
    const f4_t s2 = *reinterpret_cast<const f4_t*>(at + (w + 2) * next);
    sum += s0;
    sum += s1 + s2;
  }
  for (; w < splits; w++) sum += *reinterpret_cast<const f4_t*>(at + w * next);
  return sum;
}

// A product with scale * value as one operand: its 32 terms are 32 ranks, once against the
// upper and once against the lower part; or, of 16 ranks, both parts at once.  Lane h's
// eight ranks of chunk c:
template <int RB>
struct Ranks {
  static constexpr int kChunks = RB < 2 ? 1 : RB / 2;
  static __device__ __forceinline__ int of(int c, int h) {
    return RB < 2 ? (h & 1) * 8 : c * 32 + h * 8;
  }
};
// acc[i] += rows[i] times the parts of one token's values, i < M.
template <bool BF, int RB, int M>
__device__ __forceinline__ void multiply_parts(const us8_t (&rows)[M][Ranks<RB>::kChunks],
                                               const uint16_t* parts, int h, f4_t (&acc)[M]) {
#pragma unroll
  for (int q = 0; q < (RB < 2 ? 1 : 2); q++)
#pragma unroll
    for (int c = 0; c < Ranks<RB>::kChunks; c++) {
      const us8_t f = *reinterpret_cast<const us8_t*>(parts + q * RB * 16 + c * 32 + h * 8);
#pragma unroll
      for (int i = 0; i < M; i++) acc[i] = Half16<BF>::mma(rows[i][c], f, acc[i]);
    }
}
// The parts of a tile of TILE tokens, parts[token][2][RB * 16] (and 8 more), and each
// token's exponent (fp16; a result is multiplied by 2^-exponent).  `values` gives
// a token's four ranks from r on, and is called with valid ones only.
template <bool BF, int RB, int TILE, int THREADS, typename F>
__device__ __forceinline__ void spread_parts(F values, float scale, int count, int R,
                                             uint16_t (*parts)[RB * 32 + 8], int* exponent) {
  constexpr int kPerToken = THREADS / TILE;  // threads of a token
  constexpr int kQuads = (RB * 4 + kPerToken - 1) / kPerToken;
  const int t = threadIdx.x / kPerToken, s = threadIdx.x % kPerToken;
  f4_t val[kQuads];
  int top = 0;
#pragma unroll
  for (int i = 0; i < kQuads; i++) {
    const int r = (s + i * kPerToken) * 4;
    val[i] = f4_t{0, 0, 0, 0};
    if (r < R && t < count) val[i] = values(t, r) * scale;
#pragma unroll
    for (int j = 0; j < 4; j++)
      top = max(top, __builtin_bit_cast(int, (float)val[i][j]) & 0x7fffffff);
  }
  int e = 0;
  if (!BF) {
#pragma unroll
    for (int off = 1; off < kPerToken; off <<= 1) top = max(top, __shfl_xor(top, off, kWave));
    e = fp16_exponent(top);
  }
  if (s == 0) exponent[t] = e;
#pragma unroll
  for (int i = 0; i < kQuads; i++) {
    const int r = (s + i * kPerToken) * 4;
    if (r >= RB * 16) continue;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      uint16_t part[2];
      split_parts<BF>(BF ? val[i][j] : times_power(val[i][j], e), part);
      parts[t][r + j] = part[0];
      parts[t][RB * 16 + r + j] = part[1];
    }
  }
}

#endif  // __HIPCC__

}  // namespace lowbit
