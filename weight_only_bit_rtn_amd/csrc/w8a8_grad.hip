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
// keep their 11 significant bits, down to factors of 2^-29 of the token's largest.
// (a is formed in fp32; where a token's are so small that bits would be lost
// there, with scales 2^100 times as large.)  Rounding a to fp16 is the one
// rounding between the inputs and the output, and a choice: dx of fp16 inputs is
// 2.9e-4 off in the 2-norm where 32-bit factors give 2.1e-4, the output's own
// rounding (bf16 outputs: 1.7e-3 either way).  Keeping 22 bits in two fp16 terms is
// twice the products: 1000x4096x11008 92 -> 180 us, gated 64x28672x8192 116 -> 152,
// gated 4096x28672x8192 3.06 -> 6.20 ms.  bf16 factors would keep 8 bits.
//
// Two kernels: one makes a', e and r (and, for the gated block, the gradients
// of both projections on the way), one multiplies.  The gated block's two
// products are one sum over the gate rows and then the up rows.
#include "w8a8.h"

namespace lowbit {
namespace {

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
  int N, pitch, half;
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

// A condition that is the same for the whole workgroup: a branch on it is one for
// the compiler too.
__device__ __forceinline__ bool uniform(int v) { return __builtin_amdgcn_readfirstlane(v) != 0; }

// Eight values of a row from chunk c on.  WHOLE (N % 8 == 0): rows and chunks
// lie at 16 bytes.  Otherwise a row may lie at any 2-byte address, and its last
// chunk is not full.  Positions past N: zeros read, nothing written.
template <bool WHOLE>
__device__ __forceinline__ us8_t get8(const uint16_t* row, int c, int N, bool full) {
  us8_t v = {};
  if (WHOLE) {
    v = reinterpret_cast<const us8_t*>(row)[c];
  } else if (full) {
    __builtin_memcpy(&v, row + c * 8, 16);
  } else {  // no branches: all loads under way together
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const uint16_t x = row[min(c * 8 + j, N - 1)];
      v[j] = c * 8 + j < N ? x : 0;
    }
  }
  return v;
}
template <bool WHOLE>
__device__ __forceinline__ void put8(uint16_t* row, int c, int N, bool full, us8_t v) {
  if constexpr (WHOLE) {
    reinterpret_cast<us8_t*>(row)[c] = v;
  } else if (full) {
    __builtin_memcpy(row + c * 8, &v, 16);
  } else {
#pragma unroll
    for (int j = 0; j < 8; j++)
      if (c * 8 + j < N) row[c * 8 + j] = v[j];
  }
}

// What a token's factors have shown so far: the largest, which bits are set in any
// of its d (none: all are zero), and whether all of d (dg, du) are finite.
struct Seen {
  float top = 0;
  int bits = 0;
  bool finite = true;
};

// The gradient that a row's scale multiplies: d itself (d0) or, of the gated
// block, the gate's dg (d0) and the up projection's du (d1).
template <int ACT, bool BF>
__device__ __forceinline__ void gradients(uint16_t d, uint16_t g, uint16_t u, float& d0,
                                          float& d1) {
  d0 = elem_to_f32(d, BF);
  d1 = 0;
  if constexpr (ACT >= 0) {
    float f, df;
    act_value_slope(elem_to_f32(g, BF), ACT, f, df);
    d1 = d0 * f;
    d0 = d0 * elem_to_f32(u, BF) * df;
  }
}

// The factors d s of chunk c (gated: of the gate and the up part), in fp32;
// `write`: dg and du go out.
template <int ACT, bool BF, bool WHOLE>
__device__ __forceinline__ void factors8(const PrepArgs& p, int64_t row, int c, bool write,
                                         float (&a)[ACT < 0 ? 1 : 2][8], Seen& seen) {
  constexpr bool GATED = ACT >= 0;
  constexpr int M = GATED ? 2 : 1;
  const bool full = WHOLE || c * 8 + 8 <= p.N;
  us8_t d, g, u, og, ou, sc[M];
  auto read = [&](bool f) {  // one branch for all, so that they are under way together
    d = get8<WHOLE>(p.d + row * p.N, c, p.N, f);
    if constexpr (GATED) {
      g = get8<WHOLE>(p.gate + row * p.N, c, p.N, f);
      u = get8<WHOLE>(p.up + row * p.N, c, p.N, f);
    }
#pragma unroll
    for (int m = 0; m < M; m++) sc[m] = get8<WHOLE>(p.w[m].scales, c, p.N, f);
  };
  if (full)
    read(true);
  else
    read(false);
  const i4_t bits = __builtin_bit_cast(i4_t, d);
  seen.bits |= bits[0] | bits[1] | bits[2] | bits[3];
#pragma unroll
  for (int j = 0; j < 8; j++) {
    float d0, d1;
    gradients<ACT, BF>(d[j], GATED ? g[j] : 0, GATED ? u[j] : 0, d0, d1);
    a[0][j] = d0 * h_bits_to_f32(sc[0][j]);
    if constexpr (GATED) {
      og[j] = f32_to_elem(d0, BF);
      ou[j] = f32_to_elem(d1, BF);
      a[M - 1][j] = d1 * h_bits_to_f32(sc[M - 1][j]);
    }
    seen.finite = seen.finite && fabsf(d0) < INFINITY && fabsf(d1) < INFINITY;
#pragma unroll
    for (int m = 0; m < M; m++) seen.top = fmaxf(seen.top, fabsf(a[m][j]));
  }
  if (GATED && write) {
    put8<WHOLE>(p.dgate + row * p.N, c, p.N, full, og);
    put8<WHOLE>(p.dup + row * p.N, c, p.N, full, ou);
  }
}

// The preparation of a token whose factors are below 2^-110 (bf16 gradients near
// the end of its range), one value at a time: with scales 2^100 times as large no
// factor is subnormal (d is 2^-133 or more, s 2^-24), and none above 2^-10.
template <int ACT, bool BF>
__device__ __forceinline__ void tiny_factors(const PrepArgs& p, int64_t row, float* red) {
  constexpr int M = ACT < 0 ? 1 : 2, kMore = 100;
  const int tid = threadIdx.x, nt = blockDim.x;
  auto factors = [&](int n, float(&a)[M]) {
    const int64_t at = row * p.N + n;
    float d[2];
    gradients<ACT, BF>(p.d[at], ACT < 0 ? 0 : p.gate[at], ACT < 0 ? 0 : p.up[at], d[0], d[1]);
    for (int m = 0; m < M; m++)
      a[m] = d[m] * __builtin_amdgcn_ldexpf(h_bits_to_f32(p.w[m].scales[n]), kMore);
  };
  float a[M], top = 0, r = 0;
#pragma unroll 1
  for (int n = tid; n < p.N; n += nt) {
    factors(n, a);
    for (int m = 0; m < M; m++) top = fmaxf(top, fabsf(a[m]));
  }
  top = block_max(top, red, tid);
  const int e = top > 0 ? 15 - __builtin_amdgcn_frexp_expf(top) : 0;
#pragma unroll 1
  for (int n = tid; n < p.half; n += nt) {
    if (n < p.N) factors(n, a);
    for (int m = 0; m < M; m++) {
      uint16_t out = 0;
      if (n < p.N) {
        out = f32_to_h_bits(__builtin_amdgcn_ldexpf(a[m], e));
        r += h_bits_to_f32(out) * (float)(128 - p.w[m].zeros[n]);
      }
      p.a[row * p.pitch + m * p.half + n] = out;
    }
  }
  r = block_sum(r, red, tid);
  if (tid == 0) {
    p.r[row] = r;
    p.e[row] = e + kMore;
  }
}

// One workgroup per token.  ACT: the gated block's activation, or -1 for the
// linear layer.  NC > 0: the factors stay in registers, NC chunks per thread,
// between their largest and their rounding, so the inputs are read once; NC == 0
// (rows longer than that): they are made twice.  Bound by HBM with many tokens
// (4096 of 2 x 28672, dg and du written too: 338 us, 4.9 TB/s), by the vector
// ALUs of a token's CU with few (64 of 2 x 28672 13.9 us; a quarter more with the
// activation and the type decided at run time, whose branches part the values).
// Each row's scales and zero points come from L2.  Rows that lie at 2 bytes:
// 61 of 2 x 11007 16.5 us, of 2 x 11008 8.5.
template <int ACT, bool BF, int NC, bool WHOLE>
__global__ __launch_bounds__(1024) void grad_prep_kernel(const PrepArgs p) {
  __shared__ float red[16];
  constexpr int M = ACT < 0 ? 1 : 2;
  const int tid = threadIdx.x, nt = blockDim.x, chunks = (p.N + 7) / 8, all = p.half / 8;
  const int64_t row = blockIdx.x;
  float held[NC > 0 ? NC : 1][M][8];
  Seen seen;
  const bool write = p.dgate != nullptr;
  if constexpr (NC > 0) {
#pragma unroll
    for (int i = 0; i < NC; i++) {
      const int c = tid + i * nt;
      if (c < chunks) factors8<ACT, BF, WHOLE>(p, row, c, write, held[i], seen);
    }
  } else {
    for (int c = tid; c < chunks; c += nt)
      factors8<ACT, BF, WHOLE>(p, row, c, write, held[0], seen);
  }
  const float top = block_max(seen.finite ? seen.top : INFINITY, red, tid);
  // Below 2^-139 fp32 has less than 11 bits, and factors are to keep theirs down to
  // 2^-29 of the largest.  Tokens of zeros need no second look, and an fp16 value
  // by an fp16 scale is 2^-48 or more.
  if constexpr (BF || ACT >= 0) {
    if (uniform(top < 0x1p-110f) && uniform(__syncthreads_or(seen.bits & 0x7fff7fff))) {
      tiny_factors<ACT, BF>(p, row, red);
      return;
    }
  }
  const bool ok = top < INFINITY;
  const int e = ok && top > 0 ? 15 - __builtin_amdgcn_frexp_expf(top) : 0;
  float r = 0;
  auto round8 = [&](int c, const float(&a)[M][8]) {
#pragma unroll
    for (int m = 0; m < M; m++) {
      us8_t out = {};
      if (ok && c < chunks) {
        int z[8];
        if (WHOLE || c * 8 + 8 <= p.N) {
          const i4_t* zp = reinterpret_cast<const i4_t*>(p.w[m].zeros) + c * 2;
          __builtin_memcpy(z, zp, 32);
        } else {
#pragma unroll
          for (int j = 0; j < 8; j++) z[j] = p.w[m].zeros[min(c * 8 + j, p.N - 1)];
        }
#pragma unroll
        for (int j = 0; j < 8; j++) {  // positions past N: factors 0
          out[j] = f32_to_h_bits(__builtin_amdgcn_ldexpf(a[m][j], e));
          r += h_bits_to_f32(out[j]) * (float)(128 - z[j]);
        }
      }
      reinterpret_cast<us8_t*>(p.a + row * p.pitch + m * p.half)[c] = out;
    }
  };
  if constexpr (NC > 0) {
#pragma unroll
    for (int i = 0; i < NC; i++) {
      const int c = tid + i * nt;
      if (c < all) round8(c, held[i]);
    }
  } else {
    for (int c = tid; c < all; c += nt) {
      if (c < chunks) factors8<ACT, BF, WHOLE>(p, row, c, false, held[0], seen);
      round8(c, held[0]);
    }
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
  int T, N, K, pitch, half_steps, steps, bf16;
};

// Four code bytes to the exact fp16 integers code - 128: one byte permute
// drops two codes under the exponent bytes of 1024, one packed subtraction.
__device__ __forceinline__ void codes_to_f16(uint32_t w, h2_t& lo, h2_t& hi) {
  const h2_t off = {(_Float16)1152.0f, (_Float16)1152.0f};
  lo = as_h2(__builtin_amdgcn_perm(0x64646464u, w, 0x04010400u)) - off;
  hi = as_h2(__builtin_amdgcn_perm(0x64646464u, w, 0x04030402u)) - off;
}

// Where chunk c (16 bytes) of weight row n lies in its row of KT bytes: the 16
// rows that two quarters of a transposing read touch meet 16 different 16-byte
// slots of the 256 bytes that the banks span.
template <int KT>
__device__ __forceinline__ int slot_of(int n, int c) {
  if constexpr (KT % 256 == 0) return c ^ (n & 15);
  if constexpr (KT == 128) return c ^ ((n >> 1) & 7);
  return (c & ~3) | ((c + (n >> 2)) & 3);  // 192
}
template <int KT>
__device__ __forceinline__ int chunk_at(int n, int slot) {
  if constexpr (KT % 256 == 0 || KT == 128) return slot_of<KT>(n, slot);
  return (slot & ~3) | ((slot - (n >> 2)) & 3);
}

__device__ __forceinline__ void store_dx(const GradArgs& p, f4_t sum, float r, int e, int t, int k) {
  us4_t out;
#pragma unroll
  for (int q = 0; q < 4; q++)
    out[q] = f32_to_elem(__builtin_amdgcn_ldexpf(sum[q] + r, e), p.bf16);
  *reinterpret_cast<us4_t*>(static_cast<uint16_t*>(p.dx) + (int64_t)t * p.K + k) = out;
}

// One workgroup of WM x WN waves: MT tokens by KT columns of dx over its share
// of the steps, 64 weight rows each, staged in LDS by direct loads on a ring
// of NB buffers, one barrier per step.  The weight tile lies as it does in
// memory, rows of KT code bytes; the matrix cores need eight rows of one
// column per lane, which the transposing LDS read delivers (16 lanes read 8
// rows of 16 bytes and get a column each).  A step is two halves of 32 rows:
// while one half is multiplied, the operands of the next are read.
//
// 4096 x (2 x 28672) x 8192 takes 2.7-2.8 ms, 1.4 PFLOP/s: the matrix cores
// are busy in 73% of the clocks, at 1.8 GHz, which is all that power allows here
// (products from registers alone reach 2.0 PFLOP/s at 1.9 GHz).  With a part left
// out, of 2.75 ms: 2.27 without the direct loads, 2.48 without the operand reads,
// 2.12 without both, 1.49 without the products; of the 89 us of 1000x4096x11008
// 81, 85, 76 and 53.  Slower there: four waves of 128 x 128 (2.92 ms), steps of 32
// rows (3.1 ms).  The small tiles wait for the weights: 61 x (2 x 11008) x 4096
// takes 26 us on weights rotated over 1 GiB (3.5 TB/s), 20 where they lie in the
// last-level cache.
template <int MT, int KT, int WM, int WN, int NB>
__global__ __launch_bounds__(WM* WN * 64, 2) void grad_kernel(const GradArgs p, const TilePlan plan,
                                                                 f4_t* __restrict__ parts) {
  constexpr int kWaves = WM * WN;
  constexpr int MW = MT / WM, KW = KT / WN;
  constexpr int FM = MW / 16, FK = KW / 16;
  constexpr int kA = MT * kStepN * 2, kW = kStepN * KT, kBuf = kA + kW;
  // 1 KiB loads per wave and step; where the weight rows do not come out even,
  // the last go to a place of their own, so that every wave counts as many
  constexpr int LA = kA / 1024 / kWaves, kLW = kW / 1024, LW = (kLW + kWaves - 1) / kWaves;
  constexpr int kLoads = LA + LW;
  static_assert(LA * 1024 * kWaves == kA && kLW * 1024 == kW, "whole loads");
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WM, wn = wave / WM;
  const int i16 = lane & 15, h = lane >> 4;
  // a whole tile, or a share of the steps of one of the rest
  const int over = (int)blockIdx.x - plan.whole;
  const int split = over < 0 ? 0 : over % plan.splits;
  const int s0 = over < 0 ? 0 : (int)((int64_t)p.steps * split / plan.splits);
  const int s1 = over < 0 ? p.steps : (int)((int64_t)p.steps * (split + 1) / plan.splits);
  int tm, tn;
  tile_of(over < 0 ? (int)blockIdx.x : plan.whole + over / plan.splits, plan.whole, plan.tiles_m,
          plan.tiles_n, tm, tn);
  const int t0 = tm * MT, k0 = tn * KT;
  const uint32_t K = (uint32_t)p.K;

  const uint32_t pitch = (uint32_t)p.pitch * 2;
  const i4_t ra = buffer_of(p.a + (int64_t)t0 * p.pitch, (uint32_t)min(MT, p.T - t0) * pitch);
  uint32_t oa[LA], ow[LW];
  const uint32_t base = lds_address(lds);
#pragma unroll
  for (int i = 0; i < LA; i++)
    oa[i] = (uint32_t)((wave + i * kWaves) * 8 + (lane >> 3)) * pitch +
            ((lane & 7) ^ (lane >> 3)) * 16;
#pragma unroll
  for (int i = 0; i < LW; i++) {
    const int at = (wave + i * kWaves) * 64 + lane, n = at / (KT / 16);
    const int k = k0 + chunk_at<KT>(n, at % (KT / 16)) * 16;
    // columns past the end: not stored, so not loaded either
    ow[i] = k < p.K && n < kStepN ? (uint32_t)n * K + k : 0x80000000u;
  }
  // load i of step s; past the share's end it brings zeros
  auto load = [&](int s, int i) {
    const uint32_t buf = base + (uint32_t)((s - s0) % NB) * kBuf;
    if (i < LA) {
      const uint32_t at = s < s1 ? (uint32_t)s * (kStepN * 2) : 0x80000000u;
      load_to_lds(ra, buf + (wave + i * kWaves) * 1024, oa[i] + at);
    } else {
      const int m = s >= p.half_steps;
      const int n = (s - m * p.half_steps) * kStepN;
      const int rows = s < s1 ? max(0, min(kStepN, p.N - n)) : 0;
      const i4_t rs = buffer_of(p.w[m].codes + (int64_t)n * K, (uint32_t)rows * K);
      const int at = wave + (i - LA) * kWaves;
      const bool spare = kLW % kWaves != 0 && at >= kLW;
      load_to_lds(rs, spare ? base + NB * kBuf : buf + kA + at * 1024, ow[i - LA]);
    }
  };

  f4_t acc[FK][FM];
#pragma unroll
  for (int i = 0; i < FK; i++)
#pragma unroll
    for (int j = 0; j < FM; j++) acc[i][j] = f4_t{0, 0, 0, 0};

  // operands of a half step: tokens as they lie, codes transposed
  const int ra0 = (wm * MW + i16) * (kStepN * 2);
  auto tokens = [&](int s, int ks, int j) {
    const int at = ((ks * 4 + h) ^ (i16 & 7)) * 16;
    return *reinterpret_cast<const h8_t*>(lds + (s - s0) % NB * kBuf + ra0 +
                                          j * 16 * (kStepN * 2) + at);
  };
  auto rows = [&](int s, int ks, int i) {
    // lanes 2r and 2r + 1 of 16 read the two halves of row r's 16 bytes
    const int n = ks * 32 + h * 8 + (i16 >> 1);
    const uint8_t* at = lds + (s - s0) % NB * kBuf + kA + n * KT +
                        slot_of<KT>(n, wn * (KW / 16) + i) * 16 + (i16 & 1) * 8;
    return __builtin_amdgcn_ds_read_tr8_b64_v2i32(
        (__attribute__((address_space(3))) i2_t*)at);
  };
  auto multiply = [&](const i2_t w, const h8_t(&fa)[FM], int i) {
    h2_t q[4];
    codes_to_f16((uint32_t)w[0], q[0], q[1]);
    codes_to_f16((uint32_t)w[1], q[2], q[3]);
    const h8_t fw = {q[0][0], q[0][1], q[1][0], q[1][1], q[2][0], q[2][1], q[3][0], q[3][1]};
#pragma unroll
    for (int j = 0; j < FM; j++)
      acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fw, fa[j], acc[i][j], 0, 0, 0);
  };
  if (s0 < s1) {
    h8_t f0[FM], f1[FM];
    i2_t w0[FK], w1[FK];
#pragma unroll
    for (int s = 0; s < NB - 1; s++)
#pragma unroll
      for (int i = 0; i < kLoads; i++) load(s0 + s, i);
    lds_loads_left<(NB - 2) * kLoads>();
    __syncthreads();
#pragma unroll
    for (int i = 0; i < FK; i++) w0[i] = rows(s0, 0, i);
#pragma unroll
    for (int j = 0; j < FM; j++) f0[j] = tokens(s0, 0, j);
    for (int s = s0; s < s1; s++) {
#pragma unroll
      for (int i = 0; i < FK; i++) {
#pragma unroll
        for (int l = i * kLoads / FK; l < (i + 1) * kLoads / FK; l++) load(s + NB - 1, l);
        w1[i] = rows(s, 1, i);
#pragma unroll
        for (int j = i * FM / FK; j < (i + 1) * FM / FK; j++) f1[j] = tokens(s, 1, j);
        multiply(w0[i], f0, i);
        __builtin_amdgcn_sched_barrier(0);
      }
      lds_loads_left<(NB - 2) * kLoads>();  // this wave's part of the next step has landed
      __syncthreads();                      // and everyone's; step s has been read
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < FK; i++) {
        w0[i] = rows(s + 1, 0, i);
#pragma unroll
        for (int j = i * FM / FK; j < (i + 1) * FM / FK; j++) f0[j] = tokens(s + 1, 0, j);
        multiply(w1[i], f1, i);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    lds_loads_left<0>();
  }

  if (over >= 0) {
    f4_t* to = parts + ((int64_t)over * kWaves + wave) * (FK * FM * 64) + lane;
#pragma unroll
    for (int i = 0; i < FK; i++)
#pragma unroll
      for (int j = 0; j < FM; j++) to[(i * FM + j) * 64] = acc[i][j];
    return;
  }
  // lane l of a fragment holds columns k = 4 (l / 16) + 0..3 of token l % 16
#pragma unroll
  for (int j = 0; j < FM; j++) {
    const int t = t0 + wm * MW + j * 16 + i16;
    if (t >= p.T) continue;
    const float r = p.r[t];
    const int e = -p.e[t];
#pragma unroll
    for (int i = 0; i < FK; i++) {
      const int k = k0 + wn * KW + i * 16 + h * 4;
      if (k < p.K) store_dx(p, acc[i][j], r, e, t, k);
    }
  }
}

// Joins the shares of the plan's rest, in their order: one wave for each
// fragment of a tile.
template <int MT, int KT, int WM, int WN>
__global__ __launch_bounds__(256) void grad_join_kernel(const GradArgs p, const TilePlan plan,
                                                        const f4_t* __restrict__ parts) {
  constexpr int kWaves = WM * WN;
  constexpr int MW = MT / WM, KW = KT / WN, FM = MW / 16, FK = KW / 16;
  constexpr int kFragments = kWaves * FK * FM;
  const int lane = threadIdx.x & 63;
  const int at = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int tile = at / kFragments, f = at % kFragments;
  if (tile >= plan.rest) return;
  const int wave = f / (FK * FM), i = f / FM % FK, j = f % FM;
  int tm, tn;
  tile_of(plan.whole + tile, plan.whole, plan.tiles_m, plan.tiles_n, tm, tn);
  const int k = tn * KT + wave / WM * KW + i * 16 + (lane >> 4) * 4;
  const int t = tm * MT + wave % WM * MW + j * 16 + (lane & 15);
  if (k >= p.K || t >= p.T) return;
  f4_t sum = {0, 0, 0, 0};
  for (int z = 0; z < plan.splits; z += 4) {  // four loads at a time
    f4_t v[4];
#pragma unroll
    for (int u = 0; u < 4; u++) {
      const int zz = min(z + u, plan.splits - 1);
      v[u] = parts[((int64_t)(tile * plan.splits + zz) * kWaves + wave) * (FK * FM * 64) +
                   (i * FM + j) * 64 + lane];
    }
#pragma unroll
    for (int u = 0; u < 4; u++)
      if (z + u < plan.splits) sum += v[u];
  }
  store_dx(p, sum, p.r[t], -p.e[t], t, k);
}

template <int MT, int KT, int WM, int WN, int NB>
hipError_t launch_tile(const GradArgs& p, const TilePlan& plan, f4_t* parts, hipStream_t stream) {
  constexpr bool spare = kStepN * KT / 1024 % (WM * WN) != 0;
  constexpr int bytes = NB * (MT * kStepN * 2 + kStepN * KT) + (spare ? 1024 : 0);
  auto kernel = grad_kernel<MT, KT, WM, WN, NB>;
  hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(kernel), bytes);
  if (e != hipSuccess) return e;
  kernel<<<dim3((unsigned)plan.blocks()), dim3(WM * WN * 64), bytes, stream>>>(p, plan, parts);
  e = hipGetLastError();
  if (e != hipSuccess || plan.rest == 0) return e;
  constexpr int fragments = (MT / 16) * (KT / 16);
  grad_join_kernel<MT, KT, WM, WN>
      <<<dim3((unsigned)((plan.rest * fragments + 3) / 4)), dim3(256), 0, stream>>>(p, plan, parts);
  return hipGetLastError();
}

template <int ACT, bool BF, bool WHOLE>
void launch_prep_rows(const PrepArgs& q, int64_t T, hipStream_t stream) {
  const dim3 grid((unsigned)T);
  const int chunks = q.half / 8;
  int nt = 64;
  while (nt < 1024 && nt < chunks) nt *= 2;
  if (chunks <= nt)
    grad_prep_kernel<ACT, BF, 1, WHOLE><<<grid, dim3(nt), 0, stream>>>(q);
  else if (chunks <= 2 * nt)
    grad_prep_kernel<ACT, BF, 2, WHOLE><<<grid, dim3(nt), 0, stream>>>(q);
  else if (chunks <= 4 * nt)
    grad_prep_kernel<ACT, BF, 4, WHOLE><<<grid, dim3(nt), 0, stream>>>(q);
  else
    grad_prep_kernel<ACT, BF, 0, WHOLE><<<grid, dim3(nt), 0, stream>>>(q);
}
template <int ACT>
void launch_prep(const PrepArgs& q, int64_t T, bool bf16, hipStream_t stream) {
  const bool whole = q.N % 8 == 0;
  if (bf16)
    whole ? launch_prep_rows<ACT, true, true>(q, T, stream)
          : launch_prep_rows<ACT, true, false>(q, T, stream);
  else
    whole ? launch_prep_rows<ACT, false, true>(q, T, stream)
          : launch_prep_rows<ACT, false, false>(q, T, stream);
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }
int64_t padded(int64_t N) { return (N + kStepN - 1) / kStepN * kStepN; }

}  // namespace

size_t w8a8_grad_workspace_bytes(int64_t T, int64_t N, int64_t K, bool gated) {
  if (T == 0) return 0;
  const int64_t pitch = padded(N) * (gated ? 2 : 1);
  return up256((size_t)T * pitch * 2) + 2 * up256((size_t)T * 4) +
         grad_plan(T, K, (int)(pitch / kStepN), device_cu_count()).part_bytes();
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
  const bool bf16 = dtype == kBF16;
  if (!gated)
    launch_prep<-1>(q, T, bf16, stream);
  else if (act == kSilu)
    launch_prep<kSilu>(q, T, bf16, stream);
  else
    launch_prep<kGeluTanh>(q, T, bf16, stream);
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
  p.bf16 = bf16;
  const GradPlan plan = grad_plan(T, K, p.steps, device_cu_count());
  auto* parts =
      reinterpret_cast<f4_t*>(reinterpret_cast<uint8_t*>(q.e) + up256((size_t)T * 4));
  switch (plan.shape) {
    case 0:
      return launch_tile<16, 128, 1, 2, 4>(p, plan.tiles, parts, stream);
    case 1:
      return launch_tile<32, 128, 1, 4, 4>(p, plan.tiles, parts, stream);
    case 2:
      return launch_tile<64, 128, 1, 4, 4>(p, plan.tiles, parts, stream);
    case 3:
      return launch_tile<64, 256, 1, 8, 3>(p, plan.tiles, parts, stream);
    case 4:
      return launch_tile<128, 128, 2, 2, 3>(p, plan.tiles, parts, stream);
    case 5:
      return launch_tile<128, 256, 2, 4, 3>(p, plan.tiles, parts, stream);
    case 6:
      return launch_tile<256, 192, 2, 4, 3>(p, plan.tiles, parts, stream);
    default:
      return launch_tile<256, 256, 2, 4, 3>(p, plan.tiles, parts, stream);
  }
}

}  // namespace lowbit
