// lora.hip -- out = y + s_l b_l (a_l x): low-rank adapters of many requests beside a
// shared projection.
//
// Two kernels.  The first contracts over K: a workgroup takes one tile of tokens of
// one adapter and a share of K, and leaves v's share in the workspace.  The second
// adds the shares up, and expands over N: it takes a tile and a range of outputs.
// Bound by HBM: for few tokens the adapters (2 R (K + N) bytes each), for many x, y
// and out (2 T (K + 2 N) bytes).  8192 tokens of 12288x12288, 64 ranks: contraction 63 us
// (39 where the last call's outputs are not on their way to HBM, 5.1 TB/s), expansion 92
// (4.4 TB/s; 16 ranks 75, 5.4).  64 tokens of 64 adapters of 11008x4096, 16 ranks: 5.0 + 8.4 us.
// Both at once, each workgroup of the expansion contracting for itself, took 9.1 us against
// 3.7 + 4.7 for one token of 4096x4096 and 13.6 against 13.4 for these 64.
#include "lora.h"

#include <type_traits>

namespace lowbit {
namespace {

constexpr int kLoraWaves = 4;  // of the expansion

// ---------------------------------------------------------------------------
// v = a x
// ---------------------------------------------------------------------------
struct DownArgs {
  LoraArgs p;
  const uint16_t* x;
  float* shares;  // [splits][T][R], rows in the plan's order
  int k_share;    // a multiple of 64
};

// TB blocks of 16 tokens, RB of 16 ranks (blockIdx.z: which 64 ranks), W waves.  A wave's
// step is 64 of K; the next step's rows are under way while one is multiplied.  No load
// stands behind a lane's condition, which would make the compiler wait for it at once.
template <int RB, int TB, int W>
constexpr int down_bytes() {
  constexpr int stage = W * (RB + TB) * 16 * 128, reduce = reduce_bytes<RB, TB, W>();
  return stage > reduce ? stage : reduce;
}
template <bool BF, int RB, int TB, int W>
__global__ __launch_bounds__(W * 64, W == 4 ? 2 : 1) void lora_down_kernel(const DownArgs g) {
  constexpr int TILE = 16 * TB, RANKS = 16 * RB;
  extern __shared__ __align__(16) char lds[];
  const LoraArgs& p = g.p;
  LoraTile tile;
  if (!find_tile(p.starts, p.L, (int)p.T, TILE, blockIdx.x, tile) || tile.l == p.L) return;
  const int lane = threadIdx.x & 63, wave = wave_of_group();
  const int row = lane >> 3, chunk = lane & 7;
  const int64_t K = p.K;
  const int r0 = blockIdx.z * 64, ranks = min(p.R - r0, RANKS);
  uint16_t* const sx = reinterpret_cast<uint16_t*>(lds) + wave * (TILE + RANKS) * 64;
  uint16_t* const sa = sx + TILE * 64;
  const uint16_t *xr[TILE / 8], *ar[RANKS / 8];
#pragma unroll
  for (int q = 0; q < TILE / 8; q++)
    xr[q] = g.x + token_at(p.order, p.T, tile.begin + min(q * 8 + row, tile.count - 1)) * K + chunk * 8;
#pragma unroll
  for (int q = 0; q < RANKS / 8; q++)
    ar[q] = p.a + ((int64_t)tile.l * p.R + r0 + min(q * 8 + row, ranks - 1)) * K + chunk * 8;
  f4_t acc[RB][TB];
#pragma unroll
  for (int i = 0; i < RB; i++)
#pragma unroll
    for (int j = 0; j < TB; j++) acc[i][j] = f4_t{0, 0, 0, 0};
  const int k0 = blockIdx.y * g.k_share, k1 = min(k0 + g.k_share, p.K);
  us8_t vx[TILE / 8], va[RANKS / 8];
  auto load = [&](int k) {
#pragma unroll
    for (int q = 0; q < TILE / 8; q++) vx[q] = *reinterpret_cast<const us8_t*>(xr[q] + k);
#pragma unroll
    for (int q = 0; q < RANKS / 8; q++) va[q] = *reinterpret_cast<const us8_t*>(ar[q] + k);
  };
  auto stage = [&] {
    put_rows<TILE>(sx, vx);
    put_rows<RANKS>(sa, va);
    wave_lds_order();
  };
  auto multiply = [&] {
#pragma unroll
    for (int half = 0; half < 2; half++) {
      us8_t fa[RB];
#pragma unroll
      for (int i = 0; i < RB; i++) fa[i] = get_operand(sa, i, half);
#pragma unroll
      for (int j = 0; j < TB; j++) {
        const us8_t fx = get_operand(sx, j, half);
#pragma unroll
        for (int i = 0; i < RB; i++) acc[i][j] = Half16<BF>::mma(fa[i], fx, acc[i][j]);
      }
    }
    wave_lds_order();
  };
  int k = k0 + wave * 64;
  if (k + 64 <= k1) {
    load(k);
    for (; k + W * 64 + 64 <= k1; k += W * 64) {
      stage();
      load(k + W * 64);
      multiply();
    }
    stage();
    multiply();
    k += W * 64;
  }
  if (k < k1) {  // K is a multiple of 32: half a step, the other half's chunks are zero
    load(chunk < 4 ? k : k - 32);
#pragma unroll
    for (int q = 0; q < TILE / 8; q++) vx[q] = chunk < 4 ? vx[q] : us8_t{};
#pragma unroll
    for (int q = 0; q < RANKS / 8; q++) va[q] = chunk < 4 ? va[q] : us8_t{};
    stage();
    multiply();
  }
  reduce_waves<RB, TB, W>(acc, wave, lds);
  if (wave == 0)
    store_shares(acc, g.shares + ((int64_t)blockIdx.y * p.T + tile.begin) * p.R + r0, p.R,
                 tile.count, ranks);
}

// ---------------------------------------------------------------------------
// out = y + s b v
// ---------------------------------------------------------------------------
struct UpArgs {
  LoraArgs p;
  const float* shares;
  int splits;
  int n_share;  // a multiple of 64
  const uint16_t* y;
  uint16_t* out;
  float* v;
};

// A wave's step is 64 outputs, or 32 where there are more than 64 ranks, so that two
// workgroups fit a CU (1500 tokens of 8192x8192, 128 ranks: 53 -> 31 us).  The next step's rows
// of b and y are under way while one is multiplied.  Results pass through LDS too, in fp32,
// 16 tokens at a time: eight (four) lanes then hold the outputs of one token as y's rows lie.
template <int RB>
constexpr int kOut = RB < 8 ? 64 : 32;
template <int RB>
constexpr int up_wave_bytes() {
  constexpr int b = kOut<RB> * RB * 32, result = 16 * (kOut<RB> + 4) * 4;
  return b > result ? b : result;
}
template <int RB, int TB>
constexpr int up_bytes() {
  return TB * 16 * ((RB * 32 + 8) * 2 + 4) + kLoraWaves * up_wave_bytes<RB>();
}
template <bool BF, int RB, int TB>
__global__ __launch_bounds__(kLoraWaves * 64, 2) void lora_up_kernel(const UpArgs g) {
  constexpr int TILE = 16 * TB, PITCH = RB * 32 + 8, OUT = kOut<RB>, STEP = kLoraWaves * OUT;
  constexpr int C = Ranks<RB>::kChunks, CHUNKS = RB * 2;
  constexpr int LOADS = OUT * CHUNKS / 64;             // of b's rows, a lane
  constexpr int LANES = OUT / 8, ROWS = 64 / LANES;    // lanes of a row of y, rows of a load
  constexpr int ROUNDS = 16 / ROWS;                    // loads of 16 tokens
  extern __shared__ __align__(16) char lds[];
  uint16_t(*const parts)[PITCH] = reinterpret_cast<uint16_t(*)[PITCH]>(lds);
  int* const exponent = reinterpret_cast<int*>(lds + TILE * PITCH * 2);
  const LoraArgs& p = g.p;
  LoraTile tile;
  if (!find_tile(p.starts, p.L, (int)p.T, TILE, blockIdx.x, tile)) return;
  const bool none = tile.l == p.L;
  const bool in_place = g.y == g.out;
  if (none && in_place && !g.v) return;
  const int lane = threadIdx.x & 63, wave = wave_of_group();
  const int i16 = lane & 15, h = lane >> 4, row = lane / LANES, chunk = lane % LANES;
  char* const mine = lds + TILE * (PITCH * 2 + 4) + wave * up_wave_bytes<RB>();
  uint16_t* const sb = reinterpret_cast<uint16_t*>(mine);  // [OUT][CHUNKS] chunks
  float(*const result)[OUT + 4] = reinterpret_cast<float(*)[OUT + 4]>(mine);  // [16], after b is read
  const int64_t N = p.N;
  int64_t at[TILE / ROWS];  // of token ROWS q + row, this lane's eight outputs
#pragma unroll
  for (int q = 0; q < TILE / ROWS; q++)
    at[q] = token_at(p.order, p.T, tile.begin + min(q * ROWS + row, tile.count - 1)) * N + chunk * 8;
  const int n1 = min((int)(blockIdx.y + 1) * g.n_share, p.N);
  // b's rows lie in one piece: 16-byte chunk 64 q + lane of it (the last one again beyond), and
  // where it goes.
  // Chunk c of row n is in slot c ^ (n >> SHIFT) % CHUNKS, as in row_slot(): rows of 32, 64, 128 and
  // 256 bytes, eight, four, two and two of them with one slot order.
  const int per_row = p.R / 8;
  auto slot = [&](int n, int c) {
    constexpr int SHIFT = RB == 1 ? 3 : RB == 2 ? 2 : 1;
    return n * RB * 16 + ((c ^ ((n >> SHIFT) & (CHUNKS - 1))) << 3);
  };
  auto item = [&](int q) {
    return OUT == 64 ? q * 64 + lane : min(q * 64 + lane, per_row * OUT - 1);
  };
  int place[LOADS];
#pragma unroll
  for (int q = 0; q < LOADS; q++) {
    const int i = item(q);
    place[q] = slot(i / per_row % OUT, i % per_row);
  }
  us8_t vb[LOADS], had[TILE / ROWS], ahead[TILE / ROWS];
  const uint16_t* const b = p.b + (int64_t)(none ? 0 : tile.l) * N * p.R;
  auto load_b = [&](int n0) {
#pragma unroll
    for (int q = 0; q < LOADS; q++)
      if (q * 64 < per_row * OUT)
        vb[q] = *reinterpret_cast<const us8_t*>(b + (int64_t)n0 * p.R + item(q) * 8);
  };
  // without a y: read what out holds, to no one's use
  const uint16_t* const y = g.y ? g.y : g.out;
  auto load_y = [&](us8_t(&to)[TILE / ROWS], int n0) {
#pragma unroll
    for (int q = 0; q < TILE / ROWS; q++) to[q] = load8(y + at[q] + n0);
  };
  us8_t fb[OUT / 16][C];
  auto stage_b = [&] {
#pragma unroll
    for (int q = 0; q < LOADS; q++)
      if (q * 64 < per_row * OUT) *reinterpret_cast<us8_t*>(sb + place[q]) = vb[q];
    wave_lds_order();
#pragma unroll
    for (int i = 0; i < OUT / 16; i++)
#pragma unroll
      for (int c = 0; c < C; c++) {
        const int r = Ranks<RB>::of(c, h);
        fb[i][c] = *reinterpret_cast<const us8_t*>(sb + slot(i * 16 + i16, r / 8));
        if (RB * 16 > p.R && r >= p.R) fb[i][c] = us8_t{};
      }
    wave_lds_order();
  };
  // the step's outputs of token block j, whose y and places are given, `left` of a lane's eight inside
  auto finish = [&](int j, int n0, const us8_t* y2, const int64_t* at2, auto whole, int left) {
    f4_t acc[OUT / 16] = {};
    multiply_parts<BF, RB>(fb, parts[j * 16 + i16], h, acc);
#pragma unroll
    for (int i = 0; i < OUT / 16; i++)
      *reinterpret_cast<f4_t*>(&result[i16][i * 16 + h * 4]) = acc[i];
    wave_lds_order();
#pragma unroll
    for (int q = 0; q < ROUNDS; q++) {
      const int t = q * ROWS + row;
      const f4_t lo = *reinterpret_cast<const f4_t*>(&result[t][chunk * 8]);
      const f4_t hi = *reinterpret_cast<const f4_t*>(&result[t][chunk * 8 + 4]);
      const int e = BF ? 0 : exponent[j * 16 + t];
      us8_t o = g.y ? y2[q] : us8_t{};
      // a token without an adapter keeps the bits it has
      if (!none)
#pragma unroll
        for (int m = 0; m < 8; m++) {
          float f = m < 4 ? lo[m % 4] : hi[m % 4];
          if (!BF) f = times_power(f, -e);
          if (g.y) f += Half16<BF>::to(o[m]);
          o[m] = Half16<BF>::from(f);
        }
      if (j * 16 + t < tile.count) {
        if (whole)
          store8(g.out + at2[q] + n0, o);
        else
          store8(g.out + at2[q] + n0, o, left);
      }
    }
    wave_lds_order();
  };
  int n0 = blockIdx.y * g.n_share + wave * OUT;
  // the first step's loads are under way while v's shares are added up
  if (n0 + OUT <= n1) {
    load_y(had, n0);
    load_b(n0);
  }
  spread_parts<BF, RB, TILE, kLoraWaves * 64>(
      [&](int t, int r) {
        f4_t val = {0, 0, 0, 0};
        if (!none)
          val = add_shares(g.shares + ((int64_t)tile.begin + t) * p.R + r, p.T * p.R, g.splits);
        if (g.v && blockIdx.y == 0)
          *reinterpret_cast<f4_t*>(g.v + token_at(p.order, p.T, tile.begin + t) * p.R + r) = val;
        return val;
      },
      none ? 0.0f : p.scales[tile.l], tile.count, p.R, parts, exponent);
  __syncthreads();
  if (none && in_place) return;
  for (; n0 + OUT <= n1; n0 += STEP) {
    stage_b();
    if (n0 + STEP + OUT <= n1) {
      load_y(ahead, n0 + STEP);
      load_b(n0 + STEP);
    }
#pragma unroll
    for (int j = 0; j < TB; j++) {
      if (j * 16 >= tile.count) break;
      finish(j, n0, had + j * ROUNDS, at + j * ROUNDS, std::true_type(), 8);
    }
#pragma unroll
    for (int q = 0; q < TILE / ROWS; q++) had[q] = ahead[q];
  }
  if (n0 < n1) {  // the last outputs, fewer than a step's
    const int left = n1 - n0 - chunk * 8, most = (n1 - n0) * per_row - 1;
#pragma unroll
    for (int q = 0; q < LOADS; q++)  // beyond the last row: for outputs that nobody stores
      if (q * 64 < per_row * OUT)
        vb[q] = *reinterpret_cast<const us8_t*>(b + (int64_t)n0 * p.R + min(item(q), most) * 8);
    stage_b();
#pragma unroll 1
    for (int j = 0; j * 16 < tile.count; j++) {
      int64_t at2[ROUNDS];
      us8_t y2[ROUNDS];
#pragma unroll
      for (int q = 0; q < ROUNDS; q++) {
        const int t = min(j * 16 + q * ROWS + row, tile.count - 1);
        at2[q] = token_at(p.order, p.T, tile.begin + t) * N + chunk * 8;
        y2[q] = load8(y + at2[q] + n0, left);
      }
      finish(j, n0, y2, at2, std::false_type(), left);
    }
  }
}

template <bool BF, int RB, int TB>
hipError_t run(const DownArgs& down, const UpArgs& up, const LoraDivision& d, hipStream_t stream) {
  // The contraction in eight waves where few ranks and tokens leave each little to load (us of both
  // kernels with four / eight: 64 tokens of 64 adapters of 11008x4096, 16 ranks 14.8 / 14.3; 64 of
  // 4096x12288, 32 ranks 11.5 / 11.0; one token 7.5 / 7.6; 64 of 8 adapters, 64 ranks 11.3 / 11.4).
  constexpr int DOWN = RB < 4 ? RB : 4, W = TB == 1 && RB <= 2 ? 8 : 4;
  const hipError_t e = launch_lds(lora_down_kernel<BF, DOWN, TB, W>,
                                  dim3((unsigned)d.tiles, d.splits, (down.p.R + 63) / 64), W * 64,
                                  down_bytes<DOWN, TB, W>(), stream, down);
  if (e != hipSuccess) return e;
  return launch_lds(lora_up_kernel<BF, RB, TB>, dim3((unsigned)d.tiles, d.ranges), kLoraWaves * 64,
                    up_bytes<RB, TB>(), stream, up);
}
template <bool BF, int RB>
hipError_t run(const DownArgs& down, const UpArgs& up, const LoraDivision& d, hipStream_t stream) {
  return d.tile == 16 ? run<BF, RB, 1>(down, up, d, stream) : run<BF, RB, 4>(down, up, d, stream);
}
template <bool BF>
hipError_t run(const DownArgs& down, const UpArgs& up, const LoraDivision& d, hipStream_t stream) {
  const int blocks = (down.p.R + 15) / 16;
  if (blocks <= 1) return run<BF, 1>(down, up, d, stream);
  if (blocks <= 2) return run<BF, 2>(down, up, d, stream);
  if (blocks <= 4) return run<BF, 4>(down, up, d, stream);
  return run<BF, 8>(down, up, d, stream);
}

}  // namespace

size_t lora_workspace_bytes(const LoraSizes& s) {
  if (s.T == 0) return 0;
  return (size_t)divide_lora(s).splits * s.T * s.R * sizeof(float);
}

hipError_t launch_lora(const void* x, int dtype, const LoraArgs& p, const void* y, void* out,
                       float* v, void* workspace, hipStream_t stream) {
  const LoraDivision d = divide_lora({p.T, p.N, p.K, p.R, p.L});
  float* const shares = static_cast<float*>(workspace);
  const DownArgs down = {p, static_cast<const uint16_t*>(x), shares, d.k_share};
  const UpArgs up = {p,           shares, d.splits, d.n_share, static_cast<const uint16_t*>(y),
                     static_cast<uint16_t*>(out), v};
  return dtype == kBF16 ? run<true>(down, up, d, stream) : run<false>(down, up, d, stream);
}

}  // namespace lowbit
