// lora_grad.hip -- the gradients of out = y + s_l b_l (a_l x):
//
//   u_t = b_l^T dy_t,  dx_t = base_t + s_l a_l^T u_t,
//   da_l = s_l sum_t u_t x_t^T,  db_l = s_l sum_t dy_t v_t^T.
//
// Three launches: u; then dx, da and db side by side; then the join of da's and db's
// shares where an adapter has more than one chunk of tokens.  Bound by HBM: dy is read
// twice, x and base once, dx is written, 2 T (2 N + 3 K) bytes.
//
// The sums over tokens need, for a lane's operand, eight tokens' elements of one
// column, where rows lie along the columns.  A lane loads eight rows' 16 bytes at
// eight columns and pairs them up with byte permutes: an 8 x 8 transpose in its own
// registers, 32 permutes for 8 products, and x and dy never pass through LDS.
#include "lora.h"

namespace lowbit {
namespace {

constexpr int kGradWaves = 4;
constexpr int kTile = 64;   // tokens of u's and dx's tiles
constexpr int kCols = kGradWaves * 128;  // columns of a workgroup of dx, da or db

// ---------------------------------------------------------------------------
// u = b^T dy
// ---------------------------------------------------------------------------
struct BackArgs {
  LoraArgs p;
  const uint16_t* dy;
  float* shares;  // [splits][T][R], rows in the plan's order
  int n_share;    // a multiple of 256
};

// A wave's step is 64 outputs: it turns b's 64 rows of RB * 16 ranks around in LDS
// (rows of b hold the ranks of one output, an operand needs eight outputs of one rank).
template <bool BF, int RB>
__global__ __launch_bounds__(kGradWaves * 64) void lora_back_kernel(const BackArgs g) {
  constexpr int TB = kTile / 16, PITCH = RB * 16 + 4, TURN = 64 + 8;
  constexpr int kTurned = kGradWaves * RB * 16 * TURN * 2;
  constexpr int kReduced = kGradWaves / 2 * kTile * PITCH * 4;
  __shared__ __align__(16) char lds[kTurned > kReduced ? kTurned : kReduced];
  const LoraArgs& p = g.p;
  LoraTile tile;
  if (!find_tile(p.starts, p.L, (int)p.T, kTile, blockIdx.x, tile) || tile.l == p.L) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i16 = lane & 15, h = lane >> 4;
  const int r0 = blockIdx.z * 64, ranks = min(p.R - r0, RB * 16);
  uint16_t(*turn)[TURN] = reinterpret_cast<uint16_t(*)[TURN]>(lds + wave * RB * 16 * TURN * 2);
  const int blocks = (tile.count + 15) / 16;
  const uint16_t* dr[TB];
#pragma unroll
  for (int j = 0; j < TB; j++)
    dr[j] = g.dy +
            token_at(p.order, p.T, tile.begin + min(j * 16 + i16, tile.count - 1)) * p.N;
  f4_t acc[RB][TB];
#pragma unroll
  for (int i = 0; i < RB; i++)
#pragma unroll
    for (int j = 0; j < TB; j++) acc[i][j] = f4_t{0, 0, 0, 0};
  const int n1 = min((int)(blockIdx.y + 1) * g.n_share, p.N);
  for (int base = blockIdx.y * g.n_share; base < n1; base += kGradWaves * 64) {
    const int n0 = base + wave * 64;
    // two outputs' eight ranks to a lane, written as pairs
    const int pair = lane & 31;
    const uint16_t* br = p.b + ((int64_t)tile.l * p.N + n0 + pair * 2) * p.R + r0;
#pragma unroll
    for (int q = 0; q < RB; q++) {
      const int r = (q * 2 + (lane >> 5)) * 8;
      us8_t lo = {}, hi = {};
      if (r < ranks && n0 + pair * 2 < n1) lo = *reinterpret_cast<const us8_t*>(br + r);
      if (r < ranks && n0 + pair * 2 + 1 < n1) hi = *reinterpret_cast<const us8_t*>(br + p.R + r);
#pragma unroll
      for (int i = 0; i < 8; i++)
        *reinterpret_cast<uint32_t*>(&turn[r + i][pair * 2]) = lo[i] | (uint32_t)hi[i] << 16;
    }
    __syncthreads();
#pragma unroll
    for (int half = 0; half < 2; half++) {
      const int at = half * 32 + h * 8;
      us8_t fb[RB];
#pragma unroll
      for (int i = 0; i < RB; i++)
        fb[i] = *reinterpret_cast<const us8_t*>(&turn[i * 16 + i16][at]);
#pragma unroll
      for (int j = 0; j < TB; j++) {
        if (j >= blocks) break;
        const us8_t fd = load8(dr[j] + n0 + at, n1 - n0 - at);
#pragma unroll
        for (int i = 0; i < RB; i++) acc[i][j] = Half16<BF>::mma(fb[i], fd, acc[i][j]);
      }
    }
    __syncthreads();
  }
  float(*red)[kTile][PITCH] = reinterpret_cast<float(*)[kTile][PITCH]>(lds);
#pragma unroll
  for (int left = kGradWaves / 2; left > 0; left >>= 1) {
    if (wave >= left && wave < 2 * left)
#pragma unroll
      for (int i = 0; i < RB; i++)
#pragma unroll
        for (int j = 0; j < TB; j++)
          *reinterpret_cast<f4_t*>(&red[wave - left][j * 16 + i16][i * 16 + h * 4]) = acc[i][j];
    __syncthreads();
    if (wave < left)
#pragma unroll
      for (int i = 0; i < RB; i++)
#pragma unroll
        for (int j = 0; j < TB; j++)
          acc[i][j] += *reinterpret_cast<const f4_t*>(&red[wave][j * 16 + i16][i * 16 + h * 4]);
    __syncthreads();
  }
  if (wave > 0) return;
  float* out = g.shares + ((int64_t)blockIdx.y * p.T + tile.begin) * p.R + r0;
#pragma unroll
  for (int i = 0; i < RB; i++)
#pragma unroll
    for (int j = 0; j < TB; j++)
      if (j * 16 + i16 < tile.count && i * 16 + h * 4 < ranks)
        *reinterpret_cast<f4_t*>(out + (j * 16 + i16) * p.R + i * 16 + h * 4) = acc[i][j];
}

// ---------------------------------------------------------------------------
// dx, da, db
// ---------------------------------------------------------------------------
struct SpreadArgs {
  LoraArgs p;
  const uint16_t *dy, *x, *base;
  const float *v, *shares;  // shares of u
  int splits;
  uint16_t* dx;
  float *da, *db;
  float *part_a, *part_b;  // [share][R][K], [share][N][R] of adapters with several chunks
  int chunk;               // tokens
  int64_t tiles, chunks;   // bounds
  int k_cols, n_cols;      // workgroups along K and N
};

// Eight rows' eight elements each, rows[i] for row i, turned around: cols[j] holds
// element j of the eight rows.
__device__ __forceinline__ void transpose8(const us8_t (&rows)[8], us8_t (&cols)[8]) {
  typedef uint32_t u4_t __attribute__((ext_vector_type(4)));
  u4_t in[8], out[8];
#pragma unroll
  for (int i = 0; i < 8; i++) in[i] = __builtin_bit_cast(u4_t, rows[i]);
#pragma unroll
  for (int j = 0; j < 8; j++)
#pragma unroll
    for (int i = 0; i < 4; i++)
      out[j][i] = __builtin_amdgcn_perm(in[2 * i + 1][j / 2], in[2 * i][j / 2],
                                        j % 2 ? 0x07060302u : 0x05040100u);
#pragma unroll
  for (int j = 0; j < 8; j++) cols[j] = __builtin_bit_cast(us8_t, out[j]);
}

// dx of one tile and 512 columns, 128 to a wave.  As in the forward pass a product's
// 32 terms are 16 ranks against the upper and lower part of s u.
template <bool BF, int RB>
__device__ __forceinline__ void dx_part(const SpreadArgs& g, int index, int col, char* lds) {
  constexpr int PITCH = RB * 32 + 8, TB = kTile / 16;
  constexpr int kPerToken = kGradWaves * 64 / kTile;
  uint16_t(*parts)[PITCH] = reinterpret_cast<uint16_t(*)[PITCH]>(lds);
  int* exponent = reinterpret_cast<int*>(lds + kTile * PITCH * 2);
  const LoraArgs& p = g.p;
  LoraTile tile;
  if (!find_tile(p.starts, p.L, (int)p.T, kTile, index, tile)) return;
  const bool none = tile.l == p.L;
  if (none && g.base == g.dx) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i16 = lane & 15, h = lane >> 4;
  {
    const int t = threadIdx.x / kPerToken, s = threadIdx.x % kPerToken;
    const float scale = none ? 0.0f : p.scales[tile.l];
    f4_t val[RB];
    int top = 0;
#pragma unroll
    for (int i = 0; i < RB; i++) {
      const int r = (s + i * kPerToken) * 4;
      val[i] = f4_t{0, 0, 0, 0};
      if (r >= p.R || t >= tile.count || none) continue;
      for (int w = 0; w < g.splits; w++)
        val[i] += *reinterpret_cast<const f4_t*>(
            g.shares + ((int64_t)w * p.T + tile.begin + t) * p.R + r);
      val[i] *= scale;
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
    for (int i = 0; i < RB; i++) {
      const int r = (s + i * kPerToken) * 4;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        uint16_t part[2];
        split_parts<BF>(BF ? val[i][j] : times_power(val[i][j], e), part);
        const int at = r / 16 * 32 + r % 16 + j;
        parts[t][at] = part[0];
        parts[t][at + 16] = part[1];
      }
    }
  }
  __syncthreads();
  const int64_t K = p.K;
  const int k0 = col * kCols + wave * 128;
  if (k0 >= p.K) return;
  // lane i16 = 4 a + b loads columns 8 (4 b + a) on: its results are then pieces of eight
  // columns that lie side by side for the four lanes of a token
  const int mine = k0 + (i16 % 4 * 4 + i16 / 4) * 8;
  us8_t fa[RB][8];
#pragma unroll
  for (int c = 0; c < RB; c++) {
    us8_t rows[8];
    const int r = c * 16 + (h & 1) * 8;
#pragma unroll
    for (int i = 0; i < 8; i++) {
      rows[i] = us8_t{};
      if (!none && r < p.R && mine < p.K)
        rows[i] = *reinterpret_cast<const us8_t*>(p.a + ((int64_t)tile.l * p.R + r + i) * K + mine);
    }
    transpose8(rows, fa[c]);
  }
  for (int j = 0; j < TB; j++) {
    const int t = j * 16 + i16;
    if (j * 16 >= tile.count) break;
    us8_t fu[RB];
#pragma unroll
    for (int c = 0; c < RB; c++)
      fu[c] = *reinterpret_cast<const us8_t*>(&parts[t][c * 32 + h * 8]);
    f4_t acc[8];
#pragma unroll
    for (int m = 0; m < 8; m++) {
      acc[m] = f4_t{0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < RB; c++) acc[m] = Half16<BF>::mma(fa[c][m], fu[c], acc[m]);
    }
    if (t >= tile.count) continue;
    const int64_t row = token_at(p.order, p.T, tile.begin + t) * K;
    const int e = exponent[t];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      // result row 4 h + i is lane 4 h + i's columns
      const int k = k0 + (i * 4 + h) * 8;
      if (k >= p.K) continue;
      us8_t had = {};
      if (g.base) had = *reinterpret_cast<const us8_t*>(g.base + row + k);
      us8_t o;
#pragma unroll
      for (int m = 0; m < 8; m++) {
        float f = acc[m][i];
        if (!BF) f = times_power(f, -e);
        if (g.base) f += Half16<BF>::to(had[m]);
        o[m] = Half16<BF>::from(f);
      }
      *reinterpret_cast<us8_t*>(g.dx + row + k) = none ? had : o;
    }
  }
}

// The first of an adapter's shares where it has several chunks, its tokens beginning at
// `first`: n >= 2 chunks of more than n - 1 whole ones are at most twice their whole
// ones, so adapters' shares never overlap, and there are 2 T / chunk + 1 in all.
__device__ __forceinline__ int64_t share_of(int first, int chunk) { return 2 * (int64_t)first / chunk; }

// da (ROWS_X: sums of u_t x_t) or db (v_t dy_t) of one chunk of tokens, 64 ranks from
// r0 on and 512 columns, 128 to a wave.  64 tokens at a time pass through LDS as parts
// of u or v, turned around so that an operand's eight tokens lie side by side; their
// rows of x or dy go straight to the registers.  fp16: the parts stand for values times
// 2^e, e by the largest value so far; the sums follow when it changes.
template <bool BF, int RB, bool ROWS_X>
__device__ __forceinline__ void sum_part(const SpreadArgs& g, int index, int col, int r0,
                                         char* lds) {
  constexpr int PARTS = BF ? 3 : 2, TURN = kTile + 8;
  constexpr int kPerToken = kGradWaves * 64 / kTile;
  typedef uint16_t Turned[RB * 16][TURN];
  Turned* const turned = reinterpret_cast<Turned*>(lds);
  int* const places = reinterpret_cast<int*>(lds + PARTS * sizeof(Turned));  // tokens
  int* const tops = places + kTile;
  const LoraArgs& p = g.p;
  LoraTile tile;
  if (!find_tile(p.starts, p.L, (int)p.T, g.chunk, index, tile) || tile.l == p.L) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i16 = lane & 15, h = lane >> 4;
  const int64_t C = ROWS_X ? p.K : p.N;
  const uint16_t* const rows_of = ROWS_X ? g.x : g.dy;
  const int ranks = min(p.R - r0, RB * 16);
  const int c0 = col * kCols + wave * 128 + i16 * 8;  // this lane's eight columns
  f4_t acc[RB][8];
#pragma unroll
  for (int i = 0; i < RB; i++)
#pragma unroll
    for (int m = 0; m < 8; m++) acc[i][m] = f4_t{0, 0, 0, 0};
  int e = 0;
  bool any = false;  // whether e was chosen
  for (int t0 = 0; t0 < tile.count; t0 += kTile) {
    const int t = threadIdx.x / kPerToken, s = threadIdx.x % kPerToken;
    const bool has = t0 + t < tile.count;
    const int64_t token = has ? token_at(p.order, p.T, tile.begin + t0 + t) : 0;
    f4_t val[RB];
    int top = 0;
#pragma unroll
    for (int i = 0; i < RB; i++) {
      const int r = (s + i * kPerToken) * 4;
      val[i] = f4_t{0, 0, 0, 0};
      if (!has || r >= ranks) continue;
      if (ROWS_X) {
        for (int w = 0; w < g.splits; w++)
          val[i] += *reinterpret_cast<const f4_t*>(
              g.shares + ((int64_t)w * p.T + tile.begin + t0 + t) * p.R + r0 + r);
      } else {
        val[i] = *reinterpret_cast<const f4_t*>(g.v + token * p.R + r0 + r);
      }
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const int bits = __builtin_bit_cast(int, (float)val[i][j]) & 0x7fffffff;
        if (bits < 0x7f800000) top = max(top, bits);
      }
    }
    if (!BF) {
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) top = max(top, __shfl_xor(top, off, kWave));
      if (lane == 0) tops[wave] = top;
    }
    __syncthreads();  // the tile before has been read; the tops are there
    if (!BF) {
#pragma unroll
      for (int w = 0; w < kGradWaves; w++) top = max(top, tops[w]);
      const int next = fp16_exponent(top);
      if (top != 0 && (!any || next < e)) {
        const int by = any ? next - e : 0;
        e = next;
        any = true;
        if (by != 0)
#pragma unroll
          for (int i = 0; i < RB; i++)
#pragma unroll
            for (int m = 0; m < 8; m++)
#pragma unroll
              for (int j = 0; j < 4; j++) acc[i][m][j] = times_power(acc[i][m][j], by);
      }
    }
    if (s == 0) places[t] = (int)token;
#pragma unroll
    for (int i = 0; i < RB; i++) {
      const int r = (s + i * kPerToken) * 4;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        uint16_t part[PARTS];
        split_parts<BF>(BF ? val[i][j] : times_power(val[i][j], e), part);
#pragma unroll
        for (int q = 0; q < PARTS; q++) turned[q][r + j][t] = part[q];
      }
    }
    __syncthreads();
    if (c0 - i16 * 8 < C) {
#pragma unroll
      for (int half = 0; half < kTile / 32; half++) {
        const int at = half * 32 + h * 8;
        if (t0 + half * 32 >= tile.count) break;
        us8_t rows[8], cols[8];
#pragma unroll
        for (int i = 0; i < 8; i++) {
          rows[i] = us8_t{};
          if (t0 + at + i < tile.count) {
            const uint16_t* from = rows_of + places[at + i] * C + c0;
            if (ROWS_X) {
              if (c0 < C) rows[i] = *reinterpret_cast<const us8_t*>(from);
            } else {
              rows[i] = load8(from, C - c0);
            }
          }
        }
        transpose8(rows, cols);
#pragma unroll
        for (int i = 0; i < RB; i++)
#pragma unroll
          for (int q = 0; q < PARTS; q++) {
            const us8_t fu = *reinterpret_cast<const us8_t*>(&turned[q][i * 16 + i16][at]);
#pragma unroll
            for (int m = 0; m < 8; m++) acc[i][m] = Half16<BF>::mma(fu, cols[m], acc[i][m]);
          }
      }
    }
    __syncthreads();
  }
  const float scale = p.scales[tile.l];
  const int64_t size = (int64_t)p.R * C;
  // an adapter's only chunk is its whole sum
  const int64_t share = share_of(tile.first, g.chunk) + (tile.begin - tile.first) / g.chunk;
  float* out = tile.tiles == 1 ? (ROWS_X ? g.da : g.db) + tile.l * size
                               : (ROWS_X ? g.part_a : g.part_b) + share * size;
#pragma unroll
  for (int i = 0; i < RB; i++) {
    const int r = i * 16 + h * 4;
    if (r >= ranks) continue;
    float f[8][4];
#pragma unroll
    for (int m = 0; m < 8; m++)
#pragma unroll
      for (int j = 0; j < 4; j++) {
        f[m][j] = acc[i][m][j];
        if (!BF) f[m][j] = times_power(f[m][j], -e);
        f[m][j] *= scale;
      }
    if (ROWS_X) {
      if (c0 < C)
#pragma unroll
        for (int j = 0; j < 4; j++) {
          float* at = out + (r0 + r + j) * C + c0;
          *reinterpret_cast<f4_t*>(at) = f4_t{f[0][j], f[1][j], f[2][j], f[3][j]};
          *reinterpret_cast<f4_t*>(at + 4) = f4_t{f[4][j], f[5][j], f[6][j], f[7][j]};
        }
    } else {
#pragma unroll
      for (int m = 0; m < 8; m++)
        if (c0 + m < C)
          *reinterpret_cast<f4_t*>(out + (c0 + m) * p.R + r0 + r) =
              f4_t{f[m][0], f[m][1], f[m][2], f[m][3]};
    }
  }
}

template <bool BF, int RB>
__global__ __launch_bounds__(kGradWaves * 64) void lora_spread_kernel(const SpreadArgs g) {
  constexpr int RS = RB < 4 ? RB : 4;  // ranks of the sums, in blocks
  constexpr int kDx = kTile * (RB * 32 + 8) * 2 + kTile * 4;
  constexpr int kSum = (BF ? 3 : 2) * RS * 16 * (kTile + 8) * 2 + kTile * 4 + kGradWaves * 4;
  __shared__ __align__(16) char lds[kDx > kSum ? kDx : kSum];
  int64_t at = blockIdx.x;
  const int groups = (g.p.R + 63) / 64;
  const int64_t sums_a = g.chunks * g.k_cols * groups, sums_b = g.chunks * g.n_cols * groups;
  if (at < sums_a) {
    const int cg = g.k_cols * groups;
    sum_part<BF, RS, true>(g, (int)(at / cg), (int)(at % cg / groups), (int)(at % groups) * 64, lds);
    return;
  }
  at -= sums_a;
  if (at < sums_b) {
    const int cg = g.n_cols * groups;
    sum_part<BF, RS, false>(g, (int)(at / cg), (int)(at % cg / groups), (int)(at % groups) * 64, lds);
    return;
  }
  at -= sums_b;
  dx_part<BF, RB>(g, (int)(at / g.k_cols), (int)(at % g.k_cols), lds);
}

// ---------------------------------------------------------------------------
// the join: da and db of adapters with several chunks, or none
// ---------------------------------------------------------------------------
struct JoinArgs {
  const int32_t* starts;
  int T, L, chunk;
  int64_t size_a, size_b;
  const float *part_a, *part_b;
  float *da, *db;
};
__global__ __launch_bounds__(256) void lora_join_kernel(const JoinArgs g) {
  const int l = blockIdx.y;
  int s0 = 0, s1 = 0;
  if (g.T > 0) {
    s0 = min(max(g.starts[l], 0), g.T);
    s1 = min(max(g.starts[l + 1], s0), g.T);
  }
  const int mine = (s1 - s0 + g.chunk - 1) / g.chunk;
  if (mine == 1) return;
  const int64_t before = share_of(s0, g.chunk);
  int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  const float* part = g.part_a;
  float* out = g.da;
  int64_t size = g.size_a;
  if (at >= size) {
    at -= size;
    part = g.part_b;
    out = g.db;
    size = g.size_b;
    if (at >= size) return;
  }
  f4_t sum = {0, 0, 0, 0};
  for (int c = 0; c < mine; c++)
    sum += *reinterpret_cast<const f4_t*>(part + (before + c) * size + at);
  *reinterpret_cast<f4_t*>(out + l * size + at) = sum;
}

// How a call is divided: shares of N for u, tokens of a chunk of the sums.
struct Division {
  int64_t tiles;
  int splits, n_share;
  int chunk;
  int64_t chunks, shares;
  int k_cols, n_cols;
};
Division divide(const LoraSizes& s) {
  Division d;
  d.tiles = lora_tiles(s.T, s.L, kTile);
  const int64_t most = (s.N + 255) / 256;
  int64_t n = (512 + d.tiles - 1) / d.tiles;
  if (n > most) n = most;
  d.n_share = (int)(((s.N + n - 1) / n + 255) / 256 * 256);
  d.splits = (int)((s.N + d.n_share - 1) / d.n_share);
  d.k_cols = (int)((s.K + kCols - 1) / kCols);
  d.n_cols = (int)((s.N + kCols - 1) / kCols);
  // chunks enough for 512 workgroups, of 256 tokens at least
  const int64_t cols = (d.k_cols + d.n_cols) * ((s.R + 63) / 64);
  const int64_t wanted = (512 + cols - 1) / cols;
  int64_t chunk = ((s.T + wanted - 1) / wanted + kTile - 1) / kTile * kTile;
  if (chunk < 256) chunk = 256;
  d.chunk = (int)chunk;
  d.chunks = lora_tiles(s.T, s.L, d.chunk);
  d.shares = s.T > d.chunk ? 2 * s.T / d.chunk + 1 : 0;
  return d;
}
// floats of u's shares, rounded up to 16 bytes, and of da's and db's
int64_t u_floats(const LoraSizes& s, const Division& d) { return d.splits * s.T * s.R; }

template <bool BF, int RB>
hipError_t run(const BackArgs& back, const SpreadArgs& spread, const Division& d,
               hipStream_t stream) {
  constexpr int RU = RB < 4 ? RB : 4;
  const int groups = (back.p.R + 63) / 64;
  lora_back_kernel<BF, RU><<<dim3((unsigned)d.tiles, d.splits, groups), kGradWaves * 64, 0, stream>>>(back);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t grid =
      d.chunks * (d.k_cols + d.n_cols) * groups + d.tiles * d.k_cols;
  lora_spread_kernel<BF, RB><<<(unsigned)grid, kGradWaves * 64, 0, stream>>>(spread);
  return hipGetLastError();
}
template <bool BF>
hipError_t run(const BackArgs& back, const SpreadArgs& spread, const Division& d,
               hipStream_t stream) {
  const int blocks = (back.p.R + 15) / 16;
  if (blocks <= 1) return run<BF, 1>(back, spread, d, stream);
  if (blocks <= 2) return run<BF, 2>(back, spread, d, stream);
  if (blocks <= 4) return run<BF, 4>(back, spread, d, stream);
  return run<BF, 8>(back, spread, d, stream);
}

}  // namespace

size_t lora_grad_workspace_bytes(const LoraSizes& s) {
  if (s.T == 0) return 0;
  const Division d = divide(s);
  const int64_t parts = d.shares * s.R * (s.K + s.N);
  return (size_t)(u_floats(s, d) + parts) * sizeof(float);
}

hipError_t launch_lora_grad(const void* dy, const void* x, const float* v, int dtype,
                            const LoraArgs& p, const void* base, void* dx, float* da, float* db,
                            void* workspace, hipStream_t stream) {
  const LoraSizes s = {p.T, p.N, p.K, p.R, p.L};
  const Division d = s.T > 0 ? divide(s) : Division{};
  float* const shares = static_cast<float*>(workspace);
  float* const part_a = shares + u_floats(s, d);
  float* const part_b = part_a + d.shares * s.R * s.K;
  const auto* dyp = static_cast<const uint16_t*>(dy);
  const BackArgs back = {p, dyp, shares, d.n_share};
  const SpreadArgs spread = {p,        dyp,     static_cast<const uint16_t*>(x),
                             static_cast<const uint16_t*>(base),
                             v,        shares,  d.splits,
                             static_cast<uint16_t*>(dx),
                             da,       db,      part_a,
                             part_b,   d.chunk, d.tiles,
                             d.chunks, d.k_cols, d.n_cols};
  if (s.T > 0) {
    const hipError_t e = dtype == kBF16 ? run<true>(back, spread, d, stream)
                                        : run<false>(back, spread, d, stream);
    if (e != hipSuccess) return e;
  }
  const JoinArgs join = {p.starts, (int)p.T, p.L, s.T > 0 ? d.chunk : 1, s.R * s.K, s.R * s.N,
                         part_a,   part_b,   da,  db};
  const int64_t quads = (s.R * (s.K + s.N)) / 4;
  lora_join_kernel<<<dim3((unsigned)((quads + 255) / 256), (unsigned)s.L), 256, 0, stream>>>(join);
  return hipGetLastError();
}

}  // namespace lowbit
