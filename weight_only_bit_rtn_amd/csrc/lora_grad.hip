// lora_grad.hip -- the gradients of out = y + s_l b_l (a_l x):
//
//   u_t = b_l^T dy_t,  dx_t = base_t + s_l a_l^T u_t,
//   da_l = s_l sum_t u_t x_t^T,  db_l = s_l sum_t dy_t v_t^T.
//
// Three launches: u; then da and db; then dx, and beside it the join of da's and db's
// shares where an adapter has more than one chunk of tokens.  Bound by HBM: dy is read
// twice, x and base once, dx is written, 2 T (2 N + 3 K) bytes.  8192 tokens of 12288x12288,
// 64 ranks: 75 + 114 + 85 us (200, 400 and 400 MB: 2.7, 3.5 and 4.7 TB/s); 16 ranks 59 + 71 + 68, 3.4, 5.7
// and 5.9 TB/s.
// With 64 ranks the sums are held up by the products (27% of the matrix cores' time) and the
// parts' making between barriers: without the latter they take 8 us less, without two of
// three parts 3 less.
//
// The sums over tokens need, for a lane's operand, eight tokens' elements of one
// column, where rows lie along the columns.  A lane loads eight rows' 16 bytes at
// eight columns and pairs them up with byte permutes: an 8 x 8 transpose in its own
// registers, 32 permutes for 8 products, and the rows never pass through LDS.
#include "lora.h"

namespace lowbit {
namespace {

// ---------------------------------------------------------------------------
// u = b^T dy
// ---------------------------------------------------------------------------
struct BackArgs {
  LoraArgs p;
  const uint16_t* dy;
  float* shares;  // [splits][T][R], rows in the plan's order
  int n_share;    // a multiple of 64
};

// A wave's step is 64 outputs: 64 tokens' rows of dy, and b's 64 rows of RB * 16 ranks, which
// lie in one piece and are turned around on their way into LDS (rows of b hold the ranks of
// one output, an operand needs eight outputs of one rank): a lane takes eight ranks of two
// outputs and writes pairs.  The next step's are under way while one is multiplied.
template <int RB>
constexpr int back_bytes() {
  constexpr int TB = kTile / 16;
  constexpr int stage = kBackWaves * (kTile * 128 + RB * 16 * 144);
  constexpr int reduce = reduce_bytes<RB, TB, kBackWaves>();
  return stage > reduce ? stage : reduce;
}
template <bool BF, int RB>
__global__ __launch_bounds__(kBackWaves * 64) void lora_back_kernel(const BackArgs g) {
  constexpr int TB = kTile / 16, TURN = 64 + 8, RANKS = RB * 16;
  extern __shared__ __align__(16) char lds[];
  const LoraArgs& p = g.p;
  LoraTile tile;
  if (!find_tile(p.starts, p.L, (int)p.T, kTile, blockIdx.x, tile) || tile.l == p.L) return;
  const int lane = threadIdx.x & 63, wave = wave_of_group();
  const int i16 = lane & 15, h = lane >> 4, row = lane >> 3, chunk = lane & 7;
  const int r0 = blockIdx.z * 64, ranks = min(p.R - r0, RANKS);
  uint16_t* const sd = reinterpret_cast<uint16_t*>(lds + wave * (kTile * 128 + RANKS * 144));
  uint16_t(*const turn)[TURN] = reinterpret_cast<uint16_t(*)[TURN]>(sd + kTile * 64);
  const uint16_t* dr[kTile / 8];
#pragma unroll
  for (int q = 0; q < kTile / 8; q++)
    dr[q] = g.dy + chunk * 8 +
            token_at(p.order, p.T, tile.begin + min(q * 8 + row, tile.count - 1)) * p.N;
  // item 64 q + lane of a step: eight ranks from 8 (item % RB2) on, outputs 2 (item / RB2) and
  // the next.  The slots of a row's 16-byte chunks are dealt by its eight ranks, so that the
  // lanes' writes take different banks.
  constexpr int RB2 = RB * 2, ITEMS = 32 * RB2 / 64;
  const uint16_t* br[ITEMS];
  int place[ITEMS];
#pragma unroll
  for (int q = 0; q < ITEMS; q++) {
    const int item = q * 64 + lane, oct = item % RB2, pair = item / RB2;
    // beyond the last rank: read within the row, and turned into rows of no one's results
    br[q] = p.b + ((int64_t)tile.l * p.N + pair * 2) * p.R + r0 + min(oct * 8, ranks - 8);
    place[q] = oct * 8 * TURN + ((((pair >> 2) ^ oct) & 7) << 3) + (pair & 3) * 2;
  }
  f4_t acc[RB][TB];
#pragma unroll
  for (int i = 0; i < RB; i++)
#pragma unroll
    for (int j = 0; j < TB; j++) acc[i][j] = f4_t{0, 0, 0, 0};
  us8_t vd[kTile / 8], vb[ITEMS][2];
  auto load = [&](int n) {
#pragma unroll
    for (int q = 0; q < kTile / 8; q++) vd[q] = load8(dr[q] + n);
#pragma unroll
    for (int q = 0; q < ITEMS; q++) {
      vb[q][0] = *reinterpret_cast<const us8_t*>(br[q] + (int64_t)n * p.R);
      vb[q][1] = *reinterpret_cast<const us8_t*>(br[q] + (int64_t)n * p.R + p.R);
    }
  };
  auto stage = [&] {
    put_rows<kTile>(sd, vd);
#pragma unroll
    for (int q = 0; q < ITEMS; q++)
#pragma unroll
      for (int i = 0; i < 8; i++)
        *reinterpret_cast<uint32_t*>(&turn[0][0] + place[q] + i * TURN) =
            vb[q][0][i] | (uint32_t)vb[q][1][i] << 16;
    wave_lds_order();
  };
  auto multiply = [&] {
#pragma unroll
    for (int half = 0; half < 2; half++) {
      us8_t fb[RB];
#pragma unroll
      for (int i = 0; i < RB; i++)
        fb[i] = *reinterpret_cast<const us8_t*>(
            &turn[i * 16 + i16][((half * 4 + h) ^ ((i * 2 + (i16 >> 3)) & 7)) << 3]);
#pragma unroll
      for (int j = 0; j < TB; j++) {
        const us8_t fd = get_operand(sd, j, half);
#pragma unroll
        for (int i = 0; i < RB; i++) acc[i][j] = Half16<BF>::mma(fb[i], fd, acc[i][j]);
      }
    }
    wave_lds_order();
  };
  const int n0 = blockIdx.y * g.n_share, n1 = min(n0 + g.n_share, p.N);
  constexpr int STEP = kBackWaves * 64;
  int n = n0 + wave * 64;
  if (n + 64 <= n1) {
    load(n);
    for (; n + STEP + 64 <= n1; n += STEP) {
      stage();
      load(n + STEP);
      multiply();
    }
    stage();
    multiply();
    n += STEP;
  }
  if (n < n1) {  // the last outputs, fewer than 64
    const int left = n1 - n;
#pragma unroll
    for (int q = 0; q < kTile / 8; q++) vd[q] = load8(dr[q] + n, left - chunk * 8);
#pragma unroll
    for (int q = 0; q < ITEMS; q++) {
      const int pair = (q * 64 + lane) / RB2;
#pragma unroll
      for (int i = 0; i < 2; i++)
        vb[q][i] = pair * 2 + i < left
                       ? *reinterpret_cast<const us8_t*>(br[q] + ((int64_t)n + i) * p.R)
                       : us8_t{};
    }
    stage();
    multiply();
  }
  reduce_waves<RB, TB, kBackWaves>(acc, wave, lds);
  if (wave == 0)
    store_shares(acc, g.shares + ((int64_t)blockIdx.y * p.T + tile.begin) * p.R + r0, p.R,
                 tile.count, ranks);
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
  int dx_cols;             // columns of one of dx, in units of kCols
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

// dx of one tile and `cols` times 512 columns, 128 to a wave, with s u in two parts as s v in the
// forward pass.  Results pass through LDS as there: sixteen lanes then hold the 128
// columns of one token.
template <int RB>
constexpr int dx_bytes() {
  return kTile * ((RB * 32 + 8) * 2 + 4) + kGradWaves * 16 * 132 * 4;
}
template <bool BF, int RB>
__device__ __forceinline__ void dx_part(const SpreadArgs& g, int index, int col, int cols,
                                        char* lds) {
  constexpr int PITCH = RB * 32 + 8, TB = kTile / 16, C = Ranks<RB>::kChunks;
  uint16_t(*const parts)[PITCH] = reinterpret_cast<uint16_t(*)[PITCH]>(lds);
  int* const exponent = reinterpret_cast<int*>(lds + kTile * PITCH * 2);
  const LoraArgs& p = g.p;
  LoraTile tile;
  if (!find_tile(p.starts, p.L, (int)p.T, kTile, index, tile)) return;
  const bool none = tile.l == p.L;
  if (none && g.base == g.dx) return;
  const int lane = threadIdx.x & 63, wave = wave_of_group();
  const int i16 = lane & 15, h = lane >> 4;
  float(*const result)[132] =
      reinterpret_cast<float(*)[132]>(lds + kTile * (PITCH * 2 + 4) + wave * 16 * 132 * 4);
  const int64_t K = p.K;
  int k0 = col * kCols + wave * 128;
  int64_t row[TB][4];  // of token 16 j + 4 q + h
#pragma unroll
  for (int j = 0; j < TB; j++)
#pragma unroll
    for (int q = 0; q < 4; q++)
      row[j][q] = token_at(p.order, p.T, tile.begin + min(j * 16 + q * 4 + h, tile.count - 1)) * K;
  // without a base: read what dx holds, to no one's use
  const uint16_t* const base = g.base ? g.base : g.dx;
  us8_t had[2][4];
  auto mine = [&] { return min(k0 + i16 * 8, p.K - 8); };  // beyond the last: for no one's results
  auto load_base = [&](us8_t(&to)[4], int j) {
#pragma unroll
    for (int q = 0; q < 4; q++)
      to[q] = *reinterpret_cast<const us8_t*>(base + row[j][q] + mine());
  };
  us8_t fa[8][C];  // rows of a first, then turned around
  auto load_a = [&] {
#pragma unroll
    for (int c = 0; c < C; c++) {
      // beyond the last rank: read within the pool, cleared before the product
      const uint16_t* from =
          p.a + ((int64_t)(none ? 0 : tile.l) * p.R + min(Ranks<RB>::of(c, h), p.R - 8)) * K + mine();
#pragma unroll
      for (int i = 0; i < 8; i++) fa[i][c] = *reinterpret_cast<const us8_t*>(from + i * K);
    }
  };
  load_base(had[0], 0);
  load_a();
  spread_parts<BF, RB, kTile, kGradWaves * 64>(
      [&](int t, int r) {
        return none ? f4_t{0, 0, 0, 0}
                    : add_shares(g.shares + ((int64_t)tile.begin + t) * p.R + r, p.T * p.R, g.splits);
      },
      none ? 0.0f : p.scales[tile.l], tile.count, p.R, parts, exponent);
  __syncthreads();
  for (; cols > 0 && k0 < p.K; cols--) {
#pragma unroll
    for (int c = 0; c < C; c++) {
      us8_t rows[8], turned[8];
#pragma unroll
      for (int i = 0; i < 8; i++) rows[i] = fa[i][c];
      transpose8(rows, turned);
      const bool none_such = Ranks<RB>::of(c, h) >= p.R;
#pragma unroll
      for (int i = 0; i < 8; i++) fa[i][c] = none_such ? us8_t{} : turned[i];
    }
#pragma unroll
    for (int j = 0; j < TB; j++) {
      if (j * 16 >= tile.count) break;
      if (j + 1 < TB) load_base(had[(j + 1) % 2], j + 1);
      f4_t acc[8] = {};
      multiply_parts<BF, RB>(fa, parts[j * 16 + i16], h, acc);
      // row 4 h + i of product m is column 8 (4 h + i) + m
#pragma unroll
      for (int i = 0; i < 4; i++) {
        float* const to = &result[i16][(h * 4 + i) * 8];
        *reinterpret_cast<f4_t*>(to) = f4_t{acc[0][i], acc[1][i], acc[2][i], acc[3][i]};
        *reinterpret_cast<f4_t*>(to + 4) = f4_t{acc[4][i], acc[5][i], acc[6][i], acc[7][i]};
      }
      wave_lds_order();
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const int t = q * 4 + h;
        const f4_t lo = *reinterpret_cast<const f4_t*>(&result[t][i16 * 8]);
        const f4_t hi = *reinterpret_cast<const f4_t*>(&result[t][i16 * 8 + 4]);
        const int e = BF ? 0 : exponent[j * 16 + t];
        us8_t o = g.base ? had[j % 2][q] : us8_t{};
        if (!none)
#pragma unroll
          for (int m = 0; m < 8; m++) {
            float f = m < 4 ? lo[m % 4] : hi[m % 4];
            if (!BF) f = times_power(f, -e);
            if (g.base) f += Half16<BF>::to(o[m]);
            o[m] = Half16<BF>::from(f);
          }
        if (k0 + i16 * 8 < p.K && j * 16 + t < tile.count)
          *reinterpret_cast<us8_t*>(g.dx + row[j][q] + mine()) = o;
      }
      wave_lds_order();
    }
    k0 += kCols;
    if (cols > 1 && k0 < p.K) {
      load_base(had[0], 0);
      load_a();
    }
  }
}

// The first of an adapter's shares where it has several chunks, its tokens beginning at
// `first`: n >= 2 chunks of more than n - 1 whole ones are at most twice their whole
// ones, so adapters' shares never overlap, and there are 2 T / chunk + 1 in all.
__device__ __forceinline__ int64_t share_of(int first, int chunk) { return 2 * (int64_t)first / chunk; }

// da (ROWS_X: sums of u_t x_t) or db (v_t dy_t) of one chunk of tokens, 64 ranks from
// r0 on and 512 columns, 128 to a wave.  64 tokens at a time pass through LDS as parts
// of u or v, turned around so that an operand's eight tokens lie side by side, in two
// buffers; their rows of x or dy go straight to the registers, where the next 64 tokens'
// are under way while these are multiplied.  fp16: the parts stand for values times 2^e, e
// by the largest value of the chunk so far (all of this workgroup's ranks, and a chunk's length has
// no upper limit); the sums follow when it changes.
// At most two blocks of ranks to a wave: four double the waves, two for each 128 columns, whose
// second reading of a row the vector cache serves.
template <int RB>
struct SumWaves {
  static constexpr int kBlocks = RB < 2 ? 1 : 2, kCount = kGradWaves * RB / kBlocks;
};
template <bool BF, int RB, bool ROWS_X>
__device__ __forceinline__ void sum_part(const SpreadArgs& g, int index, int col, int r0,
                                         char* lds) {
  constexpr int PARTS = BF ? 3 : 2, TURN = kTile + 8, HALVES = kTile / 32;
  constexpr int RW = SumWaves<RB>::kBlocks, WAVES = SumWaves<RB>::kCount;
  constexpr int kPerToken = WAVES * 64 / kTile;
  typedef uint16_t Turned[PARTS][RB * 16][TURN];
  Turned* const turned = reinterpret_cast<Turned*>(lds);                       // [2]
  int(*const places)[kTile] = reinterpret_cast<int(*)[kTile]>(lds + 2 * sizeof(Turned));  // [2]
  int(*const tops)[WAVES] = reinterpret_cast<int(*)[WAVES]>(places + 2);     // [2]
  const LoraArgs& p = g.p;
  LoraTile tile;
  if (!find_tile(p.starts, p.L, (int)p.T, g.chunk, index, tile) || tile.l == p.L) return;
  const int lane = threadIdx.x & 63, wave = wave_of_group();
  const int i16 = lane & 15, h = lane >> 4;
  const int64_t C = ROWS_X ? p.K : p.N;
  const uint16_t* const rows_of = ROWS_X ? g.x : g.dy;
  const int ranks = min(p.R - r0, RB * 16);
  const int w0 = col * kCols + wave % kGradWaves * 128;  // the wave's columns
  const int b0 = wave / kGradWaves * RW;                 // and its blocks of ranks
  // this lane's eight; beyond the last column the last eight again, which somebody else
  // stores, and where C is no multiple of eight an overlap with the lane before
  const int wanted = w0 + i16 * 8, c0 = (int)min((int64_t)wanted, C - 8);
  const bool active = w0 < C;
  const int t = threadIdx.x / kPerToken, s = threadIdx.x % kPerToken;
  f4_t acc[RW][8];
#pragma unroll
  for (int i = 0; i < RW; i++)
#pragma unroll
    for (int m = 0; m < 8; m++) acc[i][m] = f4_t{0, 0, 0, 0};
  // this thread's token and its values of u or v among the 64 from t0 on
  auto token_of = [&](int t0) {
    return (int)token_at(p.order, p.T, tile.begin + min(t0 + t, tile.count - 1));
  };
  f4_t val[RW][ROWS_X ? kMostSplits : 1];
  auto load_values = [&](int t0, int token) {
    // beyond the last token or rank: read within the buffer, cleared when they are used
    const int64_t at = ROWS_X ? tile.begin + min(t0 + t, tile.count - 1) : token;
#pragma unroll
    for (int i = 0; i < RW; i++) {
      const int r = r0 + min((s + i * kPerToken) * 4, ranks - 4);
      if (ROWS_X) {
#pragma unroll
        for (int w = 0; w < kMostSplits; w++)
          if (w < g.splits)
            val[i][w] = *reinterpret_cast<const f4_t*>(g.shares + (w * p.T + at) * p.R + r);
      } else {
        val[i][0] = *reinterpret_cast<const f4_t*>(g.v + at * p.R + r);
      }
    }
  };
  f4_t sum[RW];
  auto add_values = [&](int t0) {
#pragma unroll
    for (int i = 0; i < RW; i++) {
      sum[i] = val[i][0];
      if (ROWS_X)
#pragma unroll
        for (int w = 1; w < kMostSplits; w++)
          if (w < g.splits) sum[i] += val[i][w];
      if (t0 + t >= tile.count || (s + i * kPerToken) * 4 >= ranks) sum[i] = f4_t{0, 0, 0, 0};
    }
  };
  us8_t rows[HALVES][8];
  // One path for all loads: where two meet, the compiler waits for either's.  A place beyond
  // the last token holds the last one's row, cleared before the product.
  auto load_rows = [&](int half, const int (&place)[kTile]) {
    int tok[8];
#pragma unroll
    for (int i = 0; i < 8; i++) tok[i] = place[half * 32 + h * 8 + i];
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const uint16_t* from = rows_of + tok[i] * C + c0;
      rows[half][i] = ROWS_X ? *reinterpret_cast<const us8_t*>(from) : load8(from);
    }
  };
  int e = 0;
  bool any = false;  // whether e was chosen
  int token = token_of(0), next = token_of(kTile);
  load_values(0, token);
  if (s == 0) places[0][t] = token;
  __syncthreads();
#pragma unroll
  for (int half = 0; half < HALVES; half++) {
    load_rows(half, places[0]);
    loads_stay();
  }
  for (int t0 = 0, b = 0; t0 < tile.count; t0 += kTile, b ^= 1) {
    add_values(t0);
    if (!BF) {
      int top = 0;
#pragma unroll
      for (int i = 0; i < RW; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const int bits = __builtin_bit_cast(int, (float)sum[i][j]) & 0x7fffffff;
          if (bits < 0x7f800000) top = max(top, bits);
        }
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) top = max(top, __shfl_xor(top, off, kWave));
      if (lane == 0) tops[b][wave] = top;
      __syncthreads();
      top = 0;
#pragma unroll
      for (int w = 0; w < WAVES; w++) top = max(top, tops[b][w]);
      const int wanted = fp16_exponent(top);
      if (top != 0 && (!any || wanted < e)) {
        const int by = any ? wanted - e : 0;
        e = wanted;
        any = true;
        if (by != 0)
#pragma unroll
          for (int i = 0; i < RW; i++)
#pragma unroll
            for (int m = 0; m < 8; m++)
#pragma unroll
              for (int j = 0; j < 4; j++) acc[i][m][j] = times_power(acc[i][m][j], by);
      }
    }
#pragma unroll
    for (int i = 0; i < RW; i++) {
      const int r = (s + i * kPerToken) * 4;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        uint16_t part[PARTS];
        split_parts<BF>(BF ? sum[i][j] : times_power(sum[i][j], e), part);
#pragma unroll
        for (int q = 0; q < PARTS; q++) turned[b][q][r + j][t] = part[q];
      }
    }
    if (s == 0) places[b ^ 1][t] = next;
    __syncthreads();  // the parts and the next places are there; the buffers before have been read
    load_values(t0 + kTile, next);
    loads_stay();
    next = token_of(t0 + 2 * kTile);
#pragma unroll
    for (int half = 0; half < HALVES; half++) {
      const int at = half * 32 + h * 8;
      us8_t cols[8];
      if (t0 + half * 32 + 32 > tile.count)
#pragma unroll
        for (int i = 0; i < 8; i++)
          if (t0 + at + i >= tile.count) rows[half][i] = us8_t{};
      transpose8(rows[half], cols);
      if (t0 + kTile < tile.count) load_rows(half, places[b ^ 1]);
      loads_stay();
      if (!active || t0 + half * 32 >= tile.count) continue;
#pragma unroll
      for (int i = 0; i < RW; i++)
#pragma unroll
        for (int q = 0; q < PARTS; q++) {
          const us8_t fu = *reinterpret_cast<const us8_t*>(&turned[b][q][(b0 + i) * 16 + i16][at]);
#pragma unroll
          for (int m = 0; m < 8; m++) acc[i][m] = Half16<BF>::mma(fu, cols[m], acc[i][m]);
        }
    }
  }
  if (!active) return;
  const float scale = p.scales[tile.l];
  const int64_t size = (int64_t)p.R * C;
  // an adapter's only chunk is its whole sum
  const int64_t share = share_of(tile.first, g.chunk) + (tile.begin - tile.first) / g.chunk;
  float* out = tile.tiles == 1 ? (ROWS_X ? g.da : g.db) + tile.l * size
                               : (ROWS_X ? g.part_a : g.part_b) + share * size;
#pragma unroll
  for (int i = 0; i < RW; i++) {
    const int r = (b0 + i) * 16 + h * 4;
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
      if (wanted < C)
#pragma unroll
        for (int j = 0; j < 4; j++) {
          float* at = out + (r0 + r + j) * C + c0;
          *reinterpret_cast<f4_t*>(at) = f4_t{f[0][j], f[1][j], f[2][j], f[3][j]};
          *reinterpret_cast<f4_t*>(at + 4) = f4_t{f[4][j], f[5][j], f[6][j], f[7][j]};
        }
    } else {
#pragma unroll
      for (int m = 0; m < 8; m++)
        if (wanted < C && c0 + m >= wanted)
          *reinterpret_cast<f4_t*>(out + (int64_t)(c0 + m) * p.R + r0 + r) =
              f4_t{f[m][0], f[m][1], f[m][2], f[m][3]};
    }
  }
}

template <bool BF, int RB>
__global__ __launch_bounds__(SumWaves<RB>::kCount * 64) void lora_sums_kernel(const SpreadArgs g) {
  constexpr int kSum =
      2 * ((BF ? 3 : 2) * RB * 16 * (kTile + 8) * 2 + kTile * 4 + SumWaves<RB>::kCount * 4);
  __shared__ __align__(16) char lds[kSum];
  const int groups = (g.p.R + 63) / 64, cols = (g.k_cols + g.n_cols) * groups;
  const int index = blockIdx.x / cols, at = blockIdx.x % cols;
  const int col = at / groups, r0 = at % groups * 64;
  if (col < g.k_cols)
    sum_part<BF, RB, true>(g, index, col, r0, lds);
  else
    sum_part<BF, RB, false>(g, index, col - g.k_cols, r0, lds);
}

// ---------------------------------------------------------------------------
// the join: da and db of adapters with several chunks, or none; dx beside it
// ---------------------------------------------------------------------------
struct JoinArgs {
  const int32_t* starts;
  int T, L, chunk;
  int64_t size_a, size_b;
  const float *part_a, *part_b;
  float *da, *db;
  int64_t blocks;  // of an adapter
};
__device__ __forceinline__ void join_part(const JoinArgs& g, int64_t index) {
  const int l = (int)(index / g.blocks);
  int s0 = 0, s1 = 0;
  if (g.T > 0) {
    s0 = min(max(g.starts[l], 0), g.T);
    s1 = min(max(g.starts[l + 1], s0), g.T);
  }
  const int mine = (s1 - s0 + g.chunk - 1) / g.chunk;
  if (mine == 1) return;
  const int64_t before = share_of(s0, g.chunk);
  for (int64_t i = index % g.blocks; i * 1024 < g.size_a + g.size_b; i += g.blocks) {
    int64_t at = (i * 256 + threadIdx.x) * 4;
    const bool b = at >= g.size_a;
    if (b) at -= g.size_a;
    const int64_t size = b ? g.size_b : g.size_a;
    if (at >= size) break;
    const float* part = (b ? g.part_b : g.part_a) + before * size + at;
    f4_t sum = {0, 0, 0, 0};
#pragma unroll 4
    for (int c = 0; c < mine; c++) sum += *reinterpret_cast<const f4_t*>(part + c * size);
    *reinterpret_cast<f4_t*>((b ? g.db : g.da) + l * size + at) = sum;
  }
}
__global__ __launch_bounds__(256) void lora_join_kernel(const JoinArgs g) {
  join_part(g, blockIdx.x);
}
template <bool BF, int RB>
__global__ __launch_bounds__(kGradWaves * 64, 2) void lora_finish_kernel(const SpreadArgs g,
                                                                      const JoinArgs join) {
  extern __shared__ __align__(16) char lds[];
  const int ranges = (g.k_cols + g.dx_cols - 1) / g.dx_cols;
  const int64_t dx = g.tiles * ranges, at = blockIdx.x;
  if (at < dx)
    dx_part<BF, RB>(g, (int)(at / ranges), (int)(at % ranges) * g.dx_cols, g.dx_cols, lds);
  else
    join_part(join, at - dx);
}

// floats of u's shares
int64_t u_floats(const LoraSizes& s, const LoraGradDivision& d) { return d.splits * s.T * s.R; }

template <bool BF, int RB>
hipError_t run(const BackArgs& back, const SpreadArgs& spread, const JoinArgs& join,
               const LoraGradDivision& d, hipStream_t stream) {
  constexpr int RU = RB < 4 ? RB : 4;
  const int groups = (back.p.R + 63) / 64;
  hipError_t e = launch_lds(lora_back_kernel<BF, RU>, dim3((unsigned)d.tiles, d.splits, groups),
                            kBackWaves * 64, back_bytes<RU>(), stream, back);
  if (e != hipSuccess) return e;
  lora_sums_kernel<BF, RU><<<(unsigned)(d.chunks * (d.k_cols + d.n_cols) * groups),
                             SumWaves<RU>::kCount * 64, 0, stream>>>(spread);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_lds(lora_finish_kernel<BF, RB>,
                    dim3((unsigned)(d.tiles * ((d.k_cols + d.dx_cols - 1) / d.dx_cols) +
                                    join.blocks * join.L)), kGradWaves * 64,
                    dx_bytes<RB>(), stream, spread, join);
}
template <bool BF>
hipError_t run(const BackArgs& back, const SpreadArgs& spread, const JoinArgs& join,
               const LoraGradDivision& d, hipStream_t stream) {
  const int blocks = (back.p.R + 15) / 16;
  if (blocks <= 1) return run<BF, 1>(back, spread, join, d, stream);
  if (blocks <= 2) return run<BF, 2>(back, spread, join, d, stream);
  if (blocks <= 4) return run<BF, 4>(back, spread, join, d, stream);
  return run<BF, 8>(back, spread, join, d, stream);
}

}  // namespace

size_t lora_grad_workspace_bytes(const LoraSizes& s) {
  if (s.T == 0) return 0;
  const LoraGradDivision d = divide_lora_grad(s);
  const int64_t parts = d.shares * s.R * (s.K + s.N);
  return (size_t)(u_floats(s, d) + parts) * sizeof(float);
}

hipError_t launch_lora_grad(const void* dy, const void* x, const float* v, int dtype,
                            const LoraArgs& p, const void* base, void* dx, float* da, float* db,
                            void* workspace, hipStream_t stream) {
  const LoraSizes s = {p.T, p.N, p.K, p.R, p.L};
  const LoraGradDivision d = s.T > 0 ? divide_lora_grad(s) : LoraGradDivision{};
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
                             d.chunks, d.k_cols, d.n_cols, d.dx_cols};
  // 1024 values a round; of many adapters, workgroups take several rounds each
  int64_t blocks = (s.R * (s.K + s.N) + 1023) / 1024;
  if (blocks > (1 << 20) / s.L) blocks = (1 << 20) / s.L;
  const JoinArgs join = {p.starts, (int)p.T, p.L, s.T > 0 ? d.chunk : 1, s.R * s.K, s.R * s.N,
                         part_a,   part_b,   da,  db, blocks};
  if (s.T > 0)
    return dtype == kBF16 ? run<true>(back, spread, join, d, stream)
                          : run<false>(back, spread, join, d, stream);
  lora_join_kernel<<<(unsigned)(join.blocks * s.L), 256, 0, stream>>>(join);
  return hipGetLastError();
}

}  // namespace lowbit
