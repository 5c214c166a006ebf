// lora.hip -- out = y + s_l b_l (a_l x): low-rank adapters of many requests beside a
// shared projection.
//
// Two kernels.  The first contracts over K: a workgroup takes one tile of tokens of
// one adapter and a share of K, and leaves v's share in the workspace.  The second
// adds the shares up, and expands over N: it takes a tile and a range of outputs.
// Both read the large operands (x and a; b and y) from memory straight into the
// matrix cores' registers: a lane's operand is eight consecutive elements of a row,
// which is how rows lie, and an element of x or y is used by one wave only.
// Bound by HBM: for few tokens the adapters (2 R (K + N) bytes each), for many x, y
// and out (2 T (K + 2 N) bytes).
#include "lora.h"

namespace lowbit {
namespace {

constexpr int kLoraWaves = 4;

// ---------------------------------------------------------------------------
// v = a x
// ---------------------------------------------------------------------------
struct DownArgs {
  LoraArgs p;
  const uint16_t* x;
  float* shares;  // [splits][T][R], rows in the plan's order
  int k_share;    // a multiple of 64
};

// TB blocks of 16 tokens, RB of 16 ranks (blockIdx.z: which 64 ranks).  A wave's step
// is 64 of K: lane h of a row's four takes 16 consecutive elements, so that the four
// lanes read whole 128-byte lines.
template <bool BF, int RB, int TB>
__global__ __launch_bounds__(kLoraWaves * 64) void lora_down_kernel(const DownArgs g) {
  constexpr int TILE = 16 * TB, PITCH = RB * 16 + 4;
  __shared__ float red[kLoraWaves / 2][TILE][PITCH];
  const LoraArgs& p = g.p;
  LoraTile tile;
  if (!find_tile(p.starts, p.L, (int)p.T, TILE, blockIdx.x, tile) || tile.l == p.L) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i16 = lane & 15, h = lane >> 4;
  const int64_t K = p.K;
  const int r0 = blockIdx.z * 64, ranks = min(p.R - r0, RB * 16);
  const uint16_t* ar[RB];
  const uint16_t* xr[TB];
#pragma unroll
  for (int i = 0; i < RB; i++)
    ar[i] = p.a + ((int64_t)tile.l * p.R + r0 + min(i * 16 + i16, ranks - 1)) * K;
#pragma unroll
  for (int j = 0; j < TB; j++)
    xr[j] = g.x + token_at(p.order, p.T, tile.begin + min(j * 16 + i16, tile.count - 1)) * K;
  f4_t acc[RB][TB];
#pragma unroll
  for (int i = 0; i < RB; i++)
#pragma unroll
    for (int j = 0; j < TB; j++) acc[i][j] = f4_t{0, 0, 0, 0};
  const int k0 = blockIdx.y * g.k_share, k1 = min(k0 + g.k_share, p.K);
  for (int k = k0 + wave * 64; k < k1; k += kLoraWaves * 64) {
#pragma unroll
    for (int half = 0; half < 2; half++) {
      const int at = k + h * 16 + half * 8;
      const bool inside = at < k1;
      us8_t fa[RB], fx[TB];
#pragma unroll
      for (int i = 0; i < RB; i++)
        fa[i] = inside ? *reinterpret_cast<const us8_t*>(ar[i] + at) : us8_t{};
#pragma unroll
      for (int j = 0; j < TB; j++)
        fx[j] = inside ? *reinterpret_cast<const us8_t*>(xr[j] + at) : us8_t{};
#pragma unroll
      for (int i = 0; i < RB; i++)
#pragma unroll
        for (int j = 0; j < TB; j++) acc[i][j] = Half16<BF>::mma(fa[i], fx[j], acc[i][j]);
    }
  }
  // the waves' sums in two steps, each half of them into the other
#pragma unroll
  for (int left = kLoraWaves / 2; left > 0; left >>= 1) {
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

// A product's 32 terms are 16 ranks twice: against the upper and the lower part of
// s v.  A wave's step is 64 outputs; the rows of b are dealt to the products so that a
// lane's results are eight consecutive outputs of one token.
template <bool BF, int RB, int TB>
__global__ __launch_bounds__(kLoraWaves * 64) void lora_up_kernel(const UpArgs g) {
  constexpr int TILE = 16 * TB, PITCH = RB * 32 + 8;
  constexpr int kPerToken = kLoraWaves * 64 / TILE;  // threads of a token
  constexpr int kQuads = (RB * 4 + kPerToken - 1) / kPerToken;
  __shared__ uint16_t parts[TILE][PITCH];
  __shared__ int exponent[TILE];
  const LoraArgs& p = g.p;
  LoraTile tile;
  if (!find_tile(p.starts, p.L, (int)p.T, TILE, blockIdx.x, tile)) return;
  const bool none = tile.l == p.L;
  const bool in_place = g.y == g.out;
  if (none && in_place && !g.v) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i16 = lane & 15, h = lane >> 4;
  {
    const int t = threadIdx.x / kPerToken, s = threadIdx.x % kPerToken;
    const float scale = none ? 0.0f : p.scales[tile.l];
    f4_t val[kQuads];
    int top = 0;
#pragma unroll
    for (int i = 0; i < kQuads; i++) {
      const int r = (s + i * kPerToken) * 4;
      val[i] = f4_t{0, 0, 0, 0};
      if (r >= p.R || t >= tile.count) continue;
      if (!none)
        for (int w = 0; w < g.splits; w++)
          val[i] += *reinterpret_cast<const f4_t*>(
              g.shares + ((int64_t)w * p.T + tile.begin + t) * p.R + r);
      if (g.v && blockIdx.y == 0)
        *reinterpret_cast<f4_t*>(g.v + token_at(p.order, p.T, tile.begin + t) * p.R + r) = val[i];
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
    for (int i = 0; i < kQuads; i++) {
      const int r = (s + i * kPerToken) * 4;
      if (r >= RB * 16) continue;
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
  if (none && in_place) return;
  const int64_t N = p.N;
  const int blocks = (tile.count + 15) / 16;
  int64_t row[TB];
  int e[TB];
#pragma unroll
  for (int j = 0; j < TB; j++) {
    const int t = j * 16 + i16;
    row[j] = token_at(p.order, p.T, tile.begin + min(t, tile.count - 1)) * N;
    e[j] = exponent[t];
  }
  const int n1 = min((int)(blockIdx.y + 1) * g.n_share, p.N);
  for (int n0 = blockIdx.y * g.n_share + wave * 64; n0 < n1; n0 += kLoraWaves * 64) {
    us8_t fb[4][RB];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      // pair i / 2 covers 32 outputs: row m of its product i % 2 is output 8 (m / 4) + 4 (i % 2) + m % 4
      const int n = n0 + i / 2 * 32 + i16 / 4 * 8 + i % 2 * 4 + i16 % 4;
      const uint16_t* br = p.b + ((int64_t)(none ? 0 : tile.l) * N + min(n, p.N - 1)) * p.R;
#pragma unroll
      for (int c = 0; c < RB; c++) {
        const int r = c * 16 + (h & 1) * 8;
        fb[i][c] = r < p.R && !none ? *reinterpret_cast<const us8_t*>(br + r) : us8_t{};
      }
    }
#pragma unroll
    for (int j = 0; j < TB; j++) {
      if (j >= blocks) break;
      us8_t fv[RB];
#pragma unroll
      for (int c = 0; c < RB; c++)
        fv[c] = *reinterpret_cast<const us8_t*>(&parts[j * 16 + i16][c * 32 + h * 8]);
#pragma unroll
      for (int pair = 0; pair < 2; pair++) {
        f4_t acc[2] = {f4_t{0, 0, 0, 0}, f4_t{0, 0, 0, 0}};
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
          for (int c = 0; c < RB; c++)
            acc[i] = Half16<BF>::mma(fb[pair * 2 + i][c], fv[c], acc[i]);
        const int n = n0 + pair * 32 + h * 8;
        if (j * 16 + i16 >= tile.count || n >= n1) continue;
        const int left = p.N - n;
        us8_t had = {};
        if (g.y) had = load8(g.y + row[j] + n, left);
        us8_t o;
#pragma unroll
        for (int q = 0; q < 8; q++) {
          float f = acc[q / 4][q % 4];
          if (!BF) f = times_power(f, -e[j]);
          if (g.y) f += Half16<BF>::to(had[q]);
          o[q] = Half16<BF>::from(f);
        }
        // a token without an adapter keeps the bits it has
        store8(g.out + row[j] + n, none ? had : o, left);
      }
    }
  }
}

// How a call is divided: tokens in a tile, shares of K, outputs of a workgroup.
struct Division {
  int tile;
  int64_t tiles;
  int splits, k_share;
  int ranges, n_share;
};
Division divide(const LoraSizes& s) {
  Division d;
  d.tile = s.T <= 256 ? 16 : 64;
  d.tiles = lora_tiles(s.T, s.L, d.tile);
  auto shares = [&](int64_t length, int64_t wanted, int& count, int& share) {
    const int64_t most = (length + 255) / 256;
    int64_t n = (wanted + d.tiles - 1) / d.tiles;
    if (n > most) n = most;
    share = (int)(((length + n - 1) / n + 63) / 64 * 64);
    count = (int)((length + share - 1) / share);
  };
  shares(s.K, 512, d.splits, d.k_share);
  shares(s.N, 1024, d.ranges, d.n_share);
  return d;
}

template <bool BF, int RB, int TB>
hipError_t run(const DownArgs& down, const UpArgs& up, const Division& d, hipStream_t stream) {
  constexpr int DOWN = RB < 4 ? RB : 4;
  lora_down_kernel<BF, DOWN, TB><<<dim3((unsigned)d.tiles, d.splits, (down.p.R + 63) / 64),
                                   kLoraWaves * 64, 0, stream>>>(down);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  lora_up_kernel<BF, RB, TB>
      <<<dim3((unsigned)d.tiles, d.ranges), kLoraWaves * 64, 0, stream>>>(up);
  return hipGetLastError();
}
template <bool BF, int RB>
hipError_t run(const DownArgs& down, const UpArgs& up, const Division& d, hipStream_t stream) {
  return d.tile == 16 ? run<BF, RB, 1>(down, up, d, stream) : run<BF, RB, 4>(down, up, d, stream);
}
template <bool BF>
hipError_t run(const DownArgs& down, const UpArgs& up, const Division& d, hipStream_t stream) {
  const int blocks = (down.p.R + 15) / 16;
  if (blocks <= 1) return run<BF, 1>(down, up, d, stream);
  if (blocks <= 2) return run<BF, 2>(down, up, d, stream);
  if (blocks <= 4) return run<BF, 4>(down, up, d, stream);
  return run<BF, 8>(down, up, d, stream);
}

}  // namespace

size_t lora_workspace_bytes(const LoraSizes& s) {
  if (s.T == 0) return 0;
  return (size_t)divide(s).splits * s.T * s.R * sizeof(float);
}

hipError_t launch_lora(const void* x, int dtype, const LoraArgs& p, const void* y, void* out,
                       float* v, void* workspace, hipStream_t stream) {
  const Division d = divide({p.T, p.N, p.K, p.R, p.L});
  float* const shares = static_cast<float*>(workspace);
  const DownArgs down = {p, static_cast<const uint16_t*>(x), shares, d.k_share};
  const UpArgs up = {p,           shares, d.splits, d.n_share, static_cast<const uint16_t*>(y),
                     static_cast<uint16_t*>(out), v};
  return dtype == kBF16 ? run<true>(down, up, d, stream) : run<false>(down, up, d, stream);
}

}  // namespace lowbit
