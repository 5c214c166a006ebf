// lora_division.h -- how the adapter calls are divided into tiles, shares and chunks: host
// arithmetic on sizes, without HIP, so that a program without a GPU can ask too.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace lowbit {

// Every bound on a number of tiles counts one for each adapter that has tokens, whose last
// tile may be a part, and one for the tokens without an adapter.
struct LoraSizes {
  int64_t T, N, K, R, L;
};
inline int64_t lora_tiles(int64_t T, int64_t L, int tile) {
  const int64_t most = (T + tile - 1) / tile + L;
  return most < T ? most : T;
}

// The forward pass: tokens in a tile, shares of K, outputs of a workgroup.
struct LoraDivision {
  int tile;
  int64_t tiles;
  int splits, k_share;
  int ranges, n_share;
};
inline LoraDivision divide_lora(const LoraSizes& s) {
  LoraDivision d;
  // Small tiles up to 256 tokens, large ones beyond (us of both kernels, tiles of 16 / 64, 4096
  // outputs and K unless given: 64 tokens, 16 ranks 8.9 / 11.4; 256 tokens 10.2 / 12.5; 2000 of
  // 11008x4096, 64 ranks 50.5 / 43.2; 8192 of 12288x12288, 64 ranks 234 / 156).  The border is a plain
  // one: small tiles lead further on where adapters have few tokens or ranks are few (512 tokens of
  // 64 adapters, 64 ranks 26.3 / 36.2; 1333 of 4096x11008, 24 ranks 25.5 / 28.7; 4096, 16 ranks 28.8 / 31.7).
  d.tile = s.T <= 256 ? 16 : 64;
  d.tiles = lora_tiles(s.T, s.L, d.tile);
  auto shares = [&](int64_t length, int64_t n, int& count, int& share) {
    share = (int)(((length + n - 1) / n + 63) / 64 * 64);
    count = (int)((length + share - 1) / share);
  };
  auto over_tiles = [&](int64_t workgroups) { return (workgroups + d.tiles - 1) / d.tiles; };
  // Shares of K: 512 workgroups (us of both kernels with 256 / 512 / 1024: 8192 tokens of 12288x12288,
  // 64 ranks 186 / 156 / 156, 16 ranks 154 / 136 / 135; from 4096 tokens down the limits decide and it is one),
  // a step for every wave at the least, and few, as every workgroup of the expansion
  // adds them up again (us of both kernels with 8 / 4 at most: 1500 tokens of 8192x8192, 128 ranks
  // 85 / 71, 700 of 11008x4096, 64 ranks 31 / 29; in small tiles 200 of 4096x8192, 64 ranks 13.8 / 15.3).
  const int64_t step = d.tile == 16 ? 512 : 256;
  int64_t n = over_tiles(512);
  if (n > s.K / (4 * step)) n = std::max(s.K / (4 * step), over_tiles(256));
  n = std::max<int64_t>(1, std::min({n, (s.K + step - 1) / step, d.tile == 16 ? (int64_t)8 : 4}));
  shares(s.K, n, d.splits, d.k_share);
  // Small tiles: many short workgroups (64 tokens of 64 adapters, 11008 outputs, 16 ranks: 8.4 us
  // with 1024, 9.7 with 512).  Large ones: as many as the card holds at once (1024 / 512 / 256 of
  // them: 8192x12288, 64 ranks 101 / 92 / 127; 4096x4096, 128 ranks, one to a CU, 84 / 58 / 42).
  n = std::min(over_tiles(d.tile == 16 ? 1024 : 512), (s.N + 255) / 256);
  shares(s.N, n, d.ranges, d.n_share);
  return d;
}

constexpr int kGradWaves = 4;                // of dx; of da and db with up to 32 ranks
constexpr int kTile = 64;                    // tokens of u's and dx's tiles
constexpr int kCols = kGradWaves * 128;  // columns of a workgroup of dx, da or db
constexpr int kBackWaves = 8;                // of u
constexpr int kMostSplits = 4;               // shares of u: the sums hold them in registers

// The gradients: shares of N for u, tokens of a chunk of the sums, columns of a workgroup of dx.
struct LoraGradDivision {
  int64_t tiles;
  int splits, n_share;
  int chunk;
  int64_t chunks, shares;
  int k_cols, n_cols, dx_cols;
};
inline LoraGradDivision divide_lora_grad(const LoraSizes& s) {
  LoraGradDivision d;
  d.tiles = lora_tiles(s.T, s.L, kTile);
  const int64_t most = (s.N + kBackWaves * 64 - 1) / (kBackWaves * 64);
  // shares of N: the sums read them all again (us of u / sums, 64 ranks: 8192 tokens of 12288x12288
  // with 4 of four waves, 2 of eight, 1: 66 / 120, 74 / 107, 91 / 106; 4096 of 4096x4096 with 4 and 2:
  // 20 / 37, 21 / 33).  192 workgroups (the whole gradient with 96 / 192 / 384: 8192 of 12288x12288, 64
  // ranks 272 / 264 / 281; 2000 of 11008x4096, 16 ranks 48.6 / 46.3 / 46.2; 4096 of 11008x4096, 16 ranks
  // 74.5 / 72.8 / 69.6; fewer tokens have the most shares with any of them)
  int64_t n = (192 + d.tiles - 1) / d.tiles;
  if (n > kMostSplits) n = kMostSplits;
  if (n > most) n = most;
  d.n_share = (int)(((s.N + n - 1) / n + 63) / 64 * 64);
  d.splits = (int)((s.N + d.n_share - 1) / d.n_share);
  d.k_cols = (int)((s.K + kCols - 1) / kCols);
  d.n_cols = (int)((s.N + kCols - 1) / kCols);
  // dx: two workgroups to a CU at once (us of the whole gradient with 256 / 512 / 1024 workgroups: 8192
  // tokens of 12288x12288, 64 ranks 281 / 261 / 264, 16 ranks 232 / 207 / 207; 1500 of 8192x8192, 128 ranks
  // 93 / 87 / 88; 700 of 11008x4096 one)
  const int64_t ranges = 512 / ((s.T + kTile - 1) / kTile);
  d.dx_cols = ranges < 1 ? d.k_cols : (int)((d.k_cols + ranges - 1) / ranges);
  // chunks as many as the card holds workgroups at once, of 128 tokens at least (us of the
  // sums with 256 / 128: 400 tokens 4096x4096, 16 ranks 12.5 / 8.6; 700 of 11008x4096, 64 ranks
  // 20.1 / 16.3, where the join takes 1.9 more).  Above 32 ranks they have twice the waves, and one
  // fills a CU (us of the whole gradient with 256 / 512 held: 64 ranks, 8192 tokens of 12288x12288 261 / 276,
  // 4096 of 4096x4096 84 / 93; 16 ranks, 8192 of 12288x12288 211 / 206, 4096 of 4096x4096 52.4 / 52.0,
  // 8192 of 4096x4096 80 / 85)
  const int64_t cols = (d.k_cols + d.n_cols) * ((s.R + 63) / 64);
  const int64_t held = s.R > 32 ? 256 : 512;
  const int64_t wanted = held > cols ? held / cols : 1;
  int64_t chunk = ((s.T + wanted - 1) / wanted + kTile - 1) / kTile * kTile;
  if (chunk < 128) chunk = 128;
  d.chunk = (int)chunk;
  d.chunks = lora_tiles(s.T, s.L, d.chunk);
  d.shares = s.T > d.chunk ? 2 * s.T / d.chunk + 1 : 0;
  return d;
}

}  // namespace lowbit
