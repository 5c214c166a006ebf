// w8a8_skinny.hip -- the 8-bit products for at most 64 tokens, where reading
// the weights is what takes time.
//
// One persistent workgroup of four waves per CU walks tiles of 16 weight rows
// (gated: 16 of each matrix); its waves share out K, and each streams its own
// part through a ring of its own in LDS: direct loads of 256 (or 128)
// consecutive bytes of each row, weights and the tokens' codes alike, with no
// barrier, only the wave's own load counter between arrival and use.  The
// matrix cores take 16 rows by up to four times 16 tokens from there.  The
// waves' integer sums meet in LDS once per tile.
//
// Measured, kernel alone, on weights rotated over 1 GiB: linear 8x28672x8192 41 us
// (5.7 TB/s), gated 8x28672x8192 78 (6.0).  Short rows end the wave's stream before
// it is in full flow: 8x4096x4096 7.8 (2.1).  The more tokens, the more of what a
// workgroup reads are their codes, again for each 16 weight rows: for 48 tokens
// three bytes from L2 for each byte of weights, 45x4096x11008 from codes 18 us, or 14
// where the weights lie in the last-level cache (reading both operands into
// registers in 64-byte pieces took 23-25).
#include "w8a8.h"

namespace lowbit {
namespace {

// Shape of the ring: waves, bytes of a row per step, steps.
template <int NT, bool GATED>
struct Ring {
  static constexpr int FR = GATED ? 2 : 1;
  static constexpr int OPS = FR + NT;  // 16-row operands per step
  static constexpr int W = 4;
  static constexpr int CH = OPS <= 4 ? 256 : 128;
  static constexpr int D = OPS == 2 ? 4 : OPS == 3 || OPS == 5 ? 3 : 2;
  static constexpr int kOp = 16 * CH;                // bytes of an operand
  static constexpr int kRing = W * D * OPS * kOp;
  static constexpr int kSums = W * FR * NT * 1024;
};

// 16 weight rows (of each matrix) per tile, NT token tiles.  The
// workgroup walks tiles blockIdx.x, blockIdx.x + gridDim.x, ...; a wave's
// loads run ahead into its next tile.
template <int NT, bool GATED>
__global__ __launch_bounds__((Ring<NT, GATED>::W * 64)) void skinny_kernel(const GemmArgs p) {
  using R = Ring<NT, GATED>;
  constexpr int FR = R::FR, OPS = R::OPS, CH = R::CH, D = R::D, kWaves = R::W;
  constexpr int kSlots = CH / 16, kLoads = CH / 64;
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  // the waves' rings, and their sums
  i4_t* sums = reinterpret_cast<i4_t*>(lds + R::kRing);

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i16 = lane & 15, h = lane >> 4;
  const uint32_t K = (uint32_t)p.K;
  const int steps = (p.K + kWaves * CH - 1) / (kWaves * CH);  // of each wave and tile
  const int tiles = (p.N + 15) / 16;
  const i4_t ra = buffer_of(p.a, (uint32_t)p.T * K);

  // load q of an operand: rows q * (1024 / CH) + ..., chunk c of a row at slot c ^ row
  uint32_t off[kLoads], kc[kLoads];
#pragma unroll
  for (int q = 0; q < kLoads; q++) {
    const int row = q * (1024 / CH) + lane / kSlots;
    kc[q] = ((lane % kSlots) ^ (row & (kSlots < 16 ? 7 : 15))) * 16;
    off[q] = row * K + kc[q];
  }
  const uint32_t ring = lds_address(lds) + wave * D * OPS * R::kOp;
  int lt = blockIdx.x, ls = 0;  // tile and step of the next load
  // values past the row's end come as zeros, and so do rows and tiles past the last
  auto load = [&](int slot) {
    const int n0 = lt * 16;
    const uint32_t bytes = (uint32_t)max(0, min(16, p.N - n0)) * K;
    const uint32_t k0 = (uint32_t)(ls * kWaves + wave) * CH;
    const uint32_t to = ring + slot * OPS * R::kOp;
#pragma unroll
    for (int o = 0; o < OPS; o++) {
      const i4_t rs = o < FR ? buffer_of(p.w[o].codes + (int64_t)n0 * K, bytes) : ra;
#pragma unroll
      for (int q = 0; q < kLoads; q++) {
        uint32_t at = off[q] + k0 + (o < FR ? 0 : (o - FR) * 16 * K);
        if (k0 + kc[q] >= K) at = 0x80000000u;
        load_to_lds<true>(rs, to + o * R::kOp + q * 1024, at);
      }
    }
    if (++ls == steps) {
      ls = 0;
      lt += gridDim.x;
    }
  };
#pragma unroll
  for (int d = 0; d < D; d++) load(d);
  i4_t acc[FR][NT];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < FR; i++)
#pragma unroll
      for (int j = 0; j < NT; j++) acc[i][j] = i4_t{0, 0, 0, 0};
  };
  clear();
  // joins the waves' sums of a tile; the waves take turns to finish its
  // NT fragments: lane l holds outputs n = 4 (l / 16) + 0..3 of token l % 16
  auto finish = [&](int tile, int round) {
    __syncthreads();  // the last tile's sums have been read
#pragma unroll
    for (int i = 0; i < FR; i++)
#pragma unroll
      for (int j = 0; j < NT; j++) sums[(wave * FR * NT + i * NT + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    for (int o = (wave + round) % kWaves; o < NT; o += kWaves) {
      const int n = tile * 16 + h * 4, t = o * 16 + i16;
      if (n >= p.N || t >= p.T) continue;
      i4_t sum[2] = {i4_t{0, 0, 0, 0}, i4_t{0, 0, 0, 0}};
#pragma unroll
      for (int v = 0; v < kWaves; v++) {
        sum[0] += sums[(v * FR * NT + o) * 64 + lane];
        if constexpr (GATED) sum[1] += sums[(v * FR * NT + NT + o) * 64 + lane];
      }
      store4<GATED>(p, Columns<GATED>(p, n), sum[0], sum[1], n, t, p.xs[t], p.xsum[t]);
    }
    clear();
  };

  int tile = blockIdx.x, step = 0, round = 0;
  const uint8_t* mine = lds + wave * D * OPS * R::kOp + i16 * CH;
  const int turn = i16 & (kSlots < 16 ? 7 : 15);
  while (tile < tiles) {
#pragma unroll
    for (int d = 0; d < D; d++) {
      lds_loads_left<(D - 1) * OPS * kLoads>();
      const uint8_t* buf = mine + d * OPS * R::kOp;
#pragma unroll
      for (int s = 0; s < CH / 64; s++) {
        const int at = ((s * 4 + h) ^ turn) * 16;
        i4_t a[NT];
#pragma unroll
        for (int j = 0; j < NT; j++) {
          a[j] = *reinterpret_cast<const i4_t*>(buf + (FR + j) * R::kOp + at);
        }
#pragma unroll
        for (int i = 0; i < FR; i++) {
          const i4_t w = *reinterpret_cast<const i4_t*>(buf + i * R::kOp + at) ^ (int)0x80808080;
#pragma unroll
          for (int j = 0; j < NT; j++)
            acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w, a[j], acc[i][j], 0, 0, 0);
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read: free for the next load
      load(d);
      if (++step == steps) {
        if (tile < tiles) finish(tile, round);  // the same for all waves
        step = 0;
        tile += gridDim.x;
        round++;
      }
    }
  }
  lds_loads_left<0>();
}

template <int NT, bool GATED>
hipError_t launch_one(const GemmArgs& p, hipStream_t stream) {
  using R = Ring<NT, GATED>;
  constexpr int bytes = R::kRing + R::kSums;
  static_assert(bytes <= 160 * 1024, "LDS of a CU");
  auto kernel = skinny_kernel<NT, GATED>;
  hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(kernel), bytes);
  if (e != hipSuccess) return e;
  const int tiles = (p.N + 15) / 16;
  // whole rounds of tiles, as even as they can be
  const int most_groups = device_cu_count();
  const int rounds = (tiles + most_groups - 1) / most_groups;
  kernel<<<dim3((unsigned)((tiles + rounds - 1) / rounds)), dim3(R::W * 64), bytes, stream>>>(p);
  return hipGetLastError();
}

template <bool GATED>
hipError_t launch_tokens(const GemmArgs& p, hipStream_t stream) {
  if (p.T <= 16) return launch_one<1, GATED>(p, stream);
  if (p.T <= 32) return launch_one<2, GATED>(p, stream);
  if (p.T <= 48) return launch_one<3, GATED>(p, stream);
  return launch_one<4, GATED>(p, stream);
}

}  // namespace

hipError_t launch_skinny(const GemmArgs& p, bool gated, hipStream_t stream) {
  return gated ? launch_tokens<true>(p, stream) : launch_tokens<false>(p, stream);
}

}  // namespace lowbit
