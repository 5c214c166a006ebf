// w8a8_gemm.hip -- products in 8-bit integers on the matrix cores
// (v_mfma_i32_16x16x64_i8 of gfx950): the linear layer and the gated block.
//
//   y[t][n] = S_t s_n (sum_k a[t][k] c'[n][k] + (128 - z_n) A_t)
//
// a are a token's codes, S its scale, A the sum of its codes; c' = code - 128
// is the code byte with its top bit flipped, a signed byte; the zero point
// enters once for each output.  Both grids of the weight quantizers are
// covered and every integer sum is exact.
#include "w8a8.h"

namespace lowbit {
namespace {

// One workgroup of WM x WN waves computes MT tokens by NT weight rows (gated:
// NT / 2 rows of each matrix, the wave's first half gate, its second half up,
// so a lane holds both projections of an output).
//
// Steps of 64 SUB k are staged in LDS by direct loads on a ring of NB buffers,
// one barrier per step.  A row of a step is 4 SUB chunks of 16 bytes; chunk c of
// row r lies at c ^ (-(r / 4) & 3), or c ^ (r & 7) with SUB == 2, so that the
// rows one operand read touches at a time lie in different banks (no conflicts
// counted).  Values past the row's end, tokens past T and rows past N come as
// zeros from the buffers' range check.
//
// What bounds the large tiles: no one thing.  4096x12288x12288 takes 500-533 us in
// tiles of 256 x 384 (2.3-2.5 POP/s; 128 x 96 per wave is the most that 256
// registers hold), the whole call 531, and 577 with tiles of 256 x 256 at most.
// Power holds the clock at 1.9 GHz, and 63% of the clocks are products.  With a part
// left out: 423 us without the direct loads (of 192 steps' 40 KiB a tile),
// 501 without the operand reads (112 KiB a step; LDS gives 230 bytes a clock and CU
// and is busy with them for a fifth of the time), 402 without both, 396 without the
// products.  Slower there, against 541 us for 256 x 256 at the time: 128 x 128 per wave
// with one wave per SIMD (a third fewer reads, but a lone wave cannot issue fast
// enough: 577), weights straight from L2 into registers (750), 32x32x32 products (620).
//
// Short inputs pay as much around the steps: gated 333x11008x4096 with its
// projections kept takes 44 us in 192 x 192 tiles, 0.88 us for each of 32 steps
// (half of it products) and 16 us before and after them (the first loads, the
// activation, three outputs of 7.3 MB); 12.5 where only h goes out.
template <int MT, int NT, int WM, int WN, int NB, int SUB, bool GATED>
__global__ __launch_bounds__(WM* WN * 64, 2) void w8a8_kernel(const GemmArgs p, const TilePlan plan,
                                                                 i4_t* __restrict__ parts) {
  constexpr int kWaves = WM * WN;
  constexpr int MW = MT / WM, NW = NT / WN;  // wave tile
  constexpr int FM = MW / 16, FN = NW / 16;  // its fragments
  constexpr int NO = GATED ? NT / 2 : NT;    // output columns of a tile
  constexpr int kStep = 64 * SUB, kChunks = 4 * SUB;  // bytes and chunks of a row per step
  // 1 KiB loads of 16 / SUB rows; where the weights' do not come out even among the
  // waves, the last go to a place of their own, so that every wave counts as many
  constexpr int kRows = 16 / SUB;
  constexpr int kA = MT / kRows, kB = NT / kRows;
  constexpr int LA = kA / kWaves, LB = (kB + kWaves - 1) / kWaves, kLoads = LA + LB;
  static_assert(LA * kWaves == kA && MT % (16 * WM) == 0 && NT % (16 * WN) == 0, "whole loads");
  static_assert(!GATED || FN % 2 == 0, "gate and up halves");
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  constexpr int kBuf = (MT + NT) * kStep;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WM, wn = wave / WM;
  const int i16 = lane & 15, h = lane >> 4;
  const int steps = (p.K + kStep - 1) / kStep;
  // a whole tile, or a share of the steps of one of the rest
  const int over = (int)blockIdx.x - plan.whole;
  const int split = over < 0 ? 0 : over % plan.splits;
  const int s0 = over < 0 ? 0 : (int)((int64_t)steps * split / plan.splits);
  const int s1 = over < 0 ? steps : (int)((int64_t)steps * (split + 1) / plan.splits);
  int tm, tn;
  tile_of(over < 0 ? (int)blockIdx.x : plan.whole + over / plan.splits, plan.whole,
          plan.tiles_m, plan.tiles_n, tm, tn);
  const int t0 = tm * MT, n0 = tn * NO;
  const uint32_t K = (uint32_t)p.K;

  const auto ra = buffer_of(p.a + (int64_t)t0 * K, (uint32_t)min(MT, p.T - t0) * K);
  const uint32_t wbytes = (uint32_t)min(NO, p.N - n0) * K;
  const auto rg = buffer_of(p.w[0].codes + (int64_t)n0 * K, wbytes);
  const auto ru = GATED ? buffer_of(p.w[1].codes + (int64_t)n0 * K, wbytes) : rg;

  // lane l of a load brings the chunk that lies at slot l % kChunks of its row l / kChunks
  auto swizzle = [](int r) { return SUB == 1 ? -(r >> 2) & 3 : r & 7; };
  const uint32_t rl = lane / kChunks;
  const uint32_t chunk = ((lane % kChunks) ^ swizzle(rl)) * 16;
  uint32_t oa[LA], ob[LB];
  uint32_t la[LA], lb[LB];
  bool up[LB], spare[LB];
  const uint32_t base = lds_address(lds);
  const uint32_t kend = min((uint32_t)s1 * kStep, K);
#pragma unroll
  for (int i = 0; i < LA; i++) {
    const int row = (wave + i * kWaves) * kRows;
    oa[i] = (row + rl) * K + chunk;
    la[i] = base + row * kStep;
  }
#pragma unroll
  for (int i = 0; i < LB; i++) {
    // LDS rows of the weight tile, in order; of each wave's NW rows the first
    // half is gate rows, the second up rows
    const int slot = (wave + i * kWaves) * kRows, in = slot % NW;
    up[i] = GATED && in >= NW / 2;
    spare[i] = kB % kWaves != 0 && slot >= NT;
    const int row = GATED ? slot / NW * (NW / 2) + in % (NW / 2) : slot;
    ob[i] = spare[i] ? 0x80000000u : (row + rl) * K + chunk;
    lb[i] = base + (spare[i] ? NB * kBuf : (MT + slot) * kStep);
  }
  // load i of the LA + LB of step s; past the share's last step it brings zeros
  auto load = [&](int s, int i) {
    const uint32_t k0 = (uint32_t)s * kStep, buf = (uint32_t)(s % NB) * kBuf;
    const uint32_t add = k0 + chunk < kend ? k0 : 0x80000000u;
    if (i < LA)
      load_to_lds(ra, la[i] + buf, oa[i] + add);
    else
      load_to_lds(up[i - LA] ? ru : rg, lb[i - LA] + (spare[i - LA] ? 0 : buf),
                  spare[i - LA] ? ob[i - LA] : ob[i - LA] + add);
  };

  i4_t acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; i++)
#pragma unroll
    for (int j = 0; j < FM; j++) acc[i][j] = i4_t{0, 0, 0, 0};

  // operands from LDS: row lane % 16, chunk lane / 16 of each 64 bytes
  const uint32_t ra0 = (wm * MW + i16) * kStep, rb0 = (MT + wn * NW + i16) * kStep;
  uint32_t at[SUB];
#pragma unroll
  for (int q = 0; q < SUB; q++) at[q] = ((q * 4 + h) ^ swizzle(i16)) * 16;
  auto tokens = [&](int s, int q, int j) {
    return *reinterpret_cast<const i4_t*>(lds + s % NB * kBuf + ra0 + at[q] + j * 16 * kStep);
  };
  auto rows = [&](int s, int q, int i) {
    return *reinterpret_cast<const i4_t*>(lds + s % NB * kBuf + rb0 + at[q] + i * 16 * kStep);
  };
  // One step: its first tokens are in fa and its first two row operands in fb.
  // The last row operand's products of each 64 bytes are the last to use the
  // tokens; each token's is followed by the read of the next, in the step's last
  // products behind its barrier.
  constexpr int kAll = SUB * FN;
  i4_t fa[FM], fb[2];
  auto step = [&](int s) {
#pragma unroll
    for (int o = 0; o < kAll; o++) {
      const int q = o / FN, i = o % FN;
      if (o == kAll - 1) {
        lds_loads_left<(NB - 2) * kLoads>();  // this wave's part of the next step has landed
        __syncthreads();                      // and everyone's; this step has been read
        __builtin_amdgcn_sched_barrier(0);
      } else {
#pragma unroll
        for (int l = o * kLoads / (kAll - 1); l < (o + 1) * kLoads / (kAll - 1); l++)
          load(s + NB - 1, l);
      }
      const i4_t w = fb[o % 2] ^ (int)0x80808080;
      if (o + 2 < kAll) fb[o % 2] = rows(s, (o + 2) / FN, (o + 2) % FN);
      if (o == kAll - 1) {
        fb[0] = rows(s + 1, 0, 0);
        fb[1] = rows(s + 1, 1 / FN, 1 % FN);
      }
#pragma unroll
      for (int j = 0; j < FM; j++) {
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w, fa[j], acc[i][j], 0, 0, 0);
        if (i == FN - 1) fa[j] = q + 1 < SUB ? tokens(s, (q + 1) % SUB, j) : tokens(s + 1, 0, j);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
#pragma unroll
  for (int s = 0; s < NB - 1; s++)
#pragma unroll
    for (int i = 0; i < kLoads; i++) load(s0 + s, i);
  lds_loads_left<(NB - 2) * kLoads>();
  __syncthreads();
#pragma unroll
  for (int j = 0; j < FM; j++) fa[j] = tokens(s0, 0, j);
  fb[0] = rows(s0, 0, 0);
  fb[1] = rows(s0, 1 / FN, 1 % FN);
  for (int s = s0; s < s1; s++) step(s);
  lds_loads_left<0>();

  if (over >= 0) {
    i4_t* to = parts + ((int64_t)over * kWaves + wave) * (FN * FM * 64) + lane;
#pragma unroll
    for (int i = 0; i < FN; i++)
#pragma unroll
      for (int j = 0; j < FM; j++) to[(i * FM + j) * 64] = acc[i][j];
    return;
  }
  // lane l of a fragment holds outputs n = 4 (l / 16) + 0..3 of token l % 16
  constexpr int FO = GATED ? FN / 2 : FN;
  const int nb = n0 + wn * (GATED ? NW / 2 : NW);
#pragma unroll
  for (int i = 0; i < FO; i++) {
    const int n = nb + i * 16 + h * 4;
    if (n >= p.N) continue;
    const Columns<GATED> c(p, n);
#pragma unroll
    for (int j = 0; j < FM; j++) {
      const int t = t0 + wm * MW + j * 16 + i16;
      if (t >= p.T) continue;
      store4<GATED>(p, c, acc[i][j], acc[FN - FO + i][j], n, t, p.xs[t], p.xsum[t]);
    }
  }
}

// Joins the shares of the plan's rest: one wave for each fragment of a tile.
template <int MT, int NT, int WM, int WN, bool GATED>
__global__ __launch_bounds__(256) void w8a8_join_kernel(const GemmArgs p, const TilePlan plan,
                                                        const i4_t* __restrict__ parts) {
  constexpr int kWaves = WM * WN;
  constexpr int MW = MT / WM, NW = NT / WN, FM = MW / 16, FN = NW / 16;
  constexpr int NO = GATED ? NT / 2 : NT, FO = GATED ? FN / 2 : FN;
  constexpr int kFragments = kWaves * FO * FM;
  const int lane = threadIdx.x & 63;
  const int at = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int tile = at / kFragments, f = at % kFragments;
  if (tile >= plan.rest) return;
  const int wave = f / (FO * FM), i = f / FM % FO, j = f % FM;
  int tm, tn;
  tile_of(plan.whole + tile, plan.whole, plan.tiles_m, plan.tiles_n, tm, tn);
  const int n = tn * NO + wave / WM * (GATED ? NW / 2 : NW) + i * 16 + (lane >> 4) * 4;
  const int t = tm * MT + wave % WM * MW + j * 16 + (lane & 15);
  if (n >= p.N || t >= p.T) return;
  i4_t sum[2] = {i4_t{0, 0, 0, 0}, i4_t{0, 0, 0, 0}};
  const Columns<GATED> columns(p, n);
  const float xs = p.xs[t];
  const int total = p.xsum[t];
  for (int z = 0; z < plan.splits; z += 4) {  // four shares' loads at a time
    i4_t v[4][2];
#pragma unroll
    for (int u = 0; u < 4; u++) {
      const int zz = min(z + u, plan.splits - 1);
      const i4_t* from =
          parts + ((int64_t)(tile * plan.splits + zz) * kWaves + wave) * (FN * FM * 64) + lane;
      v[u][0] = from[(i * FM + j) * 64];
      if constexpr (GATED) v[u][1] = from[((FO + i) * FM + j) * 64];
    }
#pragma unroll
    for (int u = 0; u < 4; u++)
      if (z + u < plan.splits) {
        sum[0] += v[u][0];
        if constexpr (GATED) sum[1] += v[u][1];
      }
  }
  store4<GATED>(p, columns, sum[0], sum[1], n, t, xs, total);
}

template <int MT, int NT, int WM, int WN, int NB, int SUB, bool GATED>
hipError_t launch_tile(const GemmArgs& p, const TilePlan& plan, i4_t* parts, hipStream_t stream) {
  constexpr bool spare = NT * SUB / 16 % (WM * WN) != 0;
  constexpr int bytes = NB * (MT + NT) * 64 * SUB + (spare ? 1024 : 0);
  auto kernel = w8a8_kernel<MT, NT, WM, WN, NB, SUB, GATED>;
  hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(kernel), bytes);
  if (e != hipSuccess) return e;
  kernel<<<dim3((unsigned)plan.blocks()), dim3(WM * WN * 64), bytes, stream>>>(p, plan, parts);
  e = hipGetLastError();
  if (e != hipSuccess || plan.rest == 0) return e;
  constexpr int fragments = (MT / 16) * (NT / 16) / (GATED ? 2 : 1);
  w8a8_join_kernel<MT, NT, WM, WN, GATED>
      <<<dim3((unsigned)(plan.rest * fragments / 4)), dim3(256), 0, stream>>>(p, plan, parts);
  return hipGetLastError();
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// Codes, scales and sums of the activations in the workspace.
size_t code_bytes(int64_t T, int64_t K) { return up256(T * K) + 2 * up256(T * 4); }

// Few activations are quantized inside the product's kernel.
bool fused(int64_t T, int64_t K, int dtype, bool gated) {
  return dtype != kI8 && few_takes(T, K, gated) && T * K <= kFusedMost;
}

template <bool GATED>
hipError_t launch(const Activations& x, int64_t T, const W8& w0, const W8& w1, int64_t N,
                  int64_t K, int act, void* y, void* g, void* u, int out_dtype, void* workspace,
                  hipStream_t stream) {
  GemmArgs p{};
  if (x.dtype == kI8) {
    p.a = static_cast<const int8_t*>(x.x);
    p.xs = x.scales;
    p.xsum = x.sums;
  } else if (fused(T, K, x.dtype, GATED)) {
    p.x = static_cast<const uint16_t*>(x.x);
    p.x_bf16 = x.dtype == kBF16;
  } else {
    auto* ws = static_cast<uint8_t*>(workspace);
    auto* codes = reinterpret_cast<int8_t*>(ws);
    auto* xs = reinterpret_cast<float*>(ws + up256(T * K));
    auto* sums = reinterpret_cast<int32_t*>(ws + up256(T * K) + up256(T * 4));
    hipError_t e = launch_quantize_act(x.x, x.dtype, T, K, codes, xs, sums, stream);
    if (e != hipSuccess) return e;
    p.a = codes;
    p.xs = xs;
    p.xsum = sums;
  }
  p.w[0] = w0;
  p.w[1] = w1;
  p.y = y;
  p.g = g;
  p.u = u;
  p.T = (int)T;
  p.N = (int)N;
  p.K = (int)K;
  p.act = act;
  p.bf16 = out_dtype == kBF16;
  if (few_takes(T, K, GATED)) return launch_few(p, GATED, stream);
  const GemmPlan plan = gemm_plan(T, N, K, GATED, device_cu_count());
  if (plan.shape < 0) return launch_skinny(p, GATED, stream);
  auto* parts = reinterpret_cast<i4_t*>(static_cast<uint8_t*>(workspace) +
                                        (x.dtype == kI8 ? 0 : code_bytes(T, K)));
  switch (plan.shape) {
    case 0:
      return launch_tile<64, 128, 2, 4, 3, 2, GATED>(p, plan.tiles, parts, stream);
    case 1:
      return launch_tile<128, 128, 2, 4, 3, 2, GATED>(p, plan.tiles, parts, stream);
    case 2:
      return launch_tile<256, 128, 4, 2, 3, 2, GATED>(p, plan.tiles, parts, stream);
    case 3:
      return launch_tile<192, 192, 4, 2, 3, 2, GATED>(p, plan.tiles, parts, stream);
    case 4:
      return launch_tile<256, 192, 4, 2, 4, 1, GATED>(p, plan.tiles, parts, stream);
    case 5:
      return launch_tile<256, 256, 2, 4, 4, 1, GATED>(p, plan.tiles, parts, stream);
    default:
      return launch_tile<256, 384, 2, 4, 4, 1, GATED>(p, plan.tiles, parts, stream);
  }
}

}  // namespace

size_t w8a8_workspace_bytes(int64_t T, int64_t N, int64_t K, int dtype, bool gated) {
  if (T == 0 || N == 0) return 0;
  const size_t codes = dtype == kI8 || fused(T, K, dtype, gated) ? 0 : code_bytes(T, K);
  if (few_takes(T, K, gated)) return codes;
  return codes + gemm_plan(T, N, K, gated, device_cu_count()).part_bytes();
}

hipError_t launch_linear_w8a8(const Activations& x, int64_t T, const W8& w, int64_t N, int64_t K,
                              void* y, int out_dtype, void* workspace, hipStream_t stream) {
  return launch<false>(x, T, w, w, N, K, 0, y, nullptr, nullptr, out_dtype, workspace, stream);
}

hipError_t launch_gated_w8a8(const Activations& x, int64_t T, const W8& gate, const W8& up,
                             int64_t N, int64_t K, int act, void* h, void* g, void* u,
                             int out_dtype, void* workspace, hipStream_t stream) {
  return launch<true>(x, T, gate, up, N, K, act, h, g, u, out_dtype, workspace, stream);
}

}  // namespace lowbit
