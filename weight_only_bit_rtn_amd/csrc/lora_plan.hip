// lora_plan.hip -- the tokens of a batch sorted by adapter: a stable counting sort
// in one workgroup.
//
// Each wave owns a run of tokens and counts its own adapters in LDS; a scan over
// (adapter, wave) turns the counts into places, and a second pass hands the places
// out.  Among 64 tokens, a token's rank within its adapter is the number of lanes
// before it with the same id: one ballot for each bit of the id, so the work does not
// depend on how many adapters meet.  No order depends on timing: the places of a
// wave's run are its own.  4 bytes read (twice) and 4 written a token; bound by the
// latency of one workgroup's passes.
#include "lora.h"

namespace lowbit {
namespace {

constexpr int kPlanWaves = 16;

__global__ __launch_bounds__(kPlanWaves * 64) void lora_plan_kernel(
    const int32_t* __restrict__ ids, int64_t T, int L, int bits, int32_t* __restrict__ order,
    int32_t* __restrict__ starts) {
  extern __shared__ int place[];  // [kPlanWaves][L + 1]: counts, then next places
  __shared__ int wave_total[kPlanWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, keys = L + 1;
  for (int i = tid; i < kPlanWaves * keys; i += kPlanWaves * 64) place[i] = 0;
  __syncthreads();
  const int64_t run = (T + kPlanWaves * 64 - 1) / (kPlanWaves * 64) * 64;
  const int64_t t0 = wave * run, t1 = min(T, t0 + run);
  int* const mine = place + wave * keys;
  // lanes with this lane's id, of the lanes that have a token
  auto same_ids = [&](int key, bool has) {
    uint64_t same = __ballot(has);
    for (int b = 0; b < bits; b++) {
      const uint64_t ones = __ballot((key >> b) & 1);
      same &= (key >> b) & 1 ? ones : ~ones;
    }
    return same;
  };
  auto key_of = [&](int64_t t) {
    if (t >= t1) return L;
    const int id = ids[t];
    return id >= 0 && id < L ? id : L;
  };
  const uint64_t below = ((uint64_t)1 << lane) - 1;
  for (int64_t t = t0; t < t1; t += 64) {
    const bool has = t + lane < t1;
    const int key = key_of(t + lane);
    const uint64_t same = same_ids(key, has);
    if (has && !(same & below)) mine[key] += __popcll(same);
  }
  __syncthreads();
  // places: all of an adapter's tokens before the next one's, wave by wave
  int total = 0;
  if (tid < L)
    for (int w = 0; w < kPlanWaves; w++) total += place[w * keys + tid];
  int sum = total;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int other = __shfl_up(sum, off, kWave);
    if (lane >= off) sum += other;
  }
  if (lane == 63) wave_total[wave] = sum;
  __syncthreads();
  int first = sum - total, all = 0;
  for (int w = 0; w < kPlanWaves; w++) {
    if (w < wave) first += wave_total[w];
    all += wave_total[w];
  }
  if (tid < L) starts[tid] = first;
  if (tid == 0) starts[L] = all;
  // the key L is nobody's thread where L fills the workgroup: thread 0 takes it besides
  auto hand_out = [&](int key, int from) {
    for (int w = 0; w < kPlanWaves; w++) {
      const int n = place[w * keys + key];
      place[w * keys + key] = from;
      from += n;
    }
  };
  if (tid < L) hand_out(tid, first);
  if (tid == 0) hand_out(L, all);
  __syncthreads();
  for (int64_t t = t0; t < t1; t += 64) {
    const bool has = t + lane < t1;
    const int key = key_of(t + lane);
    const uint64_t same = same_ids(key, has);
    const int leader = same ? __ffsll((unsigned long long)same) - 1 : 0;
    int at = 0;
    if (has && lane == leader) at = atomicAdd(&mine[key], (int)__popcll(same));
    at = __shfl(at, leader, kWave) + (int)__popcll(same & below);
    if (has) order[at] = (int32_t)(t + lane);
  }
}

}  // namespace

hipError_t launch_lora_plan(const int32_t* ids, int64_t T, int64_t L, int32_t* order,
                            int32_t* starts, hipStream_t stream) {
  int bits = 1;
  while ((1 << bits) <= L) bits++;
  const int lds = (int)(kPlanWaves * (L + 1) * sizeof(int));
  constexpr int kMostLds = kPlanWaves * (kPlanWaves * 64 + 1) * (int)sizeof(int);
  const hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(&lora_plan_kernel), kMostLds);
  if (e != hipSuccess) return e;
  lora_plan_kernel<<<1, kPlanWaves * 64, lds, stream>>>(ids, T, (int)L, bits, order, starts);
  return hipGetLastError();
}

}  // namespace lowbit
