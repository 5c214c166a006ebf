// lora_plan.hip -- the tokens of a batch sorted by adapter: a stable counting sort
// in one workgroup.
//
// Each wave owns a run of tokens and counts its own adapters in LDS; a scan over
// (adapter, wave) turns the counts into places, and a second pass hands the places
// out.  Among 64 tokens, a token's rank within its adapter is the number of lanes
// before it with the same id: one ballot for each bit of the id, so the work does not
// depend on how many adapters meet.  No order depends on timing: the places of a
// wave's run are its own.  4 bytes read (twice) and 4 written a token; bound by the
// latency of one workgroup's passes: 3.7 us for 64 tokens, 12.8 for 16384 in prompts (20.5
// before prompts went without ballots), 16.6 for 16384 one by one.
#include "lora.h"

namespace lowbit {
namespace {

constexpr int kPlanWaves = 16;

__global__ __launch_bounds__(kPlanWaves * 64) void lora_plan_kernel(
    const int32_t* __restrict__ ids, int64_t T, int L, int bits, int32_t* __restrict__ order,
    int32_t* __restrict__ starts) {
  extern __shared__ int place[];  // [kPlanWaves][L + 1]: counts, then next places
  __shared__ int wave_total[kPlanWaves], nobody[kPlanWaves][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_of_group(), keys = L + 1;
  for (int i = tid; i < kPlanWaves * keys; i += kPlanWaves * 64) place[i] = 0;
  __syncthreads();
  const int64_t run = (T + kPlanWaves * 64 - 1) / (kPlanWaves * 64) * 64;
  const int64_t t0 = wave * run, t1 = min(T, t0 + run);
  int* const mine = place + wave * keys;
  // lanes with this lane's id, of the lanes that have a token
  auto same_ids = [&](int key, bool has) {
    uint64_t same = __ballot(has);
    // most steps are one request's prompt
    if (__ballot(has && key != __builtin_amdgcn_readfirstlane(key)) == 0) return has ? same : 0;
    for (int b = 0; b < bits; b++) {
      const uint64_t ones = __ballot((key >> b) & 1);
      same &= (key >> b) & 1 ? ones : ~ones;
    }
    return same;
  };
  auto key_of = [&](int64_t t) {  // the last token's again beyond the run: no condition on a load
    const int id = ids[min(t, T - 1)];
    return (uint32_t)id < (uint32_t)L ? id : L;
  };
  const uint64_t below = ((uint64_t)1 << lane) - 1;
  // eight steps' ids are under way at a time
  constexpr int kAhead = 8;
  for (int64_t t = t0; t < t1; t += 64 * kAhead) {
    int key[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; i++) key[i] = key_of(t + i * 64 + lane);
#pragma unroll
    for (int i = 0; i < kAhead; i++) {
      if (t + i * 64 >= t1) break;
      const bool has = t + i * 64 + lane < t1;
      // additions to one place come one after the other: one for all of a prompt's
      const bool one = __ballot(has && key[i] != __builtin_amdgcn_readfirstlane(key[i])) == 0;
      const int n = one ? (int)__popcll(__ballot(has)) : 1;
      if (one ? lane == 0 : has) atomicAdd(&mine[key[i]], n);
    }
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
  // An adapter's first lane of 64 takes the places of all; the other lanes' additions go to
  // nobody, so that eight steps' may be under way.
  for (int64_t t = t0; t < t1; t += 64 * kAhead) {
    int key[kAhead], at[kAhead];
    uint64_t same[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; i++) key[i] = key_of(t + i * 64 + lane);
#pragma unroll
    for (int i = 0; i < kAhead; i++) {
      if (t + i * 64 >= t1) break;
      same[i] = same_ids(key[i], t + i * 64 + lane < t1);
      const bool first_of = (same[i] >> lane & 1) && !(same[i] & below);
      at[i] = atomicAdd(first_of ? &mine[key[i]] : &nobody[wave][lane], (int)__popcll(same[i]));
    }
#pragma unroll
    for (int i = 0; i < kAhead; i++) {
      if (t + i * 64 >= t1) break;
      const int first_of = same[i] ? __ffsll((unsigned long long)same[i]) - 1 : 0;
      const int from = __shfl(at[i], first_of, kWave);
      if (t + i * 64 + lane < t1)
        order[from + (int)__popcll(same[i] & below)] = (int32_t)(t + i * 64 + lane);
    }
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
