// What the attention kernels share: how the work of requests of any lengths is cut
// into even runs of units.
#pragma once

#include "divisor.h"
#include "seedlm_internal.h"

namespace seedlm {

// The first unit of a slot among `units`, and the slot of a unit: the largest i
// with i * units / slots <= u, that is i * units < (u + 1) * slots.
// (A 64-bit division takes half a microsecond, so it is left to the largest numbers.)
__host__ __device__ inline int slot_begin(int slot, int units, int slots) {
  const uint64_t x = (uint64_t)slot * (uint32_t)units;
  if (x >> 32 == 0) return (int)((uint32_t)x / (uint32_t)slots);
  return (int)(x / (uint32_t)slots);
}
__host__ __device__ inline int slot_of(int u, int units, int slots) {
  const uint64_t x = ((uint64_t)u + 1) * (uint32_t)slots - 1;
  if (x >> 32 == 0) return (int)((uint32_t)x / (uint32_t)units);
  return (int)(x / (uint32_t)units);
}

// The same with runs of several lengths: GENS workgroups of a compute unit run side by
// side, and those that started first get the larger part of its loads, so of GENS equal
// parts of the slots (workgroups start in the order of their numbers) each has longer
// runs than the next.  Where units are few all runs are even.
template <int GENS>
struct Runs {
  int units, slots, per;  // per: slots of a generation, the last one's but at least

  __host__ __device__ Runs(int most, int u) : units(u), slots(most < u ? most : u) {
    per = GENS > 1 && units >= 3 * slots ? slots / GENS : slots;
  }
  __host__ __device__ static constexpr int weight(int gen) {
    return GENS == 1 ? 1 : (GENS == 2 ? 3 - gen : 4 - gen);  // 3 : 2, 4 : 3 : 2
  }
  // The weights of the slots before `slot`.
  __host__ __device__ int before(int slot) const {
    int sum = 0;
#pragma unroll
    for (int g = 0; g < GENS; ++g) {
      const int left = slot - g * per, n = g + 1 < GENS && left > per ? per : left;
      if (n > 0) sum += n * weight(g);
    }
    return sum;
  }
  __host__ __device__ int begin(int slot) const { return slot_begin(before(slot), units, before(slots)); }
  __host__ __device__ int slot_of(int u) const {
    int x = seedlm::slot_of(u, units, before(slots)), slot = 0;
#pragma unroll
    for (int g = 0; g < GENS; ++g) {
      const bool last = g + 1 == GENS || x < per * weight(g);
      slot += last ? x / weight(g) : per;
      if (last) break;
      x -= per * weight(g);
    }
    return slot < slots ? slot : slots - 1;
  }
};

// Inclusive sums of units_of(0), ..., units_of(n - 1) into ends[0..n), by all
// THREADS threads, each taking consecutive numbers.
template <int THREADS, typename F>
__device__ void sum_units(int n, int32_t* ends, F units_of) {
  __shared__ int s_wave[THREADS / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int per = (n + THREADS - 1) / THREADS;
  const int b0 = min((int)threadIdx.x * per, n), b1 = min(b0 + per, n);
  int mine = 0;
  for (int b = b0; b < b1; ++b) {
    mine += units_of(b);
    ends[b] = mine;
  }
  int upto = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 63) s_wave[wave] = upto;
  __syncthreads();
  int before = upto - mine;
  for (int w = 0; w < wave; ++w) before += s_wave[w];
  for (int b = b0; b < b1; ++b) ends[b] += before;
  __syncthreads();
}

// x plus those of all lower lanes of the wave.
__device__ inline int wave_sums(int x) {
#define SEEDLM_ADD_DPP(ctrl, rows) x += __builtin_amdgcn_update_dpp(0, x, ctrl, rows, 0xF, false)
  SEEDLM_ADD_DPP(0x111, 0xF);  // the lane 1, 2, 4 and 8 before in the same 16
  SEEDLM_ADD_DPP(0x112, 0xF);
  SEEDLM_ADD_DPP(0x114, 0xF);
  SEEDLM_ADD_DPP(0x118, 0xF);
  SEEDLM_ADD_DPP(0x142, 0xA);  // the last lane of the 16 before, into the second and fourth 16
  SEEDLM_ADD_DPP(0x143, 0xC);  // the last lane of the first half, into the second
#undef SEEDLM_ADD_DPP
  return x;
}

// The first request whose inclusive sum exceeds u.
__device__ inline int request_of(const int32_t* ends, int n, int u) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ends[mid] > u) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

}  // namespace seedlm
