// One serving step's bookkeeping of a paged cache (seedlm_cache_plan): pages
// for new tokens, pages of finished requests back to the queue, and the row,
// position and slot of every new token.
//
// With n_b new tokens of request b, its held pages h_b = ceil(len_b / S) and
// its need w_b = ceil((len_b + n_b) / S) - h_b, everything follows from three
// prefix sums over the requests: of n_b (where tokens start), of w_b (which
// queue entries are a request's) and of the h_b of finished requests (where
// their pages join the queue).  A request is granted its pages if its inclusive
// sum of w is at most the queue's count; the sum never falls, so the granted
// requests with w > 0 take one contiguous run of the queue.
//
// The path is bound by latency, not bytes (a step of 16 requests moves under a
// kilobyte and takes 3.8 us, one of 1000 requests and 80,000 token entries 7.9 us for
// 1.03 MB), so it is one launch: every workgroup forms the prefix sums of all
// requests again (at most kMaxRequests, 8 per thread, out of L2) and then
// handles its share of the pages and tokens, each finding its request by
// bisection in LDS.  No workgroup depends on another's writes: popped queue
// entries are read from the queue itself, not from the table, and pages that
// join the queue lie outside the entries that are popped.  Workgroup 0 writes
// the per-request outputs.
#include "seedlm_internal.h"

namespace seedlm {
namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxRequests = SEEDLM_MAX_REQUESTS;
constexpr int kPerThread = kMaxRequests / kThreads;

struct PlanArgs {
  seedlm_cache_plan_args a;
  int32_t* lens_dst;   // lens_out, or scratch that a copy follows
  int32_t* state_dst;  // ring_state_out, likewise
};

// Sums saturate at 2^32 - 1, past every bound they are compared with (saturating
// sums of counts are still associative, but cannot be taken apart again).
__device__ uint32_t add(uint32_t a, uint32_t b) { return __builtin_elementwise_add_sat(a, b); }

template <int kCtrl, int kRows>
__device__ uint32_t add_dpp(uint32_t v) {
  return add(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, kRows, 0xF, false));
}

// Inclusive sum over the wave's lanes: within rows of 16, then across them.
__device__ uint32_t wave_scan(uint32_t v) {
  v = add_dpp<0x111, 0xF>(v);  // row_shr:1, 2, 4, 8
  v = add_dpp<0x112, 0xF>(v);
  v = add_dpp<0x114, 0xF>(v);
  v = add_dpp<0x118, 0xF>(v);
  v = add_dpp<0x142, 0xA>(v);  // row_bcast:15
  return add_dpp<0x143, 0xC>(v);  // row_bcast:31
}

// Sums of N values over the threads before this one (v), in thread order, and over
// all of them (total).  lds is free on entry and may be used again after the next
// barrier.
template <int N>
__device__ void block_scan(uint32_t (&v)[N], uint32_t (*lds)[N], uint32_t (&total)[N]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const uint32_t upto = wave_scan(v[k]);
    if (lane == 63) lds[wave][k] = upto;
    v[k] = __shfl_up(upto, 1);
    if (lane == 0) v[k] = 0;
    total[k] = 0;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    uint32_t before = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const uint32_t s = lds[w][k];
      if (w == wave) before = total[k];
      total[k] = add(total[k], s);
    }
    v[k] = add(v[k], before);
  }
}

// The first i of [0, n) with ends[i] > x (n if none); ends never falls.
__device__ int first_above(const int32_t* ends, int n, int32_t x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ends[mid] > x) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// ceil(len / S) and the queue index i places behind `at` (i < pool), whose sums
// may pass 2^31 but not 2^32.
__device__ int pages_of(int len, int S) {
  return (int)(((uint32_t)len + (uint32_t)S - 1u) / (uint32_t)S);
}
__device__ uint32_t ring_at(int at, int i, int pool) {
  const uint32_t x = (uint32_t)at + (uint32_t)i;
  return x >= (uint32_t)pool ? x - (uint32_t)pool : x;
}

__device__ int32_t saturate(uint32_t v) { return v > INT32_MAX ? INT32_MAX : (int32_t)v; }

__global__ __launch_bounds__(kThreads) void cache_plan_kernel(const PlanArgs p) {
  // Inclusive ends of each request's new tokens, new pages and returned pages
  // (saturated: ends past the arrays are never looked for), its length and ok.
  __shared__ int32_t s_tok[kMaxRequests], s_need[kMaxRequests], s_back[kMaxRequests];
  __shared__ int32_t s_len[kMaxRequests];
  __shared__ uint8_t s_ok[kMaxRequests];
  __shared__ uint32_t s_first[kWaves][2], s_second[kWaves][1];
  __shared__ int s_taken;
  const seedlm_cache_plan_args& a = p.a;
  const int n = a.requests, S = a.page_size, tid = threadIdx.x;
  const int64_t cap = (int64_t)a.max_pages * S;
  const int per = (n + kThreads - 1) / kThreads;  // consecutive requests of a thread
  // The queue as found, taken into its ranges.
  const int pool = a.pool;
  int head = a.ring_state[0] % pool;
  if (head < 0) head += pool;
  const int count = min(max(a.ring_state[1], 0), pool);
  const int tail = (int)ring_at(head, count, pool);
  if (tid == 0) s_taken = 0;

  // First sums: tokens and returned pages.
  int len[kPerThread], fresh[kPerThread];
  uint32_t mine[2] = {0, 0};  // new tokens, returned pages
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    if (i >= per) break;
    const int b = tid * per + i;
    len[i] = fresh[i] = 0;
    if (b < n) {
      len[i] = (int)min<int64_t>(max(a.lens[b], 0), cap);
      fresh[i] = a.fresh[b];
    }
    mine[0] = add(mine[0], (uint32_t)max(fresh[i], 0));
    if (fresh[i] < 0) mine[1] = add(mine[1], (uint32_t)pages_of(len[i], S));
  }
  uint32_t total[2];
  block_scan(mine, s_first, total);
  // Second sum: pages needed by the requests whose tokens fit.
  int need[kPerThread];
  uint32_t wanted[1] = {0};
  uint32_t end = mine[0], back = mine[1];
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    if (i >= per) break;
    const int b = tid * per + i;
    const int held = pages_of(len[i], S);
    const int64_t grown = (int64_t)len[i] + max(fresh[i], 0);
    end = add(end, (uint32_t)max(fresh[i], 0));
    const bool fits = fresh[i] >= 0 && grown <= cap && end <= (uint32_t)a.tokens;
    need[i] = fits ? pages_of((int)grown, S) - held : (fresh[i] < 0 ? 0 : -1);
    wanted[0] = add(wanted[0], (uint32_t)max(need[i], 0));
    if (fresh[i] < 0) back = add(back, (uint32_t)held);
    if (b < n) {
      s_tok[b] = saturate(end);
      s_back[b] = saturate(back);
      s_len[b] = len[i];
    }
  }
  uint32_t all_wanted[1];
  block_scan(wanted, s_second, all_wanted);
  uint32_t cum = wanted[0];
  int taken = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    if (i >= per) break;
    const int b = tid * per + i;
    if (b >= n) break;
    cum = add(cum, (uint32_t)max(need[i], 0));
    const bool ok = need[i] == 0 || (need[i] > 0 && cum <= (uint32_t)count);
    if (ok && need[i] > 0) taken = (int)cum;
    s_need[b] = saturate(cum);
    s_ok[b] = ok;
    if (blockIdx.x == 0) {
      a.ok[b] = ok;
      a.offsets[b + 1] = s_tok[b];
      p.lens_dst[b] = fresh[i] < 0 ? 0 : (ok ? len[i] + fresh[i] : len[i]);
    }
  }
  if (taken > 0) atomicMax(&s_taken, taken);
  __syncthreads();
  taken = s_taken;
  // Pages that come back find room: pool - count entries are free of any page
  // in the queue (more than that come back only if the inputs were wrong).
  const int returned = (int)min(total[1], (uint32_t)(pool - count));
  if (blockIdx.x == 0 && tid == 0) {
    a.offsets[0] = 0;
    p.state_dst[0] = (int)ring_at(head, taken, pool);
    p.state_dst[1] = count - taken + returned;
  }
  const int first = blockIdx.x * kThreads + tid, step = gridDim.x * kThreads;
  for (int i = first; i < taken; i += step) {
    const int b = first_above(s_need, n, i);
    const int held = pages_of(s_len[b], S);
    const int nth = i - (b > 0 ? s_need[b - 1] : 0);
    a.table[b * a.table_stride + held + nth] = a.ring[ring_at(head, i, pool)];
  }
  for (int i = first; i < returned; i += step) {
    const int b = first_above(s_back, n, i);
    const int nth = i - (b > 0 ? s_back[b - 1] : 0);
    a.ring[ring_at(tail, i, pool)] = a.table[b * a.table_stride + nth];
  }
  const int live = min(s_tok[n - 1], a.tokens);
  for (int t = first; t < a.tokens; t += step) {
    int row = -1, pos = 0, slot = -1;
    if (t < live) {
      row = first_above(s_tok, n, t);
      const int len_b = s_len[row];
      pos = len_b + t - (row > 0 ? s_tok[row - 1] : 0);
      if (s_ok[row]) {
        const int page_nr = pos / S, held = pages_of(len_b, S);
        const int before = row > 0 ? s_need[row - 1] : 0;
        const int page = page_nr < held
                             ? a.table[row * a.table_stride + page_nr]
                             : a.ring[ring_at(head, before + page_nr - held, pool)];
        // a page outside the cache, in a table or queue that was wrong, has no slots
        if (page >= 0 && page < pool) slot = page * S + pos % S;
      }
    }
    a.rows[t] = row;
    a.positions[t] = pos;
    a.slots[t] = slot;
    if (a.spans) a.spans[t] = slot >= 0 ? pos + 1 : 0;
  }
}

__global__ __launch_bounds__(256) void copy_plan_kernel(const int32_t* __restrict__ src,
                                                        int32_t* __restrict__ lens, int n,
                                                        int32_t* __restrict__ state) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < n) lens[i] = src[i];
  if (i < 2) state[i] = src[n + i];
}

// Workgroups of a call: a token per thread, since a thread's tokens would wait for
// one another's bisection and page number (80,000 tokens: 7.3 us a call, 12 with four
// tokens each), up to two workgroups per compute unit.
int plan_grid(const seedlm_cache_plan_args& a) {
  const int g = (a.tokens + kThreads - 1) / kThreads;
  const int most = 2 * device_cu_count();
  return g < 1 ? 1 : (g > most ? most : g);
}

}  // namespace

// Outputs on top of their own inputs are safe inside one workgroup, which reads
// all of them before it writes; several workgroups write to scratch first.
size_t cache_plan_scratch_bytes(const seedlm_cache_plan_args& a) {
  const bool in_place = a.lens_out == a.lens || a.ring_state_out == a.ring_state;
  return in_place && plan_grid(a) > 1 ? ((size_t)a.requests + 2) * sizeof(int32_t) : 0;
}

int launch_cache_plan(const seedlm_cache_plan_args& a, int32_t* scratch, hipStream_t s) {
  PlanArgs p{a, a.lens_out, a.ring_state_out};
  if (scratch) {
    p.lens_dst = scratch;
    p.state_dst = scratch + a.requests;
  }
  hipLaunchKernelGGL(cache_plan_kernel, dim3(plan_grid(a)), dim3(kThreads), 0, s, p);
  if (scratch)
    hipLaunchKernelGGL(copy_plan_kernel, dim3((a.requests + 255) / 256), dim3(256), 0, s, scratch,
                       a.lens_out, a.requests, a.ring_state_out);
  return hipGetLastError() == hipSuccess ? SEEDLM_OK : SEEDLM_E_DEVICE;
}

}  // namespace seedlm
