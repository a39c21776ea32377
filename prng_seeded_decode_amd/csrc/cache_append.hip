// Rotary positions on q and k, and k and v written into their slots of a paged
// cache (seedlm_cache_append).
//
// A pair (a, b) of a head turns by its position's angle:
// (a cos - b sin, b cos + a sin), in fp32, rounded once to the output's type.
// Each element is read and written once with three flops, so memory bandwidth
// bounds the path.  A workgroup takes one token, whose slot and position are
// the same for all its lanes, and its lanes take (head, unit) pairs: a unit is
// 16 elements of a head, two 16-byte fp16 loads (the two halves of eight pairs)
// and two 16-byte stores, so that a wave covers whole lines.  The cosines and
// sines of a token (head_dim * 4 bytes) come from L1 after their first use.
// Shapes or addresses that rule 16-byte accesses out use units of one pair.
//
// Measured: 4097 tokens of 32 query and 32 cache heads of 128 dimensions, fp16 (203
// MB), in 38.4 us, 5.3 TB/s; 16 tokens of 64 and 8 heads in 2.8 us, a launch's time;
// 2048 tokens of 32 and 8 heads, fp32 (93 MB), in 18.2 us, 5.1 TB/s, and fp16 with 120
// of the 128 dimensions rotated, so by units of one pair (51 MB), in 24.6 us, 2.1 TB/s:
// their 2-byte accesses take 16 times the instructions.
#include "rotary.h"

namespace seedlm {
namespace {

constexpr int kThreads = 256;

struct AppendArgs {
  seedlm_cache_append_args a;
  int units;           // units of a head: head_dim / (2 N)
  int heads_per_pass;  // heads that a workgroup's lanes cover at once
};

// N pairs per unit: 8, or 1 for any shape and alignment.
template <int N, typename T>
__global__ __launch_bounds__(kThreads) void cache_append_kernel(const AppendArgs p) {
  const seedlm_cache_append_args& a = p.a;
  const int64_t t = blockIdx.x;
  const int unit = threadIdx.x % p.units, lane_head = threadIdx.x / p.units;
  if (lane_head >= p.heads_per_pass) return;
  const int D = a.cache.head_dim, kv = a.cache.kv_heads, all = a.heads + 2 * kv;
  const int pos = a.positions[t], slot = a.slots[t];
  const bool turns = pos >= 0 && pos < a.table_len;
  const bool keeps = turns && slot >= 0 && slot < a.cache.pages * a.cache.page_size;
  int64_t cache_at = 0;
  if (keeps) {
    const int page = slot / a.cache.page_size;
    cache_at = page * a.cache.page_stride +
               (slot - page * a.cache.page_size) * a.cache.token_stride;
  }
  // The unit's two runs of N elements: the halves of N rotated pairs, or (as
  // interleaved pairs and unrotated elements are) 2N in a row.
  const int e0 = unit * 2 * N;
  const bool rotated = e0 < a.rot;
  const bool split = rotated && !a.interleaved;
  const int lo = split ? unit * N : e0, hi = split ? lo + a.rot / 2 : e0 + N;
  float c[N], s[N];
  if (rotated && turns) {
    const int64_t at = (int64_t)pos * (a.rot / 2) + unit * N;
    load<N>(a.cos + at, c);
    load<N>(a.sin + at, s);
  }
  const int h = blockIdx.y * p.heads_per_pass + lane_head;
  if (h >= all) return;
  const bool is_q = h < a.heads, is_v = h >= a.heads + kv;
  if (!is_q && !keeps) return;
  const int hk = is_v ? h - a.heads - kv : h - a.heads;  // head of k or v
  const T* src = is_q ? static_cast<const T*>(a.q) + t * a.q_stride + h * D
                      : (is_v ? static_cast<const T*>(a.v) + t * a.v_stride + hk * D
                              : static_cast<const T*>(a.k) + t * a.k_stride + hk * D);
  float x[N], y[N];
  load<N>(src + lo, x);
  load<N>(src + hi, y);
  if (rotated && !is_v && turns) {
    if (split) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float u = x[i], w = y[i];
        x[i] = u * c[i] - w * s[i];
        y[i] = w * c[i] + u * s[i];
      }
    } else {
      // elements 2i, 2i + 1 of the 2N in a row
      float z[2 * N];
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = x[i], z[N + i] = y[i];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float u = z[2 * i], w = z[2 * i + 1];
        z[2 * i] = u * c[i] - w * s[i];
        z[2 * i + 1] = w * c[i] + u * s[i];
      }
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = z[i], y[i] = z[N + i];
    }
  }
  if (is_q) {
    T* dst = static_cast<T*>(a.q_out) + t * a.q_out_stride + h * D;
    if (!turns) {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = y[i] = 0.f;
    }
    store<N>(dst + lo, x);
    store<N>(dst + hi, y);
  } else {
    __half* dst = static_cast<__half*>(is_v ? a.cache.v : a.cache.k) + cache_at +
                  hk * a.cache.head_stride;
    store<N>(dst + lo, x);
    store<N>(dst + hi, y);
  }
}

// Whether every access of the 8-pair units is aligned to 16 bytes.
bool wide_units(const seedlm_cache_append_args& a) {
  const int64_t per = a.x_dtype == SEEDLM_F16 ? 8 : 4;  // elements of 16 bytes
  const seedlm_cache_t& c = a.cache;
  for (int64_t s : {a.q_stride, a.k_stride, a.v_stride, a.q_out_stride})
    if (s % per != 0) return false;
  for (int64_t s : {c.page_stride, c.token_stride, c.head_stride})
    if (s % 8 != 0) return false;
  for (const void* p : {a.q, a.k, a.v, (const void*)a.q_out, (const void*)a.cos,
                        (const void*)a.sin, (const void*)c.k, (const void*)c.v})
    if (!aligned16(p)) return false;
  return c.head_dim % 16 == 0 && a.rot % 16 == 0;
}

template <int N, typename T>
void launch(const seedlm_cache_append_args& a, hipStream_t s) {
  AppendArgs p{a, a.cache.head_dim / (2 * N), 0};
  p.heads_per_pass = kThreads / p.units;
  const int all = a.heads + 2 * a.cache.kv_heads;
  const int passes = (all + p.heads_per_pass - 1) / p.heads_per_pass;
  hipLaunchKernelGGL((cache_append_kernel<N, T>), dim3(a.tokens, passes), dim3(kThreads), 0, s, p);
}

}  // namespace

int launch_cache_append(const seedlm_cache_append_args& a, hipStream_t s) {
  const bool f16 = a.x_dtype == SEEDLM_F16;
  if (wide_units(a)) {
    if (f16) launch<8, __half>(a, s);
    else launch<8, float>(a, s);
  } else {
    if (f16) launch<1, __half>(a, s);
    else launch<1, float>(a, s);
  }
  return hipGetLastError() == hipSuccess ? SEEDLM_OK : SEEDLM_E_DEVICE;
}

}  // namespace seedlm
