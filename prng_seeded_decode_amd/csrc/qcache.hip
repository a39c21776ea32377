// A quantised cache: rotary positions on q and k with k and v quantised into their
// slots (seedlm_qcache_append), and slots read back (seedlm_qcache_read).
//
// A group of x of a row gets offset o = min x, scale s = fp16((max x - o) / levels) and
// codes c = rint((x - o) / s); it reads back as o + s c.  The x are fp16 numbers, so o
// is exact.  Each element is read and written once, so memory bandwidth bounds both.
#include <hip/hip_fp16.h>

#include "seedlm_internal.h"

namespace seedlm {
namespace {

constexpr int kThreads = 256;

// Element d of a row: its unit, its place in the unit.
__device__ int byte_of(int d, int dim, int bits) { return ((d % 16) * (dim / 16) + d / 16) * bits / 8; }

// Element e of a head at `x` turned by a token's cosines and sines, each operation
// rounded: codes next to a border must not depend on how the compiler joins them.
template <typename T>
__device__ float turned(const T* x, int e, int rot, bool interleaved, const float* cos,
                        const float* sin) {
#pragma clang fp contract(off)
  if (e >= rot) return (float)x[e];
  const int half = rot / 2;
  const int pair = interleaved ? e / 2 : e % half;
  const bool second = interleaved ? e % 2 : e >= half;
  const float a = (float)x[interleaved ? 2 * pair : pair];
  const float b = (float)x[interleaved ? 2 * pair + 1 : pair + half];
  const float c = cos[pair], s = sin[pair];
  return second ? b * c + a * s : a * c - b * s;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void qcache_append_kernel(const seedlm_qcache_append_args a) {
  const int64_t t = blockIdx.x;
  const seedlm_qcache_t& c = a.cache;
  const int D = c.head_dim, groups = D / c.group;
  const int pos = a.positions[t], slot = a.slots[t];
  const bool turns = pos >= 0 && pos < a.table_len;
  const float* cos = a.cos + (turns ? (int64_t)pos * (a.rot / 2) : 0);
  const float* sin = a.sin + (turns ? (int64_t)pos * (a.rot / 2) : 0);
  // every thread keeps its head's unrotated elements until all have been read (q_out
  // may be q), so a head is a workgroup's turn
  for (int h = 0; h < a.heads; ++h) {
    const T* q = static_cast<const T*>(a.q) + t * a.q_stride + (int64_t)h * D;
    T* out = static_cast<T*>(a.q_out) + t * a.q_out_stride + (int64_t)h * D;
    const int e = threadIdx.x;
    float x = 0.f;
    if (e < D && turns) x = turned(q, e, a.rot, a.interleaved, cos, sin);
    __syncthreads();
    if (e < D) out[e] = (T)x;
  }
  if (!turns || slot < 0 || slot >= c.pages * c.page_size) return;
  const int page = slot / c.page_size, nth = slot % c.page_size;
  const float levels = (float)((1 << c.bits) - 1);
  for (int i = threadIdx.x; i < 2 * c.kv_heads * groups; i += kThreads) {
    const int g = i % groups, h = i / groups % c.kv_heads;
    const bool is_v = i >= c.kv_heads * groups;
    const T* src = (is_v ? static_cast<const T*>(a.v) + t * a.v_stride
                         : static_cast<const T*>(a.k) + t * a.k_stride) + (int64_t)h * D;
    const int rot = is_v ? 0 : a.rot;
    auto value = [&](int e) { return (float)(_Float16)turned(src, e, rot, a.interleaved, cos, sin); };
    float low = INFINITY, high = -INFINITY, sum = 0.f;
    for (int e = g * c.group; e < (g + 1) * c.group; ++e) {
      const float x = value(e);
      low = fminf(low, x), high = fmaxf(high, x), sum += x * 0.f;
    }
    const bool finite = sum == 0.f;
    const _Float16 scale = finite ? (_Float16)((high - low) / levels) : (_Float16)NAN;
    const float s = (float)scale;
    auto code = [&](int e) -> uint32_t {
      return finite && s > 0.f ? (uint32_t)fminf(rintf((value(e) - low) / s), levels) : 0;
    };
    uint8_t* row = static_cast<uint8_t*>(is_v ? c.v : c.k) + page * c.page_stride +
                   nth * c.token_stride + h * c.head_stride;
    for (int e = g * c.group; e < (g + 1) * c.group; ++e) {
      if (c.bits == 8) row[byte_of(e, D, 8)] = (uint8_t)code(e);
      else if (e / 16 % 2 == 0) row[byte_of(e, D, 4)] = (uint8_t)(code(e) | code(e + 16) << 4);
    }
    _Float16* pair = static_cast<_Float16*>(is_v ? c.v_scale : c.k_scale) +
                     2 * (page * c.scale_page_stride + nth * c.scale_token_stride +
                          h * c.scale_head_stride + g);
    pair[0] = scale;
    pair[1] = finite ? (_Float16)low : (_Float16)0.f;
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void qcache_read_kernel(const seedlm_qcache_read_args a) {
  const int64_t t = blockIdx.x;
  const seedlm_qcache_t& c = a.cache;
  const int D = c.head_dim, slot = a.slots[t];
  const bool live = slot >= 0 && slot < c.pages * c.page_size;
  const int page = live ? slot / c.page_size : 0, nth = live ? slot % c.page_size : 0;
  for (int i = threadIdx.x; i < 2 * c.kv_heads * D; i += kThreads) {
    const int e = i % D, h = i / D % c.kv_heads;
    const bool is_v = i >= c.kv_heads * D;
    T* out = static_cast<T*>(is_v ? a.v_out : a.k_out);
    if (!out) continue;
    float x = 0.f;
    if (live) {
      const uint8_t* row = static_cast<const uint8_t*>(is_v ? c.v : c.k) + page * c.page_stride +
                           nth * c.token_stride + h * c.head_stride;
      const _Float16* pair = static_cast<const _Float16*>(is_v ? c.v_scale : c.k_scale) +
                             2 * (page * c.scale_page_stride + nth * c.scale_token_stride +
                                  h * c.scale_head_stride + e / c.group);
      const uint32_t byte = row[byte_of(e, D, c.bits)];
      const uint32_t code = c.bits == 8 ? byte : byte >> (e / 16 % 2 * 4) & 15;
      x = (float)pair[1] + (float)pair[0] * (float)code;
    }
    out[t * (is_v ? a.v_stride : a.k_stride) + (int64_t)h * D + e] = (T)x;
  }
}

}  // namespace

int launch_qcache_append(const seedlm_qcache_append_args& a, hipStream_t s) {
  const auto kernel = a.x_dtype == SEEDLM_F16 ? qcache_append_kernel<__half> : qcache_append_kernel<float>;
  hipLaunchKernelGGL(kernel, dim3(a.tokens), dim3(kThreads), 0, s, a);
  return hipGetLastError() == hipSuccess ? SEEDLM_OK : SEEDLM_E_DEVICE;
}

int launch_qcache_read(const seedlm_qcache_read_args& a, hipStream_t s) {
  const auto kernel = a.y_dtype == SEEDLM_F16 ? qcache_read_kernel<__half> : qcache_read_kernel<float>;
  hipLaunchKernelGGL(kernel, dim3(a.tokens), dim3(kThreads), 0, s, a);
  return hipGetLastError() == hipSuccess ? SEEDLM_OK : SEEDLM_E_DEVICE;
}

}  // namespace seedlm
