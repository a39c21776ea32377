// Attention of query tokens over their requests' pages of a quantised cache
// (seedlm_qcache_attend): out = sum_t softmax_t(scale q . k_t) v_t.
//
// A workgroup takes one query and head.  Its threads score 256 tokens at a time, a
// token each, and then sum the values by dimension under a running maximum.
#include <hip/hip_fp16.h>

#include "seedlm_internal.h"

namespace seedlm {
namespace {

constexpr int kThreads = 256;

__device__ float element(const uint8_t* row, const _Float16* pair, int e, const seedlm_qcache_t& c) {
  const int at = (e % 16) * (c.head_dim / 16) + e / 16;
  const uint32_t code = c.bits == 8 ? row[at] : row[at / 2] >> (at % 2 * 4) & 15;
  const _Float16* so = pair + 2 * (e / c.group);
  return (float)so[1] + (float)so[0] * (float)code;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void qcache_attend_kernel(const seedlm_qcache_attend_args a,
                                                                 int cap) {
  __shared__ float s_x[kThreads];
  __shared__ int64_t s_row[kThreads], s_pair[kThreads];
  const seedlm_qcache_t& c = a.cache;
  const int b = blockIdx.y, head = blockIdx.x, D = c.head_dim, i = threadIdx.x;
  const int hk = head / (a.heads / c.kv_heads);
  const int row = a.rows ? a.rows[b] : b;
  const int len = (uint32_t)row < (uint32_t)a.table_rows ? min(max(a.lens[b], 0), cap) : 0;
  const T* q = static_cast<const T*>(a.q) + b * a.q_stride + (int64_t)head * D;
  float top = -INFINITY, sum = 0.f, acc = 0.f;
  for (int t0 = 0; t0 < len; t0 += kThreads) {
    const int t = t0 + i;
    int page = -1;
    if (t < len) page = a.table[(int64_t)row * a.table_stride + t / c.page_size];
    const bool live = page >= 0 && page < c.pages;
    s_row[i] = s_pair[i] = -1;
    float x = -INFINITY;
    if (live) {
      const int nth = t % c.page_size;
      s_row[i] = page * c.page_stride + nth * c.token_stride + hk * c.head_stride;
      s_pair[i] = 2 * (page * c.scale_page_stride + nth * c.scale_token_stride + hk * c.scale_head_stride);
      x = 0.f;
      for (int e = 0; e < D; ++e)
        x += (float)q[e] * element(static_cast<const uint8_t*>(c.k) + s_row[i],
                                   static_cast<const _Float16*>(c.k_scale) + s_pair[i], e, c);
      x *= a.scale;
    }
    s_x[i] = x;
    __syncthreads();
    float up = top;
    bool nan = false;
    for (int j = 0; j < kThreads; ++j) up = fmaxf(up, s_x[j]), nan = nan || s_x[j] != s_x[j];
    if (nan) up = NAN;
    const float shrink = up == -INFINITY ? 0.f : expf(top - up);
    top = up;
    float part = 0.f, part_acc = 0.f;  // sums of a tile first: fewer roundings beside a heavy token
    for (int j = 0; j < kThreads; ++j) {
      if (s_row[j] < 0) continue;
      const float p = expf(s_x[j] - top);
      part += p;
      if (i < D)
        part_acc += p * element(static_cast<const uint8_t*>(c.v) + s_row[j],
                           static_cast<const _Float16*>(c.v_scale) + s_pair[j], i, c);
    }
    sum = sum * shrink + part, acc = acc * shrink + part_acc;
    __syncthreads();
  }
  if (i < D)
    static_cast<T*>(a.out)[b * a.out_stride + (int64_t)head * D + i] = (T)(sum == 0.f ? 0.f : acc / sum);
}

}  // namespace

size_t qcache_attend_scratch_bytes(const seedlm_qcache_attend_args&) { return 0; }

int launch_qcache_attend(const seedlm_qcache_attend_args& a, void*, hipStream_t s) {
  const int64_t room = (int64_t)a.max_pages * a.cache.page_size;
  const int cap = (int)(a.max_len < room ? a.max_len : room);
  const auto kernel = a.x_dtype == SEEDLM_F16 ? qcache_attend_kernel<__half> : qcache_attend_kernel<float>;
  hipLaunchKernelGGL(kernel, dim3(a.heads, a.queries), dim3(kThreads), 0, s, a, cap);
  return hipGetLastError() == hipSuccess ? SEEDLM_OK : SEEDLM_E_DEVICE;
}

}  // namespace seedlm
