// Argument checks that the serving entry points share (seedlm_serve.h).
#pragma once

#include "seedlm_internal.h"

namespace seedlm {

inline bool dtype_ok(int d) { return d == SEEDLM_F32 || d == SEEDLM_F16; }
inline int64_t dtype_bytes(int d) { return d == SEEDLM_F32 ? 4 : 2; }
inline bool aligned(const void* p, uintptr_t n) { return (uintptr_t)p % n == 0; }

// Scratch of `bytes` bytes on `s` (NULL for none), held for the call's launches.
inline int scratch_for(ScratchHold* hold, hipStream_t s, size_t bytes, void** out) {
  *out = nullptr;
  if (bytes == 0) return SEEDLM_OK;
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess) return SEEDLM_E_DEVICE;
  return hold->take(dev, s, bytes, out);
}

// Both append calls, whose arguments differ by their cache alone; check_geometry checks that.
template <typename Args, typename Geometry>
int check_append(const Args* a, Geometry check_geometry) {
  if (!a) return SEEDLM_E_INVALID;
  if (!dtype_ok(a->x_dtype)) return SEEDLM_E_UNSUPPORTED;
  const int st = check_geometry(a->cache);
  if (st != SEEDLM_OK) return st;
  if (a->tokens < 0 || a->heads < 1 || a->table_len < 0 || a->rot < 0) return SEEDLM_E_INVALID;
  const int64_t D = a->cache.head_dim;
  if (a->rot > D) return SEEDLM_E_INVALID;
  if (a->rot % 2 != 0 || D % 2 != 0 || D > 512) return SEEDLM_E_UNSUPPORTED;
  // Bounds of the grid: a workgroup per token and, at the least, per head.
  if (a->heads > 16384 || a->cache.kv_heads > 16384 || a->tokens >= 1 << 24)
    return SEEDLM_E_UNSUPPORTED;
  const int64_t q = a->heads * D, kv = a->cache.kv_heads * D;
  if (a->q_stride < q || a->q_out_stride < q || a->k_stride < kv || a->v_stride < kv)
    return SEEDLM_E_INVALID;
  if (a->tokens == 0) return SEEDLM_OK;
  if (!a->q || !a->k || !a->v || !a->q_out || !a->positions || !a->slots) return SEEDLM_E_INVALID;
  if (a->rot > 0 && a->table_len > 0 && (!a->cos || !a->sin)) return SEEDLM_E_INVALID;
  const uintptr_t e = (uintptr_t)dtype_bytes(a->x_dtype);
  if (!aligned(a->q, e) || !aligned(a->k, e) || !aligned(a->v, e) || !aligned(a->q_out, e) ||
      !aligned(a->cos, 4) || !aligned(a->sin, 4) || !aligned(a->positions, 4) ||
      !aligned(a->slots, 4))
    return SEEDLM_E_INVALID;
  if (a->q_out == a->q && a->q_out_stride != a->q_stride) return SEEDLM_E_INVALID;
  return SEEDLM_OK;
}

// Both attention calls, but for their caches' alignment and spans.
template <typename Args, typename Geometry>
int check_attend(const Args* a, Geometry check_geometry) {
  if (!a) return SEEDLM_E_INVALID;
  if (!dtype_ok(a->x_dtype)) return SEEDLM_E_UNSUPPORTED;
  const auto& c = a->cache;
  const int st = check_geometry(c);
  if (st != SEEDLM_OK) return st;
  if (!a->q || !a->out || !a->table || !a->lens) return SEEDLM_E_INVALID;
  if (a->queries < 1 || a->queries > SEEDLM_MAX_REQUESTS || a->heads < 1 || a->max_pages < 1 ||
      a->max_len < 0 || a->table_stride < a->max_pages || a->heads % c.kv_heads != 0 ||
      a->table_rows < 1 || (!a->rows && a->table_rows < a->queries))
    return SEEDLM_E_INVALID;
  if (!(a->scale - a->scale == 0.f)) return SEEDLM_E_INVALID;  // NaN or infinite
  const int64_t row = (int64_t)a->heads * c.head_dim;
  if (a->q_stride < row || a->out_stride < row) return SEEDLM_E_INVALID;
  if (a->out == a->q && a->out_stride != a->q_stride) return SEEDLM_E_INVALID;
  if (!aligned(a->table, 4) || !aligned(a->lens, 4) || !aligned(a->rows, 4) ||
      !aligned(a->out, (uintptr_t)dtype_bytes(a->x_dtype)))
    return SEEDLM_E_INVALID;
  if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) return SEEDLM_E_UNSUPPORTED;
  if (a->heads > 16384) return SEEDLM_E_UNSUPPORTED;
  if (!aligned(a->q, 16) || a->q_stride % (16 / dtype_bytes(a->x_dtype)) != 0)
    return SEEDLM_E_UNSUPPORTED;
  const int64_t room = (int64_t)a->max_pages * c.page_size;
  // Token numbers, and the sums of 128-token units over the requests, are 32-bit.
  const int64_t cap = a->max_len < room ? a->max_len : room;
  if (cap > (int64_t)1 << 30 || (cap / 128 + 1) * a->queries > INT32_MAX)
    return SEEDLM_E_UNSUPPORTED;
  return SEEDLM_OK;
}

}  // namespace seedlm
