// C-ABI entry points of the serving operators (seedlm_serve.h): argument checks,
// scratch and the launches.  Nothing here allocates host memory or throws.
#include "seedlm_internal.h"

namespace seedlm {
namespace {

bool dtype_ok(int d) { return d == SEEDLM_F32 || d == SEEDLM_F16; }
int64_t dtype_bytes(int d) { return d == SEEDLM_F32 ? 4 : 2; }
bool aligned(const void* p, uintptr_t n) { return (uintptr_t)p % n == 0; }

// Whether [p, p + n) and [q, q + m) int32 ranges share an entry.
bool overlap(const int32_t* p, int64_t n, const int32_t* q, int64_t m) {
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  return a < b + (uintptr_t)m * 4 && b < a + (uintptr_t)n * 4;
}

// Scratch of `bytes` bytes on `s` (NULL for none), held for the call's launches.
int scratch_for(ScratchHold* hold, hipStream_t s, size_t bytes, void** out) {
  *out = nullptr;
  if (bytes == 0) return SEEDLM_OK;
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess) return SEEDLM_E_DEVICE;
  return hold->take(dev, s, bytes, out);
}

int check_plan(const seedlm_cache_plan_args* a) {
  if (!a || !a->lens || !a->fresh || !a->table || !a->ring || !a->ring_state || !a->lens_out ||
      !a->ring_state_out || !a->offsets || !a->ok)
    return SEEDLM_E_INVALID;
  if (a->requests < 1 || a->requests > SEEDLM_MAX_REQUESTS || a->page_size < 1 ||
      a->max_pages < 1 || a->pool < 1 || a->tokens < 0 || a->table_stride < a->max_pages)
    return SEEDLM_E_INVALID;
  if (a->tokens > 0 && (!a->rows || !a->positions || !a->slots)) return SEEDLM_E_INVALID;
  for (const void* p : {(const void*)a->lens, (const void*)a->fresh, (const void*)a->table,
                        (const void*)a->ring, (const void*)a->ring_state,
                        (const void*)a->lens_out, (const void*)a->ring_state_out,
                        (const void*)a->offsets, (const void*)a->ok, (const void*)a->rows,
                        (const void*)a->positions, (const void*)a->slots, (const void*)a->spans})
    if (!aligned(p, 4)) return SEEDLM_E_INVALID;
  if (a->lens_out != a->lens && overlap(a->lens_out, a->requests, a->lens, a->requests))
    return SEEDLM_E_INVALID;
  if (a->ring_state_out != a->ring_state && overlap(a->ring_state_out, 2, a->ring_state, 2))
    return SEEDLM_E_INVALID;
  // Token positions, slots and the kernels' counters are 32-bit.
  if ((int64_t)a->max_pages * a->page_size + a->tokens > INT32_MAX ||
      (int64_t)a->pool * a->page_size > INT32_MAX || a->tokens > 1 << 30 || a->pool > 1 << 30)
    return SEEDLM_E_UNSUPPORTED;
  return SEEDLM_OK;
}

// Geometry of a cache; strides may be any that keep its elements apart, which
// only the caller knows, so no more than their signs are checked.
int check_cache(const seedlm_cache_t& c) {
  if (!c.k || !c.v || !aligned(c.k, 2) || !aligned(c.v, 2)) return SEEDLM_E_INVALID;
  if (c.pages < 1 || c.page_size < 1 || c.kv_heads < 1 || c.head_dim < 1) return SEEDLM_E_INVALID;
  if (c.page_stride < 0 || c.token_stride < 0 || c.head_stride < 0) return SEEDLM_E_INVALID;
  if (c.pages > INT32_MAX / c.page_size) return SEEDLM_E_UNSUPPORTED;
  return SEEDLM_OK;
}

int check_append(const seedlm_cache_append_args* a) {
  if (!a) return SEEDLM_E_INVALID;
  if (!dtype_ok(a->x_dtype)) return SEEDLM_E_UNSUPPORTED;
  const int st = check_cache(a->cache);
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

int check_attend(const seedlm_cache_attend_args* a) {
  if (!a) return SEEDLM_E_INVALID;
  if (!dtype_ok(a->x_dtype)) return SEEDLM_E_UNSUPPORTED;
  const seedlm_cache_t& c = a->cache;
  const int st = check_cache(c);
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
  if (!aligned(a->q, 16) || a->q_stride % (16 / dtype_bytes(a->x_dtype)) != 0 ||
      !aligned(c.k, 16) || !aligned(c.v, 16) || c.page_stride % 8 != 0 ||
      c.token_stride % 8 != 0 || c.head_stride % 8 != 0)
    return SEEDLM_E_UNSUPPORTED;
  // Token offsets are 32-bit counts of 8 elements.
  constexpr int64_t kMost = (int64_t)1 << 35;
  // (each stride's own bound first, so that the products fit 64 bits)
  if (c.page_stride >= kMost / c.pages || c.token_stride >= kMost / c.page_size ||
      c.head_stride >= kMost / c.kv_heads ||
      c.page_stride * (c.pages - 1) + c.token_stride * (c.page_size - 1) >=
          kMost - 8 - c.head_stride * (c.kv_heads - 1) - c.head_dim)
    return SEEDLM_E_UNSUPPORTED;
  const int64_t room = (int64_t)a->max_pages * c.page_size;
  // Token numbers, and the sums of 128-token units over the requests, are 32-bit.
  const int64_t cap = a->max_len < room ? a->max_len : room;
  if (cap > (int64_t)1 << 30 || (cap / 128 + 1) * a->queries > INT32_MAX)
    return SEEDLM_E_UNSUPPORTED;
  return SEEDLM_OK;
}

int check_lora_sizes(const seedlm_lora_site* sites, int n, int64_t tokens, int xdt, int ydt) {
  if (n < 0 || tokens < 0 || (n > 0 && !sites)) return SEEDLM_E_INVALID;
  if (!dtype_ok(xdt) || !dtype_ok(ydt)) return SEEDLM_E_UNSUPPORTED;
  constexpr int64_t kMost = (int64_t)1 << 24;
  for (int i = 0; i < n; ++i) {
    const seedlm_lora_site& s = sites[i];
    if (s.rows < 1 || s.cols < 1 || s.rank < 1 || s.rank > SEEDLM_MAX_RANK)
      return SEEDLM_E_INVALID;
    if (s.rows >= kMost || s.cols >= kMost) return SEEDLM_E_UNSUPPORTED;
  }
  return tokens >= (int64_t)1 << 20 ? SEEDLM_E_UNSUPPORTED : SEEDLM_OK;
}

}  // namespace
}  // namespace seedlm

using namespace seedlm;

extern "C" {

int seedlm_cache_plan(const seedlm_cache_plan_args* args, void* stream) {
  int st = check_plan(args);
  if (st != SEEDLM_OK) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  ScratchHold hold;
  void* scratch = nullptr;
  st = scratch_for(&hold, s, cache_plan_scratch_bytes(*args), &scratch);
  if (st != SEEDLM_OK) return st;
  return launch_cache_plan(*args, static_cast<int32_t*>(scratch), s);
}

int seedlm_cache_append(const seedlm_cache_append_args* args, void* stream) {
  const int st = check_append(args);
  if (st != SEEDLM_OK || args->tokens == 0) return st;
  return launch_cache_append(*args, static_cast<hipStream_t>(stream));
}

int seedlm_cache_attend(const seedlm_cache_attend_args* args, void* stream) {
  int st = check_attend(args);
  if (st != SEEDLM_OK) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  ScratchHold hold;
  void* scratch = nullptr;
  st = scratch_for(&hold, s, cache_attend_scratch_bytes(*args), &scratch);
  if (st != SEEDLM_OK) return st;
  return launch_cache_attend(*args, scratch, s);
}

int seedlm_cache_attend_scratch_bytes(const seedlm_cache_attend_args* args, size_t* bytes) {
  if (!bytes) return SEEDLM_E_INVALID;
  const int st = check_attend(args);
  if (st != SEEDLM_OK) return st;
  *bytes = cache_attend_scratch_bytes(*args);
  return SEEDLM_OK;
}

int seedlm_lora_many(const seedlm_lora_site* sites, int n, const int32_t* adapter,
                     const float* scales, int64_t tokens, int adapters, int x_dtype, int y_dtype,
                     void* stream) {
  int st = check_lora_sizes(sites, n, tokens, x_dtype, y_dtype);
  if (st != SEEDLM_OK) return st;
  if (adapters < 1) return SEEDLM_E_INVALID;
  if (n == 0 || tokens == 0) return SEEDLM_OK;
  if (!adapter || !scales || !aligned(adapter, 4) || !aligned(scales, 4)) return SEEDLM_E_INVALID;
  const uintptr_t xe = (uintptr_t)dtype_bytes(x_dtype), ye = (uintptr_t)dtype_bytes(y_dtype);
  for (int i = 0; i < n; ++i) {
    const seedlm_lora_site& s = sites[i];
    if (!s.x || !s.A || !s.B || !s.base || !s.y) return SEEDLM_E_INVALID;
    if (!aligned(s.x, xe) || !aligned(s.A, 2) || !aligned(s.B, 2) || !aligned(s.base, ye) ||
        !aligned(s.y, ye))
      return SEEDLM_E_INVALID;
  }
  const hipStream_t s = static_cast<hipStream_t>(stream);
  ScratchHold hold;
  void* scratch = nullptr;
  st = scratch_for(&hold, s, lora_scratch_bytes(sites, n, tokens, adapters, x_dtype, y_dtype),
                   &scratch);
  if (st != SEEDLM_OK) return st;
  return launch_lora(sites, n, adapter, scales, tokens, adapters, x_dtype, y_dtype,
                     static_cast<float*>(scratch), s);
}

int seedlm_lora_scratch_bytes(const seedlm_lora_site* sites, int n, int64_t tokens, int adapters,
                              int x_dtype, int y_dtype, size_t* bytes) {
  if (!bytes || adapters < 1) return SEEDLM_E_INVALID;
  const int st = check_lora_sizes(sites, n, tokens, x_dtype, y_dtype);
  if (st != SEEDLM_OK) return st;
  *bytes = lora_scratch_bytes(sites, n, tokens, adapters, x_dtype, y_dtype);
  return SEEDLM_OK;
}

}  // extern "C"
