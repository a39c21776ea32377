// C-ABI entry points of the quantised cache (seedlm_serve.h): argument checks, scratch
// and the launches.  Nothing here allocates host memory or throws.
#include "serve_checks.h"

namespace seedlm {
namespace {

// Geometry of a quantised cache, all of which the kernels rely on.
int check_qcache(const seedlm_qcache_t& c) {
  if (!c.k || !c.v || !c.k_scale || !c.v_scale) return SEEDLM_E_INVALID;
  if (c.pages < 1 || c.page_size < 1 || c.kv_heads < 1 || c.head_dim < 1 || c.group < 1)
    return SEEDLM_E_INVALID;
  if (c.page_stride < 0 || c.token_stride < 0 || c.head_stride < 0 || c.scale_page_stride < 0 ||
      c.scale_token_stride < 0 || c.scale_head_stride < 0)
    return SEEDLM_E_INVALID;
  if (c.pages > INT32_MAX / c.page_size || c.kv_heads > 16384) return SEEDLM_E_UNSUPPORTED;
  if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) return SEEDLM_E_UNSUPPORTED;
  if (c.bits != 4 && c.bits != 8) return SEEDLM_E_UNSUPPORTED;
  if (c.group < 32 || c.head_dim % c.group != 0) return SEEDLM_E_UNSUPPORTED;
  const int groups = c.head_dim / c.group;
  if (groups != 1 && groups != 2 && groups != 4) return SEEDLM_E_UNSUPPORTED;
  if (!aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(c.k_scale, 4 * groups) ||
      !aligned(c.v_scale, 4 * groups) || c.page_stride % 16 != 0 || c.token_stride % 16 != 0 ||
      c.head_stride % 16 != 0 || c.scale_page_stride % groups != 0 ||
      c.scale_token_stride % groups != 0 || c.scale_head_stride % groups != 0)
    return SEEDLM_E_UNSUPPORTED;
  // Rows are counted in 32 bits, by 16 bytes of codes and by a row's pairs (each
  // stride's own bound first, so that the sum fits 64 bits).
  auto fits = [](int64_t stride, int64_t n, int64_t most) { return stride <= (most - 1) / n; };
  auto spans = [&](int64_t page, int64_t token, int64_t head, int64_t row, int64_t most) {
    return fits(page, c.pages, most) && fits(token, c.page_size, most) && fits(head, c.kv_heads, most) &&
           page * (c.pages - 1) + token * (c.page_size - 1) + head * (c.kv_heads - 1) + row <= most;
  };
  if (!spans(c.page_stride, c.token_stride, c.head_stride, c.head_dim * c.bits / 8,
             (int64_t)1 << 36) ||
      !spans(c.scale_page_stride, c.scale_token_stride, c.scale_head_stride, groups,
             (int64_t)groups << 32))
    return SEEDLM_E_UNSUPPORTED;
  return SEEDLM_OK;
}

int check_read(const seedlm_qcache_read_args* a) {
  if (!a) return SEEDLM_E_INVALID;
  if (!dtype_ok(a->y_dtype)) return SEEDLM_E_UNSUPPORTED;
  const int st = check_qcache(a->cache);
  if (st != SEEDLM_OK) return st;
  if (a->tokens < 0) return SEEDLM_E_INVALID;
  if (a->tokens >= 1 << 24) return SEEDLM_E_UNSUPPORTED;
  const int64_t row = (int64_t)a->cache.kv_heads * a->cache.head_dim;
  if ((a->k_out && a->k_stride < row) || (a->v_out && a->v_stride < row)) return SEEDLM_E_INVALID;
  if (a->tokens > 0 && (!a->slots || (!a->k_out && !a->v_out))) return SEEDLM_E_INVALID;
  const uintptr_t e = (uintptr_t)dtype_bytes(a->y_dtype);
  if (!aligned(a->k_out, e) || !aligned(a->v_out, e) || !aligned(a->slots, 4))
    return SEEDLM_E_INVALID;
  return SEEDLM_OK;
}

int check_qattend(const seedlm_qcache_attend_args* a) {
  const int st = check_attend(a, check_qcache);
  if (st != SEEDLM_OK) return st;
  // The split's units, with what starting each query counts for, are 32-bit.
  const int64_t room = (int64_t)a->max_pages * a->cache.page_size;
  const int64_t cap = a->max_len < room ? a->max_len : room;
  return (cap / 128 + 1 + kQcacheItemUnits) * a->queries > INT32_MAX ? SEEDLM_E_UNSUPPORTED
                                                                      : SEEDLM_OK;
}

}  // namespace
}  // namespace seedlm

using namespace seedlm;

extern "C" {

int seedlm_qcache_append(const seedlm_qcache_append_args* args, void* stream) {
  const int st = check_append(args, check_qcache);
  if (st != SEEDLM_OK || args->tokens == 0) return st;
  return launch_qcache_append(*args, static_cast<hipStream_t>(stream));
}

int seedlm_qcache_read(const seedlm_qcache_read_args* args, void* stream) {
  const int st = check_read(args);
  if (st != SEEDLM_OK || args->tokens == 0) return st;
  return launch_qcache_read(*args, static_cast<hipStream_t>(stream));
}

int seedlm_qcache_attend(const seedlm_qcache_attend_args* args, void* stream) {
  int st = check_qattend(args);
  if (st != SEEDLM_OK) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  ScratchHold hold;
  void* scratch = nullptr;
  st = scratch_for(&hold, s, qcache_attend_scratch_bytes(*args), &scratch);
  if (st != SEEDLM_OK) return st;
  return launch_qcache_attend(*args, scratch, s);
}

int seedlm_qcache_attend_scratch_bytes(const seedlm_qcache_attend_args* args, size_t* bytes) {
  if (!bytes) return SEEDLM_E_INVALID;
  const int st = check_qattend(args);
  if (st != SEEDLM_OK) return st;
  *bytes = qcache_attend_scratch_bytes(*args);
  return SEEDLM_OK;
}

}  // extern "C"
