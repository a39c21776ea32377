// Launches of seedlm_qcache_attend; the kernels and how they work are in qcache_attend.h.
#include "qcache_attend.h"

namespace seedlm {

using namespace qattend;

namespace {

int cap_of(const seedlm_qcache_attend_args& a) {
  const int64_t room = (int64_t)a.max_pages * a.cache.page_size;
  return (int)(a.max_len < room ? a.max_len : room);
}

int group_of(const seedlm_qcache_attend_args& a) { return a.heads / a.cache.kv_heads; }
int qtiles_of(const seedlm_qcache_attend_args& a) { return (group_of(a) + 15) / 16; }

// Whether items are the workgroups.
bool unsplit(const seedlm_qcache_attend_args& a) {
  const int64_t workgroups = (int64_t)a.queries * a.cache.kv_heads * qtiles_of(a);
  int steps = 4 * 128 / a.cache.head_dim;
  if (2 * workgroups >= device_cu_count() && steps < 8) steps *= 2;
  return cap_of(a) <= steps * kUnit;
}

// Runs of units per cache head: what the chip holds at once.
int slots_of(const seedlm_qcache_attend_args& a) {
  if (unsplit(a)) return 0;
  const int held = device_cu_count() *
                   waves_per_simd(a.cache.head_dim, a.cache.bits, a.cache.head_dim / a.cache.group,
                                  a.x_dtype == SEEDLM_F32);
  const int across = a.cache.kv_heads * qtiles_of(a);
  return (held + across - 1) / across;
}

struct Scratch {
  size_t joins, ml, acc;  // byte offsets and the total size
  size_t bytes;
};

Scratch scratch_of(const seedlm_qcache_attend_args& a) {
  const size_t n = (size_t)2 * slots_of(a) * a.cache.kv_heads * qtiles_of(a) * 16;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  Scratch r;
  r.joins = 0;
  r.ml = up((size_t)a.queries * sizeof(int4));
  r.acc = r.ml + up(n * sizeof(float2));
  r.bytes = n == 0 ? 0 : r.acc + n * a.cache.head_dim * sizeof(float);
  return r;
}

}  // namespace

size_t qcache_attend_scratch_bytes(const seedlm_qcache_attend_args& a) { return scratch_of(a).bytes; }

int launch_qcache_attend(const seedlm_qcache_attend_args& a, void* scratch, hipStream_t s) {
  const seedlm_qcache_t& c = a.cache;
  const int groups = c.head_dim / c.group;
  Args p{};
  p.a = a;
  p.group = group_of(a);
  p.qtiles = qtiles_of(a);
  p.shared = a.rows && p.group < 16 ? 16 / p.group : 1;
  p.slots = slots_of(a);
  p.cap = cap_of(a);
  p.page_unit = (uint32_t)(c.page_stride / 16);
  p.token_unit = (uint32_t)(c.token_stride / 16);
  p.page_pair = (uint32_t)(c.scale_page_stride / groups);
  p.token_pair = (uint32_t)(c.scale_token_stride / groups);
  p.page_size = divisor((uint32_t)c.page_size);
  p.per_head = (uint32_t)((65536 + p.group - 1) / p.group);
  const Scratch r = scratch_of(a);
  char* base = static_cast<char*>(scratch);
  if (base) {
    p.joins = reinterpret_cast<int4*>(base + r.joins);
    p.ml = reinterpret_cast<float2*>(base + r.ml);
    p.acc = reinterpret_cast<float*>(base + r.acc);
  }
  const bool wide = a.x_dtype == SEEDLM_F32;
  if (c.bits == 4) return wide ? run_4_wide(p, s) : run_4(p, s);
  return wide ? run_8_wide(p, s) : run_8(p, s);
}

}  // namespace seedlm
