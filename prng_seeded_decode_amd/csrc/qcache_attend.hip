// Launches of seedlm_qcache_attend; the kernels and how they work are in qcache_attend.h.
#include <algorithm>

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

// Queries of an item at most: as many as fill the 16 columns, where rows can repeat.
int shared_of(const seedlm_qcache_attend_args& a) {
  return a.rows && group_of(a) < 16 ? 16 / group_of(a) : 1;
}

// Queries of a row of the table, as far as the call's sizes say (which query has which row
// lies in device memory), and of an item.
int per_row(const seedlm_qcache_attend_args& a) {
  return a.rows ? std::max(1, a.queries / a.table_rows) : 1;
}
int in_item(const seedlm_qcache_attend_args& a) { return std::min(shared_of(a), per_row(a)); }

// Whether items are the workgroups: then an item's steps of kUnit tokens follow one
// another, but the sums, the partials and the second launch (4 to 5 us) fall away.  That
// pays up to so many steps, and up to twice as many where items fill half the chip.  Time
// of a call, unsplit against split, lengths alike: one request of 8 cache heads and 128
// dimensions, 4 bits, 8.3 and 9.8 us at 512 tokens, 10.1 and 9.8 at 768, 11.9 and 9.9
// at 1024; 16 requests 12.7 and 14.1 at 1024, 16.3 and 16.8 at 1536, 19.8 and 17.7 at
// 2048; 4 of 2 heads and 256 dimensions, 8 bits, 10.5 and 11.9 at 384, 12.0 and 11.9 at
// 512.  Lengths that differ shift the balance, since a call is as long as its longest item
// and the runs share the sum: 16 requests ragged up to 1536 16.3 and 14.5.  64 dimensions
// could go on past their 14 steps (1792 tokens) where lengths are alike (8 requests of 32
// heads, 8 bits, 15.7 and 20.8 at 2048), not where they are ragged, as requests that are
// served are (15.5 and 15.6; 4 requests 15.3 and 14.0; in fp32 17.5 and 16.5).  With two
// workgroups for every compute unit runs of even length gain nothing until lengths differ
// much: 64 requests 31.8 and 36.4 at 2048.  Items of several queries are as long as their
// neighbours: 128 queries of one request of 2048 tokens (256 workgroups) 22.4 and 27.7,
// 512 of 2048 48.7 and 58.7, 512 of 8192 167 and 175.  That holds from twice as many queries
// of a row as an item takes (4 of 128 in a table of 64 rows 42.2 and 48.9); with fewer the
// items may be single tokens of requests that have nothing in common (64 rows of 8 queries,
// ragged up to 8000, 135 and 118, but 128 of 4000 125 and 131).
bool unsplit(const seedlm_qcache_attend_args& a) {
  const int64_t items = (a.queries + in_item(a) - 1) / in_item(a);
  const int64_t workgroups = items * a.cache.kv_heads * qtiles_of(a);
  int steps = a.cache.head_dim == 64 ? 7 : (a.cache.head_dim == 128 ? 6 : 4);
  const int cus = device_cu_count();
  if (2 * workgroups >= cus) steps *= 2;
  if (workgroups >= 2 * cus) steps = std::max(steps, 16 * 128 / a.cache.head_dim);
  if (per_row(a) >= 2 * shared_of(a) && shared_of(a) > 1 && workgroups >= cus)
    steps = workgroups >= 4 * cus ? 64 : 32;
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
  p.shared = shared_of(a);
  p.slots = slots_of(a);
  p.rows = p.slots > 0 ? p.slots : a.queries;
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
