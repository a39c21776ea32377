// Host-side driver for test_host_qcache_launch.py: the launch that seedlm_qcache_attend makes
// of a call's sizes, caught where its kernels would start.  One token of each request with
// `rows`, as a plan gives them, has to have the workgroups, the split and the scratch of the
// call without; a call without a split has to have a workgroup row for every query, so that
// no query waits for another's item; and a call that shares items keeps its runs within what
// the chip holds.  Exit status 0 when every launch does.
#include <stdio.h>

#include "../prng_seeded_decode_amd/csrc/qcache_attend.h"

namespace {
seedlm::qattend::Args g_seen;
int g_failures = 0;
long g_calls = 0;
alignas(64) int32_t g_mem[1024];  // addresses only
int see(const seedlm::qattend::Args& p) {
  g_seen = p;
  return SEEDLM_OK;
}
}  // namespace

namespace seedlm {
int device_cu_count() { return 256; }
int ScratchHold::take(int, hipStream_t, size_t, void** base) {
  *base = g_mem;
  return SEEDLM_OK;
}
int launch_qcache_append(const seedlm_qcache_append_args&, hipStream_t) { return 77; }
int launch_qcache_read(const seedlm_qcache_read_args&, hipStream_t) { return 78; }
namespace qattend {
int run_4(const Args& p, hipStream_t) { return see(p); }
int run_4_wide(const Args& p, hipStream_t) { return see(p); }
int run_8(const Args& p, hipStream_t) { return see(p); }
int run_8_wide(const Args& p, hipStream_t) { return see(p); }
}  // namespace qattend
}  // namespace seedlm

extern "C" hipError_t hipGetDevice(int* device) {
  *device = 0;
  return hipSuccess;
}

namespace {

struct Launch {
  int status, slots, rows;
  size_t scratch;
};

Launch launch(const seedlm_qcache_attend_args& a) {
  Launch l{};
  g_seen = {};
  l.status = seedlm_qcache_attend(&a, nullptr);
  l.slots = g_seen.slots, l.rows = g_seen.rows;
  seedlm_qcache_attend_scratch_bytes(&a, &l.scratch);
  ++g_calls;
  return l;
}

void fail(const char* what, const seedlm_qcache_attend_args& a, int got, int want) {
  if (++g_failures > 20) return;
  fprintf(stderr, "FAIL %s: %d, expected %d (%d queries of %d rows, %d/%d heads, %d dimensions, %d tokens)\n",
          what, got, want, a.queries, a.table_rows, a.heads, a.cache.kv_heads, a.cache.head_dim, a.max_len);
}

void check(int kv, int group, int dim, int queries, int len) {
  seedlm_qcache_attend_args a{};
  a.q = a.out = g_mem;
  a.table = a.lens = g_mem;
  const int64_t row = (int64_t)kv * dim / 2;
  a.cache = {g_mem, g_mem, g_mem, g_mem, 10, 16 * row, row, dim / 2, 16 * 2 * kv, 2 * kv, 2, 16, kv, dim, 4, dim};
  a.heads = kv * group;
  a.q_stride = a.out_stride = (int64_t)a.heads * dim;
  a.table_stride = a.max_pages = (len + 15) / 16;
  a.queries = a.table_rows = queries, a.max_len = len, a.x_dtype = SEEDLM_F16, a.scale = 0.1f;
  const Launch plain = launch(a);
  if (plain.status != SEEDLM_OK) return fail("status", a, plain.status, SEEDLM_OK);
  a.rows = g_mem;
  const Launch with = launch(a);
  if (with.slots != plain.slots) fail("runs of a token a request", a, with.slots, plain.slots);
  if (with.rows != plain.rows) fail("workgroup rows of a token a request", a, with.rows, plain.rows);
  if (with.scratch != plain.scratch) fail("scratch of a token a request", a, (int)with.scratch, (int)plain.scratch);
  // pieces of every length of a few requests, and a table that is longer than the batch
  for (int rows : {1, 2, 3, 8, 64, 512}) {
    a.table_rows = rows;
    const Launch l = launch(a);
    if (l.status != SEEDLM_OK) fail("status", a, l.status, SEEDLM_OK);
    if (l.slots == 0 && l.rows != queries) fail("workgroup rows without a split", a, l.rows, queries);
    if (l.slots > 0 && l.rows != l.slots) fail("workgroup rows of a split", a, l.rows, l.slots);
    if ((l.slots > 0) != (l.scratch > 0)) fail("scratch", a, (int)l.scratch, l.slots);
    if ((l.slots - 1) * (int64_t)kv * ((group + 15) / 16) >= 256 * 3) fail("runs", a, l.slots, 256 * 3);
  }
}

}  // namespace

int main() {
  for (int kv : {1, 2, 4, 8, 32})
    for (int group : {1, 3, 4, 8, 16, 40})
      for (int dim : {64, 128, 256})
        for (int queries : {1, 2, 4, 15, 16, 17, 63, 64, 65, 128, 129, 512, 1000})
          for (int len : {1, 128, 500, 512, 768, 1024, 1500, 1792, 2000, 2048, 4000, 8192, 40000})
            check(kv, group, dim, queries, len);
  printf("launches: %ld made, %d failure(s)\n", g_calls, g_failures);
  return g_failures ? 1 : 0;
}
