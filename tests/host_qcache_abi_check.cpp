// Host-side driver for test_host_qcache_sanitizers.py.  It is linked against objects of
// the quantised cache's entry points and of its attention's launch, whose host side is
// built with AddressSanitizer and UndefinedBehaviorSanitizer, and calls every entry point
// with arguments that are refused, at and past the limits of their types, and the size
// query with the largest that are taken.  No call launches anything; what the sources need
// of the rest of the library is defined here, and the current device.
//
// Exit status 0 when every status is the documented one; a report aborts the run.
#include <limits.h>
#include <stdio.h>

#include "../prng_seeded_decode_amd/csrc/qcache_attend.h"

namespace seedlm {
int device_cu_count() { return 256; }
int ScratchHold::take(int, hipStream_t, size_t, void**) { return SEEDLM_E_NOMEM; }
int launch_qcache_append(const seedlm_qcache_append_args&, hipStream_t) { return 77; }
int launch_qcache_read(const seedlm_qcache_read_args&, hipStream_t) { return 78; }
namespace qattend {
int run_4(const Args&, hipStream_t) { return 79; }
int run_4_wide(const Args&, hipStream_t) { return 79; }
int run_8(const Args&, hipStream_t) { return 79; }
int run_8_wide(const Args&, hipStream_t) { return 79; }
}  // namespace qattend
}  // namespace seedlm

extern "C" hipError_t hipGetDevice(int* device) {
  *device = 0;
  return hipSuccess;
}

namespace {

int g_failures = 0;

void expect(const char* what, int got, int want) {
  if (got == want) return;
  fprintf(stderr, "FAIL %s: status %d, expected %d\n", what, got, want);
  ++g_failures;
}

alignas(64) int32_t g_mem[1024];  // addresses only
void* const kP = g_mem;

// 64 dimensions, 4 bits, two groups, token-major
seedlm_qcache_t cache() { return {kP, kP, kP, kP, 10, 1024, 64, 32, 64, 4, 2, 16, 2, 64, 4, 32}; }

seedlm_qcache_append_args append() {
  seedlm_qcache_append_args a{};
  a.q = a.k = a.v = a.q_out = kP;
  a.cos = a.sin = reinterpret_cast<float*>(kP);
  a.positions = a.slots = g_mem;
  a.cache = cache();
  a.q_stride = a.q_out_stride = 256, a.k_stride = a.v_stride = 128;
  a.tokens = 3, a.heads = 4, a.rot = 64, a.table_len = 9, a.x_dtype = SEEDLM_F16;
  return a;
}

seedlm_qcache_read_args read_args() {
  seedlm_qcache_read_args a{};
  a.k_out = a.v_out = kP;
  a.slots = g_mem;
  a.cache = cache();
  a.k_stride = a.v_stride = 128;
  a.tokens = 3, a.y_dtype = SEEDLM_F16;
  return a;
}

seedlm_qcache_attend_args attend() {
  seedlm_qcache_attend_args a{};
  a.q = a.out = kP;
  a.table = a.lens = g_mem;
  a.cache = cache();
  a.q_stride = a.out_stride = 256;
  a.table_stride = a.max_pages = 8;
  a.queries = a.table_rows = 3, a.heads = 4, a.max_len = 100, a.x_dtype = SEEDLM_F16;
  a.scale = 0.1f;
  return a;
}

// Every entry point with this cache and outer strides that fit any.
void expect_cache(const char* what, const seedlm_qcache_t& c, int want) {
  seedlm_qcache_append_args p = append();
  seedlm_qcache_read_args r = read_args();
  seedlm_qcache_attend_args q = attend();
  p.cache = r.cache = q.cache = c;
  const int64_t row = (int64_t)1 << 40;
  p.q_stride = p.q_out_stride = p.k_stride = p.v_stride = r.k_stride = r.v_stride = row;
  q.q_stride = q.out_stride = row;
  size_t bytes = 0;
  expect(what, seedlm_qcache_append(&p, nullptr), want);
  expect(what, seedlm_qcache_read(&r, nullptr), want);
  expect(what, seedlm_qcache_attend(&q, nullptr), want);
  expect(what, seedlm_qcache_attend_scratch_bytes(&q, &bytes), want);
}

void check_caches() {
  for (int64_t seedlm_qcache_t::*stride :
       {&seedlm_qcache_t::page_stride, &seedlm_qcache_t::token_stride, &seedlm_qcache_t::head_stride,
        &seedlm_qcache_t::scale_page_stride, &seedlm_qcache_t::scale_token_stride,
        &seedlm_qcache_t::scale_head_stride}) {
    seedlm_qcache_t c = cache();
    c.*stride = INT64_MAX / 16 * 16;
    expect_cache("largest stride", c, SEEDLM_E_UNSUPPORTED);
    c.*stride = INT64_MIN;
    expect_cache("smallest stride", c, SEEDLM_E_INVALID);
  }
  seedlm_qcache_t c = cache();
  c.pages = INT64_MAX;
  expect_cache("pages", c, SEEDLM_E_UNSUPPORTED);
  c = cache();
  c.page_size = c.kv_heads = c.head_dim = c.bits = c.group = INT_MAX;
  expect_cache("largest sizes", c, SEEDLM_E_UNSUPPORTED);
  c = cache();
  c.page_size = c.kv_heads = c.head_dim = c.bits = c.group = INT_MIN;
  expect_cache("smallest sizes", c, SEEDLM_E_INVALID);
  c = cache();
  c.pages = INT_MAX, c.page_size = 1, c.page_stride = 32;  // 2^36 bytes and no more
  c.token_stride = c.head_stride = 16, c.scale_page_stride = 2;
  seedlm_qcache_read_args r = read_args();
  r.cache = c;
  expect("largest pool", seedlm_qcache_read(&r, nullptr), 78);
  r.cache.page_stride = 48;
  expect("a larger pool", seedlm_qcache_read(&r, nullptr), SEEDLM_E_UNSUPPORTED);
}

void check_append() {
  expect("append null", seedlm_qcache_append(nullptr, nullptr), SEEDLM_E_INVALID);
  seedlm_qcache_append_args a = append();
  expect("append", seedlm_qcache_append(&a, nullptr), 77);
  for (int64_t most : {INT64_MAX, INT64_MIN}) {
    a = append();
    a.q_stride = a.k_stride = a.v_stride = a.q_out_stride = most, a.tokens = INT_MAX;
    expect("append strides", seedlm_qcache_append(&a, nullptr), SEEDLM_E_UNSUPPORTED);
  }
  a = append();
  a.heads = a.rot = INT_MAX;
  expect("append heads", seedlm_qcache_append(&a, nullptr), SEEDLM_E_INVALID);
  a = append();
  a.tokens = 0, a.q = nullptr;
  expect("append of no tokens", seedlm_qcache_append(&a, nullptr), SEEDLM_OK);
}

void check_read() {
  expect("read null", seedlm_qcache_read(nullptr, nullptr), SEEDLM_E_INVALID);
  seedlm_qcache_read_args a = read_args();
  a.k_out = nullptr, a.k_stride = INT64_MIN;
  expect("read of values", seedlm_qcache_read(&a, nullptr), 78);
  a.v_stride = INT64_MIN;
  expect("read stride", seedlm_qcache_read(&a, nullptr), SEEDLM_E_INVALID);
  a = read_args();
  a.tokens = INT_MAX;
  expect("read tokens", seedlm_qcache_read(&a, nullptr), SEEDLM_E_UNSUPPORTED);
}

void check_attend() {
  size_t bytes = 0;
  expect("attend null", seedlm_qcache_attend(nullptr, nullptr), SEEDLM_E_INVALID);
  seedlm_qcache_attend_args a = attend();
  expect("attend", seedlm_qcache_attend(&a, nullptr), 79);
  expect("bytes null", seedlm_qcache_attend_scratch_bytes(&a, nullptr), SEEDLM_E_INVALID);
  a.max_pages = a.max_len = INT_MAX, a.table_stride = INT64_MAX;
  expect("attend longest", seedlm_qcache_attend(&a, nullptr), SEEDLM_E_UNSUPPORTED);
  a = attend();
  a.queries = a.table_rows = SEEDLM_MAX_REQUESTS, a.max_pages = a.max_len = 1 << 30;
  a.table_stride = 1 << 30;
  expect("attend longest of most queries", seedlm_qcache_attend(&a, nullptr), SEEDLM_E_UNSUPPORTED);
  // the most units that a split may have: 2^31 - 1, with what starting an item counts for
  a.queries = a.table_rows = 255;
  a.max_len = 1 << 30;
  expect("attend most units", seedlm_qcache_attend_scratch_bytes(&a, &bytes), SEEDLM_OK);
  a.queries = a.table_rows = 256;
  expect("attend too many units", seedlm_qcache_attend_scratch_bytes(&a, &bytes), SEEDLM_E_UNSUPPORTED);
  a.queries = a.table_rows = SEEDLM_MAX_REQUESTS;
  a.max_len = 1 << 25;
  expect("attend bytes of the most", seedlm_qcache_attend_scratch_bytes(&a, &bytes), SEEDLM_OK);
  expect("attend without scratch", seedlm_qcache_attend(&a, nullptr), SEEDLM_E_NOMEM);
  a.heads = 16384, a.q_stride = a.out_stride = 1 << 20;
  expect("attend bytes of the most heads", seedlm_qcache_attend_scratch_bytes(&a, &bytes), SEEDLM_OK);
  a = attend();
  a.queries = a.heads = a.table_rows = a.max_pages = a.max_len = INT_MIN;
  expect("attend smallest", seedlm_qcache_attend(&a, nullptr), SEEDLM_E_INVALID);
}

}  // namespace

int main() {
  check_caches();
  check_append();
  check_read();
  check_attend();
  printf("quantised cache checks: %d failure(s)\n", g_failures);
  return g_failures ? 1 : 0;
}
