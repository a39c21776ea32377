// Host-side driver for test_host_serve_sanitizers.py.  It is linked against objects
// of the serving operators' sources whose host side is built with AddressSanitizer
// and UndefinedBehaviorSanitizer, and calls every entry point of seedlm_serve.h with
// arguments that are refused, at and past the limits of their types, and the size
// queries with the largest that are taken.  No call launches anything; what the
// sources need of the rest of the library is defined here, and the current device.
//
// Exit status 0 when every status is the documented one; a report aborts the run.
#include <limits.h>
#include <stdio.h>

#include "../prng_seeded_decode_amd/csrc/seedlm_internal.h"

namespace seedlm {
int device_cu_count() { return 256; }
int ScratchHold::take(int, hipStream_t, size_t, void**) { return SEEDLM_E_NOMEM; }
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

seedlm_cache_plan_args plan() {
  seedlm_cache_plan_args a{};
  a.lens = a.fresh = a.ring_state = g_mem;
  a.table = a.ring = a.offsets = a.rows = a.positions = a.slots = a.ok = g_mem;
  a.lens_out = a.ring_state_out = g_mem + 512;
  a.table_stride = a.max_pages = 8;
  a.requests = 4, a.page_size = 16, a.pool = 100, a.tokens = 32;
  return a;
}

seedlm_cache_t cache() {
  return {kP, kP, 10, 16 * 2 * 64, 2 * 64, 64, 16, 2, 64};
}

seedlm_cache_append_args append() {
  seedlm_cache_append_args a{};
  a.q = a.k = a.v = a.q_out = kP;
  a.cos = a.sin = reinterpret_cast<float*>(kP);
  a.positions = a.slots = g_mem;
  a.cache = cache();
  a.q_stride = a.q_out_stride = 256, a.k_stride = a.v_stride = 128;
  a.tokens = 3, a.heads = 4, a.rot = 64, a.table_len = 9, a.x_dtype = SEEDLM_F16;
  return a;
}

seedlm_cache_attend_args attend() {
  seedlm_cache_attend_args a{};
  a.q = a.out = kP;
  a.table = a.lens = g_mem;
  a.cache = cache();
  a.q_stride = a.out_stride = 256;
  a.table_stride = a.max_pages = 8;
  a.queries = a.table_rows = 3, a.heads = 4, a.max_len = 100, a.x_dtype = SEEDLM_F16;
  a.scale = 0.1f;
  return a;
}

void check_plan() {
  expect("plan null", seedlm_cache_plan(nullptr, nullptr), SEEDLM_E_INVALID);
  seedlm_cache_plan_args a = plan();
  a.lens = nullptr;
  expect("plan null lens", seedlm_cache_plan(&a, nullptr), SEEDLM_E_INVALID);
  a = plan();
  a.requests = INT_MAX;
  expect("plan requests", seedlm_cache_plan(&a, nullptr), SEEDLM_E_INVALID);
  a = plan();
  a.max_pages = a.page_size = a.pool = a.tokens = INT_MAX, a.table_stride = INT64_MAX;
  expect("plan largest sizes", seedlm_cache_plan(&a, nullptr), SEEDLM_E_UNSUPPORTED);
  a = plan();
  a.page_size = INT_MIN, a.tokens = INT_MIN, a.table_stride = INT64_MIN;
  expect("plan smallest sizes", seedlm_cache_plan(&a, nullptr), SEEDLM_E_INVALID);
  a = plan();
  a.requests = SEEDLM_MAX_REQUESTS, a.tokens = 1 << 30, a.lens_out = const_cast<int32_t*>(a.lens);
  expect("plan without scratch", seedlm_cache_plan(&a, nullptr), SEEDLM_E_NOMEM);
}

void check_append() {
  expect("append null", seedlm_cache_append(nullptr, nullptr), SEEDLM_E_INVALID);
  for (int64_t most : {INT64_MAX, INT64_MIN}) {
    seedlm_cache_append_args a = append();
    a.cache.pages = most;
    a.cache.page_stride = a.cache.token_stride = a.cache.head_stride = most;
    expect("append cache", seedlm_cache_append(&a, nullptr),
           most < 0 ? SEEDLM_E_INVALID : SEEDLM_E_UNSUPPORTED);
    a = append();
    a.q_stride = a.k_stride = a.v_stride = a.q_out_stride = most, a.tokens = INT_MAX;
    expect("append strides", seedlm_cache_append(&a, nullptr),
           SEEDLM_E_UNSUPPORTED);
  }
  seedlm_cache_append_args a = append();
  a.heads = a.cache.kv_heads = a.cache.page_size = a.cache.head_dim = a.rot = INT_MAX;
  a.cache.pages = 1;
  expect("append largest sizes", seedlm_cache_append(&a, nullptr), SEEDLM_E_UNSUPPORTED);
  a = append();
  a.tokens = 0, a.q = nullptr;
  expect("append of no tokens", seedlm_cache_append(&a, nullptr), SEEDLM_OK);
}

void refuse_attend(const char* what, const seedlm_cache_attend_args& a, int want) {
  size_t bytes = 0;
  expect(what, seedlm_cache_attend(&a, nullptr), want);
  expect(what, seedlm_cache_attend_scratch_bytes(&a, &bytes), want);
}

void check_attend() {
  size_t bytes = 0;
  expect("attend null", seedlm_cache_attend(nullptr, nullptr), SEEDLM_E_INVALID);
  seedlm_cache_attend_args a = attend();
  expect("attend bytes null", seedlm_cache_attend_scratch_bytes(&a, nullptr), SEEDLM_E_INVALID);
  constexpr int64_t kMost = INT64_MAX / 8 * 8;
  a.cache.head_stride = kMost;
  refuse_attend("attend head stride", a, SEEDLM_E_UNSUPPORTED);
  a.cache.kv_heads = a.heads = 16384, a.q_stride = a.out_stride = 1 << 20;
  refuse_attend("attend head stride of many heads", a, SEEDLM_E_UNSUPPORTED);
  a = attend();
  a.cache.token_stride = kMost;
  refuse_attend("attend token stride", a, SEEDLM_E_UNSUPPORTED);
  a = attend();
  a.cache.page_stride = kMost;
  refuse_attend("attend page stride", a, SEEDLM_E_UNSUPPORTED);
  a.cache.page_stride = a.cache.token_stride = a.cache.head_stride = kMost;
  refuse_attend("attend strides", a, SEEDLM_E_UNSUPPORTED);
  a = attend();  // each below its own bound, their sum above 2^35
  a.cache.page_stride = ((int64_t)1 << 35) / 10 / 8 * 8 - 8;
  a.cache.token_stride = ((int64_t)1 << 31) - 8;
  a.cache.head_stride = ((int64_t)1 << 34) - 8;
  refuse_attend("attend sum of strides", a, SEEDLM_E_UNSUPPORTED);
  a = attend();
  a.max_pages = a.max_len = INT_MAX, a.table_stride = INT64_MAX;
  refuse_attend("attend longest", a, SEEDLM_E_UNSUPPORTED);
  a = attend();
  a.queries = a.table_rows = SEEDLM_MAX_REQUESTS, a.max_pages = a.max_len = 1 << 30;
  a.table_stride = 1 << 30;
  refuse_attend("attend longest of most queries", a, SEEDLM_E_UNSUPPORTED);
  a.max_len = 1 << 25;
  expect("attend bytes of the most", seedlm_cache_attend_scratch_bytes(&a, &bytes), SEEDLM_OK);
  expect("attend without scratch", seedlm_cache_attend(&a, nullptr), SEEDLM_E_NOMEM);
  a = attend();
  a.queries = a.heads = a.table_rows = a.max_pages = a.max_len = INT_MIN;
  refuse_attend("attend smallest", a, SEEDLM_E_INVALID);
}

void check_lora() {
  size_t bytes = 0;
  const float* scales = reinterpret_cast<float*>(kP);
  auto call = [&](const char* what, const seedlm_lora_site* s, int n, int64_t tokens, int adapters,
                  int want) {
    expect(what, seedlm_lora_many(s, n, g_mem, scales, tokens, adapters, SEEDLM_F16, SEEDLM_F16,
                                  nullptr), want);
  };
  const seedlm_lora_site site{kP, kP, kP, kP, kP, 64, 32, 8};
  call("lora null", nullptr, 1, 4, 2, SEEDLM_E_INVALID);
  call("lora none", nullptr, 0, 4, 2, SEEDLM_OK);
  call("lora no tokens", &site, 1, 0, 2, SEEDLM_OK);
  call("lora negative", &site, INT_MIN, 4, 2, SEEDLM_E_INVALID);
  call("lora adapters", &site, 1, 4, INT_MIN, SEEDLM_E_INVALID);
  call("lora tokens", &site, 1, INT64_MAX, 2, SEEDLM_E_UNSUPPORTED);
  seedlm_lora_site big = site;
  big.rows = big.cols = INT64_MAX;
  call("lora largest site", &big, 1, 4, 2, SEEDLM_E_UNSUPPORTED);
  big.rank = INT_MAX;
  call("lora rank", &big, 1, 4, 2, SEEDLM_E_INVALID);
  seedlm_lora_site most[9];
  for (seedlm_lora_site& s : most) {
    s = site;
    s.rows = s.cols = (1 << 24) - 8, s.rank = SEEDLM_MAX_RANK;
  }
  for (int adapters : {1, 8191, 8192, INT_MAX})
    for (int64_t tokens : {1, 64, (1 << 20) - 1})
      for (int dt : {SEEDLM_F16, SEEDLM_F32})
        expect("lora bytes of the most",
               seedlm_lora_scratch_bytes(most, 9, tokens, adapters, dt, dt, &bytes), SEEDLM_OK);
  call("lora without scratch", most, 9, (1 << 20) - 1, INT_MAX, SEEDLM_E_NOMEM);
  expect("lora bytes null", seedlm_lora_scratch_bytes(most, 9, 4, 2, 1, 1, nullptr),
         SEEDLM_E_INVALID);
}

}  // namespace

int main() {
  check_plan();
  check_append();
  check_attend();
  check_lora();
  printf("serving checks: %d failure(s)\n", g_failures);
  return g_failures ? 1 : 0;
}
