// Host-side driver for test_host_stream_order.py.  It defines the HIP runtime
// calls that libseedlm.so makes (launches do nothing but note who made them,
// device memory is heap memory), loads the library on top of them, and calls it
// from several host threads.  No GPU is used.
//
//   host_stream_order_check <libseedlm.so> same
//       threads on one stream: the launches of each call have to follow one
//       another without another call's between them, since they hand partial
//       results on through the stream's scratch
//   host_stream_order_check <libseedlm.so> other
//       calls on two streams: neither waits for the other
//   host_stream_order_check <libseedlm.so> release
//       seedlm_scratch_release beside a call: no launch gets freed memory
//   host_stream_order_check <libseedlm.so> loads
//       attention whose queries may share their tokens runs the kernel whose loads
//       stay in the caches, whatever the bound on its lengths
//
// Exit status 0 when the check holds.
#include <dlfcn.h>
#include <hip/hip_runtime_api.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include <unistd.h>

#include <atomic>
#include <condition_variable>
#include <functional>
#include <map>
#include <mutex>
#include <string>
#include <thread>
#include <vector>

#include "seedlm_serve.h"

namespace {

struct Launch {
  hipStream_t stream;
  int call;
  const void* kernel;
};
std::mutex g_mu;
std::condition_variable g_changed;
std::vector<Launch> g_launches;
std::map<char*, size_t> g_live;  // device allocations
std::atomic<int> g_failures{0}, g_calls{0};
thread_local int t_call = -1;         // the call that this thread is in
thread_local int t_nth = 0;           // launches of it so far
std::function<void(void** args)> g_on_launch;

struct Config {
  dim3 grid, block;
  size_t lds;
  hipStream_t stream;
};
thread_local Config t_config;

void fail(const char* what) {
  fprintf(stderr, "FAIL %s\n", what);
  ++g_failures;
}

hipError_t launch(const void* kernel, hipStream_t stream, void** args) {
  {
    std::lock_guard<std::mutex> lock(g_mu);
    g_launches.push_back({stream, t_call, kernel});
  }
  ++t_nth;
  g_changed.notify_all();
  if (g_on_launch) g_on_launch(args);
  return hipSuccess;
}

bool live(const void* p) {
  std::lock_guard<std::mutex> lock(g_mu);
  for (const auto& a : g_live)
    if (p >= a.first && p < a.first + a.second) return true;
  return false;
}

}  // namespace

extern "C" {

hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, hipStream_t stream) {
  t_config = {grid, block, lds, stream};
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* stream) {
  *grid = t_config.grid;
  *block = t_config.block;
  *lds = t_config.lds;
  *stream = t_config.stream;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void* kernel, dim3, dim3, void** args, size_t, hipStream_t stream) {
  return launch(kernel, stream, args);
}
hipError_t hipExtLaunchKernel(const void* kernel, dim3, dim3, void** args, size_t, hipStream_t stream,
                              hipEvent_t, hipEvent_t, int) {
  return launch(kernel, stream, args);
}
hipError_t hipMalloc(void** p, size_t n) {
  *p = aligned_alloc(256, (n + 255) / 256 * 256);
  std::lock_guard<std::mutex> lock(g_mu);
  if (*p) g_live[static_cast<char*>(*p)] = n;
  return *p ? hipSuccess : hipErrorOutOfMemory;
}
hipError_t hipFree(void* p) {
  {
    std::lock_guard<std::mutex> lock(g_mu);
    g_live.erase(static_cast<char*>(p));
  }
  free(p);
  return hipSuccess;
}
hipError_t hipHostMalloc(void** p, size_t n, unsigned) {
  *p = malloc(n);
  return *p ? hipSuccess : hipErrorOutOfMemory;
}
hipError_t hipHostFree(void* p) {
  free(p);
  return hipSuccess;
}
hipError_t hipMemcpy(void* to, const void* from, size_t n, hipMemcpyKind) {
  memcpy(to, from, n);
  return hipSuccess;
}
hipError_t hipGetDevice(int* d) {
  *d = 0;
  return hipSuccess;
}
hipError_t hipSetDevice(int) { return hipSuccess; }
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) {
  *v = 256;
  return hipSuccess;
}
hipError_t hipDeviceSynchronize() { return hipSuccess; }
hipError_t hipStreamSynchronize(hipStream_t) { return hipSuccess; }
hipError_t hipGetLastError() { return hipSuccess; }

}  // extern "C"

namespace {

template <typename F>
F symbol(void* lib, const char* name) {
  F f = reinterpret_cast<F>(dlsym(lib, name));
  if (!f) {
    fprintf(stderr, "no %s\n", name);
    exit(2);
  }
  return f;
}

struct Call {
  std::string name;
  std::function<int(void* stream)> run;
};

// The library's calls that take more than one launch.  The pointers are never
// dereferenced: no kernel runs.
struct Calls {
  void* const p = reinterpret_cast<void*>(4096);
  void* const q = reinterpret_cast<void*>(1 << 20);
  int32_t* const i = static_cast<int32_t*>(p);
  int32_t* const j = static_cast<int32_t*>(q);
  std::vector<Call> all;

  explicit Calls(void* lib) {
    const auto plan = symbol<decltype(&seedlm_cache_plan)>(lib, "seedlm_cache_plan");
    const auto attend = symbol<decltype(&seedlm_cache_attend)>(lib, "seedlm_cache_attend");
    const auto lora = symbol<decltype(&seedlm_lora_many)>(lib, "seedlm_lora_many");
    const auto pack = symbol<decltype(&seedlm_pack)>(lib, "seedlm_pack");
    const auto gemv = symbol<decltype(&seedlm_gemv)>(lib, "seedlm_gemv");
    const auto gemm = symbol<decltype(&seedlm_gemm)>(lib, "seedlm_gemm");

    seedlm_cache_plan_args a{};
    a.lens = i, a.fresh = j, a.table = j, a.ring = j, a.ring_state = j + 64;
    a.lens_out = i, a.ring_state_out = j + 64, a.offsets = j, a.ok = j;
    a.rows = a.positions = a.slots = j;
    a.table_stride = a.max_pages = 64;
    a.requests = 8, a.page_size = 16, a.pool = 512, a.tokens = 5000;
    all.push_back({"cache_plan", [=](void* s) { return plan(&a, s); }});

    seedlm_cache_attend_args t{};
    t.q = p, t.out = q, t.table = i, t.lens = j;
    t.cache = {p, q, 1000, 16 * 2 * 128, 2 * 128, 128, 16, 2, 128};
    t.q_stride = t.out_stride = 4 * 128;
    t.table_stride = t.max_pages = 512;
    t.queries = t.table_rows = 3, t.heads = 4, t.max_len = 8192;
    t.x_dtype = SEEDLM_F16, t.scale = 0.1f;
    all.push_back({"cache_attend", [=](void* s) { return attend(&t, s); }});

    for (int64_t tokens : {5, 2048}) {  // the row kernels, and the tiles
      const seedlm_lora_site site{p, p, p, q, q, 4096, 4096, 32};
      all.push_back({"lora_many of " + std::to_string(tokens), [=](void* s) {
                       return lora(&site, 1, i, static_cast<float*>(p), tokens, 4, SEEDLM_F16,
                                   SEEDLM_F16, s);
                     }});
    }

    const int64_t rows = 2048, cols = 4096, blocks = rows * cols / 8;
    std::vector<uint16_t> seeds(blocks, 1);
    std::vector<int8_t> coeffs(blocks * 3, 1), exps(blocks, 0);
    seedlm_handle h = nullptr;
    if (pack(seeds.data(), coeffs.data(), exps.data(), rows, cols, 8, 3, 16, &h) != SEEDLM_OK)
      fail("pack");
    all.push_back({"gemv", [=](void* s) {
                     return gemv(h, p, q, 4, SEEDLM_F16, SEEDLM_F16, s);
                   }});
    all.push_back({"gemm", [=](void* s) {
                     return gemm(h, p, q, 100, SEEDLM_F16, SEEDLM_F16, s);
                   }});
  }
};

void make(const Call& c, void* stream) {
  t_call = g_calls++;
  t_nth = 0;
  if (c.run(stream) != SEEDLM_OK) fail(c.name.c_str());
  if (t_nth < 2) fail((c.name + ": one launch, which shows nothing").c_str());
}

int same(const Calls& calls) {
  g_on_launch = [](void**) { usleep(300); };  // the others' turn
  std::vector<std::thread> threads;
  for (const Call& c : calls.all)
    threads.emplace_back([&c] {
      for (int k = 0; k < 20; ++k) make(c, nullptr);
    });
  for (std::thread& t : threads) t.join();
  std::map<int, bool> ended;
  int mixed = 0;
  for (size_t k = 0; k < g_launches.size(); ++k) {
    if (k > 0 && g_launches[k].call != g_launches[k - 1].call) ended[g_launches[k - 1].call] = true;
    mixed += ended.count(g_launches[k].call) ? 1 : 0;
  }
  if (mixed) fprintf(stderr, "%d of %zu launches follow another call's\n", mixed, g_launches.size());
  if (mixed) fail("calls on one stream mix their launches");
  return g_failures != 0;
}

int other(const Calls& calls) {
  // The first launch on stream 16 waits for one on stream 32.
  std::atomic<bool> first{true};
  g_on_launch = [&](void**) {
    if (t_call != 0 || !first.exchange(false)) return;
    std::unique_lock<std::mutex> lock(g_mu);
    const bool met = g_changed.wait_for(lock, std::chrono::seconds(20), [] {
      for (const Launch& l : g_launches)
        if (l.stream == reinterpret_cast<hipStream_t>(32)) return true;
      return false;
    });
    if (!met) fail("a call on one stream waits for a call on another");
  };
  std::thread one([&] { make(calls.all[1], reinterpret_cast<void*>(16)); });
  while (true) {
    std::lock_guard<std::mutex> lock(g_mu);
    if (!g_launches.empty()) break;
  }
  std::thread two([&] { make(calls.all[1], reinterpret_cast<void*>(32)); });
  one.join();
  two.join();
  return g_failures != 0;
}

int release(const Calls& calls, void* lib) {
  const auto free_all = symbol<decltype(&seedlm_scratch_release)>(lib, "seedlm_scratch_release");
  std::thread beside;
  g_on_launch = [&](void** args) {
    if (t_nth == 1) {  // after the plan's main launch, before its copy out of scratch
      beside = std::thread([&] {
        if (free_all() != SEEDLM_OK) fail("release");
      });
      usleep(100000);
    } else if (!live(*static_cast<void**>(args[0]))) {
      fail("a launch got scratch that had been freed");
    }
  };
  make(calls.all[0], nullptr);
  beside.join();
  g_on_launch = nullptr;
  make(calls.all[0], nullptr);  // allocates again
  return g_failures != 0;
}

int loads(void* lib) {
  const auto attend = symbol<decltype(&seedlm_cache_attend)>(lib, "seedlm_cache_attend");
  int32_t* const i = reinterpret_cast<int32_t*>(4096);
  auto kernel_of = [&](int queries, const int32_t* rows, int dim, int dtype) {
    seedlm_cache_attend_args t{};
    t.q = i, t.out = i, t.table = i, t.lens = i, t.rows = rows;
    t.cache = {i, i, 100000, 16 * 2 * dim, 2 * dim, dim, 16, 2, dim};
    t.q_stride = t.out_stride = 4 * dim;
    t.table_stride = t.max_pages = 512;
    t.queries = t.table_rows = queries, t.heads = 4, t.max_len = 8192;
    t.x_dtype = dtype, t.scale = 0.1f;
    g_launches.clear();
    if (attend(&t, nullptr) != SEEDLM_OK || g_launches.empty()) fail("attend");
    return g_launches.empty() ? nullptr : g_launches[0].kernel;
  };
  for (int dim : {128, 256})
    for (int dtype : {SEEDLM_F32, SEEDLM_F16}) {
      const void* cached = kernel_of(3, nullptr, dim, dtype);  // 25 and 50 MB at most
      if (kernel_of(64, nullptr, dim, dtype) == cached) fail("64 requests of 8192 tokens are small");
      if (kernel_of(64, i, dim, dtype) != cached) fail("queries that may share tokens pass the caches");
    }
  return g_failures != 0;
}

}  // namespace

int main(int argc, char** argv) {
  if (argc != 3) return 2;
  void* lib = dlopen(argv[1], RTLD_NOW | RTLD_LOCAL);
  if (!lib) {
    fprintf(stderr, "%s\n", dlerror());
    return 2;
  }
  const Calls calls(lib);
  g_launches.clear();
  const std::string mode = argv[2];
  const int rc = mode == "same" ? same(calls) : mode == "other" ? other(calls)
               : mode == "release" ? release(calls, lib) : mode == "loads" ? loads(lib) : 2;
  printf("%s: %d failure(s)\n", argv[2], g_failures.load());
  return rc;
}
