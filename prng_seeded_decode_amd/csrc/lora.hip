// Low-rank adapters of many requests beside shared projections
// (seedlm_lora_many): y[t] = base[t] + scales[a] B_a (A_a x[t]), a = adapter[t],
// for up to 8 sites (projections) in one pair of launches.
//
// First launch: h = A x, cut along the columns into chunks so that few rows
// still fill the chip; chunk sums go to scratch as fp32 [site][chunk][token][rank].
// Second launch: adds the chunks in order, multiplies with B, scales, adds base
// and rounds once.  At a few rows the bytes of A and B bound both; at many the
// bytes of x, base and y.
#include <hip/hip_fp16.h>

#include "seedlm_internal.h"

namespace seedlm {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kChunk = 1024;  // columns of a workgroup of the row kernels

struct Site {
  const void* x;
  const __half* A;
  const __half* B;
  const void* base;
  void* y;
  float* h;       // [chunks][tokens][rank]
  int rows, cols, rank;
  int chunks;
  int wide;       // 16-byte accesses fit
  int first_down; // first workgroup (x dimension) of this site in the two launches
  int first_up;
};

struct LoraArgs {
  Site s[kLoraGroup];
  const int32_t* adapter;
  const float* scales;
  int n, tokens, adapters;
};

__device__ const Site& site_of(const LoraArgs& p, bool up, int block) {
  int i = 0;
  for (int k = 1; k < p.n; ++k)
    if (block >= (up ? p.s[k].first_up : p.s[k].first_down)) i = k;
  return p.s[i];
}

__device__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

template <typename T>
__device__ void load8(const T* p, float (&v)[8]) {
  if constexpr (sizeof(T) == 2) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const __half* h = reinterpret_cast<const __half*>(&u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __half2float(h[i]);
  } else {
    const float4 a = reinterpret_cast<const float4*>(p)[0];
    const float4 b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}

// h of one token and one chunk of columns: a wave takes the ranks in turn, its
// lanes 8 neighbouring columns each (one by one where 16-byte loads do not fit).
template <typename XT>
__global__ __launch_bounds__(kThreads) void lora_down_rows_kernel(const LoraArgs p) {
  const Site& s = site_of(p, false, blockIdx.x);
  const int chunk = blockIdx.x - s.first_down;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int t = blockIdx.y; t < p.tokens; t += gridDim.y) {
    const int a = p.adapter[t];
    if (a < 0 || a >= p.adapters) continue;
    const int c0 = chunk * kChunk, c1 = min(s.cols, c0 + kChunk);
    const XT* x = static_cast<const XT*>(s.x) + (int64_t)t * s.cols;
    const __half* A = s.A + (int64_t)a * s.rank * s.cols;
    float* h = s.h + ((int64_t)chunk * p.tokens + t) * s.rank;
    if (s.wide) {
      constexpr int kSteps = kChunk / 512;
      float xv[kSteps][8];
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        const int c = c0 + k * 512 + lane * 8;
        if (c < c1) load8(x + c, xv[k]);
        else
#pragma unroll
          for (int i = 0; i < 8; ++i) xv[k][i] = 0.f;
      }
#pragma unroll 2
      for (int j = wave; j < s.rank; j += kWaves) {
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          const int c = c0 + k * 512 + lane * 8;
          if (c < c1) {
            float av[8];
            load8(A + (int64_t)j * s.cols + c, av);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(av[i], xv[k][i], sum);
          }
        }
        sum = wave_sum(sum);
        if (lane == 0) h[j] = sum;
      }
    } else {
      for (int j = wave; j < s.rank; j += kWaves) {
        float sum = 0.f;
        for (int c = c0 + lane; c < c1; c += 64)
          sum = fmaf(__half2float(A[(int64_t)j * s.cols + c]), (float)x[c], sum);
        sum = wave_sum(sum);
        if (lane == 0) h[j] = sum;
      }
    }
  }
}

// y of one token and kThreads rows, a row per thread.
template <typename YT>
__global__ __launch_bounds__(kThreads) void lora_up_rows_kernel(const LoraArgs p) {
  __shared__ float s_h[SEEDLM_MAX_RANK];
  const Site& s = site_of(p, true, blockIdx.x);
  const int r = (blockIdx.x - s.first_up) * kThreads + threadIdx.x;
  for (int t = blockIdx.y; t < p.tokens; t += gridDim.y) {
    const int a = p.adapter[t];
    const bool has = a >= 0 && a < p.adapters;
    if (!has && s.y == s.base) continue;
    if (has) {
      __syncthreads();  // s_h of the token before has been read
      const float scale = p.scales[a];
      for (int j = threadIdx.x; j < s.rank; j += kThreads) {
        float sum = 0.f;
        for (int c = 0; c < s.chunks; ++c) sum += s.h[((int64_t)c * p.tokens + t) * s.rank + j];
        s_h[j] = sum * scale;
      }
      __syncthreads();
    }
    if (r >= s.rows) continue;
    const int64_t at = (int64_t)t * s.rows + r;
    float sum = (float)static_cast<const YT*>(s.base)[at];
    if (has) {
      const __half* B = s.B + ((int64_t)a * s.rows + r) * s.rank;
      float d = 0.f;
      if (s.wide) {
        for (int j = 0; j < s.rank; j += 8) {
          float bv[8];
          load8(B + j, bv);
#pragma unroll
          for (int i = 0; i < 8; ++i) d = fmaf(bv[i], s_h[j + i], d);
        }
      } else {
        for (int j = 0; j < s.rank; ++j) d = fmaf(__half2float(B[j]), s_h[j], d);
      }
      sum += d;
    }
    static_cast<YT*>(s.y)[at] = (YT)sum;
  }
}

bool aligned16(const void* p) { return (uintptr_t)p % 16 == 0; }

size_t site_floats(const seedlm_lora_site& s, int64_t tokens) {
  const int64_t chunks = (s.cols + kChunk - 1) / kChunk;
  return (size_t)((chunks * tokens * s.rank + 63) / 64 * 64);
}

template <typename XT, typename YT>
int run(const LoraArgs& p, int down, int up, hipStream_t s) {
  const int rows = p.tokens < 65535 ? p.tokens : 65535;
  hipLaunchKernelGGL(lora_down_rows_kernel<XT>, dim3(down, rows), dim3(kThreads), 0, s, p);
  hipLaunchKernelGGL(lora_up_rows_kernel<YT>, dim3(up, rows), dim3(kThreads), 0, s, p);
  return hipGetLastError() == hipSuccess ? SEEDLM_OK : SEEDLM_E_DEVICE;
}

}  // namespace

// The groups run one after another and share the scratch of the largest.
size_t lora_scratch_bytes(const seedlm_lora_site* sites, int n, int64_t tokens, int xdt, int ydt) {
  size_t most = 0;
  for (int i = 0; i < n; i += kLoraGroup) {
    size_t floats = 0;
    for (int k = i; k < n && k < i + kLoraGroup; ++k) floats += site_floats(sites[k], tokens);
    if (floats > most) most = floats;
  }
  return most * sizeof(float);
}

int launch_lora(const seedlm_lora_site* sites, int n, const int32_t* adapter, const float* scales,
                int64_t tokens, int adapters, int xdt, int ydt, float* scratch, hipStream_t s) {
  for (int i = 0; i < n; i += kLoraGroup) {
    LoraArgs p{};
    p.adapter = adapter;
    p.scales = scales;
    p.tokens = (int)tokens;
    p.adapters = adapters;
    float* h = scratch;
    int down = 0, up = 0;
    for (; p.n < kLoraGroup && i + p.n < n; ++p.n) {
      const seedlm_lora_site& in = sites[i + p.n];
      Site& o = p.s[p.n];
      o.x = in.x;
      o.A = static_cast<const __half*>(in.A);
      o.B = static_cast<const __half*>(in.B);
      o.base = in.base;
      o.y = in.y;
      o.h = h;
      o.rows = (int)in.rows;
      o.cols = (int)in.cols;
      o.rank = in.rank;
      o.chunks = (int)((in.cols + kChunk - 1) / kChunk);
      o.wide = in.cols % 8 == 0 && in.rank % 8 == 0 && aligned16(in.x) && aligned16(in.A) &&
               aligned16(in.B);
      o.first_down = down;
      o.first_up = up;
      down += o.chunks;
      up += (int)((in.rows + kThreads - 1) / kThreads);
      h += site_floats(in, tokens);
    }
    int st;
    if (xdt == SEEDLM_F16)
      st = ydt == SEEDLM_F16 ? run<__half, __half>(p, down, up, s) : run<__half, float>(p, down, up, s);
    else
      st = ydt == SEEDLM_F16 ? run<float, __half>(p, down, up, s) : run<float, float>(p, down, up, s);
    if (st != SEEDLM_OK) return st;
  }
  return SEEDLM_OK;
}

}  // namespace seedlm
