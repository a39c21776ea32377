// Units of rotated elements: their loads and stores in both append kernels, and their
// rotation in that of the quantised cache.
#pragma once

#include <hip/hip_fp16.h>

#include "seedlm_internal.h"

namespace seedlm {

// N elements at p as fp32, and back; N * sizeof(T) bytes, aligned to 16 where
// that is a multiple of 16.
template <int N, typename T>
__device__ void load(const T* p, float (&v)[N]) {
  if constexpr (N == 8 && sizeof(T) == 2) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const __half* h = reinterpret_cast<const __half*>(&u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __half2float(h[i]);
  } else if constexpr (N == 8) {
    const float4 a = reinterpret_cast<const float4*>(p)[0];
    const float4 b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    static_assert(N == 1, "");
    v[0] = (float)p[0];
  }
}

// STREAM: past the caches.
template <int N, bool STREAM = false, typename T>
__device__ void store(T* p, const float (&v)[N]) {
  typedef uint32_t v4u __attribute__((ext_vector_type(4)));
  [[maybe_unused]] auto put = [&](auto x, int i) {
    v4u* at = reinterpret_cast<v4u*>(p) + i;
    if (STREAM) __builtin_nontemporal_store(__builtin_bit_cast(v4u, x), at);
    else *at = __builtin_bit_cast(v4u, x);
  };
  if constexpr (N == 8 && sizeof(T) == 2) {
    uint4 u;
    __half* h = reinterpret_cast<__half*>(&u);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = __float2half_rn(v[i]);
    put(u, 0);
  } else if constexpr (N == 8) {
    put(make_float4(v[0], v[1], v[2], v[3]), 0);
    put(make_float4(v[4], v[5], v[6], v[7]), 1);
  } else {
    p[0] = (T)v[0];
  }
}

// A unit's two runs of N elements: the halves of N rotated pairs, or (as interleaved
// pairs and unrotated elements are) 2N in a row.
template <int N>
struct RotaryUnit {
  int lo, hi;
  bool rotated, split;
  __device__ RotaryUnit(int unit, int rot, bool interleaved) {
    const int e0 = unit * 2 * N;
    rotated = e0 < rot;
    split = rotated && !interleaved;
    lo = split ? unit * N : e0;
    hi = split ? lo + rot / 2 : e0 + N;
  }
  // Turns the unit's runs x and y by the angles of cosines c and sines s.
  __device__ void turn(float (&x)[N], float (&y)[N], const float (&c)[N], const float (&s)[N]) const {
    if (split) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float u = x[i], w = y[i];
        x[i] = u * c[i] - w * s[i];
        y[i] = w * c[i] + u * s[i];
      }
    } else {
      // elements 2i, 2i + 1 of the 2N in a row
      float z[2 * N];
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = x[i], z[N + i] = y[i];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float u = z[2 * i], w = z[2 * i + 1];
        z[2 * i] = u * c[i] - w * s[i];
        z[2 * i + 1] = w * c[i] + u * s[i];
      }
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = z[i], y[i] = z[N + i];
    }
  }
};

inline bool aligned16(const void* p) { return (uintptr_t)p % 16 == 0; }

}  // namespace seedlm
