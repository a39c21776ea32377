// A quantised cache: rotary positions on q and k with k and v quantised into their
// slots (seedlm_qcache_append), and slots read back (seedlm_qcache_read).
//
// A group of x of a row gets offset o = min x, scale s = fp16((max x - o) / levels) and
// codes c = rint((x - o) / s); it reads back as o + s c.  The x are fp16 numbers, so o
// is exact.  Each element is read and written once with some 20 operations, so memory
// bandwidth bounds both.
//
// Four lanes take a row, four units each: for every i elements 16i + 4u .. 16i + 4u + 3
// of lane u, one load of 8 or 16 bytes.  A lane then has whole units of codes, which it
// packs in registers, and a group's extremes are its own over some i and two exchanges
// with its neighbours.  The other half of a rotated pair is loaded too (it is in the
// caches) and not exchanged, so that any part of a head may turn.  q goes through the
// units of rotary.h in workgroups of its own.
//
// Measured (medians, one MI355X): append of 4097 tokens, 32/32 heads of 128, 4 bits, a
// group a row: 34.5 us; read of the same 21.6; read of 32771 tokens, two groups: 28.1 us
// for 170 MB, 6.0 TB/s, the rate of a streaming read.  Small calls are a launch and a
// chain of loads: append of 16 tokens 4.2, read of 300 tokens 3.2.  Dropped: a read with
// four rows to a thread (47 us where this form had 43), an append with six waves to a
// SIMD or four (46 and 38.3, five 34.5).
#include <type_traits>

#include "divisor.h"
#include "rotary.h"

namespace seedlm {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = kThreads / 4;  // rows of a workgroup
constexpr int64_t kL2Bytes = 32 << 20;  // of all XCDs: larger outputs pass the caches

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

// Four elements at p as fp32; VEC: aligned to their size.
template <bool VEC, typename T>
__device__ void load4(const T* p, float (&v)[4]) {
  if constexpr (VEC && sizeof(T) == 2) {
    const v2u u = *reinterpret_cast<const v2u*>(p);
    const __half* h = reinterpret_cast<const __half*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __half2float(h[i]);
  } else if constexpr (VEC) {
    const float4 u = *reinterpret_cast<const float4*>(p);
    v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (float)p[i];
  }
}

template <bool VEC, typename T>
__device__ void store4(T* p, const float (&v)[4]) {
  if constexpr (VEC && sizeof(T) == 2) {
    v2u u;
    __half* h = reinterpret_cast<__half*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __float2half_rn(v[i]);
    *reinterpret_cast<v2u*>(p) = u;
  } else if constexpr (VEC) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = (T)v[i];
  }
}

// A lane's elements 16i + 4u .. 16i + 4u + 3 of its head's row, in y[i], turned by a
// token's cosines and sines where they lie below rot.  Each operation is rounded: codes
// next to a border must not depend on how the compiler joins them.  All loads of a step
// are requested before the first is used.
template <int kI, typename T>
__device__ void turn_fours(const T* x, int u, int rot, bool interleaved, bool is_k, const float* cos,
                           const float* sin, float (&y)[kI][4]) {
#pragma clang fp contract(off)
  if (interleaved) {
    constexpr int kStep = 4;
#pragma unroll
    for (int i0 = 0; i0 < kI; i0 += kStep) {
      float2 c[kStep], s[kStep];
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        const int e = min(16 * (i0 + i) + 4 * u, rot - 4);
        c[i] = *reinterpret_cast<const float2*>(cos + e / 2);
        s[i] = *reinterpret_cast<const float2*>(sin + e / 2);
      }
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        float(&z)[4] = y[i0 + i];
        const bool on = is_k && 16 * (i0 + i) + 4 * u < rot;
        const float a0 = z[0], b0 = z[1], a1 = z[2], b1 = z[3];
        const float w[4] = {a0 * c[i].x - b0 * s[i].x, b0 * c[i].x + a0 * s[i].x,
                            a1 * c[i].y - b1 * s[i].y, b1 * c[i].y + a1 * s[i].y};
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j] = on ? w[j] : z[j];
      }
    }
  } else if (rot == 16 * kI) {  // the whole head: both halves of a pair are the lane's
    float c[kI / 2][4], s[kI / 2][4];
#pragma unroll
    for (int i = 0; i < kI / 2; ++i) {
      load4<true>(cos + 16 * i + 4 * u, c[i]);
      load4<true>(sin + 16 * i + 4 * u, s[i]);
    }
#pragma unroll
    for (int i = 0; i < kI / 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = y[i][j], b = y[i + kI / 2][j];
        const float za = a * c[i][j] - b * s[i][j], zb = b * c[i][j] + a * s[i][j];
        y[i][j] = is_k ? za : a;
        y[i + kI / 2][j] = is_k ? zb : b;
      }
  } else {  // the other half of a pair is in the caches
    const int half = rot / 2;
    constexpr int kStep = 2;
#pragma unroll
    for (int i0 = 0; i0 < kI; i0 += kStep) {
      float o[kStep][4], c[kStep][4], s[kStep][4];
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        const int e = min(16 * (i0 + i) + 4 * u, rot - 4);
        load4<true>(x + (e >= half ? e - half : e + half), o[i]);
        load4<true>(cos + (e >= half ? e - half : e), c[i]);
        load4<true>(sin + (e >= half ? e - half : e), s[i]);
      }
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        const int e = 16 * (i0 + i) + 4 * u;
        const bool on = is_k && e < rot;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float v = y[i0 + i][j] * c[i][j], w = o[i][j] * (e >= half ? s[i][j] : -s[i][j]);
          y[i0 + i][j] = on ? v + w : y[i0 + i][j];
        }
      }
    }
  }
}

// The same for rows and angles at any address, element by element.
template <int kI, typename T>
__device__ void turn_each(const T* x, int u, int rot, bool interleaved, const float* cos,
                          const float* sin, float (&y)[kI][4]) {
#pragma clang fp contract(off)
  const int half = rot / 2;
#pragma unroll
  for (int i = 0; i < kI; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = 16 * i + 4 * u + j;
      if (e >= rot) continue;
      const int pair = interleaved ? e / 2 : e % half;
      const bool second = interleaved ? e % 2 : e >= half;
      const float a = (float)x[interleaved ? 2 * pair : pair];
      const float b = (float)x[interleaved ? 2 * pair + 1 : pair + half];
      const float c = cos[pair], s = sin[pair];
      y[i][j] = second ? b * c + a * s : a * c - b * s;
    }
}

// The value of another lane of the same four; CTRL: its place, two bits a lane.
template <int CTRL>
__device__ uint32_t in_row(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
constexpr int kSwapOne = 0xB1, kSwapTwo = 0x4E;  // lanes 1, 0, 3, 2 and 2, 3, 0, 1

// The least and the largest of both halves of x over the four lanes of a row; NaN if
// there is one.
__device__ float least(half2v x) {
  float y = __builtin_elementwise_minimum((float)x[0], (float)x[1]);
  y = __builtin_elementwise_minimum(y, __builtin_bit_cast(float, in_row<kSwapOne>(__builtin_bit_cast(uint32_t, y))));
  return __builtin_elementwise_minimum(y, __builtin_bit_cast(float, in_row<kSwapTwo>(__builtin_bit_cast(uint32_t, y))));
}
__device__ float largest(half2v x) { return -least(-x); }

// N dwords at p, aligned to their size up to 16 bytes.
template <int N>
__device__ void load_dwords(const void* p, uint32_t (&v)[N]) {
  if constexpr (N == 1) {
    v[0] = *static_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const v2u u = *static_cast<const v2u*>(p);
    v[0] = u[0], v[1] = u[1];
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const v4u u = static_cast<const v4u*>(p)[i / 4];
      v[i] = u[0], v[i + 1] = u[1], v[i + 2] = u[2], v[i + 3] = u[3];
    }
  }
}
template <int N>
__device__ void store_dwords(void* p, const uint32_t (&v)[N]) {
  if constexpr (N == 1) {
    *static_cast<uint32_t*>(p) = v[0];
  } else if constexpr (N == 2) {
    *static_cast<v2u*>(p) = v2u{v[0], v[1]};
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) static_cast<v4u*>(p)[i / 4] = v4u{v[i], v[i + 1], v[i + 2], v[i + 3]};
  }
}

// Where a slot's row of a head lies: byte of its codes, number of its first pair.
struct RowAt {
  int64_t codes, pair;
  __device__ RowAt(const seedlm_qcache_t& c, Divisor page_size, int slot, int head) {
    const int page = (int)page_size.of(slot), nth = slot - page * c.page_size;
    codes = page * c.page_stride + nth * c.token_stride + head * c.head_stride;
    pair = page * c.scale_page_stride + nth * c.scale_token_stride + head * c.scale_head_stride;
  }
};

// Rows of k and v lie token after token, a token's keys before its values; a workgroup
// takes whole tokens, or 64 rows of one.
struct RowSplit {
  int tokens;  // of a workgroup
  int passes;  // workgroups of a token
  Divisor rows;  // of a token
  explicit RowSplit(int kv_heads) {
    tokens = 2 * kv_heads < kRows ? kRows / (2 * kv_heads) : 1;
    passes = (2 * kv_heads + kRows - 1) / kRows;
    rows = divisor((uint32_t)(2 * kv_heads));
  }
  // The token (counted in the workgroup) and the row of it that thread row `r` of pass
  // `pass` takes; false for none.
  __device__ bool at(int r, int pass, int kv_heads, int* token, int* row) const {
    *token = passes > 1 ? 0 : (int)rows.of(r);
    *row = passes > 1 ? pass * kRows + r : r - *token * 2 * kv_heads;
    return *token < tokens && *row < 2 * kv_heads;
  }
};

struct AppendArgs {
  seedlm_qcache_append_args a;
  RowSplit split;
  Divisor page_size;
  int units;            // units of a head of q
  Divisor token_units;  // units of a token of q
  bool stream;          // q passes the caches
};

// VEC: k, v and the angles in aligned fours.  N: pairs of a unit of q, 8 with VEC, else 1.
// Waves side by side: five in 128 dimensions (38.3 us for 4097 tokens of 32 heads with four,
// 34.5 with five, 46 with six, whose loads no longer fit the registers together).
template <int D, int BITS, int NG, bool VEC, int N, typename T>
__global__ __launch_bounds__(kThreads, D == 64 ? 8 : (D == 128 ? 5 : 2)) void qcache_append_kernel(const AppendArgs p) {
  const seedlm_qcache_append_args& a = p.a;
  const seedlm_qcache_t& c = a.cache;
  const int64_t t0 = (int64_t)blockIdx.x * p.split.tokens;
  if ((int)blockIdx.y >= p.split.passes) {  // q
    const int i = (blockIdx.y - p.split.passes) * kThreads + threadIdx.x;
    const int token = (int)p.token_units.of(i);
    const int64_t t = t0 + token;
    if (token >= p.split.tokens || t >= a.tokens) return;
    const int j = i - token * p.units * a.heads, h = j / p.units;
    const RotaryUnit<N> u(j - h * p.units, a.rot, a.interleaved);
    const int pos = a.positions[t];
    const bool turns = pos >= 0 && pos < a.table_len;
    const T* src = static_cast<const T*>(a.q) + t * a.q_stride + (int64_t)h * D;
    T* dst = static_cast<T*>(a.q_out) + t * a.q_out_stride + (int64_t)h * D;
    float x[N], y[N];
#pragma unroll
    for (int k = 0; k < N; ++k) x[k] = y[k] = 0.f;
    if (turns) {
      load<N>(src + u.lo, x);
      load<N>(src + u.hi, y);
      if (u.rotated) {
        float co[N], si[N];
        const int64_t at = (int64_t)pos * (a.rot / 2) + (j - h * p.units) * N;
        load<N>(a.cos + at, co);
        load<N>(a.sin + at, si);
        u.turn(x, y, co, si);
      }
    }
    if (N == 8 && p.stream) {
      store<N, true>(dst + u.lo, x);
      store<N, true>(dst + u.hi, y);
    } else {
      store<N>(dst + u.lo, x);
      store<N>(dst + u.hi, y);
    }
    return;
  }
  constexpr int kI = D / 16;                 // codes of a unit
  constexpr int kUnitBytes = kI * BITS / 8;
  constexpr int KD = kUnitBytes;             // dwords of 4 units
  constexpr float kLevels = (1 << BITS) - 1;
  const int u = threadIdx.x & 3;
  int token, row;
  if (!p.split.at(threadIdx.x >> 2, blockIdx.y, c.kv_heads, &token, &row)) return;
  const int64_t t = t0 + token;
  if (t >= a.tokens) return;
  const int pos = a.positions[t], slot = a.slots[t];
  const bool is_v = row >= c.kv_heads;
  const int h = is_v ? row - c.kv_heads : row;
  const T* src = (is_v ? static_cast<const T*>(a.v) + t * a.v_stride
                       : static_cast<const T*>(a.k) + t * a.k_stride) + (int64_t)h * D;
  float y[kI][4];
#pragma unroll
  for (int i = 0; i < kI; ++i) load4<VEC>(src + 16 * i + 4 * u, y[i]);
  if (pos < 0 || pos >= a.table_len || slot < 0 || slot >= c.pages * c.page_size) return;
  const int64_t angle = (int64_t)pos * (a.rot / 2);
  if constexpr (VEC) {
    if (a.rot > 0 && __any(!is_v))
      turn_fours<kI>(src, u, a.rot, a.interleaved, !is_v, a.cos + angle, a.sin + angle, y);
  } else {
    turn_each<kI>(src, u, is_v ? 0 : a.rot, a.interleaved, a.cos + angle, a.sin + angle, y);
  }
  half2v x[kI][2];
#pragma unroll
  for (int i = 0; i < kI; ++i) {
    x[i][0] = half2v{(_Float16)y[i][0], (_Float16)y[i][1]};
    x[i][1] = half2v{(_Float16)y[i][2], (_Float16)y[i][3]};
  }

  uint32_t even[KD], odd[KD], pair[NG];  // bytes of codes of even and of odd i
#pragma unroll
  for (int k = 0; k < KD; ++k) even[k] = odd[k] = 0;
#pragma unroll
  for (int n = 0; n < NG; ++n) {
    constexpr int kN = kI / NG;
    half2v lows = x[n * kN][0], highs = lows;
#pragma unroll
    for (int i = n * kN; i < (n + 1) * kN; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        lows = __builtin_elementwise_minimum(lows, x[i][j]);
        highs = __builtin_elementwise_maximum(highs, x[i][j]);
      }
    const float low = least(lows), high = largest(highs);
    const bool finite = high - low < INFINITY;
    const _Float16 scale = (_Float16)((high - low) / kLevels);
    const float s = (float)scale;
    // (x - o) / s by way of 1 / s is off by less than 2^-22 of itself, 2^-14 here, so it
    // rounds to the same code but within that of the middle between two.  There, and
    // where the last code might be passed, the wave divides.
    const bool codes = finite && s > 0.f;
    const float inverse = codes ? 1.f / s : 0.f;
    const bool passes = (high - low) * inverse > kLevels + 0.25f;
#pragma unroll
    for (int i = n * kN; i < (n + 1) * kN; ++i) {
      float d[4], code[4], off = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        d[j] = (float)x[i][j / 2][j % 2] - low;
        const float y = d[j] * inverse;
        code[j] = rintf(y);
        off = fmaxf(off, fabsf(y - code[j]));
      }
      if (__any(passes || off > 0.5f - 0x1p-14f)) {
#pragma unroll
        for (int j = 0; j < 4; ++j) code[j] = codes ? fminf(rintf(d[j] / s), kLevels) : 0.f;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int byte = j * kUnitBytes + i * BITS / 8;
        uint32_t& w = BITS == 4 && i % 2 ? odd[byte / 4] : even[byte / 4];
        w = __builtin_amdgcn_cvt_pk_u8_f32(code[j], byte % 4, w);
      }
    }
    const uint32_t lo = __builtin_bit_cast(uint16_t, scale);
    const uint32_t hi = __builtin_bit_cast(uint16_t, (_Float16)low);
    pair[n] = finite ? lo | hi << 16 : 0x7E00u;
  }
#pragma unroll
  for (int k = 0; k < KD; ++k) even[k] |= odd[k] << 4;
  const RowAt at(c, p.page_size, slot, h);
  store_dwords(static_cast<uint8_t*>(is_v ? c.v : c.k) + at.codes + u * 4 * KD, even);
  if (u == 0) store_dwords(static_cast<uint32_t*>(is_v ? c.v_scale : c.k_scale) + at.pair, pair);
}

struct ReadArgs {
  seedlm_qcache_read_args a;
  RowSplit split;
  Divisor page_size;
};

// How a row's elements are written: one by one, by aligned fours, or (rows aligned to 16
// bytes) through LDS and past the caches, by 1 KB in a row where the four lanes of a row
// alone write 32 or 64 bytes.
enum Out { kEach, kFours, kStream };

template <int D, int BITS, int NG, Out OUT, typename T>
__global__ __launch_bounds__(kThreads) void qcache_read_kernel(const ReadArgs p) {
  constexpr int kI = D / 16, kUnitBytes = kI * BITS / 8, KD = kUnitBytes;
  constexpr int kRowBytes = D * sizeof(T), kChunk = kRowBytes < 256 ? kRowBytes : 256;
  constexpr int kChunkI = kChunk / (16 * (int)sizeof(T));  // i of a chunk
  constexpr int kSteps = 16 * kChunk / 1024;               // stores of a wave's chunk
  constexpr int kStride = kChunk + 32;                     // LDS row stride: two rows to 64 banks
  __shared__ __align__(16) uint8_t s_out[OUT == kStream ? kThreads / 64 : 1][OUT == kStream ? 16 * kStride : 16];
  const seedlm_qcache_read_args& a = p.a;
  const seedlm_qcache_t& c = a.cache;
  const int u = threadIdx.x & 3, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // The output row of the workgroup's row r, or NULL.
  int token = 0, row = 0;
  auto out_of = [&](int r) -> T* {
    if (!p.split.at(r, blockIdx.y, c.kv_heads, &token, &row)) return nullptr;
    const int64_t t = (int64_t)blockIdx.x * p.split.tokens + token;
    const bool is_v = row >= c.kv_heads;
    T* out = static_cast<T*>(is_v ? a.v_out : a.k_out);
    if (t >= a.tokens || !out) return nullptr;
    return out + t * (is_v ? a.v_stride : a.k_stride) + (int64_t)(is_v ? row - c.kv_heads : row) * D;
  };
  T* out = out_of(threadIdx.x >> 2);
  uint32_t code[KD], pair[NG];
#pragma unroll
  for (int k = 0; k < KD; ++k) code[k] = 0;
#pragma unroll
  for (int n = 0; n < NG; ++n) pair[n] = 0;
  if (out) {
    const int slot = a.slots[(int64_t)blockIdx.x * p.split.tokens + token];
    if (slot >= 0 && slot < c.pages * c.page_size) {
      const bool is_v = row >= c.kv_heads;
      const RowAt at(c, p.page_size, slot, is_v ? row - c.kv_heads : row);
      load_dwords(static_cast<const uint8_t*>(is_v ? c.v : c.k) + at.codes + u * 4 * KD, code);
      load_dwords(static_cast<const uint32_t*>(is_v ? c.v_scale : c.k_scale) + at.pair, pair);
    }
  }
  [[maybe_unused]] T* to[kSteps];  // where the lane's 16 bytes of each store go
  if constexpr (OUT == kStream) {
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int byte = k * 1024 + lane * 16;
      to[k] = out_of(wave * 16 + byte / kChunk);
      if (to[k]) to[k] += byte % kChunk / (int)sizeof(T);
    }
  }
  float s[NG], o[NG];
#pragma unroll
  for (int n = 0; n < NG; ++n) {
    s[n] = (float)__builtin_bit_cast(_Float16, (uint16_t)pair[n]);
    o[n] = (float)__builtin_bit_cast(_Float16, (uint16_t)(pair[n] >> 16));
  }
  auto elements = [&](int i, float (&x)[4]) {
    const int n = i * NG / kI;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int byte = j * kUnitBytes + i * BITS / 8;
      uint32_t d = code[byte / 4];
      if (BITS == 4) d = (i % 2 ? d >> 4 : d) & 0x0F0F0F0Fu;
      x[j] = o[n] + s[n] * (float)(d >> (8 * (byte % 4)) & 0xFF);
    }
  };
  if constexpr (OUT == kStream) {
#pragma unroll
    for (int i0 = 0; i0 < kI; i0 += kChunkI) {
      uint8_t* mine = s_out[wave] + (lane >> 2) * kStride;
#pragma unroll
      for (int i = 0; i < kChunkI; ++i) {
        float x[4];
        elements(i0 + i, x);
        store4<true>(reinterpret_cast<T*>(mine) + 16 * i + 4 * u, x);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        const int byte = k * 1024 + lane * 16;
        const v4u v = *reinterpret_cast<const v4u*>(s_out[wave] + byte / kChunk * kStride + byte % kChunk);
        v4u* at = reinterpret_cast<v4u*>(to[k] + 16 * i0);
        if (to[k]) __builtin_nontemporal_store(v, at);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
  } else if (out) {
#pragma unroll
    for (int i = 0; i < kI; ++i) {
      float x[4];
      elements(i, x);
      store4<OUT == kFours>(out + 16 * i + 4 * u, x);
    }
  }
}

bool fours(const void* p, int64_t stride, int dtype) {
  return stride % 4 == 0 && (uintptr_t)p % (dtype == SEEDLM_F16 ? 8 : 16) == 0;
}

// Whether q's rows and angles can go by units of 8 pairs.
bool wide_units(const seedlm_qcache_append_args& a) {
  const int64_t per = a.x_dtype == SEEDLM_F16 ? 8 : 4;  // elements of 16 bytes
  return a.rot % 16 == 0 && a.q_stride % per == 0 && a.q_out_stride % per == 0 && aligned16(a.q) &&
         aligned16(a.q_out) && aligned16(a.cos) && aligned16(a.sin);
}

// f with the cache's row as compile-time numbers: f(D, BITS, NG).
template <typename F>
int with_row(const seedlm_qcache_t& c, F f) {
  auto groups = [&](auto d, auto bits) {
    const int n = c.head_dim / c.group;
    if (n == 1) return f(d, bits, std::integral_constant<int, 1>());
    if (n == 2) return f(d, bits, std::integral_constant<int, 2>());
    if constexpr (decltype(d)::value > 64) return f(d, bits, std::integral_constant<int, 4>());
    return (int)SEEDLM_E_UNSUPPORTED;
  };
  auto width = [&](auto d) {
    return c.bits == 4 ? groups(d, std::integral_constant<int, 4>())
                       : groups(d, std::integral_constant<int, 8>());
  };
  if (c.head_dim == 64) return width(std::integral_constant<int, 64>());
  if (c.head_dim == 128) return width(std::integral_constant<int, 128>());
  return width(std::integral_constant<int, 256>());
}

int launched() { return hipGetLastError() == hipSuccess ? SEEDLM_OK : SEEDLM_E_DEVICE; }

}  // namespace

int launch_qcache_append(const seedlm_qcache_append_args& a, hipStream_t s) {
  const int D = a.cache.head_dim;
  const bool vec = fours(a.k, a.k_stride, a.x_dtype) && fours(a.v, a.v_stride, a.x_dtype) &&
                   a.rot % 8 == 0 && aligned16(a.cos) && aligned16(a.sin);
  // One form for all of a call: what keeps q from units of 8 pairs (rot no multiple of 16, a row
  // or an angle off 16 bytes) nearly always does the same to k and v, which a projection wrote
  // beside it.  4097 tokens of 32/32 heads of 128, fp16, 36.7 us and by single elements 109,
  // 16 tokens of 32/8 4.8 and 11.2, whichever tensor it is that does not fit.
  const bool wide = vec && wide_units(a);
  AppendArgs p{a, RowSplit(a.cache.kv_heads), divisor((uint32_t)a.cache.page_size), wide ? D / 16 : D / 2, {}, false};
  if (a.heads > 1024) p.split.tokens = 1;  // the grid's second dimension is short
  p.stream = (int64_t)a.tokens * a.heads * D * (a.x_dtype == SEEDLM_F16 ? 2 : 4) > kL2Bytes;
  const int token_units = a.heads * p.units;
  p.token_units = divisor((uint32_t)token_units);
  const int q_passes = (p.split.tokens * token_units + kThreads - 1) / kThreads;
  const dim3 grid((a.tokens + p.split.tokens - 1) / p.split.tokens, p.split.passes + q_passes);
  return with_row(a.cache, [&](auto d, auto bits, auto groups) {
    constexpr int kD = decltype(d)::value, kBits = decltype(bits)::value, kG = decltype(groups)::value;
    const bool f16 = a.x_dtype == SEEDLM_F16;
    const auto kernel =
        wide ? (f16 ? qcache_append_kernel<kD, kBits, kG, true, 8, __half>
                    : qcache_append_kernel<kD, kBits, kG, true, 8, float>)
             : (f16 ? qcache_append_kernel<kD, kBits, kG, false, 1, __half>
                    : qcache_append_kernel<kD, kBits, kG, false, 1, float>);
    hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, s, p);
    return launched();
  });
}

int launch_qcache_read(const seedlm_qcache_read_args& a, hipStream_t s) {
  const ReadArgs p{a, RowSplit(a.cache.kv_heads), divisor((uint32_t)a.cache.page_size)};
  const int64_t per = a.y_dtype == SEEDLM_F16 ? 8 : 4;  // elements of 16 bytes
  const bool wide = (!a.k_out || (a.k_stride % per == 0 && aligned16(a.k_out))) &&
                    (!a.v_out || (a.v_stride % per == 0 && aligned16(a.v_out)));
  const int64_t bytes = (int64_t)a.tokens * a.cache.kv_heads * a.cache.head_dim *
                        (a.y_dtype == SEEDLM_F16 ? 2 : 4) * ((a.k_out != nullptr) + (a.v_out != nullptr));
  const bool stream = wide && bytes > kL2Bytes;
  const dim3 grid((a.tokens + p.split.tokens - 1) / p.split.tokens, p.split.passes);
  return with_row(a.cache, [&](auto d, auto bits, auto groups) {
    constexpr int kD = decltype(d)::value, kBits = decltype(bits)::value, kG = decltype(groups)::value;
    const bool f16 = a.y_dtype == SEEDLM_F16;
    const auto kernel =
        stream ? (f16 ? qcache_read_kernel<kD, kBits, kG, kStream, __half>
                      : qcache_read_kernel<kD, kBits, kG, kStream, float>)
        : wide ? (f16 ? qcache_read_kernel<kD, kBits, kG, kFours, __half>
                      : qcache_read_kernel<kD, kBits, kG, kFours, float>)
               : (f16 ? qcache_read_kernel<kD, kBits, kG, kEach, __half>
                      : qcache_read_kernel<kD, kBits, kG, kEach, float>);
    hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, s, p);
    return launched();
  });
}

}  // namespace seedlm
