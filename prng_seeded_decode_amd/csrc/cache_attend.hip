// Attention of query tokens over their requests' pages of an fp16 cache
// (seedlm_cache_attend): out = sum_t softmax_t(scale q . k_t) v_t.  A query is
// called a request here; rows of the table tell which pages it has.
//
// A query reads each of its keys and values once, with 4 flops per query head of
// the group that shares it (4 to 8 flops per byte at 8 query heads), so memory
// bandwidth bounds the path once there is enough work, and latency below that.
//
// Split.  The lengths lie on the GPU, so every workgroup forms the split itself.
// A request of len tokens is ceil(len / kUnit) units; the units of all requests,
// one after another, are cut into `slots` even runs, one per workgroup and cache
// head, with as many slots as the chip holds at once.  Ragged batches and one
// long request then fill it alike, in one round.  A workgroup walks the requests
// in its run; a request wholly inside the run is finished there, and of one that
// is cut the (maximum, sum, unnormalised output) go to scratch, at most two per
// run (where it starts and where it ends), and attend_join_kernel weighs them by
// 2^(m_piece - m).  Where no request can be long (unsplit), requests are the
// workgroups and there is no second launch.  Within a workgroup four waves take
// 32-token tiles in turn, each with its own running maximum and sum, and join
// them through LDS.
//
// Tile.  Both products run on v_mfma_f32_16x16x32_f16 without LDS:
//   S^T = K Q^T   A = 16 tokens' keys, B = 16 query heads (the group, padded
//                 with zeros): lane l gets head l%16, tokens 4(l/16)+i
//   O^T = V^T P^T A = V^T, B = P^T: lane l supplies, for head l%16, 8 of the 32
//                 tokens - the ones that it holds scores of, as any order of
//                 the contracted index fits when A and B agree.
// For V^T a lane loads VD = D/16 consecutive dimensions of its 8 tokens (16
// lanes read one token's whole row) and transposes them in registers: element
// j of the 8 tokens is the operand row of dimension VD (l%16) + j.
// A tile's keys are requested when the previous tile's have been used, its
// values likewise, its page numbers one tile earlier still.
//
// Precision.  exp2 of the fp32 scores, scaled by 2^15 (their maximum is 1, and
// fp16 has few bits below 2^-14), enters the second product as a sum of two
// fp16 numbers, which keeps 22 bits; one fp16 number alone would add as much
// error as the rounding of an fp16 output does.  fp32 queries are split alike,
// after scaling each row by a power of two.
//
// Measured (main launch, then the join; a streaming read reaches 6.2 TB/s), 8 cache
// heads: one request of 131071 tokens, 128 dimensions, 537 MB, 98 + 4.8 us, 5.5 TB/s,
// reading 541 MB; 64 ragged requests of up to 16384 tokens, 2.12 GB, 372 + 6.0 us, 5.7
// TB/s; 16 of up to 8192, 252 MB, 51 + 4.6 us, with fp32 q the same; in 256 dimensions,
// 505 MB, 88 + 4.8 us, 5.8 TB/s, with fp32 q the same; in 64 dimensions, 126 MB, 32 + 4.9
// us, 3.9 TB/s; 8 ragged requests of up to 2047 tokens of 32 heads of 64, fp32 q, 51 MB,
// 13.3 + 4.0 us.  Matrix cores are busy 5% of the
// time and vector units 13%: what is left is the start of each run (lengths, page
// numbers, first keys: 7 to 9 us before the reads are at full rate) and its end.
#include <hip/hip_fp16.h>

#include <type_traits>

#include "seedlm_internal.h"

namespace seedlm {
namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kTile = 32;             // tokens of a wave's step
constexpr int kUnit = kWaves * kTile; // tokens of a workgroup's step
constexpr uint32_t kNoToken = 0xFFFFFFFFu;
constexpr float kLog2e = 1.44269504088896340736f;

struct AttendArgs {
  seedlm_cache_attend_args a;
  int group;            // query heads per cache head
  int qtiles;           // ceil(group / 16)
  int slots;            // runs of units; 0: one workgroup per request
  int cap;              // largest length: min(max_len, max_pages * page_size)
  uint32_t page_unit, token_unit;  // strides in units of 8 elements
  uint32_t div_mul, div_shift;     // x / page_size = x * div_mul >> div_shift
  int32_t* ends;        // [requests] inclusive sums of units, for the join
  float2* ml;           // [2 * slots][heads] maximum (log2) and sum
  float* acc;           // [2 * slots][heads][D]
};

// A query's tokens; 0 for one without a row of the table.
__device__ int length_of(const AttendArgs& p, int b) {
  const int len = min(max(p.a.lens[b], 0), p.cap);
  return !p.a.rows || (uint32_t)p.a.rows[b] < (uint32_t)p.a.table_rows ? len : 0;
}

// The first unit of a slot among `units`, and the slot of a unit: the largest i
// with i * units / slots <= u, that is i * units < (u + 1) * slots.
__device__ int slot_begin(int slot, int units, int slots) {
  return (int)((int64_t)slot * units / slots);
}
__device__ int slot_of(int u, int units, int slots) {
  return (int)((((int64_t)u + 1) * slots - 1) / units);
}

// Inclusive sums of the requests' units into ends[0..n), by all threads, each
// taking consecutive requests.
__device__ void sum_units(const AttendArgs& p, int32_t* ends) {
  __shared__ int s_wave[kWaves];
  const int n = p.a.queries, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int per = (n + kThreads - 1) / kThreads;
  const int b0 = min((int)threadIdx.x * per, n), b1 = min(b0 + per, n);
  int mine = 0;
  for (int b = b0; b < b1; ++b) {
    mine += (length_of(p, b) + kUnit - 1) / kUnit;
    ends[b] = mine;
  }
  int upto = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 63) s_wave[wave] = upto;
  __syncthreads();
  int before = upto - mine;
  for (int w = 0; w < wave; ++w) before += s_wave[w];
  for (int b = b0; b < b1; ++b) ends[b] += before;
  __syncthreads();
}

// The first request whose inclusive sum exceeds u.
__device__ int request_of(const int32_t* ends, int n, int u) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ends[mid] > u) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

__device__ half8 as_half8(v4u v) { return __builtin_bit_cast(half8, v); }

__device__ uint32_t pack_rtz(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(a, b));
}

template <bool STREAM, typename T>
__device__ T load(const uint16_t* p) {
  const T* q = reinterpret_cast<const T*>(p);
  return STREAM ? __builtin_nontemporal_load(q) : *q;
}

template <typename T>
__device__ void store4(T* p, floatx4 v) {
  if constexpr (sizeof(T) == 4) {
    p[0] = v[0], p[1] = v[1], p[2] = v[2], p[3] = v[3];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = __float2half_rn(v[i]);
  }
}

// Waves of attend_kernel per SIMD, and so workgroups per compute unit: what the
// registers of each form allow.
__host__ __device__ constexpr int waves_per_simd(int D) {
  return D == 64 ? 3 : (D == 128 ? 2 : 1);
}

// WIDE: fp32 q and out, else fp16.  STREAM: keys and values pass the caches.
template <int D, bool WIDE, bool STREAM>
__global__ __launch_bounds__(kThreads, waves_per_simd(D)) void attend_kernel(const AttendArgs p) {
  using T = std::conditional_t<WIDE, float, __half>;
  constexpr int KC = D / 32;              // key operands of a token
  constexpr int VD = D < 128 ? D / 16 : 8;  // consecutive dimensions of a value load
  constexpr int VU = D / 16 / VD;         // value loads of a token
  using VT = std::conditional_t<VD == 4, v2u, v4u>;
  constexpr int kRow = D + 4;             // LDS row stride (floats)
  __shared__ uint32_t s_off[kWaves][kTile];
  __shared__ float2 s_ml[kWaves][16];
  __shared__ __align__(16) float s_acc[kWaves][16][kRow];
  const seedlm_cache_attend_args& a = p.a;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int m = lane & 15, g = lane >> 4;
  const int hk = blockIdx.x / p.qtiles, qt = blockIdx.x % p.qtiles;
  const int heads = min(16, p.group - qt * 16);     // of this tile
  const int head0 = hk * p.group + qt * 16;

  extern __shared__ int32_t s_ends[];  // of the requests' units
  int unit = 0, unit_end = 1, run_begin = 0;
  if (p.slots > 0) {
    sum_units(p, s_ends);
    const int units = s_ends[a.queries - 1];
    if (blockIdx.x == 0 && blockIdx.y == 0)
      for (int b = threadIdx.x; b < a.queries; b += kThreads) p.ends[b] = s_ends[b];
    const int slots = min(p.slots, units);  // none is empty
    if ((int)blockIdx.y >= slots) return;
    run_begin = unit = slot_begin(blockIdx.y, units, slots);
    unit_end = slot_begin(blockIdx.y + 1, units, slots);
  }
  while (unit < unit_end) {
    // The next request of the run and the tokens of it that lie in the run.
    int request = blockIdx.y, begin = 0, end;
    bool whole = true;
    const bool starts_run = unit == run_begin;
    if (p.slots > 0) {
      request = request_of(s_ends, a.queries, unit);
      const int u0 = request > 0 ? s_ends[request - 1] : 0, u1 = s_ends[request];
      const int upto = min(u1, unit_end);
      begin = (unit - u0) * kUnit;
      end = min(length_of(p, request), (upto - u0) * kUnit);
      whole = unit == u0 && upto == u1;
      unit = upto;
    } else {
      end = length_of(p, request);
      unit = unit_end;
    }

    // Query operands: head m, dimensions 32 c + 8 g + (0..7).
    half8 qh[KC], ql[WIDE ? KC : 1];
    float sc = a.scale * kLog2e;
    {
      const T* q = static_cast<const T*>(a.q) + (int64_t)request * a.q_stride +
                   (int64_t)(head0 + min(m, heads - 1)) * D + g * 8;
      if constexpr (WIDE) {
        float f[KC][8], top = 0.f;
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          const floatx4 u = *reinterpret_cast<const floatx4*>(q + 32 * c);
          const floatx4 w = *reinterpret_cast<const floatx4*>(q + 32 * c + 4);
#pragma unroll
          for (int i = 0; i < 4; ++i) f[c][i] = u[i], f[c][4 + i] = w[i];
#pragma unroll
          for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(f[c][i]));
        }
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        // the row's largest element into [2^9, 2^10), so that the low parts have
        // all their bits
        int e = 10;
        if (top > 0.f && top < INFINITY) (void)frexpf(top, &e);
        const int up = 10 - e;
        sc = ldexpf(sc, -up);
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float x = m < heads ? ldexpf(f[c][i], up) : 0.f;
            qh[c][i] = (_Float16)x;
            ql[c][i] = (_Float16)(x - (float)qh[c][i]);
          }
      } else {
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          const v4u z = {0, 0, 0, 0};
          const v4u v = *reinterpret_cast<const v4u*>(q + 32 * c);
          qh[c] = as_half8(m < heads ? v : z);
        }
      }
    }

    const int64_t head_at = hk * a.cache.head_stride;
    const uint16_t* kbase = static_cast<const uint16_t*>(a.cache.k) + head_at + g * 8;
    const uint16_t* vbase = static_cast<const uint16_t*>(a.cache.v) + head_at + m * VD;
    const int32_t* table = a.table + (a.rows ? a.rows[request] : request) * a.table_stride;

    // Tile i of this wave: tokens first + 128 i + (0..31); lane l looks after
    // token l % 32.
    const int first = begin + wave * kTile;
    const int tiles = first < end ? (end - first + kUnit - 1) / kUnit : 0;
    int page = -1, nth = 0;  // of this lane's token in the next tile
    auto look_up = [&](int i) {
      const int tok = first + i * kUnit + (lane & 31);
      page = -1;
      if (tok < end) {
        const uint32_t nr = (uint32_t)(((uint64_t)(uint32_t)tok * p.div_mul) >> p.div_shift);
        nth = tok - (int)nr * a.cache.page_size;
        page = table[nr];
      }
    };
    v4u kreg[2][KC];
    VT vreg[VU][8];
    uint32_t koff[2], voff[8];
    uint32_t live = 0xFF, live_next = 0xFF;  // bit j: this lane's token j of the tile exists
    // Offsets of the tile that was looked up, and its keys requested.
    auto next_keys = [&]() {
      const bool ok = (uint32_t)page < (uint32_t)a.cache.pages;
      const uint32_t at = (uint32_t)page * p.page_unit + (uint32_t)nth * p.token_unit;
      const uint32_t off = ok ? at : kNoToken;
      if (lane < kTile) s_off[wave][lane] = off;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      koff[0] = s_off[wave][m];
      koff[1] = s_off[wave][16 + m];
#pragma unroll
      for (int j = 0; j < 8; ++j) voff[j] = s_off[wave][(j >> 2) * 16 + g * 4 + (j & 3)];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      live_next = 0xFF;
      if (__any(!ok)) {  // tokens that do not exist read token 0 of page 0 and are masked
        live_next = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          live_next |= (voff[j] != kNoToken) << j;
          voff[j] = voff[j] != kNoToken ? voff[j] : 0;
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) koff[s] = koff[s] != kNoToken ? koff[s] : 0;
      }
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int c = 0; c < KC; ++c)
          kreg[s][c] = load<STREAM, v4u>(kbase + (uint64_t)koff[s] * 8 + c * 32);
    };
    auto next_values = [&]() {
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int u = 0; u < VU; ++u)
          vreg[u][j] = load<STREAM, VT>(vbase + (uint64_t)voff[j] * 8 + u * 128);
    };

    float top = -INFINITY, sum = 0.f;  // running maximum (log2) and this lane's share of the sum
    floatx4 acc[VU][VD];
#pragma unroll
    for (int u = 0; u < VU; ++u)
#pragma unroll
      for (int j = 0; j < VD; ++j) acc[u][j] = floatx4{0.f, 0.f, 0.f, 0.f};

    if (tiles > 0) {
      look_up(0);
      next_keys();
      next_values();
      if (tiles > 1) look_up(1);
    }
    for (int i = 0; i < tiles; ++i) {
      live = live_next;
      floatx4 s[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const half8 k = as_half8(kreg[h][c]);
          s[h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, qh[c], s[h], 0, 0, 0);
          if constexpr (WIDE)
            s[h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, ql[c], s[h], 0, 0, 0);
        }
      if (i + 1 < tiles) {
        next_keys();
        if (i + 2 < tiles) look_up(i + 2);
      }
      float x[8], most = -INFINITY;
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = s[j >> 2][j & 3] * sc;
      const bool full = __all(live == 0xFF);
      if (!full) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = (live >> j) & 1 ? x[j] : -INFINITY;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) most = fmaxf(most, x[j]);
      most = fmaxf(most, __shfl_xor(most, 16));
      most = fmaxf(most, __shfl_xor(most, 32));
      if (__any(most > top)) {
        const float up = fmaxf(top, most);
        const float shrink = up == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(top - up);
        top = up;
        sum *= shrink;
#pragma unroll
        for (int u = 0; u < VU; ++u)
#pragma unroll
          for (int j = 0; j < VD; ++j) acc[u][j] *= shrink;
      }
      const float ref = top == -INFINITY ? 0.f : top - 15.f;
      v4u ph, pl;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float p0 = __builtin_amdgcn_exp2f(x[2 * w] - ref);
        const float p1 = __builtin_amdgcn_exp2f(x[2 * w + 1] - ref);
        sum += p0 + p1;
        const auto h = __builtin_amdgcn_cvt_pkrtz(p0, p1);
        ph[w] = __builtin_bit_cast(uint32_t, h);
        pl[w] = pack_rtz(p0 - (float)h[0], p1 - (float)h[1]);
      }
      if (!full) {  // 0 * (whatever a page holds beyond the length) must be 0
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (!((live >> j) & 1)) {
#pragma unroll
            for (int u = 0; u < VU; ++u)
#pragma unroll
              for (int w = 0; w < VD / 2; ++w) vreg[u][j][w] = 0;
          }
      }
#pragma unroll
      for (int u = 0; u < VU; ++u)
#pragma unroll
        for (int w = 0; w < VD / 2; ++w) {
          v4u even, odd;
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            even[t] = __builtin_amdgcn_perm(vreg[u][2 * t + 1][w], vreg[u][2 * t][w], 0x05040100u);
            odd[t] = __builtin_amdgcn_perm(vreg[u][2 * t + 1][w], vreg[u][2 * t][w], 0x07060302u);
          }
          floatx4& e = acc[u][2 * w];
          floatx4& o = acc[u][2 * w + 1];
          e = __builtin_amdgcn_mfma_f32_16x16x32_f16(as_half8(even), as_half8(ph), e, 0, 0, 0);
          o = __builtin_amdgcn_mfma_f32_16x16x32_f16(as_half8(odd), as_half8(ph), o, 0, 0, 0);
          e = __builtin_amdgcn_mfma_f32_16x16x32_f16(as_half8(even), as_half8(pl), e, 0, 0, 0);
          o = __builtin_amdgcn_mfma_f32_16x16x32_f16(as_half8(odd), as_half8(pl), o, 0, 0, 0);
        }
      if (i + 1 < tiles) next_values();
    }

    // Join the four waves.
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    if (g == 0) s_ml[wave][m] = make_float2(top, sum);
    if (m < heads) {
#pragma unroll
      for (int u = 0; u < VU; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < VD; j += 4)
            *reinterpret_cast<floatx4*>(&s_acc[wave][m][u * 128 + (g * 4 + i) * VD + j]) =
                floatx4{acc[u][j][i], acc[u][j + 1][i], acc[u][j + 2][i], acc[u][j + 3][i]};
    }
    __syncthreads();
    for (int e = threadIdx.x; e < heads * (D / 4); e += kThreads) {
      const int h = e / (D / 4), d = e % (D / 4) * 4;
      float mx = -INFINITY, total = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) mx = fmaxf(mx, s_ml[w][h].x);
      const float ref = mx == -INFINITY ? 0.f : mx;
      floatx4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f(s_ml[w][h].x - ref);
        total += f * s_ml[w][h].y;
        o += f * *reinterpret_cast<const floatx4*>(&s_acc[w][h][d]);
      }
      if (whole) {
        T* out = static_cast<T*>(a.out) + (int64_t)request * a.out_stride +
                 (int64_t)(head0 + h) * D + d;
        store4(out, o * (total == 0.f ? 0.f : 1.f / total));
      } else {
        const int64_t at = (int64_t)(2 * blockIdx.y + (starts_run ? 0 : 1)) * a.heads + head0 + h;
        *reinterpret_cast<floatx4*>(p.acc + at * D + d) = o;
        if (d == 0) p.ml[at] = make_float2(mx, total);
      }
    }
    __syncthreads();  // s_ml and s_acc have been read
  }
}

// Joins the pieces of one request and query head, and writes zeros for requests
// without any.  Every wave forms the maximum and the sum itself; groups of D/4
// lanes take the pieces in turn.
template <int D, bool WIDE>
__global__ __launch_bounds__(kThreads) void attend_join_kernel(const AttendArgs p) {
  using T = std::conditional_t<WIDE, float, __half>;
  constexpr int kLanes = D / 4, kGroups = kThreads / kLanes;
  __shared__ __align__(16) floatx4 s_part[kGroups][kLanes];
  const seedlm_cache_attend_args& a = p.a;
  const int b = blockIdx.y, head = blockIdx.x;
  const int units = p.ends[a.queries - 1], slots = min(p.slots, units);
  const int u0 = b > 0 ? p.ends[b - 1] : 0, u1 = p.ends[b];
  // Its pieces lie in the slots first_slot .. first_slot + pieces - 1: in each
  // but the first they start the slot's run.
  int first_slot = 0, pieces = 0, skip = 0;
  if (u1 > u0) {
    first_slot = slot_of(u0, units, slots);
    pieces = slot_of(u1 - 1, units, slots) - first_slot + 1;
    skip = slot_begin(first_slot, units, slots) != u0;
  }
  if (pieces == 1) return;
  T* out = static_cast<T*>(a.out) + (int64_t)b * a.out_stride + (int64_t)head * D;
  const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  auto partial = [&](int s) {
    return (int64_t)(2 * (first_slot + s) + (s == 0 ? skip : 0)) * a.heads + head;
  };
  float top = -INFINITY, total = 0.f;
  for (int s = threadIdx.x & 63; s < pieces; s += 64) top = fmaxf(top, p.ml[partial(s)].x);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
  const float ref = top == -INFINITY ? 0.f : top;
  for (int s = threadIdx.x & 63; s < pieces; s += 64) {
    const float2 ml = p.ml[partial(s)];
    total += __builtin_amdgcn_exp2f(ml.x - ref) * ml.y;
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) total += __shfl_xor(total, d);
  floatx4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = group; s < pieces; s += kGroups) {
    const int64_t i = partial(s);
    const float f = __builtin_amdgcn_exp2f(p.ml[i].x - ref);
    o += f * *reinterpret_cast<const floatx4*>(p.acc + i * D + lane * 4);
  }
  s_part[group][lane] = o;
  __syncthreads();
  if (group != 0) return;
#pragma unroll
  for (int k = 1; k < kGroups; ++k) o += s_part[k][lane];
  store4(out + lane * 4, o * (total == 0.f ? 0.f : 1.f / total));
}

int cap_of(const seedlm_cache_attend_args& a) {
  const int64_t room = (int64_t)a.max_pages * a.cache.page_size;
  return (int)(a.max_len < room ? a.max_len : room);
}

int qtiles_of(const seedlm_cache_attend_args& a) {
  return (a.heads / a.cache.kv_heads + 15) / 16;
}

// Whether requests are the workgroups: then a request's steps of kUnit tokens
// follow one another, but the sums, the partials and the second launch (4 to 5 us)
// fall away.  That pays up to four steps of 128 dimensions, and up to eight where
// requests fill half the chip.  GPU time of a call, unsplit against split: one
// request of 8 cache heads and 128 dimensions 6.6 and 8.9 us at 300 tokens, 8.0
// and 9.0 at 512, 10.2 and 8.9 at 768; 16 requests 9.7 and 13.3 at 512, 15.5 and
// 19.4 at 1024; 4 requests of 2 heads and 256 dimensions 9.4 and 11.4 at 256, 13.9
// and 11.5 at 512; 8 requests of 32 heads and 64 dimensions, lengths up to 2047, 22
// and 18.
bool unsplit(const seedlm_cache_attend_args& a) {
  const int64_t workgroups = (int64_t)a.queries * a.cache.kv_heads * qtiles_of(a);
  int steps = 4 * 128 / a.cache.head_dim;
  if (2 * workgroups >= device_cu_count() && steps < 8) steps *= 2;
  return cap_of(a) <= steps * kUnit;
}

// Runs of units per cache head: what the chip holds at once.
int slots_of(const seedlm_cache_attend_args& a) {
  if (unsplit(a)) return 0;
  const int held = device_cu_count() * waves_per_simd(a.cache.head_dim);
  const int across = a.cache.kv_heads * qtiles_of(a);
  return (held + across - 1) / across;
}

struct Scratch {
  size_t ends, ml, acc;  // byte offsets and the total size
  size_t bytes;
};

Scratch scratch_of(const seedlm_cache_attend_args& a) {
  const size_t n = (size_t)2 * slots_of(a) * a.heads;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  Scratch r;
  r.ends = 0;
  r.ml = up((size_t)a.queries * sizeof(int32_t));
  r.acc = r.ml + up(n * sizeof(float2));
  r.bytes = n == 0 ? 0 : r.acc + n * a.cache.head_dim * sizeof(float);
  return r;
}

// Whether keys and values pass the caches: a call that may read more than the 256
// MB of the memory-side cache finds nothing of it there the next time.  Where rows are
// given, queries may share a request's tokens, which the caches then serve to all but
// the first.  Time of a call, passing the caches against not, 8 cache heads, fp16: one
// request of 131071 tokens in 128 dimensions 102 and 105 us, 64 of up to 16384 (32 heads)
// 357 and 361, 16 of 16384 in 256 dimensions 325 and 338; 64 dimensions gain nothing (442
// and 456).  A cache that fits would lose: 16 requests of 2048 in 128 dimensions, read
// again and again, 33 and 29.  So would prompts: 2048 queries of one request 1025 and
// 947, 512 queries behind 8192 cached tokens (64 heads) 2323 and 1226.
bool streams(const seedlm_cache_attend_args& a) {
  const int64_t most = (int64_t)a.queries * cap_of(a) * a.cache.kv_heads * a.cache.head_dim * 4;
  return !a.rows && a.cache.head_dim > 64 && most > (int64_t)256 << 20;
}

template <int D, bool WIDE>
int run(const AttendArgs& p, hipStream_t s) {
  const seedlm_cache_attend_args& a = p.a;
  const bool split = p.slots > 0;
  const auto kernel = streams(a) ? attend_kernel<D, WIDE, (D > 64)> : attend_kernel<D, WIDE, false>;
  hipLaunchKernelGGL(kernel, dim3(a.cache.kv_heads * p.qtiles, split ? p.slots : a.queries),
                     dim3(kThreads), split ? a.queries * sizeof(int32_t) : 0, s, p);
  if (split)
    hipLaunchKernelGGL((attend_join_kernel<D, WIDE>), dim3(a.heads, a.queries), dim3(kThreads), 0,
                       s, p);
  return hipGetLastError() == hipSuccess ? SEEDLM_OK : SEEDLM_E_DEVICE;
}

}  // namespace

size_t cache_attend_scratch_bytes(const seedlm_cache_attend_args& a) { return scratch_of(a).bytes; }

int launch_cache_attend(const seedlm_cache_attend_args& a, void* scratch, hipStream_t s) {
  AttendArgs p{};
  p.a = a;
  p.group = a.heads / a.cache.kv_heads;
  p.qtiles = qtiles_of(a);
  p.slots = slots_of(a);
  p.cap = cap_of(a);
  p.page_unit = (uint32_t)(a.cache.page_stride / 8);
  p.token_unit = (uint32_t)(a.cache.token_stride / 8);
  // x / d for 0 <= x < 2^31, with 2^(L-1) < d <= 2^L: ceil(2^(31+L) / d) is less
  // than 1 above 2^(31+L) / d, so the product is less than x / 2^(31+L) < 2^-L
  // above x / d.  That is at most 1/d, which no quotient's fraction lacks less
  // than to the next whole number, so the floor is the quotient's.
  const uint32_t d = (uint32_t)a.cache.page_size;
  uint32_t L = 0;
  while (((uint64_t)1 << L) < d) ++L;
  p.div_mul = (uint32_t)((((uint64_t)1 << (31 + L)) + d - 1) / d);
  p.div_shift = 31 + L;
  const Scratch r = scratch_of(a);
  char* base = static_cast<char*>(scratch);
  if (base) {
    p.ends = reinterpret_cast<int32_t*>(base + r.ends);
    p.ml = reinterpret_cast<float2*>(base + r.ml);
    p.acc = reinterpret_cast<float*>(base + r.acc);
  }
  const bool wide = a.x_dtype == SEEDLM_F32;
  switch (a.cache.head_dim) {
    case 64: return wide ? run<64, true>(p, s) : run<64, false>(p, s);
    case 128: return wide ? run<128, true>(p, s) : run<128, false>(p, s);
    case 256: return wide ? run<256, true>(p, s) : run<256, false>(p, s);
    default: return SEEDLM_E_UNSUPPORTED;
  }
}

}  // namespace seedlm
