// Attention of query tokens over their requests' pages of a quantised cache
// (seedlm_qcache_attend): out = sum_t softmax_t(scale q . k_t) v_t, where element d of
// k_t is o_tj + s_tj c_td with j the group of d, and v_t likewise.
//
// Mathematics.  The codes go into the matrix products as they are:
//   q . k_t     = sum_j (s_tj sum_{d in j} q_d c_td + o_tj sum_{d in j} q_d)
//   sum_t p_t v_td = sum_t (p_t s_tj) c_td + sum_t p_t o_tj
// so a group costs its pair's products and not a multiplication per element, and
// no dequantised value is rounded.  A code in the low bits of an fp16 number is a
// subnormal one: c 2^-24 of 8 bits, 16 c 2^-24 of 4 bits in the bits 4 to 7, so a byte
// permutation, a mask and for every second code of 4 bits a shift unpack two codes.
//
// Split.  As in cache_attend.hip: the 128-token units of all items, one after another,
// are cut into even runs, one per workgroup and cache head, and what is cut is joined by
// qcache_attend_join_kernel; short calls are not split.  An item is one query, or
// where rows are given up to 16 / group consecutive queries of one row: their heads share
// the 16 columns of the matrix products and what is read and unpacked.
//
// Tile.  A wave takes 32 tokens:
//   S^T = K Q^T   A = 16 tokens' codes, B = 16 columns: lane l gets column l%16, tokens
//                 4(l/16)+i.  Lane l holds units 4(l/16)..+3 of token l%16, and product
//                 step c contracts the codes 2c and 2c+1 of all units, elements 32c to
//                 32c+31: a group is whole steps and its sum comes out by itself.
//   O^T = V^T P^T A = code i of unit l%16 of 8 tokens, the ones that lane l holds scores
//                 of, B = their weights: element 16i + l%16, so a group is whole products
//                 and each has its own weights p s.
// Tile i+1's codes and pairs are requested before tile i is computed, its page numbers one
// tile earlier still and before those loads (a wait for a load is one for all before it).
// Pairs pass through LDS, where 4 tokens' are one read.
//
// Precision.  p s enters the second product as the sum of two fp16 numbers, 22 bits down to a
// smallest step, so what p s is relative to follows the scales of the values (`shift`).  Tiles
// in which that does not do - one scale above it, or the largest weights on scales far
// below the others, of all groups or of one - go through a general form of the loop's body, in
// which each column and group has its own.  What subnormal codes cost the sums, and which
// calls avoid it, is at Row.  fp32 outputs over 8 ragged requests err by 5.2 to 5.7e-7 of their
// norm, 32-bit sums of dequantised values by 5.4 to 6.0e-7.
//
// Measured (traced kernels, three inputs in turn; one MI355X).  One request of 131071 tokens,
// 64/8 heads of 128, 4 bits, 143 MB: 33.0 us and 5.3 of the join, 4.3 TB/s, where a streaming
// read has 6.2; 64 ragged ones up to 16384, 32/8 heads, 600 MB: 132 and 5.4 (118 for both
// where calls follow one another); 16 ragged ones up to 8192, 64/8 heads, two groups: 24.4
// and 4.6.  Memory and the vector units bound them together: in 67 to 78% of the SIMDs' busy
// cycles a vector instruction goes on (unpacking, the softmax of 16 columns), in a fifth or
// less a matrix one.  Pieces of prompts (128 queries, four groups, 55 us) read little and
// spend as large a share on vector instructions; 256 dimensions of 8 bits only a third, with
// one wave per SIMD to cover the waits (18.9 us and 4.4 for 57 MB).
#pragma once

#include <hip/hip_fp16.h>

#include <type_traits>

#include "attend_split.h"

namespace seedlm {
namespace qattend {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half4v __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kTile = 32;              // tokens of a wave's step
constexpr int kUnit = kWaves * kTile;  // tokens of a workgroup's step
constexpr int kItemUnits = kQcacheItemUnits;
constexpr uint32_t kNoToken = 0xFFFFFFFFu;
constexpr float kLog2e = 1.44269504088896340736f;

struct Args {
  seedlm_qcache_attend_args a;
  int group;    // query heads per cache head
  int qtiles;   // ceil(group / 16)
  int shared;   // queries of an item at most
  int slots;    // runs of units; 0: a workgroup per query, those that go on with another's item idle
  int rows;     // of the grid
  int cap;      // largest length: min(max_len, max_pages * page_size)
  uint32_t page_unit, token_unit;  // strides of codes in units of 16 bytes
  uint32_t page_pair, token_pair;  // strides of pairs in rows of pairs
  Divisor page_size;
  uint32_t per_head;  // 2^16 / group, rounded up
  int4* joins;    // [queries] see join_of
  float2* ml;     // [2 * slots][kv_heads * qtiles][16] maximum (log2) and sum
  float* acc;     // [2 * slots][kv_heads * qtiles][16][D]
};

// A query's tokens; 0 for one without a row of the table.
__device__ inline int length_of(const Args& p, int b) {
  const int len = min(max(p.a.lens[b], 0), p.cap);
  return !p.a.rows || (uint32_t)p.a.rows[b] < (uint32_t)p.a.table_rows ? len : 0;
}

// What is kept of query b in LDS: its tokens, negative (-1 - tokens) where it goes on with
// the item of the query before.
__device__ inline int item_entry(const Args& p, int b) {
  const int len = length_of(p, b);
  const bool goes_on = p.shared > 1 && b % p.shared != 0 && p.a.rows[b] == p.a.rows[b - 1];
  return goes_on ? -1 - len : len;
}

// The queries of the item whose first entry is e[0], of n entries, and the longest of
// their lengths.
__device__ inline int2 item_of(const int32_t* e, int n) {
  int k = 1, len = e[0];
  while (k < n && e[k] < 0) len = max(len, -1 - e[k]), ++k;
  return make_int2(k, len);
}

// Units of an item in the split.
__device__ inline int units_of(int len) { return len > 0 ? kItemUnits + (len + kUnit - 1) / kUnit : 0; }

// What the join has to know of the queries of the item of units [u0, u1) that starts with
// query `first`: that query, the first slot of its tokens, its pieces, and which of the two
// of that slot its first piece is.  The pieces lie in consecutive slots: in each but the
// first, whose run may have begun before the item, they start the slot's run.
template <int GENS>
__device__ int4 join_of(const Runs<GENS>& runs, int first, int u0, int u1) {
  if (u1 == u0) return make_int4(first, 0, 0, 0);
  const int slot = runs.slot_of(u0 + kItemUnits);
  return make_int4(first, slot, runs.slot_of(u1 - 1) - slot + 1, runs.begin(slot) < u0);
}

__device__ inline half8 as_half8(v4u v) { return __builtin_bit_cast(half8, v); }
__device__ inline half2v as_half2(uint32_t v) { return __builtin_bit_cast(half2v, v); }

__device__ inline uint32_t pack(float a, float b) {  // rounded to nearest
  return __builtin_bit_cast(uint32_t, half2v{(_Float16)a, (_Float16)b});
}

// Magnitudes of fp16 scales as numbers: of what follows the finite ones, and from one exponent
// to the next.  Scales of the least exponent are below 2^-14.
constexpr uint32_t kScaleInf = 0x7C00u, kScaleExponent = 0x400u;
constexpr float kLeastShift = -14.f - 15.f;
// Weights times scales are held to 2^-24 below 2^15 times the power of 2 above all scales.  Scales
// from 2^-8 of that on are normal, which leaves 2^-31 of the largest weight; a tile whose largest
// weight is at most 2^4 times one of a token with normal scales has products of 2^2 and more.  The
// magnitudes of smaller scales, less 1, lie below far_below().  (Where all are of the least
// exponent, 2^-24 on from 2^-14, none is.)
constexpr float kFarBelow = 8.f, kNear = 4.f;
__device__ inline uint32_t far_below(uint32_t exponent) {
  return exponent == 0 ? 0 : (exponent < 8 ? 1u << (exponent + 2) : kScaleExponent * (exponent - 7)) - 1;
}

// Scores of this and more (in powers of 2) are held in fp32 to steps of a half or more, which a
// shift is lost in.  Their maximum is the largest of the rounded products, so it is taken from
// those.
constexpr float kFar = 0x1p22f;
__device__ inline float minus(float x, float scale, float from) {
#pragma clang fp contract(off)
  return x * scale - from;
}

// The largest x of lanes l, l ^ 16, l ^ 32 and l ^ 48.
__device__ inline float max_of_column(float x) {
  auto largest = [](auto swapped) {
    const uint32_t a = swapped[0], b = swapped[1];
    return fmaxf(__uint_as_float(a), __uint_as_float(b));
  };
  uint32_t u = __float_as_uint(x);
  u = __float_as_uint(largest(__builtin_amdgcn_permlane16_swap(u, u, false, false)));
  return largest(__builtin_amdgcn_permlane32_swap(u, u, false, false));
}

// The largest x of lanes 32..63.
__device__ inline uint32_t largest_of_half(uint32_t x) {
#define SEEDLM_MAX_DPP(ctrl, rows) \
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, ctrl, rows, 0xF, false))
  SEEDLM_MAX_DPP(0x111, 0xF);  // the lane 1, 2, 4 and 8 before in the same 16
  SEEDLM_MAX_DPP(0x112, 0xF);
  SEEDLM_MAX_DPP(0x114, 0xF);
  SEEDLM_MAX_DPP(0x118, 0xF);
#undef SEEDLM_MAX_DPP
  return max((uint32_t)__builtin_amdgcn_readlane((int)x, 47), (uint32_t)__builtin_amdgcn_readlane((int)x, 63));
}

// The least x of the 16 lanes of a row.
__device__ inline int least_of_row(int x) {
#define SEEDLM_MIN_DPP(ctrl) x = min(x, __builtin_amdgcn_update_dpp(x, x, ctrl, 0xF, 0xF, false))
  SEEDLM_MIN_DPP(0x121);  // rotated by 1, 2, 4 and 8 lanes
  SEEDLM_MIN_DPP(0x122);
  SEEDLM_MIN_DPP(0x124);
  SEEDLM_MIN_DPP(0x128);
#undef SEEDLM_MIN_DPP
  return __builtin_amdgcn_readfirstlane(x);
}

// Keeps what a rare branch does in the branch: the compiler would rather do it always
// and select.
__device__ inline void rare() { asm volatile(""); }

// A number that all lanes of a wave hold alike, which the compiler cannot know.
__device__ inline int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// A number that the compiler forms where it is used, with all that follows from it, and does not
// keep in registers through a loop.
__device__ inline int own(int x) {
  asm volatile("" : "+v"(x));
  return x;
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

// Byte n of a and of b in the low bytes of the two halves; the bytes above them are 0.
__device__ inline uint32_t pair_bytes(uint32_t a, uint32_t b, int n) {
  return __builtin_amdgcn_perm(b, a, 0x0C040C00u + 0x00010001u * n);
}

constexpr uint32_t kHigh = 0x00F000F0u;  // 16 c of two bytes' high codes

template <int D, int BITS, bool WIDE>
struct Row {
  // What a code of 1 is in an operand.  The matrix instructions take a subnormal number as one
  // of the smallest normal ones and line the products up by that, so a small code costs its
  // sums low bits, the same way in all of them.  Codes of 4 bits are therefore all put where
  // the high ones are, and those of fp32 calls are made normal numbers, at one more
  // instruction for two codes.  (Weights of one token over others, the sums' relative errors:
  // 4 bits at 2^-24 7e-7, of mean -6e-7, at 2^-20 1e-7 without a mean; normal 1e-7.)
  static constexpr float kCode = (BITS == 4 ? 0x1p-20f : 0x1p-24f) * (WIDE ? 0x1p15f : 1.f);
  __device__ static half8 operand(v4u r) {
    if constexpr (!WIDE) return as_half8(r);
    return as_half8(r) * (_Float16)0x1p15f;
  }


  static constexpr int kBytes = D * BITS / 8;
  static constexpr int kUnitBytes = kBytes / 16;
  static constexpr int KD = kBytes / 16;                             // dwords of 4 units
  static constexpr int VD = kUnitBytes < 4 ? 1 : kUnitBytes / 4;     // dwords of a unit
  static constexpr int kSteps = D / 32, kAccs = D / 16;

  // The operand of step c from 4 units of a token: (u0, u1) code 2c, (u0, u1) code
  // 2c + 1, (u2, u3) code 2c, (u2, u3) code 2c + 1.
  __device__ static half8 keys(const uint32_t (&k)[KD], int c) {
    v4u r;
    if constexpr (BITS == 8) {
      const int d = c / 2, n = 2 * (c % 2);
      r = v4u{pair_bytes(k[d], k[VD + d], n), pair_bytes(k[d], k[VD + d], n + 1),
              pair_bytes(k[2 * VD + d], k[3 * VD + d], n),
              pair_bytes(k[2 * VD + d], k[3 * VD + d], n + 1)};
    } else {
      uint32_t lo, hi;
      if constexpr (kUnitBytes == 2) {  // two units to a dword
        lo = k[0] >> (8 * c), hi = k[1] >> (8 * c);
      } else {
        const int d = c / 4, n = c % 4;
        lo = pair_bytes(k[d], k[VD + d], n), hi = pair_bytes(k[2 * VD + d], k[3 * VD + d], n);
      }
      r = v4u{(lo << 4) & kHigh, lo & kHigh, (hi << 4) & kHigh, hi & kHigh};
    }
    return operand(r);
  }

  // The operand of code i from a unit of 8 tokens.
  __device__ static half8 values(const uint32_t (&v)[8][VD], int i) {
    v4u r;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int byte = i * BITS / 8;
      const uint32_t b = pair_bytes(v[2 * x][byte / 4], v[2 * x + 1][byte / 4], byte % 4);
      r[x] = BITS == 8 ? b : (i % 2 ? b : b << 4) & kHigh;
    }
    return operand(r);
  }

  // The operand of keys() whose codes are all 1, divided by kCode: the offsets carry what its
  // products lose into every score (6.8e-7 of their magnitudes' sum with subnormal 1s, nothing
  // with 1s).
  __device__ static half8 ones() {
    const uint32_t one = 0x3C003C00u;
    return as_half8(v4u{one, one, one, one});
  }
};

template <bool STREAM, typename T>
__device__ T load(const uint8_t* p) {
  const T* q = reinterpret_cast<const T*>(p);
  return STREAM ? __builtin_nontemporal_load(q) : *q;
}

// BYTES bytes at p as N dwords (2 bytes as one); STREAM: past the caches.
template <int BYTES, bool STREAM, int N>
__device__ void load_codes(const uint8_t* p, uint32_t (&out)[N]) {
  if constexpr (BYTES == 2) {
    out[0] = load<STREAM, uint16_t>(p);
  } else if constexpr (BYTES == 4) {
    out[0] = load<STREAM, uint32_t>(p);
  } else if constexpr (BYTES == 8) {
    const v2u v = load<STREAM, v2u>(p);
    out[0] = v[0], out[1] = v[1];
  } else {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      const v4u v = load<STREAM, v4u>(p + 16 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) out[4 * i + j] = v[j];
    }
  }
}

// Waves of the kernel per SIMD, and so workgroups per compute unit: what the registers
// of each form allow.  (One more of the 128-dimensional forms spills and is slower.)
__host__ __device__ constexpr int waves_per_simd(int D, int bits, int groups, bool wide) {
  if (D == 256) return bits == 8 || wide || groups > 1 ? 1 : 2;
  return D == 128 && (bits == 8 || wide || groups > 1) ? 2 : 3;
}

// WIDE: fp32 q and out, else fp16.  STREAM: codes pass the caches.
template <int D, int BITS, int NG, bool WIDE, bool STREAM>
__global__ __launch_bounds__(kThreads, waves_per_simd(D, BITS, NG, WIDE)) void qcache_attend_kernel(
    const Args p) {
  using T = std::conditional_t<WIDE, float, __half>;
  using R = Row<D, BITS, WIDE>;
  constexpr int kSteps = R::kSteps, kAccs = R::kAccs, KD = R::KD, VD = R::VD;
  constexpr int kStride = D + 4;  // LDS row stride (floats)
  constexpr int kGens = waves_per_simd(D, BITS, NG, WIDE);
  __shared__ __align__(16) uint32_t s_off[kWaves][kTile];
  __shared__ __align__(16) uint32_t s_pair[kWaves][NG][2 * kTile];
  __shared__ float2 s_ml[kWaves][16];
  __shared__ __align__(16) float s_acc[kWaves][16][kStride];
  extern __shared__ int32_t s_ends[];  // inclusive sums of the items' units, then the entries
  const seedlm_qcache_attend_args& a = p.a;
  const seedlm_qcache_t& c = a.cache;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int m = lane & 15, g = lane >> 4;
  const int hk = blockIdx.x / p.qtiles, qt = blockIdx.x % p.qtiles;
  const int heads = min(16, p.group - qt * 16);  // of a query in this tile
  const int head0 = hk * p.group + qt * 16;

  // The inclusive sums of the items' units, then the entries.  Up to 64 queries of which none goes
  // on with another's item are a lane each: every wave forms and writes the sums itself (all write
  // the same numbers, so none waits for another).
  bool few = p.slots > 0 && a.queries <= 64;
  int unit = 0, unit_end = 1, run_begin = 0;
  int block_query = blockIdx.y, block_row = 0;  // of a call without a split
  int32_t* s_entry = s_ends;
  if (p.slots > 0) {
    s_entry = s_ends + a.queries;
    int units;
    const int len = few && lane < a.queries ? item_entry(p, lane) : 0;
    few = few && !__any(len < 0);
    if (few) {
      const int upto = wave_sums(units_of(len));
      if (lane < a.queries) s_ends[lane] = upto, s_entry[lane] = len;
      units = __builtin_amdgcn_readlane(upto, 63);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    } else {
      for (int b = threadIdx.x; b < a.queries; b += kThreads) s_entry[b] = item_entry(p, b);
      __syncthreads();
      sum_units<kThreads>(a.queries, s_ends, [&](int b) {
        return s_entry[b] < 0 ? 0 : units_of(item_of(s_entry + b, a.queries - b).y);
      });
      units = uniform(s_ends[a.queries - 1]);
    }
    const Runs<kGens> runs(p.slots, units);  // none is empty
    if (blockIdx.x == 0 && blockIdx.y == 0) {
      for (int b = threadIdx.x; b < a.queries; b += kThreads) {
        int first = b;
        while (s_entry[first] < 0) --first;
        p.joins[b] = join_of(runs, first, first > 0 ? s_ends[first - 1] : 0, s_ends[first]);
      }
    }
    if ((int)blockIdx.y >= runs.slots) return;
    run_begin = unit = runs.begin(blockIdx.y);
    unit_end = runs.begin(blockIdx.y + 1);
  } else if (p.shared > 1) {
    // First the queries that certainly start an item, then the others, so that those which only
    // find that they do not end while the items go on.  Every wave writes the entries of the
    // query and of those that may go on with it.  A workgroup for `shared` queries would take
    // their items one after another: 16 requests of a token each, 32 cache heads, 500 tokens, 88
    // against 10.9 us; where all are pieces the idle workgroups cost up to 1.2 of 49 us.
    int nth = 0;  // of the `shared` queries that may be one item
    const int starts = (a.queries + p.shared - 1) / p.shared;
    if (block_query < starts) {
      block_query *= p.shared;
    } else {
      const int other = block_query - starts, of = other / (p.shared - 1);
      nth = 1 + other - of * (p.shared - 1);
      block_query = of * p.shared + nth;
    }
    const int n = min(p.shared - nth, a.queries - block_query);
    const int entry = lane < n ? item_entry(p, block_query + lane) : 0;
    block_row = a.rows[block_query];
    if (uniform(entry) < 0) return;
    if (lane < n) s_entry[lane] = entry;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    unit_end = n;
  }
  while (unit < unit_end) {
    // The next item of the run and the tokens of it that lie in the run.
    int first_query, begin = 0, end;
    bool whole = true;
    const bool starts_run = unit == run_begin;
    int2 item;
    if (p.slots > 0) {
      first_query = few ? __ffsll(__ballot(lane >= a.queries || s_ends[lane] > unit)) - 1
                        : request_of(s_ends, a.queries, unit);
      item = item_of(s_entry + first_query, a.queries - first_query);
      const int u0 = first_query > 0 ? s_ends[first_query - 1] : 0, u1 = s_ends[first_query];
      const int upto = min(u1, unit_end);
      // of the item's units those that stand for its start hold no tokens
      begin = max(unit - u0 - kItemUnits, 0) * kUnit;
      end = min(item.y, (upto - u0 - kItemUnits) * kUnit);
      whole = begin == 0 && upto == u1;
      unit = upto;
      if (begin >= end) continue;  // the run ends before the item's tokens do begin
    } else {
      first_query = block_query;
      item = p.shared > 1 ? item_of(s_entry, unit_end) : make_int2(1, length_of(p, first_query));
      end = item.y;
      unit = unit_end;
    }

    first_query = uniform(first_query);
    item = make_int2(uniform(item.x), uniform(item.y));
    begin = uniform(begin), end = uniform(end), unit = uniform(unit);
    const uint8_t* kbase = static_cast<const uint8_t*>(c.k) + hk * c.head_stride + g * (R::kBytes / 4);
    const uint8_t* vbase = static_cast<const uint8_t*>(c.v) + hk * c.head_stride + m * R::kUnitBytes;
    // lanes 0..31 fetch the keys' pairs of the tile's tokens, lanes 32..63 the values'
    const uint32_t* pairs = static_cast<const uint32_t*>(lane < kTile ? c.k_scale : c.v_scale) +
                            hk * c.scale_head_stride;
    int row = first_query;
    if (a.rows) row = p.slots == 0 && p.shared > 1 ? block_row : a.rows[first_query];
    const int32_t* table = a.table + (int64_t)row * a.table_stride;

    // Tile i of this wave: tokens first + 128 i + (0..31); lane l looks after token l % 32.
    const int first = begin + wave * kTile;
    const int tiles = first < end ? (end - first + kUnit - 1) / kUnit : 0;
    int page = -1, nth = -1;  // of this lane's token in the tile after the next
    auto look_up = [&](int i) {
      const int tok = first + i * kUnit + (lane & 31), at = min(tok, end - 1);
      const uint32_t nr = p.page_size.of(at);
      nth = tok < end ? at - (int)nr * c.page_size : -1;
      page = table[nr];
    };
    struct Tile {
      uint32_t k[2][KD], v[8][VD], pair[NG];
      uint32_t live;  // bit i: token i exists (the same in all lanes)
    };
    // Requests the tile that was looked up, and looks up tile `next`.
    auto request = [&](Tile& t, int next) {
      const bool ok = nth >= 0 && (uint32_t)page < (uint32_t)c.pages;
      const uint32_t off = (uint32_t)page * p.page_unit + (uint32_t)nth * p.token_unit;
      uint32_t row = (uint32_t)page * p.page_pair + (uint32_t)nth * p.token_pair;
      row = ok ? row : 0;
      s_off[wave][lane & 31] = ok ? off : kNoToken;  // twice the same
      look_up(next);
      t.live = (uint32_t)__ballot(ok);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      uint32_t koff[2] = {s_off[wave][m], s_off[wave][16 + m]};
      const v4u o[2] = {*reinterpret_cast<const v4u*>(&s_off[wave][4 * g]),
                        *reinterpret_cast<const v4u*>(&s_off[wave][16 + 4 * g])};
      uint32_t voff[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) voff[j] = o[j >> 2][j & 3];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (t.live != ~0u) {  // tokens that do not exist read token 0 of page 0 and are masked
        rare();
#pragma unroll
        for (int j = 0; j < 8; ++j) voff[j] = voff[j] != kNoToken ? voff[j] : 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) koff[h] = koff[h] != kNoToken ? koff[h] : 0;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) load_codes<R::kBytes / 4, STREAM>(kbase + (uint64_t)koff[h] * 16, t.k[h]);
      load_codes<4 * NG, false>(reinterpret_cast<const uint8_t*>(pairs + (uint64_t)row * NG), t.pair);
#pragma unroll
      for (int j = 0; j < 8; ++j) load_codes<R::kUnitBytes, STREAM>(vbase + (uint64_t)voff[j] * 16, t.v[j]);
    };

    Tile even, odd;
    int i = 0;
    if (tiles > 0) {
      look_up(0);
      request(even, 1);
    }

    // This lane's column: a query and a head; columns past the last repeat it.
    const int columns = item.x * heads;
    const int column = min(m, columns - 1);
    const int nth_query = p.shared > 1 ? (int)(column * p.per_head >> 16) : 0;
    const int query = first_query + nth_query, head = head0 + column - nth_query * heads;
    int length = item.y;
    if (p.shared > 1) {
      length = s_entry[p.slots > 0 ? query : query - block_query];
      length = length < 0 ? -1 - length : length;
    }

    // Query operands of step s: elements 16 (2s) + 4g + (0..3) and 16 (2s + 1) + 4g +
    // (0..3), in the order of Row::keys.
    half8 qh[kSteps], ql[WIDE ? kSteps : 1];
    float sc = a.scale * kLog2e * (1.f / R::kCode);  // of products, to scores in powers of 2
    float qsum[NG];  // of a group's elements, in the units of its products with codes
    {
      using Four = std::conditional_t<WIDE, floatx4, v2u>;
      const T* q = static_cast<const T*>(a.q) + (int64_t)query * a.q_stride + (int64_t)head * D + g * 4;
      Four raw[2 * kSteps];
#pragma unroll
      for (int s = 0; s < 2 * kSteps; ++s) raw[s] = *reinterpret_cast<const Four*>(q + 16 * s);
      // fp16 goes in as it is.  fp32 rows are multiplied by a power of two that puts their
      // largest element into [2^9, 2^10), and go in as the sum of two fp16 numbers.
      if constexpr (!WIDE) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
          qh[s] = as_half8(v4u{raw[2 * s][0], raw[2 * s + 1][0], raw[2 * s][1], raw[2 * s + 1][1]});
      } else {
        float most = 0.f;
#pragma unroll
        for (int s = 0; s < 2 * kSteps; ++s)
#pragma unroll
          for (int j = 0; j < 4; ++j) most = fmaxf(most, fabsf(raw[s][j]));
        most = max_of_column(most);
        int e = 10;
        if (most > 0.f && most < INFINITY) (void)frexpf(most, &e);
        sc = ldexpf(sc, e - 10);
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float x = ldexpf(raw[2 * s + (j >> 1 & 1)][(j >> 2) * 2 + (j & 1)], 10 - e);
            qh[s][j] = (_Float16)x;
            ql[s][j] = (_Float16)(x - (float)qh[s][j]);
          }
      }
      // Scores times sc have to grow with the products: a negative scale turns the query, and
      // one of 0 leaves nothing of it.
      if (!(sc > 0.f)) {
        rare();
        const _Float16 sign = sc < 0.f ? -1.f : 0.f;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          qh[s] *= sign;
          if constexpr (WIDE) ql[s] *= sign;
        }
        sc = sc < 0.f ? -sc : 1.f;
      }
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        floatx4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = j * kSteps / NG; i < (j + 1) * kSteps / NG; ++i) {
          s = __builtin_amdgcn_mfma_f32_16x16x32_f16(R::ones(), qh[i], s, 0, 0, 0);
          if constexpr (WIDE) s = __builtin_amdgcn_mfma_f32_16x16x32_f16(R::ones(), ql[i], s, 0, 0, 0);
        }
        qsum[j] = s[0] * R::kCode;
      }
    }

    float sum = 0.f, osum[NG];  // this lane's share of the weights, and of them times offsets
    floatx4 acc[kAccs];
    // A weight is 2 to the power of score - base, with base the running maximum rounded up to a
    // whole number, so that it changes by powers of 2, and `shift`: E - 15, with 2^E above the
    // finite scales of the values of a tile.
    float base = -INFINITY, shift = kLeastShift;
    // Magnitudes of scales, as numbers: those from the first on raise the shift, those of which 1
    // less is below the second are far below 2^E.
    uint32_t raises = 0, falls = 0;
    // Columns whose maximum and shift have no sum in fp32: base is the maximum, weights are of
    // (score - base) - shift.
    uint64_t far = 0;
    auto is_far = [&] { return (far >> lane & 1) != 0; };
#pragma unroll
    for (int j = 0; j < NG; ++j) osum[j] = 0.f;
#pragma unroll
    for (int i = 0; i < kAccs; ++i) acc[i] = floatx4{0.f, 0.f, 0.f, 0.f};

    // Products of half a pair are fused sums with a zero that the compiler does not see: one
    // mixed-precision instruction in the place of a conversion and a product.
    float zero;
    asm("s_mov_b32 %0, 0" : "=s"(zero));
    // Adds tile i.  A tile that only the general form (`any`) can add ends the other's loop, which
    // adds nothing of it: `bound`.  Where both can, their results are the same bits.
    int bound = tiles;
    bool again = false;  // whether the general form was needed
    auto compute = [&](const Tile& t, int i, auto any) {
      // Pairs: none of a token that does not exist, NaN for what is not finite.
      uint32_t e = 0, low = ~0u;  // the token's largest scale (or NaN), and its least but 0, less 1
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        uint32_t so = (t.live >> (lane & 31)) & 1 ? t.pair[n] : 0;
        if ((so & 0x7FFFu) >= kScaleInf || (so & 0x7C000000u) == 0x7C000000u) so = 0x7E007E00u;
        e = max(e, so & 0x7FFFu), low = min(low, (so & 0x7FFFu) - 1);
        s_pair[wave][n][lane] = so;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      // The pairs of group n of this lane's 8 tokens, of the keys (at 0) or the values (32).
      auto read_pairs = [&](int n, int at, uint32_t (&out)[8]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const v4u v = *reinterpret_cast<const v4u*>(&s_pair[wave][n][at + 16 * h + 4 * g]);
#pragma unroll
          for (int j = 0; j < 4; ++j) out[4 * h + j] = v[j];
        }
      };

      float x[8], most = -INFINITY;
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        uint32_t kp[8];
        read_pairs(n, 0, kp);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          floatx4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = n * kSteps / NG; k < (n + 1) * kSteps / NG; ++k) {
            const half8 codes = R::keys(t.k[h], k);
            s = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes, qh[k], s, 0, 0, 0);
            if constexpr (WIDE) s = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes, ql[k], s, 0, 0, 0);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const half2v so = as_half2(kp[4 * h + j]);
            float& y = x[4 * h + j];
            y = fmaf((float)so[1], qsum[n], n == 0 ? zero : y);
            y = fmaf((float)so[0], s[j], y);
          }
        }
      }
      const int tile_first = first + i * kUnit;
      const bool masked = t.live != ~0u || __any(tile_first + kTile > length);
      // bit j: this lane's token j exists and its column attends to it
      uint32_t on = (t.live >> (4 * g) & 15) | (t.live >> (16 + 4 * g) & 15) << 4;
      if (masked) {
        rare();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int tok = tile_first + (j >> 2) * 16 + 4 * g + (j & 3);
          on &= ~((uint32_t)(tok >= length) << j);
          x[j] = (on >> j) & 1 ? x[j] : -INFINITY;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) most = fmaxf(most, x[j]);
      most = max_of_column(most) * sc;
      // (lanes 32..63 hold values' scales)
      auto raised = [&] { return (uint32_t)(__ballot(e >= raises) >> 32); };
      auto fallen = [&] { return (uint32_t)(__ballot(low < falls) >> 32); };
      auto shift_to = [&](uint32_t exponent) {
        shift = kLeastShift + (float)(int)exponent;
        raises = kScaleExponent * (exponent + 1);
        falls = far_below(exponent);
      };
      auto times = [&](float f) {
        sum *= f;
#pragma unroll
        for (int n = 0; n < NG; ++n) osum[n] *= f;
#pragma unroll
        for (int n = 0; n < kAccs; ++n) acc[n] *= f;
      };
      // Scales of group n, as numbers; 0 where the column does not attend to the token.
      auto scales = [&](int n, uint32_t (&s)[8]) {
        read_pairs(n, kTile, s);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] &= (uint32_t)((int32_t)(on << (31 - j)) >> 31) & 0x7FFFu;
      };
      // The shift follows the scales of the tokens that all columns attend to which attend to any
      // of the tile (none must know of others'), with room for 4 times as much.
      auto follow = [&] {
        uint32_t common = ~0u;
        if (p.shared > 1) {
          const int left = least_of_row(length > tile_first ? length : INT32_MAX) - tile_first;
          common = left < kTile ? (1u << (left & 31)) - 1 : ~0u;
        }
        const uint32_t largest = largest_of_half((common >> (lane & 31)) & 1 ? e : 0);
        if (raises == 0 || largest >= raises || (largest != 0 && largest - 1 < falls))
          shift_to(largest / kScaleExponent + (largest < kScaleExponent ? 0 : 2));
      };
      // The maximum may pass what base stands for by a power of 2: twice 2^15 is still what the two
      // fp16 numbers of a product hold.
      auto rises = [&](float base) { return any && is_far() ? most > base : most + (shift - 1.f) > base; };
      [[maybe_unused]] float followed = shift;
      float ref = base == -INFINITY ? 0.f : base;
      if ((raised() | fallen() | far | __ballot(rises(base))) != 0) {
        rare();
        if (__any(e >= kScaleInf)) {  // the largest of the finite ones
          rare();
          e = 0;
#pragma unroll
          for (int n = 0; n < NG; ++n) {
            const uint32_t so = (t.live >> (lane & 31)) & 1 ? t.pair[n] : 0;
            if ((so & 0x7FFFu) < kScaleInf && (so & 0x7C000000u) != 0x7C000000u) e = max(e, so & 0x7FFFu);
          }
        }
        float up;
        if constexpr (!any) {
          if (raises == 0) {
            rare();
            follow();
          }
          up = rises(base) ? ceilf(most) + shift : base;
          uint64_t other = raised() | far | __ballot(fabsf(up) >= kFar && up != -INFINITY);
          if (fallen() != 0) {  // do weights of tokens without such scales come near the largest?
            rare();
            uint32_t least = ~0u;
#pragma unroll
            for (int n = 0; n < NG; ++n) least = min(least, t.pair[n] & 0x7FFFu);
            const uint32_t normal = __ballot(least > falls) >> 32;
            const uint32_t mine = on & ((normal >> (4 * g) & 15) | (normal >> (16 + 4 * g) & 15) << 4);
            float next = -INFINITY;
#pragma unroll
            for (int j = 0; j < 8; ++j) next = fmaxf(next, (mine >> j) & 1 ? x[j] : -INFINITY);
            other |= __ballot(max_of_column(next) * sc + kNear < most);
          }
          // (selections: with branches here the loop would copy its sums from register to register)
          bound = other != 0 ? i : bound;
          up = other != 0 ? base : up;
          times(up == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(base - up));
          ref = other != 0 ? INFINITY : (up == -INFINITY ? 0.f : up);
        } else {
          const float was = shift;
          if ((raised() | fallen()) != 0) follow();
          followed = shift;
          if (raised() != 0) shift_to(largest_of_half(e) / kScaleExponent);
          const float here = is_far() ? base : base + (shift - was);
          up = rises(here) ? ceilf(most) + (is_far() ? 0.f : shift) : here;
          const float top = is_far() ? up : up - shift, had = is_far() ? was : 0.f;
          far = __ballot(fabsf(top) >= kFar && top != -INFINITY);
          up = is_far() ? top : top + shift;
          times(up == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((base - up) + (had - (is_far() ? shift : 0.f))));
          ref = up == -INFINITY ? 0.f : up;
        }
        base = up;
      }
      // Powers of 2 of the weights: from the shift that the column knows of to the common one, and
      // of each group's products to their own.
      [[maybe_unused]] float unit = 1.f, lift[NG];
      if constexpr (any) {
        float mine = followed;
        if (shift != followed) {
          uint32_t largest = 0;
#pragma unroll
          for (int n = 0; n < NG; ++n) {
            uint32_t s[8];
            scales(n, s);
#pragma unroll
            for (int j = 0; j < 8; ++j) largest = max(largest, s[j] < kScaleInf ? s[j] : 0);
          }
          mine = fmaxf(mine, kLeastShift + max_of_column((float)(largest / kScaleExponent)));
        }
        unit = ldexpf(1.f, (int)(mine - shift));
        float weight = -INFINITY;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float y = fmaf(x[j], sc, (shift - mine) - ref);
          x[j] = is_far() ? minus(x[j], sc, ref) - mine : y;
          weight = fmaxf(weight, x[j]);
        }
        weight = max_of_column(weight);
        float most_lift = 1.f;
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          // Where scales far below the largest leave a group's largest product as far below what
          // the weight allows, it is lifted to below 2^15, but by no more than exponents of scales
          // differ by.  (NaN gives NaN with any lift; a scale of 0 counts as 2^-126.)
          uint32_t s[8], least = ~0u;
          scales(n, s);
          float product = -INFINITY;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int exponent = (int)(__float_as_uint((float)as_half2(s[j])[0]) >> 23) - 126;
            product = fmaxf(product, x[j] + exponent);
            least = min(least, s[j] - 1);
          }
          product = max_of_column(product);
          const float below = max_of_column(least < far_below((uint32_t)(mine - kLeastShift)) ? 1.f : 0.f);
          const bool needs = below > 0.f && product < weight + mine + (15.f - kFarBelow - 1.f - kNear);
          lift[n] = needs ? ldexpf(1.f, (int)fminf(fmaxf(15.f - product, 0.f), 40.f)) : 1.f;
          most_lift = fmaxf(most_lift, lift[n]);
        }
        again = (far | __ballot(most_lift > 1.f)) != 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __builtin_amdgcn_exp2f(x[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __builtin_amdgcn_exp2f(fmaf(x[j], sc, -ref));
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += any ? x[j] * unit : x[j];
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        uint32_t vp[8];
        read_pairs(n, kTile, vp);
        if (masked) {  // NaN of a token that this column does not attend to
          rare();
#pragma unroll
          for (int j = 0; j < 8; ++j) vp[j] = (on >> j) & 1 ? vp[j] : 0;
        }
        v4u ph, pl;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const half2v a0 = as_half2(vp[2 * w]), a1 = as_half2(vp[2 * w + 1]);
          float x0 = x[2 * w], x1 = x[2 * w + 1];
          osum[n] = fmaf((float)a0[1], any ? x0 * unit : x0, osum[n]);
          osum[n] = fmaf((float)a1[1], any ? x1 * unit : x1, osum[n]);
          if constexpr (any) x0 *= lift[n], x1 *= lift[n];
          // (The first is cut, which keeps it finite, the second rounded: cut too, sums would come
          // out low by 7.5e-8 on average.)
          const auto h = __builtin_amdgcn_cvt_pkrtz(fmaf((float)a0[0], x0, zero), fmaf((float)a1[0], x1, zero));
          ph[w] = __builtin_bit_cast(uint32_t, h);
          pl[w] = pack(fmaf((float)a0[0], x0, -(float)h[0]), fmaf((float)a1[0], x1, -(float)h[1]));
        }
#pragma unroll
        for (int k = n * kAccs / NG; k < (n + 1) * kAccs / NG; ++k) {
          const half8 v = R::values(t.v, k);
          if constexpr (any) acc[k] *= lift[n] / unit;
          acc[k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, as_half8(ph), acc[k], 0, 0, 0);
          acc[k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, as_half8(pl), acc[k], 0, 0, 0);
          if constexpr (any) acc[k] *= unit / lift[n];
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    };

    // (A request past the last tile reads the masked token of page 0; without it the paths
    // through the loop would have to wait for one another's loads.)
    constexpr std::false_type kFast;
    constexpr std::true_type kAny;
    while (i < tiles) {
      bound = tiles;
      for (;;) {
        request(odd, i + 2);
        compute(even, i, kFast);
        if (++i >= bound) break;
        request(even, i + 2);
        compute(odd, i, kFast);
        if (++i >= bound) break;
      }
      if (bound != tiles) {  // from that tile on in the general form, as long as it is needed
        rare();
        i = bound;
        look_up(i);
        request(even, i + 1);
        do {
          request(odd, i + 2);
          compute(even, i, kAny);
          even = odd;
        } while (++i < tiles && again);
      }
    }

    // Join the four waves.
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      osum[n] += __shfl_xor(osum[n], 16);
      osum[n] += __shfl_xor(osum[n], 32);
    }
    if (far != 0) {  // sums of weights with the shift in their base
      rare();
      const float unit = is_far() ? ldexpf(1.f, (int)shift) : 1.f;
      sum *= unit;
#pragma unroll
      for (int n = 0; n < NG; ++n) osum[n] *= unit;
#pragma unroll
      for (int n = 0; n < kAccs; ++n) acc[n] *= unit;
    }
    if (g == 0) s_ml[wave][m] = make_float2(base, sum);
    if (m < columns) {
#pragma unroll
      for (int i = 0; i < kAccs; ++i)
        *reinterpret_cast<floatx4*>(&s_acc[wave][m][i * 16 + g * 4]) =
            acc[i] * (1.f / R::kCode) + osum[i * NG / kAccs];
    }
    __syncthreads();
    for (int e = own(threadIdx.x); e < columns * (D / 4); e += kThreads) {
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
        T* out = static_cast<T*>(a.out) + (int64_t)(first_query + (p.shared > 1 ? h / heads : 0)) * a.out_stride +
                 (int64_t)(head0 + (p.shared > 1 ? h % heads : h)) * D + d;
        store4(out, o * (total == 0.f ? 0.f : 1.f / total));
      } else {
        const int64_t at =
            ((int64_t)(2 * blockIdx.y + (starts_run ? 0 : 1)) * gridDim.x + blockIdx.x) * 16 + h;
        *reinterpret_cast<floatx4*>(p.acc + at * D + d) = o;
        if (d == 0) p.ml[at] = make_float2(mx, total);
      }
    }
    __syncthreads();  // s_ml and s_acc have been read
  }
}

// Joins the pieces of one query and head, and writes zeros for queries without any.
// THREADS threads take a head, of 4 in a workgroup or alone; every wave forms the maximum
// and the sum itself, and groups of D/4 lanes take the pieces in turn.
template <int D, bool WIDE, int THREADS>
__global__ __launch_bounds__(kThreads) void qcache_attend_join_kernel(const Args p) {
  using T = std::conditional_t<WIDE, float, __half>;
  constexpr int kLanes = D / 4, kGroups = THREADS / kLanes, kHeads = kThreads / THREADS;
  __shared__ __align__(16) floatx4 s_part[kHeads][kGroups][kLanes];
  const seedlm_qcache_attend_args& a = p.a;
  const int thread = threadIdx.x % THREADS, nth = threadIdx.x / THREADS;
  const int query = blockIdx.y, head = blockIdx.x * kHeads + nth;
  if (head >= a.heads) return;
  const int4 join = p.joins[query];
  const int first_slot = join.y, pieces = join.z, skip = join.w;
  if (pieces == 1) return;
  T* out = static_cast<T*>(a.out) + (int64_t)query * a.out_stride + (int64_t)head * D;
  const int lane = thread % kLanes, group = thread / kLanes;
  const int in_group = head % p.group, heads = min(16, p.group - in_group / 16 * 16);
  const int block = head / p.group * p.qtiles + in_group / 16;
  const int column = (query - join.x) * heads + in_group % 16;
  const int blocks = a.cache.kv_heads * p.qtiles;
  auto partial = [&](int s) {
    return ((int64_t)(2 * (first_slot + s) + (s == 0 ? skip : 0)) * blocks + block) * 16 + column;
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
  s_part[nth][group][lane] = o;
  if constexpr (THREADS == kThreads) {
    __syncthreads();
  } else {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
  if (group != 0) return;
#pragma unroll
  for (int k = 1; k < kGroups; ++k) o += s_part[nth][k][lane];
  store4(out + lane * 4, o * (total == 0.f ? 0.f : 1.f / total));
}

// Whether codes pass the caches: calls that read so much find little of it there the next
// time, when the call has gone round other layers' caches.  Against caching, 16 requests
// alike, three inputs in turn: 128 dimensions, 4 bits, 31.9 and 33.0 us at 120 MB, 64.5 and
// 67.5 at 300, 175 and 179 at 900, 8 bits 30.9 and 32.1, 58.8 and 64.1, 154 and 169; 256, 4
// bits, 64.4 and 67.2 at 300.  Below, all inputs may lie in the memory-side cache: 24.6
// and 23.5 at 68 MB; the lengths are not known here, and ragged ones of half the bound lose
// 2 to 4%.  64 dimensions of 8 bits gain as much (58.3 and 64.2 at 300), rows of
// 32 bytes nothing (81.8 and 80.6), and rows of 256 bytes lose (39 and 34, 73 and 65, 187
// and 169).  Calls with `rows` stay in the caches, since queries of one row that lie in
// different items read its pages again: 256 pieces of 8 queries 243 and 225, 16 of 16 68 and
// 62.  Where each row has one token, that costs them the gain (128 requests of 32 cache
// heads and 64 dimensions at 2000 tokens 184 and 197).
constexpr bool may_stream(int row_bits) { return row_bits == 512 || row_bits == 1024; }

inline bool streams(const seedlm_qcache_attend_args& a, int cap) {
  const seedlm_qcache_t& c = a.cache;
  const int64_t row = c.head_dim * c.bits / 8 + 4 * (c.head_dim / c.group);
  return !a.rows && may_stream(c.head_dim * c.bits) &&
         (int64_t)a.queries * cap * c.kv_heads * 2 * row > (int64_t)110 << 20;
}

// Joins of so many queries and heads take a wave each, fewer a workgroup, which reads the
// many pieces of long requests faster.  Calls, waves against workgroups: 64 requests of 32
// heads 50.5 and 51.7 us, 256 of 32 167 and 169; 16 of 64 22.0 and 21.7, one of 100000
// tokens 34.3 and 31.4.
constexpr int64_t kManyJoins = 2048;

template <int D, int BITS, int NG, bool WIDE>
int run_groups(const Args& p, hipStream_t s) {
  const seedlm_qcache_attend_args& a = p.a;
  const bool split = p.slots > 0;
  const auto kernel = streams(a, p.cap) ? qcache_attend_kernel<D, BITS, NG, WIDE, may_stream(D * BITS)>
                                        : qcache_attend_kernel<D, BITS, NG, WIDE, false>;
  hipLaunchKernelGGL(kernel, dim3(a.cache.kv_heads * p.qtiles, p.rows), dim3(kThreads),
                     (split ? 2 * a.queries : p.shared) * sizeof(int32_t), s, p);
  if (split && (int64_t)a.heads * a.queries >= kManyJoins)
    hipLaunchKernelGGL((qcache_attend_join_kernel<D, WIDE, 64>), dim3((a.heads + 3) / 4, a.queries),
                       dim3(kThreads), 0, s, p);
  else if (split)
    hipLaunchKernelGGL((qcache_attend_join_kernel<D, WIDE, kThreads>), dim3(a.heads, a.queries),
                       dim3(kThreads), 0, s, p);
  return hipGetLastError() == hipSuccess ? SEEDLM_OK : SEEDLM_E_DEVICE;
}

// A checked call of one code width and one type of queries; each is a source of its own.
template <int BITS, bool WIDE>
int run(const Args& p, hipStream_t s) {
  const int groups = p.a.cache.head_dim / p.a.cache.group;
  switch (p.a.cache.head_dim) {
    case 64: return groups == 1 ? run_groups<64, BITS, 1, WIDE>(p, s)
                                : run_groups<64, BITS, 2, WIDE>(p, s);
    case 128: return groups == 1 ? run_groups<128, BITS, 1, WIDE>(p, s)
                   : groups == 2 ? run_groups<128, BITS, 2, WIDE>(p, s)
                                 : run_groups<128, BITS, 4, WIDE>(p, s);
    case 256: return groups == 1 ? run_groups<256, BITS, 1, WIDE>(p, s)
                   : groups == 2 ? run_groups<256, BITS, 2, WIDE>(p, s)
                                 : run_groups<256, BITS, 4, WIDE>(p, s);
    default: return SEEDLM_E_UNSUPPORTED;
  }
}
int run_4(const Args& p, hipStream_t s);
int run_4_wide(const Args& p, hipStream_t s);
int run_8(const Args& p, hipStream_t s);
int run_8_wide(const Args& p, hipStream_t s);

}  // namespace qattend
}  // namespace seedlm
