// Low-rank adapters of many requests beside shared projections
// (seedlm_lora_many): y[t] = base[t] + scales[a] B_a (A_a x[t]), a = adapter[t],
// for up to 8 sites (projections) in one pair of launches.
//
// Two launches: "down" is h = A x, cut along the columns into chunks so that few
// rows still fill the chip, its chunk sums going to scratch as fp32
// [site][chunk][token][rank]; "up" adds the chunks in order, multiplies with B,
// scales, adds base and rounds once.  Few rows with a small A take one launch, whose
// workgroups each form h.
//
// Few rows (any types, any sizes): a workgroup per row, chunk and 16 ranks, its lanes
// along the columns, the 16 sums exchanged by halves across the wave; then a thread
// per output.  The bytes of A and B, once per row, bound it.
//
// Many rows (fp16): v_mfma_f32_16x16x32_f16, with A (then B) as the first operand
// and 16 rows as the second, so that a lane's results belong to one row:
//   sort  rows gathered by adapter into tiles of 32, so that a tile has one adapter
//         however the rows lie
//   down  a tile and up to 64 ranks per workgroup, x and A staged through LDS
//   up    a tile and 64 outputs per wave and step; the sums turn over in LDS.  h
//         enters as two fp16 numbers, h 2^-e = hi + lo (22 bits; e from the row's
//         largest finite |h|).  Infinities are in hi alone, and lo meets a finite B
//         alone, so that they give what the formula does.  Up to rank 16 the 16 high
//         and 16 low parts fill the 32 products of one MFMA against the same 16
//         elements of B twice.
// The bytes of x, base and y bound these.  Many rows of fp32, and ranks that are no
// multiple of 8, take the row kernels, which read A and B once per row.
//
// Measured: 16 requests on q, k and v of a 70B layer at rank 16 (18.7 MB) 8.1 us in
// one launch; 2049 rows on gate and up of an 8B layer at rank 16, sort 6.7, down 10.4,
// up 55 us for 235 MB (4.3 TB/s; a large copy reaches 4.8), 70 us a call; at rank 4, by
// the row kernels, 54 and 310 us; 512 rows of fp32 at rank 16, likewise, 18 and 84 us;
// 1159 rows on q, k and v of the 70B layer at rank 64 (102 MB), sort 5.1, down 18.9, up
// 32 us.
#include <hip/hip_fp16.h>

#include "seedlm_internal.h"

namespace seedlm {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kChunk = 8 * kThreads;  // columns of a workgroup of the row kernels
constexpr int kTileRows = 32;         // rows of a tile, of one adapter
constexpr int kDownRanks = 64;        // ranks at most of a down workgroup
constexpr int kDownStep = 256;        // columns staged at once
constexpr int kUpRows = 2 * kTileRows;  // rows of an up workgroup, two waves per tile
constexpr int kUpStep = 128;            // outputs of its step
static_assert(kWaves == 4, "the tile kernels share tiles out to four waves");

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

struct Site {
  const void* x;
  const __half* A;
  const __half* B;
  const void* base;
  void* y;
  float* h;        // [chunks][tokens][rank]
  int rows, cols, rank;
  int chunks;
  int chunk_cols;  // columns of a chunk
  int up_outputs;  // outputs of an up workgroup
  int wide;        // 16-byte accesses fit
  int first_down;  // first workgroup (x dimension) of this site in the two launches
  int first_up;
};

struct LoraArgs {
  Site s[kLoraGroup];
  const int32_t* adapter;
  const float* scales;
  int32_t* tile_count;  // tiles of the many-row form, their adapters and rows
  int32_t* tiles;
  int32_t* order;
  int32_t* place;
  int n, tokens, adapters;
};

__device__ const Site& site_of(const LoraArgs& p, bool up, int block) {
  int i = 0;
  for (int k = 1; k < p.n; ++k)
    if (block >= (up ? p.s[k].first_up : p.s[k].first_down)) i = k;
  return p.s[i];
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

// Adds v[i] over the wave's lanes; lane l returns the sum of element l / 4 (halves
// of the elements are exchanged at each of four steps, then two plain ones).
__device__ float wave_sums16(float (&v)[16]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int step = 0; step < 4; ++step) {
    constexpr int kHalf = 8;
    const int n = kHalf >> step, d = 32 >> step;
    const bool up = lane & d;
#pragma unroll
    for (int i = 0; i < kHalf; ++i) {
      if (i >= n) continue;
      const float a = v[i], b = v[i + n];  // copies: a choice of elements is one by address
      v[i] = (up ? b : a) + __shfl_xor(up ? a : b, d);
    }
  }
  v[0] += __shfl_xor(v[0], 2);
  return v[0] + __shfl_xor(v[0], 1);
}

// v[j] += A[j][c] x[c] for `ranks` <= 16 rows of A (past them the last one's again)
// over the columns c0 + 8 tid + (0..7), c0 + 8 (tid + kBlock) + .., below c1 (one by
// one where 16-byte loads do not fit).
template <int kBlock, typename XT>
__device__ void contract16(const XT* x, const __half* A, int cols, int ranks, bool wide, int c0,
                           int c1, float (&v)[16]) {
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = 0.f;
  if (wide) {
    for (int c = c0 + (int)threadIdx.x * 8; c < c1; c += kBlock * 8) {
      half8 av[16];
#pragma unroll
      for (int j = 0; j < 16; ++j)
        av[j] = *reinterpret_cast<const half8*>(A + (int64_t)min(j, ranks - 1) * cols + c);
      float xv[8];
      load8(x + c, xv);
#pragma unroll
      for (int j = 0; j < 16; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j] = fmaf((float)av[j][i], xv[i], v[j]);
    }
  } else {
    for (int c = c0 + (int)threadIdx.x; c < c1; c += kBlock) {
      const float xc = (float)x[c];
#pragma unroll
      for (int j = 0; j < 16; ++j)
        v[j] = fmaf(__half2float(A[(int64_t)min(j, ranks - 1) * cols + c]), xc, v[j]);
    }
  }
}

// 16 ranks of h of one token over one chunk of columns.
template <typename XT>
__global__ __launch_bounds__(kThreads) void lora_down_rows_kernel(const LoraArgs p) {
  __shared__ float s_part[kWaves][16];
  const Site& s = site_of(p, false, blockIdx.x);
  const int rank_blocks = (s.rank + 15) / 16;
  const int chunk = (blockIdx.x - s.first_down) / rank_blocks;
  const int j0 = (blockIdx.x - s.first_down) % rank_blocks * 16;
  const int ranks = min(16, s.rank - j0);
  const int c0 = chunk * s.chunk_cols, c1 = min(s.cols, c0 + s.chunk_cols);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int t = blockIdx.y; t < p.tokens; t += gridDim.y) {
    const int a = p.adapter[t];
    if (a < 0 || a >= p.adapters) continue;
    float v[16];
    const XT* x = static_cast<const XT*>(s.x) + (int64_t)t * s.cols;
    const __half* A = s.A + ((int64_t)a * s.rank + j0) * s.cols;
    contract16<kThreads>(x, A, s.cols, ranks, s.wide, c0, c1, v);
    const float sum = wave_sums16(v);
    __syncthreads();  // s_part of the token before has been read
    if ((lane & 3) == 0) s_part[wave][lane >> 2] = sum;
    __syncthreads();
    const int j = threadIdx.x;
    if (j < ranks) {
      float h = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) h += s_part[w][j];
      s.h[((int64_t)chunk * p.tokens + t) * s.rank + j0 + j] = h;
    }
  }
}

// Row r of B_a times h (in LDS).
__device__ float dot_b(const Site& s, int a, int r, const float* h) {
  const __half* B = s.B + ((int64_t)a * s.rows + r) * s.rank;
  float d = 0.f;
  if (s.wide) {
#pragma unroll 4
    for (int j = 0; j < s.rank; j += 8) {
      float bv[8];
      load8(B + j, bv);
#pragma unroll
      for (int i = 0; i < 8; ++i) d = fmaf(bv[i], h[j + i], d);
    }
  } else {
    for (int j = 0; j < s.rank; ++j) d = fmaf(__half2float(B[j]), h[j], d);
  }
  return d;
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
    if (has) sum += dot_b(s, a, r, s_h);
    static_cast<YT*>(s.y)[at] = (YT)sum;
  }
}

// ---- fewest rows: one launch ----

constexpr int kOneThreads = 1024;
constexpr int kOneRank = 16;  // ranks at most
constexpr int kOneWaves = kOneThreads / 64;

// y of one token and a block of outputs of one site, h included: every workgroup of
// a token forms h again, its waves sharing the columns, which costs less than a
// second launch while the repeated reads of A are few.
template <typename XT, typename YT>
__global__ __launch_bounds__(kOneThreads) void lora_one_kernel(const LoraArgs p, int blocks) {
  __shared__ float s_part[kOneWaves][kOneRank];
  __shared__ float s_h[kOneRank];
  // 8 tokens or more: a token's workgroups take one XCD (block number mod 8), whose
  // L2 then serves the repeats
  const int padded = (p.tokens + 7) / 8 * 8;
  const bool near = p.tokens >= 8;
  const int t = near ? blockIdx.x % padded : blockIdx.x / blocks;
  const int block = near ? blockIdx.x / padded : blockIdx.x % blocks;
  if (t >= p.tokens) return;
  const Site& s = site_of(p, true, block);
  const int a = p.adapter[t];
  const bool has = a >= 0 && a < p.adapters;
  if (!has && s.y == s.base) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int first = (block - s.first_up) * s.up_outputs;
  const int end = min(s.rows, first + s.up_outputs);
  const YT* base = static_cast<const YT*>(s.base) + (int64_t)t * s.rows;
  YT* y = static_cast<YT*>(s.y) + (int64_t)t * s.rows;
  // What the thread's first output needs, requested before A x.
  const int mine = first + tid;
  const float base0 = mine < end ? (float)base[mine] : 0.f;
  const bool ahead = has && s.wide && mine < end;
  half8 b_lo = {0, 0, 0, 0, 0, 0, 0, 0}, b_hi = b_lo;
  if (ahead) {
    const half8* B = reinterpret_cast<const half8*>(s.B + ((int64_t)a * s.rows + mine) * s.rank);
    b_lo = B[0];
    if (s.rank > 8) b_hi = B[1];
  }
  if (has) {
    float v[16];
    contract16<kOneThreads>(static_cast<const XT*>(s.x) + (int64_t)t * s.cols,
                            s.A + (int64_t)a * s.rank * s.cols, s.cols, s.rank, s.wide, 0, s.cols,
                            v);
    const float sum = wave_sums16(v);
    if ((lane & 3) == 0) s_part[wave][lane >> 2] = sum;
    __syncthreads();
    if (tid < kOneRank) {
      float h = 0.f;
#pragma unroll
      for (int w = 0; w < kOneWaves; ++w) h += s_part[w][tid];
      s_h[tid] = tid < s.rank ? h * p.scales[a] : 0.f;
    }
    __syncthreads();
  }
  for (int r = first + tid; r < end; r += kOneThreads) {
    float sum = r == mine ? base0 : (float)base[r], d = 0.f;
    if (ahead && r == mine) {
#pragma unroll
      for (int i = 0; i < 8; ++i) d = fmaf((float)b_lo[i], s_h[i], d);
      if (s.rank > 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) d = fmaf((float)b_hi[i], s_h[8 + i], d);
      }
    } else if (has) {
      d = dot_b(s, a, r, s_h);
    }
    y[r] = (YT)(sum + d);
  }
}

// ---- many rows: the matrix cores ----

__device__ floatx4 mfma(v4u a, v4u b, floatx4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a),
                                                __builtin_bit_cast(half8, b), c, 0, 0, 0);
}

// Gathers the rows into tiles of kTileRows rows of one adapter (and of rows without
// one, whose adapter is -1): tile i has adapter tiles[i] and rows order[kTileRows * i
// + ..], -1 past its last one.  A counting sort by one workgroup, LDS counters being
// advanced once per wave and adapter; which place a row gets in its adapter's tiles
// depends on the order of these, its results do not.
constexpr int kSortThreads = 1024;
constexpr int kSortAtOnce = 4;  // rows of a thread requested together
constexpr int kSortAdapters = 8191;

__global__ __launch_bounds__(kSortThreads) void lora_sort_kernel(const LoraArgs p) {
  extern __shared__ int s_count[];  // [buckets] rows, then [buckets] first tiles
  __shared__ int s_wave[kSortThreads / 64];
  const int buckets = p.adapters + 1;  // the last one: none
  int* s_first = s_count + buckets;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int b = tid; b < buckets; b += kSortThreads) s_count[b] = 0;
  __syncthreads();
  auto bucket_of = [&](int t) {
    const int a = t < p.tokens ? p.adapter[t] : -1;
    return t >= p.tokens ? -1 : (a < 0 || a >= p.adapters ? p.adapters : a);
  };
  // Count the rows; place[t] is a row's place in its bucket.
  for (int t0 = 0; t0 < p.tokens; t0 += kSortThreads * kSortAtOnce) {
    int b[kSortAtOnce];
#pragma unroll
    for (int i = 0; i < kSortAtOnce; ++i) b[i] = bucket_of(t0 + i * kSortThreads + tid);
#pragma unroll
    for (int i = 0; i < kSortAtOnce; ++i) {
      for (uint64_t todo = __ballot(b[i] >= 0); todo;) {
        const int leader = (int)__builtin_ctzll(todo);
        const int one = __builtin_amdgcn_readlane(b[i], leader);
        const uint64_t own = __ballot(b[i] == one);
        todo &= ~own;
        int first = 0;
        if (lane == leader) first = atomicAdd(&s_count[one], __popcll(own));
        first = __builtin_amdgcn_readlane(first, leader);
        if (b[i] == one)
          p.place[t0 + i * kSortThreads + tid] =
              first + __popcll(own & (((uint64_t)1 << lane) - 1));
      }
    }
  }
  __syncthreads();
  // First tiles: sums of the buckets' tiles, a run of buckets per thread.
  const int per = (buckets + kSortThreads - 1) / kSortThreads;
  const int b0 = min(tid * per, buckets), b1 = min(b0 + per, buckets);
  int mine = 0;
  for (int b = b0; b < b1; ++b) mine += (s_count[b] + kTileRows - 1) / kTileRows;
  int upto = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 63) s_wave[wave] = upto;
  __syncthreads();
  int first = upto - mine, all = 0;
  for (int w = 0; w < kSortThreads / 64; ++w) {
    if (w < wave) first += s_wave[w];
    all += s_wave[w];
  }
  if (tid == 0) *p.tile_count = all;
  for (int b = b0; b < b1; ++b) {
    const int rows = s_count[b], tiles = (rows + kTileRows - 1) / kTileRows;
    for (int i = rows; i < tiles * kTileRows; ++i) p.order[(int64_t)first * kTileRows + i] = -1;
    s_first[b] = first;
    first += tiles;
  }
  __syncthreads();
#pragma unroll kSortAtOnce
  for (int t = tid; t < p.tokens; t += kSortThreads) {
    const int b = bucket_of(t), place = p.place[t];
    const int tile = s_first[b] + place / kTileRows;
    p.order[(int64_t)tile * kTileRows + place % kTileRows] = t;
    if (place % kTileRows == 0) p.tiles[tile] = b < p.adapters ? b : -1;
  }
}

// h of one tile's rows, RT * 16 ranks and one chunk.  x and A pass through LDS, so
// that a wave loads two rows of 512 bytes at once: read straight into operands, 16
// rows of 64 bytes whose stride is a multiple of 4 KiB fall on few cache sets and
// channels.  Wave w contracts rows 16 (w%2) + (0..15) over half w/2 of each step.
template <int RT>
__global__ __launch_bounds__(kThreads) void lora_down_tile_kernel(const LoraArgs p) {
  constexpr int kRow = kDownStep + 8;  // halves between rows in LDS
  constexpr int kRanks = RT * 16;
  constexpr int kXLoads = kTileRows * kDownStep / 8 / kThreads;
  constexpr int kALoads = kRanks * kDownStep / 8 / kThreads;
  __shared__ __align__(16) uint16_t s_x[kTileRows * kRow];
  __shared__ __align__(16) uint16_t s_a[kRanks * kRow];
  __shared__ __align__(16) float s_h[kTileRows][kRanks + 4];  // of the second half
  const int tile = blockIdx.y;
  if (tile >= *p.tile_count) return;
  const int a = p.tiles[tile];
  if (a < 0) return;
  const int32_t* order = p.order + (int64_t)tile * kTileRows;
  const Site& s = site_of(p, false, blockIdx.x);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int m = lane & 15, g = lane >> 4;
  const int rank_blocks = (s.rank + kRanks - 1) / kRanks;
  const int chunk = (blockIdx.x - s.first_down) / rank_blocks;
  const int j0 = (blockIdx.x - s.first_down) % rank_blocks * kRanks;
  const int ranks = min(kRanks, s.rank - j0);  // a multiple of 8
  const int c0 = chunk * s.chunk_cols, c1 = min(s.cols, c0 + s.chunk_cols);
  // Thread tid stages 8 columns (tid % 32) of rows tid / 32 + 8 i; rows that are none
  // stage the first one again.
  const int col = tid % (kDownStep / 8) * 8, row = tid / (kDownStep / 8);
  constexpr int kRowsAtOnce = kThreads / (kDownStep / 8);
  const __half* x[kXLoads];
#pragma unroll
  for (int i = 0; i < kXLoads; ++i) {
    const int t = order[row + kRowsAtOnce * i];
    x[i] = static_cast<const __half*>(s.x) + (int64_t)(t >= 0 ? t : order[0]) * s.cols + col;
  }
  const __half* A = s.A + ((int64_t)a * s.rank + j0) * s.cols + col;
  v4u xv[kXLoads], av[kALoads];
  auto request = [&](int c) {
    const v4u z = {0, 0, 0, 0};
    const bool in = c + col < c1;
#pragma unroll
    for (int i = 0; i < kXLoads; ++i) xv[i] = in ? *reinterpret_cast<const v4u*>(x[i] + c) : z;
#pragma unroll
    for (int i = 0; i < kALoads; ++i) {
      const int j = min(row + kRowsAtOnce * i, ranks - 1);
      av[i] = in ? *reinterpret_cast<const v4u*>(A + (int64_t)j * s.cols + c) : z;
    }
  };
  floatx4 acc[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) acc[r] = floatx4{0.f, 0.f, 0.f, 0.f};
  request(c0);
  for (int c = c0; c < c1; c += kDownStep) {
    __syncthreads();  // the step before has been read
#pragma unroll
    for (int i = 0; i < kXLoads; ++i)
      *reinterpret_cast<v4u*>(&s_x[(row + kRowsAtOnce * i) * kRow + col]) = xv[i];
#pragma unroll
    for (int i = 0; i < kALoads; ++i)
      *reinterpret_cast<v4u*>(&s_a[(row + kRowsAtOnce * i) * kRow + col]) = av[i];
    if (c + kDownStep < c1) request(c + kDownStep);
    __syncthreads();
    const int k0 = (wave >> 1) * (kDownStep / 2) + g * 8;
#pragma unroll
    for (int k = 0; k < kDownStep / 2; k += 32) {
      const v4u xk = *reinterpret_cast<const v4u*>(&s_x[((wave & 1) * 16 + m) * kRow + k0 + k]);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const v4u ak = *reinterpret_cast<const v4u*>(&s_a[(r * 16 + m) * kRow + k0 + k]);
        acc[r] = mfma(ak, xk, acc[r]);
      }
    }
  }
  // the second half's sums pass to the first's waves, which hold the same rows
  const int place = (wave & 1) * 16 + m;
  if (wave >= 2) {
#pragma unroll
    for (int r = 0; r < RT; ++r) *reinterpret_cast<floatx4*>(&s_h[place][r * 16 + g * 4]) = acc[r];
  }
  __syncthreads();
  const int t = order[place];
  if (wave >= 2 || t < 0) return;
  float* h = s.h + ((int64_t)chunk * p.tokens + t) * s.rank + j0;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int j = r * 16 + g * 4;
    if (j < ranks)
      *reinterpret_cast<floatx4*>(h + j) =
          acc[r] + *reinterpret_cast<const floatx4*>(&s_h[place][j]);
  }
}

// The chosen 16-bit halves of 8 words, packed.
__device__ v4u parts(v4u p0, v4u p1, uint32_t select) {
  const auto pick = [&](uint32_t hi, uint32_t lo) { return __builtin_amdgcn_perm(hi, lo, select); };
  return v4u{pick(p0[1], p0[0]), pick(p0[3], p0[2]), pick(p1[1], p1[0]), pick(p1[3], p1[2])};
}

// fp16 values with +-65504 for infinities and NaN (as integers fp16 values of one sign
// are in order; negative ones lie below the positive as int16, above them as uint16).
typedef int16_t short8 __attribute__((ext_vector_type(8)));
typedef uint16_t ushort8 __attribute__((ext_vector_type(8)));
__device__ v4u limit(v4u v) {
  const short8 p = __builtin_elementwise_min(__builtin_bit_cast(short8, v), (short8)(int16_t)0x7BFF);
  return __builtin_bit_cast(
      v4u, __builtin_elementwise_min(__builtin_bit_cast(ushort8, p), (ushort8)(uint16_t)0xFBFF));
}

// y of two tiles' rows and s.up_outputs outputs; of a step, a wave has its tile's rows
// and 64 outputs, so that B is loaded once for 32 rows (the vector cache's accesses
// bound higher ranks).  BLOCK: ranks of a pass, 16 (for at most 16: high and low parts
// in one MFMA, B twice) or 32 (an MFMA each, on one load of B).
template <int BLOCK>
__global__ __launch_bounds__(kThreads) void lora_up_tile_kernel(const LoraArgs p) {
  constexpr int kOut = kUpStep / 2;  // outputs of a wave's step
  // h of the rows, each value as hi | lo << 16, ranks padded with zeros to BLOCKs;
  // the factor scales[a] * 2^e of each row; and a wave's sums of a step, turned over
  // so that base and y are read and written in runs of 128 bytes
  extern __shared__ __align__(16) uint32_t s_all_pairs[];
  __shared__ float s_all_factors[kUpRows];
  __shared__ __align__(16) float s_all_sums[kWaves][kTileRows][kOut + 4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int m = lane & 15, g = lane >> 4, half = wave & 1;
  const int tiles = *p.tile_count;
  if ((int)blockIdx.y * 2 >= tiles) return;
  const Site& s = site_of(p, true, blockIdx.x);
  const int tile = min((int)blockIdx.y * 2 + (wave >> 1), tiles - 1);
  const int a = __builtin_amdgcn_readfirstlane(p.tiles[tile]);
  const bool idle = (int)blockIdx.y * 2 + (wave >> 1) >= tiles || (a < 0 && s.y == s.base);
  const int32_t* order = p.order + (int64_t)tile * kTileRows;
  const int ranks = (s.rank + BLOCK - 1) / BLOCK * BLOCK, stride = ranks + 4;
  uint32_t* s_pair = s_all_pairs + (wave >> 1) * kTileRows * stride;
  float* s_factor = s_all_factors + (wave >> 1) * kTileRows;
  auto& s_sum = s_all_sums[wave];
  // In base and y lane l has outputs 8 (l%8) + (0..7) of rows order[8 i + l/8].
  const int o_begin = (blockIdx.x - s.first_up) * s.up_outputs;
  const int o_end = min(s.rows, o_begin + s.up_outputs);
  const int o_lane = half * kOut + (lane & 7) * 8;
  int rows[4];
  v4u bases[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) rows[i] = idle ? -1 : order[8 * i + (lane >> 3)];
  auto request = [&](int o0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (o0 + o_lane < s.rows && rows[i] >= 0)
        bases[i] = __builtin_nontemporal_load(
            reinterpret_cast<const v4u*>(static_cast<const __half*>(s.base) +
                                         (int64_t)rows[i] * s.rows + o0 + o_lane));
  };
  request(o_begin);
  if (a >= 0) {
    // a wave has 16 of its tile's rows: four lanes a row, four ranks at a time
    constexpr int kAtOnce = 8;
    const int row = half * 16 + (lane >> 2), part = lane & 3, t = max(order[row], 0);
    uint32_t* pair = s_pair + row * stride;
    float top = 0.f;          // the row's largest |h|
    uint32_t low = ~0u;       // and the bits of its smallest one but zero, times 2, less 1
#pragma unroll 2
    for (int j = part * 4; j < ranks; j += 16) {
      floatx4 sum = {0.f, 0.f, 0.f, 0.f};
      for (int c0 = 0; j < s.rank && c0 < s.chunks; c0 += kAtOnce) {
        floatx4 v[kAtOnce];  // requested together
#pragma unroll
        for (int c = 0; c < kAtOnce; ++c) {
          v[c] = floatx4{0.f, 0.f, 0.f, 0.f};
          if (c0 + c < s.chunks)
            v[c] = *reinterpret_cast<const floatx4*>(
                s.h + ((int64_t)(c0 + c) * p.tokens + t) * s.rank + j);
        }
#pragma unroll
        for (int c = 0; c < kAtOnce; ++c) sum += v[c];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        top = fmaxf(top, fabsf(sum[i]));
        low = min(low, (__float_as_uint(sum[i]) << 1) - 1u);
      }
      *reinterpret_cast<floatx4*>(&pair[j]) = sum;
    }
    top = fmaxf(top, __shfl_xor(top, 1));
    top = fmaxf(top, __shfl_xor(top, 2));
    // the row's largest finite value into [2^9, 2^10): the low parts keep all bits
    auto exponent = [&] {
      top = fmaxf(top, __shfl_xor(top, 1));
      top = fmaxf(top, __shfl_xor(top, 2));
      int e = 10;
      if (top > 0.f && top < INFINITY) (void)frexpf(top, &e);
      return e;
    };
    int e = exponent();
    // rows with an infinity, or with a value that is too small for fp16 beside the largest
    const float least = __uint_as_float((low + 1u) >> 1);
    const bool odd = __any(top == INFINITY || (least > 0.f && ldexpf(least, 10 - e) < 0x1p-24f));
    if (odd) {
      top = 0.f;
      for (int j = part * 4; j < ranks; j += 16)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float h = fabsf(__uint_as_float(pair[j + i]));
          top = fmaxf(top, h < INFINITY ? h : 0.f);
        }
      e = exponent();
    }
    for (int j = part * 4; j < ranks; j += 16) {
      v4u* at = reinterpret_cast<v4u*>(&pair[j]);
      v4u v = *at;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float h = __uint_as_float(v[i]), f = ldexpf(h, 10 - e);
        _Float16 hi = (_Float16)f, lo = (_Float16)(f - (float)hi);
        if (odd) {  // the formula's infinity or NaN comes from hi, which is 0 for 0 alone
          if (hi == (_Float16)0.f && h != 0.f) hi = (_Float16)copysignf(0x1p-14f, h);
          lo = (_Float16)(fabsf(f) < INFINITY ? f - (float)hi : 0.f);
        }
        v[i] = __builtin_bit_cast(uint16_t, hi) | (uint32_t)__builtin_bit_cast(uint16_t, lo) << 16;
      }
      *at = v;
    }
    if (part == 0) s_factor[row] = ldexpf(p.scales[a], e - 10);
  }
  __syncthreads();
  if (idle) return;
  // This lane's 8 ranks of a block, and which parts: all high ones, or with BLOCK 16
  // the low ones for the upper half of the lanes.
  const int at = BLOCK == 16 ? (g & 1) * 8 : g * 8;
  const uint32_t high = 0x05040100u, low = 0x07060302u;
  const uint32_t select = BLOCK == 16 && g >= 2 ? low : high;
  const __half* B = s.B + (int64_t)max(a, 0) * s.rows * s.rank + at;
  __half* y = static_cast<__half*>(s.y);
  // a wave's own LDS accesses stay in order
  auto settle = [] {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  };
  for (int o0 = o_begin; o0 < o_end; o0 += kUpStep) {
    if (a >= 0) {
      floatx4 acc[2][kOut / 16];
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int u = 0; u < kOut / 16; ++u) acc[r][u] = floatx4{0.f, 0.f, 0.f, 0.f};
      for (int j = 0; j < ranks; j += BLOCK) {
        v4u bv[kOut / 16];
#pragma unroll
        for (int u = 0; u < kOut / 16; ++u) {
          const int o = min(o0 + half * kOut + 16 * u + m, s.rows - 1);
          bv[u] = v4u{0, 0, 0, 0};
          if (j + at < s.rank)
            bv[u] = *reinterpret_cast<const v4u*>(B + (int64_t)o * s.rank + j);
        }
        // B for the low parts is finite: an infinity, which the high part shows, times a
        // low part that is zero or of the other sign would be NaN
        v4u bl[kOut / 16];
#pragma unroll
        for (int u = 0; u < kOut / 16; ++u) {
          bl[u] = limit(bv[u]);
          if constexpr (BLOCK == 16) bv[u] = select == low ? bl[u] : bv[u];
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t* pair = &s_pair[(16 * r + m) * stride + j + at];
          const v4u p0 = *reinterpret_cast<const v4u*>(pair);
          const v4u p1 = *reinterpret_cast<const v4u*>(pair + 4);
          const v4u hv = parts(p0, p1, select);
#pragma unroll
          for (int u = 0; u < kOut / 16; ++u) acc[r][u] = mfma(bv[u], hv, acc[r][u]);
          if constexpr (BLOCK == 32) {
            const v4u lv = parts(p0, p1, low);
#pragma unroll
            for (int u = 0; u < kOut / 16; ++u) acc[r][u] = mfma(bl[u], lv, acc[r][u]);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float f = s_factor[16 * r + m];
#pragma unroll
        for (int u = 0; u < kOut / 16; ++u)
          *reinterpret_cast<floatx4*>(&s_sum[16 * r + m][16 * u + 4 * g]) = f * acc[r][u];
      }
    }
    settle();
    v4u out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      out[i] = bases[i];
      if (a < 0) continue;
      const float* sum = &s_sum[8 * i + (lane >> 3)][(lane & 7) * 8];
      const floatx4 lo = *reinterpret_cast<const floatx4*>(sum);
      const floatx4 hi = *reinterpret_cast<const floatx4*>(sum + 4);
      const __half* b = reinterpret_cast<const __half*>(&bases[i]);
      __half* q = reinterpret_cast<__half*>(&out[i]);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        q[k] = __float2half_rn(__half2float(b[k]) + (k < 4 ? lo[k & 3] : hi[k & 3]));
    }
    settle();
    if (o0 + kUpStep < o_end) request(o0 + kUpStep);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (o0 + o_lane < s.rows && rows[i] >= 0)
        *reinterpret_cast<v4u*>(y + (int64_t)rows[i] * s.rows + o0 + o_lane) = out[i];
  }
}

// ---- host ----

bool aligned16(const void* p) { return (uintptr_t)p % 16 == 0; }

// 16-byte loads of x, A and B fit.
bool wide_site(const seedlm_lora_site& s) {
  return s.cols % 8 == 0 && s.rank % 8 == 0 && aligned16(s.x) && aligned16(s.A) && aligned16(s.B);
}

// How the sites [0, n) of one group run.
enum Kind { kOne, kRows, kTiles };

// Tiles need rows enough to fill them and products enough to repay the sort and the
// set-up.  GPU time of a call, tiles against rows, all rows of one adapter (and rows
// alternating among 16): q, k and v of a 70B layer at rank 16, 96 rows (107 MB) 13.4
// (21) and 16 us, 128 rows 13.6 (21) and 21; gate and up of an 8B layer at rank 64, 64
// rows (302 MB) 18 (47) and 36 (46), 128 rows 21 (47) and 69 (88); 4096 x 11008 at rank
// 32, 96 rows (93 MB) 15.4 (20) and 13.
constexpr int64_t kTileTokens = 64;
constexpr int64_t kTileBytes = 128 << 20;  // A and B, once per row
// One launch pays while A is small for a workgroup to read whole and the workgroups
// are at most the compute units (every one reads A).  Time of a call, one launch against
// two, by A's bytes at rank 16 and 4096 rows, fp16 (fp32): 8192 columns, 256 KiB, 6.4 us
// at 1 row; 14336, 448 KiB, 7.4 and 9.2 at 1 row (7.5 and 10.4), 9.0 and 10.6 at 16 (9.0
// and 12.9), 10.3 and 13.7 at 64; 16384, 512 KiB, 7.9 and 9.2 at 1 (8.1 and 10.5), 9.6
// and 9.7 at 4, 9.2 and 11.2 at 16, 11.3 and 14.4 at 64; 20480, 640 KiB, 8.9 and 9.4 at
// 1, 11.7 and 10.5 at 4 (11.7 and 11.7); 24576 9.6 and 9.5 at 1, 12.5 and 11.0 at 4;
// 8192 x 28672 12.7 and 10.0 at 1.  By the workgroups: gate and up of an 8B layer 7.7 and
// 9.9 at 32 rows (256 workgroups), 13.8 and 13.5 at 64.
constexpr int64_t kOneBytes = 512 << 10;  // of one adapter's A

// Outputs of a workgroup of lora_one_kernel: a row per thread, or up to four where
// there are more workgroups than compute units; *workgroups gets their number.
int one_outputs(const seedlm_lora_site* s, int n, int64_t tokens, int64_t* workgroups) {
  for (int per = kOneThreads;; per *= 2) {
    *workgroups = 0;
    for (int i = 0; i < n; ++i) *workgroups += (s[i].rows + per - 1) / per * tokens;
    if (*workgroups <= device_cu_count() || per == 4 * kOneThreads) return per;
  }
}

Kind kind_of(const seedlm_lora_site* s, int n, int64_t tokens, int adapters, int xdt, int ydt) {
  int64_t bytes = 0, workgroups = 0;
  bool one = true, tile = tokens >= kTileTokens && xdt == SEEDLM_F16 && ydt == SEEDLM_F16 &&
                          adapters <= kSortAdapters;
  for (int i = 0; i < n; ++i) {
    bytes += tokens * s[i].rank * (s[i].rows + s[i].cols) * 2;
    one = one && s[i].rank <= kOneRank && s[i].rank * s[i].cols * 2 <= kOneBytes;
    tile = tile && wide_site(s[i]) && s[i].rows % 8 == 0 && aligned16(s[i].base) &&
           aligned16(s[i].y);
  }
  (void)one_outputs(s, n, tokens, &workgroups);
  if (one && workgroups <= device_cu_count()) return kOne;
  return tile && bytes >= kTileBytes ? kTiles : kRows;
}

// Column chunks of a site of an n-site group: kChunk columns each for the row
// kernels; for the tiles as few as give four workgroups per compute unit, of at
// least 512 columns, and not so many that an up workgroup reads more than 64 KiB of
// their sums (128 where few rows leave few such workgroups).
int chunk_cols_of(const seedlm_lora_site& s, int n, int64_t tokens, Kind kind) {
  if (kind != kTiles) return kChunk;
  const int64_t across = (tokens + kTileRows - 1) / kTileRows * n;
  int64_t chunks = (4 * device_cu_count() + across - 1) / across;
  const int64_t sums = tokens <= 2 * kUpRows ? 512 : 256;
  for (int64_t most : {(s.cols + 511) / 512, sums / s.rank})
    if (chunks > most) chunks = most > 0 ? most : 1;
  const int64_t cols = (s.cols + chunks - 1) / chunks;
  return (int)((cols + kDownStep - 1) / kDownStep * kDownStep);
}

size_t site_floats(const seedlm_lora_site& s, int chunk_cols, int64_t tokens) {
  const int64_t chunks = (s.cols + chunk_cols - 1) / chunk_cols;
  return (size_t)((chunks * tokens * s.rank + 63) / 64 * 64);
}

// Outputs of an up workgroup, which forms the rows' h first: so many steps that the
// workgroups run in one round of three per compute unit, at most 4; more, while that
// leaves one per compute unit, where the chunks' sums are more than a step's base and
// y (32 KiB).
int up_outputs_of(const seedlm_lora_site& s, int n, int64_t tokens, int chunks) {
  const int64_t all = (tokens + kUpRows - 1) / kUpRows * ((s.rows + kUpStep - 1) / kUpStep) * n;
  const int64_t cus = device_cu_count(), round = (all + 3 * cus - 1) / (3 * cus);
  int64_t each = round > 4 ? 4 : round;
  const int64_t sums = ((int64_t)s.rank * chunks + 127) / 128, most = all / cus;
  if (each < sums) each = sums < most ? sums : most;
  return (int)(each < 1 ? 1 : each) * kUpStep;
}

// Tiles at most: each adapter, and the rows without one, may leave one part-filled.
int64_t tiles_most(int64_t tokens, int adapters) {
  const int64_t buckets = (int64_t)adapters + 1, some = tokens < buckets ? tokens : buckets;
  return (tokens + kTileRows - 1) / kTileRows + some;
}
// Scratch of the tiles: their number, adapters and rows, and the rows' places.
int64_t tile_floats(int64_t tokens, int adapters) {
  return (64 + tiles_most(tokens, adapters) * (1 + kTileRows) + tokens + 63) / 64 * 64;
}

int group_size(int n, int i) { return n - i < kLoraGroup ? n - i : kLoraGroup; }

template <typename XT, typename YT>
void run_one(const LoraArgs& p, int blocks, hipStream_t s) {
  const int rows = p.tokens >= 8 ? (p.tokens + 7) / 8 * 8 : p.tokens;
  hipLaunchKernelGGL((lora_one_kernel<XT, YT>), dim3(rows * blocks), dim3(kOneThreads), 0, s, p,
                     blocks);
}

template <typename XT, typename YT>
void run_rows(const LoraArgs& p, int down, int up, hipStream_t s) {
  const int rows = p.tokens < 65535 ? p.tokens : 65535;
  hipLaunchKernelGGL(lora_down_rows_kernel<XT>, dim3(down, rows), dim3(kThreads), 0, s, p);
  hipLaunchKernelGGL(lora_up_rows_kernel<YT>, dim3(up, rows), dim3(kThreads), 0, s, p);
}

}  // namespace

// The groups run one after another and share the scratch of the largest.
size_t lora_scratch_bytes(const seedlm_lora_site* sites, int n, int64_t tokens, int adapters,
                          int xdt, int ydt) {
  size_t most = 0;
  for (int i = 0; i < n; i += kLoraGroup) {
    const int k = group_size(n, i);
    const Kind kind = kind_of(sites + i, k, tokens, adapters, xdt, ydt);
    size_t floats = kind == kTiles ? tile_floats(tokens, adapters) : 0;
    for (int j = i; j < i + k && kind != kOne; ++j)
      floats += site_floats(sites[j], chunk_cols_of(sites[j], k, tokens, kind), tokens);
    if (floats > most) most = floats;
  }
  return most * sizeof(float);
}

int launch_lora(const seedlm_lora_site* sites, int n, const int32_t* adapter, const float* scales,
                int64_t tokens, int adapters, int xdt, int ydt, float* scratch, hipStream_t s) {
  for (int i = 0; i < n; i += kLoraGroup) {
    LoraArgs p{};
    p.n = group_size(n, i);
    p.adapter = adapter;
    p.scales = scales;
    p.tokens = (int)tokens;
    p.adapters = adapters;
    const Kind kind = kind_of(sites + i, p.n, tokens, adapters, xdt, ydt);
    const bool tile = kind == kTiles;
    const int64_t tiles = tiles_most(tokens, adapters);
    float* h = scratch;
    if (tile) {
      p.tile_count = reinterpret_cast<int32_t*>(scratch);
      p.tiles = p.tile_count + 64;
      p.order = p.tiles + tiles;
      p.place = p.order + tiles * kTileRows;
      h += tile_floats(tokens, adapters);
    }
    int top_rank = 0;
    for (int k = 0; k < p.n; ++k)
      if (sites[i + k].rank > top_rank) top_rank = sites[i + k].rank;
    const int rank_tiles = top_rank <= 16 ? 1 : (top_rank <= 32 ? 2 : kDownRanks / 16);
    const int down_ranks = tile ? rank_tiles * 16 : 16;
    int64_t workgroups = 0;
    const int outputs = one_outputs(sites + i, p.n, tokens, &workgroups);
    int down = 0, up = 0;
    for (int k = 0; k < p.n; ++k) {
      const seedlm_lora_site& in = sites[i + k];
      Site& o = p.s[k];
      o.x = in.x;
      o.A = static_cast<const __half*>(in.A);
      o.B = static_cast<const __half*>(in.B);
      o.base = in.base;
      o.y = in.y;
      o.h = h;
      o.rows = (int)in.rows;
      o.cols = (int)in.cols;
      o.rank = in.rank;
      o.chunk_cols = chunk_cols_of(in, p.n, tokens, kind);
      o.chunks = (o.cols + o.chunk_cols - 1) / o.chunk_cols;
      o.up_outputs = kind == kOne ? outputs
                     : tile       ? up_outputs_of(in, p.n, tokens, o.chunks)
                                  : kThreads;
      o.wide = wide_site(in);
      o.first_down = down;
      o.first_up = up;
      down += o.chunks * ((o.rank + down_ranks - 1) / down_ranks);
      up += (o.rows + o.up_outputs - 1) / o.up_outputs;
      if (kind != kOne) h += site_floats(in, o.chunk_cols, tokens);
    }
    if (kind == kOne) {
      if (xdt == SEEDLM_F16) {
        if (ydt == SEEDLM_F16) run_one<__half, __half>(p, up, s);
        else run_one<__half, float>(p, up, s);
      } else {
        if (ydt == SEEDLM_F16) run_one<float, __half>(p, up, s);
        else run_one<float, float>(p, up, s);
      }
    } else if (tile) {
      const int buckets = adapters + 1;
      hipLaunchKernelGGL(lora_sort_kernel, dim3(1), dim3(kSortThreads),
                         2 * buckets * sizeof(int), s, p);
      const dim3 dg(down, tiles), ug(up, (tiles + kUpRows / kTileRows - 1) / (kUpRows / kTileRows));
      const auto down_kernel = rank_tiles == 1   ? lora_down_tile_kernel<1>
                               : rank_tiles == 2 ? lora_down_tile_kernel<2>
                                                 : lora_down_tile_kernel<kDownRanks / 16>;
      hipLaunchKernelGGL(down_kernel, dg, dim3(kThreads), 0, s, p);
      const int block = top_rank <= 16 ? 16 : 32;
      const size_t lds = (size_t)kUpRows * ((top_rank + block - 1) / block * block + 4) * 4;
      const auto up_kernel = block == 16 ? lora_up_tile_kernel<16> : lora_up_tile_kernel<32>;
      hipLaunchKernelGGL(up_kernel, ug, dim3(kThreads), lds, s, p);
    } else if (xdt == SEEDLM_F16) {
      if (ydt == SEEDLM_F16) run_rows<__half, __half>(p, down, up, s);
      else run_rows<__half, float>(p, down, up, s);
    } else {
      if (ydt == SEEDLM_F16) run_rows<float, __half>(p, down, up, s);
      else run_rows<float, float>(p, down, up, s);
    }
    if (hipGetLastError() != hipSuccess) return SEEDLM_E_DEVICE;
  }
  return SEEDLM_OK;
}

}  // namespace seedlm
