// Low-rank adapters of many requests beside shared projections
// (seedlm_lora_many): y[t] = base[t] + scales[a] B_a (A_a x[t]), a = adapter[t],
// for up to 8 sites (projections) in one pair of launches.
//
// First launch ("down"): h = A x, cut along the columns into chunks so that few
// rows still fill the chip; chunk sums go to scratch as fp32
// [site][chunk][token][rank].  Second launch ("up"): adds the chunks in order,
// multiplies with B, scales, adds base and rounds once.
//
// Few rows (any types): a workgroup per row and chunk, lanes along the columns;
// then a thread per output element.  The bytes of A and B bound it, once per row.
//
// Many rows (fp16): v_mfma_f32_16x16x32_f16, with A (then B) as the first operand
// and 16 rows as the second, so that a lane's results belong to one row:
//   down  32 rows and up to 64 ranks per workgroup, its waves splitting a chunk
//         of columns, added through LDS
//   up    64 rows (a row per lane of the bookkeeping) and 64 outputs per wave; B
//         is loaded once per adapter for all 64.  Operand row i of MFMA u is
//         output 32 (u/2) + 8 (i/4) + 4 (u%2) + i%4, so that a lane's results of
//         two MFMAs are 8 neighbouring outputs: 16-byte loads of base and stores
//         of y.  h enters as two fp16 numbers, h 2^-e = hi + lo (22 bits; e from
//         the row's largest |h|), the 16 high and 16 low parts of 16 ranks filling
//         the 32 products of one MFMA against the same 16 elements of B twice.
// A tile whose rows have several adapters takes them one after another and keeps
// each result for its own rows only, so no adapter's values reach another's rows.
// The bytes of x, base and y bound these.
#include <hip/hip_fp16.h>

#include "seedlm_internal.h"

namespace seedlm {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kChunk = 1024;     // columns of a workgroup of the row kernels
constexpr int kDownRows = 32;    // rows, and ranks at most, of a down tile
constexpr int kDownRanks = 64;
constexpr int kUpRows = 64;      // rows and outputs of an up step
constexpr int kUpOutputs = 64 * kWaves;

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

struct Site {
  const void* x;
  const __half* A;
  const __half* B;
  const void* base;
  void* y;
  float* h;       // [chunks][tokens][rank]
  int rows, cols, rank;
  int chunks;
  int chunk_cols; // columns of a chunk
  int up_outputs; // outputs of an up workgroup of the tile kernels
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

// ---- many rows: the matrix cores ----

__device__ floatx4 mfma(v4u a, v4u b, floatx4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a),
                                                __builtin_bit_cast(half8, b), c, 0, 0, 0);
}

// The adapter of row t0 + lane (lane < n), -1 for none.
__device__ int adapter_of_lane(const LoraArgs& p, int t0, int n, int lane) {
  const int t = t0 + lane;
  const int a = lane < n && t < p.tokens ? p.adapter[t] : -1;
  return a < p.adapters ? a : -1;
}

// h of kDownRows rows, RT * 16 ranks and one chunk.  Lane l supplies 8 columns
// (8 (l/16) of each 32) of rank l%16 and of rows l%16 and 16 + l%16.
template <int RT>
__global__ __launch_bounds__(kThreads) void lora_down_tile_kernel(const LoraArgs p) {
  __shared__ __align__(16) float s_h[kWaves][kDownRows][RT * 16 + 4];
  const Site& s = site_of(p, false, blockIdx.x);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int m = lane & 15, g = lane >> 4;
  constexpr int kDownSteps = 4;  // of 32 columns, requested together
  const int t0 = blockIdx.y * kDownRows;
  const int rank_blocks = (s.rank + RT * 16 - 1) / (RT * 16);
  const int chunk = (blockIdx.x - s.first_down) / rank_blocks;
  const int j0 = (blockIdx.x - s.first_down) % rank_blocks * (RT * 16);
  // this wave's columns
  const int quarter = s.chunk_cols / kWaves;
  const int c0 = chunk * s.chunk_cols + wave * quarter;
  const int c1 = min(s.cols, c0 + quarter);
  const int id = adapter_of_lane(p, t0, kDownRows, lane);
  const __half* x[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    x[h] = static_cast<const __half*>(s.x) + (int64_t)min(t0 + h * 16 + m, p.tokens - 1) * s.cols;
  uint64_t todo = __ballot(id >= 0);
  const uint64_t any = todo;
  while (todo) {
    const int a = __builtin_amdgcn_readlane(id, (int)__ffsll((unsigned long long)todo) - 1);
    const uint64_t own = __ballot(id == a);
    todo &= ~own;
    floatx4 acc[2][RT];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[h][r] = floatx4{0.f, 0.f, 0.f, 0.f};
    const __half* A[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
      A[r] = s.A + ((int64_t)a * s.rank + min(j0 + r * 16 + m, s.rank - 1)) * s.cols;
    for (int k = c0; k < c1; k += 32 * kDownSteps) {
      v4u xv[kDownSteps][2], av[kDownSteps][RT];
#pragma unroll
      for (int u = 0; u < kDownSteps; ++u) {
        const int c = k + 32 * u + 8 * g;
        const bool in = c < c1;
        const v4u z = {0, 0, 0, 0};
#pragma unroll
        for (int h = 0; h < 2; ++h) xv[u][h] = in ? *reinterpret_cast<const v4u*>(x[h] + c) : z;
#pragma unroll
        for (int r = 0; r < RT; ++r) av[u][r] = in ? *reinterpret_cast<const v4u*>(A[r] + c) : z;
      }
#pragma unroll
      for (int u = 0; u < kDownSteps; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < RT; ++r) acc[h][r] = mfma(av[u][r], xv[u][h], acc[h][r]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if ((own >> (h * 16 + m)) & 1) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
          *reinterpret_cast<floatx4*>(&s_h[wave][h * 16 + m][r * 16 + g * 4]) = acc[h][r];
      }
  }
  __syncthreads();
  const int ranks = min(RT * 16, s.rank - j0);  // a multiple of 8
  for (int e = threadIdx.x; e < kDownRows * RT * 4; e += kThreads) {
    const int t = e / (RT * 4), j = e % (RT * 4) * 4;
    if (!((any >> t) & 1) || j >= ranks) continue;
    floatx4 sum = *reinterpret_cast<const floatx4*>(&s_h[0][t][j]);
#pragma unroll
    for (int w = 1; w < kWaves; ++w) sum += *reinterpret_cast<const floatx4*>(&s_h[w][t][j]);
    *reinterpret_cast<floatx4*>(s.h + ((int64_t)chunk * p.tokens + t0 + t) * s.rank + j0 + j) = sum;
  }
}

// y of kUpRows rows and s.up_outputs outputs.
__global__ __launch_bounds__(kThreads, 2) void lora_up_tile_kernel(const LoraArgs p) {
  // h of the rows, each value as hi | lo << 16, ranks padded with zeros to
  // sixteens; and the factor scales[a] * 2^e of each row
  extern __shared__ __align__(16) uint32_t s_pair[];
  __shared__ float s_factor[kUpRows];
  const Site& s = site_of(p, true, blockIdx.x);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int m = lane & 15, g = lane >> 4;
  const int t0 = blockIdx.y * kUpRows;
  const int ranks = (s.rank + 15) / 16 * 16, stride = ranks + 4;
  const int id = adapter_of_lane(p, t0, kUpRows, lane);
  {
    // four threads a row, four ranks at a time
    const int t = threadIdx.x >> 2, part = threadIdx.x & 3;
    const int a = __shfl(id, t);
    float top = 0.f;
    if (a >= 0) {
      for (int j = part * 4; j < ranks; j += 16) {
        floatx4 sum = {0.f, 0.f, 0.f, 0.f};
        if (j < s.rank)
          for (int c = 0; c < s.chunks; ++c)
            sum += *reinterpret_cast<const floatx4*>(
                s.h + ((int64_t)c * p.tokens + t0 + t) * s.rank + j);
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, fabsf(sum[i]));
        *reinterpret_cast<floatx4*>(&s_pair[t * stride + j]) = sum;
      }
    }
    top = fmaxf(top, __shfl_xor(top, 1));
    top = fmaxf(top, __shfl_xor(top, 2));
    // the row's largest value into [2^9, 2^10): the low parts keep all bits
    int e = 10;
    if (top > 0.f && top < INFINITY) (void)frexpf(top, &e);
    if (a >= 0) {
      for (int j = part * 4; j < ranks; j += 16) {
        v4u* at = reinterpret_cast<v4u*>(&s_pair[t * stride + j]);
        v4u v = *at;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float f = ldexpf(__uint_as_float(v[i]), 10 - e);
          const _Float16 hi = (_Float16)f, lo = (_Float16)(f - (float)hi);
          v[i] = __builtin_bit_cast(uint16_t, hi) |
                 (uint32_t)__builtin_bit_cast(uint16_t, lo) << 16;
        }
        *at = v;
      }
      if (part == 0) s_factor[t] = ldexpf(p.scales[a], e - 10);
    }
  }
  __syncthreads();
  const bool copies = s.y != s.base;
  const uint32_t select = g < 2 ? 0x05040100u : 0x07060302u;  // high or low parts
  const int o_end = min(s.rows, (int)(blockIdx.x - s.first_up + 1) * s.up_outputs);
  for (int o0 = (blockIdx.x - s.first_up) * s.up_outputs + wave * 64; o0 < o_end; o0 += kUpOutputs) {
    // base of rows 16 k + m, outputs o0 + 32 v + 8 g + (0..7)
    v4u base[4][2];
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const int t = min(t0 + 16 * k + m, p.tokens - 1), o = min(o0 + 32 * v + 8 * g, s.rows - 8);
        base[k][v] = *reinterpret_cast<const v4u*>(static_cast<const __half*>(s.base) +
                                                   (int64_t)t * s.rows + o);
      }
    __half* y = static_cast<__half*>(s.y);
    uint64_t todo = __ballot(id >= 0);
    if (copies) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int t = t0 + 16 * k + m;
        if (t >= p.tokens || (todo >> (16 * k + m)) & 1) continue;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const int o = o0 + 32 * v + 8 * g;
          if (o < s.rows) *reinterpret_cast<v4u*>(y + (int64_t)t * s.rows + o) = base[k][v];
        }
      }
    }
    while (todo) {
      const int a = __builtin_amdgcn_readlane(id, (int)__ffsll((unsigned long long)todo) - 1);
      const uint64_t own = __ballot(id == a);
      todo &= ~own;
      const __half* B[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int o = o0 + 32 * (u >> 1) + 8 * (m >> 2) + 4 * (u & 1) + (m & 3);
        B[u] = s.B + ((int64_t)a * s.rows + min(o, s.rows - 1)) * s.rank + (g & 1) * 8;
      }
      floatx4 acc[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int u = 0; u < 4; ++u) acc[k][u] = floatx4{0.f, 0.f, 0.f, 0.f};
      for (int j = 0; j < ranks; j += 16) {
        v4u bv[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          bv[u] = v4u{0, 0, 0, 0};
          if (j + (g & 1) * 8 < s.rank) bv[u] = *reinterpret_cast<const v4u*>(B[u] + j);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (((own >> (16 * k)) & 0xFFFF) == 0) continue;
          const uint32_t* pair = &s_pair[(16 * k + m) * stride + j + (g & 1) * 8];
          const v4u p0 = *reinterpret_cast<const v4u*>(pair);
          const v4u p1 = *reinterpret_cast<const v4u*>(pair + 4);
          const v4u hv = {__builtin_amdgcn_perm(p0[1], p0[0], select),
                          __builtin_amdgcn_perm(p0[3], p0[2], select),
                          __builtin_amdgcn_perm(p1[1], p1[0], select),
                          __builtin_amdgcn_perm(p1[3], p1[2], select)};
#pragma unroll
          for (int u = 0; u < 4; ++u) acc[k][u] = mfma(bv[u], hv, acc[k][u]);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (!((own >> (16 * k + m)) & 1)) continue;
        const float f = s_factor[16 * k + m];
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const int o = o0 + 32 * v + 8 * g;
          if (o >= s.rows) continue;
          const __half* b = reinterpret_cast<const __half*>(&base[k][v]);
          v4u out;
          __half* q = reinterpret_cast<__half*>(&out);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            q[i] = __float2half_rn(fmaf(f, acc[k][2 * v + (i >> 2)][i & 3], __half2float(b[i])));
          *reinterpret_cast<v4u*>(y + (int64_t)(t0 + 16 * k + m) * s.rows + o) = out;
        }
      }
    }
  }
}

// ---- host ----

bool aligned16(const void* p) { return (uintptr_t)p % 16 == 0; }

// 16-byte loads of x, A and B fit.
bool wide_site(const seedlm_lora_site& s) {
  return s.cols % 8 == 0 && s.rank % 8 == 0 && aligned16(s.x) && aligned16(s.A) && aligned16(s.B);
}

// Rows from which a call runs on the matrix cores.
constexpr int64_t kTileTokens = 33;

// Whether the sites [0, n) of one pair of launches run on the matrix cores.
bool tiles(const seedlm_lora_site* s, int n, int64_t tokens, int xdt, int ydt) {
  if (tokens < kTileTokens || xdt != SEEDLM_F16 || ydt != SEEDLM_F16) return false;
  for (int i = 0; i < n; ++i)
    if (!wide_site(s[i]) || s[i].rows % 8 != 0 || !aligned16(s[i].base) || !aligned16(s[i].y))
      return false;
  return true;
}

// Column chunks of a site of an n-site group: 1024 columns each for the row
// kernels; for the tiles as few as give two workgroups per compute unit, of at
// least 512 columns.
int chunk_cols_of(const seedlm_lora_site& s, int n, int64_t tokens, bool tile) {
  if (!tile) return kChunk;
  const int64_t across = (tokens + kDownRows - 1) / kDownRows * n;
  int64_t chunks = (2 * device_cu_count() + across - 1) / across;
  const int64_t most = (s.cols + 511) / 512;
  if (chunks > most) chunks = most;
  const int64_t cols = (s.cols + chunks - 1) / chunks;
  return (int)((cols + 127) / 128 * 128);
}

size_t site_floats(const seedlm_lora_site& s, int chunk_cols, int64_t tokens) {
  const int64_t chunks = (s.cols + chunk_cols - 1) / chunk_cols;
  return (size_t)((chunks * tokens * s.rank + 63) / 64 * 64);
}

int group_size(int n, int i) { return n - i < kLoraGroup ? n - i : kLoraGroup; }

template <typename XT, typename YT>
void run_rows(const LoraArgs& p, int down, int up, hipStream_t s) {
  const int rows = p.tokens < 65535 ? p.tokens : 65535;
  hipLaunchKernelGGL(lora_down_rows_kernel<XT>, dim3(down, rows), dim3(kThreads), 0, s, p);
  hipLaunchKernelGGL(lora_up_rows_kernel<YT>, dim3(up, rows), dim3(kThreads), 0, s, p);
}

}  // namespace

// The groups run one after another and share the scratch of the largest.
size_t lora_scratch_bytes(const seedlm_lora_site* sites, int n, int64_t tokens, int xdt, int ydt) {
  size_t most = 0;
  for (int i = 0; i < n; i += kLoraGroup) {
    const int k = group_size(n, i);
    const bool tile = tiles(sites + i, k, tokens, xdt, ydt);
    size_t floats = 0;
    for (int j = i; j < i + k; ++j)
      floats += site_floats(sites[j], chunk_cols_of(sites[j], k, tokens, tile), tokens);
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
    const bool tile = tiles(sites + i, p.n, tokens, xdt, ydt);
    float* h = scratch;
    int top_rank = 0;
    for (int k = 0; k < p.n; ++k)
      if (sites[i + k].rank > top_rank) top_rank = sites[i + k].rank;
    const int rank_tiles = top_rank <= 16 ? 1 : (top_rank <= 32 ? 2 : kDownRanks / 16);
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
      o.chunk_cols = chunk_cols_of(in, p.n, tokens, tile);
      o.chunks = (o.cols + o.chunk_cols - 1) / o.chunk_cols;
      o.up_outputs = tile ? 2 * kUpOutputs : kThreads;
      o.wide = wide_site(in);
      o.first_down = down;
      o.first_up = up;
      down += o.chunks * (tile ? (o.rank + rank_tiles * 16 - 1) / (rank_tiles * 16) : 1);
      up += (o.rows + o.up_outputs - 1) / o.up_outputs;
      h += site_floats(in, o.chunk_cols, tokens);
    }
    if (tile) {
      const dim3 dg(down, (p.tokens + kDownRows - 1) / kDownRows);
      const dim3 ug(up, (p.tokens + kUpRows - 1) / kUpRows);
      if (rank_tiles == 1) hipLaunchKernelGGL(lora_down_tile_kernel<1>, dg, dim3(kThreads), 0, s, p);
      else if (rank_tiles == 2) hipLaunchKernelGGL(lora_down_tile_kernel<2>, dg, dim3(kThreads), 0, s, p);
      else hipLaunchKernelGGL(lora_down_tile_kernel<4>, dg, dim3(kThreads), 0, s, p);
      const size_t lds = (size_t)kUpRows * ((top_rank + 15) / 16 * 16 + 4) * sizeof(uint32_t);
      hipLaunchKernelGGL(lora_up_tile_kernel, ug, dim3(kThreads), lds, s, p);
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
