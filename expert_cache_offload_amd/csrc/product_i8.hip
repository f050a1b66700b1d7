// Product of 8-bit integers with a scale per row of the left operand and per channel (row) of the
// weight: c[m][n] = (sum_k a[m][k] w[n][k]) * a_scale[m] * w_scale[n], for one weight or, over rows
// sorted by expert, one weight per group of rows.  The sum is exact in 32-bit integers (K < 2^17,
// so |sum| < 2^31); it is converted to fp32 once, scaled in fp32 and rounded once more to a
// 16-bit output.  SwiGLU epilogue: channels 2i and 2i + 1 are gate and up of output i (the order
// of an expert blob's gate/up rows), out[m][i] = silu(c[m][2i]) * c[m][2i + 1].
//
// The weight's rows are the rows of the matrix instruction and the activations its columns, so a
// lane of the 32 x 32 result holds one output row and, with the weight's rows dealt to the
// instruction's in the order below, 16 neighbouring channels of it: gate and up meet in a lane
// and the output is stored in 16-byte pieces.
#include <algorithm>

#include "row_ops.h"

namespace moe {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

constexpr int kMaxK = 131071;  // 128 * 128 * K stays below 2^31
constexpr int kMaxGroups = 1024;
constexpr int kMaxN = 1 << 20;
constexpr int kMaxM = 1 << 24;

struct ProdArgs {
  const int8_t* a;
  int64_t as;
  const float* a_scale;
  int M, K;
  const int8_t* w;
  int64_t ws;
  const float* w_scale;
  int N, groups;
  const int* offsets;  // null: one group of M rows
  void* out;
  int64_t os;
};

// exp(-z) to fp32 accuracy: exp2 of the rounded exponent times the first-order term of what the
// rounding left (|rest| < 2^-17, so its square is below 2^-34).
__device__ __forceinline__ float exp_neg(float z) {
  constexpr float kL = 1.44269504088896341f, kLlo = 1.92596299e-8f;  // log2(e) in two parts
  const float t = -z * kL;
  const float rest = fmaf(-z, kL, -t) - z * kLlo;
  const float e = __builtin_amdgcn_exp2f(t);
  // |t| beyond exp2's range: e is 0 or infinity already, and the term must not make it a NaN
  return fabsf(t) < 126.f ? fmaf(e, rest * 0.693147181f, e) : e;
}
__device__ __forceinline__ float silu_f32(float z) {
  return z * __builtin_amdgcn_rcpf(1.0f + exp_neg(z));
}

// Channel (row of a 32-row weight tile) that row r of the matrix instruction holds: a lane's 16
// results, rows 8 (i / 4) + 4 (lane / 32) + i % 4, are then channels 16 (lane / 32) + i.
__device__ __forceinline__ int channel_of_row(int r) {
  return 16 * ((r >> 2) & 1) + 4 * (r >> 3) + (r & 3);
}

__device__ __forceinline__ int row_of_channel(int n) {
  return 8 * ((n >> 2) & 3) + 4 * ((n >> 4) & 1) + (n & 3);
}

// Row range of group g.
__device__ __forceinline__ int2 group_rows(const ProdArgs& a, int g) {
  if (!a.offsets) return make_int2(0, a.M);
  const int lo = min(max(a.offsets[g], 0), a.M);
  return make_int2(lo, min(max(a.offsets[g + 1], lo), a.M));
}

// s_mt[g] = first row tile (of BM rows) of group g, s_mt[groups] = their number.
template <int BM>
__device__ void tile_prefix(const ProdArgs& a, int* s_mt, int* s_wave, int tid, int nthr) {
  const int per = (a.groups + nthr - 1) / nthr;
  int sum = 0;
  for (int i = 0; i < per; ++i) {
    const int g = tid * per + i;
    if (g < a.groups) {
      const int2 r = group_rows(a, g);
      sum += (r.y - r.x + BM - 1) / BM;
    }
  }
  int inc = sum;
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const int o = __shfl_up(inc, s);
    if ((tid & 63) >= s) inc += o;
  }
  if ((tid & 63) == 63) s_wave[tid >> 6] = inc;
  __syncthreads();
  int first = inc - sum;
  for (int w = 0; w < (tid >> 6); ++w) first += s_wave[w];
  for (int i = 0; i < per; ++i) {
    const int g = tid * per + i;
    if (g < a.groups) {
      s_mt[g] = first;
      const int2 r = group_rows(a, g);
      first += (r.y - r.x + BM - 1) / BM;
      if (g == a.groups - 1) s_mt[a.groups] = first;
    }
  }
  __syncthreads();
}

__device__ __forceinline__ int find_group(const int* s_mt, int groups, int mt) {
  int lo = 0, hi = groups - 1;  // last g with s_mt[g] <= mt
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s_mt[mid] <= mt) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Stores a lane's 16 channels n .. n + 15 of output row m (sums acc, scaled by sa and the
// group's channel scales).
template <class E, bool SWIGLU>
__device__ __forceinline__ void store_channels(const ProdArgs& a, int64_t m, int n,
                                               const float* w_scale, float sa,
                                               const i32x16& acc) {
  constexpr int V = Chunk<E>::V;
  const int have = a.N - n;
  if (have <= 0) return;
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = (float)acc[i] * sa * w_scale[n + min(i, have - 1)];
  if constexpr (SWIGLU) {
    E* out = (E*)a.out + m * a.os + n / 2;
#pragma unroll
    for (int c = 0; c < 8; c += V) {
      Chunk<E> o;
#pragma unroll
      for (int i = 0; i < V; ++i)
        o.e[i] = from_f32<E>(silu_f32(v[2 * (c + i)]) * v[2 * (c + i) + 1]);
      if (have / 2 > c) store_chunk(out + c, have / 2 - c, o);
    }
  } else {
    E* out = (E*)a.out + m * a.os + n;
#pragma unroll
    for (int c = 0; c < 16; c += V) {
      Chunk<E> o;
#pragma unroll
      for (int i = 0; i < V; ++i) o.e[i] = from_f32<E>(v[c + i]);
      if (have > c) store_chunk(out + c, have - c, o);
    }
  }
}

// ------------------------------------------------------------------ general tile
// 128 rows x 128 channels, four waves of 64 x 64, stages of 64 contraction elements through
// registers into LDS: any stride, alignment and length.  Rows past a group's end load its last
// row, channels past N the last channel; bytes past K are zero.
constexpr int GT = 256, GM = 128, GN = 128, GK = 64;

__device__ __forceinline__ int g_swz(int row, int chunk) {  // byte of (row, 16-byte chunk)
  return row * GK + ((chunk ^ ((row >> 2) & 3)) << 4);
}

template <class E, bool SWIGLU>
__global__ __launch_bounds__(GT) void product_any_kernel(ProdArgs a) {
  __shared__ __align__(16) int8_t s_t[2][(GM + GN) * GK];  // channels, then rows
  __shared__ int s_mt[kMaxGroups + 1];
  __shared__ int s_wave[GT / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  tile_prefix<GM>(a, s_mt, s_wave, tid, GT);
  const int NT = (a.N + GN - 1) / GN;
  const int mt = blockIdx.x / NT, nt = blockIdx.x - mt * NT;
  if (mt >= s_mt[a.groups]) return;
  const int g = find_group(s_mt, a.groups, mt);
  const int2 rr = group_rows(a, g);
  const int m0 = rr.x + (mt - s_mt[g]) * GM, n0 = nt * GN;
  const int8_t* w = a.w + (int64_t)g * a.N * a.ws;
  // thread: chunk tid % 4 of rows tid / 4 + 64 i of the stage
  const int8_t* src[4];
  const int ck = (tid & 3) * 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = (tid >> 2) + 64 * i;
    if (r < GN)
      src[i] = w + (int64_t)min(n0 + r, a.N - 1) * a.ws + ck;
    else
      src[i] = a.a + (int64_t)min(m0 + r - GN, rr.y - 1) * a.as + ck;
  }
  Chunk<int8_t> st[4];
  auto load = [&](int k0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = a.K - k0 - ck;
      if (n >= 16) {
        st[i].q = *(const u32x4_any*)(src[i] + k0);
      } else {
        st[i].q = u32x4{0, 0, 0, 0};
        for (int b = 0; b < n; ++b) {  // the end of the row
          const uint32_t v = (uint32_t)(uint8_t)src[i][k0 + b] << (8 * (b & 3));
          const int d = b >> 2;
          st[i].q.x |= d == 0 ? v : 0;
          st[i].q.y |= d == 1 ? v : 0;
          st[i].q.z |= d == 2 ? v : 0;
          st[i].q.w |= d == 3 ? v : 0;
        }
      }
    }
  };
  auto put = [&](int buf) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *(u32x4*)(s_t[buf] + g_swz((tid >> 2) + 64 * i, tid & 3)) = st[i].q;
  };
  const int wn = (wave & 1) * 64, wm = (wave >> 1) * 64;
  i32x16 acc[2][2];  // [channel tile][row tile]
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0;
  const int stages = (a.K + GK - 1) / GK;
  load(0);
  put(0);
  __syncthreads();
  const int wrow = channel_of_row(lane & 31), arow = lane & 31, half = lane >> 5;
  for (int s = 0; s < stages; ++s) {
    if (s + 1 < stages) load((s + 1) * GK);
    const int8_t* t = s_t[s & 1];
#pragma unroll
    for (int kk = 0; kk < GK / 32; ++kk) {
      i32x4 fw[2], fa[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        fw[i] = *(const i32x4*)(t + g_swz(wn + 32 * i + wrow, 2 * kk + half));
        fa[i] = *(const i32x4*)(t + g_swz(GN + wm + 32 * i + arow, 2 * kk + half));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[i], fa[j], acc[i][j], 0, 0, 0);
    }
    if (s + 1 < stages) {
      put((s + 1) & 1);  // last read in stage s - 1, before the barrier that ended it
      __syncthreads();
    }
  }
  const float* w_scale = a.w_scale + (int64_t)g * a.N;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int m = m0 + wm + 32 * j + arow;
    if (m >= rr.y) continue;
    const float sa = a.a_scale[m];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      store_channels<E, SWIGLU>(a, m, n0 + wn + 32 * i + 16 * half, w_scale, sa, acc[i][j]);
  }
}

// ------------------------------------------------------------------ few rows
// Up to RT * 16 rows of one group times 16 channels per workgroup, the contraction split over its
// four waves and joined in LDS (integers: in any order the same).  Operands go straight from
// memory into the registers of a 16 x 16 x 64 matrix instruction; every weight byte is read once
// for the group's rows, and that stream is the bound.
constexpr int FT = 256, FN = 16, FU = 8;  // threads, channels, steps in flight

__device__ __forceinline__ i32x4 load_k(const int8_t* p, int n) {  // n bytes of the row are left
  if (n >= 16) return *(const i32x4*)&(*(const u32x4_any*)p);
  uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
  for (int b = 0; b < 15; ++b)
    if (b < n) v[b >> 2] |= (uint32_t)(uint8_t)p[b] << (8 * (b & 3));
  return i32x4{(int)v[0], (int)v[1], (int)v[2], (int)v[3]};
}

template <class E, bool SWIGLU, int RT>
__global__ __launch_bounds__(FT) void product_few_kernel(ProdArgs a) {
  __shared__ __align__(16) int s_acc[FT / 64][RT][16][FN];  // [wave][row tile][row][channel]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n0 = blockIdx.x * FN;
  int g = 0, m0 = blockIdx.y * (16 * RT), end = a.M;
  if (a.offsets) {
    // workgroup row y starts at row y of the batch if its group's row tiles do: the last group
    // that holds the row (each lane looks at one group of 64)
    m0 = blockIdx.y;
    g = -1;
    int lo = 0, hi = 0;
    for (int g0 = 0; g0 < a.groups; g0 += 64) {
      int2 r = make_int2(0, 0);
      if (g0 + lane < a.groups) r = group_rows(a, g0 + lane);
      const uint64_t in = __ballot(r.x <= m0 && m0 < r.y);
      if (in) {
        const int l = 63 - __clzll(in);
        g = g0 + l;
        lo = __shfl(r.x, l);
        hi = __shfl(r.y, l);
      }
    }
    if (g < 0 || (m0 - lo) % (16 * RT) != 0) return;
    end = hi;
  }
  const int rows = min(end - m0, 16 * RT);
  // lane: channel (or row) lane % 16, 16-byte piece lane / 16 of a 64-byte step
  const int r16 = lane & 15, piece = (lane >> 4) * 16;
  const int8_t* pw = a.w + ((int64_t)g * a.N + min(n0 + r16, a.N - 1)) * a.ws + piece;
  const int8_t* pa[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t)
    pa[t] = a.a + (int64_t)(m0 + min(16 * t + r16, rows - 1)) * a.as + piece;
  i32x4 acc[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) acc[t] = i32x4{0, 0, 0, 0};
  const int steps = (a.K + 63) / 64, per = (steps + FT / 64 - 1) / (FT / 64);
  const int s1 = min(steps, (wave + 1) * per);
  int s = wave * per;
  for (; s + FU <= s1 && (s + FU) * 64 <= a.K; s += FU) {
    i32x4 fw[FU], fa[FU][RT];
#pragma unroll
    for (int u = 0; u < FU; ++u) {
      fw[u] = load_k(pw + (s + u) * 64, 16);
#pragma unroll
      for (int t = 0; t < RT; ++t) fa[u][t] = load_k(pa[t] + (s + u) * 64, 16);
    }
#pragma unroll
    for (int u = 0; u < FU; ++u)
#pragma unroll
      for (int t = 0; t < RT; ++t)
        acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[u], fa[u][t], acc[t], 0, 0, 0);
  }
  for (; s < s1; ++s) {
    const int n = a.K - s * 64 - piece;
    const i32x4 fw = load_k(pw + s * 64, n);
#pragma unroll
    for (int t = 0; t < RT; ++t)
      acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw, load_k(pa[t] + s * 64, n), acc[t], 0, 0,
                                                    0);
  }
  // lane: row lane % 16 of the tile, channels 4 (lane / 16) + 0..3
#pragma unroll
  for (int t = 0; t < RT; ++t) *(i32x4*)&s_acc[wave][t][r16][piece / 4] = acc[t];
  __syncthreads();
  const float* w_scale = a.w_scale + (int64_t)g * a.N;
  constexpr int NO = SWIGLU ? FN / 2 : FN;  // outputs per row
  for (int o = tid; o < rows * NO; o += FT) {
    const int m = o / NO, c = o % NO;
    const float sa = a.a_scale[m0 + m];
    auto value = [&](int ch) {
      int v = 0;
#pragma unroll
      for (int w = 0; w < FT / 64; ++w) v += s_acc[w][m >> 4][m & 15][ch];
      return (float)v * sa * w_scale[n0 + ch];
    };
    E* out = (E*)a.out + (int64_t)(m0 + m) * a.os;
    if constexpr (SWIGLU) {
      if (n0 + 2 * c < a.N)
        out[n0 / 2 + c] = from_f32<E>(silu_f32(value(2 * c)) * value(2 * c + 1));
    } else {
      if (n0 + c < a.N) out[n0 + c] = from_f32<E>(value(c));
    }
  }
}

// ------------------------------------------------------------------ large tiles
// 64 MI rows x 64 NI channels, four waves in a 2 x 2 arrangement of 32 MI rows x 32 NI channels
// each.  Stages of 128 contraction bytes go from memory straight into LDS (16-byte
// global-to-LDS loads), double buffered: the loads of stage s + 2 are issued when every wave has
// read stage s.  Rows are 128 bytes unpadded; 16-byte chunk c of a row sits at chunk
// c ^ ((r / 2) % 8), r the row's place in its matrix instruction: the 16 lanes that LDS serves
// at once then read 16 distinct 16-byte bank slots.  Fragments of a 32-deep step are read while
// the previous step's matrix instructions run, also across a stage's end.
// The loads are asm so that the compiler does not hold LDS reads back for them; they return
// nothing to registers, and the waits for them are the stage's own.
// Needs 16-byte aligned operands and strides and K a multiple of 16.
constexpr int LT = 256, LK = 128;

__device__ __forceinline__ void load_to_lds(uint32_t lds, uint32_t off, const int8_t* base) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, %2"
      :
      : "s"(lds), "v"(off), "s"(base)
      : "memory");
}

// Every LDS access of this wave done, its loads to LDS landed, and the same for the others.
__device__ __forceinline__ void stage_barrier() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

typedef __attribute__((address_space(3))) int8_t lds_i8_t;

__device__ __forceinline__ int xcd_order() {
  return (int)(blockIdx.x % 8) * (int)(gridDim.x / 8) + (int)(blockIdx.x / 8);
}

template <class E, bool SWIGLU, int MI, int NI>
__global__ __launch_bounds__(LT, MI * NI >= 16 ? 1 : 2) void product_tile_kernel(ProdArgs a) {
  constexpr int BM = 64 * MI, BN = 64 * NI, ROWS = BM + BN, STAGE = ROWS * LK;
  constexpr int LPW = ROWS / 8 / (LT / 64);  // loads of a wave per stage, 8 rows each
  extern __shared__ __align__(16) int8_t l_smem[];  // 2 stages: channels, then rows
  __shared__ int s_mt[kMaxGroups + 1];
  __shared__ int s_wave[LT / 64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  tile_prefix<BM>(a, s_mt, s_wave, tid, LT);
  const int NT = (a.N + BN - 1) / BN, MT = s_mt[a.groups];
  const int ntiles = MT * NT;
  const int nst = (a.K + LK - 1) / LK;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_i8_t*)l_smem;
  const int wn = (wave & 1) * 32 * NI, wm = (wave >> 1) * 32 * MI;
  const int r32 = lane & 31, half = lane >> 5;
  for (int tile = xcd_order(); tile < ntiles; tile += gridDim.x) {
    const int mt = tile / NT, nt = tile - mt * NT;
    const int g = __builtin_amdgcn_readfirstlane(find_group(s_mt, a.groups, mt));
    const int2 gr = group_rows(a, g);
    const int2 rr = make_int2(__builtin_amdgcn_readfirstlane(gr.x),
                              __builtin_amdgcn_readfirstlane(gr.y));
    const int m0 = __builtin_amdgcn_readfirstlane(rr.x + (mt - s_mt[g]) * BM), n0 = nt * BN;
    const int8_t* wbase = a.w + ((int64_t)g * a.N + n0) * a.ws;
    const int8_t* abase = a.a + (int64_t)m0 * a.as;
    // load i of this wave: stage rows 8 (wave * LPW + i) .. + 7, lane l brings row + l / 8, chunk
    // l % 8 in LDS; rows past the group or past N load the last valid one
    auto chunk_of = [&](int i) {
      const int row = (wave * LPW + i) * 8 + (lane >> 3);
      const int r = row < BN ? row_of_channel(row & 31) : row & 31;
      return (lane & 7) ^ ((r >> 1) & 7);
    };
    uint32_t off[LPW];
#pragma unroll
    for (int i = 0; i < LPW; ++i) {
      const int row = (wave * LPW + i) * 8 + (lane >> 3);
      off[i] = (row < BN ? (uint32_t)min(row, a.N - 1 - n0) * (uint32_t)a.ws
                         : (uint32_t)min(row - BN, rr.y - 1 - m0) * (uint32_t)a.as) +
               16 * chunk_of(i);
    }
    auto load_stage = [&](int st) {
      const uint32_t dst = lds0 + (st & 1) * STAGE + wave * LPW * 1024;
      const int8_t* wk = wbase + st * LK;
      const int8_t* ak = abase + st * LK;
      const int left = (a.K - st * LK) / 16;  // chunks of the row in this stage
      if (left >= LK / 16) {
#pragma unroll
        for (int i = 0; i < LPW; ++i)
          load_to_lds(dst + i * 1024, off[i], (wave * LPW + i) * 8 < BN ? wk : ak);
      } else {
#pragma unroll 1
        for (int i = 0; i < LPW; ++i) {
          const int row = (wave * LPW + i) * 8 + (lane >> 3), c = chunk_of(i);
          const int8_t* src =
              row < BN ? wk + (int64_t)min(row, a.N - 1 - n0) * a.ws
                       : ak + (int64_t)min(row - BN, rr.y - 1 - m0) * a.as;
          i32x4 v = i32x4{0, 0, 0, 0};  // past K
          if (c < left) v = *(const i32x4*)(src + 16 * c);
          *(i32x4*)(l_smem + (st & 1) * STAGE + (wave * LPW + i) * 1024 + lane * 16) = v;
        }
      }
    };
    i32x16 acc[NI][MI];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < MI; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][j][q] = 0;
    const int8_t* rw = l_smem + (wn + channel_of_row(r32)) * LK;
    const int8_t* ra = l_smem + (BN + wm + r32) * LK;
    auto read = [&](i32x4 (&fw)[NI], i32x4 (&fa)[MI], int buf, int kk) {
      const int o = buf * STAGE + (((2 * kk + half) ^ ((r32 >> 1) & 7)) << 4);
#pragma unroll
      for (int i = 0; i < NI; ++i) fw[i] = *(const i32x4*)(rw + o + i * 32 * LK);
#pragma unroll
      for (int j = 0; j < MI; ++j) fa[j] = *(const i32x4*)(ra + o + j * 32 * LK);
    };
    auto multiply = [&](const i32x4 (&fw)[NI], const i32x4 (&fa)[MI]) {
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < MI; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[i], fa[j], acc[i][j], 0, 0, 0);
    };
    i32x4 fw0[NI], fa0[MI], fw1[NI], fa1[MI];
    load_stage(0);
    stage_barrier();
    if (nst > 1) load_stage(1);
    read(fw0, fa0, 0, 0);
    for (int st = 0; st < nst; ++st) {
      const int b = st & 1;
      read(fw1, fa1, b, 1);
      multiply(fw0, fa0);
      read(fw0, fa0, b, 2);
      multiply(fw1, fa1);
      read(fw1, fa1, b, 3);
      multiply(fw0, fa0);
      stage_barrier();
      if (st + 2 < nst) load_stage(st + 2);
      if (st + 1 < nst) read(fw0, fa0, b ^ 1, 0);
      multiply(fw1, fa1);
    }
    const float* w_scale = a.w_scale + (int64_t)g * a.N;
#pragma unroll
    for (int j = 0; j < MI; ++j) {
      const int m = m0 + wm + 32 * j + r32;
      if (m >= rr.y) continue;
      const float sa = a.a_scale[m];
#pragma unroll
      for (int i = 0; i < NI; ++i)
        store_channels<E, SWIGLU>(a, m, n0 + wn + 32 * i + 16 * half, w_scale, sa, acc[i][j]);
    }
  }
}

template <class E, bool SWIGLU, int MI, int NI>
void launch_tile(const ProdArgs& a, hipStream_t s) {
  constexpr int BM = 64 * MI, BN = 64 * NI;
  const int64_t mt = a.M / BM + (a.offsets ? min(a.groups, a.M) : 1);
  const int64_t tiles = mt * ((a.N + BN - 1) / BN);
  constexpr int lds = 2 * (BM + BN) * LK;
  constexpr int per_cu = lds > 80 * 1024 ? 1 : 2;
  static const bool big_lds = hipFuncSetAttribute(
      (const void*)product_tile_kernel<E, SWIGLU, MI, NI>,
      hipFuncAttributeMaxDynamicSharedMemorySize, lds) == hipSuccess;
  (void)big_lds;
  const int grid = (int)std::min<int64_t>((tiles + 7) / 8 * 8, 256 * per_cu);
  hipLaunchKernelGGL((product_tile_kernel<E, SWIGLU, MI, NI>), dim3(grid), dim3(LT), lds, s, a);
}

template <class E, bool SWIGLU>
void launch_product(const ProdArgs& a, hipStream_t s) {
  const int nf = (a.N + FN - 1) / FN;
  if (a.M <= 64) {
    if (a.offsets || a.M <= 16)
      hipLaunchKernelGGL((product_few_kernel<E, SWIGLU, 1>), dim3(nf, a.offsets ? a.M : 1),
                         dim3(FT), 0, s, a);
    else if (a.M <= 32)
      hipLaunchKernelGGL((product_few_kernel<E, SWIGLU, 2>), dim3(nf), dim3(FT), 0, s, a);
    else
      hipLaunchKernelGGL((product_few_kernel<E, SWIGLU, 4>), dim3(nf), dim3(FT), 0, s, a);
    return;
  }
  const bool aligned = !(((uintptr_t)a.a | (uintptr_t)a.w | (uintptr_t)a.as | (uintptr_t)a.ws |
                          (uintptr_t)a.K) & 15) &&
                       a.as < (1 << 23) && a.ws < (1 << 23);
  if (aligned) {
    const int64_t avg = a.M / a.groups;
    if (avg >= 512)
      launch_tile<E, SWIGLU, 4, 4>(a, s);
    else
      launch_tile<E, SWIGLU, 2, 2>(a, s);
    return;
  }
  const int64_t mt = a.M / GM + (a.offsets ? min(a.groups, a.M) : 1);
  const int64_t nt = (a.N + GN - 1) / GN;
  hipLaunchKernelGGL((product_any_kernel<E, SWIGLU>), dim3((unsigned)(mt * nt)), dim3(GT), 0, s,
                     a);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_product_i8(const int8_t* a, int64_t a_stride, const float* a_scale,
                                     int32_t M, int32_t K, const int8_t* w, int64_t w_stride,
                                     const float* w_scale, int32_t N, int32_t groups,
                                     const int32_t* offsets, int32_t epilogue, void* out,
                                     int64_t out_stride, int32_t out_type, void* stream) {
  const bool swiglu = epilogue == MOE_EPI_SWIGLU;
  if (M < 0 || M > kMaxM || K < 1 || K > kMaxK || N < 1 || N > kMaxN || groups < 1 ||
      groups > kMaxGroups || (epilogue != MOE_EPI_NONE && !swiglu) || (swiglu && N % 2) ||
      (!offsets && groups != 1))
    return MOE_E_INVALID;
  if (out_type < MOE_T_BF16 || out_type > MOE_T_FP32) return MOE_E_INVALID;
  if (M == 0) return MOE_OK;
  if (!rows_ok(a, a_stride, K, MOE_T_I8) || !rows_ok(w, w_stride, K, MOE_T_I8) ||
      !rows_ok(out, out_stride, swiglu ? N / 2 : N, out_type) || !a_scale || !w_scale ||
      ((uintptr_t)a_scale & 3) || ((uintptr_t)w_scale & 3) || ((uintptr_t)offsets & 3) ||
      !on_current_device(out))
    return MOE_E_INVALID;
  ProdArgs p{a, a_stride, a_scale, M,       K,   w,         w_stride,
             w_scale, N, groups, offsets, out, out_stride};
  const hipStream_t s = (hipStream_t)stream;
  if (out_type == MOE_T_BF16)
    swiglu ? launch_product<bf16_t, true>(p, s) : launch_product<bf16_t, false>(p, s);
  else if (out_type == MOE_T_FP16)
    swiglu ? launch_product<fp16_t, true>(p, s) : launch_product<fp16_t, false>(p, s);
  else
    swiglu ? launch_product<float, true>(p, s) : launch_product<float, false>(p, s);
  return launched();
}
