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
#include <atomic>
#include <cmath>
#include <type_traits>

#include "row_ops.h"

namespace moe {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

constexpr int kMaxK = 131071;  // 128 * 128 * K stays below 2^31
constexpr int kMaxGroups = 1024;
constexpr int kMaxGroups320 = 512;  // of the 256 x 320 tiles (LDS)
constexpr int kMaxN = 1 << 20;
constexpr int kMaxM = (1 << 24) - 1;

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
  return fabsf(t) < 128.f ? fmaf(e, rest * 0.693147181f, e) : e;
}
// silu(z) for an output of type E.  For 16-bit outputs exp2 of the rounded exponent is enough: its
// error, below 2^-17 where the result is not negligible, is far inside half a step (2^-12).
// The reciprocal instruction returns 0 for what lies above 2^126, so it is given a sixteenth.
template <class E>
__device__ __forceinline__ float silu_for(float z) {
  const float e = sizeof(E) == 2 ? __builtin_amdgcn_exp2f(-1.44269504f * z) : exp_neg(z);
  return z * (__builtin_amdgcn_rcpf(fmaf(e, 0.0625f, 0.0625f)) * 0.0625f);
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

// s_mt[g] = first row tile (of BM rows) of group g, s_mt[groups] = their number; s_rows[g] = the
// group's rows.
template <int BM>
__device__ void tile_prefix(const ProdArgs& a, int* s_mt, int2* s_rows, int* s_wave, int tid,
                            int nthr) {
  const int per = (a.groups + nthr - 1) / nthr;
  int sum = 0;
  for (int i = 0; i < per; ++i) {
    const int g = tid * per + i;
    if (g < a.groups) {
      const int2 r = group_rows(a, g);
      s_rows[g] = r;
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
      const int2 r = s_rows[g];  // this thread's own
      first += (r.y - r.x + BM - 1) / BM;
      if (g == a.groups - 1) s_mt[a.groups] = first;
    }
  }
  __syncthreads();
}

// The last g with s_mt[g] <= mt, by a whole wave: each lane looks at one group of 64.
__device__ __forceinline__ int find_group(const int* s_mt, int groups, int mt, int lane) {
  int n = 0;
  for (int g0 = 0; g0 < groups; g0 += 64) {
    const int v = s_mt[min(g0 + lane, groups - 1)];
    n += __popcll(__ballot(g0 + lane < groups && v <= mt));
  }
  return n - 1;
}

// The values of a lane's 16 channels (8 outputs with SwiGLU): sums acc, scaled by the row's sa and
// the channels' sw.
template <class E, bool SWIGLU>
__device__ __forceinline__ void channel_values(float (&v)[16], const float (&sw)[16], float sa,
                                               const i32x16& acc) {
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = (float)acc[i] * sa * sw[i];
  if constexpr (SWIGLU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = silu_for<E>(v[2 * i]) * v[2 * i + 1];
  }
}

// A wave's LDS accesses execute in order; this keeps the compiler, which sees one lane's only, from
// reordering or merging them where lanes read what others wrote.
__device__ __forceinline__ void wave_lds_order() { asm volatile("" ::: "memory"); }

// 32 output rows of RB bytes each that a wave has put into its LDS (row r's 16-byte chunk c at
// chunk c ^ out_swz(r)) go to memory with neighbouring lanes on neighbouring chunks: a request per
// 64 bytes instead of one per 16, which is what the stores of a tile cost otherwise (a launch
// that writes 403 MB: 165 us with a lane per row, 126 so).
template <int RB>
__device__ __forceinline__ int out_swz(int row) {
  return RB == 64 ? (row >> 2) & 3 : (row >> 3) & 1;
}
// The first n elements of a chunk (n >= its size: all).
template <class E>
__device__ __forceinline__ void store_part(E* p, int n, const Chunk<E>& c) {
  if (n >= kChunk<E>) {
    store_chunk(p, c);
  } else {
#pragma unroll
    for (int i = 0; i < kChunk<E>; ++i)
      if (i < n) p[i] = c.e[i];
  }
}
template <class E, int RB>
__device__ __forceinline__ void store_rows(const int8_t* stage, int lane, E* out, int64_t os,
                                           int rows, int cols) {
  constexpr int CPR = RB / 16, V = kChunk<E>;
  Chunk<E> v[CPR / 2];
  wave_lds_order();
#pragma unroll
  for (int t = 0; t < CPR / 2; ++t) v[t].q = *(const u32x4*)(stage + t * 1024 + lane * 16);
  wave_lds_order();
#pragma unroll
  for (int t = 0; t < CPR / 2; ++t) {
    const int row = t * (64 / CPR) + lane / CPR, c = (lane % CPR) ^ out_swz<RB>(row);
    if (row < rows && c * V < cols) store_part(out + row * os + c * V, cols - c * V, v[t]);
  }
}

// ------------------------------------------------------------------ few rows
// Up to RT * 16 rows of one group times 16 channels per workgroup, the contraction split over its
// four waves and joined in LDS (integers: in any order the same).  Operands go straight from
// memory into the registers of a 16 x 16 x 64 matrix instruction, eight steps of 64 bytes in
// flight; every weight byte is read once for the group's rows, and that stream is the bound: gate
// and up of one token's eight experts (25.2 MB of 2048-wide rows) take 6.6 us, 3.8 TB/s, of
// which launch, the search of the group and the first load's way are about half.
constexpr int FT = 256, FN = 16, FU = 8;  // threads, channels, steps in flight

__device__ __forceinline__ i32x4 load_16(const int8_t* p) {
  return __builtin_bit_cast(i32x4, *(const u32x4_any*)p);
}

// 16 bytes for a step of the product from p on, where n bytes of a row of K >= 16 are left: all 16,
// or the row's last 16 with those before p zeroed (which byte of a step is which does not matter,
// as long as both operands agree), or zeros.
__device__ __forceinline__ i32x4 load_end(const int8_t* p, int n) {
  i32x4 q = load_16(n >= 16 ? p : p + n - 16);
  const int cut = 16 - min(max(n, 0), 16);
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const int b = cut - 4 * d;  // bytes of this word that lie before p
    q[d] = b >= 4 ? 0 : b <= 0 ? q[d] : q[d] & (int)(~0u << (8 * b));
  }
  return q;
}
// The same for rows of K < 16 bytes, n = K of them at p (or none).
__device__ __forceinline__ i32x4 load_short(const int8_t* p, int n) {
  uint64_t lo = 0, hi = 0;
#pragma unroll 1
  for (int b = n - 1; b >= 0; --b) {
    hi = hi << 8 | lo >> 56;
    lo = lo << 8 | (uint8_t)p[b];
  }
  return i32x4{(int)lo, (int)(lo >> 32), (int)hi, (int)(hi >> 32)};
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
      fw[u] = load_16(pw + (s + u) * 64);
#pragma unroll
      for (int t = 0; t < RT; ++t) fa[u][t] = load_16(pa[t] + (s + u) * 64);
    }
#pragma unroll
    for (int u = 0; u < FU; ++u)
#pragma unroll
      for (int t = 0; t < RT; ++t)
        acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[u], fa[u][t], acc[t], 0, 0, 0);
  }
  for (; s < s1; ++s) {
    const int n = a.K - s * 64 - piece;
    const i32x4 fw = a.K >= 16 ? load_end(pw + s * 64, n) : load_short(pw, n);
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const i32x4 fa = a.K >= 16 ? load_end(pa[t] + s * 64, n) : load_short(pa[t], n);
      acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw, fa, acc[t], 0, 0, 0);
    }
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
        out[n0 / 2 + c] = from_f32<E>(silu_for<E>(value(2 * c)) * value(2 * c + 1));
    } else {
      if (n0 + c < a.N) out[n0 + c] = from_f32<E>(value(c));
    }
  }
}

// ------------------------------------------------------------------ tiles
// 32 WM MI rows x 32 WN NI channels per tile, WM x WN waves of 32 MI rows x 32 NI channels,
// workgroups persistent over the tiles; with KS > 1 as many sets of waves share the stages of K
// and add up in LDS, for launches of few tiles.  Stages of 128 contraction bytes go from memory
// straight into LDS (16-byte global-to-LDS loads), double buffered: the loads of stage s + 2 are
// issued when every wave has read stage s, and a tile's first stage and scales while the previous
// tile's epilogue runs.  Rows are 128 bytes unpadded; 16-byte chunk c of a row sits at chunk
// c ^ ((r / 2) % 8), r the row's place in its matrix instruction: the 16 lanes that LDS serves at
// once then read 16 distinct 16-byte bank slots.  Fragments of a 32-deep step are read while the
// previous step's matrix instructions run, also across a stage's end.  A wave whose rows (or
// channels) lie past the group's end loads and waits with the others but multiplies nothing.
// The loads are asm so that the compiler does not hold LDS reads back for them; they return
// nothing to registers, and the waits for them are the stage's own.
// They need 16-byte aligned operands and strides and K a multiple of 16; for others (ANY) a stage
// goes through registers, fetched one stage before it is put into LDS.
//
// What bounds the large dense shapes is power: 8192 x 8192 x 8192 runs at 2.37 to 2.46 POP/s with
// normally distributed codes and at 3.48 with zeros; with the former the clock falls to 1.6 GHz of
// 2.4 while the matrix units are 67% busy (a vendor library's plain 8-bit product: 2.08, zeros 3.26).
// Stages of 64 bytes four deep, 128 x 128 per wave, four waves of 64 x 64 per SIMD and fixed
// orders of reads and products were within 15% of this or slower.  With few stages per tile it is
// what lies outside them: 131072 rows over 128 experts x 1536 channels, SwiGLU, bf16 out take 104,
// 181, 272 and 455 us at K = 128, 512, 1024 and 2048 (437 to 482 by the card), 23 us for each stage
// and 90 besides; x 2048 channels, plain, 168 and 338 at K = 128 and 768, 34 for each stage and
// 134 besides.  There a tile's stores hold up the next one's first product: every stage's barrier
// waits for all that is outstanding, stores too.
// Registers: the 256 x 320 kernels spill 45 to 51 vector registers (184 to 208 bytes a lane, mostly
// in taking up a tile and in the epilogue), of those for any alignment (ANY, with a 64-bit address
// for each load) 128 x 128 spills 22 to 25 and 64 x 64 over two or four sets of waves 11 to 16.
constexpr int LK = 128;

// 16 bytes per lane from base + off to the LDS bytes from lds + 16 * lane on.  The instruction takes
// the LDS address from m0: an operand of the statement, so the compiler writes the register and
// knows what it holds (a wait state has to lie between that and the load).
__device__ __forceinline__ void load_to_lds(uint32_t lds, uint32_t off, const int8_t* base) {
  asm volatile(
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, %2"
      :
      : "{m0}"(lds), "v"(off), "s"(base)
      : "memory");
}

// The same with 4 bytes per lane.
__device__ __forceinline__ void load4_to_lds(uint32_t lds, uint32_t off, const float* base) {
  asm volatile(
      "s_nop 0\n\t"
      "global_load_lds_dword %1, %2"
      :
      : "{m0}"(lds), "v"(off), "s"(base)
      : "memory");
}

// Every LDS access of this wave done, its loads to LDS landed, and the same for the others.
__device__ __forceinline__ void stage_barrier() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

typedef __attribute__((address_space(3))) int8_t lds_i8_t;
typedef __attribute__((address_space(3))) float lds_f32_t;

__device__ __forceinline__ int xcd_order() {
  return (int)(blockIdx.x % 8) * (int)(gridDim.x / 8) + (int)(blockIdx.x / 8);
}

// Tiles in blocks of four row tiles, channel tiles ascending inside: the 32 tiles that an XCD's
// CUs work on at once then share 4 row and 8 channel operands in its L2.
__device__ __forceinline__ void tile_of(int tile, int MT, int NT, int& mt, int& nt) {
  const int block = tile / (4 * NT), in = tile - block * 4 * NT;
  const int rows = min(4, MT - block * 4);
  nt = in / rows;
  mt = block * 4 + in - nt * rows;
}

template <class E, bool SWIGLU, bool ANY, int WM, int WN, int MI, int NI, int KS, int PER_CU>
__global__ __launch_bounds__(64 * WM * WN * KS, WM * WN * KS * PER_CU / 4)
void product_tile_kernel(ProdArgs a) {
  constexpr int TW = WM * WN, LT = 64 * TW * KS;  // waves of a tile; threads
  constexpr int BM = 32 * WM * MI, BN = 32 * WN * NI, ROWS = BM + BN, STAGE = ROWS * LK;
  constexpr int LPW = ROWS / 8 / TW;  // loads of a wave per stage, 8 rows each
  static_assert(LPW * 8 * TW == ROWS && BN % 64 == 0 && BM % 64 == 0);
  // KS times 2 stages (channels, then rows), the groups' rows and first tiles
  extern __shared__ __align__(16) int8_t l_smem[];
  int2* const s_rows = (int2*)(l_smem + 2 * KS * STAGE);
  int* const s_mt = (int*)(s_rows + a.groups);
  __shared__ __align__(16) float s_scale[2][ROWS];  // of the tile's channels, then of its rows
  __shared__ int s_wave[LT / 64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave_all = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ks = KS == 1 ? 0 : wave_all / TW, wave = KS == 1 ? wave_all : wave_all % TW;
  tile_prefix<BM>(a, s_mt, s_rows, s_wave, tid, LT);
  const int NT = (a.N + BN - 1) / BN, MT = __builtin_amdgcn_readfirstlane(s_mt[a.groups]);
  const int ntiles = MT * NT;
  // stages of K; rounds of KS stages, stage KS * round + ks is this wave's
  const int nst = (a.K + LK - 1) / LK, nfull = a.K / LK, rounds = (nst + KS - 1) / KS;
  int8_t* const stages = l_smem + ks * 2 * STAGE;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_i8_t*)stages;
  const int wn = (wave % WN) * 32 * NI, wm = (wave / WN) * 32 * MI;
  const int r32 = lane & 31, half = lane >> 5;

  int tile = xcd_order();
  if (tile >= ntiles) return;
  int m0, n0, end;  // the tile's first row and channel, its group's last row + 1
  const int8_t *wbase, *abase;
  // load i of this wave: stage rows 8 (wave * LPW + i) .. + 7, lane l brings row + l / 8, chunk
  // l % 8 in LDS; rows past the group or past N load the last valid one, bytes past K are zero
  auto chunk_of = [&](int i) {
    const int row = (wave * LPW + i) * 8 + (lane >> 3);
    const int r = row < BN ? row_of_channel(row & 31) : row & 31;
    return (lane & 7) ^ ((r >> 1) & 7);
  };
  uint32_t off[LPW];        // aligned: the rows' byte offsets,
  const int8_t* src[LPW];   // else their addresses, and the stage under way to LDS
  i32x4 held[LPW];
  auto load_stage = [&](int round, int buf) {
    const int st = round * KS + ks;
    const uint32_t dst = lds0 + buf * STAGE + wave * LPW * 1024;
    const int8_t* wk = wbase + st * LK;
    const int8_t* ak = abase + st * LK;
    if (st < nfull) {
#pragma unroll
      for (int i = 0; i < LPW; ++i)
        load_to_lds(dst + i * 1024, off[i], (wave * LPW + i) * 8 < BN ? wk : ak);
    } else if (st < nst) {
      const int left = (a.K - st * LK) / 16;  // chunks of the row in this stage
#pragma unroll
      for (int i = 0; i < LPW; ++i) {
        if (chunk_of(i) < left)
          load_to_lds(dst + i * 1024, off[i], (wave * LPW + i) * 8 < BN ? wk : ak);
        else
          *(i32x4*)(stages + buf * STAGE + (wave * LPW + i) * 1024 + lane * 16) =
              i32x4{0, 0, 0, 0};
      }
    }
  };
  auto fetch = [&](int round) {
    const int k0 = (round * KS + ks) * LK;
    if (k0 + LK <= a.K) {
#pragma unroll
      for (int i = 0; i < LPW; ++i) held[i] = load_16(src[i] + k0);
    } else if (a.K >= 16) {
#pragma unroll
      for (int i = 0; i < LPW; ++i)
        held[i] = load_end(src[i] + k0, a.K - k0 - 16 * chunk_of(i));
    } else {
#pragma unroll
      for (int i = 0; i < LPW; ++i)
        held[i] = load_short(src[i], chunk_of(i) == 0 && k0 == 0 ? a.K : 0);
    }
  };
  // Takes up a tile: its scales (into half sb of their arrays) and its first stage.
  auto begin = [&](int t, int sb) {
    int mt, nt;
    tile_of(t, MT, NT, mt, nt);
    const int g = find_group(s_mt, a.groups, mt, lane);
    const int2 gr = s_rows[g];
    end = __builtin_amdgcn_readfirstlane(gr.y);
    m0 = __builtin_amdgcn_readfirstlane(gr.x + (mt - s_mt[g]) * BM);
    n0 = nt * BN;
    wbase = a.w + ((int64_t)g * a.N + n0) * a.ws;
    abase = a.a + (int64_t)m0 * a.as;
    const uint32_t dst = (uint32_t)(uintptr_t)(lds_f32_t*)s_scale[sb];
    for (int i = wave_all; i < ROWS / 64; i += LT / 64) {
      const int r = i * 64 + lane;
      if (i * 64 < BN)
        load4_to_lds(dst + i * 256, 4 * min(r, a.N - 1 - n0),
                     a.w_scale + (int64_t)g * a.N + n0);
      else
        load4_to_lds(dst + i * 256, 4 * min(r - BN, end - 1 - m0), a.a_scale + m0);
    }
#pragma unroll
    for (int i = 0; i < LPW; ++i) {
      const int row = (wave * LPW + i) * 8 + (lane >> 3);
      const int64_t at = row < BN ? (int64_t)min(row, a.N - 1 - n0) * a.ws
                                  : (int64_t)min(row - BN, end - 1 - m0) * a.as;
      if constexpr (ANY)
        src[i] = (row < BN ? wbase : abase) + at + 16 * chunk_of(i);
      else
        off[i] = (uint32_t)at + 16 * chunk_of(i);
    }
    if constexpr (ANY)
      fetch(0);
    else
      load_stage(0, 0);
  };
  if constexpr (!ANY) begin(tile, 0);
  const int8_t* rw = stages + (wn + channel_of_row(r32)) * LK;
  const int8_t* ra = stages + (BN + wm + r32) * LK;
  auto read = [&](i32x4 (&fw)[NI], i32x4 (&fa)[MI], int buf, int kk) {
    const int o = buf * STAGE + (((2 * kk + half) ^ ((r32 >> 1) & 7)) << 4);
#pragma unroll
    for (int i = 0; i < NI; ++i) fw[i] = *(const i32x4*)(rw + o + i * 32 * LK);
#pragma unroll
    for (int j = 0; j < MI; ++j) fa[j] = *(const i32x4*)(ra + o + j * 32 * LK);
  };
  for (int sb = 0;; sb ^= 1) {
    i32x16 acc[NI][MI];
    auto multiply = [&](const i32x4 (&fw)[NI], const i32x4 (&fa)[MI]) {
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < MI; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[i], fa[j], acc[i][j], 0, 0, 0);
    };
    if constexpr (ANY) begin(tile, sb);
    const int m1 = m0 + wm, n1 = n0 + wn, end1 = end;
    const bool active = m1 < end && n1 < a.N;
    const int mine = active ? (nst - ks + KS - 1) / KS : 0;  // rounds this wave multiplies in
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < MI; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][j][q] = 0;
    i32x4 fw0[NI], fa0[MI], fw1[NI], fa1[MI];
    // a round's products up to its last step, whose fragments are then in registers
    const auto most = [&](int buf) {
      read(fw1, fa1, buf, 1);
      multiply(fw0, fa0);
      read(fw0, fa0, buf, 2);
      multiply(fw1, fa1);
      read(fw1, fa1, buf, 3);
      multiply(fw0, fa0);
    };
    if constexpr (ANY) {
      // the two rounds before the first only bring the first two stages in
      for (int rd = -2; rd < rounds; ++rd) {
        const bool on = rd >= 0 && rd < mine;
        if (on) most(rd & 1);
        stage_barrier();
        if (rd + 2 < rounds) {
#pragma unroll
          for (int i = 0; i < LPW; ++i)
            *(i32x4*)(stages + (rd & 1) * STAGE + (wave * LPW + i) * 1024 + lane * 16) = held[i];
          if (rd + 3 < rounds) fetch(rd + 3);
        }
        if (rd >= -1 && rd + 1 < mine) read(fw0, fa0, (rd + 1) & 1, 0);
        if (on) multiply(fw1, fa1);
      }
    } else {
      stage_barrier();
      if (rounds > 1) load_stage(1, 1);
      if (mine > 0) read(fw0, fa0, 0, 0);
      int rd = 0;
      for (; rd < mine; ++rd) {
        const int buf = rd & 1;
        most(buf);
        stage_barrier();
        if (rd + 2 < rounds) load_stage(rd + 2, buf);
        if (rd + 1 < mine) read(fw0, fa0, buf ^ 1, 0);
        multiply(fw1, fa1);
      }
      for (; rd < rounds; ++rd) {
        stage_barrier();
        if (rd + 2 < rounds) load_stage(rd + 2, rd & 1);
      }
    }
    if constexpr (KS > 1) {  // the parts of K added up by the first (integers: exact)
      static_assert(NI == 1 && MI == 1 && (KS - 1) * TW * 4096 <= 2 * KS * STAGE);
      if (ks > 0) {
        i32x4* const part = (i32x4*)(l_smem + ((ks - 1) * TW + wave) * 4096) + lane;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          part[64 * q] = i32x4{acc[0][0][4 * q], acc[0][0][4 * q + 1], acc[0][0][4 * q + 2],
                               acc[0][0][4 * q + 3]};
      }
      stage_barrier();
      if (ks == 0) {
#pragma unroll
        for (int p = 1; p < KS; ++p)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const i32x4 v = *((const i32x4*)(l_smem + ((p - 1) * TW + wave) * 4096) + lane +
                              64 * q);
#pragma unroll
            for (int b = 0; b < 4; ++b) acc[0][0][4 * q + b] += v[b];
          }
      }
      stage_barrier();
    }
    tile += gridDim.x;
    const bool more = tile < ntiles;
    // the first half of the stages is free, and the other half of the scales
    if (!ANY && more) begin(tile, sb ^ 1);
    if (active && ks == 0) {
      // the second half of the stages is free until the next tile's first barrier: 2 KiB a wave
      constexpr int V = kChunk<E>, OB = 16 * (int)sizeof(E) / (SWIGLU ? 2 : 1);
      static_assert(TW * 2048 <= STAGE);
      int8_t* const stage = l_smem + STAGE + wave * 2048;
      const float* psw = s_scale[sb] + wn + 16 * half;
      const float* psa = s_scale[sb] + BN + wm + r32;
      const auto put = [&](auto rb, int chunk, const float* v) {
        constexpr int RB = decltype(rb)::value;
        *(u32x4*)(stage + r32 * RB + ((chunk ^ out_swz<RB>(r32)) << 4)) = round_chunk<E>(v).q;
      };
#pragma unroll
      for (int j = 0; j < MI; ++j) {
        const int rows = end1 - m1 - 32 * j;  // of the group from this row tile on
        E* const out = (E*)a.out + (int64_t)(m1 + 32 * j) * a.os;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int n = n1 + 32 * i;
          float sw[16], v[16];
#pragma unroll
          for (int q = 0; q < 16; ++q) sw[q] = psw[32 * i + q];
          channel_values<E, SWIGLU>(v, sw, psa[32 * j], acc[i][j]);
          if constexpr (OB == 16) {  // two channel tiles fill 64 bytes of a row
            constexpr bool odd_end = NI % 2 == 1;
            if (odd_end && i == NI - 1) {
              put(std::integral_constant<int, 32>{}, half, v);
              store_rows<E, 32>(stage, lane, out + n / 2, a.os, rows, (a.N - n) / 2);
            } else {
              put(std::integral_constant<int, 64>{}, 2 * (i & 1) + half, v);
              if (i & 1)
                store_rows<E, 64>(stage, lane, out + (n - 32) / 2, a.os, rows,
                                  (a.N - n + 32) / 2);
            }
          } else if constexpr (OB == 32) {
            put(std::integral_constant<int, 64>{}, 2 * half, v);
            put(std::integral_constant<int, 64>{}, 2 * half + 1, v + V);
            const int c = SWIGLU ? n / 2 : n;
            store_rows<E, 64>(stage, lane, out + c, a.os, rows, (SWIGLU ? a.N / 2 : a.N) - c);
          } else {  // fp32: a lane holds 64 bytes of its row; one half of the wave at a time
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (half == h) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  put(std::integral_constant<int, 64>{}, c, v + 4 * c);
              }
              store_rows<E, 64>(stage, lane, out + n + 16 * h, a.os, rows, a.N - n - 16 * h);
            }
          }
        }
      }
    }
    if (!more) return;
  }
}

template <class E, bool SWIGLU, bool ANY, int WM, int WN, int MI, int NI, int KS, int PER_CU>
hipError_t launch_tile(const ProdArgs& a, hipStream_t s) {
  constexpr int BM = 32 * WM * MI, BN = 32 * WN * NI, LT = 64 * WM * WN * KS;
  constexpr int stages = 2 * KS * (BM + BN) * LK;
  const int lds = stages + 12 * a.groups + 4;
  const auto kernel = product_tile_kernel<E, SWIGLU, ANY, WM, WN, MI, NI, KS, PER_CU>;
  // More than 64 KiB of LDS has to be allowed, for a kernel on a device as a whole: calls of other
  // threads launch under the limit that is set, so it is the largest that any call needs.
  constexpr int most = stages + 12 * (BN == 320 ? kMaxGroups320 : kMaxGroups) + 4;
  if constexpr (most > 64 * 1024) {
    static std::atomic<uint64_t> allowed{0};  // a bit per device
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (e == hipSuccess && !(allowed.load(std::memory_order_relaxed) & bit)) {
      e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, most);
      if (e == hipSuccess) allowed.fetch_or(bit, std::memory_order_relaxed);
    }
    if (e != hipSuccess) return e;
  }
  const int64_t mt = a.M / BM + (a.offsets ? std::min(a.groups, a.M) : 1);
  const int64_t tiles = mt * ((a.N + BN - 1) / BN);
  const int grid = (int)std::min<int64_t>((tiles + 7) / 8 * 8, 256 * PER_CU);
  return launch_kernel(kernel, dim3(grid), dim3(LT), lds, s, a);
}

// The tile shapes, and what the choice among them goes by: microseconds of one round of KS
// stages with one tile on a CU (low) and what each further tile there adds (more), or with a
// tile on most CUs, where the chip's power limit lowers the clock (full); microseconds a tile
// spends outside its stages (rest).  Measured with K = 768 .. 8192 and 64 to 131072 rows, one
// weight and up to 128: the shape of the smallest sum over the launch's rounds was the fastest
// measured one, or within a few percent of it (600 x 2 rows over 8 experts, 2000 x 1024: 12.4 us
// with 64 x 64, 14.9 with 128 x 128, 19.4 with 256 x 256; 4001 x 5000 x 4096: 145 us with
// 256 x 256, 134 with 128 x 128, 95 with 256 x 320, one round; 256 x 5000 x 4096: 45, 26, 20 with
// 64 x 64, 17.4 with two and 22.7 with four sets of waves).
struct TileShape {
  int bm, bn, ks, per_cu;
  float low, more, full, rest;
};
constexpr TileShape kShapes[] = {
    {256, 256, 1, 1, 1.3f, 0.f, 1.8f, 5.f},  {256, 320, 1, 1, 1.6f, 0.f, 2.2f, 6.f},
    {128, 128, 1, 2, 0.63f, 0.46f, 0.f, 2.5f}, {64, 64, 1, 4, 0.45f, 0.16f, 0.f, 1.5f},
    {64, 64, 2, 2, 0.62f, 0.33f, 0.f, 1.5f}, {64, 64, 4, 1, 1.06f, 0.f, 0.f, 1.5f}};

float tile_cost(const TileShape& t, const ProdArgs& a) {
  // row tiles: the sizes of the groups are only known on the device, so all M rows are taken as
  // placed and the groups as equal (rows whose experts are elsewhere, or a skewed routing, can make
  // another shape the fastest)
  const float rows = (float)a.M / (float)a.groups;
  const float mt = a.offsets ? (float)std::min(a.groups, a.M) * std::max(1.08f, rows / t.bm + 0.5f)
                             : (float)((a.M + t.bm - 1) / t.bm);
  const float tiles = mt * (float)((a.N + t.bn - 1) / t.bn);
  const int nst = (a.K + LK - 1) / LK, k_rounds = (nst + t.ks - 1) / t.ks;
  const auto round_us = [&](float on_gpu) {  // that many tiles at once
    if (t.full > 0.f && on_gpu > 128.f) return t.full;
    return t.low + t.more * (std::ceil(on_gpu / 256.f) - 1.f);
  };
  const float slots = 256.f * t.per_cu, whole = std::floor(tiles / slots);
  const float left = tiles - whole * slots;
  float us = whole * (k_rounds * round_us(slots) + t.rest);
  if (left > 0.f) us += k_rounds * round_us(left) + t.rest;
  return us;
}

template <class E, bool SWIGLU>
hipError_t launch_product(const ProdArgs& a, hipStream_t s) {
  const bool aligned = !(((uintptr_t)a.a | (uintptr_t)a.w | (uintptr_t)a.as | (uintptr_t)a.ws |
                          (uintptr_t)a.K) & 15) &&
                       a.as < (1 << 22) && a.ws < (1 << 22);  // a tile's offsets: 31 bits
  // Few rows: the streaming kernel takes 16 of them nearly as fast as one (x 5000 channels x 4096:
  // 8.0 and 9.3 us); with more the tiles win (64 rows: 13.0 against 22.8 us) where alignment
  // allows them, and for 128 rows of 128 groups the two are equal (42.0 and 42.5 us, the weights'
  // bytes).
  if (a.M <= 16 || (a.M <= 64 && (a.offsets || !aligned))) {
    const int nf = (a.N + FN - 1) / FN;
    if (a.offsets || a.M <= 16)
      return launch_kernel(product_few_kernel<E, SWIGLU, 1>, dim3(nf, a.offsets ? a.M : 1), dim3(FT),
                           0, s, a);
    return launch_kernel(product_few_kernel<E, SWIGLU, 4>, dim3(nf), dim3(FT), 0, s, a);
  }
  int best = aligned ? 0 : 2;  // the two largest shapes would hold twice the smaller ones' addresses
  for (int i = best + 1; i < (int)(sizeof(kShapes) / sizeof(kShapes[0])); ++i)
    if (!(kShapes[i].bn == 320 && a.groups > kMaxGroups320) &&
        tile_cost(kShapes[i], a) < tile_cost(kShapes[best], a))
      best = i;
  switch (best) {
    case 0: return launch_tile<E, SWIGLU, false, 4, 2, 2, 4, 1, 1>(a, s);
    case 1: return launch_tile<E, SWIGLU, false, 4, 2, 2, 5, 1, 1>(a, s);
    case 2: return aligned ? launch_tile<E, SWIGLU, false, 4, 2, 1, 2, 1, 2>(a, s)
                           : launch_tile<E, SWIGLU, true, 4, 2, 1, 2, 1, 2>(a, s);
    case 3: return aligned ? launch_tile<E, SWIGLU, false, 2, 2, 1, 1, 1, 4>(a, s)
                           : launch_tile<E, SWIGLU, true, 2, 2, 1, 1, 1, 4>(a, s);
    case 4: return aligned ? launch_tile<E, SWIGLU, false, 2, 2, 1, 1, 2, 2>(a, s)
                           : launch_tile<E, SWIGLU, true, 2, 2, 1, 1, 2, 2>(a, s);
    default: return aligned ? launch_tile<E, SWIGLU, false, 2, 2, 1, 1, 4, 1>(a, s)
                            : launch_tile<E, SWIGLU, true, 2, 2, 1, 1, 4, 1>(a, s);
  }
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
    return launched(swiglu ? launch_product<bf16_t, true>(p, s) : launch_product<bf16_t, false>(p, s));
  if (out_type == MOE_T_FP16)
    return launched(swiglu ? launch_product<fp16_t, true>(p, s) : launch_product<fp16_t, false>(p, s));
  return launched(swiglu ? launch_product<float, true>(p, s) : launch_product<float, false>(p, s));
}
