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

template <class E, bool SWIGLU>
void launch_product(const ProdArgs& a, hipStream_t s) {
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
