// Low-rank adapters of many requests at once, added beside a shared projection: over rows sorted by
// adapter, out[m] = base[m] + f_g (x[m] A_g^T) B_g^T with A_g [rank][K] and B_g [N][rank].
//
// A workgroup takes a tile of rows of one adapter and a share of the channels.  First h = x A^T: its
// waves split the contraction and are joined in LDS; then every wave adds h B^T to blocks of channels.
// The rows are the columns of the matrix instruction, so a lane holds neighbouring channels of one
// output row.  x, base and out move once per row, A and B once per tile (they stay in the caches),
// and the products are few beside the bytes: bound by memory while the rank is small.
// h is held in fp32.  16-bit inputs multiply it as two 16-bit parts, which keep 16 bits of bf16 and
// 22 (of the row's largest) of fp16: its rounding stays far inside the output's.
#include <algorithm>

#include "row_ops.h"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 fp16x8 __attribute__((ext_vector_type(8)));

constexpr int AD_T = 256, AD_W = AD_T / 64;  // threads, waves
constexpr int kMaxRank = 128;
constexpr int kMaxAdapters = 1024;
constexpr int NT = 4, NB = 16 * NT;  // channel tiles of a block, its channels

struct AdaptArgs {
  const void* x;
  int64_t xs;
  int M, K;
  const void* a;
  int64_t as;
  const void* b;
  int64_t bs;
  int N, rank;
  const float* scale;  // may be null
  int adapters;
  const int* offsets;  // null: one adapter, all rows
  const int* order;    // null: the rows lie sorted
  const void* base;    // may be null, or out
  int64_t base_s;
  void* out;
  int64_t os;
};

// acc += a b over the 16 bytes that each lane holds of a row of a and a column of b (lane l: row or
// column l % 16, share l / 16 of the contraction).
template <class E>
__device__ __forceinline__ void mma(f32x4& acc, const u32x4& a, const u32x4& b) {
  if constexpr (__is_same(E, bf16_t)) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                  __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
  } else if constexpr (__is_same(E, fp16_t)) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(fp16x8, a),
                                                 __builtin_bit_cast(fp16x8, b), acc, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[i]), __uint_as_float(b[i]), acc,
                                                 0, 0, 0);
  }
}

template <class E>
__device__ __forceinline__ u32x4 load_full(const E* p) {
  return *(const u32x4_any*)p;
}
// 16 bytes of a contraction from p on, where n elements of a row of `len` are left: all, or (len at
// least 16 bytes) the row's last 16 bytes with what lies before p zeroed, or the elements of a
// shorter row one by one; zeros behind the end.  Both operands agree in which is which.
template <class E>
__device__ __forceinline__ u32x4 load_tail(const E* p, int n, int len) {
  constexpr int V = kChunk<E>;
  if (n <= 0) return u32x4{0, 0, 0, 0};
  Chunk<E> c;
  if (len >= V) {
    c.q = load_full(n >= V ? p : p + n - V);
    const int cut = V - min(n, V);
#pragma unroll
    for (int i = 0; i < V; ++i) c.e[i] = i < cut ? E{} : c.e[i];
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) c.e[i] = i < n ? p[i] : E{};
  }
  return c.q;
}

struct Tile {
  int g, m0, end;  // adapter, first sorted row, end of the adapter's rows
};
// Row tile `tile` of BM rows, counted over the adapters, by every wave for itself (64 adapters at a
// time); g = -1 behind the last.
template <int BM>
__device__ __forceinline__ Tile find_tile(const AdaptArgs& a, int tile, int lane) {
  if (!a.offsets) return tile * BM < a.M ? Tile{0, tile * BM, a.M} : Tile{-1, 0, 0};
  for (int g0 = 0; g0 < a.adapters; g0 += 64) {
    int lo = 0, hi = 0;
    if (g0 + lane < a.adapters) {
      lo = min(max(a.offsets[g0 + lane], 0), a.M);
      hi = min(max(a.offsets[g0 + lane + 1], lo), a.M);
    }
    const int n = (hi - lo + BM - 1) / BM;
    int inc = n;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const int o = __shfl_up(inc, s);
      if (lane >= s) inc += o;
    }
    const uint64_t past = __ballot(inc > tile);
    if (past) {
      const int l = __builtin_ctzll(past);
      const int first = __builtin_amdgcn_readlane(inc - n, l);
      return Tile{g0 + l, __builtin_amdgcn_readlane(lo, l) + (tile - first) * BM,
                  __builtin_amdgcn_readlane(hi, l)};
    }
    tile -= __builtin_amdgcn_readlane(inc, 63);
  }
  return Tile{-1, 0, 0};
}

// A tile of 16 MT rows, ranks up to 16 RT.
template <class E, int RT, int MT>
__global__ __launch_bounds__(AD_T) void adapt_rows_kernel(AdaptArgs a) {
  constexpr int V = kChunk<E>, BM = 16 * MT, UNIT = 8 * V;  // elements of 128 bytes
  constexpr bool SPLIT = sizeof(E) == 2;
  constexpr int PITCH = 16 * RT + 4;                 // of a row of h, in floats
  constexpr int R = RT == 1 && SPLIT ? 32 : 16 * RT;  // contraction of the second product, padded
  constexpr int RK = R / (4 * V);
  constexpr int HP = R + V;  // pitch of its operand
  __shared__ __align__(16) float s_part[AD_W][BM][PITCH];
  __shared__ __align__(16) E s_h[SPLIT ? 2 : 1][BM][HP];
  __shared__ float s_back[BM];  // powers of two that fp16's parts were divided by
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const Tile t = find_tile<BM>(a, blockIdx.x, lane);
  if (t.g < 0) return;
  // this lane's rows; -1: none
  int row[MT];
  const E* x[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int p = t.m0 + 16 * i + col;
    row[i] = p >= t.end ? -1 : a.order ? a.order[p] : p;
    if ((unsigned)row[i] >= (unsigned)a.M) row[i] = -1;
    x[i] = (const E*)a.x + max(row[i], 0) * a.xs + quad * 2 * V;
  }
  const E* w[RT];  // rows of A; those behind the rank repeat the last
#pragma unroll
  for (int i = 0; i < RT; ++i)
    w[i] = (const E*)a.a + ((int64_t)t.g * a.rank + min(16 * i + col, a.rank - 1)) * a.as +
           quad * 2 * V;
  f32x4 acc[RT][MT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[r][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int units = a.K / UNIT;
#pragma unroll 2
  for (int u = wave; u < units; u += AD_W) {
    u32x4 xv[MT][2], wv[RT][2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int i = 0; i < MT; ++i) xv[i][s] = load_full(x[i] + u * UNIT + s * V);
#pragma unroll
      for (int r = 0; r < RT; ++r) wv[r][s] = load_full(w[r] + u * UNIT + s * V);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < MT; ++i) mma<E>(acc[r][i], wv[r][s], xv[i][s]);
  }
  if (units * UNIT < a.K && units % AD_W == wave) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int k = units * UNIT + s * V, left = a.K - k - quad * 2 * V;
      u32x4 xv[MT];
#pragma unroll
      for (int i = 0; i < MT; ++i) xv[i] = load_tail(x[i] + k, left, a.K);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const u32x4 wv = load_tail(w[r] + k, left, a.K);
#pragma unroll
        for (int i = 0; i < MT; ++i) mma<E>(acc[r][i], wv, xv[i]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int i = 0; i < MT; ++i)
      *(f32x4*)&s_part[wave][16 * i + col][16 * r + 4 * quad] = acc[r][i];
  __syncthreads();
  {  // the waves' parts joined, scaled and laid out as an operand
    constexpr int PER = AD_T / BM;  // threads of a row
    const int m = tid / PER;
    const float f = a.scale ? a.scale[t.g] : 1.f;
    float h[R / PER], big = 0.f;
#pragma unroll
    for (int i = 0; i < R / PER; ++i) {
      // the rank's last chunk ends with it and holds zeros where the one before has been
      const int q = tid % PER + i * PER, c = q / V * V;
      const int r = c + V <= a.rank || a.rank < V ? q : a.rank - V + q % V;
      const bool in = c < a.rank && r >= c && r < a.rank;
      h[i] = 0.f;
      if (in) {
#pragma unroll
        for (int p = 0; p < AD_W; ++p) h[i] += s_part[p][m][r];
        h[i] *= f;
      }
      big = fmaxf(big, fabsf(h[i]));
    }
    float by = 1.f;
    if constexpr (__is_same(E, fp16_t)) {
#pragma unroll
      for (int s = 1; s < PER; s <<= 1) big = fmaxf(big, __shfl_xor(big, s));
      // the row's largest in [1, 2), inside the normal numbers' exponents
      const int e = (int)(__float_as_uint(big) >> 23) - 127;
      if (e > -126 && e < 127) by = __uint_as_float((uint32_t)(127 - e) << 23);
      if (tid % PER == 0) s_back[m] = 1.f / by;
    }
#pragma unroll
    for (int i = 0; i < R / PER; ++i) {
      const int q = tid % PER + i * PER;
      const float v = h[i] * by;
      const E hi = from_f32<E>(v);
      s_h[0][m][q] = hi;
      if constexpr (SPLIT) {
        const float rest = v - to_f32(hi);
        s_h[1][m][q] = from_f32<E>(rest - rest == 0.f ? rest : 0.f);  // an infinity has none
      }
    }
  }
  __syncthreads();
  u32x4 h[MT][RK][SPLIT ? 2 : 1];
  float back[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    back[i] = __is_same(E, fp16_t) ? s_back[16 * i + col] : 1.f;
#pragma unroll
    for (int s = 0; s < RK; ++s)
#pragma unroll
      for (int p = 0; p < (SPLIT ? 2 : 1); ++p)
        h[i][s][p] = *(const u32x4*)&s_h[p][16 * i + col][(s * 4 + quad) * V];
  }
  // row 4 q + i of channel tile t is channel 4 (NT q + t) + i of the block: a lane's results are
  // 4 NT neighbouring channels
  const int blocks = (a.N + NB - 1) / NB;
  const E* const bg = (const E*)a.b + (int64_t)t.g * a.N * a.bs;
  for (int nb = blockIdx.y * AD_W + wave; nb < blocks; nb += gridDim.y * AD_W) {
    f32x4 o[MT][NT];
#pragma unroll
    for (int c = 0; c < NT; ++c) {
      const int n = min(nb * NB + 4 * (NT * (col >> 2) + c) + (col & 3), a.N - 1);
      const E* const b = bg + n * a.bs;
      u32x4 bv[RK];
#pragma unroll
      for (int s = 0; s < RK; ++s) {
        const int r = (s * 4 + quad) * V;
        bv[s] = r + V <= a.rank ? load_full(b + r) : load_tail(b + r, a.rank - r, a.rank);
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        o[i][c] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < RK; ++s)
#pragma unroll
          for (int p = SPLIT ? 1 : 0; p >= 0; --p) mma<E>(o[i][c], bv[s], h[i][s][p]);
      }
    }
    const int n0 = nb * NB + 4 * NT * quad;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      if (row[i] < 0) continue;
      const E* const base = (const E*)a.base + row[i] * a.base_s;
      E* const out = (E*)a.out + row[i] * a.os;
#pragma unroll
      for (int q = 0; q < 4 * NT; q += V) {
        const int n = n0 + q, left = a.N - n;
        if (left <= 0) continue;
        Chunk<E> v;
        float f[V];
        if (a.base) {
          if (left >= V)
            v = load_chunk<V>(base + n);
          else
            for (int e = 0; e < V; ++e)
              if (e < left) v.e[e] = base[n + e];
        }
#pragma unroll
        for (int e = 0; e < V; ++e)
          f[e] = fmaf(o[i][(q + e) / 4][(q + e) % 4], back[i], a.base ? to_f32(v.e[e]) : 0.f);
        v = round_chunk<E, V>(f);
        if (left >= V)
          store_chunk(out + n, v);
        else
          for (int e = 0; e < V; ++e)
            if (e < left) out[n + e] = v.e[e];
      }
    }
  }
}

// ------------------------------------------------------------------ host side

// Row tiles are counted for the worst split of the rows over the adapters; workgroups behind the last
// tile return.  The channels are shared out until there are two workgroups for a CU.
template <class E, int RT, int MT>
hipError_t launch_adapt_by(const AdaptArgs& a, hipStream_t s) {
  constexpr int BM = 16 * MT;
  const int groups = a.offsets ? std::min(a.adapters, a.M) : 1;
  const int tiles = std::min(a.M, a.M / BM + groups);
  const int blocks = (a.N + NB - 1) / NB;
  const int full = std::max(1, a.M / BM);
  const int shares = std::max(1, std::min((blocks + AD_W - 1) / AD_W, 512 / full));
  return launch_kernel(adapt_rows_kernel<E, RT, MT>, dim3((unsigned)tiles, (unsigned)shares),
                       dim3(AD_T), 0, s, a);
}
template <class E>
hipError_t launch_adapt(const AdaptArgs& a, hipStream_t s) {
  // 32 rows a tile where the adapters have so many
  const bool wide = a.M >= 32 * (a.offsets ? a.adapters : 1);
  if (a.rank <= 16) return wide ? launch_adapt_by<E, 1, 2>(a, s) : launch_adapt_by<E, 1, 1>(a, s);
  if (a.rank <= 32) return wide ? launch_adapt_by<E, 2, 2>(a, s) : launch_adapt_by<E, 2, 1>(a, s);
  if (a.rank <= 64) return wide ? launch_adapt_by<E, 4, 2>(a, s) : launch_adapt_by<E, 4, 1>(a, s);
  return launch_adapt_by<E, 8, 1>(a, s);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_adapt_rows(const void* x, int64_t x_stride, int32_t type, int32_t M,
                                     int32_t K, const void* a, int64_t a_stride, const void* b,
                                     int64_t b_stride, int32_t N, int32_t rank, const float* scale,
                                     int32_t adapters, const int32_t* offsets,
                                     const int32_t* order, const void* base, int64_t base_stride,
                                     void* out, int64_t out_stride, void* stream) {
  if (!float_type(type) || M < 0 || M > kMaxRows || K < 1 || K > kMaxCols || N < 1 ||
      N > kMaxCols || rank < 1 || rank > kMaxRank || adapters < 1 || adapters > kMaxAdapters ||
      (!offsets && adapters != 1))
    return MOE_E_INVALID;
  if (M == 0) return MOE_OK;  // before the pointers: empty buffers have none
  if (!rows_ok(x, x_stride, K, type) || !rows_ok(a, a_stride, K, type) ||
      !rows_ok(b, b_stride, rank, type) || !rows_ok(out, out_stride, N, type) ||
      (base && !rows_ok(base, base_stride, N, type)) || !aligned4(scale) || !aligned4(offsets) ||
      !aligned4(order) || !on_current_device(out))
    return MOE_E_INVALID;
  AdaptArgs p{x, x_stride, M, K, a, a_stride, b, b_stride, N, rank, scale, adapters,
              offsets, order, base, base_stride, out, out_stride};
  const hipStream_t s = (hipStream_t)stream;
  if (type == MOE_T_BF16) return launched(launch_adapt<bf16_t>(p, s));
  if (type == MOE_T_FP16) return launched(launch_adapt<fp16_t>(p, s));
  return launched(launch_adapt<float>(p, s));
}
