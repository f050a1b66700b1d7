// Root-mean-square norm of rows with the residual's addition, in the rows' type and in 8 bits, and
// its gradient.
//
// h = x + r rounded to the rows' type, q = 1 / sqrt(mean(h^2) + eps), y = q h w.  The 8-bit codes are
// those of the unrounded y: code = 127 y / max |y| = 127 p / max |p| with p = h w, where q cancels,
// so they are exact; scale = max |p| q / 127.  Gradient: with S = sum_k w dy h,
// dx = dsum + q w dy - h q^3 S / K = dsum + q (w dy - (q h) (q S / K)), dw = sum over the rows of q dy h.
//
// A row is read once and held in registers between its sums and its outputs, so both directions
// are bound by the bytes of the matrices.  Sums over a row are held in 64 bits, over a chunk of 16
// bytes in fp32, but where a row's squares or products leave its range.
#include <algorithm>
#include <type_traits>

#include "row_ops.h"

namespace moe {
namespace {

constexpr int kMaxNormCols = 16384;  // a row is held by a workgroup
constexpr int HELD = 4;              // chunks of it that a lane holds

struct NormArgs {
  const void* x;
  int64_t xs;
  const void* res;  // may be null
  int64_t res_s;
  int M, K;
  const void* w;
  float eps;
  void* sum;  // may be null, x or res
  int64_t sum_s;
  void* y;  // may be null, x or res
  int64_t ys;
  int8_t* codes;  // may be null
  int64_t cs;
  float* scale;
};

// Calls that move more bytes than this pass the caches by: what they read is not read again soon (32768
// rows of 2048 bf16 111 us so, 120 otherwise; the gradient 93 and 106).  Stores that pass the caches by
// are not joined, so where a row's ends lie inside lines that neighbouring rows share, the lines are
// written in parts: rows that 32 lanes or fewer hold stream only where sum and y start with a half line
// (65536 rows of 1024 bf16 with codes 111 us streamed and 120 not, sum and y at a stride of 1027 143 and
// 130; of 1000 149 and 127, at a stride of 1024 120 and 135; of 512, at a stride of 515 177 and 139), those
// of 16 lanes only where the codes do too (sum and codes of 500, the codes at their own stride 109 and
// 101, at 512 93 and 108; of 1000 95 and 97).  Longer rows stream wherever they start (of 2051 131 and 129,
// of 4099 146 and 152), and so do the gradient's (of 1027 106 and 111, of 515 118 and 116).
constexpr int64_t kNormStreamBytes = 128 << 20;
// A row is held by G lanes, 16, 32, 64 or (all of) a workgroup.
constexpr int norm_threads(int G) { return G < 256 ? 256 : G; }

// v joined over the lanes of a row, in all of them.
template <int G, class T, class Join>
__device__ __forceinline__ T row_join(T v, T* s_part, Join&& join) {
  v = join16(v, join);
#pragma unroll
  for (int s = 16; s < (G < 64 ? G : 64); s <<= 1) v = join(v, __shfl_xor(v, s));
  if constexpr (G > 64) {
    __syncthreads();  // what an earlier join left has been read
    if ((threadIdx.x & 63) == 0) s_part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = s_part[0];
#pragma unroll
    for (int i = 1; i < G / 64; ++i) v = join(v, s_part[i]);
  }
  return v;
}
// Two sums at once.
template <int G>
__device__ __forceinline__ void row_sums(double& u, double& v, double (*s_part)[2]) {
  const auto add = [](double a, double b) { return a + b; };
  u = join16(u, add), v = join16(v, add);
#pragma unroll
  for (int s = 16; s < (G < 64 ? G : 64); s <<= 1) u += __shfl_xor(u, s), v += __shfl_xor(v, s);
  if constexpr (G > 64) {
    __syncthreads();  // what an earlier join left has been read
    if ((threadIdx.x & 63) == 0) s_part[threadIdx.x >> 6][0] = u, s_part[threadIdx.x >> 6][1] = v;
    __syncthreads();
    u = s_part[0][0], v = s_part[0][1];
#pragma unroll
    for (int i = 1; i < G / 64; ++i) u += s_part[i][0], v += s_part[i][1];
  }
}
template <int G>
__device__ __forceinline__ double row_sum(double v, double* s_part) {
  return row_join<G>(v, s_part, [](double a, double b) { return a + b; });
}
// The larger one; a NaN stays.
__device__ __forceinline__ double max_nan(double a, double b) { return a > b || a != a ? a : b; }
template <int G>
__device__ __forceinline__ double row_max(double v, double* s_part) {
  return row_join<G>(v, s_part, [](double a, double b) { return max_nan(a, b); });
}
template <int G>
__device__ __forceinline__ float row_max(float v, float* s_part) {
  return row_join<G>(v, s_part, [](float a, float b) { return fmaxf(a, b); });
}

// A chunk without its first n elements, which the chunk before it has too.
template <class E, int V>
__device__ __forceinline__ Chunk<E, V> without_first(Chunk<E, V> c, int n) {
  if (n > 0) {
#pragma unroll
    for (int e = 0; e < V; ++e) c.e[e] = e < n ? E{} : c.e[e];
  }
  return c;
}
// Sum of a chunk's squares.  16-bit types: two products and additions to an instruction, in fp32; fp32
// in 64 bits.
template <class E, int V>
__device__ __forceinline__ double chunk_squares(const Chunk<E, V>& c) {
  if constexpr (V == 1) {
    return (double)to_f32(c.e[0]) * (double)to_f32(c.e[0]);
  } else if constexpr (sizeof(E) == 4) {
    double s = 0.0;
#pragma unroll
    for (int e = 0; e < V; ++e) s = fma((double)c.e[e], (double)c.e[e], s);
    return s;
  } else {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (__is_same(E, bf16_t)) {
        typedef __bf16 pair_t __attribute__((ext_vector_type(2)));
        const pair_t p = __builtin_bit_cast(pair_t, (uint32_t)c.q[i]);
        s = __builtin_amdgcn_fdot2_f32_bf16(p, p, s, false);
      } else {
        typedef _Float16 pair_t __attribute__((ext_vector_type(2)));
        const pair_t p = __builtin_bit_cast(pair_t, (uint32_t)c.q[i]);
        s = __builtin_amdgcn_fdot2(p, p, s, false);
      }
    }
    return s;
  }
}
// The same far from fp32's range, in 64 bits.
template <class E, int V>
__device__ __forceinline__ double chunk_squares_f64(const Chunk<E, V>& c) {
  double s = 0.0;
#pragma unroll
  for (int e = 0; e < V; ++e) s = fma((double)to_f32(c.e[e]), (double)to_f32(c.e[e]), s);
  return s;
}
// Where sums of squares and products in fp32 lose nothing to its range.
__device__ __forceinline__ bool far_inside(double v) { return v > 0x1p-60 && v < 0x1p60; }

// The lane's share of a row's sum of squares.
template <int G, class E, int V, class Squares>
__device__ __forceinline__ double lane_squares(const Chunk<E, V> (&h)[HELD], int K, int lane, int nc,
                                               Squares&& squares) {
  double sq = 0.0;
#pragma unroll
  for (int i = 0; i < HELD; ++i) {
    const int c = lane + i * G;
    if (c < nc) sq += squares(without_first(h[i], c * V - chunk_at<V>(c, K)));
  }
  return sq;
}
template <int G, class E, int V>
__device__ __forceinline__ double lane_squares(const Chunk<E, V> (&h)[HELD], int K, int lane,
                                               int nc) {
  return lane_squares<G>(h, K, lane, nc, [](const Chunk<E, V>& c) { return chunk_squares(c); });
}
// 1 / sqrt(mean of the squares + eps), sq their sum (summed again where fp32 may have lost some).
template <int G, class E, int V>
__device__ __forceinline__ double row_factor(const Chunk<E, V> (&h)[HELD], double& sq, int K,
                                             float eps, int lane, int nc, double* s_part) {
  if (sizeof(E) == 2 && !far_inside(sq))
    sq = row_sum<G>(lane_squares<G>(h, K, lane, nc,
                                    [](const Chunk<E, V>& c) { return chunk_squares_f64(c); }),
                    s_part);
  return rsqrt(sq / K + (double)eps);
}

// A number's exponent, from 0 (zero) to 2047; 1023 from one to two.
__device__ __forceinline__ uint32_t exponent(double v) {
  return (uint32_t)(__builtin_bit_cast(uint64_t, v) >> 52) & 0x7ff;
}
// Whether a row's dot in fp32 has lost something that dx would show (fp16's never has).  Beside 2^-100
// terms below fp32's normal numbers are nothing; below 2^100 no term left the range (the dot would be
// infinite or NaN), nor does n mean(w dy n), n up to 128.  Where all terms are lost, below 2^-150, dx is
// off by up to 128 q^2 2^-150: nothing beside its normal numbers up to q = 2^8, nor in a row of zeros.
template <class E>
__device__ __forceinline__ bool dot_lost(double dot, double sq, double q) {
  if (__is_same(E, fp16_t) || exponent(dot) - (1023 - 100) < 200u) return false;
  return dot != 0.0 || (q >= 0x1p8 && sq > 0.0);
}
// 2^e, or the power of two of fp32's normal numbers that is nearest to it.
__device__ __forceinline__ float power_of_two(int e) {
  return __uint_as_float((uint32_t)(min(max(e, -126), 127) + 127) << 23);
}

// The exact code of p beside the row's largest magnitude m: p and m are products of two numbers of 24
// bits and exact in 64; the quotient's rounding is that of 64 bits.
__device__ __forceinline__ uint32_t code_f64(double p, double m) {
  return __float_as_uint((float)rint(127.0 * p / m) + 12582912.0f);
}

// Codes of a chunk of p = h w.  Where the largest |p| is far inside fp32's range (`plain`):
// 16-bit types have their products exact in fp32, and those of bf16 have 16 bits, so that 127 p is
// exact too and quant_bits' 16-bit form holds: a quotient 127 P 2^e / M that is no tie (P and M of 16
// bits) is 2^e / 2^17 from one at least, and the corrected quotient is right to half a step, below
// 2^(e - 18) where P <= M, and for e < 0 (P up to 2 M) 2^(e - 17) beside 2^e / 2^16.  fp32
// products have 48 bits: the fp32 quotient, off by less than 127 * 2^-21, decides unless it is within
// 2^-12 of a tie, and 64 bits do there.
template <class E, int V>
__device__ __forceinline__ Codes<E, V> norm_codes(const Chunk<E, V>& h, const Chunk<E, V>& w,
                                                  const RowQuant& r, double m, bool plain) {
  Codes<E, V> o;
  uint32_t b[V];
  if (plain) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float hf = to_f32(h.e[i]), wf = to_f32(w.e[i]);
      if constexpr (__is_same(E, bf16_t)) {
        b[i] = quant_bits<bf16_t>(hf * wf, r);
      } else if constexpr (sizeof(E) == 2) {
        b[i] = quant_bits<float>(hf * wf, r);
      } else {
        const float q = r.k * (hf * wf) * r.inv, n = rintf(q);
        b[i] = __float_as_uint(n + 12582912.0f);
        if (fabsf(q - n) > 0.5f - 0x1p-12f) b[i] = code_f64((double)hf * (double)wf, m);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] = code_f64((double)to_f32(h.e[i]) * (double)to_f32(w.e[i]), m);
  }
  if constexpr (V == 1) {
    o.w[0] = r.live ? b[0] : 0u;
  } else {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const uint32_t lo = __builtin_amdgcn_perm(b[4 * i + 1], b[4 * i], 0x0c0c0400u);
      const uint32_t hi = __builtin_amdgcn_perm(b[4 * i + 3], b[4 * i + 2], 0x04000c0cu);
      o.w[i] = r.live ? lo | hi : 0u;
    }
  }
  return o;
}

// The row's largest |h w|, exactly: of fp32 products' maximum (whose rounding keeps their order) those
// that round to it decide in 64 bits; where fp32 may have lost some (or w holds what is no number),
// all.  plain: fp32 has lost none that matters.
template <int G, class E, int V>
__device__ __forceinline__ double row_largest(const Chunk<E, V> (&h)[HELD],
                                              const Chunk<E, V> (&w)[HELD], bool finite, int lane,
                                              int nc, float* s_f32, double* s_f64, bool& plain) {
  float m32 = 0.f;
#pragma unroll
  for (int i = 0; i < HELD; ++i)
    if (lane + i * G < nc)
#pragma unroll
      for (int e = 0; e < V; ++e) m32 = fmaxf(m32, fabsf(to_f32(h[i].e[e]) * to_f32(w[i].e[e])));
  m32 = row_max<G>(m32, s_f32);
  plain = finite && far_inside(m32);
  if (sizeof(E) == 2 && plain) return m32;
  double m = 0.0;
#pragma unroll
  for (int i = 0; i < HELD; ++i)
    if (lane + i * G < nc)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float hf = to_f32(h[i].e[e]), wf = to_f32(w[i].e[e]);
        if (!plain || fabsf(hf * wf) == m32) m = max_nan(m, fabs((double)hf * (double)wf));
      }
  return row_max<G>(m, s_f64);
}

// Keeps the compiler from holding what it derived from a chunk (twice its registers) for later.
template <class E, int V>
__device__ __forceinline__ void forget_derived(Chunk<E, V>& c) {
  if constexpr (V > 1) asm volatile("" : "+v"(c.q));
}

// 16384 rows of 2048 bf16, all four matrices and codes: 57 us, 5.3 TB/s, a plain copy's rate (65 us
// without streaming; 95 with the sums and products element by element in 64 bits and twice the
// registers).
template <class E, int V, int G, bool STREAM>
__global__ __launch_bounds__(norm_threads(G), 4 * 256 / norm_threads(G))
void norm_rows_kernel(NormArgs a) {
  constexpr int THR = norm_threads(G), ROWS = THR / G;
  __shared__ double s_sum[THR / 64], s_max[THR / 64];
  __shared__ float s_max32[THR / 64];
  const int lane = threadIdx.x % G;
  const int nc = chunk_count<V>(a.K);
  Chunk<E, V> w[HELD];
  float w_max = 0.f;
#pragma unroll
  for (int i = 0; i < HELD; ++i)
    if (lane + i * G < nc) {
      w[i] = load_chunk<V>((const E*)a.w + chunk_at<V>(lane + i * G, a.K));
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float f = to_f32(w[i].e[e]);
        w_max = f - f == 0.f ? w_max : 1.f;
      }
    }
  const bool w_finite = a.codes && row_max<G>(w_max, s_max32) == 0.f;
  for (int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / G; row < a.M;
       row += (int64_t)gridDim.x * ROWS) {
    const E* const x = (const E*)a.x + row * a.xs;
    Chunk<E, V> h[HELD];
#pragma unroll
    for (int i = 0; i < HELD; ++i)
      if (lane + i * G < nc) h[i] = load_chunk<V, STREAM>(x + chunk_at<V>(lane + i * G, a.K));
    if (a.res) {
      const E* const res = (const E*)a.res + row * a.res_s;
      Chunk<E, V> r[HELD];
#pragma unroll
      for (int i = 0; i < HELD; ++i)
        if (lane + i * G < nc) r[i] = load_chunk<V, STREAM>(res + chunk_at<V>(lane + i * G, a.K));
#pragma unroll
      for (int i = 0; i < HELD; ++i) {
        float f[V];
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] = to_f32(h[i].e[e]) + to_f32(r[i].e[e]);
        h[i] = round_chunk<E, V>(f);
      }
    }
    double sq = row_sum<G>(lane_squares<G>(h, a.K, lane, nc), s_sum);
    const double q = row_factor<G>(h, sq, a.K, a.eps, lane, nc, s_sum);
    const float qf = (float)q;
    // every lane has read its part of the row (it may be overwritten now)
    if (a.sum) {
      E* const sum = (E*)a.sum + row * a.sum_s;
#pragma unroll
      for (int i = 0; i < HELD; ++i)
        if (lane + i * G < nc) store_chunk<STREAM>(sum + chunk_at<V>(lane + i * G, a.K), h[i]);
    }
    if (a.y) {
      E* const y = (E*)a.y + row * a.ys;
#pragma unroll
      for (int i = 0; i < HELD; ++i) {
        if (lane + i * G >= nc) continue;
        forget_derived(h[i]);
        forget_derived(w[i]);
        float f[V];
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] = to_f32(h[i].e[e]) * qf * to_f32(w[i].e[e]);
        store_chunk<STREAM>(y + chunk_at<V>(lane + i * G, a.K), round_chunk<E, V>(f));
      }
    }
    if (a.codes) {
#pragma unroll
      for (int i = 0; i < HELD; ++i) forget_derived(h[i]), forget_derived(w[i]);
      bool plain;
      const double m = row_largest<G>(h, w, w_finite && q > 0.0, lane, nc, s_max32, s_max, plain);
      RowQuant r = row_quant(__float_as_uint((float)m));
      r.live = m > 0.0 && m < __builtin_inf();
      int8_t* const codes = a.codes + row * a.cs;
#pragma unroll
      for (int i = 0; i < HELD; ++i) {
        if (lane + i * G >= nc) continue;
        forget_derived(h[i]);
        forget_derived(w[i]);
        store_codes<STREAM>(codes + chunk_at<V>(lane + i * G, a.K), norm_codes(h[i], w[i], r, m, plain));
      }
      if (lane == 0)
        a.scale[row] = m < __builtin_inf() ? (float)(m * q / 127.0) : __uint_as_float(0x7fc00000u);
    }
  }
}

struct NormGradArgs {
  const void* dy;
  int64_t dys;
  const void* dsum;  // may be null
  int64_t dsum_s;
  const void* h;
  int64_t hs;
  int M, K;
  const void* w;
  float eps;
  void* dx;  // may be null, dy, dsum or h
  int64_t dxs;
  float* part;  // [workgroups][K] sums of q dy h over a workgroup's rows; null: no dweight
};

// dx of the workgroup's rows, one after the other, and the part of dw that they give: each lane adds up
// its own columns in fp32 over its rows, the row groups of the workgroup are joined in LDS.  The
// registers allow two waves a SIMD, so the next row is under way while one is worked on (16384 rows of
// 2048 bf16 with dsum: 59 us without, 48 with, 5.6 TB/s; three waves with spills 92).  A row whose
// products h w dy leave fp32's range is summed again in 64 bits, w dy beside a power of two; looking for
// such rows costs half a microsecond of that, in fp32 (8192 such rows) 1 of 45.
template <class E, int V, int G, bool STREAM>
__global__ __launch_bounds__(norm_threads(G), 2)
void norm_rows_grad_kernel(NormGradArgs a) {
  constexpr int THR = norm_threads(G), ROWS = THR / G;
  __shared__ double s_part[THR / 64], s_both[THR / 64][2];
  __shared__ float s_big[THR / 64];
  constexpr bool AHEAD = THR < 1024;  // a thousand threads have no registers for it
  extern __shared__ __align__(16) float s_dw[];  // [ROWS][K], where ROWS > 1
  const int lane = threadIdx.x % G, group = threadIdx.x / G;
  const int nc = chunk_count<V>(a.K);
  Chunk<E, V> w[HELD];
  float dw[HELD][V];
#pragma unroll
  for (int i = 0; i < HELD; ++i) {
    if (lane + i * G < nc) w[i] = load_chunk<V>((const E*)a.w + chunk_at<V>(lane + i * G, a.K));
#pragma unroll
    for (int e = 0; e < V; ++e) dw[i][e] = 0.f;
  }
  const auto load = [&](int64_t row, Chunk<E, V>(&h)[HELD], Chunk<E, V>(&g)[HELD],
                        Chunk<E, V>(&d)[HELD]) {
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      if (lane + i * G >= nc) continue;
      const int at = chunk_at<V>(lane + i * G, a.K);
      h[i] = load_chunk<V, STREAM>((const E*)a.h + row * a.hs + at);
      g[i] = load_chunk<V, STREAM>((const E*)a.dy + row * a.dys + at);
      if (a.dsum && a.dx) d[i] = load_chunk<V, STREAM>((const E*)a.dsum + row * a.dsum_s + at);
    }
  };
  const int64_t step = (int64_t)gridDim.x * ROWS;
  Chunk<E, V> h[HELD], g[HELD], d[HELD], next_h[HELD], next_g[HELD], next_d[HELD];
  int64_t row = (int64_t)blockIdx.x * ROWS + group;
  if (AHEAD && row < a.M) load(row, next_h, next_g, next_d);
  for (; row < a.M; row += step) {
    if constexpr (AHEAD) {
#pragma unroll
      for (int i = 0; i < HELD; ++i) h[i] = next_h[i], g[i] = next_g[i], d[i] = next_d[i];
      if (row + step < a.M) load(row + step, next_h, next_g, next_d);
    } else {
      load(row, h, g, d);
    }
    double dot = 0.0;
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      const int c = lane + i * G;
      if (c >= nc) continue;
      const Chunk<E, V> once = without_first(h[i], c * V - chunk_at<V>(c, a.K));
      float part = 0.f;
#pragma unroll
      for (int e = 0; e < V; ++e)
        part = fmaf(to_f32(once.e[e]), to_f32(w[i].e[e]) * to_f32(g[i].e[e]), part);
      dot += part;
    }
    double sq = lane_squares<G>(h, a.K, lane, nc);
    row_sums<G>(sq, dot, s_both);
    const double q = row_factor<G>(h, sq, a.K, a.eps, lane, nc, s_part);
    const float qf = (float)q;
    float by = 1.f, qb = qf;  // a power of two that brings w dy into fp32's range, and q / by
    const bool far = dot_lost<E>(dot, sq, q);
    if (far) {
      dot = 0.0;
      int big = 0;
#pragma unroll
      for (int i = 0; i < HELD; ++i) {
        const int c = lane + i * G;
        if (c >= nc) continue;
        forget_derived(h[i]);
        forget_derived(g[i]);
        forget_derived(w[i]);
        const int had = c * V - chunk_at<V>(c, a.K);  // elements that the chunk before has
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const double wg = (double)to_f32(w[i].e[e]) * (double)to_f32(g[i].e[e]);
          dot = fma((double)to_f32(h[i].e[e]), e < had ? 0.0 : wg, dot);
          big = max(big, (int)exponent(wg));
        }
      }
      dot = row_sum<G>(dot, s_part);
      big = (int)row_max<G>((float)big, s_big);
      by = big > 0 ? power_of_two(1023 - big) : 1.f;
      qb = (float)(q / by);
      dot *= by;
    }
    const float along = (float)(q * dot / a.K);  // mean of w dy (q h)
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      if (lane + i * G >= nc) continue;
      forget_derived(h[i]);
      forget_derived(g[i]);
      forget_derived(w[i]);
      float f[V];
      if (far) {
#pragma unroll
        for (int e = 0; e < V; ++e)
          f[e] = (float)((double)to_f32(w[i].e[e]) * (double)to_f32(g[i].e[e]) * (double)by);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] = to_f32(w[i].e[e]) * to_f32(g[i].e[e]);
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float n = to_f32(h[i].e[e]) * qf;
        dw[i][e] = fmaf(to_f32(g[i].e[e]), n, dw[i][e]);
        const float own = a.dsum ? to_f32(d[i].e[e]) : 0.f;
        f[e] = fmaf(qb, fmaf(-n, along, f[e]), own);
      }
      if (a.dx)
        store_chunk<STREAM>((E*)a.dx + row * a.dxs + chunk_at<V>(lane + i * G, a.K),
                    round_chunk<E, V>(f));
    }
  }
  if (!a.part) return;
  float* const part = a.part + (int64_t)blockIdx.x * a.K;
  float* const own = ROWS > 1 ? s_dw + group * a.K : part;
#pragma unroll
  for (int i = 0; i < HELD; ++i) {
    if (lane + i * G >= nc) continue;
    const int at = chunk_at<V>(lane + i * G, a.K);
#pragma unroll
    for (int e = 0; e < V; ++e) own[at + e] = dw[i][e];  // an overlap twice, with the same value
  }
  if constexpr (ROWS > 1) {
    __syncthreads();
    for (int k = threadIdx.x; k < a.K; k += THR) {
      float sum = 0.f;
#pragma unroll
      for (int r = 0; r < ROWS; ++r) sum += s_dw[r * a.K + k];
      part[k] = sum;
    }
  }
}

// dw[k] = sum of the workgroups' parts, in 64 bits: a workgroup takes 32 columns, each of its 32 half
// waves a share of the parts.  parts = 0: zeros.
constexpr int PART_COLS = 32, PART_SHARES = 32;
__global__ __launch_bounds__(PART_COLS * PART_SHARES) void norm_rows_parts_kernel(
    const float* part, int parts, int K, float* dw) {
  __shared__ double s_sum[PART_SHARES][PART_COLS];
  const int col = threadIdx.x % PART_COLS, share = threadIdx.x / PART_COLS;
  const int k = blockIdx.x * PART_COLS + col;
  double sum = 0.0;
  if (k < K) {
#pragma unroll 8
    for (int p = share; p < parts; p += PART_SHARES) sum += part[(int64_t)p * K + k];
  }
  s_sum[share][col] = sum;
  __syncthreads();
  if (share == 0 && k < K) {
#pragma unroll
    for (int s = 1; s < PART_SHARES; ++s) sum += s_sum[s][col];
    dw[k] = (float)sum;
  }
}

// ------------------------------------------------------------------ host side

// As few lanes per row as hold it: f(elements of a chunk, lanes).
template <int N>
using Int = std::integral_constant<int, N>;
template <class E, class F>
auto by_width(int K, F&& f) {
  constexpr int V = kChunk<E>;
  const int nc = chunk_count<V>(K);
  if (K < V) return f(Int<1>{}, Int<16>{});
  if (nc <= 16 * HELD) return f(Int<V>{}, Int<16>{});
  if (nc <= 32 * HELD) return f(Int<V>{}, Int<32>{});
  if (nc <= 64 * HELD) return f(Int<V>{}, Int<64>{});
  if (nc <= 256 * HELD) return f(Int<V>{}, Int<256>{});
  return f(Int<V>{}, Int<kMaxNormCols / V / HELD>{});
}

// Workgroups of a launch over M rows, `rows` at a time each.
int norm_grid(int M, int rows, int most) { return std::min((M + rows - 1) / rows, most); }

// Every row of an output (if there is one) starts with half a line.
bool starts_half_line(const void* out, int64_t row_bytes) {
  return !out || ((uintptr_t)out % 64 == 0 && row_bytes % 64 == 0);
}

template <class E>
hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
  return by_width<E>(a.K, [&](auto v, auto g) {
    constexpr int V = decltype(v)::value, G = decltype(g)::value, THR = norm_threads(G);
    const int64_t row = (int64_t)sizeof(E) * (1 + !!a.res + !!a.sum + !!a.y) + !!a.codes;
    const bool starts = starts_half_line(a.sum, a.sum_s * (int64_t)sizeof(E)) &&
                        starts_half_line(a.y, a.ys * (int64_t)sizeof(E)) &&
                        (G > 16 || starts_half_line(a.codes, a.cs));
    const bool stream = row * a.K * a.M > kNormStreamBytes && (G > 32 || starts);
    // rows below 16 bytes are never streamed: their kernel is bound by their number
    const auto kernel = V > 1 && stream ? norm_rows_kernel<E, V, G, V != 1>
                                        : norm_rows_kernel<E, V, G, false>;
    return launch_kernel(kernel, dim3((unsigned)norm_grid(a.M, THR / G, 256 * 8)), dim3(THR), 0, s,
                         a);
  });
}

// Parts of dw (workgroups of the gradient's launch): as many as the CUs hold at once, and so many that a
// lane adds up no more than kPartRows rows in fp32.
constexpr int kMaxParts = 512, kPartRows = 256;
template <class E>
int grad_parts(int M, int K) {
  return by_width<E>(K, [&](auto, auto g) {
    constexpr int G = decltype(g)::value, ROWS = norm_threads(G) / G;
    const int few = (M + ROWS * kPartRows - 1) / (ROWS * kPartRows);
    return norm_grid(M, ROWS, std::max(few, G > 256 ? 256 : kMaxParts));
  });
}

template <class E>
hipError_t launch_norm_grad(NormGradArgs& a, float* dweight, float* ws, hipStream_t s) {
  const int parts = grad_parts<E>(a.M, a.K);
  if (dweight) a.part = parts == 1 ? dweight : ws;
  hipError_t e = hipSuccess;
  if (parts > 0)
    e = by_width<E>(a.K, [&](auto v, auto g) {
      constexpr int V = decltype(v)::value, G = decltype(g)::value, THR = norm_threads(G);
      const size_t lds = THR > G && dweight ? sizeof(float) * (THR / G) * a.K : 0;
      const int64_t row = (int64_t)sizeof(E) * (2 + !!a.dsum + !!a.dx);
      const bool stream = row * a.K * a.M > kNormStreamBytes;
      const auto kernel = V > 1 && stream ? norm_rows_grad_kernel<E, V, G, V != 1>
                                          : norm_rows_grad_kernel<E, V, G, false>;
      return launch_kernel(kernel, dim3((unsigned)parts), dim3(THR), lds, s, a);
    });
  if (e != hipSuccess || !dweight || parts == 1) return e;
  return launch_kernel(norm_rows_parts_kernel, dim3((unsigned)((a.K + PART_COLS - 1) / PART_COLS)),
                       dim3(PART_COLS * PART_SHARES), 0, s, (const float*)ws, parts, a.K, dweight);
}

bool norm_ok(int type, int M, int K, float eps) {
  return float_type(type) && M >= 0 && M <= kMaxRows && K >= 1 && K <= kMaxNormCols && eps > 0.f &&
         eps < __builtin_inff();
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_norm_rows(const void* x, int64_t x_stride, const void* residual,
                         int64_t residual_stride, int32_t type, int32_t M, int32_t K,
                         const void* weight, float eps, void* sum, int64_t sum_stride, void* y,
                         int64_t y_stride, int8_t* codes, int64_t codes_stride, float* scale,
                         void* stream) {
  if (!norm_ok(type, M, K, eps)) return MOE_E_INVALID;
  if (M == 0) return MOE_OK;  // before the pointers: empty buffers have none
  if (!rows_ok(x, x_stride, K, type) || !rows_ok(weight, K, K, type) ||
      (residual && !rows_ok(residual, residual_stride, K, type)) || (!y && !codes) ||
      (sum && (!residual || !rows_ok(sum, sum_stride, K, type))) ||
      (y && !rows_ok(y, y_stride, K, type)) ||
      (codes && (!rows_ok(codes, codes_stride, K, MOE_T_I8) || !scale || !aligned4(scale))) ||
      (sum && sum == y) || !same_rows(sum, sum_stride, x, x_stride) ||
      !same_rows(sum, sum_stride, residual, residual_stride) ||
      !same_rows(y, y_stride, x, x_stride) ||
      !same_rows(y, y_stride, residual, residual_stride) || !on_current_device(x))
    return MOE_E_INVALID;
  NormArgs a{x,   x_stride,   residual, residual_stride, M,     K,            weight, eps,
             sum, sum_stride, y,        y_stride,        codes, codes_stride, scale};
  const hipStream_t s = (hipStream_t)stream;
  if (type == MOE_T_BF16) return launched(launch_norm<bf16_t>(a, s));
  if (type == MOE_T_FP16) return launched(launch_norm<fp16_t>(a, s));
  return launched(launch_norm<float>(a, s));
}

size_t moe_norm_grad_workspace_bytes(int32_t M, int32_t K) {
  if (!norm_ok(MOE_T_FP32, M, K, 1.f)) return 0;
  const int parts = std::max(grad_parts<float>(M, K), grad_parts<bf16_t>(M, K));
  return parts > 1 ? sizeof(float) * (size_t)parts * (size_t)K : 0;
}

moe_status moe_norm_rows_grad(const void* dy, int64_t dy_stride, const void* dsum,
                              int64_t dsum_stride, const void* sum, int64_t sum_stride,
                              int32_t type, int32_t M, int32_t K, const void* weight, float eps,
                              void* dx, int64_t dx_stride, float* dweight, void* workspace,
                              size_t workspace_bytes, void* stream) {
  if (!norm_ok(type, M, K, eps) || !aligned4(dweight)) return MOE_E_INVALID;
  if (M == 0 && !dweight) return MOE_OK;
  if (M > 0 && (!rows_ok(dy, dy_stride, K, type) || !rows_ok(sum, sum_stride, K, type) ||
                !rows_ok(weight, K, K, type) || (!dx && !dweight) ||
                (dsum && !rows_ok(dsum, dsum_stride, K, type)) ||
                (dx && !rows_ok(dx, dx_stride, K, type)) ||
                !same_rows(dx, dx_stride, dy, dy_stride) ||
                !same_rows(dx, dx_stride, dsum, dsum_stride) ||
                !same_rows(dx, dx_stride, sum, sum_stride)))
    return MOE_E_INVALID;
  const size_t need = dweight ? moe_norm_grad_workspace_bytes(M, K) : 0;
  if (need && (!workspace || !aligned4(workspace))) return MOE_E_INVALID;
  if (workspace_bytes < need) return MOE_E_SCRATCH;
  if (!on_current_device(M > 0 ? dy : dweight)) return MOE_E_INVALID;
  NormGradArgs a{dy, dy_stride, dsum, dsum_stride, sum, sum_stride, M, K, weight, eps,
                 dx, dx_stride, nullptr};
  const hipStream_t s = (hipStream_t)stream;
  float* const ws = (float*)workspace;
  if (type == MOE_T_BF16) return launched(launch_norm_grad<bf16_t>(a, dweight, ws, s));
  if (type == MOE_T_FP16) return launched(launch_norm_grad<fp16_t>(a, dweight, ws, s));
  return launched(launch_norm_grad<float>(a, dweight, ws, s));
}

}  // extern "C"
