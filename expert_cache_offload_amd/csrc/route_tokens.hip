// Experts and routing weights of tokens from their logits, and the gradient for the logits.
//
// Scores s = softmax(z) or 1 / (1 + exp(-z)); an expert is chosen by its choice value, c = s + bias or,
// without a bias, z itself (which orders the scores).  Of G groups of neighbouring experts the best
// `kept` by the sum of their one or two largest choice values (scores without a bias) stay;
// of their experts the k largest c are chosen, ties to the lower id.  Weights: s of the chosen,
// divided by their sum or not, times a factor.
//
// A lane holds neighbouring experts.  Up to 512 experts and 15 choices four tokens share a wave, 16
// lanes each: one read of the logits, k + 2 rounds of a maximum over the lanes on keys that hold the
// expert's id.  Other sizes, and tokens that these keys cannot decide, take a wave each, in which the
// first lane of a ballot has the lowest id among equal values.  Both are bound by instructions, not by
// bytes: 16384 tokens of 128 bf16 logits and 8 choices 6.9 us (560 vector instructions for four tokens, 3.7
// us of the SIMDs' time, behind the launch and the read), of 256 fp32 logits with a bias 14 in groups;
// a wave to a token, of 256 with 16 choices 34, of 1024 with 8 choices 89.
#include <algorithm>

#include "row_ops.h"

namespace moe {
namespace {

constexpr int RT_T = 256;  // threads of a workgroup
constexpr int kMaxChoices = 16;
constexpr int kMaxRouted = 1024;
constexpr int kMaxRouteGroups = 64;
constexpr int kMaxRouteT = 1 << 20;

struct RouteArgs {
  const void* z;
  int64_t zs;
  int T, E, score;
  const float* bias;  // may be null
  int G, best, kept, k, renorm;
  float scale;
  int* idx;
  float* w;
};

// Keys that order as numbers do (without NaN); 0 is below every number's.
__device__ __forceinline__ uint32_t key_of(float f) {
  const uint32_t b = __float_as_uint(f + 0.f);  // -0 as 0
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ uint64_t key_of(double f) {
  const uint64_t b = __builtin_bit_cast(uint64_t, f + 0.0);
  return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}

// The wave's largest, in every lane (an SGPR).
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  const auto with = [&](uint32_t o) { v = v > o ? v : o; };
  with(__builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false));  // row_shr:1, 2, 4, 8
  with(__builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false));
  with(__builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false));
  with(__builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false));
  with(__builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false));  // row_bcast:15, 31
  with(__builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false));
  return __builtin_amdgcn_readlane(v, 63);
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
  const uint32_t hi = wave_max((uint32_t)(v >> 32));
  const uint32_t lo = wave_max((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return (uint64_t)hi << 32 | lo;
}
// Over W neighbouring lanes (16 or 64), in all of them.
template <int W, class T, class Join>
__device__ __forceinline__ T join_lanes(T v, Join&& join) {
  v = join16(v, join);
#pragma unroll
  for (int s = 16; s < W; s <<= 1) v = join(v, __shfl_xor(v, s));
  return v;
}
template <int W, class R>
__device__ __forceinline__ R sum_lanes(R v) {
  return join_lanes<W>(v, [](R a, R b) { return a + b; });
}
template <int W>
__device__ __forceinline__ float max_lanes(float v) {
  return join_lanes<W>(v, [](float a, float b) { return fmaxf(a, b); });
}

__device__ __forceinline__ float exp_fast(float x) {
  return __builtin_amdgcn_exp2f(x * 1.44269504f);
}
__device__ __forceinline__ double exp_fast(double x) { return exp(x); }
__device__ __forceinline__ float inverse(float x) { return __builtin_amdgcn_rcpf(x); }
__device__ __forceinline__ double inverse(double x) { return 1.0 / x; }

// Scores of the lane's experts (zmax: the largest logit, of softmax).
template <class R, int NPL>
__device__ __forceinline__ void route_scores(R (&s)[NPL], const float (&z)[NPL], int score,
                                             float zmax) {
  if (score == MOE_SCORE_SOFTMAX) {
    R sum = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      s[i] = exp_fast((R)z[i] - (R)zmax);
      sum += s[i];
    }
    const R inv = inverse(sum_lanes<64>(sum));
#pragma unroll
    for (int i = 0; i < NPL; ++i) s[i] *= inv;
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i) s[i] = inverse((R)1 + exp_fast(-(R)z[i]));
  }
}

// What a fp32 choice value may be off by, in units of 1 + |c|.  exp's argument x is off by 1.5 |x| 2^-24
// (2.5 below the row's largest), exp and the reciprocal by 2^-23 of themselves.  A sigmoid's
// s (1 - s) |x| and s (1 - s) stay below 1 / 4, so it is off by less than 2^-22; softmax has its sum in
// fp32 over up to 22 additions in sequence, less than 2^-19, or in 64 bits, less than 2^-21.  The
// bias' addition adds half a step of c.
__device__ __forceinline__ float error_unit(int score, bool sum_f64) {
  return score == MOE_SCORE_SIGMOID ? 0x1p-22f : sum_f64 ? 0x1p-21f : 0x1p-19f;
}

struct Chosen {
  int idx;    // of lane j: choice j (j < found)
  int found;  // uniform
  bool sure;  // fp32: no two values that decide are closer than their errors
};

// Groups kept, as bits at each group's first lane: 64 / G2 lanes share a group, G2 = 2^g_log >= G.
// c: [E] in LDS, -inf where an expert is not to be had.
template <class R>
__device__ __forceinline__ uint64_t kept_groups(const R* c, int E, int G, int g_log, int best,
                                                int kept, int lane, float unit, bool& sure) {
  const R none = -__builtin_inff();
  const int per = 64 >> g_log, g = lane / per, size = E / G;
  R m1 = none, m2 = none;
  if (g < G)
    for (int t = lane % per; t < size; t += per) {
      const R v = c[g * size + t];
      m2 = v > m1 ? m1 : v > m2 ? v : m2;
      m1 = v > m1 ? v : m1;
    }
  for (int s = 1; s < per; s <<= 1) {
    const R o1 = __shfl_xor(m1, s), o2 = __shfl_xor(m2, s);
    const R low = m1 < o1 ? m1 : o1, up = m2 > o2 ? m2 : o2;
    m1 = m1 > o1 ? m1 : o1;
    m2 = low > up ? low : up;
  }
  R value = m1;
  if (best == 2 && m2 > none) value += m2;
  int rank = 0;
  for (int o = 0; o < G; ++o) {
    const R other = __shfl(value, o * per);
    rank += other > value || (other == value && o < g);
  }
  const bool keep = g < G && rank < kept;
  if constexpr (sizeof(R) == 4) {
    float off = m1 > none ? unit * (1.f + fabsf(m1)) : 0.f;
    if (best == 2 && m2 > none) off += unit * (1.f + fabsf(m2));
    const float low = keep ? value - off : __builtin_inff();
    const float high = !keep && g < G ? value + off : none;
    const float worst = -max_lanes<64>(-low), next = max_lanes<64>(high);
    sure = kept >= G || worst > next;
  }
  return __ballot(keep && lane % per == 0);
}

// c: choice values, v: what groups are ranked by; out: experts that are not to be had.
template <class R, int NPL>
__device__ __forceinline__ Chosen choose(const RouteArgs& a, const R (&c)[NPL], const R (&v)[NPL],
                                         const bool (&out)[NPL], R* s_c, int g_log,
                                         const int (&group_lane)[NPL], int lane, bool check) {
  Chosen r{-1, 0, true};
  uint64_t groups = ~0ull;
  if (a.G > 1) {
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (lane * NPL + i < a.E) s_c[lane * NPL + i] = out[i] ? (R)-__builtin_inff() : v[i];
    asm volatile("" ::: "memory");  // a wave's LDS accesses run in order
    groups = kept_groups(s_c, a.E, a.G, g_log, a.best, a.kept, lane,
                         error_unit(a.score, false), r.sure);
    asm volatile("" ::: "memory");
  }
  using Key = decltype(key_of(R()));
  Key key[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i)
    key[i] = out[i] || !(groups >> group_lane[i] & 1) ? 0 : key_of(c[i]);
  Key own = 0, last = 0;
  for (int j = 0; j <= a.k; ++j) {
    Key m = key[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < NPL; ++i) {
      at = key[i] > m ? i : at;
      m = key[i] > m ? key[i] : m;
    }
    const Key top = wave_max(m);
    if (j == a.k || top == 0) {
      last = top;
      break;
    }
    const int win = __builtin_ctzll(__ballot(m == top));
    const int e = win * NPL + __builtin_amdgcn_readlane(at, win);
    if (lane == j) {
      r.idx = e;
      own = top;
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (lane * NPL + i == e) key[i] = 0;
    r.found = j + 1;
  }
  if constexpr (sizeof(R) == 4)
    if (check) {
      Key next = __shfl_down(own, 1);
      next = lane == r.found - 1 ? last : next;
      const float hi = value_of(own), lo = value_of(next);
      const bool open = lane < r.found && next != 0 &&
                        !(hi - lo > error_unit(a.score, false) * (2.f + fabsf(hi) + fabsf(lo)));
      r.sure = r.sure && __ballot(open) == 0;
    }
  return r;
}

template <class E, int NPL>
__device__ __forceinline__ void load_logits(float (&z)[NPL], const E* row, int lane, int n,
                                            float fill) {
#pragma unroll
  for (int i = 0; i < NPL; ++i) z[i] = fill;
  if (lane * NPL >= n) return;
  constexpr int B = NPL * (int)sizeof(E);
  if (lane * NPL + NPL <= n && B >= 4) {
    if constexpr (B >= 16) {
      constexpr int V = kChunk<E>;
#pragma unroll
      for (int q = 0; q < NPL / V; ++q) {
        const Chunk<E> c = load_chunk<V>(row + lane * NPL + q * V);
#pragma unroll
        for (int i = 0; i < V; ++i) z[q * V + i] = to_f32(c.e[i]);
      }
    } else if constexpr (B >= 4) {
      struct Part {
        E e[NPL];
      };
      typedef uint32_t part_t __attribute__((ext_vector_type(B / 4)));
      typedef part_t part_any __attribute__((aligned(1)));
      const Part p = __builtin_bit_cast(Part, (part_t) * (const part_any*)(row + lane * NPL));
#pragma unroll
      for (int i = 0; i < NPL; ++i) z[i] = to_f32(p.e[i]);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < NPL; ++i)
    if (lane * NPL + i < n) z[i] = to_f32(row[lane * NPL + i]);
}

// Sigmoid of a logit in 64 bits: for the chosen, which are few.
template <class E>
__device__ __forceinline__ double sigmoid_f64(E z) {
  return 1.0 / (1.0 + exp(-(double)z));
}

// Choice `lane` of a token (has: there is one), by 16 neighbouring lanes: its weight in 64 bits, the
// chosen being few.  zmax and sum: of softmax that is not renormalised.
template <class E>
__device__ __forceinline__ void write_choice(const RouteArgs& a, const E* row, int64_t at, int lane,
                                             bool has, int e, float zmax, double sum) {
  const float zc = has ? to_f32(row[e]) : -__builtin_inff();
  double w;
  if (a.score == MOE_SCORE_SOFTMAX) {
    const float top = a.renorm ? max_lanes<kMaxChoices>(zc) : zmax;
    w = has ? exp((double)zc - (double)top) : 0.0;
    if (a.renorm) sum = sum_lanes<kMaxChoices>(w);
    w /= sum;
  } else {
    w = has ? sigmoid_f64(zc) : 0.0;
    if (a.renorm) {
      sum = sum_lanes<kMaxChoices>(w);
      w = sum == 0.0 ? 0.0 : w / sum;
    }
  }
  if (lane < a.k) {
    a.idx[at] = has ? e : -1;
    a.w[at] = has ? (float)(w * (double)a.scale) : 0.f;
  }
}

// Choice values are scores (with a bias or not), not the logits alone.
__device__ __forceinline__ bool by_score(const RouteArgs& a) {
  return a.bias || (a.G > 1 && a.best == 2);
}

// Token t by a whole wave, each choice exact: fp32 (TRY) where no two values that decide are closer than
// their errors, else 64 bits.  s_choice: NPL * 64 numbers of the wave's own.
template <class E, int NPL, bool TRY>
__device__ void route_exact(const RouteArgs& a, int t, double* s_choice, int lane) {
  const float none = -__builtin_inff();
  const E* const row = (const E*)a.z + (int64_t)t * a.zs;
  int g_log = 0;
  while ((1 << g_log) < a.G) ++g_log;
  float z[NPL], bias[NPL], zmax = none;
  int group_lane[NPL];
  load_logits(z, row, lane, a.E, none);
  bool out[NPL], nan = false;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = lane * NPL + i;
    bias[i] = e >= a.E ? none : a.bias ? a.bias[e] : 0.f;
    group_lane[i] = a.G > 1 && e < a.E ? e / (a.E / a.G) * (64 >> g_log) : 0;
    out[i] = z[i] == none || bias[i] == none;
    zmax = fmaxf(zmax, z[i]);
    nan |= z[i] != z[i] && (!out[i] || a.score == MOE_SCORE_SOFTMAX);
    nan |= bias[i] != bias[i] && !out[i];
    nan |= z[i] == __builtin_inff() && a.score == MOE_SCORE_SOFTMAX;
  }
  const int64_t at = (int64_t)t * a.k + lane;
  if (__ballot(nan)) {
    if (lane < a.k) {
      a.idx[at] = lane;
      a.w[at] = __uint_as_float(0x7fc00000u);
    }
    return;
  }
  if (a.score == MOE_SCORE_SOFTMAX) zmax = max_lanes<64>(zmax);
  Chosen r;
  if (by_score(a)) {
    if constexpr (TRY) {
      float c[NPL], v[NPL];
      route_scores(v, z, a.score, zmax);
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        v[i] += bias[i];
        c[i] = a.bias ? v[i] : z[i];
      }
      r = choose(a, c, v, out, (float*)s_choice, g_log, group_lane, lane, a.bias != nullptr);
    }
    if (!TRY || !r.sure) {
      double cd[NPL], vd[NPL];
      route_scores(vd, z, a.score, zmax);
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        vd[i] += (double)bias[i];
        cd[i] = a.bias ? vd[i] : (double)z[i];
      }
      r = choose(a, cd, vd, out, s_choice, g_log, group_lane, lane, false);
    }
  } else {
    r = choose(a, z, z, out, (float*)s_choice, g_log, group_lane, lane, false);
  }
  double sum = 0.0;
  if (a.score == MOE_SCORE_SOFTMAX && !a.renorm) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) sum += exp((double)z[i] - (double)zmax);
    sum = sum_lanes<64>(sum);
  }
  const bool has = lane < r.found;
  write_choice(a, row, at, lane, has, r.idx, zmax, sum);
}

// A wave to every token, for sizes that the kernel below does not take.
template <class E, int NPL>
__global__ __launch_bounds__(RT_T) void route_tokens_wave_kernel(RouteArgs a) {
  __shared__ double s_choice[RT_T / 64][NPL * 64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int t = blockIdx.x * (RT_T / 64) + wave; t < a.T; t += gridDim.x * (RT_T / 64))
    route_exact<E, NPL, true>(a, t, s_choice[wave], lane);
}

// The nearest integer below, 0 for what is negative or no number.
__device__ __forceinline__ uint32_t steps_of(float f) {
  uint32_t u;
  asm("v_cvt_u32_f32 %0, %1" : "=v"(u) : "v"(f));
  return u;
}

// Four neighbouring elements of a row (the experts are a multiple of four and four of them a piece
// of 8 or 16 bytes), or those that there are.
template <class E>
__device__ __forceinline__ void load_four(float* f, const E* p, int n, bool fours, float fill) {
  if (fours) {
    typedef uint32_t part_t __attribute__((ext_vector_type(sizeof(E))));
    typedef part_t part_any __attribute__((aligned(1)));
    struct Part {
      E e[4];
    };
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = fill;
    if (n > 0) {
      const Part q = __builtin_bit_cast(Part, (part_t) * (const part_any*)p);
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = to_f32(q.e[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = j < n ? to_f32(p[j]) : fill;
  }
}

// Rank among the G groups of a token's 16 lanes, group_lanes each, by their one or two largest values:
// of this lane's group.  m1 >= m2: the lane's own two largest.
template <class R>
__device__ __forceinline__ int group_rank(R& m1, R& m2, const RouteArgs& a, int group_lanes,
                                          int lane) {
  const R none = -__builtin_inff();
  for (int s = 1; s < group_lanes; s <<= 1) {
    const R o1 = __shfl_xor(m1, s), o2 = __shfl_xor(m2, s);
    const R low = m1 < o1 ? m1 : o1, up = m2 > o2 ? m2 : o2;
    m1 = m1 > o1 ? m1 : o1;
    m2 = low > up ? low : up;
  }
  const R value = a.best == 2 && m2 > none ? m1 + m2 : m1;
  const int g = (lane & 15) / group_lanes;
  int rank = 0;
  for (int o = 0; o < a.G; ++o) {
    const R other = __shfl(value, (lane & 48) + o * group_lanes);
    rank += other > value || (other == value && o < g);
  }
  return rank;
}

// A choice value in 64 bits (zmax, sum: of softmax).
__device__ __forceinline__ double choice_f64(const RouteArgs& a, float z, int e, float zmax,
                                             double sum) {
  const double s = a.score == MOE_SCORE_SOFTMAX ? exp((double)z - (double)zmax) / sum
                                                : sigmoid_f64(z);
  return s + (a.bias ? (double)a.bias[e] : 0.0);
}

// Four tokens to a wave, 16 lanes each, a lane with n_lane (up to NE, a multiple of 4) neighbouring
// experts.  A choice value becomes a number of up to 31 bits with the expert's id, inverted, in the
// low ones: keys are distinct, the largest is the best choice, the next the largest below it, which
// is the largest of key - last in 32 bits' arithmetic (keys above wrap to the lower half).
// 16-bit logits go in whole and are exact.  Others go in as fixed-point distances from the row's
// largest; where some of the k + 1 best are equal or, of scores, too close, these are ranked in 64
// bits, and so are groups that are too close.  What else may be wrong (the border among more than two
// experts, NaN, fewer experts than choices) is left to route_exact.
template <class E, int NE>
__global__ __launch_bounds__(RT_T) void route_tokens_kernel(RouteArgs a, int n_lane, int id_bits,
                                                            int group_lanes) {
  constexpr int NPL = NE / 4;
  // fixed point: with 9 bits of an id below 2^31; the largest is kTop, whose rounding leaves it inside
  constexpr float kTop = (1 << 22) - (1 << 12);
  __shared__ double s_choice[RT_T / 64][NPL * 64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l = lane & 15;
  const float none = -__builtin_inff(), inf = __builtin_inff();
  const bool scores = by_score(a), whole = sizeof(E) == 2 && !a.bias, fours = a.E % 4 == 0;
  const uint32_t id_mask = (1u << id_bits) - 1;
  const int first = l * n_lane, mine = min(n_lane, a.E - first);  // this lane's experts
  const int t = (blockIdx.x * (RT_T / 64) + wave) * 4 + (lane >> 4);
  const E* const row = (const E*)a.z + (int64_t)min(t, a.T - 1) * a.zs;
  float z[NE], v[NE];  // logits; scores, with the bias
  uint32_t key[NE];
#pragma unroll
  for (int i = 0; i < NE; i += 4) load_four(z + i, row + first + i, mine - i, fours, none);
  bool rest = false;  // left to route_exact
  float zmax = none;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    rest |= !(z[i] < inf);
    zmax = fmaxf(zmax, z[i]);
  }
  zmax = max_lanes<16>(zmax);
  float cmax = zmax;  // the largest of what is ranked
  double sum = 1.0;
  if (a.score == MOE_SCORE_SOFTMAX && (scores || !a.renorm)) {
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < NE; ++i) sum += exp((double)z[i] - (double)zmax);
    sum = sum_lanes<16>(sum);
  }
  if (scores) {
    if (a.score == MOE_SCORE_SOFTMAX) {
      const float inv = (float)(1.0 / sum);
#pragma unroll
      for (int i = 0; i < NE; ++i) v[i] = exp_fast(z[i] - zmax) * inv;
    } else {
#pragma unroll
      for (int i = 0; i < NE; ++i) v[i] = inverse(1.f + exp_fast(-z[i]));
    }
    float vmax = none;
#pragma unroll
    for (int i = 0; i < NE; i += 4) {
      float bias[4] = {0.f, 0.f, 0.f, 0.f};
      if (a.bias) load_four(bias, a.bias + first + i, mine - i, fours, none);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[i + j] = z[i + j] > none ? v[i + j] + bias[j] : none;
        rest |= !(v[i + j] < inf);
        vmax = fmaxf(vmax, v[i + j]);
      }
    }
    if (a.bias) cmax = max_lanes<16>(vmax);
  }
  const float unit = error_unit(a.score, true);
  bool keep = true;
  if (a.G > 1) {
    float m1 = none, m2 = none;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const float c = scores ? v[i] : z[i];
      m2 = __builtin_amdgcn_fmed3f(m1, m2, c);
      m1 = fmaxf(m1, c);
    }
    const bool in = l < a.G * group_lanes;
    keep = group_rank(m1, m2, a, group_lanes, lane) < a.kept && in;
    if (scores) {
      float value = m1, off = unit * (1.f + fabsf(m1));
      if (a.best == 2 && m2 > none) {
        value += m2;
        off += unit * (1.f + fabsf(m2));
      }
      const float low = -max_lanes<16>(keep ? off - value : none);
      const float high = max_lanes<16>(in && !keep ? value + off : none);
      if (__ballot(!(low > high))) {
        double d1 = none, d2 = none;
#pragma unroll 4
        for (int i = 0; i < mine; ++i) {
          const float zi = to_f32(row[first + i]);
          double c = choice_f64(a, zi, first + i, zmax, sum);
          c = zi > none ? c : (double)none;
          const double low = d1 < c ? d1 : c;
          d2 = d2 > low ? d2 : low;
          d1 = d1 > c ? d1 : c;
        }
        keep = group_rank(d1, d2, a, group_lanes, lane) < a.kept && in;
      }
    }
  }
  // values down to 2 (logits: 32) below the largest in steps; twice the error of scores that near, in
  // steps, and the roundings to these; a largest whose own steps are not exact enough is left
  const float step = a.bias ? 0x1p21f : 0x1p17f;
  rest |= !(fabsf(cmax) < 1024.f);
  const uint32_t close = a.bias ? (uint32_t)(2.f * unit * (3.f + fabsf(cmax)) * step + 4.f) : 0u;
  const uint32_t id0 = id_mask - (uint32_t)first;
  if (whole) {
    constexpr int DROP = __is_same(E, bf16_t) ? 16 : 13;  // bits that these types leave zero
#pragma unroll
    for (int i = 0; i < NE; ++i)
      key[i] = keep ? (((key_of(z[i]) >> DROP) - (key_of(none) >> DROP)) << id_bits) +
                          (id0 - i & id_mask)
                    : 0u;
  } else {
    const float top_step = keep ? kTop - cmax * step : none;
#pragma unroll
    for (int i = 0; i < NE; ++i)
      key[i] = (steps_of(fmaf(a.bias ? v[i] : z[i], step, top_step)) << id_bits) +
               (id0 - i & id_mask);
  }
  uint32_t top = 1u << 31, own = 0;  // own: lane j's the j-th best
  for (int j = 0; j <= a.k + 1; ++j) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NE; ++i) m = max(m, key[i] - top);
    top += join16(m, [](uint32_t x, uint32_t y) { return max(x, y); });
    own = l == j ? top : own;
  }
  // where the keys ran out (id bits alone) all that follows does not count
  const uint64_t out = __ballot(own <= id_mask) >> (lane & 48) & 0xffff;
  const bool valid = l <= a.k && (out & ((2u << l) - 1)) == 0;
  const int e = (int)(id_mask - (own & id_mask));
  int place = l;
  if (!whole) {
    const uint32_t f = own >> id_bits, next = __shfl_down(own, 1) >> id_bits;
    rest |= l < a.k && !valid;
    // the one behind the k + 1 best, which are ranked below, is far enough from the k-th
    rest |= l == a.k - 1 && f - (top >> id_bits) <= close;
    const bool next_valid = (out & ((4u << l) - 1)) == 0;
    if (__ballot(l < a.k && valid && next_valid && f - next <= close)) {
      double c = none;
      if (valid) {
        const float zc = to_f32(row[e]);
        c = a.bias ? choice_f64(a, zc, e, zmax, sum) : (double)zc;
      }
      int rank = 0;
      for (int j = 0; j <= a.k; ++j) {
        const double oc = __shfl(c, (lane & 48) + j);
        const int oe = __shfl(e, (lane & 48) + j);
        rank += oc > c || (oc == c && oe < e);
      }
      place = l <= a.k ? rank : l;
    }
  }
  const uint64_t left = __ballot(rest);
  const bool fast = (left >> (lane & 48) & 0xffff) == 0 && t < a.T;
  const bool has = valid && place < a.k && fast;
  write_choice(a, row, (int64_t)t * a.k + place, fast ? place : 16, has, e, zmax, sum);
  for (int q = 0; q < 4; ++q)
    if (left >> (16 * q) & 0xffff) {
      const int tq = (blockIdx.x * (RT_T / 64) + wave) * 4 + q;
      if (tq < a.T) route_exact<E, NPL, false>(a, tq, s_choice[wave], lane);
    }
}

struct RouteGradArgs {
  const void* z;
  int64_t zs;
  int T, E, score;
  const int* idx;
  int k, renorm;
  float scale;
  const float* dw;
  void* dz;
  int64_t dzs;
};

// With W the chosen scores divided by their sum and D = sum_j W_j dw_j: softmax renormalised
// dz_j = f W_j (dw_j - D); sigmoid renormalised the same times (1 - s_j); sigmoid
// dz_j = f s_j (1 - s_j) dw_j; softmax dz_e = f p_e (dw_e - sum_j p_j dw_j) for every expert (dw_e = 0
// where e was not chosen), otherwise 0.  The chosen are few: 64 bits, four tokens to a wave, 16 lanes
// each.  A token's row is put together in LDS (the logits of the others are read where softmax needs
// them, their exponentials held there in fp32) and written in 16-byte pieces.  16384 tokens of 256 fp32
// logits: 6.8 us, softmax that is not renormalised 14.5 (its 64-bit exponentials of every expert; bytes
// at a copy's rate 6.3).
template <class E>
__global__ __launch_bounds__(RT_T) void route_tokens_grad_kernel(RouteGradArgs a, int pitch) {
  constexpr int V = kChunk<E>;
  extern __shared__ __align__(16) float s_rows[];  // [RT_T / 16][pitch], pitch a multiple of V
  const int l = threadIdx.x & 15, slot = threadIdx.x >> 4;
  const float none = -__builtin_inff();
  const bool all = a.score == MOE_SCORE_SOFTMAX && !a.renorm;
  const int tokens = RT_T / 16, t = min(blockIdx.x * tokens + slot, (unsigned)a.T - 1);
  // behind the last token its lanes do the last one's work again, and write nothing
  const bool live = blockIdx.x * tokens + slot < (unsigned)a.T;
  const E* const row = (const E*)a.z + (int64_t)t * a.zs;
  float* const s_row = s_rows + slot * pitch;
  const int64_t at = (int64_t)t * a.k + l;
  const int e = l < a.k ? a.idx[at] : -1;
  const bool has = (unsigned)e < (unsigned)a.E;
  const float zc = has ? to_f32(row[e]) : none;
  const double dw = has ? (double)a.dw[at] * (double)a.scale : 0.0;
  double own;
  if (all) {
    float zmax = none;
    for (int c = l * V; c < a.E; c += 16 * V) {
      float f[V];
      if (c + V <= a.E) {
        const Chunk<E> q = load_chunk<V>(row + c);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = to_f32(q.e[i]);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = c + i < a.E ? to_f32(row[c + i]) : none;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        zmax = fmaxf(zmax, f[i]);
        s_row[c + i] = f[i];
      }
    }
    zmax = max_lanes<16>(zmax);
    double sum = 0.0;
    for (int c = l * V; c < a.E; c += 16 * V)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float z = s_row[c + i];
        const double p = z == none ? 0.0 : exp((double)z - (double)zmax);
        sum += p;
        s_row[c + i] = (float)p;
      }
    sum = sum_lanes<16>(sum);
    sum = sum == 0.0 ? 0.0 : 1.0 / sum;  // no expert at all: zeros
    const double w = has ? exp((double)zc - (double)zmax) * sum : 0.0;
    const double along = sum_lanes<16>(w * dw);
    own = w * (dw - along);
    const double by = -sum * along;
    for (int c = l * V; c < a.E; c += 16 * V)
#pragma unroll
      for (int i = 0; i < V; ++i) s_row[c + i] = (float)((double)s_row[c + i] * by);
  } else {
    for (int c = l * 4; c < pitch; c += 64) *(float4*)(s_row + c) = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.score == MOE_SCORE_SOFTMAX) {
      const float top = max_lanes<16>(zc);
      double w = has ? exp((double)zc - (double)top) : 0.0;
      w /= sum_lanes<16>(w);
      own = w * (dw - sum_lanes<16>(w * dw));
    } else {
      // 1 - s without its cancellation: s(-z) = exp(-z) s(z), with the smaller of the exponentials
      const double f = exp(-fabs((double)zc)), big = 1.0 / (1.0 + f), small = f * big;
      const double s = !has ? 0.0 : zc < 0.f ? small : big;
      double w = s, along = 0.0;
      if (a.renorm) {
        const double sum = sum_lanes<16>(s);
        w = sum == 0.0 ? 0.0 : s / sum;
        along = sum_lanes<16>(w * dw);
      }
      own = w * (zc < 0.f ? big : small) * (dw - along);
      if (zc != zc) own = zc;
    }
  }
  asm volatile("" ::: "memory");  // a wave's LDS accesses run in order
  if (has) s_row[e] = (float)own;
  asm volatile("" ::: "memory");
  if (!live) return;
  E* const out = (E*)a.dz + (int64_t)t * a.dzs;
  for (int c = l * V; c < a.E; c += 16 * V) {
    const Chunk<E> q = round_chunk<E, V>(s_row + c);
    if (c + V <= a.E) {
      store_chunk(out + c, q);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c + i < a.E) out[c + i] = q.e[i];
    }
  }
}

// ------------------------------------------------------------------ host side

constexpr int kRouteGrid = 256 * 8;
unsigned route_grid(int T) {
  return (unsigned)std::min((T + RT_T / 64 - 1) / (RT_T / 64), kRouteGrid);
}

template <class E>
hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
  // experts of a lane: with groups, so many that a group has 1, 2, 4, 8 or 16 lanes
  int n_lane = (a.E + 63) / 64 * 4, group_lanes = 1;
  if (a.G > 1) {
    const int size = a.E / a.G;
    n_lane = 0;
    for (group_lanes = 16; group_lanes > 1; group_lanes >>= 1)
      if (size % (4 * group_lanes) == 0 && a.G * group_lanes <= 16) break;
    if (size % (4 * group_lanes) == 0 && a.G * group_lanes <= 16) n_lane = size / group_lanes;
  }
  int id_bits = 1;
  while ((1 << id_bits) < a.E) ++id_bits;
  if (n_lane > 0 && n_lane <= 32 && a.k < 16) {
    const auto kernel = n_lane <= 4    ? route_tokens_kernel<E, 4>
                        : n_lane <= 8  ? route_tokens_kernel<E, 8>
                        : n_lane <= 16 ? route_tokens_kernel<E, 16>
                                       : route_tokens_kernel<E, 32>;
    constexpr int tokens = RT_T / 16;
    return launch_kernel(kernel, dim3((unsigned)((a.T + tokens - 1) / tokens)), dim3(RT_T), 0, s, a,
                         n_lane, id_bits, group_lanes);
  }
  const auto kernel = a.E <= 64    ? route_tokens_wave_kernel<E, 1>
                      : a.E <= 128 ? route_tokens_wave_kernel<E, 2>
                      : a.E <= 256 ? route_tokens_wave_kernel<E, 4>
                      : a.E <= 512 ? route_tokens_wave_kernel<E, 8>
                                   : route_tokens_wave_kernel<E, 16>;
  return launch_kernel(kernel, dim3(route_grid(a.T)), dim3(RT_T), 0, s, a);
}
template <class E>
hipError_t launch_route_grad(const RouteGradArgs& a, hipStream_t s) {
  constexpr int tokens = RT_T / 16;
  const int pitch = (a.E + 7) / 8 * 8;
  return launch_kernel(route_tokens_grad_kernel<E>, dim3((unsigned)((a.T + tokens - 1) / tokens)),
                       dim3(RT_T), sizeof(float) * tokens * pitch, s, a, pitch);
}

bool route_ok(int type, int T, int E, int score, int k, float scale) {
  return float_type(type) && T >= 0 && T <= kMaxRouteT && E >= 1 && E <= kMaxRouted &&
         (score == MOE_SCORE_SOFTMAX || score == MOE_SCORE_SIGMOID) && k >= 1 &&
         k <= std::min(E, kMaxChoices) && scale - scale == 0.f;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_route_tokens(const void* logits, int64_t logits_stride, int32_t type, int32_t T,
                            int32_t experts, int32_t score, const float* bias, int32_t groups,
                            int32_t group_best, int32_t top_groups, int32_t top_k,
                            int32_t renormalise, float scale, int32_t* topk_idx, float* topk_w,
                            void* stream) {
  if (!route_ok(type, T, experts, score, top_k, scale) || !aligned4(bias) || groups < 1 ||
      groups > kMaxRouteGroups || experts % groups != 0 || group_best < 1 || group_best > 2 ||
      top_groups < 1 || top_groups > groups)
    return MOE_E_INVALID;
  if (T == 0) return MOE_OK;  // before the pointers: empty buffers have none
  if (!rows_ok(logits, logits_stride, experts, type) || !topk_idx || !topk_w ||
      !aligned4(topk_idx) || !aligned4(topk_w) || !on_current_device(topk_idx))
    return MOE_E_INVALID;
  // where every group stays there is nothing to rank
  const int G = top_groups == groups ? 1 : groups;
  RouteArgs a{logits, logits_stride, T, experts, score, bias, G, group_best, top_groups,
              top_k, renormalise, scale, topk_idx, topk_w};
  const hipStream_t s = (hipStream_t)stream;
  if (type == MOE_T_BF16) return launched(launch_route<bf16_t>(a, s));
  if (type == MOE_T_FP16) return launched(launch_route<fp16_t>(a, s));
  return launched(launch_route<float>(a, s));
}

moe_status moe_route_tokens_grad(const void* logits, int64_t logits_stride, int32_t type,
                                 int32_t T, int32_t experts, int32_t score,
                                 const int32_t* topk_idx, int32_t top_k, int32_t renormalise,
                                 float scale, const float* dweights, void* dlogits,
                                 int64_t dlogits_stride, void* stream) {
  if (!route_ok(type, T, experts, score, top_k, scale)) return MOE_E_INVALID;
  if (T == 0) return MOE_OK;  // before the pointers: empty buffers have none
  if (!rows_ok(logits, logits_stride, experts, type) || !topk_idx || !dweights ||
      !aligned4(topk_idx) || !aligned4(dweights) ||
      !rows_ok(dlogits, dlogits_stride, experts, type) ||
      !same_rows(dlogits, dlogits_stride, logits, logits_stride) || !on_current_device(dlogits))
    return MOE_E_INVALID;
  RouteGradArgs a{logits, logits_stride, T, experts, score, topk_idx, top_k,
                  renormalise, scale, dweights, dlogits, dlogits_stride};
  const hipStream_t s = (hipStream_t)stream;
  if (type == MOE_T_BF16) return launched(launch_route_grad<bf16_t>(a, s));
  if (type == MOE_T_FP16) return launched(launch_route_grad<fp16_t>(a, s));
  return launched(launch_route_grad<float>(a, s));
}

}  // extern "C"
