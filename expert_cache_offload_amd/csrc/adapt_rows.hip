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
#include <cmath>

#include "row_ops.h"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 fp16x8 __attribute__((ext_vector_type(8)));

constexpr int kMaxRank = 128;
constexpr int kMaxAdapters = 1024;
// Calls whose x, base and out are more than this together pass the caches by: they would push out the
// adapters (2048 to 2048 of rank 64: 16384 rows, 201 MB, 57.7 us without, 52.3 with; 8192 rows 33.3 and
// 29.5; 6144 rows, 75 MB, 21.1 and 24.4).  Only where rows of out start with a half line: a store that
// passes the caches by is not joined with its neighbour's part of the line (16384 rows, 1024 to 3000
// of rank 32, 100 us with and 69 without; 1024 to 2976 equal).
constexpr int64_t kAdaptStreamBytes = 80 << 20;

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
template <bool STREAM, class E>
__device__ __forceinline__ u32x4 load_x(const E* p) {
  return load_chunk<kChunk<E>, STREAM>(p).q;
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
  int g, m0, end;   // adapter, first sorted row, end of the adapter's rows
  int part, parts;  // which part of the channels, of how many
};
// Tiles left over when every CU has had the same number of them are shared out over the channels, as
// many parts as there are CUs for, of 256 channels at least; each part computes h for itself.  Whole,
// the last ones keep a few CUs busy while the others wait (2048 to 2048, 11 requests of 16384 rows: rank
// 64 59 us whole, 53 shared out, rank 16 50 and 47; 16032 rows, 512 tiles at most, 47 and 42; 8192 rows of
// rank 64 36 and 30.  With 1024 channels a part at least 55, 48 and 32).
constexpr int kCus = 256;
__host__ __device__ constexpr int parts_of_rest(int rest, int most) {
  return rest > 0 && kCus / rest > 1 ? (kCus / rest < most ? kCus / rest : most) : 1;
}
__host__ __device__ constexpr int most_parts(int N) {
  return N / 256 > kCus ? kCus : N / 256 > 1 ? N / 256 : 1;
}
// The row tile (of BM rows, counted over the adapters) of workgroup column b, by every wave for itself,
// 64 adapters at a time; g = -1 where there is none.  Workgroups go round the eight dies, so each
// die is given a run of neighbouring tiles: its L2 then holds the one or two adapters that they
// share (16384 rows over 11 adapters of 512 KiB read 144 MB from behind the L2, 185 with the tiles dealt
// out in order).
constexpr int kDies = 8;
template <int BM>
__device__ __forceinline__ Tile find_tile(const AdaptArgs& a, int b, int lane) {
  int2 rows = make_int2(0, 0);  // this lane's adapter's, of the 64 from g0 on
  int inc = 0, n = 0;           // tiles up to and with it; its own
  const auto look = [&](int g0) {
    rows = make_int2(0, 0);
    if (!a.offsets) {
      if (lane == 0) rows.y = a.M;
    } else if (g0 + lane < a.adapters) {
      rows.x = min(max(a.offsets[g0 + lane], 0), a.M);
      rows.y = min(max(a.offsets[g0 + lane + 1], rows.x), a.M);
    }
    n = inc = (rows.y - rows.x + BM - 1) / BM;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const int o = __shfl_up(inc, s);
      if (lane >= s) inc += o;
    }
    return __builtin_amdgcn_readlane(inc, 63);
  };
  int total = look(0);
  for (int g0 = 64; g0 < a.adapters; g0 += 64) total += look(g0);
  const int rest = gridDim.y == 1 && total > kCus ? total % kCus : 0;
  int parts = parts_of_rest(rest, most_parts(a.N)), part = 0, tile;
  const int whole = parts > 1 ? total - rest : total, per = (whole + kDies - 1) / kDies;
  if (b < per * kDies) {
    tile = b % kDies * per + b / kDies;
    if (tile >= whole) return Tile{-1, 0, 0, 0, 1};
    parts = gridDim.y;
    part = blockIdx.y;
  } else {  // the parts of a tile on one die too
    if (parts == 1) return Tile{-1, 0, 0, 0, 1};
    const int i = (b - whole) / kDies, left = i / parts * kDies + b % kDies;
    if (left >= rest) return Tile{-1, 0, 0, 0, 1};
    tile = whole + left;
    part = i % parts;
  }
  for (int g0 = 0; g0 < a.adapters; g0 += 64) {
    const int here = a.adapters > 64 ? look(g0) : total;
    if (tile < here) {
      const int l = __builtin_ctzll(__ballot(inc > tile));
      const int before = __builtin_amdgcn_readlane(inc - n, l);
      return Tile{g0 + l, __builtin_amdgcn_readlane(rows.x, l) + (tile - before) * BM,
                  __builtin_amdgcn_readlane(rows.y, l), part, parts};
    }
    tile -= here;
  }
  return Tile{-1, 0, 0, 0, 1};
}

// A wave's LDS accesses execute in order; this keeps the compiler, which sees one lane's only, from
// reordering or merging them where lanes read what others wrote.
__device__ __forceinline__ void wave_lds_order() { asm volatile("" ::: "memory"); }

// 16-byte chunks of a row of UC in LDS are dealt by the row's number, so that the sixteen rows of an
// operand do not meet in the same banks.
template <int UC>
__device__ __forceinline__ int dealt(int chunk, int row) {
  return UC == 8 ? chunk ^ (row & 7) : chunk ^ ((row >> 1) & 3);
}

// A tile of 16 MT rows, ranks up to 16 RT, UC 16-byte chunks of a row's contraction at a time, W waves.
// Neighbouring lanes load neighbouring chunks (a lane per row, as the matrix instruction has them,
// costs an access of the cache for each lane: 93 us where this took 67), which go through the
// wave's own part of LDS into the instruction's order, and its results back the same way.  Both
// products have the loads of their next step under way in registers.
template <class E, int RT, int MT, int UC, int W, bool STREAM>
__global__ __launch_bounds__(64 * W) void adapt_rows_kernel(AdaptArgs a) {
  constexpr int V = kChunk<E>, BM = 16 * MT, UNIT = UC * V;
  constexpr bool SPLIT = sizeof(E) == 2;
  constexpr int PARTS = SPLIT ? 2 : 1;
  constexpr int RPL = 64 / UC;                        // rows of a load of all lanes
  constexpr int NX = BM / RPL, NA = 16 * RT / RPL;    // loads of a step
  // steps under way (twice as many cost the registers of a wave more a SIMD: 2000 rows of rank 8, 1024 to
  // 8192, 23.7 us so and 21.4; 7254 rows of rank 16, 6888 to 920, 37 and 39)
  constexpr int BATCH = NX + NA <= 4 ? 2 : 1;
  constexpr int PITCH = 16 * RT + 4;                  // of a row of h, in floats
  constexpr int R = RT == 1 && SPLIT ? 32 : 16 * RT;  // contraction of the second product, padded
  constexpr int RC = R / V, RK = RC / 4;              // its chunks, and steps
  constexpr int HP = R + V;                           // pitch of its operands
  // channel tiles of a block; half where LDS holds eight waves'
  constexpr int NT = (RC <= 8 ? 4 : RC <= 16 ? 2 : 1) / (W > 4 && RC <= 16 ? 2 : 1);
  constexpr int NB = 16 * NT, CPR = NB / V;           // channels, chunks of a row of the output
  constexpr int NBL = NB * RC / 64;                   // loads of a block's B
  constexpr int RPO = 64 / CPR, NO = BM / RPO;        // rows of a load of the base; loads
  constexpr int OP = NB + 4;                          // pitch of the results
  // the wave's LDS: a step's operands, or its part of h, or a block's B, then its results
  constexpr int STEP_B = (BM + 16 * RT) * UC * 16, PART_B = BM * PITCH * 4;
  constexpr int BLOCK_B = NB * HP * (int)sizeof(E), RESULT_B = 16 * OP * 4;
  constexpr int WAVE_B = std::max({STEP_B, PART_B, BLOCK_B, RESULT_B});
  static_assert(WAVE_B % 16 == 0 && NX * RPL == BM && NA * RPL == 16 * RT);
  __shared__ __align__(16) uint8_t s_wave[W][WAVE_B];
  __shared__ __align__(16) E s_h[PARTS][BM][HP];
  __shared__ float s_back[BM];  // powers of two that fp16's parts were divided by
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const Tile t = find_tile<BM>(a, blockIdx.x, lane);
  if (t.g < 0) return;
  uint8_t* const mem = s_wave[wave];
  // The tile's rows, a lane each.  Behind the adapter's last row, and where a place is no row, another
  // row of the tile is computed and written again, so that no store depends on its lane: a wait for a
  // load would otherwise count on none of the stores after it, and wait for these too.
  int mine = t.m0 + lane % BM;
  if (mine >= t.end) mine = t.end - 1;
  if (a.order) mine = a.order[mine];
  const uint64_t rows = __ballot((unsigned)mine < (unsigned)a.M);
  if (rows == 0) return;
  const int other = __builtin_amdgcn_readlane(mine, __builtin_ctzll(rows));
  if ((unsigned)mine >= (unsigned)a.M) mine = other;
  const auto row_of = [&](int m) { return __shfl(mine, m); };
  const E* src[NX + NA];  // this lane's chunk of its rows of x, and of A (behind the rank: the last)
  const int lr = lane / UC, lc = lane % UC;
#pragma unroll
  for (int i = 0; i < NX; ++i)
    src[i] = (const E*)a.x + row_of(lr + RPL * i) * a.xs + lc * V;
#pragma unroll
  for (int i = 0; i < NA; ++i)
    src[NX + i] = (const E*)a.a +
                  ((int64_t)t.g * a.rank + min(lr + RPL * i, a.rank - 1)) * a.as + lc * V;

  f32x4 acc[RT][MT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[r][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  struct Step {
    u32x4 q[NX + NA];
  };
  const auto load_step = [&](Step& k, int u) {
#pragma unroll
    for (int i = 0; i < NX + NA; ++i)
      k.q[i] = i < NX ? load_x<STREAM>(src[i] + u * UNIT) : load_full(src[i] + u * UNIT);
  };
  const auto use_step = [&](const Step& k) {
    wave_lds_order();
#pragma unroll
    for (int i = 0; i < NX + NA; ++i) {
      const int row = lr + RPL * i;
      *(u32x4*)(mem + (row * UC + dealt<UC>(lc, row)) * 16) = k.q[i];
    }
    wave_lds_order();
#pragma unroll
    for (int s = 0; s < UC / 4; ++s) {
      const auto frag = [&](int row) {
        return *(const u32x4*)(mem + (row * UC + dealt<UC>(4 * s + quad, row)) * 16);
      };
      u32x4 xf[MT];
#pragma unroll
      for (int i = 0; i < MT; ++i) xf[i] = frag(16 * i + col);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const u32x4 wf = frag(BM + 16 * r + col);
#pragma unroll
        for (int i = 0; i < MT; ++i) mma<E>(acc[r][i], wf, xf[i]);
      }
    }
  };

  // A block of channels: its rows of B, a lane a chunk of NBL of them, and the base's chunks
  const int blocks = (a.N + NB - 1) / NB, step = t.parts * W;
  const bool short_rank = a.rank < V;
  // whole blocks; of the others (the last where N is no multiple, all where the rank is below 16
  // bytes) a lane's chunk may be short
  const int whole = short_rank ? 0 : a.N / NB;
  const int bc = lane % RC * V;  // first element of this lane's chunk of a row of B
  const E* const bg = (const E*)a.b + (int64_t)t.g * a.N * a.bs;
  const int oc = lane % CPR * V;
  E* out[NO];
  const E* base[NO];
#pragma unroll
  for (int i = 0; i < NO; ++i) {
    const int r = row_of(lane / CPR + RPO * i);
    out[i] = (E*)a.out + r * a.os + oc;
    // without a base any 16 bytes of the output's row serve: nothing takes them
    base[i] = a.base ? (const E*)a.base + r * a.base_s + oc : (const E*)a.out + r * a.os;
  }
  const int base_n = a.base ? -1 : 0;
  const auto block_at = [&](int i) { return min(i, whole - 1); };
  // two blocks of B and one of the base are under way (with the base two or four blocks ahead, a tile
  // of 32 rows took 8 to 10 us longer)
  u32x4 bq[2][NBL];
  Chunk<E> bases[NO];
  const auto load_b = [&](u32x4(&k)[NBL], int nb) {
#pragma unroll
    for (int i = 0; i < NBL; ++i)
      k[i] = load_full(bg + (nb * NB + (i * 64 + lane) / RC) * a.bs + min(bc, a.rank - V));
  };
  const auto load_base = [&](Chunk<E>(&k)[NO], int nb) {
#pragma unroll
    for (int i = 0; i < NO; ++i) k[i] = load_chunk<V, STREAM>(base[i] + (nb * NB & base_n));
  };

  const int units = a.K / UNIT, batches = units / BATCH;
  const int ib = t.part * W + wave;
  {
    Step k[2][BATCH];  // in turn; behind the last the last is loaded again
    const auto load_batch = [&](Step(&k)[BATCH], int i) {
      const int u = min(i, batches - 1) * BATCH;
#pragma unroll
      for (int j = 0; j < BATCH; ++j) load_step(k[j], u + j);
    };
    const auto use_batch = [&](const Step(&k)[BATCH]) {
#pragma unroll
      for (int j = 0; j < BATCH; ++j) use_step(k[j]);
    };
    if (wave < batches) load_batch(k[0], wave);
    for (int i = wave; i < batches; i += 2 * W) {
      load_batch(k[1], i + W);
      use_batch(k[0]);
      if (i + W >= batches) break;
      load_batch(k[0], i + 2 * W);
      use_batch(k[1]);
    }
    static_assert(BATCH - 1 <= W);
    if (BATCH > 1 && batches * BATCH + wave < units) {  // steps short of a batch, one each
      load_step(k[0][0], batches * BATCH + wave);
      use_step(k[0][0]);
    }
    if (units * UNIT < a.K && wave == W - 1) {
      const int n = a.K - units * UNIT - lc * V;
#pragma unroll
      for (int i = 0; i < NX + NA; ++i) k[0][0].q[i] = load_tail(src[i] + units * UNIT, n, a.K);
      use_step(k[0][0]);
    }
  }
  if (whole > 0) {
    load_b(bq[0], block_at(ib));
    load_b(bq[1], block_at(ib + step));
    load_base(bases, block_at(ib));
  }
  wave_lds_order();
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int i = 0; i < MT; ++i)
      *(f32x4*)(mem + ((16 * i + col) * PITCH + 16 * r + 4 * quad) * 4) = acc[r][i];
  __syncthreads();
  {  // the waves' parts joined, scaled and laid out as an operand
    constexpr int PER = 16;  // threads of a row
    const float f = a.scale ? a.scale[t.g] : 1.f;
#pragma unroll
    for (int m = tid / PER; m < BM; m += 64 * W / PER) {
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
          for (int p = 0; p < W; ++p) h[i] += ((const float*)s_wave[p])[m * PITCH + r];
          h[i] *= f;
        }
        big = fmaxf(big, fabsf(h[i]));
      }
      float by = 1.f;
      if constexpr (__is_same(E, fp16_t)) {
        big = join16(big, [](float p, float q) { return fmaxf(p, q); });
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
  }
  __syncthreads();
  u32x4 h[MT][RK][PARTS];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int s = 0; s < RK; ++s)
#pragma unroll
      for (int p = 0; p < PARTS; ++p)
        h[i][s][p] = *(const u32x4*)&s_h[p][16 * i + col][(s * 4 + quad) * V];

  // what counts of a lane's chunk of B: nothing behind the rank and, in its last chunk, nothing that
  // the one before has
  Chunk<E> count;
  count.q = u32x4{~0u, ~0u, ~0u, ~0u};
  if (!short_rank) {
    const int gone = bc - min(bc, a.rank - V);
#pragma unroll
    for (int e = 0; e < V; ++e) count.e[e] = e < gone ? E{} : count.e[e];
  }
  const auto put_b = [&](u32x4(&k)[NBL]) {
    wave_lds_order();
#pragma unroll
    for (int i = 0; i < NBL; ++i)
      *(u32x4*)(mem + ((i * 64 + lane) / RC * HP + bc) * (int)sizeof(E)) = k[i] & count.q;
    wave_lds_order();
  };
  const auto use_block = [&](const Chunk<E>(&bk)[NO], int nb, bool all) {
    u32x4 bf[NT][RK];
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
      for (int s = 0; s < RK; ++s)
        bf[c][s] = *(const u32x4*)(mem + ((16 * c + col) * HP + (s * 4 + quad) * V) * (int)sizeof(E));
    float* const res = (float*)mem;  // where B was, which is in registers
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      wave_lds_order();
#pragma unroll
      for (int c = 0; c < NT; ++c) {
        f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < RK; ++s)
#pragma unroll
          for (int p = PARTS - 1; p >= 0; --p) mma<E>(o, bf[c][s], h[i][s][p]);
        *(f32x4*)(res + col * OP + 16 * c + 4 * quad) = o;
      }
      wave_lds_order();
#pragma unroll
      for (int j = 0; j < 16 / RPO; ++j) {
        const int at = i * (16 / RPO) + j, m = lane / CPR + RPO * j;
        float f[V];
#pragma unroll
        for (int e = 0; e < V; e += 4) *(f32x4*)(f + e) = *(const f32x4*)(res + m * OP + oc + e);
        const float back = __is_same(E, fp16_t) ? s_back[16 * i + m] : 1.f;
#pragma unroll
        for (int e = 0; e < V; ++e)
          f[e] = fmaf(f[e], back, a.base ? to_f32(bk[at].e[e]) : 0.f);
        const Chunk<E> v = round_chunk<E, V>(f);
        const int n = a.N - nb * NB - oc;
        if (all || n >= V) {
          store_chunk<STREAM>(out[at] + nb * NB, v);
        } else {
#pragma unroll
          for (int e = 0; e < V - 1; ++e)
            if (e < n) out[at][nb * NB + e] = v.e[e];
        }
      }
    }
  };
  const auto turn = [&](u32x4(&k)[NBL], int nb) {
    put_b(k);
    load_b(k, block_at(nb + 2 * step));
    use_block(bases, nb, true);
    load_base(bases, block_at(nb + step));
  };
  for (int nb = ib; nb < whole; nb += 2 * step) {
    turn(bq[0], nb);
    if (nb + step >= whole) break;
    turn(bq[1], nb + step);
  }
  for (int nb = ib; nb < blocks; nb += step) {
    if (nb < whole) continue;
#pragma unroll
    for (int i = 0; i < NBL; ++i) {
      const E* const b = bg + min(nb * NB + (i * 64 + lane) / RC, a.N - 1) * a.bs;
      bq[0][i] = short_rank ? load_tail(b + bc, a.rank - bc, a.rank)
                            : load_full(b + min(bc, a.rank - V));
    }
#pragma unroll
    for (int i = 0; i < NO; ++i) {
      bases[i].q = u32x4{0, 0, 0, 0};
      const int n = a.base ? a.N - nb * NB - oc : 0;
      if (n >= V) {
        bases[i] = load_chunk<V, STREAM>(base[i] + nb * NB);
      } else {
#pragma unroll
        for (int e = 0; e < V - 1; ++e)
          if (e < n) bases[i].e[e] = base[i][nb * NB + e];
      }
    }
    put_b(bq[0]);
    use_block(bases, nb, false);
  }
}

// ------------------------------------------------------------------ host side

// Row tiles are counted for the worst split of the rows over the adapters; workgroups behind the last
// tile return.  The channels of a tile are shared out over several workgroups, each of which
// computes the tile's h for itself.  With p1 elements that h reads and p2 that the rest moves, a
// workgroup's own time goes with p1 + p2 / shares, what all of them read with tiles (p1 shares + p2): the
// best number is the root of p2 / (p1 tiles) times a constant, which measures 200 to 400 (1024 rows of
// rank 64, 2048 to 2048: 15.5, 12.6 and 15.7 us with 1, 2 and 4; 664 rows, 864 to 3080: 20.5, 16.0,
// 13.7 and 12.4 with 1, 2, 4 and 8; 4096 rows, 2048 to 2048: 20.5 and 23.4 with 1 and 2), up to four
// workgroups for a CU (4480 rows of rank 32, 112 to 7072, in 140 tiles: 55, 48 and 51 us with 1, 8
// and 14); all by four waves.
constexpr double kShareRate = 215.0;
int adapt_shares(const AdaptArgs& a, int tiles, int rows, int blocks, int waves) {
  const double p1 = (double)a.K * (rows + a.rank), p2 = (double)a.N * (a.rank + 2 * rows);
  const int best = (int)std::lround(std::sqrt(kShareRate * p2 / (p1 * tiles)));
  return std::max(1, std::min({(blocks + waves - 1) / waves, 1024 / tiles, best}));
}
template <class E>
bool streams(const AdaptArgs& a) {
  return (int64_t)a.M * (a.K + (a.base ? 2 : 1) * (int64_t)a.N) * (int)sizeof(E) >
             kAdaptStreamBytes &&
         (uintptr_t)a.out % 64 == 0 && a.os * (int64_t)sizeof(E) % 64 == 0;
}
template <class E, int RT, int MT, int UC, int W>
hipError_t launch_adapt_by(const AdaptArgs& a, hipStream_t s) {
  constexpr int BM = 16 * MT;
  const int groups = a.offsets ? std::min(a.adapters, a.M) : 1;
  const int most = std::min(a.M, a.M / BM + groups);
  int tiles = (most + kDies - 1) / kDies * kDies;
  const int shares = adapt_shares(a, std::min(tiles, a.M / BM + 1), BM, (a.N + 63) / 64, W);
  if (shares == 1 && most > kCus) {  // enough for every number of tiles that there may be
    const int p = most_parts(a.N), even = most / kCus * kCus;
    tiles = std::max(tiles, (even + std::min(kCus, most % kCus * p) + (kDies - 1) * p + kDies - 1) /
                                kDies * kDies);
  }
  constexpr bool MAY = W == 4;  // the few rows of eight waves are never that much
  const auto kernel = MAY && streams<E>(a) ? adapt_rows_kernel<E, RT, MT, UC, W, MAY>
                                           : adapt_rows_kernel<E, RT, MT, UC, W, false>;
  return launch_kernel(kernel, dim3((unsigned)tiles, (unsigned)shares), dim3(64 * W), 0, s, a);
}
template <class E>
hipError_t launch_adapt(const AdaptArgs& a, hipStream_t s) {
  // 32 rows a tile read A and B half as often, but leave a CU half as many waves: taken for many rows of a
  // high rank (rank 64, 2048 to 2048: 4096 rows 19.4 us with 16 rows a tile, 20.2 with 32, 6144 rows
  // 23.6 and 21.1, 16384 60.9 and 51.5; rank 32: 8192 rows, 2048 to 4096, 41.9 and 47.0, 20000 rows,
  // 2048 to 2048, 55.0 and 51.3; rank 16: 16384 rows 41.0 and 45.4), where an adapter has so many
  const bool wide = (int64_t)a.M * (a.rank <= 32 ? 32 : 64) >= 6144 * 64 &&
                    a.M >= 32 * (a.offsets ? a.adapters : 1);
  // Eight waves where tiles are few and the work of each long: ranks up to 32 with long rows of x (rank 32,
  // N = 2048: one row of 6144 10.0 us with four waves, 9.6 with eight; 256 rows of 512 5.6 and 6.0, of
  // 4096 11.4 and 10.2; 1024 rows of 4096 15.2 and 13.3; but 4000 rows, 4096 to 4096, 35 and 45), rank 64
  // with short ones, whose channels eight waves share (256 rows of 512 7.8 and 7.4, of 6144 19.8 and
  // 22.8: a step holds half as much of a row there, for the LDS), or with very few
  const int64_t row = (int64_t)a.K * (int)sizeof(E);
  const bool few = a.M <= 1024 && !streams<E>(a);
  const bool deep = few && (a.rank <= 32 ? row >= (a.M < 256 ? 8192 : 2048) : row <= 4096 || a.M <= 64);
  if (a.rank <= 16)
    return deep ? launch_adapt_by<E, 1, 1, 8, 8>(a, s) : launch_adapt_by<E, 1, 1, 8, 4>(a, s);
  if (a.rank <= 32)
    return wide   ? launch_adapt_by<E, 2, 2, 8, 4>(a, s)
           : deep ? launch_adapt_by<E, 2, 1, 8, 8>(a, s)
                  : launch_adapt_by<E, 2, 1, 8, 4>(a, s);
  if (a.rank <= 64)
    return wide   ? launch_adapt_by<E, 4, 2, 8, 4>(a, s)
           : deep ? launch_adapt_by<E, 4, 1, 4, 8>(a, s)
                  : launch_adapt_by<E, 4, 1, 8, 4>(a, s);
  return launch_adapt_by<E, 8, 1, 4, 4>(a, s);
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
      (base && !rows_ok(base, base_stride, N, type)) ||
      !same_rows(out, out_stride, base, base_stride) || !aligned4(scale) || !aligned4(offsets) ||
      !aligned4(order) || !on_current_device(out))
    return MOE_E_INVALID;
  AdaptArgs p{x, x_stride, M, K, a, a_stride, b, b_stride, N, rank, scale, adapters,
              offsets, order, base, base_stride, out, out_stride};
  const hipStream_t s = (hipStream_t)stream;
  if (type == MOE_T_BF16) return launched(launch_adapt<bf16_t>(p, s));
  if (type == MOE_T_FP16) return launched(launch_adapt<fp16_t>(p, s));
  return launched(launch_adapt<float>(p, s));
}
