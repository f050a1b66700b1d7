// Tokens sorted by expert and back, with routing weights, their gradients, and the 8-bit
// quantisation of rows.
//
// With id[a] the expert of assignment a = t * k + j (choice j of token t), the sort is stable by
// expert: place[a] = #{b : id[b] < id[a]} + #{b < a : id[b] = id[a]} over the assignments whose
// id is in [0, E); the others are dropped (place -1).  Row place[a] of the sorted matrix is
// token t's row.  Back: y[t] = sum_j w[t][j] * rows[place[t][j]].  Gradients: of the sort, the same
// sum with w = 1; of the sum, drows[place[a]] = w[a] dy[t] and dw[a] = <dy[t], rows[place[a]]>.
//
// All of it is movement: every kernel is bound by the bytes of the rows it reads and writes.
// Every count is an integer (of ballots, or of atomics on counters in LDS), so nothing depends on the
// order of execution.
#include <algorithm>

#include "row_ops.h"

namespace moe {
namespace {

constexpr int TOK_T = 256;          // threads of every kernel here but the scan
constexpr int kSmallIds = 2048;     // assignments that one kernel sorts (each workgroup counts
                                    // all of them for the ids of its own token): 2048 take
                                    // 11.1 us so and 11.7 with a launch more, 4096 18.8 and 12.5
constexpr int kMaxTopK = 16;
constexpr int kMaxExperts = 1024;
constexpr int kChunkIds = 1024;     // assignments of a counted chunk (whole tokens)
constexpr int kChunkWaves = kChunkIds / 64;
constexpr int kSubTokens = 16;      // tokens a workgroup of the move kernel sorts and moves,
constexpr int kSubIds = 256;        // and the most assignments
constexpr int kSelfChunks = 16;     // most chunks whose counts the move kernel adds up itself
constexpr int kMaxT = 1 << 20;
constexpr int kMaxRows = (1 << 24) - 1;  // a workgroup each stays a launch's size
// A rows matrix above this is streamed past the caches (non-temporal loads and stores): it would
// not be there any more for whoever reads it next, and the chip moves it faster so (16384 tokens
// of 8 rows, 2048 bf16: sort 137 -> 116 us, combine 118 -> 102, its gradient 226 -> 207, 131072 rows
// of 768 quantised 54.7 -> 52.0; a gradient over 34 MB, which stays in the 256 MB cache, got slower
// so, 13.7 -> 15.4 us).  Two exceptions: combine below a wave per token, and sorts whose last launch
// adds up the counts itself (up to 16 chunks, 16384 assignments), never stream.
constexpr int64_t kStreamBytes = 128 << 20;
constexpr int kScanExperts = 16, kScanSegs = 64;  // of a workgroup of the scan
constexpr int SCAN_T = kScanExperts * kScanSegs;
constexpr int kScanHeld = 16;

struct SortArgs {
  const int* ids;
  int T, k, E, N;
  const void* x;  // null: integers only
  int64_t xs;
  int H;
  int* offsets;
  int* order;  // may be null
  int* place;
  void* rows;
  int64_t rs;
  float* row_scale;
  int* base;    // [nblk][E] counts of each chunk, or those of the chunks before it
  int* total;   // [E] counts of all chunks
  int tok_blk;  // tokens of a chunk
  int nblk;
};

// Dropped assignments get a key above every expert's.
__device__ __forceinline__ int key_of_id(int id, int E) {
  return (unsigned)id < (unsigned)E ? id : 0x7fffffff;
}

// Chunks of a row that a thread holds at once.
constexpr int kHeld = 4;

// Loads chunks c, c + nthr, ... below c1 of a row.
template <class E, int V>
__device__ __forceinline__ void load_row(Chunk<E, V> (&v)[kHeld], const E* x, int H, int c,
                                         int c1, int nthr) {
#pragma unroll
  for (int h = 0; h < kHeld; ++h)
    if (c + h * nthr < c1) v[h] = load_chunk<V>(x + chunk_at<V>(c + h * nthr, H));
}

// Copies a row's chunks [c0, c1) to its k places, threads tid of nthr, each with kHeld loads in
// flight before its first store (the first of them in v already).  A choice that was dropped
// has place -1.
template <bool STREAM, class E, int V>
__device__ __forceinline__ void copy_row(const E* x, int H, const int* place, int k, E* rows,
                                         int64_t rs, int c0, int c1, int tid, int nthr,
                                         Chunk<E, V> (&v)[kHeld]) {
  for (int c = c0 + tid; c < c1; c += kHeld * nthr) {
    if (c != c0 + tid) load_row(v, x, H, c, c1, nthr);
    for (int j = 0; j < k; ++j) {
      const int p = place[j];
      if (p < 0) continue;
      E* const out = rows + (int64_t)p * rs;
#pragma unroll
      for (int h = 0; h < kHeld; ++h)
        if (c + h * nthr < c1) store_chunk<STREAM>(out + chunk_at<V>(c + h * nthr, H), v[h]);
    }
  }
}

// A row of H elements by G neighbouring lanes (G > 64: the whole workgroup): its scale and its
// codes, computed once.  The row stays in registers between the maximum and the codes if G lanes
// hold it (kHeld chunks each, loaded by load_row before), else the rest is read twice.
// put(at, codes): the codes of the chunk that starts at element `at`.
template <int G, class E, int V, class Put>
__device__ __forceinline__ RowQuant quant_row(const E* x, int H, int lane, uint32_t* s_max,
                                              const Chunk<E, V> (&v)[kHeld], Put&& put) {
  const int nc = chunk_count<V>(H);
  uint32_t m = 0;
#pragma unroll
  for (int h = 0; h < kHeld; ++h)
    if (lane + h * G < nc) m = chunk_max_bits(v[h], m);
  for (int c = lane + kHeld * G; c < nc; c += G)
    m = chunk_max_bits(load_chunk<V>(x + chunk_at<V>(c, H)), m);
  if constexpr (G <= 64) {
    m = group_max_u32<G>(m);
  } else {
    m = group_max_u32<64>(m);
    if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < G / 64; ++w) m = m > s_max[w] ? m : s_max[w];
  }
  const RowQuant r = row_quant(m);
#pragma unroll
  for (int h = 0; h < kHeld; ++h)
    if (lane + h * G < nc) put(chunk_at<V>(lane + h * G, H), quant_chunk(v[h], r));
  for (int c = lane + kHeld * G; c < nc; c += G) {
    const int at = chunk_at<V>(c, H);
    put(at, quant_chunk(load_chunk<V>(x + at), r));
  }
  return r;
}

// The codes of a token's row to its k places.
template <int G, bool STREAM, class E, int V>
__device__ __forceinline__ void quant_row_to(const E* x, int H, const int* place, int k,
                                             int8_t* rows, int64_t rs, float* row_scale, int lane,
                                             uint32_t* s_max, const Chunk<E, V> (&v)[kHeld]) {
  const RowQuant r =
      quant_row<G>(x, H, lane, s_max, v, [&](int at, const Codes<E, V>& codes) {
        for (int j = 0; j < k; ++j) {
          const int p = place[j];
          if (p >= 0) store_codes<STREAM>(rows + (int64_t)p * rs + at, codes);
        }
      });
  if (lane < k && place[lane] >= 0) row_scale[place[lane]] = r.scale;
}

// first_of[0..E] (LDS or global) = exclusive prefix of total[0..E-1] (LDS), by one workgroup of nthr
// threads, whose writes are not synchronised yet when it returns.
__device__ void prefix_counts(const int* total, int E, int* first_of, int* s_wave, int tid,
                              int nthr) {
  const int per = (E + nthr - 1) / nthr;
  int sum = 0;
  for (int i = 0; i < per; ++i) {
    const int e = tid * per + i;
    if (e < E) sum += total[e];
  }
  int inc = sum;  // inclusive over the lanes of the wave
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
    const int e = tid * per + i;
    if (e < E) {
      first_of[e] = first;
      first += total[e];
      if (e == E - 1) first_of[E] = first;
    }
  }
}

// Few assignments: one launch.  Workgroup (t, y) counts, over all N ids, those before each of
// token t's k assignments (a wave takes 64 ids at a time and adds up ballots), and moves column
// slice y of the token's row; workgroup (T, 0) writes the offsets.  Latency is what it costs: one
// read of the ids (L2), one barrier, one read and k writes of the row.
template <class E, int V, bool I8>
__global__ __launch_bounds__(TOK_T) void sort_small_kernel(SortArgs a) {
  __shared__ int s_cnt[TOK_T / 64][kMaxTopK];
  __shared__ int s_place[kMaxTopK];
  __shared__ int s_hist[kMaxExperts];
  __shared__ int s_wave[TOK_T / 64];
  __shared__ uint32_t s_max[TOK_T / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int t = blockIdx.x;
  if (t == a.T) {
    if (blockIdx.y != 0) return;
    for (int e = tid; e < a.E; e += TOK_T) s_hist[e] = 0;
    __syncthreads();
    for (int i = tid; i < a.N; i += TOK_T) {
      const int id = a.ids[i];
      if ((unsigned)id < (unsigned)a.E) atomicAdd(&s_hist[id], 1);
    }
    __syncthreads();
    prefix_counts(s_hist, a.E, a.offsets, s_wave, tid, TOK_T);
    return;
  }
  const E* x = (const E*)a.x + (int64_t)t * a.xs;
  // this workgroup's slice of the row, under way while the ids are counted
  const int nc = a.x ? chunk_count<V>(a.H) : 0;
  const int per = (nc + gridDim.y - 1) / gridDim.y;
  const int c0 = blockIdx.y * per, c1 = min(nc, c0 + per);
  Chunk<E, V> v[kHeld];
  load_row(v, x, a.H, c0 + tid, c1, TOK_T);
  int own[kMaxTopK], cnt[kMaxTopK];
  const int mine = lane < a.k ? key_of_id(a.ids[t * a.k + lane], a.E) : 0;
#pragma unroll
  for (int j = 0; j < kMaxTopK; ++j) {
    own[j] = __builtin_amdgcn_readlane(mine, j);
    cnt[j] = 0;
  }
  constexpr int AHEAD = 8;  // ids of a lane in flight
  for (int i0 = wave * 64; i0 < a.N; i0 += AHEAD * TOK_T) {
    int id[AHEAD];
#pragma unroll
    for (int h = 0; h < AHEAD; ++h) {
      const int i = i0 + h * TOK_T + lane;
      id[h] = i < a.N ? a.ids[i] : -1;
    }
#pragma unroll
    for (int h = 0; h < AHEAD; ++h) {
      const int i = i0 + h * TOK_T + lane;
      if (i - lane >= a.N) break;
      const int key = key_of_id(id[h], a.E);
#pragma unroll
      for (int j = 0; j < kMaxTopK; ++j)
        if (j < a.k)
          cnt[j] += __popcll(__ballot(key < own[j] || (key == own[j] && i < t * a.k + j)));
    }
  }
#pragma unroll
  for (int j = 0; j < kMaxTopK; ++j)
    if (j < a.k && lane == 0)
      s_cnt[wave][j] = own[j] == 0x7fffffff ? -kSmallIds : cnt[j];
  __syncthreads();
  if (tid < a.k) {
    int p = 0;
#pragma unroll
    for (int w = 0; w < TOK_T / 64; ++w) p += s_cnt[w][tid];
    const int at = t * a.k + tid;
    if (p < 0) p = -1;
    s_place[tid] = p;
    if (blockIdx.y == 0) {
      a.place[at] = p;
      if (a.order && p >= 0) a.order[p] = at;
    }
  }
  __syncthreads();
  if (!a.x) return;
  if constexpr (I8)  // one slice
    quant_row_to<TOK_T, false>(x, a.H, s_place, a.k, (int8_t*)a.rows, a.rs, a.row_scale, tid,
                               s_max, v);
  else
    copy_row<false>(x, a.H, s_place, a.k, (E*)a.rows, a.rs, c0, c1, tid, TOK_T, v);
}

// Many assignments, first of two or three launches: the ids of each chunk counted by expert.
__global__ __launch_bounds__(TOK_T) void sort_count_kernel(SortArgs a) {
  __shared__ int s_hist[kMaxExperts];
  const int b = blockIdx.x;
  for (int e = threadIdx.x; e < a.E; e += TOK_T) s_hist[e] = 0;
  __syncthreads();
  const int i1 = min(a.N, (b + 1) * a.tok_blk * a.k);
  for (int i = b * a.tok_blk * a.k + threadIdx.x; i < i1; i += TOK_T) {
    const int id = a.ids[i];
    if ((unsigned)id < (unsigned)a.E) atomicAdd(&s_hist[id], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += TOK_T) a.base[(int64_t)b * a.E + e] = s_hist[e];
}

// Second, where there are more than kSelfChunks chunks: a workgroup takes 16 experts and turns the
// counts of each chunk into those of the chunks before it.  Thread (g, e) adds up segment g of the
// chunks of expert e, a wave per expert scans the segments, and the running count is written
// over each chunk's.  128 chunks of 128 experts 4.8 us, 1024 of 1024 6.2 (one workgroup for all
// experts took 412).
__global__ __launch_bounds__(SCAN_T) void sort_scan_kernel(SortArgs a) {
  __shared__ int s_seg[kScanExperts][kScanSegs + 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int el = tid % kScanExperts, g = tid / kScanExperts;
  const int e = blockIdx.x * kScanExperts + el;
  const int per = (a.nblk + kScanSegs - 1) / kScanSegs;
  const int b0 = min(a.nblk, g * per), n = e < a.E ? min(a.nblk, b0 + per) - b0 : 0;
  int* const base = a.base + (int64_t)b0 * a.E + e;
  // the counts of up to kScanHeld chunks stay in registers between the passes
  int held[kScanHeld];
  int sum = 0;
#pragma unroll
  for (int i = 0; i < kScanHeld; ++i) held[i] = i < n ? base[(int64_t)i * a.E] : 0;
#pragma unroll
  for (int i = 0; i < kScanHeld; ++i) sum += held[i];
#pragma unroll 8
  for (int i = kScanHeld; i < n; ++i) sum += base[(int64_t)i * a.E];
  s_seg[el][g] = sum;
  __syncthreads();
  {
    static_assert(kScanSegs == 64 && SCAN_T / 64 == kScanExperts);
    const int v = s_seg[wave][lane];
    int inc = v;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const int o = __shfl_up(inc, s);
      if (lane >= s) inc += o;
    }
    s_seg[wave][lane] = inc - v;
    const int mine = blockIdx.x * kScanExperts + wave;
    if (lane == 63 && mine < a.E) a.total[mine] = inc;
  }
  __syncthreads();
  int run = s_seg[el][g];
#pragma unroll
  for (int i = 0; i < kScanHeld; ++i) {
    if (i < n) base[(int64_t)i * a.E] = run;
    run += held[i];
  }
  for (int i = kScanHeld; i < n; ++i) {
    const int v = base[(int64_t)i * a.E];
    base[(int64_t)i * a.E] = run;
    run += v;
  }
}

// Last: a workgroup takes `sub` tokens of a chunk, ranks the chunk's ids up to its own last one (a
// wave finds the lanes that hold its id by ballots over the id's bits; counts per wave and expert
// in LDS), writes their places and moves their rows, a wave per token or (WIDE) all waves on one
// token after the other, the next token's row under way while one is written.  SELF: the counts
// are few enough that each workgroup adds them up itself instead of a launch between (1024 tokens
// of 8: 16 us in all, 24 with the launch and 16 tokens per workgroup).  16384 tokens of 8 rows of
// 2048 bf16: 104 us for 605 MB, 5.8 TB/s, the rate of writes.
template <class E, int V, bool I8, bool WIDE, bool STREAM, bool SELF>
__global__ __launch_bounds__(TOK_T) void sort_move_kernel(SortArgs a, int sub, int subs) {
  extern __shared__ __align__(16) uint16_t s_cnt[];  // [kChunkWaves][E]
  static_assert(kSubTokens * kMaxTopK <= kSubIds && kSubIds <= TOK_T);
  __shared__ int s_id[kSubIds], s_rank[kSubIds], s_place[kSubIds];
  __shared__ uint32_t s_max[2][TOK_T / 64];
  __shared__ int s_first[kMaxExperts + 1], s_total[kMaxExperts];
  __shared__ int s_wave[TOK_T / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int b = blockIdx.x / subs;
  const int t_blk = b * a.tok_blk;
  const int t0 = t_blk + (blockIdx.x % subs) * sub;
  const int t1 = min(min(a.T, t_blk + a.tok_blk), t0 + sub);
  if (t0 >= t1) return;
  int before[kMaxExperts / TOK_T];  // SELF: in the chunks before this one
#pragma unroll
  for (int q = 0; q < kMaxExperts / TOK_T; ++q) {
    const int e = tid + q * TOK_T;
    before[q] = 0;
    if (e >= a.E) continue;
    if constexpr (SELF) {
      int cnt[kSelfChunks], sum = 0;
#pragma unroll
      for (int c = 0; c < kSelfChunks; ++c) cnt[c] = c < a.nblk ? a.base[c * a.E + e] : 0;
#pragma unroll
      for (int c = 0; c < kSelfChunks; ++c) {
        before[q] += c < b ? cnt[c] : 0;
        sum += cnt[c];
      }
      s_total[e] = sum;
    } else {
      s_total[e] = a.total[e];
    }
  }
  __syncthreads();
  prefix_counts(s_total, a.E, s_first, s_wave, tid, TOK_T);
  __syncthreads();
  if (blockIdx.x == 0)
    for (int e = tid; e <= a.E; e += TOK_T) a.offsets[e] = s_first[e];
  if constexpr (SELF) {
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kMaxExperts / TOK_T; ++q)
      if (tid + q * TOK_T < a.E) s_first[tid + q * TOK_T] += before[q];
  }
  const int first = t_blk * a.k, own0 = (t0 - t_blk) * a.k, own1 = (t1 - t_blk) * a.k;
  const int waves = (own1 + 63) / 64;
  for (int i = tid; i < waves * a.E; i += TOK_T) s_cnt[i] = 0;
  __syncthreads();
  for (int it = wave; it < waves; it += TOK_T / 64) {
    const int i = it * 64 + lane;
    const int id = i < own1 ? a.ids[first + i] : -1;
    const bool ok = (unsigned)id < (unsigned)a.E;
    uint64_t same = __ballot(ok);
    for (int bit = 0; (a.E - 1) >> bit; ++bit) {
      const uint64_t set = __ballot((id >> bit) & 1);
      same &= (id >> bit) & 1 ? set : ~set;
    }
    const int rank = __popcll(same & lanemask_lt());
    if (ok && rank == 0) s_cnt[it * a.E + id] = (uint16_t)__popcll(same);
    if (i >= own0 && i < own1) {
      s_id[i - own0] = ok ? id : -1;
      s_rank[i - own0] = rank;
    }
  }
  __syncthreads();
  if (tid < own1 - own0) {
    const int i = own0 + tid, id = s_id[tid];
    int p = -1;
    if (id >= 0) {
      p = s_rank[tid] + s_first[id];
      if constexpr (!SELF) p += a.base[(int64_t)b * a.E + id];
      for (int it = 0; it < i / 64; ++it) p += s_cnt[it * a.E + id];
      if (a.order) a.order[p] = first + i;
    }
    a.place[first + i] = p;
    s_place[tid] = p;
  }
  __syncthreads();
  if (!a.x) return;
  const int nc = chunk_count<V>(a.H);
  constexpr int G = WIDE ? TOK_T : 64;
  constexpr int STEP = WIDE ? 1 : TOK_T / 64;
  const int l = WIDE ? tid : lane;
  const E* x = (const E*)a.x + (int64_t)t0 * a.xs;
  int t = WIDE ? 0 : wave;  // of the workgroup's tokens
  Chunk<E, V> v[kHeld], next[kHeld];
  if (t < t1 - t0) load_row(v, x + (int64_t)t * a.xs, a.H, l, nc, G);
  for (; t < t1 - t0; t += STEP) {
    if (t + STEP < t1 - t0) load_row(next, x + (int64_t)(t + STEP) * a.xs, a.H, l, nc, G);
    const int* place = s_place + t * a.k;
    if constexpr (I8)
      quant_row_to<G, STREAM>(x + (int64_t)t * a.xs, a.H, place, a.k, (int8_t*)a.rows, a.rs,
                              a.row_scale, l, s_max[t & 1], v);
    else
      copy_row<STREAM>(x + (int64_t)t * a.xs, a.H, place, a.k, (E*)a.rows, a.rs, 0, nc, l, G, v);
#pragma unroll
    for (int h = 0; h < kHeld; ++h) v[h] = next[h];
  }
}

struct CombineArgs {
  const void* rows;
  int64_t rs;
  int n_rows;
  const int* place;
  const float* w;  // null: 1
  int T, k, H;
  void* out;
  int64_t os;
  int tpt_log;  // log2 of the threads per token
};

// y[t] = sum_j w[t][j] rows[place[t][j]], fp32, j ascending, rounded once.  A thread holds one
// 16-byte chunk of one token's row and has the loads of eight choices in flight; 2^tpt_log
// threads share a token (UNI: whole waves do, so places and weights are scalar loads).  16384
// tokens of 8 rows of 2048 bf16: 104 us, 5.8 TB/s, bound by the rows' reads.
template <class E, int V, bool W, bool UNI, bool STREAM>
__global__ __launch_bounds__(TOK_T) void combine_kernel(CombineArgs a) {
  constexpr int HELD = 8;
  const int64_t g = (int64_t)blockIdx.x * TOK_T + threadIdx.x;
  int t = (int)(g >> a.tpt_log);
  if constexpr (UNI) t = __builtin_amdgcn_readfirstlane(t);
  const int c = (int)(g & ((1 << a.tpt_log) - 1)) + ((int)blockIdx.y << a.tpt_log);
  if (t >= a.T || c >= chunk_count<V>(a.H)) return;
  const int col = chunk_at<V>(c, a.H);
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  const int* place = a.place + (int64_t)t * a.k;
  const float* w = W ? a.w + (int64_t)t * a.k : nullptr;
  const E* rows = (const E*)a.rows + col;
  for (int j0 = 0; j0 < a.k; j0 += HELD) {
    Chunk<E, V> v[HELD];
    bool in[HELD];
#pragma unroll
    for (int h = 0; h < HELD; ++h) {
      const int p = j0 + h < a.k ? place[j0 + h] : -1;
      in[h] = (unsigned)p < (unsigned)a.n_rows;
      if (in[h]) v[h] = load_chunk<V, STREAM>(rows + (int64_t)p * a.rs);
    }
#pragma unroll
    for (int h = 0; h < HELD; ++h) {
      if (!in[h]) continue;
      const float wj = W ? w[j0 + h] : 1.f;
#pragma unroll
      for (int i = 0; i < V; ++i)
        acc[i] = W ? fmaf(wj, to_f32(v[h].e[i]), acc[i]) : acc[i] + to_f32(v[h].e[i]);
    }
  }
  store_chunk((E*)a.out + (int64_t)t * a.os + col, round_chunk<E, V>(acc));
}

struct CombineGradArgs {
  const void* dout;
  int64_t ds;
  const void* rows;  // null without dw
  int64_t rs;
  int n_rows;
  const int* place;
  const float* w;  // null: 1
  int T, k, H;
  void* drows;  // may be null
  int64_t drs;
  float* dw;  // may be null
};

// A wave per assignment: drows[p] = w dy, dw = <dy, rows[p]> (fp32 within a chunk, 64 bits over
// the chunks and lanes, where a long sum may cancel; joined by shuffles in a fixed order), four
// chunks of each row in flight.  The waves of a token read its dy row together: of 16384 tokens of
// 8 rows of 2048 bf16 1.22 GB move for 1.14, in 205 us.
template <class E, int V, bool STREAM>
__global__ __launch_bounds__(TOK_T) void combine_grad_kernel(CombineGradArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t at = (int64_t)blockIdx.x * (TOK_T / 64) +
                     __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (at >= (int64_t)a.T * a.k) return;
  const int p = a.place[at];
  if ((unsigned)p >= (unsigned)a.n_rows) {
    if (a.dw && lane == 0) a.dw[at] = 0.f;
    return;
  }
  const float w = a.w[at];
  const E* dy = (const E*)a.dout + at / a.k * a.ds;
  const E* r = (const E*)a.rows + (int64_t)p * a.rs;
  E* dr = (E*)a.drows + (int64_t)p * a.drs;
  const int nc = chunk_count<V>(a.H);
  double sum = 0.0;
  for (int c0 = lane; c0 < nc; c0 += 64 * kHeld) {
    Chunk<E, V> g[kHeld], v[kHeld];
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
      const int c = c0 + 64 * h;
      if (c < nc) {
        g[h] = load_chunk<V>(dy + chunk_at<V>(c, a.H));
        if (a.dw) v[h] = load_chunk<V, STREAM>(r + chunk_at<V>(c, a.H));
      }
    }
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
      const int c = c0 + 64 * h;
      if (c >= nc) continue;
      const int at = chunk_at<V>(c, a.H);
      if (a.drows) {
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = w * to_f32(g[h].e[i]);
        store_chunk<STREAM>(dr + at, round_chunk<E, V>(o));
      }
      if (a.dw) {
        const int twice = c * V - at;  // elements that the chunk before has added up
        float part = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float f = fmaf(to_f32(g[h].e[i]), to_f32(v[h].e[i]), part);
          part = i >= twice ? f : part;
        }
        sum += part;
      }
    }
  }
  if (a.dw) {
    sum = wave_sum(sum);
    if (lane == 0) a.dw[at] = (float)sum;
  }
}

struct QuantArgs {
  const void* x;
  int64_t xs;
  int M, K;
  int8_t* codes;
  int64_t cs;
  float* scale;
  const int* rows_end;  // may be null
};

// G lanes per row (G = 256: a workgroup); one read of the row where they hold it.  131072 rows of
// 768 bf16: 51 us, 5.9 TB/s; about eight instructions per element keep the arithmetic below that
// (a fully rounded division each took 104 us).
template <class E, int V, int G, bool STREAM>
__global__ __launch_bounds__(TOK_T) void quantise_kernel(QuantArgs a) {
  __shared__ uint32_t s_max[TOK_T / 64];
  const int lane = threadIdx.x % G, row = blockIdx.x * (TOK_T / G) + threadIdx.x / G;
  const int end = a.rows_end ? min(*a.rows_end, a.M) : a.M;
  if (row >= end) return;
  int8_t* codes = a.codes + (int64_t)row * a.cs;
  const E* x = (const E*)a.x + (int64_t)row * a.xs;
  Chunk<E, V> v[kHeld];
  load_row(v, x, a.K, lane, chunk_count<V>(a.K), G);
  const RowQuant r = quant_row<G>(x, a.K, lane, s_max, v, [&](int at, const Codes<E, V>& q) {
    store_codes<STREAM>(codes + at, q);
  });
  if (lane == 0) a.scale[row] = r.scale;
}

// ------------------------------------------------------------------ host side

bool tokens_ok(int T, int k, int E) {
  return T >= 0 && T <= kMaxT && k >= 1 && k <= kMaxTopK && E >= 1 && E <= kMaxExperts;
}
bool float_type(int type) { return type >= MOE_T_BF16 && type <= MOE_T_FP32; }
bool aligned4(const void* p) { return ((uintptr_t)p & 3) == 0; }
constexpr int kMaxCols = 1 << 20;

int block_tokens(int k) { return kChunkIds / k; }
int block_count(int T, int k) { return (T + block_tokens(k) - 1) / block_tokens(k); }

// The move kernel of a launch.  Rows below 16 bytes (V = 1) are never streamed as codes (2^24 rows of 7
// stay below kStreamBytes), nor where tokens are few enough for WIDE.
template <class E, int V, bool I8, bool WIDE>
auto move_kernel(bool self, bool stream) {
  if (self) return sort_move_kernel<E, V, I8, WIDE, false, true>;
  if constexpr (V > 1 || !(I8 || WIDE))
    if (stream) return sort_move_kernel<E, V, I8, WIDE, true, false>;
  return sort_move_kernel<E, V, I8, WIDE, false, false>;
}

template <class E, int V, bool I8>
hipError_t launch_sort_by(SortArgs& a, hipStream_t s) {
  const int nc = a.x ? chunk_count<V>(a.H) : 0;
  if (a.N <= kSmallIds) {
    const int slices = I8 ? 1 : std::max(1, std::min(64, (nc + TOK_T - 1) / TOK_T));
    return launch_kernel(sort_small_kernel<E, V, I8>, dim3(a.T + 1, slices), dim3(TOK_T), 0, s, a);
  }
  // each reads what the one before leaves in the workspace, so none follows a failed one
  hipError_t e = launch_kernel(sort_count_kernel, dim3(a.nblk), dim3(TOK_T), 0, s, a);
  const bool self = a.nblk <= kSelfChunks;
  if (e == hipSuccess && !self)
    e = launch_kernel(sort_scan_kernel, dim3((a.E + kScanExperts - 1) / kScanExperts), dim3(SCAN_T),
                      0, s, a);
  if (e != hipSuccess) return e;
  // a wave per token, unless there are too few tokens for that to fill the chip, or rows of codes
  // that a wave cannot hold; 16 tokens per workgroup amortise its counting, fewer fill the chip
  // (8 rows of 2048 bf16 per token: 4096 tokens 36 us with 4, 41 with 4 and whole workgroups per
  // token; 1024 tokens of 8 rows of 4096, quantised: 18 us with one per workgroup, 64 with 16)
  const bool wide = a.T < 2048 || (I8 && nc > 64 * kHeld);
  int sub = a.T < 2048 ? 1 : a.T < 8192 ? 4 : kSubTokens;
  // and where few choices make for few ids per token, as many as leave 1024 workgroups
  if (a.T > 1024 * kSubTokens) sub = std::max(sub, std::min(a.T / 1024, kSubIds / 2 / a.k));
  const bool stream = (int64_t)a.N * a.H * (I8 ? 1 : (int)sizeof(E)) > kStreamBytes;
  const auto kernel = wide ? move_kernel<E, V, I8, true>(self, stream)
                           : move_kernel<E, V, I8, false>(self, stream);
  const int subs = (a.tok_blk + sub - 1) / sub;
  return launch_kernel(kernel, dim3(a.nblk * subs), dim3(TOK_T), (size_t)kChunkWaves * a.E * 2, s, a,
                       sub, subs);
}

// Rows shorter than a chunk go element by element, in all the launches.
template <class E, bool I8>
hipError_t launch_sort(SortArgs& a, hipStream_t s) {
  return a.H >= kChunk<E> || !a.x ? launch_sort_by<E, kChunk<E>, I8>(a, s)
                                  : launch_sort_by<E, 1, I8>(a, s);
}

// A row of 16 bytes at least may have a wave to itself (uni), a shorter one never has.
template <class E, int V, bool W>
auto combine_kernel_for(bool uni, bool stream) {
  if constexpr (V > 1)
    if (uni) return stream ? combine_kernel<E, V, W, true, true> : combine_kernel<E, V, W, true, false>;
  return combine_kernel<E, V, W, false, false>;
}

template <class E, int V>
hipError_t launch_combine_by(CombineArgs& a, hipStream_t s) {
  const int nc = chunk_count<V>(a.H);
  a.tpt_log = 0;
  while (a.tpt_log < 8 && (1 << a.tpt_log) < nc) ++a.tpt_log;
  const int64_t thr = (int64_t)a.T << a.tpt_log;
  const dim3 grid((unsigned)((thr + TOK_T - 1) / TOK_T),
                  (unsigned)((nc + (1 << a.tpt_log) - 1) >> a.tpt_log));
  const bool uni = a.tpt_log >= 6;
  const bool stream = (int64_t)a.T * a.k * a.H * (int)sizeof(E) > kStreamBytes;
  const auto kernel = a.w ? combine_kernel_for<E, V, true>(uni, stream)
                          : combine_kernel_for<E, V, false>(uni, stream);
  return launch_kernel(kernel, grid, dim3(TOK_T), 0, s, a);
}
template <class E>
hipError_t launch_combine(CombineArgs& a, hipStream_t s) {
  return a.H >= kChunk<E> ? launch_combine_by<E, kChunk<E>>(a, s) : launch_combine_by<E, 1>(a, s);
}

template <class E>
hipError_t launch_combine_grad(const CombineGradArgs& a, hipStream_t s) {
  const bool stream = (int64_t)a.T * a.k * a.H * (int)sizeof(E) > kStreamBytes;
  const auto kernel = a.H < kChunk<E> ? combine_grad_kernel<E, 1, false>
                      : stream        ? combine_grad_kernel<E, kChunk<E>, true>
                                      : combine_grad_kernel<E, kChunk<E>, false>;
  return launch_kernel(kernel, dim3((unsigned)((a.T * a.k + TOK_T / 64 - 1) / (TOK_T / 64))),
                       dim3(TOK_T), 0, s, a);
}

template <class E, int V, int G>
hipError_t launch_quantise_by(const QuantArgs& a, hipStream_t s) {
  constexpr int rows = TOK_T / G;
  const bool stream = (int64_t)a.M * a.K * (int)sizeof(E) > kStreamBytes;
  const auto kernel = stream ? quantise_kernel<E, V, G, true> : quantise_kernel<E, V, G, false>;
  return launch_kernel(kernel, dim3((unsigned)(((int64_t)a.M + rows - 1) / rows)), dim3(TOK_T), 0, s,
                       a);
}

// As few lanes per row as hold it in kHeld chunks each.
template <class E>
hipError_t launch_quantise(const QuantArgs& a, hipStream_t s) {
  constexpr int V = kChunk<E>;
  const int nc = chunk_count<V>(a.K);
  if (a.K < V) return launch_quantise_by<E, 1, 16>(a, s);
  if (nc <= 16 * kHeld) return launch_quantise_by<E, V, 16>(a, s);
  if (nc <= 32 * kHeld) return launch_quantise_by<E, V, 32>(a, s);
  if (nc <= 64 * kHeld) return launch_quantise_by<E, V, 64>(a, s);
  return launch_quantise_by<E, V, 256>(a, s);
}

moe_status combine(const void* rows, int64_t rs, int n_rows, int type, const int* place,
                   const float* w, int T, int k, int H, void* out, int64_t os, hipStream_t s) {
  if (!float_type(type) || !tokens_ok(T, k, 1) || H < 1 || H > kMaxCols || n_rows < 0)
    return MOE_E_INVALID;
  if (T == 0) return MOE_OK;  // before the pointers: empty buffers have none
  if (!place || !aligned4(place) || !aligned4(w) || !rows_ok(out, os, H, type) ||
      (n_rows > 0 && !rows_ok(rows, rs, H, type)) || !on_current_device(out))
    return MOE_E_INVALID;
  CombineArgs a{rows, rs, n_rows, place, w, T, k, H, out, os, 0};
  if (type == MOE_T_BF16) return launched(launch_combine<bf16_t>(a, s));
  if (type == MOE_T_FP16) return launched(launch_combine<fp16_t>(a, s));
  return launched(launch_combine<float>(a, s));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_sort_workspace_bytes(int32_t T, int32_t top_k, int32_t experts) {
  if (!tokens_ok(T, top_k, experts) || T * top_k <= kSmallIds) return 0;
  return sizeof(int) * (size_t)(block_count(T, top_k) + 1) * (size_t)experts;
}

moe_status moe_sort_tokens(const int32_t* topk_idx, int32_t T, int32_t top_k, int32_t experts,
                           int32_t* offsets, int32_t* order, int32_t* place, const void* x,
                           int64_t x_stride, int32_t hidden, int32_t x_type, void* rows,
                           int64_t rows_stride, int32_t rows_type, float* row_scale,
                           void* workspace, size_t workspace_bytes, void* stream) {
  if (!tokens_ok(T, top_k, experts) || !offsets || !aligned4(offsets) || !aligned4(order))
    return MOE_E_INVALID;
  if (T > 0 && (!topk_idx || !place || !aligned4(topk_idx) || !aligned4(place)))
    return MOE_E_INVALID;
  const bool i8 = (x || rows) && rows_type == MOE_T_I8;
  if ((x || rows) && (!float_type(x_type) || (rows_type != x_type && !i8) || hidden < 1 ||
                      hidden > kMaxCols))
    return MOE_E_INVALID;
  if (T == 0) x = rows = nullptr;  // either may be an empty buffer, which has no address
  if ((x == nullptr) != (rows == nullptr)) return MOE_E_INVALID;
  if (x) {
    if (!rows_ok(x, x_stride, hidden, x_type) || !rows_ok(rows, rows_stride, hidden, rows_type))
      return MOE_E_INVALID;
    if (i8 && (!row_scale || !aligned4(row_scale))) return MOE_E_INVALID;
  }
  const size_t need = moe_sort_workspace_bytes(T, top_k, experts);
  if (need && (!workspace || !aligned4(workspace))) return MOE_E_INVALID;
  if (workspace_bytes < need) return MOE_E_SCRATCH;
  if (!on_current_device(offsets)) return MOE_E_INVALID;
  const int nblk = block_count(T, top_k);
  int* const base = (int*)workspace;
  SortArgs a{topk_idx, T,     top_k, experts, T * top_k, x,           x_stride,  hidden,
             offsets,  order, place, rows,    rows_stride, row_scale, base,
             need ? base + (size_t)nblk * experts : nullptr, block_tokens(top_k), nblk};
  const hipStream_t s = (hipStream_t)stream;
  const int type = x ? x_type : MOE_T_FP32;
  if (type == MOE_T_BF16)
    return launched(i8 ? launch_sort<bf16_t, true>(a, s) : launch_sort<bf16_t, false>(a, s));
  if (type == MOE_T_FP16)
    return launched(i8 ? launch_sort<fp16_t, true>(a, s) : launch_sort<fp16_t, false>(a, s));
  return launched(i8 ? launch_sort<float, true>(a, s) : launch_sort<float, false>(a, s));
}

moe_status moe_sort_tokens_grad(const void* drows, int64_t drows_stride, int32_t n_rows,
                                int32_t type, const int32_t* place, int32_t T, int32_t top_k,
                                int32_t hidden, void* dx, int64_t dx_stride, void* stream) {
  return combine(drows, drows_stride, n_rows, type, place, nullptr, T, top_k, hidden, dx,
                 dx_stride, (hipStream_t)stream);
}

moe_status moe_combine_tokens(const void* rows, int64_t rows_stride, int32_t n_rows, int32_t type,
                              const int32_t* place, const float* weights, int32_t T,
                              int32_t top_k, int32_t hidden, void* out, int64_t out_stride,
                              void* stream) {
  if (!weights && T != 0) return MOE_E_INVALID;
  return combine(rows, rows_stride, n_rows, type, place, weights, T, top_k, hidden, out,
                 out_stride, (hipStream_t)stream);
}

moe_status moe_combine_tokens_grad(const void* dout, int64_t dout_stride, const void* rows,
                                   int64_t rows_stride, int32_t n_rows, int32_t type,
                                   const int32_t* place, const float* weights, int32_t T,
                                   int32_t top_k, int32_t hidden, void* drows,
                                   int64_t drows_stride, float* dweights, void* stream) {
  if (!float_type(type) || !tokens_ok(T, top_k, 1) || hidden < 1 || hidden > kMaxCols || n_rows < 0)
    return MOE_E_INVALID;
  if (T == 0) return MOE_OK;  // before the pointers: empty buffers have none
  if (!place || !weights || !aligned4(place) || !aligned4(weights) || !aligned4(dweights) ||
      (!drows && !dweights && n_rows > 0) || !rows_ok(dout, dout_stride, hidden, type) ||
      (drows && !rows_ok(drows, drows_stride, hidden, type)) ||
      (dweights && n_rows > 0 && !rows_ok(rows, rows_stride, hidden, type)) ||
      !on_current_device(dout))
    return MOE_E_INVALID;
  if (!drows && !dweights) return MOE_OK;  // no rows to give a gradient to
  CombineGradArgs a{dout, dout_stride, rows, rows_stride, n_rows, place, weights, T,
                    top_k, hidden, drows, drows_stride, dweights};
  const hipStream_t s = (hipStream_t)stream;
  if (type == MOE_T_BF16) return launched(launch_combine_grad<bf16_t>(a, s));
  if (type == MOE_T_FP16) return launched(launch_combine_grad<fp16_t>(a, s));
  return launched(launch_combine_grad<float>(a, s));
}

moe_status moe_quantise_rows(const void* x, int64_t x_stride, int32_t type, int32_t M, int32_t K,
                             int8_t* codes, int64_t codes_stride, float* scale,
                             const int32_t* rows_end, void* stream) {
  if (!float_type(type) || M < 0 || M > kMaxRows || K < 1 || K > kMaxCols) return MOE_E_INVALID;
  if (M == 0) return MOE_OK;  // before the pointers: empty buffers have none
  if (!rows_ok(x, x_stride, K, type) || !rows_ok(codes, codes_stride, K, MOE_T_I8) || !scale ||
      !aligned4(scale) || !aligned4(rows_end) || !on_current_device(codes))
    return MOE_E_INVALID;
  QuantArgs a{x, x_stride, M, K, codes, codes_stride, scale, rows_end};
  const hipStream_t s = (hipStream_t)stream;
  if (type == MOE_T_BF16) return launched(launch_quantise<bf16_t>(a, s));
  if (type == MOE_T_FP16) return launched(launch_quantise<fp16_t>(a, s));
  return launched(launch_quantise<float>(a, s));
}

}  // extern "C"
