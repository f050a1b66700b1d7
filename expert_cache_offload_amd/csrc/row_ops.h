// Rows of activations in bf16, fp16 or fp32: element types, 16-byte chunks and the 8-bit
// quantisation of a row, shared by the token kernels and the 8-bit product.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moe_offload.h"
#include "moe_dev.h"

namespace moe {

struct bf16_t {
  uint16_t v;
};
typedef _Float16 fp16_t;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// Rows start at any element, so a chunk is only as aligned as an element is; gfx950 loads and
// stores 16 bytes at any byte address in one instruction (the HSA target enables it), and an
// address that happens to be aligned costs nothing extra.
typedef u32x4 u32x4_any __attribute__((aligned(1)));
typedef uint64_t u64_any __attribute__((aligned(1)));
typedef uint32_t u32_any __attribute__((aligned(1)));

__device__ __forceinline__ float to_f32(bf16_t e) { return __uint_as_float((uint32_t)e.v << 16); }
__device__ __forceinline__ float to_f32(fp16_t e) { return (float)e; }
__device__ __forceinline__ float to_f32(float e) { return e; }
template <class E>
__device__ __forceinline__ E from_f32(float f);
template <>
__device__ __forceinline__ bf16_t from_f32<bf16_t>(float f) {
  return bf16_t{__builtin_bit_cast(uint16_t, (__bf16)f)};  // v_cvt_pk_bf16_f32: to nearest even
}
template <>
__device__ __forceinline__ fp16_t from_f32<fp16_t>(float f) {
  return (fp16_t)f;
}
template <>
__device__ __forceinline__ float from_f32<float>(float f) {
  return f;
}

// A chunk of a row: V elements, 16 bytes (or one element, for rows shorter than that).  Chunk c of
// a row of H >= V elements starts at element chunk_at(c): the last one ends with the row and, where
// H is no multiple of V, overlaps the one before; what both write there is the same.
template <class E>
constexpr int kChunk = 16 / (int)sizeof(E);
template <class E, int V = kChunk<E>>
union Chunk {
  u32x4 q;
  E e[V];
};
template <class E>
union Chunk<E, 1> {
  E e[1];
};
template <int V>
__device__ __forceinline__ int chunk_at(int c, int H) {
  return min(c * V, H - V);
}
template <int V>
__host__ __device__ __forceinline__ int chunk_count(int H) {
  return (H + V - 1) / V;
}

// V values rounded to a chunk (two at a time: one instruction converts a pair).
template <class E, int V = kChunk<E>>
__device__ __forceinline__ Chunk<E, V> round_chunk(const float* v) {
  Chunk<E, V> c;
  if constexpr (V == 1) {
    c.e[0] = from_f32<E>(v[0]);
  } else if constexpr (sizeof(E) == 2) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    typedef _Float16 fp16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x2 p = {v[2 * i], v[2 * i + 1]};
      if constexpr (__is_same(E, bf16_t))
        c.q[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf16x2));
      else
        c.q[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, fp16x2));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) c.e[i] = v[i];
  }
  return c;
}

// STREAM: nothing reads these bytes again soon, so they pass the caches by.
template <int V, bool STREAM = false, class E>
__device__ __forceinline__ Chunk<E, V> load_chunk(const E* p) {
  Chunk<E, V> c;
  if constexpr (V == 1)
    c.e[0] = p[0];
  else if constexpr (STREAM)
    c.q = __builtin_nontemporal_load((const u32x4_any*)p);
  else
    c.q = *(const u32x4_any*)p;
  return c;
}
template <bool STREAM = false, class E, int V>
__device__ __forceinline__ void store_chunk(E* p, const Chunk<E, V>& c) {
  if constexpr (V == 1)
    p[0] = c.e[0];
  else if constexpr (STREAM)
    __builtin_nontemporal_store(c.q, (u32x4_any*)p);
  else
    *(u32x4_any*)p = c.q;
}

// 8-bit quantisation of a row with m = max |x|: scale = m / 127 and code = 127 x / m rounded to
// the nearest integer, ties to even, exactly (as if computed without rounding).  A row of
// zeros has scale 0 and codes 0; a row that holds a NaN or an infinity has scale NaN and codes
// 0, so that whatever is computed from it is NaN.
struct RowQuant {
  float m, inv;  // largest magnitude and its reciprocal, scaled by a power of two
  float k;       // 127 times that power: 127 x and 1 / m stay normal numbers of fp32
  float scale;
  bool live;     // false: the codes are zero
};

__device__ __forceinline__ uint32_t abs_bits(float f) { return __float_as_uint(f) & 0x7fffffffu; }

// max_bits: the largest abs_bits() of the row (a NaN's are above infinity's, above a number's).
__device__ __forceinline__ RowQuant row_quant(uint32_t max_bits) {
  RowQuant r;
  const float m = __uint_as_float(max_bits);
  // elements so small beside m that the scaling rounds them have code 0 either way
  const float by = m < 0x1p-60f ? 0x1p100f : m > 0x1p60f ? 0x1p-60f : 1.0f;
  r.m = m * by;
  r.inv = 1.0f / r.m;
  r.k = 127.0f * by;
  r.live = max_bits != 0 && max_bits < 0x7f800000u;
  r.scale = max_bits < 0x7f800000u ? m / 127.0f : __uint_as_float(0x7fc00000u);
  return r;
}

// The bits of 1.5 * 2^23 + code, whose low byte is the code (fp32 addition rounds to nearest even
// at that size).  t = 127 x, y = t / m up to 2 roundings.
// 16-bit inputs: y + (t - y m) / m is the quotient to half a step; t is exact (18 bits), and where
// the quotient is a tie it is a number of fp32 and comes out exactly.  A quotient 127 X 2^e / M that
// is no tie (X and M of 11 bits) is 2^e / 4094 from one at least, its error below
// 127 * 2^(e - 22): the rounding is right.
// fp32 inputs: t + u = 127 x exactly, and so is the remainder t - q m of the candidate q = rint(y),
// a multiple of m's last place below m; its double against m, with u, decides.
template <class E>
__device__ __forceinline__ uint32_t quant_bits(float x, const RowQuant& r) {
  const float t = r.k * x;
  float y = t * r.inv;
  if constexpr (sizeof(E) == 2) {
    y = fmaf(fmaf(-y, r.m, t), r.inv, y);
  } else {
    const float u = -2.0f * fmaf(r.k, x, -t);
    y = rintf(y);
    const float rest = fmaf(-y, r.m, t);
    const float up = fmaf(2.0f, rest, -r.m), down = fmaf(2.0f, rest, r.m);
    const bool odd = (int)y & 1;
    if (up > u || (up == u && odd)) y += 1.0f;
    if (down < u || (down == u && odd)) y -= 1.0f;
  }
  return __float_as_uint(y + 12582912.0f);
}

// The codes of one chunk, four to a word.
template <class E, int V>
struct Codes {
  uint32_t w[(V + 3) / 4];
};
template <class E, int V>
__device__ __forceinline__ Codes<E, V> quant_chunk(const Chunk<E, V>& c, const RowQuant& r) {
  Codes<E, V> o;
  if constexpr (V == 1) {
    o.w[0] = r.live ? quant_bits<E>(to_f32(c.e[0]), r) : 0u;
  } else {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      uint32_t b[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) b[k] = quant_bits<E>(to_f32(c.e[4 * i + k]), r);
      const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u);
      const uint32_t hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
      o.w[i] = r.live ? lo | hi : 0u;
    }
  }
  return o;
}
template <bool STREAM = false, class E, int V>
__device__ __forceinline__ void store_codes(int8_t* p, const Codes<E, V>& c) {
  if constexpr (V == 1) {
    p[0] = (int8_t)c.w[0];
  } else if constexpr (V == 8) {
    const uint64_t v = (uint64_t)c.w[1] << 32 | c.w[0];
    if constexpr (STREAM)
      __builtin_nontemporal_store(v, (u64_any*)p);
    else
      *(u64_any*)p = v;
  } else {
    if constexpr (STREAM)
      __builtin_nontemporal_store(c.w[0], (u32_any*)p);
    else
      *(u32_any*)p = c.w[0];
  }
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) v += __shfl_xor(v, s);
  return v;
}

// The larger of m and the largest abs_bits() of a chunk.
template <class E, int V>
__device__ __forceinline__ uint32_t chunk_max_bits(const Chunk<E, V>& c, uint32_t m) {
  if constexpr (V == 1) {
    const uint32_t b = abs_bits(to_f32(c.e[0]));
    m = m > b ? m : b;
  } else if constexpr (sizeof(E) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t b = c.q[i] & 0x7fffffffu;
      m = m > b ? m : b;
    }
  } else {  // magnitudes of 16 bits order as their bits do: pairs at a time
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 p = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p = __builtin_elementwise_max(p, __builtin_bit_cast(u16x2, c.q[i] & 0x7fff7fffu));
    Chunk<E, V> big;
    big.q.x = p[0] > p[1] ? p[0] : p[1];
    const uint32_t b = abs_bits(to_f32(big.e[0]));
    m = m > b ? m : b;
  }
  return m;
}

// The largest of m over groups of G neighbouring lanes (G <= 64).
template <int G>
__device__ __forceinline__ uint32_t group_max_u32(uint32_t v) {
#pragma unroll
  for (int s = G / 2; s > 0; s >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)v, s);
    v = v > o ? v : o;
  }
  return v;
}

inline size_t elem_bytes(int type) {
  return type == MOE_T_FP32 ? 4 : type == MOE_T_I8 ? 1 : 2;
}
// A row operand: rows of `cols` elements, `stride` elements apart, element aligned.
inline bool rows_ok(const void* p, int64_t stride, int64_t cols, int type) {
  return p && stride >= cols && stride <= ((int64_t)1 << 40) &&
         (uintptr_t)p % elem_bytes(type) == 0;
}

// The buffers' device has to be the current one: kernels are launched there.  Looked up only
// where there is more than one device.
inline bool on_current_device(const void* p) {
  static const int devices = [] {
    int n = 0;
    return hipGetDeviceCount(&n) == hipSuccess ? n : 0;
  }();
  if (devices <= 1) return true;
  int dev = -1;
  hipPointerAttribute_t at{};
  if (hipGetDevice(&dev) != hipSuccess || hipPointerGetAttributes(&at, p) != hipSuccess) {
    (void)hipGetLastError();
    return false;
  }
  return at.device == dev;
}

// A plain launch without the call configuration that the triple-bracket form pushes and pops (0.2 us
// of the host's 3.1 per launch), and its own status: an error that an earlier call of the thread has
// left behind is another's.
template <class... P>
inline hipError_t launch_kernel(void (*kernel)(P...), dim3 grid, dim3 block, size_t lds,
                                hipStream_t s, P... args) {
  void* p[] = {(void*)&args...};
  return hipLaunchKernel((const void*)kernel, grid, block, p, lds, s);
}
inline moe_status launched(hipError_t e) {
  if (e == hipSuccess) return MOE_OK;
  (void)hipGetLastError();  // reported here
  return MOE_E_HIP;
}

}  // namespace moe
