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

// One 16-byte chunk of a row: V elements.
template <class E>
union Chunk {
  static constexpr int V = 16 / (int)sizeof(E);
  u32x4 q;
  E e[V];
};

// V values rounded to a chunk (two at a time: one instruction converts a pair).
template <class E>
__device__ __forceinline__ Chunk<E> round_chunk(const float* v) {
  Chunk<E> c;
  if constexpr (sizeof(E) == 2) {
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

// The chunk at p, of which the first n elements belong to the row (n >= V: all); elements past
// the row are not touched and read as zero.  STREAM: nothing reads these bytes again soon, so they
// pass the caches by.
template <class E, bool STREAM = false>
__device__ __forceinline__ Chunk<E> load_chunk(const E* p, int n) {
  Chunk<E> c;
  if (n >= Chunk<E>::V) {
    if constexpr (STREAM)
      c.q = __builtin_nontemporal_load((const u32x4_any*)p);
    else
      c.q = *(const u32x4_any*)p;
  } else {
    c.q = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < Chunk<E>::V; ++i)
      if (i < n) c.e[i] = p[i];
  }
  return c;
}
template <class E, bool STREAM = false>
__device__ __forceinline__ void store_chunk(E* p, int n, const Chunk<E>& c) {
  if (n >= Chunk<E>::V) {
    if constexpr (STREAM)
      __builtin_nontemporal_store(c.q, (u32x4_any*)p);
    else
      *(u32x4_any*)p = c.q;
  } else {
#pragma unroll
    for (int i = 0; i < Chunk<E>::V; ++i)
      if (i < n) p[i] = c.e[i];
  }
}

// 8-bit quantisation of a row with m = max |x|: scale = m / 127 and code = 127 x / m rounded to
// the nearest integer, ties to even, exactly (as if computed without rounding).  A row of
// zeros has scale 0 and codes 0; a row that holds a NaN or an infinity has scale NaN and codes
// 0, so that whatever is computed from it is NaN.
struct RowQuant {
  float m, inv, scale;
  int mode;  // 0: codes are zero, 1: fp32 arithmetic, 2: 64-bit arithmetic
};

__device__ __forceinline__ uint32_t abs_bits(float f) { return __float_as_uint(f) & 0x7fffffffu; }

// max_bits: the largest abs_bits() of the row (a NaN's are above infinity's, above a number's).
__device__ __forceinline__ RowQuant row_quant(uint32_t max_bits) {
  RowQuant r;
  r.m = __uint_as_float(max_bits);
  r.inv = 1.0f / r.m;
  r.scale = r.m / 127.0f;
  // fp32: 127 x must not overflow and 1 / m must be a normal number
  r.mode = r.m >= 0x1p-100f && r.m <= 0x1p100f ? 1 : 2;
  if (max_bits == 0) r.mode = 0;
  if (max_bits >= 0x7f800000u) {
    r.mode = 0;
    r.scale = __uint_as_float(0x7fc00000u);
  }
  return r;
}

// The bits of 1.5 * 2^23 + 127 x / m, whose low byte is the code (fp32 addition rounds to
// nearest even at that size).  t = 127 x, y = t / m up to 2 roundings, and y + (t - y m) / m is
// the quotient to half a step: where the quotient is a tie it is a number of fp32 and comes out
// exactly.  16-bit inputs: t is exact (18 bits) and a quotient 127 X 2^e / M that is no tie (X and M
// of 11 bits) is 2^e / 4094 from one at least, its error below 127 * 2^(e - 22): the rounding is
// right.  fp32 inputs: t may be rounded; quotients within 2^-14 of a tie (their error is below
// 2^-15) are decided in 64 bits, where 127 x is exact and a quotient that is no tie differs from
// one by 2^-33 at least.
template <class E>
__device__ __forceinline__ uint32_t quant_bits(float x, const RowQuant& r) {
  const float t = 127.0f * x;
  float y = t * r.inv;
  y = fmaf(fmaf(-y, r.m, t), r.inv, y);
  if constexpr (sizeof(E) == 4) {
    if (fabsf(fabsf(y - rintf(y)) - 0.5f) < 0x1p-14f) y = (float)rint(127.0 * (double)x / (double)r.m);
  }
  return __float_as_uint(y + 12582912.0f);
}
// The same for rows whose largest magnitude fp32 arithmetic does not serve.
__device__ __forceinline__ uint32_t quant_bits_wide(float x, const RowQuant& r) {
  return r.mode == 0 ? 0u : (uint32_t)(int)rint(127.0 * (double)x / (double)r.m);
}

// The codes of one chunk, four to a word.
template <class E>
struct Codes {
  static constexpr int W = Chunk<E>::V / 4;
  uint32_t w[W];
};
template <class E>
__device__ __forceinline__ Codes<E> quant_chunk(const Chunk<E>& c, const RowQuant& r) {
  Codes<E> o;
#pragma unroll
  for (int i = 0; i < Codes<E>::W; ++i) {
    uint32_t b[4];
    if (r.mode == 1) {
#pragma unroll
      for (int k = 0; k < 4; ++k) b[k] = quant_bits<E>(to_f32(c.e[4 * i + k]), r);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) b[k] = quant_bits_wide(to_f32(c.e[4 * i + k]), r);
    }
    const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
    o.w[i] = lo | hi;
  }
  return o;
}
template <class E, bool STREAM = false>
__device__ __forceinline__ void store_codes(int8_t* p, int n, const Codes<E>& c) {
  constexpr int V = Chunk<E>::V;
  if (n >= V) {
    if constexpr (V == 8) {
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
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) p[i] = (int8_t)(c.w[i / 4] >> (8 * (i % 4)));
  }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) v += __shfl_xor(v, s);
  return v;
}

// The larger of m and the largest abs_bits() of a chunk.
template <class E>
__device__ __forceinline__ uint32_t chunk_max_bits(const Chunk<E>& c, uint32_t m) {
  if constexpr (sizeof(E) == 4) {
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
    Chunk<E> big;
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

inline moe_status launched() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_E_HIP; }

}  // namespace moe
