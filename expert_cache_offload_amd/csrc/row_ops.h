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
// the row are not touched and read as zero.
template <class E>
__device__ __forceinline__ Chunk<E> load_chunk(const E* p, int n) {
  Chunk<E> c;
  if (n >= Chunk<E>::V) {
    c.q = *(const u32x4_any*)p;
  } else {
    c.q = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < Chunk<E>::V; ++i)
      if (i < n) c.e[i] = p[i];
  }
  return c;
}
template <class E>
__device__ __forceinline__ void store_chunk(E* p, int n, const Chunk<E>& c) {
  if (n >= Chunk<E>::V) {
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

// 16-bit inputs in mode 1: 127 x has at most 18 significant bits, so the residual 127 x - q m of
// the candidate q is exact in fp32 and decides the rounding.  fp32 inputs: the quotient's error
// is below 3 * 2^-24 * 127 < 2^-15; candidates that near a tie are decided in 64 bits, where
// 127 x is exact and a quotient that is no tie differs from one by 2^-33 at least.
template <class E>
__device__ __forceinline__ int quant_code(float x, const RowQuant& r) {
  if (r.mode == 0) return 0;
  if (r.mode == 2) return (int)rint(127.0 * (double)x / (double)r.m);
  const float t = 127.0f * x;
  const float y = t * r.inv;
  float q = rintf(y);
  if constexpr (sizeof(E) == 2) {
    const float d = 2.0f * fmaf(-q, r.m, t);
    const bool odd = (int)q & 1;
    if (d > r.m || (d == r.m && odd)) q += 1.0f;
    if (d < -r.m || (d == -r.m && odd)) q -= 1.0f;
    return (int)q;
  } else {
    if (fabsf(fabsf(y - q) - 0.5f) < 0x1p-14f)
      return (int)rint(127.0 * (double)x / (double)r.m);
    return (int)q;
  }
}

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
  return (uint32_t)(a & 255) | (uint32_t)(b & 255) << 8 | (uint32_t)(c & 255) << 16 |
         (uint32_t)(d & 255) << 24;
}

// Four codes of elements e[0..3].
template <class E>
__device__ __forceinline__ uint32_t quant4(const E* e, const RowQuant& r) {
  return pack4(quant_code<E>(to_f32(e[0]), r), quant_code<E>(to_f32(e[1]), r),
               quant_code<E>(to_f32(e[2]), r), quant_code<E>(to_f32(e[3]), r));
}

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)v, s);
    v = v > o ? v : o;
  }
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) v += __shfl_xor(v, s);
  return v;
}

template <class E>
__device__ __forceinline__ uint32_t chunk_max_bits(const Chunk<E>& c, uint32_t m) {
#pragma unroll
  for (int i = 0; i < Chunk<E>::V; ++i) {
    const uint32_t b = abs_bits(to_f32(c.e[i]));
    m = m > b ? m : b;
  }
  return m;
}

// The codes of one chunk, the first n of which belong to the row.
template <class E>
__device__ __forceinline__ void store_codes(int8_t* p, int n, const Chunk<E>& c,
                                            const RowQuant& r) {
  constexpr int V = Chunk<E>::V;
  uint32_t w[V / 4];
#pragma unroll
  for (int i = 0; i < V / 4; ++i) w[i] = quant4(c.e + 4 * i, r);
  if (n >= V) {
    if constexpr (V == 8)
      *(u64_any*)p = (uint64_t)w[1] << 32 | w[0];
    else
      __builtin_memcpy(p, w, 4);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) p[i] = (int8_t)(w[i / 4] >> (8 * (i % 4)));
  }
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
