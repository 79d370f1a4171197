// Building blocks of the 16-bit matrix-core kernels: the two element types,
// their MFMA instructions, rounding and cross-lane moves.
//
// Operand layouts used throughout (lane l of 64):
//   32x32x16: A holds row l % 32, B column l % 32, both k = 8 (l / 32) + 0..7;
//             D register i holds row 8 (i / 4) + 4 (l / 32) + i % 4, column l % 32.
//   16x16x32: A holds row l % 16, B column l % 16, both k = 8 (l / 16) + 0..7;
//             D register i holds row 4 (l / 16) + i, column l % 16.
// The k order inside an instruction is free as long as A and B agree, which the
// kernels use to feed one product's D straight into the next one's B.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace pit {

constexpr int WAVE = 64;

typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef short s4 __attribute__((ext_vector_type(4)));

// LOW, LAG, HIGH: powers of two of the weights in a softmax, see pi_attn.hpp.
struct H16 {                       // IEEE binary16
  static constexpr float LOW = 11.f, LAG = 4.f, HIGH = LOW + LAG;
  static constexpr uint16_t INF = 0x7c00;
  typedef _Float16 v8 __attribute__((ext_vector_type(8)));
  typedef _Float16 v2 __attribute__((ext_vector_type(2)));
  static __device__ __forceinline__ f16v mma32(u4 a, u4 b, f16v c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f4 mma16(u4 a, u4 b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {   // to nearest even
    v2 r = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, r);
  }
  static __device__ __forceinline__ float low(uint32_t w) { return (float)__builtin_bit_cast(v2, w)[0]; }
  static __device__ __forceinline__ float high(uint32_t w) { return (float)__builtin_bit_cast(v2, w)[1]; }
};

struct B16 {                       // bfloat16
  static constexpr float LOW = 0.f, LAG = 8.f, HIGH = 0.f;
  static constexpr uint16_t INF = 0x7f80;
  typedef __bf16 v8 __attribute__((ext_vector_type(8)));
  typedef __bf16 v2 __attribute__((ext_vector_type(2)));
  static __device__ __forceinline__ f16v mma32(u4 a, u4 b, f16v c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f4 mma16(u4 a, u4 b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    v2 r = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, r);
  }
  static __device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
  static __device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
};

// Combine a value with those of the lanes that hold the same column of a D
// operand: lanes l and l ^ 32 (32x32), or the four lanes l % 16 + 16 k (16x16).
__device__ __forceinline__ float max32(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum32(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float max16(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return max32(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float sum16(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return sum32(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// Inclusive prefix sum over the 64 lanes by DPP: row_shr 1, 2, 4, 8 inside each
// row of 16 lanes, then row_bcast 15 and 31 carry the rows' totals.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_add(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false);
}
__device__ __forceinline__ int scan64(int v) {
  v = dpp_add<0x111, 0xf>(v);
  v = dpp_add<0x112, 0xf>(v);
  v = dpp_add<0x114, 0xf>(v);
  v = dpp_add<0x118, 0xf>(v);
  v = dpp_add<0x142, 0xa>(v);
  return dpp_add<0x143, 0xc>(v);
}

// Two 16-bit values of two words: the low halves, and the high halves.
__device__ __forceinline__ uint32_t lows(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }
__device__ __forceinline__ uint32_t highs(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }

// A value that all lanes ask for, by a scalar load, which waits on a counter of its own: for memory that nothing writes while
// the kernel runs.
__device__ __forceinline__ int fixed(const int32_t* p, int64_t at) {
  typedef const __attribute__((address_space(4))) int32_t* memory;
  return reinterpret_cast<memory>(reinterpret_cast<uintptr_t>(p))[at];
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

}  // namespace pit
