// Matrix-core products and cross-row reductions of the context kernels.
#pragma once

#include "device_common.h"

namespace pkv {

typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// D[4 kg + r][c] += sum_k A[c][k] B[k][c]; lane l = 16 kg + c holds A row c and
// B column c, k = 8 kg .. 8 kg + 7 (k16: k = 4 kg .. 4 kg + 3).
template <bool BF16>
__device__ __forceinline__ f32x4 mfma16(const uint4& a, const uint4& b, f32x4 c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
template <bool BF16>
__device__ __forceinline__ f32x4 mfma16_k16(const uint2& a, const uint2& b, f32x4 c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(bf16x4, a),
                                                     __builtin_bit_cast(bf16x4, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x16f16(__builtin_bit_cast(f16x4, a),
                                                 __builtin_bit_cast(f16x4, b), c, 0, 0, 0);
}
// D[8 (i / 4) + 4 h + i % 4][n] += sum_k A[n][k] B[k][n]; lane l = 32 h + n
// holds A row n and B column n, k = 8 h .. 8 h + 7, and D registers i = 0..15.
template <bool BF16>
__device__ __forceinline__ f32x16 mfma32(const uint4& a, const uint4& b, f32x16 c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Two floats to 16 bits, rounded to nearest even, a in the low half.
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (BF16)
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf162_t));
  else
    return __builtin_bit_cast(uint32_t,
                              half2_t{static_cast<_Float16>(a), static_cast<_Float16>(b)});
}

// x combined with the lane 16 or 32 away (the row-swap instructions hand both
// lanes the same two values, so a symmetric operation gives both the result).
__device__ __forceinline__ float max_x16(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float max_x32(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_x16(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float sum_x32(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Largest of three, one instruction (v_maximum3_f32): fmaxf of matrix-core results
// would first quieten each operand.  A NaN wins.  Left to the compiler, which keeps
// the wait that a vector read of a matrix-core result needs; it knows of none in
// front of inline asm.
__device__ __forceinline__ float max3(float a, float b, float c) {
  return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c);
}

// Where a running maximum starts: finite, so that a score of -inf weighs
// exp2(-inf) = 0 and never meets -inf - -inf.
constexpr float kLowest = -3.402823466e38f;

// The running maximum that weights are relative to is kept `room` (log2) below
// the largest score, and only moves when a score passes it by more than room +
// slack: a weight is at most 2^(room + slack), and the largest at least 2^room.
// An f16 weight below 2^-14 is subnormal, held to 2^-25, so its type needs room,
// with 2^15 at the top; bf16 has the range of fp32 and needs none.
//  * One part a weight (prompts): room 7 keeps the 11 bits of a weight down to
//    2^-21 of the largest, and an error of 2^-32 of it below.
//  * Two parts (decode): room 12 keeps 22 bits down to 2^-15 of the largest, 11
//    down to 2^-26, and an error of 2^-37 of it below.  (With room 0, 1500
//    tokens 17.4 nats under a first one whose V is zero gave an output 6 % off.)
struct Reach {
  float room, slack;
};
template <bool BF16>
inline constexpr Reach kPromptReach = BF16 ? Reach{0.f, 8.f} : Reach{7.f, 8.f};
template <bool BF16>
inline constexpr Reach kDecodeReach = BF16 ? Reach{0.f, 8.f} : Reach{12.f, 3.f};

// A row's length as the operators take it: 0 outside [0, capacity].
__device__ __forceinline__ int clean_len(int n, int max_pages) {
  return (n < 0 || n > max_pages * 16) ? 0 : n;
}

}  // namespace pkv
