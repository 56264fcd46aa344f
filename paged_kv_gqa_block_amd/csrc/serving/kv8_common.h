// The 8-bit cache on the device: where a (token, channel) sits in a page, and
// the conversions.
//
// A block is one page of one KV head, K and V apart: 16 tokens by d channels of
// e4m3 codes (no infinities; 127 and 255 are NaN) and one scale 2^(b - 127), b
// its scale byte.  gfx950 converts two codes and a power-of-two scale to 16 bits
// in one instruction, without rounding while b stays in its type's range.
//
// One page of one KV head is 32 d consecutive bytes, ordered so that a wave of
// the attention kernels reads it in contiguous 1 KiB loads, already in the matrix
// core's operand order (lane l = 16 kg + c):
//   [0, 16d)     K codes: in 1 KiB piece x, lane l's 16 bytes hold token c,
//                channels 32 b + 8 kg .. + 7 of the blocks of channels b = 2 x, 2 x + 1
//   [16d, 32d)   V codes: in piece x, lane l's 16 bytes hold channels
//                (d/16) c .. (d/16) (c + 1) - 1 of the tokens 4 kg + T x ..
//                4 kg + T (x + 1) - 1, T = 256 / d
// Every byte belongs to one token.  The two scale bytes of a page and head (K, V)
// lie apart from it, [pages][Hkv][2]: sixteen times 8 heads' bytes fill a cache
// line, so they come out of the L2, and pages stay whole cache lines.
#pragma once

#include "device_common.h"

namespace pkv {

template <int D>
struct Kv8 {
  static constexpr int kBytes = 32 * D;
  static constexpr int kV = 16 * D;
  static constexpr int kVTokens = 256 / D;  // V tokens in a lane's 16 bytes
  // Byte of token t's K channels 8 j .. 8 j + 7 (8 bytes).
  static __device__ __forceinline__ int k_at(int t, int j) {
    return (j >> 3) * 1024 + ((j & 3) * 16 + t) * 16 + ((j >> 2) & 1) * 8;
  }
  // Byte of token t's V channels of lane column c (D / 16 bytes).
  static __device__ __forceinline__ int v_at(int t, int c) {
    const int i = t & 3;
    return kV + (i / kVTokens) * 1024 + ((t >> 2) * 16 + c) * 16 + (i % kVTokens) * (D / 16);
  }
};

// Exponents that keep every value exact in the type: the smallest subnormal code
// is 2^-9, the largest code 448.
template <bool BF16>
inline constexpr int kKv8MinExp = BF16 ? -117 : -15;
template <bool BF16>
inline constexpr int kKv8MaxExp = BF16 ? 119 : 7;

__device__ __forceinline__ float kv8_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// Two codes of w (the low or the high pair), exact in 16 bits.
template <bool BF16, bool HIGH>
__device__ __forceinline__ uint32_t kv8_pair(uint32_t w, float scale) {
  if constexpr (BF16)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, HIGH));
  else
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, scale, HIGH));
}

// The eight values of two dwords.
template <bool BF16>
__device__ __forceinline__ uint4 kv8_eight(uint32_t a, uint32_t b, float scale) {
  return make_uint4(kv8_pair<BF16, false>(a, scale), kv8_pair<BF16, true>(a, scale),
                    kv8_pair<BF16, false>(b, scale), kv8_pair<BF16, true>(b, scale));
}

// One page of one KV head as a wave holds it: channel block b of the lane's K token
// is k[2 b], k[2 b + 1]; V token 4 kg + i is the i-th D / 64 dwords of v.
template <int D>
struct Kv8Page {
  uint32_t k[D / 16], v[D / 16];
  // (Constant offsets apart from the lane's: as sums they took a register each.)
  template <int POLICY>
  static __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, int lane, int at,
                                              uint32_t (&x)[D / 16]) {
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const u32x4 y = __builtin_amdgcn_raw_buffer_load_b128(r, lane * 16, at + 1024 * i, POLICY);
      x[4 * i] = y.x, x[4 * i + 1] = y.y, x[4 * i + 2] = y.z, x[4 * i + 3] = y.w;
    }
  }
  template <int POLICY>
  __device__ __forceinline__ void load_k(__amdgpu_buffer_rsrc_t r, int lane) {
    load<POLICY>(r, lane, 0, k);
  }
  template <int POLICY>
  __device__ __forceinline__ void load_v(__amdgpu_buffer_rsrc_t r, int lane) {
    load<POLICY>(r, lane, Kv8<D>::kV, v);
  }
};

}  // namespace pkv
