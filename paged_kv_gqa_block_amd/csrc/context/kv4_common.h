// The 4-bit cache on the device: where a (token, channel) sits in a page, and
// the conversions.
//
// Elements are e2m1 codes (sign, 0 .5 1 1.5 2 3 4 6) in blocks of 32
// consecutive channels of one token and KV head; a block's scale is 2^(b -
// 127) with b its scale byte, 255 marking a block that held an infinity or a
// NaN (every value of it reads as NaN).  gfx950 converts two codes and their
// power-of-two scale to 16 bits in one instruction, without rounding.
//
// One page of one KV head is 17 d consecutive bytes, ordered so that a wave of
// the attention kernel reads it in four contiguous loads, already in the
// matrix core's operand order (lane l = 16 kg + c):
//   [0, 8d)      K codes: lane l holds token c, channels 32 b + 8 kg .. + 7
//                of every block b, 4 bytes each
//   [8d, 16d)    V codes: lane l holds tokens 4 kg .. 4 kg + 3, channels
//                (d/16) c .. (d/16) (c + 1) - 1, d/32 bytes a token
//   [16d, 16.5d) K scales: [token][block]
//   [16.5d, 17d) V scales: [kg][block][token of the four]
// Every byte belongs to one token, so tokens of a page may be written at
// different times, and by different workgroups, without reading it.
#pragma once

#include "device_common.h"

namespace pkv {

template <int D>
struct Kv4 {
  static constexpr int kBytes = 17 * D;
  static constexpr int kV = 8 * D;
  static constexpr int kKs = 16 * D;
  static constexpr int kVs = 16 * D + D / 2;
  // Byte of token t's K channels 8 j .. 8 j + 7 (4 bytes).
  static __device__ __forceinline__ int k_at(int t, int j) {
    return ((j & 3) * 16 + t) * (D / 8) + (j >> 2) * 4;
  }
  // Byte of token t's V channels of lane column c (D/32 bytes).
  static __device__ __forceinline__ int v_at(int t, int c) {
    return kV + ((t >> 2) * 16 + c) * (D / 8) + (t & 3) * (D / 32);
  }
  static __device__ __forceinline__ int ks_at(int t, int b) { return kKs + t * (D / 32) + b; }
  static __device__ __forceinline__ int vs_at(int t, int b) {
    return kVs + (t >> 2) * (D / 8) + b * 4 + (t & 3);
  }
};

// 2^(byte - 127); byte 255 gives an infinity, which the conversions below turn
// into NaN for every code.
__device__ __forceinline__ float kv4_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// Two values of byte SEL of w (low nibble in the low half), exact in 16 bits.
template <bool BF16, int SEL>
__device__ __forceinline__ uint32_t kv4_pair(uint32_t w, float scale) {
  if constexpr (BF16)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, SEL));
  else
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, SEL));
}

// The eight values of a dword.
template <bool BF16>
__device__ __forceinline__ uint4 kv4_eight(uint32_t w, float scale) {
  return make_uint4(kv4_pair<BF16, 0>(w, scale), kv4_pair<BF16, 1>(w, scale),
                    kv4_pair<BF16, 2>(w, scale), kv4_pair<BF16, 3>(w, scale));
}

// One page of one KV head as a wave holds it (the lane's pieces above).
template <int D>
struct Kv4Page {
  uint32_t k[D / 32], v[D / 32];
  uint32_t ks, vs;
  template <int POLICY>
  __device__ __forceinline__ void load_k(__amdgpu_buffer_rsrc_t r, int lane) {
    const int c = lane & 15;
    if constexpr (D == 128) {
      const u32x4 x = __builtin_amdgcn_raw_buffer_load_b128(r, lane * 16, 0, POLICY);
      k[0] = x.x, k[1] = x.y, k[2] = x.z, k[3] = x.w;
      ks = __builtin_amdgcn_raw_buffer_load_b32(r, Kv4<D>::kKs + c * 4, 0, POLICY);
    } else {
      const auto x = __builtin_amdgcn_raw_buffer_load_b64(r, lane * 8, 0, POLICY);
      k[0] = x[0], k[1] = x[1];
      ks = __builtin_amdgcn_raw_buffer_load_b16(r, Kv4<D>::kKs + c * 2, 0, POLICY);
    }
  }
  template <int POLICY>
  __device__ __forceinline__ void load_v(__amdgpu_buffer_rsrc_t r, int lane) {
    const int kg = lane >> 4, c = lane & 15;
    if constexpr (D == 128) {
      const u32x4 x = __builtin_amdgcn_raw_buffer_load_b128(r, Kv4<D>::kV + lane * 16, 0, POLICY);
      v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
      const auto x = __builtin_amdgcn_raw_buffer_load_b64(r, Kv4<D>::kV + lane * 8, 0, POLICY);
      v[0] = x[0], v[1] = x[1];
    }
    // The lane's V channels lie in one block.
    vs = __builtin_amdgcn_raw_buffer_load_b32(
        r, Kv4<D>::kVs + kg * (D / 8) + (c / (512 / D)) * 4, 0, POLICY);
  }
};

}  // namespace pkv
