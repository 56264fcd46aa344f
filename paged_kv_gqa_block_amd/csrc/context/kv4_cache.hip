// Writing a run of new tokens into the paged cache, 16 bits or quantised to 4
// as they are written, and reading the 4-bit cache back (gfx950).
//
// A block's scale is 2^e, e = floor(log2 max|x|) - 2 (+ 1 where max|x| > 7 *
// 2^e, which would be off by more than half of the largest step); its elements
// are e2m1 roundings of x / 2^e, ties to even, saturating.  Bound: bytes moved;
// there is no reuse and no arithmetic to speak of.  Measured: 98000 tokens of 8
// KV heads, d = 128, f16: 117 us to quantise 401 MB into 107 MB (4.3 TB/s),
// 107 us to read them back (4.7 TB/s; a plain copy of this size reaches 4.9), 155
// to write them in 16 bits (5.2 TB/s); one token of 64 rows: 3.4, 3.1 and 3.1 us, a
// launch and its loads.
//
// One workgroup per (page of a row that the run touches, KV head): 16 tokens
// by d channels.  Thread (token, chunk) converts eight channels of K and of V;
// four neighbouring threads share a block.
#include "context_internal.h"
#include "kv4_common.h"
#include "runs.h"

namespace pkv {
namespace {

constexpr int kInfExp16[2] = {0x7c00, 0x7f80};  // exponent field of f16, bf16

// Maximum over the four threads of a block (one quad).
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
  x = max(x, uint32_t(__builtin_amdgcn_mov_dpp(int(x), kDppQuadXor1, 0xf, 0xf, true)));
  return max(x, uint32_t(__builtin_amdgcn_mov_dpp(int(x), kDppQuadXor2, 0xf, 0xf, true)));
}

// Eight channels of a block to codes (one dword) and the block's scale byte.
// Called by the whole quad.
template <bool BF16>
__device__ __forceinline__ uint32_t quantise8(const uint4& x, uint32_t* scale_byte) {
  // Magnitudes of a 16-bit float compare as integers.
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
  top = quad_max(top);
  // Bounds that keep every value exact in the type.
  constexpr int kMinExp = BF16 ? -120 : -23, kMaxExp = BF16 ? 125 : 13;
  const float a = BF16 ? Elem<true>::lo(top) : Elem<false>::lo(top);
  const uint32_t u = __float_as_uint(a);  // a > 0 is a normal fp32 number or a bf16 subnormal
  int e = static_cast<int>(u >> 23) - 127 - 2 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = min(max(e, kMinExp), kMaxExp);
  const bool fine = top < uint32_t(kInfExp16[BF16]);
  *scale_byte = fine ? uint32_t(e + 127) : 255u;
  const float s = __uint_as_float(uint32_t(e + 127) << 23);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, Elem<BF16>::lo(w[0]), Elem<BF16>::hi(w[0]), s, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, Elem<BF16>::lo(w[1]), Elem<BF16>::hi(w[1]), s, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, Elem<BF16>::lo(w[2]), Elem<BF16>::hi(w[2]), s, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, Elem<BF16>::lo(w[3]), Elem<BF16>::hi(w[3]), s, 3);
  return fine ? c : 0u;
}

// Threads of a workgroup: d / 8 chunks of 16 tokens.
template <int D, bool BF16, bool KV4>
__global__ __launch_bounds__(2 * D) void store_kernel(StoreArgs a) {
  constexpr int CH = D / 8;
  const int g = blockIdx.x % a.num_kv_heads;
  const Segment s = find_segment(a, blockIdx.x / a.num_kv_heads);
  if (s.begin >= s.end) return;
  const int id = a.block_table[int64_t(s.run.row) * a.max_pages + s.entry];
  if (static_cast<uint32_t>(id) >= static_cast<uint32_t>(a.num_pool_pages)) return;
  const int t = threadIdx.x / CH, j = threadIdx.x % CH;
  const int p = s.entry * 16 + t;
  if (p < s.begin || p >= s.end) return;  // whole quads share a token
  const int64_t tok = s.run.first + (p - (s.run.len - s.run.count));
  const uint4 k = load16(static_cast<const uint16_t*>(a.k_new) + tok * a.k_stride + g * D + 8 * j);
  const uint4 v = load16(static_cast<const uint16_t*>(a.v_new) + tok * a.v_stride + g * D + 8 * j);
  const int64_t page = int64_t(id) * a.num_kv_heads + g;
  if constexpr (KV4) {
    uint8_t* out = static_cast<uint8_t*>(a.k_pool) + page * Kv4<D>::kBytes;
    uint32_t sk, sv;
    const uint32_t ck = quantise8<BF16>(k, &sk);
    const uint32_t cv = quantise8<BF16>(v, &sv);
    *reinterpret_cast<uint32_t*>(out + Kv4<D>::k_at(t, j)) = ck;
    if constexpr (D == 128) {
      *reinterpret_cast<uint32_t*>(out + Kv4<D>::v_at(t, j)) = cv;
    } else {
      *reinterpret_cast<uint16_t*>(out + Kv4<D>::v_at(t, 2 * j)) = uint16_t(cv);
      *reinterpret_cast<uint16_t*>(out + Kv4<D>::v_at(t, 2 * j + 1)) = uint16_t(cv >> 16);
    }
    if ((j & 3) == 0) {
      out[Kv4<D>::ks_at(t, j >> 2)] = uint8_t(sk);
      out[Kv4<D>::vs_at(t, j >> 2)] = uint8_t(sv);
    }
  } else {
    const int64_t at = (page * 16 + t) * D + 8 * j;
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.k_pool) + at) = k;
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.v_pool) + at) = v;
  }
}

template <int D, bool BF16>
__global__ __launch_bounds__(2 * D) void load_kernel(LoadArgs a) {
  constexpr int CH = D / 8;
  const int g = blockIdx.x % a.num_kv_heads;
  const Segment s = find_segment(a, blockIdx.x / a.num_kv_heads);
  if (s.begin >= s.end) return;
  const int id = a.block_table[int64_t(s.run.row) * a.max_pages + s.entry];
  if (static_cast<uint32_t>(id) >= static_cast<uint32_t>(a.num_pool_pages)) return;
  const int t = threadIdx.x / CH, j = threadIdx.x % CH;
  const int p = s.entry * 16 + t;
  if (p < s.begin || p >= s.end) return;
  const int64_t tok = s.run.first + (p - (s.run.len - s.run.count));
  const uint8_t* in = static_cast<const uint8_t*>(a.pool) +
                      (int64_t(id) * a.num_kv_heads + g) * Kv4<D>::kBytes;
  const uint32_t ck = *reinterpret_cast<const uint32_t*>(in + Kv4<D>::k_at(t, j));
  uint32_t cv;
  if constexpr (D == 128)
    cv = *reinterpret_cast<const uint32_t*>(in + Kv4<D>::v_at(t, j));
  else
    cv = *reinterpret_cast<const uint16_t*>(in + Kv4<D>::v_at(t, 2 * j)) |
         (uint32_t(*reinterpret_cast<const uint16_t*>(in + Kv4<D>::v_at(t, 2 * j + 1))) << 16);
  const uint32_t sk = in[Kv4<D>::ks_at(t, j >> 2)], sv = in[Kv4<D>::vs_at(t, j >> 2)];
  const int64_t at = (tok * a.num_kv_heads + g) * D + 8 * j;
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.k_out) + at) =
      kv4_eight<BF16>(ck, kv4_scale(sk));
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.v_out) + at) =
      kv4_eight<BF16>(cv, kv4_scale(sv));
}

template <int D>
void launch_store_d(bool bf, bool kv4, const StoreArgs& a, uint32_t grid, hipStream_t s) {
  if (!kv4)  // a copy: the type does not matter
    hipLaunchKernelGGL((store_kernel<D, false, false>), dim3(grid), dim3(2 * D), 0, s, a);
  else if (bf)
    hipLaunchKernelGGL((store_kernel<D, true, true>), dim3(grid), dim3(2 * D), 0, s, a);
  else
    hipLaunchKernelGGL((store_kernel<D, false, true>), dim3(grid), dim3(2 * D), 0, s, a);
}

}  // namespace

pkv_status launch_store(const pkv_problem& p, bool kv4, const StoreArgs& a, hipStream_t s) {
  const uint32_t grid = static_cast<uint32_t>(run_groups(a));
  const bool bf = p.dtype == PKV_BF16;
  if (p.head_dim == 128) launch_store_d<128>(bf, kv4, a, grid, s);
  else launch_store_d<64>(bf, kv4, a, grid, s);
  return hipGetLastError() == hipSuccess ? PKV_OK : PKV_EHIP;
}

pkv_status launch_load(const pkv_problem& p, const LoadArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(run_groups(a)));
  const bool bf = p.dtype == PKV_BF16;
  if (p.head_dim == 128) {
    if (bf) hipLaunchKernelGGL((load_kernel<128, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((load_kernel<128, false>), grid, dim3(256), 0, s, a);
  } else {
    if (bf) hipLaunchKernelGGL((load_kernel<64, true>), grid, dim3(128), 0, s, a);
    else hipLaunchKernelGGL((load_kernel<64, false>), grid, dim3(128), 0, s, a);
  }
  return hipGetLastError() == hipSuccess ? PKV_OK : PKV_EHIP;
}

}  // namespace pkv
