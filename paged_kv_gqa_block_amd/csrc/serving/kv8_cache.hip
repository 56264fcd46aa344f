// Writing a run of new tokens into the 8-bit cache, quantised as they are written,
// and reading it back (gfx950).
//
// A block (16 tokens by d channels of one KV head, K and V apart) has one scale 2^e:
// e = floor(log2 max|x|) - 8 (+ 1 where max|x| > 448 * 2^e), the smallest that holds
// every finite element of the run's tokens in the block; its codes are x / 2^e rounded
// to e4m3, ties to even.  e4m3 is off by at most 2^-4 of an element (half a step of
// three bits of mantissa) as long as that is 2^(e - 6) or more, so always at 2^-13 of the
// block's largest (2^(e - 6) over more than 224 * 2^e).  A scale between two powers of
// two would gain nothing; whole powers keep every value exact in 16 bits, and rescaling
// exact but for what falls below 2^(e - 6) (a block's subnormal codes).  A block that
// holds earlier tokens of its row keeps at least its exponent, and those tokens are
// rounded again where it grows: by 2^(e - 10) at most each time.  The rounding before the
// first of these was of at most 2^(e - 11) (what falls below 2^(e - 6) had steps of
// 2^(e - 10)), or one of a subnormal code too, so that all make less than 2^(e - 9).
//
// Bound: bytes moved; there is no reuse.  Measured: 98000 tokens of 8 KV heads, d = 128,
// f16: 129-137 us to quantise 401 MB into 201 (4.4-4.7 TB/s), 108-113 to read them back
// (5.3-5.6; a large copy reaches 4.9); one token of 64 rows, most of them behind earlier ones of
// their page: 4.4 and 3.5 us, a launch and a chain of four loads (offsets, page number,
// scale and codes, and the store).
//
// One workgroup per (page of a row that the run touches, KV head): 16 tokens
// by d channels.  Thread (token, chunk) holds eight channels of K and of V.
#include "context/context_internal.h"
#include "context/runs.h"
#include "serving/kv8_common.h"
#include "serving/serving_internal.h"

namespace pkv {
namespace {

constexpr uint32_t kInfBits[2] = {0x7c00, 0x7f80};  // infinity of f16, bf16

// The smallest exponent that holds a largest magnitude, given as 16-bit float bits.
template <bool BF16>
__device__ __forceinline__ int exponent_for(uint32_t top) {
  const uint32_t u = __float_as_uint(Elem<BF16>::lo(top));
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, kKv8MinExp<BF16>), kKv8MaxExp<BF16>);
}

// Largest finite magnitude of eight channels, as its bits.
template <bool BF16>
__device__ __forceinline__ uint32_t top_of(const uint4& x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = w[i] & 0x7fffu, b = (w[i] >> 16) & 0x7fffu;
    top = max(top, a < kInfBits[BF16] ? a : 0u);
    top = max(top, b < kInfBits[BF16] ? b : 0u);
  }
  return top;
}

// Two values, already divided by their scale, to codes in the low or high half of `w`;
// what is not finite becomes NaN, what is too large the largest code.
template <bool HIGH>
__device__ __forceinline__ uint32_t codes2(float a, float b, uint32_t w) {
  const float x = __builtin_amdgcn_fmed3f(a, -448.f, 448.f);
  const float y = __builtin_amdgcn_fmed3f(b, -448.f, 448.f);
  uint32_t c = __builtin_amdgcn_cvt_pk_fp8_f32(x, y, static_cast<int>(w), HIGH);
  constexpr int kAt = HIGH ? 16 : 0;
  if (!(__builtin_fabsf(a) < __builtin_inff())) c |= 0x7fu << kAt;
  if (!(__builtin_fabsf(b) < __builtin_inff())) c |= 0x7fu << (kAt + 8);
  return c;
}

// Eight channels to codes at exponent e.
template <bool BF16>
__device__ __forceinline__ uint2 quantise8(const uint4& x, int e) {
  const float s = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e
  uint2 c = make_uint2(0u, 0u);
  c.x = codes2<false>(Elem<BF16>::lo(x.x) * s, Elem<BF16>::hi(x.x) * s, c.x);
  c.x = codes2<true>(Elem<BF16>::lo(x.y) * s, Elem<BF16>::hi(x.y) * s, c.x);
  c.y = codes2<false>(Elem<BF16>::lo(x.z) * s, Elem<BF16>::hi(x.z) * s, c.y);
  c.y = codes2<true>(Elem<BF16>::lo(x.w) * s, Elem<BF16>::hi(x.w) * s, c.y);
  return c;
}

// Four codes rounded again at an exponent `by` larger.
__device__ __forceinline__ uint32_t requantise4(uint32_t c, int by) {
  const float s = __uint_as_float(static_cast<uint32_t>(127 - min(by, 126)) << 23);
  const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c), false);
  const auto b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c), true);
  return codes2<true>(b[0] * s, b[1] * s, codes2<false>(a[0] * s, a[1] * s, 0u));
}

// A thread's eight codes of V: one piece of a lane, or two.
template <int D>
__device__ __forceinline__ uint2 get_v(const uint8_t* page, int t, int j) {
  if constexpr (D == 128) return *reinterpret_cast<const uint2*>(page + Kv8<D>::v_at(t, j));
  return make_uint2(*reinterpret_cast<const uint32_t*>(page + Kv8<D>::v_at(t, 2 * j)),
                    *reinterpret_cast<const uint32_t*>(page + Kv8<D>::v_at(t, 2 * j + 1)));
}
template <int D>
__device__ __forceinline__ void put_v(uint8_t* page, int t, int j, uint2 c) {
  if constexpr (D == 128) {
    *reinterpret_cast<uint2*>(page + Kv8<D>::v_at(t, j)) = c;
  } else {
    *reinterpret_cast<uint32_t*>(page + Kv8<D>::v_at(t, 2 * j)) = c.x;
    *reinterpret_cast<uint32_t*>(page + Kv8<D>::v_at(t, 2 * j + 1)) = c.y;
  }
}

template <int D, bool BF16>
__global__ __launch_bounds__(2 * D) void store8_kernel(Store8Args a) {
  constexpr int CH = D / 8, NW = 2 * D / 64;
  __shared__ int s_top[2][NW];
  const int g = blockIdx.x % a.num_kv_heads;
  const Segment s = find_segment(a, blockIdx.x / a.num_kv_heads);
  if (s.begin >= s.end) return;
  const int id = a.block_table[int64_t(s.run.row) * a.max_pages + s.entry];
  if (static_cast<uint32_t>(id) >= static_cast<uint32_t>(a.num_pool_pages)) return;
  const int t = threadIdx.x / CH, j = threadIdx.x % CH;
  const int p = s.entry * 16 + t;
  const bool fresh = p >= s.begin && p < s.end, old = p < s.begin;
  const int64_t at = int64_t(id) * a.num_kv_heads + g;
  uint8_t* page = static_cast<uint8_t*>(a.k_pool) + at * Kv8<D>::kBytes;
  uint16_t* scale = reinterpret_cast<uint16_t*>(a.scales) + at;
  const bool grows = (s.begin & 15) != 0;  // the block holds earlier tokens
  uint4 k = zero4(), v = zero4();
  uint2 ck = make_uint2(0u, 0u), cv = ck;
  uint32_t was = 0;
  if (fresh) {
    const int64_t tok = s.run.first + (p - (s.run.len - s.run.count));
    k = load16(static_cast<const uint16_t*>(a.k_new) + tok * a.k_stride + g * D + 8 * j);
    v = load16(static_cast<const uint16_t*>(a.v_new) + tok * a.v_stride + g * D + 8 * j);
  }
  if (grows) was = *scale;
  if (old) {
    ck = *reinterpret_cast<const uint2*>(page + Kv8<D>::k_at(t, j));
    cv = get_v<D>(page, t, j);
  }
  const int top_k = wave_max(static_cast<int>(top_of<BF16>(k)));
  const int top_v = wave_max(static_cast<int>(top_of<BF16>(v)));
  if ((threadIdx.x & 63) == 0) {
    s_top[0][threadIdx.x >> 6] = top_k;
    s_top[1][threadIdx.x >> 6] = top_v;
  }
  __syncthreads();
  int tops[2] = {0, 0}, e[2], by[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
#pragma unroll
    for (int w = 0; w < NW; ++w) tops[x] = max(tops[x], s_top[x][w]);
    e[x] = exponent_for<BF16>(static_cast<uint32_t>(tops[x]));
    const int e_old = min(static_cast<int>((was >> (8 * x)) & 0xff) - 127, kKv8MaxExp<BF16>);
    by[x] = 0;
    if (grows) {
      by[x] = max(e[x] - e_old, 0);
      e[x] = max(e[x], e_old);
    }
  }
  if (fresh) {
    *reinterpret_cast<uint2*>(page + Kv8<D>::k_at(t, j)) = quantise8<BF16>(k, e[0]);
    put_v<D>(page, t, j, quantise8<BF16>(v, e[1]));
  } else if (old) {
    if (by[0] > 0)
      *reinterpret_cast<uint2*>(page + Kv8<D>::k_at(t, j)) =
          make_uint2(requantise4(ck.x, by[0]), requantise4(ck.y, by[0]));
    if (by[1] > 0) put_v<D>(page, t, j, make_uint2(requantise4(cv.x, by[1]),
                                                   requantise4(cv.y, by[1])));
  }
  if (threadIdx.x == 0)
    *scale = static_cast<uint16_t>((e[0] + 127) | ((e[1] + 127) << 8));
}

template <int D, bool BF16>
__global__ __launch_bounds__(2 * D) void load8_kernel(Load8Args a) {
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
  const int64_t at = int64_t(id) * a.num_kv_heads + g;
  const uint8_t* page = static_cast<const uint8_t*>(a.pool) + at * Kv8<D>::kBytes;
  const uint32_t sc = reinterpret_cast<const uint16_t*>(a.scales)[at];
  const uint2 ck = *reinterpret_cast<const uint2*>(page + Kv8<D>::k_at(t, j));
  const uint2 cv = get_v<D>(page, t, j);
  const int64_t to = (tok * a.num_kv_heads + g) * D + 8 * j;
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.k_out) + to) =
      kv8_eight<BF16>(ck.x, ck.y, kv8_scale(sc & 0xff));
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.v_out) + to) =
      kv8_eight<BF16>(cv.x, cv.y, kv8_scale(sc >> 8));
}

}  // namespace

pkv_status launch_store8(const pkv_problem& p, const Store8Args& a, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(run_groups(a)));
  const bool bf = p.dtype == PKV_BF16;
  if (p.head_dim == 128) {
    if (bf) hipLaunchKernelGGL((store8_kernel<128, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((store8_kernel<128, false>), grid, dim3(256), 0, s, a);
  } else {
    if (bf) hipLaunchKernelGGL((store8_kernel<64, true>), grid, dim3(128), 0, s, a);
    else hipLaunchKernelGGL((store8_kernel<64, false>), grid, dim3(128), 0, s, a);
  }
  return hipGetLastError() == hipSuccess ? PKV_OK : PKV_EHIP;
}

pkv_status launch_load8(const pkv_problem& p, const Load8Args& a, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(run_groups(a)));
  const bool bf = p.dtype == PKV_BF16;
  if (p.head_dim == 128) {
    if (bf) hipLaunchKernelGGL((load8_kernel<128, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((load8_kernel<128, false>), grid, dim3(256), 0, s, a);
  } else {
    if (bf) hipLaunchKernelGGL((load8_kernel<64, true>), grid, dim3(128), 0, s, a);
    else hipLaunchKernelGGL((load8_kernel<64, false>), grid, dim3(128), 0, s, a);
  }
  return hipGetLastError() == hipSuccess ? PKV_OK : PKV_EHIP;
}

}  // namespace pkv
