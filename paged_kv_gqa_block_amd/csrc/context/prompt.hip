// Prompt attention (gfx950): many query tokens per row over the paged cache,
// causal, with a sliding window and sinks; 16-bit pages or the 4-bit pool.
//
//   out_i = sum_t exp(x_it - M_i) v_t / L_i,  x_it = scale <q_i, k_t>
// over t <= p_i with t > p_i - window or t < sinks: one pass over the visible
// keys with the running maximum and sum of every query.
//
// Bound: the matrix core, 4 d flops per visible (query, key).  A workgroup owns
// 128 packed query rows (token-major, the G heads of a KV head side by side, so
// that they share its keys) and walks the pages that any of them sees, 64 keys
// at a time through two LDS buffers; each of its four waves owns 32 rows.
//  * S^T = K Q^T on v_mfma_f32_32x32x16: a lane holds one query's scores for 16
//    of 32 keys, so maximum and sum need one exchange with the lane 32 away.
//  * O^T += V^T P^T: the lane's own probabilities are the B operand as they
//    stand (the order of the keys inside a product is free), and V^T comes out
//    of row-major LDS by the transposing read ds_read_b64_tr_b16.
//  * O is rescaled only when a score passes the running maximum by more than
//    2^8: below that, exp2 stays exact enough in fp32 and fits in f16.
// The probabilities enter the second product rounded to the problem's type (a
// relative 2^-9 (bf16) or 2^-12 (f16) each, of the size of the output's own
// rounding); maxima, sums and outputs are fp32 until the last rounding.
#include "context_internal.h"
#include "kv4_common.h"
#include "mfma.h"
#include "runs.h"

namespace pkv {
namespace {

constexpr int kKeys = 64;             // keys per step: four pages
constexpr int kNoPage = 0x7ffffff0;   // token base of an absent page: behind every query

// Physical 16-byte chunk of chunk ch of key t.  K is read 32 keys at a time at
// one chunk, V four keys at a time over 64 bytes: in both, lanes that are
// served together fall on distinct banks.
template <int D>
__device__ __forceinline__ int k_chunk(int t, int ch) {
  return D == 128 ? ch ^ (t & 15) : ch ^ ((t >> 1) & 7);
}
template <int D>
__device__ __forceinline__ int v_chunk(int t, int ch) {
  return D == 128 ? ch ^ ((t & 3) << 2) : ch ^ (((t >> 1) & 1) << 2);
}

template <int D>
struct PromptShared {
  uint4 k[2][kKeys][D / 8];
  uint4 v[2][kKeys][D / 8];
};

// Token bases of the four pages of a step (kNoPage where there is none).
struct Pages {
  int base[4];
};

// One step's keys and values on their way to LDS.  Load x covers pages x (d =
// 128) or 2 x and 2 x + 1 (d = 64, one for each half of the workgroup).
template <int D, bool BF16, bool KV4>
struct Stage {
  static constexpr int NL = D / 32;
  uint4 k[KV4 ? 1 : NL], v[KV4 ? 1 : NL];
  uint32_t ck[KV4 ? NL : 1], cv[KV4 ? NL : 1], sk[KV4 ? NL : 1], sv[KV4 ? NL : 1];

  static __device__ __forceinline__ int page(int x, int wave) {
    return D == 128 ? x : 2 * x + (wave >> 1);
  }
  // Thread's index among those of its page.
  static __device__ __forceinline__ int slot(int tid) { return D == 128 ? tid : tid & 127; }

  // `id`: this load's pool page or -1; `len - base` tokens of it exist.
  __device__ __forceinline__ void load(int x, const PromptArgs& a, int g, int id, int left,
                                       int tid) {
    const int u = slot(tid);
    const int64_t at = int64_t(max(id, 0)) * a.num_kv_heads + g;
    if constexpr (KV4) {
      const uint8_t* p = static_cast<const uint8_t*>(a.k_pool) + at * Kv4<D>::kBytes;
      const auto r = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<uint8_t*>(p), (short)0, id >= 0 ? Kv4<D>::kBytes : 0, kBufferFlags);
      const int l = u / (D / 32), w = u % (D / 32);  // lane piece and dword of it
      const int kg = l >> 4, c = l & 15;
      ck[x] = __builtin_amdgcn_raw_buffer_load_b32(r, u * 4, 0, 0);
      cv[x] = __builtin_amdgcn_raw_buffer_load_b32(r, Kv4<D>::kV + u * 4, 0, 0);
      sk[x] = __builtin_amdgcn_raw_buffer_load_b8(r, Kv4<D>::ks_at(c, w), 0, 0);
      if constexpr (D == 128)
        sv[x] = __builtin_amdgcn_raw_buffer_load_b8(r, Kv4<D>::vs_at(4 * kg + w, c >> 2), 0, 0);
      else
        sv[x] = __builtin_amdgcn_raw_buffer_load_b16(r, Kv4<D>::vs_at(4 * kg + 2 * w, c >> 3), 0,
                                                     0);
    } else {
      const int bytes = id >= 0 ? min(16, left) * D * 2 : 0;
      const uint16_t* kp = static_cast<const uint16_t*>(a.k_pool) + at * 16 * D;
      const uint16_t* vp = static_cast<const uint16_t*>(a.v_pool) + at * 16 * D;
      const auto kr = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(kp), (short)0, bytes,
                                                        kBufferFlags);
      const auto vr = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(vp), (short)0, bytes,
                                                        kBufferFlags);
      const u32x4 kk = __builtin_amdgcn_raw_buffer_load_b128(kr, u * 16, 0, 0);
      const u32x4 vv = __builtin_amdgcn_raw_buffer_load_b128(vr, u * 16, 0, 0);
      k[x] = make_uint4(kk.x, kk.y, kk.z, kk.w);
      v[x] = make_uint4(vv.x, vv.y, vv.z, vv.w);
    }
  }

  // To LDS.  seen(t): whether some query of the tile sees token t of the page;
  // the others' V is cleared, because 0 * NaN is not 0.
  template <typename Seen>
  __device__ __forceinline__ void put(int x, PromptShared<D>& sh, int buf, int tid, int wave,
                                      bool all_seen, Seen seen) {
    const int u = slot(tid), key0 = 16 * page(x, wave);
    if constexpr (KV4) {
      const int l = u / (D / 32), w = u % (D / 32);
      const int kg = l >> 4, c = l & 15;
      sh.k[buf][key0 + c][k_chunk<D>(key0 + c, 4 * w + kg)] =
          kv4_eight<BF16>(ck[x], kv4_scale(sk[x]));
      if constexpr (D == 128) {
        const int t = 4 * kg + w;
        uint4 e = kv4_eight<BF16>(cv[x], kv4_scale(sv[x]));
        if (!all_seen && !seen(t)) e = zero4();
        sh.v[buf][key0 + t][v_chunk<D>(key0 + t, c)] = e;
      } else {
        const int t = 4 * kg + 2 * w;
        const float s0 = kv4_scale(sv[x] & 0xff), s1 = kv4_scale((sv[x] >> 8) & 0xff);
        uint2 e0 = make_uint2(kv4_pair<BF16, 0>(cv[x], s0), kv4_pair<BF16, 1>(cv[x], s0));
        uint2 e1 = make_uint2(kv4_pair<BF16, 2>(cv[x], s1), kv4_pair<BF16, 3>(cv[x], s1));
        if (!all_seen && !seen(t)) e0 = make_uint2(0u, 0u);
        if (!all_seen && !seen(t + 1)) e1 = make_uint2(0u, 0u);
        reinterpret_cast<uint2*>(&sh.v[buf][key0 + t][v_chunk<D>(key0 + t, c >> 1)])[c & 1] = e0;
        reinterpret_cast<uint2*>(&sh.v[buf][key0 + t + 1][v_chunk<D>(key0 + t + 1, c >> 1)])[c & 1] =
            e1;
      }
    } else {
      const int t = u / (D / 8), c = u % (D / 8);
      sh.k[buf][key0 + t][k_chunk<D>(key0 + t, c)] = k[x];
      uint4 e = v[x];
      if (!all_seen && !seen(t)) e = zero4();
      sh.v[buf][key0 + t][v_chunk<D>(key0 + t, c)] = e;
    }
  }
};

typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;

// Four keys by 16 channels per 16 lanes, transposed: lane a of the 16 passes
// the address of key a / 4, channels 4 (a % 4) .., and gets channel a of the
// four keys.
__device__ __forceinline__ uint2 read_transposed(const void* p) {
  return __builtin_bit_cast(
      uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                 (lds_bf16x4*)(__attribute__((address_space(3))) void*)(const_cast<void*>(p))));
}

template <int D, bool BF16, bool KV4>
__global__ __launch_bounds__(256, 2) void prompt_kernel(PromptArgs a, int tiles) {
  constexpr int NQ = D / 16;  // products over the channels
  constexpr int NC = D / 32;  // channel blocks of the output
  using St = Stage<D, BF16, KV4>;
  __shared__ PromptShared<D> sh;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 31, h = lane >> 5;
  const int g = blockIdx.x % a.num_kv_heads;
  // Late tiles of a causal row see the most keys: they start first.
  const int item = tiles - 1 - static_cast<int>(blockIdx.x / a.num_kv_heads);
  const int G = a.group;

  int row = item, k_tile = 0;
  if (a.tok_offsets) {
    row = find_row(a.tok_offsets, a.batch, a.num_tokens, item, [&](int64_t off, int64_t r) {
      return tile_base(off, r, G);
    });
  }
  const Run run = run_of(a.tok_offsets, a.seq_lens, row, a.num_tokens, a.max_pages);
  if (a.tok_offsets) k_tile = item - static_cast<int>(tile_base(run.first, row, G));
  const int64_t rows64 = int64_t(run.count) * G;
  if (k_tile < 0 || int64_t(k_tile) * kTileRows >= rows64) return;
  const int r0 = k_tile * kTileRows;
  const int rows = static_cast<int>(min(rows64 - r0, int64_t(kTileRows)));  // of this tile
  const int shift = run.len - run.count;  // position of the run's first token
  const int p_first = max(shift + r0 / G, 0);  // negative positions see nothing
  const int p_last = shift + (r0 + rows - 1) / G;

  // This lane's query.
  const int wr = 32 * wave;  // the wave's first row in the tile
  const int my = wr + n;
  const int j = (r0 + min(my, rows - 1)) / G;
  const int head = (r0 + min(my, rows - 1)) - j * G;
  const int p = max(shift + j, -1);
  const int64_t qh = (int64_t(run.first) + j) * a.num_q_heads + g * G + head;
  const bool mine = my < rows;

  if (p_last < 0) {  // no query of the tile is at a position of the row
    if (mine) {
      for (int e = h; e < D / 4; e += 2)
        reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + qh * D)[e] = make_uint2(0u, 0u);
      if (a.lse && h == 0) a.lse[qh] = kNegInf;
    }
    return;
  }
  const SeenPages sp = seen_pages(p_first, p_last, a.window, a.sinks);
  const int steps = (sp.count + 3) >> 2;
  const int32_t* bt = a.block_table + int64_t(row) * a.max_pages;

  // B operand of the scores: channels 16 t + 8 h .. of this lane's query.
  uint4 qf[NQ];
  {
    const uint16_t* qp = static_cast<const uint16_t*>(a.q) + qh * D + 8 * h;
#pragma unroll
    for (int t = 0; t < NQ; ++t) {
      qf[t] = mine ? load16(qp + 16 * t) : zero4();
      qf[t].x ^= a.q_flip, qf[t].y ^= a.q_flip, qf[t].z ^= a.q_flip, qf[t].w ^= a.q_flip;
    }
  }
  // Positions of the wave's first and last query (empty when it has none).
  const bool busy = wr < rows;
  const int pw_first = max(shift + (r0 + min(wr, rows - 1)) / G, -1);
  const int pw_last = max(shift + (r0 + min(wr + 31, rows - 1)) / G, -1);

  // ---- staging ----------------------------------------------------------------
  St st;
  Pages next;  // of the step in `st`
  int ids = -1;
  auto issue = [&](int s) {
    if ((s & 15) == 0) {  // pool pages of 16 steps, one per lane
      const int v = 4 * s + lane;
      const int id = v < sp.count ? bt[v < sp.ahead ? v : v + sp.skip] : -1;
      ids = (static_cast<uint32_t>(id) < static_cast<uint32_t>(a.num_pool_pages)) ? id : -1;
    }
    int id[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int v = 4 * s + x;
      id[x] = __builtin_amdgcn_readlane(ids, v & 63);
      next.base[x] = id[x] >= 0 ? 16 * (v < sp.ahead ? v : v + sp.skip) : kNoPage;
    }
#pragma unroll
    for (int x = 0; x < St::NL; ++x) {
      // Selected without an index into registers.
      const int i0 = D == 128 ? id[x] : (wave >> 1) ? id[2 * x + 1] : id[2 * x];
      const int b0 = D == 128 ? next.base[x] : (wave >> 1) ? next.base[2 * x + 1] : next.base[2 * x];
      st.load(x, a, g, i0, run.len - b0, tid);
    }
  };
  auto put = [&](int buf) {
#pragma unroll
    for (int x = 0; x < St::NL; ++x) {
      const int b0 = D == 128 ? next.base[x] : (wave >> 1) ? next.base[2 * x + 1] : next.base[2 * x];
      const bool all_seen = b0 + 15 <= p_last && (a.window == 0 || b0 > p_first - a.window ||
                                                  b0 + 15 < a.sinks);
      st.put(x, sh, buf, tid, wave, all_seen, [&](int t) {
        return b0 + t <= p_last &&
               (a.window == 0 || b0 + t > p_first - a.window || b0 + t < a.sinks);
      });
    }
  };

  float m_run = kLowest, l_part = 0.f;
  f32x16 acc[NC];
#pragma unroll
  for (int cb = 0; cb < NC; ++cb)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[cb][i] = 0.f;

  auto compute = [&](int buf, const Pages& pg) {
    bool full = true, any = false;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int b0 = pg.base[x];
      full &= b0 + 15 <= pw_first && (a.window == 0 || b0 > pw_last - a.window ||
                                      b0 + 15 < a.sinks);
      any |= b0 <= pw_last && (a.window == 0 || b0 + 15 > pw_first - a.window || b0 < a.sinks);
    }
    if (!any || !busy) return;
    f32x16 s[2];
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
#pragma unroll
      for (int i = 0; i < 16; ++i) s[sub][i] = 0.f;
#pragma unroll
      for (int t = 0; t < NQ; ++t) {
        const int key = 32 * sub + n;
        s[sub] = mfma32<BF16>(sh.k[buf][key][k_chunk<D>(key, 2 * t + h)], qf[t], s[sub]);
      }
    }
    if (!full) {
#pragma unroll
      for (int sub = 0; sub < 2; ++sub)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int t = pg.base[2 * sub + (i >> 3)] + 8 * ((i >> 2) & 1) + 4 * h + (i & 3);
          if (!sees(p, t, a.window, a.sinks)) s[sub][i] = kNegInf;
        }
    }
    float top = fmaxf(s[0][0], s[1][0]);
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, fmaxf(s[0][i], s[1][i]));
    top = max_x32(top) * a.scale_log2;
    if (__builtin_amdgcn_ballot_w64(top > m_run + kSlack) != 0) {
      const float mn = fmaxf(m_run, top);
      const float alpha = fast_exp2(m_run - mn);
      l_part *= alpha;
#pragma unroll
      for (int cb = 0; cb < NC; ++cb)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[cb][i] *= alpha;
      m_run = mn;
    }
    uint32_t pb[2][8];
#pragma unroll
    for (int sub = 0; sub < 2; ++sub)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float e0 = fast_exp2(fmaf(s[sub][2 * i], a.scale_log2, -m_run));
        const float e1 = fast_exp2(fmaf(s[sub][2 * i + 1], a.scale_log2, -m_run));
        l_part += e0 + e1;
        pb[sub][i] = pack2<BF16>(e0, e1);
      }
    // Lane's share of a transposed read: key lane % 16 / 4 of four, 16-byte
    // chunk 2 (lane / 16 % 2) + lane % 4 / 2 of a channel block, half lane % 2.
    const int kq = (lane & 15) >> 2, cq = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      const uint4 bv = make_uint4(pb[ks >> 1][4 * (ks & 1)], pb[ks >> 1][4 * (ks & 1) + 1],
                                  pb[ks >> 1][4 * (ks & 1) + 2], pb[ks >> 1][4 * (ks & 1) + 3]);
#pragma unroll
      for (int cb = 0; cb < NC; ++cb) {
        const int key = 16 * ks + 4 * h + kq;
        const uint2* p0 =
            reinterpret_cast<const uint2*>(&sh.v[buf][key][v_chunk<D>(key, 4 * cb + cq)]) +
            (lane & 1);
        const uint2* p1 =
            reinterpret_cast<const uint2*>(&sh.v[buf][key + 8][v_chunk<D>(key + 8, 4 * cb + cq)]) +
            (lane & 1);
        const uint2 v0 = read_transposed(p0), v1 = read_transposed(p1);
        acc[cb] = mfma32<BF16>(make_uint4(v0.x, v0.y, v1.x, v1.y), bv, acc[cb]);
      }
    }
  };

  issue(0);
  put(0);
  Pages cur = next;
  if (steps > 1) issue(1);
  __syncthreads();
  for (int s = 0; s < steps; ++s) {
    compute(s & 1, cur);
    if (s + 1 < steps) {
      put((s + 1) & 1);
      cur = next;
      if (s + 2 < steps) issue(s + 2);
    }
    __syncthreads();
  }

  // ---- outputs ----------------------------------------------------------------
  const float l = sum_x32(l_part);
  if (!mine) return;
  const bool none = l == 0.f;
  const float inv = none ? 0.f : 1.f / l;
  uint16_t* out = static_cast<uint16_t*>(a.out) + qh * D;
#pragma unroll
  for (int cb = 0; cb < NC; ++cb)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<uint2*>(out + 32 * cb + 8 * i + 4 * h) =
          make_uint2(pack2<BF16>(acc[cb][4 * i] * inv, acc[cb][4 * i + 1] * inv),
                     pack2<BF16>(acc[cb][4 * i + 2] * inv, acc[cb][4 * i + 3] * inv));
  if (a.lse && h == 0) a.lse[qh] = none ? kNegInf : m_run * kLn2 + __logf(l);
}

template <int D, bool BF16>
void launch_fmt(bool kv4, const PromptArgs& a, int tiles, uint32_t grid, hipStream_t s) {
  if (kv4)
    hipLaunchKernelGGL((prompt_kernel<D, BF16, true>), dim3(grid), dim3(256), 0, s, a, tiles);
  else
    hipLaunchKernelGGL((prompt_kernel<D, BF16, false>), dim3(grid), dim3(256), 0, s, a, tiles);
}

}  // namespace

pkv_status launch_prompt(const pkv_problem& p, bool kv4, const PromptArgs& a, hipStream_t s) {
  const int64_t tiles = prompt_tiles(a);
  const bool bf = p.dtype == PKV_BF16;
  const uint32_t n = static_cast<uint32_t>(tiles * a.num_kv_heads);
  if (p.head_dim == 128) {
    if (bf) launch_fmt<128, true>(kv4, a, static_cast<int>(tiles), n, s);
    else launch_fmt<128, false>(kv4, a, static_cast<int>(tiles), n, s);
  } else {
    if (bf) launch_fmt<64, true>(kv4, a, static_cast<int>(tiles), n, s);
    else launch_fmt<64, false>(kv4, a, static_cast<int>(tiles), n, s);
  }
  return hipGetLastError() == hipSuccess ? PKV_OK : PKV_EHIP;
}

}  // namespace pkv
