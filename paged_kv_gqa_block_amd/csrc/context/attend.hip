// Decode attention over the visible part of a paged cache (gfx950): one query
// token per row, 16-bit pages or the 4-bit pool, d = 64 or 128, G <= 16.
//
//   out = sum_t exp(x_t - M) v_t / L,  x_t = scale <q, k_t>,  L = sum_t exp(x_t - M)
// over the visible tokens t >= N - window or t < sinks.  One pass with the
// running maximum and sum; a row's list of visible pages (the sinks' pages,
// then the window's) is cut into splits; each leaves its partial state (m, l,
// o), and the last of them to finish joins the pair's states: one launch.
//
// Bound: the bytes of the visible pages, read once.  A wave takes its pages in
// units (16-bit: one page; 4-bit: two), the next unit's loads in flight while
// one is computed.
//  * Scores: v_mfma_f32_16x16x32, A = 16 tokens x 32 channels of K, B = Q^T (16
//    heads, padded).  16-bit K arrives in coalesced rows and goes through a
//    private, XOR-swizzled LDS tile into operand order; the 4-bit pool is
//    stored in operand order and needs none.
//  * P V: A = P (heads x tokens) from the lane's own scores, B = V (tokens x
//    channels) by byte permutes.  P is split into its 16-bit rounding and the
//    rounding of the rest, so the product keeps 16 bits of a weight in bf16, and
//    22 in f16 as far down as kDecodeReach says.
//  * The running maximum only moves, and O is only rescaled, when a score passes
//    it by a good deal (kDecodeReach).
// Three waves of a SIMD (at most 168 registers): with the compiler's own two,
// 96 rows x 8 heads x 8192 tokens in 4 bits took 190 us instead of 160.
// Joining in the same launch: one row of 32768 tokens in 4 bits, 8 KV heads,
// took 18.1 us with a second launch and 17.0 us so, and the host one call less
// (16 -> 9 us); with 16 states on their way at once 15.8 us.
//
// Measured (G = 8, d = 128, 64 rows, 8 KV heads, bf16): 4 bits, 1.1 million
// tokens (1.21 GB): 212-227 us, 5.3-5.7 TB/s; the same pages read and not used take
// 187 us (6.5 TB/s), the rest is conversion and matrix work that three waves do
// not hide (221 vector instructions for two pages).  Eight rows, half of them
// short (111 MB): 28-29 us.  One row of 32768: 15-16 us.  256 rows of 1024-2048 over
// one KV head 18 us (3.0 TB/s), 1024 rows of 256-512 over eight 109 (4.2).  16 bits, window 1000 and
// 5 sinks (260 MB): 44 us, 5.9 TB/s; window 4096 over eight rows (134 MB): 27 us,
// 5.0 TB/s.  Small calls: 7 us, a chain of dependent loads (length, page number,
// page, state, counter).
#include <atomic>

#include "context_internal.h"
#include "kv4_common.h"
#include "mfma.h"
#include "states.h"
#include "wave.h"

namespace pkv {
namespace {

// A workgroup's share of a row.
struct Share {
  int row;
  int split;  // negative: no share
  int pages;  // of every range but a row's last
  int n;      // the row's length
};

// Share number `item` in the list of every row's ranges, row after row.  A range
// has the longest row's visible pages over the ranges that they are worth
// (decode_ranges), the split cap at most.  Workgroups without a
// range come last in the launch: mixed in, as a grid of rows by splits has them,
// they leave compute units short of real ones (64 rows of 1024 to 32768 tokens:
// 600 resident workgroups of 768).
__device__ __forceinline__ Share find_share(const AttendArgs& a, int item) {
  Share s{item, 0, 0x7fffffff, 0};
  if (a.splits == 1) {
    s.n = clean_len(a.seq_lens[item], a.max_pages);
    return s;
  }
  const int lane = threadIdx.x & 63;
  int n, pages;
  auto load = [&](int r0) {
    const int r = r0 + lane;
    n = r < a.batch ? clean_len(a.seq_lens[r], a.max_pages) : 0;
    pages = n > 0 ? seen_pages(n - 1, n - 1, a.window, a.sinks).count : 0;
  };
  load(0);
  int t_max = pages;
  if (a.batch > 64) {
    for (int r0 = 64; r0 < a.batch; r0 += 64) {
      load(r0);
      t_max = max(t_max, pages);
    }
    load(0);
  }
  t_max = wave_max(t_max);
  const int most = min(a.splits, decode_ranges(t_max, a.fill, a.even));
  s.pages = max(1, (t_max + most - 1) / most);
  s.split = -1;
  auto ranges = [&](int r0) {
    return r0 + lane < a.batch ? max(1, (pages + s.pages - 1) / s.pages) : 0;
  };
  // A few workgroups for every compute unit, and some left over, take as long as
  // one more for each: then longer ranges that come out even, where they cost less
  // (a range is worth 8 pages more than it reads).  Eight rows, half of them short:
  // 552 ranges 34 us, 512 ranges 28 us.  (Counting again
  // takes one scan where a wave holds the rows; more than 64 leave little over.)
  if (a.batch > 1 && a.batch <= 64) {
    const int total = __builtin_amdgcn_readlane(wave_scan(ranges(0)), 63);
    const int rounds = (total * a.num_kv_heads + a.cus - 1) / a.cus;
    if (rounds >= 2 && rounds <= 4) {
      const int even = (rounds - 1) * a.cus / a.num_kv_heads, first = s.pages;
      int t = total;
      for (int i = 0; i < 3 && t > even && even >= a.batch; ++i) {
        s.pages += 1 + static_cast<int>(static_cast<float>(s.pages) *
                                        static_cast<float>(t - even) / static_cast<float>(even));
        s.pages = min(s.pages, t_max);
        t = __builtin_amdgcn_readlane(wave_scan(ranges(0)), 63);
      }
      if (t > even || (rounds - 1) * (s.pages + 8) >= rounds * (first + 8)) s.pages = first;
    }
  }
  for (int r0 = 0, before = 0;;) {
    const int mine = ranges(r0);
    const int upto = wave_scan(mine);
    const int all = __builtin_amdgcn_readlane(upto, 63);
    if (item < before + all) {
      const uint64_t past = __builtin_amdgcn_ballot_w64(before + upto > item);
      const int at = __builtin_amdgcn_readfirstlane(__builtin_ctzll(past));
      s.row = r0 + at;
      s.split = item - before - __builtin_amdgcn_readlane(upto - mine, at);
      s.n = __builtin_amdgcn_readlane(n, at);
      return s;
    }
    before += all;
    r0 += 64;
    if (r0 >= a.batch) return s;
    load(r0);
  }
}

// The loads of one page, as each format lays it out.
template <int D, bool KV4>
struct PageRegs;

template <int D>
struct PageRegs<D, true> : Kv4Page<D> {};

template <int D>
struct PageRegs<D, false> {
  uint32_t k[4][D / 32], v[4][D / 32];  // tokens kg + 4 i, channels (D/16) c ..
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t kr, __amdgpu_buffer_rsrc_t vr,
                                       int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (D == 128) {
        const uint4 x = buffer_load16(kr, lane * 16 + i * 1024);
        const uint4 y = buffer_load16(vr, lane * 16 + i * 1024);
        k[i][0] = x.x, k[i][1] = x.y, k[i][2] = x.z, k[i][3] = x.w;
        v[i][0] = y.x, v[i][1] = y.y, v[i][2] = y.z, v[i][3] = y.w;
      } else {
        const auto x = __builtin_amdgcn_raw_buffer_load_b64(kr, lane * 8 + i * 512, 0,
                                                            kCachePolicyStream);
        const auto y = __builtin_amdgcn_raw_buffer_load_b64(vr, lane * 8 + i * 512, 0,
                                                            kCachePolicyStream);
        k[i][0] = x[0], k[i][1] = x[1];
        v[i][0] = y[0], v[i][1] = y[1];
      }
    }
  }
};

// The waves' states for the final combine; the K tiles share the space, which
// they no longer need then.
template <int D, int GP, int NW>
struct AttendShared {
  float m[NW][GP];
  float l[NW][GP];
  union {
    alignas(16) float o[NW][GP][D];
    uint4 k[NW][16][D / 8];  // per-wave K tile of 16-bit pages: [token][physical chunk]
  };
};

// Physical 16-byte chunk of chunk ch of token t in a K tile: the 16 tokens that
// the matrix core reads together lie on distinct banks, and so do the four
// that a store writes.
template <int D>
__device__ __forceinline__ int ktile_chunk(int t, int ch) {
  if constexpr (D == 128)
    return ch ^ (((t & 3) << 2) | (t >> 2));
  else
    return ch ^ (((t & 3) << 1) | ((t >> 2) & 1));
}

// (m, l, o) joined with (m1, l1, o1).
__device__ __forceinline__ void join(float& m, float& l, float4& o, float m1, float l1,
                                     const float4& o1) {
  const float mn = fmaxf(m, m1);
  const float w0 = fast_exp2(m - mn), w1 = fast_exp2(m1 - mn);
  l = l * w0 + l1 * w1;
  o.x = o.x * w0 + o1.x * w1;
  o.y = o.y * w0 + o1.y * w1;
  o.z = o.z * w0 + o1.z * w1;
  o.w = o.w * w0 + o1.w * w1;
  m = mn;
}

// Four channels of a query head's output, and its lse.
template <int D, bool BF16>
__device__ __forceinline__ void write_out(const AttendArgs& a, int64_t qh, int c4, float m, float l,
                                          const float4& o) {
  const bool none = l == 0.f;  // every page of the row lies outside the pool
  const float inv = none ? 0.f : 1.f / l;
  reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + qh * D)[c4] =
      make_uint2(pack2<BF16>(o.x * inv, o.y * inv), pack2<BF16>(o.z * inv, o.w * inv));
  if (c4 == 0 && a.lse) a.lse[qh] = none ? kNegInf : m * kLn2 + __logf(l);
}

// P V for one lane column of channels: 16 tokens, or 32.
template <bool BF16>
__device__ __forceinline__ f32x4 pv(const uint32_t (&p)[2], const uint32_t (&v)[2], f32x4 c) {
  return mfma16_k16<BF16>(make_uint2(p[0], p[1]), make_uint2(v[0], v[1]), c);
}
template <bool BF16>
__device__ __forceinline__ f32x4 pv(const uint32_t (&p)[4], const uint32_t (&v)[4], f32x4 c) {
  return mfma16<BF16>(make_uint4(p[0], p[1], p[2], p[3]), make_uint4(v[0], v[1], v[2], v[3]), c);
}

template <int D, bool BF16, bool KV4, int GP, int NW, int PF>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(3, 8)))
void attend_kernel(AttendArgs a) {
  constexpr int UP = KV4 ? 2 : 1;  // pages per unit
  constexpr int VEC = D / 16;      // channels per lane
  constexpr int NT = D / 32;       // score products per page
  constexpr Reach kReach = kDecodeReach<BF16>;
  __shared__ AttendShared<D, GP, NW> sh;
  __shared__ bool s_last;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, kg = lane >> 4;
  const int g = blockIdx.x;
  const Share share = find_share(a, static_cast<int>(blockIdx.y + a.splits * blockIdx.z));
  const int row = share.row, split = share.split, n = share.n;
  const int G = a.group, hkv = a.num_kv_heads;
  if (split < 0) return;
  if (n == 0) {  // an empty row sees nothing
    const int64_t h0 = int64_t(row) * a.num_q_heads + g * G;
    for (int e = threadIdx.x; e < G * D; e += NW * 64)
      static_cast<uint16_t*>(a.out)[h0 * D + e] = 0;
    if (a.lse && threadIdx.x < G) a.lse[h0 + threadIdx.x] = kNegInf;
    return;
  }
  const SeenPages sp = seen_pages(n - 1, n - 1, a.window, a.sinks);
  const int pps = min(share.pages, sp.count);
  const int pb = split * pps;
  const int pe = min(pb + pps, sp.count);
  if (pb >= pe) return;
  const bool whole = sp.count <= pps;  // the row has one split: no state to join
  const int lo = (a.window > 0 && a.window < n) ? n - a.window : 0;

  uint4 qb[NT];
  {
    const uint16_t* qp = static_cast<const uint16_t*>(a.q) +
                         (int64_t(row) * a.num_q_heads + g * G + c) * D + 8 * kg;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      qb[t] = (c < G) ? load16(qp + 32 * t) : zero4();
      qb[t].x ^= a.q_flip, qb[t].y ^= a.q_flip, qb[t].z ^= a.q_flip, qb[t].w ^= a.q_flip;
    }
  }

  float m_run = kLowest, l_part = 0.f;  // head c: running max (log2 units), this lane's sum
  f32x4 acc[VEC];                       // O[4 kg + r][VEC c + j]
#pragma unroll
  for (int j = 0; j < VEC; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // The wave's pages: units u = wave, wave + NW, ... of UP pages from pb.
  const int32_t* bt = a.block_table + int64_t(row) * a.max_pages;
  const int n_units = (pe - pb + UP - 1) / UP;
  const int cnt = n_units > wave ? (n_units - wave + NW - 1) / NW : 0;
  constexpr int CH = 64 / UP;  // units whose page ids one register holds
  auto table_index = [&](int v) { return v < sp.ahead ? v : v + sp.skip; };
  auto page_of = [&](int k) { return pb + UP * (wave + NW * k); };  // first page of unit k
  auto load_ids = [&](int k0) {
    const int v = page_of(k0 + lane / UP) + lane % UP;
    const int id = (v < pe) ? bt[table_index(v)] : -1;
    return (static_cast<uint32_t>(id) < static_cast<uint32_t>(a.num_pool_pages)) ? id : -1;
  };
  int ids = load_ids(0), k0 = 0;

  struct Unit {
    PageRegs<D, KV4> page[UP];
  };
  auto issue = [&](int j, int n_c, Unit& u) {
#pragma unroll
    for (int x = 0; x < UP; ++x) {
      const int id = (j < n_c) ? __builtin_amdgcn_readlane(ids, UP * j + x) : -1;
      if constexpr (KV4) {
        const uint8_t* p = static_cast<const uint8_t*>(a.k_pool) +
                           (int64_t(max(id, 0)) * hkv + g) * Kv4<D>::kBytes;
        const auto r = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint8_t*>(p), (short)0, id >= 0 ? Kv4<D>::kBytes : 0, kBufferFlags);
        u.page[x].template load_k<kCachePolicyStream>(r, lane);
        u.page[x].template load_v<kCachePolicyStream>(r, lane);
      } else {
        // Tokens past the row's length are not fetched: they read as zero.
        const int base = table_index(page_of(k0 + j) + x) * 16;
        const int bytes = id >= 0 ? min(16, n - base) * D * 2 : 0;
        const int64_t at = (int64_t(max(id, 0)) * hkv + g) * 16 * D;
        const uint16_t* kp = static_cast<const uint16_t*>(a.k_pool) + at;
        const uint16_t* vp = static_cast<const uint16_t*>(a.v_pool) + at;
        u.page[x].load(__builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(kp), (short)0,
                                                         bytes, kBufferFlags),
                       __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(vp), (short)0,
                                                         bytes, kBufferFlags),
                       lane);
      }
    }
  };

  auto compute = [&](int j, Unit& u) {
    float xs[4 * UP];
#pragma unroll
    for (int x = 0; x < UP; ++x) {
      PageRegs<D, KV4>& pg = u.page[x];
      f32x4 s = {0.f, 0.f, 0.f, 0.f};
      if constexpr (KV4) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
          s = mfma16<BF16>(kv4_eight<BF16>(pg.k[t], kv4_scale((pg.ks >> (8 * t)) & 0xff)), qb[t],
                           s);
      } else {
        // K through the tile: the lane's tokens kg + 4 i, then A row m = c,
        // token (c / 4) + 4 (c % 4), so that D row 4 kg + r is token kg + 4 r.
        uint4 (&tile)[16][D / 8] = sh.k[wave];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = kg + 4 * i;
          if constexpr (D == 128)
            tile[t][ktile_chunk<D>(t, c)] = make_uint4(pg.k[i][0], pg.k[i][1], pg.k[i][2],
                                                       pg.k[i][3]);
          else
            reinterpret_cast<uint2*>(&tile[t][ktile_chunk<D>(t, c >> 1)])[c & 1] =
                make_uint2(pg.k[i][0], pg.k[i][1]);
        }
        const int at = (c >> 2) + 4 * (c & 3);
#pragma unroll
        for (int t = 0; t < NT; ++t)
          s = mfma16<BF16>(tile[at][ktile_chunk<D>(at, 4 * t + kg)], qb[t], s);
      }
      const int v = page_of(k0 + j) + x;
      const int base = table_index(v) * 16;
      const int id = __builtin_amdgcn_readlane(ids, UP * j + x);
      const bool full = id >= 0 && base + 16 <= n && (base >= lo || base + 16 <= a.sinks);
#pragma unroll
      for (int i = 0; i < 4; ++i) xs[4 * x + i] = s[i];
      if (!full) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = base + (KV4 ? 4 * kg + i : kg + 4 * i);
          const bool ok = id >= 0 && t < n && (t >= lo || t < a.sinks);
          if (!ok) xs[4 * x + i] = kNegInf;
          // An unseen token may hold anything: its V must be finite, as 0 * NaN
          // is not 0.
          if constexpr (KV4) {
            if (!ok) pg.vs &= ~(0xffu << (8 * i));
          } else {
#pragma unroll
            for (int e = 0; e < D / 32; ++e) pg.v[i][e] = ok ? pg.v[i][e] : 0u;
          }
        }
      }
    }
    float top = xs[0];
#pragma unroll
    for (int i = 1; i < 4 * UP; ++i) top = fmaxf(top, xs[i]);
    top *= a.scale_log2;
    if (__builtin_amdgcn_ballot_w64(top > m_run + (kReach.room + kReach.slack)) != 0) {  // rescale O and l
      const float mn = fmaxf(m_run, max_x32(max_x16(top)) - kReach.room);
      const float alpha = fast_exp2(m_run - mn);
      l_part *= alpha;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float ar = __int_as_float(
            __builtin_amdgcn_ds_bpermute((4 * kg + r) << 2, __float_as_int(alpha)));
#pragma unroll
        for (int jj = 0; jj < VEC; ++jj) acc[jj][r] *= ar;
      }
      m_run = mn;
    }
    uint32_t ph[2 * UP], pl[2 * UP];
#pragma unroll
    for (int i = 0; i < 2 * UP; ++i) {
      const float p0 = fast_exp2(fmaf(xs[2 * i], a.scale_log2, -m_run));
      const float p1 = fast_exp2(fmaf(xs[2 * i + 1], a.scale_log2, -m_run));
      l_part += p0 + p1;
      ph[i] = pack2<BF16>(p0, p1);
      pl[i] = pack2<BF16>(p0 - Elem<BF16>::lo(ph[i]), p1 - Elem<BF16>::hi(ph[i]));
    }
    // V of the unit as [token][channel pair].
    uint32_t w[4 * UP][VEC / 2];
#pragma unroll
    for (int x = 0; x < UP; ++x) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (KV4) {
          const float sc = kv4_scale((u.page[x].vs >> (8 * i)) & 0xff);
          if constexpr (D == 128) {
            const uint4 e = kv4_eight<BF16>(u.page[x].v[i], sc);
            w[4 * x + i][0] = e.x, w[4 * x + i][1] = e.y;
            w[4 * x + i][2] = e.z, w[4 * x + i][3] = e.w;
          } else {
            const uint32_t two = u.page[x].v[i >> 1];  // tokens 2 (i / 2) and the next
            w[4 * x + i][0] = (i & 1) ? kv4_pair<BF16, 2>(two, sc) : kv4_pair<BF16, 0>(two, sc);
            w[4 * x + i][1] = (i & 1) ? kv4_pair<BF16, 3>(two, sc) : kv4_pair<BF16, 1>(two, sc);
          }
        } else {
#pragma unroll
          for (int e = 0; e < VEC / 2; ++e) w[4 * x + i][e] = u.page[x].v[i][e];
        }
      }
    }
    uint32_t b[VEC][2 * UP];
#pragma unroll
    for (int jj = 0; jj < VEC; ++jj) {
      const uint32_t sel = (jj & 1) ? 0x07060302u : 0x05040100u;
#pragma unroll
      for (int i = 0; i < 2 * UP; ++i)
        b[jj][i] = __builtin_amdgcn_perm(w[2 * i + 1][jj >> 1], w[2 * i][jj >> 1], sel);
      acc[jj] = pv<BF16>(ph, b[jj], acc[jj]);
    }
#pragma unroll
    for (int jj = 0; jj < VEC; ++jj) acc[jj] = pv<BF16>(pl, b[jj], acc[jj]);
  };

  constexpr int R = PF + 1;
  Unit ring[R];
  for (k0 = 0; k0 < cnt; k0 += CH) {
    const int n_c = min(CH, cnt - k0);
    if (k0 > 0) ids = load_ids(k0);
#pragma unroll
    for (int u = 0; u < PF; ++u) issue(u, n_c, ring[u]);
    for (int j0 = 0; j0 < n_c; j0 += R) {
#pragma unroll
      for (int u = 0; u < R; ++u) {
        issue(j0 + u + PF, n_c, ring[(u + PF) % R]);
        if (j0 + u < n_c) compute(j0 + u, ring[u]);
      }
    }
  }

  // ---- combine the waves ------------------------------------------------------
  const float l_tot = sum_x32(sum_x16(l_part));
  __syncthreads();  // every wave is done with its K tile
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int h = 4 * kg + r;
    if (h < GP) {
#pragma unroll
      for (int jj = 0; jj < VEC; ++jj) sh.o[wave][h][VEC * c + jj] = acc[jj][r];
    }
  }
  if (lane < GP) {
    sh.m[wave][lane] = m_run;
    sh.l[wave][lane] = l_tot;
  }
  __syncthreads();
  constexpr int C4 = D / 4;
  const int64_t pair = int64_t(row) * hkv + g;
  const int64_t slot = pair * a.splits + split;
  for (int e = threadIdx.x; e < G * C4; e += NW * 64) {
    const int h = e / C4, c4 = e % C4;
    float mx = kLowest;
#pragma unroll
    for (int w = 0; w < NW; ++w) mx = fmaxf(mx, sh.m[w][h]);
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float wt = fast_exp2(sh.m[w][h] - mx);
      const float4 ow = reinterpret_cast<const float4*>(sh.o[w][h])[c4];
      l = fmaf(wt, sh.l[w][h], l);
      o.x = fmaf(wt, ow.x, o.x);
      o.y = fmaf(wt, ow.y, o.y);
      o.z = fmaf(wt, ow.z, o.z);
      o.w = fmaf(wt, ow.w, o.w);
    }
    if (whole) {
      write_out<D, BF16>(a, int64_t(row) * a.num_q_heads + g * G + h, c4, mx, l, o);
    } else {
      put_state4<D>(a.st_o + (slot * G + h) * D, c4, o);
      if (c4 == 0) put_state(a.st_ml + (slot * G + h) * 2, mx, l);
    }
  }
  if (whole) return;

  // ---- the last split of the pair to arrive joins them all -------------------------
  // Its sum runs in split order, so the result does not depend on who arrives
  // last.  M = max m_s, w_s = 2^(m_s - M), out = sum w_s o_s / sum w_s l_s.
  const int ns = (sp.count + pps - 1) / pps;
  if (!last_to_arrive(arrival_counter(a.arrivals, pair), ns, &s_last)) return;
  // Threads take (head, chunk of four channels) and, where there are more
  // threads than that, a share of the splits each.
  const int items = G * C4;
  const int sg_n = items < NW * 64 ? NW * 64 / items : 1;
  const int64_t first = pair * a.splits;
  for (int e0 = 0; e0 < items; e0 += NW * 64) {
    const int e = e0 + threadIdx.x % (sg_n * items);
    const int item = sg_n > 1 ? e % items : e;
    const int sg = sg_n > 1 ? e / items : 0;
    const bool on = sg_n > 1 ? threadIdx.x < sg_n * items : item < items;
    const int h = item / C4, c4 = item % C4;
    float m = kLowest, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on) {
      constexpr int U = D / 8;  // states in flight (d = 64: four shares, so fewer each)
      for (int s0 = 0; s0 < ns; s0 += sg_n * U) {
        float2 ml[U];
        float4 os[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (s0 + u * sg_n >= ns) break;  // for every share
          const int s = min(s0 + u * sg_n + sg, ns - 1);
          const int64_t at = (first + s) * G + h;
          ml[u] = get_state2(a.st_ml + at * 2);
          os[u] = get_state4<D>(a.st_o + at * D, c4);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (s0 + u * sg_n >= ns) break;
          if (s0 + u * sg_n + sg < ns) join(m, l, o, ml[u].x, ml[u].y, os[u]);
        }
      }
    }
    if (sg_n > 1) {  // the shares, in order, through LDS (o of `sh` is read no more)
      static_assert(sizeof(sh) - offsetof(decltype(sh), o) >= NW * 64 * 24, "room for the shares");
      float4* s_o = reinterpret_cast<float4*>(&sh.o[0][0][0]);
      float2* s_ml = reinterpret_cast<float2*>(s_o + NW * 64);
      if (on) {
        s_o[threadIdx.x] = o;
        s_ml[threadIdx.x] = make_float2(m, l);
      }
      __syncthreads();
      if (sg == 0 && on)
        for (int k = 1; k < sg_n; ++k) {
          const float2 x = s_ml[threadIdx.x + k * items];
          join(m, l, o, x.x, x.y, s_o[threadIdx.x + k * items]);
        }
    }
    if (on && sg == 0)
      write_out<D, BF16>(a, int64_t(row) * a.num_q_heads + g * G + h, c4, m, l, o);
  }
}

template <int D, bool BF16, bool KV4, int GP>
void launch_one(const AttendArgs& a, hipStream_t s) {
  const dim3 grid(a.num_kv_heads, a.splits, a.batch);
  hipLaunchKernelGGL((attend_kernel<D, BF16, KV4, GP, 4, KV4 ? 2 : 1>), grid, dim3(256), 0, s, a);
}

template <int D, bool BF16, bool KV4>
void launch_gp(const AttendArgs& a, hipStream_t s) {
  if (a.group <= 4) launch_one<D, BF16, KV4, 4>(a, s);
  else if (a.group <= 8) launch_one<D, BF16, KV4, 8>(a, s);
  else launch_one<D, BF16, KV4, 16>(a, s);
}

template <int D, bool BF16>
void launch_fmt(bool kv4, const AttendArgs& a, hipStream_t s) {
  if (kv4) launch_gp<D, BF16, true>(a, s);
  else launch_gp<D, BF16, false>(a, s);
}

}  // namespace

int current_compute_units() {
  static std::atomic<int> known[64];
  int dev = 0, cus = 0;
  if (hipGetDevice(&dev) != hipSuccess) return 0;
  if (dev < 64 && (cus = known[dev].load(std::memory_order_relaxed)) > 0) return cus;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
    return 0;
  if (dev < 64) known[dev].store(cus, std::memory_order_relaxed);
  return cus;
}

pkv_status launch_attend(const pkv_problem& p, bool kv4, const AttendArgs& args, hipStream_t s) {
  const bool bf = p.dtype == PKV_BF16;
  AttendArgs a = args;
  if (a.splits > 1) {
    if ((a.cus = current_compute_units()) <= 0) return PKV_EHIP;
    ranges_of_device(int64_t(a.batch) * a.num_kv_heads, a.cus, &a.fill, &a.even);
  }
  if (p.head_dim == 128) {
    if (bf) launch_fmt<128, true>(kv4, a, s);
    else launch_fmt<128, false>(kv4, a, s);
  } else {
    if (bf) launch_fmt<64, true>(kv4, a, s);
    else launch_fmt<64, false>(kv4, a, s);
  }
  return hipGetLastError() == hipSuccess ? PKV_OK : PKV_EHIP;
}

}  // namespace pkv
