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
// a step through two LDS buffers; each of its four waves owns 32 rows.  Few
// tiles over many keys are cut along the keys (splits, of eight steps and more), and
// the last split of a tile to finish joins the partial states.
//  * S^T = K Q^T on v_mfma_f32_32x32x16: a lane holds one query's scores for 16
//    of 32 keys, so maximum and sum need one exchange with the lane 32 away.
//  * O^T += V^T P^T: the lane's own probabilities are the B operand as they
//    stand (the order of the keys inside a product is free), and V^T comes out
//    of row-major LDS by the transposing read ds_read_b64_tr_b16.
//  * The next step's scores are started before this step's softmax, so that the
//    matrix core works while the vector unit does.
//  * 16-bit pages go to LDS directly (buffer_load ... lds); wave w brings page w
//    of the step.
//  * O is rescaled only when a score passes the running maximum by a good deal
//    (kPromptReach).
// The probabilities enter the second product rounded to the problem's type (a
// relative 2^-8 (bf16) or 2^-11 (f16) at most each, of the size of the output's
// own rounding); maxima, sums (of the unrounded ones) and outputs are fp32 until the
// last rounding.
//
// Measured (bf16, d = 128): 8192 tokens, 32 heads over 8, window 4096: 402-420 us
// for 413 GFLOP, card by card, 0.98-1.03 PFLOP/s, 0.82-0.85 of what a square product
// of 8192 reaches (over 4 bits: 409 us beside 408).  Matrix work fills half of a
// SIMD's cycles and vector work (exponentials, maxima, rounding) 47 %, and the two
// hardly overlap.  Direct loads and two scores in flight brought it from 502 us;
// deeper rings of buffers, pages touched ahead in L2 (430 us), wave priorities and
// tiles of 64 rows brought nothing.  Eight chunks of 9-54 tokens behind a window of
// 4096, 64 heads over 8: 65-69 us (4 bits: 67), of which 46 at the same rate, 8 until
// the first pages are there (dependent loads) and 8 for the last join (65 KiB of
// state a tile and range).  Eight prompts of 183-1659 tokens, d = 64, window 500:
// 20 us (4 bits: 24).
#include "context_internal.h"
#include "kv4_common.h"
#include "mfma.h"
#include "runs.h"
#include "states.h"

namespace pkv {
namespace {

constexpr int kKeys = 64;             // keys per step: four pages, one per wave

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

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;

// 16 bytes a lane from a buffer to LDS, in lane order from p on.
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t r, void* p, uint32_t lane_offset,
                                           uint32_t offset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)p, 16, lane_offset, offset, 0, 0);
}

// Four keys by 16 channels per 16 lanes, transposed: lane a of the 16 passes
// the address of key a / 4, channels 4 (a % 4) .., and gets channel a of the
// four keys.
__device__ __forceinline__ uint2 read_transposed(const void* p) {
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                       (lds_bf16x4*)(lds_void*)(const_cast<void*>(p))));
}

template <int D, bool BF16, bool KV4>
__global__ __launch_bounds__(256, 2) void prompt_kernel(PromptArgs a, int tiles, int slots) {
  constexpr int NQ = D / 16;   // products over the channels
  constexpr int NC = D / 32;   // channel blocks of the output
  constexpr int CH = D / 8;    // 16-byte chunks of a key
  constexpr int KPL = 64 / CH; // keys of one 1 KiB load
  constexpr int NL = 16 / KPL; // loads of a page
  // Objects of their own, named at compile time where they are used: the
  // compiler then knows which loads to LDS a read has to wait for.
  using Tile = uint4[kKeys][CH];
  __shared__ Tile kt0, kt1, vt0, vt1;
  __shared__ bool s_last;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 31, h = lane >> 5;
  const int g = blockIdx.x % a.num_kv_heads;
  const int ts = blockIdx.x / a.num_kv_heads;
  const int G = a.group;

  const TileRun found = find_tile(a, ts, tiles, slots);
  const int k_tile = found.tile, splits = found.splits;
  if (k_tile < 0) return;
  const Run& run = found.run;
  const int item = ts / splits, split = ts - item * splits;
  const int64_t rows64 = int64_t(run.count) * G;
  if (int64_t(k_tile) * kTileRows >= rows64) return;
  const int r0 = k_tile * kTileRows;
  const int rows = static_cast<int>(min(rows64 - r0, int64_t(kTileRows)));  // of this tile
  const int shift = run.len - run.count;  // position of the run's first token
  // Token of the tile's row r, 0 <= r < 128, in the run: x / G = x ceil(4096 / G) /
  // 4096 for x < 144 and G <= 16, as the product is off by less than 4096 / G.
  const int j0 = r0 / G, head0 = r0 - j0 * G;
  auto token_of = [&](int r) {
    return j0 + static_cast<int>(static_cast<uint32_t>(head0 + r) * a.group_inv >> 12);
  };
  const int p_first = max(shift + j0, 0);  // negative positions see nothing
  const int p_last = shift + token_of(rows - 1);

  // This lane's query.
  const int wr = 32 * wave;  // the wave's first row in the tile
  const int my = wr + n;
  const int j = token_of(min(my, rows - 1));
  const int head = (r0 + min(my, rows - 1)) - j * G;
  const int p = max(shift + j, -1);
  const int64_t qh = (int64_t(run.first) + j) * a.num_q_heads + g * G + head;
  const bool mine = my < rows;

  if (p_last < 0) {  // no query of the tile is at a position of the row
    if (mine && split == 0) {
      for (int e = h; e < D / 4; e += 2)
        reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + qh * D)[e] = make_uint2(0u, 0u);
      if (a.lse && h == 0) a.lse[qh] = kNegInf;
    }
    return;
  }
  const int window = a.window > 0 ? a.window : 0x7fffffff;
  const SeenPages sp = seen_pages(p_first, p_last, a.window, a.sinks);
  const int all_steps = (sp.count + 3) >> 2;
  const int per_split = max(found.steps, (all_steps + splits - 1) / splits);
  const int s_begin = split * per_split, s_end = min(s_begin + per_split, all_steps);
  if (s_begin >= s_end) return;
  const int32_t* bt = a.block_table + int64_t(run.row) * a.max_pages;

  // Steps whose every key is seen by every query of the wave (absent pages
  // aside): those behind the start of the last query's window and before the
  // first query's position, or those before the end of the sinks.
  const int pw_first = max(shift + token_of(min(wr, rows - 1)), -1);
  const int pw_last = max(shift + token_of(min(wr + 31, rows - 1)), -1);
  int full_lo = 0;
  if (a.window > 0) {
    const int w0 = max(pw_last - a.window + 1, 0);           // first token all of them see
    full_lo = (max(((w0 + 15) >> 4) - sp.skip, sp.ahead) + 3) >> 2;
  }
  const int full_hi = (((pw_first + 1) >> 4) - sp.skip) >> 2;  // pages that end by pw_first
  const int sink_hi = min(min(a.sinks, pw_first + 1) >> 4, sp.ahead) >> 2;

  // ---- bringing pages to LDS: wave w brings page w of a step -----------------------
  // Pool pages of 16 steps, one per lane; -1 where there is none.
  auto load_ids = [&](int s0) {
    const int v = 4 * s0 + lane;
    const int id = v < sp.count ? bt[v < sp.ahead ? v : v + sp.skip] : -1;
    return static_cast<uint32_t>(id) < static_cast<uint32_t>(a.num_pool_pages) ? id : -1;
  };
  int ids0 = s_begin, ids = load_ids(s_begin), ids_next = load_ids(s_begin + 16);
  // B operand of the scores: channels 16 t + 8 h .. of this lane's query (lanes
  // behind the tile's rows repeat its last one).
  uint4 qf[NQ];
  {
    const uint16_t* qp = static_cast<const uint16_t*>(a.q) + qh * D + 8 * h;
#pragma unroll
    for (int t = 0; t < NQ; ++t) qf[t] = load16(qp + 16 * t);
  }
  auto base_of = [&](int s) {
    const int v = 4 * s + wave;
    return 16 * (v < sp.ahead ? v : v + sp.skip);
  };
  // Offset of a lane's 16 bytes in its page, load by load, so that they land
  // where k_chunk and v_chunk say: LDS is filled in lane order.
  uint32_t k_off[NL];
  const int lk = lane / CH, lc = lane % CH;
#pragma unroll
  for (int i = 0; i < NL; ++i)
    k_off[i] = ((KPL * i + lk) * CH + k_chunk<D>(KPL * i + lk, lc)) * 16;
  const uint32_t v_off = (lk * CH + v_chunk<D>(lk, lc)) * 16;
  auto rsrc = [&](const void* pool, int id, int bytes) {
    bytes = __builtin_amdgcn_readfirstlane(bytes);
    const int64_t at = (int64_t(max(id, 0)) * a.num_kv_heads + g) * 32 * D;
    return __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(static_cast<const char*>(pool)) + at, (short)0, bytes, kBufferFlags);
  };
  // Bytes of a page up to the last token that some query sees: behind them
  // loads give zero.
  auto seen_bytes = [&](int id, int s) {
    return id < 0 ? 0 : min(max(p_last + 1 - base_of(s), 0), 16) * 2 * D;
  };
  Kv4Page<D> k4, v4;  // 4-bit: a step's page on its way (K and V travel a step apart)
  auto rsrc4 = [&](int id) {
    const int64_t at = (int64_t(max(id, 0)) * a.num_kv_heads + g) * Kv4<D>::kBytes;
    return __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(static_cast<const char*>(a.k_pool)) + at, (short)0,
        id >= 0 ? Kv4<D>::kBytes : 0, kBufferFlags);
  };
  auto issue_k = [&](int id, int s, Tile& kt) __attribute__((always_inline)) {
    if constexpr (KV4) {
      k4.template load_k<0>(rsrc4(id), lane);
    } else {
      const auto r = rsrc(a.k_pool, id, seen_bytes(id, s));
#pragma unroll
      for (int i = 0; i < NL; ++i)
        load_lds16(r, &kt[16 * wave + KPL * i][0], k_off[i], 0);
    }
  };
  auto issue_v = [&](int id, int s, Tile& vt) __attribute__((always_inline)) {
    if constexpr (KV4) {
      v4.template load_v<0>(rsrc4(id), lane);
    } else {
      const auto r = rsrc(a.v_pool, id, seen_bytes(id, s));
#pragma unroll
      for (int i = 0; i < NL; ++i)
        load_lds16(r, &vt[16 * wave + KPL * i][0], v_off, i * 1024);
    }
  };
  // A lane number whose uses are computed where they stand: the LDS offsets of a
  // conversion, kept over the loop instead, spilled (one prompt of 8192: 506 us).
  auto lane_now = [&] {
    int x = lane;
    asm volatile("" : "+v"(x));
    return x;
  };
  // 4-bit: to LDS, converted.
  auto put_k = [&](Tile& kt) __attribute__((always_inline)) {
    if constexpr (KV4) {
      const int ln = lane_now(), kg = ln >> 4, t = 16 * wave + (ln & 15);
#pragma unroll
      for (int b = 0; b < D / 32; ++b)
        kt[t][k_chunk<D>(t, 4 * b + kg)] =
            kv4_eight<BF16>(k4.k[b], kv4_scale((k4.ks >> (8 * b)) & 0xff));
    }
  };
  auto put_v = [&](Tile& vt) __attribute__((always_inline)) {
    if constexpr (KV4) {
      const int ln = lane_now(), c = ln & 15;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 16 * wave + 4 * (ln >> 4) + i;
        const float sc = kv4_scale((v4.vs >> (8 * i)) & 0xff);
        if constexpr (D == 128) {
          vt[t][v_chunk<D>(t, c)] = kv4_eight<BF16>(v4.v[i], sc);
        } else {
          const uint32_t two = v4.v[i >> 1];
          reinterpret_cast<uint2*>(&vt[t][v_chunk<D>(t, c >> 1)])[c & 1] =
              (i & 1) ? make_uint2(kv4_pair<BF16, 2>(two, sc), kv4_pair<BF16, 3>(two, sc))
                      : make_uint2(kv4_pair<BF16, 0>(two, sc), kv4_pair<BF16, 1>(two, sc));
        }
      }
    }
  };
  // Clear the V rows of this wave's page of step s that no query of the tile
  // sees, all of them where there is no page: they may hold anything, and 0 *
  // NaN is not 0.  After the page has landed, before the others read it.
  auto clear_unseen = [&](int id, int s, Tile& vt) __attribute__((always_inline)) {
    const int b0 = base_of(s);
    if (id >= 0 && b0 + 15 <= p_last && (p_first - b0 < window || b0 + 15 < a.sinks)) return;
    const int ln = lane_now();
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int r = KPL * i + ln / CH, t = b0 + r;
      if (id < 0 || t > p_last || (p_first - t >= window && t >= a.sinks))
        vt[16 * wave + r][ln % CH] = zero4();
    }
  };

  // This wave's loads have reached LDS.
  auto landed = [] { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); };

  constexpr Reach kReach = kPromptReach<BF16>;

  // ---- one step ---------------------------------------------------------------------
  float m_run = kLowest, l_part = 0.f;
  f32x16 acc[NC];
#pragma unroll
  for (int cb = 0; cb < NC; ++cb)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[cb][i] = 0.f;

  auto scores = [&](const Tile& kt, f32x16 (&s)[2]) __attribute__((always_inline)) {
#pragma unroll
    for (int sub = 0; sub < 2; ++sub)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[sub][i] = 0.f;
#pragma unroll
    for (int t = 0; t < NQ; ++t)
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
        const int key = 32 * sub + n;
        s[sub] = mfma32<BF16>(kt[key][k_chunk<D>(key, 2 * t + h)], qf[t], s[sub]);
      }
  };
  // `bad`: this step has absent pages (a bit each).  The tokens of a page that
  // this lane's query sees, a bit each: below p + 1 and not below the window's
  // start, or below the sinks' end.
  auto mask = [&](int st, uint32_t bad, f32x16 (&s)[2]) {
    const int lo = max(p + 1 - window, 0), sink = min(a.sinks, p + 1);
    auto below = [](int n) { return (1u << min(max(n, 0), 16)) - 1u; };
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int v = 4 * st + x;
      const int b0 = 16 * (v < sp.ahead ? v : v + sp.skip);
      uint32_t seen = (below(p + 1 - b0) & ~below(lo - b0)) | below(sink - b0);
      seen = ((bad >> x) & 1) ? 0u : seen >> (4 * h);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t keep = __builtin_amdgcn_sbfe(seen, 8 * (i >> 2) + (i & 3), 1);
        const uint32_t e = __float_as_uint(s[x >> 1][8 * (x & 1) + i]);
        s[x >> 1][8 * (x & 1) + i] = __uint_as_float((e & keep) | (0xff800000u & ~keep));
      }
    }
  };
  const int kq = (lane & 15) >> 2, cq = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
  auto softmax_pv = [&](const Tile& vt, const f32x16 (&s)[2]) __attribute__((always_inline)) {
    float t0 = max3(s[0][0], s[1][0], s[1][0]), t1 = max3(s[0][1], s[1][1], s[1][1]);
#pragma unroll
    for (int i = 2; i < 16; i += 2) {
      t0 = max3(t0, s[0][i], s[1][i]);
      t1 = max3(t1, s[0][i + 1], s[1][i + 1]);
    }
    const float top = max_x32(fmaxf(t0, t1)) * a.scale_log2;
    if (__builtin_amdgcn_ballot_w64(top > m_run + (kReach.room + kReach.slack)) != 0) {
      const float mn = fmaxf(m_run, top - kReach.room);
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
        pb[sub][i] = pack2<BF16>(e0, e1);
        l_part += e0 + e1;
      }
    // Lane's share of a transposed read: key lane % 16 / 4 of four, 16-byte
    // chunk 2 (lane / 16 % 2) + lane % 4 / 2 of a channel block, half lane % 2.
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      const uint4 bv = make_uint4(pb[ks >> 1][4 * (ks & 1)], pb[ks >> 1][4 * (ks & 1) + 1],
                                  pb[ks >> 1][4 * (ks & 1) + 2], pb[ks >> 1][4 * (ks & 1) + 3]);
#pragma unroll
      for (int cb = 0; cb < NC; ++cb) {
        const int key = 16 * ks + 4 * h + kq;
        const uint2 v0 = read_transposed(
            reinterpret_cast<const uint2*>(&vt[key][v_chunk<D>(key, 4 * cb + cq)]) +
            (lane & 1));
        const uint2 v1 = read_transposed(
            reinterpret_cast<const uint2*>(&vt[key + 8][v_chunk<D>(key + 8, 4 * cb + cq)]) +
            (lane & 1));
        acc[cb] = mfma32<BF16>(make_uint4(v0.x, v0.y, v1.x, v1.y), bv, acc[cb]);
      }
    }
  };

  // ---- the walk -----------------------------------------------------------------------
  // During step s, K of step s + 2 and V of step s + 1 are under way.
  uint64_t no_page = __builtin_amdgcn_ballot_w64(ids < 0);
  // This wave's page of a step, and the step's absent pages (a bit each).
  struct StepPages {
    int id;
    uint32_t bad;
  };
  auto pages_of = [&](int s) {
    StepPages r{-1, 15u};
    if (s >= s_end) return r;
    if (s - ids0 >= 16) {
      ids0 += 16;
      ids = ids_next;
      ids_next = load_ids(ids0 + 16);
      no_page = __builtin_amdgcn_ballot_w64(ids < 0);
    }
    const int at = 4 * (s - ids0);
    r.id = __builtin_amdgcn_readlane(ids, at + wave);
    r.bad = static_cast<uint32_t>(no_page >> at) & 15u;
    return r;
  };
  StepPages pg0 = pages_of(s_begin), pg1 = pages_of(s_begin + 1);
  issue_k(pg0.id, s_begin, kt0);
  issue_v(pg0.id, s_begin, vt0);
  put_k(kt0);
  issue_k(pg1.id, s_begin + 1, kt1);
  put_k(kt1);
  put_v(vt0);
#pragma unroll
  for (int t = 0; t < NQ; ++t)
    qf[t].x ^= a.q_flip, qf[t].y ^= a.q_flip, qf[t].z ^= a.q_flip, qf[t].w ^= a.q_flip;
  landed();
  clear_unseen(pg0.id, s_begin, vt0);
  __syncthreads();
  f32x16 sa[2], sb[2];
  scores(kt0, sa);
  __syncthreads();  // kt0 is free
  // One step: `sc` holds its scores, `sn` gets the next step's (of nothing
  // behind the last: not used).
  auto step = [&](int s, Tile& k_cur, Tile& k_next, Tile& v_cur, Tile& v_next, f32x16 (&sc)[2],
                  f32x16 (&sn)[2]) __attribute__((always_inline)) {
    const StepPages pg2 = pages_of(s + 2);
    if constexpr (!KV4) {
      issue_k(pg2.id, s + 2, k_cur);
      issue_v(pg1.id, s + 1, v_next);
    }
    scores(k_next, sn);
    if constexpr (KV4) {  // to registers: later, so that fewer are taken meanwhile
      issue_k(pg2.id, s + 2, k_cur);
      issue_v(pg1.id, s + 1, v_next);
    }
    const bool full = (s >= full_lo && s < full_hi) || s < sink_hi;
    if (!full || pg0.bad) mask(s, pg0.bad, sc);
    softmax_pv(v_cur, sc);
    put_k(k_cur);
    put_v(v_next);
    landed();
    clear_unseen(pg1.id, s + 1, v_next);
    pg0 = pg1, pg1 = pg2;
    __syncthreads();
  };
  for (int s = s_begin; s < s_end; s += 2) {
    step(s, kt0, kt1, vt0, vt1, sa, sb);
    if (s + 1 < s_end) step(s + 1, kt1, kt0, vt1, vt0, sb, sa);
  }

  // ---- outputs ----------------------------------------------------------------
  float l = sum_x32(l_part);
  const int ns = (all_steps + per_split - 1) / per_split;
  if (ns > 1) {
    // State of a split: [d / 2 pairs][thread][2] of O and [thread][2] of m, l.
    const int64_t tg = int64_t(item) * a.num_kv_heads + g;
    constexpr int64_t kSlot = 256 * (D / 2 + 2);
    float* mine_st = a.state + (tg * a.splits + split) * kSlot;
#pragma unroll
    for (int cb = 0; cb < NC; ++cb)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        put_state(mine_st + ((cb * 8 + i) * 256 + tid) * 2, acc[cb][2 * i], acc[cb][2 * i + 1]);
    put_state(mine_st + (NC * 8 * 256 + tid) * 2, m_run, l);
    if (!last_to_arrive(arrival_counter(a.arrivals, tg), ns, &s_last)) return;
    // Joined in split order, so that the result does not depend on the order
    // of arrival: first the maximum, then the weighted sums.
    const float* st0 = a.state + tg * a.splits * kSlot;
    constexpr int U = 8;  // splits whose m and l are under way together
    auto get_ml = [&](int s) {
      return get_state2(st0 + min(s, ns - 1) * kSlot + (NC * 8 * 256 + tid) * 2);
    };
    m_run = kLowest;
    for (int s0 = 0; s0 < ns; s0 += U) {
      float2 ml[U];
#pragma unroll
      for (int u = 0; u < U; ++u) ml[u] = get_ml(s0 + u);
#pragma unroll
      for (int u = 0; u < U; ++u) m_run = fmaxf(m_run, ml[u].x);
    }
    l = 0.f;
#pragma unroll
    for (int cb = 0; cb < NC; ++cb)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[cb][i] = 0.f;
    for (int s = 0; s < ns; ++s) {
      const float* st = st0 + s * kSlot;
      const float2 ml = get_ml(s);
      const float w = fast_exp2(ml.x - m_run);
      l = fmaf(w, ml.y, l);
#pragma unroll
      for (int cb = 0; cb < NC; ++cb)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 o = get_state2(st + ((cb * 8 + i) * 256 + tid) * 2);
          acc[cb][2 * i] = fmaf(w, o.x, acc[cb][2 * i]);
          acc[cb][2 * i + 1] = fmaf(w, o.y, acc[cb][2 * i + 1]);
        }
    }
  }
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
void launch_fmt(bool kv4, const PromptArgs& a, int tiles, int slots, uint32_t grid,
                hipStream_t s) {
  if (kv4)
    hipLaunchKernelGGL((prompt_kernel<D, BF16, true>), dim3(grid), dim3(256), 0, s, a, tiles,
                       slots);
  else
    hipLaunchKernelGGL((prompt_kernel<D, BF16, false>), dim3(grid), dim3(256), 0, s, a, tiles,
                       slots);
}

}  // namespace

pkv_status launch_prompt(const pkv_problem& p, bool kv4, const PromptArgs& a, hipStream_t s) {
  const int64_t tiles = prompt_tiles(a);
  const bool bf = p.dtype == PKV_BF16;
  const uint32_t n = static_cast<uint32_t>(tiles * a.num_kv_heads * a.splits);
  // Workgroups a KV head that run at the same time: two a compute unit.
  int slots = 0;
  if (a.splits > 1) {
    const int cus = current_compute_units();
    if (cus <= 0) return PKV_EHIP;
    slots = 2 * cus / a.num_kv_heads;
  }
  if (p.head_dim == 128) {
    if (bf) launch_fmt<128, true>(kv4, a, static_cast<int>(tiles), slots, n, s);
    else launch_fmt<128, false>(kv4, a, static_cast<int>(tiles), slots, n, s);
  } else {
    if (bf) launch_fmt<64, true>(kv4, a, static_cast<int>(tiles), slots, n, s);
    else launch_fmt<64, false>(kv4, a, static_cast<int>(tiles), slots, n, s);
  }
  return hipGetLastError() == hipSuccess ? PKV_OK : PKV_EHIP;
}

}  // namespace pkv
