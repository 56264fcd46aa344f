// Prompt attention (gfx950): many query tokens per row over the paged cache,
// causal, with a sliding window and sinks; 16-bit pages, the 4-bit or the 8-bit
// pool.  CROSS: every query sees the whole row.
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
// Measured (bf16, d = 128): 8192 tokens, 32 heads over 8, window 4096, 413 GFLOP: 392-445
// us, card by card, 0.93-1.05 PFLOP/s, 0.73-0.80 of what a square product of 8192
// reaches on the same card (1.28-1.39; over 4 bits 395-460, 8 bits 405-473).  Bound by
// power: it runs at 1.96 GHz, not 2.4, and all 8192 keys for every query at 1.89, with 52
// and 55 % of the matrix core's cycles taken and 50 of the vector unit's (the product at
// 1.91 GHz, 70 and 28 %), so shorter instruction sequences move nothing there (the weights
// between the products of the scores, one after the other without a gap, took the same
// time).  Direct loads and two scores in flight brought it from 502 us; deeper rings of
// buffers, pages touched ahead in L2 (430 us), wave priorities and tiles of 64 rows
// brought nothing; waves without queries that skip their products 2 % more on full tiles.
// Eight chunks of 36 tokens behind a window of 4096, 64 heads over 8: 70-77 us (4 bits
// 75-80, 8 bits 77-88).  Eight prompts of 183-1659 tokens, d = 64, window 500: 19-21 us.
// 8 bits: 23523 tokens of eight prompts, f16, 610 GFLOP: 665-777 us, 0.63-0.70 of the
// product's rate, at 2.09 GHz with 43 % of the matrix core's cycles and 52 of the vector
// unit's, which converts as well.  K and V of a page share one page's registers in turn: with both in hand
// the kernel spilled (one prompt 498 us).  289 tokens behind 1024-32768 and a window of
// 4096: 70-77 us, bound by latency (2.39 GHz, 25 and 34 %).
// CROSS: 2969 queries of eight rows of 1024-8192 states, 253 GFLOP: 277-320 us (with the
// rows as they come 303-306 where sorted take 288-292), 2.09 GHz, 43 and 40 %: 96 tiles of
// 29-124 steps for 64 places a KV head end at 148 steps, 123.5 on the average.
#pragma once

#include <type_traits>

#include "context/context_internal.h"
#include "context/kv4_common.h"
#include "context/mfma.h"
#include "context/runs.h"
#include "context/states.h"
#include "serving/kv8_common.h"
#include "serving/shares.h"

namespace pkv {

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

// One of equal ranges of a tile's steps (find_tile).
struct SplitPart {
  int item;   // of the tile among those that the launch lists
  int split, splits;
  int steps;  // of a range at least
};

// A share's part of a tile: [from, to) of its cost on the line, the parts of other shares
// ending at multiples of `each`.  In LDS, a copy for each wave: its registers are needed
// for the tile.
struct LinePart {
  int64_t start, cost, slot;  // as in SharePart
  int64_t from, to, each, end;
  __device__ __forceinline__ int step_at(int64_t v, int all_steps) const {
    return __builtin_amdgcn_readfirstlane(
        static_cast<int>(static_cast<double>(min(max(v, int64_t(0)), cost)) * all_steps /
                         static_cast<double>(cost)));
  }
};

// A tile of a run, or a part of its steps.  Part: SplitPart or LinePart.
template <int D, bool BF16, Cache F, bool CROSS, typename Part>
__device__ __forceinline__ void prompt_tile(const PromptArgs& a, int g, const Run& run, int k_tile,
                                            const Part& part, uint4 (&kt0)[kKeys][D / 8],
                                            uint4 (&kt1)[kKeys][D / 8], uint4 (&vt0)[kKeys][D / 8],
                                            uint4 (&vt1)[kKeys][D / 8], bool* s_last) {
  constexpr bool kLine = std::is_same_v<Part, LinePart>;
  constexpr bool KV4 = F == Cache::k4, KV8 = F == Cache::k8;
  // 16-bit pages: scores and weights in one stretch of code, in the order that the
  // groups below set.  A launch of few workgroups takes 4 % less (chunks of 36 tokens 72.6
  // and 69.6 us); a full one is bound by power, not by cycles, and takes the same.
  // (With a page's registers between, 4 and 8 bits took 2-4 % more.)
  constexpr bool kInterleave = F == Cache::k16 && D == 128;
  constexpr int kVector = 0x402, kMfma = 0x008, kDsRead = 0x100;  // classes of instructions
  constexpr int NQ = D / 16;   // products over the channels
  constexpr int NC = D / 32;   // channel blocks of the output
  constexpr int CH = D / 8;    // 16-byte chunks of a key
  constexpr int KPL = 64 / CH; // keys of one 1 KiB load
  constexpr int NL = 16 / KPL; // loads of a page
  using Tile = uint4[kKeys][CH];
  int thread = threadIdx.x;
  // New to every tile: what depends on it alone, kept over the loop of a share's tiles,
  // spilled.
  if constexpr (kLine) asm volatile("" : "+v"(thread));
  const int tid = thread, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 31, h = lane >> 5;
  const int G = a.group;
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
  // Position of the run's token j; CROSS: every query stands behind the whole row.
  auto position = [&](int j) { return CROSS ? run.len - 1 : shift + j; };
  const int p_first = max(position(j0), 0);  // negative positions see nothing
  const int p_last = position(token_of(rows - 1));

  // This lane's query.
  const int wr = 32 * wave;  // the wave's first row in the tile
  const bool busy = wr < rows;  // else the wave's results are nobody's: no states of O
  const int my = wr + n;
  const int j = token_of(min(my, rows - 1));
  const int head = (r0 + min(my, rows - 1)) - j * G;
  const int p = max(position(j), -1);
  const int64_t qh = (int64_t(run.first) + j) * a.num_q_heads + g * G + head;
  const bool mine = my < rows;

  if (p_last < 0) {  // no query of the tile is at a position of the row
    bool writes;
    if constexpr (kLine) writes = part.from == 0;
    else writes = part.split == 0;
    if (mine && writes) {
      for (int e = h; e < D / 4; e += 2)
        reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + qh * D)[e] = make_uint2(0u, 0u);
      if (a.lse && h == 0) a.lse[qh] = kNegInf;
    }
    return;
  }
  const int window = a.window > 0 ? a.window : 0x7fffffff;
  const SeenPages sp = seen_pages(p_first, p_last, a.window, a.sinks);
  const int all_steps = (sp.count + 3) >> 2;
  int s_begin, s_end, per_split = 0;
  if constexpr (kLine) {
    s_begin = part.step_at(part.from, all_steps), s_end = part.step_at(part.to, all_steps);
  } else {
    per_split = max(part.steps, (all_steps + part.splits - 1) / part.splits);
    s_begin = part.split * per_split, s_end = min(s_begin + per_split, all_steps);
  }
  // A part of a cut tile may be too short for a step: it leaves a state of nothing.
  if constexpr (kLine) {
    if (all_steps == 0 || (s_begin >= s_end && part.to - part.from == part.cost)) return;
  } else {
    if (s_begin >= s_end) return;
  }
  const int32_t* bt = a.block_table + int64_t(run.row) * a.max_pages;

  // Steps whose every key is seen by every query of the wave (absent pages
  // aside): those behind the start of the last query's window and before the
  // first query's position, or those before the end of the sinks.
  const int pw_first = max(position(token_of(min(wr, rows - 1))), -1);
  const int pw_last = max(position(token_of(min(wr + 31, rows - 1))), -1);
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
  // 8 bits: the two scale bytes of each of those pages.
  auto load_scales = [&](int id) -> uint32_t {
    if constexpr (!KV8) return 0;
    return id >= 0 ? reinterpret_cast<const uint16_t*>(
                         a.scales)[int64_t(id) * a.num_kv_heads + g] : 0;
  };
  uint32_t scales = load_scales(ids), scales_next = load_scales(ids_next);
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
  // 4 and 8 bits: a step's page on its way (K and V travel a step apart).
  std::conditional_t<KV8, Kv8Page<D>, Kv4Page<D>> kp, vp;
  auto rsrc_packed = [&](int id) {
    constexpr int kBytes = KV8 ? Kv8<D>::kBytes : Kv4<D>::kBytes;
    const int64_t at = (int64_t(max(id, 0)) * a.num_kv_heads + g) * kBytes;
    return __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(static_cast<const char*>(a.k_pool)) + at, (short)0,
        id >= 0 ? kBytes : 0, kBufferFlags);
  };
  auto issue_k = [&](int id, int s, Tile& kt) __attribute__((always_inline)) {
    if constexpr (KV4 || KV8) {
      kp.template load_k<0>(rsrc_packed(id), lane);
    } else {
      const auto r = rsrc(a.k_pool, id, seen_bytes(id, s));
#pragma unroll
      for (int i = 0; i < NL; ++i)
        load_lds16(r, &kt[16 * wave + KPL * i][0], k_off[i], 0);
    }
  };
  auto issue_v = [&](int id, int s, Tile& vt) __attribute__((always_inline)) {
    if constexpr (KV4 || KV8) {
      vp.template load_v<0>(rsrc_packed(id), lane);
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
  // 4 and 8 bits: to LDS, converted.
  // (8 bits: `sc`, the scale bytes of the page.)
  auto put_k = [&](Tile& kt, uint32_t sc) __attribute__((always_inline)) {
    if constexpr (KV4 || KV8) {
      const int ln = lane_now(), kg = ln >> 4, t = 16 * wave + (ln & 15);
#pragma unroll
      for (int b = 0; b < D / 32; ++b) {
        uint4& to = kt[t][k_chunk<D>(t, 4 * b + kg)];
        if constexpr (KV8)
          to = kv8_eight<BF16>(kp.k[2 * b], kp.k[2 * b + 1], kv8_scale(sc & 0xff));
        else
          to = kv4_eight<BF16>(kp.k[b], kv4_scale((kp.ks >> (8 * b)) & 0xff));
      }
    }
  };
  auto put_v = [&](Tile& vt, uint32_t scales_v) __attribute__((always_inline)) {
    if constexpr (KV4) {
      const int ln = lane_now(), c = ln & 15;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 16 * wave + 4 * (ln >> 4) + i;
        const float sc = kv4_scale((vp.vs >> (8 * i)) & 0xff);
        if constexpr (D == 128) {
          vt[t][v_chunk<D>(t, c)] = kv4_eight<BF16>(vp.v[i], sc);
        } else {
          const uint32_t two = vp.v[i >> 1];
          reinterpret_cast<uint2*>(&vt[t][v_chunk<D>(t, c >> 1)])[c & 1] =
              (i & 1) ? make_uint2(kv4_pair<BF16, 2>(two, sc), kv4_pair<BF16, 3>(two, sc))
                      : make_uint2(kv4_pair<BF16, 0>(two, sc), kv4_pair<BF16, 1>(two, sc));
        }
      }
    } else if constexpr (KV8) {
      const int ln = lane_now(), c = ln & 15;
      const float sc = kv8_scale(scales_v >> 8);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 16 * wave + 4 * (ln >> 4) + i;
        if constexpr (D == 128) {
          vt[t][v_chunk<D>(t, c)] = kv8_eight<BF16>(vp.v[2 * i], vp.v[2 * i + 1], sc);
        } else {
          reinterpret_cast<uint2*>(&vt[t][v_chunk<D>(t, c >> 1)])[c & 1] =
              make_uint2(kv8_pair<BF16, false>(vp.v[i], sc), kv8_pair<BF16, true>(vp.v[i], sc));
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
  // The running maximum of the query, moved where a step's scores pass it.
  auto raise = [&](const f32x16 (&s)[2]) __attribute__((always_inline)) {
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
  };
  auto weigh = [&](const Tile& vt, const f32x16 (&s)[2]) __attribute__((always_inline)) {
    uint32_t pb[2][8];
#pragma unroll
    for (int sub = 0; sub < 2; ++sub)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float e0 = fast_exp2(fmaf(s[sub][2 * i], a.scale_log2, -m_run));
        const float e1 = fast_exp2(fmaf(s[sub][2 * i + 1], a.scale_log2, -m_run));
        pb[sub][i] = pack2<BF16>(e0, e1);
        l_part += e0 + e1;
        // The sum with the weights: left to the step's end, it kept all of them.
        if constexpr (kInterleave) asm("" : "+v"(pb[sub][i]), "+v"(l_part));
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
  // During step s, K of step s + 2 and V of step s + 1 are under way (8 bits: V from
  // the end of step s - 1 to the scores, K from then on, one page's registers for both).
  uint64_t no_page = __builtin_amdgcn_ballot_w64(ids < 0);
  // This wave's page of a step, and the step's absent pages (a bit each).
  struct StepPages {
    int id;
    uint32_t bad;
    uint32_t scales;  // 8 bits: the page's
  };
  auto pages_of = [&](int s) {
    StepPages r{-1, 15u, 0u};
    if (s >= s_end) return r;
    if (s - ids0 >= 16) {
      ids0 += 16;
      ids = ids_next;
      ids_next = load_ids(ids0 + 16);
      scales = scales_next;
      scales_next = load_scales(ids_next);
      no_page = __builtin_amdgcn_ballot_w64(ids < 0);
    }
    const int at = 4 * (s - ids0);
    r.id = __builtin_amdgcn_readlane(ids, at + wave);
    r.bad = static_cast<uint32_t>(no_page >> at) & 15u;
    if constexpr (KV8) r.scales = __builtin_amdgcn_readlane(scales, at + wave);
    return r;
  };
  if (!kLine || s_begin < s_end) {
  StepPages pg0 = pages_of(s_begin), pg1 = pages_of(s_begin + 1);
  issue_k(pg0.id, s_begin, kt0);
  issue_v(pg0.id, s_begin, vt0);
  put_k(kt0, pg0.scales);
  issue_k(pg1.id, s_begin + 1, kt1);
  put_k(kt1, pg1.scales);
  put_v(vt0, pg0.scales);
#pragma unroll
  for (int t = 0; t < NQ; ++t)
    qf[t].x ^= a.q_flip, qf[t].y ^= a.q_flip, qf[t].z ^= a.q_flip, qf[t].w ^= a.q_flip;
  landed();
  clear_unseen(pg0.id, s_begin, vt0);
  __syncthreads();
  f32x16 sa[2], sb[2];
  if constexpr (KV8) issue_v(pg1.id, s_begin + 1, vt1);
  scores(kt0, sa);
  __syncthreads();  // kt0 is free
  // One step: `sc` holds its scores, `sn` gets the next step's (of nothing
  // behind the last: not used).
  auto step = [&](int s, Tile& k_cur, Tile& k_next, Tile& v_cur, Tile& v_next, f32x16 (&sc)[2],
                  f32x16 (&sn)[2]) __attribute__((always_inline)) {
    const StepPages pg2 = pages_of(s + 2);
    if constexpr (!KV4 && !KV8) {
      issue_k(pg2.id, s + 2, k_cur);
      issue_v(pg1.id, s + 1, v_next);
    }
    const bool full = (s >= full_lo && s < full_hi) || s < sink_hi;
    auto settle = [&] {
      if (!full || pg0.bad) mask(s, pg0.bad, sc);
      raise(sc);
    };
    if constexpr (kInterleave) settle();
    scores(k_next, sn);
    if constexpr (KV4) {  // to registers: later, so that fewer are taken meanwhile
      issue_k(pg2.id, s + 2, k_cur);
      issue_v(pg1.id, s + 1, v_next);
    }
    if constexpr (KV8) {  // V came under the last step's end and the scores; now K
      put_v(v_next, pg1.scales);
      issue_k(pg2.id, s + 2, k_cur);
    }
    if constexpr (!kInterleave) settle();
    weigh(v_cur, sc);
    if constexpr (kInterleave) {
      // Between two products of the next scores: an LDS read four products ahead and a
      // share of this step's weights (32 exponentials, 80 other instructions).
      __builtin_amdgcn_sched_group_barrier(kDsRead, 4, 0);
#pragma unroll
      for (int i = 0; i < 2 * NQ; ++i) {
        __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
        __builtin_amdgcn_sched_group_barrier(kDsRead, 1, 0);
        __builtin_amdgcn_sched_group_barrier(kVector, 112 / (2 * NQ), 0);
      }
#pragma unroll
      for (int i = 0; i < 4 * NC; ++i) {
        __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
        __builtin_amdgcn_sched_group_barrier(kDsRead, 2, 0);
      }
    }
    put_k(k_cur, pg2.scales);
    if constexpr (!KV8) put_v(v_next, 0u);
    if constexpr (KV8) issue_v(pg2.id, s + 2, v_cur);
    else landed();
    clear_unseen(pg1.id, s + 1, v_next);
    pg0 = pg1, pg1 = pg2;
    __syncthreads();
  };
  for (int s = s_begin; s < s_end; s += 2) {
    step(s, kt0, kt1, vt0, vt1, sa, sb);
    if (s + 1 < s_end) step(s + 1, kt1, kt0, vt1, vt0, sb, sa);
  }
  }

  // ---- outputs ----------------------------------------------------------------
  float l = sum_x32(l_part);
  bool whole;
  if constexpr (kLine) whole = part.to - part.from == part.cost;
  else whole = per_split >= all_steps;
  if (!whole) {
    // State of a part: [d / 2 pairs][thread][2] of O and [thread][2] of m, l.
    constexpr int64_t kSlot = 256 * (D / 2 + 2);
    int64_t tg, slot0, slot1;      // tile and KV head; slots of a part of it and of the next
    int mine_at, first_at = 0, last_at;  // parts: this one, and those of the tile
    if constexpr (kLine) {
      tg = part.slot * a.num_kv_heads + g;
      slot0 = tg, slot1 = tg + a.num_kv_heads;
      mine_at = static_cast<int>((part.start + part.from) / part.each);
      first_at = static_cast<int>(part.start / part.each);
      last_at = static_cast<int>((part.start + part.cost - 1) / part.each);
    } else {
      tg = int64_t(part.item) * a.num_kv_heads + g;
      slot0 = tg * a.splits, slot1 = slot0 + 1;
      mine_at = part.split, last_at = (all_steps + per_split - 1) / per_split - 1;
    }
    const float* st0 = a.state + slot0 * kSlot;
    const int64_t next = (slot1 - slot0) * kSlot;
    float* mine_st = a.state + slot0 * kSlot + mine_at * next;
    if (busy) {
#pragma unroll
      for (int cb = 0; cb < NC; ++cb)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          put_state(mine_st + ((cb * 8 + i) * 256 + tid) * 2, acc[cb][2 * i], acc[cb][2 * i + 1]);
    }  // (16 new tokens behind 32768, 64 rows of 128: 114 us with the states of all, 94 so)
    put_state(mine_st + (NC * 8 * 256 + tid) * 2, m_run, l);
    if (!last_to_arrive(arrival_counter(a.arrivals, tg), last_at - first_at + 1, s_last)) return;
    if (!busy) return;
    // Joined in order, so that the result does not depend on the order
    // of arrival: first the maximum, then the weighted sums.
    constexpr int U = 8;  // parts whose m and l are under way together
    auto get_ml = [&](int s) {
      return get_state2(st0 + min(s, last_at) * next + (NC * 8 * 256 + tid) * 2);
    };
    m_run = kLowest;
    for (int s0 = first_at; s0 <= last_at; s0 += U) {
      float2 ml[U];
#pragma unroll
      for (int u = 0; u < U; ++u) ml[u] = get_ml(s0 + u);
#pragma unroll
      for (int u = 0; u < U; ++u)
        m_run = fmaxf(m_run, ml[u].x);
    }
    l = 0.f;
#pragma unroll
    for (int cb = 0; cb < NC; ++cb)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[cb][i] = 0.f;
    for (int s = first_at; s <= last_at; ++s) {
      const float* st = st0 + s * next;
      const float2 ml = get_ml(s);
      // All of a state on its way at once: one load after the other took 7 us a state.
      float2 o[NC][8];
#pragma unroll
      for (int cb = 0; cb < NC; ++cb)
#pragma unroll
        for (int i = 0; i < 8; ++i) o[cb][i] = get_state2(st + ((cb * 8 + i) * 256 + tid) * 2);
#pragma unroll
      for (int cb = 0; cb < NC; ++cb)
        asm volatile("" : "+v"(o[cb][0].x), "+v"(o[cb][1].x), "+v"(o[cb][2].x), "+v"(o[cb][3].x),
                          "+v"(o[cb][4].x), "+v"(o[cb][5].x), "+v"(o[cb][6].x), "+v"(o[cb][7].x));
      const float w = fast_exp2(ml.x - m_run);
      l = fmaf(w, ml.y, l);
#pragma unroll
      for (int cb = 0; cb < NC; ++cb)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          acc[cb][2 * i] = fmaf(w, o[cb][i].x, acc[cb][2 * i]);
          acc[cb][2 * i + 1] = fmaf(w, o[cb][i].y, acc[cb][2 * i + 1]);
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

template <int D, bool BF16, Cache F, bool CROSS>
__global__ __launch_bounds__(256, 2) void prompt_kernel(PromptArgs a, int tiles, int slots) {
  // Objects of their own, named at compile time where they are used: the
  // compiler then knows which loads to LDS a read has to wait for.
  __shared__ uint4 kt0[kKeys][D / 8], kt1[kKeys][D / 8], vt0[kKeys][D / 8], vt1[kKeys][D / 8];
  __shared__ bool s_last;
  const int g = blockIdx.x % a.num_kv_heads;
  const int ts = blockIdx.x / a.num_kv_heads;
  const TileRun found = find_tile<CROSS>(a, ts, tiles, slots);
  if (found.tile < 0) return;
  SplitPart part{ts / found.splits, 0, found.splits, found.steps};
  part.split = ts - part.item * found.splits;
  prompt_tile<D, BF16, F, CROSS>(a, g, found.run, found.tile, part, kt0, kt1, vt0, vt1, &s_last);
}

// The same in even shares: workgroup i of a KV head takes [i each, (i + 1) each) of the
// line of its tiles (serving/shares.h).
template <int D, bool BF16, Cache F, bool CROSS>
__global__ __launch_bounds__(256, 2) void prompt_shares_kernel(PromptArgs a, int slots) {
  __shared__ uint4 kt0[kKeys][D / 8], kt1[kKeys][D / 8], vt0[kKeys][D / 8], vt1[kKeys][D / 8];
  __shared__ bool s_last;
  __shared__ LinePart s_part[4];
  const int g = blockIdx.x % a.num_kv_heads;
  const int share = blockIdx.x / a.num_kv_heads;
  LinePart& part = s_part[threadIdx.x >> 6];
  Shares shares;
  int64_t at;
  SharePart p = find_part<CROSS>(a, share, slots, at, shares);
  if (p.cost == 0) return;
  part.each = shares.each;
  part.end = min(shares.total, at + shares.each);
  for (;;) {
    part.start = p.start, part.cost = p.cost, part.slot = p.slot;
    part.from = at - p.start;
    part.to = min(p.cost, part.end - p.start);
    prompt_tile<D, BF16, F, CROSS>(a, g, p.run, p.tile, part, kt0, kt1, vt0, vt1, &s_last);
    at = readlane64(part.start + part.to, 0);
    if (at >= readlane64(part.end, 0)) return;
    p = find_part<CROSS>(a, -1, slots, at, shares);
    if (p.cost == 0) return;
  }
}

// Workgroups a KV head that run at the same time: two a compute unit.
inline int prompt_slots(int cus, int num_kv_heads) { return 2 * cus / num_kv_heads; }

template <int D, bool BF16, Cache F, bool CROSS>
inline pkv_status launch_prompt_kernel(const PromptArgs& a, hipStream_t s) {
  const int64_t tiles = prompt_tiles(a);
  int slots = 0;
  if (a.splits > 1) {
    const int cus = current_compute_units();
    if (cus <= 0) return PKV_EHIP;
    slots = prompt_slots(cus, a.num_kv_heads);
  }
  hipLaunchKernelGGL((prompt_kernel<D, BF16, F, CROSS>),
                     dim3(static_cast<uint32_t>(tiles * a.num_kv_heads * a.splits)), dim3(256), 0,
                     s, a, static_cast<int>(tiles), slots);
  return hipGetLastError() == hipSuccess ? PKV_OK : PKV_EHIP;
}

// One workgroup a tile, or with more than one split in even shares.
template <int D, bool BF16, Cache F, bool CROSS>
inline pkv_status launch_prompt_shares(const PromptArgs& a, hipStream_t s) {
  if (a.splits == 1) return launch_prompt_kernel<D, BF16, F, CROSS>(a, s);
  const int cus = current_compute_units();
  if (cus <= 0) return PKV_EHIP;
  const int slots = std::max(prompt_slots(cus, a.num_kv_heads), 1);
  // Whole tiles: a workgroup each.
  const int64_t n = std::max<int64_t>(std::min(a.splits, slots), prompt_tiles(a));
  hipLaunchKernelGGL((prompt_shares_kernel<D, BF16, F, CROSS>),
                     dim3(static_cast<uint32_t>(n * a.num_kv_heads)), dim3(256), 0, s, a, slots);
  return hipGetLastError() == hipSuccess ? PKV_OK : PKV_EHIP;
}

}  // namespace pkv
