// Work of prompt and cross-attention tiles in even shares, on the device.
//
// The tiles of a KV head lie one behind the other on a line, each as long as it is
// expensive: units of pages times heads of a group that its last query sees, and what
// starting a tile costs.  Each of S workgroups takes one S-th of the line, whatever
// tiles that cuts; the last workgroup of a cut tile to finish joins its states.  So few
// tiles, or tiles of uneven lengths, keep every compute unit busy to the end.
#pragma once

#include "context/context_internal.h"
#include "context/mfma.h"
#include "context/runs.h"
#include "context/wave.h"

namespace pkv {

// A tile, or the part of it that a share covers.
struct SharePart {
  Run run;
  int tile;       // of the run
  int64_t slot;   // its number: below tile_base(num_tokens, batch, group), or batch
  int64_t start;  // where the tile begins on the line
  int64_t cost;   // its length there
};

struct Shares {
  int64_t total;  // length of the line
  int64_t each;   // of a share
  int even;       // length of every tile; 0: by what it costs
};

__device__ __forceinline__ int64_t moved_sum(int64_t x, int64_t y_lo, int64_t y_hi) {
  return x + static_cast<int64_t>((static_cast<uint64_t>(static_cast<uint32_t>(y_hi)) << 32) |
                                  static_cast<uint32_t>(y_lo));
}

// Inclusive sum over the wave.
__device__ __forceinline__ int64_t wave_scan64(int64_t x) {
#define PKV_ADD_MOVED(CTRL, ROWS)                                             \
  x = moved_sum(x, moved<CTRL, ROWS>(static_cast<int>(x)), moved<CTRL, ROWS>( \
                                                               static_cast<int>(x >> 32)))
  PKV_ADD_MOVED(kDppRowShr + 1, 0xf);
  PKV_ADD_MOVED(kDppRowShr + 2, 0xf);
  PKV_ADD_MOVED(kDppRowShr + 4, 0xf);
  PKV_ADD_MOVED(kDppRowShr + 8, 0xf);
  PKV_ADD_MOVED(kDppRowBcast15, 0xa);
  PKV_ADD_MOVED(kDppRowBcast31, 0xc);
#undef PKV_ADD_MOVED
  return x;
}

__device__ __forceinline__ int64_t readlane64(int64_t x, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(x), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(x >> 32), lane);
  return static_cast<int64_t>((static_cast<uint64_t>(hi) << 32) | lo);
}

// Costs of a row's tiles: first, first + 8, ... (128 / 16 pages times heads a tile), most
// at the highest.
struct TileCosts {
  int64_t first, most;
  // Of tiles 0 .. k - 1.
  __device__ __forceinline__ int64_t before(int64_t k) const {
    const int64_t n = min((most - first + 7) >> 3, k);  // those below `most`
    return first * n + 4 * n * (n - 1) + most * (k - n);
  }
};

// What joining adds to a workgroup's steps, in steps.  (Twelve shapes, 0, 16 and 1000 for
// the second: eight rows of 4096 tokens and 100 new ones, 33 tiles for 64 workgroups, 105, 86
// and 87 us; rows of 3000 to 31000, 36 new ones each, 266, 268 and 477.)
constexpr float kEvenJoin = 8.f, kShareJoin = 16.f;

// The part of the line at `at`; or, with `share` >= 0, the line is measured, for a.splits
// shares at most of `slots` that run at once, and `at` is where that share begins.
// cost == 0: behind its end.
//  * A tile's start costs as much as four steps: loads that nothing hides.
//  * A share keeps 8 steps, or the root of the longest tile's: a join reads 65 KiB a part,
//    as much time as a step, and a tile in p parts takes steps / p + p of them.
//  * Tiles of like cost stay whole or are cut into the same number of parts, a workgroup
//    each: cut anywhere, more of them are joined.  Whole ones are launched as they come,
//    the late tiles of a row first.
template <bool CROSS>
__device__ __forceinline__ SharePart find_part(const PromptArgs& a, int share, int slots,
                                               int64_t& at, Shares& shares) {
  const int lane = threadIdx.x & 63;
  const int G = a.group;
  const bool measure = share >= 0;
  if (measure) shares.even = 0;
  int first, count, len, tiles;
  TileCosts costs;
  auto load = [&](int r0) {
    const int r = r0 + lane;
    int next = r + 1;
    first = r;
    len = a.seq_lens[min(r, a.batch - 1)];
    if (a.tok_offsets) {
      first = a.tok_offsets[min(r, a.batch)];
      next = a.tok_offsets[min(r + 1, a.batch)];
      asm volatile("" : "+v"(first), "+v"(next), "+v"(len));  // one wait for the three
      first = clamp_offset(first, a.num_tokens), next = clamp_offset(next, a.num_tokens);
    }
    count = r < a.batch ? max(next - first, 0) : 0;
    len = clean_len(len, a.max_pages);
    tiles = static_cast<int>((int64_t(count) * G + kTileRows - 1) / kTileRows);
    const int64_t all = (int64_t(len) * G >> 4) + 1;
    costs.first = costs.most = all;
    if constexpr (!CROSS) {
      costs.first = min((max((int64_t(len) - count) * G + kTileRows, int64_t(0)) >> 4) + 1, all);
      if (a.window > 0)
        costs.most = min(all, ((int64_t(a.window) + a.sinks + 64) * G + kTileRows) >> 4);
      costs.first = min(costs.first, costs.most);
    }
    costs.first += 16 * G;
    costs.most += 16 * G;
    if (shares.even > 0) costs.first = costs.most = shares.even;
  };
  load(0);
  if (measure) {
    int64_t total = costs.before(tiles);
    int64_t most = tiles > 0 ? costs.most : 0;
    int all_tiles = tiles;
    if (a.batch > 64) {
      for (int r0 = 64; r0 < a.batch; r0 += 64) {
        load(r0);
        total += costs.before(tiles);
        all_tiles += tiles;
        if (tiles > 0) most = max(most, costs.most);
      }
      load(0);
    }
    total = readlane64(wave_scan64(total), 63);
    all_tiles = __builtin_amdgcn_readlane(wave_scan(all_tiles), 63);
    const float unit = 4.f * static_cast<float>(G);  // of a step
    const int longest = wave_max(static_cast<int>(static_cast<float>(most) / unit));
    const int least = max(kRangeSteps, static_cast<int>(__builtin_sqrtf(longest)));
    const int n = min(a.splits, slots);
    shares.total = total;
    shares.each = max(static_cast<int64_t>(static_cast<double>(total) / n) + 1,
                      int64_t(least) * 4 * G);
    // Either way in steps, with what joining costs.
    const int parts = max(min(n / max(all_tiles, 1), longest / least), 1);
    const float average = static_cast<float>(total) / unit / static_cast<float>(max(all_tiles, 1));
    const float rounds = __builtin_ceilf(static_cast<float>(all_tiles) / static_cast<float>(n));
    const float even = parts > 1
                           ? static_cast<float>(longest) / static_cast<float>(parts) + kEvenJoin
                           : fmaxf(static_cast<float>(longest), average * rounds);
    if (__builtin_amdgcn_readfirstlane(
            even <= static_cast<float>(shares.each) / unit + kShareJoin)) {
      shares.even = __builtin_amdgcn_readfirstlane(parts);
      shares.total = int64_t(all_tiles) * shares.even;
      shares.each = 1;
      costs.first = costs.most = shares.even;
    }
    at = share * shares.each;
  }
  SharePart p{};
  if (at >= shares.total) return p;
  int64_t base = 0;  // the line before the rows in hand
  for (int r0 = 0;;) {
    const int64_t mine = costs.before(tiles);
    const int64_t upto = base + wave_scan64(mine);
    const int64_t all = readlane64(upto, 63);
    if (at < all) {
      const uint64_t past = __builtin_amdgcn_ballot_w64(upto > at);
      const int in = __builtin_amdgcn_readfirstlane(__builtin_ctzll(past));
      p.run = make_run(r0 + in, __builtin_amdgcn_readlane(first, in),
                       __builtin_amdgcn_readlane(first + count, in),
                       __builtin_amdgcn_readlane(len, in), a.max_pages);
      const TileCosts c{readlane64(costs.first, in), readlane64(costs.most, in)};
      const int64_t row0 = readlane64(upto - mine, in);
      const int last = __builtin_amdgcn_readlane(tiles, in) - 1;
      // The last tile that starts at or before `at`.
      int lo = 0, hi = last;
      if (shares.even > 0) {
        lo = static_cast<int>(at - row0) / shares.even;
      } else {
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (row0 + c.before(mid) <= at) lo = mid;
          else hi = mid - 1;
        }
      }
      p.start = row0 + c.before(lo);
      p.cost = c.before(lo + 1) - c.before(lo);
      p.tile = shares.even > 0 ? last - lo : lo;
      // By the tile's place on the line: then slot plus share names one part alone.
      p.slot = a.tok_offsets ? tile_base(p.run.first, p.run.row, G) + lo : p.run.row;
      return p;
    }
    base = all;
    r0 += 64;
    if (r0 >= a.batch) return p;
    load(r0);
  }
}

}  // namespace pkv
