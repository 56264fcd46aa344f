// Finding a workgroup's row in a batch of ragged runs, on the device.
#pragma once

#include "context_internal.h"
#include "mfma.h"
#include "wave.h"

namespace pkv {

// One row's run of new tokens.
struct Run {
  int row;
  int first;  // its first row in the token-major arrays
  int count;
  int len;    // the row's length after the run (0 when invalid)
};

__device__ __forceinline__ int clamp_offset(int off, int num_tokens) {
  return min(max(off, 0), num_tokens);
}

__device__ __forceinline__ Run make_run(int row, int first, int next, int len, int max_pages) {
  Run r;
  r.row = row;
  r.first = __builtin_amdgcn_readfirstlane(first);
  r.count = max(__builtin_amdgcn_readfirstlane(next) - r.first, 0);
  r.len = clean_len(__builtin_amdgcn_readfirstlane(len), max_pages);
  return r;
}

// The run of work item `item`: that of the last row i with base(off_i, i) <=
// item, where base grows with i.  Every wave finds it by itself, 64 rows at a
// time; offsets and lengths of the first 64 come with one round of loads.
template <typename Args, typename Base>
__device__ __forceinline__ Run find_run(const Args& a, int64_t item, Base base) {
  const int lane = threadIdx.x & 63;
  int below = 0, off = 0, len = 0, r0 = 0;
  for (;; r0 += 64) {
    const int r = r0 + lane;
    off = r <= a.batch ? clamp_offset(a.tok_offsets[r], a.num_tokens) : a.num_tokens;
    len = r < a.batch ? a.seq_lens[r] : 0;
    const bool in = r < a.batch && base(off, r) <= item;
    const int k = __popcll(__builtin_amdgcn_ballot_w64(in));
    below += k;
    if (k < 64 || r0 + 64 >= a.batch) break;
  }
  const int row = max(__builtin_amdgcn_readfirstlane(below) - 1, 0);
  const int at = row - r0;  // 0 .. 62: the row and its successor are in hand
  if (at >= 0 && at < 63)
    return make_run(row, __builtin_amdgcn_readlane(off, at), __builtin_amdgcn_readlane(off, at + 1),
                    __builtin_amdgcn_readlane(len, at), a.max_pages);
  return make_run(row, clamp_offset(a.tok_offsets[row], a.num_tokens),
                  clamp_offset(a.tok_offsets[row + 1], a.num_tokens), a.seq_lens[row],
                  a.max_pages);
}

// The one new token of a row, without offsets.
template <typename Args>
__device__ __forceinline__ Run single_run(const Args& a, int row) {
  return make_run(row, row, row + 1, a.seq_lens[row], a.max_pages);
}

// Query tiles of a prompt: row after row, the late tiles of a row first.
// Counted from the offsets, not from the bound that sizes the grid: launched
// workgroups without a tile then all lie behind the others, which come out even
// on the compute units.
struct TileRun {
  Run run;
  int tile;    // of the run; negative: none
  int splits;  // ranges that a tile's keys are cut into, at most,
  int steps;   // each of this many steps at least
};

// The share of workgroup `ts` of one KV head.  With max_splits > 1 the tiles are
// counted first, so that tiles times ranges fill `slots` workgroups a KV head
// and no more, and no more ranges than the longest row's steps are worth; a shorter
// tile's ranges are as long as the longest one's.
template <typename Args>
__device__ __forceinline__ TileRun find_tile(const Args& a, int ts, int tiles, int slots) {
  const int lane = threadIdx.x & 63;
  TileRun t;
  t.tile = -1;
  t.splits = a.splits;
  t.steps = a.splits > 1 ? kRangeSteps : 0;
  if (!a.tok_offsets) {
    if (a.splits > 1) t.splits = min(a.splits, max(slots / a.batch, 1));
    const int row = ts / t.splits;
    if (row < a.batch) {
      t.run = single_run(a, row);
      t.tile = 0;
    }
    return t;
  }
  int first, next, len, count;
  auto load = [&](int r0) {  // 64 rows from r0 on; count: tiles up to and with a lane's row
    const int r = r0 + lane;
    first = a.tok_offsets[min(r, a.batch)];
    next = a.tok_offsets[min(r + 1, a.batch)];
    len = a.seq_lens[min(r, a.batch - 1)];
    asm volatile("" : "+v"(first), "+v"(next), "+v"(len));  // one wait for the three
    first = clamp_offset(first, a.num_tokens), next = clamp_offset(next, a.num_tokens);
    const int64_t rows = int64_t(max(next - first, 0)) * a.group;
    count = wave_scan(r < a.batch ? static_cast<int>((rows + kTileRows - 1) / kTileRows) : 0);
  };
  load(0);
  if (a.splits > 1) {
    int total = __builtin_amdgcn_readlane(count, 63);
    int longest = next > first ? clean_len(len, a.max_pages) : 0;  // of rows with new tokens
    if (a.batch > 64) {
      for (int r0 = 64; r0 < a.batch; r0 += 64) {
        load(r0);
        total += __builtin_amdgcn_readlane(count, 63);
        if (next > first) longest = max(longest, clean_len(len, a.max_pages));
      }
      load(0);
    }
    longest = wave_max(longest);
    const int steps = min((longest >> 6) + ((longest & 63) ? 1 : 0), (a.tile_pages + 3) >> 2);
    t.splits = min(min(a.splits, prompt_ranges(steps)), max(slots / max(total, 1), 1));
    t.steps = (steps + t.splits - 1) / t.splits;
  }
  const int item = ts / t.splits;
  if (item >= tiles) return t;
  for (int r0 = 0, before = 0;;) {
    const int in_all = __builtin_amdgcn_readlane(count, 63);
    if (item < before + in_all) {
      const uint64_t past = __builtin_amdgcn_ballot_w64(before + count > item);
      const int at = __builtin_amdgcn_readfirstlane(__builtin_ctzll(past));
      t.run = make_run(r0 + at, __builtin_amdgcn_readlane(first, at),
                       __builtin_amdgcn_readlane(next, at), __builtin_amdgcn_readlane(len, at),
                       a.max_pages);
      t.tile = before + __builtin_amdgcn_readlane(count, at) - 1 - item;
      return t;
    }
    before += in_all;
    r0 += 64;
    if (r0 >= a.batch) return t;
    load(r0);
  }
}

// A page's share of a run: tokens [begin, end) of block-table entry `entry`
// (begin >= end: none), as positions.
struct Segment {
  Run run;
  int entry;
  int begin;
  int end;
};

template <typename Args>
__device__ __forceinline__ Segment find_segment(const Args& a, int item) {
  Segment s;
  int k = 0;
  if (a.tok_offsets) {
    s.run = find_run(a, item, [](int64_t off, int64_t r) { return segment_base(off, r); });
    k = item - static_cast<int>(segment_base(s.run.first, s.run.row));
  } else {
    s.run = single_run(a, item);
  }
  const int p0 = max(s.run.len - s.run.count, 0);  // negative positions are not in the cache
  s.entry = (p0 >> 4) + k;
  s.begin = max(p0, s.entry * 16);
  s.end = min(s.run.len, s.entry * 16 + 16);
  if (k < 0) s.end = s.begin;
  return s;
}

}  // namespace pkv
