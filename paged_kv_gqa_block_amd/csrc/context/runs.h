// Finding a workgroup's row in a batch of ragged runs, on the device.
#pragma once

#include "context_internal.h"
#include "mfma.h"

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

// The last row i with base(off_i, i) <= item, where base grows with i: every
// wave counts the rows below by itself, 64 at a time.
template <typename Base>
__device__ __forceinline__ int find_row(const int32_t* tok_offsets, int batch, int num_tokens,
                                        int64_t item, Base base) {
  const int lane = threadIdx.x & 63;
  int below = 0;
  for (int r0 = 0; r0 < batch; r0 += 64) {
    const int r = r0 + lane;
    const bool in = r < batch && base(clamp_offset(tok_offsets[r], num_tokens), r) <= item;
    const int k = __popcll(__builtin_amdgcn_ballot_w64(in));
    below += k;
    if (k < 64) break;
  }
  return max(__builtin_amdgcn_readfirstlane(below) - 1, 0);
}

__device__ __forceinline__ Run run_of(const int32_t* tok_offsets, const int32_t* seq_lens, int row,
                                      int num_tokens, int max_pages) {
  Run r;
  r.row = row;
  if (tok_offsets) {
    r.first = clamp_offset(tok_offsets[row], num_tokens);
    r.count = max(clamp_offset(tok_offsets[row + 1], num_tokens) - r.first, 0);
  } else {
    r.first = row;
    r.count = 1;
  }
  r.len = clean_len(seq_lens[row], max_pages);
  r.first = __builtin_amdgcn_readfirstlane(r.first);
  r.count = __builtin_amdgcn_readfirstlane(r.count);
  r.len = __builtin_amdgcn_readfirstlane(r.len);
  return r;
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
    const int row = find_row(a.tok_offsets, a.batch, a.num_tokens, item,
                             [](int64_t off, int64_t r) { return segment_base(off, r); });
    s.run = run_of(a.tok_offsets, a.seq_lens, row, a.num_tokens, a.max_pages);
    k = item - static_cast<int>(segment_base(s.run.first, row));
  } else {
    s.run = run_of(nullptr, a.seq_lens, item, a.num_tokens, a.max_pages);
  }
  const int p0 = max(s.run.len - s.run.count, 0);  // negative positions are not in the cache
  s.entry = (p0 >> 4) + k;
  s.begin = max(p0, s.entry * 16);
  s.end = min(s.run.len, s.entry * 16 + 16);
  if (k < 0) s.end = s.begin;
  return s;
}

}  // namespace pkv
