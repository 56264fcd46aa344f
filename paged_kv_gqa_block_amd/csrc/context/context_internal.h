// Internal declarations of the context operators (include/pkv_context.h):
// kernel arguments, launchers and the view arithmetic that host and device
// share.  Not part of the public ABI.
#pragma once

#include <cstdint>

#include "pkv_context.h"

#if defined(__HIP__) || defined(__HIPCC__)
#define PKV_HD __host__ __device__ __forceinline__
#else
#define PKV_HD inline
#endif

namespace pkv {

// The pages of one row that some query of a run sees, in reading order: the
// sinks' pages, then the window's.  Page v of that list is block-table entry
// v < ahead ? v : v + skip.
struct SeenPages {
  int ahead;  // pages that hold sinks only
  int skip;   // pages between them and the window
  int count;
};

// Queries at positions first_q .. last_q (0 <= first_q <= last_q).
PKV_HD SeenPages seen_pages(int first_q, int last_q, int window, int sinks) {
  const int begin = (window > 0 && first_q >= window) ? (first_q - window + 1) >> 4 : 0;
  const int sink_pages = (sinks >> 4) + ((sinks & 15) ? 1 : 0);
  SeenPages s;
  s.ahead = sink_pages < begin ? sink_pages : begin;
  s.skip = begin - s.ahead;
  s.count = (last_q >> 4) + 1 - s.skip;
  return s;
}

// Whether the query at position p sees token t.
PKV_HD bool sees(int p, int t, int window, int sinks) {
  return t <= p && (window == 0 || t > p - window || t < sinks);
}

// Ranges that the longest row of a decode call, `pages` visible pages, is worth
// cutting into: `fill` of them fill the compute units once, `even` take them
// several times.
//  * Up to 40 pages stay whole: joining waits for stores, a counter and loads, 3
//    us.  One row, 8 heads, in one range and in as many as fill: 24 pages 6.0 and
//    7.5 us, 40 pages 7.8 and 7.7 (16 bits: 6.3 and 7.4, 8.4 and 7.6), 64 pages 10.3
//    and 7.9.
//  * One range for every compute unit, as long as a range keeps eight pages (one
//    unit for each wave); beyond that ranges of at least 96 pages, so that rows of
//    different lengths even out (the launch takes fewer where that comes out even).
//    Joining costs more than it gives where ranges are shorter: 512 pairs of 64 to
//    2048 pages took 237 us in up to 4, 222 in 6, 212 in 10 and 231 in 24 ranges each.
// The host asks for the pages of a table, the launch again for those that there are:
// under a table of 131072 tokens, with the table's ranges and with the rows' own,
// 8 rows of 2048 tokens (4 bits, 8 heads) took 40 and 12 us, 64 rows of 1024 52 and 21.
PKV_HD int decode_ranges(int pages, int fill, int even) {
  const int own = pages <= 40 ? 1 : (fill < (pages + 7) / 8 ? fill : (pages + 7) / 8);
  const int more = even < pages / 96 ? even : pages / 96;
  return own > more ? own : (more > 1 ? more : 1);
}

// The same of a prompt's longest tile, `steps` of four visible pages: a range keeps
// kRangeSteps (16 new tokens behind 2048, 64 heads over 8, the same table: 54 us with
// the table's ranges, 23 with the rows').
constexpr int kRangeSteps = 8;
PKV_HD int prompt_ranges(int steps) {
  return steps >= 2 * kRangeSteps ? steps / kRangeSteps : 1;
}

struct AttendArgs {
  const void* q;        // [B][Hq][d]
  const void* k_pool;   // 16-bit pages, or the 4-bit pool (v_pool unused)
  const void* v_pool;
  const int32_t* block_table;
  const int32_t* seq_lens;
  int32_t cus;          // compute units of the device; set by the launcher, as the
  int32_t fill;         // next two, for decode_ranges
  int32_t even;
  float* st_ml;         // [slots][G][2]: running max (log2 units) and sum
  float* st_o;          // [slots][G][d]
  int32_t* arrivals;    // [B * Hkv], zero between calls
  void* out;
  float* lse;           // may be null
  int32_t batch;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t group;
  int32_t max_pages;
  int32_t num_pool_pages;
  int32_t splits;
  int32_t window;       // 0: everything
  int32_t sinks;
  float scale_log2;     // |scale| log2(e), above zero (subnormal where need be)
  uint32_t q_flip;      // sign bits of a negative scale, moved to the queries
};

struct PromptArgs {
  const void* q;        // [num_tokens][Hq][d]
  const void* k_pool;
  const void* v_pool;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* tok_offsets;  // [B + 1]
  float* state;         // splits' states, see prompt.hip
  int32_t* arrivals;    // [tiles * Hkv], zero between calls
  void* out;
  float* lse;
  int32_t batch;
  int32_t num_tokens;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t group;
  uint32_t group_inv;   // ceil(4096 / group)
  int32_t max_pages;
  int32_t num_pool_pages;
  int32_t splits;
  int32_t tile_pages;   // that one tile sees at most
  int32_t window;
  int32_t sinks;
  float scale_log2;     // |scale| log2(e), above zero (subnormal where need be)
  uint32_t q_flip;      // sign bits of a negative scale, moved to the queries
};

struct StoreArgs {
  const void* k_new;    // token stride k_stride elements, heads contiguous
  const void* v_new;
  int64_t k_stride;
  int64_t v_stride;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* tok_offsets;  // null: one token per row
  void* k_pool;         // 16-bit pages, or the 4-bit pool (v_pool unused)
  void* v_pool;
  int32_t batch;
  int32_t num_tokens;
  int32_t num_kv_heads;
  int32_t max_pages;
  int32_t num_pool_pages;
};

struct LoadArgs {
  const void* pool;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* tok_offsets;
  void* k_out;          // [num_tokens][Hkv][d]
  void* v_out;
  int32_t batch;
  int32_t num_tokens;
  int32_t num_kv_heads;
  int32_t max_pages;
  int32_t num_pool_pages;
};

// Page segments of a run: a bound that needs only the token count.  Row i owns
// the segments [off_i / 16 + 2 i, off_{i+1} / 16 + 2 (i + 1)), at least the
// ceil(n_i / 16) + 1 pages its run can touch.
PKV_HD int64_t segment_base(int64_t off, int64_t row) { return (off >> 4) + 2 * row; }

// Workgroups of a store or load launch: every segment of every KV head.
template <typename Args>
inline int64_t run_groups(const Args& a) {
  return (a.tok_offsets ? segment_base(a.num_tokens, a.batch) : a.batch) * a.num_kv_heads;
}

// Query tiles of a prompt, by the same rule over packed rows (token, head of
// the group).
constexpr int kTileRows = 128;
PKV_HD int64_t tile_base(int64_t off, int64_t row, int group) {
  return off * group / kTileRows + row;
}
// Floats of one split's state of one tile and KV head (prompt.hip).
inline size_t prompt_state_floats(int head_dim) { return 256 * (size_t(head_dim) / 2 + 2); }
inline int64_t prompt_tiles(const PromptArgs& a) {
  return a.tok_offsets ? tile_base(a.num_tokens, a.batch, a.group) : int64_t(a.batch);
}

// `fill` and `even` of decode_ranges, for pairs of row and KV head.  Up to twenty
// ranges a compute unit; eight pairs a unit come out even whole: 1024 pairs of up to
// 1024 pages 235 us whole and 219 in 3 to 5 ranges, 2048 of up to 512 222 and 222, 4096
// of up to 256 213 and 253 in 2.
inline void ranges_of_device(int64_t pairs, int cus, int32_t* fill, int32_t* even) {
  *fill = static_cast<int32_t>((cus + pairs - 1) / pairs);
  *even = pairs >= 8 * int64_t(cus) ? 1 : static_cast<int32_t>(20 * int64_t(cus) / pairs);
}

// Compute units of the current device; 0 where the query fails.
int current_compute_units();

pkv_status launch_attend(const pkv_problem& p, bool kv4, const AttendArgs& a, hipStream_t s);
pkv_status launch_prompt(const pkv_problem& p, bool kv4, const PromptArgs& a, hipStream_t s);
pkv_status launch_store(const pkv_problem& p, bool kv4, const StoreArgs& a, hipStream_t s);
pkv_status launch_load(const pkv_problem& p, const LoadArgs& a, hipStream_t s);

}  // namespace pkv
