// Internal declarations of the serving operators (include/pkv_serving.h): kernel
// arguments and launchers.  Not part of the public ABI.
#pragma once

#include "context/context_internal.h"
#include "pkv_serving.h"

namespace pkv {

struct Store8Args : StoreArgs {  // k_pool: the 8-bit pool
  uint8_t* scales;               // [pages][Hkv][2]
};

struct Load8Args : LoadArgs {
  const uint8_t* scales;
};

// Words of the page state (include/pkv_serving.h).
constexpr int kStateFree = 0, kStateDenied = 1, kStateArrivals = 2;

struct TakeArgs {
  const int32_t* counts;
  int32_t* lens;
  int32_t* block_table;
  const int32_t* free_pages;
  int32_t* state;
  int32_t* seq_lens;
  int32_t* tok_offsets;
  int64_t* slots;      // may be null
  int32_t* positions;  // may be null
  int32_t batch;
  int32_t num_tokens;
  int32_t max_pages;
  int32_t num_pool_pages;
};

struct ReleaseArgs {
  const int32_t* keep;
  int32_t* lens;
  int32_t* block_table;
  int32_t* free_pages;
  int32_t* state;
  int32_t batch;
  int32_t max_pages;
  int32_t num_pool_pages;
};

// Queries of a row up to which cross attention takes tiles of sixteen.
constexpr int kFewQueries = 32;

// Tiles of sixteen queries: a bound that needs only the token count.
inline int64_t cross_tiles(const pkv_problem& p, int32_t num_tokens, bool one_per_row) {
  return one_per_row ? p.batch
                     : cross_tile_base(num_tokens, p.batch, p.num_q_heads / p.num_kv_heads);
}

// Whether a cross-attention call takes tiles of sixteen queries (attend_kernel.h)
// rather than of 128 (prompt_kernel.h): by the average of its rows' packed queries.
inline bool cross_takes_few(const pkv_problem& p, int32_t num_tokens, bool one_per_row) {
  const int64_t rows = int64_t(num_tokens) * (p.num_q_heads / p.num_kv_heads);
  return rows <= int64_t(kFewQueries) * p.batch && cross_tiles(p, num_tokens, one_per_row) <= 65535;
}

pkv_status launch_attend8(const pkv_problem& p, const AttendArgs& a, hipStream_t s);
pkv_status launch_prompt8(const pkv_problem& p, const PromptArgs& a, hipStream_t s);
pkv_status launch_cross_few(const pkv_problem& p, Cache kind, int64_t tiles, const AttendArgs& a,
                            hipStream_t s);
pkv_status launch_cross_many(const pkv_problem& p, Cache kind, const PromptArgs& a, hipStream_t s);
pkv_status launch_store8(const pkv_problem& p, const Store8Args& a, hipStream_t s);
pkv_status launch_load8(const pkv_problem& p, const Load8Args& a, hipStream_t s);
pkv_status launch_take(const TakeArgs& a, hipStream_t s);
pkv_status launch_release(const ReleaseArgs& a, hipStream_t s);

}  // namespace pkv
