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

// Tiles of sixteen queries: a bound that needs only the token count.
inline int64_t cross_tiles(const pkv_problem& p, int32_t num_tokens, bool one_per_row) {
  return one_per_row ? p.batch
                     : cross_tile_base(num_tokens, p.batch, p.num_q_heads / p.num_kv_heads);
}

// Whether a cross-attention call takes tiles of sixteen queries (attend_kernel.h)
// rather than of 128 (prompt_kernel.h): up to 32 packed queries a row on the average, 64
// where few pairs of row and KV head leave room for more tiles.
//  us, tiles of sixteen / of 128, d = 128, 16 bits: 16 rows x 8 KV heads of 3000-4000
//  states, 16 queries each 43 / 64, 32 62 / 64, 48 88 / 65 (8 bits: 35 / 57 at 32, 49 / 57
//  at 48); 8 rows, 32 queries 31 / 52, 64 49 / 52, 96 73 / 53; one row of 20000, 64 queries
//  53 / 59, 96 73 / 59.  64 rows of 500-8000 in 8 bits: 16 queries 110 / 185, 32 192 / 185.
inline bool cross_takes_few(const pkv_problem& p, int32_t num_tokens, bool one_per_row) {
  const int64_t rows = int64_t(num_tokens) * (p.num_q_heads / p.num_kv_heads);
  const int64_t few = int64_t(p.batch) * p.num_kv_heads <= 64 ? 64 : 32;
  return rows <= few * p.batch && cross_tiles(p, num_tokens, one_per_row) <= 65535;
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
