// Host side of the attention calls over a paged cache: argument checks, workspace
// sizes and kernel arguments, shared by the entry points of every kind of cache.
#pragma once

#include <algorithm>
#include <cmath>
#include <limits>

#include "context/context_internal.h"
#include "launch_limits.h"
#include "pkv_internal.h"

namespace pkv {

constexpr float kLog2e = 1.4426950408889634f;

inline bool aligned(const void* p, uintptr_t to) {
  return reinterpret_cast<uintptr_t>(p) % to == 0;
}

// The cache of a call: two 16-bit pools, the 4-bit pool, or the 8-bit pool and its
// scales.
struct Pools {
  Cache kind;
  const void* k;
  const void* v;       // 16 bits alone
  const void* scales;  // 8 bits alone
  bool given() const {
    return k && (kind != Cache::k16 || v) && (kind != Cache::k8 || scales);
  }
  bool placed() const { return aligned(k, 16) && aligned(v, 16) && aligned(scales, 2); }
  template <typename Args>
  void fill(Args* a) const {
    a->k_pool = k;
    a->v_pool = v;
    a->scales = static_cast<const uint8_t*>(scales);
  }
};

inline pkv_status check_view(const pkv_view* view) {
  return view && (view->window < 0 || view->sinks < 0) ? PKV_EINVAL : PKV_OK;
}

// The window the kernels get: 0 where it covers every position of the table,
// so that positions minus the window stay in 32 bits.
inline int32_t clean_window(const pkv_problem* p, const pkv_view* view) {
  if (!view) return 0;
  return view->window >= int64_t(p->max_pages_per_row) * p->page_size ? 0 : view->window;
}

// The kernels take maxima of unscaled scores, so their scale is positive: the
// sign of a negative one moves to the queries, and zero becomes the smallest
// number there is, which takes every finite score to 5e-7 or less: a weight of 1
// within fp32.  (The smallest normal number took scores of 2^125 to 1/2.)
template <typename Args>
void set_scale(const pkv_problem* p, Args* a) {
  const float x = p->sm_scale * kLog2e;
  a->q_flip = x < 0.f ? 0x80008000u : 0u;
  a->scale_log2 = std::max(std::fabs(x), std::numeric_limits<float>::denorm_min());
}

// Largest number of pages that one query of this problem sees.
inline int64_t most_pages(const pkv_problem* p, const pkv_view* view) {
  const int64_t all = p->max_pages_per_row;
  const int32_t w = clean_window(p, view);
  if (w == 0) return all;
  return std::min(all, ceil_div(w, 16) + 1 + ceil_div(view->sinks, 16));
}

inline int64_t attend_slots(const pkv_problem* p, int32_t splits) {
  return int64_t(p->batch) * p->num_kv_heads * splits;
}

// Workspace of both attention calls: the arrival counters, at one place for every
// problem, so that calls of any sizes find them as zero as the last one left
// them; then the states (decode: (m, l) of every slot, then o).
constexpr int64_t kCounters = 65536;
constexpr size_t kCounterBytes = kCounters * sizeof(int32_t);

struct Workspace {
  size_t ml, o, bytes;
};

inline Workspace workspace_of(const pkv_problem* p, int32_t splits) {
  const auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
  const size_t slots = static_cast<size_t>(attend_slots(p, splits));
  const size_t g = static_cast<size_t>(p->num_q_heads / p->num_kv_heads);
  Workspace w;
  w.ml = kCounterBytes;
  w.o = w.ml + up(slots * g * 2 * sizeof(float));
  w.bytes = w.o + slots * g * p->head_dim * sizeof(float);
  return w;
}

inline pkv_status check_run(const pkv_problem* prob, const int32_t* tok_offsets, int32_t num_tokens,
                     const int32_t* seq_lens, const int32_t* block_table) {
  const pkv_status st = check_problem(prob);
  if (st != PKV_OK) return st;
  if (num_tokens < 0 || (!tok_offsets && num_tokens != prob->batch)) return PKV_EINVAL;
  if (!seq_lens || !block_table) return PKV_EINVAL;
  return PKV_OK;
}

// Rows are the third grid dimension of the launch; pairs in splits take a counter.
inline pkv_status check_attend_size(const pkv_problem* p, int32_t splits) {
  if (p->batch > 65535 || p->num_q_heads > 65535 || attend_slots(p, splits) > kMaxGridGroups ||
      (splits > 1 && int64_t(p->batch) * p->num_kv_heads > kCounters))
    return PKV_ERANGE;
  return PKV_OK;
}

// Checks of a decode call and its kernel arguments.
inline pkv_status fill_attend(const pkv_problem* prob, const pkv_view* view,
                              const int32_t* seq_lens, int32_t max_splits, const void* q,
                              Pools pools, const int32_t* block_table, void* workspace,
                              size_t workspace_bytes, void* out, float* lse, AttendArgs* args) {
  pkv_status st = check_problem(prob);
  if (st != PKV_OK) return st;
  st = check_view(view);
  if (st != PKV_OK) return st;
  if (max_splits < 1 || max_splits > 65535) return PKV_EINVAL;
  if (!seq_lens || !q || !pools.given() || !block_table || !workspace || !out) return PKV_EINVAL;
  if (!aligned(q, 16) || !pools.placed() || !aligned(out, 16) || !aligned(workspace, 16))
    return PKV_ESHAPE;
  st = check_attend_size(prob, max_splits);
  if (st != PKV_OK) return st;
  const Workspace w = workspace_of(prob, max_splits);
  if (workspace_bytes < w.bytes) return PKV_ENOSPC;
  char* ws = static_cast<char*>(workspace);
  AttendArgs& a = *args;
  a = AttendArgs{};
  a.q = q;
  pools.fill(&a);
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.arrivals = reinterpret_cast<int32_t*>(ws);
  a.st_ml = reinterpret_cast<float*>(ws + w.ml);
  a.st_o = reinterpret_cast<float*>(ws + w.o);
  a.out = out;
  a.lse = lse;
  a.batch = prob->batch;
  a.num_q_heads = prob->num_q_heads;
  a.num_kv_heads = prob->num_kv_heads;
  a.group = prob->num_q_heads / prob->num_kv_heads;
  a.max_pages = prob->max_pages_per_row;
  a.num_pool_pages = prob->num_pool_pages;
  a.splits = max_splits;
  a.window = clean_window(prob, view);
  a.sinks = view ? view->sinks : 0;
  set_scale(prob, &a);
  return PKV_OK;
}

// How the tiles of a prompt are divided: each into up to max_splits ranges, or all of a KV
// head's into max_splits even shares (serving/shares.h).
enum class Divide { kRanges, kShares };

// Launch size of a prompt, and its counters where it is split.
inline bool prompt_fits(const pkv_problem* p, int64_t tiles, int32_t splits, Divide by) {
  const int64_t pairs = tiles * p->num_kv_heads;
  const int64_t parts = by == Divide::kShares ? (tiles + splits - 1) * p->num_kv_heads
                                              : pairs * splits;
  return parts <= kMaxGridGroups && (splits == 1 || pairs <= kCounters);
}

// Shares: a part of a tile has the state tile + share, and no two of them the same.
inline size_t prompt_workspace_of(const pkv_problem* p, int64_t tiles, int32_t splits, Divide by) {
  const int64_t states = by == Divide::kShares ? tiles + splits - 1 : tiles * splits;
  return kCounterBytes + static_cast<size_t>(states) * p->num_kv_heads *
                             prompt_state_floats(p->head_dim) * sizeof(float);
}

// Checks of a prompt call and its kernel arguments; no tokens: num_tokens stays 0, and
// there is nothing to launch.
inline pkv_status fill_prompt(const pkv_problem* prob, const pkv_view* view,
                              const int32_t* tok_offsets, int32_t num_tokens,
                              const int32_t* seq_lens, int32_t max_splits, const void* q,
                              Pools pools, const int32_t* block_table, void* workspace,
                              size_t workspace_bytes, void* out, float* lse, Divide by,
                              PromptArgs* args) {
  PromptArgs& a = *args;
  a = PromptArgs{};
  pkv_status st = check_run(prob, tok_offsets, num_tokens, seq_lens, block_table);
  if (st != PKV_OK) return st;
  st = check_view(view);
  if (st != PKV_OK) return st;
  if (max_splits < 1 || max_splits > 65535) return PKV_EINVAL;
  if (num_tokens == 0) return PKV_OK;
  if (!q || !pools.given() || !out || (max_splits > 1 && !workspace)) return PKV_EINVAL;
  if (!aligned(q, 16) || !pools.placed() || !aligned(out, 16) || !aligned(workspace, 16))
    return PKV_ESHAPE;
  a.q = q;
  pools.fill(&a);
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.tok_offsets = tok_offsets;
  a.out = out;
  a.lse = lse;
  a.batch = prob->batch;
  a.num_tokens = num_tokens;
  a.num_q_heads = prob->num_q_heads;
  a.num_kv_heads = prob->num_kv_heads;
  a.group = prob->num_q_heads / prob->num_kv_heads;
  a.group_inv = static_cast<uint32_t>(ceil_div(4096, a.group));
  a.max_pages = prob->max_pages_per_row;
  a.num_pool_pages = prob->num_pool_pages;
  a.window = clean_window(prob, view);
  a.sinks = view ? view->sinks : 0;
  set_scale(prob, &a);
  a.splits = max_splits;
  // Its first token's view, and a page more for every 16 tokens behind that.
  a.tile_pages = static_cast<int32_t>(
      std::min<int64_t>(most_pages(prob, view) + kTileRows / a.group / 16 + 2, a.max_pages));
  const int64_t tiles = prompt_tiles(a);
  if (!prompt_fits(prob, tiles, max_splits, by)) return PKV_ERANGE;
  if (max_splits > 1) {
    if (workspace_bytes < prompt_workspace_of(prob, tiles, max_splits, by)) return PKV_ENOSPC;
    a.arrivals = static_cast<int32_t*>(workspace);
    a.state = reinterpret_cast<float*>(static_cast<char*>(workspace) + kCounterBytes);
  }
  return PKV_OK;
}

// pkv_prompt_workspace_bytes and its like.
inline size_t prompt_bytes(const pkv_problem* p, int64_t tiles, int32_t max_splits, Divide by) {
  if (tiles < 0 || max_splits < 2 || max_splits > 65535 || !prompt_fits(p, tiles, max_splits, by))
    return 0;
  return prompt_workspace_of(p, tiles, max_splits, by);
}

// Query tiles of a run batch, from the host's numbers alone; -1 when invalid.
inline int64_t tiles_of(const pkv_problem* p, int32_t num_tokens, int32_t one_per_row) {
  if (check_problem(p) != PKV_OK || num_tokens < 0 || (one_per_row && num_tokens != p->batch))
    return -1;
  return one_per_row ? p->batch
                     : tile_base(num_tokens, p->batch, p->num_q_heads / p->num_kv_heads);
}

}  // namespace pkv
