// Entry points of include/pkv_context.h: argument checks on the host, then
// launches on the caller's stream.
#include <algorithm>
#include <cmath>
#include <limits>

#include "context_internal.h"
#include "launch_limits.h"
#include "pkv_internal.h"

using namespace pkv;

namespace {

constexpr float kLog2e = 1.4426950408889634f;

bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

pkv_status check_view(const pkv_view* view) {
  return view && (view->window < 0 || view->sinks < 0) ? PKV_EINVAL : PKV_OK;
}

// The window the kernels get: 0 where it covers every position of the table,
// so that positions minus the window stay in 32 bits.
int32_t clean_window(const pkv_problem* p, const pkv_view* view) {
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
int64_t most_pages(const pkv_problem* p, const pkv_view* view) {
  const int64_t all = p->max_pages_per_row;
  const int32_t w = clean_window(p, view);
  if (w == 0) return all;
  return std::min(all, ceil_div(w, 16) + 1 + ceil_div(view->sinks, 16));
}

int64_t attend_slots(const pkv_problem* p, int32_t splits) {
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

Workspace workspace_of(const pkv_problem* p, int32_t splits) {
  const auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
  const size_t slots = static_cast<size_t>(attend_slots(p, splits));
  const size_t g = static_cast<size_t>(p->num_q_heads / p->num_kv_heads);
  Workspace w;
  w.ml = kCounterBytes;
  w.o = w.ml + up(slots * g * 2 * sizeof(float));
  w.bytes = w.o + slots * g * p->head_dim * sizeof(float);
  return w;
}

pkv_status check_run(const pkv_problem* prob, const int32_t* tok_offsets, int32_t num_tokens,
                     const int32_t* seq_lens, const int32_t* block_table) {
  const pkv_status st = check_problem(prob);
  if (st != PKV_OK) return st;
  if (num_tokens < 0 || (!tok_offsets && num_tokens != prob->batch)) return PKV_EINVAL;
  if (!seq_lens || !block_table) return PKV_EINVAL;
  return PKV_OK;
}

// Rows are the third grid dimension of the launch; pairs in splits take a counter.
pkv_status check_attend_size(const pkv_problem* p, int32_t splits) {
  if (p->batch > 65535 || p->num_q_heads > 65535 || attend_slots(p, splits) > kMaxGridGroups ||
      (splits > 1 && int64_t(p->batch) * p->num_kv_heads > kCounters))
    return PKV_ERANGE;
  return PKV_OK;
}

pkv_status attend(const pkv_problem* prob, const pkv_view* view, const int32_t* seq_lens,
                  int32_t max_splits, const void* q, bool kv4, const void* k_pool,
                  const void* v_pool, const int32_t* block_table, void* workspace,
                  size_t workspace_bytes, void* out, float* lse, hipStream_t stream) {
  pkv_status st = check_problem(prob);
  if (st != PKV_OK) return st;
  st = check_view(view);
  if (st != PKV_OK) return st;
  if (max_splits < 1 || max_splits > 65535) return PKV_EINVAL;
  if (!seq_lens || !q || !k_pool || (!kv4 && !v_pool) || !block_table || !workspace || !out)
    return PKV_EINVAL;
  if (!aligned(q, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(out, 16) ||
      !aligned(workspace, 16))
    return PKV_ESHAPE;
  st = check_attend_size(prob, max_splits);
  if (st != PKV_OK) return st;
  const Workspace w = workspace_of(prob, max_splits);
  if (workspace_bytes < w.bytes) return PKV_ENOSPC;
  char* ws = static_cast<char*>(workspace);
  AttendArgs a{};
  a.q = q;
  a.k_pool = k_pool;
  a.v_pool = v_pool;
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
  return launch_attend(*prob, kv4, a, stream);
}

// Launch size of a prompt, and its counters where it is split.
bool prompt_fits(const pkv_problem* p, int64_t tiles, int32_t splits) {
  const int64_t pairs = tiles * p->num_kv_heads;
  return pairs * splits <= kMaxGridGroups && (splits == 1 || pairs <= kCounters);
}

size_t prompt_workspace_of(const pkv_problem* p, int64_t tiles, int32_t splits) {
  return kCounterBytes + static_cast<size_t>(tiles) * p->num_kv_heads * splits *
                             prompt_state_floats(p->head_dim) * sizeof(float);
}

pkv_status prompt(const pkv_problem* prob, const pkv_view* view, const int32_t* tok_offsets,
                  int32_t num_tokens, const int32_t* seq_lens, int32_t max_splits, const void* q,
                  bool kv4, const void* k_pool, const void* v_pool, const int32_t* block_table,
                  void* workspace, size_t workspace_bytes, void* out, float* lse,
                  hipStream_t stream) {
  pkv_status st = check_run(prob, tok_offsets, num_tokens, seq_lens, block_table);
  if (st != PKV_OK) return st;
  st = check_view(view);
  if (st != PKV_OK) return st;
  if (max_splits < 1 || max_splits > 65535) return PKV_EINVAL;
  if (num_tokens == 0) return PKV_OK;
  if (!q || !k_pool || (!kv4 && !v_pool) || !out || (max_splits > 1 && !workspace))
    return PKV_EINVAL;
  if (!aligned(q, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(out, 16) ||
      !aligned(workspace, 16))
    return PKV_ESHAPE;
  PromptArgs a{};
  a.q = q;
  a.k_pool = k_pool;
  a.v_pool = v_pool;
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
  if (!prompt_fits(prob, tiles, max_splits)) return PKV_ERANGE;
  if (max_splits > 1) {
    if (workspace_bytes < prompt_workspace_of(prob, tiles, max_splits)) return PKV_ENOSPC;
    a.arrivals = static_cast<int32_t*>(workspace);
    a.state = reinterpret_cast<float*>(static_cast<char*>(workspace) + kCounterBytes);
  }
  return launch_prompt(*prob, kv4, a, stream);
}

pkv_status store(const pkv_problem* prob, const int32_t* tok_offsets, int32_t num_tokens,
                 const int32_t* seq_lens, const void* k_new, int64_t k_stride, const void* v_new,
                 int64_t v_stride, const int32_t* block_table, bool kv4, void* k_pool,
                 void* v_pool, hipStream_t stream) {
  const pkv_status st = check_run(prob, tok_offsets, num_tokens, seq_lens, block_table);
  if (st != PKV_OK) return st;
  if (num_tokens == 0) return PKV_OK;
  if (!k_new || !v_new || !k_pool || (!kv4 && !v_pool)) return PKV_EINVAL;
  const int64_t width = int64_t(prob->num_kv_heads) * prob->head_dim;
  if (k_stride < width || v_stride < width || k_stride % 8 != 0 || v_stride % 8 != 0)
    return PKV_ESHAPE;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16))
    return PKV_ESHAPE;
  StoreArgs a{};
  a.k_new = k_new;
  a.v_new = v_new;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.tok_offsets = tok_offsets;
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.batch = prob->batch;
  a.num_tokens = num_tokens;
  a.num_kv_heads = prob->num_kv_heads;
  a.max_pages = prob->max_pages_per_row;
  a.num_pool_pages = prob->num_pool_pages;
  if (run_groups(a) > kMaxGridGroups) return PKV_ERANGE;
  return launch_store(*prob, kv4, a, stream);
}

}  // namespace

extern "C" size_t pkv_kv4_page_bytes(int32_t head_dim) {
  return head_dim == 64 || head_dim == 128 ? size_t(17) * head_dim : 0;
}

extern "C" pkv_status pkv_store_kv(const pkv_problem* prob, const int32_t* tok_offsets,
                                   int32_t num_tokens, const int32_t* seq_lens_dev,
                                   const void* k_new, int64_t k_stride, const void* v_new,
                                   int64_t v_stride, const int32_t* block_table, void* k_pool,
                                   void* v_pool, hipStream_t stream) {
  return store(prob, tok_offsets, num_tokens, seq_lens_dev, k_new, k_stride, v_new, v_stride,
               block_table, false, k_pool, v_pool, stream);
}

extern "C" pkv_status pkv_kv4_store(const pkv_problem* prob, const int32_t* tok_offsets,
                                    int32_t num_tokens, const int32_t* seq_lens_dev,
                                    const void* k_new, int64_t k_stride, const void* v_new,
                                    int64_t v_stride, const int32_t* block_table, void* kv4_pool,
                                    hipStream_t stream) {
  return store(prob, tok_offsets, num_tokens, seq_lens_dev, k_new, k_stride, v_new, v_stride,
               block_table, true, kv4_pool, nullptr, stream);
}

extern "C" pkv_status pkv_kv4_load(const pkv_problem* prob, const int32_t* tok_offsets,
                                   int32_t num_tokens, const int32_t* seq_lens_dev,
                                   const int32_t* block_table, const void* kv4_pool, void* k_out,
                                   void* v_out, hipStream_t stream) {
  const pkv_status st = check_run(prob, tok_offsets, num_tokens, seq_lens_dev, block_table);
  if (st != PKV_OK) return st;
  if (num_tokens == 0) return PKV_OK;
  if (!kv4_pool || !k_out || !v_out) return PKV_EINVAL;
  if (!aligned(kv4_pool, 16) || !aligned(k_out, 16) || !aligned(v_out, 16)) return PKV_ESHAPE;
  LoadArgs a{};
  a.pool = kv4_pool;
  a.block_table = block_table;
  a.seq_lens = seq_lens_dev;
  a.tok_offsets = tok_offsets;
  a.k_out = k_out;
  a.v_out = v_out;
  a.batch = prob->batch;
  a.num_tokens = num_tokens;
  a.num_kv_heads = prob->num_kv_heads;
  a.max_pages = prob->max_pages_per_row;
  a.num_pool_pages = prob->num_pool_pages;
  if (run_groups(a) > kMaxGridGroups) return PKV_ERANGE;
  return launch_load(*prob, a, stream);
}

extern "C" size_t pkv_attend_workspace_bytes(const pkv_problem* prob, int32_t max_splits) {
  if (check_problem(prob) != PKV_OK || max_splits < 1 || max_splits > 65535 ||
      check_attend_size(prob, max_splits) != PKV_OK)
    return 0;
  return workspace_of(prob, max_splits).bytes;
}

extern "C" int32_t pkv_attend_splits(const pkv_problem* prob, const pkv_view* view,
                                     int32_t num_cus) {
  if (check_problem(prob) != PKV_OK || check_view(view) != PKV_OK) return 0;
  if (num_cus < 1 || num_cus > 1024) return 0;
  int32_t fill, even;
  ranges_of_device(int64_t(prob->batch) * prob->num_kv_heads, num_cus, &fill, &even);
  const int ranges = decode_ranges(static_cast<int>(most_pages(prob, view)), fill, even);
  return std::min(ranges, 1024);
}

extern "C" pkv_status pkv_attend_window(const pkv_problem* prob, const pkv_view* view,
                                        const int32_t* seq_lens_dev, int32_t max_splits,
                                        const void* q, const void* k_pool, const void* v_pool,
                                        const int32_t* block_table, void* workspace,
                                        size_t workspace_bytes, void* out, float* lse,
                                        hipStream_t stream) {
  return attend(prob, view, seq_lens_dev, max_splits, q, false, k_pool, v_pool, block_table,
                workspace, workspace_bytes, out, lse, stream);
}

extern "C" pkv_status pkv_attend_kv4(const pkv_problem* prob, const pkv_view* view,
                                     const int32_t* seq_lens_dev, int32_t max_splits,
                                     const void* q, const void* kv4_pool,
                                     const int32_t* block_table, void* workspace,
                                     size_t workspace_bytes, void* out, float* lse,
                                     hipStream_t stream) {
  return attend(prob, view, seq_lens_dev, max_splits, q, true, kv4_pool, nullptr, block_table,
                workspace, workspace_bytes, out, lse, stream);
}

extern "C" pkv_status pkv_prompt_window(const pkv_problem* prob, const pkv_view* view,
                                        const int32_t* tok_offsets, int32_t num_tokens,
                                        const int32_t* seq_lens_dev, int32_t max_splits,
                                        const void* q, const void* k_pool, const void* v_pool,
                                        const int32_t* block_table, void* workspace,
                                        size_t workspace_bytes, void* out, float* lse,
                                        hipStream_t stream) {
  return prompt(prob, view, tok_offsets, num_tokens, seq_lens_dev, max_splits, q, false, k_pool,
                v_pool, block_table, workspace, workspace_bytes, out, lse, stream);
}

extern "C" pkv_status pkv_prompt_kv4(const pkv_problem* prob, const pkv_view* view,
                                     const int32_t* tok_offsets, int32_t num_tokens,
                                     const int32_t* seq_lens_dev, int32_t max_splits,
                                     const void* q, const void* kv4_pool,
                                     const int32_t* block_table, void* workspace,
                                     size_t workspace_bytes, void* out, float* lse,
                                     hipStream_t stream) {
  return prompt(prob, view, tok_offsets, num_tokens, seq_lens_dev, max_splits, q, true, kv4_pool,
                nullptr, block_table, workspace, workspace_bytes, out, lse, stream);
}

namespace {

// Query tiles of a run batch, from the host's numbers alone; -1 when invalid.
int64_t tiles_of(const pkv_problem* p, int32_t num_tokens, int32_t one_per_row) {
  if (check_problem(p) != PKV_OK || num_tokens < 0 || (one_per_row && num_tokens != p->batch))
    return -1;
  return one_per_row ? p->batch
                     : tile_base(num_tokens, p->batch, p->num_q_heads / p->num_kv_heads);
}

}  // namespace

extern "C" size_t pkv_prompt_workspace_bytes(const pkv_problem* prob, int32_t num_tokens,
                                             int32_t one_per_row, int32_t max_splits) {
  const int64_t tiles = tiles_of(prob, num_tokens, one_per_row);
  if (tiles < 0 || max_splits < 2 || max_splits > 65535 ||
      !prompt_fits(prob, tiles, max_splits))
    return 0;
  return prompt_workspace_of(prob, tiles, max_splits);
}

extern "C" int32_t pkv_prompt_splits(const pkv_problem* prob, const pkv_view* view,
                                     int32_t num_tokens, int32_t one_per_row, int32_t num_cus) {
  const int64_t tiles = tiles_of(prob, num_tokens, one_per_row);
  if (tiles < 0 || check_view(view) != PKV_OK || num_cus < 1 || num_cus > 1024) return 0;
  if (tiles == 0) return 1;
  // Two workgroups a compute unit, as long as a split keeps its steps.  Tiles: half of a row's last one on the average; the launch counts the
  // real ones and cuts into fewer ranges where there are more.
  const int64_t rows = int64_t(num_tokens) * (prob->num_q_heads / prob->num_kv_heads);
  const int64_t likely = one_per_row ? tiles
                                     : std::max<int64_t>({1, ceil_div(rows, kTileRows),
                                                          rows / kTileRows + prob->batch / 2});
  const int64_t fill = 2 * int64_t(num_cus) / (likely * prob->num_kv_heads);
  const int64_t keys = std::min<int64_t>(most_pages(prob, view) + ceil_div(num_tokens, 16),
                                         prob->max_pages_per_row);
  return static_cast<int32_t>(
      std::max<int64_t>(1, std::min<int64_t>(fill, prompt_ranges(static_cast<int>(keys / 4)))));
}
