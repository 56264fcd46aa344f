// Entry points of include/pkv_serving.h: argument checks on the host, then
// launches on the caller's stream.
#include "context/context_host.h"
#include "serving/serving_internal.h"

using namespace pkv;

extern "C" size_t pkv_kv8_page_bytes(int32_t head_dim) {
  return head_dim == 64 || head_dim == 128 ? size_t(32) * head_dim : 0;
}

extern "C" pkv_status pkv_kv8_store(const pkv_problem* prob, const int32_t* tok_offsets,
                                    int32_t num_tokens, const int32_t* seq_lens_dev,
                                    const void* k_new, int64_t k_stride, const void* v_new,
                                    int64_t v_stride, const int32_t* block_table, void* kv8_pool,
                                    void* kv8_scales, hipStream_t stream) {
  const pkv_status st = check_run(prob, tok_offsets, num_tokens, seq_lens_dev, block_table);
  if (st != PKV_OK) return st;
  if (num_tokens == 0) return PKV_OK;
  if (!k_new || !v_new || !kv8_pool || !kv8_scales) return PKV_EINVAL;
  const int64_t width = int64_t(prob->num_kv_heads) * prob->head_dim;
  if (k_stride < width || v_stride < width || k_stride % 8 != 0 || v_stride % 8 != 0)
    return PKV_ESHAPE;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(kv8_pool, 16) ||
      !aligned(kv8_scales, 2))
    return PKV_ESHAPE;
  Store8Args a{};
  a.k_new = k_new;
  a.v_new = v_new;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.block_table = block_table;
  a.seq_lens = seq_lens_dev;
  a.tok_offsets = tok_offsets;
  a.k_pool = kv8_pool;
  a.scales = static_cast<uint8_t*>(kv8_scales);
  a.batch = prob->batch;
  a.num_tokens = num_tokens;
  a.num_kv_heads = prob->num_kv_heads;
  a.max_pages = prob->max_pages_per_row;
  a.num_pool_pages = prob->num_pool_pages;
  if (run_groups(a) > kMaxGridGroups) return PKV_ERANGE;
  return launch_store8(*prob, a, stream);
}

extern "C" pkv_status pkv_kv8_load(const pkv_problem* prob, const int32_t* tok_offsets,
                                   int32_t num_tokens, const int32_t* seq_lens_dev,
                                   const int32_t* block_table, const void* kv8_pool,
                                   const void* kv8_scales, void* k_out, void* v_out,
                                   hipStream_t stream) {
  const pkv_status st = check_run(prob, tok_offsets, num_tokens, seq_lens_dev, block_table);
  if (st != PKV_OK) return st;
  if (num_tokens == 0) return PKV_OK;
  if (!kv8_pool || !kv8_scales || !k_out || !v_out) return PKV_EINVAL;
  if (!aligned(kv8_pool, 16) || !aligned(kv8_scales, 2) || !aligned(k_out, 16) ||
      !aligned(v_out, 16))
    return PKV_ESHAPE;
  Load8Args a{};
  a.pool = kv8_pool;
  a.scales = static_cast<const uint8_t*>(kv8_scales);
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
  return launch_load8(*prob, a, stream);
}

extern "C" pkv_status pkv_attend_kv8(const pkv_problem* prob, const pkv_view* view,
                                     const int32_t* seq_lens_dev, int32_t max_splits,
                                     const void* q, const void* kv8_pool, const void* kv8_scales,
                                     const int32_t* block_table, void* workspace,
                                     size_t workspace_bytes, void* out, float* lse,
                                     hipStream_t stream) {
  AttendArgs a;
  const pkv_status st =
      fill_attend(prob, view, seq_lens_dev, max_splits, q,
                  {Cache::k8, kv8_pool, nullptr, kv8_scales}, block_table, workspace,
                  workspace_bytes, out, lse, &a);
  return st == PKV_OK ? launch_attend8(*prob, a, stream) : st;
}

extern "C" pkv_status pkv_prompt_kv8(const pkv_problem* prob, const pkv_view* view,
                                     const int32_t* tok_offsets, int32_t num_tokens,
                                     const int32_t* seq_lens_dev, int32_t max_splits,
                                     const void* q, const void* kv8_pool, const void* kv8_scales,
                                     const int32_t* block_table, void* workspace,
                                     size_t workspace_bytes, void* out, float* lse,
                                     hipStream_t stream) {
  PromptArgs a;
  const pkv_status st =
      fill_prompt(prob, view, tok_offsets, num_tokens, seq_lens_dev, max_splits, q,
                  {Cache::k8, kv8_pool, nullptr, kv8_scales}, block_table, workspace,
                  workspace_bytes, out, lse, Divide::kShares, &a);
  if (st != PKV_OK || a.num_tokens == 0) return st;
  return launch_prompt8(*prob, a, stream);
}

namespace {

// Shares a KV head of tiles of 128 queries: as many workgroups as run at once, as long as
// they get eight steps each.  Where the tiles alone may be as many, they stay whole:
// the tiles of a row then walk its keys together and read them out of the L2 (8 rows of
// 1024-8192 states, 97 tiles for 64 workgroups, 16 bits: 306 us whole, 326 in shares;
// 24 tiles for 64, 8 bits, 3000-31000 states: 582 whole, 258 in shares).  A prompt, or
// cross attention (view null: every query sees the whole table).
int32_t shares_for(const pkv_problem* p, const pkv_view* view, int32_t num_tokens, int64_t tiles,
                   int32_t num_cus) {
  const int64_t slots = std::max<int64_t>(2 * int64_t(num_cus) / p->num_kv_heads, 1);
  const int64_t pages = std::min<int64_t>(most_pages(p, view) + ceil_div(num_tokens, 16),
                                          p->max_pages_per_row);
  const int64_t shares = std::min(slots, tiles * (ceil_div(pages, 4) / kRangeSteps));
  if (tiles > slots || shares < 2 ||
      !prompt_fits(p, tiles, static_cast<int32_t>(shares), Divide::kShares))
    return 1;
  return static_cast<int32_t>(shares);
}

}  // namespace

extern "C" size_t pkv_prompt_kv8_workspace_bytes(const pkv_problem* prob, int32_t num_tokens,
                                                 int32_t one_per_row, int32_t max_splits) {
  return prompt_bytes(prob, tiles_of(prob, num_tokens, one_per_row), max_splits, Divide::kShares);
}

extern "C" int32_t pkv_prompt_kv8_splits(const pkv_problem* prob, const pkv_view* view,
                                         int32_t num_tokens, int32_t one_per_row,
                                         int32_t num_cus) {
  const int64_t tiles = tiles_of(prob, num_tokens, one_per_row);
  if (tiles < 0 || check_view(view) != PKV_OK || num_cus < 1 || num_cus > 1024) return 0;
  return num_tokens == 0 ? 1 : shares_for(prob, view, num_tokens, tiles, num_cus);
}

// ---- cross attention -------------------------------------------------------------

namespace {

// Launch size of tiles of sixteen queries, and their counters where they are split.
bool cross_fits(const pkv_problem* p, int64_t tiles, int32_t splits) {
  const int64_t pairs = tiles * p->num_kv_heads;
  return pairs * splits <= kMaxGridGroups && (splits == 1 || pairs <= kCounters);
}

// As workspace_of, with kCrossRows states a slot.
Workspace cross_workspace_of(const pkv_problem* p, int64_t tiles, int32_t splits) {
  const auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
  const size_t states = static_cast<size_t>(tiles) * p->num_kv_heads * splits * kCrossRows;
  Workspace w;
  w.ml = kCounterBytes;
  w.o = w.ml + up(states * 2 * sizeof(float));
  w.bytes = w.o + states * p->head_dim * sizeof(float);
  return w;
}

// The ranges, up to max_splits, whose states a workspace holds; 1: not even two.  A
// workspace for two ranges or more of a call of many queries holds two of any call of
// few over the same problem, so it is never too small for a smaller step: up to 64 (32)
// queries a row make 5 (3) tiles of 16 states a row and range, more of them 1.5 (1.25) and
// more tiles of 128 a row.
int32_t cross_splits_in(const pkv_problem* p, int64_t tiles, int32_t max_splits, size_t bytes) {
  const size_t one = static_cast<size_t>(tiles) * p->num_kv_heads * kCrossRows *
                     (p->head_dim + 2) * sizeof(float);
  if (bytes < kCounterBytes) return 1;
  size_t s = std::min<size_t>((bytes - kCounterBytes) / one, max_splits);
  while (s > 1 && cross_workspace_of(p, tiles, static_cast<int32_t>(s)).bytes > bytes) --s;
  return static_cast<int32_t>(std::max<size_t>(s, 1));
}

pkv_status cross(const pkv_problem* prob, const int32_t* tok_offsets, int32_t num_tokens,
                 const int32_t* seq_lens, int32_t max_splits, const void* q, Pools pools,
                 const int32_t* block_table, void* workspace, size_t workspace_bytes, void* out,
                 float* lse, hipStream_t stream) {
  const pkv_status run = check_run(prob, tok_offsets, num_tokens, seq_lens, block_table);
  if (run != PKV_OK) return run;
  if (!cross_takes_few(*prob, num_tokens, !tok_offsets)) {
    PromptArgs a;
    const pkv_status st = fill_prompt(prob, nullptr, tok_offsets, num_tokens, seq_lens, max_splits,
                                      q, pools, block_table, workspace, workspace_bytes, out, lse,
                                      Divide::kShares, &a);
    if (st != PKV_OK || a.num_tokens == 0) return st;
    return launch_cross_many(*prob, pools.kind, a, stream);
  }
  if (max_splits < 1 || max_splits > 65535) return PKV_EINVAL;
  if (num_tokens == 0) return PKV_OK;
  if (!q || !pools.given() || !out || (max_splits > 1 && !workspace)) return PKV_EINVAL;
  if (!aligned(q, 16) || !pools.placed() || !aligned(out, 16) || !aligned(workspace, 16))
    return PKV_ESHAPE;
  const int64_t tiles = cross_tiles(*prob, num_tokens, !tok_offsets);
  if (!cross_fits(prob, tiles, max_splits)) return PKV_ERANGE;
  AttendArgs a{};
  if (max_splits > 1) {
    max_splits = cross_splits_in(prob, tiles, max_splits, workspace_bytes);
    if (max_splits < 2) return PKV_ENOSPC;
    const Workspace w = cross_workspace_of(prob, tiles, max_splits);
    char* ws = static_cast<char*>(workspace);
    a.arrivals = reinterpret_cast<int32_t*>(ws);
    a.st_ml = reinterpret_cast<float*>(ws + w.ml);
    a.st_o = reinterpret_cast<float*>(ws + w.o);
  }
  a.q = q;
  pools.fill(&a);
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.tok_offsets = tok_offsets;
  a.num_tokens = num_tokens;
  a.out = out;
  a.lse = lse;
  a.batch = prob->batch;
  a.num_q_heads = prob->num_q_heads;
  a.num_kv_heads = prob->num_kv_heads;
  a.group = prob->num_q_heads / prob->num_kv_heads;
  a.group_inv = static_cast<uint32_t>(ceil_div(4096, a.group));
  a.max_pages = prob->max_pages_per_row;
  a.num_pool_pages = prob->num_pool_pages;
  a.splits = max_splits;
  set_scale(prob, &a);
  return launch_cross_few(*prob, pools.kind, tiles, a, stream);
}

}  // namespace

extern "C" size_t pkv_cross_workspace_bytes(const pkv_problem* prob, int32_t num_tokens,
                                            int32_t one_per_row, int32_t max_splits) {
  if (tiles_of(prob, num_tokens, one_per_row) < 0 || max_splits < 2 || max_splits > 65535)
    return 0;
  if (!cross_takes_few(*prob, num_tokens, one_per_row != 0))
    return pkv_prompt_kv8_workspace_bytes(prob, num_tokens, one_per_row, max_splits);
  const int64_t tiles = cross_tiles(*prob, num_tokens, one_per_row != 0);
  return cross_fits(prob, tiles, max_splits) ? cross_workspace_of(prob, tiles, max_splits).bytes
                                             : 0;
}

extern "C" int32_t pkv_cross_splits(const pkv_problem* prob, int32_t num_tokens,
                                    int32_t one_per_row, int32_t num_cus) {
  if (tiles_of(prob, num_tokens, one_per_row) < 0 || num_cus < 1 || num_cus > 1024) return 0;
  if (num_tokens == 0) return 1;
  if (!cross_takes_few(*prob, num_tokens, one_per_row != 0))
    return pkv_prompt_kv8_splits(prob, nullptr, num_tokens, one_per_row, num_cus);
  // The launch counts the real tiles; there are at least these.
  const int64_t rows = int64_t(num_tokens) * (prob->num_q_heads / prob->num_kv_heads);
  const int64_t likely = std::max(ceil_div(rows, kCrossRows),
                                  std::min<int64_t>(num_tokens, ceil_div(prob->batch, 2)));
  int32_t fill, even;
  ranges_of_device(likely * prob->num_kv_heads, num_cus, &fill, &even);
  const int ranges = std::min(decode_ranges(prob->max_pages_per_row, fill, even), 1024);
  const int64_t tiles = cross_tiles(*prob, num_tokens, one_per_row != 0);
  return cross_fits(prob, tiles, ranges) ? ranges : 1;
}

extern "C" pkv_status pkv_cross(const pkv_problem* prob, const int32_t* tok_offsets,
                                int32_t num_tokens, const int32_t* seq_lens_dev,
                                int32_t max_splits, const void* q, const void* k_pool,
                                const void* v_pool, const int32_t* block_table, void* workspace,
                                size_t workspace_bytes, void* out, float* lse,
                                hipStream_t stream) {
  return cross(prob, tok_offsets, num_tokens, seq_lens_dev, max_splits, q,
               {Cache::k16, k_pool, v_pool, nullptr}, block_table, workspace, workspace_bytes, out,
               lse, stream);
}

extern "C" pkv_status pkv_cross_kv4(const pkv_problem* prob, const int32_t* tok_offsets,
                                    int32_t num_tokens, const int32_t* seq_lens_dev,
                                    int32_t max_splits, const void* q, const void* kv4_pool,
                                    const int32_t* block_table, void* workspace,
                                    size_t workspace_bytes, void* out, float* lse,
                                    hipStream_t stream) {
  return cross(prob, tok_offsets, num_tokens, seq_lens_dev, max_splits, q,
               {Cache::k4, kv4_pool, nullptr, nullptr}, block_table, workspace, workspace_bytes,
               out, lse, stream);
}

extern "C" pkv_status pkv_cross_kv8(const pkv_problem* prob, const int32_t* tok_offsets,
                                    int32_t num_tokens, const int32_t* seq_lens_dev,
                                    int32_t max_splits, const void* q, const void* kv8_pool,
                                    const void* kv8_scales, const int32_t* block_table,
                                    void* workspace, size_t workspace_bytes, void* out, float* lse,
                                    hipStream_t stream) {
  return cross(prob, tok_offsets, num_tokens, seq_lens_dev, max_splits, q,
               {Cache::k8, kv8_pool, nullptr, kv8_scales}, block_table, workspace, workspace_bytes,
               out, lse, stream);
}

// ---- page tables -------------------------------------------------------------------

extern "C" pkv_status pkv_pages_take(const pkv_problem* prob, const int32_t* counts,
                                     int32_t num_tokens, int32_t* lens, int32_t* block_table,
                                     const int32_t* free_pages, int32_t* state, int32_t* seq_lens,
                                     int32_t* tok_offsets, int64_t* slots, int32_t* positions,
                                     hipStream_t stream) {
  const pkv_status st = check_problem(prob);
  if (st != PKV_OK) return st;
  if (!counts || num_tokens < 0 || !lens || !block_table || !free_pages || !state || !seq_lens ||
      !tok_offsets)
    return PKV_EINVAL;
  if (num_tokens > 1 << 30) return PKV_ERANGE;
  TakeArgs a{};
  a.counts = counts;
  a.lens = lens;
  a.block_table = block_table;
  a.free_pages = free_pages;
  a.state = state;
  a.seq_lens = seq_lens;
  a.tok_offsets = tok_offsets;
  a.slots = slots;
  a.positions = positions;
  a.batch = prob->batch;
  a.num_tokens = num_tokens;
  a.max_pages = prob->max_pages_per_row;
  a.num_pool_pages = prob->num_pool_pages;
  return launch_take(a, stream);
}

extern "C" pkv_status pkv_pages_release(const pkv_problem* prob, const int32_t* keep,
                                        int32_t* lens, int32_t* block_table, int32_t* free_pages,
                                        int32_t* state, hipStream_t stream) {
  const pkv_status st = check_problem(prob);
  if (st != PKV_OK) return st;
  if (!keep || !lens || !block_table || !free_pages || !state) return PKV_EINVAL;
  ReleaseArgs a{};
  a.keep = keep;
  a.lens = lens;
  a.block_table = block_table;
  a.free_pages = free_pages;
  a.state = state;
  a.batch = prob->batch;
  a.max_pages = prob->max_pages_per_row;
  a.num_pool_pages = prob->num_pool_pages;
  return launch_release(a, stream);
}
