// Entry points of include/pkv_context.h: argument checks on the host, then
// launches on the caller's stream.
#include "context/context_host.h"

using namespace pkv;

namespace {

pkv_status attend(const pkv_problem* prob, const pkv_view* view, const int32_t* seq_lens,
                  int32_t max_splits, const void* q, Pools pools, const int32_t* block_table,
                  void* workspace, size_t workspace_bytes, void* out, float* lse,
                  hipStream_t stream) {
  AttendArgs a;
  const pkv_status st = fill_attend(prob, view, seq_lens, max_splits, q, pools, block_table,
                                    workspace, workspace_bytes, out, lse, &a);
  return st == PKV_OK ? launch_attend(*prob, pools.kind == Cache::k4, a, stream) : st;
}

pkv_status prompt(const pkv_problem* prob, const pkv_view* view, const int32_t* tok_offsets,
                  int32_t num_tokens, const int32_t* seq_lens, int32_t max_splits, const void* q,
                  Pools pools, const int32_t* block_table, void* workspace,
                  size_t workspace_bytes, void* out, float* lse, hipStream_t stream) {
  PromptArgs a;
  const pkv_status st = fill_prompt(prob, view, tok_offsets, num_tokens, seq_lens, max_splits, q,
                                    pools, block_table, workspace, workspace_bytes, out, lse,
                                    Divide::kRanges, &a);
  if (st != PKV_OK || a.num_tokens == 0) return st;
  return launch_prompt(*prob, pools.kind == Cache::k4, a, stream);
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
  return attend(prob, view, seq_lens_dev, max_splits, q, {Cache::k16, k_pool, v_pool, nullptr},
                block_table, workspace, workspace_bytes, out, lse, stream);
}

extern "C" pkv_status pkv_attend_kv4(const pkv_problem* prob, const pkv_view* view,
                                     const int32_t* seq_lens_dev, int32_t max_splits,
                                     const void* q, const void* kv4_pool,
                                     const int32_t* block_table, void* workspace,
                                     size_t workspace_bytes, void* out, float* lse,
                                     hipStream_t stream) {
  return attend(prob, view, seq_lens_dev, max_splits, q, {Cache::k4, kv4_pool, nullptr, nullptr},
                block_table, workspace, workspace_bytes, out, lse, stream);
}

extern "C" pkv_status pkv_prompt_window(const pkv_problem* prob, const pkv_view* view,
                                        const int32_t* tok_offsets, int32_t num_tokens,
                                        const int32_t* seq_lens_dev, int32_t max_splits,
                                        const void* q, const void* k_pool, const void* v_pool,
                                        const int32_t* block_table, void* workspace,
                                        size_t workspace_bytes, void* out, float* lse,
                                        hipStream_t stream) {
  return prompt(prob, view, tok_offsets, num_tokens, seq_lens_dev, max_splits, q,
                {Cache::k16, k_pool, v_pool, nullptr}, block_table, workspace, workspace_bytes,
                out, lse, stream);
}

extern "C" pkv_status pkv_prompt_kv4(const pkv_problem* prob, const pkv_view* view,
                                     const int32_t* tok_offsets, int32_t num_tokens,
                                     const int32_t* seq_lens_dev, int32_t max_splits,
                                     const void* q, const void* kv4_pool,
                                     const int32_t* block_table, void* workspace,
                                     size_t workspace_bytes, void* out, float* lse,
                                     hipStream_t stream) {
  return prompt(prob, view, tok_offsets, num_tokens, seq_lens_dev, max_splits, q,
                {Cache::k4, kv4_pool, nullptr, nullptr}, block_table, workspace, workspace_bytes,
                out, lse, stream);
}

extern "C" size_t pkv_prompt_workspace_bytes(const pkv_problem* prob, int32_t num_tokens,
                                             int32_t one_per_row, int32_t max_splits) {
  return prompt_bytes(prob, tiles_of(prob, num_tokens, one_per_row), max_splits, Divide::kRanges);
}

extern "C" int32_t pkv_prompt_splits(const pkv_problem* prob, const pkv_view* view,
                                     int32_t num_tokens, int32_t one_per_row, int32_t num_cus) {
  const int64_t tiles = tiles_of(prob, num_tokens, one_per_row);
  if (tiles < 0 || check_view(view) != PKV_OK || num_cus < 1 || num_cus > 1024) return 0;
  if (tiles == 0) return 1;
  // Two workgroups a compute unit, as long as a split keeps its steps.  Tiles: half of a
  // row's last one on the average; the launch counts the real ones and cuts into fewer
  // ranges where there are more.
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
