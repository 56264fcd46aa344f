// Page tables kept on the device (gfx950): pages for a step's new tokens, with the
// offsets, lengths, slots and positions that the step's calls read, and pages given
// back.
//
//   off_i = sum_{k<i} c_k,  need_i = ceil((n_i + c_i) / 16) - ceil(n_i / 16),
// row i is served where its tokens fit the call's arrays and the table and the sum of
// need_k, k <= i, fits the free list; its page of rank m among all that are asked for
// is free[count - 1 - m].  Released pages go on top, the last row's last page first, so
// that giving back what a call took restores the list.  Entries of a table that name no
// page of the pool go there too and come out again: where a workgroup met one, the last to
// finish closes the list's gaps.
//
// Bound: latency.  A step of 64 rows reads and writes a few KB behind a chain of three
// dependent loads (lengths, free list, table); 256 rows of 130000 tokens write
// 1.6 MB.  So: one launch; every workgroup scans all rows by itself (1024 at a time,
// four a thread) and does 512 tokens or its share of the pages.  Nothing that
// the others read is written before all are done: the last of several workgroups to
// finish writes lengths and counts; one workgroup needs nobody.  64 rows of a token each
// take 4.2-4.6 us and give their pages back in 3.5, most of it launch and the chain of
// loads; 132465 tokens of 256 rows take 9.2-9.4 and 6.2 (7600 pages).  (With the rows
// scanned again for their results 10.6.)
#include "context/states.h"
#include "context/wave.h"
#include "serving/serving_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerThread = 4;
constexpr int kChunk = kThreads * kRowsPerThread;  // rows of one scan
constexpr int kTokens = 512;                       // new tokens of a workgroup
constexpr int kFewPages = 1024;                    // released by one workgroup alone

__device__ __forceinline__ int pages_of(int tokens) {
  return (tokens >> 4) + ((tokens & 15) ? 1 : 0);
}

// Inclusive sum over the wave, no higher than `most` (below 2^31, so that two such sums add
// up within 32 bits).
__device__ __forceinline__ uint32_t capped_scan(uint32_t x, uint32_t most) {
  auto add = [&](int y) { x = min(x + static_cast<uint32_t>(y), most); };
  add(moved<kDppRowShr + 1>(static_cast<int>(x)));
  add(moved<kDppRowShr + 2>(static_cast<int>(x)));
  add(moved<kDppRowShr + 4>(static_cast<int>(x)));
  add(moved<kDppRowShr + 8>(static_cast<int>(x)));
  add(moved<kDppRowBcast15, 0xa>(static_cast<int>(x)));
  add(moved<kDppRowBcast31, 0xc>(static_cast<int>(x)));
  return x;
}

// Sums before a thread's own values `x` over the workgroup, from `carry` on, which
// becomes the sum of all; none above `most`.
__device__ __forceinline__ uint32_t scan_before(uint32_t x, uint32_t& carry, uint32_t most,
                                                uint32_t (&s_wave)[4]) {
  const int wave = threadIdx.x >> 6;
  const uint32_t upto = capped_scan(x, most);
  __syncthreads();
  if ((threadIdx.x & 63) == 63) s_wave[wave] = upto;
  // The lane below, 0 in the first.
  uint32_t before = static_cast<uint32_t>(__builtin_amdgcn_ds_bpermute(
      ((static_cast<int>(threadIdx.x & 63) - 1) & 63) << 2, static_cast<int>(upto)));
  if ((threadIdx.x & 63) == 0) before = 0;
  __syncthreads();
  uint32_t all = carry;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (w == wave) before = min(before + all, most);
    all = min(all + s_wave[w], most);
  }
  carry = all;
  return before;
}

// Index of the first entry of v[0, n) above x, v not decreasing, its last above x.
__device__ __forceinline__ int first_above(const uint32_t* v, int n, uint32_t x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] > x) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

__device__ __forceinline__ int free_count(const int32_t* state, int pool) {
  return min(max(state[kStateFree], 0), pool);
}

__global__ __launch_bounds__(kThreads) void take_kernel(TakeArgs a) {
  __shared__ uint32_t s_upto[kChunk];  // tokens up to and with a row
  __shared__ uint32_t s_off[kChunk];   // tokens before it
  __shared__ uint32_t s_rank[kChunk];  // pages asked for before it
  __shared__ int s_len[kChunk];        // tokens it holds; negative: not served
  __shared__ uint32_t s_wave[4];
  __shared__ bool s_last;
  const int cap = a.max_pages * 16;
  const uint32_t most = static_cast<uint32_t>(a.num_tokens) + 1;
  const uint32_t begin = blockIdx.x * uint32_t(kTokens), end = begin + kTokens;
  const int free = free_count(a.state, a.num_pool_pages);
  uint32_t tokens = 0, asked = 0, granted = 0, denied = 0;
  // One chunk of rows, four a thread.
  int cnt[kRowsPerThread], len[kRowsPerThread], need[kRowsPerThread];
  uint32_t upto[kRowsPerThread];
  bool ok[kRowsPerThread];
  auto scan = [&](int r0) {
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) {
      const int r = r0 + int(threadIdx.x) * kRowsPerThread + i;
      cnt[i] = r < a.batch ? max(a.counts[r], 0) : 0;
      len[i] = r < a.batch ? a.lens[r] : 0;
    }
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i)
      mine = min(mine + min(static_cast<uint32_t>(cnt[i]), most), most);
    uint32_t before = scan_before(mine, tokens, most, s_wave);
    uint32_t wants = 0;
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) {
      s_off[int(threadIdx.x) * kRowsPerThread + i] = before;
      upto[i] = before = min(before + min(static_cast<uint32_t>(cnt[i]), most), most);
      // (A row without tokens has none outside the arrays, whatever the rows before it bring.)
      ok[i] = len[i] >= 0 && len[i] <= cap && cnt[i] <= cap - len[i] &&
              (cnt[i] == 0 || upto[i] < most);
      need[i] = ok[i] ? pages_of(len[i] + cnt[i]) - pages_of(len[i]) : 0;
      wants += static_cast<uint32_t>(need[i]);
    }
    uint32_t rank = scan_before(wants, asked, 0x7fffffffu, s_wave);
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) {
      const int at = int(threadIdx.x) * kRowsPerThread + i;
      ok[i] = ok[i] && (need[i] == 0 || rank + need[i] <= static_cast<uint32_t>(free));
      s_upto[at] = upto[i];
      s_rank[at] = rank;
      s_len[at] = ok[i] ? len[i] : -1;
      rank += static_cast<uint32_t>(need[i]);
    }
  };
  auto write_rows = [&](int r0) {
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) {
      const int r = r0 + int(threadIdx.x) * kRowsPerThread + i;
      if (r >= a.batch) break;
      if (ok[i]) granted += static_cast<uint32_t>(need[i]);
      if (!ok[i] && cnt[i] > 0) ++denied;
      a.seq_lens[r] = ok[i] ? len[i] + cnt[i] : 0;
      a.tok_offsets[r + 1] = static_cast<int>(min(upto[i], most - 1));
      if (ok[i]) a.lens[r] = len[i] + cnt[i];
    }
  };

  int groups = gridDim.x;  // that have tokens of the step
  for (int r0 = 0; r0 < a.batch; r0 += kChunk) {
    const uint32_t tokens0 = tokens;
    scan(r0);
    if (a.batch <= kChunk) {
      groups = max(1, static_cast<int>((min(tokens, most - 1) + kTokens - 1) / kTokens));
      if (static_cast<int>(blockIdx.x) >= groups) return;
    }
    __syncthreads();
    const int rows = min(a.batch - r0, kChunk);
    const uint32_t stop = min(min(tokens, most - 1), end);
    for (uint32_t t = begin + threadIdx.x; t < stop; t += kThreads) {
      if (t < tokens0) continue;
      const int at = first_above(s_upto, rows, t);
      const int held = s_len[at];
      int64_t slot = -1;
      int p = -1;
      if (held >= 0) {
        const int64_t row = int64_t(r0 + at) * a.max_pages;
        p = held + static_cast<int>(t - s_off[at]);
        const int entry = p >> 4, had = pages_of(held);
        int page;
        if (entry >= had) {
          page = a.free_pages[free - 1 - static_cast<int>(s_rank[at]) - (entry - had)];
          if ((p & 15) == 0) a.block_table[row + entry] = page;
        } else {
          page = a.block_table[row + entry];
        }
        if (static_cast<uint32_t>(page) < static_cast<uint32_t>(a.num_pool_pages))
          slot = int64_t(page) * 16 + (p & 15);
      }
      if (a.slots) a.slots[t] = slot;
      if (a.positions) a.positions[t] = p;
    }
    if (groups == 1) write_rows(r0);
    else if (tokens >= end) break;  // the rows behind have none of its tokens
  }
  if (groups > 1) {
    if (!last_to_arrive(a.state + kStateArrivals, groups, &s_last)) return;
    if (a.batch <= kChunk) {
      write_rows(0);  // as scanned
    } else {
      tokens = asked = 0;
      for (int r0 = 0; r0 < a.batch; r0 += kChunk) {
        scan(r0);
        write_rows(r0);
      }
    }
  }
  const uint32_t all = static_cast<uint32_t>(wave_sum_i(static_cast<int>(granted)));
  const uint32_t no = static_cast<uint32_t>(wave_sum_i(static_cast<int>(denied)));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) {
    s_wave[threadIdx.x >> 6] = all;
    s_rank[threadIdx.x >> 6] = no;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    a.tok_offsets[0] = 0;
    a.state[kStateFree] = free - static_cast<int>(s_wave[0] + s_wave[1] + s_wave[2] + s_wave[3]);
    a.state[kStateDenied] = static_cast<int>(s_rank[0] + s_rank[1] + s_rank[2] + s_rank[3]);
  }
}

// Past the L2, for the workgroup that closes gaps (7600 pages of many workgroups: 0.4 us more
// than into the L2).
__device__ __forceinline__ void put_page(int32_t* p, int page) {
  __hip_atomic_store(p, page, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// As last_to_arrive; in the last workgroup `any` becomes true where it was in one of them
// (the counter's upper half counts those).
__device__ __forceinline__ bool last_of_any(int32_t* counter, int ns, bool& any, int* s_last) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0) {
    const int was = __hip_atomic_fetch_add(counter, any ? 0x10001 : 1, __ATOMIC_RELAXED,
                                           __HIP_MEMORY_SCOPE_AGENT);
    const bool last = (was & 0xffff) == ns - 1;
    if (last) __hip_atomic_store(counter, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *s_last = !last ? 0 : any || was > 0xffff ? 2 : 1;
  }
  __syncthreads();
  any = *s_last == 2;
  return *s_last != 0;
}

__global__ __launch_bounds__(kThreads) void release_kernel(ReleaseArgs a) {
  __shared__ uint32_t s_upto[kChunk];  // pages up to and with a row, from the last row on
  __shared__ int s_end[kChunk];        // block-table entry behind its last page
  __shared__ uint32_t s_wave[4];
  __shared__ bool s_gap;               // an entry released here names no page of the pool
  __shared__ int s_last;
  const int cap = a.max_pages * 16;
  const int free = free_count(a.state, a.num_pool_pages);
  if (threadIdx.x == 0) s_gap = false;
  // The new length of a row: `keep` where that is shorter.
  auto kept = [&](int r, int& len) {
    len = a.lens[r];
    const int keep = a.keep[r];
    return (len < 0 || len > cap || keep < 0 || keep >= len) ? len : keep;
  };
  auto pages_between = [&](int keep, int len) {
    return (len < 0 || len > cap) ? 0 : pages_of(len) - pages_of(keep);
  };

  // With more than one chunk of rows, or many pages, the pages are divided among the
  // workgroups; a few are moved by the first alone, and the others need not wait for it:
  // rows that it has shortened already count as nothing to them.
  uint32_t total = 0;
  bool alone = gridDim.x == 1;
  uint32_t next = blockIdx.x * uint32_t(kThreads) + threadIdx.x;
  uint32_t stride = gridDim.x * uint32_t(kThreads);
  for (int r0 = 0; r0 < a.batch; r0 += kChunk) {
    const uint32_t total0 = total;
    int count[kRowsPerThread];
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) {
      const int at = int(threadIdx.x) * kRowsPerThread + i, r = a.batch - 1 - r0 - at;
      count[i] = 0;
      s_end[at] = 0;
      if (r >= 0) {
        int len;
        const int keep = kept(r, len);
        count[i] = pages_between(keep, len);
        s_end[at] = pages_of(len);
      }
      mine += static_cast<uint32_t>(count[i]);
    }
    uint32_t upto = scan_before(mine, total, 0x7fffffffu, s_wave);
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) {
      upto += static_cast<uint32_t>(count[i]);
      s_upto[int(threadIdx.x) * kRowsPerThread + i] = upto;
    }
    __syncthreads();
    if (a.batch <= kChunk && !alone && total <= kFewPages) {
      if (blockIdx.x != 0) return;
      alone = true;
      next = threadIdx.x;
      stride = kThreads;
    }
    const int rows = min(a.batch - r0, kChunk);
    for (; next < total; next += stride) {
      const int at = first_above(s_upto, rows, next);
      const uint32_t before = at > 0 ? s_upto[at - 1] : total0;
      const int entry = s_end[at] - 1 - static_cast<int>(next - before);
      int32_t* from = a.block_table + int64_t(a.batch - 1 - r0 - at) * a.max_pages + entry;
      const int64_t to = int64_t(free) + next;
      const int page = *from;
      if (to < a.num_pool_pages) {
        put_page(a.free_pages + to, page);
        if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.num_pool_pages)) s_gap = true;
      }
      *from = -1;
    }
    __syncthreads();
  }
  bool gap = s_gap;
  if (!alone && !last_of_any(a.state + kStateArrivals, gridDim.x, gap, &s_last)) return;
  uint32_t listed = min(total, static_cast<uint32_t>(a.num_pool_pages - free));
  if (gap) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this workgroup's pages are in the list
    __syncthreads();
    const uint32_t upto = listed;
    listed = 0;
    for (uint32_t i0 = 0; i0 < upto; i0 += kThreads) {
      const uint32_t i = i0 + threadIdx.x;
      const int page = i < upto ? __hip_atomic_load(a.free_pages + free + i, __ATOMIC_RELAXED,
                                                    __HIP_MEMORY_SCOPE_AGENT)
                                : -1;
      const bool in = static_cast<uint32_t>(page) < static_cast<uint32_t>(a.num_pool_pages);
      // No page moves up, and all of these are read before the first is written.
      const uint32_t to = scan_before(in ? 1 : 0, listed, 0x7fffffffu, s_wave);
      if (in) put_page(a.free_pages + free + to, page);
    }
  }
  for (int r = threadIdx.x; r < a.batch; r += kThreads) {
    int len;
    const int keep = kept(r, len);
    if (keep != len) a.lens[r] = keep;
  }
  if (threadIdx.x == 0) a.state[kStateFree] = free + static_cast<int>(listed);
}

}  // namespace

pkv_status launch_take(const TakeArgs& a, hipStream_t s) {
  const int64_t groups = std::max<int64_t>(1, (int64_t(a.num_tokens) + kTokens - 1) / kTokens);
  hipLaunchKernelGGL(take_kernel, dim3(static_cast<uint32_t>(groups)), dim3(kThreads), 0, s, a);
  return hipGetLastError() == hipSuccess ? PKV_OK : PKV_EHIP;
}

pkv_status launch_release(const ReleaseArgs& a, hipStream_t s) {
  const int64_t most = std::min<int64_t>(a.num_pool_pages, int64_t(a.batch) * a.max_pages);
  const int64_t groups = std::min<int64_t>(64, (most + 2 * kFewPages - 1) / (2 * kFewPages));
  hipLaunchKernelGGL(release_kernel, dim3(static_cast<uint32_t>(std::max<int64_t>(1, groups))),
                     dim3(kThreads), 0, s, a);
  return hipGetLastError() == hipSuccess ? PKV_OK : PKV_EHIP;
}

}  // namespace pkv
