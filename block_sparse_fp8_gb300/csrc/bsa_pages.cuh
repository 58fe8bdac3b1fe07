// Pages for new tokens, and pages given back.
//
// Sequence b holds c_b tokens and gets n_b more: it needs w_b = ceil((c_b + n_b) / ps) - ceil(c_b / ps)
// more pages.  They come from the top of a stack of free pages in the order of the sequences: with
// W_b the sum of w up to b (inclusive), page j of the call is free[count - 1 - j] and sequence b takes
// j in [W_b - w_b, W_b), if W_b <= count.  Giving back walks the same order the other way, so that
// pages taken by a call and given back by the next leave the stack as it was.
//
// Two prefix sums over the sequences and 8 bytes written per new token: nothing but latency for a
// decode step, one CTA then does it all.  With more rows than two a thread, eight CTAs, a cluster, share
// the pages out (each sums up all the lengths for itself), and the rows are written by as many CTAs
// as they fill (fill_kernel), from the lengths and the table that the first kernel has written.
//
// Measured (device time, calls back to back in a graph): 256 sequences of a token or none each, assigned
// and released, 8.3 us for the two calls; 64 prompts of 0.7-16K tokens (562K rows, 8.8K pages),
// assigned and released, 12.1 us, 20.2 with one CTA for the pages, of which the rows' 4.5 MB are
// 0.7 us at the copy rate: launches, and chains of dependent reads.
#pragma once

#include <cstdint>

#include "bsa_common.cuh"
#include "bsa_decode.cuh"

namespace bsa {
namespace pages {

constexpr int THREADS = 1024;
constexpr int WARPS = THREADS / 32;
constexpr unsigned CLUSTER = 8;   // CTAs of a call with many pages to move
constexpr int FEW_PAGES = 2 * THREADS, FEW_ROWS = 2 * THREADS;  // ... and what one CTA does as well
constexpr int AT_ONCE = 4;  // pages in flight per thread
constexpr int FILL_THREADS = 256;
constexpr int FILL_ROWS = 4 * FILL_THREADS;  // of a CTA

struct Params {
  const int *new_lens, *cache_seqlens;
  int *block_table;
  int *free_pages, *free_count;
  int *cu_seqlens, *seqused_kv, *positions, *slot_map;
  const int *seq_lens, *keep_lens;  // release
  int *lens_out;
  int *dev_status;
  int B, ps_shift, num_pages, L, total;
  int fill;  // the token rows as well
};

__device__ __forceinline__ void report(const Params &p, int bits) {
  if (p.dev_status) atomicOr(p.dev_status, bits);
}

// The CTAs of the call are one cluster: each sums up all the lengths for itself and takes its share of
// the pages and rows; what one of them changes that the others read waits for the cluster's barrier.
__device__ __forceinline__ int cluster_rank() {
  int r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ int cluster_size() {
  int r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

// Inclusive sums of (a, b) over the CTA's threads, and the totals; a barrier before the next call.
__device__ __forceinline__ void scan2(long long &a, long long &b, long long &all_a,
                                      long long &all_b) {
  __shared__ long long s_a[WARPS], s_b[WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) {
      a += x;
      b += y;
    }
  }
  if (lane == 31) {
    s_a[warp] = a;
    s_b[warp] = b;
  }
  __syncthreads();
  long long x = s_a[lane], y = s_b[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += u;
      y += v;
    }
  }
  if (warp > 0) {
    a += __shfl_sync(0xffffffffu, x, warp - 1);
    b += __shfl_sync(0xffffffffu, y, warp - 1);
  }
  all_a = __shfl_sync(0xffffffffu, x, 31);
  all_b = __shfl_sync(0xffffffffu, y, 31);
}

// The last i in [lo, hi] with first[i] <= x (first[lo] <= x).
template <typename T>
__device__ __forceinline__ int last_at_most(const T *first, int lo, int hi, T x) {
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Position and slot of token row `row` of sequence b, whose rows begin at `first`.
__device__ __forceinline__ int2 token(const Params &p, int b, int row, int first, int cached,
                                      int used) {
  const int i = row - first, pos = (int)((unsigned)cached + (unsigned)i);
  int slot = -1;
  if (pos >= 0 && pos < used) {  // the sequence was served
    const int page = p.block_table[(size_t)b * p.L + (pos >> p.ps_shift)];
    if (page >= 0 && page < p.num_pages)
      slot = (page << p.ps_shift) + (pos & ((1 << p.ps_shift) - 1));
    else
      report(p, BSA_DEV_BAD_PAGE);
  }
  return make_int2(pos, slot);
}

__global__ void __launch_bounds__(THREADS) assign_kernel(const Params p) {
  // of the THREADS sequences at hand: first new page and first token row, tokens held before and after
  __shared__ long long s_page[THREADS];
  __shared__ int s_row[THREADS], s_old[THREADS], s_used[THREADS], s_take[THREADS], s_popped;
  const int tid = threadIdx.x;
  const int ps_mask = (1 << p.ps_shift) - 1;
  const long long room = (long long)p.L << p.ps_shift;
  const int rank = cluster_rank(), all_threads = cluster_size() * THREADS;
  decode::pdl_wait();
  decode::pdl_launch_dependents();
  const int count = min(max(*p.free_count, 0), p.num_pages);
  long long rows = 0, taken = 0;  // of the sequences before these
  if (tid == 0) {
    if (rank == 0) p.cu_seqlens[0] = 0;
    s_popped = 0;
  }
  __syncthreads();
  for (int b0 = 0; b0 < p.B; b0 += THREADS) {
    const int b = b0 + tid;
    int n = 0, old = 0;
    long long want = 0;
    bool good = true;
    if (b < p.B) {
      n = p.new_lens[b];
      old = p.cache_seqlens[b];
      good = n >= 0 && old >= 0 && (long long)old + n <= room;
      n = max(n, 0);
      if (good) want = (((long long)old + n + ps_mask) >> p.ps_shift) - (((long long)old + ps_mask) >> p.ps_shift);
    }
    long long row_end = n, page_end = want, all_rows, all_pages;
    scan2(row_end, page_end, all_rows, all_pages);
    row_end += rows;
    page_end += taken;
    if (b < p.B) {
      // rows beyond the buffers have no place: their sequence gets none
      if (row_end > p.total) good = false;
      const bool some = page_end <= count;
      if (!good) report(p, BSA_DEV_BAD_SEQLEN);
      else if (want > 0 && !some) report(p, BSA_DEV_NO_PAGES);
      const bool served = good && (want == 0 || some);
      const int used = served ? old + n : max(old, 0);
      if (rank == 0) {
        p.cu_seqlens[b + 1] = (int)min(row_end, (long long)p.total);
        p.seqused_kv[b] = used;
      }
      s_page[tid] = page_end - want;
      s_row[tid] = (int)min(row_end - n, (long long)p.total);
      s_old[tid] = old;
      s_used[tid] = used;
      s_take[tid] = served ? (int)want : 0;
      // (who wants pages is served up to some sequence and not beyond it: what is taken is a prefix)
      if (served && want > 0) atomicMax(&s_popped, (int)page_end);
    }
    const int here = min(p.B - b0, THREADS);
    __syncthreads();
    // the pages of these sequences, a thread a page, some of them at once
    const long long last = min(taken + all_pages, (long long)count);
    for (long long j0 = taken + rank * THREADS + tid; j0 < last; j0 += all_threads * AT_ONCE) {
      int page[AT_ONCE], at[AT_ONCE];
#pragma unroll
      for (int u = 0; u < AT_ONCE; ++u) {
        const long long j = j0 + u * all_threads;
        page[u] = j < last ? p.free_pages[count - 1 - (int)j] : 0;
        at[u] = j < last ? last_at_most(s_page, 0, here - 1, j) : -1;
      }
#pragma unroll
      for (int u = 0; u < AT_ONCE; ++u) {
        if (at[u] < 0) continue;
        const int k = (int)(j0 + u * all_threads - s_page[at[u]]);
        if (k >= s_take[at[u]]) continue;  // not served after all
        if (page[u] < 0 || page[u] >= p.num_pages) report(p, BSA_DEV_BAD_PAGE);
        const long long col = (((long long)s_old[at[u]] + ps_mask) >> p.ps_shift) + k;
        p.block_table[(size_t)(b0 + at[u]) * p.L + col] = page[u];
      }
    }
    cluster_barrier();  // (a barrier of the CTA as well)
    if (p.fill) {
      const int r1 = (int)min(rows + all_rows, (long long)p.total);
      for (int r = (int)min(rows, (long long)p.total) + rank * THREADS + tid; r < r1;
           r += all_threads) {
        const int i = last_at_most(s_row, 0, here - 1, r);
        const int2 at = token(p, b0 + i, r, s_row[i], s_old[i], s_used[i]);
        p.positions[r] = at.x;
        p.slot_map[r] = at.y;
      }
      __syncthreads();
    }
    rows += all_rows;
    taken += all_pages;
  }
  if (p.B == 0) cluster_barrier();  // every CTA has read the count
  if (rank == 0 && tid == 0) *p.free_count = count - s_popped;
  if (p.fill)
    for (long long r = min(rows, (long long)p.total) + rank * THREADS + tid; r < p.total;
         r += all_threads) {
      p.positions[r] = 0;
      p.slot_map[r] = -1;
    }
}

// The token rows, once the lengths and the table are there.
__global__ void __launch_bounds__(FILL_THREADS) fill_kernel(const Params p) {
  __shared__ int s_seq[2];
  const int tid = threadIdx.x;
  const long long r0 = (long long)blockIdx.x * FILL_ROWS;
  decode::pdl_wait();
  decode::pdl_launch_dependents();
  const int rows = p.cu_seqlens[p.B];
  if (tid < 2 && r0 < rows)  // the sequences of the CTA's first and last row
    s_seq[tid] = last_at_most(p.cu_seqlens, 0, p.B - 1,
                              tid == 0 ? (int)r0 : (int)min(r0 + FILL_ROWS, (long long)rows) - 1);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < FILL_ROWS / FILL_THREADS; ++i) {
    const long long r = r0 + i * FILL_THREADS + tid;
    if (r >= p.total) break;
    int2 at = make_int2(0, -1);
    if (r < rows) {
      const int b = last_at_most(p.cu_seqlens, s_seq[0], s_seq[1], (int)r);
      at = token(p, b, (int)r, p.cu_seqlens[b], p.cache_seqlens[b], p.seqused_kv[b]);
    }
    p.positions[r] = at.x;
    p.slot_map[r] = at.y;
  }
}

// Tokens beyond keep_lens given up, and the pages that hold none any more put on the stack.
__global__ void __launch_bounds__(THREADS) release_kernel(const Params p) {
  __shared__ long long s_page[THREADS];
  __shared__ int s_col[THREADS];
  const int tid = threadIdx.x;
  const int ps_mask = (1 << p.ps_shift) - 1;
  const long long room = (long long)p.L << p.ps_shift;
  const int rank = cluster_rank(), all_threads = cluster_size() * THREADS;
  decode::pdl_wait();
  decode::pdl_launch_dependents();
  const int count = min(max(*p.free_count, 0), p.num_pages);
  // the pages' places on the stack count down from the last one: how many there are comes first, in a
  // pass of its own if one sum does not take in all sequences
  long long total = 0, none = 0;
  for (int pass = p.B <= THREADS ? 1 : 0; pass < 2; ++pass) {
    long long given = 0;
    for (int b0 = 0; b0 < p.B; b0 += THREADS) {
      const int b = b0 + tid;
      long long back = 0;
      int len = 0, keep = 0;
      if (b < p.B) {
        len = p.seq_lens[b];
        keep = min(max(p.keep_lens[b], 0), max(len, 0));
        const bool good = len >= 0 && len <= room;
        if (!good && pass == 1) report(p, BSA_DEV_BAD_SEQLEN);
        if (!good) keep = len;  // left as it is
        else
          back = (((long long)len + ps_mask) >> p.ps_shift) -
                 (((long long)keep + ps_mask) >> p.ps_shift);
      }
      long long end = back, all;
      scan2(end, none, all, none);
      if (pass == 1) {
        s_page[tid] = given + end - back;
        s_col[tid] = (int)(((long long)keep + ps_mask) >> p.ps_shift);
        __syncthreads();
        const int here = min(p.B - b0, THREADS);
        if (p.B <= THREADS) total = all;
        for (long long j0 = given + rank * THREADS + tid; j0 < given + all;
             j0 += all_threads * AT_ONCE) {
          int page[AT_ONCE];
#pragma unroll
          for (int u = 0; u < AT_ONCE; ++u) {
            const long long j = j0 + u * all_threads;
            page[u] = 0;
            if (j < given + all) {
              const int i = last_at_most(s_page, 0, here - 1, j);
              page[u] = p.block_table[(size_t)(b0 + i) * p.L + s_col[i] + (j - s_page[i])];
            }
          }
#pragma unroll
          for (int u = 0; u < AT_ONCE; ++u) {
            const long long j = j0 + u * all_threads, at = count + total - 1 - j;
            if (j >= given + all) continue;
            if (page[u] < 0 || page[u] >= p.num_pages) {
              report(p, BSA_DEV_BAD_PAGE);
              page[u] = -1;
            }
            if (at < p.num_pages) p.free_pages[at] = page[u];
          }
        }
        // (the lengths may be given up in place: every CTA has read these)
        cluster_barrier();
        if (rank == 0 && b < p.B) p.lens_out[b] = keep;
      }
      __syncthreads();
      given += all;
    }
    total = given;
  }
  // more pages than there are: some are held twice
  if (tid == 0 && count + total > p.num_pages) report(p, BSA_DEV_BAD_PAGE);
  if (rank == 0 && tid == 0) *p.free_count = (int)min(count + total, (long long)p.num_pages);
}

}  // namespace pages
}  // namespace bsa
