// Attention of one new token per sequence over the paged e4m3 cache.
//
//   s_j = (q . k_j) * qd * kd_j * softmax_scale * log2(e),  O = vd * sum_j 2^(s_j - m) v_j / l
//
// Bound by HBM: a KV head's token is 256 bytes of codes for 4 * 128 flop per query head, 16 flop
// per byte at eight query heads, a tenth of the ridge.  So everything serves a steady stream of
// loads:
//
//   * Work is cut evenly whatever the batch's lengths are.  Every (sequence, KV head) is a task of
//     128-token tiles; the grid's CTAs (two per SM, resident at once) take equal runs of the
//     batch's tiles in task order, each finding its run by a scan of the lengths.  A task that
//     lies inside one run is finished there; a task cut by run borders leaves one partial (m, l,
//     O in fp32) per run, which the join kernel combines.  No atomics: results do not depend on
//     timing.  Where no sequence has more than WHOLE_TILES tiles and there is a CTA for every
//     task, the runs are whole tasks instead, with nothing to scan and nothing to join.
//   * Within a tile each of the CTA's four warps owns 32 tokens and keeps its own (m, l, O), so
//     warps never wait for one another inside a task.  A warp fetches its own K and V rows, 32 slots
//     of a page each, by TMA (one lane, one instruction each) into a ring STAGES deep.  A bad page is
//     fetched from beyond the pool, which reads as zeros; what lies past a sequence's end is
//     replaced before it is used, so nothing there can reach the result.
//   * The products run on mma.sync m16n8k16 with tokens (K) or dimensions (V) as the 16 rows and
//     up to eight query heads as the 8 columns: with one token per sequence there is no
//     128-row operand for tcgen05.mma to work on, and the tensor pipe is far from its limit.
//     e4m3 codes convert to fp16 exactly, and so do bf16 queries times a power of two per row
//     (values below 2^-28 of the row's largest lose bits).  P goes in as two fp16 terms, the
//     rounded value and what the rounding left, together 2^-22 relative or 2^-40 of the largest
//     weight, whichever is more; one term alone moves one result in fifteen by a bf16 step.
//     Accumulation, maxima and sums are fp32.  A tile's products start from zero and are added to
//     the sums outside: mma.sync cuts off what lies below its accumulator's last bit, some 2^-25
//     of it each time, which pulled a run of 1000 products 2^-15 towards zero.
//   * The 128-byte swizzle (a row's 16-byte chunks XORed with the row number) keeps the fragment
//     reads of K (a thread: 32 dimensions of one token) and V (16 dimensions of one token) free of
//     bank conflicts.
//
// Measured (mean of back-to-back calls, inputs from HBM): 64 sequences of 8-16K tokens, 64/8 heads
// (1655 MB) 245 us, 6.75 TB/s, 99% of the measured copy rate; a bare loop of the same copies reaches
// 6.99 TB/s, which would be 237 us.  The alternatives there, measured in an earlier form of 245 us:
// 16-byte cp.async by all lanes 257 us, three stages 266 us, three CTAs per SM 260 us, one CTA of four
// stages 316 us (more in flight spoils the DRAM's pattern, less does not fill it).  2 x 128K
// tokens, 32/4 heads (268 MB) 47.5 us; 8 x 50-64K at a quarter of the tiles (243 MB) 49.5 us; 16
// ragged sequences (62 MB) 18.4 us; one of 300 tokens 5.3 us: the first tile is done after 4 to 5 us
// (length, page, rows: a chain of reads), the join takes 2.5.  That HBM is the bound holds up to eight
// query heads per KV head.  Sixteen double the products and the softmax, on the same eight warps an SM:
// 16 x 32K tokens, 64/4 heads (545 MB, 80 us at the copy rate) 113 us, 125 us under masks that leave
// each head a quarter of the tiles (and all heads together nearly all): bound by issue and latency.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <cstdint>

#include "bsa_common.cuh"
#include "ptx_sm103.cuh"

namespace bsa {
namespace decode {

constexpr int WARPS = 4;
constexpr int THREADS = WARPS * 32;
constexpr int TOK = TILE / WARPS;  // tokens of a tile that one warp owns: one mma row block pair
constexpr int STAGES = 2;
constexpr int CTAS_PER_SM = 2;
// one warp's stage: K rows, V rows (1024-byte aligned, as the swizzle wants)
constexpr int OFF_V = TOK * HEAD_DIM;
constexpr int STAGE_BYTES = 2 * TOK * HEAD_DIM;
constexpr int SMEM_ALIGN = 1024;
constexpr int SMEM_BYTES = WARPS * STAGES * STAGE_BYTES + SMEM_ALIGN;
// fp16 probabilities are kept as 2^(s - m + P_SHIFT): the largest, 2^15, fits, and weights down to
// 2^-29 of it are normal numbers
constexpr float P_SHIFT = 15.f;
constexpr int MAX_G = 16;
constexpr int WHOLE_TILES = 4;

struct Params {
  const void *q;
  const float *q_descale;
  const uint8_t *k_pages, *v_pages;
  const float *k_descale, *v_descale;
  const int *seqused_kv, *block_table;
  const uint8_t *block_mask;
  const int *sparse_indices, *sparse_seq_len;
  __nv_bfloat16 *out;
  float *lse;
  int *dev_status;
  // workspace: per slot (two per CTA) and head of the group a partial (m, l) and O; with lists, per
  // task {the count of its tiles, the sequence's tokens} and the tiles, ascending, the heads that
  // enable them in the upper half
  float2 *part_ml;
  float *part_o;
  int2 *counts;
  uint32_t *tiles;
  long long q_stride;  // elements
  int B, N1, N2, G, ps, ps_shift, num_pages, L, Kb, max_kv_len;
  int q_e4m3, k_per_token, v_per_head;
  int kv_nhd;
  int whole;  // a run is a task, whatever its length
  float scale_log2;  // softmax_scale * log2(e)
  unsigned long long wait_limit_ns;
};

__device__ __forceinline__ void report(const Params &p, int bits) {
  if (p.dev_status) atomicOr(p.dev_status, bits);
}

// Tokens of sequence b; a bad length counts as none.  Read past L1: the join looks before it has
// waited for the kernel that it joins.
__device__ __forceinline__ int seq_len(const Params &p, int b) {
  const int kv = __ldcg(p.seqused_kv + b);
  if (kv >= 0 && kv <= p.max_kv_len) return kv;  // max_kv_len <= L * ps is checked on the host
  report(p, BSA_DEV_BAD_SEQLEN);
  return 0;
}

// Tiles of a task that takes no part still number one, so that a CTA comes by and writes its
// empty result.
__device__ __forceinline__ int dense_tiles(int kv) { return max((kv + TILE - 1) / TILE, 1); }

__device__ __forceinline__ void pdl_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// The first probe of a barrier: the thread is suspended, up to the limit, while the phase is
// incomplete.  A suspension outlasts a limit of some microseconds, so such a one is polled for.
__device__ __forceinline__ bool wait_first(uint64_t *bar, uint32_t parity,
                                           unsigned long long limit_ns) {
  if (limit_ns < 20000) return ptx::mbar_test_wait(bar, parity);
  return ptx::mbar_try_wait_hint(bar, parity,
                                 (uint32_t)min(limit_ns, (unsigned long long)WAIT_LIMIT_NS));
}

// Polls for a phase that the first probe did not see complete, at most limit_ns; false when that
// runs out.
__device__ __noinline__ bool wait_more(uint64_t *bar, uint32_t parity, unsigned long long limit_ns) {
  const unsigned long long t0 = ptx::globaltimer_ns();
  while (!ptx::mbar_test_wait(bar, parity))
    if (ptx::globaltimer_ns() - t0 > limit_ns) return false;
  return true;
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

__device__ __forceinline__ void prefetch_l2(const void *a) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(a));
}
__device__ __forceinline__ void prefetch_l1(const void *a) {
  asm volatile("prefetch.global.L1 [%0];" ::"l"(a));
}

// Four e4m3 codes -> two f16 pairs, exactly.
__device__ __forceinline__ void f16_of_e4m3x4(uint32_t w, uint32_t &lo, uint32_t &hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The 8 x 8 matrix of 16-bit elements held across the warp, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// The two fp16 values of a pair as fp32.
__device__ __forceinline__ float2 f32x2(uint32_t v) {
  __half2 h;
  memcpy(&h, &v, 4);
  return __half22float2(h);
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Head g of (b, kvh)'s result from a warp's (m, l, O), four dimensions a lane, and its LSE.
__device__ __forceinline__ void write_row(const Params &p, int b, int kvh, int g, int lane, float m,
                                          float l, float4 o) {
  const int h = kvh * p.G + g;
  const bool some = l != 0.f;  // a NaN sum is a result, not an empty row
  // (the quotient first: a small descale over a large sum may leave fp32's normal numbers)
  const float vd = !some ? 0.f : p.v_per_head ? p.v_descale[kvh] : p.v_descale[0];
  const float f = 1.f / (some ? l : 1.f);
  if (!some) o = make_float4(0.f, 0.f, 0.f, 0.f);
  const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * f * vd, o.y * f * vd);
  const __nv_bfloat162 hi = __floats2bfloat162_rn(o.z * f * vd, o.w * f * vd);
  uint2 w;
  memcpy(&w.x, &lo, 4);
  memcpy(&w.y, &hi, 4);
  reinterpret_cast<uint2 *>(p.out)[((size_t)b * p.N1 + h) * 32 + lane] = w;
  if (lane == 0 && p.lse)
    p.lse[(size_t)h * p.B + b] =
        some ? (m + log2f(l) - P_SHIFT) * 0.6931471805599453f : -FLT_MAX;
}

// (m, l, O) += a partial of its own maximum.
__device__ __forceinline__ void add_part(float &m, float &l, float4 &o, float2 ml, float4 v) {
  const float mn = fmaxf(m, ml.x), base = mn == -INFINITY ? 0.f : mn;
  const float a = ptx::ex2_approx(m - base), f = ptx::ex2_approx(ml.x - base);
  m = mn;
  l = l * a + f * ml.y;
  o = make_float4(o.x * a + f * v.x, o.y * a + f * v.y, o.z * a + f * v.z, o.w * a + f * v.w);
}

// ------------------------------------------------------------------------------------------
// Tile lists of the sparse forms: one CTA per (sequence, KV head) forms the union of its query
// heads' tiles below the sequence's end, each with a mask of the heads that enable it.  Nothing but
// latency: the lengths, a mask's bytes of all heads and the first entries of all lists are read at
// once (what lies past the end is in the row all the same, and dropped after the length is known).
// ------------------------------------------------------------------------------------------
constexpr int PLAN_WARPS = 16;  // a warp per query head of the group
constexpr int PLAN_THREADS = PLAN_WARPS * 32;
constexpr int PLAN_AHEAD = 8;   // list entries in flight per lane

template <bool MASK>  // block_mask, or sparse_indices
__global__ void __launch_bounds__(PLAN_THREADS, 2) plan_kernel(const Params p) {
  extern __shared__ uint32_t heads[];  // [Kb]
  __shared__ int warp_n[PLAN_WARPS];
  pdl_wait();
  pdl_launch_dependents();
  const int task = blockIdx.x, b = task / p.N2, kvh = task % p.N2;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const size_t first = (size_t)b * p.N1 + (size_t)kvh * p.G;  // the group's first (b, h)
  const bool lists = !MASK && warp < p.G;
  const int *row = p.sparse_indices + (first + warp) * p.Kb;
  int len = lists ? p.sparse_seq_len[first + warp] : 0;
  const int kv = seq_len(p, b);
  int t[PLAN_AHEAD];
#pragma unroll
  for (int u = 0; u < PLAN_AHEAD; ++u)
    t[u] = lists && lane + 32 * u < p.Kb ? row[lane + 32 * u] : 0;
  for (int i = tid; i < p.Kb; i += PLAN_THREADS) {
    uint32_t on = 0;
    if (MASK) {
      const uint8_t *col = p.block_mask + first * p.Kb + i;
      uint8_t byte[MAX_G];
#pragma unroll
      for (int g = 0; g < MAX_G; ++g) byte[g] = g < p.G ? col[g * p.Kb] : 0;  // below 2^16 bytes
#pragma unroll
      for (int g = 0; g < MAX_G; ++g) on |= byte[g] != 0 ? 1u << g : 0u;
    }
    heads[i] = on;
  }
  const int kend = (kv + TILE - 1) / TILE;
  __syncthreads();
  if (!MASK) {
    if (len < 0 || len > p.Kb) {
      if (lane == 0) report(p, BSA_DEV_BAD_INDEX);
      len = len < 0 ? 0 : p.Kb;
    }
    for (int e0 = lane; e0 < len; e0 += 32 * PLAN_AHEAD) {
      if (e0 >= 32 * PLAN_AHEAD) {
#pragma unroll
        for (int u = 0; u < PLAN_AHEAD; ++u) t[u] = e0 + 32 * u < len ? row[e0 + 32 * u] : 0;
      }
#pragma unroll
      for (int u = 0; u < PLAN_AHEAD; ++u) {
        if (e0 + 32 * u >= len) continue;
        if (t[u] < 0 || t[u] >= p.Kb)
          report(p, BSA_DEV_BAD_INDEX);
        else if (t[u] < kend)
          atomicOr(&heads[t[u]], 1u << warp);
      }
    }
    __syncthreads();
  }
  uint32_t *list = p.tiles + (size_t)task * p.Kb;
  int n = 0;
  for (int base = 0; base < kend; base += PLAN_THREADS) {
    const int t = base + tid;
    const uint32_t on = t < kend ? heads[t] : 0u;
    const unsigned bal = __ballot_sync(0xffffffffu, on != 0);
    if (lane == 0) warp_n[warp] = __popc(bal);
    __syncthreads();
    int at = n + __popc(bal & ((1u << lane) - 1u));
#pragma unroll
    for (int w = 0; w < PLAN_WARPS; ++w) {
      if (w < warp) at += warp_n[w];
      n += warp_n[w];
    }
    if (on) list[at] = (uint32_t)t | on << 16;
    __syncthreads();
  }
  if (tid == 0) p.counts[task] = make_int2(n, kv);
}

// Tiles that task's list holds (one for an empty list, as above).  Bounded by the list's room, as the
// walks below are by the batch: lengths that someone changes under a running call spoil its
// results, but lead it nowhere outside its tensors.
__device__ __forceinline__ int listed_tiles(const Params &p, int task, int &kv) {
  const int2 c = __ldcg(p.counts + task);
  kv = c.y;
  return min(max(c.x, 1), p.Kb);
}

// The batch's tiles, in task order, cut into even runs for `grid` CTAs (as many runs as there are
// tiles, if those are fewer).
struct Cut {
  int runs, size, larger;  // runs have `size` tiles, the first `larger` of them one more
  __device__ __forceinline__ int begin(int i) const { return i * size + min(i, larger); }
  __device__ __forceinline__ int of(int x) const {  // the run that holds tile x
    const int edge = larger * (size + 1);
    return x < edge ? x / (size + 1) : larger + (x - edge) / size;
  }
};

// Finds the cut, and the item in which a wanted tile lies.  Items are sequences, all of whose KV heads
// have the same tiles, or tasks when every task has a list of its own.  want(cut) names the tile, or
// is negative: none wanted, the item is -1.  With by_item the item is given instead and its first
// tile is returned.  Called by all of a CTA's warps; every thread sums a stretch of the items.
struct Found {
  int item, off;  // the item, the wanted tile's offset in it (by_item: the item's first tile)
  int kv;         // the tokens of the item's sequence
};

constexpr int MAX_WARPS = 8;

template <bool SPARSE, typename Want>
__device__ __forceinline__ Found find_tile(const Params &p, int grid, int threads, Cut &cut,
                                           bool by_item, Want &&want) {
  __shared__ int s_sum[MAX_WARPS], s_item, s_off, s_kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int items = SPARSE ? p.B * p.N2 : p.B;
  const int per = (items + threads - 1) / threads, i0 = min(tid * per, items),
            i1 = min(i0 + per, items);
  int kv = 0;  // of the item looked at last
  const auto tiles = [&](int i) {
    if (SPARSE) return listed_tiles(p, i, kv);
    kv = seq_len(p, i);
    return p.N2 * dense_tiles(kv);
  };
  int sum = 0;
  for (int i = i0; i < i1; ++i) sum += tiles(i);
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_sum[warp] = incl;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < MAX_WARPS; ++w) {
    if (w >= threads / 32) break;
    if (w < warp) incl += s_sum[w];
    total += s_sum[w];
  }
  cut.runs = min(grid, total);
  cut.size = total / cut.runs;
  cut.larger = total - cut.runs * cut.size;
  const int x = want(cut);
  if (x < 0) return Found{-1, 0, 0};
  int before = incl - sum, i = i0;
  if (by_item ? x >= i0 && x < i1 : x >= before && x < incl) {
    if (per > 1) {  // (a single item has just been looked at)
      for (;; ++i) {
        const int w = tiles(i);
        if (i + 1 >= i1 || (by_item ? i == x : x < before + w)) break;
        before += w;
      }
    }
    s_item = i;
    s_off = by_item ? before : x - before;
    s_kv = kv;
  }
  __syncthreads();
  return Found{s_item, s_off, s_kv};
}

// A position in the batch's run of tiles, moved along by the copying side of a warp.
template <bool SPARSE>
struct Cursor {
  int b, kvh, idx, n, kv;  // task, tile position in it, its tiles, the sequence's tokens
  int pos, heads, page;    // of the current tile: the warp's first token, heads, physical page

  // The current tile's entry and page (the page still unchecked; -1: nothing to read).
  __device__ __forceinline__ void look(const Params &p, int warp) {
    int tile = idx;
    heads = 0xffff;
    if (SPARSE) {
      const size_t task = (size_t)b * p.N2 + kvh;
      const uint32_t e = p.counts[task].x > 0 ? p.tiles[task * p.Kb + idx] : 0u;
      tile = e & 0xffffu;
      heads = e >> 16;
    }
    pos = tile * TILE + warp * TOK;
    page = pos < kv && heads != 0 ? p.block_table[(size_t)b * p.L + (pos >> p.ps_shift)] : -1;
  }
  __device__ __forceinline__ void next(const Params &p, int warp) {
    if (++idx == n) {
      idx = 0;
      if (++kvh == p.N2) {
        kvh = 0;
        b = min(b + 1, p.B - 1);
        if (!SPARSE) kv = seq_len(p, b);
      }
      n = SPARSE ? listed_tiles(p, b * p.N2 + kvh, kv) : dense_tiles(kv);
    }
    look(p, warp);
  }
};

template <int NT, bool SPARSE>  // NT: blocks of eight query heads per KV head
__global__ void __launch_bounds__(THREADS, CTAS_PER_SM)
    decode_kernel(const Params p, const __grid_constant__ CUtensorMap tk,
                  const __grid_constant__ CUtensorMap tv) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ float2 s_ml[WARPS][MAX_G];
  __shared__ __align__(16) float s_kd[WARPS][STAGES][TOK];
  // {heads, tokens left, last tile of its task (1) and of the run (2), page bad}
  __shared__ __align__(16) int4 s_meta[WARPS][STAGES];
  __shared__ uint64_t s_full[WARPS][STAGES];
  uint8_t *const smem = smem_raw + (-ptx::smem_u32(smem_raw) & (SMEM_ALIGN - 1));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = lane >> 2, q4 = lane & 3;  // mma fragment coordinates
  if (lane == 0) {
    for (int i = 0; i < STAGES; ++i) ptx::mbar_init(&s_full[warp][i], 1);
    ptx::fence_mbarrier_init();
    if (warp == 0 && p.Kb > 0) {
      ptx::prefetch_tmap(&tk);
      ptx::prefetch_tmap(&tv);
    }
  }
  __syncwarp();
  if (SPARSE) {
    // while the lists are being made: the queries and the block table into L2, a line a thread
    const size_t line = ((size_t)blockIdx.x * THREADS + tid) * 128;
    const size_t q_end = (size_t)(p.B - 1) * p.q_stride + (size_t)p.N1 * HEAD_DIM;  // elements
    if (line < q_end * (p.q_e4m3 ? 1 : 2)) prefetch_l2(static_cast<const uint8_t *>(p.q) + line);
    if (line < (size_t)p.B * p.L * 4)
      prefetch_l2(reinterpret_cast<const uint8_t *>(p.block_table) + line);
  }
  pdl_wait();               // what the stream ran before: the tile lists among it
  pdl_launch_dependents();  // the join, which reads the lengths and counts as well: only now

  // this CTA's run: its first tile's place, and the tiles left of it
  const int cta = blockIdx.x;
  int tiles_left;
  Cursor<SPARSE> cur;
  if (p.whole) {  // the grid has a CTA for every task
    cur.b = cta / p.N2;
    cur.kvh = cta % p.N2;
    cur.idx = 0;
    if (!SPARSE) cur.kv = seq_len(p, cur.b);
    cur.n = SPARSE ? listed_tiles(p, cta, cur.kv) : dense_tiles(cur.kv);
    tiles_left = cur.n;
  } else {
    Cut cut;
    const Found at = find_tile<SPARSE>(p, (int)gridDim.x, THREADS, cut, false, [&](const Cut &c) {
      return cta < c.runs ? c.begin(cta) : -1;
    });
    if (at.item < 0) return;
    tiles_left = cut.begin(cta + 1) - cut.begin(cta);
    cur.b = SPARSE ? at.item / p.N2 : at.item;
    cur.kv = at.kv;
    if (SPARSE) cur.kvh = at.item % p.N2;
    cur.n = SPARSE ? listed_tiles(p, at.item, cur.kv) : dense_tiles(cur.kv);
    if (!SPARSE) cur.kvh = min(at.off / cur.n, p.N2 - 1);
    cur.idx = SPARSE ? min(at.off, cur.n - 1) : at.off % cur.n;
  }
  int b = cur.b, kvh = cur.kvh;      // the computing side's task
  bool from_start = cur.idx == 0;    // the segment begins its task
  // ---- the group's queries as B fragments: column r is head r, a thread's 32 dimensions
  // 32 q4 .. 32 q4 + 31 in steps of four (the order of K's reads below).  Fetched raw first (16
  // words of bf16, or 8 of e4m3), converted once the copies in flight are on their way.
  uint32_t qf[NT][16];
  float fac[NT][2];  // score factors of the thread's columns 2 q4, 2 q4 + 1
  float qd[NT];
  const auto fetch_q = [&](int qb, int qh) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int g = nt * 8 + r;
      qd[nt] = 1.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) qf[nt][i] = 0u;
      if (g >= p.G) continue;
      const size_t at = (size_t)qb * p.q_stride + (size_t)(qh * p.G + g) * HEAD_DIM + q4 * 32;
      const uint4 *src = p.q_e4m3 ? reinterpret_cast<const uint4 *>(
                                        static_cast<const uint8_t *>(p.q) + at)
                                  : reinterpret_cast<const uint4 *>(
                                        static_cast<const __nv_bfloat16 *>(p.q) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i >= 2 && p.q_e4m3) break;
        const uint4 v = src[i];
        qf[nt][4 * i] = v.x;
        qf[nt][4 * i + 1] = v.y;
        qf[nt][4 * i + 2] = v.z;
        qf[nt][4 * i + 3] = v.w;
      }
      if (p.q_e4m3) qd[nt] = p.q_descale[(size_t)qb * p.N1 + qh * p.G + g];
    }
  };
  const auto convert_q = [&]() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float f = p.scale_log2;
      if (p.q_e4m3) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = qf[nt][i];
#pragma unroll
        for (int i = 0; i < 8; ++i) f16_of_e4m3x4(w[i], qf[nt][2 * i], qf[nt][2 * i + 1]);
        f *= qd[nt];
      } else {
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(qf[nt][i] << 16)),
                                   fabsf(__uint_as_float(qf[nt][i] & 0xffff0000u))));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // times 2^(14 - e), e the exponent of the row's largest value: it lands in
        // [2^14, 2^15), and only values below 2^-28 of it lose bits to fp16's subnormals
        const int e = max((int)(__float_as_uint(amax) >> 23) - 127, -110);
        const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
        f *= __uint_as_float((uint32_t)(127 + e - 14) << 23);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          qf[nt][i] = f16x2(__uint_as_float(qf[nt][i] << 16) * up,
                            __uint_as_float(qf[nt][i] & 0xffff0000u) * up);
      }
      fac[nt][0] = __shfl_sync(0xffffffffu, f, 8 * q4);
      fac[nt][1] = __shfl_sync(0xffffffffu, f, 8 * q4 + 4);
    }
  };

  fetch_q(b, kvh);
  cur.look(p, warp);

  const uint32_t ring = ptx::smem_u32(smem) + warp * STAGES * STAGE_BYTES;
  uint32_t phases = 0, in_flight = 0;  // a bit a stage

  const int q_size = p.q_e4m3 ? 1 : 2, q_lines = p.G * q_size;  // 128-byte lines of a group
  const auto q_row = [&](int qb, int qh) {
    return static_cast<const uint8_t *>(p.q) +
           ((size_t)qb * p.q_stride + (size_t)qh * p.G * HEAD_DIM) * q_size;
  };

  const auto issue = [&](int stage) {
    if (tiles_left == 0) return;
    const int left = cur.heads != 0 ? cur.kv - cur.pos : 0;
    const bool bad = cur.page < 0 || cur.page >= p.num_pages;
    const bool last = cur.idx + 1 == cur.n, end = tiles_left == 1;
    if (left > 0) in_flight |= 1u << stage;
    if (lane == 0) {
      s_meta[warp][stage] = make_int4(cur.heads, left, (last ? 1 : 0) | (end ? 2 : 0), bad);
      if (left > 0) {
        if (bad) report(p, BSA_DEV_BAD_PAGE);
        const int page = bad ? p.num_pages : cur.page, slot = cur.pos & (p.ps - 1);
        const int c1 = p.kv_nhd ? cur.kvh : slot, c2 = p.kv_nhd ? slot : cur.kvh;
        const bool kd = p.k_per_token && !bad;
        uint64_t *bar = &s_full[warp][stage];
        uint8_t *dst = smem + (warp * STAGES + stage) * STAGE_BYTES;
        ptx::mbar_arrive_expect_tx(bar, STAGE_BYTES + (kd ? TOK * 4 : 0));
        ptx::tma_load_4d(dst, &tk, bar, 0, c1, c2, page);
        ptx::tma_load_4d(dst + OFF_V, &tv, bar, 0, c1, c2, page);
        if (kd)
          ptx::bulk_load(s_kd[warp][stage],
                         p.k_descale + ((size_t)page * p.N2 + cur.kvh) * p.ps + slot, TOK * 4,
                         bar);
      }
    }
    if (--tiles_left > 0) {
      cur.next(p, warp);
      // the next task's queries, wanted when the computing side gets there
      if (cur.idx == 0 && lane < q_lines) prefetch_l1(q_row(cur.b, cur.kvh) + lane * 128);
    }
  };

#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) issue(s);

  float m[NT][2], l[NT][2], acc[NT][8][4];
  const auto reset = [&]() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[nt][i][c] = 0.f;
    }
  };

  // ---- one warp's 32 tokens of a tile
  const float kd_all = p.k_per_token || !p.k_descale ? 1.f : p.k_descale[0];
  const int group = (1 << p.G) - 1;
  const auto compute = [&](uint32_t st, const float *kds, int heads, int left, bool bad) {
    float s[NT][2][4];  // [head block][16 tokens][token r | r + 8, head 2 q4 | + 1]
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[nt][mt][c] = 0.f;
      const uint32_t row = st + (mt * 16 + r) * HEAD_DIM;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t chunk = ((2 * q4 + i) ^ r) << 4;
        const uint4 a = lds128(row + chunk), c = lds128(row + 8 * HEAD_DIM + chunk);
        const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wc[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t a0, a1, a2, a3;
          f16_of_e4m3x4(wa[w], a0, a2);
          f16_of_e4m3x4(wc[w], a1, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816(s[nt][mt], a0, a1, a2, a3, qf[nt][2 * (4 * i + w)],
                     qf[nt][2 * (4 * i + w) + 1]);
        }
      }
    }
    // scores, masked; a masked value is replaced, never multiplied
    const bool whole = left >= TOK && (!SPARSE || heads == group) && !bad;
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int t = mt * 16 + half * 8 + r;
        const float kd = p.k_per_token ? kds[t] : kd_all;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float &x = s[nt][mt][2 * half + c];
            x *= kd * fac[nt][c];
            if (!whole) {
              if (bad) x = 0.f;  // no descale was fetched
              if (t >= left || (SPARSE && !((heads >> (nt * 8 + 2 * q4 + c)) & 1))) x = -INFINITY;
            }
          }
      }
    }
    // P as B fragments: [16 tokens][rounded, rest][tokens 2 q4 | 2 q4 + 8, head r]
    uint32_t pf[NT][2][2][2];
    float alpha[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float ref[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float mx = fmaxf(fmaxf(s[nt][0][c], s[nt][0][2 + c]), fmaxf(s[nt][1][c], s[nt][1][2 + c]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        const float mn = fmaxf(m[nt][c], mx);
        const float base = mn == -INFINITY ? 0.f : mn;
        alpha[nt][c] = ptx::ex2_approx(m[nt][c] - base);
        m[nt][c] = mn;
        // rounded up: beyond 2^24 the nearest number may lie 16 below, where the largest weight,
        // 2^16, is no fp16 number (the shift is then less than 15, scores are whole numbers)
        ref[c] = __fadd_ru(base, -P_SHIFT);
      }
      float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        float e[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) e[c] = ptx::ex2_approx(s[nt][mt][c] - ref[c & 1]);
        sum0 += e[0] + e[2];
        sum1 += e[1] + e[3];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t hi = f16x2(e[2 * half], e[2 * half + 1]);
          const float2 x = f32x2(hi);
          pf[nt][mt][0][half] = transpose8x8(hi);
          pf[nt][mt][1][half] =
              transpose8x8(f16x2(e[2 * half] - x.x, e[2 * half + 1] - x.y));
        }
      }
      l[nt][0] = l[nt][0] * alpha[nt][0] + sum0;
      l[nt][1] = l[nt][1] * alpha[nt][1] + sum1;
    }
    // With `masked` the columns of heads that mask the tile keep their sums: their weights are zero,
    // but zero times a NaN of the tile's V would reach them through the shared product.
    const auto pv = [&](const bool masked) {
      uint4 v[2][4];  // [16 tokens][tokens 2 q4, 2 q4 + 1 and those + 8], dimensions 16 r .. 16 r + 15
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const uint32_t t0 = st + OFF_V + (mt * 16 + 2 * q4) * HEAD_DIM;
        const uint32_t c0 = (r ^ (2 * q4)) << 4, c1 = (r ^ (2 * q4 + 1)) << 4;
        v[mt][0] = lds128(t0 + c0);
        v[mt][1] = lds128(t0 + HEAD_DIM + c1);
        v[mt][2] = lds128(t0 + 8 * HEAD_DIM + c0);
        v[mt][3] = lds128(t0 + 9 * HEAD_DIM + c1);
        if (left < TOK) {  // whatever lies past the end, NaN codes too, counts as zero
          const int t = mt * 16 + 2 * q4;
          const uint4 zero = make_uint4(0, 0, 0, 0);
          if (t >= left) v[mt][0] = zero;
          if (t + 1 >= left) v[mt][1] = zero;
          if (t + 8 >= left) v[mt][2] = zero;
          if (t + 9 >= left) v[mt][3] = zero;
        }
      }
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        float o[2][NT][4] = {};
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          uint32_t x[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            x[k] = w == 0 ? v[mt][k].x : w == 1 ? v[mt][k].y : w == 2 ? v[mt][k].z : v[mt][k].w;
          // bytes of two tokens interleaved: a fragment pairs tokens within a dimension
          uint32_t a[2][4];
          f16_of_e4m3x4(__byte_perm(x[0], x[1], 0x5140), a[0][0], a[0][1]);
          f16_of_e4m3x4(__byte_perm(x[0], x[1], 0x7362), a[1][0], a[1][1]);
          f16_of_e4m3x4(__byte_perm(x[2], x[3], 0x5140), a[0][2], a[0][3]);
          f16_of_e4m3x4(__byte_perm(x[2], x[3], 0x7362), a[1][2], a[1][3]);
#pragma unroll
          for (int part = 1; part >= 0; --part)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma16816(o[i][nt], a[i][0], a[i][1], a[i][2], a[i][3], pf[nt][mt][part][0],
                         pf[nt][mt][part][1]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (!masked || ((heads >> (nt * 8 + 2 * q4 + (c & 1))) & 1))
                acc[nt][2 * w + i][c] = fmaf(acc[nt][2 * w + i][c], alpha[nt][c & 1], o[i][nt][c]);
      }
    };
    if (!SPARSE || heads == group)
      pv(false);
    else
      pv(true);
  };

  // ---- the end of a segment: the four warps' states combined; written out when the segment is
  // its whole task, left as a partial otherwise.  O goes through the stage just consumed, the one
  // that the next copy will overwrite.
  bool first_segment = true;
  const auto flush = [&](int stage, bool to_end) {
    const uint32_t buf = ring + stage * STAGE_BYTES;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float t = l[nt][c];
        t += __shfl_xor_sync(0xffffffffu, t, 4);
        t += __shfl_xor_sync(0xffffffffu, t, 8);
        t += __shfl_xor_sync(0xffffffffu, t, 16);
        const int g = nt * 8 + 2 * q4 + c;
        if (r == 0) s_ml[warp][g] = make_float2(m[nt][c], t);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                           buf + g * (HEAD_DIM * 4) + (((4 * r + k) ^ q4) << 4)),
                       "f"(acc[nt][2 * k][c]), "f"(acc[nt][2 * k][2 + c]),
                       "f"(acc[nt][2 * k + 1][c]), "f"(acc[nt][2 * k + 1][2 + c])
                       : "memory");
      }
    __syncthreads();
    const bool complete = from_start && to_end;
    const size_t slot = 2 * (size_t)cta + (first_segment ? 0 : 1);
    const uint8_t *o0 = smem + stage * STAGE_BYTES;
#pragma unroll 2
    for (int g = warp; g < p.G; g += WARPS) {  // a head a warp, four dimensions a lane
      float mm = -INFINITY, ll = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WARPS; ++w)
        add_part(mm, ll, o, s_ml[w][g],
                 *reinterpret_cast<const float4 *>(o0 + w * STAGES * STAGE_BYTES +
                                                   g * (HEAD_DIM * 4) +
                                                   ((lane ^ ((g >> 1) & 3)) << 4)));
      if (complete) {
        write_row(p, b, kvh, g, lane, mm, ll, o);
      } else {
        if (lane == 0) p.part_ml[slot * MAX_G + g] = make_float2(mm, ll);
        reinterpret_cast<float4 *>(p.part_o)[(slot * p.G + g) * 32 + lane] = o;
      }
    }
    // the stage's next contents come through the async proxy
    ptx::fence_proxy_async_smem();
    __syncthreads();
  };

  convert_q();
  reset();
  int stage = 0;
  for (;;) {
    __syncwarp();  // the stage before this one has been read by every lane, and is refilled
    issue(stage == 0 ? STAGES - 1 : stage - 1);
    const int4 meta = s_meta[warp][stage];
    const int heads = meta.x, left = meta.y;
    const bool last = meta.z & 1, end = meta.z & 2;
    if (left > 0) {
      uint64_t *bar = &s_full[warp][stage];
      const uint32_t parity = (phases >> stage) & 1u;
      bool ok = __all_sync(0xffffffffu, wait_first(bar, parity, p.wait_limit_ns));
      if (!ok) ok = __all_sync(0xffffffffu, wait_more(bar, parity, p.wait_limit_ns));
      if (!ok) {
        // out of time: report, see the copies in flight land (with the default limit), leave
        if (lane == 0) report(p, BSA_DEV_TIMEOUT);
        for (int i = 0; i < STAGES; ++i)
          if ((in_flight >> i) & 1u)
            wait_more(&s_full[warp][i], (phases >> i) & 1u, WAIT_LIMIT_NS);
        return;
      }
      phases ^= 1u << stage;
      in_flight &= ~(1u << stage);
      compute(ring + stage * STAGE_BYTES, s_kd[warp][stage], heads, left, meta.w != 0);
    }
    if (last || end) {
      flush(stage, last);
      if (end) return;
      first_segment = false;
      from_start = true;
      if (++kvh == p.N2) {
        kvh = 0;
        b = min(b + 1, p.B - 1);
      }
      fetch_q(b, kvh);
      convert_q();
      reset();
    }
    stage = stage == STAGES - 1 ? 0 : stage + 1;
  }
}

// ------------------------------------------------------------------------------------------
// The join of the cut tasks.  A task's partials are its first run's last slot and the first slots of
// the runs that follow, up to the one that holds its last tile.  Launched while the attention kernel
// runs: the blocks find their partials in that kernel's shadow, in the registers it leaves free (up
// to eight heads per KV head; the kernels for more leave none), and then wait for its writes.
// With fewer tasks than runs (`by_task`) a task has many partials: a block joins one head of one task,
// its warps sharing the partials out.  Otherwise most cut tasks have two or three, but a long
// sequence among short ones may have one in every run, so a task is joined by the blocks of the
// runs that it leaves unfinished, as many as there are heads: they deal the heads out among them, a
// head a warp, or, with more partials than a warp reads at once, a head a block, whose warps
// share the partials out (one sequence of 512K tokens among 319 of 500, one KV head, 8 query heads: 48
// us, with all heads in the first run's block 92).
// ------------------------------------------------------------------------------------------
constexpr int JOIN_AHEAD = 5;  // partials in flight per warp

template <bool SPARSE>
__global__ void __launch_bounds__(MAX_WARPS * 32) join_kernel(const Params p, bool by_task,
                                                              int grid) {
  __shared__ float2 s_ml[MAX_WARPS];
  __shared__ float4 s_o[MAX_WARPS][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const int index = blockIdx.x;
  Cut cut;
  const Found at = find_tile<SPARSE>(p, grid, (int)blockDim.x, cut, by_task, [&](const Cut &c) {
    return by_task ? (SPARSE ? index : index / p.N2) : index < c.runs ? c.begin(index + 1) - 1 : -1;
  });
  if (at.item < 0) return;  // (never block 0)
  int kv = at.kv;
  const int n = SPARSE ? listed_tiles(p, at.item, kv) : dense_tiles(kv);
  int task, t0;  // the task and its first tile
  if (by_task) {
    task = index;
    t0 = at.off + (SPARSE ? 0 : index % p.N2 * n);
  } else {
    task = SPARSE ? at.item : at.item * p.N2 + min(at.off / n, p.N2 - 1);
    t0 = max(cut.begin(index + 1) - 1 - (SPARSE ? min(at.off, n - 1) : at.off % n), 0);
  }
  const int c = min(cut.of(t0), cut.runs - 1);
  const int parts = min(cut.of(t0 + n - 1), cut.runs - 1) - c + 1;
  // the blocks of one task, and this one's number among them; the run with the task's last tile is
  // not asked: it may begin the next cut task
  const int blocks = by_task ? p.G : min(parts - 1, p.G);
  const int block = by_task ? (int)blockIdx.y : index - c;
  if (parts <= 1 || block >= blocks) {  // not cut, or enough others
    // one block always waits, so that the join never ends before the kernel it belongs to
    if (index == 0 && blockIdx.y == 0) pdl_wait();
    return;
  }
  const int first = 2 * c + (t0 > cut.begin(c) ? 1 : 0);  // after a finished segment: the second slot
  const int b = task / p.N2, kvh = task % p.N2;
  pdl_wait();

  const bool together = by_task || parts > JOIN_AHEAD;  // a block's warps share a head's partials
  const int j0 = together ? warp : 0, step = together ? warps : 1;
  for (int g = block + (together ? 0 : warp * blocks); g < p.G; g += blocks * (together ? 1 : warps)) {
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = j0; j < parts; j += step * JOIN_AHEAD) {
      float2 ml[JOIN_AHEAD];
      float4 v[JOIN_AHEAD];
#pragma unroll
      for (int u = 0; u < JOIN_AHEAD; ++u) {
        const int ju = j + u * step;
        ml[u] = make_float2(-INFINITY, 0.f);
        v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (ju < parts) {
          const size_t slot = ju == 0 ? first : 2 * (size_t)(c + ju);
          ml[u] = p.part_ml[slot * MAX_G + g];
          v[u] = reinterpret_cast<const float4 *>(p.part_o)[(slot * p.G + g) * 32 + lane];
        }
      }
#pragma unroll
      for (int u = 0; u < JOIN_AHEAD; ++u) add_part(m, l, o, ml[u], v[u]);
    }
    if (together) {
      s_o[warp][lane] = o;
      if (lane == 0) s_ml[warp] = make_float2(m, l);
      __syncthreads();
      if (warp == 0)
        for (int w = 1; w < warps; ++w) add_part(m, l, o, s_ml[w], s_o[w][lane]);
    }
    if (!together || warp == 0) write_row(p, b, kvh, g, lane, m, l, o);
    if (together) __syncthreads();  // the next head's states go where these were
  }
}

}  // namespace decode
}  // namespace bsa
