// Attention of one new token per sequence over the 4-bit cache (bsa_fp4.cuh): bsa_decode.cuh's cut of the
// work, join, queries and precision, over rows of 64 bytes of e2m1 codes and 8 e4m3 scales.
//
//   s_j = (q . k_j) * qd * kd * softmax_scale * log2(e),  O = vd * sum_j 2^(s_j - m) v_j / l
//
// A KV head's token is 144 bytes against 260 and the work on it the same and more, so HBM is no longer
// the bound: the instructions are.  Every code is converted (e2m1 -> fp16, exactly) and multiplied
// by its block's scale (exactly: two bits times four); 256 conversions and 256 packed products a warp
// for 64 tokens, each of which keeps its pipe for two cycles, and mma.sync, which takes as much of the
// issue as four other instructions.  What is here to spend fewer:
//
//   * A warp owns 64 tokens of a tile (32 in the e4m3 kernel), so that the softmax's reductions, the
//     rescaling of O and the loop are paid half as often (all figures: 64 sequences of 8-16K tokens,
//     64/8 heads, 917 MB, 137 us at the copy rate; mean of back-to-back calls): 259 -> 220 us.
//   * Copies are 16-byte cp.async by all lanes, their places looked up for sixteen tiles at once, a lane
//     a box of 32 tokens: 18 instructions a tile and no barrier to wait at.  TMA by one lane takes
//     fewer copies, but their operands go through uniform registers: 211 -> 189.  They go through
//     L1: past it (.cg) every 32-byte sector is fetched once for either half (303 MB for 151), 174
//     against 164.  L2 is asked for no more than a row's 64 bytes, beside which NHD pages have other
//     heads' rows (2 x 128K tokens, 32/4 heads: 43.8 -> 40.6; HND 35.5 either way).
//   * The score factor is kept above zero (its sign goes into the queries), so that the maximum is
//     taken of the bare products.  A weight is 2^((s - max) * factor + 15): the difference comes before
//     the product, so that the largest score's weight is 2^15 whatever its size (of rounded products
//     beyond 2^24 it is not: the exponent loses the 15, or the score itself lies below its maximum).
//     Differences in pairs, products singly: 164 us, as with one fma for both; both in pairs 166.
//   * P goes in as one fp16 number, 2^-12 of it off (bf16's own rounding of the result is 2^-9): the
//     rest as a second term, as over e4m3 pages, costs 19 us more (183 against 164) for what four bits
//     have long lost; 6 to 8% of the results then lie a bf16 step from the rounded fp64 value (0.1% in
//     plain fp32), 1.7e-3 off in norm like those.
//
// What did not help: twelve warps an SM in place of eight (64 tokens a warp: no room for L1, 233; 32
// tokens: 175), sixteen (201), six (207), three stages (220: no room for L1), products of K side by
// side, fp32 arithmetic in pairs (no change), codes converted by shifts and masks (305 against 259).
//
// Measured: the case above 164 us, 84% of the copy rate; 2 x 128K tokens, 32/4 heads (151 MB) 35.5 us,
// 40.6 in NHD pages; a quarter of the tiles of 8 x 50-64K tokens (118 MB) 37.4 us.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <cstdint>

#include "bsa_common.cuh"
#include "bsa_decode.cuh"
#include "bsa_fp4.cuh"

namespace bsa {
namespace decode4 {

using decode::add_part;
using decode::Cut;
using decode::f16_of_e4m3x4;
using decode::f16x2;
using decode::Found;
using decode::lds128;
using decode::mma16816;
using decode::MAX_G;
using decode::P_SHIFT;
using decode::transpose8x8;

constexpr int WARPS = 2;
constexpr int THREADS = WARPS * 32;
constexpr int TOK = TILE / WARPS;  // tokens of a tile that one warp owns
constexpr int MT = TOK / 16;
constexpr int BOX = 32;            // tokens that are sure to lie in one page
constexpr int BOXES = TOK / BOX;
constexpr int STAGES = 2;
constexpr int CTAS_PER_SM = 4;
constexpr int ROW = fp4::ROW_BYTES;
// one warp's stage: K rows, V rows, K scales, V scales
constexpr int BOX_BYTES = BOX * ROW;
constexpr int OFF_V = TOK * ROW;
constexpr int OFF_KS = 2 * TOK * ROW;
constexpr int SCALE_BYTES = TOK * fp4::BLOCKS;
constexpr int OFF_VS = OFF_KS + SCALE_BYTES;
constexpr int STAGE_BYTES = OFF_VS + SCALE_BYTES;
constexpr int SMEM_BYTES = WARPS * STAGES * STAGE_BYTES;
static_assert(STAGE_BYTES >= MAX_G * HEAD_DIM * 4, "a segment's sums pass through a stage");

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global.L2::64B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copies_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>  // all but the last N groups of copies have landed
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// Two e4m3 codes (the low half word) -> an f16 pair.
__device__ __forceinline__ uint32_t f16_of_e4m3x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}

// Eight e2m1 codes -> four f16 pairs, exactly.
__device__ __forceinline__ void f16_of_e2m1x8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// d = a b, from nothing
__device__ __forceinline__ void mma16816_new(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

template <int NT, bool SPARSE, typename P>  // NT: blocks of eight query heads per KV head
__global__ void __launch_bounds__(THREADS, CTAS_PER_SM) decode_kernel(const P p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float2 s_ml[WARPS][MAX_G];
  // {heads, tokens left, last tile of its task (1) and of the run (2), -}
  __shared__ __align__(16) int4 s_meta[WARPS][STAGES];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = lane >> 2, q4 = lane & 3;  // mma fragment coordinates
  if (SPARSE) {
    // while the lists are being made: the queries and the block table into L2, a line a thread
    const size_t line = ((size_t)blockIdx.x * THREADS + tid) * 128;
    const size_t q_end = (size_t)(decode::rows_of(p) - 1) * p.q_stride + (size_t)p.N1 * HEAD_DIM;  // elements
    if (line < q_end * (p.q_e4m3 ? 1 : 2))
      decode::prefetch_l2(static_cast<const uint8_t *>(p.q) + line);
    if (line < (size_t)p.B * p.L * 4)
      decode::prefetch_l2(reinterpret_cast<const uint8_t *>(p.block_table) + line);
  }
  decode::pdl_wait();               // what the stream ran before: the tile lists among it
  decode::pdl_launch_dependents();  // the join, which reads the lengths and counts as well: only now

  // this CTA's run: its first tile's place (the copying side's), and the tiles left of it
  const int cta = blockIdx.x;
  int tiles_left;
  int c_b, c_kvh, c_idx, c_n, c_kv = 0;
  if (p.whole) {  // the grid has a CTA for every task
    c_b = cta / p.N2;
    c_kvh = cta % p.N2;
    c_idx = 0;
    if (!SPARSE) c_kv = decode::seq_len(p, c_b);
    c_n = SPARSE ? decode::listed_tiles(p, cta, c_kv) : decode::dense_tiles(c_kv);
    tiles_left = c_n;
  } else {
    Cut cut;
    const Found at =
        decode::find_tile<SPARSE>(p, (int)gridDim.x, THREADS, cut, false, [&](const Cut &c) {
          return cta < c.runs ? c.begin(cta) : -1;
        });
    if (at.item < 0) {
      if constexpr (P::PACKED) decode::clear_rows(p);
      return;
    }
    tiles_left = cut.begin(cta + 1) - cut.begin(cta);
    c_b = SPARSE ? at.item / p.N2 : at.item;
    c_kv = at.kv;
    c_n = SPARSE ? decode::listed_tiles(p, at.item, c_kv) : decode::dense_tiles(c_kv);
    c_kvh = SPARSE ? at.item % p.N2 : min(at.off / c_n, p.N2 - 1);
    c_idx = SPARSE ? min(at.off, c_n - 1) : at.off % c_n;
  }
  int b = c_b, kvh = c_kvh;      // the computing side's task
  bool from_start = c_idx == 0;  // the segment begins its task

  // ---- the group's queries as B fragments: column r is head r, a thread's 32 dimensions
  // 32 q4 .. 32 q4 + 31 in steps of four (the order of K's reads below).  Fetched raw first (16
  // words of bf16, or 8 of e4m3), converted once the copies in flight are on their way.
  uint32_t qf[NT][16];
  float fac[NT][2];  // score factors of the thread's columns 2 q4, 2 q4 + 1, above zero
  float qd[NT], kd = 1.f;
  const auto fetch_q = [&](int qb, int qh) {
    if (p.k_descale) kd = p.k_descale[p.k_per_head ? qh : 0];
    const size_t row = decode::row_of(p, qb);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int g = nt * 8 + r;
      qd[nt] = 1.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) qf[nt][i] = 0u;
      if (g >= p.G) continue;
      const size_t at = row * p.q_stride + (size_t)(qh * p.G + g) * HEAD_DIM + q4 * 32;
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
      if (p.q_e4m3) qd[nt] = p.q_descale[row * p.N1 + qh * p.G + g];
    }
  };
  const auto convert_q = [&]() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float f = p.scale_log2 * kd;
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
      // the factor above zero, its sign in the queries: the largest product is then the largest
      // score, and -inf stays -inf (a factor of zero becomes one that leaves no trace in fp32)
      if (f < 0.f) {
#pragma unroll
        for (int i = 0; i < 16; ++i) qf[nt][i] ^= 0x80008000u;
      }
      f = f == 0.f ? 1e-30f : fabsf(f);
      fac[nt][0] = __shfl_sync(0xffffffffu, f, 8 * q4);
      fac[nt][1] = __shfl_sync(0xffffffffu, f, 8 * q4 + 4);
    }
  };

  if constexpr (!P::PACKED) fetch_q(b, kvh);

  const int q_size = p.q_e4m3 ? 1 : 2, q_lines = p.G * q_size;  // 128-byte lines of a group
  const auto prefetch_q = [&](int qb, int qh) {
    if (lane < q_lines)
      decode::prefetch_l1(static_cast<const uint8_t *>(p.q) +
                          ((size_t)decode::row_of(p, qb) * p.q_stride + (size_t)qh * p.G * HEAD_DIM) *
                              q_size +
                          lane * 128);
  };

  // ---- the copying side.  Tiles of one task are looked up a lane a box, as many at once as lanes
  // reach; a tile then costs its copies.
  constexpr int AHEAD = 32 / BOXES;
  int b_heads = 0, b_left = 0, b_page = -1, b_slot = 0;  // of the lane's box; b_left: of its tile
  uint32_t b_row = 0, b_srow = 0;                        // its first row among codes and scales
  int at = 0, n_at = 0;       // tile at hand of those looked up, their number
  int kvh_at = 0;             // their KV head
  bool to_end = false;        // the last of them ends its task
  uint32_t alive = 0;         // boxes whose tile holds tokens
  uint32_t there = 0;         // boxes with something to copy
  int unseen = tiles_left;    // tiles not looked up yet
  const auto look = [&]() {
    n_at = min(min(c_n - c_idx, AHEAD), unseen);
    at = 0;
    unseen -= n_at;
    kvh_at = c_kvh;
    const int i = lane / BOXES, box = lane % BOXES;
    b_left = 0;
    b_page = -1;
    if (i < n_at) {
      int tile = c_idx + i;
      b_heads = 0xffff;
      if (SPARSE) {
        const size_t task = (size_t)c_b * p.N2 + c_kvh;
        const uint32_t e = p.counts[task].x > 0 ? p.tiles[task * p.Kb + tile] : 0u;
        tile = e & 0xffffu;
        b_heads = e >> 16;
      }
      const int pos = tile * TILE + warp * TOK, pos_box = pos + box * BOX;
      b_left = b_heads != 0 ? c_kv - pos : 0;
      b_slot = pos_box & (p.ps - 1);
      if (b_left > box * BOX) b_page = p.block_table[(size_t)c_b * p.L + (pos_box >> p.ps_shift)];
    }
    c_idx += n_at;
    to_end = c_idx == c_n;
    if (to_end && unseen > 0) {
      c_idx = 0;
      if (++c_kvh == p.N2) {
        c_kvh = 0;
        c_b = min(c_b + 1, p.B - 1);
        if (!SPARSE) c_kv = decode::seq_len(p, c_b);
      }
      c_n = SPARSE ? decode::listed_tiles(p, c_b * p.N2 + c_kvh, c_kv) : decode::dense_tiles(c_kv);
      prefetch_q(c_b, c_kvh);  // wanted when the computing side gets there
    }
  };
  // ... and, once the pages have come, are turned into places.  A bad page's rows are zeros.
  const auto looked = [&]() {
    const bool mine = b_left > (lane % BOXES) * BOX, good = b_page >= 0 && b_page < p.num_pages;
    if (mine && !good) decode::report(p, BSA_DEV_BAD_PAGE);
    alive = __ballot_sync(0xffffffffu, b_left > 0);
    there = __ballot_sync(0xffffffffu, mine && good);
    if (!good) b_page = 0;
    b_srow = ((uint32_t)b_page * p.N2 + kvh_at) * p.ps + b_slot;
    b_row = p.kv_nhd ? ((uint32_t)b_page * p.ps + b_slot) * p.N2 + kvh_at : b_srow;
  };

  // a lane's part of a box: 16 bytes of every eighth row.  A row's 16-byte chunks are XORed with half
  // the row's number.
  const uint32_t ring =
      static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * STAGES * STAGE_BYTES;
  const uint32_t step = 8u * (p.kv_nhd ? (uint32_t)p.N2 * ROW : ROW);
  const uint32_t to = r * ROW + ((q4 ^ ((r >> 1) & 3)) << 4);
  const uint8_t *const k_lane = p.k_pages + (size_t)r * (step / 8) + q4 * 16;
  const uint8_t *const v_lane = p.v_pages + (size_t)r * (step / 8) + q4 * 16;
  const uint8_t *const ks_lane = p.k_scales + (lane & 15) * 16;
  const uint8_t *const vs_lane = p.v_scales + (lane & 15) * 16;

  const auto issue = [&](int stage) {
    if (tiles_left > 0) {
      if (at == 0) looked();
      const int first = at * BOXES;
      const bool last = at + 1 == n_at && to_end, end = tiles_left == 1;
      const uint32_t st = ring + stage * STAGE_BYTES;
      if (lane == first)
        s_meta[warp][stage] = make_int4(b_heads, b_left, (last ? 1 : 0) | (end ? 2 : 0), 0);
      if ((alive >> first) & 1u) {
#pragma unroll
        for (int box = 0; box < BOXES; ++box) {
          const uint32_t row = __shfl_sync(0xffffffffu, b_row, first + box);
          const uint32_t bytes = (there >> (first + box)) & 1u ? 16u : 0u;  // none: zeros
          const uint8_t *k = k_lane + (size_t)row * ROW, *v = v_lane + (size_t)row * ROW;
          const uint32_t dst = st + box * BOX_BYTES + to;
#pragma unroll
          for (int i = 0; i < BOX / 8; ++i) {
            copy16(dst + i * 8 * ROW, k + i * step, bytes);
            copy16(dst + OFF_V + i * 8 * ROW, v + i * step, bytes);
          }
        }
        static_assert(BOX * fp4::BLOCKS == 16 * 16 && BOXES == 2, "half a warp has a box's scales");
        const int from = first + (lane >> 4);
        const uint32_t row = __shfl_sync(0xffffffffu, b_srow, from);
        const uint32_t bytes = (there >> from) & 1u ? 16u : 0u;
        copy16(st + OFF_KS + lane * 16, ks_lane + (size_t)row * fp4::BLOCKS, bytes);
        copy16(st + OFF_VS + lane * 16, vs_lane + (size_t)row * fp4::BLOCKS, bytes);
      }
      --tiles_left;
      if (++at == n_at && tiles_left > 0) look();
    }
    copies_close();
  };

  look();
  if constexpr (P::PACKED) fetch_q(b, kvh);  // (a read more in the chain: not in front of the pages')
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) issue(s);
  if constexpr (P::PACKED) decode::clear_rows(p);

  float m[NT][2], l[NT][2], acc[NT][8][4];  // m: of the bare products
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

  // ---- one warp's tokens of a tile.  A product's row i is a token, the eight of a half in the order
  // 0 3 1 2 4 7 5 6: whatever rows a phase of the fragment reads touches, of K (two) or of V
  // (four), lie in different banks.
  constexpr uint32_t ORDER = 0x65742130u;
  const int tok_k = (ORDER >> (4 * r)) & 7;
  const int tok_v[2] = {(int)((ORDER >> (8 * q4)) & 7), (int)((ORDER >> (8 * q4 + 4)) & 7)};
  const uint32_t k_off = tok_k * ROW + ((q4 ^ (tok_k >> 1)) << 4);
  const uint32_t ks_off = OFF_KS + tok_k * fp4::BLOCKS + 2 * q4;
  uint32_t v_off[2], vs_off[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    v_off[j] = OFF_V + tok_v[j] * ROW + (((r >> 1) ^ (tok_v[j] >> 1)) << 4) + (r & 1) * 8;
    vs_off[j] = OFF_VS + tok_v[j] * fp4::BLOCKS + r;
  }
  const int group = (1 << p.G) - 1;
  const auto compute = [&](uint32_t st, int heads, int left) {
    float s[NT][MT][4];  // [head block][16 tokens][token r | r + 8, head 2 q4 | + 1]
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      // a thread's 32 dimensions of a token: 16 bytes of codes, two scales
      const uint4 a = lds128(st + k_off + mt * 16 * ROW), c = lds128(st + k_off + (mt * 16 + 8) * ROW);
      const uint32_t sa = f16_of_e4m3x2(lds16(st + ks_off + mt * 16 * fp4::BLOCKS)),
                     sb = f16_of_e4m3x2(lds16(st + ks_off + (mt * 16 + 8) * fp4::BLOCKS));
      const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wc[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t pick = w < 2 ? 0x1010 : 0x3232;
        const uint32_t fa = __byte_perm(sa, 0, pick), fb = __byte_perm(sb, 0, pick);
        uint32_t ha[4], hc[4];
        f16_of_e2m1x8(wa[w], ha);
        f16_of_e2m1x8(wc[w], hc);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          ha[k] = mul_f16x2(ha[k], fa);
          hc[k] = mul_f16x2(hc[k], fb);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint32_t b0 = qf[nt][2 * (2 * w + k)], b1 = qf[nt][2 * (2 * w + k) + 1];
            if (w == 0 && k == 0)
              mma16816_new(s[nt][mt], ha[0], hc[0], ha[1], hc[1], b0, b1);
            else
              mma16816(s[nt][mt], ha[2 * k], hc[2 * k], ha[2 * k + 1], hc[2 * k + 1], b0, b1);
          }
      }
    }
    // a masked score is replaced, never multiplied
    if (left < TOK || (SPARSE && heads != group)) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (mt * 16 + (c >> 1) * 8 + tok_k >= left ||
                (SPARSE && !((heads >> (nt * 8 + 2 * q4 + (c & 1))) & 1)))
              s[nt][mt][c] = -INFINITY;
    }
    // P as B fragments: [16 tokens][tokens 2 q4 | 2 q4 + 8, head r]
    uint32_t pf[NT][MT][2];
    float alpha[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float base[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float mx = fmaxf(s[nt][0][c], s[nt][0][2 + c]);
#pragma unroll
        for (int mt = 1; mt < MT; ++mt) mx = ptx::max3(mx, s[nt][mt][c], s[nt][mt][2 + c]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        const float mn = fmaxf(m[nt][c], mx);
        base[c] = mn == -INFINITY ? 0.f : mn;
        alpha[nt][c] = ptx::ex2_approx((m[nt][c] - base[c]) * fac[nt][c]);
        m[nt][c] = mn;
      }
      const uint64_t below = ptx::pk(-base[0], -base[1]);
      float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float e[4];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint64_t x = ptx::pk(s[nt][mt][2 * half], s[nt][mt][2 * half + 1]);
          float x0, x1;
          ptx::upk(ptx::add2(x, below), x0, x1);
          e[2 * half] = ptx::ex2_approx(fmaf(x0, fac[nt][0], P_SHIFT));
          e[2 * half + 1] = ptx::ex2_approx(fmaf(x1, fac[nt][1], P_SHIFT));
        }
        sum0 += e[0] + e[2];
        sum1 += e[1] + e[3];
#pragma unroll
        for (int half = 0; half < 2; ++half)
          pf[nt][mt][half] = transpose8x8(f16x2(e[2 * half], e[2 * half + 1]));
      }
      l[nt][0] = l[nt][0] * alpha[nt][0] + sum0;
      l[nt][1] = l[nt][1] * alpha[nt][1] + sum1;
    }
    // With `masked` the columns of heads that mask the tile keep their sums: their weights are zero,
    // but zero times a NaN of the tile's V would reach them through the shared product.
    const auto pv = [&](const bool masked) {
      uint32_t f[MT][2];  // scales of block r: tokens 2 q4, 2 q4 + 1 | those + 8
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t c[2];
#pragma unroll
          for (int j = 0; j < 2; ++j)
            c[j] = lds8(st + vs_off[j] + (mt * 16 + half * 8) * fp4::BLOCKS);
          if (left < TOK) {
            // whatever lies past the end counts as zero (a code is a number, a scale may be a NaN)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              if (mt * 16 + half * 8 + tok_v[j] >= left) c[j] = 0u;
          }
          f[mt][half] = f16_of_e4m3x2(c[0] | c[1] << 8);
        }
      uint2 v[MT][2][2];  // dimensions 16 r .. 16 r + 15 of those tokens
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            v[mt][half][j] = lds64(st + v_off[j] + (mt * 16 + half * 8) * ROW);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        float o[4][NT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          uint32_t h[4][4];  // dimensions 8 w + 0 2 4 6 | + 1 of tokens 2 q4, 2 q4 + 1 | of those + 8
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t x = w == 0 ? v[mt][half][0].x : v[mt][half][0].y;
            const uint32_t y = w == 0 ? v[mt][half][1].x : v[mt][half][1].y;
            // the codes of two tokens interleaved: a fragment pairs tokens within a dimension
            f16_of_e2m1x8((x & 0x0f0f0f0fu) | ((y << 4) & 0xf0f0f0f0u), h[2 * half]);
            f16_of_e2m1x8(((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u), h[2 * half + 1]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              h[2 * half][k] = mul_f16x2(h[2 * half][k], f[mt][half]);
              h[2 * half + 1][k] = mul_f16x2(h[2 * half + 1][k], f[mt][half]);
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              if (mt == 0)
                mma16816_new(o[k][nt], h[0][k], h[1][k], h[2][k], h[3][k], pf[nt][mt][0],
                             pf[nt][mt][1]);
              else
                mma16816(o[k][nt], h[0][k], h[1][k], h[2][k], h[3][k], pf[nt][mt][0],
                         pf[nt][mt][1]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (!masked || ((heads >> (nt * 8 + 2 * q4 + (c & 1))) & 1))
                acc[nt][4 * w + k][c] = fmaf(acc[nt][4 * w + k][c], alpha[nt][c & 1], o[k][nt][c]);
      }
    };
    if (!SPARSE || heads == group)
      pv(false);
    else
      pv(true);
  };

  // ---- the end of a segment: the warps' states combined; written out when the segment is its whole
  // task, left as a partial otherwise.  O goes through the stage just consumed, the one that the next
  // copy will overwrite.
  bool first_segment = true;
  const auto flush = [&](int stage, bool to_end_) {
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
        if (r == 0) s_ml[warp][g] = make_float2(m[nt][c] * fac[nt][c], t);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                           buf + g * (HEAD_DIM * 4) + (((4 * r + k) ^ q4) << 4)),
                       "f"(acc[nt][2 * k][c]), "f"(acc[nt][2 * k][2 + c]),
                       "f"(acc[nt][2 * k + 1][c]), "f"(acc[nt][2 * k + 1][2 + c])
                       : "memory");
      }
    __syncthreads();
    const bool complete = from_start && to_end_;
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
        decode::write_row(p, b, kvh, g, lane, mm, ll, o);
      } else {
        if (lane == 0) p.part_ml[slot * MAX_G + g] = make_float2(mm, ll);
        reinterpret_cast<float4 *>(p.part_o)[(slot * p.G + g) * 32 + lane] = o;
      }
    }
    __syncthreads();
  };

  convert_q();
  reset();
  int stage = 0;
  for (;;) {
    copies_wait<STAGES - 2>();
    __syncwarp();  // every lane's copies are there, and the stage before has been read by every lane
    issue(stage == 0 ? STAGES - 1 : stage - 1);
    const int4 meta = s_meta[warp][stage];
    const bool last = meta.z & 1, end = meta.z & 2;
    if (meta.y > 0) compute(ring + stage * STAGE_BYTES, meta.x, meta.y);
    if (last || end) {
      flush(stage, last);
      if (end) break;
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
  copies_wait<0>();
}

}  // namespace decode4
}  // namespace bsa
