// Join of attention results over disjoint sets of keys:
//   M = max_i LSE_i, w_i = exp(LSE_i - M), O = sum_i w_i O_i / sum_i w_i, LSE = M + ln sum_i w_i.
//
// HBM-bound: every O is read once, one is written.  A block takes a tile of tokens x heads.  The LSEs
// lie head-major and the O rows token-major, so the tile's weights are worked out first, a thread per
// (token, head) with neighbouring threads on neighbouring tokens, and left in shared memory; then 16
// lanes to a row stream the parts, a thread's 16 bytes of every part of two rows in flight at once.
// out may be one of the parts and lse one of their LSEs: whoever writes an element has read all of
// its sources before.
//
// Measured (mean of back-to-back calls): five parts of 16K tokens x 64 heads (1636 MB) 231 us, 7.1
// TB/s, 104% of the measured copy rate (which writes as much as it reads; one block a row, the first
// form: 1232 us); two of 8K x 32 (204 MB) 34 us, 89%, the rest launch and ramp.
#pragma once

#include <cuda_bf16.h>

#include <cfloat>
#include <cstdint>

#include "bsa_common.cuh"

namespace bsa {
namespace merge {

constexpr int THREADS = 256;
constexpr int MAX_ROWS = 256;  // rows (token, head) of a tile

struct Params {
  // no __restrict__: out may be one of outs, lse one of lses
  const __nv_bfloat16 *outs[BSA_MAX_MERGE];
  const float *lses[BSA_MAX_MERGE];
  __nv_bfloat16 *out;
  float *lse;
  int T, N1;
  int head_shift, tok_shift;  // log2 of the tile's heads and tokens
  int head_tiles;
};

template <int N>  // parts
__global__ void __launch_bounds__(THREADS) merge_kernel(const Params p) {
  __shared__ float s_w[N][MAX_ROWS];
  const int heads = 1 << p.head_shift, toks = 1 << p.tok_shift, rows = heads * toks;
  const int t0 = (int)(blockIdx.x / p.head_tiles) * toks;
  const int h0 = (int)(blockIdx.x % p.head_tiles) * heads, tid = threadIdx.x;
  for (int i = tid; i < rows; i += THREADS) {
    const int t = i & (toks - 1), h = i >> p.tok_shift;  // neighbouring threads: tokens
    if (t0 + t >= p.T || h0 + h >= p.N1) continue;
    const size_t at = (size_t)(h0 + h) * p.T + t0 + t;
    float x[N], m = -INFINITY;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      x[j] = p.lses[j][at];
      if (x[j] == -FLT_MAX) x[j] = -INFINITY;
      m = fmaxf(m, x[j]);
    }
    const float base = m == -INFINITY ? 0.f : m;
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      x[j] = expf(x[j] - base);  // exp(-inf) = 0
      sum += x[j];
    }
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) s_w[j][(t << p.head_shift) + h] = x[j] * inv;
    if (p.lse) p.lse[at] = sum != 0.f ? base + logf(sum) : -FLT_MAX;
  }
  __syncthreads();
  const int li = tid & 15;
  for (int i0 = tid >> 4; i0 < rows; i0 += 2 * (THREADS / 16)) {
    uint4 v[2][N];
    size_t at[2];
    bool live[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = i0 + u * (THREADS / 16), t = t0 + (i >> p.head_shift),
                h = h0 + (i & (heads - 1));
      live[u] = i < rows && t < p.T && h < p.N1;
      at[u] = ((size_t)t * p.N1 + h) * 16 + li;
#pragma unroll
      for (int j = 0; j < N; ++j)
        v[u][j] = live[u] ? reinterpret_cast<const uint4 *>(p.outs[j])[at[u]]
                          : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (!live[u]) continue;
      float o[8] = {};
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float w = s_w[j][i0 + u * (THREADS / 16)];
        if (w == 0.f) continue;  // an empty part's O is not used, whatever it holds
        const uint32_t c[4] = {v[u][j].x, v[u][j].y, v[u][j].z, v[u][j].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          o[2 * k] += w * __uint_as_float(c[k] << 16);
          o[2 * k + 1] += w * __uint_as_float(c[k] & 0xffff0000u);
        }
      }
      uint32_t r[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(o[2 * k], o[2 * k + 1]);
        memcpy(&r[k], &b, 4);
      }
      __stcs(reinterpret_cast<uint4 *>(p.out) + at[u], make_uint4(r[0], r[1], r[2], r[3]));
    }
  }
}

}  // namespace merge
}  // namespace bsa
