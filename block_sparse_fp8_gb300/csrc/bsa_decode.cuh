// Attention of one new token per sequence over the paged e4m3 cache.
//
//   s_j = (q . k_j) * qd * kd_j * softmax_scale,  O = vd * sum_j 2^(s_j - m) v_j / l
//
// The simplest form: one CTA per (sequence, query head) walks the enabled tiles with a running
// maximum m and sum l; a thread owns one token's score, then one dimension of O.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cfloat>
#include <cstdint>

#include "bsa_common.cuh"

namespace bsa {
namespace decode {

constexpr int THREADS = 128;

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
  long long q_stride;                            // elements
  long long page_bytes, head_bytes, slot_bytes;  // strides inside the page pool
  int B, N1, N2, G, ps, num_pages, L, Kb, max_kv_len;
  int q_e4m3, k_per_token, v_per_head;
  float scale;
};

__device__ __forceinline__ void report(const Params &p, int bits) {
  if (p.dev_status) atomicOr(p.dev_status, bits);
}

__device__ __forceinline__ float e4m3_value(uint8_t c) {
  __nv_fp8_e4m3 x;
  x.__x = c;
  return static_cast<float>(x);
}

__global__ void __launch_bounds__(THREADS) decode_kernel(const Params p) {
  __shared__ float qs[HEAD_DIM], ps[TILE], red[THREADS / 32];
  __shared__ uint32_t on[KB_MAX / 32];
  __shared__ long long base[TILE];
  const int b = blockIdx.x / p.N1, h = blockIdx.x % p.N1, kvh = h / p.G, tid = threadIdx.x;
  int kv = p.seqused_kv[b];
  if (kv < 0 || kv > p.max_kv_len || (long long)kv > (long long)p.L * p.ps) {
    if (tid == 0) report(p, BSA_DEV_BAD_SEQLEN);
    kv = 0;
  }
  qs[tid] = p.q_e4m3
                ? e4m3_value(static_cast<const uint8_t *>(p.q)[b * p.q_stride + h * HEAD_DIM + tid]) *
                      p.q_descale[b * p.N1 + h]
                : __bfloat162float(static_cast<const __nv_bfloat16 *>(
                      p.q)[b * p.q_stride + h * HEAD_DIM + tid]);
  const size_t row = ((size_t)b * p.N1 + h) * p.Kb;
  const int nt = (kv + TILE - 1) / TILE;
  if (p.sparse_indices) {
    for (int w = tid; w < KB_MAX / 32; w += THREADS) on[w] = 0;
    __syncthreads();
    int len = p.sparse_seq_len[(size_t)b * p.N1 + h];
    if (len < 0 || len > p.Kb) {
      if (tid == 0) report(p, BSA_DEV_BAD_INDEX);
      len = len < 0 ? 0 : p.Kb;
    }
    for (int e = tid; e < len; e += THREADS) {
      const int t = p.sparse_indices[row + e];
      if (t < 0 || t >= p.Kb)
        report(p, BSA_DEV_BAD_INDEX);
      else
        atomicOr(&on[t >> 5], 1u << (t & 31));
    }
  }
  __syncthreads();
  float m = -INFINITY, l = 0.f, acc = 0.f;
  for (int t = 0; t < nt; ++t) {
    if (p.block_mask && p.block_mask[row + t] == 0) continue;
    if (p.sparse_indices && !((on[t >> 5] >> (t & 31)) & 1u)) continue;
    const int pos = t * TILE + tid;
    float s = -INFINITY;
    long long at = -1;
    if (pos < kv) {
      const int pg = p.block_table[(size_t)b * p.L + pos / p.ps];
      const int slot = pos % p.ps;
      s = 0.f;
      if (pg < 0 || pg >= p.num_pages) {
        report(p, BSA_DEV_BAD_PAGE);
      } else {
        at = pg * p.page_bytes + kvh * p.head_bytes + slot * p.slot_bytes;
        for (int d = 0; d < HEAD_DIM; ++d) s += qs[d] * e4m3_value(p.k_pages[at + d]);
        s *= p.k_per_token ? p.k_descale[((size_t)pg * p.N2 + kvh) * p.ps + slot] : p.k_descale[0];
        s *= p.scale;
      }
    }
    base[tid] = at;
    float mx = s;
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if ((tid & 31) == 0) red[tid >> 5] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float mn = fmaxf(m, mx), ms = mn == -INFINITY ? 0.f : mn;
    ps[tid] = pos < kv ? expf(s - ms) : 0.f;
    __syncthreads();
    const float alpha = expf(m - ms);
    acc *= alpha;
    l *= alpha;
    m = mn;
    for (int j = 0; j < TILE && t * TILE + j < kv; ++j) {
      l += ps[j];
      if (base[j] >= 0) acc += ps[j] * e4m3_value(p.v_pages[base[j] + tid]);
    }
    __syncthreads();
  }
  const bool some = l != 0.f;
  const float o = some ? acc / l * (p.v_per_head ? p.v_descale[kvh] : p.v_descale[0]) : 0.f;
  p.out[((size_t)b * p.N1 + h) * HEAD_DIM + tid] = __float2bfloat16(o);
  if (tid == 0 && p.lse) p.lse[(size_t)h * p.B + b] = some ? m + logf(l) : -FLT_MAX;
}

}  // namespace decode
}  // namespace bsa
