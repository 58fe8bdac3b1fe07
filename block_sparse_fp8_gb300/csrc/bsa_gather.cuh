// The paged e4m3 cache read back into contiguous rows: value = code * descale, one fp32 product,
// rounded once more for bf16.
//
// HBM-bound (a KV head's token: 256 bytes of codes and 4 of descale in, 512 or 1024 out).  A block
// takes a run of tokens.  Its first threads look the tokens up -- the sequence by binary search over
// cu_seqlens, then the block table -- and leave page and slot in shared memory, so that the
// dependent reads are paid once a token and not once a row.  Then a row of 128 values belongs to
// 16 lanes (bf16) or 32 (fp32), each of which turns 8 or 4 codes into one 16-byte store; a thread has
// the K and V codes of ROWS rows in flight.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "bsa_common.cuh"

namespace bsa {
namespace gather {

constexpr int THREADS = 256;
constexpr int MAX_TOKENS = 32;  // tokens of a block
constexpr int ROWS = 4;         // rows in flight per thread

struct Params {
  const uint8_t *k_pages, *v_pages;
  const float *k_descale, *v_descale;
  const int *cu_seqlens, *cache_starts, *block_table;
  void *k_out, *v_out;
  int *dev_status;
  long long page_bytes, head_bytes, slot_bytes;
  int B, N2, ps, num_pages, L, total;
  int k_per_token, v_per_head;
  int tokens;  // of a block, a power of two up to MAX_TOKENS
};

// Two e4m3 codes (the low 16 bits) as fp32.
__device__ __forceinline__ float2 values2(uint32_t codes) {
  uint32_t h;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t}"
      : "=r"(h)
      : "r"(codes));
  __half2 x;
  memcpy(&x, &h, 4);
  return __half22float2(x);
}

__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
  uint32_t r;
  memcpy(&r, &x, 4);
  return r;
}

template <bool F32>
struct Codes;  // a thread's share of a row
template <>
struct Codes<false> {
  uint2 c;
  __device__ __forceinline__ void load(const uint8_t *p) { c = *reinterpret_cast<const uint2 *>(p); }
  __device__ __forceinline__ void zero() { c = make_uint2(0, 0); }
  __device__ __forceinline__ uint4 scaled(float s) const {
    const float2 a = values2(c.x), b = values2(c.x >> 16), d = values2(c.y), e = values2(c.y >> 16);
    return make_uint4(bf16x2(a.x * s, a.y * s), bf16x2(b.x * s, b.y * s), bf16x2(d.x * s, d.y * s),
                      bf16x2(e.x * s, e.y * s));
  }
};
template <>
struct Codes<true> {
  uint32_t c;
  __device__ __forceinline__ void load(const uint8_t *p) {
    c = *reinterpret_cast<const uint32_t *>(p);
  }
  __device__ __forceinline__ void zero() { c = 0; }
  __device__ __forceinline__ uint4 scaled(float s) const {
    const float2 a = values2(c), b = values2(c >> 16);
    return make_uint4(__float_as_uint(a.x * s), __float_as_uint(a.y * s), __float_as_uint(b.x * s),
                      __float_as_uint(b.y * s));
  }
};

template <bool F32>
__global__ void __launch_bounds__(THREADS) gather_kernel(const Params p) {
  constexpr int LANES = F32 ? 32 : 16;  // of a row
  constexpr int STEP = THREADS / LANES;
  __shared__ int s_page[MAX_TOKENS], s_slot[MAX_TOKENS];
  const int tid = threadIdx.x, t0 = blockIdx.x * p.tokens;
  if (tid < p.tokens) {
    const int tok = t0 + tid;
    int page = -2, slot = 0;  // -2: a row behind the last sequence, left as it is
    if (tok < p.total && tok >= p.cu_seqlens[0] && tok < p.cu_seqlens[p.B]) {
      int lo = 0, hi = p.B - 1;  // the last b with cu_seqlens[b] <= tok
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.cu_seqlens[mid] <= tok) lo = mid; else hi = mid - 1;
      }
      const long long pos =
          (long long)(p.cache_starts ? p.cache_starts[lo] : 0) + (tok - p.cu_seqlens[lo]);
      const long long lp = pos / p.ps;
      page = pos >= 0 && lp < p.L ? p.block_table[(size_t)lo * p.L + lp] : -1;
      slot = (int)(pos & (p.ps - 1));
      if (page < 0 || page >= p.num_pages) {
        if (p.dev_status) atomicOr(p.dev_status, BSA_DEV_BAD_PAGE);
        page = -1;
      }
    }
    s_page[tid] = page;
    s_slot[tid] = slot;
  }
  __syncthreads();
  const int li = tid % LANES, rows = p.tokens * p.N2;
  for (int r0 = tid / LANES; r0 < rows; r0 += STEP * ROWS) {
    Codes<F32> k[ROWS], v[ROWS];
    float ks[ROWS], vs[ROWS];
    int page[ROWS];
    size_t at[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int r = r0 + i * STEP, t = r / p.N2, g = r - t * p.N2;
      page[i] = r < rows ? s_page[t] : -2;
      at[i] = ((size_t)(t0 + t) * p.N2 + g) * HEAD_DIM + li * (HEAD_DIM / LANES);
      k[i].zero();
      v[i].zero();
      ks[i] = vs[i] = 0.f;
      if (page[i] >= 0) {
        const int slot = s_slot[t];
        const long long off = page[i] * p.page_bytes + g * p.head_bytes + slot * p.slot_bytes +
                              li * (HEAD_DIM / LANES);
        if (p.k_out) {
          k[i].load(p.k_pages + off);
          ks[i] = p.k_per_token ? p.k_descale[((size_t)page[i] * p.N2 + g) * p.ps + slot]
                                : p.k_descale[0];
        }
        if (p.v_out) {
          v[i].load(p.v_pages + off);
          vs[i] = p.v_per_head ? p.v_descale[g] : p.v_descale[0];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      if (page[i] == -2) continue;
      constexpr int SIZE = F32 ? 4 : 2;
      if (p.k_out)
        __stcs(reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.k_out) + at[i] * SIZE),
               k[i].scaled(ks[i]));
      if (p.v_out)
        __stcs(reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.v_out) + at[i] * SIZE),
               v[i].scaled(vs[i]));
    }
  }
}

}  // namespace gather
}  // namespace bsa
