// The 4-bit cache: a row of 128 values is 64 bytes of e2m1 codes (two to a byte, the first in the low
// half) and eight e4m3 scales, one for every 16 codes; value = code * scale * descale, with one fp32
// descale per tensor or KV head.  Here: new bf16 tokens quantised into it.
//
//   scale = the e4m3 number nearest to amax / (6 descale),  code = the e2m1 number nearest to
//   x / (scale * descale), ties to the even code, 448 and 6 the largest
//
// decided exactly, not on rounded quotients.  That matters more than it seems to: a descale is often some
// largest value over 6 * 448 = 2^7 * 21, so that quotients next to the borders at 7/4 and 7/2 are
// common (one value in six hundred), and fp32 puts them on the border.  A quotient estimated to
// 2^-21 is converted twice, nudged up and down by 2^-20; where the two codes differ the border between
// them, times scale and descale, is compared with the value itself by the sign of one fma, which rounds
// but never crosses zero.
//
// HBM-bound: 256 bytes of a row read, 72 written.  A thread has one block of 16 values of K and the
// same of V, eight threads a row.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "bsa_common.cuh"
#include "bsa_quant.cuh"

namespace bsa {
namespace fp4 {

constexpr int BLOCK = 16;                     // codes to a scale
constexpr int BLOCKS = HEAD_DIM / BLOCK;      // scales of a row
constexpr int ROW_BYTES = HEAD_DIM / 2;       // codes of a row
constexpr int THREADS = 256;

struct AppendParams {
  const __nv_bfloat16 *k_new, *v_new;
  long long k_stride, v_stride;  // elements from token to token
  const int *slot_map;
  const float *k_descale, *v_descale;
  uint8_t *k_pages, *v_pages, *k_scales, *v_scales;
  int *dev_status;
  long long rows;  // tokens x KV heads
  int N2, ps_shift, num_pages;
  int k_per_head, v_per_head, kv_nhd;
};

__device__ __forceinline__ uint32_t e4m3_of(float x) {  // of one non-negative value
  uint32_t r;
  asm("{\n\t.reg .b16 c;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 c, %1, %1;\n\t"
      "cvt.u32.u16 %0, c;\n\t}"
      : "=r"(r)
      : "f"(x));
  return r & 0xffu;
}

__device__ __forceinline__ float value_of_e4m3(uint32_t c) {
  uint32_t h;
  asm("{\n\t.reg .b16 a;\n\t"
      "cvt.u16.u32 a, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t}"
      : "=r"(h)
      : "r"(c & 0xffu));
  return __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
}

// e2m1 codes of two values, the first in the low half of the byte.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 c;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %2, %1;\n\t"
      "cvt.u32.u8 %0, c;\n\t}"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return r;
}

// The size of an e2m1 code (0 .. 7), doubled: 0 1 2 3 4 6 8 12.
__device__ __forceinline__ int twice_e2m1(uint32_t c) {
  const int e = c >> 1, m = c & 1;
  return e == 0 ? m : (2 + m) << (e - 1);
}

constexpr float NUDGE_UP = 1.f + 0x1p-20f, NUDGE_DOWN = 1.f - 0x1p-20f;

// Which of two neighbouring codes (`down`, `down` + 1) is nearer: the sign of the value less the border
// between them, zero for a tie.
__device__ __forceinline__ uint32_t settle(uint32_t down, float above) {
  return above > 0.f || (above == 0.f && (down & 1u)) ? down + 1 : down;
}

// The scale of a block whose largest magnitude is amax, as a code.
__device__ __forceinline__ uint32_t scale_of(float amax, float descale, float inv6) {
  const float t = amax * inv6;
  const uint32_t up = e4m3_of(t * NUDGE_UP), down = e4m3_of(t * NUDGE_DOWN);
  if (up == down) return up;
  const float border = 0.5f * (value_of_e4m3(down) + value_of_e4m3(up));
  return settle(down, fmaf(-6.f * border, descale, amax));
}

// The codes of a block's 16 values under its scale.
__device__ __forceinline__ uint2 codes_of(const float (&x)[16], float scale, float descale) {
  const float d = scale * descale, r = d > 0.f ? __frcp_rn(d) : 0.f;
  uint32_t w[2] = {0u, 0u}, other[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = x[2 * i] * r, b = x[2 * i + 1] * r;
    w[i >> 2] |= e2m1x2(a * NUDGE_UP, b * NUDGE_UP) << (8 * (i & 3));
    other[i >> 2] |= e2m1x2(a * NUDGE_DOWN, b * NUDGE_DOWN) << (8 * (i & 3));
  }
  if (w[0] != other[0] || w[1] != other[1]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int at = 4 * (i & 7);
      const uint32_t up = (w[i >> 3] >> at) & 7u, down = (other[i >> 3] >> at) & 7u;
      if (up == down) continue;
      // the border is (twice one + twice the other) / 4, exact with the scale
      const float border = 0.25f * (float)(twice_e2m1(up) + twice_e2m1(down)) * scale;
      const uint32_t c = settle(down, fmaf(-border, descale, fabsf(x[i])));
      w[i >> 3] = (w[i >> 3] & ~(7u << at)) | c << at;
    }
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void store_block(const uint4 &a, const uint4 &b, float descale,
                                            float inv6, uint8_t *codes, uint8_t *scale_at) {
  float lo[8], hi[8], x[16];
  quant::unpack8(a, lo);
  quant::unpack8(b, hi);
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = lo[i];
    x[8 + i] = hi[i];
    amax = fmaxf(amax, fmaxf(fabsf(lo[i]), fabsf(hi[i])));
  }
  const uint32_t s = scale_of(amax, descale, inv6);
  *reinterpret_cast<uint2 *>(codes) = codes_of(x, value_of_e4m3(s), descale);
  *scale_at = (uint8_t)s;
}

__global__ void __launch_bounds__(THREADS) append_kernel(const AppendParams p) {
  const int block = threadIdx.x & (BLOCKS - 1);
  const long long row = (long long)blockIdx.x * (THREADS / BLOCKS) + threadIdx.x / BLOCKS;
  if (row >= p.rows) return;
  const long long tok = row / p.N2;
  const int g = (int)(row % p.N2);
  const long long at = (long long)g * HEAD_DIM + block * BLOCK;
  const uint4 *k = reinterpret_cast<const uint4 *>(p.k_new + tok * p.k_stride + at);
  const uint4 *v = reinterpret_cast<const uint4 *>(p.v_new + tok * p.v_stride + at);
  const uint4 k0 = k[0], k1 = k[1], v0 = v[0], v1 = v[1];
  const int slot = p.slot_map[tok];
  const float kg = p.k_descale[p.k_per_head ? g : 0], vg = p.v_descale[p.v_per_head ? g : 0];
  if (slot < 0) return;  // a row without a place
  const int page = slot >> p.ps_shift, in = slot & ((1 << p.ps_shift) - 1);
  if (page >= p.num_pages) {
    if (p.dev_status) atomicOr(p.dev_status, BSA_DEV_BAD_PAGE);
    return;
  }
  const long long hnd = (((long long)page * p.N2 + g) << p.ps_shift) + in;
  const long long dst = p.kv_nhd ? (((long long)page << p.ps_shift) + in) * p.N2 + g : hnd;
  store_block(k0, k1, kg, __frcp_rn(6.f * kg), p.k_pages + dst * ROW_BYTES + block * (BLOCK / 2),
              p.k_scales + hnd * BLOCKS + block);
  store_block(v0, v1, vg, __frcp_rn(6.f * vg), p.v_pages + dst * ROW_BYTES + block * (BLOCK / 2),
              p.v_scales + hnd * BLOCKS + block);
}

}  // namespace fp4
}  // namespace bsa
