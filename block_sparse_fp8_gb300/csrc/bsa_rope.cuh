// Rotary positions: pairs of a head's first R values are turned by position x frequency,
//   (x, y) -> amplitude * (x cos a - y sin a, y cos a + x sin a),  a = 2 pi frac(position f_i),
// pair i being (i, i + R/2) or (2i, 2i + 1); the rest of the head is copied.  Either bf16 -> bf16 for Q
// and K at once, or bf16 -> e4m3 codes and a descale per row for Q (bsa_quant.cuh's rule on the
// turned values, which are not rounded to bf16 in between).
//
// A frequency is a 64-bit fixed-point fraction of a turn, and the product with the position is taken
// modulo a turn by the integers' own overflow, exactly for any 32-bit position, where an fp32 product at
// position 500,000 is off by up to 0.03 radians.  Of the product the upper 32 bits go on (2^-32 turns)
// and are rounded to fp32 (2^-26 turns at most, next to half a turn).  The frequencies come from double
// arithmetic, within 2^-55 turns a position of their formulas (2^-24 turns at position 2^31).
//
// HBM-bound (a row of 128 values: 256 bytes in, 256 or 132 out).  Eight threads have a row, two
// 16-byte vectors each, chosen so that a thread's vectors hold whole pairs and eight threads' loads
// lie side by side; eight frequencies serve a thread's sixteen values in either layout.  A thread works
// its sines and cosines out once for the heads that it serves, up to eight, its first loads in
// flight meanwhile; the arithmetic runs on pairs (fma.f32x2).
//
// Measured (mean of back-to-back calls): 8192 tokens x 40 heads in bf16, half of each head turned (168
// MB) 29 us, 86% of the measured copy rate, 26.7 in a graph (94%); 16K tokens x 64 heads to e4m3 (407
// MB) 81 us, 75%: latency at 95 registers, 18 warps an SM (of it the sines 4 us; blocks of 128
// threads 83, two parts of two heads in turn 91, 80 registers 104, fp32 in single values 116); 16
// tokens x 40 heads 2.2 us.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "bsa_common.cuh"
#include "bsa_div.cuh"
#include "bsa_quant.cuh"
#include "ptx_sm103.cuh"

namespace bsa {
namespace rope {

constexpr int THREADS = 64;
constexpr int LANES = 8;    // threads of a row
constexpr int VEC = 8;      // values of a 16-byte vector
constexpr int VECS = HEAD_DIM / VEC;

struct Params {
  const __nv_bfloat16 *q, *k;
  __nv_bfloat16 *q_out, *k_out;
  uint2 *codes;
  float *descale;
  const int *positions;
  const unsigned long long *freqs;
  long long q_stride, k_stride, q_out_stride, k_out_stride;  // elements from token to token
  uint32_t units;  // tokens x groups of heads, below 2^31
  Divisor by_groups;
  int N1, N2, R;
  int groups, heads;  // groups of `heads` heads that one thread serves
  int interleaved, ue8m0;
  float amplitude;
};

// Two bf16 values as a pair of fp32, and back.
__device__ __forceinline__ uint64_t pair_of(uint32_t w) {
  return ptx::pk(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t bf16_of(uint64_t v) {
  float lo, hi;
  ptx::upk(v, lo, hi);
  const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
  uint32_t r;
  memcpy(&r, &x, 4);
  return r;
}
__device__ __forceinline__ uint4 pack8(const uint64_t (&v)[4]) {
  return make_uint4(bf16_of(v[0]), bf16_of(v[1]), bf16_of(v[2]), bf16_of(v[3]));
}
__device__ __forceinline__ uint64_t swapped(uint64_t v) {
  float lo, hi;
  ptx::upk(v, lo, hi);
  return ptx::pk(hi, lo);
}

// The codes of eight values, as quant::codes8 makes them: rounded quotients (Markstein's correction of
// the product with the rounded reciprocal).
__device__ __forceinline__ uint2 codes8(const uint64_t (&v)[4], float scale, uint64_t inv,
                                        uint64_t neg) {
  float q[8];
  if (scale >= 0x1p-90f && scale <= 0x1p90f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t q0 = ptx::mul2(v[i], inv);
      ptx::upk(ptx::fma2(ptx::fma2(q0, neg, v[i]), inv, q0), q[2 * i], q[2 * i + 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ptx::upk(v[i], q[2 * i], q[2 * i + 1]);
      q[2 * i] = __fdiv_rn(q[2 * i], scale);
      q[2 * i + 1] = __fdiv_rn(q[2 * i + 1], scale);
    }
  }
  return make_uint2(ptx::cvt_e4m3x4(q[0], q[1], q[2], q[3]), ptx::cvt_e4m3x4(q[4], q[5], q[6], q[7]));
}

constexpr int AHEAD = 4;  // heads in flight per thread

template <bool QUANT>
__global__ void __launch_bounds__(THREADS) rope_kernel(const Params p) {
  const int lane = threadIdx.x & (LANES - 1);
  // whole warps stay to the end: the rows' maxima go by shuffles
  const uint32_t unit = blockIdx.x * (THREADS / LANES) + threadIdx.x / LANES;
  const bool live = unit < p.units;
  const long long t = live ? p.by_groups.quotient(unit) : 0;
  const int group = live ? (int)(unit - (uint32_t)t * p.groups) : 0;
  const int heads = p.N1 + p.N2, h0 = group * p.heads,
            h1 = live ? min(h0 + p.heads, heads) : h0;

  // the thread's vectors, and whether they are turned
  const int turned = p.R / VEC;  // vectors that hold pairs
  int v0 = lane, v1 = lane + LANES;
  bool turn0 = v0 < turned, turn1 = v1 < turned;
  if (!p.interleaved) {
    const int half = turned / 2, rest = lane - half;
    turn0 = turn1 = rest < 0;
    v0 = turn0 ? lane : turned + rest;
    v1 = turn0 ? lane + half : turned + rest + LANES - half;
  }

  const uint4 *const q_row = reinterpret_cast<const uint4 *>(p.q + t * p.q_stride);
  const uint4 *const k_row =
      QUANT ? nullptr : reinterpret_cast<const uint4 *>(p.k + t * p.k_stride) - p.N1 * VECS;
  uint4 a[AHEAD], b[AHEAD];
  const auto load = [&](int h) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      a[i] = b[i] = make_uint4(0, 0, 0, 0);
      if (h + i < h1) {
        const uint4 *x = (QUANT || h + i < p.N1 ? q_row : k_row) + (h + i) * VECS;
        a[i] = x[v0];
        b[i] = x[v1];
      }
    }
  };
  load(h0);

  // cosines and sines: in halves pair j of both vectors, interleaved four pairs of each vector
  float c[8], s[8];
  const unsigned long long pos = live ? (unsigned long long)(long long)p.positions[t] : 0ull;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int i = p.interleaved ? (j < 4 ? 4 * v0 + j : 4 * v1 + j - 4) : 8 * v0 + j;
    const bool on = j < 4 || !p.interleaved ? turn0 : turn1;
    const unsigned long long turns = on ? pos * p.freqs[i] : 0ull;
    // the nearer way round: [-1/2, 1/2) of a turn
    sincospif((float)(int)(turns >> 32) * 0x1p-31f, &s[j], &c[j]);
    c[j] = on ? c[j] * p.amplitude : 1.f;
    s[j] = on ? s[j] * p.amplitude : 0.f;
  }

  uint2 *const codes = QUANT ? p.codes + t * p.N1 * VECS : nullptr;
  float *const descale = QUANT ? p.descale + t * p.N1 : nullptr;
  // (with codes to make, whole warps walk the same heads: groups may be short, rows not)
  const int steps = (p.heads + AHEAD - 1) / AHEAD;
  for (int step = 0; step < steps; ++step) {
    const int h = h0 + step * AHEAD;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const uint32_t wa[4] = {a[i].x, a[i].y, a[i].z, a[i].w},
                     wb[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
      uint64_t x[4], y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = pair_of(wa[j]);
        y[j] = pair_of(wb[j]);
      }
      if (p.interleaved) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // (x0, x1) (c, c) + (x1, x0) (-s, s)
          x[j] = ptx::fma2(swapped(x[j]), ptx::pk(-s[j], s[j]), ptx::mul2(x[j], ptx::pk(c[j], c[j])));
          y[j] = ptx::fma2(swapped(y[j]), ptx::pk(-s[4 + j], s[4 + j]),
                           ptx::mul2(y[j], ptx::pk(c[4 + j], c[4 + j])));
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t u = x[j], v = y[j], cc = ptx::pk(c[2 * j], c[2 * j + 1]);
          x[j] = ptx::fma2(v, ptx::pk(-s[2 * j], -s[2 * j + 1]), ptx::mul2(u, cc));
          y[j] = ptx::fma2(u, ptx::pk(s[2 * j], s[2 * j + 1]), ptx::mul2(v, cc));
        }
      }
      if constexpr (QUANT) {
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float x0, x1, y0, y1;
          ptx::upk(x[j], x0, x1);
          ptx::upk(y[j], y0, y1);
          m = fmaxf(fmaxf(m, fmaxf(fabsf(x0), fabsf(x1))), fmaxf(fabsf(y0), fabsf(y1)));
        }
#pragma unroll
        for (int o = LANES / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (h + i < h1) {
          const float d = quant::descale_of(m, p.ue8m0), r = __frcp_rn(d);
          const uint64_t inv = ptx::pk(r, r), neg = ptx::pk(-d, -d);
          uint2 *o = codes + (h + i) * VECS;
          o[v0] = codes8(x, d, inv, neg);
          o[v1] = codes8(y, d, inv, neg);
          if (lane == 0) descale[h + i] = d;
        }
      } else if (h + i < h1) {
        uint4 *o = reinterpret_cast<uint4 *>(
            h + i < p.N1 ? p.q_out + t * p.q_out_stride + (long long)(h + i) * HEAD_DIM
                         : p.k_out + t * p.k_out_stride + (long long)(h + i - p.N1) * HEAD_DIM);
        o[v0] = turn0 ? pack8(x) : a[i];
        o[v1] = turn1 ? pack8(y) : b[i];
      }
    }
    if (step + 1 < steps) load(h + AHEAD);
  }
}

}  // namespace rope
}  // namespace bsa
