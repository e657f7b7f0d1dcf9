// act_codec.h -- the activation codes (Q8_0, MXFP8) of 32-value blocks.
#pragma once

#include "device_common.h"

namespace coli {

// E8M0 shared exponent of a 32-block with maximum magnitude amax:
// floor(log2 amax) - 8 (the largest E4M3 exponent) + 127, clamped to
// [0, 254]; 0 for an all-zero block.  floor(log2) comes from the fp32
// exponent field; a subnormal amax clamps to 0 anyway.
COLI_DEV uint32_t mx8_exponent(float amax) {
  const int ex = (int)((__float_as_uint(amax) >> 23) & 0xffu);  // biased; 0 for 0 / subnormal
  const int E = ex - 127 - 8 + 127;
  return amax > 0.0f ? (uint32_t)max(0, min(254, E)) : 0u;
}

// ---- blocks held by neighbouring lanes, N = 8 or 4 values each ---------------
// Codes and scales are bit for bit those of the prefill path's quantisers,
// which hold a block in one thread.

// Maximum of a >= 0 over aligned groups of 32 / N lanes, by DPP moves
// (non-negative floats order as their bit patterns do).
template <int CTRL>
COLI_DEV uint32_t dpp_max(uint32_t u) {
  return max(u, (uint32_t)__builtin_amdgcn_mov_dpp((int)u, CTRL, 0xf, 0xf, false));
}
template <int N>
COLI_DEV float block_max(const float (&v)[N]) {
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) a = fmaxf(a, fabsf(v[i]));
  uint32_t u = dpp_max<0x4E>(dpp_max<0xB1>(__float_as_uint(a)));  // swap neighbours, then pairs
  if (N == 4) u = dpp_max<0x141>(u);                              // mirror halves of 8
  return __uint_as_float(u);
}

// Q8_0: d = max / 127, q = round half away from zero of v / d, both divisions
// IEEE; 0 for an all-zero block.  Returns d as fp16 bits.
template <int N>
COLI_DEV uint16_t q8_0_lane(const float (&v)[N], uint32_t (&q)[N / 4]) {
  const float a = block_max(v);
  const float d = __fdiv_rn(a, 127.0f);
#pragma unroll
  for (int w = 0; w < N / 4; ++w) q[w] = 0u;
  if (a != 0.0f) {
    // 2 v / d = v / (d / 2), halves being exact: the divisor's reciprocal with
    // one Newton step, then a product and two exact-residual corrections per
    // value give the IEEE quotient while no step leaves the normal range,
    // which a d outside [2^-60, 2^100] could.  t = trunc(2 v / d) rounds half
    // away from zero as (t + 1) / 2 below; |v| <= 127.0000077 d, so codes
    // stay within 127.
    const bool mid = d >= 0x1p-60f && d <= 0x1p100f;
    const float h = 0.5f * d;
    const float y0 = __builtin_amdgcn_rcpf(h);
    const float y = fmaf(fmaf(-h, y0, 1.0f), y0, y0);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float t = v[i] * y;
      t = fmaf(fmaf(-h, t, v[i]), y, t);
      t = fmaf(fmaf(-h, t, v[i]), y, t);
      if (!mid) t = 2.0f * __fdiv_rn(v[i], d);
      const int n = max(-254, min(254, (int)t));
      const int r = (n + 1 + (n >> 31)) >> 1;
      q[i >> 2] |= (uint32_t)(r & 0xff) << (8 * (i & 3));
    }
  }
  return f32_to_f16_bits(d);
}

// MXFP8: E4M3 codes of v / 2^(E - 127), nearest with ties to even, saturating
// at 448, the sign kept.  The scaling is by a power of two (exact but far
// below the smallest code) and the hardware conversion rounds as the format
// asks; it does not saturate, so the values are clamped first (all that lie in
// (448, 512) round to 448).  Returns E.
template <int N>
COLI_DEV uint32_t mx8_lane(const float (&v)[N], uint32_t (&q)[N / 4]) {
  const uint32_t E = mx8_exponent(block_max(v));
  const float f = __uint_as_float((254u - E) << 23);  // 2^(127 - E), E <= 247
#pragma unroll
  for (int w = 0; w < N / 4; ++w) {
    float m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      m[i] = __builtin_amdgcn_fmed3f(v[4 * w + i] * f, -448.0f, 448.0f);
    const int p = __builtin_amdgcn_cvt_pk_fp8_f32(m[0], m[1], 0, false);
    q[w] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(m[2], m[3], p, true);
  }
  return E;
}

}  // namespace coli
