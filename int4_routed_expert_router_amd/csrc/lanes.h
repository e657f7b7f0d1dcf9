// lanes.h -- rows spread over lanes: sums over the lanes that share a row.
#pragma once

#include "device_common.h"

namespace coli {

template <int CTRL>
COLI_DEV float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, false));
}

// Sum over aligned groups of N = 8, 16, 32 or 64 lanes, in every one of them.
// Up to 16 lanes by DPP moves (swap neighbours, swap pairs, mirror halves of
// 8, mirror the row of 16), without LDS.
template <int N>
COLI_DEV float lanes_sum(float v) {
  static_assert(N == 8 || N == 16 || N == 32 || N == 64, "");
  v = dpp_add<0xB1>(v);
  v = dpp_add<0x4E>(v);
  v = dpp_add<0x141>(v);
  if (N >= 16) v = dpp_add<0x140>(v);
  if (N >= 32) v += __shfl_xor(v, 16, 64);
  if (N >= 64) v += __shfl_xor(v, 32, 64);
  return v;
}

// Sums of NV values over the LPR lanes of a row, in every one of them; the
// workgroup holds RPB rows, this lane's being the ri-th.  Rows of more than 64
// lanes need the whole workgroup here, and red is its LDS for this; two calls in
// a row need no barrier between them if they use two of them.
constexpr int waves_of(int lanes) { return lanes > 64 ? lanes / 64 : 1; }
template <int LPR, int NV, int RPB = 1>
COLI_DEV void row_sums(float (&v)[NV], float (*red)[RPB * waves_of(LPR)], int ri = 0) {
#pragma unroll
  for (int n = 0; n < NV; ++n) v[n] = lanes_sum<(LPR < 64 ? LPR : 64)>(v[n]);
  if (LPR <= 64) return;
  constexpr int W = waves_of(LPR);
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int n = 0; n < NV; ++n) red[n][wave] = v[n];
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    v[n] = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) v[n] += red[n][(RPB > 1 ? ri * W : 0) + w];
  }
}

}  // namespace coli
