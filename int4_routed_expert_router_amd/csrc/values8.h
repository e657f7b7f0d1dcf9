// values8.h -- eight neighbouring values of a bf16 or fp32 array, the unit in
// which the row kernels move data (16 or 32 bytes).
#pragma once

#include "device_common.h"

namespace coli {

// Loads and stores that leave the caches to others (NT), for buffers that are
// several times the 256 MB of the chip's last cache: their own next reader
// finds nothing of them there anyway.
typedef unsigned int coli_u32x4 __attribute__((ext_vector_type(4)));
template <bool NT>
COLI_DEV uint4 load16(const uint4 *p) {
  if (!NT) return *p;
  const coli_u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const coli_u32x4 *>(p));
  return make_uint4(v.x, v.y, v.z, v.w);
}
template <bool NT>
COLI_DEV void store16(uint4 *p, uint4 a) {
  const coli_u32x4 v = {a.x, a.y, a.z, a.w};
  if (NT)
    __builtin_nontemporal_store(v, reinterpret_cast<coli_u32x4 *>(p));
  else
    *p = a;
}

COLI_DEV void unpack8(const uint4 u, float v[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// Two fp32 -> bf16, round to nearest even, by the hardware's conversion (one
// instruction for what takes a dozen in integers).
COLI_DEV uint32_t pack2(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, coli_bf16x2));
}

COLI_DEV uint4 pack8(const float v[8]) {
  return make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}

// Values 8i .. 8i+7 of p.
template <bool F32>
COLI_DEV void load8(const void *p, int64_t i, float v[8]) {
  if (F32) {
    const float4 a = reinterpret_cast<const float4 *>(p)[2 * i];
    const float4 b = reinterpret_cast<const float4 *>(p)[2 * i + 1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    unpack8(reinterpret_cast<const uint4 *>(p)[i], v);
  }
}

template <bool F32>
COLI_DEV void store8(void *p, int64_t i, const float v[8]) {
  if (F32) {
    reinterpret_cast<float4 *>(p)[2 * i] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[2 * i + 1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    reinterpret_cast<uint4 *>(p)[i] = pack8(v);
  }
}

}  // namespace coli
