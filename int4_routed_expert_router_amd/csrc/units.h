// units.h -- neighbouring values of a bf16 or fp32 array, the units in which
// the row kernels move data: eight values (16 or 32 bytes) or four.
#pragma once

#include "device_common.h"

namespace coli {

// Loads and stores that leave the caches to others (NT), for buffers that take
// up much of the 256 MB of the chip's last cache.
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

// U = 4 or 8 values as loaded, and U of them from index U * i on.  Rows of fp32
// go in fours, so that each load and store of a wave is one run of memory: of
// two 16-byte halves at 32-byte distance, past the caches, each would be half a
// line.
typedef unsigned int coli_u32x2 __attribute__((ext_vector_type(2)));
template <int U, bool F32>
struct Unit {
  uint32_t w[U * (F32 ? 4 : 2) / 4];
};
template <int U, bool F32, bool NT>
COLI_DEV Unit<U, F32> load_unit(const void *p, int64_t i) {
  constexpr int N = U * (F32 ? 4 : 2) / 4;  // words
  Unit<U, F32> r;
  const uint32_t *at = reinterpret_cast<const uint32_t *>(p) + i * N;
  if (N == 2) {
    const coli_u32x2 *q = reinterpret_cast<const coli_u32x2 *>(at);
    const coli_u32x2 v = NT ? __builtin_nontemporal_load(q) : *q;
    r.w[0] = v.x, r.w[1] = v.y;
  } else {
#pragma unroll
    for (int h = 0; h < N / 4; ++h) {
      const uint4 v = load16<NT>(reinterpret_cast<const uint4 *>(at) + h);
      r.w[4 * h] = v.x, r.w[4 * h + 1] = v.y;
      r.w[4 * h + 2] = v.z, r.w[4 * h + 3] = v.w;
    }
  }
  return r;
}
template <int U, bool F32>
COLI_DEV void unpack(const Unit<U, F32> &r, float (&v)[U]) {
#pragma unroll
  for (int j = 0; j < U; ++j)
    v[j] = F32 ? __uint_as_float(r.w[F32 ? j : 0])
               : __uint_as_float(j & 1 ? r.w[j / 2] & 0xffff0000u : r.w[j / 2] << 16);
}
template <int U, bool F32>
COLI_DEV Unit<U, F32> pack(const float (&v)[U]) {
  Unit<U, F32> r;
  if (F32) {
#pragma unroll
    for (int j = 0; j < U; ++j) r.w[F32 ? j : 0] = __float_as_uint(v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < U; j += 2) r.w[j / 2] = pack2(v[j], v[j + 1]);
  }
  return r;
}
template <int U, bool F32, bool NT>
COLI_DEV void store_unit(void *p, int64_t i, const Unit<U, F32> &r) {
  constexpr int N = U * (F32 ? 4 : 2) / 4;
  uint32_t *at = reinterpret_cast<uint32_t *>(p) + i * N;
  if (N == 2) {
    const coli_u32x2 v = {r.w[0], r.w[1]};
    coli_u32x2 *q = reinterpret_cast<coli_u32x2 *>(at);
    if (NT)
      __builtin_nontemporal_store(v, q);
    else
      *q = v;
  } else {
#pragma unroll
    for (int h = 0; h < N / 4; ++h)
      store16<NT>(reinterpret_cast<uint4 *>(at) + h,
                  make_uint4(r.w[4 * h], r.w[4 * h + 1], r.w[4 * h + 2], r.w[4 * h + 3]));
  }
}

}  // namespace coli
