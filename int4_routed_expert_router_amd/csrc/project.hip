// project.hip -- one expert matrix times the batch with the low-rank adapters
// of many requests beside it, and the backward pass.
//
//   u[t]  = c_a A_a x[t]                   a = adapter of row t
//   y[t]  = W x[t] + B_a u[t]
// and, W frozen,
//   v[t]  = c_a B_a^T dy[t]
//   dx[t] = W^T dy[t] + A_a^T v[t]
//   dA_a  = sum of v[t] x[t]^T,  dB_a = sum of dy[t] u[t]^T  over a's rows.
//
// W is one matrix of the layer's container (codes q, a scale per group along
// K); x, dy, A and B are bf16; all sums are fp32 on the bf16 matrix cores,
// whose products of bf16 values are exact.  Codes are exact in bf16, so y
// uses w = q*s exactly: each 64-wide group's partial product is multiplied by
// its scale in fp32.  W^T in dx is contracted across groups, where the scale
// cannot be taken out of the sum: there w is rounded to bf16, half a step of
// the type that dx itself is rounded to.  u and v stay fp32 and enter the
// matrix cores as sums of two bf16 parts (16 bits of mantissa, for bf16
// results) or three (24 bits, for fp32 ones).
//
// Kernels
//  prep   : container codes -> a bf16 plane (transposed for dx; A and B too).
//  shrink : u or v, 64-row tiles, split along the long axis.
//  gemm   : y or dx, an LDS-tiled matrix-core product; the rows' adapters are
//           added in registers at the end.
//  finish : sums shrink's parts, transposes u and v for the next kernel.
//  grads  : dA and dB, contractions over the rows of one adapter.
#include "internal.h"
#include "spans.h"

namespace coli {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
#define COLI_LDS __attribute__((address_space(3)))

COLI_DEV f32x4 mfma(const uint4 &a, const uint4 &b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
COLI_DEV uint4 ld16(const void *p) { return *reinterpret_cast<const uint4 *>(p); }
COLI_DEV uint4 zero4() { return make_uint4(0, 0, 0, 0); }
COLI_DEV void dma16(const void *g, void *lds) {
  __builtin_amdgcn_global_load_lds(g, (COLI_LDS void *)lds, 16, 0, 0);
}
COLI_DEV void wait_dma() { __builtin_amdgcn_s_waitcnt(0x0F70); }  // vmcnt(0)

COLI_DEV uint32_t pack_bf16(float lo, float hi) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  b2 v;
  v[0] = (__bf16)lo;
  v[1] = (__bf16)hi;
  return __builtin_bit_cast(uint32_t, v);
}
// v as a sum of P bf16 parts, each the rounding of what the earlier ones
// leave; an infinity stays in the first part.
template <int P>
COLI_DEV void split8(const float (&v)[8], uint4 (&out)[P]) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = v[i];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    uint32_t d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      d[i] = pack_bf16(r[2 * i], r[2 * i + 1]);
      const float lo = __uint_as_float(d[i] << 16), hi = __uint_as_float(d[i] & 0xffff0000u);
      r[2 * i] = r[2 * i] == lo ? 0.0f : r[2 * i] - lo;
      r[2 * i + 1] = r[2 * i + 1] == hi ? 0.0f : r[2 * i + 1] - hi;
    }
    out[p] = make_uint4(d[0], d[1], d[2], d[3]);
  }
}

// keeps the first n of eight bf16 values
COLI_DEV uint4 keep_first(uint4 v, int n) {
  uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    d[i] = n >= 2 * i + 2 ? d[i] : (n == 2 * i + 1 ? d[i] & 0xffffu : 0u);
  return make_uint4(d[0], d[1], d[2], d[3]);
}

// Sum of A accumulators over NW wavefronts, in wavefront 0, pairwise through
// LDS (buf: NW/2 * A rows).
template <int A, int NW>
COLI_DEV void wave_sums(f32x4 *acc, f32x4 (*buf)[64], int wv, int lane) {
#pragma unroll
  for (int half = NW / 2; half > 0; half >>= 1) {
    __syncthreads();
    if (wv >= half && wv < 2 * half) {
#pragma unroll
      for (int i = 0; i < A; ++i) buf[(wv - half) * A + i][lane] = acc[i];
    }
    __syncthreads();
    if (wv < half) {
#pragma unroll
      for (int i = 0; i < A; ++i) acc[i] += buf[wv * A + i][lane];
    }
  }
}

struct Adapters {
  const uint16_t *a, *b;  // [n][R][K], [n][N][R]
  const int32_t *rank;    // [n] or NULL
  const float *scale;     // [n] or NULL
  int R;
};
COLI_DEV int rank_of(const int32_t *rank, int a, int R) {
  return rank ? min(max(rank[a], 0), R) : R;
}

// One matrix of the container.
enum { kI4 = 0, kI8 = 1, kF4 = 2 };
struct Matrix {
  const uint8_t *q;   // codes, row n at n * row_bytes
  const uint8_t *sc;  // scales: fp16 per 64, or E8M0 per 32 (kF4)
  int N, K;
};

// ------------------------------------------------------------------- prep

// Eight consecutive weights' codes (k8 a multiple of 8 inside row n) as fp32.
template <int F>
COLI_DEV void codes8(const Matrix &m, int n, int k8, float (&w)[8]) {
  if (F == kI8) {
    const uint2 v = *reinterpret_cast<const uint2 *>(m.q + (int64_t)n * m.K + k8);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = (float)(int8_t)((i < 4 ? v.x : v.y) >> (8 * (i & 3)));
    return;
  }
  const uint32_t v = *reinterpret_cast<const uint32_t *>(m.q + ((int64_t)n * m.K + k8) / 2);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t nib = (v >> (4 * i)) & 15u;
    if (F == kI4) {
      w[i] = (float)((int)(nib ^ 8u) - 8);
    } else {
      // E2M1: exponent 0 holds 0 and 0.5, else (1 + m/2) * 2^(e-1)
      const uint32_t e = (nib >> 1) & 3u, mant = nib & 1u;
      const float mag = e ? (1.0f + 0.5f * mant) * (float)(1u << e) * 0.5f : 0.5f * mant;
      w[i] = (nib & 8u) ? -mag : mag;
    }
  }
}
// Scale of weight (n, k).
template <int F>
COLI_DEV float scale_at(const Matrix &m, int n, int k) {
  if (F == kF4) {
    const uint32_t e = m.sc[(int64_t)n * (m.K / 32) + k / 32];
    return __uint_as_float(e ? e << 23 : 0x00400000u);
  }
  return f16_to_f32(reinterpret_cast<const uint16_t *>(m.sc)[(int64_t)n * (m.K / 64) + k / 64]);
}

// Plane [N][K]: the codes (int4, int8; exact), with the scales as fp32
// [K/64][N]; or the weights themselves (MXFP4: a code times a power of two).
template <int F>
__global__ void __launch_bounds__(256) prep_kernel(Matrix m, uint16_t *plane, float *sc) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t total = (int64_t)m.N * m.K / 8;
  if (i >= total) return;
  const int n = (int)(i / (m.K / 8)), k = (int)(i % (m.K / 8)) * 8;
  float w[8];
  codes8<F>(m, n, k, w);
  if (F == kF4) {
    const float s = scale_at<F>(m, n, k);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] *= s;
  } else if (k % 64 == 0) {
    sc[(int64_t)(k / 64) * m.N + n] = scale_at<F>(m, n, k);
  }
  uint32_t d[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) d[j] = pack_bf16(w[2 * j], w[2 * j + 1]);
  *reinterpret_cast<uint4 *>(plane + 8 * i) = make_uint4(d[0], d[1], d[2], d[3]);
}

// The backward pass's operands: the weights as bf16 [K][N], and A and B of
// every adapter in use transposed to [K][R] and [R][N].  One 64 x 64 tile
// per workgroup, through LDS.
struct PrepT {
  Matrix m;
  uint16_t *wt;  // [K][N] or NULL
  Adapters ad;
  Requests q;
  uint16_t *at, *bt;  // [n][K][R], [n][R][N]
  int w_tiles, a_tiles, b_tiles;  // workgroups of each kind (a, b per adapter)
};
template <int F>
__global__ void __launch_bounds__(256) prep_transposed_kernel(PrepT g) {
  __shared__ uint16_t t[64][66];
  __shared__ int used;
  const int tid = threadIdx.x;
  int b = blockIdx.x;
  const uint16_t *src;
  uint16_t *dst;
  int rows, cols;  // of the source
  int r0, c0;
  if (b < g.w_tiles) {
    const int ct = g.m.K / 64;
    r0 = b / ct * 64;
    c0 = b % ct * 64;
    rows = g.m.N;
    cols = g.m.K;
    dst = g.wt;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = (tid >> 3) + 32 * h, c = (tid & 7) * 8;
      float w[8];
      codes8<F>(g.m, r0 + r, c0 + c, w);
      const float s = scale_at<F>(g.m, r0 + r, c0 + c);
#pragma unroll
      for (int j = 0; j < 8; ++j) t[c + j][r] = (uint16_t)f32_to_bf16_bits(w[j] * s);
    }
  } else {
    b -= g.w_tiles;
    const int per = g.a_tiles + g.b_tiles, a = b / per;
    b %= per;
    if (tid == 0) used = 0;
    __syncthreads();
    for (int i = tid; i < g.q.n; i += 256)
      if (g.q.adapter[i] == a && g.q.off[i + 1] > g.q.off[i]) used = 1;
    __syncthreads();
    if (!used) return;
    const int R = g.ad.R;
    if (b < g.a_tiles) {
      const int ct = g.m.K / 64;
      rows = R;
      cols = g.m.K;
      r0 = b / ct * 64;
      c0 = b % ct * 64;
      src = g.ad.a + (int64_t)a * R * g.m.K;
      dst = g.at + (int64_t)a * R * g.m.K;
    } else {
      b -= g.a_tiles;
      const int ct = (R + 63) / 64;
      rows = g.m.N;
      cols = R;
      r0 = b / ct * 64;
      c0 = b % ct * 64;
      src = g.ad.b + (int64_t)a * R * g.m.N;
      dst = g.bt + (int64_t)a * R * g.m.N;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = (tid >> 3) + 32 * h, c = (tid & 7) * 8;
      if (r0 + r < rows && c0 + c < cols) {
        const uint4 v = ld16(src + (int64_t)(r0 + r) * cols + c0 + c);
        const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) t[c + j][r] = (uint16_t)(d[j >> 1] >> (16 * (j & 1)));
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = (tid >> 3) + 32 * h, r = (tid & 7) * 8;
    if (c0 + c < cols && r0 + r < rows) {  // rows and cols are multiples of 8
      uint32_t d[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        d[j] = (uint32_t)t[c][r + 2 * j] | (uint32_t)t[c][r + 2 * j + 1] << 16;
      *reinterpret_cast<uint4 *>(dst + (int64_t)(c0 + c) * rows + r0 + r) =
          make_uint4(d[0], d[1], d[2], d[3]);
    }
  }
}

// ----------------------------------------------------------------- shrink

// part[split][t][r] = scale * sum over the split's k of z[t][k] m[a][r][k].
struct ShrinkArgs {
  const uint16_t *z;  // [T][F]
  const uint16_t *m;  // [n][R][F]
  const int32_t *rank;
  const float *scale;
  Requests q;
  float *part;  // [splits][T][R32]
  int T, F, R, R32, splits, nsub;
};

// One workgroup per tile of 16 MI rows, split and residue of the tile's
// requests modulo nsub (so that a tile of many one-row requests spreads over
// many workgroups).  Its NW wavefronts take the split's 64-wide k blocks in
// turn; operands come straight from memory: lane (c, g) holds 16 values of
// row c at k = 16g, two matrix-core steps.
template <int RT, int MI, int NW>
COLI_DEV void shrink_tile(const ShrinkArgs &g, int tile, int sub, int split, f32x4 (*buf)[64]) {
  const int lane = threadIdx.x & 63, c = lane & 15, kg = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t0 = tile * (16 * MI), t1 = min(g.T, t0 + 16 * MI);
  const int nb = g.F / 64;
  for_requests(g.q, t0, t1, [&](int ordinal, int begin, int end, int a) {
    if (ordinal % g.nsub != sub) return;
    const int rank = rank_of(g.rank, a, g.R);
    f32x4 acc[MI][RT];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[i][r] = f32x4{0, 0, 0, 0};
    const uint16_t *mrow = g.m + ((int64_t)a * g.R + c) * g.F + 16 * kg;
    const uint16_t *zrow = g.z + (int64_t)(t0 + c) * g.F + 16 * kg;
    for (int b = split * NW + wv; b < nb; b += NW * g.splits) {
      uint4 mf[RT][2];
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          mf[r][h] = 16 * r + c < rank ? ld16(mrow + (int64_t)16 * r * g.F + 64 * b + 8 * h) : zero4();
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        if (MI > 1 && (begin >= t0 + 16 * i + 16 || end <= t0 + 16 * i)) continue;
        const int t = t0 + 16 * i + c;
        uint4 zf[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          zf[h] = t >= begin && t < end ? ld16(zrow + (int64_t)16 * i * g.F + 64 * b + 8 * h) : zero4();
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < RT; ++r) acc[i][r] = mfma(zf[h], mf[r][h], acc[i][r]);
      }
    }
    wave_sums<MI * RT, NW>(&acc[0][0], buf, wv, lane);
    if (wv == 0) {
      const float s = g.scale ? g.scale[a] : 1.0f;
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int t = t0 + 16 * i + 4 * kg + j;
            if (t >= begin && t < end && 16 * r + c < g.R32)
              g.part[((int64_t)split * g.T + t) * g.R32 + 16 * r + c] = s * acc[i][r][j];
          }
    }
  });
}

template <int RT>
__global__ void __launch_bounds__(256) shrink_kernel(ShrinkArgs g0, ShrinkArgs g1) {
  __shared__ f32x4 buf[2 * 4 * RT][64];
  // z: the first operand's splits, then the second's
  const bool second = (int)blockIdx.z >= g0.splits;
  const ShrinkArgs &g = second ? g1 : g0;
  shrink_tile<RT, 4, 4>(g, blockIdx.x, blockIdx.y, second ? blockIdx.z - g0.splits : blockIdx.z, buf);
}

// ------------------------------------------------------------------- gemm

// The adapters' side of an output: b [n][N][R] bf16 and shrink's u.
struct ExpandArgs {
  Requests q;
  const float *u;  // [splits][T][R32]
  const uint16_t *b;
  const int32_t *rank;
  int T, N, R, R32, splits;
};

// This lane's operand values u[t][k .. k+8), the splits added up, as P parts.
template <int P>
COLI_DEV void load_u(const ExpandArgs &g, int t, int k, bool live, uint4 (&uf)[P]) {
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 0.0f;
  if (live) {
    const float *p = g.u + (int64_t)t * g.R32 + k;
#pragma unroll 4
    for (int s = 0; s < g.splits; ++s) {
      const float4 lo = *reinterpret_cast<const float4 *>(p + (int64_t)s * g.T * g.R32);
      const float4 hi = *reinterpret_cast<const float4 *>(p + (int64_t)s * g.T * g.R32 + 4);
      v[0] += lo.x;
      v[1] += lo.y;
      v[2] += lo.z;
      v[3] += lo.w;
      v[4] += hi.x;
      v[5] += hi.y;
      v[6] += hi.z;
      v[7] += hi.w;
    }
  }
  split8<P>(v, uf);
}
// Ranks [k, k + 8) of the adapter's columns n0 + 4c + j.
COLI_DEV void load_b(const ExpandArgs &g, int a, int n0, int k, int rank, uint4 (&bf)[4]) {
  const int c = threadIdx.x & 15;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int n = min(n0 + 4 * c + j, g.N - 1);
    bf[j] = k < rank ? keep_first(ld16(g.b + ((int64_t)a * g.N + n) * g.R + k), rank - k) : zero4();
  }
}

// acc += the adapters' part of the wavefront's MI x 4 tiles: rows t0 + 16i +
// c, columns n0 + 4c + j.  Every request with rows here multiplies only the
// 16-row tiles that it reaches, its other rows as zeros.
template <int MI, int P>
COLI_DEV void expand(const ExpandArgs &g, int t0, int n0, f32x4 (&acc)[MI][4]) {
  const int lane = threadIdx.x & 63, c = lane & 15, kg = lane >> 4;
  const int t1 = min(g.T, t0 + 16 * MI);
  if (t0 >= t1) return;
  for_requests(g.q, t0, t1, [&](int, int begin, int end, int a) {
    const int rank = rank_of(g.rank, a, g.R);
    for (int k0 = 0; k0 < rank; k0 += 32) {
      const int k = k0 + 8 * kg;  // this lane's eight ranks
      uint4 bf[4];
      load_b(g, a, n0, k, rank, bf);
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        if (begin >= t0 + 16 * i + 16 || end <= t0 + 16 * i) continue;
        const int t = t0 + 16 * i + c;
        uint4 uf[P];
        load_u<P>(g, t, k, t >= begin && t < end && k < rank, uf);
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = mfma(uf[p], bf[j], acc[i][j]);
      }
    }
  });
}

// Four neighbouring columns of one row.
template <bool F32>
COLI_DEV void store4(void *y, int64_t at, float a, float b, float c, float d) {
  if (F32)
    *reinterpret_cast<float4 *>(static_cast<float *>(y) + at) = make_float4(a, b, c, d);
  else
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(y) + at) =
        make_uint2(pack_bf16(a, b), pack_bf16(c, d));
}

struct GemmArgs {
  const uint16_t *x;  // [T][K] bf16
  const uint16_t *w;  // [N][K] bf16
  const float *sc;    // [K/64][N] or unused
  int T, N, K;
  void *y;  // [T][N]
  ExpandArgs e;  // u NULL: no adapters
};

// BM x BN tile, wavefronts of WM x 64.  Stages of 64 k go global -> LDS by
// DMA, two in turn.  A row's 16-byte chunk q is kept at q ^ (row & 7) for x
// and at q ^ ((row >> 2) & 7) for w, whose rows are read in the order
// n = 4c + j: lane c then ends up with four neighbouring columns, stored
// together, and neither operand read meets a bank conflict.
template <int BM, int BN, int WM, bool SCALED, bool F32>
__global__ void __launch_bounds__(BM / WM *BN / 64 * 64) gemm_kernel(GemmArgs g) {
  constexpr int NW = (BM / WM) * (BN / 64), MI = WM / 16;
  constexpr int LD = (BM + BN) / 8 / NW;  // DMA instructions of a wavefront per stage
  __shared__ uint4 lds[2][(BM + BN) * 8];
  const int lane = threadIdx.x & 63, c = lane & 15, kg = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tm = blockIdx.y * BM, tn = blockIdx.x * BN;
  const int wm = (wv / (BN / 64)) * WM, wn = (wv % (BN / 64)) * 64;

  const uint16_t *src[LD];
#pragma unroll
  for (int i = 0; i < LD; ++i) {
    const int row = (wv * LD + i) * 8 + (lane >> 3), pos = lane & 7;
    if (row < BM) {
      src[i] = g.x + (int64_t)min(tm + row, g.T - 1) * g.K + 8 * (pos ^ (row & 7));
    } else {
      const int r = row - BM;
      src[i] = g.w + (int64_t)min(tn + r, g.N - 1) * g.K + 8 * (pos ^ ((r >> 2) & 7));
    }
  }
  auto issue = [&](int st) {
#pragma unroll
    for (int i = 0; i < LD; ++i) dma16(src[i] + 64 * st, &lds[st & 1][(wv * LD + i) * 64]);
  };
  f32x4 acc[MI][4];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  const int n0 = tn + wn;
  const bool cols = n0 < g.N;  // N is a multiple of 64
  const float *scp = g.sc + n0 + 4 * c;
  const int nst = g.K / 64;
  issue(0);
  for (int st = 0; st < nst; ++st) {
    float4 s4 = make_float4(1, 1, 1, 1);
    if (SCALED && cols) s4 = *reinterpret_cast<const float4 *>(scp + (int64_t)st * g.N);
    wait_dma();
    __syncthreads();
    if (st + 1 < nst) issue(st + 1);
    const uint4 *A = lds[st & 1], *B = A + BM * 8;
    uint4 bf[4][2];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        bf[j][h] = B[(wn + 4 * c + j) * 8 + ((2 * kg + h) ^ (c & 7))];
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      uint4 af[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) af[h] = A[(wm + 16 * i + c) * 8 + ((2 * kg + h) ^ (c & 7))];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (SCALED) {
          f32x4 d = mfma(af[0], bf[j][0], f32x4{0, 0, 0, 0});
          d = mfma(af[1], bf[j][1], d);
          const float s = j == 0 ? s4.x : (j == 1 ? s4.y : (j == 2 ? s4.z : s4.w));
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(d[e], s, acc[i][j][e]);
        } else {
          acc[i][j] = mfma(af[0], bf[j][0], acc[i][j]);
          acc[i][j] = mfma(af[1], bf[j][1], acc[i][j]);
        }
      }
    }
  }
  if (!cols) return;
  if (g.e.u) expand<MI, F32 ? 3 : 2>(g.e, tm + wm, n0, acc);
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = tm + wm + 16 * i + 4 * kg + e;
      if (t < g.T)
        store4<F32>(g.y, (int64_t)t * g.N + n0 + 4 * c, acc[i][0][e], acc[i][1][e], acc[i][2][e],
                    acc[i][3][e]);
    }
}

// ----------------------------------------------------------------- stream
//
// Short batches: the codes go from memory straight into registers, so that a
// call costs one pass over the container and two launches.  The first
// computes W x in parts (split along K) and u side by side; the second adds
// the parts and the adapters.

struct StreamArgs {
  Matrix m;
  const uint16_t *x;  // [T][K]
  float *part;        // [splits][T][N]
  int T, splits, per;  // per: 64-wide groups of a wavefront
  int shrink_blocks, shrink_tiles;
  ShrinkArgs s;
};

constexpr int kStreamWaves = 8;

// Raw operands of one 64-wide group of a row: 16 codes per lane (k = 16g of
// the group, g = lane / 16), in two steps of eight.
template <int F>
struct Raw {
  uint32_t w[F == kI8 ? 4 : 2];
  uint32_t s;
};
template <int F>
COLI_DEV Raw<F> load_raw(const Matrix &m, int n, int b, int kg) {
  Raw<F> r;
  if (F == kI8) {
    const uint4 v = ld16(m.q + (int64_t)n * m.K + 64 * b + 16 * kg);
    r.w[F == kI8 ? 2 : 0] = v.z;
    r.w[F == kI8 ? 3 : 0] = v.w;
    r.w[0] = v.x;
    r.w[1] = v.y;
  } else {
    const uint2 v = *reinterpret_cast<const uint2 *>(m.q + ((int64_t)n * m.K + 64 * b + 16 * kg) / 2);
    r.w[0] = v.x;
    r.w[1] = v.y;
  }
  if (F == kF4) r.s = m.sc[(int64_t)n * (m.K / 32) + 2 * b + (kg >> 1)];
  else r.s = reinterpret_cast<const uint16_t *>(m.sc)[(int64_t)n * (m.K / 64) + b];
  return r;
}
// Step h as a matrix-core operand.  int4: the bf16 value 24 + q (a nibble in
// the mantissa of 16 .. 31), pairs (k, k + 4); the bias leaves through the
// accumulator's start value, -24 times the row's sum of x.  int8: exact
// values.  MXFP4: the weights themselves.
template <int F>
COLI_DEV uint4 unpack(const Raw<F> &r, int h) {
  if (F == kI4) {
    const uint32_t w = r.w[h];
    constexpr uint32_t M = 0x00780078u, X = 0x41c041c0u;
    return make_uint4(__builtin_amdgcn_bitop3_b32(w << 3, M, X, kAndXor),
                      __builtin_amdgcn_bitop3_b32(w >> 1, M, X, kAndXor),
                      __builtin_amdgcn_bitop3_b32(w >> 5, M, X, kAndXor),
                      __builtin_amdgcn_bitop3_b32(w >> 9, M, X, kAndXor));
  }
  if (F == kI8) {
    uint32_t d[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t v = r.w[F == kI8 ? 2 * h + i : 0];
      d[2 * i] = pack_bf16((float)(int8_t)v, (float)(int8_t)(v >> 8));
      d[2 * i + 1] = pack_bf16((float)(int8_t)(v >> 16), (float)(int8_t)(v >> 24));
    }
    return make_uint4(d[0], d[1], d[2], d[3]);
  }
  const float s = __uint_as_float(r.s ? r.s << 23 : 0x00400000u);
  const uint32_t w = r.w[h];
  return make_uint4(
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3)));
}

// One workgroup: 16 MT rows x 16 NJ columns (n0 + NJ c + j) over one split of
// K; its wavefronts take neighbouring runs of `per` groups, GB of them loaded
// ahead of their use.
template <int F, int MT, int NJ, int GB>
COLI_DEV void stream_tile(const StreamArgs &g, int nt, int tt, int split, f32x4 (*buf)[64]) {
  const int lane = threadIdx.x & 63, c = lane & 15, kg = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = nt * (16 * NJ), t0 = tt * (16 * MT);
  const int b0 = (split * kStreamWaves + wv) * g.per, b1 = min(g.m.K / 64, b0 + g.per);
  f32x4 acc[MT][NJ];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  const uint16_t *xrow = g.x + (int64_t)(t0 + c) * g.m.K + 16 * kg;
  for (int b = b0; b < b1; b += GB) {
    Raw<F> raw[GB][NJ];
    uint4 xr[GB][MT][2];
#pragma unroll
    for (int i = 0; i < GB; ++i) {
      if (b + i >= b1) continue;
#pragma unroll
      for (int j = 0; j < NJ; ++j) raw[i][j] = load_raw<F>(g.m, n0 + NJ * c + j, b + i, kg);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          xr[i][m][h] = t0 + 16 * m + c < g.T
                            ? ld16(xrow + (int64_t)16 * m * g.m.K + 64 * (b + i) + 8 * h)
                            : zero4();
    }
#pragma unroll
    for (int i = 0; i < GB; ++i) {
      if (b + i >= b1) continue;
      f32x4 start[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        start[m] = f32x4{0, 0, 0, 0};
        if (F == kI4) {
          constexpr uint32_t kMinus24 = 0xc1c0c1c0u;
          const uint4 ones = make_uint4(kMinus24, kMinus24, kMinus24, kMinus24);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t d[4] = {xr[i][m][h].x, xr[i][m][h].y, xr[i][m][h].z, xr[i][m][h].w};
            uint32_t o[4];
            x8_to_pairs(d, o);
            xr[i][m][h] = make_uint4(o[0], o[1], o[2], o[3]);
            start[m] = mfma(xr[i][m][h], ones, start[m]);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const uint4 w0 = unpack<F>(raw[i][j], 0), w1 = unpack<F>(raw[i][j], 1);
        const float s = F == kF4 ? 1.0f : f16_to_f32((uint16_t)raw[i][j].s);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          f32x4 d = F == kF4 ? acc[m][j] : start[m];
          d = mfma(xr[i][m][0], w0, d);
          d = mfma(xr[i][m][1], w1, d);
          if (F == kF4) {
            acc[m][j] = d;
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[m][j][e] = fmaf(d[e], s, acc[m][j][e]);
          }
        }
      }
    }
  }
  wave_sums<MT * NJ, kStreamWaves>(&acc[0][0], buf, wv, lane);
  if (wv != 0) return;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = t0 + 16 * m + 4 * kg + e;
      if (t >= g.T) continue;
      float *p = g.part + ((int64_t)split * g.T + t) * g.m.N + n0 + NJ * c;
      if (NJ == 4) {
        *reinterpret_cast<float4 *>(p) =
            make_float4(acc[m][0][e], acc[m][NJ > 1][e], acc[m][NJ > 2 ? 2 : 0][e], acc[m][NJ > 3 ? 3 : 0][e]);
      } else {
#pragma unroll
        for (int j = 0; j < NJ; ++j) p[j] = acc[m][j][e];
      }
    }
}

template <int F, int MT, int NJ, int GB, int RT>
__global__ void __launch_bounds__(64 * kStreamWaves) stream_kernel(StreamArgs g) {
  constexpr int A = MT * NJ > RT ? MT * NJ : RT;
  __shared__ f32x4 buf[kStreamWaves / 2 * A][64];
  int b = blockIdx.x;
  if (b < g.shrink_blocks) {
    const int tile = b % g.shrink_tiles;
    b /= g.shrink_tiles;
    shrink_tile<RT, 1, kStreamWaves>(g.s, tile, b % g.s.nsub, b / g.s.nsub, buf);
    return;
  }
  b -= g.shrink_blocks;
  const int nt = g.m.N / (16 * NJ), tt = (g.T + 16 * MT - 1) / (16 * MT);
  const int n = b % nt;
  b /= nt;
  stream_tile<F, MT, NJ, GB>(g, n, b % tt, b / tt, buf);
}

// y = the sum of the parts, plus the adapters.  A wavefront takes 64 columns
// of one 16-row tile and every nsub-th request with rows there, so that one-
// row requests run side by side; the first of them also writes the rows
// without an adapter.
struct CombineArgs {
  const float *part;  // [splits][T][N]
  int splits, nsub;
  void *y;
  ExpandArgs e;
};
template <bool F32>
__global__ void __launch_bounds__(256) combine_parts_kernel(CombineArgs g) {
  const int lane = threadIdx.x & 63, c = lane & 15, kg = lane >> 4;
  const int n0 = (blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * 64;
  if (n0 >= g.e.N) return;
  const int t0 = blockIdx.y * 16, t1 = min(g.e.T, t0 + 16), sub = blockIdx.z;
  uint32_t covered = 0;
  auto rows = [&](int begin, int end, uint32_t mask, int a) {
    f32x4 acc[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = 4 * kg + e;
      const bool mine = (mask >> r) & 1u;
      float4 v = make_float4(0, 0, 0, 0);
      if (mine) {
        const float *p = g.part + (int64_t)(t0 + r) * g.e.N + n0 + 4 * c;
#pragma unroll 4
        for (int s = 0; s < g.splits; ++s) {
          const float4 o = *reinterpret_cast<const float4 *>(p + (int64_t)s * g.e.T * g.e.N);
          v.x += o.x;
          v.y += o.y;
          v.z += o.z;
          v.w += o.w;
        }
      }
      acc[0][e] = v.x;
      acc[1][e] = v.y;
      acc[2][e] = v.z;
      acc[3][e] = v.w;
    }
    if (a >= 0) {
      constexpr int P = F32 ? 3 : 2;
      const int rank = rank_of(g.e.rank, a, g.e.R);
      const int t = t0 + c;
      for (int k0 = 0; k0 < rank; k0 += 32) {
        const int k = k0 + 8 * kg;
        uint4 bf[4], uf[P];
        load_b(g.e, a, n0, k, rank, bf);
        load_u<P>(g.e, t, k, t >= begin && t < end && k < rank, uf);
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[j] = mfma(uf[p], bf[j], acc[j]);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = 4 * kg + e;
      if ((mask >> r) & 1u)
        store4<F32>(g.y, (int64_t)(t0 + r) * g.e.N + n0 + 4 * c, acc[0][e], acc[1][e], acc[2][e],
                    acc[3][e]);
    }
  };
  if (g.e.u) {
    for_requests(g.e.q, t0, t1, [&](int ordinal, int begin, int end, int a) {
      const uint32_t mask = ((1u << (end - t0)) - 1u) & ~((1u << (begin - t0)) - 1u);
      covered |= mask;
      if (ordinal % g.nsub == sub) rows(begin, end, mask, a);
    });
  }
  const uint32_t rest = ((1u << (t1 - t0)) - 1u) & ~covered;
  if (sub == 0 && rest) rows(0, 0, rest, -1);
}

// ----------------------------------------------------------------- finish

// Sums shrink's parts of u and v.  Writes v as rows (fp32 [T][R32]), both
// transposed as three bf16 parts [3][R32][Tp], and every row's adapter;
// zeros for rows without one.
struct FinishArgs {
  Requests q;
  const float *part[2];  // u, v
  int splits[2];
  float *rows;           // v
  uint16_t *planes[2];
  int32_t *owner;        // [Tp]
  int T, Tp, R32;
};
__global__ void __launch_bounds__(256) finish_kernel(FinishArgs g) {
  __shared__ float s[64][33];
  __shared__ int own[64];
  const int tid = threadIdx.x, t0 = blockIdx.x * 64, r0 = blockIdx.y * 32, w = blockIdx.z;
  if (tid < 64) {
    const int t = t0 + tid;
    int a = -1;
    if (t < g.T) {
      int lo = 0, hi = g.q.n + 1;  // first entry past t
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (g.q.off[mid] <= t) lo = mid + 1;
        else hi = mid;
      }
      if (lo > 0 && lo <= g.q.n) a = g.q.adapter[lo - 1];
      if (a < 0 || a >= g.q.n_adapters) a = -1;
    }
    own[tid] = a;
    if (w == 0 && r0 == 0) g.owner[t] = a;
  }
  __syncthreads();
  for (int i = tid; i < 64 * 32; i += 256) {
    const int tt = i >> 5, r = i & 31;
    float v = 0.0f;
    if (own[tt] >= 0) {
      const float *p = g.part[w] + (int64_t)(t0 + tt) * g.R32 + r0 + r;
      for (int k = 0; k < g.splits[w]; ++k) v += p[(int64_t)k * g.T * g.R32];
    }
    if (w == 1 && t0 + tt < g.T) g.rows[(int64_t)(t0 + tt) * g.R32 + r0 + r] = v;
    s[tt][r] = v;
  }
  __syncthreads();
  const int r = tid >> 3, tt = (tid & 7) * 8;  // eight rows' values of one rank
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = s[tt + j][r];
  uint4 parts[3];
  split8<3>(v, parts);
#pragma unroll
  for (int p = 0; p < 3; ++p)
    *reinterpret_cast<uint4 *>(g.planes[w] + ((int64_t)p * g.R32 + r0 + r) * g.Tp + t0 + tt) = parts[p];
}

// ------------------------------------------------------------------ grads

// G_a[f][r] = sum over a's rows t of z[t][f] p[t][r].
struct GradArgs {
  const uint16_t *z;       // [T][F]
  const uint16_t *planes;  // [3][R32][Tp]
  float *out;              // [splits][n][R][F] (dA) or [splits][n][F][R] (dB)
  int F;
  int transposed;          // dB's layout
  int f_tiles;
};
struct GradsArgs {
  GradArgs g[2];  // dB (dy, u), dA (x, v)
  const int32_t *owner;
  int T, Tp, R, R32, n, splits, rows;  // rows per split, a multiple of 64
};

// A workgroup takes 128 columns f, one adapter, up to 16 RT ranks and one
// range of rows; its wavefronts take the range's 64-row windows in turn and
// skip rows of other adapters.  A step contracts 32 rows: lane (c, g) loads
// eight columns of eight rows, 16 bytes each, and an 8 x 8 transposition in
// registers turns them into one operand per column, so that tile j holds
// columns 8c + j.
template <int RT>
__global__ void __launch_bounds__(256) grads_kernel(GradsArgs a) {
  __shared__ f32x4 buf[2 * RT * 8][64];
  const int lane = threadIdx.x & 63, c = lane & 15, kg = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool second = (int)blockIdx.x >= a.g[0].f_tiles;
  const GradArgs &g = a.g[second];
  const int f0 = ((int)blockIdx.x - (second ? a.g[0].f_tiles : 0)) * 128 + 8 * c;
  const int ad = blockIdx.y;
  const int split = blockIdx.z % a.splits, r0 = blockIdx.z / a.splits * (16 * RT);
  const int row0 = split * a.rows, row1 = min(a.Tp, row0 + a.rows);
  const bool cols = f0 < g.F;
  f32x4 acc[RT][8];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[r][j] = f32x4{0, 0, 0, 0};
  for (int w0 = row0 + 64 * wv; w0 < row1; w0 += 256) {
    const uint64_t mine = __ballot(a.owner[w0 + lane] == ad);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t m32 = (uint32_t)(mine >> (32 * h));
      if (!m32) continue;
      const uint32_t m8 = (m32 >> (8 * kg)) & 255u;
      const int t = w0 + 32 * h + 8 * kg;
      uint32_t z[8][4];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4 v = cols && (m8 >> i & 1u) ? ld16(g.z + (int64_t)(t + i) * g.F + f0) : zero4();
        z[i][0] = v.x;
        z[i][1] = v.y;
        z[i][2] = v.z;
        z[i][3] = v.w;
      }
      uint4 pf[3][RT];
#pragma unroll
      for (int p = 0; p < 3; ++p)
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const int rr = r0 + 16 * r + c;
          uint4 v = rr < a.R32 ? ld16(g.planes + ((int64_t)p * a.R32 + rr) * a.Tp + t) : zero4();
          // other adapters' rows may hold anything
          if (m32 != 0xffffffffu) {
            uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              d[i] &= ((m8 >> (2 * i)) & 1u ? 0xffffu : 0u) | ((m8 >> (2 * i + 1)) & 1u ? 0xffff0000u : 0u);
            v = make_uint4(d[0], d[1], d[2], d[3]);
          }
          pf[p][r] = v;
        }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
        uint4 zf;
        zf.x = __builtin_amdgcn_perm(z[1][j >> 1], z[0][j >> 1], sel);
        zf.y = __builtin_amdgcn_perm(z[3][j >> 1], z[2][j >> 1], sel);
        zf.z = __builtin_amdgcn_perm(z[5][j >> 1], z[4][j >> 1], sel);
        zf.w = __builtin_amdgcn_perm(z[7][j >> 1], z[6][j >> 1], sel);
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
          for (int r = 0; r < RT; ++r) acc[r][j] = mfma(pf[p][r], zf, acc[r][j]);
      }
    }
  }
  wave_sums<RT * 8, 4>(&acc[0][0], buf, wv, lane);
  if (wv != 0 || !cols) return;
  float *out = g.out + ((int64_t)split * a.n + ad) * a.R * g.F;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int rr = r0 + 16 * r + 4 * kg;  // four ranks; R is a multiple of 8
    if (rr >= a.R) continue;
    if (g.transposed) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        *reinterpret_cast<f32x4 *>(out + (int64_t)(f0 + j) * a.R + rr) = acc[r][j];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float *p = out + (int64_t)(rr + e) * g.F + f0;
        *reinterpret_cast<float4 *>(p) =
            make_float4(acc[r][0][e], acc[r][1][e], acc[r][2][e], acc[r][3][e]);
        *reinterpret_cast<float4 *>(p + 4) =
            make_float4(acc[r][4][e], acc[r][5][e], acc[r][6][e], acc[r][7][e]);
      }
    }
  }
}

// out = sum of the splits' partial gradients, both gradients in one launch.
struct ReduceArgs {
  const float4 *src[2];
  float4 *dst[2];
  int64_t n[2];  // float4 values
  int splits;
};
__global__ void __launch_bounds__(256) reduce_kernel(ReduceArgs a) {
  int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int w = i >= a.n[0];
  if (w) i -= a.n[0];
  if (i >= a.n[w]) return;
  float4 v = a.src[w][i];
  for (int s = 1; s < a.splits; ++s) {
    const float4 o = a.src[w][s * a.n[w] + i];
    v.x += o.x;
    v.y += o.y;
    v.z += o.z;
    v.w += o.w;
  }
  a.dst[w][i] = v;
}

// ----------------------------------------------------------------- launch

Matrix matrix_of(const Layer &L, int expert, int matrix) {
  Matrix m;
  m.N = matrix == 2 ? L.H : L.I;
  m.K = matrix == 2 ? L.I : L.H;
  m.q = L.q4 + expert * L.expert_bytes + matrix * (L.expert_bytes / 3);
  m.sc = reinterpret_cast<const uint8_t *>(L.scales + expert * L.expert_scales +
                                           matrix * (L.expert_scales / 3));
  return m;
}
int format_of(const Layer &L) { return L.w8 ? kI8 : (L.f4 ? kF4 : kI4); }

int round32(int r) { return (r + 31) / 32 * 32; }
// Splits of shrink's long axis F: enough workgroups for the chip, at least
// 256 values each.
int shrink_splits(int T, int F) {
  const int tiles = (T + 63) / 64;
  int s = 512 / tiles;
  if (s > F / 256) s = F / 256;
  return s < 1 ? 1 : (s > 8 ? 8 : s);
}
// Row ranges of the gradients: about 1,024 workgroups.
int grad_splits(int T, int N, int K, int n) {
  const int64_t blocks = (int64_t)((N + 127) / 128 + (K + 127) / 128) * n;
  const int windows = (T + 255) / 256;  // a window per wavefront
  int64_t s = (1024 + blocks - 1) / blocks;
  if (s > windows) s = windows;
  return (int)(s > 16 ? 16 : s);
}

// Batches of up to this many rows take the streaming path.
constexpr int kStreamRows = 640;
// The streaming path's tiles: columns per workgroup grow with the rows, so
// that x is not read once per 16 columns.
int stream_mt(int T) { return T <= 16 ? 1 : (T <= 32 ? 2 : 4); }
int stream_splits(int T, int N, int K) {
  const int mt = stream_mt(T);
  const int blocks = N / (16 * mt) * ((T + 16 * mt - 1) / (16 * mt));
  int s = 384 / blocks;
  const int most = K / 64 / kStreamWaves;
  if (s > most) s = most;
  return s < 1 ? 1 : (s > 8 ? 8 : s);
}

int stream_shrink_splits(int T, int F) {
  // a run of 64-wide blocks per wavefront
  int s = 64 / ((T + 15) / 16);
  const int most = (F / 64 + kStreamWaves - 1) / kStreamWaves;
  if (s > most) s = most;
  return s < 1 ? 1 : (s > 8 ? 8 : s);
}

struct Carve {
  char *p;
  size_t used = 0;
  explicit Carve(void *ws) : p(static_cast<char *>(ws)) {}
  template <typename X>
  X *take(size_t n) {
    X *r = reinterpret_cast<X *>(p + used);
    used += align_up(n * sizeof(X));
    return r;
  }
};

struct Work {
  uint16_t *plane;
  float *sc;
  float *part_u, *part_v, *rows;
  uint16_t *at, *bt, *planes_u, *planes_v;
  int32_t *owner;
  float *pa, *pb;
  float *part;
  int su, sv, sg, sp, Tp, R32;
};
// Regions of the workspace; n = R = 0 without adapters.
size_t carve(const Layer &L, int matrix, int n, int R, int T, bool backward, void *ws, Work *w) {
  const size_t N = matrix == 2 ? L.H : L.I, K = matrix == 2 ? L.I : L.H;
  Carve c(ws);
  Work o = {};
  o.R32 = round32(R);
  o.Tp = (T + 63) / 64 * 64;
  o.su = shrink_splits(T, (int)K);
  o.sv = shrink_splits(T, (int)N);
  if (!backward && T <= kStreamRows) {
    o.sp = stream_splits(T, (int)N, (int)K);
    o.su = stream_shrink_splits(T, (int)K);
    o.part = c.take<float>((size_t)o.sp * T * N);
  } else {
    o.plane = c.take<uint16_t>(N * K);
    if (!backward) o.sc = c.take<float>(N * K / 64);
  }
  if (n) {
    o.part_u = c.take<float>((size_t)o.su * T * o.R32);
    if (backward) {
      o.part_v = c.take<float>((size_t)o.sv * T * o.R32);
      o.rows = c.take<float>((size_t)T * o.R32);
      o.at = c.take<uint16_t>((size_t)n * R * K);
      o.bt = c.take<uint16_t>((size_t)n * R * N);
      o.planes_u = c.take<uint16_t>((size_t)3 * o.R32 * o.Tp);
      o.planes_v = c.take<uint16_t>((size_t)3 * o.R32 * o.Tp);
      o.owner = c.take<int32_t>(o.Tp);
      o.sg = grad_splits(T, (int)N, (int)K, n);
      if (o.sg > 1) {
        o.pa = c.take<float>((size_t)o.sg * n * R * K);
        o.pb = c.take<float>((size_t)o.sg * n * R * N);
      }
    }
  }
  if (w) *w = o;
  return c.used;
}

// Workgroups (per tile) that the requests of a tile are spread over.
int spread(int rows, int n_req) { return n_req < rows ? n_req : rows; }

int launch_shrink(const ShrinkArgs &a, const ShrinkArgs &b, hipStream_t s) {
  const dim3 grid((a.T + 63) / 64, a.nsub, a.splits + b.splits);
  if (a.R32 <= 32) launch_k(COLI_K_PROJECT_SHRINK, shrink_kernel<2>, grid, dim3(256), 0, s, a, b);
  else if (a.R32 <= 64) launch_k(COLI_K_PROJECT_SHRINK, shrink_kernel<4>, grid, dim3(256), 0, s, a, b);
  else launch_k(COLI_K_PROJECT_SHRINK, shrink_kernel<8>, grid, dim3(256), 0, s, a, b);
  return hip_status(hipGetLastError());
}

template <bool SCALED, bool F32>
int launch_gemm(const GemmArgs &g, hipStream_t s) {
  const dim3 grid((g.N + 127) / 128, (g.T + 127) / 128);
  launch_k(COLI_K_PROJECT_GEMM, gemm_kernel<128, 128, 64, SCALED, F32>, grid, dim3(256), 0, s, g);
  return hip_status(hipGetLastError());
}

template <int F, int RT>
int launch_stream(const StreamArgs &g, hipStream_t s) {
  const int mt = stream_mt(g.T);
  const unsigned grid = g.shrink_blocks +
                        g.m.N / (16 * mt) * ((g.T + 16 * mt - 1) / (16 * mt)) * g.splits;
  const dim3 b(64 * kStreamWaves);
  if (mt == 1) launch_k(COLI_K_PROJECT_STREAM, stream_kernel<F, 1, 1, 4, RT>, dim3(grid), b, 0, s, g);
  else if (mt == 2) launch_k(COLI_K_PROJECT_STREAM, stream_kernel<F, 2, 2, 2, RT>, dim3(grid), b, 0, s, g);
  else launch_k(COLI_K_PROJECT_STREAM, stream_kernel<F, 4, 4, 1, RT>, dim3(grid), b, 0, s, g);
  return hip_status(hipGetLastError());
}
template <int F>
int launch_stream_rank(const StreamArgs &g, int R32, hipStream_t s) {
  if (R32 <= 32) return launch_stream<F, 2>(g, s);
  if (R32 <= 64) return launch_stream<F, 4>(g, s);
  return launch_stream<F, 8>(g, s);
}

Requests requests_of(const coli_moe_adapters_t *ad, const coli_moe_requests_t *rq) {
  Requests q = {};
  q.off = rq->offsets;
  q.adapter = rq->adapter;
  q.n = rq->n_requests;
  q.n_adapters = ad->n_adapters;
  return q;
}

}  // namespace

size_t project_workspace(const Layer &L, int matrix, int n, int R, int T, int backward) {
  return carve(L, matrix, n, R, T, backward != 0, nullptr, nullptr);
}

int launch_project(const Layer &L, int expert, int matrix, const coli_moe_adapters_t *ad,
                   const coli_moe_requests_t *rq, const uint16_t *x, int T, void *y, int y_dtype,
                   void *ws, hipStream_t s) {
  const Matrix m = matrix_of(L, expert, matrix);
  Work w;
  carve(L, matrix, ad ? ad->n_adapters : 0, ad ? ad->max_rank : 0, T, false, ws, &w);
  const int fmt = format_of(L);
  const bool f32 = y_dtype == COLI_OUT_F32;
  ExpandArgs e = {};
  e.T = T;
  e.N = m.N;
  ShrinkArgs sh = {};
  if (ad) {
    e.q = requests_of(ad, rq);
    e.u = w.part_u;
    e.b = ad->b;
    e.rank = ad->rank;
    e.R = ad->max_rank;
    e.R32 = w.R32;
    e.splits = w.su;
    sh = {x, ad->a, ad->rank, ad->scale, e.q, w.part_u, T, m.K, e.R, e.R32, w.su, 1};
  }
  int rc;
  if (T <= kStreamRows) {
    StreamArgs g = {};
    g.m = m;
    g.x = x;
    g.part = w.part;
    g.T = T;
    g.splits = w.sp;
    g.per = (m.K / 64 + kStreamWaves * w.sp - 1) / (kStreamWaves * w.sp);
    g.shrink_tiles = (T + 15) / 16;
    g.s = sh;
    CombineArgs c = {};
    c.part = w.part;
    c.splits = w.sp;
    c.nsub = 1;
    c.y = y;
    c.e = e;
    if (ad) {
      c.nsub = g.s.nsub = spread(16, e.q.n);
      g.shrink_blocks = g.shrink_tiles * g.s.nsub * w.su;
    }
    rc = fmt == kI4 ? launch_stream_rank<kI4>(g, w.R32, s)
                    : (fmt == kI8 ? launch_stream_rank<kI8>(g, w.R32, s)
                                  : launch_stream_rank<kF4>(g, w.R32, s));
    if (rc) return rc;
    const dim3 grid((m.N + 255) / 256, (T + 15) / 16, c.nsub);
    if (f32) launch_k(COLI_K_PROJECT_COMBINE, combine_parts_kernel<true>, grid, dim3(256), 0, s, c);
    else launch_k(COLI_K_PROJECT_COMBINE, combine_parts_kernel<false>, grid, dim3(256), 0, s, c);
    return hip_status(hipGetLastError());
  }
  const unsigned pb = (unsigned)(((int64_t)m.N * m.K / 8 + 255) / 256);
  if (fmt == kI4) launch_k(COLI_K_PROJECT_PREP, prep_kernel<kI4>, dim3(pb), dim3(256), 0, s, m, w.plane, w.sc);
  else if (fmt == kI8) launch_k(COLI_K_PROJECT_PREP, prep_kernel<kI8>, dim3(pb), dim3(256), 0, s, m, w.plane, w.sc);
  else launch_k(COLI_K_PROJECT_PREP, prep_kernel<kF4>, dim3(pb), dim3(256), 0, s, m, w.plane, w.sc);
  if ((rc = hip_status(hipGetLastError()))) return rc;
  if (ad && (rc = launch_shrink(sh, ShrinkArgs{}, s))) return rc;
  const GemmArgs g = {x, w.plane, w.sc, T, m.N, m.K, y, e};
  if (fmt == kF4) return f32 ? launch_gemm<false, true>(g, s) : launch_gemm<false, false>(g, s);
  return f32 ? launch_gemm<true, true>(g, s) : launch_gemm<true, false>(g, s);
}

int launch_project_backward(const Layer &L, int expert, int matrix, const coli_moe_adapters_t *ad,
                            const coli_moe_requests_t *rq, const uint16_t *x, const uint16_t *dy,
                            int T, uint16_t *dx, float *d_a, float *d_b, void *ws, hipStream_t s) {
  const Matrix m = matrix_of(L, expert, matrix);
  const int n = ad ? ad->n_adapters : 0, R = ad ? ad->max_rank : 0;
  Work w;
  carve(L, matrix, n, R, T, true, ws, &w);
  int rc;
  PrepT p = {};
  p.m = m;
  p.wt = w.plane;
  p.w_tiles = dx ? (m.N / 64) * (m.K / 64) : 0;
  if (ad) {
    p.ad = {ad->a, ad->b, ad->rank, ad->scale, R};
    p.q = requests_of(ad, rq);
    p.at = w.at;
    p.bt = w.bt;
    p.a_tiles = (R + 63) / 64 * (m.K / 64);
    p.b_tiles = (R + 63) / 64 * (m.N / 64);
  }
  const dim3 pg((unsigned)(p.w_tiles + (int64_t)n * (p.a_tiles + p.b_tiles)));
  const int fmt = format_of(L);
  if (fmt == kI4) launch_k(COLI_K_PROJECT_PREP, prep_transposed_kernel<kI4>, pg, dim3(256), 0, s, p);
  else if (fmt == kI8) launch_k(COLI_K_PROJECT_PREP, prep_transposed_kernel<kI8>, pg, dim3(256), 0, s, p);
  else launch_k(COLI_K_PROJECT_PREP, prep_transposed_kernel<kF4>, pg, dim3(256), 0, s, p);
  if ((rc = hip_status(hipGetLastError()))) return rc;
  if (ad) {
    const Requests q = p.q;
    const int nsub = T <= 1024 ? spread(16, q.n) : 1;
    const ShrinkArgs u = {x, ad->a, ad->rank, ad->scale, q, w.part_u, T, m.K, R, w.R32, w.su, nsub};
    const ShrinkArgs v = {dy, w.bt, ad->rank, ad->scale, q, w.part_v, T, m.N, R, w.R32, w.sv, nsub};
    if ((rc = launch_shrink(u, v, s))) return rc;
    FinishArgs f = {};
    f.q = q;
    f.part[0] = w.part_u;
    f.part[1] = w.part_v;
    f.splits[0] = w.su;
    f.splits[1] = w.sv;
    f.rows = w.rows;
    f.planes[0] = w.planes_u;
    f.planes[1] = w.planes_v;
    f.owner = w.owner;
    f.T = T;
    f.Tp = w.Tp;
    f.R32 = w.R32;
    launch_k(COLI_K_PROJECT_FINISH, finish_kernel, dim3(w.Tp / 64, w.R32 / 32, 2), dim3(256), 0, s, f);
    if ((rc = hip_status(hipGetLastError()))) return rc;
  }
  if (d_a) {
    GradsArgs a = {};
    a.g[0] = {dy, w.planes_u, w.sg > 1 ? w.pb : d_b, m.N, 1, (m.N + 127) / 128};
    a.g[1] = {x, w.planes_v, w.sg > 1 ? w.pa : d_a, m.K, 0, (m.K + 127) / 128};
    a.owner = w.owner;
    a.T = T;
    a.Tp = w.Tp;
    a.R = R;
    a.R32 = w.R32;
    a.n = n;
    a.splits = w.sg;
    a.rows = ((w.Tp / 64 + w.sg - 1) / w.sg) * 64;
    const int rt = w.R32 <= 32 ? 2 : 4;
    const dim3 grid(a.g[0].f_tiles + a.g[1].f_tiles, n, w.sg * ((w.R32 + 16 * rt - 1) / (16 * rt)));
    if (rt == 2) launch_k(COLI_K_PROJECT_GRADS, grads_kernel<2>, grid, dim3(256), 0, s, a);
    else launch_k(COLI_K_PROJECT_GRADS, grads_kernel<4>, grid, dim3(256), 0, s, a);
    if ((rc = hip_status(hipGetLastError()))) return rc;
    if (w.sg > 1) {
      ReduceArgs r = {};
      r.src[0] = reinterpret_cast<const float4 *>(w.pb);
      r.src[1] = reinterpret_cast<const float4 *>(w.pa);
      r.dst[0] = reinterpret_cast<float4 *>(d_b);
      r.dst[1] = reinterpret_cast<float4 *>(d_a);
      r.n[0] = (int64_t)n * R * m.N / 4;
      r.n[1] = (int64_t)n * R * m.K / 4;
      r.splits = w.sg;
      launch_k(COLI_K_PROJECT_REDUCE, reduce_kernel, dim3((unsigned)((r.n[0] + r.n[1] + 255) / 256)),
               dim3(256), 0, s, r);
      if ((rc = hip_status(hipGetLastError()))) return rc;
    }
  }
  if (!dx) return COLI_OK;
  ExpandArgs e = {};
  if (ad) e = {p.q, w.rows, w.at, ad->rank, T, m.K, R, w.R32, 1};
  return launch_gemm<false, false>({dy, w.plane, nullptr, T, m.K, m.N, dx, e}, s);
}

}  // namespace coli
