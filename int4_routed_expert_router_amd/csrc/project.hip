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
// the type that dx itself is rounded to (MXFP4 weights are exact; a second part
// of w would double the long batches' product, and dx uses the same W for
// every T).  u and v stay fp32 and enter the
// matrix cores as sums of two bf16 parts (16 bits of mantissa, for bf16
// results) or three (24 bits, for fp32 ones).
//
// Three paths by the batch (path_of):
//  short    stream: codes from memory into registers, W x in parts along K, u
//           in the same launch; a second launch joins parts and adapters.
//  between  direct: the same with x staged in LDS.
//  long     prep (codes -> a bf16 plane), shrink (u), gemm (LDS-tiled, the
//           adapters added in registers at its end).
// The backward pass has W, A and B transposed first (prep), takes the same
// three paths for dx with v for u, and adds
//  finish   sums the parts of u and v and lays them out for
//  grads    dA and dB, contractions over the rows of one adapter, split into
//           row ranges that reduce adds up.
#include "copy_ring.h"
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

constexpr int kMaxSplits = 4;  // parts of a sum along K

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
enum { kI4 = 0, kI8 = 1, kF4 = 2, kBF = 3 };  // kBF: a bf16 plane instead of codes
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
// Bound by its writes: 12.6 M weights, 25 MB out, 9 us, 4 % of the product it is
// for (kernel times here are between two events on the stream).
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

// The backward pass's operands: the weights rounded to bf16 (see the top) [K][N], and A and B of
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
constexpr int kMaxLook = 1024;  // requests that each workgroup looks through
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
    // adapters that no request names are left out where looking is cheap
    if (g.q.n <= kMaxLook) {
      if (tid == 0) used = 0;
      __syncthreads();
      for (int i = tid; i < g.q.n; i += 256)
        if (g.q.adapter[i] == a && g.q.off[i + 1] > g.q.off[i]) used = 1;
      __syncthreads();
      if (!used) return;
    }
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

// One of two, field by field: a reference chosen at run time would have the
// compiler copy both to scratch memory and read every use from there.
COLI_DEV ShrinkArgs pick(const ShrinkArgs &a, const ShrinkArgs &b, bool second) {
  ShrinkArgs g = a;  // masks, sizes and the rest are the same for both
  g.z = second ? b.z : a.z;
  g.m = second ? b.m : a.m;
  g.part = second ? b.part : a.part;
  g.F = second ? b.F : a.F;
  g.splits = second ? b.splits : a.splits;
  return g;
}

// One workgroup per tile of 16 rows, split and residue of the tile's requests
// modulo nsub (so that a tile of many one-row requests spreads over many
// workgroups).  Its NW wavefronts take the split's 64-wide k blocks in turn;
// operands come straight from memory: lane (c, g) holds 16 values of row c at
// k = 16g, two matrix-core steps.  Short requests are bound by the adapters
// they read and by latency, which this spreads as far as it goes.
template <int RT, int NW>
COLI_DEV void shrink_tile(const ShrinkArgs &g, int tile, int sub, int split, f32x4 (*buf)[64]) {
  const int lane = threadIdx.x & 63, c = lane & 15, kg = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t0 = tile * 16, t1 = min(g.T, t0 + 16);
  const int nb = g.F / 64;
  for_requests(g.q, t0, t1, [&](int ordinal, int begin, int end, int a) {
    if (ordinal % g.nsub != sub) return;
    const int rank = rank_of(g.rank, a, g.R);
    f32x4 acc[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r] = f32x4{0, 0, 0, 0};
    const bool mine = t0 + c >= begin && t0 + c < end;
    const uint16_t *mrow = g.m + ((int64_t)a * g.R + c) * g.F + 16 * kg;
    const uint16_t *zrow = g.z + (int64_t)(t0 + c) * g.F + 16 * kg;
    for (int b = split * NW + wv; b < nb; b += NW * g.splits) {
      uint4 mf[RT][2], zf[2];
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          mf[r][h] = 16 * r + c < rank ? ld16(mrow + (int64_t)16 * r * g.F + 64 * b + 8 * h) : zero4();
#pragma unroll
      for (int h = 0; h < 2; ++h) zf[h] = mine ? ld16(zrow + 64 * b + 8 * h) : zero4();
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[r] = mfma(zf[h], mf[r][h], acc[r]);
    }
    wave_sums<RT, NW>(acc, buf, wv, lane);
    if (wv == 0) {
      const float s = g.scale ? g.scale[a] : 1.0f;
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = t0 + 4 * kg + j;
          if (t >= begin && t < end && 16 * r + c < g.R32)
            g.part[((int64_t)split * g.T + t) * g.R32 + 16 * r + c] =
                16 * r + c < rank ? s * acc[r][j] : 0.0f;  // also for rows that are not finite
        }
    }
  });
}

// Long requests: z and the adapter staged in LDS, 128 k at a time, two stages
// in turn, for 64 rows; each of the four wavefronts takes 16 of them against
// all ranks.  (Operand loads straight from memory touch 16 rows per
// instruction, which the memory pipeline takes in four lanes at a time: they
// held this pass at 2 TB/s.)  Bound by its reads of z: 8192 x 6144 (100 MB), rank
// 64, 24 us, 4.2 TB/s.  16-byte chunk q of a row is kept at q ^ 2 (row &
// 7), so that the chunks that LDS serves together fall on distinct banks.
// Rows of z outside the request are only copied in groups of four.
template <int RT>
__global__ void __launch_bounds__(256) shrink_kernel(ShrinkArgs g0, ShrinkArgs g1) {
  constexpr int kRowsA = 64, kChunks = 16, kRows = kRowsA + 16 * RT;
  constexpr int LD = kRows / 16;  // DMA instructions (four rows) of a wavefront per stage
  __shared__ uint4 stage0[kRows * kChunks], stage1[kRows * kChunks];
  const bool second = (int)blockIdx.z >= g0.splits;  // the first operand's splits, then the second's
  const ShrinkArgs g = pick(g0, g1, second);
  const int split = second ? blockIdx.z - g0.splits : blockIdx.z;
  const int lane = threadIdx.x & 63, c = lane & 15, kg = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t0 = blockIdx.x * 64, t1 = min(g.T, t0 + 64);
  const int nb = g.F / 64, per = (nb + g.splits - 1) / g.splits;
  const int b0 = split * per, b1 = min(nb, b0 + per), nst = (b1 - b0 + 1) / 2;
  for_requests(g.q, t0, t1, [&](int ordinal, int begin, int end, int a) {
    if (ordinal % g.nsub != (int)blockIdx.y) return;
    const int rank = rank_of(g.rank, a, g.R);
    const uint16_t *src[LD];
#pragma unroll
    for (int i = 0; i < LD; ++i) {
      const int row = (wv * LD + i) * 4 + (lane >> 4), q = (lane & 15) ^ (2 * (row & 7));
      const uint16_t *p = (wv * LD + i) * 4 < kRowsA
                              ? g.z + (int64_t)min(t0 + row, g.T - 1) * g.F
                              : g.m + ((int64_t)a * g.R + min(row - kRowsA, g.R - 1)) * g.F;
      src[i] = p + 64 * b0 + 8 * q;
    }
    auto issue = [&](uint4 *to, int st) {
      // an odd last stage copies its one block twice; the copy is not used
      const bool half = b0 + 2 * st + 1 >= b1;
#pragma unroll
      for (int i = 0; i < LD; ++i) {
        const int r0 = (wv * LD + i) * 4, row = r0 + (lane >> 4);
        if (r0 < kRowsA && (t0 + r0 + 4 <= begin || t0 + r0 >= end)) continue;
        const int back = half && (((lane & 15) ^ (2 * (row & 7))) >> 3) ? 64 : 0;
        dma16(src[i] + 128 * st - back, to + r0 * kChunks);
      }
    };
    f32x4 acc[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r] = f32x4{0, 0, 0, 0};
    // rows of other requests and ranks past the adapter's multiply whatever is
    // there: a sum depends on its own row and rank alone, and theirs are not used
    auto compute = [&](const uint4 *A, int st) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (s == 2 && b0 + 2 * st + 1 >= b1) break;
        const int q = (kg + 4 * s) ^ (2 * (c & 7));
        const uint4 zf = A[(16 * wv + c) * kChunks + q];
#pragma unroll
        for (int r = 0; r < RT; ++r)
          acc[r] = mfma(zf, A[(kRowsA + 16 * r + c) * kChunks + q], acc[r]);
      }
    };
    __syncthreads();  // the buffers may still be read for the request before
    if (nst > 0) issue(stage0, 0);
    for (int st = 0; st < nst; st += 2) {
      wait_dma();
      __syncthreads();
      if (st + 1 < nst) issue(stage1, st + 1);
      compute(stage0, st);
      if (st + 1 >= nst) break;
      wait_dma();
      __syncthreads();
      if (st + 2 < nst) issue(stage0, st + 2);
      compute(stage1, st + 1);
    }
    const float s = g.scale ? g.scale[a] : 1.0f;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = t0 + 16 * wv + 4 * kg + j, rr = 16 * r + c;
        if (t >= begin && t < end && rr < g.R32)
          g.part[((int64_t)split * g.T + t) * g.R32 + rr] = rr < rank ? s * acc[r][j] : 0.0f;
      }
  });
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

// Sums of up to four parts, in order, at M places.  All loads of all places
// are requested before any is used, and no more parts than there are.
static_assert(kMaxSplits == 4, "sum_parts");
COLI_DEV void add4(float4 &v, const float4 &o) {
  v.x += o.x;
  v.y += o.y;
  v.z += o.z;
  v.w += o.w;
}
template <int M>
COLI_DEV void sum_parts(const float *const (&p)[M], int64_t stride, int splits, float4 (&v)[M]) {
  auto load = [&](int s, float4 (&o)[M]) {
#pragma unroll
    for (int m = 0; m < M; ++m) o[m] = *reinterpret_cast<const float4 *>(p[m] + s * stride);
  };
  load(0, v);
  if (splits == 1) return;
  float4 a[M], b[M], c[M];
  load(1, a);
  if (splits > 2) {
    load(2, b);
    load(splits > 3 ? 3 : 2, c);
  }
#pragma unroll
  for (int m = 0; m < M; ++m) {
    add4(v[m], a[m]);
    if (splits > 2) add4(v[m], b[m]);
    if (splits > 3) add4(v[m], c[m]);
  }
}

// This lane's operand values u[t][k .. k+8), the splits added up, as P parts;
// zeros where not live.  Every lane loads (row t is in the batch, k in the
// padded width): a branch around the loads would have each wait for the last.
template <int P>
COLI_DEV void load_u(const ExpandArgs &g, int t, int k, bool live, uint4 (&uf)[P]) {
  const float *p = g.u + (int64_t)min(t, g.T - 1) * g.R32 + k;
  const int64_t stride = (int64_t)g.T * g.R32;
  const float *const at[2] = {p, p + 4};
  float4 q[2];
  sum_parts<2>(at, stride, g.splits, q);
  float v[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w};
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = live ? v[e] : 0.0f;
  split8<P>(v, uf);
}
// Ranks [k, k + 8) of the adapter's columns n0 + NJ c + j, zeros past its rank.
template <int NJ>
COLI_DEV void load_b(const ExpandArgs &g, int a, int n0, int k, int rank, uint4 (&bf)[NJ]) {
  const int c = threadIdx.x & 15;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int n = min(n0 + NJ * c + j, g.N - 1);
    bf[j] = ld16(g.b + ((int64_t)a * g.N + n) * g.R + min(k, g.R - 8));
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) bf[j] = keep_first(bf[j], rank - k);
}

// acc += the adapters' part of the wavefront's MI x NJ tiles: rows t0 + 16i +
// c, columns n0 + NJ c + j.  Every request with rows here multiplies only the
// 16-row tiles that it reaches.  Other requests' rows in a tile are multiplied
// as zeros and keep their sums: a zero times an infinity or NaN of b would not
// be zero.
template <int MI, int NJ, int P>
COLI_DEV void expand(const ExpandArgs &g, int t0, int n0, f32x4 (&acc)[MI][NJ]) {
  const int lane = threadIdx.x & 63, c = lane & 15, kg = lane >> 4;
  const int t1 = min(g.T, t0 + 16 * MI);
  if (t0 >= t1) return;
  for_requests(g.q, t0, t1, [&](int, int begin, int end, int a) {
    const int rank = rank_of(g.rank, a, g.R);
    for (int k0 = 0; k0 < rank; k0 += 32) {
      const int k = k0 + 8 * kg;  // this lane's eight ranks
      uint4 bf[NJ];
      load_b<NJ>(g, a, n0, k, rank, bf);
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        if (begin >= t0 + 16 * i + 16 || end <= t0 + 16 * i) continue;
        const int t = t0 + 16 * i + c;
        uint4 uf[P];
        load_u<P>(g, t, k, t >= begin && t < end && k < rank, uf);
        f32x4 d[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) d[j] = acc[i][j];
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int j = 0; j < NJ; ++j) d[j] = mfma(uf[p], bf[j], d[j]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = t0 + 16 * i + 4 * kg + e;
          const bool own = row >= begin && row < end;
#pragma unroll
          for (int j = 0; j < NJ; ++j) acc[i][j][e] = own ? d[j][e] : acc[i][j][e];
        }
      }
    }
  });
}

// NJ neighbouring columns of one row.
template <int NJ, bool F32>
COLI_DEV void store_cols(void *y, int64_t at, const float (&v)[NJ]) {
  if (F32) {
    float *p = static_cast<float *>(y) + at;
    if (NJ == 4) *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[NJ > 1], v[NJ > 2 ? 2 : 0], v[NJ > 3 ? 3 : 0]);
    else if (NJ == 2) *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[NJ > 1]);
    else *p = v[0];
  } else {
    uint16_t *p = static_cast<uint16_t *>(y) + at;
    if (NJ == 4)
      *reinterpret_cast<uint2 *>(p) =
          make_uint2(pack_bf16(v[0], v[NJ > 1]), pack_bf16(v[NJ > 2 ? 2 : 0], v[NJ > 3 ? 3 : 0]));
    else if (NJ == 2) *reinterpret_cast<uint32_t *>(p) = pack_bf16(v[0], v[NJ > 1]);
    else *p = (uint16_t)pack_bf16(v[0], 0.0f);
  }
}
template <int MI, int NJ, bool F32>
COLI_DEV void store_tile(void *y, int T, int N, int t0, int n0, const f32x4 (&acc)[MI][NJ]) {
  const int c = threadIdx.x & 15, kg = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = t0 + 16 * i + 4 * kg + e;
      if (t >= T) continue;
      float v[NJ];
#pragma unroll
      for (int j = 0; j < NJ; ++j) v[j] = acc[i][j][e];
      store_cols<NJ, F32>(y, (int64_t)t * N + n0 + NJ * c, v);
    }
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
// DMA, two buffers in turn, and from there to registers one stage ahead:
// while a stage is multiplied, the next one's operands are read from LDS and
// the one after it is copied into the buffer that was emptied a stage ago.
//
// Lane (c, g) of a 16 x 16 x 32 step h holds k = 32h + 8g of row c: chunk g +
// 4h of the row's eight 16-byte chunks, kept at (g + 4h) ^ (row & 7).  LDS
// serves the chunks of lanes g and g + 1 of eight rows together, which then
// fall on distinct banks (with chunks 2g + h, two apart, they collide: the
// reads took 1.5 times as long).
//
// Bound by the matrix cores and, with scales, by the vector ALUs beside them
// (one fp32 FMA per output and 64-wide group): 8192 x 2048 x 6144 takes 164 to
// 168 us on a plane of weights (1240 TFLOP/s, matrix cores busy in 65 % of the
// cycles; the library's bf16 product of that size 153 us), 188 us on codes
// with scales, and 201 to 218 us with five requests' rank-64 adapters (51 % busy; 2.5
// times the vector instructions).  Steps on the way, on the plane: 201 us at
// first, conflict-free reads 183 us, the third buffer 181 us, copies spread
// between the matrix-core steps 164 us.  A 256 x 256 tile has no registers
// left for the operands of the next stage.  w's rows are kept in the order n =
// 4c + j, so that lane c ends up with four neighbouring columns, stored
// together.
template <int BM, int BN, int WM, bool SCALED, bool F32>
__global__ void __launch_bounds__(BM / WM * BN) gemm_kernel(GemmArgs g) {
  constexpr int NW = (BM / WM) * (BN / 64), MI = WM / 16;
  constexpr int LD = (BM + BN) / 8 / NW;  // DMA instructions of a wavefront per stage
  // operations of a wavefront that may be in flight: before the first stages are
  // read the third one's copies, in a step those and the scale load before them
  constexpr int kFirst = LD, VM = LD + (SCALED ? 1 : 0);
  static_assert(ring_waits_hold(LD, SCALED, kFirst, VM) && VM < 16, "waits of the ring");
  // three objects, so that the compiler sees that one is read while others fill
  __shared__ uint4 stage0[(BM + BN) * 8], stage1[(BM + BN) * 8], stage2[(BM + BN) * 8];
  const int lane = threadIdx.x & 63, c = lane & 15, kg = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Workgroups go to the 8 XCDs in turn; each XCD gets a run of neighbouring
  // tiles (all columns of a few row tiles), so that its L2 holds those rows
  // of x once instead of every row.
  const int cols_t = (g.N + BN - 1) / BN;
  const int tile = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
  const int tm = tile / cols_t * BM, tn = tile % cols_t * BN;
  if (tm >= g.T) return;
  const int wm = (wv / (BN / 64)) * WM, wn = (wv % (BN / 64)) * 64;

  uint32_t src[LD];  // byte offsets: a matrix has at most 2^31 bytes
#pragma unroll
  for (int i = 0; i < LD; ++i) {
    const int row = (wv * LD + i) * 8 + (lane >> 3), pos = lane & 7;
    if ((wv * LD + i) * 8 < BM) {
      src[i] = (uint32_t)min(tm + row, g.T - 1) * (uint32_t)g.K * 2u + 16u * (pos ^ (row & 7));
    } else {
      const int r = row - BM, n = (r & ~63) + 4 * (r & 15) + ((r >> 4) & 3);
      src[i] = (uint32_t)min(tn + n, g.N - 1) * (uint32_t)g.K * 2u + 16u * (pos ^ (r & 7));
    }
  }
  const int n0 = tn + wn;
  const float *scp = g.sc + min(n0, g.N - 64) + 4 * c;  // N is a multiple of 64
  const int nst = g.K / 64;
  // past the last stage the copies repeat it, so that every stage leaves the
  // same number of operations in flight
  auto issue_one = [&](uint4 *to, int st, int i) {
    const char *base = reinterpret_cast<const char *>((wv * LD + i) * 8 < BM ? g.x : g.w);
    dma16(base + 128 * min(st, nst - 1) + src[i], to + (wv * LD + i) * 64);
  };
  auto issue = [&](uint4 *to, int st) {
#pragma unroll
    for (int i = 0; i < LD; ++i) issue_one(to, st, i);
  };
  f32x4 acc[MI][4];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  // with scales: a row tile's partial products join the sums (plain floats,
  // which the compiler keeps in place) while the matrix cores work on the
  // next row tile's
  float sums[MI][4][4];
  f32x4 dprev[4];
  float4 sprev = make_float4(0, 0, 0, 0), s0 = sprev, s1 = sprev, s2 = sprev;
#pragma unroll
  for (int j = 0; j < 4; ++j) dprev[j] = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < MI * 16; ++i) (&sums[0][0][0])[i] = 0.0f;
  auto add_scaled = [&](float (&to)[4][4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float s = j == 0 ? sprev.x : (j == 1 ? sprev.y : (j == 2 ? sprev.z : sprev.w));
#pragma unroll
      for (int e = 0; e < 4; ++e) to[j][e] = fmaf(dprev[j][e], s, to[j][e]);
    }
  };
  // with scales there are registers for one set of w's operands: the last row
  // tile reads each one's successor as soon as it has used it
  uint4 af[MI][2], bf[SCALED ? 1 : 2][4][2];
  auto read_a = [&](const uint4 *A, int i) {
#pragma unroll
    for (int h = 0; h < 2; ++h) af[i][h] = A[(wm + 16 * i + c) * 8 + ((kg + 4 * h) ^ (c & 7))];
  };
  auto read_b = [&](const uint4 *A, int j, uint4 (&to)[4][2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) to[j][h] = A[(BM + wn + 16 * j + c) * 8 + ((kg + 4 * h) ^ (c & 7))];
  };
  // Stage st: its operands are in af and b; `next` holds the next stage, the
  // one after that is on its way, and `to` (this stage's buffer, emptied)
  // takes the third.
  // Its scales are in s4; those of stage st + 2 are loaded into s6.
  auto compute = [&](uint4 (&b)[4][2], uint4 (&bnext)[4][2], const uint4 *next, uint4 *to,
                     const float4 &s4, float4 &s6, int st) {
    // the next stage is there, this one's reads are done
    __builtin_amdgcn_s_waitcnt(0x0070 | (VM & 15));
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (SCALED) s6 = *reinterpret_cast<const float4 *>(scp + (int64_t)min(st + 2, nst - 1) * g.N);
    __builtin_amdgcn_sched_barrier(0);
    // the copies are spread over the stage: issued in one go, they would hold
    // up every wavefront's start while the memory pipeline takes them in
#pragma unroll
    for (int i = 0; i < MI; ++i) {
#pragma unroll
      for (int q = i * LD / MI; q < (i + 1) * LD / MI; ++q) issue_one(to, st + 3, q);
      if (SCALED) {
        f32x4 d[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          d[j] = mfma(af[i][0], b[j][0], f32x4{0, 0, 0, 0});
          d[j] = mfma(af[i][1], b[j][1], d[j]);
          if (i == MI - 1) read_b(next, j, b);
        }
        add_scaled(sums[(i + MI - 1) % MI]);
        if (i == 0) sprev = s4;
#pragma unroll
        for (int j = 0; j < 4; ++j) dprev[j] = d[j];
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = mfma(af[i][h], b[j][h], acc[i][j]);
      }
      // past the last stage this reads what is there, unused
      read_a(next, i);
      if (!SCALED) {
#pragma unroll
        for (int j = 4 * i / MI; j < 4 * (i + 1) / MI; ++j) read_b(next, j, bnext);
      }
      if (SCALED) {
        __builtin_amdgcn_sched_barrier(0);
        continue;
      }
      constexpr int R = 2 + 8 / MI;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        if (q * R / 8 != (q + 1) * R / 8) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        if (q == 2 || q == 6) __builtin_amdgcn_sched_group_barrier(0x10, 1, 0);
      }
    }
  };
  issue(stage0, 0);
  if (SCALED) {
    s0 = *reinterpret_cast<const float4 *>(scp);
    s1 = *reinterpret_cast<const float4 *>(scp + (int64_t)min(1, nst - 1) * g.N);
  }
  issue(stage1, 1);
  issue(stage2, 2);
  // stages 0 and 1: no scale load follows stage 1's copies, so the first step's
  // wait alone would let its last copy be in flight
  __builtin_amdgcn_s_waitcnt(0x0F70 | kFirst);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < MI; ++i) read_a(stage0, i);
#pragma unroll
  for (int j = 0; j < 4; ++j) read_b(stage0, j, bf[0]);
  constexpr int B1 = SCALED ? 0 : 1;
  int st = 0;
  for (; st + 6 <= nst; st += 6) {
    compute(bf[0], bf[B1], stage1, stage0, s0, s2, st);
    compute(bf[B1], bf[0], stage2, stage1, s1, s0, st + 1);
    compute(bf[0], bf[B1], stage0, stage2, s2, s1, st + 2);
    compute(bf[B1], bf[0], stage1, stage0, s0, s2, st + 3);
    compute(bf[0], bf[B1], stage2, stage1, s1, s0, st + 4);
    compute(bf[B1], bf[0], stage0, stage2, s2, s1, st + 5);
  }
  if (st < nst) compute(bf[0], bf[B1], stage1, stage0, s0, s2, st);
  if (st + 1 < nst) compute(bf[B1], bf[0], stage2, stage1, s1, s0, st + 1);
  if (st + 2 < nst) compute(bf[0], bf[B1], stage0, stage2, s2, s1, st + 2);
  if (st + 3 < nst) compute(bf[B1], bf[0], stage1, stage0, s0, s2, st + 3);
  if (st + 4 < nst) compute(bf[0], bf[B1], stage2, stage1, s1, s0, st + 4);
  wait_dma();  // nothing may land in LDS after the workgroup has ended
  if (SCALED) {
    add_scaled(sums[MI - 1]);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = sums[i][j][e];
  }
  if (n0 >= g.N) return;
  if (g.e.u) expand<MI, 4, F32 ? 3 : 2>(g.e, tm + wm, n0, acc);
  store_tile<MI, 4, F32>(g.y, g.T, g.N, tm + wm, n0, acc);
}

// ----------------------------------------------------------------- stream
//
// Short batches: the codes go from memory straight into registers, so that a
// call costs one pass over the container and two launches.  The first
// computes W x in parts (split along K) and u side by side; the second adds
// the parts and the adapters.  Bound by latency: two launches, each a chain of
// two or three dependent loads (1 token, 6144 x 2048 int4, rank 16: 11.7 us in
// all, against 1.3 us for its bytes; unpacking first and multiplying then took
// 151 us).

struct StreamArgs {
  Matrix m;
  const uint16_t *x;  // [T][K]
  float *part;        // [splits][T][N]
  int T, splits, per;  // per: 64-wide groups of a wavefront
  int shrink_blocks, shrink_tiles;
  ShrinkArgs s[2];  // u, and in the backward pass v
};

constexpr int kStreamWaves = 8;

// Raw operands of one 64-wide group of a row: 16 codes per lane (k = 16g of
// the group, g = lane / 16), in two steps of eight.
template <int F>
struct Raw {
  uint32_t w[F == kBF ? 8 : (F == kI8 ? 4 : 2)];
  uint32_t s;
};
template <int F>
COLI_DEV Raw<F> load_raw(const Matrix &m, int n, int b, int kg) {
  Raw<F> r;
  if (F == kBF) {
    const uint16_t *p = reinterpret_cast<const uint16_t *>(m.q) + (int64_t)n * m.K + 64 * b + 16 * kg;
    const uint4 v[2] = {ld16(p), ld16(p + 8)};
    __builtin_memcpy(r.w, v, sizeof(r.w));
    r.s = 0;
    return r;
  }
  if (F == kI8) {
    const uint4 v = ld16(m.q + (int64_t)n * m.K + 64 * b + 16 * kg);
    __builtin_memcpy(r.w, &v, F == kI8 ? 16 : 8);
  } else {
    const uint2 v = *reinterpret_cast<const uint2 *>(m.q + ((int64_t)n * m.K + 64 * b + 16 * kg) / 2);
    r.w[0] = v.x;
    r.w[1] = v.y;
  }
  if (F == kF4) r.s = m.sc[(int64_t)n * (m.K / 32) + 2 * b + (kg >> 1)];
  else r.s = reinterpret_cast<const uint16_t *>(m.sc)[(int64_t)n * (m.K / 64) + b];
  return r;
}
// Step h as a matrix-core operand, exact in bf16.  int4: 16 q, a nibble in the
// upper half of a signed byte (a biased form such as 24 + q takes half the
// instructions, but its bias times sum(x) has to leave the fp32 sums again:
// where large x meet small codes, little else than rounding stays).  int8: q.
// MXFP4: the weights themselves.
template <int F>
COLI_DEV uint4 unpack(const Raw<F> &r, int h) {
  if (F == kBF) {
    uint4 v;
    __builtin_memcpy(&v, &r.w[F == kBF ? 4 * h : 0], F == kBF ? 16 : 8);
    return v;
  }
  if (F == kI4) {
    const uint32_t w = r.w[h], even = (w << 4) & 0xf0f0f0f0u, odd = w & 0xf0f0f0f0u;
    uint32_t d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      d[i] = pack_bf16((float)(int8_t)(even >> (8 * i)), (float)(int8_t)(odd >> (8 * i)));
    return make_uint4(d[0], d[1], d[2], d[3]);
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

// What a group's sum of products with unpack's operands is multiplied by.
template <int F>
COLI_DEV float group_scale(const Raw<F> &r) {
  const float s = f16_to_f32((uint16_t)r.s);
  return F == kI4 ? s * 0.0625f : s;
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
  constexpr bool exact = F == kF4 || F == kBF;  // operands are whole weights
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
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const uint4 w0 = unpack<F>(raw[i][j], 0), w1 = unpack<F>(raw[i][j], 1);
        const float s = exact ? 1.0f : group_scale(raw[i][j]);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          f32x4 d = exact ? acc[m][j] : f32x4{0, 0, 0, 0};
          d = mfma(xr[i][m][0], w0, d);
          d = mfma(xr[i][m][1], w1, d);
          if (exact) {
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
      if (NJ == 2) {
        *reinterpret_cast<float2 *>(p) = make_float2(acc[m][0][e], acc[m][NJ > 1][e]);
      } else if (NJ == 4) {
        *reinterpret_cast<float4 *>(p) =
            make_float4(acc[m][0][e], acc[m][NJ > 1][e], acc[m][NJ > 2 ? 2 : 0][e], acc[m][NJ > 3 ? 3 : 0][e]);
      } else {
#pragma unroll
        for (int j = 0; j < NJ; ++j) p[j] = acc[m][j][e];
      }
    }
}

// Workgroup b of the u (and v) side.
template <int RT, int NW>
COLI_DEV void shrink_block(const StreamArgs &g, int b, f32x4 (*buf)[64]) {
  const int tile = b % g.shrink_tiles;
  b /= g.shrink_tiles;
  const int sub = b % g.s[0].nsub, split = b / g.s[0].nsub;
  if (split < g.s[0].splits) shrink_tile<RT, NW>(g.s[0], tile, sub, split, buf);
  else shrink_tile<RT, NW>(g.s[1], tile, sub, split - g.s[0].splits, buf);
}

template <int F, int MT, int NJ, int GB, int RT>
__global__ void __launch_bounds__(64 * kStreamWaves) stream_kernel(StreamArgs g) {
  constexpr int A = MT * NJ > RT ? MT * NJ : RT;
  __shared__ f32x4 buf[kStreamWaves / 2 * A][64];
  int b = blockIdx.x;
  if (b < g.shrink_blocks) {
    shrink_block<RT, kStreamWaves>(g, b, buf);
    return;
  }
  b -= g.shrink_blocks;
  const int nt = g.m.N / (16 * NJ), tt = (g.T + 16 * MT - 1) / (16 * MT);
  const int n = b % nt;
  b /= nt;
  stream_tile<F, MT, NJ, GB>(g, n, b % tt, b / tt, buf);
}

// ----------------------------------------------------------------- direct
//
// The codes again go from memory straight into registers, but x is staged in
// LDS (two 64-wide groups per stage, two stages in turn) and shared by the
// workgroup's four wavefronts, 64 rows x 32 columns each.  Otherwise as the
// streaming path: parts and u first, joined by the second launch.  Bound by
// the latency of a stage (0.8 us per 64 k with one stage in flight), which the
// splits along K spread: 517 rows, 2048 x 1024 int4, 37 requests 17 us, the second
// launch 9 us.
constexpr int kDirectM = 4, kDirectN = 2, kDirectWaves = 4, kDirectGroups = 2;
constexpr int kDirectRows = 16 * kDirectM, kDirectCols = 16 * kDirectN * kDirectWaves;

template <int F>
COLI_DEV void direct_tile(const StreamArgs &g, int nt, int tt, int split, uint4 *stage0,
                          uint4 *stage1) {
  constexpr int MT = kDirectM, NJ = kDirectN, NW = kDirectWaves, KS = kDirectGroups;
  constexpr int RB = 8 * KS;                      // 16-byte chunks of a staged row
  constexpr int LD = kDirectRows * RB / 64 / NW;  // DMA instructions of a wavefront per stage
  constexpr bool exact = F == kF4 || F == kBF;
  const int lane = threadIdx.x & 63, c = lane & 15, kg = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tm = tt * kDirectRows, n0 = nt * kDirectCols + wv * (16 * NJ);
  const int ns = min(n0, g.m.N - 16 * NJ);  // wavefronts past the last column read that one's
  const int g0 = split * g.per, g1 = min(g.m.K / 64, g0 + g.per);  // groups of this split
  const int nst = (g1 - g0 + KS - 1) / KS;
  // Chunk p of row r is kept at p ^ key(r): LDS serves eight rows' chunks of
  // lanes kg and kg + 1 together, which are two apart.
  auto key = [](int r) {
    return KS == 1 ? ((r >> 1) & 1) | ((r >> 2) & 1) << 2 : (r & 1) | ((r >> 1) & 3) << 2;
  };
  static_assert(KS <= 2, "keys for rows of 8 and 16 chunks");
  const uint16_t *src[LD];
#pragma unroll
  for (int i = 0; i < LD; ++i) {
    const int q = (wv * LD + i) * 64 + lane, row = q / RB, pos = q % RB;
    src[i] = g.x + (int64_t)min(tm + row, g.T - 1) * g.m.K + 64 * g0 + 8 * (pos ^ key(row));
  }
  const int nb = g1 - g0;
  Raw<F> raw[KS][NJ];
  auto issue = [&](uint4 *to, int st) {
#pragma unroll
    for (int i = 0; i < LD; ++i) {
      // the last stage may be short: its missing groups are not used
      const int q = (wv * LD + i) * 64 + lane, pos = (q % RB) ^ key(q / RB);
      const int over = KS > 1 ? max(0, 64 * (KS * st + pos / 8 - nb + 1)) : 0;
      dma16(src[i] + 64 * KS * st - over, to + (wv * LD + i) * 64);
    }
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        raw[s][j] = load_raw<F>(g.m, ns + NJ * c + j, g0 + min(KS * st + s, nb - 1), kg);
  };
  f32x4 acc[MT][NJ];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  auto compute = [&](const uint4 *A, uint4 *to, int st) {
    uint4 w[KS][NJ][2];
    float sc[KS][NJ];
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        w[s][j][0] = unpack<F>(raw[s][j], 0);
        w[s][j][1] = unpack<F>(raw[s][j], 1);
        sc[s][j] = exact ? 1.0f : group_scale(raw[s][j]);
      }
    if (st + 1 < nst) issue(to, st + 1);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      if (KS > 1 && KS * st + s >= nb) continue;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        uint4 af[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) af[h] = A[(16 * i + c) * RB + ((8 * s + 2 * kg + h) ^ key(c))];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          f32x4 d = exact ? acc[i][j] : f32x4{0, 0, 0, 0};
          d = mfma(af[0], w[s][j][0], d);
          d = mfma(af[1], w[s][j][1], d);
          if (exact) {
            acc[i][j] = d;
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(d[e], sc[s][j], acc[i][j][e]);
          }
        }
      }
    }
  };
  if (nb > 0) {
    issue(stage0, 0);
    for (int st = 0; st < nst; st += 2) {
      wait_dma();
      __syncthreads();
      compute(stage0, stage1, st);
      if (st + 1 == nst) break;
      wait_dma();
      __syncthreads();
      compute(stage1, stage0, st + 1);
    }
  }
  if (n0 >= g.m.N) return;
  store_tile<MT, NJ, true>(g.part + (int64_t)split * g.T * g.m.N, g.T, g.m.N, tm, n0, acc);
}

template <int F, int RT>
__global__ void __launch_bounds__(64 * kDirectWaves) direct_kernel(StreamArgs g) {
  __shared__ uint4 stage0[kDirectRows * 8 * kDirectGroups], stage1[kDirectRows * 8 * kDirectGroups];
  __shared__ f32x4 buf[kDirectWaves / 2 * RT][64];
  int b = blockIdx.x;
  if (b < g.shrink_blocks) {
    shrink_block<RT, kDirectWaves>(g, b, buf);
    return;
  }
  b -= g.shrink_blocks;
  const int nt = (g.m.N + kDirectCols - 1) / kDirectCols, tt = (g.T + kDirectRows - 1) / kDirectRows;
  const int n = b % nt;
  b /= nt;
  direct_tile<F>(g, n, b % tt, b / tt, stage0, stage1);
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
COLI_DEV void combine_tile(const CombineArgs &g, int nx, int ty, int sub) {
  const int lane = threadIdx.x & 63, c = lane & 15, kg = lane >> 4;
  const int n0 = (nx * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * 64;
  if (n0 >= g.e.N) return;
  const int t0 = ty * 16, t1 = min(g.e.T, t0 + 16);
  uint32_t covered = 0;
  auto rows = [&](int begin, int end, uint32_t mask, int a) {
    // the four rows of this lane, if any of them is wanted
    f32x4 acc[4] = {};
    if ((mask >> (4 * kg)) & 15u) {
      const float *at[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        at[e] = g.part + (int64_t)min(t0 + 4 * kg + e, g.e.T - 1) * g.e.N + n0 + 4 * c;
      float4 v[4];
      sum_parts<4>(at, (int64_t)g.e.T * g.e.N, g.splits, v);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[0][e] = v[e].x;
        acc[1][e] = v[e].y;
        acc[2][e] = v[e].z;
        acc[3][e] = v[e].w;
      }
    }
    if (a >= 0) {
      constexpr int P = F32 ? 3 : 2;
      const int rank = rank_of(g.e.rank, a, g.e.R);
      const int t = t0 + c;
      for (int k0 = 0; k0 < rank; k0 += 32) {
        const int k = k0 + 8 * kg;
        uint4 bf[4], uf[P];
        load_b<4>(g.e, a, n0, k, rank, bf);
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
      if ((mask >> r) & 1u) {
        const float v[4] = {acc[0][e], acc[1][e], acc[2][e], acc[3][e]};
        store_cols<4, F32>(g.y, (int64_t)(t0 + r) * g.e.N + n0 + 4 * c, v);
      }
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

template <bool F32>
__global__ void __launch_bounds__(256) combine_parts_kernel(CombineArgs g) {
  combine_tile<F32>(g, blockIdx.x, blockIdx.y, blockIdx.z);
}

// The same for short requests, decode's single rows above all: a wavefront takes
// 64 columns of one row, with plain fp32 products instead of matrix-core tiles
// of which one row would be used.  B's rows come in whole cache lines (P lanes
// to a row of at most P chunks of eight ranks, 64 / P rows per load), and
// everything that does not need the request is on its way before it is known.
// 64 users, 32 adapters of rank 64, 6144 x 2048: the second launch takes 7.9
// us, with the tiles 16.3 us.
template <bool F32>
__global__ void __launch_bounds__(256) combine_rows_kernel(CombineArgs g) {
  const int lane = threadIdx.x & 63;
  const int n0 = (blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * 64;
  const int t = blockIdx.y;
  const ExpandArgs &e = g.e;
  if (n0 >= e.N) return;
  const float *pp = g.part + (int64_t)t * e.N + n0 + lane;
  const int64_t stride = (int64_t)e.T * e.N;
  float part[kMaxSplits];
#pragma unroll
  for (int s = 0; s < kMaxSplits; ++s) part[s] = pp[min(s, g.splits - 1) * stride];
  const int chunks = e.R / 8;
  int lg = 0;  // P = 1 << lg
  while ((1 << lg) < chunks) ++lg;
  const int P = 1 << lg, sub = lane & (P - 1), per = 64 >> lg;
  const int k = 8 * min(sub, chunks - 1);
  const float *up = e.u + (int64_t)t * e.R32 + k;
  const float *const at[2] = {up, up + 4};
  float4 uq[2];
  sum_parts<2>(at, (int64_t)e.T * e.R32, e.splits, uq);
  // the request of this row
  int a = -1;
  if (e.q.n <= 64) {
    const int i = min(lane, e.q.n - 1);
    const int b = e.q.off[i], end = e.q.off[i + 1], who = e.q.adapter[i];
    const uint64_t hit = __ballot(lane < e.q.n && b <= t && t < end);
    if (hit) a = __builtin_amdgcn_readlane(who, __ffsll((long long)hit) - 1);
  } else {
    const int s = last_at_or_before(e.q.off, e.q.n + 1, t);
    if (s >= 0 && s < e.q.n) a = __builtin_amdgcn_readfirstlane(e.q.adapter[s]);
  }
  float y = part[0];
#pragma unroll
  for (int s = 1; s < kMaxSplits; ++s) y += s < g.splits ? part[s] : 0.0f;
  if (a >= 0 && a < e.q.n_adapters) {
    const uint16_t *bp = e.b + ((int64_t)a * e.N + n0 + (lane >> lg)) * e.R + k;
    const int rank = rank_of(e.rank, a, e.R);
    const int live = sub < chunks ? rank - k : 0;  // ranks of this lane's chunk in use
    float u[8] = {uq[0].x, uq[0].y, uq[0].z, uq[0].w, uq[1].x, uq[1].y, uq[1].z, uq[1].w};
    for (int i0 = 0; i0 < P; i0 += 4) {
      uint4 q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = ld16(bp + (int64_t)min(i0 + i, P - 1) * per * e.R);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        q[i] = keep_first(q[i], live);
        const uint32_t d[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
        float v = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // ranks past the adapter's: u is zero there, b was made so
          v = fmaf(__uint_as_float(d[j] << 16), u[2 * j], v);
          v = fmaf(__uint_as_float(d[j] & 0xffff0000u), u[2 * j + 1], v);
        }
        for (int o = P >> 1; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
        // column i * per + r, summed by lanes r P .. r P + P - 1, goes to its own lane
        v = __shfl(v, (lane & (per - 1)) << lg, 64);
        if (lane / per == i0 + i) y += v;
      }
    }
  }
  if (F32) static_cast<float *>(g.y)[(int64_t)t * e.N + n0 + lane] = y;
  else static_cast<uint16_t *>(g.y)[(int64_t)t * e.N + n0 + lane] = (uint16_t)pack_bf16(y, 0.0f);
}

// ----------------------------------------------------------------- finish

// Index of a lane's eight values of part p in the planes of u and v.
COLI_DEV int64_t plane_at(int window, int p, int rank_tile, int R32, int lane) {
  return (((int64_t)window * 3 + p) * (R32 / 16) + rank_tile) * 64 + lane;
}

// Sums shrink's parts of u and v.  Writes v as rows (fp32 [T][R32]), both
// as three bf16 parts in the order of the matrix-core operands that grads
// loads -- [Tp/32][3][R32/16][lane][8 rows], lane (c, g) holding rows 8g .. 8g
// + 7 of a window of 32 at rank c: whole KiBs instead of 16-byte pieces of 16
// lines -- and every row's adapter; zeros for rows without one.
struct FinishArgs {
  Requests q;
  const float *part[2];  // u, v
  int splits[2];
  float *rows;           // v
  uint16_t *planes[2];
  int32_t *owner;        // [Tp]
  int T, Tp, R32;
};
COLI_DEV void finish_tile(const FinishArgs &g, int tile, int rank_block, int w) {
  __shared__ float s[64][33];
  __shared__ int own[64];
  const int tid = threadIdx.x, t0 = tile * 64, r0 = rank_block * 32;
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
#pragma unroll 2
  for (int i = tid; i < 64 * 32; i += 256) {
    const int tt = i >> 5, r = i & 31;
    float v = 0.0f;
    if (own[tt] >= 0) {
      const float *p = g.part[w] + (int64_t)(t0 + tt) * g.R32 + r0 + r;
#pragma unroll
      for (int k = 0; k < kMaxSplits; ++k)
        if (k < g.splits[w]) v += p[(int64_t)k * g.T * g.R32];
    }
    if (g.rows && w == 1 && t0 + tt < g.T) g.rows[(int64_t)(t0 + tt) * g.R32 + r0 + r] = v;
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
    reinterpret_cast<uint4 *>(g.planes[w])[plane_at((t0 + tt) / 32, p, (r0 + r) / 16, g.R32,
                                                    (tt % 32) / 8 * 16 + r % 16)] = parts[p];
}

__global__ void __launch_bounds__(256) finish_kernel(FinishArgs g) {
  finish_tile(g, blockIdx.x, blockIdx.y, blockIdx.z);
}

// The backward pass's third launch for short batches: dx from its parts, and
// finish.
__global__ void __launch_bounds__(256) combine_finish_kernel(CombineArgs c, FinishArgs f,
                                                             int combine_blocks) {
  int b = blockIdx.x;
  if (b < combine_blocks) {
    const int nx = (c.e.N + 255) / 256, ny = (c.e.T + 15) / 16;
    combine_tile<false>(c, b % nx, b / nx % ny, b / nx / ny);
    return;
  }
  b -= combine_blocks;
  finish_tile(f, b % (f.Tp / 64), b / (f.Tp / 64) % (f.R32 / 32), b / (f.Tp / 64) / (f.R32 / 32));
}

// ------------------------------------------------------------------ grads

// G_a[f][r] = sum over a's rows t of z[t][f] p[t][r].
struct GradArgs {
  const uint16_t *z;       // [T][F]
  const uint16_t *planes;  // see finish_tile
  float *out;              // [splits][n][R][F] (dA) or [splits][n][F][R] (dB)
  int F;
  int transposed;          // dB's layout
  int f_tiles;
};
struct GradsArgs {
  GradArgs g[2];  // dB (dy, u), dA (x, v)
  const int32_t *owner, *rank;
  int T, Tp, R, R32, n, splits, rows;  // rows per split, a multiple of 64
};

// A workgroup takes 128 columns f, one adapter, up to 16 RT ranks and one
// range of rows; its wavefronts take the range's 64-row windows in turn and
// skip rows of other adapters.  A step contracts 32 rows: lane (c, g) loads
// eight columns of eight rows, 16 bytes each, and an 8 x 8 transposition in
// registers turns them into one operand per column, so that tile j holds
// columns 8c + j.  Bound by its reads of z and of the operands of u and v: 8192
// rows, columns 6144 and 2048, two adapters of rank 64, 25 to 27 us for 134 MB.
template <int RT>
__global__ void __launch_bounds__(256) grads_kernel(GradsArgs a) {
  __shared__ f32x4 buf[2 * RT * 8][64];
  const int lane = threadIdx.x & 63, c = lane & 15, kg = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool second = (int)blockIdx.x >= a.g[0].f_tiles;
  GradArgs g = a.g[0];  // field by field, as in pick()
  g.z = second ? a.g[1].z : g.z;
  g.planes = second ? a.g[1].planes : g.planes;
  g.out = second ? a.g[1].out : g.out;
  g.F = second ? a.g[1].F : g.F;
  g.transposed = second ? a.g[1].transposed : g.transposed;
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
          const int rt = min(r0 / 16 + r, a.R32 / 16 - 1);  // ranks past R32 are not stored
          uint4 v = reinterpret_cast<const uint4 *>(g.planes)[plane_at(w0 / 32 + h, p, rt, a.R32, lane)];
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
  const int rank = rank_of(a.rank, ad, a.R);
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int rr = r0 + 16 * r + 4 * kg;  // four ranks; R is a multiple of 8
    if (rr >= a.R) continue;
    // past the rank: zeros, also from rows that are not finite
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[r][j][e] = rr + e < rank ? acc[r][j][e] : 0.0f;
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
  const bool second = i >= a.n[0];
  if (second) i -= a.n[0];
  const int64_t n = second ? a.n[1] : a.n[0];
  if (i >= n) return;
  const float4 *src = second ? a.src[1] : a.src[0];
  float4 v = src[i];
#pragma unroll 4
  for (int s = 1; s < a.splits; ++s) {
    const float4 o = src[s * n + i];
    v.x += o.x;
    v.y += o.y;
    v.z += o.z;
    v.w += o.w;
  }
  (second ? a.dst[1] : a.dst[0])[i] = v;
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
  int s = 256 / tiles;
  if (s > F / 256) s = F / 256;
  return s < 1 ? 1 : (s > kMaxSplits ? kMaxSplits : s);
}
// Row ranges of the gradients: about 512 workgroups, which run in two rounds
// (at rank 64 a wavefront takes 384 registers, so a CU holds one workgroup).
// 8192 rows, two adapters of rank 64, 6144 and 2048 columns: 26.8 us, against
// 37.8 us with 1,024 and 32.8 us with 256.
int grad_splits(int T, int N, int K, int n) {
  const int64_t blocks = (int64_t)((N + 127) / 128 + (K + 127) / 128) * n;
  const int windows = (T + 255) / 256;  // a window per wavefront
  int64_t s = (512 + blocks - 1) / blocks;
  if (s > windows) s = windows;
  return (int)(s > 16 ? 16 : s);
}

// Which kernels compute T x K times N x K.  Measured on int4 (us, stream /
// direct / gemm, each with the launches it needs):
//   N 2048 K 6144, T  64: 21 / 25 / 85   T 256: 33 / 28 / 82   T 1024: 102 / 70 / 77
//   N 6144 K 2048, T  64: 18 / 15 / 44   T 256: 42 / 29 / 43   T 1024: 118 / 68 / 41
//   N 2048 K 1024, T  64: 13 / 10 / 19   T 517: 25 / 20 / 21   T 2048: the gemm
// The streaming kernel reads x once per 16-64 columns, which pays only for
// few rows (more of them where K is long and its splits keep the chip busy);
// the gemm needs its 256 x 128 tiles to reach most CUs and a pass that
// unpacks the weights.  Narrow matrices (us, direct / gemm, 8 requests of
// rank 32; the bound of 96 tiles is what wide ones need, and in between these
// are on the slower side of it):
//   N  128 K 2048, T 1024: 16 / 44   T 4096: 33 / 47   T 8192: 47 / 46   T 16384: 80 / 49
//   N  512 K 2048, T 1024: 24 / 45   T 2048: 34 / 46   T 4096: 60 / 49
//   N  512 K 6144, T 1024: 51 / 94   T 2048: 77 / 95   T 4096: 141 / 97
//   N 1024 K 2048, T  600: 23 / 48   T 1024: 30 / 48   T 2048: 54 / 49
enum Path { kStream, kDirect, kGemm };
Path path_of(int T, int N, int K) {
  if (T <= (K > 4096 ? 128 : 32)) return kStream;
  const int tiles = (T + 255) / 256 * ((N + 127) / 128);
  return T > 512 && tiles >= 96 ? kGemm : kDirect;
}
constexpr int kLastPartRows = 96 * 256;  // from here on one column of tiles is enough
// The streaming path's tiles: columns per workgroup grow with the rows, so
// that x is not read once per 16 columns.
int stream_mt(int T) { return T <= 16 ? 1 : (T <= 32 ? 2 : 4); }
int clamp_splits(int s, int most) {
  if (s > most) s = most;
  return s < 1 ? 1 : (s > kMaxSplits ? kMaxSplits : s);
}
int part_splits(int T, int N, int K) {
  if (path_of(T, N, K) == kDirect) {
    const int tiles = (N + kDirectCols - 1) / kDirectCols * ((T + kDirectRows - 1) / kDirectRows);
    return clamp_splits(512 / tiles, K / 64 / (2 * kDirectGroups));
  }
  const int mt = stream_mt(T);
  const int blocks = N / (16 * mt) * ((T + 16 * mt - 1) / (16 * mt));
  return clamp_splits(256 / blocks, K / 64 / kStreamWaves);
}
// 64-wide groups of a split (direct) or of a split's wavefront (stream).
int part_groups(int T, int N, int K, int splits) {
  const int over = path_of(T, N, K) == kDirect ? splits : splits * kStreamWaves;
  return (K / 64 + over - 1) / over;
}
// Four 64-wide blocks per wavefront of u's and v's workgroups beside the parts.
int part_shrink_splits(int T, int N, int K, int F) {
  const int waves = path_of(T, N, K) == kDirect ? kDirectWaves : kStreamWaves;
  return clamp_splits((F / 64 + 4 * waves - 1) / (4 * waves), kMaxSplits);
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
  const bool stream = (backward ? path_of(T, (int)K, (int)N) : path_of(T, (int)N, (int)K)) != kGemm;
  if (stream) {  // backward: dx [T][K], contracted over N
    o.sp = backward ? part_splits(T, (int)K, (int)N) : part_splits(T, (int)N, (int)K);
    const int n_out = (int)(backward ? K : N), n_in = (int)(backward ? N : K);
    o.su = part_shrink_splits(T, n_out, n_in, (int)K);
    o.sv = part_shrink_splits(T, n_out, n_in, (int)N);
    o.part = c.take<float>((size_t)o.sp * T * (backward ? K : N));
  }
  if (backward || !stream) o.plane = c.take<uint16_t>(N * K);
  if (!backward && !stream) o.sc = c.take<float>(N * K / 64);
  if (n) {
    o.part_u = c.take<float>((size_t)o.su * T * o.R32);
    if (backward) {
      o.part_v = c.take<float>((size_t)o.sv * T * o.R32);
      if (!stream) o.rows = c.take<float>((size_t)T * o.R32);
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

// Whether the second launch goes row by row (its cost: rows times rank) or by
// tiles (tiles times the requests in each).  us by tiles / by rows:
//   256 rows, rank  64,  4 rows per request: 13.0 /  9.8    8: 10.3 /  9.6
//   517 rows, rank  64, 14 rows per request: 11.3 / 13.2
//   517 rows, rank  24,  4 rows per request: 14.9 / 10.4   14: 10.2 /  8.9   21: 10.3 / 9.2
//    64 rows, rank  16, 16 rows per request:  5.9 /  4.7
//   512 rows, rank 128,  3 rows per request: 23.0 / 22.0    8: 35.2 / 53.0
bool row_wise(int T, int n_req, int R) {
  return T <= (int64_t)n_req * (R <= 64 ? 512 / (R < 16 ? 16 : R) : 2);
}

// Workgroups (per tile) that the requests of a tile are spread over.
int spread(int rows, int n_req) { return n_req < rows ? n_req : rows; }
// The same for the long requests' 64-row tiles: what a tile holds on average,
// and one more for tiles that a boundary cuts.
int spread_long(int T, int n_req) {
  const int tiles = (T + 63) / 64;
  return spread(16, n_req < 2 ? n_req : (n_req + tiles - 1) / tiles + 1);
}

int launch_shrink(const ShrinkArgs &a, const ShrinkArgs &b, hipStream_t s) {
  const dim3 grid((a.T + 63) / 64, a.nsub, a.splits + b.splits), block(256);
  if (a.R32 <= 32) launch_k(COLI_K_PROJECT_SHRINK, shrink_kernel<2>, grid, block, 0, s, a, b);
  else if (a.R32 <= 64) launch_k(COLI_K_PROJECT_SHRINK, shrink_kernel<4>, grid, block, 0, s, a, b);
  else launch_k(COLI_K_PROJECT_SHRINK, shrink_kernel<8>, grid, block, 0, s, a, b);
  return hip_status(hipGetLastError());
}

template <int BM, int BN, int WM, bool SCALED, bool F32>
int launch_gemm_cfg(const GemmArgs &g, hipStream_t s) {
  const unsigned tiles = (unsigned)(((g.N + BN - 1) / BN) * ((g.T + BM - 1) / BM));
  launch_k(COLI_K_PROJECT_GEMM, gemm_kernel<BM, BN, WM, SCALED, F32>, dim3((tiles + 7) / 8 * 8),
           dim3(BM / WM * BN), 0, s, g);
  return hip_status(hipGetLastError());
}

template <bool SCALED, bool F32>
int launch_gemm(const GemmArgs &g, hipStream_t s) {
  return launch_gemm_cfg<256, 128, 64, SCALED, F32>(g, s);
}

template <int F, int RT>
int launch_stream(const StreamArgs &g, int N, hipStream_t s) {  // N: the columns the path was chosen for
  if (path_of(g.T, N, g.m.K) == kDirect) {
    const int tiles = (g.m.N + kDirectCols - 1) / kDirectCols * ((g.T + kDirectRows - 1) / kDirectRows);
    launch_k(COLI_K_PROJECT_STREAM, direct_kernel<F, RT>, dim3(g.shrink_blocks + tiles * g.splits),
             dim3(64 * kDirectWaves), 0, s, g);
    return hip_status(hipGetLastError());
  }
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
int launch_stream_rank(const StreamArgs &g, int N, int R32, hipStream_t s) {
  if (R32 <= 32) return launch_stream<F, 2>(g, N, s);
  if (R32 <= 64) return launch_stream<F, 4>(g, N, s);
  return launch_stream<F, 8>(g, N, s);
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

// The most that any batch of up to T rows needs: the parts of a batch in
// between can take more than a long batch's unpacked weights.  Sizes grow
// with T between multiples of 16 (every tile's and path's bound is one).
size_t project_workspace_upto(const Layer &L, int matrix, int n, int R, int T, int backward) {
  size_t most = project_workspace(L, matrix, n, R, T, backward);
  for (int t = 16; t < T && t <= kLastPartRows; t += 16) {
    const size_t need = project_workspace(L, matrix, n, R, t, backward);
    if (need > most) most = need;
  }
  return most;
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
    sh = {x, ad->a, ad->rank, ad->scale, e.q, w.part_u, T, m.K, e.R, e.R32, w.su,
          path_of(T, m.N, m.K) == kGemm ? spread_long(T, e.q.n) : spread(16, e.q.n)};
  }
  int rc;
  if (path_of(T, m.N, m.K) != kGemm) {
    StreamArgs g = {};
    g.m = m;
    g.x = x;
    g.part = w.part;
    g.T = T;
    g.splits = w.sp;
    g.per = part_groups(T, m.N, m.K, w.sp);
    g.shrink_tiles = (T + 15) / 16;
    g.s[0] = sh;
    CombineArgs c = {};
    c.part = w.part;
    c.splits = w.sp;
    c.nsub = 1;
    c.y = y;
    c.e = e;
    if (ad) {
      c.nsub = sh.nsub;
      g.shrink_blocks = g.shrink_tiles * c.nsub * w.su;
    }
    rc = fmt == kI4 ? launch_stream_rank<kI4>(g, m.N, w.R32, s)
                    : (fmt == kI8 ? launch_stream_rank<kI8>(g, m.N, w.R32, s)
                                  : launch_stream_rank<kF4>(g, m.N, w.R32, s));
    if (rc) return rc;
    if (ad && row_wise(T, e.q.n, e.R)) {
      const dim3 rows((m.N + 255) / 256, T);
      if (f32) launch_k(COLI_K_PROJECT_COMBINE, combine_rows_kernel<true>, rows, dim3(256), 0, s, c);
      else launch_k(COLI_K_PROJECT_COMBINE, combine_rows_kernel<false>, rows, dim3(256), 0, s, c);
      return hip_status(hipGetLastError());
    }
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
  const bool stream = path_of(T, m.K, m.N) != kGemm;
  ShrinkArgs u = {}, v = {};
  FinishArgs f = {};
  if (ad) {
    const int nsub = stream ? spread(16, p.q.n) : spread_long(T, p.q.n);
    u = {x, ad->a, ad->rank, ad->scale, p.q, w.part_u, T, m.K, R, w.R32, w.su, nsub};
    v = {dy, w.bt, ad->rank, ad->scale, p.q, w.part_v, T, m.N, R, w.R32, w.sv, nsub};
    f.q = p.q;
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
  }
  if (stream) {
    StreamArgs g = {};
    g.m = {reinterpret_cast<const uint8_t *>(w.plane), nullptr, dx ? m.K : 0, m.N};
    g.x = dy;
    g.part = w.part;
    g.T = T;
    g.splits = w.sp;
    g.per = part_groups(T, m.K, m.N, w.sp);
    g.shrink_tiles = (T + 15) / 16;
    g.s[0] = u;
    g.s[1] = v;
    g.shrink_blocks = g.shrink_tiles * u.nsub * (u.splits + v.splits);
    if ((rc = launch_stream_rank<kBF>(g, m.K, w.R32, s))) return rc;
    CombineArgs c = {};
    c.part = w.part;
    c.splits = w.sp;
    c.nsub = ad ? u.nsub : 1;
    c.y = dx;
    c.e.T = T;
    c.e.N = m.K;
    if (ad) c.e = {p.q, w.part_v, w.at, ad->rank, T, m.K, R, w.R32, w.sv};
    const int cb = dx ? (m.K + 255) / 256 * ((T + 15) / 16) * c.nsub : 0;
    const int fb = d_a ? w.Tp / 64 * (w.R32 / 32) * 2 : 0;
    launch_k(COLI_K_PROJECT_COMBINE, combine_finish_kernel, dim3(cb + fb), dim3(256), 0, s, c, f, cb);
    if ((rc = hip_status(hipGetLastError()))) return rc;
  } else if (ad) {
    if ((rc = launch_shrink(u, v, s))) return rc;
    launch_k(COLI_K_PROJECT_FINISH, finish_kernel, dim3(w.Tp / 64, w.R32 / 32, 2), dim3(256), 0, s, f);
    if ((rc = hip_status(hipGetLastError()))) return rc;
  }
  if (d_a) {
    GradsArgs a = {};
    a.g[0] = {dy, w.planes_u, w.sg > 1 ? w.pb : d_b, m.N, 1, (m.N + 127) / 128};
    a.g[1] = {x, w.planes_v, w.sg > 1 ? w.pa : d_a, m.K, 0, (m.K + 127) / 128};
    a.owner = w.owner;
    a.rank = ad->rank;
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
  if (!dx || stream) return COLI_OK;
  ExpandArgs e = {};
  if (ad) e = {p.q, w.rows, w.at, ad->rank, T, m.K, R, w.R32, 1};
  return launch_gemm<false, false>({dy, w.plane, nullptr, T, m.K, m.N, dx, e}, s);
}

}  // namespace coli
