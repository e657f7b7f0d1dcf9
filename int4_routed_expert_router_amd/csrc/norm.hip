// norm.hip -- the root-mean-square norm in front of the layer: the residual's
// addition, the norm and the prefill path's codes in one pass; its gradients.
//
//   s = residual + x;  y = s r w,  r = 1 / sqrt(mean s^2 + eps)
//   d = r (n - h mean(n h)) + d_total,  n = dy w,  h = s r;  d_w = sum dy h
//
// Memory bounds both: a row stays in registers between its sum and its
// results, so everything moves once.  16,384 x 6144 with MXFP8 codes (909 MB):
// 157 to 161 us, 5.7 TB/s (a copy of 1 GiB on this card: 5.1); the gradients at
// 8,192 with an fp32 stream (805 MB): 150 us.  A row lies over as many lanes as keep a
// lane's share at one chunk of eight values (forward: up to four, with more
// rows at work instead); up to 64 lanes several rows share a workgroup and sum
// without LDS.
#include "act_codec.h"
#include "internal.h"
#include "lanes.h"
#include "units.h"

namespace coli {
namespace {

constexpr int kThreads = 256;
constexpr int block_of(int lanes) { return lanes > 64 ? lanes : kThreads; }

// Values of a lane's units: fours where the stream is fp32, else eights.
constexpr int unit_of(bool f32) { return f32 ? 4 : 8; }

template <int U>
COLI_DEV void load_weight(const void *w, int f32, int i, float (&v)[U]) {
  if (!w) {
#pragma unroll
    for (int j = 0; j < U; ++j) v[j] = 1.0f;
  } else if (f32) {
    unpack(load_unit<U, true, false>(w, i), v);
  } else {
    unpack(load_unit<U, false, false>(w, i), v);
  }
}

// ------------------------------------------------------------------ forward

struct NormArgs {
  const uint16_t *x;
  const void *residual;
  void *total;
  const void *weight;
  uint16_t *y;
  uint8_t *q;
  void *scales;
  int T, units;  // rows, and units of a row
  int weight_f32, format;
  float eps, inv_h;
};

// RES: 0 no residual, 1 bf16, 2 fp32.  A row is held by LPR lanes, NU units each.
template <int LPR, int NU, int RES, bool NT>
__global__ void __launch_bounds__(block_of(LPR)) norm_kernel(NormArgs g) {
  constexpr int U = unit_of(RES == 2);
  constexpr int B = block_of(LPR), RPB = B / LPR;  // rows of a workgroup
  __shared__ float red[2][1][waves_of(LPR)];
  const int li = threadIdx.x % LPR;
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / LPR; row < g.T;
       row += (int64_t)gridDim.x * RPB, turn ^= 1) {
    const int64_t base = row * g.units;
    float v[NU][U];
    float sum[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < NU; ++c) {
      const int i = li + c * LPR;
#pragma unroll
      for (int j = 0; j < U; ++j) v[c][j] = 0.0f;
      if (i < g.units) {
        unpack(load_unit<U, false, NT>(g.x, base + i), v[c]);
        if (RES) {
          float r[U];
          unpack(load_unit<U, RES == 2, NT>(g.residual, base + i), r);
#pragma unroll
          for (int j = 0; j < U; ++j) v[c][j] += r[j];
          const auto p = pack<U, RES == 2>(v[c]);
          store_unit<U, RES == 2, NT>(g.total, base + i, p);
          unpack(p, v[c]);  // the stored sum is what is normed
        }
      }
#pragma unroll
      for (int j = 0; j < U; ++j) sum[0] = fmaf(v[c][j], v[c][j], sum[0]);
    }
    row_sums<LPR, 1>(sum, red[turn]);
    const float r = rsqrtf(fmaf(sum[0], g.inv_h, g.eps));
#pragma unroll
    for (int c = 0; c < NU; ++c) {
      const int i = li + c * LPR;
      if (i >= g.units) continue;  // with codes, whole blocks of lanes
      float w[U];
      load_weight(g.weight, g.weight_f32, i, w);
#pragma unroll
      for (int j = 0; j < U; ++j) w[j] *= v[c][j] * r;
      const auto p = pack<U, false>(w);
      if (g.y) store_unit<U, false, NT>(g.y, base + i, p);
      if (g.format != COLI_NORM_PLAIN) {
        uint32_t q[U / 4];
        constexpr int L = 32 / U;  // lanes of a block
        unpack(p, w);
        if (g.format == COLI_NORM_Q8_0) {
          const uint16_t d = q8_0_lane(w, q);
          if (i % L == 0) reinterpret_cast<uint16_t *>(g.scales)[(base + i) / L] = d;
        } else {
          const uint32_t e = mx8_lane(w, q);
          if (i % L == 0) reinterpret_cast<uint8_t *>(g.scales)[(base + i) / L] = (uint8_t)e;
        }
        uint32_t *to = reinterpret_cast<uint32_t *>(g.q) + (base + i) * (U / 4);
        if (U == 8)
          *reinterpret_cast<uint2 *>(to) = make_uint2(q[0], q[U / 4 - 1]);
        else
          *to = q[0];
      }
    }
  }
}

// NC: chunks of eight values to a lane.
template <int RES, int LPR, int NC>
void run_norm(const NormArgs &g, hipStream_t s) {
  constexpr int B = block_of(LPR), RPB = B / LPR, U = unit_of(RES == 2), NU = NC * 8 / U;
  const int64_t blocks = ((int64_t)g.T + RPB - 1) / RPB;
  // From half as much again as the last cache on, x, residual, total and y go
  // past it: 8,192 x 6144 in 69 us instead of 76, and 172 instead of 178 with a
  // reader of y behind; fp32 16,384 x 2048 67 instead of 73, and 135 instead of
  // 146 with the next norm behind; bf16 16,384 x 2048 (268 MB) 44 against 41.
  const int64_t bytes = (int64_t)g.T * g.units * U * (RES == 2 ? 12 : RES ? 8 : 4);
  launch_k(COLI_K_NORM,
           bytes >= int64_t(384) << 20 ? norm_kernel<LPR, NU, RES, true>
                                       : norm_kernel<LPR, NU, RES, false>,
           dim3((unsigned)(blocks < (1 << 20) ? blocks : (1 << 20))), dim3(B), 0, s, g);
}

template <int RES>
void pick_norm(const NormArgs &g, hipStream_t s) {
  const int n = g.units * unit_of(RES == 2) / 8;
  if (n <= 8) return run_norm<RES, 8, 1>(g, s);
  if (n <= 16) return run_norm<RES, 16, 1>(g, s);
  if (n <= 32) return run_norm<RES, 32, 1>(g, s);
  if (n <= 64) return run_norm<RES, 64, 1>(g, s);
  if (n <= 128) return run_norm<RES, 64, 2>(g, s);
  if (n <= 256) return run_norm<RES, 256, 1>(g, s);
  if (n <= 512) return run_norm<RES, 256, 2>(g, s);
  if (n <= 768) return run_norm<RES, 256, 3>(g, s);
  if (n <= 1024) return run_norm<RES, 256, 4>(g, s);
  run_norm<RES, 1024, 2>(g, s);
}

// ----------------------------------------------------------------- backward

struct NormBackArgs {
  const void *total;
  const uint16_t *dy;
  const void *d_total;
  const void *weight;
  uint16_t *dx;
  void *d_residual;
  float *parts;  // of d_weight [gridDim.x][H] (one workgroup: d_weight itself), or NULL
  int T, units;
  int weight_f32;
  float eps, inv_h;
};

// One lane's share of a row, as loaded.
template <int NU, bool F32>
struct BackRow {
  Unit<unit_of(F32), F32> s[NU], o[NU];
  Unit<unit_of(F32), false> dy[NU];
};

template <int LPR, int NU, bool F32, bool NT>
COLI_DEV void load_row(const NormBackArgs &g, int64_t row, int li, BackRow<NU, F32> &r) {
  constexpr int U = unit_of(F32);
  const int64_t base = row * g.units;
#pragma unroll
  for (int c = 0; c < NU; ++c) {
    const int i = li + c * LPR;
    r.s[c] = r.o[c] = {};
    r.dy[c] = {};
    if (row < g.T && i < g.units) {
      r.s[c] = load_unit<U, F32, NT>(g.total, base + i);
      r.dy[c] = load_unit<U, false, NT>(g.dy, base + i);
      if (g.d_total) r.o[c] = load_unit<U, F32, NT>(g.d_total, base + i);
    }
  }
}

// d = r (n - h mean(n h)) + d_total with h = s r: both row sums, of s^2 and of
// n s, come from the one pass that loads the row.  A workgroup goes over rows
// with the next one's loads in flight (up to 8192 values), and keeps its part
// of d_weight in registers.
template <int LPR, int NU, bool F32, bool NT, int B>
__global__ void __launch_bounds__(B) norm_backward_kernel(NormBackArgs g) {
  constexpr int U = unit_of(F32), RPB = B / LPR;  // rows of a workgroup
  __shared__ float red[2][2][(LPR > 64 ? RPB : 1) * waves_of(LPR)];
  const int li = threadIdx.x % LPR, ri = threadIdx.x / LPR;
  float dw[NU][U];
#pragma unroll
  for (int c = 0; c < NU; ++c)
#pragma unroll
    for (int j = 0; j < U; ++j) dw[c][j] = 0.0f;
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t first = (int64_t)blockIdx.x * RPB;  // the same for the whole workgroup
  // two chunks to a lane leave no registers for a second row (fp32 4,096 x 16,384:
  // 218 us, with it 272)
  constexpr bool kAhead = NU * U == 8;
  BackRow<NU, F32> a, next;
  if (kAhead) load_row<LPR, NU, F32, NT>(g, first + ri, li, a);
  int turn = 0;
  for (; first < g.T; first += step, turn ^= 1) {
    const int64_t row = first + ri;  // past the last: zeros, and no results
    if (kAhead)
      load_row<LPR, NU, F32, NT>(g, row + step, li, next);
    else
      load_row<LPR, NU, F32, NT>(g, row, li, a);
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < NU; ++c) {
      const int i = li + c * LPR;
      float v[U], dy[U], w[U];
      unpack(a.s[c], v);
      unpack(a.dy[c], dy);
      load_weight(i < g.units ? g.weight : nullptr, g.weight_f32, i, w);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        sum[0] = fmaf(v[j], v[j], sum[0]);
        sum[1] = fmaf(dy[j] * w[j], v[j], sum[1]);
      }
    }
    row_sums<LPR, 2, (LPR > 64 ? RPB : 1)>(sum, red[turn], ri);
    const float r = rsqrtf(fmaf(sum[0], g.inv_h, g.eps));
    const float m = sum[1] * g.inv_h * r;  // mean(n h)
    const int64_t base = row * g.units;
#pragma unroll
    for (int c = 0; c < NU; ++c) {
      const int i = li + c * LPR;
      if (i >= g.units || (RPB > 1 && row >= g.T)) continue;
      float v[U], dy[U], o[U], w[U], d[U];
      unpack(a.s[c], v);
      unpack(a.o[c], o);
      unpack(a.dy[c], dy);
      load_weight(g.weight, g.weight_f32, i, w);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const float h = v[j] * r;
        dw[c][j] = fmaf(dy[j], h, dw[c][j]);
        d[j] = fmaf(r, fmaf(-h, m, dy[j] * w[j]), o[j]);
      }
      if (g.dx) store_unit<U, false, NT>(g.dx, base + i, pack<U, false>(d));
      if (g.d_residual) store_unit<U, F32, NT>(g.d_residual, base + i, pack<U, F32>(d));
    }
    if (kAhead) a = next;
  }
  if (!g.parts) return;
  if (RPB == 1) {
#pragma unroll
    for (int c = 0; c < NU; ++c) {
      const int i = li + c * LPR;
      if (i < g.units)
        store_unit<U, true, false>(g.parts, (int64_t)blockIdx.x * g.units + i, pack<U, true>(dw[c]));
    }
    return;
  }
  // the rows of a workgroup that went side by side
  __shared__ float side[RPB > 1 ? RPB : 1][RPB > 1 ? LPR * NU * U : 1];
#pragma unroll
  for (int c = 0; c < NU; ++c)
#pragma unroll
    for (int j = 0; j < U; ++j)
      side[RPB > 1 ? ri : 0][RPB > 1 ? U * (li + c * LPR) + j : 0] = dw[c][j];
  __syncthreads();
  for (int c = threadIdx.x; c < U * g.units; c += B) {
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < RPB; ++k) sum += side[k][RPB > 1 ? c : 0];
    g.parts[(int64_t)blockIdx.x * U * g.units + c] = sum;
  }
}

// Sums n parts of H columns: COLS columns to a workgroup, every (1024 / COLS)th
// part to COLS lanes, sixteen loads in flight.  16 columns keep the chip busy
// with many parts of short rows (1,536 of 1024: 4.9 us with an empty launch's
// 3.9; 64 columns 6.7), 64 read whole lines of long ones (256 of 16,384: 4.1
// against 6.9).  In between, 768 parts of 2048, 512 of 4096 and 256 of 6144 take
// 4.0 to 4.1 either way.
template <int COLS>
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float *__restrict__ parts, int n,
                                                           int H, float *__restrict__ out) {
  constexpr int G = 1024 / COLS;
  __shared__ float red[G][COLS];
  const int col = threadIdx.x % COLS, first = threadIdx.x / COLS;
  const int c = blockIdx.x * COLS + col;
  float a = 0.0f;
  if (c < H) {
    for (int p0 = first; p0 < n; p0 += 16 * G) {
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int p = p0 + G * i;
        v[i] = p < n ? parts[(int64_t)p * H + c] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) a += v[i];
    }
  }
  red[first][col] = a;
  __syncthreads();
  if (first != 0 || c >= H) return;
  a = 0.0f;
#pragma unroll
  for (int j = 0; j < G; ++j) a += red[j][col];
  out[c] = a;
}

// Lanes of a row in the backward pass: one chunk each up to 8192 values, as what
// a lane keeps of a chunk (the row, the next one, d_weight) is 80 to 90
// registers (8,192 x 6144: 256 lanes with three chunks 90 us, 768 with one 87;
// 65,536 x 1024: 64 lanes with two 127, 128 with one 113).
int backward_lanes(int chunks) {
  if (chunks <= 8) return 8;
  if (chunks <= 16) return 16;
  if (chunks <= 32) return 32;
  if (chunks <= 64) return 64;
  if (chunks <= 128) return 128;
  if (chunks <= 256) return 256;
  if (chunks <= 512) return 512;
  return chunks <= 768 ? 768 : 1024;
}
// Workgroups, and parts of d_weight: some 768 lanes to each of the 256 CUs.
// More would be more parts and fewer rows to each (65,536 x 2048: 768
// workgroups 219 us, 1,024 and 1,280 226; x 1024: 1,024 141, 1,536 and 2,048
// 113; 8,192 x 6144: 256 87, 512 89).
int backward_groups(int chunks, int T) {
  const int lanes = backward_lanes(chunks), block = block_of(lanes);
  const int groups = (T + block / lanes - 1) / (block / lanes);
  const int most = 256 * ((768 + block - 1) / block);
  return groups < most ? groups : most;
}

// Whether one workgroup of few_of threads takes all rows where d_weight is asked
// for: it writes that itself, and the call is one launch instead of two.  Up to
// four turns of its rows: in a row of calls 16 rows of 2048 in 6.9 us instead of
// 8.6, alone 20.1 against 19.4 with the wait, 12 rows 18.9 against 19.4; two of
// 16,384 7.1, three 9.4.
constexpr int few_of(int lanes) { return lanes == 768 ? 768 : 1024; }
bool few_rows(int chunks, int T) {
  const int lanes = backward_lanes(chunks);
  return T <= (chunks <= 1024 ? 4 : 2) * (few_of(lanes) / lanes);
}

// NC: chunks of eight values to a lane.
template <int LPR, int NC, bool F32>
void run_norm_backward(const NormBackArgs &g, hipStream_t s) {
  constexpr int U = unit_of(F32), NU = NC * 8 / U, B = block_of(LPR), FEW = few_of(LPR);
  const int chunks = g.units * U / 8;
  if (g.parts && few_rows(chunks, g.T)) {
    launch_k(COLI_K_NORM_BACKWARD, norm_backward_kernel<LPR, NU, F32, false, FEW>, dim3(1),
             dim3(FEW), 0, s, g);
    return;
  }
  // As in the forward pass: fp32 16,384 x 2048 (512 MB) in 95 us instead of 102,
  // and 190 instead of 204 with the next layer's behind; 8,192 x 2048 (256 MB) 51
  // against 49.
  const bool nt = (int64_t)g.T * g.units * U * (F32 ? 16 : 8) >= int64_t(384) << 20;
  launch_k(COLI_K_NORM_BACKWARD,
           nt ? norm_backward_kernel<LPR, NU, F32, true, B>
              : norm_backward_kernel<LPR, NU, F32, false, B>,
           dim3(backward_groups(chunks, g.T)), dim3(B), 0, s, g);
}

template <bool F32>
void pick_norm_backward(const NormBackArgs &g, hipStream_t s) {
  const int chunks = g.units * unit_of(F32) / 8;
  switch (backward_lanes(chunks)) {
    case 8: return run_norm_backward<8, 1, F32>(g, s);
    case 16: return run_norm_backward<16, 1, F32>(g, s);
    case 32: return run_norm_backward<32, 1, F32>(g, s);
    case 64: return run_norm_backward<64, 1, F32>(g, s);
    case 128: return run_norm_backward<128, 1, F32>(g, s);
    case 256: return run_norm_backward<256, 1, F32>(g, s);
    case 512: return run_norm_backward<512, 1, F32>(g, s);
    case 768: return run_norm_backward<768, 1, F32>(g, s);
    default:
      return chunks <= 1024 ? run_norm_backward<1024, 1, F32>(g, s)
                            : run_norm_backward<1024, 2, F32>(g, s);
  }
}

}  // namespace

size_t norm_workspace(int H, int T) {
  return align_up((size_t)backward_groups(H / 8, T) * H * sizeof(float));
}

int launch_norm(const coli_moe_norm_t &n, const uint16_t *x, const void *residual,
                int residual_dtype, int T, void *total, uint16_t *y, int format, void *q,
                void *scales, hipStream_t s) {
  NormArgs g{};
  g.x = x;
  g.residual = residual;
  g.total = total;
  g.weight = n.weight;
  g.y = y;
  g.q = reinterpret_cast<uint8_t *>(q);
  g.scales = scales;
  g.T = T;
  g.units = n.hidden / unit_of(residual && residual_dtype == COLI_SRC_F32);
  g.weight_f32 = n.weight_dtype == COLI_SRC_F32;
  g.format = format;
  g.eps = n.eps;
  g.inv_h = 1.0f / (float)n.hidden;
  if (!residual)
    pick_norm<0>(g, s);
  else if (residual_dtype == COLI_SRC_BF16)
    pick_norm<1>(g, s);
  else
    pick_norm<2>(g, s);
  return hip_status(hipGetLastError());
}

int launch_norm_backward(const coli_moe_norm_t &n, const void *total, int total_dtype,
                         const uint16_t *dy, const void *d_total, int T, uint16_t *dx,
                         void *d_residual, float *d_weight, void *ws, hipStream_t s) {
  NormBackArgs g{};
  g.total = total;
  g.dy = dy;
  g.d_total = d_total;
  g.weight = n.weight;
  g.dx = dx;
  g.d_residual = d_residual;
  const bool few = few_rows(n.hidden / 8, T);
  g.parts = few || !d_weight ? d_weight : reinterpret_cast<float *>(ws);
  g.T = T;
  g.units = n.hidden / unit_of(total_dtype == COLI_SRC_F32);
  g.weight_f32 = n.weight_dtype == COLI_SRC_F32;
  g.eps = n.eps;
  g.inv_h = 1.0f / (float)n.hidden;
  if (total_dtype == COLI_SRC_F32)
    pick_norm_backward<true>(g, s);
  else
    pick_norm_backward<false>(g, s);
  if (hipGetLastError() != hipSuccess) return COLI_E_HIP;
  if (!d_weight || few) return COLI_OK;
  const int H = n.hidden;
  launch_k(COLI_K_NORM_REDUCE, H <= 2048 ? norm_reduce_kernel<16> : norm_reduce_kernel<64>,
           dim3(H <= 2048 ? (H + 15) / 16 : (H + 63) / 64), dim3(1024), 0, s, (const float *)ws,
           backward_groups(H / 8, T), H, d_weight);
  return hip_status(hipGetLastError());
}

}  // namespace coli
