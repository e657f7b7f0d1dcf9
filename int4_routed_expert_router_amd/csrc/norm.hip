// norm.hip -- the root-mean-square norm in front of the layer: the residual's
// addition, the norm and the prefill path's codes in one pass; its gradients.
#include "act_codec.h"
#include "internal.h"
#include "values8.h"

namespace coli {
namespace {

constexpr int kThreads = 256;

COLI_DEV void weight8(const void *w, int f32, int i, float v[8]) {
  if (!w) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 1.0f;
  } else if (f32) {
    load8<true>(w, i, v);
  } else {
    load8<false>(w, i, v);
  }
}

// Sums of N values over the W waves that share a row (W = 1: the wave itself).
template <int W, int N>
COLI_DEV void row_sums(float (&v)[N], float (*red)[W]) {
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = wave_sum(v[n]);
  if (W == 1) return;
  const int wave = threadIdx.x >> 6;
  __syncthreads();  // the last row's sums have been read
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int n = 0; n < N; ++n) red[n][wave] = v[n];
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    v[n] = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) v[n] += red[n][w];
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
  int T, chunks;  // rows, and chunks of eight values in a row
  int weight_f32, format;
  float eps, inv_h;
};

// RES: 0 no residual, 1 bf16, 2 fp32.  A row is held by 256 lanes, NC chunks
// of eight values each.
template <int NC, int RES>
__global__ void __launch_bounds__(kThreads) norm_kernel(NormArgs g) {
  __shared__ float red[1][4];
  for (int64_t row = blockIdx.x; row < g.T; row += gridDim.x) {
    const int64_t base = row * g.chunks;
    float v[NC][8];
    float sum[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = threadIdx.x + c * kThreads;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] = 0.0f;
      if (i < g.chunks) {
        load8<false>(g.x, base + i, v[c]);
        if (RES) {
          float r[8];
          load8<RES == 2>(g.residual, base + i, r);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[c][j] += r[j];
          if (RES == 1) {  // the stored sum is what is normed
            const uint4 p = pack8(v[c]);
            reinterpret_cast<uint4 *>(g.total)[base + i] = p;
            unpack8(p, v[c]);
          } else {
            store8<true>(g.total, base + i, v[c]);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[0] = fmaf(v[c][j], v[c][j], sum[0]);
    }
    row_sums<4, 1>(sum, red);
    const float r = rsqrtf(fmaf(sum[0], g.inv_h, g.eps));
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = threadIdx.x + c * kThreads;
      if (i >= g.chunks) continue;  // with codes, whole quads of lanes
      float w[8];
      weight8(g.weight, g.weight_f32, i, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] *= v[c][j] * r;
      const uint4 p = pack8(w);
      if (g.y) reinterpret_cast<uint4 *>(g.y)[base + i] = p;
      if (g.format != COLI_NORM_PLAIN) {
        uint32_t q[2];
        unpack8(p, w);
        if (g.format == COLI_NORM_Q8_0) {
          const uint16_t d = q8_0_lane(w, q);
          if ((i & 3) == 0) reinterpret_cast<uint16_t *>(g.scales)[(base + i) >> 2] = d;
        } else {
          const uint32_t e = mx8_lane(w, q);
          if ((i & 3) == 0) reinterpret_cast<uint8_t *>(g.scales)[(base + i) >> 2] = (uint8_t)e;
        }
        reinterpret_cast<uint2 *>(g.q)[base + i] = make_uint2(q[0], q[1]);
      }
    }
  }
}

template <int RES>
void pick_norm(const NormArgs &g, hipStream_t s) {
  const int nc = (g.chunks + kThreads - 1) / kThreads;
  const int grid = g.T < (1 << 16) ? g.T : (1 << 16);
  launch_k(COLI_K_NORM,
           nc == 1   ? norm_kernel<1, RES>
           : nc == 2 ? norm_kernel<2, RES>
           : nc == 3 ? norm_kernel<3, RES>
           : nc == 4 ? norm_kernel<4, RES>
                     : norm_kernel<8, RES>,
           dim3(grid), dim3(kThreads), 0, s, g);
}

// ----------------------------------------------------------------- backward

struct NormBackArgs {
  const void *total;
  const uint16_t *dy;
  const void *d_total;
  const void *weight;
  uint16_t *dx;
  void *d_residual;
  float *parts;  // [gridDim.x][H] or NULL
  int T, chunks;
  int weight_f32;
  float eps, inv_h;
};

// d = r (n - h mean(n h)) + d_total with h = s r: both row sums, of s^2 and of
// n s, come from the one pass that loads the row.  A workgroup takes the rows
// blockIdx, blockIdx + grid, ... and keeps its part of d_weight in registers.
template <int NC, bool F32>
__global__ void __launch_bounds__(kThreads) norm_backward_kernel(NormBackArgs g) {
  __shared__ float red[2][4];
  float dw[NC][8];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[c][j] = 0.0f;
  for (int64_t row = blockIdx.x; row < g.T; row += gridDim.x) {
    const int64_t base = row * g.chunks;
    float v[NC][8], dy[NC][8];
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = threadIdx.x + c * kThreads;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] = dy[c][j] = 0.0f;
      if (i < g.chunks) {
        float w[8];
        load8<F32>(g.total, base + i, v[c]);
        load8<false>(g.dy, base + i, dy[c]);
        weight8(g.weight, g.weight_f32, i, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          sum[0] = fmaf(v[c][j], v[c][j], sum[0]);
          sum[1] = fmaf(dy[c][j] * w[j], v[c][j], sum[1]);
        }
      }
    }
    row_sums<4, 2>(sum, red);
    const float r = rsqrtf(fmaf(sum[0], g.inv_h, g.eps));
    const float m = sum[1] * g.inv_h * r;  // mean(n h)
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = threadIdx.x + c * kThreads;
      if (i >= g.chunks) continue;
      float w[8], d[8];
      weight8(g.weight, g.weight_f32, i, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float h = v[c][j] * r;
        dw[c][j] = fmaf(dy[c][j], h, dw[c][j]);
        d[j] = r * fmaf(-h, m, dy[c][j] * w[j]);
      }
      if (g.d_total) {
        float o[8];
        load8<F32>(g.d_total, base + i, o);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] += o[j];
      }
      if (g.dx) store8<false>(g.dx, base + i, d);
      if (g.d_residual) store8<F32>(g.d_residual, base + i, d);
    }
  }
  if (!g.parts) return;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int i = threadIdx.x + c * kThreads;
    if (i < g.chunks) store8<true>(g.parts, (int64_t)blockIdx.x * g.chunks + i, dw[c]);
  }
}

// Sums n parts of H columns in the order of the parts: 64 columns to a
// workgroup, every 16th part to a wave.
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float *__restrict__ parts, int n,
                                                           int H, float *__restrict__ out) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  float a = 0.0f;
  if (c < H)
    for (int p = wave; p < n; p += 16) a += parts[(int64_t)p * H + c];
  red[wave][lane] = a;
  __syncthreads();
  if (wave || c >= H) return;
  a = 0.0f;
#pragma unroll
  for (int w = 0; w < 16; ++w) a += red[w][lane];
  out[c] = a;
}

// Workgroups of the backward pass, and parts of d_weight.
int backward_groups(int T) { return T < 512 ? T : 512; }

template <bool F32>
void pick_norm_backward(const NormBackArgs &g, hipStream_t s) {
  const int nc = (g.chunks + kThreads - 1) / kThreads;
  launch_k(COLI_K_NORM_BACKWARD,
           nc == 1   ? norm_backward_kernel<1, F32>
           : nc == 2 ? norm_backward_kernel<2, F32>
           : nc == 3 ? norm_backward_kernel<3, F32>
           : nc == 4 ? norm_backward_kernel<4, F32>
                     : norm_backward_kernel<8, F32>,
           dim3(backward_groups(g.T)), dim3(kThreads), 0, s, g);
}

}  // namespace

size_t norm_workspace(int H, int T) {
  return align_up((size_t)backward_groups(T) * H * sizeof(float));
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
  g.chunks = n.hidden / 8;
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
  g.parts = d_weight ? reinterpret_cast<float *>(ws) : nullptr;
  g.T = T;
  g.chunks = n.hidden / 8;
  g.weight_f32 = n.weight_dtype == COLI_SRC_F32;
  g.eps = n.eps;
  g.inv_h = 1.0f / (float)n.hidden;
  if (total_dtype == COLI_SRC_F32)
    pick_norm_backward<true>(g, s);
  else
    pick_norm_backward<false>(g, s);
  if (hipGetLastError() != hipSuccess) return COLI_E_HIP;
  if (!d_weight) return COLI_OK;
  launch_k(COLI_K_NORM_REDUCE, norm_reduce_kernel, dim3((n.hidden + 63) / 64), dim3(1024), 0, s,
           (const float *)ws, backward_groups(T), n.hidden, d_weight);
  return hip_status(hipGetLastError());
}

}  // namespace coli
