// rows.hip -- a batch's rows sorted by expert and back, with the routing
// weights, and the gradients of both.
//
// Pair p = t*k + j owns row pos[p] of a buffer of n_rows rows; a pos outside
// [0, n_rows) is a pair without a row.  Each kernel goes over tokens, so that
// what belongs to a token (x, y, dy) moves once and the k rows of its pairs
// move once each.
#include "device_common.h"
#include "internal.h"
#include "values8.h"

namespace coli {
namespace {

constexpr int kThreads = 256;

struct RowArgs {
  const int32_t *pos;
  const float *w;
  const void *rows;    // rows by expert (input)
  void *out_rows;      // rows by expert (output)
  const void *token;   // what belongs to tokens: x, beside or dy
  void *out_token;     // y or dx
  float *d_w;
  int64_t n_rows;
  int T, k, chunks;    // chunks of a row: 16 bytes (dispatch) or 8 values
  int out_f32;         // type of out_token
};

// Chunks of a row over the threads of a workgroup: blockIdx is a token's
// ordinal times the workgroups of a row, plus one of those.
COLI_DEV bool my_chunk(const RowArgs &g, int &t, int &i) {
  const int per = (g.chunks + kThreads - 1) / kThreads;
  t = blockIdx.x / per;
  i = (blockIdx.x - t * per) * kThreads + threadIdx.x;
  return i < g.chunks;
}

// ----------------------------------------------------------------- dispatch

__global__ void __launch_bounds__(kThreads) dispatch_kernel(RowArgs g) {
  int t, i;
  if (!my_chunk(g, t, i)) return;
  const uint4 v = reinterpret_cast<const uint4 *>(g.token)[(int64_t)t * g.chunks + i];
  for (int j = 0; j < g.k; ++j) {
    const int64_t p = g.pos[(int64_t)t * g.k + j];
    if (p >= 0 && p < g.n_rows) reinterpret_cast<uint4 *>(g.out_rows)[p * g.chunks + i] = v;
  }
}

// ------------------------------------------------------------------ combine

template <bool F32, bool WEIGHTED>
__global__ void __launch_bounds__(kThreads) rows_combine_kernel(RowArgs g) {
  int t, i;
  if (!my_chunk(g, t, i)) return;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < g.k; ++j) {
    const int64_t p = g.pos[(int64_t)t * g.k + j];
    if (p < 0 || p >= g.n_rows) continue;
    const float w = WEIGHTED ? g.w[(int64_t)t * g.k + j] : 1.0f;
    float v[8];
    load8<F32>(g.rows, p * g.chunks + i, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = fmaf(w, v[e], acc[e]);
  }
  if (g.token) {
    float v[8];
    load8<F32>(g.token, (int64_t)t * g.chunks + i, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += v[e];
  }
  if (g.out_f32)
    store8<true>(g.out_token, (int64_t)t * g.chunks + i, acc);
  else
    store8<false>(g.out_token, (int64_t)t * g.chunks + i, acc);
}

// ----------------------------------------------------------------- backward

// One workgroup per token: its dy stays in registers while the rows of its
// pairs pass.  F32: type of the rows, DF32 of dy.
template <bool F32, bool DF32>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(RowArgs g) {
  constexpr int NC = 8;  // 16,384 values
  __shared__ float red[32][kThreads / 64];
  const int t = blockIdx.x;
  float dy[NC][8];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int i = threadIdx.x + c * kThreads;
    if (i < g.chunks) load8<DF32>(g.token, (int64_t)t * g.chunks + i, dy[c]);
  }
  for (int j = 0; j < g.k; ++j) {
    const int64_t p = g.pos[(int64_t)t * g.k + j];
    const bool has = p >= 0 && p < g.n_rows;
    const float w = g.w[(int64_t)t * g.k + j];
    float dot = 0.0f;
    if (has) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int i = threadIdx.x + c * kThreads;
        if (i >= g.chunks) continue;
        if (g.d_w) {
          float v[8];
          load8<F32>(g.rows, p * g.chunks + i, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) dot = fmaf(v[e], dy[c][e], dot);
        }
        if (g.out_rows) {
          float d[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) d[e] = w * dy[c][e];
          store8<F32>(g.out_rows, p * g.chunks + i, d);
        }
      }
    }
    dot = wave_sum(dot);
    if ((threadIdx.x & 63) == 0) red[j][threadIdx.x >> 6] = dot;
  }
  __syncthreads();
  if (g.d_w && (int)threadIdx.x < g.k) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) s += red[threadIdx.x][w];
    g.d_w[(int64_t)t * g.k + threadIdx.x] = s;
  }
}

}  // namespace

int launch_dispatch(const Layer &L, const int32_t *pos, const void *x, int dtype, int T,
                    void *rows, int64_t n_rows, hipStream_t s) {
  RowArgs g{};
  g.pos = pos;
  g.token = x;
  g.out_rows = rows;
  g.n_rows = n_rows;
  g.T = T;
  g.k = L.k;
  g.chunks = L.H * (dtype == COLI_SRC_F32 ? 4 : 2) / 16;
  launch_k(COLI_K_DISPATCH, dispatch_kernel, dim3((g.chunks + kThreads - 1) / kThreads * T),
           dim3(kThreads), 0, s, g);
  return hip_status(hipGetLastError());
}

int launch_rows_combine(const Layer &L, const int32_t *pos, const float *w, const void *rows,
                        int rows_dtype, int64_t n_rows, const void *beside, int T, void *y,
                        int y_dtype, hipStream_t s) {
  RowArgs g{};
  g.pos = pos;
  g.w = w;
  g.rows = rows;
  g.n_rows = n_rows;
  g.token = beside;
  g.out_token = y;
  g.out_f32 = y_dtype == COLI_SRC_F32;
  g.T = T;
  g.k = L.k;
  g.chunks = L.H / 8;
  const bool f32 = rows_dtype == COLI_SRC_F32;
  launch_k(COLI_K_ROWS_COMBINE,
           w ? (f32 ? rows_combine_kernel<true, true> : rows_combine_kernel<false, true>)
             : (f32 ? rows_combine_kernel<true, false> : rows_combine_kernel<false, false>),
           dim3((g.chunks + kThreads - 1) / kThreads * T), dim3(kThreads), 0, s, g);
  return hip_status(hipGetLastError());
}

int launch_combine_backward(const Layer &L, const int32_t *pos, const float *w, const void *rows,
                            int rows_dtype, int64_t n_rows, const void *dy, int dy_dtype, int T,
                            void *d_rows, float *d_w, hipStream_t s) {
  RowArgs g{};
  g.pos = pos;
  g.w = w;
  g.rows = rows;
  g.out_rows = d_rows;
  g.n_rows = n_rows;
  g.token = dy;
  g.d_w = d_w;
  g.T = T;
  g.k = L.k;
  g.chunks = L.H / 8;
  const bool f32 = rows_dtype == COLI_SRC_F32;
  launch_k(COLI_K_ROWS_BACKWARD,
           dy_dtype == COLI_SRC_F32
               ? (f32 ? combine_backward_kernel<true, true> : combine_backward_kernel<false, true>)
               : (f32 ? combine_backward_kernel<true, false>
                      : combine_backward_kernel<false, false>),
           dim3(T), dim3(kThreads), 0, s, g);
  return hip_status(hipGetLastError());
}

}  // namespace coli
