// rows.hip -- a batch's rows sorted by expert and back, with the routing
// weights, and the gradients of both.
//
// Pair p = t*k + j owns row pos[p] of a buffer of n_rows rows; a pos outside
// [0, n_rows) is a pair without a row.  Each kernel goes over tokens, so that
// what belongs to a token (x, y, dy) moves once and the k rows of its pairs
// move once each.  Memory bounds all of them: 16,384 tokens x 8 rows of 2048
// dispatched in 104 us (5.8 TB/s), 8,192 x 8 of 6144 combined in 165 us (5.5),
// the gradients of 8,192 x 8 of 2048 in 120 us (4.7; a copy on this card: 5.1).
#include "device_common.h"
#include "internal.h"
#include "lanes.h"
#include "units.h"

namespace coli {
namespace {

constexpr int kThreads = 256;
constexpr int block_of(int lanes) { return lanes > kThreads ? lanes : kThreads; }
constexpr int kBatch = 8;  // rows of a token that are in flight together

struct RowArgs {
  const int32_t *pos;
  const float *w;
  const void *rows;    // rows by expert (input)
  void *out_rows;      // rows by expert (output)
  const void *token;   // what belongs to tokens: x, beside or dy
  void *out_token;     // y or dx
  float *d_w;
  int64_t n_rows;
  int T, k, units;     // units of a row: 16 bytes (dispatch), or 4 or 8 values
  int out_f32;         // type of out_token
};

// Which unit of which token a thread of the kernels without a row sum takes:
// LPR lanes to a token (256: as many workgroups as its units need), several
// tokens of short rows to a workgroup.
template <int LPR>
COLI_DEV bool my_unit(const RowArgs &g, int &t, int &i) {
  if (LPR == kThreads) {  // the token is the same for the whole workgroup
    const int per = (g.units + kThreads - 1) / kThreads;
    t = blockIdx.x / per;
    i = (blockIdx.x - t * per) * kThreads + threadIdx.x;
  } else {
    t = blockIdx.x * (kThreads / LPR) + threadIdx.x / LPR;
    i = threadIdx.x % LPR;
  }
  return t < g.T && i < g.units;
}

// ----------------------------------------------------------------- dispatch

template <int LPR, bool NT>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(RowArgs g) {
  int t, i;
  if (!my_unit<LPR>(g, t, i)) return;
  const uint4 v = reinterpret_cast<const uint4 *>(g.token)[(int64_t)t * g.units + i];
  const int32_t *pos = g.pos + (int64_t)t * g.k;
  for (int j0 = 0; j0 < g.k; j0 += kBatch) {
    int p[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) p[j] = j0 + j < g.k ? pos[j0 + j] : -1;
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (p[j] >= 0 && p[j] < g.n_rows)
        store16<NT>(reinterpret_cast<uint4 *>(g.out_rows) + (int64_t)p[j] * g.units + i, v);
  }
}

// ------------------------------------------------------------------ combine

// Values of a lane's units: fours of fp32 rows, eights of bf16 ones.
constexpr int unit_of(bool f32) { return f32 ? 4 : 8; }

// A batch of a token's rows is requested before the first is used.
template <int LPR, bool F32, bool WEIGHTED, bool NT>
__global__ void __launch_bounds__(kThreads) rows_combine_kernel(RowArgs g) {
  constexpr int U = unit_of(F32);
  int t, i;
  if (!my_unit<LPR>(g, t, i)) return;
  const int64_t own = (int64_t)t * g.units + i;
  float acc[U], f[U];
#pragma unroll
  for (int e = 0; e < U; ++e) acc[e] = 0.0f;
  Unit<U, F32> beside{};
  if (g.token) beside = load_unit<U, F32, false>(g.token, own);
  for (int j0 = 0; j0 < g.k; j0 += kBatch) {
    bool has[kBatch];
    float w[kBatch];
    Unit<U, F32> v[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int64_t p = (int64_t)t * g.k + j0 + j;
      const int r = j0 + j < g.k ? g.pos[p] : -1;
      has[j] = r >= 0 && r < g.n_rows;
      w[j] = WEIGHTED && has[j] ? g.w[p] : 1.0f;
      v[j] = {};
      if (has[j]) v[j] = load_unit<U, F32, NT>(g.rows, (int64_t)r * g.units + i);
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (!has[j]) continue;
      unpack(v[j], f);
#pragma unroll
      for (int e = 0; e < U; ++e) acc[e] = fmaf(w[j], f[e], acc[e]);
    }
  }
  if (g.token) {
    unpack(beside, f);
#pragma unroll
    for (int e = 0; e < U; ++e) acc[e] += f[e];
  }
  if (g.out_f32)
    store_unit<U, true, false>(g.out_token, own, pack<U, true>(acc));
  else
    store_unit<U, false, false>(g.out_token, own, pack<U, false>(acc));
}

// ----------------------------------------------------------------- backward

// LPR lanes hold a token's dy, NU units each, while the rows of its pairs pass,
// a batch of them in flight.  With few tokens their pairs are spread over
// gridDim.y workgroups (one token: 4.0 us instead of 7.8 to 15).  F32: type of
// the rows, DF32 of dy.
template <int LPR, int NU, bool F32, bool DF32>
__global__ void __launch_bounds__(block_of(LPR)) combine_backward_kernel(RowArgs g) {
  constexpr int U = unit_of(F32);
  constexpr int B = block_of(LPR), W = LPR > 64 ? LPR / 64 : 1;
  // Rows of a batch: two, and more waves instead (2,051 x 6 of 2048: 17.4 us,
  // with one row 19.1, with eight 20.4; 65,536 x 2 of 256: 36, 38, 43).
  constexpr int JB = 2;
  __shared__ float red[LPR > 64 ? 32 : 1][W];
  const int li = threadIdx.x % LPR;
  const int t = blockIdx.x * (B / LPR) + threadIdx.x / LPR;
  const int per = (g.k + gridDim.y - 1) / gridDim.y;
  const int first = blockIdx.y * per, last = min(g.k, first + per);
  if (LPR <= 64 && t >= g.T) return;  // whole rows of lanes; no barrier follows
  Unit<U, DF32> dy[NU];
#pragma unroll
  for (int c = 0; c < NU; ++c) {
    const int i = li + c * LPR;
    dy[c] = {};
    if (i < g.units) dy[c] = load_unit<U, DF32, false>(g.token, (int64_t)t * g.units + i);
  }
  const int64_t pair = (int64_t)t * g.k;
  for (int j0 = first; j0 < last; j0 += JB) {
    int row[JB];
    float w[JB], dot[JB];
    Unit<U, F32> v[JB][NU];
#pragma unroll
    for (int j = 0; j < JB; ++j) {
      const int r = j0 + j < last ? g.pos[pair + j0 + j] : -1;
      row[j] = r >= 0 && r < g.n_rows ? r : -1;
      w[j] = row[j] >= 0 ? g.w[pair + j0 + j] : 0.0f;
      dot[j] = 0.0f;
#pragma unroll
      for (int c = 0; c < NU; ++c) {
        const int i = li + c * LPR;
        v[j][c] = {};
        if (g.d_w && row[j] >= 0 && i < g.units)
          v[j][c] = load_unit<U, F32, false>(g.rows, (int64_t)row[j] * g.units + i);
      }
    }
#pragma unroll
    for (int c = 0; c < NU; ++c) {
      const int i = li + c * LPR;
      float f[U];
      unpack(dy[c], f);
#pragma unroll
      for (int j = 0; j < JB; ++j) {
        if (j0 + j >= last) break;
        float e[U];
        unpack(v[j][c], e);
        float d = 0.0f;
#pragma unroll
        for (int x = 0; x < U; ++x) d = fmaf(e[x], f[x], d);
        // a row that is not there, or units past the row, must not meet a dy
        // that is not finite
        if (row[j] >= 0 && i < g.units) {
          dot[j] += d;
          if (g.out_rows) {
#pragma unroll
            for (int x = 0; x < U; ++x) e[x] = w[j] * f[x];
            store_unit<U, F32, false>(g.out_rows, (int64_t)row[j] * g.units + i, pack<U, F32>(e));
          }
        }
      }
    }
    if (!g.d_w) continue;
#pragma unroll
    for (int j = 0; j < JB; ++j) {
      if (j0 + j >= last) break;
      const float s = lanes_sum<(LPR < 64 ? LPR : 64)>(dot[j]);
      if (LPR <= 64) {
        if (li == 0) g.d_w[pair + j0 + j] = s;
      } else if ((threadIdx.x & 63) == 0) {
        red[LPR > 64 ? j0 + j : 0][LPR > 64 ? threadIdx.x >> 6 : 0] = s;
      }
    }
  }
  if (LPR <= 64 || !g.d_w) return;
  __syncthreads();
  const int j = first + (int)threadIdx.x;
  if (j < last) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) s += red[LPR > 64 ? j : 0][w];
    g.d_w[pair + j] = s;
  }
}

// Lanes of a row of n units: the next power of two, up to a workgroup.
int lanes_of(int n) { return n <= 8 ? 8 : n <= 16 ? 16 : n <= 32 ? 32 : n <= 64 ? 64 : kThreads; }

// Workgroups of the kernels that spread units over all tokens.
unsigned unit_groups(int units, int lanes, int T) {
  return lanes == kThreads ? (unsigned)((units + kThreads - 1) / kThreads * T)
                           : (unsigned)((T + kThreads / lanes - 1) / (kThreads / lanes));
}

// NC: chunks of eight values to a lane.
template <int LPR, int NC, bool F32, bool DF32>
void run_backward(const RowArgs &g, hipStream_t s) {
  constexpr int B = block_of(LPR), per = B / LPR, NU = NC * 8 / unit_of(F32);
  const int groups = (g.T + per - 1) / per;
  const int split = groups >= 512 ? 1 : (512 + groups - 1) / groups;
  launch_k(COLI_K_ROWS_BACKWARD, combine_backward_kernel<LPR, NU, F32, DF32>,
           dim3(groups, split < g.k ? split : g.k), dim3(B), 0, s, g);
}

template <bool F32, bool DF32>
void pick_backward(const RowArgs &g, hipStream_t s) {
  const int n = g.units * unit_of(F32) / 8;
  if (n <= 8) return run_backward<8, 1, F32, DF32>(g, s);
  if (n <= 16) return run_backward<16, 1, F32, DF32>(g, s);
  if (n <= 32) return run_backward<32, 1, F32, DF32>(g, s);
  if (n <= 64) return run_backward<64, 1, F32, DF32>(g, s);
  if (n <= 128) return run_backward<64, 2, F32, DF32>(g, s);
  if (n <= 256) return run_backward<256, 1, F32, DF32>(g, s);
  if (n <= 512) return run_backward<256, 2, F32, DF32>(g, s);
  if (n <= 768) return run_backward<256, 3, F32, DF32>(g, s);
  if (n <= 1024) return run_backward<512, 2, F32, DF32>(g, s);
  run_backward<1024, 2, F32, DF32>(g, s);
}

// Bytes of the rows of all pairs.
int64_t row_bytes(const Layer &L, int T, int dtype) {
  return (int64_t)T * L.k * L.H * (dtype == COLI_SRC_F32 ? 4 : 2);
}

template <bool NT>
void pick_dispatch(const RowArgs &g, hipStream_t s) {
  const int lanes = lanes_of(g.units);
  launch_k(COLI_K_DISPATCH,
           lanes == 8    ? dispatch_kernel<8, NT>
           : lanes == 16 ? dispatch_kernel<16, NT>
           : lanes == 32 ? dispatch_kernel<32, NT>
           : lanes == 64 ? dispatch_kernel<64, NT>
                         : dispatch_kernel<kThreads, NT>,
           dim3(unit_groups(g.units, lanes, g.T)), dim3(kThreads), 0, s, g);
}

template <bool F32, bool WEIGHTED, bool NT>
void pick_combine(const RowArgs &g, hipStream_t s) {
  const int lanes = lanes_of(g.units);
  launch_k(COLI_K_ROWS_COMBINE,
           lanes == 8    ? rows_combine_kernel<8, F32, WEIGHTED, NT>
           : lanes == 16 ? rows_combine_kernel<16, F32, WEIGHTED, NT>
           : lanes == 32 ? rows_combine_kernel<32, F32, WEIGHTED, NT>
           : lanes == 64 ? rows_combine_kernel<64, F32, WEIGHTED, NT>
                         : rows_combine_kernel<kThreads, F32, WEIGHTED, NT>,
           dim3(unit_groups(g.units, lanes, g.T)), dim3(kThreads), 0, s, g);
}
template <bool F32, bool WEIGHTED>
void pick_combine(const RowArgs &g, bool nt, hipStream_t s) {
  nt ? pick_combine<F32, WEIGHTED, true>(g, s) : pick_combine<F32, WEIGHTED, false>(g, s);
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
  g.units = L.H * (dtype == COLI_SRC_F32 ? 4 : 2) / 16;
  // Rows of twice the last cache or more are written past it: 16,384 tokens x 8
  // rows of 2048 in 105 us instead of 122, and with a reader behind 403 against
  // 396; at 384 MB the reader loses more (206 against 195 with it).
  if (row_bytes(L, T, dtype) >= int64_t(512) << 20)
    pick_dispatch<true>(g, s);
  else
    pick_dispatch<false>(g, s);
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
  const bool f32 = rows_dtype == COLI_SRC_F32;
  g.units = L.H / unit_of(f32);
  // Rows that fill half of the last cache or more are read past it, as they are
  // read once: 8,192 tokens x 8 rows of 6144 in 170 us instead of 183, after
  // their writer 150 instead of 197 (4,096 tokens); rows of 64 MB and less would
  // be found there (8,192 x 8 of 256: 7.9 us, past it 9.6).
  const bool nt = row_bytes(L, T, rows_dtype) >= int64_t(128) << 20;
  if (w)
    f32 ? pick_combine<true, true>(g, nt, s) : pick_combine<false, true>(g, nt, s);
  else
    f32 ? pick_combine<true, false>(g, nt, s) : pick_combine<false, false>(g, nt, s);
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
  const bool f32 = rows_dtype == COLI_SRC_F32;
  g.units = L.H / unit_of(f32);
  if (dy_dtype == COLI_SRC_F32)
    f32 ? pick_backward<true, true>(g, s) : pick_backward<false, true>(g, s);
  else
    f32 ? pick_backward<true, false>(g, s) : pick_backward<false, false>(g, s);
  return hip_status(hipGetLastError());
}

}  // namespace coli
