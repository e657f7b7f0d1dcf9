// balance.hip -- the router's balance loss with per-expert counts, and the
// gradient of the route.
//
// Sequence s has n_s counted tokens and c_se choices of expert e.  With
// p_t = softmax(l_t), or for sigmoid routing p_te = sig(l_te) / sum_j sig(l_tj):
//   P_se = mean_t p_te,  f_se = E c_se / (k n_s)
//   balance = mean over non-empty s of sum_e f_se P_se
//   z       = mean over counted t of (log sum_e exp l_te)^2
// and, f a constant,
//   d balance / d l_tj = p_tj D_tj (f_sj - sum_e f_se p_te) / (S n_s),
//     D = 1 (softmax) or 1 - sig(l_tj)
//   d z / d l_tj = 2 lse_t softmax(l_t)_j / N.
//
// Both are bound by memory: one read of the logits (and one write of their
// gradient), so a row stays in registers between its loads and its stores.
// W lanes share a row, each with C chunks of V neighbouring experts (16-byte
// accesses where E and the pointers allow them); small E puts several rows
// into a wavefront.
//
// Sums over tokens take a fixed order (no floating-point atomics): a
// workgroup adds up the rows of a tile; sequences that end inside the tile
// are finished there, the others leave one partial row per tile (at most the
// tile's first and its last sequence), which a second kernel adds up.
#include <float.h>

#include "internal.h"
#include "spans.h"

namespace coli {
namespace {

constexpr int kFwdThreads = 512;
constexpr int kMaxTiles = 512;
constexpr int kMaxFinish = 512;  // workgroups of the second kernel
constexpr int kSoloRows = 64;    // up to here one workgroup does everything
constexpr int kCols = 16;        // experts per item of the second kernel

template <int W>
COLI_DEV float sum_w(float v) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}
template <int W>
COLI_DEV float max_w(float v) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}

template <int V>
COLI_DEV void load_v(const float *p, float *out) {
  if (V == 4) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    out[0] = v.x;
    out[1] = v.y;
    out[2] = v.z;
    out[3] = v.w;
  } else {
    out[0] = p[0];
  }
}
template <int V>
COLI_DEV void store_v(float *p, const float *v) {
  if (V == 4) *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
  else p[0] = v[0];
}

// This lane's share of a row: experts V * (lane + W * c) + v.
template <int W, int C, int V>
COLI_DEV void load_row(const float *__restrict__ row, int E, int gl, float (&l)[C * V]) {
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int e = V * (gl + W * c);
    if (e < E) {
      load_v<V>(row + e, l + V * c);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) l[V * c + v] = -INFINITY;
    }
  }
}

// exp(-|l|), from which both the sigmoid and its complement follow without
// cancellation.
COLI_DEV float sig_part(float l) { return __expf(-fabsf(l)); }
COLI_DEV float sig(float l, float q) { return (l >= 0.0f ? 1.0f : q) / (1.0f + q); }
COLI_DEV float one_minus_sig(float l, float q) { return (l >= 0.0f ? q : 1.0f) / (1.0f + q); }

// Unnormalised probability of an entry with logit l, in a row whose largest
// logit is m: exp(l - m), or the sigmoid -- where all logits are negative
// times exp(-m), so that the row's sum does not underflow.
template <bool SIGMOID>
COLI_DEV float score(float l, float m, float e1) {
  if (!SIGMOID) return e1;
  const float q = sig_part(l);
  return m >= 0.0f ? sig(l, q) : e1 / (1.0f + q);
}

// p (normalised probabilities) and the log-sum-exp of a row.  A row without
// a finite logit has p = 0 and lse = 0.
template <int W, int C, int V, bool SIGMOID>
COLI_DEV void row_probs(const float (&l)[C * V], float (&p)[C * V], float &m, float &sum,
                        float &lse) {
  m = -INFINITY;
#pragma unroll
  for (int i = 0; i < C * V; ++i) m = fmaxf(m, l[i]);
  m = max_w<W>(m);
  const bool any = m > -INFINITY;
  float s = 0.0f, z = 0.0f;
#pragma unroll
  for (int i = 0; i < C * V; ++i) {
    const float e1 = any ? __expf(l[i] - m) : 0.0f;
    s += e1;
    p[i] = any ? score<SIGMOID>(l[i], m, e1) : 0.0f;
    if (SIGMOID) z += p[i];
  }
  sum = sum_w<W>(s);
  if (SIGMOID) z = sum_w<W>(z);
  else z = sum;
  lse = any ? m + __logf(sum) : 0.0f;
  const float inv = any ? 1.0f / z : 0.0f;
#pragma unroll
  for (int i = 0; i < C * V; ++i) p[i] *= inv;
}

// ---------------------------------------------------------------- forward

struct FwdArgs {
  const float *logits;
  const int32_t *idx;
  const int32_t *off;
  const uint8_t *valid;
  int T, E, k, n_seq, tile;  // rows per tile
  int n_tiles;
  int32_t *counts;
  float *mean_prob;
  int32_t *tokens;
  int32_t *totals;
  float *loss;
  // workspace
  float *part_p;      // [2 * n_tiles][E] sums of p of a tile's first / last sequence
  int32_t *part_c;    // [2 * n_tiles][E] choices
  int32_t *part_n;    // [2 * n_tiles] counted tokens
  double *tile_z;     // [n_tiles] sums of lse^2
  int32_t *tile_n;    // [n_tiles] counted tokens of the tile
  double *fin_term;   // [kMaxFinish]
  int32_t *fin_live;  // [kMaxFinish] non-empty sequences
  uint32_t *ticket;
};

// Row range of sequence s, clipped to the batch.
COLI_DEV int seq_begin(const FwdArgs &g, int s) { return g.off ? min(max(g.off[s], 0), g.T) : 0; }
COLI_DEV int seq_end(const FwdArgs &g, int s) {
  return g.off ? min(max(g.off[s + 1], 0), g.T) : g.T;
}

struct FinShared {
  float p[kFwdThreads];
  int c[kFwdThreads];
  double d[kFwdThreads];
  int n[kFwdThreads];
  int last;
};

template <typename X>
COLI_DEV X block_sum(X v, X *buf) {
  buf[threadIdx.x] = v;
  __syncthreads();
  for (int o = kFwdThreads / 2; o > 0; o >>= 1) {
    if ((int)threadIdx.x < o) buf[threadIdx.x] += buf[threadIdx.x + o];
    __syncthreads();
  }
  const X r = buf[0];
  __syncthreads();
  return r;
}

// Finishes the sequences (items of kCols experts of one sequence): adds the
// tiles' partial rows of those that several tiles share, writes zeros for
// empty ones, and sums c * P; the last workgroup adds up the losses.
__device__ void finish_sequences(const FwdArgs &g, FinShared &sh, int block, int n_blocks,
                                 bool solo) {
  const int tid = threadIdx.x;
  const int chunks = (g.E + kCols - 1) / kCols;
  const int64_t items = (int64_t)g.n_seq * chunks;
  constexpr int kRows = kFwdThreads / kCols;
  const int col = tid % kCols, rg = tid / kCols;
  double term = 0.0;
  int live = 0;
  for (int64_t it = block; it < items; it += n_blocks) {
    const int s = (int)(it / chunks), e = (int)(it % chunks) * kCols + col;
    const int b = seq_begin(g, s), t = seq_end(g, s);
    const bool empty = b >= t;
    const int tile0 = b / g.tile, tile1 = empty ? tile0 : (t - 1) / g.tile;
    float p = 0.0f;
    int c = 0, n = 0;
    if (!empty && tile0 != tile1) {
      // rows of partials: tile0 (its last sequence, or its first if the
      // sequence starts with the tile), then the first of every later tile
      for (int i = tile0 + rg; i <= tile1; i += kRows) {
        const int64_t row = 2 * (int64_t)i + (i == tile0 && b != tile0 * g.tile ? 1 : 0);
        if (e < g.E) {
          p += g.part_p[row * g.E + e];
          c += g.part_c[row * g.E + e];
        }
        n += g.part_n[row];
      }
      sh.p[tid] = p;
      sh.c[tid] = c;
      sh.n[tid] = n;
      __syncthreads();
      if (rg == 0) {
        p = 0.0f;
        c = n = 0;
        for (int r = 0; r < kRows; ++r) {
          p += sh.p[r * kCols + col];
          c += sh.c[r * kCols + col];
          n += sh.n[r * kCols + col];
        }
        p = n ? p / (float)n : 0.0f;
      }
      __syncthreads();
    } else if (!empty && rg == 0) {
      n = g.tokens[s];
      if (e < g.E) {
        p = g.mean_prob[(int64_t)s * g.E + e];
        c = g.counts[(int64_t)s * g.E + e];
      }
    }
    if (rg == 0) {
      if (e < g.E && (empty || tile0 != tile1)) {
        g.mean_prob[(int64_t)s * g.E + e] = p;
        g.counts[(int64_t)s * g.E + e] = c;
      }
      if (e == 0 && (empty || tile0 != tile1)) g.tokens[s] = n;
      if (e < g.E && n) term += (double)p * (double)c / (double)n;
      if (e == 0 && n) ++live;
    }
  }
  term = block_sum(term, sh.d);
  live = block_sum(live, sh.n);
  if (!solo) {
    // the partial sums pass between workgroups of different L2s: device
    // scope on both sides of the ticket
    if (tid == 0) {
      __hip_atomic_store(&g.fin_term[block], term, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __hip_atomic_store(&g.fin_live[block], live, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __threadfence();
      sh.last = atomicAdd(g.ticket, 1u) == (uint32_t)n_blocks - 1u;
    }
    __syncthreads();
    if (!sh.last) return;
    __threadfence();
    term = 0.0;
    live = 0;
    for (int i = tid; i < n_blocks; i += kFwdThreads) {
      term += __hip_atomic_load(&g.fin_term[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      live += __hip_atomic_load(&g.fin_live[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    term = block_sum(term, sh.d);
    live = block_sum(live, sh.n);
  }
  double z = 0.0;
  int n = 0;
  for (int i = tid; i < g.n_tiles; i += kFwdThreads) {
    z += g.tile_z[i];
    n += g.tile_n[i];
  }
  z = block_sum(z, sh.d);
  n = block_sum(n, sh.n);
  if (tid == 0) {
    g.loss[0] = live ? (float)(term * g.E / g.k / live) : 0.0f;
    g.loss[1] = n ? (float)(z / n) : 0.0f;
    g.totals[0] = n;
    g.totals[1] = live;
  }
}

template <int W, int C, int V, bool SIGMOID, bool SOLO>
__global__ void __launch_bounds__(kFwdThreads) balance_kernel(FwdArgs g) {
  constexpr int G = kFwdThreads / W;  // rows in flight
  constexpr int S = W * C * V;        // experts, padded
  __shared__ float red[G * S];
  __shared__ int hist[S];
  __shared__ int counted;
  __shared__ FinShared fin;
  const int tid = threadIdx.x, gl = tid % W, grp = tid / W;
  const int E = g.E;
  const int row0 = blockIdx.x * g.tile, row1 = min(g.T, row0 + g.tile);
  if (blockIdx.x == 0 && tid == 0) *g.ticket = 0u;  // for the kernel after this one
  double zsum = 0.0;
  int ntile = 0;
  for (int pos = row0; pos < row1;) {
    // the piece [pos, end) of sequence s, or rows of no sequence (s < 0)
    int s = 0, begin = 0, end = g.T;
    if (g.off) {
      s = last_at_or_before(g.off, g.n_seq + 1, pos);
      begin = s >= 0 ? max(g.off[s], 0) : 0;
      end = s < g.n_seq ? min(g.off[s + 1], g.T) : g.T;
      if (s == g.n_seq) s = -1;
    }
    const bool whole = begin >= row0 && end <= row1;
    end = min(max(end, pos + 1), row1);
    if (s >= 0) {
      float acc[C * V];
#pragma unroll
      for (int i = 0; i < C * V; ++i) acc[i] = 0.0f;
      for (int i = tid; i < S; i += kFwdThreads) hist[i] = 0;
      if (tid == 0) counted = 0;
      __syncthreads();
      int mine = 0;
      for (int t = pos + grp; t < end; t += G) {
        if (g.valid && !g.valid[t]) continue;
        float l[C * V], p[C * V], m, sum, lse;
        load_row<W, C, V>(g.logits + (int64_t)t * E, E, gl, l);
        row_probs<W, C, V, SIGMOID>(l, p, m, sum, lse);
#pragma unroll
        for (int i = 0; i < C * V; ++i) acc[i] += p[i];
        for (int j = gl; j < g.k; j += W) {
          const int e = g.idx[(int64_t)t * g.k + j];
          if (e >= 0 && e < E) atomicAdd(&hist[e], 1);
        }
        if (gl == 0) {
          zsum += (double)lse * (double)lse;
          ++mine;
        }
      }
      if (gl == 0 && mine) atomicAdd(&counted, mine);
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int v = 0; v < V; ++v) red[grp * S + V * (gl + W * c) + v] = acc[V * c + v];
      __syncthreads();
      const int n = counted;
      ntile += n;
      const int64_t row = 2 * (int64_t)blockIdx.x + (pos == row0 ? 0 : 1);
      for (int e = tid; e < E; e += kFwdThreads) {
        float p = 0.0f;
#pragma unroll 8
        for (int r = 0; r < G; ++r) p += red[r * S + e];
        if (whole) {
          g.mean_prob[(int64_t)s * E + e] = n ? p / (float)n : 0.0f;
          g.counts[(int64_t)s * E + e] = hist[e];
        } else {
          g.part_p[row * E + e] = p;
          g.part_c[row * E + e] = hist[e];
        }
      }
      if (tid == 0) {
        if (whole) g.tokens[s] = n;
        else g.part_n[row] = n;
      }
      __syncthreads();
    }
    pos = end;
  }
  zsum = block_sum(zsum, fin.d);
  if (tid == 0) {
    g.tile_z[blockIdx.x] = zsum;
    g.tile_n[blockIdx.x] = ntile;
  }
  if (SOLO) {
    __syncthreads();
    finish_sequences(g, fin, 0, 1, true);
  }
}

__global__ void __launch_bounds__(kFwdThreads) balance_finish_kernel(FwdArgs g) {
  __shared__ FinShared fin;
  finish_sequences(g, fin, blockIdx.x, gridDim.x, false);
}

// ---------------------------------------------------------------- backward

struct BwdArgs {
  const float *logits;
  const int32_t *idx;
  const float *d_w;      // gradient of the routing weights, or NULL
  float routed_scale;
  int T, E, k;
  // the balance part (counts NULL: none)
  const int32_t *off;
  const uint8_t *valid;
  int n_seq;
  const int32_t *counts;
  const int32_t *tokens;
  const int32_t *totals;
  const float *d_loss;
  float *d_logits;
  int rows;  // per wavefront
};

constexpr int kBwdThreads = 256;

// Gradients of the routing weights with respect to the chosen logits, added
// into the row's LDS entries; returns sum_j g_j w_j of the plain softmax.
template <int W, bool SIGMOID, bool RENORM>
COLI_DEV float route_part(const BwdArgs &g, int64_t t, int gl, float m, float inv, float *row) {
  const float *lrow = g.logits + t * g.E;
  const int32_t *idx = g.idx + t * g.k;
  const float *dw = g.d_w + t * g.k;
  const float c = g.routed_scale;
  float out = 0.0f;
  if (!RENORM) {
    for (int j = gl; j < g.k; j += W) {
      const int e = idx[j];
      if (e < 0 || e >= g.E) continue;
      const float l = lrow[e];
      float d;
      if (SIGMOID) {
        const float q = sig_part(l);
        d = c * dw[j] * sig(l, q) * one_minus_sig(l, q);
      } else {
        d = c * dw[j] * __expf(l - m) * inv;
        out += d;
      }
      atomicAdd(&row[e], d);
    }
    return SIGMOID ? 0.0f : sum_w<W>(out);
  }
  float ms = -INFINITY;
  for (int j = gl; j < g.k; j += W) {
    const int e = idx[j];
    if (e >= 0 && e < g.E) ms = fmaxf(ms, lrow[e]);
  }
  ms = max_w<W>(ms);
  if (!(ms > -INFINITY)) return 0.0f;
  float z = 0.0f, gw = 0.0f;
  for (int j = gl; j < g.k; j += W) {
    const int e = idx[j];
    if (e < 0 || e >= g.E) continue;
    const float w = score<SIGMOID>(lrow[e], ms, __expf(lrow[e] - ms));
    z += w;
    gw += w * dw[j];
  }
  z = 1.0f / sum_w<W>(z);
  gw = sum_w<W>(gw) * z;
  for (int j = gl; j < g.k; j += W) {
    const int e = idx[j];
    if (e < 0 || e >= g.E) continue;
    const float l = lrow[e];
    float d = c * score<SIGMOID>(l, ms, __expf(l - ms)) * z * (dw[j] - gw);
    if (SIGMOID) d *= one_minus_sig(l, sig_part(l));
    atomicAdd(&row[e], d);
  }
  return 0.0f;
}

template <int W, int C, int V, bool SIGMOID, bool RENORM>
__global__ void __launch_bounds__(kBwdThreads) route_backward_kernel(BwdArgs g) {
  constexpr int G = 64 / W;     // rows of a wavefront in flight
  constexpr int S = W * C * V;
  __shared__ float rows[kBwdThreads / W][S];
  const int lane = threadIdx.x & 63, gl = lane % W, grp = lane / W;
  const int wave = __builtin_amdgcn_readfirstlane(blockIdx.x * (kBwdThreads / 64) + (threadIdx.x >> 6));
  const int E = g.E;
  float *row = rows[threadIdx.x / W];
  const bool balance = g.counts != nullptr;
  // rows are cleared once here and again by whoever read them
  for (int i = gl; i < S; i += W) row[i] = 0.0f;
  const int64_t first = (int64_t)wave * g.rows;
  if (first >= g.T) return;
  const int row0 = (int)first, row1 = min(g.T, row0 + g.rows);
  float zc = 0.0f, bc = 0.0f;
  if (balance) {
    bc = g.d_loss[0] / (float)max(1, g.totals[1]) * (float)E / (float)g.k;
    zc = 2.0f * g.d_loss[1] / (float)max(1, g.totals[0]);
  }
  for (int pos = row0; pos < row1;) {
    int s = 0, end = g.T;
    float f[C * V];
#pragma unroll
    for (int i = 0; i < C * V; ++i) f[i] = 0.0f;
    if (balance) {
      if (g.off) {
        s = last_at_or_before(g.off, g.n_seq + 1, pos);
        end = s < g.n_seq ? g.off[s + 1] : g.T;
        if (s == g.n_seq) s = -1;
      }
      if (s >= 0) {
        const float n = (float)max(1, g.tokens[s]);
        const float fc = bc / n / n;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const int e = V * (gl + W * c) + v;
            if (e < E) f[V * c + v] = fc * (float)g.counts[(int64_t)s * E + e];
          }
      }
    }
    end = min(max(end, pos + 1), row1);
    for (int t = pos + grp; t < end; t += G) {
      const bool live = !balance || (s >= 0 && !(g.valid && !g.valid[t]));
      float d[C * V];
#pragma unroll
      for (int i = 0; i < C * V; ++i) d[i] = 0.0f;
      if (live) {
        const bool full = balance || (!SIGMOID && !RENORM);
        float p[C * V], m = 0.0f, inv = 0.0f;
        if (full) {
          float l[C * V], sum, lse;
          load_row<W, C, V>(g.logits + (int64_t)t * E, E, gl, l);
          row_probs<W, C, V, SIGMOID>(l, p, m, sum, lse);
          inv = sum > 0.0f ? 1.0f / sum : 0.0f;
          if (balance) {
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < C * V; ++i) dot += f[i] * p[i];
            dot = sum_w<W>(dot);
            const float zr = zc * lse * inv;
#pragma unroll
            for (int i = 0; i < C * V; ++i) {
              float b = p[i] * (f[i] - dot);
              if (SIGMOID) b *= one_minus_sig(l[i], sig_part(l[i]));
              d[i] = b + (sum > 0.0f ? zr * __expf(l[i] - m) : 0.0f);
            }
          }
        }
        if (g.d_w) {
          const float gw = route_part<W, SIGMOID, RENORM>(g, t, gl, m, inv, row);
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const int e = V * (gl + W * c);
#pragma unroll
            for (int v = 0; v < V; ++v) {
              d[V * c + v] += row[e + v];
              if (!SIGMOID && !RENORM) d[V * c + v] -= p[V * c + v] * gw;
              row[e + v] = 0.0f;
            }
          }
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int e = V * (gl + W * c);
        if (e < E) store_v<V>(g.d_logits + (int64_t)t * E + e, d + V * c);
      }
    }
    pos = end;
  }
}

// ---------------------------------------------------------------- launch

template <int W, int C, int V, bool SIGMOID>
int launch_fwd(FwdArgs g, hipStream_t s) {
  constexpr int G = kFwdThreads / W;
  if (g.T <= kSoloRows) {
    g.tile = kSoloRows;
    g.n_tiles = 1;
    launch_k(COLI_K_BALANCE, balance_kernel<W, C, V, SIGMOID, true>, dim3(1), dim3(kFwdThreads), 0,
             s, g);
    return hip_status(hipGetLastError());
  }
  g.tile = G * ((g.T + kMaxTiles * G - 1) / (kMaxTiles * G));
  g.n_tiles = (g.T + g.tile - 1) / g.tile;
  launch_k(COLI_K_BALANCE, balance_kernel<W, C, V, SIGMOID, false>, dim3(g.n_tiles),
           dim3(kFwdThreads), 0, s, g);
  const int64_t items = (int64_t)g.n_seq * ((g.E + kCols - 1) / kCols);
  launch_k(COLI_K_BALANCE_FINISH, balance_finish_kernel,
           dim3((unsigned)(items < kMaxFinish ? items : kMaxFinish)), dim3(kFwdThreads), 0, s, g);
  return hip_status(hipGetLastError());
}

template <int W, int C, int V, bool SIGMOID, bool RENORM>
int launch_bwd(BwdArgs g, hipStream_t s) {
  constexpr int G = 64 / W;
  // up to 8,192 wavefronts
  g.rows = G * ((g.T + 8192 * G - 1) / (8192 * G));
  const int waves = (g.T + g.rows - 1) / g.rows;
  launch_k(COLI_K_ROUTE_BACKWARD, route_backward_kernel<W, C, V, SIGMOID, RENORM>,
           dim3((waves + 3) / 4), dim3(kBwdThreads), 0, s, g);
  return hip_status(hipGetLastError());
}

// Calls f(W, C, V as integral constants) for the row layout of E experts:
// 16-byte accesses when every row starts on 16 bytes, as few lanes per row
// as hold it.
template <int N>
struct Int {
  static constexpr int value = N;
};
template <class F>
int with_layout(int E, bool vec, F f) {
  if (vec) {
    if (E <= 16) return f(Int<4>{}, Int<1>{}, Int<4>{});
    if (E <= 32) return f(Int<8>{}, Int<1>{}, Int<4>{});
    if (E <= 64) return f(Int<16>{}, Int<1>{}, Int<4>{});
    if (E <= 128) return f(Int<32>{}, Int<1>{}, Int<4>{});
    if (E <= 256) return f(Int<64>{}, Int<1>{}, Int<4>{});
    if (E <= 512) return f(Int<64>{}, Int<2>{}, Int<4>{});
    return f(Int<64>{}, Int<4>{}, Int<4>{});
  }
  if (E <= 16) return f(Int<16>{}, Int<1>{}, Int<1>{});
  if (E <= 64) return f(Int<64>{}, Int<1>{}, Int<1>{});
  if (E <= 256) return f(Int<64>{}, Int<4>{}, Int<1>{});
  return f(Int<64>{}, Int<16>{}, Int<1>{});
}

}  // namespace

size_t balance_workspace(const Layer &L, int T) {
  (void)T;
  const size_t rows = 2 * (size_t)kMaxTiles;
  return 2 * align_up(rows * L.E * 4) + align_up(rows * 4) + align_up((size_t)kMaxTiles * 8) +
         align_up((size_t)kMaxTiles * 4) + align_up((size_t)kMaxFinish * 8) +
         align_up((size_t)kMaxFinish * 4) + 256;
}

int launch_balance(const Layer &L, const float *logits, const int32_t *idx, int T,
                   const coli_moe_balance_t &b, void *ws, hipStream_t s) {
  char *p = static_cast<char *>(ws);
  auto take = [&](size_t n) {
    char *r = p;
    p += align_up(n);
    return r;
  };
  const size_t rows = 2 * (size_t)kMaxTiles;
  FwdArgs g = {};
  g.logits = logits;
  g.idx = idx;
  g.off = b.seq_offsets;
  g.valid = b.valid;
  g.T = T;
  g.E = L.E;
  g.k = L.k;
  g.n_seq = b.n_seq;
  g.counts = b.counts;
  g.mean_prob = b.mean_prob;
  g.tokens = b.tokens;
  g.totals = b.totals;
  g.loss = b.loss;
  g.part_p = reinterpret_cast<float *>(take(rows * L.E * 4));
  g.part_c = reinterpret_cast<int32_t *>(take(rows * L.E * 4));
  g.part_n = reinterpret_cast<int32_t *>(take(rows * 4));
  g.tile_z = reinterpret_cast<double *>(take((size_t)kMaxTiles * 8));
  g.tile_n = reinterpret_cast<int32_t *>(take((size_t)kMaxTiles * 4));
  g.fin_term = reinterpret_cast<double *>(take((size_t)kMaxFinish * 8));
  g.fin_live = reinterpret_cast<int32_t *>(take((size_t)kMaxFinish * 4));
  g.ticket = reinterpret_cast<uint32_t *>(take(256));
  const bool vec = L.E % 4 == 0 && reinterpret_cast<uintptr_t>(logits) % 16 == 0;
  return with_layout(L.E, vec, [&](auto w, auto c, auto v) {
    constexpr int W = decltype(w)::value, C = decltype(c)::value, V = decltype(v)::value;
    return (L.flags & COLI_ROUTE_SIGMOID) ? launch_fwd<W, C, V, true>(g, s)
                                          : launch_fwd<W, C, V, false>(g, s);
  });
}

int launch_route_backward(const Layer &L, const float *logits, const int32_t *idx, int T,
                          const float *d_w, const coli_moe_balance_t *b, const float *d_loss,
                          float *d_logits, hipStream_t s) {
  BwdArgs g = {};
  g.logits = logits;
  g.idx = idx;
  g.d_w = d_w;
  g.routed_scale = L.routed_scale;
  g.T = T;
  g.E = L.E;
  g.k = L.k;
  if (b) {
    g.off = b->seq_offsets;
    g.valid = b->valid;
    g.n_seq = b->n_seq;
    g.counts = b->counts;
    g.tokens = b->tokens;
    g.totals = b->totals;
    g.d_loss = d_loss;
  }
  g.d_logits = d_logits;
  const bool vec = L.E % 4 == 0 && reinterpret_cast<uintptr_t>(logits) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(d_logits) % 16 == 0;
  return with_layout(L.E, vec, [&](auto w, auto c, auto v) {
    constexpr int W = decltype(w)::value, C = decltype(c)::value, V = decltype(v)::value;
    const bool renorm = (L.flags & COLI_ROUTE_RENORM) != 0;
    if (L.flags & COLI_ROUTE_SIGMOID)
      return renorm ? launch_bwd<W, C, V, true, true>(g, s) : launch_bwd<W, C, V, true, false>(g, s);
    return renorm ? launch_bwd<W, C, V, false, true>(g, s) : launch_bwd<W, C, V, false, false>(g, s);
  });
}

}  // namespace coli
