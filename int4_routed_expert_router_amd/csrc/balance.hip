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
// into a wavefront.  65,536 x 256 logits (67 MB): the loss 26 us (19 us for the
// rows, 3.5 TB/s, and the second launch), the gradient of a sigmoid layer with
// renormalised weights 38 us, 3.6 TB/s over read and write; its vector ALUs
// issue in 68 % of the cycles (272 instructions per row).  Rows whose largest
// logit is beyond kOneExp, with a second exponential, take 40 to 41.5 us.
// Smaller batches are bound by latency: 5 to 7 us per launch.
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
constexpr int kCols = 16;        // experts per item of the second kernel
// One workgroup does everything for few rows and few items (sequences times
// kCols experts), which it takes one after another, 0.6 us each.  us by one
// launch / two, 40 rows (4 and 64 rows alike):
//   1 item  6.8 / 9.3   4: 7.5 / 10.0   8: 11.1 / 11.4   16: 15.3 / 10.1
//   64 items 44 / 13   1,024: 579 / 26   4,800: 2,519 / 30
constexpr int kSoloRows = 64, kSoloItems = 8;

// Reductions over aligned groups of W lanes, the result in every lane: DPP
// moves within 16 lanes (neighbours, pairs, mirrored halves, mirrored row),
// then the row and half swaps, no LDS round trips.
template <int CTRL>
COLI_DEV float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int W, class Op>
COLI_DEV float reduce_w(float v, Op op) {
  if (W >= 2) v = op(v, dpp<0xB1>(v));    // quad_perm 1,0,3,2
  if (W >= 4) v = op(v, dpp<0x4E>(v));    // quad_perm 2,3,0,1
  if (W >= 8) v = op(v, dpp<0x141>(v));   // row_half_mirror
  if (W >= 16) v = op(v, dpp<0x140>(v));  // row_mirror
  if (W >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  if (W >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  return v;
}
template <int W>
COLI_DEV float sum_w(float v) {
  return reduce_w<W>(v, [](float a, float b) { return a + b; });
}
template <int W>
COLI_DEV float max_w(float v) {
  return reduce_w<W>(v, [](float a, float b) { return fmaxf(a, b); });
}
COLI_DEV float rcp(float v) { return __builtin_amdgcn_rcpf(v); }  // 1 ulp

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

// Sigmoid and its complement without cancellation, from one exponential.
struct Sig {
  float s, c;  // sig(l), 1 - sig(l)
  float r;     // 1 / (1 + exp(-|l|)), which is sig(l) exp(-l) where l < 0
};
COLI_DEV Sig sigmoid(float l) {
  const float q = __expf(-fabsf(l));
  const float r = rcp(1.0f + q);
  return {l >= 0.0f ? r : q * r, l >= 0.0f ? q * r : r, r};
}

// Unnormalised probability of an entry with logit l, in a row whose largest
// logit is m: e1 = exp(l - m), or the sigmoid -- where all logits are
// negative times exp(-m), so that the row's sum does not underflow.
template <bool SIGMOID>
COLI_DEV float score(const Sig &g, float m, float e1) {
  return !SIGMOID ? e1 : (m >= 0.0f ? g.s : e1 * g.r);
}

// Rows whose largest logit is within this of zero take one exponential per
// expert for sigmoid and softmax, others two.
constexpr float kOneExp = 20.0f;

// A row's probabilities p, exponentials e1 = exp(l - m), sigmoid complements
// and log-sum-exp.  A row without a finite logit has p = e1 = 0 and lse = 0.
template <int N>
struct Row {
  float p[N], e1[N], c[N];
  float m, inv, lse;  // inv: 1 / sum of e1
};
// `f` given: also *dot = sum_e f_e p_e.
template <int W, int N, bool SIGMOID>
COLI_DEV void row_probs(const float (&l)[N], Row<N> &o, const float *f = nullptr,
                        float *dot = nullptr) {
  float m = l[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = fmaxf(m, l[i]);
  m = max_w<W>(m);
  const bool any = m > -INFINITY;
  float s = 0.0f, z = 0.0f;
  if (SIGMOID && fabsf(m) <= kOneExp) {
    // one exponential for both, as 1 / (1 + e^l) and e^l / (1 + e^l) are exact
    // to a few steps.  The hardware exponential gives 0 below 2^-126, for l <
    // -87.3: at a largest logit of -kOneExp or more that is less than e^-67
    // of it (nearer to -87 it would be seen: 255 experts 8.5 below a largest
    // one of -79.5 are 5 % of their row).  e^l e^-m is off by (|l| + |m|)
    // 2^-24, up to 2 kOneExp more than e^(l - m).
    const float em = __expf(-m);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float t = __expf(l[i]);
      o.c[i] = rcp(1.0f + t);
      o.p[i] = t * o.c[i];
      o.e1[i] = t * em;
      s += o.e1[i];
      z += o.p[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      o.e1[i] = any ? __expf(l[i] - m) : 0.0f;
      s += o.e1[i];
      Sig g = {};
      if (SIGMOID) g = sigmoid(l[i]);
      o.c[i] = g.c;
      o.p[i] = any ? score<SIGMOID>(g, m, o.e1[i]) : 0.0f;
      if (SIGMOID) z += o.p[i];
    }
  }
  float fp = 0.0f;
  if (f) {
#pragma unroll
    for (int i = 0; i < N; ++i) fp += f[i] * o.p[i];
    fp = sum_w<W>(fp);
  }
  s = sum_w<W>(s);
  z = SIGMOID ? sum_w<W>(z) : s;
  o.m = m;
  o.inv = any ? rcp(s) : 0.0f;
  o.lse = any ? m + __logf(s) : 0.0f;
  const float inv = any ? rcp(z) : 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) o.p[i] *= inv;
  if (f) *dot = fp * inv;
}

// Choices of a row that a lane holds: k <= min(E, 32).
constexpr int lane_choices(int W) { return W >= 32 ? 1 : (W == 16 ? 2 : 4); }

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
  int n[kFwdThreads];
  double d[kFwdThreads / 64];
  int i[kFwdThreads / 64];
  int last;
};

// Sums over the workgroup, the same in every thread.
COLI_DEV void block_sums(double &v, int &n, FinShared &sh) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    v += __shfl_xor(v, o, 64);
    n += __shfl_xor(n, o, 64);
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 0) {
    sh.d[threadIdx.x >> 6] = v;
    sh.i[threadIdx.x >> 6] = n;
  }
  __syncthreads();
  v = 0.0;
  n = 0;
#pragma unroll
  for (int w = 0; w < kFwdThreads / 64; ++w) {
    v += sh.d[w];
    n += sh.i[w];
  }
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
#pragma unroll 4
      for (int i = tile0 + rg; i <= tile1; i += kRows) {
        const int64_t row = 2 * (int64_t)i + (i == tile0 && b != tile0 * g.tile ? 1 : 0);
        p += g.part_p[row * g.E + min(e, g.E - 1)];
        c += g.part_c[row * g.E + min(e, g.E - 1)];
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
  block_sums(term, live, sh);
  if (!solo) {
    // The partial sums pass between workgroups of different L2s: device-scope
    // stores and loads, which go past the L2s, and between store and ticket a
    // wait until the stores are done.  (A fence would also write back what
    // else is in the L2s, which nobody here reads.)
    if (tid == 0) {
      __hip_atomic_store(&g.fin_term[block], term, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __hip_atomic_store(&g.fin_live[block], live, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      sh.last = __hip_atomic_fetch_add(g.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                (uint32_t)n_blocks - 1u;
    }
    __syncthreads();
    if (!sh.last) return;
    term = 0.0;
    live = 0;
    for (int i = tid; i < n_blocks; i += kFwdThreads) {
      term += __hip_atomic_load(&g.fin_term[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      live += __hip_atomic_load(&g.fin_live[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    block_sums(term, live, sh);
  }
  double z = 0.0;
  int n = 0;
  for (int i = tid; i < g.n_tiles; i += kFwdThreads) {
    z += g.tile_z[i];
    n += g.tile_n[i];
  }
  block_sums(z, n, sh);
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
      // the next row's inputs are on their way while this one is summed
      constexpr int KL = lane_choices(W);
      struct In {
        float l[C * V];
        int e[KL];
        int valid;
      };
      auto fetch = [&](int t, In &o) {
        t = min(t, end - 1);
        load_row<W, C, V>(g.logits + (int64_t)t * E, E, gl, o.l);
#pragma unroll
        for (int i = 0; i < KL; ++i)
          o.e[i] = gl + W * i < g.k ? g.idx[(int64_t)t * g.k + gl + W * i] : -1;
        o.valid = g.valid ? g.valid[t] : 1;
      };
      In cur, next;
      fetch(pos + grp, cur);
      for (int t = pos + grp; t < end; t += G) {
        fetch(t + G, next);
        if (cur.valid) {
#pragma unroll
          for (int i = 0; i < KL; ++i)
            if (cur.e[i] >= 0 && cur.e[i] < E) atomicAdd(&hist[cur.e[i]], 1);
          Row<C * V> r;
          row_probs<W, C * V, SIGMOID>(cur.l, r);
#pragma unroll
          for (int i = 0; i < C * V; ++i) acc[i] += r.p[i];
          if (gl == 0) {
            zsum += (double)r.lse * (double)r.lse;
            ++mine;
          }
        }
        cur = next;
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
  int unused = 0;
  block_sums(zsum, unused, fin);
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

// A row's choices, KL to a lane: expert (-1: none) and gradient of its weight.
template <int KL>
struct Chosen {
  int e[KL];
  float d[KL];
};
template <int W, int KL>
COLI_DEV void load_chosen(const BwdArgs &g, int64_t t, int gl, Chosen<KL> &o) {
#pragma unroll
  for (int i = 0; i < KL; ++i) {
    const int j = gl + W * i;
    o.e[i] = -1;
    o.d[i] = 0.0f;
    if (j < g.k) {
      const int e = g.idx[t * g.k + j];
      o.e[i] = e >= 0 && e < g.E ? e : -1;
      o.d[i] = g.d_w[t * g.k + j];
    }
  }
}

// Adds the gradients of the routing weights with respect to the chosen
// logits l into the row's LDS entries (an LDS add, so that an expert named
// twice gets both); returns sum_j g_j w_j of the plain softmax, whose
// p_j-weighted part every entry of the row loses.
template <int W, int KL, bool SIGMOID, bool RENORM>
COLI_DEV float route_part(const Chosen<KL> &ch, const float (&l)[KL], float c, float m, float inv,
                          float *row) {
  float out = 0.0f;
  if (!RENORM) {
#pragma unroll
    for (int i = 0; i < KL; ++i) {
      if (ch.e[i] < 0) continue;
      float d = c * ch.d[i];
      if (SIGMOID) {
        const Sig s = sigmoid(l[i]);
        d *= s.s * s.c;
      } else {
        // a row of -inf alone has no probabilities, and -inf - -inf no value
        d = m > -INFINITY ? d * (__expf(l[i] - m) * inv) : 0.0f;
        out += d;
      }
      atomicAdd(&row[ch.e[i]], d);
    }
    return SIGMOID ? 0.0f : sum_w<W>(out);
  }
  float ms = -INFINITY;
#pragma unroll
  for (int i = 0; i < KL; ++i)
    if (ch.e[i] >= 0) ms = fmaxf(ms, l[i]);
  ms = max_w<W>(ms);
  const bool any = ms > -INFINITY;
  float w[KL], comp[KL], z = 0.0f, gw = 0.0f;
#pragma unroll
  for (int i = 0; i < KL; ++i) {
    w[i] = comp[i] = 0.0f;
    if (ch.e[i] < 0 || !any) continue;
    Sig s = {};
    if (SIGMOID) s = sigmoid(l[i]);
    comp[i] = SIGMOID ? s.c : 1.0f;
    w[i] = score<SIGMOID>(s, ms, __expf(l[i] - ms));
    z += w[i];
    gw += w[i] * ch.d[i];
  }
  z = sum_w<W>(z);
  gw = sum_w<W>(gw);
  const float iz = any ? rcp(z) : 0.0f;
  gw *= iz;
#pragma unroll
  for (int i = 0; i < KL; ++i)
    if (ch.e[i] >= 0) atomicAdd(&row[ch.e[i]], c * w[i] * iz * comp[i] * (ch.d[i] - gw));
  return 0.0f;
}

template <int W, int C, int V, bool SIGMOID, bool RENORM>
__global__ void __launch_bounds__(kBwdThreads) route_backward_kernel(BwdArgs g) {
  constexpr int G = 64 / W;  // rows of a wavefront in flight
  constexpr int S = W * C * V;
  constexpr int KL = lane_choices(W);
  __shared__ __align__(16) float grads[kBwdThreads / W][S];
  __shared__ __align__(16) float logit[kBwdThreads / W][S];
  const int lane = threadIdx.x & 63, gl = lane % W, grp = lane / W;
  const int wave = __builtin_amdgcn_readfirstlane(blockIdx.x * (kBwdThreads / 64) + (threadIdx.x >> 6));
  const int E = g.E;
  float *row = grads[threadIdx.x / W], *lrow = logit[threadIdx.x / W];
  const bool balance = g.counts != nullptr;
  const bool full = balance || (!SIGMOID && !RENORM);  // needs the whole row
  // gradient rows are cleared once here and again by whoever read them
  for (int i = gl; i < S; i += W) row[i] = 0.0f;
  const int64_t first = (int64_t)wave * g.rows;
  if (first >= g.T) return;
  const int row0 = (int)first, row1 = min(g.T, row0 + g.rows);
  float zc = 0.0f, bc = 0.0f;
  if (balance) {
    bc = g.d_loss[0] / (float)max(1, g.totals[1]) * (float)E / (float)g.k;
    zc = 2.0f * g.d_loss[1] / (float)max(1, g.totals[0]);
  }
  // the next row's inputs are on their way while this one is worked on
  float l[C * V];
  Chosen<KL> ch = {};
  int live = 0;
  auto fetch = [&](int t, float (&lo)[C * V], Chosen<KL> &co, int &vo) {
    t = min(t, row1 - 1);
    if (full) load_row<W, C, V>(g.logits + (int64_t)t * E, E, gl, lo);
    if (g.d_w) load_chosen<W, KL>(g, t, gl, co);
    vo = g.valid ? g.valid[t] : 1;
  };
  for (int pos = row0; pos < row1;) {
    int s = 0, end = g.T;
    float f[C * V];
#pragma unroll
    for (int i = 0; i < C * V; ++i) f[i] = 0.0f;
    fetch(pos + grp, l, ch, live);
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
      float ln[C * V];
      Chosen<KL> cn = {};
      int vn;
      fetch(t + G, ln, cn, vn);
      const bool counts = !balance || (s >= 0 && live);
      float d[C * V];
#pragma unroll
      for (int i = 0; i < C * V; ++i) d[i] = 0.0f;
      if (counts) {
        Row<C * V> r;
        r.m = r.inv = 0.0f;
        if (full) {
          float dot;
          row_probs<W, C * V, SIGMOID>(l, r, f, &dot);
          if (balance) {
            const float zr = zc * r.lse * r.inv;
#pragma unroll
            for (int i = 0; i < C * V; ++i) {
              const float b = r.p[i] * (f[i] - dot);
              d[i] = (SIGMOID ? b * r.c[i] : b) + zr * r.e1[i];
            }
          }
        }
        if (g.d_w) {
          float lc[KL];
          if (full) {
#pragma unroll
            for (int c = 0; c < C; ++c) store_v<V>(lrow + V * (gl + W * c), l + V * c);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
          }
#pragma unroll
          for (int i = 0; i < KL; ++i) {
            const int e = max(ch.e[i], 0);
            lc[i] = full ? lrow[e] : g.logits[(int64_t)t * E + e];
          }
          const float gw = route_part<W, KL, SIGMOID, RENORM>(ch, lc, g.routed_scale, r.m, r.inv, row);
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
          for (int c = 0; c < C; ++c) {
            float *p = row + V * (gl + W * c);
            float v4[V], zero[V] = {};
            load_v<V>(p, v4);
            store_v<V>(p, zero);
#pragma unroll
            for (int v = 0; v < V; ++v) {
              d[V * c + v] += v4[v];
              if (!SIGMOID && !RENORM) d[V * c + v] -= r.p[V * c + v] * gw;
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
#pragma unroll
      for (int i = 0; i < C * V; ++i) l[i] = ln[i];
      ch = cn;
      live = vn;
    }
    pos = end;
  }
}

// ---------------------------------------------------------------- launch

template <int W, int C, int V, bool SIGMOID>
int launch_fwd(FwdArgs g, hipStream_t s) {
  constexpr int G = kFwdThreads / W;
  const int64_t items = (int64_t)g.n_seq * ((g.E + kCols - 1) / kCols);
  if (g.T <= kSoloRows && items <= kSoloItems) {
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
