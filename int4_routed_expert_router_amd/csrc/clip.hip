// clip.hip -- the norm over many gradients, and clipping.
//
// A plan cuts the gradients into items of a few thousand values on the host,
// so that one launch goes over any number of tensors of any sizes.  One kernel
// adds up squares, a partial sum to a workgroup, and another scales: up to some
// thousand items its workgroups add the partial sums up themselves, in the same
// order, beyond that a small kernel in between does.  A few items are one
// workgroup's work, and one launch.  Memory bounds large ones: 656 MB in 305 to
// 326 us, read at 6.8 TB/s for the sum, then read and written at 6.0.
#include <math.h>

#include <algorithm>

#include "clip_rules.h"
#include "internal.h"
#include "units.h"

namespace coli {
namespace {

constexpr int kThreads = 256;
constexpr int kGroups = 1024;  // partial sums
constexpr int kItem = 8192;    // values of an item, at most (and up to 7 in front of the first)
constexpr int kFew = 16;       // items that one workgroup takes alone, a wave each
enum { kGradF32 = 1, kOutF32 = 2 };

// ------------------------------------------------------------------- device

template <bool F32>
COLI_DEV float load1(const void *p, int64_t i) {
  return F32 ? reinterpret_cast<const float *>(p)[i]
             : bf16_to_f32(reinterpret_cast<const uint16_t *>(p)[i]);
}
template <bool F32>
COLI_DEV void store1(void *p, int64_t i, float v) {
  if (F32)
    reinterpret_cast<float *>(p)[i] = v;
  else
    reinterpret_cast<uint16_t *>(p)[i] = (uint16_t)f32_to_bf16_bits(v);
}

// Values in front of the first 16-byte boundary.
template <bool F32>
COLI_DEV int head_of(const void *p, int n) {
  const int past = (int)(reinterpret_cast<uintptr_t>(p) & 15) / (F32 ? 4 : 2);
  return min(n, past ? (F32 ? 4 : 8) - past : 0);
}

// 16 bytes of bf16 or fp32 values.
template <bool F32>
COLI_DEV void values(uint4 u, float (&v)[F32 ? 4 : 8]) {
  if (F32) {
    v[0] = __uint_as_float(u.x), v[1] = __uint_as_float(u.y);
    v[2] = __uint_as_float(u.z), v[3] = __uint_as_float(u.w);
  } else {
    float w[8];
    unpack8(u, w);
#pragma unroll
    for (int i = 0; i < (F32 ? 4 : 8); ++i) v[i] = w[i];
  }
}

COLI_DEV double square(float v) { return (double)v * (double)v; }

constexpr int kFlight = 4;  // 16-byte loads of a lane in flight (8: 355 us for 656 MB, 4: 349)

// Squares of an item, over THREADS threads of which this is the tid-th.
template <bool F32, int THREADS, bool NT>
COLI_DEV double item_squares(const void *g, int n, int tid) {
  constexpr int V = F32 ? 4 : 8;
  double a = 0.0;
  const int head = head_of<F32>(g, n), body = (n - head) / V;
  const uint4 *at = reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(g) +
                                                    head * (F32 ? 4 : 2));
  auto add = [&](uint4 u) {
    float v[V];
    values<F32>(u, v);
#pragma unroll
    for (int j = 0; j < V; ++j) a += square(v[j]);
  };
  int i0 = tid;
  for (; i0 - tid + kFlight * THREADS <= body; i0 += kFlight * THREADS) {
    uint4 u[kFlight];
#pragma unroll
    for (int c = 0; c < kFlight; ++c) u[c] = load16<NT>(at + i0 + c * THREADS);
#pragma unroll
    for (int c = 0; c < kFlight; ++c) add(u[c]);
  }
  for (; i0 < body; i0 += 2 * THREADS) {
    const bool two = i0 + THREADS < body;
    const uint4 u = load16<NT>(at + i0);
    uint4 w = make_uint4(0, 0, 0, 0);
    if (two) w = load16<NT>(at + i0 + THREADS);
    add(u);
    add(w);
  }
  const int rest = head + V * body;
  if (tid < head) a += square(load1<F32>(g, tid));
  if (tid < n - rest) a += square(load1<F32>(g, rest + tid));
  return a;
}

template <bool F32, bool OF32, int THREADS, bool NT>
COLI_DEV void item_scale(const void *g, void *o, int n, float f, int tid) {
  constexpr int V = F32 ? 4 : 8;
  int head = head_of<F32>(g, n), body = (n - head) / V;
  const uint4 *gat = reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(g) +
                                                     head * (F32 ? 4 : 2));
  char *oat = reinterpret_cast<char *>(o) + head * (OF32 ? 4 : 2);
  // out's boundaries elsewhere: value by value
  if (reinterpret_cast<uintptr_t>(oat) & (V * (OF32 ? 4 : 2) >= 16 ? 15 : 7)) head = body = 0;
  auto put = [&](uint4 u, int i) {
    float v[V];
    values<F32>(u, v);
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] *= f;
    if (OF32) {
#pragma unroll
      for (int j = 0; j < V; j += 4)
        store16<NT && F32>(reinterpret_cast<uint4 *>(oat) + (V * i + j) / 4,
                           make_uint4(__float_as_uint(v[j]), __float_as_uint(v[j + 1]),
                                      __float_as_uint(v[j + 2]), __float_as_uint(v[j + 3])));
    } else if (F32) {
      reinterpret_cast<uint2 *>(oat)[i] = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
    } else {
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = v[F32 ? 0 : j];
      store16<NT>(reinterpret_cast<uint4 *>(oat) + i, pack8(w));
    }
  };
  int i0 = tid;
  for (; i0 - tid + kFlight * THREADS <= body; i0 += kFlight * THREADS) {
    uint4 u[kFlight];
#pragma unroll
    for (int c = 0; c < kFlight; ++c) u[c] = load16<NT>(gat + i0 + c * THREADS);
#pragma unroll
    for (int c = 0; c < kFlight; ++c) put(u[c], i0 + c * THREADS);
  }
  for (; i0 < body; i0 += 2 * THREADS) {
    const bool two = i0 + THREADS < body;
    const uint4 u = gat[i0];
    uint4 w = make_uint4(0, 0, 0, 0);
    if (two) w = gat[i0 + THREADS];
    put(u, i0);
    if (two) put(w, i0 + THREADS);
  }
  if (tid < head) store1<OF32>(o, tid, load1<F32>(g, tid) * f);
  for (int i = head + V * body + tid; i < n; i += THREADS)
    store1<OF32>(o, i, load1<F32>(g, i) * f);
}

template <int THREADS, bool NT>
COLI_DEV double squares_of(const coli_moe_clip_item_t &it, int tid) {
  return it.dtypes & kGradF32 ? item_squares<true, THREADS, NT>(it.grad, it.n, tid)
                              : item_squares<false, THREADS, NT>(it.grad, it.n, tid);
}

// Whether an item's grad is of that many bytes or more.
COLI_DEV bool from_bytes(const coli_moe_clip_item_t &it, int from) {
  return clip_item_bytes(it.n, it.dtypes & kGradF32) >= from;
}

template <int THREADS, bool NT>
COLI_DEV void scale(const coli_moe_clip_item_t &it, float f, int tid) {
  if (it.out == it.grad && f == 1.0f) return;
  switch (it.dtypes) {
    case 0: item_scale<false, false, THREADS, NT>(it.grad, it.out, it.n, f, tid); break;
    case kGradF32: item_scale<true, false, THREADS, NT>(it.grad, it.out, it.n, f, tid); break;
    case kOutF32: item_scale<false, true, THREADS, NT>(it.grad, it.out, it.n, f, tid); break;
    default: item_scale<true, true, THREADS, NT>(it.grad, it.out, it.n, f, tid); break;
  }
}

// Sum over the workgroup, in every thread; red has a place for each wave.
template <int THREADS>
COLI_DEV double group_sum64(double a, double *red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) a += __shfl_xor(a, o, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = a;
  __syncthreads();
  a = 0.0;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) a += red[w];
  return a;
}

// The factor of a sum of squares; the first workgroup reports it.
COLI_DEV float factor(double squares, float max_norm, float *norm) {
  const float total = (float)sqrt(squares);
  // false for NaN; an infinite norm is left to the caller too
  const float f = total > max_norm && total <= 3.402823466e38f ? __fdiv_rn(max_norm, total) : 1.0f;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    norm[0] = total;
    norm[1] = f;
  }
  return f;
}

__global__ void __launch_bounds__(kThreads) clip_norm_kernel(
    const coli_moe_clip_item_t *__restrict__ items, int64_t n_items, int past_from,
    double *__restrict__ parts) {
  __shared__ double red[kThreads / 64];
  double a = 0.0;
  for (int64_t i = blockIdx.x; i < n_items; i += gridDim.x) {
    const coli_moe_clip_item_t it = items[i];
    a += from_bytes(it, past_from) ? squares_of<kThreads, true>(it, threadIdx.x)
                                   : squares_of<kThreads, false>(it, threadIdx.x);
  }
  a = group_sum64<kThreads>(a, red);
  if (threadIdx.x == 0) parts[blockIdx.x] = a;
}

// One item to a workgroup: with the norm's grid, several to each, 656 MB take
// 254 us instead of 222.  Every workgroup adds the partial sums up itself.
__global__ void __launch_bounds__(kThreads) clip_scale_kernel(
    const coli_moe_clip_item_t *__restrict__ items, const double *__restrict__ parts, int n_parts,
    float max_norm, float *__restrict__ norm) {
  __shared__ double red[kThreads / 64];
  double a = 0.0;
  for (int i = threadIdx.x; i < n_parts; i += kThreads) a += parts[i];
  const float f = factor(group_sum64<kThreads>(a, red), max_norm, norm);
  scale<kThreads, false>(items[blockIdx.x], f, threadIdx.x);
}

// For many items that sum is a launch of its own, of one workgroup ...
__global__ void __launch_bounds__(kThreads) clip_finish_kernel(const double *__restrict__ parts,
                                                               int n_parts, float max_norm,
                                                               float *__restrict__ norm) {
  __shared__ double red[kThreads / 64];
  double a = 0.0;
  for (int i = threadIdx.x; i < n_parts; i += kThreads) a += parts[i];
  factor(group_sum64<kThreads>(a, red), max_norm, norm);
}

// ... whose factor is all that the others read.
__global__ void __launch_bounds__(kThreads) clip_scale_many_kernel(
    const coli_moe_clip_item_t *__restrict__ items, int past_from, const float *__restrict__ norm) {
  const coli_moe_clip_item_t it = items[blockIdx.x];
  const float f = norm[1];
  if (from_bytes(it, past_from))
    scale<kThreads, true>(it, f, threadIdx.x);
  else
    scale<kThreads, false>(it, f, threadIdx.x);
}

// Both in one workgroup, for a few items: a wave to an item.  16 items take 6.8 us
// in a row of calls instead of 8.4, 8 take 4.9; alone, 16 are even (18.7 and 18.2
// with the wait).
__global__ void __launch_bounds__(64 * kFew) clip_few_kernel(
    const coli_moe_clip_item_t *__restrict__ items, int n_items, float max_norm,
    float *__restrict__ norm) {
  __shared__ double red[kFew];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  coli_moe_clip_item_t it{};
  if (wave < n_items) it = items[wave];
  const double a = wave < n_items ? squares_of<64, false>(it, lane) : 0.0;
  const float f = factor(group_sum64<64 * kFew>(a, red), max_norm, norm);
  if (wave < n_items) scale<64, false>(it, f, lane);
}

// --------------------------------------------------------------------- plan

constexpr int64_t kMaxValues = int64_t(1) << 36;  // the items of one launch: below 2^24

int64_t bytes_of(int dtype) { return dtype == COLI_SRC_F32 ? 4 : 2; }

int check_gradients(const coli_moe_gradient_t *g, int32_t n, int64_t *total) {
  if (n < 0 || n > (1 << 20) || (n && !g)) return COLI_E_INVALID;
  *total = 0;
  for (int32_t i = 0; i < n; ++i) {
    const coli_moe_gradient_t &t = g[i];
    if (t.n < 0 || t.n > kMaxValues) return COLI_E_INVALID;
    if ((t.grad_dtype != COLI_SRC_BF16 && t.grad_dtype != COLI_SRC_F32) ||
        (t.out_dtype != COLI_SRC_BF16 && t.out_dtype != COLI_SRC_F32))
      return COLI_E_INVALID;
    if (t.n == 0) continue;
    if (!t.grad || !t.out) return COLI_E_INVALID;
    if (t.grad == t.out && t.grad_dtype != t.out_dtype) return COLI_E_INVALID;
    if (reinterpret_cast<uintptr_t>(t.grad) % bytes_of(t.grad_dtype) ||
        reinterpret_cast<uintptr_t>(t.out) % bytes_of(t.out_dtype))
      return COLI_E_ALIGN;
    *total += t.n;
    if (*total > kMaxValues) return COLI_E_INVALID;
  }
  return COLI_OK;
}

// Values of an item: several items to a workgroup where there is enough to do,
// so that the last ones end together, and at least 2,048.
int64_t item_values(int64_t total) {
  const int64_t per = (total / (2 * kGroups) + 2047) / 2048 * 2048;
  return std::min<int64_t>(std::max<int64_t>(per, 2048), kItem);
}

// Values of a gradient's first item: up to a 16-byte boundary of grad, and a
// whole item behind it.
int64_t first_values(const coli_moe_gradient_t &t, int64_t per) {
  const int64_t size = bytes_of(t.grad_dtype);
  const int64_t past = (int64_t)(reinterpret_cast<uintptr_t>(t.grad) & 15) / size;
  return per + (past ? 16 / size - past : 0);
}

uintptr_t addr(const void *p) { return reinterpret_cast<uintptr_t>(p); }
uintptr_t out_end(const coli_moe_clip_item_t &i) {
  return addr(i.out) + (uintptr_t)i.n * (i.dtypes & kOutF32 ? 4 : 2);
}
uintptr_t grad_end(const coli_moe_clip_item_t &i) {
  return addr(i.grad) + (uintptr_t)i.n * (i.dtypes & kGradF32 ? 4 : 2);
}

}  // namespace

int64_t clip_items(const coli_moe_gradient_t *g, int32_t n) {
  int64_t total, items = 0;
  const int rc = check_gradients(g, n, &total);
  if (rc) return rc;
  const int64_t per = item_values(total);
  for (int32_t i = 0; i < n; ++i)
    if (g[i].n) {
      const int64_t rest = std::max<int64_t>(g[i].n - first_values(g[i], per), 0);
      items += 1 + (rest + per - 1) / per;
    }
  return items;
}

int clip_plan(const coli_moe_gradient_t *g, int32_t n, coli_moe_clip_item_t *items,
              int64_t n_items) {
  const int64_t want = clip_items(g, n);
  if (want < 0) return (int)want;
  if (n_items != want || (want && !items)) return COLI_E_INVALID;
  int64_t total, at = 0;
  check_gradients(g, n, &total);
  const int64_t per = item_values(total);
  for (int32_t i = 0; i < n; ++i) {
    const coli_moe_gradient_t &t = g[i];
    for (int64_t o = 0; o < t.n;) {
      const int64_t c = std::min(t.n - o, o ? per : first_values(t, per));
      coli_moe_clip_item_t &it = items[at];
      it.grad = reinterpret_cast<const char *>(t.grad) + o * bytes_of(t.grad_dtype);
      it.out = reinterpret_cast<char *>(t.out) + o * bytes_of(t.out_dtype);
      it.n = (int32_t)c;
      it.dtypes = (t.grad_dtype == COLI_SRC_F32 ? kGradF32 : 0) |
                  (t.out_dtype == COLI_SRC_F32 ? kOutF32 : 0);
      it.order = at++;
      o += c;
    }
  }
  // No out may overlap another, or a grad that is not its own: sorted by out,
  // neighbours tell the former, and a search for each grad the latter.
  using Item = coli_moe_clip_item_t;
  std::sort(items, items + want, [](const Item &a, const Item &b) { return addr(a.out) < addr(b.out); });
  bool bad = false;
  for (int64_t i = 0; i + 1 < want; ++i) bad = bad || out_end(items[i]) > addr(items[i + 1].out);
  for (int64_t i = 0; i < want && !bad; ++i) {
    const Item *hit = std::lower_bound(items, items + want, addr(items[i].grad),
                                       [](const Item &a, uintptr_t p) { return out_end(a) <= p; });
    for (; hit < items + want && addr(hit->out) < grad_end(items[i]) && !bad; ++hit)
      bad = hit != items + i || hit->out != hit->grad;
  }
  std::sort(items, items + want, [](const Item &a, const Item &b) { return a.order < b.order; });
  return bad ? COLI_E_INVALID : COLI_OK;
}

size_t clip_workspace() { return kGroups * sizeof(double); }

int launch_clip(const coli_moe_clip_item_t *items, int64_t n_items, float max_norm, float *norm,
                void *ws, hipStream_t s) {
  if (n_items <= kFew) {
    launch_k(COLI_K_CLIP_SCALE, clip_few_kernel, dim3(1), dim3(64 * kFew), 0, s, items, (int)n_items,
             max_norm, norm);
    return hip_status(hipGetLastError());
  }
  double *parts = reinterpret_cast<double *>(ws);
  // every workgroup the same number of items, up to one
  const int64_t rounds = (n_items + kGroups - 1) / kGroups;
  const int grid = (int)((n_items + rounds - 1) / rounds);
  launch_k(COLI_K_CLIP_NORM, clip_norm_kernel, dim3(grid), dim3(kThreads), 0, s, items, n_items,
           clip_item_from(kSumPast, n_items), parts);
  if (hipGetLastError() != hipSuccess) return COLI_E_HIP;
  if (n_items < kSumOnce) {
    launch_k(COLI_K_CLIP_SCALE, clip_scale_kernel, dim3((unsigned)n_items), dim3(kThreads), 0, s,
             items, (const double *)parts, grid, max_norm, norm);
    return hip_status(hipGetLastError());
  }
  launch_k(COLI_K_CLIP_FINISH, clip_finish_kernel, dim3(1), dim3(kThreads), 0, s,
           (const double *)parts, grid, max_norm, norm);
  if (hipGetLastError() != hipSuccess) return COLI_E_HIP;
  launch_k(COLI_K_CLIP_SCALE, clip_scale_many_kernel, dim3((unsigned)n_items), dim3(kThreads), 0, s,
           items, clip_item_from(kScalePast, n_items), (const float *)norm);
  return hip_status(hipGetLastError());
}

}  // namespace coli
