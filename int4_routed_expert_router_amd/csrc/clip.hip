// clip.hip -- the norm over many gradients, and clipping.
//
// A plan cuts the gradients into items of a few thousand values on the host,
// so that one launch goes over any number of tensors of any sizes.  The first
// kernel adds up squares, a partial sum to a workgroup; every workgroup of the
// second adds the partial sums up again, in the same order, and scales its
// items.
#include <math.h>

#include <algorithm>

#include "internal.h"
#include "values8.h"

namespace coli {
namespace {

constexpr int kThreads = 256;
constexpr int kGroups = 1024;  // partial sums
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

COLI_DEV double square(float v) { return (double)v * (double)v; }

template <bool F32>
COLI_DEV double item_squares(const void *g, int n) {
  double a = 0.0;
  const int head = head_of<F32>(g, n);
  const int body = (n - head) / 8;
  const char *at = reinterpret_cast<const char *>(g) + head * (F32 ? 4 : 2);
  for (int i = threadIdx.x; i < body; i += kThreads) {
    float v[8];
    load8<F32>(at, i, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) a += square(v[j]);
  }
  const int rest = head + 8 * body;
  if ((int)threadIdx.x < head) a += square(load1<F32>(g, threadIdx.x));
  if ((int)threadIdx.x < n - rest) a += square(load1<F32>(g, rest + threadIdx.x));
  return a;
}

// Sum over the workgroup, in every thread.
COLI_DEV double group_sum64(double a, double *red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) a += __shfl_xor(a, o, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = a;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

__global__ void __launch_bounds__(kThreads) clip_norm_kernel(
    const coli_moe_clip_item_t *__restrict__ items, int64_t n_items, double *__restrict__ parts) {
  __shared__ double red[kThreads / 64];
  double a = 0.0;
  for (int64_t i = blockIdx.x; i < n_items; i += gridDim.x) {
    const coli_moe_clip_item_t it = items[i];
    a += it.dtypes & kGradF32 ? item_squares<true>(it.grad, it.n)
                              : item_squares<false>(it.grad, it.n);
  }
  a = group_sum64(a, red);
  if (threadIdx.x == 0) parts[blockIdx.x] = a;
}

template <bool F32, bool OF32>
COLI_DEV void item_scale(const void *g, void *o, int n, float f) {
  int head = head_of<F32>(g, n);
  const char *gat = reinterpret_cast<const char *>(g) + head * (F32 ? 4 : 2);
  char *oat = reinterpret_cast<char *>(o) + head * (OF32 ? 4 : 2);
  int body = (n - head) / 8;
  if (reinterpret_cast<uintptr_t>(oat) & 15) head = body = 0;  // value by value
  for (int i = threadIdx.x; i < body; i += kThreads) {
    float v[8];
    load8<F32>(gat, i, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= f;
    store8<OF32>(oat, i, v);
  }
  if ((int)threadIdx.x < head) store1<OF32>(o, threadIdx.x, load1<F32>(g, threadIdx.x) * f);
  for (int i = head + 8 * body + threadIdx.x; i < n; i += kThreads)
    store1<OF32>(o, i, load1<F32>(g, i) * f);
}

__global__ void __launch_bounds__(kThreads) clip_scale_kernel(
    const coli_moe_clip_item_t *__restrict__ items, int64_t n_items,
    const double *__restrict__ parts, int n_parts, float max_norm, float *__restrict__ norm) {
  __shared__ double red[kThreads / 64];
  double a = 0.0;
  for (int i = threadIdx.x; i < n_parts; i += kThreads) a += parts[i];
  const float total = (float)sqrt(group_sum64(a, red));
  // false for NaN; an infinite norm is left to the caller too
  const float f = total > max_norm && total <= 3.402823466e38f ? __fdiv_rn(max_norm, total) : 1.0f;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    norm[0] = total;
    norm[1] = f;
  }
  for (int64_t i = blockIdx.x; i < n_items; i += gridDim.x) {
    const coli_moe_clip_item_t it = items[i];
    if (it.out == it.grad && f == 1.0f) continue;
    switch (it.dtypes) {
      case 0: item_scale<false, false>(it.grad, it.out, it.n, f); break;
      case kGradF32: item_scale<true, false>(it.grad, it.out, it.n, f); break;
      case kOutF32: item_scale<false, true>(it.grad, it.out, it.n, f); break;
      default: item_scale<true, true>(it.grad, it.out, it.n, f); break;
    }
  }
}

// --------------------------------------------------------------------- plan

int64_t bytes_of(int dtype) { return dtype == COLI_SRC_F32 ? 4 : 2; }

int check_gradients(const coli_moe_gradient_t *g, int32_t n, int64_t *total) {
  if (n < 0 || n > (1 << 20) || (n && !g)) return COLI_E_INVALID;
  *total = 0;
  for (int32_t i = 0; i < n; ++i) {
    const coli_moe_gradient_t &t = g[i];
    if (t.n < 0 || t.n > (int64_t(1) << 40)) return COLI_E_INVALID;
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
    if (*total > int64_t(1) << 42) return COLI_E_INVALID;
  }
  return COLI_OK;
}

// Values of an item: enough items for every partial sum where there is enough
// to do, at least one pass of a workgroup.
int64_t item_values(int64_t total) {
  const int64_t per = (total / kGroups + 2047) / 2048 * 2048;
  return std::min<int64_t>(std::max<int64_t>(per, 2048), 32768);
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
  double *parts = reinterpret_cast<double *>(ws);
  const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(n_items, kGroups));
  launch_k(COLI_K_CLIP_NORM, clip_norm_kernel, dim3(grid), dim3(kThreads), 0, s, items, n_items,
           parts);
  if (hipGetLastError() != hipSuccess) return COLI_E_HIP;
  launch_k(COLI_K_CLIP_SCALE, clip_scale_kernel, dim3(grid), dim3(kThreads), 0, s, items, n_items,
           (const double *)parts, grid, max_norm, norm);
  return hip_status(hipGetLastError());
}

}  // namespace coli
