// gradnorm.hip -- the norm of many gradients together, and clipping.
//
//   norm = max |g|, sum |g| or (sum g^2)^(1/2) over all elements of all tensors
//   g <- g min(1, max_norm / (norm + 1e-6))
//
// Two passes over the data: k_norm_parts leaves one float64 a workgroup,
// k_clip adds them in a fixed order (every workgroup the same way, so no one waits
// for another) and scales; without clipping k_norm_end adds them alone.
// Squares are exact in float64, whatever the magnitudes.  The tensors' addresses,
// new in every step of a training loop, come with the kernel's arguments.
//
// Bound by HBM: 80 million bfloat16 elements in 64 tensors, 27 us for the norm (5.9 TB/s)
// and 51 for scaling (6.3: part of them are in the last cache from the first pass); 1.5
// million in 120 tensors 5 and 5.5 us, launches.
#include <algorithm>
#include <new>
#include <vector>

#include "encoder.h"

namespace semicrf {

namespace {

constexpr int kThreads = 256;
constexpr int kBlock = 4096;  // elements a workgroup takes at a time
// Tensors of a launch: 15 bytes each fill 3.9 of the 4 KB of arguments.
constexpr int kTensors = 256;
constexpr int kParts = 2048;  // workgroups of a launch, one partial each

struct NormArgs {
  double *parts;
  int count, order;
  int blocks;              // of the launch's tensors
  int at, all;             // the launch's first partial, and how many there are
  void *p[kTensors];
  uint32_t end[kTensors];  // blocks up to the tensor's last
  uint16_t tail[kTensors];  // elements of its last block, less one
  uint8_t dtype[kTensors];
};
struct ClipArgs {
  NormArgs n;
  double max_norm;
  float *norm, *coefficient;
};

// Sixteen elements a thread of a block, 16 bytes at a time where aligned:
// f(value) -> value, stored if WRITE.
template <bool WRITE, typename T, typename F>
__device__ __forceinline__ void over(T *p, int n, F f) {
  constexpr int V = 16 / sizeof(T);
  if ((uintptr_t)p % 16 == 0) {
    const int whole = n / V;
    for (int i = threadIdx.x; i < whole; i += kThreads) {
      Pack<T, V> x = reinterpret_cast<const Pack<T, V> *>(p)[i];
#pragma unroll
      for (int e = 0; e < V; ++e) x.v[e] = (T)f((float)x.v[e]);
      if (WRITE) reinterpret_cast<Pack<T, V> *>(p)[i] = x;
    }
    const int i = whole * V + threadIdx.x;
    if (i < n) {
      const float y = f((float)p[i]);
      if (WRITE) p[i] = (T)y;
    }
  } else {
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const float y = f((float)p[i]);
      if (WRITE) p[i] = (T)y;
    }
  }
}
// All blocks of this workgroup.
template <bool WRITE, typename F>
__device__ __forceinline__ void over_all(const NormArgs &a, F f) {
  int t = 0;
  for (uint32_t b = blockIdx.x; b < (uint32_t)a.blocks; b += gridDim.x) {
    int last = a.count - 1;  // the first tensor that ends after block b
    while (t < last) {
      const int mid = (t + last) / 2;
      if (a.end[mid] <= b)
        t = mid + 1;
      else
        last = mid;
    }
    const uint32_t first = t ? a.end[t - 1] : 0;
    const int64_t at = (int64_t)(b - first) * kBlock;
    const int n = b + 1 == a.end[t] ? a.tail[t] + 1 : kBlock;
    if (a.dtype[t] == SEMICRF_F32)
      over<WRITE>((float *)a.p[t] + at, n, f);
    else if (a.dtype[t] == SEMICRF_BF16)
      over<WRITE>((bf16 *)a.p[t] + at, n, f);
    else
      over<WRITE>((f16 *)a.p[t] + at, n, f);
  }
}

// Magnitudes are compared as bit patterns, so that a NaN wins.
__device__ __forceinline__ double larger(double x, double y) {
  return __double_as_longlong(x) > __double_as_longlong(y) ? x : y;
}
__device__ __forceinline__ double join(double x, double y, int order) {
  return order == SEMICRF_NORM_MAX ? larger(x, y) : x + y;
}
__device__ __forceinline__ double join_all(double x, int order, double *lds) {
#pragma unroll
  for (int o = 32; o; o >>= 1) x = join(x, __shfl_xor(x, o), order);
  if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = x;
  __syncthreads();
  x = lds[0];
#pragma unroll
  for (int w = 1; w < kThreads / 64; ++w) x = join(x, lds[w], order);
  return x;
}

__device__ __forceinline__ float norm_of(const NormArgs &a, double *lds) {
  double x = 0;
  for (int i = threadIdx.x; i < a.all; i += kThreads) x = join(x, a.parts[i], a.order);
  x = join_all(x, a.order, lds);
  return (float)(a.order == SEMICRF_NORM_2 ? sqrt(x) : x);
}
__device__ __forceinline__ float coefficient_of(const ClipArgs &a, float norm) {
  const double c = a.max_norm / ((double)norm + 1e-6);
  return c >= 1 ? 1.f : (float)c;  // not-a-number stays one
}

}  // namespace

__global__ __launch_bounds__(kThreads) void k_norm_parts(NormArgs a) {
  __shared__ double lds[kThreads / 64];
  double x = 0;
  if (a.order == SEMICRF_NORM_2)
    over_all<false>(a, [&](float g) { x = fma((double)g, (double)g, x); return g; });
  else if (a.order == SEMICRF_NORM_1)
    over_all<false>(a, [&](float g) { x += fabs((double)g); return g; });
  else
    over_all<false>(a, [&](float g) { x = larger(x, fabs((double)g)); return g; });
  x = join_all(x, a.order, lds);
  if (threadIdx.x == 0) a.parts[a.at + blockIdx.x] = x;
}

__global__ __launch_bounds__(kThreads) void k_clip(ClipArgs a) {
  __shared__ double lds[kThreads / 64];
  const float norm = norm_of(a.n, lds), c = coefficient_of(a, norm);
  if (blockIdx.x == 0 && threadIdx.x == 0 && a.n.at == 0) {
    if (a.norm) *a.norm = norm;
    if (a.coefficient) *a.coefficient = c;
  }
  if (c == 1.f) return;
  over_all<true>(a.n, [&](float g) { return g * c; });
}

// all partials, one workgroup
__global__ __launch_bounds__(kThreads) void k_norm_end(ClipArgs a) {
  __shared__ double lds[kThreads / 64];
  const float norm = norm_of(a.n, lds);
  if (threadIdx.x == 0) {
    if (a.norm) *a.norm = norm;
    if (a.coefficient) *a.coefficient = coefficient_of(a, norm);
  }
}

namespace {

int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }

// Calls f(first, last, blocks) for the launches' tensors: up to kTensors with
// elements, up to 2^31 - 1 blocks.
template <typename F>
semicrf_status_t launches(const int64_t *sizes, int count, F f) {
  int i = 0;
  while (i < count) {
    int64_t blocks = 0;
    int there = 0, j = i;
    for (; j < count && there < kTensors; ++j) {
      if (sizes[j] < 0) return SEMICRF_ERR_SHAPE;
      if (!sizes[j]) continue;
      if (blocks_of(sizes[j]) > 0x7fffffff) return SEMICRF_ERR_SHAPE;
      if (blocks + blocks_of(sizes[j]) > 0x7fffffff) break;
      blocks += blocks_of(sizes[j]), ++there;
    }
    if (blocks) {
      const semicrf_status_t e = f(i, j, (int)blocks);
      if (e != SEMICRF_OK) return e;
    }
    i = j;
  }
  return SEMICRF_OK;
}
int parts_of(int blocks) { return blocks < kParts ? blocks : kParts; }

semicrf_status_t total_parts(const int64_t *sizes, int count, int64_t *all) {
  *all = 0;
  const semicrf_status_t e = launches(sizes, count, [&](int, int, int blocks) {
    *all += parts_of(blocks);
    return SEMICRF_OK;
  });
  return e != SEMICRF_OK ? e : *all > 0x7fffffff ? SEMICRF_ERR_SHAPE : SEMICRF_OK;
}

// Whether two tensors share memory.
bool overlap(void *const *p, const int64_t *sizes, const uint8_t *dtypes, int count) {
  std::vector<std::pair<uintptr_t, uintptr_t>> at;
  at.reserve(count);
  for (int i = 0; i < count; ++i)
    if (sizes[i]) at.push_back({(uintptr_t)p[i], (uintptr_t)p[i] + sizes[i] * elem_size(dtypes[i])});
  std::sort(at.begin(), at.end());
  for (size_t i = 1; i < at.size(); ++i)
    if (at[i].first < at[i - 1].second) return true;
  return false;
}

}  // namespace

}  // namespace semicrf

using namespace semicrf;

extern "C" {

semicrf_status_t semicrf_grad_norm_workspace_size(const int64_t *sizes, int count, size_t *bytes) {
  if (!bytes || (count > 0 && !sizes)) return SEMICRF_ERR_NULL;
  if (count < 0) return SEMICRF_ERR_SHAPE;
  int64_t all;
  const semicrf_status_t e = total_parts(sizes, count, &all);
  if (e == SEMICRF_OK) *bytes = all * sizeof(double);
  return e;
}

semicrf_status_t semicrf_grad_norm(void *const *grads, const int64_t *sizes,
                                   const uint8_t *dtypes, int count, int order, double max_norm,
                                   int clip, float *norm, float *coefficient, void *workspace,
                                   size_t workspace_bytes, void *stream) try {
  size_t need;
  const semicrf_status_t e = semicrf_grad_norm_workspace_size(sizes, count, &need);
  if (e != SEMICRF_OK) return e;
  if (count && (!grads || !dtypes)) return SEMICRF_ERR_NULL;
  if (order < SEMICRF_NORM_MAX || order > SEMICRF_NORM_2 || !(max_norm >= 0))
    return SEMICRF_ERR_ARG;
  for (int i = 0; i < count; ++i) {
    if (!dtype_ok(dtypes[i])) return SEMICRF_ERR_ARG;
    if (sizes[i] && !grads[i]) return SEMICRF_ERR_NULL;
  }
  if (need && (!workspace || workspace_bytes < need)) return SEMICRF_ERR_WORKSPACE;
  if (clip && overlap(grads, sizes, dtypes, count)) return SEMICRF_ERR_ARG;
  (void)hipGetLastError();
  hipStream_t st = (hipStream_t)stream;
  ClipArgs a = {};
  a.n.parts = (double *)workspace;
  a.n.order = order;
  a.n.all = (int)(need / sizeof(double));
  a.max_norm = max_norm, a.norm = norm, a.coefficient = coefficient;
  auto pass = [&](bool scale) {
    a.n.at = 0;
    return launches(sizes, count, [&](int first, int last, int blocks) {
      int n = 0;
      uint32_t end = 0;
      for (int i = first; i < last; ++i) {
        if (!sizes[i]) continue;
        end += (uint32_t)blocks_of(sizes[i]);
        a.n.p[n] = grads[i];
        a.n.end[n] = end;
        a.n.tail[n] = (uint16_t)((sizes[i] - 1) % kBlock);
        a.n.dtype[n++] = dtypes[i];
      }
      a.n.count = n, a.n.blocks = blocks;
      if (scale)
        k_clip<<<parts_of(blocks), kThreads, 0, st>>>(a);
      else
        k_norm_parts<<<parts_of(blocks), kThreads, 0, st>>>(a.n);
      a.n.at += parts_of(blocks);
      return launch_status();
    });
  };
  semicrf_status_t r = pass(false);
  if (r != SEMICRF_OK) return r;
  if (clip && a.n.all) return pass(true);
  k_norm_end<<<1, kThreads, 0, st>>>(a);
  return launch_status();
} catch (const std::bad_alloc &) {
  return SEMICRF_ERR_WORKSPACE;
}

}  // extern "C"
