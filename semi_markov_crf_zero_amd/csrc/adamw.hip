// adamw.hip -- one AdamW step over many tensors, states in 32 bits or in 8.
//
//   m <- b1 m + (1 - b1) g,  v <- b2 v + ((1 - b2) g) g
//   p <- p (1 - lr wd) - (lr / (1 - b1^t)) (m / (sqrt(v) c + eps))
//
// Every operation is rounded to float32 by itself (no contraction), in the
// order the header gives, so the codes of an 8-bit state do not depend on
// how a compiler fuses them.
//
// Bound by HBM: 28 bytes a parameter in 32 bits; in 8 bits with float32
// parameters and bfloat16 gradients 14, and a state's 256 values, their scale
// and their largest magnitude stay in one wave's registers, so a step is one
// pass.  Measured: 80 million parameters in 8 bits, 205 us at best (5.4 TB/s);
// 1.5 million in 120 tensors in 32 bits, 10 us.
//
// One launch covers up to kGrads tensors: a workgroup finds its tensor in
// the table's map and steps SEMICRF_ADAMW_BLOCK elements of it.  The
// gradients' addresses, new in every step of a training loop, come with the
// kernel's arguments, so a step copies nothing to the device first.
#include <math.h>

#include <string.h>

#include "encoder.h"

namespace semicrf {

namespace {

constexpr int kThreads = 256;
constexpr int kBlock8 = 256;  // elements of one scale: 4 a lane of one wave
// Gradients of a launch: their addresses and types fill 3.7 of the 4 KB of
// arguments.
constexpr int kGrads = 416;
constexpr float kTiny = 0x1p-100f;  // a block with nothing above holds zeros

struct AdamwArgs {
  const semicrf_adamw_tensor_t *table;
  const int32_t *map;  // tensor of each workgroup
  const float *grad_scale;
  int64_t block0;  // the launch's first workgroup of the table
  int first;       // and its first tensor
  float keep, rate, b1, a1, b2, a2, c, eps;  // 1 - lr wd, lr / (1 - b1^t), 1 - b1, ...
  const void *grads[kGrads];
  uint8_t grad_dtypes[kGrads];
};

// Four elements from i on as float32 (0 past n); one load where aligned.
template <typename T>
__device__ __forceinline__ f32x4_t load4(const T *p, int64_t i, int64_t n) {
  f32x4_t x = {0.f, 0.f, 0.f, 0.f};
  if (i + 4 <= n && (uintptr_t)(p + i) % (4 * sizeof(T)) == 0) {
    const Pack<T, 4> d = *reinterpret_cast<const Pack<T, 4> *>(p + i);
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = (float)d.v[k];
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k < n) x[k] = (float)p[i + k];
  }
  return x;
}
template <typename T>
__device__ __forceinline__ void store4(T *p, int64_t i, int64_t n, f32x4_t x) {
  if (i + 4 <= n && (uintptr_t)(p + i) % (4 * sizeof(T)) == 0) {
    Pack<T, 4> d;
#pragma unroll
    for (int k = 0; k < 4; ++k) d.v[k] = (T)x[k];
    *reinterpret_cast<Pack<T, 4> *>(p + i) = d;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k < n) p[i + k] = (T)x[k];
  }
}
__device__ __forceinline__ f32x4_t load4(const void *p, int dtype, int64_t i, int64_t n) {
  if (dtype == SEMICRF_F32) return load4((const float *)p, i, n);
  if (dtype == SEMICRF_BF16) return load4((const bf16 *)p, i, n);
  return load4((const f16 *)p, i, n);
}
__device__ __forceinline__ void store4(void *p, int dtype, int64_t i, int64_t n, f32x4_t x) {
  if (dtype == SEMICRF_F32)
    store4((float *)p, i, n, x);
  else if (dtype == SEMICRF_BF16)
    store4((bf16 *)p, i, n, x);
  else
    store4((f16 *)p, i, n, x);
}

// The 8-bit forms.  m: the hardware's e4m3 conversions.
__device__ __forceinline__ f32x4_t from_signed8(uint32_t c) {
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(c, false);
  const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(c, true);
  return f32x4_t{lo[0], lo[1], hi[0], hi[1]};
}
__device__ __forceinline__ uint32_t to_signed8(f32x4_t x) {
  int c = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], c, true);
}
// v's root: the top bits of a float32 with its exponent moved, below 2^-6
// steps of 2^-10.
__device__ __forceinline__ float from_root8(uint32_t c) {
  return c >= 16 ? __uint_as_float((c + (120u << 4)) << 19) : (float)c * 0x1p-10f;
}
__device__ __forceinline__ uint32_t to_root8(float x) {
  const uint32_t b = __float_as_uint(x);
  const uint32_t normal = ((b + 0x3FFFFu + ((b >> 19) & 1u)) >> 19) - (120u << 4);
  const uint32_t small = (uint32_t)(int)rintf(x * 1024.f);
  return (x >= 0x1p-6f ? normal : small) & 255u;
}

// Largest magnitude of a wave; as bit patterns, so that a NaN wins.
__device__ __forceinline__ float wave_max(f32x4_t x) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) m = max(m, __float_as_uint(x[k]) & 0x7fffffffu);
#pragma unroll
  for (int o = 32; o; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
  return __uint_as_float(m);
}
__device__ __forceinline__ float block_inv(float top, float most) {
#pragma clang fp contract(off)
  // not-a-number stays one: 0 times it is what the codes and the scale get
  return top > kTiny ? (1.f / top) * most : 0.f;
}

}  // namespace

template <int BITS>
__global__ __launch_bounds__(kThreads) void k_adamw(AdamwArgs a) {
#pragma clang fp contract(off)
  const int64_t blk = a.block0 + blockIdx.x;
  const int ti = a.map[blk];
  const void *grad = a.grads[ti - a.first];
  if (!grad) return;
  const int gtype = a.grad_dtypes[ti - a.first];
  const semicrf_adamw_tensor_t t = a.table[ti];
  const int64_t base = (blk - t.first) * SEMICRF_ADAMW_BLOCK;
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  for (int k = w; k < SEMICRF_ADAMW_BLOCK / kBlock8; k += kThreads / 64) {
    const int64_t b0 = base + k * kBlock8, i = b0 + 4 * lane;
    if (b0 >= t.n) break;
    f32x4_t g = load4(grad, gtype, i, t.n);
    f32x4_t p = t.master ? load4(t.master, i, t.n) : load4(t.p, t.dtype, i, t.n);
    f32x4_t m, v;
    if (BITS == 8) {
      const uint8_t *mc = (const uint8_t *)t.m, *vc = (const uint8_t *)t.v;
      const float ms = t.m_scale[b0 / kBlock8], vs = t.v_scale[b0 / kBlock8];
      uint32_t cm = 0, cv = 0;
      if (i + 4 <= t.n && ((uintptr_t)(mc + i) | (uintptr_t)(vc + i)) % 4 == 0) {
        cm = *(const uint32_t *)(mc + i);
        cv = *(const uint32_t *)(vc + i);
      } else {
        for (int e = 0; e < 4; ++e)
          if (i + e < t.n) {
            cm |= (uint32_t)mc[i + e] << (8 * e);
            cv |= (uint32_t)vc[i + e] << (8 * e);
          }
      }
      m = from_signed8(cm);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        m[e] = m[e] * ms;
        const float r = from_root8((cv >> (8 * e)) & 255u) * vs;
        v[e] = r * r;
      }
    } else {
      m = load4((const float *)t.m, i, t.n);
      v = load4((const float *)t.v, i, t.n);
    }
    f32x4_t root;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (a.grad_scale) g[e] = g[e] * gs;
      m[e] = m[e] * a.b1 + a.a1 * g[e];
      v[e] = v[e] * a.b2 + (a.a2 * g[e]) * g[e];
      root[e] = sqrtf(v[e]);
      p[e] = p[e] * a.keep - (m[e] / (root[e] * a.c + a.eps)) * a.rate;
    }
    if (t.master) store4(t.master, i, t.n, p);
    store4(t.p, t.dtype, i, t.n, p);
    if (BITS == 8) {
      // past the end m and v are 0: they take part in no maximum
      const float tm = wave_max(m), tv = wave_max(root);
      const float im = block_inv(tm, 448.f), iv = block_inv(tv, 496.f);
      f32x4_t x;
      uint32_t cv = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = m[e] * im;
        cv |= to_root8(root[e] * iv) << (8 * e);
      }
      const uint32_t cm = to_signed8(x);
      uint8_t *mc = (uint8_t *)t.m, *vc = (uint8_t *)t.v;
      if (i + 4 <= t.n && ((uintptr_t)(mc + i) | (uintptr_t)(vc + i)) % 4 == 0) {
        *(uint32_t *)(mc + i) = cm;
        *(uint32_t *)(vc + i) = cv;
      } else {
        for (int e = 0; e < 4; ++e)
          if (i + e < t.n) {
            mc[i + e] = (uint8_t)(cm >> (8 * e));
            vc[i + e] = (uint8_t)(cv >> (8 * e));
          }
      }
      if (lane == 0) {
        t.m_scale[b0 / kBlock8] = tm * (1.f / 448.f);
        t.v_scale[b0 / kBlock8] = tv * (1.f / 496.f);
      }
    } else {
      store4((float *)t.m, i, t.n, m);
      store4((float *)t.v, i, t.n, v);
    }
  }
}

template <int ROOT>
__global__ __launch_bounds__(kThreads) void k_adamw_values(const uint8_t *codes,
                                                           const float *scale, int64_t n,
                                                           float *values) {
#pragma clang fp contract(off)
  for (int64_t i = 4 * (blockIdx.x * (int64_t)kThreads + threadIdx.x); i < n;
       i += 4 * (int64_t)gridDim.x * kThreads) {
    uint32_t c = 0;
    if (i + 4 <= n && (uintptr_t)(codes + i) % 4 == 0)
      c = *(const uint32_t *)(codes + i);
    else
      for (int e = 0; e < 4; ++e)
        if (i + e < n) c |= (uint32_t)codes[i + e] << (8 * e);
    const float s = scale[i / kBlock8];
    f32x4_t x;
    if (ROOT) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float r = from_root8((c >> (8 * e)) & 255u) * s;
        x[e] = r * r;
      }
    } else {
      x = from_signed8(c);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = x[e] * s;
    }
    store4(values, i, n, x);
  }
}

namespace {

int64_t blocks_of(int64_t n) { return (n + SEMICRF_ADAMW_BLOCK - 1) / SEMICRF_ADAMW_BLOCK; }

semicrf_status_t check(const semicrf_adamw_tensor_t *t, int count, int bits, int64_t *blocks) {
  if (!t) return SEMICRF_ERR_NULL;
  if (count < 1) return SEMICRF_ERR_SHAPE;
  if (bits != 32 && bits != 8) return SEMICRF_ERR_ARG;
  int64_t sum = 0;
  for (int i = 0; i < count; ++i) {
    if (t[i].n < 0) return SEMICRF_ERR_SHAPE;
    if (!dtype_ok(t[i].dtype)) return SEMICRF_ERR_ARG;
    if (t[i].n && (!t[i].p || !t[i].m || !t[i].v ||
                   (bits == 8 && (!t[i].m_scale || !t[i].v_scale))))
      return SEMICRF_ERR_NULL;
    sum += blocks_of(t[i].n);
    if (sum > 0x7fffffff) return SEMICRF_ERR_SHAPE;
  }
  *blocks = sum;
  return SEMICRF_OK;
}

}  // namespace

}  // namespace semicrf

using namespace semicrf;

extern "C" {

semicrf_status_t semicrf_adamw_table_size(const semicrf_adamw_tensor_t *tensors, int count,
                                          int bits, size_t *bytes) {
  if (!bytes) return SEMICRF_ERR_NULL;
  int64_t blocks;
  const semicrf_status_t e = check(tensors, count, bits, &blocks);
  if (e != SEMICRF_OK) return e;
  *bytes = (size_t)count * sizeof(semicrf_adamw_tensor_t) + (size_t)blocks * sizeof(int32_t);
  return SEMICRF_OK;
}

semicrf_status_t semicrf_adamw_table(const semicrf_adamw_tensor_t *tensors, int count, int bits,
                                     void *host_table, size_t bytes) {
  size_t need;
  const semicrf_status_t e = semicrf_adamw_table_size(tensors, count, bits, &need);
  if (e != SEMICRF_OK) return e;
  if (!host_table) return SEMICRF_ERR_NULL;
  if (bytes < need) return SEMICRF_ERR_WORKSPACE;
  semicrf_adamw_tensor_t *t = (semicrf_adamw_tensor_t *)host_table;
  int32_t *map = (int32_t *)(t + count);
  int64_t at = 0;
  for (int i = 0; i < count; ++i) {
    t[i] = tensors[i];
    t[i].first = at;
    const int64_t end = at + blocks_of(t[i].n);
    while (at < end) map[at++] = i;
  }
  return SEMICRF_OK;
}

semicrf_status_t semicrf_adamw_step(const void *host_table, const void *device_table,
                                    const void *const *grads, const uint8_t *grad_dtypes, int count,
                                    int bits, int64_t step,
                                    double lr, double beta1, double beta2, double eps,
                                    double weight_decay, const float *grad_scale, void *stream) {
  if (!host_table || !device_table || !grads || !grad_dtypes) return SEMICRF_ERR_NULL;
  if (count < 1) return SEMICRF_ERR_SHAPE;
  if ((bits != 32 && bits != 8) || step < 1 || !(beta1 >= 0 && beta1 < 1) ||
      !(beta2 >= 0 && beta2 < 1) || !(eps >= 0))
    return SEMICRF_ERR_ARG;
  for (int i = 0; i < count; ++i)
    if (grads[i] && !dtype_ok(grad_dtypes[i])) return SEMICRF_ERR_ARG;
  (void)hipGetLastError();
  const semicrf_adamw_tensor_t *t = (const semicrf_adamw_tensor_t *)host_table;
  AdamwArgs a;
  a.table = (const semicrf_adamw_tensor_t *)device_table;
  a.map = (const int32_t *)(a.table + count);
  a.grad_scale = grad_scale;
  a.keep = (float)(1.0 - lr * weight_decay);
  a.rate = (float)(lr / (1.0 - pow(beta1, (double)step)));
  a.b1 = (float)beta1;
  a.a1 = (float)(1.0 - beta1);
  a.b2 = (float)beta2;
  a.a2 = (float)(1.0 - beta2);
  a.c = (float)(1.0 / sqrt(1.0 - pow(beta2, (double)step)));
  a.eps = (float)eps;
  for (int i = 0; i < count; i += kGrads) {
    const int n = count - i < kGrads ? count - i : kGrads;
    memset(a.grads, 0, sizeof(a.grads));
    memcpy(a.grads, grads + i, n * sizeof(void *));
    memcpy(a.grad_dtypes, grad_dtypes + i, n);
    a.first = i;
    a.block0 = t[i].first;
    const int64_t blocks = t[i + n - 1].first + blocks_of(t[i + n - 1].n) - a.block0;
    if (!blocks) continue;
    if (bits == 8)
      k_adamw<8><<<(unsigned)blocks, kThreads, 0, (hipStream_t)stream>>>(a);
    else
      k_adamw<32><<<(unsigned)blocks, kThreads, 0, (hipStream_t)stream>>>(a);
    const semicrf_status_t e = launch_status();
    if (e != SEMICRF_OK) return e;
  }
  return SEMICRF_OK;
}

semicrf_status_t semicrf_adamw_values(const void *codes, const float *scale, int64_t n, int root,
                                      float *values, void *stream) {
  if (!codes || !scale || !values) return SEMICRF_ERR_NULL;
  if (n < 1) return SEMICRF_ERR_SHAPE;
  (void)hipGetLastError();
  const int64_t wg = (n + 4 * kThreads - 1) / (4 * kThreads);
  const unsigned grid = (unsigned)(wg < 8192 ? wg : 8192);
  if (root)
    k_adamw_values<1><<<grid, kThreads, 0, (hipStream_t)stream>>>((const uint8_t *)codes, scale, n,
                                                                 values);
  else
    k_adamw_values<0><<<grid, kThreads, 0, (hipStream_t)stream>>>((const uint8_t *)codes, scale, n,
                                                                 values);
  return launch_status();
}

}  // extern "C"
