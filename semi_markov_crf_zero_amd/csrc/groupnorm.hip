// groupnorm.hip -- group norm with an activation over channels-last
// sequences [B][T][C], and its gradient.
//
//   h = (x - mean) rstd over the lengths[b] positions and C/G channels of a
//   group;  z = h w + b;  y = act(z)
//   dz = dy act'(z),  d = dz w:
//   dx = rstd (d - mean(d) - h mean(d h)),  dw = sum dz h,  db = sum dz
//
// A thread owns V neighbouring channels (one 16-byte load of the tensor's
// type) of every R-th position, so a wave's load covers whole rows.  The
// sums over a sequence are split over workgroups (slabs of positions) that
// leave one partial per channel vector; a small kernel adds them in a fixed
// order in float64, and the last pass reads x again and writes the result.
//
// Bound by HBM: a forward pass reads x twice and writes y, a backward pass
// reads x and dy twice and writes dx; what the first pass left in the caches
// serves the second in part.  Measured: 2^20 positions of 64 channels in
// float32, sums 60 to 78 us (4.5 to 3.5 TB/s), result 88 us (6.1 TB/s of reads
// and writes); 16 sequences of 4096 positions (three quarters of them valid) of
// 256 channels in bfloat16 with SiLU, forward 9 + 4 + 15 us, backward 22 + 5 +
// 21 + 4 us.  Fewer than eight positions a thread cost more in their channels'
// parameters than they give (result 21 us at four, 15 at eight, 14.5 at 16).
//
// Short sequences (a norm of each position by itself above all) take another
// way: a workgroup holds NS whole sequences, a stretch of memory without
// gaps, in LDS, so x is read once, whatever C and the groups are.  Positions
// past a length lie in the stretch: they are loaded and then left out by a
// select.
//
// Sums.  mean and var come from sums of (x - pivot) and its square in
// float64, the pivot the group's first element: the subtraction takes the
// common offset out before anything is squared.  It is one in float64 too: where
// the first element is far from the others, a float32 difference would lose
// the same part of each of them.
#include "encoder.h"

namespace semicrf {

namespace {

constexpr int kThreads = 256;

struct GnArgs {
  int B, T, C, G, Cg;
  int cv;     // channel vectors = C / V
  int cvt;    // of them in one workgroup's tile
  int tiles;  // of a row
  int rows;   // positions a workgroup takes at once = kThreads / cvt
  int slab;   // positions of one workgroup
  int slabs;  // of a sequence
  int lanes;  // threads that sum one group's partials
  float eps;
  const int32_t *lengths;
  const float *weight, *bias;
};

// 1 / (1 + e^-z) from the hardware's base-2 exponential and reciprocal, each
// within an ulp: the exponent's rounding adds |z| 2^-24 of e^-z.
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * -1.44269504088896341f));
}

template <int ACT>
__device__ __forceinline__ float act(float z) {
  if (ACT == SEMICRF_ACT_SILU) return z * sigmoid(z);
  if (ACT == SEMICRF_ACT_GELU) return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
  if (ACT == SEMICRF_ACT_RELU) return z > 0.f ? z : z == z ? 0.f : z;
  return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if (ACT == SEMICRF_ACT_SILU) {
    const float e = sigmoid(z);
    return e * (1.f + z * (1.f - e));
  }
  if (ACT == SEMICRF_ACT_GELU)
    return 0.5f * (1.f + erff(z * 0.70710678118654752f)) +
           z * __builtin_amdgcn_exp2f(z * z * -0.72134752044448170f) * 0.39894228040143268f;
  if (ACT == SEMICRF_ACT_RELU) return z > 0.f ? 1.f : 0.f;
  return 1.f;
}

// What a thread needs of its V channels: ONE group holds them all, or each
// has its own statistics.
template <int V, bool ONE>
struct Channels {
  float mean[ONE ? 1 : V], rstd[ONE ? 1 : V], w[V], b[V];
  __device__ __forceinline__ Channels(const GnArgs &p, float2 st, int ch) {
    mean[0] = st.x;
    rstd[0] = st.y;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      w[i] = p.weight ? p.weight[ch + i] : 1.f;
      b[i] = p.bias ? p.bias[ch + i] : 0.f;
    }
  }
  __device__ __forceinline__ Channels(const GnArgs &p, const float *stats, int64_t seq, int ch) {
#pragma unroll
    for (int i = 0; i < (ONE ? 1 : V); ++i) {
      const int64_t bg = seq * p.G + (ch + i) / p.Cg;
      mean[i] = stats[2 * bg];
      rstd[i] = stats[2 * bg + 1];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      w[i] = p.weight ? p.weight[ch + i] : 1.f;
      b[i] = p.bias ? p.bias[ch + i] : 0.f;
    }
  }
  __device__ __forceinline__ float h(float x, int i) const {
    return (x - mean[ONE ? 0 : i]) * rstd[ONE ? 0 : i];
  }
};

constexpr int kUnroll = 4;  // positions a thread has loads in flight for

}  // namespace

// Partial sums of x - pivot and its square, one pair for a vector of channels
// or, where groups part it, for each: part[b][slab][pairs].
template <typename T, int V, bool ONE>
__global__ __launch_bounds__(kThreads) void k_gn_sums(GnArgs p, const T *x, double2 *part) {
  constexpr int N = ONE ? 1 : V;
  __shared__ double2 red[kThreads];
  const int b = blockIdx.x / (p.slabs * p.tiles), s = blockIdx.x / p.tiles % p.slabs;
  const int c = threadIdx.x % p.cvt, r = threadIdx.x / p.cvt;
  const int v = blockIdx.x % p.tiles * p.cvt + c;
  const int len = max(valid_length(p.lengths, b, p.T), 0);
  const int t1 = min(len, (s + 1) * p.slab);
  double sum[N] = {}, sq[N] = {};
  if (r < p.rows && v < p.cv && len > 0) {
    const T *row = x + (int64_t)b * p.T * p.C;
    double pivot[N];
#pragma unroll
    for (int i = 0; i < N; ++i) pivot[i] = (float)row[(v * V + i) / p.Cg * p.Cg];
    row += (int64_t)v * V;
    auto one = [&](const Pack<T, V> &d) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int k = ONE ? 0 : i;
        const double e = (double)(float)d.v[i] - pivot[k];
        sum[k] += e;
        sq[k] += e * e;
      }
    };
    int t = s * p.slab + r;
    for (; t + (kUnroll - 1) * p.rows < t1; t += kUnroll * p.rows) {
      Pack<T, V> d[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k)
        d[k] = *reinterpret_cast<const Pack<T, V> *>(row + (int64_t)(t + k * p.rows) * p.C);
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) one(d[k]);
    }
    for (; t < t1; t += p.rows)
      one(*reinterpret_cast<const Pack<T, V> *>(row + (int64_t)t * p.C));
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (i) __syncthreads();
    red[threadIdx.x] = make_double2(sum[i], sq[i]);
    __syncthreads();
    if (r == 0 && v < p.cv) {
      double a1 = sum[i], a2 = sq[i];
      for (int k = 1; k < p.rows; ++k) {
        a1 += red[k * p.cvt + c].x;
        a2 += red[k * p.cvt + c].y;
      }
      part[((int64_t)b * p.slabs + s) * p.cv * N + v * N + i] = make_double2(a1, a2);
    }
  }
}

// Sums of two values over teams of `lanes` neighbouring threads (a power of
// two up to 64, or the whole workgroup), in a fixed order; all of them get it.
__device__ __forceinline__ double2 team_sum(double a, double b, int lanes) {
  for (int o = (lanes < 64 ? lanes : 64) / 2; o; o >>= 1) {
    a += __shfl_xor(a, o);
    b += __shfl_xor(b, o);
  }
  if (lanes <= 64) return make_double2(a, b);
  __shared__ double2 red[kThreads / 64];
  if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = make_double2(a, b);
  __syncthreads();
  double2 s = red[0];
  for (int k = 1; k < kThreads / 64; ++k) {
    s.x += red[k].x;
    s.y += red[k].y;
  }
  return s;
}

// mean and 1/sqrt(var + eps) from the sums of x - pivot and its square over m
// values; 0, 0 of nothing, NaN of a length that is none (m < 0).
__device__ __forceinline__ float2 stats_of(double2 sum, int64_t m, double pivot, float eps) {
  if (m <= 0) {
    const float x = m < 0 ? __builtin_nanf("") : 0.f;
    return make_float2(x, x);
  }
  const double n = 1.0 / (double)m, mean = sum.x * n, var = sum.y * n - mean * mean;
  const double v = (var > 0 ? var : var == var ? 0.0 : var) + (double)eps;
  return make_float2((float)(pivot + mean), (float)(1.0 / sqrt(v)));  // v may pass float32's range
}

// A team of p.lanes threads per sequence and group: its statistics.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_gn_stats(GnArgs p, int pairs, const T *x,
                                                       const double2 *part, float *stats) {
  const int64_t bg = blockIdx.x * (int64_t)(kThreads / p.lanes) + threadIdx.x / p.lanes;
  const int b = (int)(bg / p.G), g = (int)(bg % p.G), lane = threadIdx.x % p.lanes;
  if (b >= p.B) return;
  const int vg = pairs / p.G;  // pairs of a group
  const int len = valid_length(p.lengths, b, p.T);
  double sum = 0, sq = 0;
#pragma unroll 4
  for (int e = lane; e < p.slabs * vg; e += p.lanes) {
    const double2 d = part[((int64_t)b * p.slabs + e / vg) * pairs + g * vg + e % vg];
    sum += d.x;
    sq += d.y;
  }
  const double2 all = team_sum(sum, sq, p.lanes);
  if (lane == 0)
    reinterpret_cast<float2 *>(stats)[bg] =
        stats_of(all, (int64_t)len * p.Cg, (float)x[(int64_t)b * p.T * p.C + g * p.Cg], p.eps);
}

// y over positions t0.. of a thread's channels.
template <typename T, int V, int ACT, bool ONE>
__device__ __forceinline__ void apply_rows(const GnArgs &p, const Channels<V, ONE> &u, int t, int t1,
                                           int valid, const T *x, T *y) {
  const int len = min(t1, max(valid, 0));
  auto one = [&](int t, Pack<T, V> d) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      d.v[i] = (T)act<ACT>(u.h((float)d.v[i], i) * u.w[i] + u.b[i]);
    *reinterpret_cast<Pack<T, V> *>(y + (int64_t)t * p.C) = d;
  };
  for (; t + (kUnroll - 1) * p.rows < len; t += kUnroll * p.rows) {
    Pack<T, V> d[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k)
      d[k] = *reinterpret_cast<const Pack<T, V> *>(x + (int64_t)(t + k * p.rows) * p.C);
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) one(t + k * p.rows, d[k]);
  }
  for (; t < len; t += p.rows)
    one(t, *reinterpret_cast<const Pack<T, V> *>(x + (int64_t)t * p.C));
  Pack<T, V> none;
#pragma unroll
  for (int i = 0; i < V; ++i) none.v[i] = (T)(valid < 0 ? __builtin_nanf("") : 0.f);
  for (; t < t1; t += p.rows) *reinterpret_cast<Pack<T, V> *>(y + (int64_t)t * p.C) = none;
}

template <typename T, int V, int ACT, bool ONE>
__global__ __launch_bounds__(kThreads) void k_gn_apply(GnArgs p, const T *x, const float *stats,
                                                       T *y) {
  const int b = blockIdx.x / (p.slabs * p.tiles), s = blockIdx.x / p.tiles % p.slabs;
  const int c = threadIdx.x % p.cvt, r = threadIdx.x / p.cvt;
  const int v = blockIdx.x % p.tiles * p.cvt + c;
  if (r >= p.rows || v >= p.cv) return;
  const Channels<V, ONE> u(p, stats, b, v * V);
  const int64_t base = (int64_t)b * p.T * p.C + (int64_t)v * V;
  apply_rows<T, V, ACT, ONE>(p, u, s * p.slab + r, min(p.T, (s + 1) * p.slab),
                             valid_length(p.lengths, b, p.T), x + base, y + base);
}

// The same where a sequence has few partials: every workgroup adds them up
// itself and no launch between the sums and this is needed (one tile of
// vectors a row, each within a group).
template <typename T, int V, int ACT>
__global__ __launch_bounds__(kThreads) void k_gn_apply_sums(GnArgs p, const T *x,
                                                            const double2 *part, float *stats,
                                                            T *y) {
  __shared__ double2 red[kThreads];
  const int b = blockIdx.x / p.slabs, s = blockIdx.x % p.slabs;
  const int v = threadIdx.x % p.cvt, r = threadIdx.x / p.cvt, vg = p.Cg / V;
  const int valid = valid_length(p.lengths, b, p.T);
  double2 sum = make_double2(0, 0);
  if (r < p.rows)
    for (int k = r; k < p.slabs; k += p.rows) {
      const double2 d = part[((int64_t)b * p.slabs + k) * p.cv + v];
      sum.x += d.x;
      sum.y += d.y;
    }
  red[threadIdx.x] = sum;
  __syncthreads();
  if (r >= p.rows) return;
  const int g = v / vg;
  sum = make_double2(0, 0);
  for (int k = 0; k < p.rows; ++k)
    for (int i = 0; i < vg; ++i) {
      const double2 d = red[k * p.cvt + g * vg + i];
      sum.x += d.x;
      sum.y += d.y;
    }
  const float2 st = stats_of(sum, (int64_t)valid * p.Cg,
                             (float)x[(int64_t)b * p.T * p.C + g * p.Cg], p.eps);
  if (s == 0 && r == 0 && v % vg == 0) reinterpret_cast<float2 *>(stats)[(int64_t)b * p.G + g] = st;
  const Channels<V, true> u(p, st, v * V);
  const int64_t base = (int64_t)b * p.T * p.C + (int64_t)v * V;
  apply_rows<T, V, ACT, true>(p, u, s * p.slab + r, min(p.T, (s + 1) * p.slab), valid, x + base,
                              y + base);
}

// Positions a thread sums in float32 before it goes on in float64; without an
// end their rounding grows with the sequence.  16 x 4096 x 256 in bfloat16: 21.5
// us, 20.5 without the second level.
constexpr int kRun = 64;

// Partial sums of dz and dz h per channel: part[b][slab][C].
template <typename T, int V, int ACT, bool ONE>
__global__ __launch_bounds__(kThreads) void k_gn_bwd_sums(GnArgs p, const T *x, const T *dy,
                                                          const float *stats, float2 *part) {
  __shared__ float2 red[kThreads * V];
  const int b = blockIdx.x / (p.slabs * p.tiles), s = blockIdx.x / p.tiles % p.slabs;
  const int c = threadIdx.x % p.cvt, r = threadIdx.x / p.cvt;
  const int v = blockIdx.x % p.tiles * p.cvt + c;
  const int len = max(valid_length(p.lengths, b, p.T), 0);
  const int t1 = min(len, (s + 1) * p.slab);
  double s1[V] = {}, s2[V] = {};
  if (r < p.rows && v < p.cv) {
    const Channels<V, ONE> u(p, stats, b, v * V);
    const int64_t base = (int64_t)b * p.T * p.C + (int64_t)v * V;
    // in float32 over kRun positions, in float64 over those
    float f1[V], f2[V];
    auto one = [&](const Pack<T, V> &d, const Pack<T, V> &e) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float h = u.h((float)d.v[i], i);
        const float dz = (float)e.v[i] * act_slope<ACT>(h * u.w[i] + u.b[i]);
        f1[i] += dz;
        f2[i] += dz * h;
      }
    };
    for (int t = s * p.slab + r; t < t1;) {
#pragma unroll
      for (int i = 0; i < V; ++i) f1[i] = f2[i] = 0.f;
      const int stop = min(t1, t + kRun * p.rows);
      for (; t + p.rows < stop; t += 2 * p.rows) {
        Pack<T, V> d[2], e[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int64_t at = base + (int64_t)(t + k * p.rows) * p.C;
          d[k] = *reinterpret_cast<const Pack<T, V> *>(x + at);
          e[k] = *reinterpret_cast<const Pack<T, V> *>(dy + at);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) one(d[k], e[k]);
      }
      for (; t < stop; t += p.rows) {
        const int64_t at = base + (int64_t)t * p.C;
        one(*reinterpret_cast<const Pack<T, V> *>(x + at),
            *reinterpret_cast<const Pack<T, V> *>(dy + at));
      }
#pragma unroll
      for (int i = 0; i < V; ++i) s1[i] += f1[i], s2[i] += f2[i];
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) red[threadIdx.x * V + i] = make_float2((float)s1[i], (float)s2[i]);
  __syncthreads();
  if (r == 0 && v < p.cv) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      double a1 = s1[i], a2 = s2[i];
      for (int k = 1; k < p.rows; ++k) {
        a1 += red[(k * p.cvt + c) * V + i].x;
        a2 += red[(k * p.cvt + c) * V + i].y;
      }
      part[((int64_t)b * p.slabs + s) * p.C + v * V + i] = make_float2((float)a1, (float)a2);
    }
  }
}

// A team of p.lanes threads per sequence and group: its mean(d), mean(d h).
__global__ __launch_bounds__(kThreads) void k_gn_bwd_group(GnArgs p, const float2 *part,
                                                           float2 *coef) {
  const int64_t bg = blockIdx.x * (int64_t)(kThreads / p.lanes) + threadIdx.x / p.lanes;
  const int b = (int)(bg / p.G), g = (int)(bg % p.G), lane = threadIdx.x % p.lanes;
  if (b >= p.B) return;
  const int len = valid_length(p.lengths, b, p.T);
  double m1 = 0, m2 = 0;
#pragma unroll 4
  for (int e = lane; e < p.slabs * p.Cg; e += p.lanes) {
    const int ch = g * p.Cg + e % p.Cg;
    const float2 d = part[((int64_t)b * p.slabs + e / p.Cg) * p.C + ch];
    const double w = p.weight ? p.weight[ch] : 1.0;
    m1 += w * d.x;
    m2 += w * d.y;
  }
  const double2 all = team_sum(m1, m2, p.lanes);
  if (lane == 0) {
    const double n = 1.0 / ((double)max(len, 1) * p.Cg);
    coef[bg] = make_float2((float)(all.x * n), (float)(all.y * n));
  }
}

// The parameters' gradients: rows of partials [n][C] added in float64, 16
// channels and n / splits rows a workgroup; then the splits.
constexpr int kParamThreads = 1024;
__global__ __launch_bounds__(kParamThreads) void k_gn_bwd_params(int C, int64_t n, int splits,
                                                                 const float2 *part, double2 *sums,
                                                                 float *dw, float *db) {
  __shared__ double2 red[kParamThreads / 4];
  const int tiles = (C + 15) / 16, s = blockIdx.x / tiles;
  const int ch = blockIdx.x % tiles * 16 + threadIdx.x % 16, q = threadIdx.x / 16;
  const int64_t r0 = n * s / splits, r1 = n * (s + 1) / splits;
  double a1 = 0, a2 = 0;
  if (ch < C)
#pragma unroll 8
    for (int64_t r = r0 + q; r < r1; r += kParamThreads / 16) {
      const float2 d = part[r * C + ch];
      a1 += d.x;
      a2 += d.y;
    }
  for (int o = 16; o < 64; o <<= 1) {
    a1 += __shfl_xor(a1, o);
    a2 += __shfl_xor(a2, o);
  }
  if (threadIdx.x % 64 < 16) red[threadIdx.x / 64 * 16 + threadIdx.x % 16] = make_double2(a1, a2);
  __syncthreads();
  if (threadIdx.x < 16 && ch < C) {
    a1 = a2 = 0;
    for (int k = 0; k < kParamThreads / 64; ++k) {
      a1 += red[k * 16 + threadIdx.x].x;
      a2 += red[k * 16 + threadIdx.x].y;
    }
    if (splits > 1) {
      sums[(int64_t)s * C + ch] = make_double2(a1, a2);
    } else {
      if (db) db[ch] = (float)a1;
      if (dw) dw[ch] = (float)a2;
    }
  }
}
__global__ __launch_bounds__(64) void k_gn_bwd_params_sum(int C, int splits, const double2 *sums,
                                                          float *dw, float *db) {
  const int ch = blockIdx.x * 64 + threadIdx.x;
  if (ch >= C) return;
  double a1 = 0, a2 = 0;
#pragma unroll 8
  for (int s = 0; s < splits; ++s) {
    a1 += sums[(int64_t)s * C + ch].x;
    a2 += sums[(int64_t)s * C + ch].y;
  }
  if (db) db[ch] = (float)a1;
  if (dw) dw[ch] = (float)a2;
}

template <typename T, int V, int ACT, bool ONE>
__global__ __launch_bounds__(kThreads) void k_gn_bwd_apply(GnArgs p, const T *x, const T *dy,
                                                           const float *stats, const float2 *coef,
                                                           T *dx) {
  const int b = blockIdx.x / (p.slabs * p.tiles), s = blockIdx.x / p.tiles % p.slabs;
  const int c = threadIdx.x % p.cvt, r = threadIdx.x / p.cvt;
  const int v = blockIdx.x % p.tiles * p.cvt + c;
  if (r >= p.rows || v >= p.cv) return;
  const int t1 = min(p.T, (s + 1) * p.slab);
  const int len = min(t1, max(valid_length(p.lengths, b, p.T), 0));
  const Channels<V, ONE> u(p, stats, b, v * V);
  float2 m[ONE ? 1 : V];
#pragma unroll
  for (int i = 0; i < (ONE ? 1 : V); ++i) m[i] = coef[(int64_t)b * p.G + (v * V + i) / p.Cg];
  const int64_t base = (int64_t)b * p.T * p.C + (int64_t)v * V;
  auto one = [&](int t, Pack<T, V> d, const Pack<T, V> &e) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float h = u.h((float)d.v[i], i);
      const float dh = (float)e.v[i] * act_slope<ACT>(h * u.w[i] + u.b[i]) * u.w[i];
      const int k = ONE ? 0 : i;
      d.v[i] = (T)(u.rstd[k] * (dh - m[k].x - h * m[k].y));
    }
    *reinterpret_cast<Pack<T, V> *>(dx + base + (int64_t)t * p.C) = d;
  };
  int t = s * p.slab + r;
  for (; t + p.rows < len; t += 2 * p.rows) {
    Pack<T, V> d[2], e[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int64_t at = base + (int64_t)(t + k * p.rows) * p.C;
      d[k] = *reinterpret_cast<const Pack<T, V> *>(x + at);
      e[k] = *reinterpret_cast<const Pack<T, V> *>(dy + at);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) one(t + k * p.rows, d[k], e[k]);
  }
  for (; t < len; t += p.rows) {
    const int64_t at = base + (int64_t)t * p.C;
    one(t, *reinterpret_cast<const Pack<T, V> *>(x + at),
        *reinterpret_cast<const Pack<T, V> *>(dy + at));
  }
  Pack<T, V> none;
#pragma unroll
  for (int i = 0; i < V; ++i) none.v[i] = (T)0.f;
  for (; t < t1; t += p.rows) *reinterpret_cast<Pack<T, V> *>(dx + base + (int64_t)t * p.C) = none;
}

// ---- short sequences -------------------------------------------------------

namespace {

// x / d for x < 2^16 and 1 <= d < 2^16: the high word of x times
// ceil(2^32 / d); 2^32 itself stands as 0.
__device__ __forceinline__ int div_small(int x, uint32_t m) {
  return m ? (int)__umulhi((uint32_t)x, m) : x;
}

struct SmallArgs {
  GnArgs g;
  int ns, TC;             // sequences of a workgroup, elements of one
  uint32_t mTC, mC, mCg;  // for div_small
};

// Walks through consecutive elements of a workgroup's stretch: sequence,
// position, channel and group.
struct Walk {
  int s, t, c, g, in_g;
  __device__ __forceinline__ Walk(const SmallArgs &p, int e) {
    s = div_small(e, p.mTC);
    const int r = e - s * p.TC;
    t = div_small(r, p.mC);
    c = r - t * p.g.C;
    g = div_small(c, p.mCg);
    in_g = c - g * p.g.Cg;
  }
  __device__ __forceinline__ void next(const SmallArgs &p) {
    ++c;
    if (++in_g == p.g.Cg) in_g = 0, ++g;
    if (c == p.g.C) {
      c = g = 0;
      if (++t == p.g.T) t = 0, ++s;
    }
  }
};

// LDS: n floats of data (twice backwards), weight and bias, a pair a group.
__device__ __forceinline__ void load_params(const GnArgs &p, float *w, float *b) {
  for (int c = threadIdx.x; c < p.C; c += kThreads) {
    w[c] = p.weight ? p.weight[c] : 1.f;
    b[c] = p.bias ? p.bias[c] : 0.f;
  }
}

}  // namespace

// 16384 positions of 250 channels in 10 groups, float32: 18 us forward, 25
// backward (2 and 3 times 16 MB moved: 2 TB/s); the walk over channels and the
// teams' sums in LDS are what remains.
template <typename T, int V, int ACT>
__global__ __launch_bounds__(kThreads) void k_gn_small(SmallArgs p, const T *x, T *y,
                                                       float *stats) {
  extern __shared__ float lds[];
  const int most = p.ns * p.TC;
  float *xs = lds, *w = xs + (most + 1) / 2 * 2, *bi = w + p.g.C, *st = bi + p.g.C;
  const int b0 = blockIdx.x * p.ns, ns = min(p.ns, p.g.B - b0), n = ns * p.TC;
  x += (int64_t)b0 * p.TC;
  y += (int64_t)b0 * p.TC;
  load_params(p.g, w, bi);
  for (int e = threadIdx.x * V; e < n; e += kThreads * V) {
    const Pack<T, V> d = *reinterpret_cast<const Pack<T, V> *>(x + e);
#pragma unroll
    for (int i = 0; i < V; ++i) xs[e + i] = (float)d.v[i];
  }
  __syncthreads();
  const int lanes = p.g.lanes, lane = threadIdx.x % lanes;
  for (int pair = threadIdx.x / lanes; pair < ns * p.g.G; pair += kThreads / lanes) {
    const int s = pair / p.g.G, g = pair % p.g.G;
    const int len = valid_length(p.g.lengths, b0 + s, p.g.T), m = len * p.g.Cg;
    const float *u = xs + s * p.TC + g * p.g.Cg;
    const double pivot = u[0];
    double sum = 0, sq = 0;
    for (int j = lane; j < m; j += lanes) {
      const int t = p.g.T == 1 ? 0 : div_small(j, p.mCg);
      const double d = u[t * p.g.C + j - t * p.g.Cg] - pivot;
      sum += d;
      sq += d * d;
    }
    const double2 all = team_sum(sum, sq, lanes);
    if (lane == 0) {
      const float2 a = stats_of(all, m, pivot, p.g.eps);
      reinterpret_cast<float2 *>(st)[pair] = a;
      reinterpret_cast<float2 *>(stats)[(int64_t)b0 * p.g.G + pair] = a;
    }
  }
  __syncthreads();
  for (int e = threadIdx.x * V; e < n; e += kThreads * V) {
    Walk k(p, e);
    Pack<T, V> d;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int len = valid_length(p.g.lengths, b0 + k.s, p.g.T);
      const float2 a = *reinterpret_cast<const float2 *>(st + 2 * (k.s * p.g.G + k.g));
      const float v = act<ACT>((xs[e + i] - a.x) * a.y * w[k.c] + bi[k.c]);
      d.v[i] = (T)(k.t < len ? v : len < 0 ? __builtin_nanf("") : 0.f);
      k.next(p);
    }
    *reinterpret_cast<Pack<T, V> *>(y + e) = d;
  }
}

// dx, and the workgroup's sums of dz and dz h per channel: part[workgroup][C].
template <typename T, int V, int ACT>
__global__ __launch_bounds__(kThreads) void k_gn_small_bwd(SmallArgs p, const T *x, const T *dy,
                                                           const float *stats, T *dx,
                                                           float2 *part) {
  extern __shared__ float lds[];
  const int most = p.ns * p.TC;
  float *hs = lds, *dz = hs + most, *w = dz + most, *bi = w + p.g.C, *st = bi + p.g.C;
  __shared__ double2 red[kThreads];
  const int b0 = blockIdx.x * p.ns, ns = min(p.ns, p.g.B - b0), n = ns * p.TC;
  x += (int64_t)b0 * p.TC;
  dy += (int64_t)b0 * p.TC;
  dx += (int64_t)b0 * p.TC;
  stats += 2 * (int64_t)b0 * p.g.G;
  load_params(p.g, w, bi);
  __syncthreads();
  for (int e = threadIdx.x * V; e < n; e += kThreads * V) {
    const Pack<T, V> d = *reinterpret_cast<const Pack<T, V> *>(x + e);
    const Pack<T, V> q = *reinterpret_cast<const Pack<T, V> *>(dy + e);
    Walk k(p, e);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int len = valid_length(p.g.lengths, b0 + k.s, p.g.T);
      const float2 a = *reinterpret_cast<const float2 *>(stats + 2 * (k.s * p.g.G + k.g));
      const float h = ((float)d.v[i] - a.x) * a.y;
      const bool in = k.t < len;
      hs[e + i] = in ? h : 0.f;
      dz[e + i] = in ? (float)q.v[i] * act_slope<ACT>(h * w[k.c] + bi[k.c]) : 0.f;
      k.next(p);
    }
  }
  __syncthreads();
  const int lanes = p.g.lanes, lane = threadIdx.x % lanes;
  for (int pair = threadIdx.x / lanes; pair < ns * p.g.G; pair += kThreads / lanes) {
    const int s = pair / p.g.G, g = pair % p.g.G;
    const int m = max(valid_length(p.g.lengths, b0 + s, p.g.T), 0) * p.g.Cg;
    const int at = s * p.TC + g * p.g.Cg;
    double m1 = 0, m2 = 0;
    for (int j = lane; j < m; j += lanes) {
      const int t = p.g.T == 1 ? 0 : div_small(j, p.mCg), c = j - t * p.g.Cg;
      const float d = dz[at + t * p.g.C + c] * w[g * p.g.Cg + c];
      m1 += d;
      m2 += (double)d * hs[at + t * p.g.C + c];
    }
    const double2 all = team_sum(m1, m2, lanes);
    if (lane == 0) {
      const float n = 1.f / (float)max(m, 1);
      st[2 * pair] = (float)all.x * n;
      st[2 * pair + 1] = (float)all.y * n;
    }
  }
  __syncthreads();
  for (int e = threadIdx.x * V; e < n; e += kThreads * V) {
    Walk k(p, e);
    Pack<T, V> d;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float2 a = *reinterpret_cast<const float2 *>(st + 2 * (k.s * p.g.G + k.g));
      const float rstd = stats[2 * (k.s * p.g.G + k.g) + 1];
      const bool in = k.t < valid_length(p.g.lengths, b0 + k.s, p.g.T);
      d.v[i] = (T)(in ? rstd * (dz[e + i] * w[k.c] - a.x - hs[e + i] * a.y) : 0.f);
      k.next(p);
    }
    *reinterpret_cast<Pack<T, V> *>(dx + e) = d;
  }
  if (!part) return;
  // the channels' sums over the rows: as many row groups as there are threads
  const int rows = ns * p.g.T, groups = max(1, min(kThreads / p.g.C, rows));
  for (int c0 = 0; c0 < p.g.C; c0 += kThreads) {
    const int c = c0 + (p.g.C < kThreads ? threadIdx.x % p.g.C : threadIdx.x);
    const int q = p.g.C < kThreads ? threadIdx.x / p.g.C : 0;
    double a1 = 0, a2 = 0;
    if (c < p.g.C && q < groups)
      for (int r = q; r < rows; r += groups) {
        const float d = dz[r * p.g.C + c];
        a1 += d;
        a2 += (double)d * hs[r * p.g.C + c];
      }
    red[threadIdx.x] = make_double2(a1, a2);
    __syncthreads();
    if (c < p.g.C && q == 0) {
      for (int k = 1; k < groups; ++k) {
        a1 += red[k * p.g.C + c].x;
        a2 += red[k * p.g.C + c].y;
      }
      part[(int64_t)blockIdx.x * p.g.C + c] = make_float2((float)a1, (float)a2);
    }
    __syncthreads();
  }
}

namespace {

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

semicrf_status_t check(const semicrf_groupnorm_shape_t *s) {
  if (!s) return SEMICRF_ERR_NULL;
  if (s->B < 1 || s->T < 1 || s->C < 1 || s->G < 1 || s->C % s->G)
    return SEMICRF_ERR_SHAPE;
  if (s->B > 1 << 30 || s->T > 1 << 30 || s->C > 1 << 30) return SEMICRF_ERR_SHAPE;
  if (!dtype_ok(s->dtype) || s->act < SEMICRF_ACT_NONE || s->act > SEMICRF_ACT_RELU ||
      !(s->eps >= 0.f))
    return SEMICRF_ERR_ARG;
  return SEMICRF_OK;
}

// Channels of a thread: 16 bytes of them, or the largest power of two below
// that divides a row and that every pointer is aligned for.
int vector_width(const semicrf_groupnorm_shape_t *s, const void *const *ptrs, int n) {
  const int size = elem_size(s->dtype);
  int V = 16 / size;
  while (V > 1 && s->C % V) V /= 2;
  for (int i = 0; i < n; ++i)
    while (V > 1 && (uintptr_t)ptrs[i] % (V * size)) V /= 2;
  return V;
}

GnArgs args(const semicrf_groupnorm_shape_t *s, int V) {
  GnArgs p = {};
  p.B = s->B, p.T = s->T, p.C = s->C, p.G = s->G, p.Cg = s->C / s->G;
  p.cv = s->C / V;
  p.cvt = p.cv < kThreads ? p.cv : kThreads;
  p.tiles = (p.cv + p.cvt - 1) / p.cvt;
  p.rows = kThreads / p.cvt;
  // slabs: enough workgroups to fill the GPU several times over, but no
  // shorter than eight positions a thread
  const int64_t tiles = (int64_t)s->B * p.tiles;
  const int64_t most = (s->T + 8 * p.rows - 1) / (8 * p.rows);
  int64_t slabs = (2048 + tiles - 1) / tiles;
  if (slabs > most) slabs = most;
  if (slabs < 1) slabs = 1;
  p.slab = (int)((s->T + slabs - 1) / slabs);
  p.slabs = (s->T + p.slab - 1) / p.slab;
  p.eps = s->eps;
  return p;
}

// Threads that sum `entries` values: about four each, 64 at most, or the
// workgroup for many (4096 of them: 12 us with 64 threads, 6 with 256) of few
// groups: a million groups fill the GPU with a wave each.
int team(int64_t entries, int64_t groups) {
  int n = 1;
  while (n < 64 && 4 * n < entries) n *= 2;
  return entries > 256 && groups < 1 << 20 ? kThreads : n;
}
unsigned team_grid(const GnArgs &p) {
  const int64_t teams = kThreads / p.lanes;
  return (unsigned)(((int64_t)p.B * p.G + teams - 1) / teams);
}

// Short sequences go NS at a time through LDS: about kStretch elements a
// workgroup, NS a power of two so that a stretch is a whole number of
// vectors; where 64 KB of LDS hold what the backward pass keeps of one.
constexpr int kStretch = 4096;
uint32_t magic(int d) { return d == 1 ? 0 : (uint32_t)(((1ull << 32) + d - 1) / d); }
SmallArgs small_args(const semicrf_groupnorm_shape_t *s) {
  SmallArgs p = {};
  p.g = args(s, 1);
  p.TC = s->T * s->C;
  p.ns = 1;
  while (2 * p.ns * p.TC <= kStretch && p.ns < s->B) p.ns *= 2;
  p.mTC = magic(p.TC);
  p.mC = magic(s->C);
  p.mCg = magic(p.g.Cg);
  // a team for each group; wider ones where the groups are few
  const int n = team((int64_t)s->T * p.g.Cg, (int64_t)s->B * s->G);
  p.g.lanes = n > 64 ? 64 : n;
  while (p.g.lanes < 64 && 2 * p.g.lanes * p.ns * s->G <= kThreads) p.g.lanes *= 2;
  return p;
}
// LDS of a short-sequence workgroup with `arrays` copies of its data.
size_t small_lds(const SmallArgs &p, int arrays) {
  return sizeof(float) * ((size_t)arrays * p.ns * p.TC + 2 * (size_t)p.g.C +
                          2 * (size_t)p.ns * p.g.G + 2);
}
bool small_path(const semicrf_groupnorm_shape_t *s) {
  return (int64_t)s->T * s->C <= 2 * kStretch &&
         small_lds(small_args(s), 2) + kThreads * sizeof(double2) <= 65536;
}
int64_t small_blocks(const semicrf_groupnorm_shape_t *s) {
  const int ns = small_args(s).ns;
  return ((int64_t)s->B + ns - 1) / ns;
}
// Elements a thread moves at once there: groups do not matter, only whole
// aligned pieces of a stretch.
int small_width(const semicrf_groupnorm_shape_t *s, const void *const *ptrs, int n) {
  const int size = elem_size(s->dtype), stretch = small_args(s).ns * s->T * s->C;
  int V = 16 / size;
  while (V > 1 && (stretch % V || (int64_t)s->B * s->T * s->C % V)) V /= 2;
  for (int i = 0; i < n; ++i)
    while (V > 1 && (uintptr_t)ptrs[i] % (V * size)) V /= 2;
  return V;
}

// Workgroups that share the rows of partials of the parameters' gradients: one
// up to 4096 rows (eight of its loops of eight loads: about 5 us, as much as
// the second launch that more of them need), 64 at most.
int param_splits(int64_t rows) {
  if (rows <= 4096) return 1;
  const int64_t n = rows / 2048;
  return n > 64 ? 64 : (int)n;
}
size_t param_bytes(const semicrf_groupnorm_shape_t *s, int64_t rows) {
  const int n = param_splits(rows);
  return n > 1 ? align256((size_t)n * s->C * sizeof(double2)) : 0;
}

// Whether the launches with vectors of V channels are within a grid's 2^32 - 1
// threads.
bool fits(const semicrf_groupnorm_shape_t *s, int V) {
  constexpr int64_t most = 0xffffffff;
  int64_t rows;
  if (small_path(s)) {
    rows = small_blocks(s);
    if (rows * kThreads > most) return false;
  } else {
    const GnArgs p = args(s, V);
    rows = (int64_t)p.B * p.slabs;
    if (rows * p.tiles * kThreads > most) return false;
    const int64_t groups = (int64_t)p.B * p.G;
    if (groups * team((int64_t)p.slabs * p.Cg, groups) + kThreads > most) return false;
  }
  return (s->C + 15ll) / 16 * param_splits(rows) * kParamThreads <= most;
}

// Workspace for the narrowest vectors (the widest partials).
size_t need(const semicrf_groupnorm_shape_t *s, int backward) {
  if (small_path(s)) {
    const int64_t rows = small_blocks(s);
    return backward ? align256((size_t)rows * s->C * sizeof(float2)) + param_bytes(s, rows) : 0;
  }
  size_t n = 0;
  for (int V = 1; V <= 8; V *= 2) {
    if (s->C % V) break;
    const GnArgs p = args(s, V);
    const int pairs = (s->C / s->G) % V ? p.C : p.cv;
    size_t m;
    if (backward)
      m = align256((size_t)p.B * p.slabs * p.C * sizeof(float2)) +
          param_bytes(s, (int64_t)p.B * p.slabs) + align256((size_t)p.B * p.G * sizeof(float2));
    else
      m = align256((size_t)p.B * p.slabs * pairs * sizeof(double2));
    if (m > n) n = m;
  }
  return n;
}

template <typename T, int V, int ACT, bool ONE>
semicrf_status_t run_fwd(GnArgs p, const void *x, void *y, float *stats, void *ws,
                         hipStream_t st) {
  const unsigned grid = (unsigned)p.B * p.slabs * p.tiles;
  k_gn_sums<T, V, ONE><<<grid, kThreads, 0, st>>>(p, (const T *)x, (double2 *)ws);
  // the statistics with the result, where a workgroup reads at most 1024
  // partials and a thread adds at most 32 of its group's (32 sequences of 512
  // positions of 256 channels: 20 -> 19 us)
  if (ONE && p.tiles == 1 && p.slabs * p.cv <= 1024 && p.rows * p.Cg / V <= 32) {
    k_gn_apply_sums<T, V, ACT><<<grid, kThreads, 0, st>>>(p, (const T *)x, (const double2 *)ws,
                                                         stats, (T *)y);
    return launch_status();
  }
  p.lanes = team((int64_t)p.slabs * (ONE ? p.cv : p.C) / p.G, (int64_t)p.B * p.G);
  k_gn_stats<T><<<team_grid(p), kThreads, 0, st>>>(p, ONE ? p.cv : p.C, (const T *)x,
                                                         (const double2 *)ws, stats);
  k_gn_apply<T, V, ACT, ONE><<<grid, kThreads, 0, st>>>(p, (const T *)x, stats, (T *)y);
  return launch_status();
}

// part [rows][C] to dw and db.
void run_params(int C, int64_t rows, const float2 *part, double2 *sums, float *dw, float *db,
                hipStream_t st) {
  if (!dw && !db) return;
  const int splits = param_splits(rows), tiles = (C + 15) / 16;
  k_gn_bwd_params<<<(unsigned)(tiles * splits), kParamThreads, 0, st>>>(C, rows, splits, part, sums, dw, db);
  if (splits > 1) k_gn_bwd_params_sum<<<(C + 63) / 64, 64, 0, st>>>(C, splits, sums, dw, db);
}

template <typename T, int V, int ACT, bool ONE>
semicrf_status_t run_bwd(GnArgs p, const void *x, const void *dy, const float *stats,
                         void *dx, float *dw, float *db, void *ws, size_t sums_bytes,
                         hipStream_t st) {
  const unsigned grid = (unsigned)p.B * p.slabs * p.tiles;
  char *w = (char *)ws;
  float2 *part = (float2 *)w;
  w += align256((size_t)p.B * p.slabs * p.C * sizeof(float2));
  double2 *sums = (double2 *)w;
  float2 *coef = (float2 *)(w + sums_bytes);
  k_gn_bwd_sums<T, V, ACT, ONE><<<grid, kThreads, 0, st>>>(p, (const T *)x, (const T *)dy, stats,
                                                           part);
  p.lanes = team((int64_t)p.slabs * p.Cg, (int64_t)p.B * p.G);
  k_gn_bwd_group<<<team_grid(p), kThreads, 0, st>>>(p, part, coef);
  k_gn_bwd_apply<T, V, ACT, ONE><<<grid, kThreads, 0, st>>>(p, (const T *)x, (const T *)dy, stats,
                                                            coef, (T *)dx);
  run_params(p.C, (int64_t)p.B * p.slabs, part, sums, dw, db, st);
  return launch_status();
}

// f<T, V, ACT>() for the call's type, vector width and activation.
template <typename T, int V, typename F>
semicrf_status_t by_act(int act, F f) {
  switch (act) {
    case SEMICRF_ACT_SILU: return f.template run<T, V, SEMICRF_ACT_SILU>();
    case SEMICRF_ACT_GELU: return f.template run<T, V, SEMICRF_ACT_GELU>();
    case SEMICRF_ACT_RELU: return f.template run<T, V, SEMICRF_ACT_RELU>();
    default: return f.template run<T, V, SEMICRF_ACT_NONE>();
  }
}
template <typename F>
semicrf_status_t dispatch(int dtype, int V, int act, F f) {
  if (dtype == SEMICRF_F32) {
    if (V == 4) return by_act<float, 4>(act, f);
    return V == 2 ? by_act<float, 2>(act, f) : by_act<float, 1>(act, f);
  }
  if (dtype == SEMICRF_BF16) {
    if (V == 8) return by_act<bf16, 8>(act, f);
    if (V == 4) return by_act<bf16, 4>(act, f);
    return V == 2 ? by_act<bf16, 2>(act, f) : by_act<bf16, 1>(act, f);
  }
  if (V == 8) return by_act<f16, 8>(act, f);
  if (V == 4) return by_act<f16, 4>(act, f);
  return V == 2 ? by_act<f16, 2>(act, f) : by_act<f16, 1>(act, f);
}

struct Fwd {
  GnArgs p;
  SmallArgs small;  // ns 0: the long way
  const void *x;
  void *y;
  float *stats;
  void *ws;
  hipStream_t st;
  template <typename T, int V, int ACT>
  semicrf_status_t run() {
    if (!small.ns)
      return p.Cg % V ? run_fwd<T, V, ACT, V == 1>(p, x, y, stats, ws, st)
                      : run_fwd<T, V, ACT, true>(p, x, y, stats, ws, st);
    const unsigned grid = (unsigned)((small.g.B + small.ns - 1) / small.ns);
    k_gn_small<T, V, ACT><<<grid, kThreads, small_lds(small, 1), st>>>(small, (const T *)x,
                                                                       (T *)y, stats);
    return launch_status();
  }
};

struct Bwd {
  GnArgs p;
  SmallArgs small;
  size_t sums_bytes;
  const void *x, *dy;
  const float *stats;
  void *dx;
  float *dw, *db;
  void *ws;
  hipStream_t st;
  template <typename T, int V, int ACT>
  semicrf_status_t run() {
    if (!small.ns)
      return p.Cg % V ? run_bwd<T, V, ACT, V == 1>(p, x, dy, stats, dx, dw, db, ws, sums_bytes, st)
                      : run_bwd<T, V, ACT, true>(p, x, dy, stats, dx, dw, db, ws, sums_bytes, st);
    const unsigned grid = (unsigned)((small.g.B + small.ns - 1) / small.ns);
    float2 *part = dw || db ? (float2 *)ws : nullptr;
    k_gn_small_bwd<T, V, ACT><<<grid, kThreads, small_lds(small, 2), st>>>(
        small, (const T *)x, (const T *)dy, stats, (T *)dx, part);
    double2 *sums = (double2 *)((char *)ws + align256((size_t)grid * small.g.C * sizeof(float2)));
    run_params(small.g.C, grid, part, sums, dw, db, st);
    return launch_status();
  }
};

}  // namespace

}  // namespace semicrf

using namespace semicrf;

extern "C" {

semicrf_status_t semicrf_groupnorm_workspace_size(const semicrf_groupnorm_shape_t *s, int backward,
                                                  size_t *bytes) {
  if (!bytes) return SEMICRF_ERR_NULL;
  const semicrf_status_t e = check(s);
  if (e != SEMICRF_OK) return e;
  if (!fits(s, vector_width(s, nullptr, 0))) return SEMICRF_ERR_SHAPE;
  *bytes = need(s, backward);
  return SEMICRF_OK;
}

semicrf_status_t semicrf_groupnorm_fwd(const semicrf_groupnorm_shape_t *s, const void *x,
                                       const float *weight, const float *bias,
                                       const int32_t *lengths, void *y, float *stats,
                                       void *workspace, size_t workspace_bytes, void *stream) {
  if (!s || !x || !y || !stats) return SEMICRF_ERR_NULL;
  const semicrf_status_t e = check(s);
  if (e != SEMICRF_OK) return e;
  const size_t bytes = need(s, 0);
  if (bytes && (!workspace || workspace_bytes < bytes)) return SEMICRF_ERR_WORKSPACE;
  (void)hipGetLastError();
  const void *ptrs[] = {x, y};
  const bool small = small_path(s);
  const int V = small ? small_width(s, ptrs, 2) : vector_width(s, ptrs, 2);
  if (!fits(s, V)) return SEMICRF_ERR_SHAPE;
  Fwd f = {args(s, small ? 1 : V), {}, x, y, stats, workspace, (hipStream_t)stream};
  if (small) f.small = small_args(s);
  f.p.lengths = f.small.g.lengths = lengths;
  f.p.weight = f.small.g.weight = weight;
  f.p.bias = f.small.g.bias = bias;
  return dispatch(s->dtype, V, s->act, f);
}

semicrf_status_t semicrf_groupnorm_bwd(const semicrf_groupnorm_shape_t *s, const void *x,
                                       const float *weight, const float *bias,
                                       const int32_t *lengths, const void *grad_y,
                                       const float *stats, void *grad_x, float *grad_weight,
                                       float *grad_bias, void *workspace, size_t workspace_bytes,
                                       void *stream) {
  if (!s || !x || !grad_y || !stats || !grad_x) return SEMICRF_ERR_NULL;
  const semicrf_status_t e = check(s);
  if (e != SEMICRF_OK) return e;
  const size_t bytes = need(s, 1);
  if (bytes && (!workspace || workspace_bytes < bytes)) return SEMICRF_ERR_WORKSPACE;
  (void)hipGetLastError();
  const void *ptrs[] = {x, grad_y, grad_x};
  const bool small = small_path(s);
  const int V = small ? small_width(s, ptrs, 3) : vector_width(s, ptrs, 3);
  if (!fits(s, V)) return SEMICRF_ERR_SHAPE;
  Bwd f = {args(s, small ? 1 : V), {}, 0, x, grad_y, stats, grad_x, grad_weight, grad_bias, workspace,
           (hipStream_t)stream};
  if (small) f.small = small_args(s);
  f.sums_bytes = param_bytes(s, (int64_t)f.p.B * f.p.slabs);
  f.p.lengths = f.small.g.lengths = lengths;
  f.p.weight = f.small.g.weight = weight;
  f.p.bias = f.small.g.bias = bias;
  return dispatch(s->dtype, V, s->act, f);
}

}  // extern "C"
