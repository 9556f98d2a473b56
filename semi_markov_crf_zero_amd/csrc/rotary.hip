// rotary.hip -- rotary positions.
//
//   (a, b) <- scale (a cos z - b sin z, a sin z + b cos z),  z = position * frequency
//
// for the planes of a row, which are the same for all heads of a position: a
// workgroup takes a few positions, works their cosines and sines out once in LDS
// and then turns every head of both tensors, 16 bytes a load where the layout
// allows.  Angles are formed and reduced to a turn in float64 (at 2^20 a float32
// angle is off by a 16th): r = z / 2 pi less its nearest whole number, sine and
// cosine of r's float32 part and one term for the rest of it.
//
// Bound by HBM: 2^20 positions of 4 + 4 heads of 64 in bfloat16, half of each turned,
// 2.15 GB: 402 to 411 us, 5.2 TB/s, a copy's rate.  Two loads a lane also where a
// row is copied (one of them twice: 600 us), without branches around them (695 us).
// 80004 positions of 4 + 2 heads of 40 in float32 28 to 33 us; 256 of 16 + 16 heads of 128
// 5.5 us, a launch.
#include "encoder.h"

namespace semicrf {

namespace {

constexpr int kThreads = 256;
constexpr int kPlanes = 1024;  // planes of the positions of a workgroup, in LDS
constexpr int kMaxPlanes = 4096;  // of a position: then in more of it
constexpr int kAhead = 4;
constexpr int64_t kMaxGrid = 1 << 20;

// n / d by a product where n d < 2^32 (m = ceil(2^32 / d)); m = 0: the quotient itself.
struct Divisor {
  uint32_t d, m;
};
__device__ __forceinline__ uint32_t quotient(uint32_t n, Divisor v) {
  return v.m ? __umulhi(n, v.m) : n / v.d;
}

struct RotaryArgs {
  semicrf_rotary_shape_t s;
  const void *x[2];
  void *y[2];
  const double *frequency;
  const int32_t *position;
  int rows;           // positions of a workgroup at a time
  int turned;         // vectors of a head that are turned
  Divisor units, per;  // vectors of a head, and of all heads of a position
};

struct Turn {
  float c, s;
};
// A position: its number, and where its rows lie in both tensors.
struct Row {
  int64_t position, x[2];
};

__device__ __forceinline__ Turn turn_of(int64_t position, double frequency, float scale,
                                        bool inverse) {
  const double r = (double)position * frequency * 0.15915494309189533577;
  const double f = r - rint(r);
  const float hi = (float)f, rest = (float)((f - (double)hi) * 6.283185307179586477);
  float s, c;
  sincospif(2.f * hi, &s, &c);
  Turn t;
  t.c = scale * fmaf(-s, rest, c);
  t.s = scale * fmaf(c, rest, s);
  if (inverse) t.s = -t.s;
  return t;
}

}  // namespace

template <typename T, int V, bool HALF>
__global__ __launch_bounds__(kThreads) void k_rotary(RotaryArgs p) {
  extern __shared__ __align__(16) unsigned char lds[];
  Row *const at = (Row *)lds;
  Turn *const turns = (Turn *)(at + p.rows);
  const semicrf_rotary_shape_t &s = p.s;
  const int half = s.turn / 2;
  const int64_t all = (int64_t)s.B * s.T;
  for (int64_t first = (int64_t)blockIdx.x * p.rows; first < all;
       first += (int64_t)gridDim.x * p.rows) {
    const int rows = (int)min((int64_t)p.rows, all - first);
    __syncthreads();
    for (int r = threadIdx.x; r < rows; r += kThreads) {
      const int64_t row = first + r, b = row / s.T, t = row - b * s.T;
      at[r].position = s.positions == SEMICRF_POSITION_EACH       ? p.position[row]
                       : s.positions == SEMICRF_POSITION_SEQUENCE ? p.position[b] + t
                                                                  : t;
      at[r].x[0] = b * s.stride[0] + t * s.stride[1];
      at[r].x[1] = b * s.stride2[0] + t * s.stride2[1];
    }
    __syncthreads();
    // kAhead vectors (pairs of them) a thread on their way, the first ones while the
    // cosines and sines are worked out
    constexpr int W = HALF ? V : V == 1 ? 2 : V;  // elements from one turned unit to the next
    constexpr int C = HALF || V == 1 ? 2 * V : V;  // of a copied one: two loads where turning has two
    const int all_units = rows * (int)p.per.d;
    Pack<T, V> lo[kAhead], hi[kAhead];
    T *to[kAhead];
    int unit[kAhead], row_of[kAhead];
    auto load = [&](int e0) {
#pragma unroll
      for (int n = 0; n < kAhead; ++n) {
        // loads without branches: past the end the last one again
        const int e = min(e0 + n * kThreads, all_units - 1);
        const int r = (int)quotient(e, p.per), left = e - r * (int)p.per.d;
        const int head = (int)quotient(left, p.units), u = left - head * (int)p.units.d;
        const bool second = head >= s.heads;
        const int h = second ? head - s.heads : head;
        const T *x = (const T *)p.x[second] + at[r].x[second] + h * (second ? s.stride2 : s.stride)[2];
        to[n] = (T *)p.y[second] + ((first + r) * (second ? s.heads2 : s.heads) + h) * s.D;
        unit[n] = u, row_of[n] = r;
        const int d = u < p.turned ? u * W : s.turn + (u - p.turned) * C;
        lo[n] = *reinterpret_cast<const Pack<T, V> *>(x + d);
        if (HALF || V == 1)
          hi[n] = *reinterpret_cast<const Pack<T, V> *>(
              x + (u < p.turned ? d + (HALF ? half : 1) : min(d + V, s.D - V)));
      }
    };
    load(threadIdx.x);
    for (int e = threadIdx.x; e < rows * half; e += kThreads) {
      const int r = e / half;
      turns[e] = turn_of(at[r].position, p.frequency[e - r * half], s.scale, s.inverse);
    }
    __syncthreads();
    for (int e0 = threadIdx.x; e0 < all_units; e0 += kAhead * kThreads) {
      if (e0 >= kAhead * kThreads) load(e0);
#pragma unroll
      for (int n = 0; n < kAhead; ++n) {
        if (e0 + n * kThreads >= all_units) break;
        T *y = to[n];
        const int u = unit[n];
        const Turn *turn = turns + row_of[n] * half;
        if (u >= p.turned) {
          const int d = s.turn + (u - p.turned) * C;
          *reinterpret_cast<Pack<T, V> *>(y + d) = lo[n];
          if (C > V && d + V < s.D) *reinterpret_cast<Pack<T, V> *>(y + d + V) = hi[n];
        } else if (HALF || V == 1) {
          // vectors of first and of second elements; one by one, a plane
          const int d = u * W;
          Pack<T, V> a, c;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const Turn z = turn[HALF ? d + i : u];
            const float f = (float)lo[n].v[i], g = (float)hi[n].v[i];
            a.v[i] = (T)(f * z.c - g * z.s);
            c.v[i] = (T)(f * z.s + g * z.c);
          }
          *reinterpret_cast<Pack<T, V> *>(y + d) = a;
          *reinterpret_cast<Pack<T, V> *>(y + d + (HALF ? half : 1)) = c;
        } else {
          Pack<T, V> a;
#pragma unroll
          for (int i = 0; i + 1 < V; i += 2) {
            const Turn z = turn[(u * V + i) / 2];
            const float f = (float)lo[n].v[i], g = (float)lo[n].v[i + 1];
            a.v[i] = (T)(f * z.c - g * z.s);
            a.v[i + 1] = (T)(f * z.s + g * z.c);
          }
          *reinterpret_cast<Pack<T, V> *>(y + u * V) = a;
        }
      }
    }
  }
}

namespace {

// The widest vector, up to 16 bytes, that the planes, rows, strides and
// addresses allow.
int vector_of(const RotaryArgs &p, int size) {
  const semicrf_rotary_shape_t &s = p.s;
  int v = 16 / size;
  auto fits = [&](int64_t n) {
    while (n % v) v /= 2;
  };
  fits(s.layout == SEMICRF_ROTARY_HALF ? s.turn / 2 : s.turn);
  fits(s.D);
  for (int i = 0; i < 2; ++i) {
    if (!p.x[i]) continue;
    const int64_t *st = i ? s.stride2 : s.stride;
    for (int j = 0; j < 3; ++j) fits(st[j]);
    fits((uintptr_t)p.x[i] / size);
    fits((uintptr_t)p.y[i] / size);
  }
  return v;
}

template <typename T, int V>
semicrf_status_t launch(RotaryArgs p, hipStream_t st) {
  const semicrf_rotary_shape_t &s = p.s;
  const bool half = s.layout == SEMICRF_ROTARY_HALF;
  p.turned = half || V == 1 ? s.turn / 2 / (half ? V : 1) : s.turn / V;
  const int copied = half || V == 1 ? 2 * V : V;
  const int units = p.turned + (s.D - s.turn + copied - 1) / copied;
  // four vectors a thread, as far as the planes fit
  const int64_t per = (int64_t)(s.heads + s.heads2) * units, all = (int64_t)s.B * s.T;
  int64_t rows = kAhead * kThreads / per;
  if (rows > kPlanes / (s.turn / 2)) rows = kPlanes / (s.turn / 2);
  if (rows < 1) rows = 1;
  p.rows = (int)rows;
  auto divisor = [](int64_t d, int64_t most) {
    return Divisor{(uint32_t)d, d > 1 && most * d < (int64_t)1 << 32
                                    ? (uint32_t)((((int64_t)1 << 32) + d - 1) / d) : 0};
  };
  p.per = divisor(per, rows * per), p.units = divisor(units, per);
  const size_t lds = rows * (sizeof(Row) + s.turn / 2 * sizeof(Turn));
  int64_t grid = (all + rows - 1) / rows;
  if (grid > kMaxGrid) grid = kMaxGrid;
  if (half)
    k_rotary<T, V, true><<<(unsigned)grid, kThreads, lds, st>>>(p);
  else
    k_rotary<T, V, false><<<(unsigned)grid, kThreads, lds, st>>>(p);
  return launch_status();
}
template <typename T>
semicrf_status_t launch_type(const RotaryArgs &p, hipStream_t st) {
  switch (vector_of(p, sizeof(T))) {
    case 1: return launch<T, 1>(p, st);
    case 2: return launch<T, 2>(p, st);
    case 4: return launch<T, 4>(p, st);
    default: return launch<T, 16 / sizeof(T)>(p, st);
  }
}

}  // namespace

}  // namespace semicrf

using namespace semicrf;

extern "C" semicrf_status_t semicrf_rotary(const semicrf_rotary_shape_t *s, const void *x,
                                           const void *x2, const double *frequency,
                                           const int32_t *position, void *y, void *y2,
                                           void *stream) {
  if (!s || !x || !y || !frequency) return SEMICRF_ERR_NULL;
  const int most = 1 << 30;
  if (s->B < 1 || s->T < 1 || s->heads < 1 || s->heads2 < 0 || s->D < 2 || s->B > most ||
      s->T > most || s->heads > most || s->heads2 > most)
    return SEMICRF_ERR_SHAPE;
  if (s->turn < 2 || s->turn % 2 || s->turn > s->D) return SEMICRF_ERR_SHAPE;
  if (s->D > 2 * kMaxPlanes) return SEMICRF_ERR_UNSUPPORTED;
  const int64_t heads = (int64_t)s->heads + s->heads2;
  if (heads * s->D >= 1 << 28) return SEMICRF_ERR_SHAPE;
  if (!dtype_ok(s->dtype) || s->layout < 0 || s->layout > SEMICRF_ROTARY_INTERLEAVED ||
      s->positions < 0 || s->positions > SEMICRF_POSITION_EACH)
    return SEMICRF_ERR_ARG;
  if ((s->heads2 && (!x2 || !y2)) || (s->positions && !position)) return SEMICRF_ERR_NULL;
  (void)hipGetLastError();
  RotaryArgs p = {};
  p.s = *s;
  p.x[0] = x, p.y[0] = y;
  if (s->heads2) p.x[1] = x2, p.y[1] = y2;
  p.frequency = frequency, p.position = position;
  switch (s->dtype) {
    case SEMICRF_F32: return launch_type<float>(p, (hipStream_t)stream);
    case SEMICRF_BF16: return launch_type<bf16>(p, (hipStream_t)stream);
    default: return launch_type<f16>(p, (hipStream_t)stream);
  }
}
