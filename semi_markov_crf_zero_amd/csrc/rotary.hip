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
#include "encoder.h"

namespace semicrf {

namespace {

constexpr int kThreads = 256;
constexpr int kPlanes = 4096;  // planes of the positions of a workgroup, in LDS
constexpr int64_t kMaxGrid = 1 << 20;

struct RotaryArgs {
  semicrf_rotary_shape_t s;
  const void *x[2];
  void *y[2];
  const double *frequency;
  const int32_t *position;
  int rows;       // positions of a workgroup at a time
  int turned, units;  // vectors of a head that are turned, and all of them
};

struct Turn {
  float c, s;
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
  __shared__ Turn turns[kPlanes];
  const semicrf_rotary_shape_t &s = p.s;
  const int half = s.turn / 2, heads = s.heads + s.heads2;
  const int64_t all = (int64_t)s.B * s.T;
  for (int64_t first = (int64_t)blockIdx.x * p.rows; first < all;
       first += (int64_t)gridDim.x * p.rows) {
    const int rows = (int)min((int64_t)p.rows, all - first);
    __syncthreads();
    for (int e = threadIdx.x; e < rows * half; e += kThreads) {
      const int64_t row = first + e / half;
      const int64_t b = row / s.T, t = row % s.T;
      const int64_t at = s.positions == SEMICRF_POSITION_EACH       ? p.position[row]
                         : s.positions == SEMICRF_POSITION_SEQUENCE ? p.position[b] + t
                                                                    : t;
      turns[e] = turn_of(at, p.frequency[e % half], s.scale, s.inverse);
    }
    __syncthreads();
    const int per = heads * p.units;
    for (int e = threadIdx.x; e < rows * per; e += kThreads) {
      const int r = e / per, left = e % per, head = left / p.units, u = left % p.units;
      const int64_t row = first + r, b = row / s.T, t = row % s.T;
      const bool second = head >= s.heads;
      const int h = second ? head - s.heads : head;
      const int64_t *st = second ? s.stride2 : s.stride;
      const T *x = (const T *)p.x[second] + b * st[0] + t * st[1] + h * st[2];
      T *y = (T *)p.y[second] + (row * (second ? s.heads2 : s.heads) + h) * s.D;
      const Turn *turn = turns + r * half;
      if (u >= p.turned) {
        const int d = s.turn + (u - p.turned) * V;
        *reinterpret_cast<Pack<T, V> *>(y + d) = *reinterpret_cast<const Pack<T, V> *>(x + d);
      } else if (HALF) {
        const int d = u * V;
        const Pack<T, V> lo = *reinterpret_cast<const Pack<T, V> *>(x + d);
        const Pack<T, V> hi = *reinterpret_cast<const Pack<T, V> *>(x + d + half);
        Pack<T, V> a, c;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const Turn z = turn[d + i];
          const float f = (float)lo.v[i], g = (float)hi.v[i];
          a.v[i] = (T)(f * z.c - g * z.s);
          c.v[i] = (T)(f * z.s + g * z.c);
        }
        *reinterpret_cast<Pack<T, V> *>(y + d) = a;
        *reinterpret_cast<Pack<T, V> *>(y + d + half) = c;
      } else {
        // V neighbours hold V / 2 planes; one by one, a unit is a plane
        constexpr int W = V == 1 ? 2 : V;
        const int d = u * W;
        T in[W], out[W];
        if (V == 1) {
          in[0] = x[d], in[1] = x[d + 1];
        } else {
          const Pack<T, V> a = *reinterpret_cast<const Pack<T, V> *>(x + d);
#pragma unroll
          for (int i = 0; i < V; ++i) in[i] = a.v[i];
        }
#pragma unroll
        for (int i = 0; i < W; i += 2) {
          const Turn z = turn[(d + i) / 2];
          const float f = (float)in[i], g = (float)in[i + 1];
          out[i] = (T)(f * z.c - g * z.s);
          out[i + 1] = (T)(f * z.s + g * z.c);
        }
        if (V == 1) {
          y[d] = out[0], y[d + 1] = out[1];
        } else {
          Pack<T, V> a;
#pragma unroll
          for (int i = 0; i < V; ++i) a.v[i] = out[i];
          *reinterpret_cast<Pack<T, V> *>(y + d) = a;
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
  p.units = p.turned + (s.D - s.turn) / V;
  // four vectors a thread, as far as the planes fit
  const int64_t per = (int64_t)(s.heads + s.heads2) * p.units, all = (int64_t)s.B * s.T;
  int64_t rows = 4 * kThreads / per;
  if (rows > kPlanes / (s.turn / 2)) rows = kPlanes / (s.turn / 2);
  if (rows < 1) rows = 1;
  p.rows = (int)rows;
  int64_t grid = (all + rows - 1) / rows;
  if (grid > kMaxGrid) grid = kMaxGrid;
  if (half)
    k_rotary<T, V, true><<<(unsigned)grid, kThreads, 0, st>>>(p);
  else
    k_rotary<T, V, false><<<(unsigned)grid, kThreads, 0, st>>>(p);
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
  if (s->D > 2 * kPlanes) return SEMICRF_ERR_UNSUPPORTED;
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
