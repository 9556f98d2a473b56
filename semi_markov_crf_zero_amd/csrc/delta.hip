// delta.hip -- the gated delta rule.
//
//   S_t = e^{g_t} (I - b_t k_t k_t^T) S_{t-1} + b_t k_t v_t^T,  o_t = scale S_t^T q_t
//
// In chunks of L positions.  With G the sums of g from the chunk's start, S the
// state before it, E = diag(e^G), D_ij = e^{G_i - G_j} (j <= i) and
//   m = strict lower part of D * (K K^T),  X = (I + diag(b) m)^-1 diag(b),
// what the positions write is U = X (V - E K S), and
//   O = scale (E Q S + (D * Q K^T) U)
//   S' = e^{G_L} S + Kh^T U,  Kh = diag(e^{G_L - G}) K
//      = (e^{G_L} + A) S + B,  A = -Kh^T X E K,  B = Kh^T X V.
// A and B do not depend on the state, so the chunks are worked on side by side:
//   k_delta_prepare  X, A and B of each chunk;
//   k_delta_scan     S before each chunk, one product with A a chunk;
//   k_delta_out      O of each chunk.
// Backward, with P = D * Q K^T and dS' the gradient of the state after a chunk:
//   dU = scale P^T dO + Kh dS',  dR = X^T dU,  dV = dR
//   dS = (e^{G_L} + A^T) dS' + C,  C = scale (E Q)^T dO - (E K)^T X^T (scale P^T dO)
//   dP = scale D * (dO U^T),  dM = -(strict lower part of D) * (dR U^T)
//   dQ = scale E dO S^T + dP K
//   dK = (dM K - E dR S^T) + (dP^T Q + dM^T K + diag(e^{G_L - G}) U dS'^T)
//   db_i = (dR_i / b_i) . (U_i / b_i)
// The first bracket of dK comes from k as what asks (its position decays from the
// state: +G), the second from k as what is written (-G), so with c_i = q_i . dq_i +
// k_i . (first - second), dg_i = sum_{j >= i} c_j + S' . dS' over the chunk.
//   k_delta_prepare_back  C of each chunk;
//   k_delta_scan          dS' of each chunk, backwards, with A^T;
//   k_delta_grads         the gradients of each chunk.
//
// b = 0 would make the quotient in db 0 / 0: it counts as 2^-96, whose writes
// are below any rounding.  e^g below float32's range counts as 2^-288.
// Differences of G are taken in float64: no quotient of decays is formed.
#include "encoder.h"

namespace semicrf {

namespace {

constexpr int L = 32;  // positions of a chunk
constexpr int kThreads = 256;
constexpr int64_t kMaxThreads = 0xffffffff;  // of a grid
constexpr int kMaxHead = 128;

struct DeltaArgs {
  View q, k, v;
  const void *go;  // gradient of o [B][T][H][Dv]
  const float *log_decay, *beta;
  const int32_t *lengths;
  const float *state_in;
  float *X, *A, *S, *D;  // of each chunk: [L][L], [Dk][Dk], [Dk][Dv] twice (S has one more)
  double *all;           // e^{G_L} of each chunk
  void *o, *dq, *dk, *dv;
  float *state_out, *dg, *db;
  int part_q, part_k, part_v;  // gradients go to float32 [B][T][H][D]: of shared heads
  int rev;
  float bad, scale;
  int B, T, H, Dk, Dv, N;
};

__device__ __forceinline__ f32x4_t mfma(float a, float b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// put(row, col, sum over k of a(row, k) b(k, col)) for M x N values, K deep;
// multiples of 16, a multiple of 4.  One tile of 16 x 16 a wave at a time.
template <typename FA, typename FB, typename FO>
__device__ __forceinline__ void product(int M, int N, int K, FA a, FB b, FO put) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, g = lane >> 4, l16 = lane & 15;
  const int mt = M / 16, all = mt * (N / 16);
  for (int t = w; t < all; t += kThreads / 64) {
    const int r0 = t % mt * 16, c0 = t / mt * 16;
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < K; k += 4) acc = mfma(a(r0 + l16, k + g), b(k + g, c0 + l16), acc);
#pragma unroll
    for (int r = 0; r < 4; ++r) put(r0 + 4 * g + r, c0 + l16, acc[r]);
  }
}

__device__ __forceinline__ int up16(int n) { return (n + 15) & ~15; }

// A matrix in LDS, rows padded against bank conflicts.
struct Mat {
  float *p;
  int ld;
  __device__ __forceinline__ float &operator()(int r, int c) const { return p[r * ld + c]; }
};
struct Lds {
  float *p;
  __device__ __forceinline__ Mat mat(int rows, int cols) {
    Mat m = {p, cols + 4};
    p += rows * (cols + 4);
    return m;
  }
};
__host__ __device__ constexpr int mat_floats(int rows, int cols) { return rows * (cols + 4); }

struct Gates {
  double G[L];
  float from[L], to[L], beta[L];  // e^{G_i}, e^{G_L - G_i}
  float g[L];
  __device__ __forceinline__ float decay(int i, int j) const { return expf((float)(G[i] - G[j])); }
};

// rows n.. and columns D.. are 0
template <typename T>
__device__ __forceinline__ void load(Mat m, const T *src, int64_t st, int n, int D) {
  const int cols = up16(D);
  for (int e = threadIdx.x; e < L * cols; e += kThreads) {
    const int i = e / cols, d = e % cols;
    m(i, d) = i < n && d < D ? (float)src[i * st + d] : 0.f;
  }
}

__device__ __forceinline__ void load_gates(Gates &s, const DeltaArgs &p, int b, int h, int t0,
                                           int n) {
  const int i = threadIdx.x;
  if (i < L) {
    float g = 0.f, beta = 0.f;
    if (i < n) {
      const int64_t at = ((int64_t)b * p.T + t0 + i) * p.H + h;
      g = p.log_decay[at], beta = p.beta[at];
      if (g < -200.f) g = -200.f;
      if (fabsf(beta) < 0x1p-96f) beta = copysignf(0x1p-96f, beta);
    }
    s.g[i] = g, s.beta[i] = beta;
  }
  __syncthreads();
  if (i < L) {
    double G = 0;
    for (int j = 0; j <= i; ++j) G += s.g[j];
    s.G[i] = G;
  }
  __syncthreads();
  if (i < L) {
    s.from[i] = (float)exp(s.G[i]);
    s.to[i] = (float)exp(s.G[L - 1] - s.G[i]);
  }
  __syncthreads();
}

struct Where {
  int n, h, b, t0, count;  // chunk; positions of it within the length
  int64_t bh, at;          // sequence and head, and chunk of all
};
__device__ __forceinline__ Where where(const DeltaArgs &p) {
  Where w;
  w.h = blockIdx.x % p.H;
  w.n = blockIdx.x / p.H % p.N;
  w.b = blockIdx.x / p.H / p.N;
  w.t0 = w.n * L;
  w.bh = (int64_t)w.b * p.H + w.h;
  w.at = w.bh * p.N + w.n;
  w.count = min(L, max(valid_length(p.lengths, w.b, p.T), 0) - w.t0);
  return w;
}
template <typename T>
__device__ __forceinline__ const T *rows(const View &v, const Where &w) {
  return (const T *)v.p + w.b * v.sb + w.t0 * v.st + w.h / v.share * v.sh;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_delta_prepare(DeltaArgs p) {
  extern __shared__ float lds[];
  __shared__ Gates s;
  const Where w = where(p);
  if (w.count <= 0) return;
  const int dk = up16(p.Dk), dv = up16(p.Dv);
  Lds at = {lds};
  const Mat K = at.mat(L, dk), V = at.mat(L, dv), M = at.mat(L, L), X = at.mat(L, L);
  load(K, rows<T>(p.k, w), p.k.st, w.count, p.Dk);
  load(V, rows<T>(p.v, w), p.v.st, w.count, p.Dv);
  load_gates(s, p, w.b, w.h, w.t0, w.count);
  product(L, L, dk, [&](int i, int k) { return K(i, k); }, [&](int k, int j) { return K(j, k); },
          [&](int i, int j, float x) { M(i, j) = j < i ? s.beta[i] * s.decay(i, j) * x : 0.f; });
  __syncthreads();
  // column j of the inverse, from the diagonal down
  if (threadIdx.x < L) {
    const int j = threadIdx.x;
    for (int i = 0; i < L; ++i) {
      float x = i == j ? 1.f : 0.f;
      for (int l = j; l < i; ++l) x -= M(i, l) * X(l, j);
      X(i, j) = x;
    }
    for (int i = 0; i < L; ++i) X(i, j) *= s.beta[j];
    if (j == 0) p.all[w.at] = exp(s.G[L - 1]);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < L * L; e += kThreads) p.X[w.at * L * L + e] = X(e / L, e % L);
  const Mat W = at.mat(L, dk), U = at.mat(L, dv);
  product(L, dk, L, [&](int i, int j) { return X(i, j) * s.from[j]; },
          [&](int j, int d) { return K(j, d); },
          [&](int i, int d, float x) { W(i, d) = -s.to[i] * x; });
  product(L, dv, L, [&](int i, int j) { return X(i, j); }, [&](int j, int c) { return V(j, c); },
          [&](int i, int c, float x) { U(i, c) = s.to[i] * x; });
  __syncthreads();
  float *A = p.A + w.at * p.Dk * p.Dk, *B = p.S + (w.bh * (p.N + 1) + w.n) * p.Dk * p.Dv;
  product(dk, dk, L, [&](int d, int i) { return K(i, d); }, [&](int i, int e) { return W(i, e); },
          [&](int d, int e, float x) { if (d < p.Dk && e < p.Dk) A[d * p.Dk + e] = x; });
  product(dk, dv, L, [&](int d, int i) { return K(i, d); }, [&](int i, int c) { return U(i, c); },
          [&](int d, int c, float x) { if (d < p.Dk && c < p.Dv) B[d * p.Dv + c] = x; });
}

// X <- e^{G_L} X + A X + B over the chunks, 16 columns a workgroup; X before a
// chunk takes the place of its B.  rev: from the last chunk to the first, with
// A^T, D's C in the place of B.
__global__ __launch_bounds__(kThreads) void k_delta_scan(DeltaArgs p) {
  __shared__ float xs[2][kMaxHead][17];
  const int ct = (p.Dv + 15) / 16, c0 = blockIdx.x % ct * 16;
  const int64_t bh = blockIdx.x / ct;
  const int valid = valid_length(p.lengths, (int)(bh / p.H), p.T);
  const int chunks = (max(valid, 0) + L - 1) / L, dk = up16(p.Dk);
  const int64_t size = (int64_t)p.Dk * p.Dv;
  for (int e = threadIdx.x; e < dk * 16; e += kThreads) {
    const int d = e / 16, c = c0 + e % 16;
    xs[0][d][e % 16] = p.state_in && d < p.Dk && c < p.Dv ? p.state_in[bh * size + d * p.Dv + c] : 0.f;
    xs[1][d][e % 16] = 0.f;
  }
  __syncthreads();
  int now = 0;
  for (int i = 0; i < chunks; ++i) {
    const int n = p.rev ? chunks - 1 - i : i;
    const float *A = p.A + (bh * p.N + n) * p.Dk * p.Dk;
    float *slot = p.rev ? p.D + (bh * p.N + n) * size : p.S + (bh * (p.N + 1) + n) * size;
    const double all = p.all[bh * p.N + n];
    const float a = (float)all, low = (float)(all - a);
    product(dk, 16, dk,
            [&](int d, int k) {
              return d < p.Dk && k < p.Dk ? A[p.rev ? k * p.Dk + d : d * p.Dk + k] : 0.f;
            },
            [&](int k, int c) { return xs[now][k][c]; },
            [&](int d, int c, float x) {
              if (d >= p.Dk || c0 + c >= p.Dv) return;
              float *to = slot + d * p.Dv + c0 + c;
              const float old = xs[now][d][c];
              xs[now ^ 1][d][c] = fmaf(old, a, fmaf(old, low, x + *to));
              *to = old;
            });
    now ^= 1;
    __syncthreads();
  }
  for (int e = threadIdx.x; e < dk * 16; e += kThreads) {
    const int d = e / 16, c = c0 + e % 16;
    if (d >= p.Dk || c >= p.Dv) continue;
    const float x = xs[now][d][e % 16];
    if (!p.rev) p.S[(bh * (p.N + 1) + chunks) * size + d * p.Dv + c] = x;
    if (p.state_out) p.state_out[bh * size + d * p.Dv + c] = valid < 0 ? p.bad : x;
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_delta_out(DeltaArgs p) {
  extern __shared__ float lds[];
  __shared__ Gates s;
  const Where w = where(p);
  const int dk = up16(p.Dk), dv = up16(p.Dv);
  T *o = (T *)p.o + (((int64_t)w.b * p.T + w.t0) * p.H + w.h) * p.Dv;
  const int64_t so = (int64_t)p.H * p.Dv;
  const int rest = min(L, p.T - w.t0);
  const T fill = (T)(valid_length(p.lengths, w.b, p.T) < 0 ? p.bad : 0.f);
  for (int e = threadIdx.x; e < rest * p.Dv; e += kThreads)
    if (e / p.Dv >= w.count) o[e / p.Dv * so + e % p.Dv] = fill;
  if (w.count <= 0) return;
  Lds at = {lds};
  const Mat Q = at.mat(L, dk), K = at.mat(L, dk), R = at.mat(L, dv), U = at.mat(L, dv);
  const Mat X = at.mat(L, L), P = at.mat(L, L);
  load(Q, rows<T>(p.q, w), p.q.st, w.count, p.Dk);
  load(K, rows<T>(p.k, w), p.k.st, w.count, p.Dk);
  load(R, rows<T>(p.v, w), p.v.st, w.count, p.Dv);
  for (int e = threadIdx.x; e < L * L; e += kThreads) X(e / L, e % L) = p.X[w.at * L * L + e];
  load_gates(s, p, w.b, w.h, w.t0, w.count);
  const float *S = p.S + (w.bh * (p.N + 1) + w.n) * p.Dk * p.Dv;
  auto state = [&](int d, int c) { return d < p.Dk && c < p.Dv ? S[d * p.Dv + c] : 0.f; };
  product(L, L, dk, [&](int i, int k) { return Q(i, k); }, [&](int k, int j) { return K(j, k); },
          [&](int i, int j, float x) { P(i, j) = j <= i ? s.decay(i, j) * x : 0.f; });
  product(L, dv, dk, [&](int i, int k) { return K(i, k); }, state,
          [&](int i, int c, float x) { R(i, c) -= s.from[i] * x; });
  __syncthreads();
  product(L, dv, L, [&](int i, int j) { return X(i, j); }, [&](int j, int c) { return R(j, c); },
          [&](int i, int c, float x) { U(i, c) = x; });
  __syncthreads();
  product(L, dv, dk + L,
          [&](int i, int k) { return k < dk ? s.from[i] * Q(i, k) : P(i, k - dk); },
          [&](int k, int c) { return k < dk ? state(k, c) : U(k - dk, c); },
          [&](int i, int c, float x) {
            if (i < w.count && c < p.Dv) o[i * so + c] = (T)(p.scale * x);
          });
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_delta_prepare_back(DeltaArgs p) {
  extern __shared__ float lds[];
  __shared__ Gates s;
  const Where w = where(p);
  if (w.count <= 0) return;
  const int dk = up16(p.Dk), dv = up16(p.Dv);
  Lds at = {lds};
  const Mat Q = at.mat(L, dk), K = at.mat(L, dk), dO = at.mat(L, dv), Z = at.mat(L, dv),
            Y = at.mat(L, dv), X = at.mat(L, L), P = at.mat(L, L);
  load(Q, rows<T>(p.q, w), p.q.st, w.count, p.Dk);
  load(K, rows<T>(p.k, w), p.k.st, w.count, p.Dk);
  load(dO, (const T *)p.go + (((int64_t)w.b * p.T + w.t0) * p.H + w.h) * p.Dv,
       (int64_t)p.H * p.Dv, w.count, p.Dv);
  for (int e = threadIdx.x; e < L * L; e += kThreads) X(e / L, e % L) = p.X[w.at * L * L + e];
  load_gates(s, p, w.b, w.h, w.t0, w.count);
  product(L, L, dk, [&](int i, int k) { return Q(i, k); }, [&](int k, int j) { return K(j, k); },
          [&](int i, int j, float x) { P(i, j) = j <= i ? s.decay(i, j) * x : 0.f; });
  __syncthreads();
  product(L, dv, L, [&](int j, int i) { return P(i, j); }, [&](int i, int c) { return dO(i, c); },
          [&](int j, int c, float x) { Z(j, c) = x; });
  __syncthreads();
  product(L, dv, L, [&](int j, int i) { return X(i, j); }, [&](int i, int c) { return Z(i, c); },
          [&](int j, int c, float x) { Y(j, c) = -s.from[j] * x; });
  __syncthreads();
  float *C = p.D + w.at * p.Dk * p.Dv;
  product(dk, dv, 2 * L, [&](int d, int i) { return i < L ? s.from[i] * Q(i, d) : K(i - L, d); },
          [&](int i, int c) { return i < L ? dO(i, c) : Y(i - L, c); },
          [&](int d, int c, float x) {
            if (d < p.Dk && c < p.Dv) C[d * p.Dv + c] = p.scale * x;
          });
}

template <typename T>
__device__ __forceinline__ void put(void *to, int part, int64_t i, float x) {
  if (part)
    ((float *)to)[i] = x;
  else
    ((T *)to)[i] = (T)x;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_delta_grads(DeltaArgs p) {
  extern __shared__ float lds[];
  __shared__ Gates s;
  __shared__ double red[kThreads / 64];
  const Where w = where(p);
  const int dk = up16(p.Dk), dv = up16(p.Dv), rest = min(L, p.T - w.t0);
  const int64_t row0 = ((int64_t)w.b * p.T + w.t0) * p.H + w.h;
  for (int e = threadIdx.x; e < rest * max(p.Dk, p.Dv); e += kThreads) {
    const int i = e / max(p.Dk, p.Dv), d = e % max(p.Dk, p.Dv);
    if (i < w.count) continue;
    const int64_t row = row0 + (int64_t)i * p.H;
    if (d < p.Dk && p.dq) put<T>(p.dq, p.part_q, row * p.Dk + d, 0.f);
    if (d < p.Dk && p.dk) put<T>(p.dk, p.part_k, row * p.Dk + d, 0.f);
    if (d < p.Dv && p.dv) put<T>(p.dv, p.part_v, row * p.Dv + d, 0.f);
    if (d == 0 && p.dg) p.dg[row] = 0.f;
    if (d == 0 && p.db) p.db[row] = 0.f;
  }
  if (w.count <= 0) return;
  Lds at = {lds};
  const Mat Q = at.mat(L, dk), K = at.mat(L, dk), R = at.mat(L, dv), U = at.mat(L, dv),
            dO = at.mat(L, dv), dU = at.mat(L, dv), dR = at.mat(L, dv), X = at.mat(L, L),
            P = at.mat(L, L), dP = at.mat(L, L), dM = at.mat(L, L);
  load(Q, rows<T>(p.q, w), p.q.st, w.count, p.Dk);
  load(K, rows<T>(p.k, w), p.k.st, w.count, p.Dk);
  load(R, rows<T>(p.v, w), p.v.st, w.count, p.Dv);
  load(dO, (const T *)p.go + row0 * p.Dv, (int64_t)p.H * p.Dv, w.count, p.Dv);
  for (int e = threadIdx.x; e < L * L; e += kThreads) X(e / L, e % L) = p.X[w.at * L * L + e];
  load_gates(s, p, w.b, w.h, w.t0, w.count);
  const int64_t size = (int64_t)p.Dk * p.Dv;
  const float *S = p.S + (w.bh * (p.N + 1) + w.n) * size, *D = p.D + w.at * size;
  auto state = [&](int d, int c) { return d < p.Dk && c < p.Dv ? S[d * p.Dv + c] : 0.f; };
  auto after = [&](int d, int c) { return d < p.Dk && c < p.Dv ? D[d * p.Dv + c] : 0.f; };
  // S' . dS'
  double dot = 0;
  for (int e = threadIdx.x; e < size; e += kThreads) dot += (double)S[size + e] * D[e];
#pragma unroll
  for (int o = 32; o; o >>= 1) dot += __shfl_xor(dot, o);
  if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = dot;
  product(L, L, dk, [&](int i, int k) { return Q(i, k); }, [&](int k, int j) { return K(j, k); },
          [&](int i, int j, float x) { P(i, j) = j <= i ? s.decay(i, j) * x : 0.f; });
  product(L, dv, dk, [&](int i, int k) { return K(i, k); }, state,
          [&](int i, int c, float x) { R(i, c) -= s.from[i] * x; });
  __syncthreads();
  product(L, dv, L, [&](int i, int j) { return X(i, j); }, [&](int j, int c) { return R(j, c); },
          [&](int i, int c, float x) { U(i, c) = x; });
  product(L, dv, L + dk,
          [&](int j, int i) { return i < L ? p.scale * P(i, j) : s.to[j] * K(j, i - L); },
          [&](int i, int c) { return i < L ? dO(i, c) : after(i - L, c); },
          [&](int j, int c, float x) { dU(j, c) = x; });
  __syncthreads();
  product(L, dv, L, [&](int j, int i) { return X(i, j); }, [&](int i, int c) { return dU(i, c); },
          [&](int j, int c, float x) {
            dR(j, c) = x;
            if (p.dv && j < w.count && c < p.Dv)
              put<T>(p.dv, p.part_v, (row0 + (int64_t)j * p.H) * p.Dv + c, x);
          });
  __syncthreads();
  product(L, L, dv, [&](int i, int c) { return dO(i, c); }, [&](int c, int j) { return U(j, c); },
          [&](int i, int j, float x) { dP(i, j) = j <= i ? p.scale * s.decay(i, j) * x : 0.f; });
  product(L, L, dv, [&](int i, int c) { return dR(i, c); }, [&](int c, int j) { return U(j, c); },
          [&](int i, int j, float x) { dM(i, j) = j < i ? -s.decay(i, j) * x : 0.f; });
  __syncthreads();
  double mine = 0;  // c of row threadIdx.x
  auto rows_of = [&](Mat z, int D) {
    if (threadIdx.x < L)
      for (int d = 0; d < D; ++d) mine += z(threadIdx.x, d);
  };
  const Mat c = at.mat(L, dk);
  product(L, dk, dv + L,
          [&](int i, int e) { return e < dv ? p.scale * s.from[i] * dO(i, e) : dP(i, e - dv); },
          [&](int e, int d) { return e < dv ? state(d, e) : K(e - dv, d); },
          [&](int i, int d, float x) {
            c(i, d) = Q(i, d) * x;
            if (p.dq && i < w.count && d < p.Dk)
              put<T>(p.dq, p.part_q, (row0 + (int64_t)i * p.H) * p.Dk + d, x);
          });
  __syncthreads();
  rows_of(c, dk);
  __syncthreads();
  product(L, dk, dv + L,
          [&](int i, int e) { return e < dv ? -s.from[i] * dR(i, e) : dM(i, e - dv); },
          [&](int e, int d) { return e < dv ? state(d, e) : K(e - dv, d); },
          [&](int i, int d, float x) { c(i, d) = x; });
  __syncthreads();
  product(L, dk, dv + 2 * L,
          [&](int j, int e) {
            return e < dv ? s.to[j] * U(j, e) : e < dv + L ? dP(e - dv, j) : dM(e - dv - L, j);
          },
          [&](int e, int d) {
            return e < dv ? after(d, e) : e < dv + L ? Q(e - dv, d) : K(e - dv - L, d);
          },
          [&](int j, int d, float x) {
            const float first = c(j, d);
            if (p.dk && j < w.count && d < p.Dk)
              put<T>(p.dk, p.part_k, (row0 + (int64_t)j * p.H) * p.Dk + d, first + x);
            c(j, d) = K(j, d) * (first - x);
          });
  __syncthreads();
  rows_of(c, dk);
  __shared__ double cs[L];
  if (threadIdx.x < L) {
    const int i = threadIdx.x;
    cs[i] = mine;
    if (i < w.count && p.db) {
      double x = 0;
      const float inv = 1.f / s.beta[i];
      for (int e = 0; e < dv; ++e) x += (double)(dR(i, e) * inv) * (U(i, e) * inv);
      p.db[row0 + (int64_t)i * p.H] = (float)x;
    }
  }
  __syncthreads();
  if (threadIdx.x < w.count && p.dg) {
    double x = 0;
    for (int i = 0; i < kThreads / 64; ++i) x += red[i];
    for (int j = L - 1; j >= (int)threadIdx.x; --j) x += cs[j];
    p.dg[row0 + (int64_t)threadIdx.x * p.H] = s.g[threadIdx.x] < -104.f ? 0.f : (float)x;
  }
}

// One position: a workgroup per stream and head, a thread V neighbouring
// columns of R rows of the state, which stays in registers between the dot
// products with the key and its update; what the query reads of the new state
// follows from the old one: q . S' = q . S + (q . k) b (v - k . S).
template <typename T, int V, int R>
__global__ __launch_bounds__(256) void k_delta_step(semicrf_linattn_shape_t s, const T *q,
                                                    const T *k, const T *v,
                                                    const float *log_decay, const float *beta,
                                                    const int32_t *slots, int nslots, float *state,
                                                    T *o) {
  __shared__ float qs[kMaxHead], ks[kMaxHead], qk;
  __shared__ Pack<float, V> red[2][256];
  const int b = blockIdx.x / s.H, h = blockIdx.x % s.H;
  const int slot = slots ? slots[b] : b;
  T *const ob = o + ((int64_t)b * s.H + h) * s.Dv;
  if (slot < 0 || slot >= nslots) {
    for (int c = threadIdx.x; c < s.Dv; c += 256) ob[c] = (T)0.f;
    return;
  }
  const T *vb = v + b * s.v_stride[0] + h / (s.H / s.Hv) * s.v_stride[2];
  float *const S = state + ((int64_t)slot * s.H + h) * s.Dk * s.Dv;
  const int tpr = s.Dv / V, groups = 256 / tpr;
  const int c = threadIdx.x % tpr * V, r0 = threadIdx.x / tpr;
  const bool on = r0 < groups;
  Pack<float, V> x[R];
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (on && r0 + i * groups < s.Dk)
      x[i] = *reinterpret_cast<const Pack<float, V> *>(S + (r0 + i * groups) * s.Dv + c);
  if ((int)threadIdx.x < s.Dk) {
    qs[threadIdx.x] =
        (float)q[b * s.q_stride[0] + h / (s.H / s.Hq) * s.q_stride[2] + threadIdx.x] * s.scale;
    ks[threadIdx.x] = (float)k[b * s.k_stride[0] + h / (s.H / s.Hk) * s.k_stride[2] + threadIdx.x];
  }
  // the decay in two floats: see k_linattn_step
  const double decay = exp((double)log_decay[(int64_t)b * s.H + h]);
  const float d = (float)decay, dl = (float)(decay - d), bt = beta[(int64_t)b * s.H + h];
  Pack<float, V> told, read;
#pragma unroll
  for (int e = 0; e < V; ++e) told.v[e] = read.v[e] = 0.f;
  __syncthreads();
  if (threadIdx.x < 64) {
    float y = 0.f;
    for (int i = threadIdx.x; i < s.Dk; i += 64) y += qs[i] * ks[i];
#pragma unroll
    for (int n = 32; n; n >>= 1) y += __shfl_xor(y, n);
    if (threadIdx.x == 0) qk = y;
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int row = r0 + i * groups;
    if (on && row < s.Dk)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float y = x[i].v[e];
        x[i].v[e] = fmaf(d, y, fabsf(y) < INFINITY ? dl * y : 0.f);
        told.v[e] += ks[row] * x[i].v[e];
        read.v[e] += qs[row] * x[i].v[e];
      }
  }
  red[0][threadIdx.x] = told;
  red[1][threadIdx.x] = read;
  __syncthreads();
  if (!on) return;
  // every thread sums its columns, in the same order
  told = red[0][threadIdx.x % tpr];
  for (int g = 1; g < groups; ++g)
#pragma unroll
    for (int e = 0; e < V; ++e) told.v[e] += red[0][g * tpr + threadIdx.x % tpr].v[e];
  Pack<float, V> add;
#pragma unroll
  for (int e = 0; e < V; ++e) add.v[e] = bt * ((float)vb[c + e] - told.v[e]);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int row = r0 + i * groups;
    if (row < s.Dk) {
#pragma unroll
      for (int e = 0; e < V; ++e) x[i].v[e] = fmaf(ks[row], add.v[e], x[i].v[e]);
      *reinterpret_cast<Pack<float, V> *>(S + row * s.Dv + c) = x[i];
    }
  }
  if (r0 == 0) {
    read = red[1][threadIdx.x];
    for (int g = 1; g < groups; ++g)
#pragma unroll
      for (int e = 0; e < V; ++e) read.v[e] += red[1][g * tpr + threadIdx.x].v[e];
#pragma unroll
    for (int e = 0; e < V; ++e) ob[c + e] = (T)fmaf(qk, add.v[e], read.v[e]);
  }
}

template <typename T, int V, int R>
semicrf_status_t launch_step(const semicrf_linattn_shape_t &s, const void *q, const void *k,
                             const void *v, const float *log_decay, const float *beta,
                             const int32_t *slots, int nslots, float *state, void *o,
                             hipStream_t st) {
  k_delta_step<T, V, R><<<(unsigned)s.B * s.H, 256, 0, st>>>(
      s, (const T *)q, (const T *)k, (const T *)v, log_decay, beta, slots, nslots, state, (T *)o);
  return launch_status();
}
// Rows of the state a thread holds: those of 128 columns by fours, or of 127 one
// by one.
template <typename T>
semicrf_status_t step_type(const semicrf_linattn_shape_t &s, const void *q, const void *k,
                           const void *v, const float *log_decay, const float *beta,
                           const int32_t *slots, int nslots, float *state, void *o,
                           hipStream_t st) {
  if (s.Dv % 4 == 0 && (uintptr_t)state % 16 == 0)
    return launch_step<T, 4, 16>(s, q, k, v, log_decay, beta, slots, nslots, state, o, st);
  return launch_step<T, 1, 64>(s, q, k, v, log_decay, beta, slots, nslots, state, o, st);
}

semicrf_status_t check(const semicrf_linattn_shape_t *s) {
  if (!s) return SEMICRF_ERR_NULL;
  if (s->B < 1 || s->T < 1 || s->H < 1 || s->Hq < 1 || s->Hk < 1 || s->Hv < 1 || s->Dk < 1 ||
      s->Dv < 1 || s->H % s->Hq || s->H % s->Hk || s->H % s->Hv)
    return SEMICRF_ERR_SHAPE;
  if (s->T > 1 << 30) return SEMICRF_ERR_SHAPE;
  const int64_t heads = (int64_t)s->B * s->H, chunks = (s->T + L - 1) / L;
  if (heads * kThreads > kMaxThreads || heads * chunks * kThreads > kMaxThreads)
    return SEMICRF_ERR_SHAPE;
  if (s->Dk > kMaxHead || s->Dv > kMaxHead) return SEMICRF_ERR_UNSUPPORTED;
  if (heads * ((s->Dv + 15) / 16) * kThreads > kMaxThreads) return SEMICRF_ERR_SHAPE;
  return dtype_ok(s->dtype) ? SEMICRF_OK : SEMICRF_ERR_ARG;
}

// The workspaces.  Forward: what the backward pass reads again.  Backward: D
// and the parts of shared heads' gradients.
struct Areas {
  char *at;
  template <typename T>
  T *take(int64_t n) {
    T *p = (T *)at;
    at += (n * sizeof(T) + 255) / 256 * 256;
    return p;
  }
};
size_t forward_areas(const semicrf_linattn_shape_t *s, void *ws, DeltaArgs *p) {
  Areas a = {(char *)ws};
  const int64_t heads = (int64_t)s->B * s->H, N = (s->T + L - 1) / L;
  p->X = a.take<float>(heads * N * L * L);
  p->A = a.take<float>(heads * N * s->Dk * s->Dk);
  p->S = a.take<float>(heads * (N + 1) * s->Dk * s->Dv);
  p->all = a.take<double>(heads * N);
  return a.at - (char *)ws;
}
size_t backward_areas(const semicrf_linattn_shape_t *s, void *ws, DeltaArgs *p, float *part[3]) {
  Areas a = {(char *)ws};
  const int64_t heads = (int64_t)s->B * s->H, N = (s->T + L - 1) / L, rows = heads * s->T;
  p->D = a.take<float>(heads * N * s->Dk * s->Dv);
  part[0] = a.take<float>(s->Hq == s->H ? 0 : rows * s->Dk);
  part[1] = a.take<float>(s->Hk == s->H ? 0 : rows * s->Dk);
  part[2] = a.take<float>(s->Hv == s->H ? 0 : rows * s->Dv);
  return a.at - (char *)ws;
}

void fill(DeltaArgs *p, const semicrf_linattn_shape_t *s, const void *q, const void *k,
          const void *v, const float *log_decay, const float *beta, const int32_t *lengths) {
  p->q = {q, s->q_stride[0], s->q_stride[1], s->q_stride[2], s->H / s->Hq};
  p->k = {k, s->k_stride[0], s->k_stride[1], s->k_stride[2], s->H / s->Hk};
  p->v = {v, s->v_stride[0], s->v_stride[1], s->v_stride[2], s->H / s->Hv};
  p->log_decay = log_decay, p->beta = beta, p->lengths = lengths;
  p->scale = s->scale;
  p->B = s->B, p->T = s->T, p->H = s->H, p->Dk = s->Dk, p->Dv = s->Dv;
  p->N = (s->T + L - 1) / L;
}

unsigned chunk_grid(const DeltaArgs &p) { return (unsigned)((int64_t)p.B * p.H * p.N); }
unsigned scan_grid(const DeltaArgs &p) { return (unsigned)((int64_t)p.B * p.H * ((p.Dv + 15) / 16)); }
int host_up16(int n) { return (n + 15) / 16 * 16; }

template <typename T>
semicrf_status_t forward(const DeltaArgs &p, hipStream_t st) {
  const int dk = host_up16(p.Dk), dv = host_up16(p.Dv), kk = mat_floats(L, dk),
            vv = mat_floats(L, dv), ll = mat_floats(L, L);
  k_delta_prepare<T><<<chunk_grid(p), kThreads, 4 * (2 * kk + 2 * vv + 2 * ll), st>>>(p);
  k_delta_scan<<<scan_grid(p), kThreads, 0, st>>>(p);
  k_delta_out<T><<<chunk_grid(p), kThreads, 4 * (2 * kk + 2 * vv + 2 * ll), st>>>(p);
  return launch_status();
}
template <typename T>
semicrf_status_t backward(const DeltaArgs &p, hipStream_t st) {
  const int dk = host_up16(p.Dk), dv = host_up16(p.Dv), kk = mat_floats(L, dk),
            vv = mat_floats(L, dv), ll = mat_floats(L, L);
  k_delta_prepare_back<T><<<chunk_grid(p), kThreads, 4 * (2 * kk + 3 * vv + 2 * ll), st>>>(p);
  k_delta_scan<<<scan_grid(p), kThreads, 0, st>>>(p);
  if (p.dq || p.dk || p.dv || p.dg || p.db)
    k_delta_grads<T><<<chunk_grid(p), kThreads, 4 * (3 * kk + 5 * vv + 4 * ll), st>>>(p);
  return launch_status();
}

}  // namespace

}  // namespace semicrf

using namespace semicrf;

extern "C" {

semicrf_status_t semicrf_delta_workspace_size(const semicrf_linattn_shape_t *s, int backward,
                                              size_t *bytes) {
  if (!bytes) return SEMICRF_ERR_NULL;
  const semicrf_status_t e = check(s);
  if (e != SEMICRF_OK) return e;
  DeltaArgs p;
  float *part[3];
  *bytes = backward ? backward_areas(s, nullptr, &p, part) : forward_areas(s, nullptr, &p);
  return SEMICRF_OK;
}

semicrf_status_t semicrf_delta_fwd(const semicrf_linattn_shape_t *s, const void *q, const void *k,
                                   const void *v, const float *log_decay, const float *beta,
                                   const int32_t *lengths, const float *state_in, void *o,
                                   float *state_out, void *workspace, size_t workspace_bytes,
                                   void *stream) {
  if (!s || !q || !k || !v || !log_decay || !beta || !o) return SEMICRF_ERR_NULL;
  size_t need;
  const semicrf_status_t e = semicrf_delta_workspace_size(s, 0, &need);
  if (e != SEMICRF_OK) return e;
  if (!workspace || workspace_bytes < need) return SEMICRF_ERR_WORKSPACE;
  (void)hipGetLastError();
  DeltaArgs p = {};
  fill(&p, s, q, k, v, log_decay, beta, lengths);
  forward_areas(s, workspace, &p);
  p.state_in = state_in, p.state_out = state_out, p.o = o;
  p.bad = __builtin_nanf("");
  hipStream_t st = (hipStream_t)stream;
  switch (s->dtype) {
    case SEMICRF_F32: return forward<float>(p, st);
    case SEMICRF_BF16: return forward<bf16>(p, st);
    default: return forward<f16>(p, st);
  }
}

semicrf_status_t semicrf_delta_bwd(const semicrf_linattn_shape_t *s, const void *q, const void *k,
                                   const void *v, const float *log_decay, const float *beta,
                                   const int32_t *lengths, const void *saved, const void *grad_o,
                                   const float *grad_state, void *grad_q, void *grad_k,
                                   void *grad_v, float *grad_log_decay, float *grad_beta,
                                   float *grad_state_in, void *workspace, size_t workspace_bytes,
                                   void *stream) {
  if (!s || !q || !k || !v || !log_decay || !beta || !saved || !grad_o) return SEMICRF_ERR_NULL;
  size_t need;
  const semicrf_status_t e = semicrf_delta_workspace_size(s, 1, &need);
  if (e != SEMICRF_OK) return e;
  if (!workspace || workspace_bytes < need) return SEMICRF_ERR_WORKSPACE;
  (void)hipGetLastError();
  DeltaArgs p = {};
  float *part[3];
  fill(&p, s, q, k, v, log_decay, beta, lengths);
  forward_areas(s, const_cast<void *>(saved), &p);  // read only
  backward_areas(s, workspace, &p, part);
  p.go = grad_o, p.state_in = grad_state, p.state_out = grad_state_in, p.rev = 1;
  void *out[3] = {grad_q, grad_k, grad_v};
  const int heads[3] = {s->Hq, s->Hk, s->Hv};
  bool shared[3];
  for (int i = 0; i < 3; ++i) shared[i] = out[i] && heads[i] != s->H;
  p.dq = shared[0] ? part[0] : grad_q, p.part_q = shared[0];
  p.dk = shared[1] ? part[1] : grad_k, p.part_k = shared[1];
  p.dv = shared[2] ? part[2] : grad_v, p.part_v = shared[2];
  p.dg = grad_log_decay, p.db = grad_beta;
  hipStream_t st = (hipStream_t)stream;
  semicrf_status_t r;
  switch (s->dtype) {
    case SEMICRF_F32: r = backward<float>(p, st); break;
    case SEMICRF_BF16: r = backward<bf16>(p, st); break;
    default: r = backward<f16>(p, st);
  }
  for (int i = 0; i < 3 && r == SEMICRF_OK; ++i)
    if (shared[i])
      r = share_sum(s->dtype, (int64_t)s->B * s->T, s->H, heads[i], i == 2 ? s->Dv : s->Dk, part[i],
                    out[i], st);
  return r;
}

semicrf_status_t semicrf_delta_step(const semicrf_linattn_shape_t *s, const void *q, const void *k,
                                    const void *v, const float *log_decay, const float *beta,
                                    const int32_t *slots, int nslots, float *state, void *o,
                                    void *stream) {
  if (!s || !q || !k || !v || !log_decay || !beta || !state || !o) return SEMICRF_ERR_NULL;
  const semicrf_status_t e = check(s);
  if (e != SEMICRF_OK) return e;
  if (s->T != 1 || nslots < 1) return SEMICRF_ERR_SHAPE;
  (void)hipGetLastError();
  hipStream_t st = (hipStream_t)stream;
  switch (s->dtype) {
    case SEMICRF_F32:
      return step_type<float>(*s, q, k, v, log_decay, beta, slots, nslots, state, o, st);
    case SEMICRF_BF16:
      return step_type<bf16>(*s, q, k, v, log_decay, beta, slots, nslots, state, o, st);
    default: return step_type<f16>(*s, q, k, v, log_decay, beta, slots, nslots, state, o, st);
  }
}

}  // extern "C"
