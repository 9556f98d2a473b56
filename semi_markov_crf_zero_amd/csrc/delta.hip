// delta.hip -- the gated delta rule.
//
//   S_t = e^{g_t} (I - b_t k_t k_t^T) S_{t-1} + b_t k_t v_t^T,  o_t = scale S_t^T q_t
//
// In chunks of L positions.  With G the sums of g from the chunk's start, S the
// state before it, E = diag(e^G), D_ij = e^{G_i - G_j} (j <= i) and
//   m = strict lower part of D * (K K^T),  X = (I + diag(b) m)^-1 diag(b),
// what the positions write is U = X (V - E K S), and
//   O = scale (E Q S + (D * Q K^T) U),  S' = e^{G_L} S + Kh^T U,  Kh = diag(e^{G_L - G}) K.
//   k_delta_inverse   X of each chunk, side by side;
//   k_delta_chunks    the chunks of a sequence one after another, products on the
//                     matrix cores, S in accumulators.
// Backward, with P = scale D * Q K^T and dS' the gradient of the state after a chunk:
//   dU = P^T dO + Kh dS',  dR = X^T dU,  dV = dR,
//   dS = e^{G_L} dS' + scale (E Q)^T dO - (E K)^T dR
//   dP = scale D * (dO U^T),  dM = -(strict lower part of D) * (dR U^T)
//   dQ = scale E dO S^T + dP K
//   dK = (dM K - E dR S^T) + (dP^T Q + dM^T K + diag(e^{G_L - G}) U dS'^T)
//   db_i = (dR_i / b_i) . (U_i / b_i)
// and the gradient of a decay from what crosses its position,
//   a_i = q_i . (scale E dO S^T)_i - k_i . (E dR S^T)_i    what i asks of the state,
//   e_j = k_j . (diag(e^{G_L - G}) U dS'^T)_j              what j gives to the state after,
//   W_ij = dP_ij q_i . k_j + dM_ij k_i . k_j               what j gives to i,
//   dg_t = sum_{i >= t} a_i + sum_{j < t} e_j + sum_{i >= t > j} W_ij + e^{G_L} S . dS',
// all of which has the factor e^{g_t}: a strong decay's gradient, as small as that, keeps its
// digits (as sums of q . dq and k . dk, in which terms on one side of t cancel, it had none).
//   k_delta_back      dS', dR and dV, the chunks one after another from the last;
//   k_delta_grads     the rest, chunks side by side.
//
// Long sequences are cut into segments so that a few heads fill the GPU: what a
// segment makes of the state before it is phi S + sum, both from one walk
// (k_delta_chunks, composing) with phi's columns started from I; k_delta_scan joins the
// segments, and each is walked from its own state.  The backward pass has its own
// sums and phi^T.
//
// b = 0 would make the quotient in db 0 / 0: it counts as 2^-64, whose writes
// are below any rounding.  e^g below float32's range counts as e^-200.
// G is summed in float64 and kept in two floats: no quotient of decays is formed.
#include "delta_kernels.h"

namespace semicrf {

namespace {

constexpr int64_t kMaxThreads = 0xffffffff;  // of a grid
constexpr int kMaxHead = 128;
constexpr int kScanThreads = 256;

// X <- phi X + sum over the segments, 16 columns a workgroup of four waves; X after
// segment s takes the place of its sum.  REV: from the last segment on, with phi^T.  A
// wave has DK / 64 tiles of rows; X is read by all from LDS, by columns.  A step is
// 500 cycles of one matrix product after the other (DK = 64) and loads take 2000:
// they are AHEAD steps ahead.  127 steps of four heads of 64: 105 us; with a branch for
// rows that are no multiple of 4, 260 (the compiler then waits for every load).
template <int DK, bool REV>
__global__ __launch_bounds__(kScanThreads) void k_delta_scan(DeltaArgs p) {
  constexpr int MT = DK / 16, MW = (MT + 3) / 4, LD = DK + 4, AHEAD = DK <= 64 ? 4 : 2;
  __shared__ alignas(16) float xs[2][16 * LD];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, g = lane >> 4, l16 = lane & 15;
  const int ct = (p.Dv + 15) / 16, c = blockIdx.x % ct * 16 + l16;
  const int64_t bh = blockIdx.x / ct, size = (int64_t)p.Dk * p.lv;
  const int steps = p.nseg - 1;
  f4 ahead[AHEAD][MW][MT], sums[AHEAD][MW];
  auto fetch = [&](int i, f4(&A)[MW][MT], f4(&sum)[MW]) {
    const int s = REV ? p.nseg - 1 - i : i;
    const auto phi = whole_range((REV ? p.phit : p.phi) + (bh * p.nseg + s) * p.Dk * p.lk);
    const auto add = whole_range(p.xs + (bh * p.nseg + s) * size);
#pragma unroll
    for (int a = 0; a < MW; ++a) {
      const int mt = w + 4 * a, row = 16 * mt + l16;
#pragma unroll
      for (int kt = 0; kt < MT; ++kt) {
        const int k = 16 * kt + 4 * g;
        const bool on = row < p.Dk && k < p.lk;
        A[a][kt] = __builtin_bit_cast(
            f4, __builtin_amdgcn_raw_buffer_load_b128(phi, on ? 4 * (row * p.lk + k) : -1, 0, 0));
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int d = 16 * mt + 4 * g + r;
        const bool on = d < p.Dk && c < p.lv;
        sum[a][r] = __builtin_bit_cast(
            float, __builtin_amdgcn_raw_buffer_load_b32(add, on ? 4 * (d * p.lv + c) : -1, 0, 0));
      }
    }
  };
#pragma unroll
  for (int n = 0; n < AHEAD; ++n)
    if (n < steps) fetch(n, ahead[n], sums[n]);
  for (int e = threadIdx.x; e < DK * 16; e += kScanThreads) {
    const int d = e / 16, col = blockIdx.x % ct * 16 + e % 16;
    xs[0][e % 16 * LD + d] =
        p.state_in && d < p.Dk && col < p.Dv ? p.state_in[(bh * p.Dk + d) * p.Dv + col] : 0.f;
  }
  __syncthreads();
  for (int i0 = 0; i0 < steps; i0 += AHEAD)
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) {
      const int i = i0 + n;
      if (i >= steps) break;
      const float *x = xs[i & 1];
      float *to = xs[(i & 1) ^ 1], *out = p.xs + (bh * p.nseg + (REV ? p.nseg - 1 - i : i)) * size;
      f4 y[MW];
#pragma unroll
      for (int a = 0; a < MW; ++a) y[a] = sums[n][a];
#pragma unroll
      for (int kt = 0; kt < MT; ++kt) {
        const f4 b = *reinterpret_cast<const f4 *>(x + l16 * LD + 16 * kt + 4 * g);
#pragma unroll
        for (int a = 0; a < MW; ++a)
#pragma unroll
          for (int r = 0; r < 4; ++r) y[a] = mfma32(ahead[n][a][kt][r], b[r], y[a]);
      }
      if (i + AHEAD < steps) fetch(i + AHEAD, ahead[n], sums[n]);
#pragma unroll
      for (int a = 0; a < MW; ++a) {
        const int mt = w + 4 * a;
        if (mt >= MT) continue;
        *reinterpret_cast<f4 *>(to + l16 * LD + 16 * mt + 4 * g) = y[a];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int d = 16 * mt + 4 * g + r;
          if (d < p.Dk && c < p.lv) out[d * p.lv + c] = y[a][r];
        }
      }
      __syncthreads();
    }
}

// One position: a workgroup per stream and head, a thread V neighbouring
// columns of R rows of the state, which stays in registers between the dot
// products with the key and its update; what the query reads of the new state
// follows from the old one: q . S' = q . S + (q . k) b (v - k . S).  Bound by the
// state's bytes: 256 streams of 16 heads of 128 x 128, 537 MB, 113 us a call, 4.8 TB/s;
// 4 streams of 4 heads of 64 x 64 6.5 us, a launch.
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


int64_t chunks_of(const semicrf_linattn_shape_t *s) {
  const int L = delta_chunk(delta_parts(s->dtype));
  return (s->T + (int64_t)L - 1) / L;
}

// Segments.  A chunk takes a walk about 6 us where it has a compute unit to itself,
// 9 where two share it (up to four waves each; more do not fit); with segments the
// walk that composes adds three quarters, and two launches and the scan 10 us and
// 0.4 a segment.  The number that this puts first, of those that give every compute
// unit 1, 2, ... walks over up to two rounds.  Measured: 32 sequences of 512 positions
// of 4 heads of 64, 73 us in one segment each, 78 in two; 1024 positions 115 us in one, 66 in four, 48 in eight;
// 2^20 positions 100 ms in one, 5.7 ms in 32, 2.4 in 128; four sequences of 20001 positions
// of 4 heads of 128 (one walk a compute unit) 538 us in 16, 597 in 32.
void segments(const semicrf_linattn_shape_t *s, int *nseg, int *seg) {
  const int NW = delta_waves(s->Dv), resident = NW <= 4 ? 2 : 1;
  const int64_t chunks = chunks_of(s), slots = 256 * resident;
  const int64_t walks = (int64_t)s->B * s->H * ((s->Dv + 16 * NW - 1) / (16 * NW));
  int64_t best_n = 1;
  double best = 0;
  for (int k = 0; k <= 2 * resident; ++k) {
    int64_t n = k ? 256 * k / walks : 1;
    if (n > chunks / 2) n = chunks / 2;
    if (n < 1) n = 1;
    const int64_t per = (chunks + n - 1) / n;
    n = (chunks + per - 1) / per;
    const int64_t all = walks * n;
    double us = (double)per * ((all + slots - 1) / slots) * (all > 256 && resident > 1 ? 9 : 6);
    if (n > 1) us = 1.75 * us + 10 + 0.4 * n;
    if (!k || us < best) best = us, best_n = n;
  }
  const int64_t per = (chunks + best_n - 1) / best_n;
  *seg = (int)per;
  *nseg = (int)((chunks + per - 1) / per);
}

semicrf_status_t check(const semicrf_linattn_shape_t *s) {
  if (!s) return SEMICRF_ERR_NULL;
  if (s->B < 1 || s->T < 1 || s->H < 1 || s->Hq < 1 || s->Hk < 1 || s->Hv < 1 || s->Dk < 1 ||
      s->Dv < 1 || s->H % s->Hq || s->H % s->Hk || s->H % s->Hv)
    return SEMICRF_ERR_SHAPE;
  if (s->T > 1 << 30) return SEMICRF_ERR_SHAPE;
  // the chunks' workgroups of 512 threads are the most: segments are few where heads
  // are many
  const int64_t heads = (int64_t)s->B * s->H, chunks = (s->T + 31) / 32;
  if (heads > kMaxThreads / (chunks * 512)) return SEMICRF_ERR_SHAPE;
  if (s->Dk > kMaxHead || s->Dv > kMaxHead) return SEMICRF_ERR_UNSUPPORTED;
  return dtype_ok(s->dtype) ? SEMICRF_OK : SEMICRF_ERR_ARG;
}

int up4(int n) { return (n + 3) / 4 * 4; }

// The workspaces' areas, each on 256 bytes.
struct Areas {
  char *at;
  float *take(int64_t n) {
    float *p = (float *)at;
    at += (n * sizeof(float) + 255) / 256 * 256;
    return p;
  }
};
// keep: what the backward pass reads again is left there.
size_t forward_areas(const semicrf_linattn_shape_t *s, void *ws, bool keep, DeltaArgs *p) {
  Areas a = {(char *)ws};
  const int L = delta_chunk(delta_parts(s->dtype));
  const int64_t heads = (int64_t)s->B * s->H, N = chunks_of(s);
  segments(s, &p->nseg, &p->seg);
  // a sequence of one chunk may be short
  p->ld = N > 1 || s->T > L - 16 ? L : (s->T + 15) / 16 * 16;
  p->X = a.take(heads * N * p->ld * p->ld);
  p->gates = a.take(heads * N * delta_gates(L));
  const int lk = up4(s->Dk), lv = up4(s->Dv);
  const int64_t parts = p->nseg > 1 ? heads * p->nseg * s->Dk : 0;
  p->phi = a.take(parts * lk);
  p->xs = a.take(parts * lv);
  p->phit = p->S = p->U = nullptr;
  if (keep) {
    p->phit = a.take(parts * lk);
    p->S = a.take(heads * N * s->Dv * lk);
    p->U = a.take(heads * N * s->Dv * L);
  }
  return a.at - (char *)ws;
}
size_t backward_areas(const semicrf_linattn_shape_t *s, void *ws, DeltaArgs *p, float *part[3]) {
  Areas a = {(char *)ws};
  const int L = delta_chunk(delta_parts(s->dtype));
  const int64_t heads = (int64_t)s->B * s->H, N = chunks_of(s), rows = heads * s->T;
  segments(s, &p->nseg, &p->seg);
  const int lk = up4(s->Dk), lv = up4(s->Dv);
  p->D = a.take(heads * N * s->Dv * lk);
  p->R = a.take(heads * N * s->Dv * L);
  p->xs = a.take(p->nseg > 1 ? heads * p->nseg * s->Dk * lv : 0);
  part[0] = a.take(s->Hq == s->H ? 0 : rows * s->Dk);
  part[1] = a.take(s->Hk == s->H ? 0 : rows * s->Dk);
  part[2] = a.take(s->Hv == s->H ? 0 : rows * s->Dv);
  return a.at - (char *)ws;
}

// Whether every row of a tensor is a whole number of aligned 16-byte pieces,
// and a chunk of rows within reach of a buffer descriptor.
bool aligned(const View &v, int D, int dtype) {
  const int size = elem_size(dtype), e = 16 / size;
  return (uintptr_t)v.p % 16 == 0 && D % e == 0 && v.sb % e == 0 && v.st % e == 0 &&
         v.sh % e == 0 && v.st >= 0 && (v.st * 64 + 256) * size < kRange;
}

void fill(DeltaArgs *p, const semicrf_linattn_shape_t *s, const void *q, const void *k,
          const void *v, const float *log_decay, const float *beta, const int32_t *lengths) {
  p->q = {q, s->q_stride[0], s->q_stride[1], s->q_stride[2], s->H / s->Hq};
  p->k = {k, s->k_stride[0], s->k_stride[1], s->k_stride[2], s->H / s->Hk};
  p->v = {v, s->v_stride[0], s->v_stride[1], s->v_stride[2], s->H / s->Hv};
  p->log_decay = log_decay, p->beta = beta, p->lengths = lengths;
  p->scale = s->scale;
  p->B = s->B, p->T = s->T, p->H = s->H, p->Dk = s->Dk, p->Dv = s->Dv;
  p->N = (int)chunks_of(s), p->lk = up4(s->Dk), p->lv = up4(s->Dv);
}

semicrf_status_t run(const DeltaArgs &p, int dtype, DeltaPass pass, hipStream_t st) {
  switch (dtype) {
    case SEMICRF_F32: return delta_f32(p, pass, st);
    case SEMICRF_BF16: return delta_bf16(p, pass, st);
    default: return delta_f16(p, pass, st);
  }
}
template <bool REV>
semicrf_status_t scan(const DeltaArgs &p, hipStream_t st) {
  const unsigned grid = (unsigned)((int64_t)p.B * p.H * ((p.Dv + 15) / 16));
  if (p.Dk <= 32)
    k_delta_scan<32, REV><<<grid, kScanThreads, 0, st>>>(p);
  else if (p.Dk <= 64)
    k_delta_scan<64, REV><<<grid, kScanThreads, 0, st>>>(p);
  else if (p.Dk <= 96)
    k_delta_scan<96, REV><<<grid, kScanThreads, 0, st>>>(p);
  else
    k_delta_scan<128, REV><<<grid, kScanThreads, 0, st>>>(p);
  return launch_status();
}

}  // namespace

}  // namespace semicrf

using namespace semicrf;

extern "C" {

semicrf_status_t semicrf_delta_workspace_size(const semicrf_linattn_shape_t *s, int pass,
                                              size_t *bytes) {
  if (!bytes) return SEMICRF_ERR_NULL;
  const semicrf_status_t e = check(s);
  if (e != SEMICRF_OK) return e;
  if (pass < SEMICRF_DELTA_FORWARD || pass > SEMICRF_DELTA_BACKWARD) return SEMICRF_ERR_ARG;
  DeltaArgs p;
  float *part[3];
  *bytes = pass == SEMICRF_DELTA_BACKWARD ? backward_areas(s, nullptr, &p, part)
                                          : forward_areas(s, nullptr, pass == SEMICRF_DELTA_KEEP, &p);
  return SEMICRF_OK;
}

semicrf_status_t semicrf_delta_fwd(const semicrf_linattn_shape_t *s, int keep, const void *q,
                                   const void *k, const void *v, const float *log_decay,
                                   const float *beta, const int32_t *lengths,
                                   const float *state_in, void *o, float *state_out,
                                   void *workspace, size_t workspace_bytes, void *stream) {
  if (!s || !q || !k || !v || !log_decay || !beta || !o) return SEMICRF_ERR_NULL;
  size_t need;
  semicrf_status_t e = semicrf_delta_workspace_size(
      s, keep ? SEMICRF_DELTA_KEEP : SEMICRF_DELTA_FORWARD, &need);
  if (e != SEMICRF_OK) return e;
  if (!workspace || workspace_bytes < need) return SEMICRF_ERR_WORKSPACE;
  (void)hipGetLastError();
  DeltaArgs p = {};
  fill(&p, s, q, k, v, log_decay, beta, lengths);
  forward_areas(s, workspace, keep, &p);
  p.state_in = state_in, p.state_out = state_out, p.o = o;
  p.bad = __builtin_nanf("");
  p.vec = aligned(p.q, p.Dk, s->dtype) && aligned(p.k, p.Dk, s->dtype) &&
          aligned(p.v, p.Dv, s->dtype) && (uintptr_t)o % 16 == 0;
  hipStream_t st = (hipStream_t)stream;
  e = run(p, s->dtype, DELTA_INVERSE, st);
  if (e == SEMICRF_OK && p.nseg > 1) {
    // the last segment's transition is of use to the backward pass only
    p.first = 0, p.count = keep ? p.nseg : p.nseg - 1;
    e = run(p, s->dtype, DELTA_COMPOSE, st);
    if (e == SEMICRF_OK) e = scan<false>(p, st);
  }
  p.first = 0, p.count = p.nseg;
  return e == SEMICRF_OK ? run(p, s->dtype, DELTA_FORWARD, st) : e;
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
  semicrf_status_t e = semicrf_delta_workspace_size(s, SEMICRF_DELTA_BACKWARD, &need);
  if (e != SEMICRF_OK) return e;
  if (!workspace || workspace_bytes < need) return SEMICRF_ERR_WORKSPACE;
  (void)hipGetLastError();
  DeltaArgs p = {};
  float *part[3];
  fill(&p, s, q, k, v, log_decay, beta, lengths);
  forward_areas(s, const_cast<void *>(saved), true, &p);  // read only
  backward_areas(s, workspace, &p, part);                 // xs its own
  p.go = grad_o, p.state_in = grad_state, p.state_out = grad_state_in;
  void *out[3] = {grad_q, grad_k, grad_v};
  const int heads[3] = {s->Hq, s->Hk, s->Hv};
  bool shared[3];
  for (int i = 0; i < 3; ++i) shared[i] = out[i] && heads[i] != s->H;
  p.dq = shared[0] ? part[0] : grad_q, p.part_q = shared[0];
  p.dk = shared[1] ? part[1] : grad_k, p.part_k = shared[1];
  p.dv = shared[2] ? part[2] : grad_v, p.part_v = shared[2];
  p.dg = grad_log_decay, p.db = grad_beta;
  const int64_t row = (int64_t)s->H * s->Dv;
  const View go = {grad_o, s->T * row, row, s->Dv, 1};
  p.vec = aligned(p.q, p.Dk, s->dtype) && aligned(p.k, p.Dk, s->dtype) &&
          aligned(go, p.Dv, s->dtype);
  p.vec_out = p.Dk % 4 == 0 && (uintptr_t)p.dq % 16 == 0 && (uintptr_t)p.dk % 16 == 0;
  hipStream_t st = (hipStream_t)stream;
  if (p.nseg > 1) {
    p.first = 1, p.count = p.nseg - 1;
    e = run(p, s->dtype, DELTA_COMPOSE_BACK, st);
    if (e == SEMICRF_OK) e = scan<true>(p, st);
  }
  p.first = 0, p.count = p.nseg;
  if (e == SEMICRF_OK) e = run(p, s->dtype, DELTA_BACK, st);
  if (e == SEMICRF_OK && (grad_q || grad_k || grad_log_decay || grad_beta))
    e = run(p, s->dtype, DELTA_GRADS, st);
  for (int i = 0; i < 3 && e == SEMICRF_OK; ++i)
    if (shared[i])
      e = share_sum(s->dtype, (int64_t)s->B * s->T, s->H, heads[i], i == 2 ? s->Dv : s->Dk, part[i],
                    out[i], st);
  return e;
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
