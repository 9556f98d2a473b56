// linattn.hip -- linear attention with a decay for each head.
//
//   S_t = e^g S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
//
// Every pass of the operator, forward or backward, is one form of the sum
//   out_i = sum_{j <= i} e^{g (i-j)} (a_i . b_j) c_j + e^{g (i + off)} X^T a_i
// over positions taken forwards or backwards:
//   o       (a, b, c) = (q, k, v), forwards, X = state_in;
//   grad_q  (grad_o, v, k), forwards, X = state_in^T;
//   grad_k  (v, grad_o, q), backwards, X = grad_state^T;
//   grad_v  (k, q, grad_o), backwards, X = grad_state;
// so one kernel serves all four.  It works in chunks of L positions:
//   P = (A B^T) * decay, lower triangle;  O = P C + decay (A X);
//   X <- e^{g L} X + (decay B)^T C,
// products on the matrix cores, X in float32 accumulators of the wave that
// owns its 16 columns, from the first chunk of a sequence to its last.
//
// Decays are e^{g n} with n >= 0 (at most 1 for g <= 0: no quotient of
// decays is ever formed), and e^{g 0} = 1 also for g = -inf.
//
// Read forwards, X enters position i with e^{g (i+1)} and a chunk adds c_j
// with e^{g (n-1-j)}; the gradient of a state, read backwards, enters with
// e^{g i'} and adds with e^{g (n-j')}: off = 1 or 0 moves one step of the
// decay from the reading to the adding side.
//
// Long sequences are cut into segments so that a few heads fill the GPU.  A
// segment's part of X does not depend on what came before: k_linattn_state
// sums it for each segment from X = 0, k_linattn_scan runs
//   X before segment s+1 = e^{g n_s} (X before segment s) + part of s
// over the segments, and k_linattn starts each one from its own X.  X^T is
// what the transposed pair adds up to, so the four passes need two sets of
// states: that of (k, v) forwards and that of (q, grad_o) backwards.
//
// The states' pass reads b and c once more, 3.2 GB in the place of 2.15 over
// 2^20 positions of 4 heads.  Without it a head would be one workgroup: 4 of
// 256 compute units, 389 ms in the place of 0.73.
//
// Positions past the length are not loaded (zeros stand in their place, so
// NaN there stays out) and their rows of the output are written as 0.
#include "linattn_kernels.h"

namespace semicrf {

namespace {
constexpr int kThreads = 256;
constexpr int64_t kMaxThreads = 0xffffffff;  // of a grid
}

// xs[s] from the part of segment s to X before segment s + 1, one element of
// X a thread.  191 segments of 4 heads of 64 x 64: 24 us, the latency of twelve
// rounds of sixteen loads.
__global__ __launch_bounds__(kThreads) void k_linattn_scan(LaArgs p) {
  const int64_t n = (int64_t)p.Da * p.Dc;
  const int64_t e = blockIdx.x * (int64_t)kThreads + threadIdx.x;
  if (e >= (int64_t)p.B * p.H * n) return;
  const int64_t bh = e / n;
  const int b = (int)(bh / p.H), h = (int)(bh % p.H);
  const int len = max(valid_length(p.lengths, b, p.T), 0);
  float *x = p.xs + bh * (p.nseg - 1) * n + e % n;
  // in float64: the same factor again and again (see Decays)
  double acc = p.x_in ? p.x_in[e] : 0.f;
  const double gd = p.log_decay[h], whole = exp(gd * p.seg);
  const int full = len / p.seg, left = len % p.seg;  // segments; positions of the one after
  const double rest = left ? exp(gd * left) : 1.0;
  // sixteen loads at a time, the next ones on their way: the sum is a chain,
  // the loads are not (past the end the last one again)
  constexpr int N = 16;
  const int last = p.nseg - 2;
  float part[N], next[N];
#pragma unroll
  for (int k = 0; k < N; ++k) next[k] = x[min(k, last) * n];
  for (int s0 = 0; s0 <= last; s0 += N) {
#pragma unroll
    for (int k = 0; k < N; ++k) part[k] = next[k];
#pragma unroll
    for (int k = 0; k < N; ++k) next[k] = x[min(s0 + N + k, last) * n];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int s = s0 + k;
      acc = (s < full ? whole : s == full ? rest : 1.0) * acc + part[k];
      if (s <= last) x[s * n] = (float)acc;
    }
  }
}

// Sum over the heads that share one: part [B*T][H][D] float32 to out
// [B*T][H / share][D].  A fixed order, no atomics; 100002 positions of four heads
// of 40 to two: 25 us.
template <typename T>
__global__ __launch_bounds__(256) void k_share_sum(const float *part, T *out, int64_t rows, int H,
                                                   int share, int D) {
  const int64_t n = rows * (H / share) * D;
  for (int64_t e = blockIdx.x * (int64_t)256 + threadIdx.x; e < n; e += (int64_t)gridDim.x * 256) {
    const int64_t rh = e / D;
    const float *s = part + rh * share * D + e % D;
    float x = 0.f;
    for (int i = 0; i < share; ++i) x += s[(int64_t)i * D];
    out[e] = (T)x;
  }
}

semicrf_status_t share_sum(int dtype, int64_t rows, int H, int heads, int D, const float *part,
                           void *out, hipStream_t st) {
  const int64_t n = rows * heads * D;
  const unsigned grid = (unsigned)(n < 256 * 8192 ? (n + 255) / 256 : 8192);
  const int share = H / heads;
  switch (dtype) {
    case SEMICRF_F32: k_share_sum<<<grid, 256, 0, st>>>(part, (float *)out, rows, H, share, D); break;
    case SEMICRF_BF16: k_share_sum<<<grid, 256, 0, st>>>(part, (bf16 *)out, rows, H, share, D); break;
    default: k_share_sum<<<grid, 256, 0, st>>>(part, (f16 *)out, rows, H, share, D);
  }
  return launch_status();
}

// One position: a workgroup per stream and head.  Bound by the state's bytes:
// 256 streams of 16 heads of 128 x 128, 537 MB, 114 us, 4.8 TB/s; 4 streams of
// 4 heads of 64 x 64 5.1 us, a launch.  The state is read and written once, V
// neighbouring columns and kStepRows rows of a thread in flight; thread t takes
// column group t % tpr of rows t / tpr, + groups, ...
constexpr int kStepRows = 8;
template <typename T, int V>
__global__ __launch_bounds__(256) void k_linattn_step(semicrf_linattn_shape_t s, const T *q,
                                                      const T *k, const T *v,
                                                      const float *log_decay,
                                                      const int32_t *slots, int nslots,
                                                      float *state, T *o) {
  __shared__ float qs[256], ks[256];
  __shared__ Pack<float, V> red[256];
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
  Pack<float, V> x[kStepRows];
  auto load = [&](int r) {
#pragma unroll
    for (int i = 0; i < kStepRows; ++i)
      if (r + i * groups < s.Dk)
        x[i] = *reinterpret_cast<const Pack<float, V> *>(S + (r + i * groups) * s.Dv + c);
  };
  if (on) load(r0);
  if ((int)threadIdx.x < s.Dk) {
    qs[threadIdx.x] =
        (float)q[b * s.q_stride[0] + h / (s.H / s.Hq) * s.q_stride[2] + threadIdx.x] * s.scale;
    ks[threadIdx.x] = (float)k[b * s.k_stride[0] + h / (s.H / s.Hk) * s.k_stride[2] + threadIdx.x];
  }
  // the decay in two floats: one would put its own rounding into a state that
  // lives for thousands of steps at each of them, always with the same sign
  const double decay = exp((double)log_decay[h]);
  const float d = (float)decay, dl = (float)(decay - d);
  float vc[V];
  Pack<float, V> acc;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    vc[i] = on ? (float)vb[c + i] : 0.f;
    acc.v[i] = 0.f;
  }
  __syncthreads();
  if (on)
    for (int r = r0; r < s.Dk; r += kStepRows * groups) {
      if (r != r0) load(r);
#pragma unroll
      for (int i = 0; i < kStepRows; ++i) {
        const int row = r + i * groups;
        if (row < s.Dk) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float y = x[i].v[e];
            const float add = fmaf(ks[row], vc[e], fabsf(y) < INFINITY ? dl * y : 0.f);
            x[i].v[e] = fmaf(d, y, add);
            acc.v[e] += qs[row] * x[i].v[e];
          }
          *reinterpret_cast<Pack<float, V> *>(S + row * s.Dv + c) = x[i];
        }
      }
    }
  red[threadIdx.x] = acc;
  __syncthreads();
  if (r0 == 0) {
    for (int g = 1; g < groups; ++g)
#pragma unroll
      for (int e = 0; e < V; ++e) acc.v[e] += red[g * tpr + threadIdx.x].v[e];
#pragma unroll
    for (int e = 0; e < V; ++e) ob[c + e] = (T)acc.v[e];
  }
}

namespace {

// Whether every row of a tensor is a whole number of aligned 16-byte pieces,
// and a chunk of rows within reach of a buffer descriptor.
bool aligned(const View &v, int D, int dtype) {
  const int size = elem_size(dtype), e = 16 / size;
  return (uintptr_t)v.p % 16 == 0 && D % e == 0 && v.sb % e == 0 && v.st % e == 0 &&
         v.sh % e == 0 && v.st >= 0 && (v.st * 64 + 256) * size < kRange;
}

semicrf_status_t launch_any(const LaArgs &p, int dtype, bool vec, bool f32_out, bool states,
                            hipStream_t st) {
  switch (dtype) {
    case SEMICRF_F32: return linattn_f32(p, vec, f32_out, states, st);
    case SEMICRF_BF16: return linattn_bf16(p, vec, f32_out, states, st);
    default: return linattn_f16(p, vec, f32_out, states, st);
  }
}

// The pass over the chunks.  f32_out: the output is float32 whatever the
// tensors are (parts of the gradient of a shared head).
semicrf_status_t launch_linattn(const LaArgs &p, int dtype, bool f32_out, hipStream_t st) {
  const bool vec = aligned(p.a, p.Da, dtype) && aligned(p.b, p.Da, dtype) &&
                   aligned(p.c, p.Dc, dtype) && (uintptr_t)p.out % 16 == 0;
  return launch_any(p, dtype, vec, f32_out, false, st);
}

// The segments' states of a pair (b, c) in p.xs.
semicrf_status_t launch_states(const LaArgs &p, int dtype, hipStream_t st) {
  if (p.nseg < 2) return SEMICRF_OK;
  const bool vec = aligned(p.b, p.Da, dtype) && aligned(p.c, p.Dc, dtype);
  const semicrf_status_t e = launch_any(p, dtype, vec, false, true, st);
  if (e != SEMICRF_OK) return e;
  const int64_t n = (int64_t)p.B * p.H * p.Da * p.Dc;
  k_linattn_scan<<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, st>>>(p);
  return launch_status();
}

// Workgroups of the chunk kernel a compute unit holds.
int resident(int Da, int Dc, int dtype) {
  const int NP = linattn_parts(dtype), DA = Da <= 128 ? (Da + 31) / 32 * 32 : 256;
  const int NW = DA > 128 ? 4 : linattn_waves(Dc);
  const int by_lds = linattn_by_lds(NP, DA, NW), occ = linattn_occupancy(NP, DA, NW);
  const int by_waves = NW < 4 ? 4 * occ / NW : occ / ((NW + 3) / 4);
  const int n = by_lds < by_waves ? by_lds : by_waves;
  return n < 1 ? 1 : n;
}

// Segments.  A chunk takes a workgroup about 3 us where it has a compute unit
// to itself and 1 us more for each that shares it (bfloat16, 64 wide); with
// segments the states' pass adds about 0.45 of that and two launches 10 us.
// The number that this puts first, of those that give every compute unit 1,
// 2, ... workgroups over up to two rounds; four chunks at least in each.
void segments(const semicrf_linattn_shape_t *s, int *nseg, int *seg) {
  const int r1 = resident(s->Dk, s->Dv, s->dtype), r2 = resident(s->Dv, s->Dk, s->dtype);
  const int res = r1 < r2 ? r1 : r2, L = 64;
  const int64_t heads = (int64_t)s->B * s->H, chunks = (s->T + L - 1) / L;
  int64_t best_n = 1;
  double best = 0;
  for (int k = 0; k <= 2 * res; ++k) {
    int64_t n = k ? 256 * k / heads : 1;
    if (n > chunks / 4) n = chunks / 4;
    if (n < 1) n = 1;
    const int64_t per = (chunks + n - 1) / n, slots = 256 * res;
    n = (chunks + per - 1) / per;
    const int64_t full = heads * n / slots, left = heads * n % slots;
    double us = (double)per * (full * (2 + res) + (left ? 2 + (left + 255) / 256 : 0));
    if (n > 1) us = 1.45 * us + 10;
    if (!k || us < best) best = us, best_n = n;
  }
  const int64_t per = (chunks + best_n - 1) / best_n;
  *seg = (int)(per * L);
  *nseg = (int)((chunks + per - 1) / per);
}

size_t state_bytes(const semicrf_linattn_shape_t *s) {
  int nseg, seg;
  segments(s, &nseg, &seg);
  return ((size_t)s->B * s->H * (nseg - 1) * s->Dk * s->Dv * sizeof(float) + 255) / 256 * 256;
}

template <typename T>
semicrf_status_t launch_step(const semicrf_linattn_shape_t &s, const void *q, const void *k,
                             const void *v, const float *log_decay, const int32_t *slots,
                             int nslots, float *state, void *o, void *stream) {
  const unsigned grid = (unsigned)s.B * s.H;
  hipStream_t st = (hipStream_t)stream;
  if (s.Dv % 4 == 0 && (uintptr_t)state % 16 == 0)
    k_linattn_step<T, 4><<<grid, 256, 0, st>>>(s, (const T *)q, (const T *)k, (const T *)v,
                                               log_decay, slots, nslots, state, (T *)o);
  else
    k_linattn_step<T, 1><<<grid, 256, 0, st>>>(s, (const T *)q, (const T *)k, (const T *)v,
                                               log_decay, slots, nslots, state, (T *)o);
  return launch_status();
}

// Threads for the Dc columns of a head: tiles of 16 a wave, as launch_nw has
// them or by fours.
int column_threads(int Dc) {
  int most = 0;
  for (int NW : {linattn_waves(Dc), 4}) {
    const int n = (Dc + 16 * NW - 1) / (16 * NW) * 64 * NW;
    if (n > most) most = n;
  }
  return most;
}

semicrf_status_t check(const semicrf_linattn_shape_t *s) {
  if (!s) return SEMICRF_ERR_NULL;
  if (s->B < 1 || s->T < 1 || s->H < 1 || s->Hq < 1 || s->Hk < 1 || s->Hv < 1 || s->Dk < 1 ||
      s->Dv < 1 || s->H % s->Hq || s->H % s->Hk || s->H % s->Hv)
    return SEMICRF_ERR_SHAPE;
  if (s->T > 1 << 30) return SEMICRF_ERR_SHAPE;
  const int64_t heads = (int64_t)s->B * s->H;
  if (heads > kMaxThreads / 256) return SEMICRF_ERR_SHAPE;  // the least a head takes
  if (s->Dk > 256 || s->Dv > 256) return SEMICRF_ERR_UNSUPPORTED;
  if (!dtype_ok(s->dtype)) return SEMICRF_ERR_ARG;
  // segments are few where heads are many, so this counts the chunk kernel's
  // threads; the scan has one for each element of a state
  int nseg, seg;
  segments(s, &nseg, &seg);
  if (heads * nseg * column_threads(s->Dk > s->Dv ? s->Dk : s->Dv) > kMaxThreads ||
      (nseg > 1 && heads * s->Dk * s->Dv + kThreads > kMaxThreads))
    return SEMICRF_ERR_SHAPE;
  return SEMICRF_OK;
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Parts of a shared head's gradient: one float32 row a head.
size_t share_bytes(const semicrf_linattn_shape_t *s, int heads, int D) {
  return heads == s->H ? 0 : align256((size_t)s->B * s->T * s->H * D * sizeof(float));
}

View view(const void *p, const int64_t *st, int share) { return {p, st[0], st[1], st[2], share}; }

}  // namespace

}  // namespace semicrf

using namespace semicrf;

extern "C" {

semicrf_status_t semicrf_linattn_workspace_size(const semicrf_linattn_shape_t *s, int backward,
                                                size_t *bytes) {
  if (!bytes) return SEMICRF_ERR_NULL;
  const semicrf_status_t e = check(s);
  if (e != SEMICRF_OK) return e;
  *bytes = state_bytes(s);
  if (backward) {  // one area: each gradient's parts are summed before the next one's are written
    size_t most = 0;
    for (const size_t n : {share_bytes(s, s->Hq, s->Dk), share_bytes(s, s->Hk, s->Dk),
                           share_bytes(s, s->Hv, s->Dv)})
      if (n > most) most = n;
    *bytes += most;
  }
  return SEMICRF_OK;
}

semicrf_status_t semicrf_linattn_fwd(const semicrf_linattn_shape_t *s, const void *q,
                                     const void *k, const void *v, const float *log_decay,
                                     const int32_t *lengths, const float *state_in, void *o,
                                     float *state_out, void *workspace, size_t workspace_bytes,
                                     void *stream) {
  if (!s || !q || !k || !v || !log_decay || !o) return SEMICRF_ERR_NULL;
  size_t need;
  const semicrf_status_t e = semicrf_linattn_workspace_size(s, 0, &need);
  if (e != SEMICRF_OK) return e;
  if (need && (!workspace || workspace_bytes < need)) return SEMICRF_ERR_WORKSPACE;
  (void)hipGetLastError();
  LaArgs p = {};
  p.a = view(q, s->q_stride, s->H / s->Hq);
  p.b = view(k, s->k_stride, s->H / s->Hk);
  p.c = view(v, s->v_stride, s->H / s->Hv);
  p.log_decay = log_decay;
  p.lengths = lengths;
  p.x_in = state_in;
  p.x_out = state_out;
  p.out = o;
  p.off = 1;
  p.bad = __builtin_nanf("");
  p.p_scale = p.x_scale = s->scale;
  p.add_scale = 1.f;
  p.B = s->B, p.T = s->T, p.H = s->H, p.Da = s->Dk, p.Dc = s->Dv;
  p.xs = (float *)workspace;
  segments(s, &p.nseg, &p.seg);
  const semicrf_status_t r = launch_states(p, s->dtype, (hipStream_t)stream);
  return r == SEMICRF_OK ? launch_linattn(p, s->dtype, false, (hipStream_t)stream) : r;
}

semicrf_status_t semicrf_linattn_bwd(const semicrf_linattn_shape_t *s, const void *q,
                                     const void *k, const void *v, const float *log_decay,
                                     const int32_t *lengths, const float *state_in,
                                     const void *states, const void *grad_o,
                                     const float *grad_state, void *grad_q, void *grad_k,
                                     void *grad_v, float *grad_state_in, void *workspace,
                                     size_t workspace_bytes, void *stream) {
  if (!s || !q || !k || !v || !log_decay || !grad_o) return SEMICRF_ERR_NULL;
  size_t need;
  semicrf_status_t e = semicrf_linattn_workspace_size(s, 1, &need);
  if (e != SEMICRF_OK) return e;
  if (need && (!workspace || workspace_bytes < need)) return SEMICRF_ERR_WORKSPACE;
  (void)hipGetLastError();
  hipStream_t st = (hipStream_t)stream;
  float *const xs = (float *)workspace;
  float *const part = (float *)((char *)workspace + state_bytes(s));
  const View vq = view(q, s->q_stride, s->H / s->Hq), vk = view(k, s->k_stride, s->H / s->Hk),
             vv = view(v, s->v_stride, s->H / s->Hv);
  const int64_t row = (int64_t)s->H * s->Dv;
  const View vg = {grad_o, s->T * row, row, s->Dv, 1};
  LaArgs p = {};
  p.log_decay = log_decay;
  p.lengths = lengths;
  p.p_scale = s->scale;
  p.B = s->B, p.T = s->T, p.H = s->H;
  p.xs = xs;
  segments(s, &p.nseg, &p.seg);
  auto set = [&](View a, View b, View c, int Da, int Dc) {
    p.a = a, p.b = b, p.c = c, p.Da = Da, p.Dc = Dc;
  };
  auto run = [&](void *out, int heads) {
    const bool shared = out && heads != s->H;
    p.out = shared ? part : out;
    semicrf_status_t r = launch_linattn(p, s->dtype, shared, st);
    if (r == SEMICRF_OK && shared)
      r = share_sum(s->dtype, (int64_t)s->B * s->T, s->H, heads, p.Dc, part, out, st);
    return r;
  };
  if (grad_q) {
    p.x_in = state_in, p.rev = 0, p.off = 1;
    p.x_scale = s->scale, p.add_scale = 1.f;
    set(vq, vk, vv, s->Dk, s->Dv);
    if (states) {
      p.xs = (float *)states;  // read only
    } else {
      e = launch_states(p, s->dtype, st);
      if (e != SEMICRF_OK) return e;
    }
    p.x_tr = 1;
    set(vg, vv, vk, s->Dv, s->Dk);
    e = run(grad_q, s->Hq);
    if (e != SEMICRF_OK) return e;
  }
  p.xs = xs;
  p.rev = 1, p.off = 0, p.x_scale = 1.f, p.add_scale = s->scale, p.x_in = grad_state, p.x_tr = 0;
  if (grad_k || grad_v || grad_state_in) {
    set(vk, vq, vg, s->Dk, s->Dv);
    e = launch_states(p, s->dtype, st);
    if (e != SEMICRF_OK) return e;
  }
  if (grad_v || grad_state_in) {
    p.x_out = grad_state_in;
    e = run(grad_v, s->Hv);
    if (e != SEMICRF_OK) return e;
  }
  if (grad_k) {
    p.x_tr = 1, p.x_out = nullptr;
    set(vv, vg, vq, s->Dv, s->Dk);
    e = run(grad_k, s->Hk);
  }
  return e;
}

semicrf_status_t semicrf_linattn_step(const semicrf_linattn_shape_t *s, const void *q,
                                      const void *k, const void *v, const float *log_decay,
                                      const int32_t *slots, int nslots, float *state, void *o,
                                      void *stream) {
  if (!s || !q || !k || !v || !log_decay || !state || !o) return SEMICRF_ERR_NULL;
  const semicrf_status_t e = check(s);
  if (e != SEMICRF_OK) return e;
  if (s->T != 1 || nslots < 1) return SEMICRF_ERR_SHAPE;
  (void)hipGetLastError();
  switch (s->dtype) {
    case SEMICRF_F32:
      return launch_step<float>(*s, q, k, v, log_decay, slots, nslots, state, o, stream);
    case SEMICRF_BF16:
      return launch_step<bf16>(*s, q, k, v, log_decay, slots, nslots, state, o, stream);
    default: return launch_step<f16>(*s, q, k, v, log_decay, slots, nslots, state, o, stream);
  }
}

}  // extern "C"
