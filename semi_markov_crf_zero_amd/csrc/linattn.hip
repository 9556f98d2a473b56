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
// Positions past the length are loaded as zeros (a select, so NaN there
// stays out) and their rows of the output are written as 0.
#include "encoder.h"

namespace semicrf {

namespace {

typedef f32x4_t f4;
typedef float f2 __attribute__((ext_vector_type(2)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef s4 __attribute__((address_space(3))) lds_s4;

typedef unsigned u4 __attribute__((ext_vector_type(4)));

constexpr int kRange = 0x7fffffff;      // bytes a buffer descriptor reaches
constexpr int kRawBuffer = 0x00027000;  // its last word: raw 32-bit data
constexpr int kThreads = 256;  // four waves, 16 output columns each
constexpr int kCols = 64;      // output columns of a workgroup

// One tensor as the kernel reads it: element strides of batch, position and
// head, and how many heads of the call share one of its heads.
struct View {
  const void *p;
  int64_t sb, st, sh;
  int share;
};

struct LaArgs {
  View a, b, c;
  const float *log_decay;
  const int32_t *lengths;
  const float *x_in;  // [B][H][Da][Dc], or [B][H][Dc][Da] if x_tr; or NULL
  float *x_out;       // [B][H][Da][Dc]; or NULL
  float *xs;          // [B][H][nseg - 1], as x_in: before segments 1..
  int nseg, seg;      // segments, positions of one (a multiple of the chunk)
  void *out;          // [B][T][H][Dc] contiguous; or NULL
  int x_tr;
  int rev, off;
  float bad;  // what a sequence without a valid length gets: NaN, or 0 for gradients
  float p_scale, x_scale, add_scale;  // of P, of A X, of what a chunk adds to X
  int B, T, H, Da, Dc;
  int ctiles;
};

// A fragment is a lane's part of one operand over a 32-wide stretch of the
// contraction: indices {4g + r} and {16 + 4g + r} (g = lane / 16, r < 4) of
// row or column lane % 16.  That is how two neighbouring 16x16 accumulator
// tiles hold their rows, so X goes from accumulators to operands in place.
template <typename T>
struct Frag;
template <>
struct Frag<bf16> {
  bf8 v;
};
template <>
struct Frag<float> {
  float v[8];
};

__device__ __forceinline__ f4 mma(const Frag<bf16> &a, const Frag<bf16> &b, f4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ f4 mma(const Frag<float> &a, const Frag<float> &b, f4 c) {
#pragma unroll
  for (int r = 0; r < 8; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[r], b.v[r], c, 0, 0, 0);
  return c;
}

// Fragment of a row whose contraction index is contiguous: p at index 4g.
__device__ __forceinline__ Frag<bf16> frag_row(const bf16 *p) {
  typedef __bf16 bf4 __attribute__((ext_vector_type(4)));
  const bf4 lo = *reinterpret_cast<const bf4 *>(p), hi = *reinterpret_cast<const bf4 *>(p + 16);
  return {__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7)};
}
__device__ __forceinline__ Frag<float> frag_row(const float *p) {
  const f4 lo = *reinterpret_cast<const f4 *>(p), hi = *reinterpret_cast<const f4 *>(p + 16);
  return {{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]}};
}

// Fragment of a column whose contraction index runs over LDS rows: the tile
// of 32 rows x 16 columns at p (row stride ld).  16-bit elements come through
// the transposing LDS read: in each group of 16 lanes, lane i names 4
// elements of row i / 4 and gets column i of the four rows.
__device__ __forceinline__ Frag<bf16> frag_col(const bf16 *p, int ld, int lane) {
  const int g = lane >> 4, i = lane & 15;
  const bf16 *q = p + (4 * g + (i >> 2)) * ld + (i & 3) * 4;
  const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(q));
  const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(q + 16 * ld));
  return {__builtin_bit_cast(bf8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7))};
}
__device__ __forceinline__ Frag<float> frag_col(const float *p, int ld, int lane) {
  const float *q = p + (4 * (lane >> 4)) * ld + (lane & 15);
  Frag<float> f;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    f.v[r] = q[r * ld];
    f.v[4 + r] = q[(16 + r) * ld];
  }
  return f;
}

// Float32 values as a sum of N fragments of the operand type.  A bfloat16
// part leaves at most 2^-8 of what it was given: two parts of P and X leave
// 2^-16, far below the rounding of a 16-bit output (2^-8 or 2^-11); three
// parts of what is added to X leave 2^-24, so the float32 state is as exact
// as one summed from float32 products.
template <typename T>
struct Parts;
template <>
struct Parts<bf16> {
  static constexpr int kRead = 2, kAdd = 3;
};
template <>
struct Parts<float> {
  static constexpr int kRead = 1, kAdd = 1;
};
// Two neighbours at a time: one instruction rounds a pair.
template <int N>
__device__ __forceinline__ void split(const float *x, Frag<bf16> *f) {
  f2 r[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) r[e] = f2{x[2 * e], x[2 * e + 1]};
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const b2 y = __builtin_convertvector(r[e], b2);
      f[n].v[2 * e] = y[0];
      f[n].v[2 * e + 1] = y[1];
      r[e] -= __builtin_convertvector(y, f2);
    }
}
template <int N>
__device__ __forceinline__ void split(const float *x, Frag<float> *f) {
#pragma unroll
  for (int e = 0; e < 8; ++e) f[0].v[e] = x[e];
}
// Four float32 values rounded to the type; x keeps what is left of them.
__device__ __forceinline__ void part4(f4 &x, Pack<bf16, 4> &y) {
  const f2 lo = {x[0], x[1]}, hi = {x[2], x[3]};
  const b2 a = __builtin_convertvector(lo, b2), b = __builtin_convertvector(hi, b2);
  const f2 ra = lo - __builtin_convertvector(a, f2), rb = hi - __builtin_convertvector(b, f2);
  x = f4{ra[0], ra[1], rb[0], rb[1]};
  y = {{a[0], a[1], b[0], b[1]}};
}
template <typename T>
__device__ __forceinline__ void part4(f4 &x, Pack<T, 4> &y) {
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    y.v[r] = (T)x[r];
    x[r] -= (float)y.v[r];
  }
}
__device__ __forceinline__ void values(const Frag<bf16> &f, float *x) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = (float)f.v[e];
}
__device__ __forceinline__ void values(const Frag<float> &f, float *x) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = f.v[e];
}

// A tile of a chunk: L rows of W columns, zeros past row n and past column
// D.  fetch() issues a thread's 16-byte loads into registers while the chunk
// before is worked on, put() writes them to LDS.  The loads go through a
// buffer descriptor whose range a row that is not wanted lies past, so it
// reads 0 without a branch, whatever memory holds there.
template <typename T, typename CT, int W, int L>
struct Tile {
  static constexpr int VE = 16 / sizeof(T), per = W / VE, NV = L * per / kThreads;
  static constexpr int ld = W + 16 / sizeof(CT);
  u4 r[NV];

  // row i of the tile is row `row0 + step * i` (step +-1) from src, rows st
  // elements apart
  __device__ __forceinline__ void fetch(const T *src, int st, int D, int n, int row0, int step,
                                        int col0) {
    const int c = threadIdx.x % per * VE, i0 = threadIdx.x / per;
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)src, 0, kRange, kRawBuffer);
    const bool col = col0 + c < D;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = i0 + k * (kThreads / per);
      const int at = ((row0 + step * i) * st + col0 + c) * (int)sizeof(T);
      r[k] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, i < n && col ? at : -1, 0, 0);
    }
  }
  __device__ __forceinline__ void put(CT *lds) const {
    const int c = threadIdx.x % per * VE, i0 = threadIdx.x / per;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const Pack<T, VE> y = __builtin_bit_cast(Pack<T, VE>, r[k]);
      Pack<CT, VE> x;
#pragma unroll
      for (int e = 0; e < VE; ++e) x.v[e] = (CT)y.v[e];
      CT *to = lds + (i0 + k * (kThreads / per)) * ld + c;
#pragma unroll
      for (int e = 0; e < VE; e += 16 / sizeof(CT))
        *reinterpret_cast<Pack<CT, 16 / sizeof(CT)> *>(to + e) =
            *reinterpret_cast<const Pack<CT, 16 / sizeof(CT)> *>(x.v + e);
    }
  }
};

// The same without the alignment 16-byte loads need: element by element,
// straight to LDS.
template <typename T, typename CT, int W, int L>
__device__ __forceinline__ void stage(CT *lds, const T *src, int64_t st, int D, int n, int col0) {
  constexpr int ld = W + 16 / sizeof(CT);
  for (int e = threadIdx.x; e < L * W; e += kThreads) {
    const int i = e / W, d = e % W;
    lds[i * ld + d] = i < n && col0 + d < D ? (CT)(float)src[i * st + col0 + d] : (CT)0.f;
  }
}

// The decays a workgroup uses, with the pass's factors in them; entries of
// negative powers are 0, so masked places need no branch.
template <int L>
struct Decays {
  float x[L + 1];       // e^{g n}: of X over n positions
  float p[2 * L];       // p_scale e^{g (n - L)}: of P
  float read[L];        // x_scale e^{g (i + off)}: of X read by position i
  float add[2 * L + 1]; // add_scale e^{g (n - L)}: of what a position adds to X

  __device__ __forceinline__ void fill(const LaArgs &a, float g) {
    auto e = [&](int n) { return n < 0 ? 0.f : n ? expf(g * n) : 1.f; };
    for (int n = threadIdx.x; n < 2 * L + 1; n += kThreads) {
      add[n] = a.add_scale * e(n - L);
      if (n <= L) x[n] = e(n);
      if (n < 2 * L) p[n] = a.p_scale * e(n - L);
      if (n < L) read[n] = a.x_scale * e(n + a.off);
    }
  }
};

// X <- e^{g n} X + sum_j e^{g (n - off - j)} b_j c_j^T over a staged chunk:
// B in rows of lda, this wave's 16 columns of C in fragments.
template <typename CT, int KB, int L>
__device__ __forceinline__ void add_chunk(f4 *X, const CT *Bm, const Frag<CT> *C,
                                          const Decays<L> &dec, int n, int off, int lane) {
  constexpr int lda = 32 * KB + 16 / sizeof(CT);
  constexpr int NA = Parts<CT>::kAdd;
  const float *add = dec.add + L + n - off - 4 * (lane >> 4);
#pragma unroll
  for (int k = 0; k < 2 * KB; ++k)
#pragma unroll
    for (int r = 0; r < 4; ++r) X[k][r] *= dec.x[n];
#pragma unroll
  for (int jb = 0; jb < L / 32; ++jb) {
    float x[8];
    values(C[jb], x);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= add[-(32 * jb + (e & 3) + (e >> 2) * 16)];
    Frag<CT> cf[NA];
    split<NA>(x, cf);
#pragma unroll
    for (int k = 0; k < 2 * KB; ++k) {
      const Frag<CT> bf = frag_col(Bm + 32 * jb * lda + 16 * k, lda, lane);
#pragma unroll
      for (int s = 0; s < NA; ++s) X[k] = mma(bf, cf[s], X[k]);
    }
  }
}

}  // namespace

// Parts of X: one workgroup per segment but the last, kCols columns.  Writes
// xs[segment]; a segment past the length leaves zeros.
template <typename T, typename CT, int DA, int L, bool VEC>
__global__ __launch_bounds__(kThreads) void k_linattn_state(LaArgs p) {
  constexpr int pad = 16 / sizeof(CT);
  constexpr int lda = DA + pad, ldc = kCols + pad, KB = DA / 32;
  __shared__ alignas(16) CT Bm[L * lda + L * ldc];
  CT *const C = Bm + L * lda;
  __shared__ Decays<L> dec;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, g = lane >> 4, l16 = lane & 15;
  const int ct = blockIdx.x % p.ctiles, s0 = blockIdx.x / p.ctiles % (p.nseg - 1);
  const int bh = blockIdx.x / p.ctiles / (p.nseg - 1);
  const int h = bh % p.H, b = bh / p.H, c0 = ct * kCols;
  const int len = max(valid_length(p.lengths, b, p.T), 0);
  const int lo = s0 * p.seg, hi = min(len, lo + p.seg);
  dec.fill(p, p.log_decay[h]);
  const T *bb = (const T *)p.b.p + (int64_t)b * p.b.sb + (int64_t)(h / p.b.share) * p.b.sh;
  const T *c = (const T *)p.c.p + (int64_t)b * p.c.sb + (int64_t)(h / p.c.share) * p.c.sh;
  f4 X[2 * KB];
#pragma unroll
  for (int k = 0; k < 2 * KB; ++k) X[k] = f4{0.f, 0.f, 0.f, 0.f};
  Tile<T, CT, DA, L> tb;
  Tile<T, CT, kCols, L> tc;
  // rows of a chunk in the order taken; `base` is the lowest position
  const int step = p.rev ? -1 : 1;
  auto fetch = [&](int t0) {
    const int n = min(L, hi - t0), row0 = p.rev ? n - 1 : 0;
    const int64_t base = p.rev ? len - t0 - n : t0;
    tb.fetch(bb + base * p.b.st, (int)p.b.st, p.Da, n, row0, step, 0);
    tc.fetch(c + base * p.c.st, (int)p.c.st, p.Dc, n, row0, step, c0);
  };
  if (VEC && lo < hi) fetch(lo);
  for (int t0 = lo; t0 < hi; t0 += L) {
    const int n = min(L, hi - t0);
    __syncthreads();
    if (VEC) {
      tb.put(Bm);
      tc.put(C);
    } else {
      const int64_t first = p.rev ? len - 1 - t0 : t0;
      stage<T, CT, DA, L>(Bm, bb + first * p.b.st, step * p.b.st, p.Da, n, 0);
      stage<T, CT, kCols, L>(C, c + first * p.c.st, step * p.c.st, p.Dc, n, c0);
    }
    __syncthreads();
    if (VEC && t0 + L < hi) fetch(t0 + L);
    Frag<CT> cf[L / 32];
#pragma unroll
    for (int jb = 0; jb < L / 32; ++jb) cf[jb] = frag_col(C + 32 * jb * ldc + 16 * w, ldc, lane);
    add_chunk<CT, KB, L>(X, Bm, cf, dec, n, p.off, lane);
  }
  const int xc = c0 + 16 * w + l16;
  float *out = p.xs + ((int64_t)bh * (p.nseg - 1) + s0) * p.Da * p.Dc;
#pragma unroll
  for (int k = 0; k < 2 * KB; ++k)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * k + 4 * g + r;
      if (row < p.Da && xc < p.Dc) out[row * p.Dc + xc] = X[k][r];
    }
}

// xs[s] from the part of segment s to X before segment s + 1, one element of
// X a thread.
__global__ __launch_bounds__(kThreads) void k_linattn_scan(LaArgs p) {
  const int64_t n = (int64_t)p.Da * p.Dc;
  const int64_t e = blockIdx.x * (int64_t)kThreads + threadIdx.x;
  if (e >= (int64_t)p.B * p.H * n) return;
  const int64_t bh = e / n;
  const int b = (int)(bh / p.H), h = (int)(bh % p.H);
  const int len = max(valid_length(p.lengths, b, p.T), 0);
  float *x = p.xs + bh * (p.nseg - 1) * n + e % n;
  float acc = p.x_in ? p.x_in[e] : 0.f;
  const float gd = p.log_decay[h], whole = expf(gd * p.seg);
  // eight loads at a time: the sum is a chain, the loads are not
  for (int s0 = 0; s0 < p.nseg - 1; s0 += 8) {
    float part[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) part[k] = s0 + k < p.nseg - 1 ? x[(s0 + k) * n] : 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int s = s0 + k, m = min(max(len - s * p.seg, 0), p.seg);
      acc = (m == p.seg ? whole : m ? expf(gd * m) : 1.f) * acc + part[k];
      if (s < p.nseg - 1) x[s * n] = acc;
    }
  }
}

// One workgroup: one segment of one sequence and head, kCols columns of the
// output, every chunk in turn.  T: the tensors' type; CT: the operands' type (bfloat16 as
// it is; float32 and float16 in float32: float16 would need its range
// watched in P and X); OT: the output's; DA: Da rounded up.
template <typename T, typename CT, typename OT, int DA, int L, bool VEC>
__global__ __launch_bounds__(kThreads) void k_linattn(LaArgs p) {
  constexpr int pad = 16 / sizeof(CT);
  constexpr int lda = DA + pad, ldc = kCols + pad, ldp = L + pad;
  constexpr int KB = DA / 32;
  constexpr int NR = Parts<CT>::kRead;
  __shared__ alignas(16) CT A[2 * L * lda + L * ldc + NR * L * ldp];
  __shared__ Decays<L> dec;
  CT *const Bm = A + L * lda;
  CT *const C = Bm + L * lda;
  CT *const P = C + L * ldc;

  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, g = lane >> 4, l16 = lane & 15;
  const int ct = blockIdx.x % p.ctiles, s0 = blockIdx.x / p.ctiles % p.nseg;
  const int bh = blockIdx.x / p.ctiles / p.nseg;
  const int h = bh % p.H, b = bh / p.H;
  const int c0 = ct * kCols;
  const int valid = valid_length(p.lengths, b, p.T);
  const int len = max(valid, 0);
  const int lo = s0 * p.seg, hi = min(len, lo + p.seg);  // of the order taken

  dec.fill(p, p.log_decay[h]);

  const T *a = (const T *)p.a.p + (int64_t)b * p.a.sb + (int64_t)(h / p.a.share) * p.a.sh;
  const T *bb = (const T *)p.b.p + (int64_t)b * p.b.sb + (int64_t)(h / p.b.share) * p.b.sh;
  const T *c = (const T *)p.c.p + (int64_t)b * p.c.sb + (int64_t)(h / p.c.share) * p.c.sh;
  OT *out = (OT *)p.out + ((int64_t)b * p.T * p.H + h) * p.Dc;
  const int64_t sot = (int64_t)p.H * p.Dc;

  // X: tile k holds rows 16k + 4g + r of column c0 + 16w + lane % 16.  All
  // loads at once, through a descriptor that reads 0 past the state
  f4 X[2 * KB];
  const int xc = c0 + 16 * w + l16;
  const int64_t xb = (int64_t)bh * p.Da * p.Dc;
  const float *x0 = s0 ? p.xs + ((int64_t)bh * (p.nseg - 1) + s0 - 1) * p.Da * p.Dc
                       : p.x_in ? p.x_in + xb : nullptr;
  const auto xr = __builtin_amdgcn_make_buffer_rsrc((void *)x0, 0, x0 ? kRange : 0, kRawBuffer);
  const int xrow = p.x_tr ? 1 : p.Dc, xcol = p.x_tr ? p.Da : 1;
#pragma unroll
  for (int k = 0; k < 2 * KB; ++k)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * k + 4 * g + r;
      const int at = 4 * (row * xrow + xc * xcol);
      X[k][r] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                              xr, row < p.Da && xc < p.Dc ? at : -1, 0, 0));
    }

  Tile<T, CT, DA, L> ta, tb;
  Tile<T, CT, kCols, L> tc;
  // rows of a chunk in the order taken: backwards, row 0 is the last
  // position not yet taken; `base` is the lowest position
  const int step = p.rev ? -1 : 1;
  auto fetch = [&](int t0) {
    const int n = min(L, hi - t0), row0 = p.rev ? n - 1 : 0;
    const int64_t base = p.rev ? len - t0 - n : t0;
    ta.fetch(a + base * p.a.st, (int)p.a.st, p.Da, n, row0, step, 0);
    tb.fetch(bb + base * p.b.st, (int)p.b.st, p.Da, n, row0, step, 0);
    tc.fetch(c + base * p.c.st, (int)p.c.st, p.Dc, n, row0, step, c0);
  };
  auto stage_chunk = [&](int t0) {
    if (VEC) {
      ta.put(A);
      tb.put(Bm);
      tc.put(C);
    } else {
      const int n = min(L, hi - t0);
      const int64_t first = p.rev ? len - 1 - t0 : t0;
      stage<T, CT, DA, L>(A, a + first * p.a.st, step * p.a.st, p.Da, n, 0);
      stage<T, CT, DA, L>(Bm, bb + first * p.b.st, step * p.b.st, p.Da, n, 0);
      stage<T, CT, kCols, L>(C, c + first * p.c.st, step * p.c.st, p.Dc, n, c0);
    }
  };
  if (lo < hi) {
    if (VEC) fetch(lo);
    stage_chunk(lo);
  }

  // Two barriers a chunk: one when its tiles and one when P is in LDS.
  // Everything that reads the tiles comes before the second, so the next
  // chunk's tiles follow it at once.
  constexpr int NT = L / 16;
  for (int t0 = lo; t0 < hi; t0 += L) {
    const int n = min(L, hi - t0);
    __syncthreads();
    if (VEC && t0 + L < hi) fetch(t0 + L);
    Frag<CT> cf[L / 32];
#pragma unroll
    for (int jb = 0; jb < L / 32; ++jb) cf[jb] = frag_col(C + 32 * jb * ldc + 16 * w, ldc, lane);
    f4 O[NT];
    if (p.out) {
      // P: wave w its rows 16w.., the tiles up to the diagonal and, as P is
      // read 32 columns at a time, the one beside it (zeros, by the table).  A
      // tile is computed transposed: a lane then holds four neighbours of a
      // row of P
      if (w < NT) {
        Frag<CT> af[KB];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
          af[kb] = frag_row(A + (16 * w + l16) * lda + 32 * kb + 4 * g);
        const int i = 16 * w + l16;
        const float *dp = dec.p + L + i - 4 * g;
        CT *to = P + i * ldp + 4 * g;
#pragma unroll
        for (int jt = 0; jt < NT; ++jt) {
          if (jt > (w | 1)) break;
          f4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int kb = 0; kb < KB; ++kb)
            acc = mma(frag_row(Bm + (16 * jt + l16) * lda + 32 * kb + 4 * g), af[kb], acc);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[r] *= dp[-(16 * jt + r)];
#pragma unroll
          for (int q = 0; q < NR; ++q) {
            Pack<CT, 4> x;
            part4(acc, x);
            *reinterpret_cast<Pack<CT, 4> *>(to + q * L * ldp + 16 * jt) = x;
          }
        }
      }
      // what X gives to each position
#pragma unroll
      for (int it = 0; it < NT; ++it) O[it] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        float x[8];
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = X[2 * kb][r], x[4 + r] = X[2 * kb + 1][r];
        Frag<CT> xf[NR];
        split<NR>(x, xf);
#pragma unroll
        for (int it = 0; it < NT; ++it) {
          const Frag<CT> af = frag_row(A + (16 * it + l16) * lda + 32 * kb + 4 * g);
#pragma unroll
          for (int q = 0; q < NR; ++q) O[it] = mma(xf[q], af, O[it]);
        }
      }
#pragma unroll
      for (int it = 0; it < NT; ++it) {
        const float d = dec.read[16 * it + l16];
#pragma unroll
        for (int r = 0; r < 4; ++r) O[it][r] *= d;
      }
    }
    add_chunk<CT, KB, L>(X, Bm, cf, dec, n, p.off, lane);
    __syncthreads();
    if (p.out) {
      const int64_t first = p.rev ? len - 1 - t0 : t0;
      const int col = c0 + 16 * w + 4 * g;
#pragma unroll
      for (int it = 0; it < NT; ++it) {
        const int i = 16 * it + l16;
#pragma unroll
        for (int jb = 0; jb <= it / 2; ++jb)
#pragma unroll
          for (int q = 0; q < NR; ++q)
            O[it] = mma(cf[jb], frag_row(P + q * L * ldp + i * ldp + 32 * jb + 4 * g), O[it]);
        if (i < n && col < p.Dc) {
          OT *to = out + (first + step * i) * sot + col;
          if (VEC) {
            Pack<OT, 4> x;
            part4(O[it], x);
            *reinterpret_cast<Pack<OT, 4> *>(to) = x;
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (col + r < p.Dc) to[r] = (OT)O[it][r];
          }
        }
      }
    }
    if (t0 + L < hi) stage_chunk(t0 + L);
  }

  if (p.out) {
    const OT fill = (OT)(valid < 0 ? p.bad : 0.f);
    const int f0 = max(len, lo), f1 = min((int64_t)p.T, (int64_t)lo + p.seg);
    for (int64_t e = threadIdx.x; e < (int64_t)(f1 - f0) * kCols; e += kThreads) {
      const int64_t t = f0 + e / kCols;
      const int col = c0 + e % kCols;
      if (col < p.Dc) out[t * sot + col] = fill;
    }
  }
  // the segment that holds the last valid position (the first, if none)
  if (p.x_out && hi == len && (lo < len || s0 == 0)) {
#pragma unroll
    for (int k = 0; k < 2 * KB; ++k)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * k + 4 * g + r;
        if (row < p.Da && xc < p.Dc)
          p.x_out[xb + (int64_t)row * p.Dc + xc] = valid >= 0 ? X[k][r] : p.bad;
      }
  }
}

// Sum over the heads that share one: part [B*T][H][D] float32 to out
// [B*T][H / share][D].
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

// One position: a workgroup per stream and head.  Thread t owns column
// t % 64 of each 64 and every fourth row.
template <typename T>
__global__ __launch_bounds__(256) void k_linattn_step(semicrf_linattn_shape_t s, const T *q,
                                                      const T *k, const T *v,
                                                      const float *log_decay,
                                                      const int32_t *slots, int nslots,
                                                      float *state, T *o) {
  __shared__ float qs[256], ks[256], red[4][64];
  const int b = blockIdx.x / s.H, h = blockIdx.x % s.H;
  const int slot = slots ? slots[b] : b;
  T *const ob = o + ((int64_t)b * s.H + h) * s.Dv;
  if (slot < 0 || slot >= nslots) {
    for (int c = threadIdx.x; c < s.Dv; c += 256) ob[c] = (T)0.f;
    return;
  }
  const T *qb = q + b * s.q_stride[0] + h / (s.H / s.Hq) * s.q_stride[2];
  const T *kb = k + b * s.k_stride[0] + h / (s.H / s.Hk) * s.k_stride[2];
  const T *vb = v + b * s.v_stride[0] + h / (s.H / s.Hv) * s.v_stride[2];
  if ((int)threadIdx.x < s.Dk) {
    qs[threadIdx.x] = (float)qb[threadIdx.x];
    ks[threadIdx.x] = (float)kb[threadIdx.x];
  }
  __syncthreads();
  const float d = expf(log_decay[h]);
  float *const S = state + ((int64_t)slot * s.H + h) * s.Dk * s.Dv;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  for (int c0 = 0; c0 < s.Dv; c0 += 64) {
    const int c = c0 + lane;
    float acc = 0.f;
    if (c < s.Dv) {
      const float vc = (float)vb[c];
      for (int r = w; r < s.Dk; r += 4) {
        const float x = d * S[(int64_t)r * s.Dv + c] + ks[r] * vc;
        S[(int64_t)r * s.Dv + c] = x;
        acc += qs[r] * x;
      }
    }
    red[w][lane] = acc;
    __syncthreads();
    if (w == 0 && c < s.Dv)
      ob[c] = (T)(s.scale * (red[0][lane] + red[1][lane] + red[2][lane] + red[3][lane]));
    __syncthreads();
  }
}

namespace {

int round_da(int D) { return D <= 32 ? 32 : D <= 64 ? 64 : D <= 128 ? 128 : 256; }

// Chunks of 64 positions; of 32 where float32 operands 256 wide would not
// leave a compute unit's 160 KB of LDS room for the tiles of 64.
template <typename CT, int DA>
constexpr int chunk_of() {
  return sizeof(CT) * DA > 512 ? 32 : 64;
}

template <typename T, typename CT, typename OT, int DA, bool VEC>
semicrf_status_t launch_da(const LaArgs &p, bool states, hipStream_t st) {
  constexpr int L = chunk_of<CT, DA>();
  if (states) {
    const int64_t grid = (int64_t)p.B * p.H * (p.nseg - 1) * p.ctiles;
    k_linattn_state<T, CT, DA, L, VEC><<<(unsigned)grid, kThreads, 0, st>>>(p);
  } else {
    const int64_t grid = (int64_t)p.B * p.H * p.nseg * p.ctiles;
    k_linattn<T, CT, OT, DA, L, VEC><<<(unsigned)grid, kThreads, 0, st>>>(p);
  }
  return launch_status();
}

template <typename T, typename CT, typename OT, bool VEC>
semicrf_status_t launch_v(const LaArgs &p, bool states, hipStream_t st) {
  switch (round_da(p.Da)) {
    case 32: return launch_da<T, CT, OT, 32, VEC>(p, states, st);
    case 64: return launch_da<T, CT, OT, 64, VEC>(p, states, st);
    case 128: return launch_da<T, CT, OT, 128, VEC>(p, states, st);
    default: return launch_da<T, CT, OT, 256, VEC>(p, states, st);
  }
}

// Whether every row of a tensor is a whole number of aligned 16-byte pieces,
// and a chunk of rows within reach of a buffer descriptor.
bool aligned(const View &v, int D, int dtype) {
  const int size = elem_size(dtype), e = 16 / size;
  return (uintptr_t)v.p % 16 == 0 && D % e == 0 && v.sb % e == 0 && v.st % e == 0 &&
         v.sh % e == 0 && v.st >= 0 && (v.st * 64 + 256) * size < kRange;
}

template <typename T, typename CT, typename OT>
semicrf_status_t launch_t(const LaArgs &p, bool vec, bool states, hipStream_t st) {
  return vec ? launch_v<T, CT, OT, true>(p, states, st) : launch_v<T, CT, OT, false>(p, states, st);
}

// The pass over the chunks.  f32_out: the output is float32 whatever the
// tensors are (parts of the gradient of a shared head).
semicrf_status_t launch_linattn(const LaArgs &p, int dtype, bool f32_out, hipStream_t st) {
  const bool vec = aligned(p.a, p.Da, dtype) && aligned(p.b, p.Da, dtype) &&
                   aligned(p.c, p.Dc, dtype) && (uintptr_t)p.out % 16 == 0;
  switch (dtype) {
    case SEMICRF_F32: return launch_t<float, float, float>(p, vec, false, st);
    case SEMICRF_BF16:
      return f32_out ? launch_t<bf16, bf16, float>(p, vec, false, st)
                     : launch_t<bf16, bf16, bf16>(p, vec, false, st);
    default:
      return f32_out ? launch_t<f16, float, float>(p, vec, false, st)
                     : launch_t<f16, float, f16>(p, vec, false, st);
  }
}

// The segments' states of a pair (b, c) in p.xs.
semicrf_status_t launch_states(const LaArgs &p, int dtype, hipStream_t st) {
  if (p.nseg < 2) return SEMICRF_OK;
  const bool vec = aligned(p.b, p.Da, dtype) && aligned(p.c, p.Dc, dtype);
  semicrf_status_t e = dtype == SEMICRF_F32    ? launch_t<float, float, float>(p, vec, true, st)
                       : dtype == SEMICRF_BF16 ? launch_t<bf16, bf16, bf16>(p, vec, true, st)
                                               : launch_t<f16, float, f16>(p, vec, true, st);
  if (e != SEMICRF_OK) return e;
  const int64_t n = (int64_t)p.B * p.H * p.Da * p.Dc;
  k_linattn_scan<<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, st>>>(p);
  return launch_status();
}

// Segments: enough for kFill workgroups, each of four chunks at least.
constexpr int kFill = 1024;
void segments(const semicrf_linattn_shape_t *s, int *nseg, int *seg) {
  const int64_t heads = (int64_t)s->B * s->H, chunks = (s->T + 63) / 64;
  int64_t n = (kFill + heads - 1) / heads;
  if (n > chunks / 4) n = chunks / 4;
  if (n < 1) n = 1;
  const int64_t per = (chunks + n - 1) / n;
  *seg = (int)(per * 64);
  *nseg = (int)((chunks + per - 1) / per);
}

size_t state_bytes(const semicrf_linattn_shape_t *s) {
  int nseg, seg;
  segments(s, &nseg, &seg);
  return ((size_t)s->B * s->H * (nseg - 1) * s->Dk * s->Dv * sizeof(float) + 255) / 256 * 256;
}

semicrf_status_t check(const semicrf_linattn_shape_t *s) {
  if (!s) return SEMICRF_ERR_NULL;
  if (s->B < 1 || s->T < 1 || s->H < 1 || s->Hq < 1 || s->Hk < 1 || s->Hv < 1 || s->Dk < 1 ||
      s->Dv < 1 || s->H % s->Hq || s->H % s->Hk || s->H % s->Hv)
    return SEMICRF_ERR_SHAPE;
  // a grid counts sequences, heads, four column tiles and the segments, which
  // are few where those are many; a state's elements over 256 threads
  if (s->T > 1 << 30 || (int64_t)s->B * s->H * 1024 > 0x7fffffff) return SEMICRF_ERR_SHAPE;
  if (s->Dk > 256 || s->Dv > 256) return SEMICRF_ERR_UNSUPPORTED;
  if (!dtype_ok(s->dtype)) return SEMICRF_ERR_ARG;
  return SEMICRF_OK;
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Parts of a shared head's gradient: one float32 row a head.
size_t share_bytes(const semicrf_linattn_shape_t *s, int heads, int D) {
  return heads == s->H ? 0 : align256((size_t)s->B * s->T * s->H * D * sizeof(float));
}

View view(const void *p, const int64_t *st, int share) { return {p, st[0], st[1], st[2], share}; }

semicrf_status_t share_sum(const semicrf_linattn_shape_t *s, const float *part, void *out,
                           int heads, int D, hipStream_t st) {
  const int64_t rows = (int64_t)s->B * s->T, n = rows * heads * D;
  const unsigned grid = (unsigned)(n < 256 * 8192 ? (n + 255) / 256 : 8192);
  const int share = s->H / heads;
  switch (s->dtype) {
    case SEMICRF_F32:
      k_share_sum<<<grid, 256, 0, st>>>(part, (float *)out, rows, s->H, share, D);
      break;
    case SEMICRF_BF16:
      k_share_sum<<<grid, 256, 0, st>>>(part, (bf16 *)out, rows, s->H, share, D);
      break;
    default: k_share_sum<<<grid, 256, 0, st>>>(part, (f16 *)out, rows, s->H, share, D);
  }
  return launch_status();
}

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
  if (backward)
    *bytes += share_bytes(s, s->Hq, s->Dk) + share_bytes(s, s->Hk, s->Dk) +
             share_bytes(s, s->Hv, s->Dv);
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
  p.ctiles = (p.Dc + kCols - 1) / kCols;
  p.xs = (float *)workspace;
  segments(s, &p.nseg, &p.seg);
  const semicrf_status_t r = launch_states(p, s->dtype, (hipStream_t)stream);
  return r == SEMICRF_OK ? launch_linattn(p, s->dtype, false, (hipStream_t)stream) : r;
}

semicrf_status_t semicrf_linattn_bwd(const semicrf_linattn_shape_t *s, const void *q,
                                     const void *k, const void *v, const float *log_decay,
                                     const int32_t *lengths, const float *state_in,
                                     const void *grad_o, const float *grad_state, void *grad_q,
                                     void *grad_k, void *grad_v, float *grad_state_in,
                                     void *workspace, size_t workspace_bytes, void *stream) {
  if (!s || !q || !k || !v || !log_decay || !grad_o) return SEMICRF_ERR_NULL;
  size_t need;
  semicrf_status_t e = semicrf_linattn_workspace_size(s, 1, &need);
  if (e != SEMICRF_OK) return e;
  if (need && (!workspace || workspace_bytes < need)) return SEMICRF_ERR_WORKSPACE;
  (void)hipGetLastError();
  hipStream_t st = (hipStream_t)stream;
  char *ws = (char *)workspace;
  float *xs = (float *)ws;
  ws += state_bytes(s);
  float *pq = (float *)ws;
  ws += share_bytes(s, s->Hq, s->Dk);
  float *pk = (float *)ws;
  ws += share_bytes(s, s->Hk, s->Dk);
  float *pv = (float *)ws;
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
    p.ctiles = (Dc + kCols - 1) / kCols;
  };
  auto run = [&](void *out, float *part, int heads) {
    const bool shared = out && heads != s->H;
    p.out = shared ? part : out;
    semicrf_status_t r = launch_linattn(p, s->dtype, shared, st);
    if (r == SEMICRF_OK && shared) r = share_sum(s, part, out, heads, p.Dc, st);
    return r;
  };
  if (grad_q) {
    p.x_in = state_in, p.rev = 0, p.off = 1;
    p.x_scale = s->scale, p.add_scale = 1.f;
    set(vq, vk, vv, s->Dk, s->Dv);
    e = launch_states(p, s->dtype, st);
    if (e != SEMICRF_OK) return e;
    p.x_tr = 1;
    set(vg, vv, vk, s->Dv, s->Dk);
    e = run(grad_q, pq, s->Hq);
    if (e != SEMICRF_OK) return e;
  }
  p.rev = 1, p.off = 0, p.x_scale = 1.f, p.add_scale = s->scale, p.x_in = grad_state, p.x_tr = 0;
  if (grad_k || grad_v || grad_state_in) {
    set(vk, vq, vg, s->Dk, s->Dv);
    e = launch_states(p, s->dtype, st);
    if (e != SEMICRF_OK) return e;
  }
  if (grad_v || grad_state_in) {
    p.x_out = grad_state_in;
    e = run(grad_v, pv, s->Hv);
    if (e != SEMICRF_OK) return e;
  }
  if (grad_k) {
    p.x_tr = 1, p.x_out = nullptr;
    set(vv, vg, vq, s->Dv, s->Dk);
    e = run(grad_k, pk, s->Hk);
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
  const unsigned grid = (unsigned)s->B * s->H;
  hipStream_t st = (hipStream_t)stream;
  switch (s->dtype) {
    case SEMICRF_F32:
      k_linattn_step<<<grid, 256, 0, st>>>(*s, (const float *)q, (const float *)k,
                                           (const float *)v, log_decay, slots, nslots, state,
                                           (float *)o);
      break;
    case SEMICRF_BF16:
      k_linattn_step<<<grid, 256, 0, st>>>(*s, (const bf16 *)q, (const bf16 *)k, (const bf16 *)v,
                                           log_decay, slots, nslots, state, (bf16 *)o);
      break;
    default:
      k_linattn_step<<<grid, 256, 0, st>>>(*s, (const f16 *)q, (const f16 *)k, (const f16 *)v,
                                           log_decay, slots, nslots, state, (f16 *)o);
  }
  return launch_status();
}

}  // extern "C"
