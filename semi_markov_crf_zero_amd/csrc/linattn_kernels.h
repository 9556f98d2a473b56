// linattn_kernels.h -- the chunked kernels of linear attention, instantiated
// by linattn_f32.hip, linattn_bf16.hip and linattn_f16.hip (linattn.hip says
// what they compute).
#pragma once

#include "encoder.h"

namespace semicrf {

// One tensor as the kernels read it: element strides of batch, position and
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

// Positions of a chunk.  The products inside a chunk grow with it, the reading
// and updating of X shrink: 64 for bfloat16 operands; 32 for float32 ones,
// whose matrix rate is a sixteenth and whose tiles of 64 would leave a
// compute unit room for one workgroup.
__host__ __device__ constexpr int linattn_chunk(bool f32_operands) { return f32_operands ? 32 : 64; }

// Waves of a workgroup: one for 16 columns of the output.
inline int linattn_waves(int Dc, bool vec) {
  const int w = (Dc + 15) / 16;
  return !vec ? 4 : w <= 2 ? 2 : w <= 6 ? w : 8;
}
// Waves a SIMD is to hold (what the registers are rationed to).
__host__ __device__ constexpr int linattn_occupancy(int DA, int NW) {
  return DA <= 64 || (DA <= 96 && NW >= 4) ? 3 : DA <= 128 ? 2 : 1;
}

// Widths of a launch: Da up to DA (a multiple of 32), NW waves for 16 NW
// columns of Dc.  vec: 16-byte loads; f32_out: float32 output whatever the
// tensors are; states: k_linattn_state instead of k_linattn.
semicrf_status_t linattn_f32(const LaArgs &p, bool vec, bool f32_out, bool states, hipStream_t st);
semicrf_status_t linattn_bf16(const LaArgs &p, bool vec, bool f32_out, bool states, hipStream_t st);
semicrf_status_t linattn_f16(const LaArgs &p, bool vec, bool f32_out, bool states, hipStream_t st);


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
template <typename T, typename CT, int W, int L, int NT>
struct Tile {
  static constexpr int VE = 16 / sizeof(T), per = W / VE, all = L * per, NV = (all + NT - 1) / NT;
  static constexpr int ld = W + 16 / sizeof(CT);
  u4 r[NV];

  // row i of the tile is row `row0 + step * i` (step +-1) from src, rows st
  // elements apart
  __device__ __forceinline__ void fetch(const T *src, int st, int D, int n, int row0, int step,
                                        int col0) {
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)src, 0, kRange, kRawBuffer);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int e = threadIdx.x + k * NT, i = e / per, c = col0 + e % per * VE;
      const int at = ((row0 + step * i) * st + c) * (int)sizeof(T);
      r[k] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, i < n && c < D ? at : -1, 0, 0);
    }
  }
  __device__ __forceinline__ void put(CT *lds) const {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int e = threadIdx.x + k * NT, i = e / per, c = e % per * VE;
      if (all % NT && e >= all) break;
      const Pack<T, VE> y = __builtin_bit_cast(Pack<T, VE>, r[k]);
      Pack<CT, VE> x;
#pragma unroll
      for (int q = 0; q < VE; ++q) x.v[q] = (CT)y.v[q];
      CT *to = lds + i * ld + c;
#pragma unroll
      for (int q = 0; q < VE; q += 16 / sizeof(CT))
        *reinterpret_cast<Pack<CT, 16 / sizeof(CT)> *>(to + q) =
            *reinterpret_cast<const Pack<CT, 16 / sizeof(CT)> *>(x.v + q);
    }
  }
};

// The same without the alignment 16-byte loads need: element by element,
// straight to LDS.
template <typename T, typename CT, int W, int L, int NT>
__device__ __forceinline__ void stage(CT *lds, const T *src, int64_t st, int D, int n, int col0) {
  constexpr int ld = W + 16 / sizeof(CT);
  for (int e = threadIdx.x; e < L * W; e += NT) {
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
    for (int n = threadIdx.x; n < 2 * L + 1; n += blockDim.x) {
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

// Parts of X: one workgroup of NW waves per segment but the last, 16 NW
// columns.  Writes
// xs[segment]; a segment past the length leaves zeros.
template <typename T, typename CT, int DA, int NW, int L, bool VEC>
__global__ __launch_bounds__(64 * NW) void k_linattn_state(LaArgs p) {
  constexpr int pad = 16 / sizeof(CT);
  constexpr int kCols = 16 * NW, kThreads = 64 * NW;
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
  Tile<T, CT, DA, L, kThreads> tb;
  Tile<T, CT, kCols, L, kThreads> tc;
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
      stage<T, CT, DA, L, kThreads>(Bm, bb + first * p.b.st, step * p.b.st, p.Da, n, 0);
      stage<T, CT, kCols, L, kThreads>(C, c + first * p.c.st, step * p.c.st, p.Dc, n, c0);
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

// One workgroup of NW waves: one segment of one sequence and head, 16 NW
// columns of the output, every chunk in turn.  T: the tensors' type; CT: the operands' type (bfloat16 as
// it is; float32 and float16 in float32: float16 would need its range
// watched in P and X); OT: the output's; DA: Da rounded up.
template <typename T, typename CT, typename OT, int DA, int NW, int L, bool VEC>
__global__ __launch_bounds__(64 * NW)
    __attribute__((amdgpu_waves_per_eu(linattn_occupancy(DA, NW)))) void k_linattn(LaArgs p) {
  constexpr int pad = 16 / sizeof(CT);
  constexpr int kCols = 16 * NW, kThreads = 64 * NW;
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

  Tile<T, CT, DA, L, kThreads> ta, tb;
  Tile<T, CT, kCols, L, kThreads> tc;
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
      stage<T, CT, DA, L, kThreads>(A, a + first * p.a.st, step * p.a.st, p.Da, n, 0);
      stage<T, CT, DA, L, kThreads>(Bm, bb + first * p.b.st, step * p.b.st, p.Da, n, 0);
      stage<T, CT, kCols, L, kThreads>(C, c + first * p.c.st, step * p.c.st, p.Dc, n, c0);
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
#pragma unroll
      for (int it = w; it < NT; it += NW) {
        Frag<CT> af[KB];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
          af[kb] = frag_row(A + (16 * it + l16) * lda + 32 * kb + 4 * g);
        const int i = 16 * it + l16;
        const float *dp = dec.p + L + i - 4 * g;
        CT *to = P + i * ldp + 4 * g;
#pragma unroll
        for (int jt = 0; jt < NT; ++jt) {
          if (jt > (it | 1)) break;
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

namespace {

template <typename T, typename CT, typename OT, int DA, int NW, bool VEC>
semicrf_status_t launch_one(LaArgs p, bool states, hipStream_t st) {
  constexpr int L = linattn_chunk(sizeof(CT) == 4);
  p.ctiles = (p.Dc + 16 * NW - 1) / (16 * NW);
  const int64_t grid = (int64_t)p.B * p.H * (states ? p.nseg - 1 : p.nseg) * p.ctiles;
  if (grid > 0x7fffffff) return SEMICRF_ERR_SHAPE;
  if (states)
    k_linattn_state<T, CT, DA, NW, L, VEC><<<(unsigned)grid, 64 * NW, 0, st>>>(p);
  else
    k_linattn<T, CT, OT, DA, NW, L, VEC><<<(unsigned)grid, 64 * NW, 0, st>>>(p);
  return launch_status();
}

template <typename T, typename CT, typename OT, int DA>
semicrf_status_t launch_nw(const LaArgs &p, bool states, hipStream_t st) {
  switch (linattn_waves(p.Dc, true)) {
    case 2: return launch_one<T, CT, OT, DA, 2, true>(p, states, st);
    case 3: return launch_one<T, CT, OT, DA, 3, true>(p, states, st);
    case 4: return launch_one<T, CT, OT, DA, 4, true>(p, states, st);
    case 5: return launch_one<T, CT, OT, DA, 5, true>(p, states, st);
    case 6: return launch_one<T, CT, OT, DA, 6, true>(p, states, st);
    default: return launch_one<T, CT, OT, DA, 8, true>(p, states, st);
  }
}

// As many waves as the output has 16-column tiles, up to eight: A, B and P
// are then read and computed once for all of it.  At Da > 128 four: eight
// would leave a lane 256 registers, and X alone takes 64.
// Without aligned rows the loads are by element and cost more than padding:
// two widths serve.
template <typename T, typename CT, typename OT>
semicrf_status_t launch_type(const LaArgs &p, bool vec, bool states, hipStream_t st) {
  if (!vec)
    return p.Da <= 64 ? launch_one<T, CT, OT, 64, 4, false>(p, states, st)
                      : launch_one<T, CT, OT, 256, 4, false>(p, states, st);
  if (p.Da <= 32) return launch_nw<T, CT, OT, 32>(p, states, st);
  if (p.Da <= 64) return launch_nw<T, CT, OT, 64>(p, states, st);
  if (p.Da <= 96) return launch_nw<T, CT, OT, 96>(p, states, st);
  if (p.Da <= 128) return launch_nw<T, CT, OT, 128>(p, states, st);
  return launch_one<T, CT, OT, 256, 4, true>(p, states, st);
}

}  // namespace

}  // namespace semicrf
