// linattn_kernels.h -- the chunked kernels of linear attention, instantiated
// by linattn_f32.hip, linattn_bf16.hip and linattn_f16.hip (linattn.hip says
// what they compute).
#pragma once

#include <type_traits>

#include "parts.h"

namespace semicrf {

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

// Operands.  The matrix cores multiply bfloat16 sixteen times as fast as
// float32, and a float32 is a sum of three bfloat16 parts (8 bits each), a
// float16 of two: so every operand is held in NP parts, and a product of two
// sums keeps the pairs of parts (i, j) whose share is above the last part's
// (i + j < the number of parts).
//   inputs       1, 2 or 3 parts: exact
//   P and X, and what is added to X   3 parts (2^-24): they are float32 whatever
//                the tensors are.  Two parts for 16-bit tensors would lose what
//                is left where terms cancel, for 3 to 8 % of the time (32
//                sequences of 512 positions of 4 heads of 64 + 64 27 us in the
//                place of 29, 2^20 positions 701 in the place of 726)
// Float32 at 64 columns: 6 products of 16 cycles in the place of 8 of 32.
__host__ __device__ constexpr int linattn_parts(int dtype) {
  return dtype == SEMICRF_F32 ? 3 : dtype == SEMICRF_F16 ? 2 : 1;
}
// Positions of a chunk.  The products inside a chunk grow with it, the reading
// and updating of X shrink: 64; 32 where more parts than one would leave a
// compute unit's LDS room for one workgroup.
__host__ __device__ constexpr int linattn_chunk(int parts) { return parts > 1 ? 32 : 64; }

// Waves of a workgroup: one for 16 columns of the output.
inline int linattn_waves(int Dc) {
  const int w = (Dc + 15) / 16;
  return w <= 2 ? 2 : w <= 6 ? w : 8;
}
// Elements of bfloat16 in LDS for the tiles of a chunk: A, B, C and P.
__host__ __device__ constexpr int linattn_tiles(int NP, int DA, int NW) {
  const int L = linattn_chunk(NP), W = 16 * NW;
  return L * (NP * (DA + 4 + DA + (W % 32 == 16 ? W : W + 16)) + 3 * (NP == 1 ? L : L + 4));
}
// Workgroups a compute unit's LDS holds (the decays beside the tiles).
__host__ __device__ constexpr int linattn_by_lds(int NP, int DA, int NW) {
  return 163840 / (2 * linattn_tiles(NP, DA, NW) + 4 * (7 * linattn_chunk(NP) + 3));
}
// Waves a SIMD is to hold (what the registers are rationed to), where LDS lets
// it.  The waves of a workgroup are dealt to the four SIMDs from the first one
// on, so one of five to eight waves needs two places there: four places hold
// two of them.
__host__ __device__ constexpr int linattn_occupancy(int NP, int DA, int NW) {
  const int waves = (linattn_by_lds(NP, DA, NW) * NW + 3) / 4;
  const int most = DA <= 64 ? (NW <= 4 ? 3 : 4) : DA <= 128 ? 2 : 1;
  return NW == 6 || most < waves ? most : waves;
}
// Twelve waves of two workgroups of six fill three places a SIMD, and the
// compiler, which counts them so, would not ration registers to four where it
// knows their LDS: it is told at the launch.  64 x 96 in bfloat16, 8 sequences
// of 4096 positions of 4 heads: 49 us in the place of 57.
__host__ __device__ constexpr bool linattn_lds_at_launch(int DA, int NW) {
  return NW == 6 && DA <= 64;
}

// Widths of a launch: Da up to DA (a multiple of 32), NW waves for 16 NW
// columns of Dc.  vec: 16-byte loads; f32_out: float32 output whatever the
// tensors are; states: k_linattn_state instead of k_linattn.
semicrf_status_t linattn_f32(const LaArgs &p, bool vec, bool f32_out, bool states, hipStream_t st);
semicrf_status_t linattn_bf16(const LaArgs &p, bool vec, bool f32_out, bool states, hipStream_t st);
semicrf_status_t linattn_f16(const LaArgs &p, bool vec, bool f32_out, bool states, hipStream_t st);

namespace {

// A lane's number as something new to the compiler: what follows from it is
// then computed again in every chunk instead of being kept in registers all
// along.  For the shapes that are short of them (workgroups of more than four
// waves have 128 a lane): the load of a spilled register would wait for every
// tile on its way.
template <int DA, int NW>
__device__ __forceinline__ int fresh(int lane) {
  if (NW > 4 || DA > 96) asm volatile("" : "+v"(lane));
  return lane;
}

// The decays a workgroup uses, with the pass's factors in them, from float64
// exponentials; entries of negative powers are 0, so masked places need no
// branch.  X is multiplied by e^{g n} once a chunk, thousands of times in a
// long sequence: there e^{g n} is a sum of two float32, or its own rounding,
// the same every time, would add up.
template <int L>
struct Decays {
  float x[L + 1], x_low[L + 1];  // e^{g n}: of X over n positions
  float p[2 * L];                // p_scale e^{g (n - L)}: of P
  float read[L];                 // x_scale e^{g (i + off)}: of X read by position i
  float add[2 * L + 1];          // add_scale e^{g (n - L)}: of what a position adds to X

  // all threads of the workgroup; the caller's next barrier ends it
  __device__ __forceinline__ void fill(const LaArgs &a, float g) {
    for (int n = threadIdx.x; n <= L; n += blockDim.x) {
      const double e = n ? exp((double)g * n) : 1.0;
      x[n] = (float)e;
      x_low[n] = (float)(e - (double)(float)e);
    }
    __syncthreads();
    for (int n = threadIdx.x; n < 2 * L + 1; n += blockDim.x) {
      const float e = n < L ? 0.f : x[n - L];
      add[n] = a.add_scale * e;
      if (n < 2 * L) p[n] = a.p_scale * e;
      if (n < L) read[n] = a.x_scale * x[n + a.off];
    }
  }
};

// X <- e^{g n} X + sum_j e^{g (n - off - j)} b_j c_j^T over a staged chunk:
// B from LDS, this wave's 16 columns of C in fragments.
template <int NP, int KB, int L>
__device__ __forceinline__ void add_chunk(f4 *X, const bf16 *Bm, const Frag<NP> *C,
                                          const Decays<L> &dec, int n, int off, int lane) {
  constexpr int DA = 32 * KB;
  const float *add = dec.add + L + n - off - 4 * (lane >> 4);
  const float all = dec.x[n], low = dec.x_low[n];
#pragma unroll
  for (int k = 0; k < 2 * KB; ++k)
#pragma unroll
    for (int r = 0; r < 4; ++r) X[k][r] = fmaf(X[k][r], low, X[k][r] * all);
#pragma unroll
  for (int jb = 0; jb < L / 32; ++jb) {
    float x[8];
    values(C[jb], x);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= add[-(32 * jb + (e & 3) + (e >> 2) * 16)];
    const Frag<3> cf = split<3>(x);
#pragma unroll
    for (int k = 0; k < 2 * KB; ++k)
      X[k] = mma<3>(frag_col<NP, ByBoth<DA>>(Bm, L * DA, 32 * jb, k, lane), cf, X[k]);
  }
}

}  // namespace

// Parts of X: one workgroup of NW waves per segment but the last, 16 NW
// columns.  Writes xs[segment]; a segment past the length leaves zeros.  Bound
// by HBM: 1.07 GB of keys and values (2^20 positions, 4 heads of 64 + 64,
// bfloat16) in 211 to 225 us, 5 TB/s.
template <typename T, int NP, int DA, int NW, int L, bool VEC>
__global__ __launch_bounds__(64 * NW) void k_linattn_state(LaArgs p) {
  constexpr int kCols = 16 * NW, kThreads = 64 * NW;
  constexpr int KB = DA / 32;
  typedef ByBoth<DA> LB;
  typedef ByColumn<kCols> LC;
  __shared__ alignas(16) bf16 Bm[NP * L * (DA + LC::row)];
  bf16 *const C = Bm + NP * L * DA;
  __shared__ Decays<L> dec;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, g = lane >> 4, l16 = lane & 15;
  const int ct = blockIdx.x % p.ctiles, s0 = blockIdx.x / p.ctiles % (p.nseg - 1);
  const int bh = blockIdx.x / p.ctiles / (p.nseg - 1);
  const int h = bh % p.H, b = bh / p.H, c0 = ct * kCols;
  const int len = max(valid_length(p.lengths, b, p.T), 0);
  const int lo = s0 * p.seg, hi = min(len, lo + p.seg);
  const T *bb = (const T *)p.b.p + (int64_t)b * p.b.sb + (int64_t)(h / p.b.share) * p.b.sh;
  const T *c = (const T *)p.c.p + (int64_t)b * p.c.sb + (int64_t)(h / p.c.share) * p.c.sh;
  f4 X[2 * KB];
#pragma unroll
  for (int k = 0; k < 2 * KB; ++k) X[k] = f4{0.f, 0.f, 0.f, 0.f};
  Tile<T, NP, LB, DA, L, kThreads> tb;
  Tile<T, NP, LC, kCols, L, kThreads> tc;
  // rows of a chunk in the order taken; `base` is the lowest position
  const int step = p.rev ? -1 : 1;
  auto fetch = [&](int t0) {
    const int n = min(L, hi - t0), row0 = p.rev ? n - 1 : 0;
    const int64_t base = p.rev ? len - t0 - n : t0;
    tb.fetch(threadIdx.x, bb + base * p.b.st, (int)p.b.st, p.Da, n, row0, step, 0);
    tc.fetch(threadIdx.x, c + base * p.c.st, (int)p.c.st, p.Dc, n, row0, step, c0);
  };
  if (VEC && lo < hi) fetch(lo);
  dec.fill(p, p.log_decay[h]);
  for (int t0 = lo; t0 < hi; t0 += L) {
    const int n = min(L, hi - t0);
    __syncthreads();
    if (VEC) {
      tb.put(threadIdx.x, Bm);
      tc.put(threadIdx.x, C);
    } else {
      const int64_t first = p.rev ? len - 1 - t0 : t0;
      stage<T, NP, LB, DA, L, kThreads>(Bm, bb + first * p.b.st, step * p.b.st, p.Da, n, 0);
      stage<T, NP, LC, kCols, L, kThreads>(C, c + first * p.c.st, step * p.c.st, p.Dc, n, c0);
    }
    __syncthreads();
    if (VEC && t0 + L < hi) fetch(t0 + L);
    Frag<NP> cf[L / 32];
#pragma unroll
    for (int jb = 0; jb < L / 32; ++jb) cf[jb] = frag_col<NP, LC>(C, L * LC::row, 32 * jb, w, lane);
    add_chunk<NP, KB, L>(X, Bm, cf, dec, n, p.off, lane);
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
// columns of the output, every chunk in turn.  T: the tensors' type, in NP
// parts; OT: the output's; DA: Da rounded up to a multiple of 32.
//
// A wave keeps its 16 columns of X in accumulators from chunk to chunk and
// reads them as operands in place; P goes through LDS, as every wave needs all
// of it.  At 64 x 64 in bfloat16 a chunk of 64 positions is 24 KB read and 8
// written against about 1250 matrix cycles, 1900 LDS cycles and 690 vector
// instructions a wave: three workgroups a compute unit (54 KB of LDS, 161
// registers), bound by HBM and nearly by the vector units.  Measured, 2^20
// positions of 4 heads: 529 us at best, 4.1 TB/s of 2.15 GB read and written (a
// large copy: 5.1); matrix cores busy 31 %, vector units 60 %, LDS 56 % (10 %
// conflicts).  In float32 (40 x 72 wide) 126 to 133 us for 330 MB: two
// workgroups of five waves, vector units busy 60 %, the splitting into parts
// and the longer sums of them.
template <typename T, int NP, typename OT, int DA, int NW, int L, bool VEC>
__global__ __launch_bounds__(64 * NW)
    __attribute__((amdgpu_waves_per_eu(linattn_occupancy(NP, DA, NW)))) void k_linattn(LaArgs p) {
  constexpr int kCols = 16 * NW, kThreads = 64 * NW;
  constexpr int KB = DA / 32;
  constexpr int NR = 3;  // parts of P and X
  typedef ByRow<DA> LA;
  typedef ByBoth<DA> LB;
  typedef ByColumn<kCols> LC;
  // without padding where that lets a compute unit hold a workgroup more; with
  // it where the addresses of the other would take registers that are short
  typedef std::conditional_t<NP == 1, ByBoth<L>, ByRow<L>> LP;
  constexpr int kTiles = linattn_tiles(NP, DA, NW);
  static_assert(kTiles == L * (NP * (LA::row + LB::row + LC::row) + NR * LP::row), "");
  constexpr bool kAtLaunch = linattn_lds_at_launch(DA, NW);
  __shared__ alignas(16) bf16 tiles[kAtLaunch ? 1 : kTiles];
  extern __shared__ __align__(16) unsigned char at_launch[];
  bf16 *const A = kAtLaunch ? (bf16 *)at_launch : tiles;
  bf16 *const Bm = A + NP * L * LA::row;
  bf16 *const C = Bm + NP * L * DA;
  bf16 *const P = C + NP * L * LC::row;
  __shared__ Decays<L> dec;

  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, g = lane >> 4, l16 = lane & 15;
  const int ct = blockIdx.x % p.ctiles, s0 = blockIdx.x / p.ctiles % p.nseg;
  const int bh = blockIdx.x / p.ctiles / p.nseg;
  const int h = bh % p.H, b = bh / p.H;
  const int c0 = ct * kCols;
  const int valid = valid_length(p.lengths, b, p.T);
  const int len = max(valid, 0);
  const int lo = s0 * p.seg, hi = min(len, lo + p.seg);  // of the order taken

  const T *a = (const T *)p.a.p + (int64_t)b * p.a.sb + (int64_t)(h / p.a.share) * p.a.sh;
  const T *bb = (const T *)p.b.p + (int64_t)b * p.b.sb + (int64_t)(h / p.b.share) * p.b.sh;
  const T *c = (const T *)p.c.p + (int64_t)b * p.c.sb + (int64_t)(h / p.c.share) * p.c.sh;
  OT *out = (OT *)p.out + ((int64_t)b * p.T * p.H + h) * p.Dc;
  const int64_t sot = (int64_t)p.H * p.Dc;

  Tile<T, NP, LA, DA, L, kThreads> ta;
  Tile<T, NP, LB, DA, L, kThreads> tb;
  Tile<T, NP, LC, kCols, L, kThreads> tc;
  // rows of a chunk in the order taken: backwards, row 0 is the last
  // position not yet taken; `base` is the lowest position
  const int step = p.rev ? -1 : 1;
  auto fetch = [&](int t0) {
    const int tid = fresh<DA, NW>(threadIdx.x);
    const int n = min(L, hi - t0), row0 = p.rev ? n - 1 : 0;
    const int64_t base = p.rev ? len - t0 - n : t0;
    ta.fetch(tid, a + base * p.a.st, (int)p.a.st, p.Da, n, row0, step, 0);
    tb.fetch(tid, bb + base * p.b.st, (int)p.b.st, p.Da, n, row0, step, 0);
    tc.fetch(tid, c + base * p.c.st, (int)p.c.st, p.Dc, n, row0, step, c0);
  };
  auto stage_chunk = [&](int t0) {
    if (VEC) {
      const int tid = fresh<DA, NW>(threadIdx.x);
      ta.put(tid, A);
      tb.put(tid, Bm);
      tc.put(tid, C);
    } else {
      const int n = min(L, hi - t0);
      const int64_t first = p.rev ? len - 1 - t0 : t0;
      stage<T, NP, LA, DA, L, kThreads>(A, a + first * p.a.st, step * p.a.st, p.Da, n, 0);
      stage<T, NP, LB, DA, L, kThreads>(Bm, bb + first * p.b.st, step * p.b.st, p.Da, n, 0);
      stage<T, NP, LC, kCols, L, kThreads>(C, c + first * p.c.st, step * p.c.st, p.Dc, n, c0);
    }
  };
  if (VEC && lo < hi) fetch(lo);

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

  dec.fill(p, p.log_decay[h]);
  if (lo < hi) stage_chunk(lo);

  // Two barriers a chunk: one when its tiles and one when P is in LDS.
  // Everything that reads the tiles comes before the second, so the next
  // chunk's tiles follow it at once.
  constexpr int NT = L / 16;
  for (int t0 = lo; t0 < hi; t0 += L) {
    const int n = min(L, hi - t0);
    __syncthreads();
    const int ln = fresh<DA, NW>(lane), g = ln >> 4, l16 = ln & 15;
    if (VEC && t0 + L < hi) fetch(t0 + L);
    Frag<NP> cf[L / 32];
#pragma unroll
    for (int jb = 0; jb < L / 32; ++jb) cf[jb] = frag_col<NP, LC>(C, L * LC::row, 32 * jb, w, ln);
    f4 O[NT];
    if (p.out) {
      // P: wave w its rows 16w.., the tiles up to the diagonal and, as P is
      // read 32 columns at a time, the one beside it (zeros, by the table).  A
      // tile is computed transposed: a lane then holds four neighbours of a
      // row of P
      for (int it = w; it < NT; it += NW) {
        Frag<NP> af[KB];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
          af[kb] = frag_row<NP, LA>(A, L * LA::row, 16 * it, kb, ln);
        const int i = 16 * it + l16;
        const float *dp = dec.p + L + i - 4 * g;
#pragma unroll
        for (int jt = 0; jt < NT; ++jt) {
          if (jt > (it | 1)) continue;
          f4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int kb = 0; kb < KB; ++kb)
            acc = mma<3>(frag_row<NP, LB>(Bm, L * DA, 16 * jt, kb, ln), af[kb], acc);
          f2 lo = {acc[0] * dp[-16 * jt], acc[1] * dp[-16 * jt - 1]};
          f2 hi = {acc[2] * dp[-16 * jt - 2], acc[3] * dp[-16 * jt - 3]};
#pragma unroll
          for (int q = 0; q < NR; ++q) {
            const b2 x = part2(lo), y = part2(hi);
            *reinterpret_cast<Pack<bf16, 4> *>(P + q * L * LP::row + LP::at(i, 4 * jt + g)) =
                Pack<bf16, 4>{{x[0], x[1], y[0], y[1]}};
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
        const Frag<NR> xf = split<NR>(x);
#pragma unroll
        for (int it = 0; it < NT; ++it)
          O[it] = mma<NR>(xf, frag_row<NP, LA>(A, L * LA::row, 16 * it, kb, ln), O[it]);
      }
#pragma unroll
      for (int it = 0; it < NT; ++it) {
        const float d = dec.read[16 * it + l16];
#pragma unroll
        for (int r = 0; r < 4; ++r) O[it][r] *= d;
      }
    }
    add_chunk<NP, KB, L>(X, Bm, cf, dec, n, p.off, ln);
    __syncthreads();
    if (p.out) {
      const int64_t first = p.rev ? len - 1 - t0 : t0;
      const int col = c0 + 16 * w + 4 * g;
#pragma unroll
      for (int it = 0; it < NT; ++it) {
        const int i = 16 * it + l16;
#pragma unroll
        for (int jb = 0; jb <= it / 2; ++jb)
          O[it] = mma<NR>(cf[jb], frag_row<NR, LP>(P, L * LP::row, 16 * it, jb, ln), O[it]);
        if (i < n && col < p.Dc) {
          OT *to = out + (first + step * i) * sot + col;
          if (VEC) {
            Pack<OT, 4> x;
#pragma unroll
            for (int r = 0; r < 4; ++r) x.v[r] = (OT)O[it][r];
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

template <typename T, int NP, typename OT, int DA, int NW, bool VEC>
semicrf_status_t launch_one(LaArgs p, bool states, hipStream_t st) {
  constexpr int L = linattn_chunk(NP);
  p.ctiles = (p.Dc + 16 * NW - 1) / (16 * NW);
  const int64_t grid = (int64_t)p.B * p.H * (states ? p.nseg - 1 : p.nseg) * p.ctiles;
  if (states)
    k_linattn_state<T, NP, DA, NW, L, VEC><<<(unsigned)grid, 64 * NW, 0, st>>>(p);
  else
    k_linattn<T, NP, OT, DA, NW, L, VEC>
        <<<(unsigned)grid, 64 * NW, linattn_lds_at_launch(DA, NW) ? 2 * linattn_tiles(NP, DA, NW) : 0,
           st>>>(p);
  return launch_status();
}

template <typename T, int NP, typename OT, int DA>
semicrf_status_t launch_nw(const LaArgs &p, bool states, hipStream_t st) {
  switch (linattn_waves(p.Dc)) {
    case 2: return launch_one<T, NP, OT, DA, 2, true>(p, states, st);
    case 3: return launch_one<T, NP, OT, DA, 3, true>(p, states, st);
    case 4: return launch_one<T, NP, OT, DA, 4, true>(p, states, st);
    case 5: return launch_one<T, NP, OT, DA, 5, true>(p, states, st);
    case 6: return launch_one<T, NP, OT, DA, 6, true>(p, states, st);
    default: return launch_one<T, NP, OT, DA, 8, true>(p, states, st);
  }
}

// As many waves as the output has 16-column tiles, up to eight: A, B and P
// are then read and computed once for all of it.  At Da > 128 four: eight
// would leave a lane 256 registers, and X alone takes 64.
// Without aligned rows the loads are by element and cost more than padding:
// two widths serve.
template <typename T, int NP, typename OT>
semicrf_status_t launch_type(const LaArgs &p, bool vec, bool states, hipStream_t st) {
  if (!vec)
    return p.Da <= 64 ? launch_one<T, NP, OT, 64, 4, false>(p, states, st)
                      : launch_one<T, NP, OT, 256, 4, false>(p, states, st);
  if (p.Da <= 32) return launch_nw<T, NP, OT, 32>(p, states, st);
  if (p.Da <= 64) return launch_nw<T, NP, OT, 64>(p, states, st);
  if (p.Da <= 96) return launch_nw<T, NP, OT, 96>(p, states, st);
  if (p.Da <= 128) return launch_nw<T, NP, OT, 128>(p, states, st);
  return launch_one<T, NP, OT, 256, 4, true>(p, states, st);
}

}  // namespace

}  // namespace semicrf
