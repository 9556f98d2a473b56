// delta_kernels.h -- the chunked kernels of the gated delta rule, instantiated
// by delta_f32.hip, delta_bf16.hip and delta_f16.hip (delta.hip says what they
// compute).
#pragma once

#include <type_traits>

#include "parts.h"

namespace semicrf {

// What is left of a chunk's gates: of each position the sum G of its log decays
// from the chunk's start in two floats, e^G, e^{G_L - G}; then e^{G_L} in two.
__host__ __device__ constexpr int delta_gates(int L) { return 4 * L + 4; }

struct DeltaArgs {
  View q, k, v;
  const void *go;  // gradient of o [B][T][H][Dv]
  const float *log_decay, *beta;
  const int32_t *lengths;
  const float *state_in;
  float *X, *gates;  // of each chunk: [ld][ld], delta_gates
  // Rows of Dk or Dv of the following are lk or lv apart, rounded up to fours (zeros there).
  float *phi, *phit, *xs;  // of each segment: [Dk][Dk], its transpose (or NULL), [Dk][Dv]
  // of each chunk, by columns, which lanes hold four neighbours of:
  float *S, *U;  // for the backward pass: [Dv][Dk], [Dv][L]; or NULL
  float *D, *R;  // and its own: the gradients of the state after it and of R
  void *o, *dq, *dk, *dv;
  float *state_out, *dg, *db;
  int part_q, part_k, part_v;  // gradients go to float32 [B][T][H][D]: of shared heads
  int vec, vec_out;            // rows are read 16 bytes at a time; dq and dk written by fours
  int nseg, seg;               // segments, chunks of one
  int first, count;            // segments of a launch
  int ld;                      // of X: L, or less where a sequence is one short chunk
  float bad, scale;
  int B, T, H, Dk, Dv, N;  // N chunks
  int lk, lv;
  int ctiles;              // column groups of a launch
};

// Operands are held in parts as linear attention's are; chunks are 64 positions
// for bfloat16, 32 where inputs have more parts than one.
__host__ __device__ constexpr int delta_parts(int dtype) {
  return dtype == SEMICRF_F32 ? 3 : dtype == SEMICRF_F16 ? 2 : 1;
}
__host__ __device__ constexpr int delta_chunk(int parts) { return parts > 1 ? 32 : 64; }
// Waves of a workgroup that walks along a sequence: one for 16 columns.
inline int delta_waves(int Dv) {
  return Dv <= 32 ? 2 : Dv <= 64 ? 4 : Dv <= 80 ? 5 : Dv <= 96 ? 6 : 8;
}

enum DeltaPass { DELTA_INVERSE, DELTA_COMPOSE, DELTA_FORWARD, DELTA_COMPOSE_BACK, DELTA_BACK, DELTA_GRADS };
semicrf_status_t delta_f32(const DeltaArgs &p, DeltaPass pass, hipStream_t st);
semicrf_status_t delta_bf16(const DeltaArgs &p, DeltaPass pass, hipStream_t st);
semicrf_status_t delta_f16(const DeltaArgs &p, DeltaPass pass, hipStream_t st);

namespace {

// part2 with one instruction for what an element's rounding leaves: the dot product
// with (-1, 0) or (0, -1), which is exact (the same bits for 2^22 values of all
// exponents).  Seven instructions in the place of eleven for a pair's three parts take
// a little longer, but fewer registers: for the operands that k_delta_grads makes of its
// accumulators, where it is short of them.  The constants are kept from being folded
// into the instruction, whose literals are not halves.
__device__ __forceinline__ b2 part2_dot(f2 &x) {
  unsigned first, second;
  asm("" : "=s"(first) : "0"(0x0000bf80u));
  asm("" : "=s"(second) : "0"(0xbf800000u));
  const b2 y = __builtin_convertvector(x, b2);
  x[0] = __builtin_amdgcn_fdot2_f32_bf16(y, __builtin_bit_cast(b2, first), x[0], false);
  x[1] = __builtin_amdgcn_fdot2_f32_bf16(y, __builtin_bit_cast(b2, second), x[1], false);
  return y;
}
template <bool DOT>
__device__ __forceinline__ b2 part2_of(f2 &x) {
  return DOT ? part2_dot(x) : part2(x);
}

template <int L>
struct Gates {
  float hi[L], lo[L], from[L], to[L], all, low, none[2];
  // e^{G_i - G_j}
  __device__ __forceinline__ float decay(int i, int j) const {
    return __expf((hi[i] - hi[j]) + (lo[i] - lo[j]));
  }
};
// Loads go through buffer descriptors, like Tile's: what is not wanted lies past the
// range and reads 0 without a branch.
__device__ __forceinline__ auto whole_range(const void *p) {
  return __builtin_amdgcn_make_buffer_rsrc((void *)p, 0, kRange, kRawBuffer);
}
template <int L, int NT>
struct GatesTile {
  static constexpr int all = delta_gates(L), N = (all + NT - 1) / NT;
  float r[N];
  __device__ __forceinline__ void fetch(int tid, const float *src) {
    const auto rsrc = whole_range(src);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int e = tid + k * NT;
      r[k] = __builtin_bit_cast(
          float, __builtin_amdgcn_raw_buffer_load_b32(rsrc, e < all ? 4 * e : -1, 0, 0));
    }
  }
  __device__ __forceinline__ void put(int tid, Gates<L> &g) const {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (tid + k * NT < all) (&g.hi[0])[tid + k * NT] = r[k];
  }
};

// A float32 matrix of `ROWS` rows (ld apart, 16 bytes aligned) and W columns, in three
// parts in LDS, zeros past n rows and D columns (a multiple of 4); LOWER: blocks of
// 32 above the diagonal are not read (nor written).
template <typename Lay, int W, int ROWS, int NT, bool LOWER>
struct Tile32 {
  static constexpr int per = W / 4, all = ROWS * per, N = (all + NT - 1) / NT;
  static constexpr int plane = ROWS * Lay::row;
  f4 r[N];
  __device__ __forceinline__ void fetch(int tid, const float *src, int ld, int n, int D) {
    const auto rsrc = whole_range(src);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int e = tid + k * NT, i = e / per, c = e % per * 4;
      const bool on = e < all && i < n && c < D && !(LOWER && c / 32 > i / 32);
      r[k] = __builtin_bit_cast(
          f4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, on ? 4 * (i * ld + c) : -1, 0, 0));
    }
  }
  __device__ __forceinline__ void put(int tid, bf16 *lds) const {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int e = tid + k * NT, i = e / per, c = e % per * 4;
      if ((all % NT && e >= all) || (LOWER && c / 32 > i / 32)) continue;
      f2 lo = {r[k][0], r[k][1]}, hi = {r[k][2], r[k][3]};
#pragma unroll
      for (int m = 0; m < 3; ++m) {
        const b2 a = part2(lo), b = part2(hi);
        *reinterpret_cast<Pack<bf16, 4> *>(lds + m * plane + Lay::at(i, c / 4)) =
            Pack<bf16, 4>{{a[0], a[1], b[0], b[1]}};
      }
    }
  }
};

// A number as something new to the compiler: what follows from it (addresses in
// LDS) is then computed again in every chunk instead of being kept in registers
// all along.  The load of a spilled register would wait for every tile on its way.
__device__ __forceinline__ int delta_fresh(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// What a beta of 0 counts as.  The write and its gradient are this times the value's and the
// incoming gradient's size and lose digits below 2^-126: those of up to 2^-62 keep theirs.
__device__ __forceinline__ float least_beta(float b) {
  return fabsf(b) < 0x1p-64f ? copysignf(0x1p-64f, b) : b;
}

// The tiles of 16 rows 2 b and 2 b + 1 of an accumulated matrix as an operand whose
// contraction runs over them.
template <bool DOT = false>
__device__ __forceinline__ Frag<3> frag_of(const f4 &a, const f4 &b) {
  Frag<3> f;
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    f2 r = e < 4 ? f2{a[e], a[e + 1]} : f2{b[e - 4], b[e - 3]};
#pragma unroll
    for (int n = 0; n < 3; ++n) {
      const b2 y = part2_of<DOT>(r);
      f.v[n][e] = y[0];
      f.v[n][e + 1] = y[1];
    }
  }
  return f;
}

// Zeros in the tiles (2 b, 2 b + 1) of three parts of an L x L matrix in LDS.
template <typename Lay, int L, int NT>
__device__ __forceinline__ void beside_diagonal(bf16 *P) {
  for (int e = threadIdx.x; e < 3 * L / 2 * 4; e += NT) {
    const int part = e / (2 * L), row = e / 4 % (L / 2), i = row / 16 * 32 + row % 16;
    *reinterpret_cast<Pack<bf16, 4> *>(P + part * L * Lay::row +
                                       Lay::at(i, row / 16 * 8 + 4 + e % 4)) = Pack<bf16, 4>{};
  }
}

template <typename T>
__device__ __forceinline__ const T *view_rows(const View &v, int b, int h) {
  return (const T *)v.p + (int64_t)b * v.sb + (int64_t)(h / v.share) * v.sh;
}

__device__ __forceinline__ f4 mfma32(float a, float b, f4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// x of another lane, 0 where there is none.
template <int CTRL, int ROWS = 15>
__device__ __forceinline__ float lanes(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, ROWS, 15, false));
}
// Sums up to a lane, of its 16 or of all 64; of those before it.
__device__ __forceinline__ float sum_row(float x) {
  x += lanes<0x111>(x);  // 1, 2, 4, 8 lanes before
  x += lanes<0x112>(x);
  x += lanes<0x114>(x);
  return x + lanes<0x118>(x);
}
__device__ __forceinline__ float sum_up(float x) {
  x = sum_row(x);
  x += lanes<0x142, 10>(x);  // the last of the row before, for the second and the fourth
  return x + lanes<0x143, 12>(x);  // the 32nd, for the upper half
}
__device__ __forceinline__ float exclusive(float x) { return lanes<0x138>(x); }  // one before

}  // namespace

// X = (I + diag(b) m)^-1 diag(b) (blocks of 32 up to the diagonal) and the gates of a
// chunk, a workgroup of four waves each.  M = diag(b) m on the matrix cores; its 16 x 16 blocks on the diagonal
// are inverted by substitution, a column a lane, and put together by
//   (I + M)^-1 = [T1, 0; -T2 M21 T1, T2]
// to 32 and 64 with float32 matrix instructions: what substitution gives, whatever
// the keys' lengths.  65536 chunks of 64 keys of 64 in bfloat16: 480 to 510 us, 1.3 GB
// read and written (2.6 TB/s).  A chunk is a chain of seven barriers, so occupancy counts: two
// workgroups a compute unit took 920 us; four, with the inverse in M's place, 710; the
// rest came from one wave for the diagonal's blocks, 16 lanes each, which left a
// lane a quarter of the registers.
template <typename T, int NP, int DK, int L>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(4))) void k_delta_inverse(
    DeltaArgs p) {
  constexpr int KB = DK / 32, NT = L / 16, LD = L + 4, LT = L / 2 + 4;
  typedef ByRow<DK> LK;
  // the inverse takes M's place block by block; T1 by columns, of tiles 0, 1 (whole)
  // and 2 (its first 16 rows); K is done with by then
  constexpr int kKeys = NP * L * LK::row, kCols = (L == 64 ? 48 : 16) * LT;
  __shared__ alignas(16) float M[L * LD];
  __shared__ alignas(16) float Xt[kCols > kKeys / 2 ? kCols : kKeys / 2];
  bf16 *const K = (bf16 *)Xt;
  __shared__ Gates<L> s;
  __shared__ float beta[L];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, g = lane >> 4, l16 = lane & 15;
  const int h = blockIdx.x % p.H, n = blockIdx.x / p.H % p.N, b = blockIdx.x / p.H / p.N;
  const int t0 = n * L, count = min(L, max(valid_length(p.lengths, b, p.T), 0) - t0);
  if (count <= 0) return;
  const int64_t at = ((int64_t)b * p.H + h) * p.N + n;
  const T *k = view_rows<T>(p.k, b, h) + t0 * p.k.st;
  Tile<T, NP, LK, DK, L, 256> tk;
  if (p.vec) tk.fetch(threadIdx.x, k, (int)p.k.st, p.Dk, count, 0, 1, 0);
  if (w == 0) {
    float gi = 0.f, bt = 0.f;
    if (lane < count) {
      const int64_t e = ((int64_t)b * p.T + t0 + lane) * p.H + h;
      gi = p.log_decay[e], bt = p.beta[e];
      if (gi < -200.f) gi = -200.f;
      bt = least_beta(bt);
    }
    double G = gi;
#pragma unroll
    for (int o = 1; o < L; o <<= 1) {
      const double y = __shfl_up(G, o);
      if (lane >= o) G += y;
    }
    if (lane < L) {
      const float hi = (float)G;
      s.hi[lane] = hi, s.lo[lane] = (float)(G - hi);
      beta[lane] = bt;
    }
  }
  if (p.vec)
    tk.put(threadIdx.x, K);
  else
    stage<T, NP, LK, DK, L, 256>(K, k, p.k.st, p.Dk, count, 0);
  __syncthreads();
  // M by rows: a tile is computed transposed, so that a lane holds four neighbours
  for (int t = w; t < NT * (NT + 1) / 2; t += 4) {
    int it = 0, jt = t;
    while (jt > it) jt -= ++it;
    f4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
      acc = mma<3>(frag_row<NP, LK>(K, L * LK::row, 16 * jt, kb, lane),
                   frag_row<NP, LK>(K, L * LK::row, 16 * it, kb, lane), acc);
    const int i = 16 * it + l16, j = 16 * jt + 4 * g;
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[r] = j + r < i ? beta[i] * s.decay(i, j + r) * acc[r] : 0.f;
    *reinterpret_cast<f4 *>(M + i * LD + j) = acc;
  }
  __syncthreads();
  if (w == 0 && g < NT) {
    float x[16];
    float *m = M + 16 * g * LD + 16 * g;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float y = i == l16 ? 1.f : 0.f;
#pragma unroll
      for (int l = 0; l < i; ++l) y = fmaf(-m[i * LD + l], x[l], y);
      x[i] = y;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) m[i * LD + l16] = x[i];
    if (g < kCols / LT / 16) {
      float *t = Xt + (16 * g + l16) * LT + 16 * g % (L / 2);
#pragma unroll
      for (int i = 0; i < 16; i += 4) *reinterpret_cast<f4 *>(t + i) = f4{x[i], x[i + 1], x[i + 2], x[i + 3]};
    }
  }
  __syncthreads();
  // blocks of n16 tiles beside each other: rows it, columns ct of the lower left
  // one of a pair
#pragma unroll
  for (int n16 = 1; n16 < NT; n16 *= 2) {
    const int pairs = NT / (2 * n16), jobs = pairs * n16 * n16;
    f4 out = {0.f, 0.f, 0.f, 0.f};
    int it = 0, ct = 0;
    if (w < jobs) {
      const int base = w / (n16 * n16) * 2 * n16;
      it = base + n16 + w / n16 % n16, ct = base + w % n16;
      for (int mt = base + n16; mt <= it; ++mt) {
        f4 y = {0.f, 0.f, 0.f, 0.f};  // rows of tile mt of M21 T1
        for (int jt = ct; jt < base + n16; ++jt) {
          const f4 a = *reinterpret_cast<const f4 *>(M + (16 * mt + l16) * LD + 16 * jt + 4 * g);
          const f4 c = *reinterpret_cast<const f4 *>(Xt + (16 * ct + l16) * LT +
                                                     (16 * jt + 4 * g) % (L / 2));
#pragma unroll
          for (int r = 0; r < 4; ++r) y = mfma32(a[r], c[r], y);
        }
        const f4 a = *reinterpret_cast<const f4 *>(M + (16 * it + l16) * LD + 16 * mt + 4 * g);
#pragma unroll
        for (int r = 0; r < 4; ++r) out = mfma32(a[r], -y[r], out);
      }
    }
    __syncthreads();
    if (w < jobs) {
#pragma unroll
      for (int r = 0; r < 4; ++r) M[(16 * it + 4 * g + r) * LD + 16 * ct + l16] = out[r];
      if (it < NT / 2) *reinterpret_cast<f4 *>(Xt + (16 * ct + l16) * LT + 16 * it + 4 * g) = out;
    }
    __syncthreads();
  }
  // the other gates, for the walks: e^{hi + lo} = e^hi (1 + lo)
  float *out = p.gates + at * delta_gates(L);
  if (lane < L) {
    const float hi = s.hi[lane], lo = s.lo[lane];
    if (w == 0) out[lane] = hi, out[L + lane] = lo;
    if (w == 1) out[2 * L + lane] = fmaf(expf(hi), lo, expf(hi));
    if (w == 2) {
      const double d = ((double)s.hi[L - 1] - hi) + ((double)s.lo[L - 1] - lo);
      const float x = (float)d, y = expf(x);
      out[3 * L + lane] = fmaf(y, (float)(d - x), y);
    }
    if (w == 3 && lane < 4) {
      const double all = exp((double)s.hi[L - 1] + s.lo[L - 1]);
      const float x = (float)all;
      out[4 * L + lane] = lane == 0 ? x : lane == 1 ? (float)(all - x) : 0.f;
    }
  }
  const int ld = p.ld;
  for (int e = threadIdx.x; e < ld * ld / 4; e += 256) {
    const int i = e / (ld / 4), j = e % (ld / 4) * 4;
    if (j / 32 > i / 32) continue;  // not read
    f4 x = *reinterpret_cast<const f4 *>(M + i * LD + j);
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] = j / 16 > i / 16 ? 0.f : x[r] * beta[j + r];
    *reinterpret_cast<f4 *>(p.X + at * ld * ld + i * ld + j) = x;
  }
}

// The chunks of a segment one after another, 16 columns of the state a wave, in
// accumulators from the first chunk to the last.  COMPOSE: 16 columns of the
// segment's transition phi, from I with values of 0, and of its sum, from 0: two
// independent chains that read the same operands; else the outputs (and what the
// backward pass reads again) from the state before it.
//
// A chunk of 64 x 64 in bfloat16 is 150 matrix instructions a wave (2400 cycles) and
// 1260 vector ones, a third of them the splitting of S, R and U into parts.  2^20
// positions of 4 heads, two workgroups of four waves a compute unit (80 KB of LDS):
// 1.06 to 1.17 ms, 9 us a chunk, vector units busy 66 %; composing 0.89 to 0.96 ms, 85 %.
// Measured on the way: addresses computed again in each chunk and no spilled register
// 1.56 -> 1.20 ms; both chains in one wave when composing 1.19 -> 0.95; part2_dot in
// the place of part2 3 % more.
template <typename T, int NP, int DK, int NW, int L, bool COMPOSE>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(2))) void k_delta_chunks(DeltaArgs p) {
  constexpr int kCols = 16 * NW, kThreads = 64 * NW;
  constexpr int KB = DK / 32, NT = L / 16, JB = L / 32, NC = COMPOSE ? 2 : 1;
  constexpr int TILES = NT * (NT + 1) / 2;
  // operands of three parts are not read far ahead (the barriers to the scheduler)
  // where 128 rows of state leave no registers for them: 250 bytes a lane were spilled
  // (4 x 8192 positions of 4 heads of 128 x 64: 333 -> 309 us)
  constexpr bool kTight = NP == 3 && DK > 64;
  typedef ByBoth<DK> LK;
  typedef ByRow<DK> LQ;
  typedef ByColumn<kCols> LV;
  typedef ByRow<L> LX;
  __shared__ alignas(16) bf16 K[NP * L * LK::row];
  __shared__ alignas(16) bf16 V[NP * L * LV::row];
  __shared__ alignas(16) bf16 X[3 * L * LX::row];
  __shared__ alignas(16) bf16 Q[COMPOSE ? 8 : NP * L * LQ::row];
  __shared__ alignas(16) bf16 P[COMPOSE ? 8 : 3 * L * LX::row];
  __shared__ Gates<L> gs;

  const int tid = threadIdx.x, w = tid >> 6, g0 = (tid & 63) >> 4, l0 = tid & 15;
  const int ct = blockIdx.x % p.ctiles;
  const int seg = p.first + blockIdx.x / p.ctiles % p.count;
  const int64_t bh = blockIdx.x / p.ctiles / p.count;
  const int h = (int)(bh % p.H), b = (int)(bh / p.H);
  const int c0 = ct * kCols, xc = c0 + 16 * w + l0;
  const int valid = valid_length(p.lengths, b, p.T), len = max(valid, 0);
  const int chunks = (len + L - 1) / L;
  const int lo = seg * p.seg, hi = min(chunks, lo + p.seg);

  const T *q = view_rows<T>(p.q, b, h), *k = view_rows<T>(p.k, b, h), *v = view_rows<T>(p.v, b, h);
  Tile<T, NP, LK, DK, L, kThreads> tk;
  Tile<T, NP, LQ, DK, L, kThreads> tq;
  Tile<T, NP, LV, kCols, L, kThreads> tv;
  Tile32<LX, L, L, kThreads, true> tx;
  GatesTile<L, kThreads> tg;
  auto fetch = [&](int n) {
    const int tid = delta_fresh(threadIdx.x);
    const int64_t t0 = (int64_t)n * L;
    const int m = (int)min((int64_t)L, len - t0);
    const int64_t at = bh * p.N + n;
    tg.fetch(tid, p.gates + at * delta_gates(L));
    tx.fetch(tid, p.X + at * p.ld * p.ld, p.ld, p.ld, p.ld);
    if (!p.vec) return;
    tk.fetch(tid, k + t0 * p.k.st, (int)p.k.st, p.Dk, m, 0, 1, 0);
    if (!COMPOSE) tq.fetch(tid, q + t0 * p.q.st, (int)p.q.st, p.Dk, m, 0, 1, 0);
    tv.fetch(tid, v + t0 * p.v.st, (int)p.v.st, p.Dv, m, 0, 1, c0);
  };
  auto put = [&](int n) {
    const int tid = delta_fresh(threadIdx.x);
    tg.put(tid, gs);
    tx.put(tid, X);
    if (p.vec) {
      tk.put(tid, K);
      if (!COMPOSE) tq.put(tid, Q);
      tv.put(tid, V);
    } else {
      const int64_t t0 = (int64_t)n * L;
      const int m = (int)min((int64_t)L, len - t0);
      stage<T, NP, LK, DK, L, kThreads>(K, k + t0 * p.k.st, p.k.st, p.Dk, m, 0);
      if (!COMPOSE) stage<T, NP, LQ, DK, L, kThreads>(Q, q + t0 * p.q.st, p.q.st, p.Dk, m, 0);
      stage<T, NP, LV, kCols, L, kThreads>(V, v + t0 * p.v.st, p.v.st, p.Dv, m, c0);
    }
  };
  if (lo < hi) fetch(lo);

  // state tile i: rows 16 i + 4 g + r of column xc
  f4 S[NC][2 * KB];
  const int64_t size = (int64_t)p.Dk * p.lv;
  const float *s0 = COMPOSE ? nullptr
                    : seg   ? p.xs + (bh * p.nseg + seg - 1) * size
                            : p.state_in ? p.state_in + bh * p.Dk * p.Dv : nullptr;
  const int l0v = seg ? p.lv : p.Dv;
#pragma unroll
  for (int i = 0; i < 2 * KB; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * i + 4 * g0 + r;
      S[0][i][r] = s0 && row < p.Dk && xc < p.Dv ? s0[row * l0v + xc] : 0.f;
      if (NC > 1) S[NC - 1][i][r] = row == xc ? 1.f : 0.f;  // phi
    }
  if (lo < hi) put(lo);
  // the tiles of P beside the diagonal that products of 32 columns read
  if (!COMPOSE) beside_diagonal<LX, L, kThreads>(P);

  T *out = (T *)p.o + ((int64_t)b * p.T * p.H + h) * p.Dv;
  const int64_t so = (int64_t)p.H * p.Dv;
  for (int n = lo; n < hi; ++n) {
    const int m = min(L, len - n * L);
    __syncthreads();
    const int lane = DK <= 64 ? tid & 63 : delta_fresh(tid & 63), g = lane >> 4, l16 = lane & 15;
    if (n + 1 < hi) fetch(n + 1);
    if (!COMPOSE && p.S && xc < p.Dv) {
      float *to = p.S + ((bh * p.N + n) * p.Dv + xc) * p.lk + 4 * g;
#pragma unroll
      for (int i = 0; i < 2 * KB; ++i)
        if (16 * i + 4 * g < p.lk) *reinterpret_cast<f4 *>(to + 16 * i) = S[0][i];
    }
    if (!COMPOSE) {
      // P, up to the diagonal, a tile a wave at a time (of bfloat16 the last one again
      // where they do not divide: without a branch, the chain's products go in between)
#pragma unroll
      for (int n = 0; n < (TILES + NW - 1) / NW; ++n) {
        if (NP > 1 && w + n * NW >= TILES) break;
        const int t = min(w + n * NW, TILES - 1);
        const int it = (t > 0) + (t > 2) + (t > 5), jt = t - it * (it + 1) / 2;
        f4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
          acc = mma<3>(frag_row<NP, LK>(K, L * LK::row, 16 * jt, kb, lane),
                       frag_row<NP, LQ>(Q, L * LQ::row, 16 * it, kb, lane), acc);
        const int i = 16 * it + l16, j = 16 * jt + 4 * g;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[r] = j + r <= i ? p.scale * gs.decay(i, j + r) * acc[r] : 0.f;
        f2 x = {acc[0], acc[1]}, y = {acc[2], acc[3]};
#pragma unroll
        for (int c = 0; c < 3; ++c) {
          const b2 a = part2(x), d = part2(y);
          *reinterpret_cast<Pack<bf16, 4> *>(P + c * L * LX::row + LX::at(i, 4 * jt + g)) =
              Pack<bf16, 4>{{a[0], a[1], d[0], d[1]}};
        }
      }
    }
    Frag<3> sf[NC][KB];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) sf[c][kb] = frag_of(S[c][2 * kb], S[c][2 * kb + 1]);
    // R = V - E K S
    Frag<3> rf[NC][JB];
#pragma unroll
    for (int jb = 0; jb < JB; ++jb) {
      f4 ks[NC][2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int c = 0; c < NC; ++c) ks[c][t] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          const Frag<NP> kf = frag_row<NP, LK>(K, L * LK::row, 32 * jb + 16 * t, kb, lane);
#pragma unroll
          for (int c = 0; c < NC; ++c) ks[c][t] = mma<3>(kf, sf[c][kb], ks[c][t]);
          if (kTight) __builtin_amdgcn_sched_barrier(0);
        }
      }
      float v8[8];
      values(frag_col<NP, LV>(V, L * LV::row, 32 * jb, w, lane), v8);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          x[e] = (c ? 0.f : v8[e]) -
                 gs.from[32 * jb + 16 * (e >> 2) + 4 * g + (e & 3)] * ks[c][e >> 2][e & 3];
        rf[c][jb] = split<3>(x);
      }
    }
    // what the state gives, transposed: a lane holds four neighbours of a row of O
    f4 O[NT];
    if (!COMPOSE) {
#pragma unroll
      for (int it = 0; it < NT; ++it) {
        O[it] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
        {
          O[it] = mma<3>(sf[0][kb], frag_row<NP, LQ>(Q, L * LQ::row, 16 * it, kb, lane), O[it]);
          if (kTight) __builtin_amdgcn_sched_barrier(0);
        }
        const float d = p.scale * gs.from[16 * it + l16];
#pragma unroll
        for (int r = 0; r < 4; ++r) O[it][r] *= d;
      }
    }
    // U = X R
    f4 U[NC][NT];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int it = 0; it < NT; ++it) U[c][it] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int jb = 0; jb < JB; ++jb)
#pragma unroll
      for (int it = 2 * jb; it < NT; ++it) {
        const Frag<3> xf = frag_row<3, LX>(X, L * LX::row, 16 * it, jb, lane);
#pragma unroll
        for (int c = 0; c < NC; ++c) U[c][it] = mma<3>(xf, rf[c][jb], U[c][it]);
      }
    if (!COMPOSE && p.U && xc < p.Dv) {
      float *to = p.U + ((bh * p.N + n) * p.Dv + xc) * L + 4 * g;
#pragma unroll
      for (int it = 0; it < NT; ++it) *reinterpret_cast<f4 *>(to + 16 * it) = U[0][it];
    }
    // S <- e^{G_L} S + K^T (e^{G_L - G} U)
    Frag<3> uf[JB];
    const float all = gs.all, low = gs.low;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 2 * KB; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[c][i][r] = fmaf(S[c][i][r], low, S[c][i][r] * all);
#pragma unroll
    for (int jb = 0; jb < JB; ++jb) {
      if (!COMPOSE) uf[jb] = frag_of(U[0][2 * jb], U[0][2 * jb + 1]);
      Frag<3> tf[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          x[e] = U[c][2 * jb + (e >> 2)][e & 3] * gs.to[32 * jb + 16 * (e >> 2) + 4 * g + (e & 3)];
        tf[c] = split<3>(x);
      }
#pragma unroll
      for (int i = 0; i < 2 * KB; ++i) {
        const Frag<NP> kf = frag_col<NP, LK>(K, L * LK::row, 32 * jb, i, lane);
#pragma unroll
        for (int c = 0; c < NC; ++c) S[c][i] = mma<3>(kf, tf[c], S[c][i]);
        if (kTight) __builtin_amdgcn_sched_barrier(0);
      }
    }
    __syncthreads();
    if (!COMPOSE) {
      const int col = c0 + 16 * w + 4 * g;
#pragma unroll
      for (int it = 0; it < NT; ++it) {
        const int i = 16 * it + l16;
#pragma unroll
        for (int jb = 0; jb <= it / 2; ++jb)
          O[it] = mma<3>(uf[jb], frag_row<3, LX>(P, L * LX::row, 16 * it, jb, lane), O[it]);
        if (i < m && col < p.Dv) {
          T *to = out + ((int64_t)n * L + i) * so + col;
          if (p.vec) {
            Pack<T, 4> x;
#pragma unroll
            for (int r = 0; r < 4; ++r) x.v[r] = (T)O[it][r];
            *reinterpret_cast<Pack<T, 4> *>(to) = x;
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (col + r < p.Dv) to[r] = (T)O[it][r];
          }
        }
      }
    }
    if (n + 1 < hi) put(n + 1);
  }

  if (COMPOSE) {
    float *sum = p.xs + (bh * p.nseg + seg) * size;
    const int64_t at = (bh * p.nseg + seg) * p.Dk * p.lk;
#pragma unroll
    for (int i = 0; i < 2 * KB; ++i) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * i + 4 * g0 + r;
        if (row < p.Dk && xc < p.lv) sum[row * p.lv + xc] = S[0][i][r];
        if (row < p.Dk && xc < p.lk) p.phi[at + row * p.lk + xc] = S[NC - 1][i][r];
      }
      if (p.phit && 16 * i + 4 * g0 < p.lk && xc < p.Dk)
        *reinterpret_cast<f4 *>(p.phit + at + xc * p.lk + 16 * i + 4 * g0) = S[NC - 1][i];
    }
    return;
  }
  const T fill = (T)(valid < 0 ? p.bad : 0.f);
  const int64_t f0 = max((int64_t)len, (int64_t)lo * L),
                f1 = min((int64_t)p.T, ((int64_t)lo + p.seg) * L);
  for (int64_t e = threadIdx.x; e < (f1 - f0) * kCols; e += kThreads) {
    const int col = c0 + (int)(e % kCols);
    if (col < p.Dv) out[(f0 + e / kCols) * so + col] = fill;
  }
  // the segment that holds the last valid position (the first, if none)
  if (p.state_out && hi == chunks && (lo < chunks || seg == 0)) {
#pragma unroll
    for (int i = 0; i < 2 * KB; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * i + 4 * g0 + r;
        if (row < p.Dk && xc < p.Dv)
          p.state_out[(bh * p.Dk + row) * p.Dv + xc] = valid < 0 ? p.bad : S[0][i][r];
      }
  }
}

// The chunks of a segment from the last to the first, 16 columns of the gradient
// of the state a wave.  COMPOSE: from 0 to what the segment adds; else from the
// gradient after the segment, leaving that after each chunk in D, the gradients of
// R in R and of the values in dv.  Bound as k_delta_chunks is: 16 x 4096 positions of 4
// heads of 64 in bfloat16 99 us, composing 64 (80004 positions of 4 heads of 40 x 72 in
// float32: 250 and 180).
template <typename T, int NP, int DK, int NW, int L, bool COMPOSE>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(2))) void k_delta_back(DeltaArgs p) {
  constexpr int kCols = 16 * NW, kThreads = 64 * NW;
  constexpr int KB = DK / 32, NT = L / 16, JB = L / 32, TILES = NT * (NT + 1) / 2;
  typedef ByBoth<DK> LK;
  typedef ByColumn<kCols> LV;
  typedef ByBoth<L> LX;
  __shared__ alignas(16) bf16 K[NP * L * LK::row];
  __shared__ alignas(16) bf16 Q[NP * L * LK::row];
  __shared__ alignas(16) bf16 G[NP * L * LV::row];
  __shared__ alignas(16) bf16 X[3 * L * LX::row];
  __shared__ alignas(16) bf16 P[3 * L * LX::row];
  __shared__ Gates<L> gs;

  const int tid = threadIdx.x, w = tid >> 6, g0 = (tid & 63) >> 4, l0 = tid & 15;
  const int ct = blockIdx.x % p.ctiles, seg = p.first + blockIdx.x / p.ctiles % p.count;
  const int64_t bh = blockIdx.x / p.ctiles / p.count;
  const int h = (int)(bh % p.H), b = (int)(bh / p.H);
  const int c0 = ct * kCols, xc = c0 + 16 * w + l0;
  const int valid = valid_length(p.lengths, b, p.T), len = max(valid, 0);
  const int chunks = (len + L - 1) / L;
  const int lo = seg * p.seg, hi = min(chunks, lo + p.seg);

  const T *q = view_rows<T>(p.q, b, h), *k = view_rows<T>(p.k, b, h);
  const int64_t so = (int64_t)p.H * p.Dv;
  const T *go = (const T *)p.go + ((int64_t)b * p.T * p.H + h) * p.Dv;
  Tile<T, NP, LK, DK, L, kThreads> tk, tq;
  Tile<T, NP, LV, kCols, L, kThreads> to;
  Tile32<LX, L, L, kThreads, true> tx;
  GatesTile<L, kThreads> tg;
  auto fetch = [&](int n) {
    const int tid = delta_fresh(threadIdx.x);
    const int64_t t0 = (int64_t)n * L;
    const int m = (int)min((int64_t)L, len - t0);
    const int64_t at = bh * p.N + n;
    tg.fetch(tid, p.gates + at * delta_gates(L));
    tx.fetch(tid, p.X + at * p.ld * p.ld, p.ld, p.ld, p.ld);
    if (!p.vec) return;
    tk.fetch(tid, k + t0 * p.k.st, (int)p.k.st, p.Dk, m, 0, 1, 0);
    tq.fetch(tid, q + t0 * p.q.st, (int)p.q.st, p.Dk, m, 0, 1, 0);
    to.fetch(tid, go + t0 * so, (int)so, p.Dv, m, 0, 1, c0);
  };
  auto put = [&](int n) {
    const int tid = delta_fresh(threadIdx.x);
    tg.put(tid, gs);
    tx.put(tid, X);
    if (p.vec) {
      tk.put(tid, K);
      tq.put(tid, Q);
      to.put(tid, G);
    } else {
      const int64_t t0 = (int64_t)n * L;
      const int m = (int)min((int64_t)L, len - t0);
      stage<T, NP, LK, DK, L, kThreads>(K, k + t0 * p.k.st, p.k.st, p.Dk, m, 0);
      stage<T, NP, LK, DK, L, kThreads>(Q, q + t0 * p.q.st, p.q.st, p.Dk, m, 0);
      stage<T, NP, LV, kCols, L, kThreads>(G, go + t0 * so, so, p.Dv, m, c0);
    }
  };
  if (lo < hi) fetch(hi - 1);
  f4 D[2 * KB];
  const int64_t size = (int64_t)p.Dk * p.lv;
  const float *d0 = COMPOSE              ? nullptr
                    : seg + 1 < p.nseg   ? p.xs + (bh * p.nseg + seg + 1) * size
                            : p.state_in ? p.state_in + bh * p.Dk * p.Dv : nullptr;
  const int l0v = seg + 1 < p.nseg ? p.lv : p.Dv;
#pragma unroll
  for (int i = 0; i < 2 * KB; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * i + 4 * g0 + r;
      D[i][r] = d0 && row < p.Dk && xc < p.Dv ? d0[row * l0v + xc] : 0.f;
    }
  if (lo < hi) put(hi - 1);
  beside_diagonal<LX, L, kThreads>(P);

  for (int n = hi - 1; n >= lo; --n) {
    const int m = min(L, len - n * L);
    __syncthreads();
    const int lane = DK <= 64 ? tid & 63 : delta_fresh(tid & 63), g = lane >> 4, l16 = lane & 15;
    if (n > lo) fetch(n - 1);
    if (!COMPOSE && xc < p.Dv) {
      float *at = p.D + ((bh * p.N + n) * p.Dv + xc) * p.lk + 4 * g;
#pragma unroll
      for (int i = 0; i < 2 * KB; ++i)
        if (16 * i + 4 * g < p.lk) *reinterpret_cast<f4 *>(at + 16 * i) = D[i];
    }
    // P, as k_delta_chunks has it
#pragma unroll
    for (int n = 0; n < (TILES + NW - 1) / NW; ++n) {
      if (NP > 1 && w + n * NW >= TILES) break;
      const int t = min(w + n * NW, TILES - 1);
      const int it = (t > 0) + (t > 2) + (t > 5), jt = t - it * (it + 1) / 2;
      f4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
        acc = mma<3>(frag_row<NP, LK>(K, L * LK::row, 16 * jt, kb, lane),
                     frag_row<NP, LK>(Q, L * LK::row, 16 * it, kb, lane), acc);
      const int i = 16 * it + l16, j = 16 * jt + 4 * g;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        acc[r] = j + r <= i ? p.scale * gs.decay(i, j + r) * acc[r] : 0.f;
      f2 x = {acc[0], acc[1]}, y = {acc[2], acc[3]};
#pragma unroll
      for (int c = 0; c < 3; ++c) {
        const b2 a = part2(x), d = part2(y);
        *reinterpret_cast<Pack<bf16, 4> *>(P + c * L * LX::row + LX::at(i, 4 * jt + g)) =
            Pack<bf16, 4>{{a[0], a[1], d[0], d[1]}};
      }
    }
    // dU = P^T dO + e^{G_L - G} K dS
    f4 dU[NT];
#pragma unroll
    for (int jt = 0; jt < NT; ++jt) dU[jt] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      const Frag<3> df = frag_of(D[2 * kb], D[2 * kb + 1]);
#pragma unroll
      for (int jt = 0; jt < NT; ++jt)
        dU[jt] = mma<3>(frag_row<NP, LK>(K, L * LK::row, 16 * jt, kb, lane), df, dU[jt]);
    }
#pragma unroll
    for (int jt = 0; jt < NT; ++jt)
#pragma unroll
      for (int r = 0; r < 4; ++r) dU[jt][r] *= gs.to[16 * jt + 4 * g + r];
    // dS <- e^{G_L} dS + scale (E Q)^T dO - (E K)^T dR
    const float all = gs.all, low = gs.low;
#pragma unroll
    for (int i = 0; i < 2 * KB; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) D[i][r] = fmaf(D[i][r], low, D[i][r] * all);
    Frag<NP> gf[JB];
#pragma unroll
    for (int ib = 0; ib < JB; ++ib) {
      gf[ib] = frag_col<NP, LV>(G, L * LV::row, 32 * ib, w, lane);
      float x[8];
      values(gf[ib], x);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[e] *= p.scale * gs.from[32 * ib + 16 * (e >> 2) + 4 * g + (e & 3)];
      const Frag<3> ef = split<3>(x);
#pragma unroll
      for (int i = 0; i < 2 * KB; ++i)
        D[i] = mma<3>(frag_col<NP, LK>(Q, L * LK::row, 32 * ib, i, lane), ef, D[i]);
    }
    __syncthreads();
#pragma unroll
    for (int ib = 0; ib < JB; ++ib)
#pragma unroll
      for (int jt = 0; jt <= 2 * ib + 1; ++jt)
        dU[jt] = mma<3>(frag_col<3, LX>(P, L * LX::row, 32 * ib, jt, lane), gf[ib], dU[jt]);
    f4 dR[NT];
#pragma unroll
    for (int jt = 0; jt < NT; ++jt) dR[jt] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ib = 0; ib < JB; ++ib) {
      const Frag<3> df = frag_of(dU[2 * ib], dU[2 * ib + 1]);
#pragma unroll
      for (int jt = 0; jt <= 2 * ib + 1; ++jt)
        dR[jt] = mma<3>(frag_col<3, LX>(X, L * LX::row, 32 * ib, jt, lane), df, dR[jt]);
    }
    if (!COMPOSE && xc < p.Dv) {
      float *at = p.R + ((bh * p.N + n) * p.Dv + xc) * L + 4 * g;
#pragma unroll
      for (int jt = 0; jt < NT; ++jt) {
        *reinterpret_cast<f4 *>(at + 16 * jt) = dR[jt];
        if (!p.dv) continue;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = 16 * jt + 4 * g + r;
          if (j >= m) continue;
          const int64_t e = (((int64_t)b * p.T + n * (int64_t)L + j) * p.H + h) * p.Dv + xc;
          if (p.part_v)
            ((float *)p.dv)[e] = dR[jt][r];
          else
            ((T *)p.dv)[e] = (T)dR[jt][r];
        }
      }
    }
#pragma unroll
    for (int jb = 0; jb < JB; ++jb) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[e] = dR[2 * jb + (e >> 2)][e & 3] * -gs.from[32 * jb + 16 * (e >> 2) + 4 * g + (e & 3)];
      const Frag<3> rf = split<3>(x);
#pragma unroll
      for (int i = 0; i < 2 * KB; ++i)
        D[i] = mma<3>(frag_col<NP, LK>(K, L * LK::row, 32 * jb, i, lane), rf, D[i]);
    }
    __syncthreads();
    if (n > lo) put(n - 1);
  }

  float *to_d = COMPOSE ? p.xs + (bh * p.nseg + seg) * size
                : p.state_out && seg == 0 ? p.state_out + bh * p.Dk * p.Dv : nullptr;
  const int ld = COMPOSE ? p.lv : p.Dv;
  if (to_d && xc < ld) {
#pragma unroll
    for (int i = 0; i < 2 * KB; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * i + 4 * g0 + r;
        if (row < p.Dk) to_d[row * ld + xc] = !COMPOSE && valid < 0 ? p.bad : D[i][r];
      }
  }
  if (!COMPOSE && p.dv) {
    const int64_t f0 = max((int64_t)len, (int64_t)lo * L),
                  f1 = min((int64_t)p.T, ((int64_t)lo + p.seg) * L);
    for (int64_t e = threadIdx.x; e < (f1 - f0) * kCols; e += kThreads) {
      const int col = c0 + (int)(e % kCols);
      if (col >= p.Dv) continue;
      const int64_t to = (((int64_t)b * p.T + f0 + e / kCols) * p.H + h) * p.Dv + col;
      if (p.part_v)
        ((float *)p.dv)[to] = 0.f;
      else
        ((T *)p.dv)[to] = (T)0.f;
    }
  }
}

// The gradients of q, k, the log decays and betas of a chunk, eight waves each.  Half
// of the waves have rows of 16 positions that ask (dq, and what dM and the state
// give to dk), half have rows that are asked (the rest of dk); for L = 32 two
// waves share the keys' columns of a row.  Contractions over the values' columns
// go in slices of 32.  dP and dM are computed by rows by the first and by columns
// by the others: the accumulators' layout is then that of the operand they become,
// and the triangles' rows and columns on a SIMD add up to the same.
//
// The decays' gradients are sums over rectangles of a triangle (i >= t > j).  With rows and columns
// in tiles of 16 they are what a row has from the tiles before its own, what a column has from
// the tiles of rows below, a whole tile, and in the diagonal tile the product with a triangle of
// ones on the matrix cores, then sums over 16 lanes: no scan along a row.
//
// Bound by the wait for its loads: 4096 chunks of 64 x 64 in bfloat16 are 430 MB, 84 us
// at a copy's rate, and take 136 to 139 with two workgroups of eight waves a compute unit (6 of them
// for the decays' rectangles; 18 with scans by shuffles, 13 with 8-byte reads of the rows, which
// conflict).  Before the rectangles: 130; 185 with four waves and all triangles twice, 177 with one
// workgroup, 225 with the next slice's loads ahead (accumulators spilled).
template <typename T, int NP, int DK, int L>
__global__ __launch_bounds__(512)
    __attribute__((amdgpu_waves_per_eu(NP == 1 && DK > 64 ? 2 : 4))) void k_delta_grads(DeltaArgs p) {
  constexpr int NT = L / 16, JB = L / 32, DS = 4 / NT, DT = DK / 16 / DS, kThreads = 512;
  typedef ByRow<32> LG;
  // 32 columns of U and R as rows of L; of S and D of DK.  Padded, they take fewer
  // registers for addresses; at DK = 128 a second workgroup has room without (but for one part).
  typedef std::conditional_t<(DK <= 64), ByColumn<L>, ByBoth<L>> LU;
  typedef std::conditional_t<(DK <= 64), ByColumn<DK>, ByBoth<DK>> LS;
  // keys and queries are read by rows and by columns: rows of one part 16 bytes at a time, which
  // the padding serves, of more parts 8, for which padded rows would have four lanes on a bank
  // (80004 positions of 4 heads of 40 x 72 in float32: 338 -> 325 us)
  typedef std::conditional_t<(NP == 1), ByColumn<DK>, ByBoth<DK>> LK;
  constexpr int PU = 32 * LU::row, PS = 32 * LS::row;
  constexpr int kSlice = 6 * PU + 6 * PS + NP * L * LG::row;
  constexpr int kKeys = 2 * NP * L * LK::row, LW = DK + 4, kAfter = kKeys + 2 * L * LW;
  __shared__ alignas(16) bf16 tiles[kSlice > kAfter ? kSlice : kAfter];
  bf16 *const U = tiles, *const R = U + 3 * PU, *const S = R + 3 * PU, *const D = S + 3 * PS,
             *const G = D + 3 * PS;
  // after the slices: the keys, the queries and the others' share of dk
  bf16 *const K = tiles, *const Q = K + NP * L * LK::row;
  float *const dks = (float *)(tiles + kKeys);
  __shared__ Gates<L> gs;
  __shared__ alignas(16) float inv[L], dbs[8][L];
  __shared__ float decays[L];
  __shared__ double red[8];
  // d g_t by its terms: what positions from t on ask of the state, what those before t
  // give to the state after, and what those before t give to those from t on (by tiles
  // of rows; a row's before its own tile)
  __shared__ float as[DS][L], es[DS][L], rs[DS][NT][L], ps[DS][L];

  const int tid = threadIdx.x, w = tid >> 6;
  const int h = blockIdx.x % p.H, n = blockIdx.x / p.H % p.N, b = blockIdx.x / p.H / p.N;
  const int t0 = n * L, count = min(L, max(valid_length(p.lengths, b, p.T), 0) - t0);
  const int rest = min(L, p.T - t0);
  const int64_t row0 = ((int64_t)b * p.T + t0) * p.H + h;
  for (int e = max(count, 0) * p.Dk + tid; e < rest * p.Dk; e += kThreads) {
    const int64_t row = row0 + (int64_t)(e / p.Dk) * p.H, to = row * p.Dk + e % p.Dk;
    if (p.dq) { if (p.part_q) ((float *)p.dq)[to] = 0.f; else ((T *)p.dq)[to] = (T)0.f; }
    if (p.dk) { if (p.part_k) ((float *)p.dk)[to] = 0.f; else ((T *)p.dk)[to] = (T)0.f; }
    if (e % p.Dk == 0 && p.dg) p.dg[row] = 0.f;
    if (e % p.Dk == 0 && p.db) p.db[row] = 0.f;
  }
  if (count <= 0) return;
  const int64_t at = ((int64_t)b * p.H + h) * p.N + n, size = (int64_t)p.Dv * p.lk;
  const T *q = view_rows<T>(p.q, b, h) + t0 * p.q.st, *k = view_rows<T>(p.k, b, h) + t0 * p.k.st;
  const int64_t so = (int64_t)p.H * p.Dv;
  const T *go = (const T *)p.go + row0 * p.Dv;
  const float *u = p.U + at * L * p.Dv, *dr = p.R + at * L * p.Dv, *s = p.S + at * size,
              *ds = p.D + at * size;
  Tile32<LU, L, 32, kThreads, false> tu, tr;
  Tile32<LS, DK, 32, kThreads, false> ts, td;
  Tile<T, NP, LG, 32, L, kThreads> tg;
  Tile<T, NP, LK, DK, L, kThreads> tk, tq;
  auto fetch = [&](int c0) {
    const int tid = delta_fresh(threadIdx.x);
    tu.fetch(tid, u + c0 * L, L, p.Dv - c0, L);
    tr.fetch(tid, dr + c0 * L, L, p.Dv - c0, L);
    ts.fetch(tid, s + c0 * p.lk, p.lk, p.Dv - c0, p.lk);
    td.fetch(tid, ds + c0 * p.lk, p.lk, p.Dv - c0, p.lk);
    if (p.vec) tg.fetch(tid, go, (int)so, p.Dv, count, 0, 1, c0);
  };
  if (tid < L) {
    float bt = 1.f, gi = 0.f;
    if (tid < count) {
      const int64_t row = row0 + (int64_t)tid * p.H;
      bt = p.beta[row], gi = p.log_decay[row];
    }
    inv[tid] = 1.f / least_beta(bt);
    decays[tid] = gi;
  }
  if (tid < delta_gates(L)) (&gs.hi[0])[tid] = p.gates[at * delta_gates(L) + tid];
  const int pt = w % NT, part = w / NT / 2, d0 = part * DT;
  const bool asks = w / NT % 2 == 0;
  // of rows that ask: dq and its like from dR; of the others: what is written
  f4 a0[DT], a1[DT], p0[NT], p1[NT];
  const f4 zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < DT; ++i) a0[i] = a1[i] = zero;
#pragma unroll
  for (int i = 0; i < NT; ++i) p0[i] = p1[i] = zero;
  static_assert(decltype(tu)::N == 1, "");
  float dot = 0.f;  // S . dS', this thread's share: a few products a slice
  f4 db4 = zero;   // (dR / b) . (U / b) of four positions, this thread's columns
  // no slice ahead: the registers it would take are worth more as the second
  // workgroup's on the compute unit
  for (int c0 = 0; c0 < p.Dv; c0 += 32) {
    fetch(c0);
    __syncthreads();
    {
      const int tid = delta_fresh(threadIdx.x);
      // one after another (the barriers to the scheduler): 128 registers are all there
      // are, and a spilled accumulator costs more than the wait
      tu.put(tid, U);
      __builtin_amdgcn_sched_barrier(0);
      tr.put(tid, R);
      __builtin_amdgcn_sched_barrier(0);
      ts.put(tid, S);
      __builtin_amdgcn_sched_barrier(0);
      td.put(tid, D);
      __builtin_amdgcn_sched_barrier(0);
      if (p.vec)
        tg.put(tid, G);
      else
        stage<T, NP, LG, 32, L, kThreads>(G, go, so, p.Dv, count, c0);
      const f4 iv = *reinterpret_cast<const f4 *>(inv + tid % (L / 4) * 4);
#pragma unroll
      for (int r = 0; r < 4; ++r) db4[r] = fmaf(tr.r[0][r] * iv[r], tu.r[0][r] * iv[r], db4[r]);
    }
#pragma unroll
    for (int i = 0; i < decltype(ts)::N; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) dot = fmaf(ts.r[i][r], td.r[i][r], dot);
    __syncthreads();
    const int lane = delta_fresh(tid & 63);
    if (asks) {
      const Frag<NP> gf = frag_row<NP, LG>(G, L * LG::row, 16 * pt, 0, lane);
      const Frag<3> rf = frag_col<3, LU>(R, PU, 0, pt, lane);
#pragma unroll
      for (int t = 0; t < NT; ++t)
        if (t <= pt) {
          const Frag<3> x = frag_col<3, LU>(U, PU, 0, t, lane);
          p0[t] = mma<3>(x, gf, p0[t]);
          p1[t] = mma<3>(x, rf, p1[t]);
        }
#pragma unroll
      for (int i = 0; i < DT; ++i) {
        const Frag<3> x = frag_col<3, LS>(S, PS, 0, d0 + i, lane);
        a0[i] = mma<3>(x, gf, a0[i]);
        a1[i] = mma<3>(x, rf, a1[i]);
      }
    } else {
      const Frag<3> uf = frag_col<3, LU>(U, PU, 0, pt, lane);
#pragma unroll
      for (int t = 0; t < NT; ++t)
        if (t >= pt) {
          p0[t] = mma<3>(frag_row<NP, LG>(G, L * LG::row, 16 * t, 0, lane), uf, p0[t]);
          p1[t] = mma<3>(frag_col<3, LU>(R, PU, 0, t, lane), uf, p1[t]);
        }
#pragma unroll
      for (int i = 0; i < DT; ++i)
        a0[i] = mma<3>(frag_col<3, LS>(D, PS, 0, d0 + i, lane), uf, a0[i]);
    }
  }
  if (p.vec) {
    const int tid = delta_fresh(threadIdx.x);
    tk.fetch(tid, k, (int)p.k.st, p.Dk, count, 0, 1, 0);
    tq.fetch(tid, q, (int)p.q.st, p.Dk, count, 0, 1, 0);
  }
  __syncthreads();
  if (p.vec) {
    const int tid = delta_fresh(threadIdx.x);
    tk.put(tid, K);
    tq.put(tid, Q);
  } else {
    stage<T, NP, LK, DK, L, kThreads>(K, k, p.k.st, p.Dk, count, 0);
    stage<T, NP, LK, DK, L, kThreads>(Q, q, p.q.st, p.Dk, count, 0);
  }
  // lanes L / 4 apart have the same positions
#pragma unroll
  for (int o = L / 4; o < 64; o <<= 1)
#pragma unroll
    for (int r = 0; r < 4; ++r) db4[r] += __shfl_xor(db4[r], o);
  if ((tid & 63) < L / 4) *reinterpret_cast<f4 *>(&dbs[w][4 * (tid & 63)]) = db4;
  const int lane = delta_fresh(tid & 63), g = lane >> 4, l16 = lane & 15;
  double all_dot = dot;
#pragma unroll
  for (int o = 32; o; o >>= 1) all_dot += __shfl_xor(all_dot, o);
  if (lane == 0) red[w] = all_dot;
  __syncthreads();
  const int mine = 16 * pt + l16;
  // four neighbours of this position's row of K or Q
  auto four = [&](const bf16 *t, int i) {
    f4 x = zero;
#pragma unroll
    for (int m = 0; m < NP; ++m) {
      const Pack<bf16, 4> y = *reinterpret_cast<const Pack<bf16, 4> *>(
          t + m * L * LK::row + LK::at(mine, 4 * (d0 + i) + g));
#pragma unroll
      for (int r = 0; r < 4; ++r) x[r] += (float)y.v[r];
    }
    return x;
  };
  // products of this wave's rows of `rows` with the keys of tile t, times y; rows 16 bytes at a
  // time where they are padded (any order of the contraction will do)
  auto scores = [&](const bf16 *rows, int t, const f4 &y) {
    f4 x = zero;
#pragma unroll
    for (int kb = 0; kb < DK / 32; ++kb) {
      if constexpr (NP == 1) {
        const int at = l16 * LK::row + 32 * kb + 8 * g;
        x = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            *reinterpret_cast<const bf8 *>(K + 16 * t * LK::row + at),
            *reinterpret_cast<const bf8 *>(rows + 16 * pt * LK::row + at), x, 0, 0, 0);
      } else {
        x = mma<3>(frag_row<NP, LK>(K, L * LK::row, 16 * t, kb, lane),
                   frag_row<NP, LK>(rows, L * LK::row, 16 * pt, kb, lane), x);
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] *= y[r];
    return x;
  };
  // sums of x over the 16 lanes that have the same four rows of tile t
  auto columns = [&](float *out, int t, const f4 &x) {
    const bool odd = l16 & 1, high = l16 & 2;
    float a = odd ? x[2] : x[0], c = odd ? x[3] : x[1];
    a += lanes<0xb1>(odd ? x[0] : x[2]), c += lanes<0xb1>(odd ? x[1] : x[3]);  // of lane ^ 1
    float y = high ? c : a;
    y += lanes<0x4e>(high ? a : c);  // ^ 2
    y += lanes<0x124>(y);            // 4 and 8 further
    y += lanes<0x128>(y);
    if (l16 < 4) out[16 * t + 4 * g + 2 * odd + high] = y;
  };
  auto give = [&](void *out, int whole, int i, const f4 &x) {
    const int d = 16 * (d0 + i) + 4 * g;
    if (mine >= count || d >= p.Dk) return;
    const int64_t to = (row0 + (int64_t)mine * p.H) * p.Dk + d;
    if (p.vec_out) {
      if (whole) {
        *reinterpret_cast<f4 *>((float *)out + to) = x;
      } else {
        Pack<T, 4> y;
#pragma unroll
        for (int r = 0; r < 4; ++r) y.v[r] = (T)x[r];
        *reinterpret_cast<Pack<T, 4> *>((T *)out + to) = y;
      }
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (d + r < p.Dk) {
          if (whole)
            ((float *)out)[to + r] = x[r];
          else
            ((T *)out)[to + r] = (T)x[r];
        }
    }
  };
  if (asks) {
    const float from = gs.from[mine];
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) a0[i][r] *= p.scale * from, a1[i][r] *= -from;
    float c = 0.f;
#pragma unroll
    for (int i = 0; i < DT; ++i) {
      const f4 kv = four(K, i), qv = four(Q, i);
#pragma unroll
      for (int r = 0; r < 4; ++r) c += qv[r] * a0[i][r] + kv[r] * a1[i][r];
    }
#pragma unroll
    for (int o = 16; o < 64; o <<= 1) c += __shfl_xor(c, o);
    if (g == 0) as[part][mine] = c;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int o = 16 * t + 4 * g + r;
        const float d = t <= pt && o <= mine ? gs.decay(mine, o) : 0.f;
        p0[t][r] *= p.scale * d;
        p1[t][r] *= o < mine ? -d : 0.f;
      }
    // W_ij, what j gives to i: sums over the columns before each of the rows from it on in
    // the diagonal tile, over rows and over columns in the others
    float row = 0.f;
#pragma unroll
    for (int t = 0; t < NT; ++t)
      if (t <= pt) {
        f4 x = zero;
        if (part == 0) x = scores(Q, t, p0[t]);
        if (part == DS - 1) x += scores(K, t, p1[t]);
        if (t == pt) {
          f4 y = zero;
#pragma unroll
          for (int r = 0; r < 4; ++r) y = mfma32(4 * g + r < l16 ? 1.f : 0.f, x[r], y);
#pragma unroll
          for (int r = 0; r < 4; ++r) x[r] = 4 * g + r <= l16 ? y[r] : 0.f;
        } else {
          row += (x[0] + x[1]) + (x[2] + x[3]);
        }
        columns(rs[part][pt], t, x);
      }
#pragma unroll
    for (int o = 16; o < 64; o <<= 1) row += __shfl_xor(row, o);
    if (g == 0) ps[part][mine] = row;
#pragma unroll
    for (int jb = 0; jb < JB; ++jb)
      if (2 * jb <= pt) {
        const Frag<3> f0 = frag_of<true>(p0[2 * jb], p0[2 * jb + 1]), f1 = frag_of<true>(p1[2 * jb], p1[2 * jb + 1]);
#pragma unroll
        for (int i = 0; i < DT; ++i) {
          const Frag<NP> x = frag_col<NP, LK>(K, L * LK::row, 32 * jb, d0 + i, lane);
          a0[i] = mma<3>(x, f0, a0[i]);
          a1[i] = mma<3>(x, f1, a1[i]);
        }
      }
#pragma unroll
    for (int i = 0; i < DT; ++i)
      if (p.dq) give(p.dq, p.part_q, i, a0[i]);
  } else {
    const float to = gs.to[mine];
    float e = 0.f;
#pragma unroll
    for (int i = 0; i < DT; ++i) {
      const f4 kv = four(K, i);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        a0[i][r] *= to;
        e += kv[r] * a0[i][r];
      }
    }
#pragma unroll
    for (int o = 16; o < 64; o <<= 1) e += __shfl_xor(e, o);
    if (g == 0) es[part][mine] = e;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int o = 16 * t + 4 * g + r;
        const float d = t >= pt && o >= mine ? gs.decay(o, mine) : 0.f;
        p0[t][r] *= p.scale * d;
        p1[t][r] *= o > mine ? -d : 0.f;
      }
#pragma unroll
    for (int ib = 0; ib < JB; ++ib)
      if (2 * ib + 1 >= pt) {
        const Frag<3> f0 = frag_of<true>(p0[2 * ib], p0[2 * ib + 1]), f1 = frag_of<true>(p1[2 * ib], p1[2 * ib + 1]);
#pragma unroll
        for (int i = 0; i < DT; ++i) {
          a0[i] = mma<3>(frag_col<NP, LK>(Q, L * LK::row, 32 * ib, d0 + i, lane), f0, a0[i]);
          a0[i] = mma<3>(frag_col<NP, LK>(K, L * LK::row, 32 * ib, d0 + i, lane), f1, a0[i]);
        }
      }
#pragma unroll
    for (int i = 0; i < DT; ++i)
      *reinterpret_cast<f4 *>(dks + mine * LW + 16 * (d0 + i) + 4 * g) = a0[i];
  }
  __syncthreads();
  if (asks && p.dk) {
#pragma unroll
    for (int i = 0; i < DT; ++i) {
      const f4 x = *reinterpret_cast<const f4 *>(dks + mine * LW + 16 * (d0 + i) + 4 * g);
      f4 y;
#pragma unroll
      for (int r = 0; r < 4; ++r) y[r] = a1[i][r] + x[r];
      give(p.dk, p.part_k, i, y);
    }
  }
  if (w == 6 && lane < count && p.db) {
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) x += dbs[i][lane];
    p.db[row0 + (int64_t)lane * p.H] = x;
  }
  if (w == 7 && p.dg) {
    const int tile = lane / 16;
    float x = 0.f, y = 0.f, z = 0.f, own = 0.f, h[NT] = {};
    if (lane < L) {
#pragma unroll
      for (int i = 0; i < DS; ++i) {
        x += as[i][L - 1 - lane], z += ps[i][L - 1 - lane], y += es[i][lane];
        own += rs[i][tile][lane];
#pragma unroll
        for (int t = 1; t < NT; ++t) h[t] += tile < t ? rs[i][t][lane] : 0.f;
      }
    }
    // sums from a position on, to the chunk's end and to its tile's; and up to it
    x = sum_up(x) + sum_row(z);
    double sum = own + exclusive(sum_up(y));
#pragma unroll
    for (int t = 1; t < NT; ++t) {
      const float u = exclusive(sum_up(h[t]));
      if (tile < t) sum += u;
    }
    sum += __shfl(x, (L - 1 - lane) & 63);
    double all = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) all += red[i];
    sum += ((double)gs.all + gs.low) * all;
    if (lane < count)
      p.dg[row0 + (int64_t)lane * p.H] = decays[lane] < -104.f ? 0.f : (float)sum;
  }
}

namespace {

template <typename T, int NP, int DK, int NW>
semicrf_status_t delta_walk(DeltaArgs p, DeltaPass pass, hipStream_t st) {
  constexpr int L = delta_chunk(NP);
  const int vt = (p.Dv + 16 * NW - 1) / (16 * NW);
  // composing, the columns of phi go beside those of the sum
  const int kt = pass == DELTA_COMPOSE ? (p.Dk + 16 * NW - 1) / (16 * NW) : 0;
  p.ctiles = kt > vt ? kt : vt;
  const int64_t grid = (int64_t)p.B * p.H * p.count * p.ctiles;
  if (pass == DELTA_COMPOSE)
    k_delta_chunks<T, NP, DK, NW, L, true><<<(unsigned)grid, 64 * NW, 0, st>>>(p);
  else if (pass == DELTA_FORWARD)
    k_delta_chunks<T, NP, DK, NW, L, false><<<(unsigned)grid, 64 * NW, 0, st>>>(p);
  else if (pass == DELTA_COMPOSE_BACK)
    k_delta_back<T, NP, DK, NW, L, true><<<(unsigned)grid, 64 * NW, 0, st>>>(p);
  else
    k_delta_back<T, NP, DK, NW, L, false><<<(unsigned)grid, 64 * NW, 0, st>>>(p);
  return launch_status();
}

template <typename T, int NP, int DK>
semicrf_status_t delta_width(const DeltaArgs &p, DeltaPass pass, hipStream_t st) {
  constexpr int L = delta_chunk(NP);
  const unsigned grid = (unsigned)((int64_t)p.B * p.H * p.N);
  if (pass == DELTA_INVERSE) {
    k_delta_inverse<T, NP, DK, L><<<grid, 256, 0, st>>>(p);
    return launch_status();
  }
  if (pass == DELTA_GRADS) {
    k_delta_grads<T, NP, DK, L><<<grid, 512, 0, st>>>(p);
    return launch_status();
  }
  switch (delta_waves(p.Dv)) {
    case 2: return delta_walk<T, NP, DK, 2>(p, pass, st);
    case 4: return delta_walk<T, NP, DK, 4>(p, pass, st);
    case 5: return delta_walk<T, NP, DK, 5>(p, pass, st);
    case 6: return delta_walk<T, NP, DK, 6>(p, pass, st);
    default: return delta_walk<T, NP, DK, 8>(p, pass, st);
  }
}

template <typename T, int NP>
semicrf_status_t delta_type(const DeltaArgs &p, DeltaPass pass, hipStream_t st) {
  if (p.Dk <= 32) return delta_width<T, NP, 32>(p, pass, st);
  if (p.Dk <= 64) return delta_width<T, NP, 64>(p, pass, st);
  if (p.Dk <= 96) return delta_width<T, NP, 96>(p, pass, st);
  return delta_width<T, NP, 128>(p, pass, st);
}

}  // namespace

}  // namespace semicrf
