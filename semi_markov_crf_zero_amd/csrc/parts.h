// parts.h -- products of matrices held as sums of bfloat16 parts: operands'
// fragments, tiles in LDS and how they are filled (linattn_kernels.h,
// delta_kernels.h).
#pragma once

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

// A fragment is a lane's part of one operand over a 32-wide stretch of the
// contraction: indices {4g + r} and {16 + 4g + r} (g = lane / 16, r < 4) of
// row or column lane % 16, in N parts.  That is how two neighbouring 16x16
// accumulator tiles hold their rows, so X goes from accumulators to operands
// in place.
template <int N>
struct Frag {
  bf8 v[N];
};

// c + a b, the pairs of parts (i, j) with i + j < K.
template <int K, int N, int M>
__device__ __forceinline__ f4 mma(const Frag<N> &a, const Frag<M> &b, f4 c) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < M; ++j)
      if (i + j < K) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[j], c, 0, 0, 0);
  return c;
}

// Tiles in LDS, by what is read of them.  A phase of an 8-byte read serves 16
// lanes from 32 banks: a fragment of rows asks for one 8-byte unit of 16 rows
// (A, P), the transposing read of columns for 4 units of 4 rows (C), both of
// B.  16 different bank pairs each time: rows an odd number of units apart;
// rows 4 or 12 units (mod 16) apart; for both, the units of a row exchanged
// by an XOR with a number that the row gives.  The first two leave one address
// and constant offsets, the XOR a handful of addresses, so only B has it.
template <int W>
struct ByRow {
  static constexpr int row = W + 4;
  __device__ static __forceinline__ int at(int r, int u) { return r * row + 4 * u; }
};
template <int W>
struct ByColumn {
  static constexpr int row = W % 32 == 16 ? W : W + 16;
  __device__ static __forceinline__ int at(int r, int u) { return r * row + 4 * u; }
};
template <int W>
struct ByBoth {
  static constexpr int row = W;
  __device__ static __forceinline__ int at(int r, int u) {
    const int key = W % 64 == 0 ? ((r & 3) << 2) | ((r >> 2) & 3) : ((r & 2) << 1) | ((r >> 2) & 3);
    return r * row + 4 * (u ^ key);
  }
};

// Fragment of row row0 + lane % 16 (row0 a multiple of 16), contraction
// indices 32 kb..; the parts lie `plane` apart.
template <int N, typename Lay>
__device__ __forceinline__ Frag<N> frag_row(const bf16 *t, int plane, int row0, int kb, int lane) {
  typedef __bf16 bf4 __attribute__((ext_vector_type(4)));
  const int r = lane & 15, u = 8 * kb + (lane >> 4);
  const bf16 *lo = t + row0 * Lay::row + Lay::at(r, u);
  const bf16 *hi = t + row0 * Lay::row + Lay::at(r, u + 4);
  Frag<N> f;
#pragma unroll
  for (int i = 0; i < N; ++i)
    f.v[i] = __builtin_shufflevector(*reinterpret_cast<const bf4 *>(lo + i * plane),
                                     *reinterpret_cast<const bf4 *>(hi + i * plane), 0, 1, 2, 3, 4,
                                     5, 6, 7);
  return f;
}

// Fragment of column 16 ct + lane % 16 whose contraction index runs over the
// 32 rows from row0, through the transposing LDS read: in each group of 16
// lanes, lane i names 4 elements of row i / 4 and gets column i of the four
// rows.
template <int N, typename Lay>
__device__ __forceinline__ Frag<N> frag_col(const bf16 *t, int plane, int row0, int ct, int lane) {
  const int r = 4 * (lane >> 4) + ((lane & 15) >> 2), u = 4 * ct + (lane & 3);
  const bf16 *q = t + row0 * Lay::row + Lay::at(r, u);
  Frag<N> f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(q + i * plane));
    const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(q + i * plane + 16 * Lay::row));
    f.v[i] = __builtin_bit_cast(bf8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
  return f;
}

// Two float32 rounded to bfloat16; x keeps what is left.  One instruction
// rounds a pair.
__device__ __forceinline__ b2 part2(f2 &x) {
  const b2 y = __builtin_convertvector(x, b2);
  x -= __builtin_convertvector(y, f2);
  return y;
}
template <int N>
__device__ __forceinline__ Frag<N> split(const float *x) {
  Frag<N> f;
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    f2 r = {x[e], x[e + 1]};
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const b2 y = part2(r);
      f.v[n][e] = y[0];
      f.v[n][e + 1] = y[1];
    }
  }
  return f;
}
template <int N>
__device__ __forceinline__ void values(const Frag<N> &f, float *x) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[e] = (float)f.v[N - 1][e];
#pragma unroll
    for (int n = N - 2; n >= 0; --n) x[e] += (float)f.v[n][e];
  }
}

// A tile of a chunk: L rows of W columns in N parts, zeros past row n and past
// column D.  fetch() issues a thread's 16-byte loads into registers while the
// chunk before is worked on, put() writes them to LDS.  The loads go through a
// buffer descriptor whose range a row that is not wanted lies past, so it
// reads 0 without a branch, whatever memory holds there.
template <typename T, int N, typename Lay, int W, int L, int NT>
struct Tile {
  static constexpr int VE = 16 / sizeof(T), per = W / VE, all = L * per, NV = (all + NT - 1) / NT;
  static constexpr int plane = L * Lay::row;
  u4 r[NV];

  // row i of the tile is row `row0 + step * i` (step +-1) from src, rows st
  // elements apart
  __device__ __forceinline__ void fetch(int tid, const T *src, int st, int D, int n, int row0,
                                        int step, int col0) {
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)src, 0, kRange, kRawBuffer);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int e = tid + k * NT, i = e / per, c = col0 + e % per * VE;
      const int at = ((row0 + step * i) * st + c) * (int)sizeof(T);
      r[k] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, i < n && c < D ? at : -1, 0, 0);
    }
  }
  __device__ __forceinline__ void put(int tid, bf16 *lds) const {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int e = tid + k * NT, i = e / per, c = e % per * VE;
      if (all % NT && e >= all) break;
      const Pack<T, VE> y = __builtin_bit_cast(Pack<T, VE>, r[k]);
#pragma unroll
      for (int q = 0; q < VE; q += 4) {
        bf16 *to = lds + Lay::at(i, (c + q) / 4);
        f2 lo = {(float)y.v[q], (float)y.v[q + 1]}, hi = {(float)y.v[q + 2], (float)y.v[q + 3]};
#pragma unroll
        for (int m = 0; m < N; ++m) {
          Pack<bf16, 4> x;
          if constexpr (N == 1) {
            x = {{y.v[q], y.v[q + 1], y.v[q + 2], y.v[q + 3]}};
          } else {
            const b2 a = part2(lo), b = part2(hi);
            x = {{a[0], a[1], b[0], b[1]}};
          }
          *reinterpret_cast<Pack<bf16, 4> *>(to + m * plane) = x;
        }
      }
    }
  }
};

// The same without the alignment 16-byte loads need: element by element,
// straight to LDS.
template <typename T, int N, typename Lay, int W, int L, int NT>
__device__ __forceinline__ void stage(bf16 *lds, const T *src, int64_t st, int D, int n,
                                      int col0) {
  constexpr int plane = L * Lay::row;
  for (int e = threadIdx.x; e < L * W; e += NT) {
    const int i = e / W, d = e % W;
    float x = i < n && col0 + d < D ? (float)src[i * st + col0 + d] : 0.f;
#pragma unroll
    for (int m = 0; m < N; ++m) {
      const bf16 y = (bf16)x;
      lds[m * plane + Lay::at(i, d / 4) + d % 4] = y;
      x -= (float)y;
    }
  }
}

}  // namespace

}  // namespace semicrf
