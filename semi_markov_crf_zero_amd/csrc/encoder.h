// encoder.h -- element types and small helpers shared by the encoder's and
// the optimiser's kernels (linattn.hip, groupnorm.hip, adamw.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "semicrf_encoder.h"

namespace semicrf {

typedef __bf16 bf16;
typedef _Float16 f16;
typedef float f32x4_t __attribute__((ext_vector_type(4)));

__host__ inline int elem_size(int dtype) { return dtype == SEMICRF_F32 ? 4 : 2; }
__host__ inline bool dtype_ok(int dtype) { return dtype >= SEMICRF_F32 && dtype <= SEMICRF_F16; }

// A launch's own error, with what an earlier call left behind cleared first.
inline semicrf_status_t launch_status() {
  return hipGetLastError() == hipSuccess ? SEMICRF_OK : SEMICRF_ERR_HIP;
}

// Valid positions of sequence b: its length, or -1 for one outside [0, T].
__device__ __forceinline__ int valid_length(const int32_t *lengths, int b, int T) {
  if (!lengths) return T;
  const int L = lengths[b];
  return L < 0 || L > T ? -1 : L;
}

// N neighbouring elements as one load or store; VEC says that the address
// allows it (N * sizeof(T) bytes, aligned to that).
template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
  T v[N];
};

}  // namespace semicrf
