// linattn_bf16.hip -- linear attention over bfloat16 tensors.
#include "linattn_kernels.h"

namespace semicrf {

semicrf_status_t linattn_bf16(const LaArgs &p, bool vec, bool f32_out, bool states, hipStream_t st) {
  return f32_out ? launch_type<bf16, 1, float>(p, vec, states, st)
                 : launch_type<bf16, 1, bf16>(p, vec, states, st);
}

}  // namespace semicrf
