// linattn_f16.hip -- linear attention over float16 tensors.
#include "linattn_kernels.h"

namespace semicrf {

semicrf_status_t linattn_f16(const LaArgs &p, bool vec, bool f32_out, bool states, hipStream_t st) {
  return f32_out ? launch_type<f16, 2, float>(p, vec, states, st)
                 : launch_type<f16, 2, f16>(p, vec, states, st);
}

}  // namespace semicrf
