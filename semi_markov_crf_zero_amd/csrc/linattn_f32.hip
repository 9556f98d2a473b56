// linattn_f32.hip -- linear attention over float32 tensors.
#include "linattn_kernels.h"

namespace semicrf {

semicrf_status_t linattn_f32(const LaArgs &p, bool vec, bool f32_out, bool states, hipStream_t st) {
  (void)f32_out;
  return launch_type<float, 3, float>(p, vec, states, st);
}

}  // namespace semicrf
