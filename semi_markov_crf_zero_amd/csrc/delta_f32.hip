// delta_f32.hip -- the gated delta rule over float32 tensors.
#include "delta_kernels.h"

namespace semicrf {

semicrf_status_t delta_f32(const DeltaArgs &p, DeltaPass pass, hipStream_t st) {
  return delta_type<float, 3>(p, pass, st);
}

}  // namespace semicrf
