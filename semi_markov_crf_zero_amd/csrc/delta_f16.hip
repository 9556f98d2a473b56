// delta_f16.hip -- the gated delta rule over float16 tensors.
#include "delta_kernels.h"

namespace semicrf {

semicrf_status_t delta_f16(const DeltaArgs &p, DeltaPass pass, hipStream_t st) {
  return delta_type<f16, 2>(p, pass, st);
}

}  // namespace semicrf
