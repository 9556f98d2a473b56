// delta_bf16.hip -- the gated delta rule over bfloat16 tensors.
#include "delta_kernels.h"

namespace semicrf {

semicrf_status_t delta_bf16(const DeltaArgs &p, DeltaPass pass, hipStream_t st) {
  return delta_type<bf16, 1>(p, pass, st);
}

}  // namespace semicrf
