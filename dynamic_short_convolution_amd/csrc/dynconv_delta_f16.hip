// Gated delta rule kernels for f16 storage.
#include "dynconv_delta_kernels.hpp"

namespace dynconv {

hipError_t delta_fwd_f16(const DeltaParams& p, hipStream_t s) { return delta::delta_fwd_et<f16_t>(p, s); }
hipError_t delta_bwd_f16(const DeltaParams& p, hipStream_t s) { return delta::delta_bwd_et<f16_t>(p, s); }

}  // namespace dynconv
