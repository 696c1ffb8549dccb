// Gated delta rule kernels for f32 storage.
#include "dynconv_delta_kernels.hpp"

namespace dynconv {

hipError_t delta_fwd_f32(const DeltaParams& p, hipStream_t s) { return delta::delta_fwd_et<float>(p, s); }
hipError_t delta_bwd_f32(const DeltaParams& p, hipStream_t s) { return delta::delta_bwd_et<float>(p, s); }

}  // namespace dynconv
