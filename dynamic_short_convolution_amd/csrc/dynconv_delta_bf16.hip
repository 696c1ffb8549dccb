// Gated delta rule kernels for bf16 storage.
#include "dynconv_delta_kernels.hpp"

namespace dynconv {

hipError_t delta_fwd_bf16(const DeltaParams& p, hipStream_t s) { return delta::delta_fwd_et<bf16_t>(p, s); }
hipError_t delta_bwd_bf16(const DeltaParams& p, hipStream_t s) { return delta::delta_bwd_et<bf16_t>(p, s); }

}  // namespace dynconv
