// The group norm's kernels for f16 storage.
#include "dynconv_groupnorm_kernels.hpp"

namespace dynconv {

hipError_t group_tokens_f16(const GroupParams& p, bool whole, bool packed, bool bwd, hipStream_t s) {
  return group::tokens<f16_t>(p, whole, packed, bwd, s);
}
hipError_t group_sequences_f16(const GroupParams& p, bool whole, bool packed, GroupStage stage, hipStream_t s) {
  return group::sequences<f16_t>(p, whole, packed, stage, s);
}

}  // namespace dynconv
