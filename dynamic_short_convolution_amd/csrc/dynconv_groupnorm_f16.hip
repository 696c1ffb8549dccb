// The group norm's kernels for f16 storage.
#include "dynconv_groupnorm_kernels.hpp"

namespace dynconv {

hipError_t group_tokens_f16(const GroupParams& p, bool vec, bool packed, bool bwd, hipStream_t s) {
  return group::tokens<f16_t>(p, vec, packed, bwd, s);
}
hipError_t group_sequences_f16(const GroupParams& p, bool vec, bool packed, GroupStage stage, hipStream_t s) {
  return group::sequences<f16_t>(p, vec, packed, stage, s);
}

}  // namespace dynconv
