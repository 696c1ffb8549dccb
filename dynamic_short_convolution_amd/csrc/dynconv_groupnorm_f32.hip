// The group norm's kernels for f32 storage.
#include "dynconv_groupnorm_kernels.hpp"

namespace dynconv {

hipError_t group_tokens_f32(const GroupParams& p, bool whole, bool packed, bool bwd, hipStream_t s) {
  return group::tokens<float>(p, whole, packed, bwd, s);
}
hipError_t group_sequences_f32(const GroupParams& p, bool whole, bool packed, GroupStage stage, hipStream_t s) {
  return group::sequences<float>(p, whole, packed, stage, s);
}

}  // namespace dynconv
