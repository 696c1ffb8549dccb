// The group norm's kernels for bf16 storage.
#include "dynconv_groupnorm_kernels.hpp"

namespace dynconv {

hipError_t group_tokens_bf16(const GroupParams& p, bool whole, bool packed, bool bwd, hipStream_t s) {
  return group::tokens<bf16_t>(p, whole, packed, bwd, s);
}
hipError_t group_sequences_bf16(const GroupParams& p, bool whole, bool packed, GroupStage stage, hipStream_t s) {
  return group::sequences<bf16_t>(p, whole, packed, stage, s);
}

}  // namespace dynconv
