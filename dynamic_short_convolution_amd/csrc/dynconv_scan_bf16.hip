// The gated linear scan's kernels for bf16 storage.
#include "dynconv_scan_kernels.hpp"

namespace dynconv {

hipError_t scan_fwd_bf16(const ScanParams& p, int vec, bool packed, hipStream_t s) { return scan::fwd<bf16_t>(p, vec, packed, s); }
hipError_t scan_bwd_bf16(const ScanParams& p, int vec, bool packed, hipStream_t s) { return scan::bwd<bf16_t>(p, vec, packed, s); }

}  // namespace dynconv
