// The gated linear scan's kernels for bf16 storage.
#include "dynconv_scan_kernels.hpp"

namespace dynconv {

hipError_t scan_fwd_bf16(const ScanParams& p, int vec, bool packed, hipStream_t s) { return scan::run<bf16_t>(p, vec, packed, false, s); }
hipError_t scan_bwd_bf16(const ScanParams& p, int vec, bool packed, hipStream_t s) { return scan::run<bf16_t>(p, vec, packed, true, s); }

}  // namespace dynconv
