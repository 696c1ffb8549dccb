// The gated linear scan's kernels for f16 storage.
#include "dynconv_scan_kernels.hpp"

namespace dynconv {

hipError_t scan_fwd_f16(const ScanParams& p, int vec, bool packed, hipStream_t s) { return scan::run<f16_t>(p, vec, packed, false, s); }
hipError_t scan_bwd_f16(const ScanParams& p, int vec, bool packed, hipStream_t s) { return scan::run<f16_t>(p, vec, packed, true, s); }

}  // namespace dynconv
