// The gated linear scan's kernels for f16 storage.
#include "dynconv_scan_kernels.hpp"

namespace dynconv {

hipError_t scan_fwd_f16(const ScanParams& p, int vec, bool packed, hipStream_t s) { return scan::fwd<f16_t>(p, vec, packed, s); }
hipError_t scan_bwd_f16(const ScanParams& p, int vec, bool packed, hipStream_t s) { return scan::bwd<f16_t>(p, vec, packed, s); }

}  // namespace dynconv
