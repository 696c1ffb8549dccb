// The gated linear scan's kernels for f32 storage.
#include "dynconv_scan_kernels.hpp"

namespace dynconv {

hipError_t scan_fwd_f32(const ScanParams& p, int vec, bool packed, hipStream_t s) { return scan::fwd<float>(p, vec, packed, s); }
hipError_t scan_bwd_f32(const ScanParams& p, int vec, bool packed, hipStream_t s) { return scan::bwd<float>(p, vec, packed, s); }

}  // namespace dynconv
