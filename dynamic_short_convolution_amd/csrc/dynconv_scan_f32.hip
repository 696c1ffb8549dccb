// The gated linear scan's kernels for f32 storage.
#include "dynconv_scan_kernels.hpp"

namespace dynconv {

hipError_t scan_fwd_f32(const ScanParams& p, int vec, bool packed, hipStream_t s) { return scan::run<float>(p, vec, packed, false, s); }
hipError_t scan_bwd_f32(const ScanParams& p, int vec, bool packed, hipStream_t s) { return scan::run<float>(p, vec, packed, true, s); }

}  // namespace dynconv
