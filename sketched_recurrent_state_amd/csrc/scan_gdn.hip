// scan_gdn.hip -- the scan kernels of the Gated DeltaNet rule.
#include "scan_rule.hpp"

namespace ssm {

template hipError_t launch_scan_rule<GDN>(const ssm_dims&, const ScanArgs&, bool, hipStream_t);

}  // namespace ssm
