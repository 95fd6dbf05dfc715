// scan_mamba2.hip -- the scan kernels of the Mamba-2 rule.
#include "scan_rule.hpp"

namespace ssm {

template hipError_t launch_scan_rule<MAMBA2>(const ssm_dims&, const ScanArgs&, bool, hipStream_t);

}  // namespace ssm
