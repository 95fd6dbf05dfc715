// scan_kda.hip -- the scan kernels of the KDA rule.
#include "scan_rule.hpp"

namespace ssm {

template hipError_t launch_scan_rule<KDA>(const ssm_dims&, const ScanArgs&, bool, hipStream_t);

}  // namespace ssm
