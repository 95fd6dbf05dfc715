// scan_rule.hpp -- the scan's launches for one rule (one translation unit per rule).
#pragma once

#include "scan_grads.hpp"
#include "scan_prep.hpp"
#include "scan_split.hpp"
#include "scan_state.hpp"

namespace ssm {

template <int RULE>
hipError_t launch_scan_rule(const ssm_dims& d, const ScanArgs& a, bool backward, hipStream_t stream) {
  return dispatch_shape(d.in_dtype, d.d_k, d.d_v, [&](auto DK, auto DV, auto T) -> hipError_t {
    using TIN = typename decltype(T)::type;
    constexpr int kDK = decltype(DK)::value, kDV = decltype(DV)::value;
    const unsigned cells = (unsigned)((size_t)a.plan.cap * d.heads);
    const unsigned units = unit_grid((long long)d.batch * d.heads, kDV / 16);
    if (!backward) {
      hipLaunchKernelGGL((scan_prep_kernel<RULE, kDK, TIN, false>), dim3(cells * NB), dim3(64), 0,
                         stream, a);
      if constexpr (kSplit<RULE, kDK, TIN>)
        hipLaunchKernelGGL((scan_split_state_kernel<RULE, kDK, false>), dim3(units), dim3(64), 0,
                           stream, a);
      else
        hipLaunchKernelGGL((scan_state_kernel<RULE, kDK, TIN, false>), dim3(units), dim3(64), 0,
                           stream, a);
      return hipGetLastError();
    }
    hipLaunchKernelGGL((scan_prep_kernel<RULE, kDK, TIN, true>), dim3(cells * NB), dim3(64), 0,
                       stream, a);
    if constexpr (kSplit<RULE, kDK, TIN>) {
      hipLaunchKernelGGL((scan_split_state_kernel<RULE, kDK, true>), dim3(units), dim3(64), 0,
                         stream, a);
      hipLaunchKernelGGL((scan_split_gradient_kernel<RULE, kDK>), dim3(units), dim3(64), 0, stream,
                         a);
    } else {
      hipLaunchKernelGGL((scan_state_kernel<RULE, kDK, TIN, true>), dim3(units), dim3(64), 0,
                         stream, a);
      hipLaunchKernelGGL((scan_gradient_kernel<RULE, kDK, TIN>), dim3(units), dim3(64), 0, stream,
                         a);
    }
    hipLaunchKernelGGL((scan_grads_kernel<RULE, kDK, kDV, TIN>), dim3(cells),
                       dim3(kDK >= 32 ? 2 * kDK : 64), 0, stream, a);
    return hipGetLastError();
  });
}

}  // namespace ssm
