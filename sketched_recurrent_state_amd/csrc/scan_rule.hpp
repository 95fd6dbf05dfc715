// scan_rule.hpp -- the scan's launches for one rule (one translation unit per rule).
#pragma once

#include "scan_grads.hpp"
#include "scan_prep.hpp"
#include "scan_state.hpp"

namespace ssm {

// Calls f(waves of a workgroup, narrow). Wide workgroups do least work; where they leave SIMDs
// (there are 1,024) without a wave, the rows of a column block are divided over as many waves
// as fill them: 32 rows a wave at least.
template <int RULE, int DK, int DV, typename F>
void split_shape(const ssm_dims& d, F&& f) {
  using std::integral_constant;
  const long long blocks = (long long)d.batch * d.heads * (DV / 16);
  if constexpr (DK == 128) {
    if (blocks <= 256) return f(integral_constant<int, 4>{}, std::true_type{});
  }
  if (blocks <= (RULE == KDA ? 256 : 512))
    f(integral_constant<int, (DK >= 64 ? 2 : 1)>{}, std::true_type{});
  else
    f(integral_constant<int, (DV >= 64 ? 4 : DV / 16)>{}, std::false_type{});
}

template <int RULE>
hipError_t launch_scan_rule(const ssm_dims& d, const ScanArgs& a, bool backward, hipStream_t stream) {
  return dispatch_shape(d.in_dtype, d.d_k, d.d_v, [&](auto DK, auto DV, auto T) -> hipError_t {
    using TIN = typename decltype(T)::type;
    constexpr int kDK = decltype(DK)::value, kDV = decltype(DV)::value;
    const unsigned cells = (unsigned)((size_t)a.plan.cap * d.heads);
    const long long units = (long long)d.batch * d.heads;
    auto prep = [&](auto B) {
      hipLaunchKernelGGL((scan_prep_kernel<RULE, kDK, TIN, decltype(B)::value>), dim3(cells * NB),
                         dim3(64), 0, stream, a);
    };
    auto state = [&](auto B) {
      split_shape<RULE, kDK, kDV>(d, [&](auto NW, auto NARROW) {
        constexpr int nw = decltype(NW)::value;
        constexpr bool narrow = decltype(NARROW)::value, bwd = decltype(B)::value;
        hipLaunchKernelGGL((scan_state_kernel<RULE, kDK, TIN, nw, narrow, bwd>),
                           dim3(unit_grid(units, kDV / 16 / (narrow ? 1 : nw))),
                           dim3(64 * (nw + (narrow && !bwd))), 0, stream, a);
      });
    };
    if (!backward) {
      prep(std::false_type{});
      state(std::false_type{});
      return hipGetLastError();
    }
    prep(std::true_type{});
    state(std::true_type{});
    split_shape<RULE, kDK, kDV>(d, [&](auto NW, auto NARROW) {
      constexpr int nw = decltype(NW)::value;
      constexpr bool narrow = decltype(NARROW)::value;
      hipLaunchKernelGGL((scan_gradient_kernel<RULE, kDK, TIN, nw, narrow>),
                         dim3(unit_grid(units, kDV / 16 / (narrow ? 1 : nw))), dim3(64 * nw), 0,
                         stream, a);
    });
    hipLaunchKernelGGL((scan_grads_kernel<RULE, kDK, kDV, TIN>), dim3(cells),
                       dim3(kGradThreads<RULE, kDK>), 0, stream, a);
    return hipGetLastError();
  });
}

}  // namespace ssm
