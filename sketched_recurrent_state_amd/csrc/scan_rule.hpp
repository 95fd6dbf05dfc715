// scan_rule.hpp -- the scan's launches for one rule (one translation unit per rule).
#pragma once

#include "scan_grads.hpp"
#include "scan_prep.hpp"
#include "scan_split.hpp"
#include "scan_state.hpp"

namespace ssm {

// Waves of a workgroup and waves per column block (NW, DS) of the split passes. One wave per
// column block does least work; where that leaves most of the 1,024 SIMDs without a wave, the
// block's rows are divided.
template <int RULE, int DK, typename F>
void split_shape(const ssm_dims& d, F&& f) {
  using std::integral_constant;
  const long long waves = (long long)d.batch * d.heads * (d.d_v / 16);
  if constexpr (DK >= 128) {
    if (waves <= 512) return f(integral_constant<int, 4>{}, integral_constant<int, 4>{});
  }
  if (d.d_v >= 64) return f(integral_constant<int, 4>{}, integral_constant<int, 1>{});
  if (d.d_v == 32) return f(integral_constant<int, 2>{}, integral_constant<int, 1>{});
  return f(integral_constant<int, 1>{}, integral_constant<int, 1>{});
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
      if constexpr (kSplit<RULE, kDK, TIN>) {
        split_shape<RULE, kDK>(d, [&](auto NW, auto DS) {
          constexpr int nw = decltype(NW)::value, ds = decltype(DS)::value;
          hipLaunchKernelGGL((scan_split_state_kernel<RULE, kDK, nw, ds, decltype(B)::value>),
                             dim3(unit_grid(units, kDV * ds / (16 * nw))), dim3(64 * nw), 0, stream, a);
        });
      } else {
        hipLaunchKernelGGL((scan_state_kernel<RULE, kDK, TIN, decltype(B)::value>),
                           dim3(unit_grid(units, kDV / 16)), dim3(64), 0, stream, a);
      }
    };
    if (!backward) {
      prep(std::false_type{});
      state(std::false_type{});
      return hipGetLastError();
    }
    prep(std::true_type{});
    state(std::true_type{});
    if constexpr (kSplit<RULE, kDK, TIN>) {
      split_shape<RULE, kDK>(d, [&](auto NW, auto DS) {
        constexpr int nw = decltype(NW)::value, ds = decltype(DS)::value;
        hipLaunchKernelGGL((scan_split_gradient_kernel<RULE, kDK, nw, ds>),
                           dim3(unit_grid(units, kDV * ds / (16 * nw))), dim3(64 * nw), 0, stream, a);
      });
    } else {
      hipLaunchKernelGGL((scan_gradient_kernel<RULE, kDK, TIN>), dim3(unit_grid(units, kDV / 16)),
                         dim3(64), 0, stream, a);
    }
    hipLaunchKernelGGL((scan_grads_kernel<RULE, kDK, kDV, TIN>), dim3(cells),
                       dim3(kDK >= 32 ? 2 * kDK : 64), 0, stream, a);
    return hipGetLastError();
  });
}

}  // namespace ssm
