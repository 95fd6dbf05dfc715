// scan_rule.hpp -- the scan's launches for one rule (one translation unit per rule).
#pragma once

#include "scan_grads.hpp"
#include "scan_prep.hpp"
#include "scan_state.hpp"

namespace ssm {

// Calls f(waves of a workgroup, narrow). Wide workgroups do least work; where they leave SIMDs
// (there are 1,024) without a wave, the rows of a column block are divided over as many waves as
// gain: at least 32 rows a wave. Measured at 1024 tokens, d_v = 128, bf16 (fp32), in us:
//   d_k = 128, column blocks      256: wide, 4 waves      512: wide, 2, 4 waves    1,024: wide, best narrow
//   Mamba-2 forward              83, 49 (119, 70)      86, 72, 62 (125, 122, 129)     93, 131 (138, 232)
//   GDN forward                 103, 68 (138, 95)     107, 95, 124 (145, 153, 178)   117, 178 (166, 296)
//   Mamba-2 backward           168, 129 (223, 164)   201, 193, 176 (278, 268, 245)  306, 339 (395, 500)
//   GDN backward               260, 212 (328, 245)   341, 335, 319 (422, 394, 376)  487, 538 (585, 729)
//   KDA forward                180, 126 (182, 130)   202, 317, 241 (212, 321, 247)  261, 467 (274, 472)
//   KDA backward               640, 529 (641, 522)  1006, 1192, 1058 (978, 1163, 1032)
//   d_k = 64: GDN forward        80, 61 (99, 81)       84, 75 (106, 101)              92, 134 (117, 182)
//             GDN backward     201, 187 (236, 222)    255, 266 (305, 312)
//             KDA forward      112, 103 (111, 101)    121, 124 (123, 125)
//   d_k = 32: GDN forward        71, 53 (84, 73)       74, 61 (87, 83)                80, 85 (94, 111)
//             KDA forward        88, 90 (87, 89)       92, 101 (91, 100)
// KDA's blocks hold three split arrays: LDS leaves a narrow workgroup or two on a CU.
template <int RULE, int DK, int DV, typename TIN, bool BWD, typename F>
void split_shape(const ssm_dims& d, F&& f) {
  using std::integral_constant;
  constexpr bool SLOW = BWD ? DK < 128 : DK == 128 && sizeof(TIN) == 4;
  constexpr int LIMIT = RULE == KDA ? (DK >= 64 ? 256 : 0) : SLOW ? 256 : 512;
  const long long blocks = (long long)d.batch * d.heads * (DV / 16);
  if constexpr (RULE == GDN && !BWD && DK == 128 && LIMIT == 512) {
    if (blocks > 256 && blocks <= LIMIT) return f(integral_constant<int, 2>{}, std::true_type{});
  }
  if constexpr (LIMIT > 0) {
    if (blocks <= LIMIT)
      return f(integral_constant<int, (DK >= 32 ? DK / 32 : 1)>{}, std::true_type{});
  }
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
                         dim3(64 * kPrepWaves<RULE, kDK>), 0, stream, a);
    };
    auto state = [&](auto B) {
      split_shape<RULE, kDK, kDV, TIN, decltype(B)::value>(d, [&](auto NW, auto NARROW) {
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
    split_shape<RULE, kDK, kDV, TIN, true>(d, [&](auto NW, auto NARROW) {
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
