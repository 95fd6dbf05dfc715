// selective.hpp -- the selective recurrence: shared by the forward, backward and single-token kernels.
//
// A wave takes 64 / S channels: S lanes a channel, each with NS = d_state / S of its states. Sixteen
// tokens ("a block") at a time are read by all lanes (lane = 4 * token + quarter, 16 / S channels
// and d_state / 4 values of B and C a lane), turned into fp32 with softplus taken once per
// token and channel, and passed through LDS of the wave's own: no workgroup barrier. Per state and
// token the recurrence is a product, an exp2, a product and two fused ones, so prompts are bound by the
// vector ALU, not by HBM.
#pragma once

#include "layer.hpp"
#include "launch.hpp"

namespace ssm {

constexpr int TB = 16;     // tokens of a block
constexpr int WAVES = 4;   // of a workgroup

// log(1 + e^x) without losing small values; above 20 it is x in fp32.
__device__ __forceinline__ float softplus(float x) { return x > 20.f ? x : log1pf(expf(x)); }

template <int S, int NS>
struct SelShape {
  static constexpr int N = S * NS, CH = 64 / S, EC = CH / 4, EN = N / 4;
};

// Sum over the S lanes of a channel.
template <int S>
__device__ __forceinline__ float state_sum(float x) {
  x += dpp<DPP_QUAD_1032>(x);
  x += dpp<DPP_QUAD_2301>(x);
  if constexpr (S >= 8) x += dpp<DPP_HALF_MIRROR>(x);
  if constexpr (S >= 16) x += dpp<DPP_ROR8>(x);
  return x;
}
// Sum over the lanes of a wave that share lane % S.
template <int S>
__device__ __forceinline__ float channel_sum(float x) {
  if constexpr (S <= 4) x += dpp<DPP_ROR4>(x);
  if constexpr (S <= 8) x += dpp<DPP_ROR8>(x);
  return xsum32(xsum16(x));
}

// The wave's tile of channels, and the lane's place in it.
struct SelTile {
  int tile, c0, group;   // first channel
  int lane, t, q;        // reading: token t of a block, quarter q
  int ch, sg;            // computing: channel ch of the tile, states sg * NS ..
};
template <int S>
__device__ __forceinline__ SelTile sel_tile(const SelectiveArgs& a, int tile) {
  SelTile w;
  w.tile = tile;
  w.c0 = tile * (64 / S);
  w.group = w.c0 / (a.channels / a.groups);
  w.lane = threadIdx.x & 63;
  w.t = w.lane >> 2;
  w.q = w.lane & 3;
  w.ch = w.lane / S;
  w.sg = w.lane % S;
  return w;
}

// E consecutive elements, zero where the row holds no token.
template <typename T, int E>
__device__ __forceinline__ void load_or_zero(Packed<T, E>& r, const T* p, bool on) {
#pragma unroll
  for (int i = 0; i < Packed<T, E>::NW; ++i) r.w[i] = 0u;
  if (on) r.load(p);
}

template <typename T, int E>
__device__ __forceinline__ void store_row(T* p, const float* v) {
  if constexpr (sizeof(T) == 4) {
    Vec<float, E>::store(p, v);
  } else if constexpr (E == 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  } else if constexpr (E == 2) {
    *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(v[0], v[1]);
  } else {
    static_assert(E == 1, "a lane's channels");
    *p = (uint16_t)pack_bf16x2(v[0], v[0]);
  }
}

// A walker's sequences: every walkers-th.
struct SelSeq {
  int seq, tok, len, slot;
};
__device__ __forceinline__ bool sel_sequence(const SelectiveArgs& a, int s, SelSeq& q) {
  int first;
  if (!a.plan.sequence(s, q.tok, q.len, first)) return false;
  q.seq = s;
  q.slot = a.slot ? a.slot[s] : s;
  return q.slot >= 0 && q.slot < a.num_slots;
}

// The states before every block, for the backward pass; sets a.walkers.
hipError_t launch_selective_states(const ssm_selective_dims& d, SelectiveArgs& a, hipStream_t stream);

// Calls f(S, NS, type) for d.d_state: S lanes a channel, NS states a lane.
template <typename F>
hipError_t selective_dispatch(const ssm_selective_dims& d, F&& f) {
  auto with = [&](auto S, auto NS) -> hipError_t {
    if (d.in_dtype == SSM_IN_BF16) return f(S, NS, type_tag<uint16_t>{});
    return f(S, NS, type_tag<float>{});
  };
  switch (d.d_state) {
    case 8: return with(std::integral_constant<int, 4>{}, std::integral_constant<int, 2>{});
    case 16: return with(std::integral_constant<int, 4>{}, std::integral_constant<int, 4>{});
    case 32: return with(std::integral_constant<int, 8>{}, std::integral_constant<int, 4>{});
    case 64: return with(std::integral_constant<int, 16>{}, std::integral_constant<int, 4>{});
  }
  return hipErrorInvalidValue;
}

}  // namespace ssm
