// selective.hpp -- the selective recurrence over packed prompts: what the forward and backward passes share.
//
// A wave takes 64 / S channels: S lanes a channel, each with NS = d_state / S of its states. Sixteen
// tokens ("a block") at a time are read by all lanes (lane = 4 * token + quarter, 16 / S channels
// and d_state / 4 values of B and C a lane), turned into fp32 with softplus taken once per
// token and channel, and passed through LDS of the wave's own: no workgroup barrier. Per state and
// token the recurrence is a product, an exp2, a product and two fused ones, so prompts are bound by the
// vector ALU, not by HBM. (exp2 takes two issue slots here: six a state and token at the least. One prompt of 8192 tokens,
// 5120 channels x 16 states: the main pass 169 us, 8.3 instructions a state and token, of which 5 are the recurrence,
// 0.75 the sum over lanes, the rest softplus, gate, conversions and LDS, all once for 16 states; its vector units
// issue all the time. The local pass 122 us, 5.6 instructions. Times are of a GPU that has been busy for 30 ms; its clock
// rises over them, and the first passes after a pause take 204 and 147 us.)
//
// Time is divided too: the plan's 64-token chunks go to `groups` of equal size, whatever sequences
// they belong to, and a wave walks one group. A sequence that crosses groups needs its state
// at each group's start: a first pass ("local") takes every group's part from a state of zero and
// notes the sum of delta, and the main pass joins the groups before its own,
//   h <- exp(A sum delta) h + local,
// which costs a few exps a group. Likewise backwards, where the gradient that leaves a group at its start
// is sum_t P_t C_t dy_t with P_t the product of the decays up to t: taken in the same forward
// walk, which also keeps the states that the walk back starts from (selective_grads.hip).
#pragma once

#include "layer.hpp"
#include "launch.hpp"

namespace ssm {

constexpr int TB = 16;     // tokens of a block
constexpr int HB = KT;     // tokens between the states that the backward pass starts from
constexpr int WAVES = 4;   // of a workgroup

// log(1 + e^x) = max(x, 0) + 2 atanh(s), s = e / (2 + e), e = e^-|x| <= 1, so small values keep their digits.
// atanh(s) / s as a polynomial in q = s^2 <= 1/9 whose largest relative error is the least (7.8e-9, 2^-26.9). x = +inf
// and NaN pass through.
__device__ __forceinline__ float softplus(float x) {
  const float e = __builtin_amdgcn_exp2f(-kLog2e * fabsf(x));
  const float s = e * __builtin_amdgcn_rcpf(2.f + e), q = s * s;
  float p = fmaf(q, 0.140891671f, 0.139803007f);
  p = fmaf(q, p, 0.200124547f);
  p = fmaf(q, p, 0.333331585f);
  p = fmaf(q, p, 1.f);
  return fmaf(2.f * s, p, fmaxf(x, 0.f));
}

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
// Sum over a block's tokens of what a lane has read: the lanes with the same quarter.
__device__ __forceinline__ float token_sum(float x) {
  x += dpp<DPP_ROR4>(x);
  x += dpp<DPP_ROR8>(x);
  return xsum32(xsum16(x));
}

// The wave's tile of channels, and the lane's place in it.
struct SelTile {
  int c0, group;         // first channel, and the group of B and C
  int lane, t, q;        // reading: token t of a block, quarter q
  int ch, sg;            // computing: channel ch of the tile, states sg * NS ..
};
template <int S>
__device__ __forceinline__ SelTile sel_tile(const SelectiveArgs& a, int tile) {
  SelTile w;
  w.c0 = tile * (64 / S);
  w.group = w.c0 / (a.channels / a.groups);
  w.lane = threadIdx.x & 63;
  w.t = w.lane >> 2;
  w.q = w.lane & 3;
  w.ch = w.lane / S;
  w.sg = w.lane % S;
  return w;
}

// One value for the wave, in a scalar register (the plan is read by vector loads).
__device__ __forceinline__ int scalar(int x) { return __builtin_amdgcn_readfirstlane(x); }

// Element `col` of row `row` (both the lane's) behind row tok0 (the wave's): a scalar base and an offset of
// 32 bits (strides are below 2^26), so that an array's place takes one vector register, not two, and the
// base one product of 32 bits by 32.
template <typename T>
__device__ __forceinline__ T* row_at(const Rows& m, int tok0, int row, int col) {
  const uint32_t pitch = (uint32_t)m.stride * (uint32_t)sizeof(T);
  char* base = static_cast<char*>(const_cast<void*>(m.p)) + (uint64_t)(uint32_t)tok0 * pitch;
  return reinterpret_cast<T*>(base + (uint32_t)((uint32_t)row * pitch + (uint32_t)col * (uint32_t)sizeof(T)));
}

template <typename T, int E>
__device__ __forceinline__ void mask_out(Packed<T, E>& r, uint32_t mask) {
#pragma unroll
  for (int i = 0; i < Packed<T, E>::NW; ++i) r.w[i] &= mask;
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

// A chunk of the plan that holds tokens.
struct SelCell {
  int entry, seq, slot, first, len, pos, count;
  __device__ __forceinline__ bool starts() const { return pos == 0; }
  __device__ __forceinline__ bool ends() const { return pos + count == len; }
};
__device__ __forceinline__ bool sel_slot(const SelectiveArgs& a, int seq, int& slot) {
  slot = a.slot ? a.slot[seq] : seq;
  return slot >= 0 && slot < a.num_slots;
}
__device__ __forceinline__ bool sel_cell(const SelectiveArgs& a, int e, SelCell& c) {
  c = SelCell{};
  int ok = a.plan.locate(e, c.seq, c.first, c.len, c.pos) && sel_slot(a, c.seq, c.slot);
  c.entry = e;
  c.seq = scalar(c.seq);
  c.slot = scalar(c.slot);
  c.first = scalar(c.first);
  c.len = scalar(c.len);
  c.pos = scalar(c.pos);
  c.count = min(c.len - c.pos, CT);
  return scalar(ok);
}
// The first such chunk in [e, end), or in (end, e] going down.
__device__ __forceinline__ bool next_cell(const SelectiveArgs& a, int e, int end, SelCell& c) {
  for (; e < end; ++e)
    if (sel_cell(a, e, c)) return true;
  return false;
}
__device__ __forceinline__ bool prev_cell(const SelectiveArgs& a, int e, int end, SelCell& c) {
  for (; e > end; --e)
    if (sel_cell(a, e, c)) return true;
  return false;
}

// A group's entries of the chunk table.
struct SelGroup {
  int g, e0, e1;
};
__device__ __forceinline__ SelGroup sel_group(const SelectiveArgs& a, int g) {
  return SelGroup{g, g * a.group_chunks, min((g + 1) * a.group_chunks, a.plan.cap)};
}
// The entries of sequence s that a plan gives it, cut to the table.
__device__ __forceinline__ int seq_entry(const SelectiveArgs& a, int s) {
  return min(max(a.plan.chunk(s), 0), a.plan.cap);
}

// f(sequence, slot) for the sequences without tokens among the group's entries' numbers (the table has an
// entry for every sequence).
template <typename F>
__device__ __forceinline__ void for_empty_sequences(const SelectiveArgs& a, const SelGroup& g, F&& f) {
  const int lane = threadIdx.x & 63;
  for (int e = g.e0; e < g.e1 && e < a.plan.seqs; e += 64) {
    int tok, len = 1, first, slot = 0;
    const int s = e + lane;
    const bool none = s < g.e1 && s < a.plan.seqs && a.plan.sequence(s, tok, len, first) && len == 0 &&
                      sel_slot(a, s, slot);
    for (uint64_t left = __ballot(none); left; left &= left - 1) {
      const int l = __builtin_ctzll(left);
      f(e + l, __builtin_amdgcn_readlane(slot, l));
    }
  }
}

template <int NS>
__device__ __forceinline__ void zero(float (&h)[NS]) {
#pragma unroll
  for (int i = 0; i < NS; ++i) h[i] = 0.f;
}

// One block of a sequence: raw inputs of the lane's token, zero where there is none (the block's last row is
// read all the same and masked out: a branch around every load costs more).
template <typename T, int S, int NS, bool C, bool Z, bool DY>
struct SelBlock {
  using SH = SelShape<S, NS>;
  Packed<T, SH::EC> x, dt, z, dy;
  Packed<T, SH::EN> b, c;
  // what the state is made of
  __device__ __forceinline__ void load_state(const SelectiveArgs& a, const SelTile& w, const SelCell& cell, int t0) {
    const int tok0 = cell.first + cell.pos + t0;
    const int left = cell.count - t0, row = min(w.t, left - 1);
    const int c0 = w.c0 + w.q * SH::EC, n0 = w.group * SH::N + w.q * SH::EN;
    x.load(row_at<T>(a.x, tok0, row, c0));
    dt.load(row_at<T>(a.dt, tok0, row, c0));
    b.load(row_at<T>(a.B, tok0, row, n0));
    if (left < TB) {
      const uint32_t mask = w.t < left ? 0xFFFFFFFFu : 0u;
      mask_out(x, mask);
      mask_out(dt, mask);
      mask_out(b, mask);
    }
  }
  // and the rest
  __device__ __forceinline__ void load_more(const SelectiveArgs& a, const SelTile& w, const SelCell& cell, int t0) {
    const int tok0 = cell.first + cell.pos + t0;
    const int left = cell.count - t0, row = min(w.t, left - 1);
    const int c0 = w.c0 + w.q * SH::EC, n0 = w.group * SH::N + w.q * SH::EN;
    if constexpr (Z) z.load(row_at<T>(a.z, tok0, row, c0));  // x where there is no gate
    if constexpr (C) c.load(row_at<T>(a.C, tok0, row, n0));
    if constexpr (DY) dy.load(row_at<T>(a.dout, tok0, row, c0));
    if (left < TB) {
      const uint32_t mask = w.t < left ? 0xFFFFFFFFu : 0u;
      if constexpr (Z) mask_out(z, mask);
      if constexpr (C) mask_out(c, mask);
      if constexpr (DY) mask_out(dy, mask);
    }
  }
  __device__ __forceinline__ void load(const SelectiveArgs& a, const SelTile& w, const SelCell& cell, int t0) {
    load_state(a, w, cell, t0);
    load_more(a, w, cell, t0);
  }
};

// Steps and gates of a lane's channels. One branch of the wave for all of them: a branch for each value
// costs more than the value.
template <int E>
__device__ __forceinline__ void steps(const SelectiveArgs& a, const float (&raw)[E], bool whole, bool on,
                                      float (&delta)[E]) {
#pragma unroll
  for (int i = 0; i < E; ++i) delta[i] = raw[i];
  if (a.softplus) {
#pragma unroll
    for (int i = 0; i < E; ++i) delta[i] = softplus(raw[i]);
  }
  if (!whole) {  // rows without a token leave the state as it is
#pragma unroll
    for (int i = 0; i < E; ++i) delta[i] = on ? delta[i] : 0.f;
  }
}
template <int E>
__device__ __forceinline__ void apply_gate(const SelectiveArgs& a, const float (&z)[E], float (&v)[E]) {
  if (a.gated) {
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] *= z[i] * sigmoid(z[i]);
  }
}

// A channel parameter of the wave's tile in LDS, zero where there is none: read by every block, and registers
// are short.
template <int CH>
__device__ __forceinline__ void stage_channels(float (&to)[CH], const float* from, const SelTile& w) {
  if (w.lane < CH) to[w.lane] = from ? from[w.c0 + w.lane] : 0.f;
}

// The state before the group's first chunk c, which is not its sequence's first: the groups before.
template <int N, int NS>
__device__ __forceinline__ void carry_in(const SelectiveArgs& a, const SelGroup& g, const SelCell& c, int my,
                                         int n0, const float (&A2)[NS], float (&h)[NS]) {
  zero(h);
  const int from = seq_entry(a, c.seq) / a.group_chunks;
  const size_t step = (size_t)a.channels * N;
  const float* p = a.w.local + ((size_t)from * a.channels + my) * N + n0;
  const float* d = a.w.sums + (size_t)from * a.channels + my;
#pragma unroll 4
  for (int i = from; i < g.g; ++i, p += step, d += a.channels) {
    float l[NS];
    Vec<float, NS>::load(p, l);
    const float sum = i > from ? *d : 0.f;  // nothing yet to decay
#pragma unroll
    for (int k = 0; k < NS; ++k) h[k] = fmaf(__builtin_amdgcn_exp2f(A2[k] * sum), h[k], l[k]);
  }
}
// The gradient that enters the group's last chunk c from behind, where its sequence goes on.
template <int N, int NS>
__device__ __forceinline__ void carry_back(const SelectiveArgs& a, const SelGroup& g, const SelCell& c, int my,
                                           int n0, const float (&A2)[NS], float (&h)[NS]) {
  zero(h);
  const int last = min(max(seq_entry(a, c.seq + 1) - 1, 0) / a.group_chunks, a.time_groups - 1);
#pragma unroll 4
  for (int i = last; i > g.g; --i) {
    float l[NS];
    Vec<float, NS>::load(a.w.back + ((size_t)i * a.channels + my) * N + n0, l);
    const float sum = i < last ? a.w.sums[(size_t)i * a.channels + my] : 0.f;  // nothing yet to decay
#pragma unroll
    for (int k = 0; k < NS; ++k) h[k] = fmaf(__builtin_amdgcn_exp2f(A2[k] * sum), h[k], l[k]);
  }
}

// Groups of the chunk table: chunks of a group, and their number.
struct SelGroups {
  int chunks, groups;
};
SelGroups selective_groups(const ssm_selective_dims& d, int cap);

inline int selective_tiles(const ssm_selective_dims& d) {  // of selective_dispatch's mapping
  const int S = d.d_state <= 16 ? 4 : d.d_state / 4;
  return d.channels * S / 64;
}

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

// Launches a pass over the groups: f(S, NS, type, grid).
template <typename F>
hipError_t over_groups(const ssm_selective_dims& d, const SelectiveArgs& a, F&& f) {
  const unsigned tile_blocks = (unsigned)(selective_tiles(d) + WAVES - 1) / WAVES;
  return selective_dispatch(d, [&](auto S, auto NS, auto T) {
    f(S, NS, T, dim3(tile_blocks * (unsigned)a.time_groups));
    return hipGetLastError();
  });
}

}  // namespace ssm
