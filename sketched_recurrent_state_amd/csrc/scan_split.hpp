// scan_split.hpp -- the passes along a sequence of scan_state.hpp on the bf16 matrix cores,
// for scalar gates and bf16 inputs (kSplit): the state, kept in fp32, is split into three
// bf16 parts once per block and multiplied by the exact keys and queries.
//
// Rows of the state's tiles: tile 2s + h holds channel 32 s + 8 g + 4 h + i in row 4g + i, so
// that the two tiles' registers are the 32-deep B operand whose slot 8g + j is channel
// 32 s + 8 g + j: the A operand is then 16 consecutive bytes of a key. The update needs the
// keys the other way round (four tokens of one channel): the block's keys go through LDS and
// come back with ds_read_b64_tr_b16.
#pragma once

#include "scan.hpp"

namespace ssm {

template <int DK>
struct KeyTile {
  // Row stride in bytes: rows 16 dwords apart modulo the 64 banks, so that the 4 rows x 4
  // pieces of 8 bytes that 16 lanes read together fall on different banks.
  static constexpr int STRIDE = DK >= 128 ? 2 * DK + 64 : DK == 64 ? 192 : 64;
  static constexpr int BYTES = SB * STRIDE;
  // Lane (m, g)'s part of the block: channels 32 s + 8 g .. + 7 of token m.
  static __device__ __forceinline__ void put(char* lds, int m, int g, const uint4 (&k)[DK / 32]) {
#pragma unroll
    for (int s = 0; s < DK / 32; ++s)
      *reinterpret_cast<uint4*>(lds + m * STRIDE + 64 * s + 16 * g) = k[s];
  }
  // Tokens 4g .. 4g + 3 of the channel in row m of tile t = 2s + h. Sixteen lanes transpose
  // four rows of 16 values: lane p + 4 r names values 4p .. 4p + 3 of row r and receives column
  // p + 4 r of the four.
  static __device__ __forceinline__ uint2 column(const char* lds, int m, int g, int t) {
    const char* p = lds + (4 * g + (m >> 2)) * STRIDE + 64 * (t >> 1) + 16 * (m & 3) + 8 * (t & 1);
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p));
  }
};

// Channel of row i (of this lane's four) of tile t.
__device__ __forceinline__ int split_channel(int t, int g, int i) {
  return 32 * (t >> 1) + 8 * g + 4 * (t & 1) + i;
}

template <int RULE, int DK, bool BWD>
struct SplitStateStep {
  static constexpr int KS = DK / 32;
  uint4 k[KS], q[KS];
  uint16_t v[4];
  Split4 A, P;
  float4 in, out, b;
  float all;

  __device__ __forceinline__ void load(const ScanArgs& a, size_t cell, int blk, int tok, int count,
                                       int h, int col, int lane, int m, int g) {
    const uint16_t* pk = static_cast<const uint16_t*>(a.k);
    const uint16_t* pq = static_cast<const uint16_t*>(a.q);
    const uint16_t* pv = static_cast<const uint16_t*>(a.v);
    const size_t at = ((size_t)(tok + min(m, count - 1)) * a.heads + h) * DK + 8 * g;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      k[s] = *reinterpret_cast<const uint4*>(pk + at + 32 * s);
      if constexpr (!BWD) q[s] = *reinterpret_cast<const uint4*>(pq + at + 32 * s);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = pv[((size_t)(tok + min(4 * g + i, count - 1)) * a.heads + h) * a.d_v + col];
    const float* row = a.w.row + cell * 3 * CT + SB * blk;
    in = *reinterpret_cast<const float4*>(row + 4 * g);
    out = *reinterpret_cast<const float4*>(row + CT + 4 * g);
    all = row[SB - 1];
    if constexpr (!BWD) load_split(a.w.P, cell * NB + blk, lane, P);
    if constexpr (RULE != MAMBA2) {
      b = *reinterpret_cast<const float4*>(row + 2 * CT + 4 * g);
      load_split(a.w.A, cell * NB + blk, lane, A);
    }
  }
  // Zero for the rows behind the sequence's end, when the block is used (a loaded value that
  // is touched has been waited for).
  __device__ __forceinline__ void clip(int count, int m, int g) {
    const uint32_t rm = row_mask(m < count);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      k[s] = masked(k[s], rm);
      if constexpr (!BWD) q[s] = masked(q[s], rm);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = masked(v[i], row_mask(4 * g + i < count));
  }
};

__device__ __forceinline__ f32x4 vec(float4 x) { return f32x4{x.x, x.y, x.z, x.w}; }

// Forwards, as scan_state_kernel.
template <int RULE, int DK, bool BWD>
__global__ void __launch_bounds__(64) scan_split_state_kernel(const ScanArgs a) {
  constexpr bool DELTA = RULE != MAMBA2;
  constexpr int T = DK / 16;
  using Step = SplitStateStep<RULE, DK, BWD>;
  using KT = KeyTile<DK>;
  __shared__ __align__(16) char sk[KT::BYTES];
  int unit, part;
  unit_of(blockIdx.x, a.d_v / 16, unit, part);
  const int seq = unit / a.heads, h = unit % a.heads;
  if (seq >= a.plan.seqs) return;
  int tok, len, first;
  if (!a.plan.sequence(seq, tok, len, first)) return;
  const int srow = a.slot ? a.slot[seq] : seq;
  if (srow < 0 || srow >= a.num_slots) return;
  const int lane = threadIdx.x, m = lane & 15, g = lane >> 4, col = 16 * part + m;
  const size_t so = ((size_t)srow * a.heads + h) * DK * a.d_v + col;

  f32x4 S[T];
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      S[t][i] = a.state_in ? a.state_in[so + (size_t)split_channel(t, g, i) * a.d_v] : 0.f;

  const int blocks = (len + SB - 1) / SB;
  auto fetch = [&](Step& s, int j) {
    s.load(a, (size_t)(first + j / NB) * a.heads + h, j % NB, tok + SB * j, len - SB * j, h, col,
           lane, m, g);
  };
  auto run = [&](Step& s, int j) {
    const size_t cell = (size_t)(first + j / NB) * a.heads + h;
    if (len - SB * j < SB) s.clip(len - SB * j, m, g);
    if constexpr (BWD) {
      if (j % NB == 0) {
        float* p = a.w.S + cell * DK * a.d_v + col;
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) p[(size_t)split_channel(t, g, i) * a.d_v] = S[t][i];
      }
    }
    KT::put(sk, m, g, s.k);
    f32x4 ks = {0.f, 0.f, 0.f, 0.f}, o = ks, w;
    if constexpr (DELTA || !BWD) {
#pragma unroll
      for (int c = 0; c < T / 2; ++c) {
        const Split4 x = split4(S[2 * c]), y = split4(S[2 * c + 1]);
        const uint4 sh = make_uint4(x.h.x, x.h.y, y.h.x, y.h.y);
        const uint4 sm = make_uint4(x.m.x, x.m.y, y.m.x, y.m.y);
        const uint4 sl = make_uint4(x.l.x, x.l.y, y.l.x, y.l.y);
        if constexpr (DELTA) {
          ks = mfma32(s.k[c], sl, ks);
          ks = mfma32(s.k[c], sm, ks);
          ks = mfma32(s.k[c], sh, ks);
        }
        if constexpr (!BWD) {
          o = mfma32(s.q[c], sl, o);
          o = mfma32(s.q[c], sm, o);
          o = mfma32(s.q[c], sh, o);
        }
      }
    }
    const f32x4 in = vec(s.in);
    if constexpr (DELTA) {
      f32x4 r;
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = to_f32(s.v[i]) - in[i] * ks[i];
      r = mfma_split(s.A, split4(r), f32x4{0.f, 0.f, 0.f, 0.f});
      if constexpr (BWD) {
#pragma unroll
        for (int i = 0; i < 4; ++i) a.w.r[(cell * CT + SB * (j % NB) + 4 * g + i) * a.d_v + col] = r[i];
      }
      w = vec(s.b) * r;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = to_f32(s.v[i]);
    }
    // S <- a_1..a_16 S + k^T (O w)
    const Split4 ow = split4(vec(s.out) * w);
#pragma unroll
    for (int t = 0; t < T; ++t) S[t] = mfma_exact(KT::column(sk, m, g, t), ow, S[t] * s.all);
    if constexpr (!BWD) {
      o *= in;
      if constexpr (DELTA) {
        o = mfma_split(s.P, split4(w), o);
      } else {  // the values are exact
        const uint2 v = make_uint2(s.v[0] | (uint32_t)s.v[1] << 16, s.v[2] | (uint32_t)s.v[3] << 16);
        o = mfma_two(s.P.l, v, make_uint2(0u, 0u), make_uint2(0u, 0u), o);
        o = mfma_two(s.P.h, v, s.P.m, v, o);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (SB * j + 4 * g + i < len)
          a.y[((size_t)(tok + SB * j + 4 * g + i) * a.heads + h) * a.d_v + col] = o[i];
    }
  };
  Step s0, s1;
  if (blocks > 0) fetch(s0, 0);
  for (int j = 0; j < blocks; j += 2) {
    if (j + 1 < blocks) fetch(s1, j + 1);
    run(s0, j);
    if (j + 1 >= blocks) break;
    if (j + 2 < blocks) fetch(s0, j + 2);
    run(s1, j + 1);
  }
  if constexpr (!BWD) {
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) a.state[so + (size_t)split_channel(t, g, i) * a.d_v] = S[t][i];
  }
}

template <int RULE, int DK>
struct SplitGradientStep {
  static constexpr int KS = DK / 32;
  uint4 k[KS], q[KS];
  float dy[4];
  Split4 A, P;  // transposed
  float4 in, out, b;
  float all;

  __device__ __forceinline__ void load(const ScanArgs& a, size_t cell, int blk, int tok, int count,
                                       int h, int col, int lane, int m, int g) {
    const uint16_t* pk = static_cast<const uint16_t*>(a.k);
    const uint16_t* pq = static_cast<const uint16_t*>(a.q);
    const size_t at = ((size_t)(tok + min(m, count - 1)) * a.heads + h) * DK + 8 * g;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      k[s] = *reinterpret_cast<const uint4*>(pk + at + 32 * s);
      q[s] = *reinterpret_cast<const uint4*>(pq + at + 32 * s);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      dy[i] = a.dy[((size_t)(tok + min(4 * g + i, count - 1)) * a.heads + h) * a.d_v + col];
    const float* row = a.w.row + cell * 3 * CT + SB * blk;
    in = *reinterpret_cast<const float4*>(row + 4 * g);
    out = *reinterpret_cast<const float4*>(row + CT + 4 * g);
    all = row[SB - 1];
    load_split(a.w.P, cell * NB + blk, lane, P);
    if constexpr (RULE != MAMBA2) {
      b = *reinterpret_cast<const float4*>(row + 2 * CT + 4 * g);
      load_split(a.w.A2, cell * NB + blk, lane, A);
    }
  }
  __device__ __forceinline__ void clip(int count, int m, int g) {
    const uint32_t rm = row_mask(m < count);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      k[s] = masked(k[s], rm);
      q[s] = masked(q[s], rm);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) dy[i] = masked(dy[i], row_mask(4 * g + i < count));
  }
};

// Backwards, as scan_gradient_kernel.
template <int RULE, int DK>
__global__ void __launch_bounds__(64) scan_split_gradient_kernel(const ScanArgs a) {
  constexpr bool DELTA = RULE != MAMBA2;
  constexpr int T = DK / 16;
  using Step = SplitGradientStep<RULE, DK>;
  using KT = KeyTile<DK>;
  __shared__ __align__(16) char sk[KT::BYTES], sq[KT::BYTES];
  int unit, part;
  unit_of(blockIdx.x, a.d_v / 16, unit, part);
  const int seq = unit / a.heads, h = unit % a.heads;
  if (seq >= a.plan.seqs) return;
  int tok, len, first;
  if (!a.plan.sequence(seq, tok, len, first)) return;
  const int lane = threadIdx.x, m = lane & 15, g = lane >> 4, col = 16 * part + m;
  const size_t so = ((size_t)seq * a.heads + h) * DK * a.d_v + col;
  uint16_t* dv = static_cast<uint16_t*>(a.dv);

  f32x4 G[T];
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      G[t][i] = a.dstate ? a.dstate[so + (size_t)split_channel(t, g, i) * a.d_v] : 0.f;

  const int blocks = (len + SB - 1) / SB;
  auto fetch = [&](Step& s, int j) {
    s.load(a, (size_t)(first + j / NB) * a.heads + h, j % NB, tok + SB * j, len - SB * j, h, col,
           lane, m, g);
  };
  auto run = [&](Step& s, int j) {
    const size_t cell = (size_t)(first + j / NB) * a.heads + h;
    if (len - SB * j < SB) s.clip(len - SB * j, m, g);
    if (j % NB == NB - 1 || j == blocks - 1) {
      float* p = a.w.G + cell * DK * a.d_v + col;
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) p[(size_t)split_channel(t, g, i) * a.d_v] = G[t][i];
    }
    KT::put(sq, m, g, s.q);
    if constexpr (DELTA) KT::put(sk, m, g, s.k);
    f32x4 w = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < T / 2; ++c) {
      const Split4 x = split4(G[2 * c]), y = split4(G[2 * c + 1]);
      w = mfma32(s.k[c], make_uint4(x.l.x, x.l.y, y.l.x, y.l.y), w);
      w = mfma32(s.k[c], make_uint4(x.m.x, x.m.y, y.m.x, y.m.y), w);
      w = mfma32(s.k[c], make_uint4(x.h.x, x.h.y, y.h.x, y.h.y), w);
    }
    const f32x4 in = vec(s.in), dy = {s.dy[0], s.dy[1], s.dy[2], s.dy[3]};
    w *= vec(s.out);
    w = mfma_split(s.P, split4(dy), w);
    const Split4 iy = split4(in * dy);
#pragma unroll
    for (int t = 0; t < T; ++t) G[t] = mfma_exact(KT::column(sq, m, g, t), iy, G[t] * s.all);
    f32x4 dr = w;
    if constexpr (DELTA) {
      const f32x4 e = mfma_split(s.A, split4(w), f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
      for (int i = 0; i < 4; ++i) a.w.e[(cell * CT + SB * (j % NB) + 4 * g + i) * a.d_v + col] = e[i];
      dr = vec(s.b) * e;
      const Split4 ir = split4(-(in * dr));
#pragma unroll
      for (int t = 0; t < T; ++t) G[t] = mfma_exact(KT::column(sk, m, g, t), ir, G[t]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (SB * j + 4 * g + i < len)
        put(dv + ((size_t)(tok + SB * j + 4 * g + i) * a.heads + h) * a.d_v + col, dr[i]);
  };
  Step s0, s1;
  if (blocks > 0) fetch(s0, blocks - 1);
  for (int j = blocks - 1; j >= 0; j -= 2) {
    if (j >= 1) fetch(s1, j - 1);
    run(s0, j);
    if (j < 1) break;
    if (j >= 2) fetch(s0, j - 2);
    run(s1, j - 1);
  }
  if (a.dstate_in) {
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) a.dstate_in[so + (size_t)split_channel(t, g, i) * a.d_v] = G[t][i];
  }
}

}  // namespace ssm
