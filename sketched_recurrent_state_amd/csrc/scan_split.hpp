// scan_split.hpp -- the passes along a sequence of scan_state.hpp on the bf16 matrix cores,
// for scalar gates and bf16 inputs (kSplit): the state, kept in fp32, is split into three
// bf16 parts once per block and multiplied by the exact keys and queries.
//
// A wave holds 16 columns of the state, or DK / DS rows of them: with few units (see
// scan_rule.hpp) DS waves share a column block, and add up their parts of k S and q S through
// LDS. The waves of a workgroup share the block's operands: they are loaded into registers
// two blocks ahead, put into the other half of a double buffer in LDS, and read from there.
//
// Rows of the state's tiles: tile 2s + h holds channel 32 s + 8 g + 4 h + i in row 4g + i, so
// that the two tiles' registers are the 32-deep B operand whose slot 8g + j is channel
// 32 s + 8 g + j: the A operand is then 16 consecutive bytes of a key. The update needs the
// keys the other way round (four tokens of one channel): ds_read_b64_tr_b16 transposes them.
//
// Rows behind the sequence's end are given the last token's keys and queries (the plan of a
// partial block has b = 0 and no P or K there), and values and dy of zero: they write nothing.
#pragma once

#include "scan.hpp"

namespace ssm {

template <int DK>
struct KeyTile {
  // Row stride in bytes: rows 16 dwords apart modulo the 64 banks, so that the 4 rows x 4
  // pieces of 8 bytes that 16 lanes read together fall on different banks.
  static constexpr int STRIDE = DK >= 128 ? 2 * DK + 64 : DK == 64 ? 192 : 64;
  static constexpr int BYTES = SB * STRIDE;
  static __device__ __forceinline__ void put(char* lds, int piece, uint4 x) {
    *reinterpret_cast<uint4*>(lds + piece / (DK / 8) * STRIDE + piece % (DK / 8) * 16) = x;
  }
  // Channels 32 s + 8 g .. + 7 of token m.
  static __device__ __forceinline__ uint4 row(const char* lds, int m, int g, int s) {
    return *reinterpret_cast<const uint4*>(lds + m * STRIDE + 64 * s + 16 * g);
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

__device__ __forceinline__ f32x4 vec(float4 x) { return f32x4{x.x, x.y, x.z, x.w}; }

// The operands of one block that the workgroup shares.
template <int DK>
struct SplitBlock {
  __align__(16) char k[KeyTile<DK>::BYTES];
  __align__(16) char q[KeyTile<DK>::BYTES];
  uint2 P[192], A[192];  // split operands, 3 x 64 lanes
  __align__(16) float row[3 * SB];  // decay in, decay out, b

  __device__ __forceinline__ Split4 split(const uint2* p, int lane) const {
    return Split4{p[lane], p[64 + lane], p[128 + lane]};
  }
  __device__ __forceinline__ f32x4 rows(int which, int g) const {
    return vec(*reinterpret_cast<const float4*>(row + SB * which + 4 * g));
  }
};

// A thread's share of a block, in registers between the load and the LDS write.
template <int DK, int NT, bool Q, bool DELTA, bool P>
struct SplitShare {
  static constexpr int KP = SB * DK / 8, NK = (KP + NT - 1) / NT, NP = (192 + NT - 1) / NT;
  uint4 k[NK], q[Q ? NK : 1];
  uint2 p[P ? NP : 1], a[DELTA ? NP : 1];
  float row;

  // A is the operand of the state's pass or of the gradient's.
  __device__ __forceinline__ void load(const ScanArgs& s, const float* A, size_t cell, int blk,
                                       int tok, int count, int h, int tid) {
    const uint16_t* pk = static_cast<const uint16_t*>(s.k);
    const uint16_t* pq = static_cast<const uint16_t*>(s.q);
#pragma unroll
    for (int n = 0; n < NK; ++n) {
      const int piece = min(tid + n * NT, KP - 1);  // the surplus threads load the last one again
      const int r = min(piece / (DK / 8), count - 1);
      const size_t at = ((size_t)(tok + r) * s.heads + h) * DK + piece % (DK / 8) * 8;
      k[n] = *reinterpret_cast<const uint4*>(pk + at);
      if constexpr (Q) q[n] = *reinterpret_cast<const uint4*>(pq + at);
    }
    const size_t block = (cell * NB + blk) * 192;
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      const int i = min(tid + n * NT, 191);
      if constexpr (P) p[n] = reinterpret_cast<const uint2*>(s.w.P)[block + i];
      if constexpr (DELTA) a[n] = reinterpret_cast<const uint2*>(A)[block + i];
    }
    const int i = min(tid, 3 * SB - 1);
    row = s.w.row[cell * 3 * CT + (i / SB) * CT + SB * blk + i % SB];
  }
  __device__ __forceinline__ void put(SplitBlock<DK>& b, int tid) const {
#pragma unroll
    for (int n = 0; n < NK; ++n) {
      const int piece = tid + n * NT;
      if (KP % NT == 0 || piece < KP) {
        KeyTile<DK>::put(b.k, piece, k[n]);
        if constexpr (Q) KeyTile<DK>::put(b.q, piece, q[n]);
      }
    }
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      const int i = tid + n * NT;
      if (192 % NT == 0 || i < 192) {
        if constexpr (P) b.P[i] = p[n];
        if constexpr (DELTA) b.A[i] = a[n];
      }
    }
    if (tid < 3 * SB) b.row[tid] = row;
  }
};

// k times the state's tiles of this wave (channels from 32 s0), in three parts.
template <int DK, int TL>
__device__ __forceinline__ void state_products(const char* k, const char* q, bool with_k, bool with_q,
                                               const f32x4 (&S)[TL], int s0, int m, int g,
                                               f32x4& ks, f32x4& qs) {
#pragma unroll
  for (int c = 0; c < TL / 2; ++c) {
    const Split4 x = split4(S[2 * c]), y = split4(S[2 * c + 1]);
    const uint4 sh = make_uint4(x.h.x, x.h.y, y.h.x, y.h.y);
    const uint4 sm = make_uint4(x.m.x, x.m.y, y.m.x, y.m.y);
    const uint4 sl = make_uint4(x.l.x, x.l.y, y.l.x, y.l.y);
    if (with_k) {
      const uint4 a = KeyTile<DK>::row(k, m, g, s0 + c);
      ks = mfma32(a, sl, ks);
      ks = mfma32(a, sm, ks);
      ks = mfma32(a, sh, ks);
    }
    if (with_q) {
      const uint4 a = KeyTile<DK>::row(q, m, g, s0 + c);
      qs = mfma32(a, sl, qs);
      qs = mfma32(a, sm, qs);
      qs = mfma32(a, sh, qs);
    }
  }
}

// The sum of x over the DS waves that share this wave's columns. `slot`: LDS for every wave's x.
template <int DS>
__device__ __forceinline__ f32x4 wave_sum(const f32x4* slot, int wave, int lane) {
  f32x4 s = slot[(wave / DS * DS) * 64 + lane];
#pragma unroll
  for (int i = 1; i < DS; ++i) s += slot[(wave / DS * DS + i) * 64 + lane];
  return s;
}

// Forwards, as scan_state_kernel.
template <int RULE, int DK, int NW, int DS, bool BWD>
__global__ void __launch_bounds__(64 * NW, 2) scan_split_state_kernel(const ScanArgs a) {
  constexpr bool DELTA = RULE != MAMBA2;
  constexpr int TL = DK / 16 / DS, NT = 64 * NW, CB = NW / DS;
  using Share = SplitShare<DK, NT, !BWD, DELTA, !BWD>;
  __shared__ SplitBlock<DK> buf[2];
  __shared__ f32x4 xk[DS > 1 && DELTA ? NT : 1], xq[DS > 1 && !BWD ? NT : 1];
  int unit, part;
  unit_of(blockIdx.x, a.d_v / (16 * CB), unit, part);
  const int seq = unit / a.heads, h = unit % a.heads;
  if (seq >= a.plan.seqs) return;
  int tok, len, first;
  if (!a.plan.sequence(seq, tok, len, first)) return;
  const int srow = a.slot ? a.slot[seq] : seq;
  if (srow < 0 || srow >= a.num_slots) return;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, m = lane & 15, g = lane >> 4;
  const int col = 16 * (part * CB + wave / DS) + m, dpart = wave % DS, s0 = dpart * TL / 2;
  const size_t so = ((size_t)srow * a.heads + h) * DK * a.d_v + (size_t)(32 * s0) * a.d_v + col;
  const size_t stride = (size_t)a.heads * a.d_v;
  const size_t ro = ((size_t)tok * a.heads + h) * a.d_v + col;  // row 0 of v and y
  const uint16_t* v = static_cast<const uint16_t*>(a.v) + ro;

  f32x4 S[TL];
#pragma unroll
  for (int t = 0; t < TL; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      S[t][i] = a.state_in ? a.state_in[so + (size_t)split_channel(t, g, i) * a.d_v] : 0.f;

  const int blocks = (len + SB - 1) / SB;
  struct Ahead {
    Share s;
    uint16_t v[4];
  };
  auto fetch = [&](Ahead& x, int j) {
    x.s.load(a, a.w.A, (size_t)(first + j / NB) * a.heads + h, j % NB, tok + SB * j, len - SB * j, h,
             tid);
#pragma unroll
    for (int i = 0; i < 4; ++i) x.v[i] = v[(size_t)min(SB * j + 4 * g + i, len - 1) * stride];
  };
  auto run = [&](const SplitBlock<DK>& b, const uint16_t (&vr)[4], int j) {
    const size_t cell = (size_t)(first + j / NB) * a.heads + h;
    if constexpr (BWD) {
      if (j % NB == 0) {
        float* p = a.w.S + (cell * DK + 32 * s0) * a.d_v + col;
#pragma unroll
        for (int t = 0; t < TL; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) p[(size_t)split_channel(t, g, i) * a.d_v] = S[t][i];
      }
    }
    f32x4 ks = {0.f, 0.f, 0.f, 0.f}, o = ks, w;
    if constexpr (DELTA || !BWD)
      state_products<DK, TL>(b.k, b.q, DELTA, !BWD, S, s0, m, g, ks, o);
    if constexpr (DS > 1 && (DELTA || !BWD)) {
      if constexpr (DELTA) xk[tid] = ks;
      if constexpr (!BWD) xq[tid] = o;
      __syncthreads();
      if constexpr (DELTA) ks = wave_sum<DS>(xk, wave, lane);
    }
    const f32x4 in = b.rows(0, g);
    f32x4 vf;
#pragma unroll
    for (int i = 0; i < 4; ++i) vf[i] = SB * j + 4 * g + i < len ? to_f32(vr[i]) : 0.f;
    if constexpr (DELTA) {
      const f32x4 r = mfma_split(b.split(b.A, lane), split4(vf - in * ks), f32x4{0.f, 0.f, 0.f, 0.f});
      if constexpr (BWD) {
        if (dpart == 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            a.w.r[(cell * CT + SB * (j % NB) + 4 * g + i) * a.d_v + col] = r[i];
        }
      }
      w = b.rows(2, g) * r;
    } else {
      w = vf;
    }
    // S <- a_1..a_16 S + k^T (O w)
    const Split4 ow = split4(b.rows(1, g) * w);
    const float all = b.row[SB - 1];
#pragma unroll
    for (int t = 0; t < TL; ++t)
      S[t] = mfma_exact(KeyTile<DK>::column(b.k, m, g, 2 * s0 + t), ow, S[t] * all);
    if constexpr (!BWD) {
      if (dpart == 0) {
        if constexpr (DS > 1) o = wave_sum<DS>(xq, wave, lane);
        o *= in;
        const Split4 P = b.split(b.P, lane);
        if constexpr (DELTA) {
          o = mfma_split(P, split4(w), o);
        } else {  // the values are exact
          const uint2 x = make_uint2(heads(vf[0], vf[1]), heads(vf[2], vf[3]));
          const uint2 none = make_uint2(0u, 0u);
          o = mfma_two(P.l, x, none, none, o);
          o = mfma_two(P.h, x, P.m, x, o);
        }
        float* y = a.y + ro + (size_t)(SB * j + 4 * g) * stride;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (SB * j + 4 * g + i < len) y[i * stride] = o[i];
      }
    }
  };
  Ahead x0, x1;
  if (blocks > 0) {
    fetch(x0, 0);
    if (blocks > 1) fetch(x1, 1);
    x0.s.put(buf[0], tid);
  }
  for (int j = 0; j < blocks; j += 2) {
    uint16_t vr[4] = {x0.v[0], x0.v[1], x0.v[2], x0.v[3]};
    if (j + 2 < blocks) fetch(x0, j + 2);
    __syncthreads();  // block j is in buf[0], and nobody reads buf[1] any more
    run(buf[0], vr, j);
    if (j + 1 >= blocks) break;
    x1.s.put(buf[1], tid);
#pragma unroll
    for (int i = 0; i < 4; ++i) vr[i] = x1.v[i];
    if (j + 3 < blocks) fetch(x1, j + 3);
    __syncthreads();
    run(buf[1], vr, j + 1);
    if (j + 2 < blocks) x0.s.put(buf[0], tid);
  }
  if constexpr (!BWD) {
#pragma unroll
    for (int t = 0; t < TL; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) a.state[so + (size_t)split_channel(t, g, i) * a.d_v] = S[t][i];
  }
}

// Backwards, as scan_gradient_kernel.
template <int RULE, int DK, int NW, int DS>
__global__ void __launch_bounds__(64 * NW, 2) scan_split_gradient_kernel(const ScanArgs a) {
  constexpr bool DELTA = RULE != MAMBA2;
  constexpr int TL = DK / 16 / DS, NT = 64 * NW, CB = NW / DS;
  using Share = SplitShare<DK, NT, true, DELTA, true>;
  __shared__ SplitBlock<DK> buf[2];
  __shared__ f32x4 xk[DS > 1 ? NT : 1];
  int unit, part;
  unit_of(blockIdx.x, a.d_v / (16 * CB), unit, part);
  const int seq = unit / a.heads, h = unit % a.heads;
  if (seq >= a.plan.seqs) return;
  int tok, len, first;
  if (!a.plan.sequence(seq, tok, len, first)) return;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, m = lane & 15, g = lane >> 4;
  const int col = 16 * (part * CB + wave / DS) + m, dpart = wave % DS, s0 = dpart * TL / 2;
  const size_t so = ((size_t)seq * a.heads + h) * DK * a.d_v + (size_t)(32 * s0) * a.d_v + col;
  const size_t stride = (size_t)a.heads * a.d_v;
  const size_t ro = ((size_t)tok * a.heads + h) * a.d_v + col;
  const float* dy = a.dy + ro;

  f32x4 G[TL];
#pragma unroll
  for (int t = 0; t < TL; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      G[t][i] = a.dstate ? a.dstate[so + (size_t)split_channel(t, g, i) * a.d_v] : 0.f;

  const int blocks = (len + SB - 1) / SB;
  struct Ahead {
    Share s;
    float dy[4];
  };
  auto fetch = [&](Ahead& x, int j) {
    x.s.load(a, a.w.A2, (size_t)(first + j / NB) * a.heads + h, j % NB, tok + SB * j, len - SB * j, h,
             tid);
#pragma unroll
    for (int i = 0; i < 4; ++i) x.dy[i] = dy[(size_t)min(SB * j + 4 * g + i, len - 1) * stride];
  };
  auto run = [&](const SplitBlock<DK>& b, const float (&yr)[4], int j) {
    const size_t cell = (size_t)(first + j / NB) * a.heads + h;
    if (j % NB == NB - 1 || j == blocks - 1) {
      float* p = a.w.G + (cell * DK + 32 * s0) * a.d_v + col;
#pragma unroll
      for (int t = 0; t < TL; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) p[(size_t)split_channel(t, g, i) * a.d_v] = G[t][i];
    }
    f32x4 w = {0.f, 0.f, 0.f, 0.f}, unused = w;
    state_products<DK, TL>(b.k, b.q, true, false, G, s0, m, g, w, unused);
    if constexpr (DS > 1) {
      xk[tid] = w;
      __syncthreads();
      w = wave_sum<DS>(xk, wave, lane);
    }
    const f32x4 in = b.rows(0, g);
    f32x4 y;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = SB * j + 4 * g + i < len ? yr[i] : 0.f;
    w = mfma_split(b.split(b.P, lane), split4(y), b.rows(1, g) * w);
    const Split4 iy = split4(in * y);
    const float all = b.row[SB - 1];
#pragma unroll
    for (int t = 0; t < TL; ++t)
      G[t] = mfma_exact(KeyTile<DK>::column(b.q, m, g, 2 * s0 + t), iy, G[t] * all);
    f32x4 dr = w;
    if constexpr (DELTA) {
      const f32x4 e = mfma_split(b.split(b.A, lane), split4(w), f32x4{0.f, 0.f, 0.f, 0.f});
      if (dpart == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          a.w.e[(cell * CT + SB * (j % NB) + 4 * g + i) * a.d_v + col] = e[i];
      }
      dr = b.rows(2, g) * e;
      const Split4 ir = split4(-(in * dr));
#pragma unroll
      for (int t = 0; t < TL; ++t)
        G[t] = mfma_exact(KeyTile<DK>::column(b.k, m, g, 2 * s0 + t), ir, G[t]);
    }
    if (dpart == 0) {
      uint16_t* dv = static_cast<uint16_t*>(a.dv) + ro + (size_t)(SB * j + 4 * g) * stride;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (SB * j + 4 * g + i < len) put(dv + i * stride, dr[i]);
    }
  };
  Ahead x0, x1;
  if (blocks > 0) {
    fetch(x0, blocks - 1);
    if (blocks > 1) fetch(x1, blocks - 2);
    x0.s.put(buf[0], tid);
  }
  for (int j = blocks - 1; j >= 0; j -= 2) {
    float yr[4] = {x0.dy[0], x0.dy[1], x0.dy[2], x0.dy[3]};
    if (j >= 2) fetch(x0, j - 2);
    __syncthreads();
    run(buf[0], yr, j);
    if (j < 1) break;
    x1.s.put(buf[1], tid);
#pragma unroll
    for (int i = 0; i < 4; ++i) yr[i] = x1.dy[i];
    if (j >= 3) fetch(x1, j - 3);
    __syncthreads();
    run(buf[1], yr, j - 1);
    if (j >= 2) x0.s.put(buf[0], tid);
  }
  if (a.dstate_in) {
#pragma unroll
    for (int t = 0; t < TL; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) a.dstate_in[so + (size_t)split_channel(t, g, i) * a.d_v] = G[t][i];
  }
}

}  // namespace ssm
