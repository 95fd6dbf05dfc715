// scan_state.hpp -- the two passes along a sequence: the state forwards
// (scan_state_kernel) and its gradient backwards (scan_gradient_kernel). Notation in
// scan.hpp.
//
// One wave holds 16 columns of one unit's state: the recurrence acts on the d_k side
// only, so columns never meet and no wave waits for another. Its d_k x 16 tile stays in
// registers from the first block to the last; the next block's operands are loaded while
// the present one is computed.
#pragma once

#include "scan.hpp"

namespace ssm {

// The element type of the decayed keys and queries: KDA's are fp32 in the workspace,
// the other rules read the inputs and scale the products' rows.
template <int RULE, typename TIN>
using KeyT = std::conditional_t<RULE == KDA, float, TIN>;

template <int RULE, int DK, typename TIN, bool BWD>
struct StateStep {
  static constexpr int T = DK / 16;
  using KT = KeyT<RULE, TIN>;
  Quad<KT> k[T], q[T];
  KT kt[T][4];
  TIN v[4];
  float A[4], P[4], in[4], out[4], b[4], all[RULE == KDA ? 4 * T : 1];

  __device__ __forceinline__ void load(const ScanArgs& a, size_t cell, int blk, int tok, int count,
                                       int h, int col, int m, int g) {
    constexpr bool DELTA = RULE != MAMBA2;
    const size_t H = a.heads;
    if constexpr (RULE == KDA) {
      const size_t o = (cell * CT + SB * blk) * DK;
#pragma unroll
      for (int t = 0; t < T; ++t) {
        k[t].load(a.w.kh + o + m * DK + 16 * t + 4 * g);
        if constexpr (!BWD) q[t].load(a.w.qh + o + m * DK + 16 * t + 4 * g);
#pragma unroll
        for (int i = 0; i < 4; ++i) kt[t][i] = a.w.kt[o + (4 * g + i) * DK + 16 * t + m];
        *reinterpret_cast<float4*>(all + 4 * t) = *reinterpret_cast<const float4*>(
            a.w.all + (cell * NB + blk) * DK + 16 * t + 4 * g);
      }
    } else {
      const TIN* pk = static_cast<const TIN*>(a.k);
      const TIN* pq = static_cast<const TIN*>(a.q);
      const bool valid = m < count;
      const size_t at = ((size_t)(tok + (valid ? m : 0)) * H + h) * DK + 4 * g;
#pragma unroll
      for (int t = 0; t < T; ++t) {
        if constexpr (DELTA) k[t].load(pk + at + 16 * t);
        if constexpr (!BWD) q[t].load(pq + at + 16 * t);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool ok = 4 * g + i < count;
        const size_t r = ((size_t)(tok + (ok ? 4 * g + i : 0)) * H + h) * DK + m;
#pragma unroll
        for (int t = 0; t < T; ++t) kt[t][i] = pk[r + 16 * t];
      }
      const float* row = a.w.row + cell * 3 * CT + SB * blk + 4 * g;
      *reinterpret_cast<float4*>(in) = *reinterpret_cast<const float4*>(row);
      *reinterpret_cast<float4*>(out) = *reinterpret_cast<const float4*>(row + CT);
      all[0] = a.w.row[cell * 3 * CT + SB * blk + SB - 1];
    }
    const TIN* pv = static_cast<const TIN*>(a.v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool ok = 4 * g + i < count;
      v[i] = pv[((size_t)(tok + (ok ? 4 * g + i : 0)) * H + h) * a.d_v + col];
    }
    const size_t o = (cell * NB + blk) * (SB * SB) + m * SB + 4 * g;
    if constexpr (!BWD) *reinterpret_cast<float4*>(P) = *reinterpret_cast<const float4*>(a.w.P + o);
    if constexpr (DELTA) {
      *reinterpret_cast<float4*>(A) = *reinterpret_cast<const float4*>(a.w.A + o);
      *reinterpret_cast<float4*>(b) =
          *reinterpret_cast<const float4*>(a.w.row + cell * 3 * CT + 2 * CT + SB * blk + 4 * g);
    }
  }

  // Zero for the rows behind the sequence's end. Applied when the block is used, not when it
  // is loaded: a loaded value that is touched has been waited for.
  __device__ __forceinline__ void clip(int count, int m, int g) {
    if constexpr (RULE != KDA) {
#pragma unroll
      for (int t = 0; t < T; ++t) {
        if constexpr (RULE != MAMBA2) k[t].mask(row_mask(m < count));
        if constexpr (!BWD) q[t].mask(row_mask(m < count));
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t ok = row_mask(4 * g + i < count);
      v[i] = masked(v[i], ok);
      if constexpr (RULE != KDA) {
#pragma unroll
        for (int t = 0; t < T; ++t) kt[t][i] = masked(kt[t][i], ok);
      }
    }
  }
};

// Forwards. Writes y and the final state, or for the backward pass (BWD) r of every
// token and the state at each chunk's start.
template <int RULE, int DK, typename TIN, bool BWD>
__global__ void __launch_bounds__(64) scan_state_kernel(const ScanArgs a) {
  constexpr bool DELTA = RULE != MAMBA2, CH = RULE == KDA;
  constexpr int T = DK / 16;
  using Step = StateStep<RULE, DK, TIN, BWD>;
  int unit, part;
  unit_of(blockIdx.x, a.d_v / 16, unit, part);
  const int seq = unit / a.heads, h = unit % a.heads;
  if (seq >= a.plan.seqs) return;
  int tok, len, first;
  if (!a.plan.sequence(seq, tok, len, first)) return;
  const int srow = a.slot ? a.slot[seq] : seq;
  if (srow < 0 || srow >= a.num_slots) return;
  const int lane = threadIdx.x, m = lane & 15, g = lane >> 4, col = 16 * part + m;
  const size_t so = ((size_t)srow * a.heads + h) * DK * a.d_v + (size_t)(4 * g) * a.d_v + col;

  f32x4 S[T];
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      S[t][i] = a.state_in ? a.state_in[so + (size_t)(16 * t + i) * a.d_v] : 0.f;

  const int blocks = (len + SB - 1) / SB;
  auto fetch = [&](Step& s, int j) {
    s.load(a, (size_t)(first + j / NB) * a.heads + h, j % NB, tok + SB * j, len - SB * j, h, col, m, g);
  };
  auto run = [&](Step& s, int j) {
    const size_t cell = (size_t)(first + j / NB) * a.heads + h;
    if (len - SB * j < SB) s.clip(len - SB * j, m, g);
    if constexpr (BWD) {
      if (j % NB == 0) {
        float* p = a.w.S + (cell * DK + 4 * g) * a.d_v + col;
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) p[(size_t)(16 * t + i) * a.d_v] = S[t][i];
      }
    }
    f32x4 ks = {0.f, 0.f, 0.f, 0.f}, o = ks, w;
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (DELTA) ks = mfma4(s.k[t][i], S[t][i], ks);
        if constexpr (!BWD) o = mfma4(s.q[t][i], S[t][i], o);
      }
    if constexpr (DELTA) {
      f32x4 r = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 4; ++i) r = mfma4(s.A[i], to_f32(s.v[i]) - (CH ? ks[i] : s.in[i] * ks[i]), r);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (BWD) a.w.r[(cell * CT + SB * (j % NB) + 4 * g + i) * a.d_v + col] = r[i];
        w[i] = s.b[i] * r[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = to_f32(s.v[i]);
    }
    if constexpr (!BWD) {
      if constexpr (!CH) {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] *= s.in[i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) o = mfma4(s.P[i], w[i], o);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (SB * j + 4 * g + i < len)
          a.y[((size_t)(tok + SB * j + 4 * g + i) * a.heads + h) * a.d_v + col] = o[i];
    }
    if constexpr (!CH) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] *= s.out[i];
    }
#pragma unroll
    for (int t = 0; t < T; ++t) {
#pragma unroll
      for (int i = 0; i < 4; ++i) S[t][i] *= CH ? s.all[CH ? 4 * t + i : 0] : s.all[0];
#pragma unroll
      for (int i = 0; i < 4; ++i) S[t] = mfma4(to_f32(s.kt[t][i]), w[i], S[t]);
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
      for (int i = 0; i < 4; ++i) a.state[so + (size_t)(16 * t + i) * a.d_v] = S[t][i];
  }
}

template <int RULE, int DK, typename TIN>
struct GradientStep {
  static constexpr int T = DK / 16;
  using KT = KeyT<RULE, TIN>;
  Quad<KT> k[T];             // KDA: O k
  KT qt[T][4], kt[T][4];     // KDA: I q, I k
  float dy[4], A[4], P[4], in[4], out[4], b[4], all[RULE == KDA ? 4 * T : 1];

  __device__ __forceinline__ void load(const ScanArgs& a, size_t cell, int blk, int tok, int count,
                                       int h, int col, int m, int g) {
    constexpr bool DELTA = RULE != MAMBA2;
    const size_t H = a.heads;
    if constexpr (RULE == KDA) {
      const size_t o = (cell * CT + SB * blk) * DK;
#pragma unroll
      for (int t = 0; t < T; ++t) {
        k[t].load(a.w.kt + o + m * DK + 16 * t + 4 * g);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          qt[t][i] = a.w.qh[o + (4 * g + i) * DK + 16 * t + m];
          kt[t][i] = a.w.kh[o + (4 * g + i) * DK + 16 * t + m];
        }
        *reinterpret_cast<float4*>(all + 4 * t) = *reinterpret_cast<const float4*>(
            a.w.all + (cell * NB + blk) * DK + 16 * t + 4 * g);
      }
    } else {
      const TIN* pk = static_cast<const TIN*>(a.k);
      const TIN* pq = static_cast<const TIN*>(a.q);
      const bool valid = m < count;
      const size_t at = ((size_t)(tok + (valid ? m : 0)) * H + h) * DK + 4 * g;
#pragma unroll
      for (int t = 0; t < T; ++t) k[t].load(pk + at + 16 * t);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool ok = 4 * g + i < count;
        const size_t r = ((size_t)(tok + (ok ? 4 * g + i : 0)) * H + h) * DK + m;
#pragma unroll
        for (int t = 0; t < T; ++t) {
          qt[t][i] = pq[r + 16 * t];
          if constexpr (DELTA) kt[t][i] = pk[r + 16 * t];
        }
      }
      const float* row = a.w.row + cell * 3 * CT + SB * blk + 4 * g;
      *reinterpret_cast<float4*>(in) = *reinterpret_cast<const float4*>(row);
      *reinterpret_cast<float4*>(out) = *reinterpret_cast<const float4*>(row + CT);
      all[0] = a.w.row[cell * 3 * CT + SB * blk + SB - 1];
    }
    const size_t o = (cell * NB + blk) * (SB * SB) + 4 * g * SB + m;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool ok = 4 * g + i < count;
      dy[i] = a.dy[((size_t)(tok + (ok ? 4 * g + i : 0)) * H + h) * a.d_v + col];
      P[i] = a.w.P[o + i * SB];  // column m: the transposed operand
      if constexpr (DELTA) A[i] = a.w.A2[o + i * SB];
    }
    if constexpr (DELTA)
      *reinterpret_cast<float4*>(b) =
          *reinterpret_cast<const float4*>(a.w.row + cell * 3 * CT + 2 * CT + SB * blk + 4 * g);
  }

  __device__ __forceinline__ void clip(int count, int m, int g) {
    if constexpr (RULE != KDA) {
#pragma unroll
      for (int t = 0; t < T; ++t) k[t].mask(row_mask(m < count));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t ok = row_mask(4 * g + i < count);
      dy[i] = masked(dy[i], ok);
      if constexpr (RULE != KDA) {
#pragma unroll
        for (int t = 0; t < T; ++t) {
          qt[t][i] = masked(qt[t][i], ok);
          if constexpr (RULE != MAMBA2) kt[t][i] = masked(kt[t][i], ok);
        }
      }
    }
  }
};

// Backwards. Writes dv, e of every token, dL/dS at each chunk's end and dL/d(initial state).
template <int RULE, int DK, typename TIN>
__global__ void __launch_bounds__(64) scan_gradient_kernel(const ScanArgs a) {
  constexpr bool DELTA = RULE != MAMBA2, CH = RULE == KDA;
  constexpr int T = DK / 16;
  using Step = GradientStep<RULE, DK, TIN>;
  int unit, part;
  unit_of(blockIdx.x, a.d_v / 16, unit, part);
  const int seq = unit / a.heads, h = unit % a.heads;
  if (seq >= a.plan.seqs) return;
  int tok, len, first;
  if (!a.plan.sequence(seq, tok, len, first)) return;
  const int lane = threadIdx.x, m = lane & 15, g = lane >> 4, col = 16 * part + m;
  const size_t so = ((size_t)seq * a.heads + h) * DK * a.d_v + (size_t)(4 * g) * a.d_v + col;
  TIN* dv = static_cast<TIN*>(a.dv);

  f32x4 G[T];
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      G[t][i] = a.dstate ? a.dstate[so + (size_t)(16 * t + i) * a.d_v] : 0.f;

  const int blocks = (len + SB - 1) / SB;
  auto fetch = [&](Step& s, int j) {
    s.load(a, (size_t)(first + j / NB) * a.heads + h, j % NB, tok + SB * j, len - SB * j, h, col, m, g);
  };
  auto run = [&](Step& s, int j) {
    const size_t cell = (size_t)(first + j / NB) * a.heads + h;
    if (len - SB * j < SB) s.clip(len - SB * j, m, g);
    if (j % NB == NB - 1 || j == blocks - 1) {
      float* p = a.w.G + (cell * DK + 4 * g) * a.d_v + col;
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) p[(size_t)(16 * t + i) * a.d_v] = G[t][i];
    }
    f32x4 w = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) w = mfma4(s.k[t][i], G[t][i], w);
    if constexpr (!CH) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] *= s.out[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) w = mfma4(s.P[i], s.dy[i], w);
    f32x4 dr;
    if constexpr (DELTA) {
      f32x4 e = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 4; ++i) e = mfma4(s.A[i], w[i], e);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a.w.e[(cell * CT + SB * (j % NB) + 4 * g + i) * a.d_v + col] = e[i];
        dr[i] = s.b[i] * e[i];
      }
    } else {
      dr = w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (SB * j + 4 * g + i < len)
        put(dv + ((size_t)(tok + SB * j + 4 * g + i) * a.heads + h) * a.d_v + col, dr[i]);
    f32x4 iy, ir;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      iy[i] = CH ? s.dy[i] : s.in[i] * s.dy[i];
      ir[i] = CH ? -dr[i] : -s.in[i] * dr[i];
    }
#pragma unroll
    for (int t = 0; t < T; ++t) {
#pragma unroll
      for (int i = 0; i < 4; ++i) G[t][i] *= CH ? s.all[CH ? 4 * t + i : 0] : s.all[0];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        G[t] = mfma4(to_f32(s.qt[t][i]), iy[i], G[t]);
        if constexpr (DELTA) G[t] = mfma4(to_f32(s.kt[t][i]), ir[i], G[t]);
      }
    }
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
      for (int i = 0; i < 4; ++i) a.dstate_in[so + (size_t)(16 * t + i) * a.d_v] = G[t][i];
  }
}

}  // namespace ssm
