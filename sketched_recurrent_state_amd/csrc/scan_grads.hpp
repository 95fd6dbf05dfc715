// scan_grads.hpp -- the gradients of q, k, the gates and beta of one chunk (64 tokens)
// of one head, all chunks at once, from the state at the chunk's start, its gradient at
// the chunk's end, and every token's r and e (notation in scan.hpp).
//
// A wave owns 32 key channels and holds the transposed state (rows v, columns d), so a
// product against it contracts the whole d_v in the wave's own registers and no sums
// cross waves. The state is carried forwards over the chunk's four blocks (its writes w
// are known), then the state's gradient backwards, which costs four blocks' updates
// instead of four times the states in memory.
#pragma once

#include "scan.hpp"

namespace ssm {

// Sum over the four lanes that differ in bits 4 and 5 of the values of lanes above this
// one, and over all four.
__device__ __forceinline__ void above(float x, int lane, int g, float& after, float& total) {
  after = total = 0.f;
#pragma unroll
  for (int o = 0; o < 4; ++o) {
    const float y = __shfl(x, (lane & 15) + 16 * o);
    total += y;
    if (o > g) after += y;
  }
}

template <int RULE, int DK, int DV, typename TIN>
__global__ void __launch_bounds__(DK >= 32 ? 2 * DK : 64) scan_grads_kernel(const ScanArgs a) {
  constexpr bool DELTA = RULE != MAMBA2, CH = RULE == KDA;
  constexpr int TD = DK >= 32 ? 2 : 1, W = DK >= 32 ? DK / 32 : 1, TV = DV / 16, LP = 20;
  __shared__ __align__(16) float sp[NB][SB * LP], sk[NB][SB * LP], sx[W][CT];
  __shared__ float send[W];
  const int cell = blockIdx.x, h = cell % a.heads;
  int tok, count;
  if (!a.plan.cell(cell / a.heads, tok, count)) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
  const int d0 = wave * 16 * TD + m;  // channel of tile u: d0 + 16 u
  const int nb = (count + SB - 1) / SB;
  const size_t H = a.heads;
  const TIN* q = static_cast<const TIN*>(a.q);
  const TIN* k = static_cast<const TIN*>(a.k);
  const TIN* v = static_cast<const TIN*>(a.v);
  const float* row = a.w.row + (size_t)cell * 3 * CT;
  const size_t base = (size_t)tok * H + h;  // token i: base + i * H

  // ---- the blocks' dP and dK, one block per wave in turn, with dbeta
  for (int blk = wave; blk < nb; blk += W) {
    const int left = count - SB * blk;
    const bool valid = m < left;
    const size_t at = base + (size_t)(SB * blk + (valid ? m : 0)) * H;
    f32x4 dP = {0.f, 0.f, 0.f, 0.f}, dK = dP;
    float db = 0.f;
    const size_t wr = ((size_t)cell * CT + SB * blk + m) * DV + 4 * g;
#pragma unroll
    for (int t = 0; t < TV; ++t) {
      Quad<float> y, r, e;
      Quad<TIN> x;
      y.load(a.dy + at * DV + 16 * t + 4 * g);
      y.mask(row_mask(valid));
      if constexpr (DELTA) {
        r.load(a.w.r + wr + 16 * t);
        e.load(a.w.e + wr + 16 * t);
      } else {
        x.load(v + at * DV + 16 * t + 4 * g);
        x.mask(row_mask(valid));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (DELTA) {
          dP = mfma4(y[i], r[i], dP);
          dK = mfma4(e[i], r[i], dK);
          db += e[i] * r[i];
        } else {
          dP = mfma4(y[i], x[i], dP);
        }
      }
    }
    float ratio[4] = {1.f, 1.f, 1.f, 1.f};
    if constexpr (!CH) {
      float in, out;
      gate_products(valid ? a.decay[at] : 1.f, m, g, in, out, ratio);
    }
    const float bj = DELTA ? row[2 * CT + SB * blk + m] : 1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * g + i;
      sp[blk][r * LP + m] = m <= r ? dP[i] * bj * ratio[i] : 0.f;
      if constexpr (DELTA)
        sk[blk][r * LP + m] = m < r ? -dK[i] * bj * row[2 * CT + SB * blk + r] * ratio[i] : 0.f;
    }
    if constexpr (DELTA) {
      db = xsum32(xsum16(db));
      if (g == 0 && valid) a.dbeta[at] = db;
    }
  }

  // ---- forwards: the state, dq and the readers' part of dk
  f32x4 S[TV][TD];
  const float* S0 = a.w.S + (size_t)cell * DK * DV;
#pragma unroll
  for (int t = 0; t < TV; ++t)
#pragma unroll
    for (int u = 0; u < TD; ++u)
      S[t][u] = *reinterpret_cast<const f32x4*>(S0 + (size_t)(d0 + 16 * u) * DV + 16 * t + 4 * g);
  __syncthreads();
  f32x4 dkr[NB][TD], x[NB][TD];

  // this lane's rows 4g + i of the block's keys, queries and gate products
  struct Rows {
    float q[TD][4], k[TD][4], in[TD][4], out[TD][4], all[TD], b[4];
    float qc[CH ? TD : 1][CH ? SB : 1], kc[CH ? TD : 1][CH ? SB : 1], ac[CH ? TD : 1][CH ? SB : 1];
  };
  auto rows = [&](Rows& z, int blk) {
    const int left = count - SB * blk;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool ok = 4 * g + i < left;
      const size_t at = (base + (size_t)(SB * blk + (ok ? 4 * g + i : 0)) * H) * DK + d0;
      z.b[i] = DELTA ? row[2 * CT + SB * blk + 4 * g + i] : 1.f;
#pragma unroll
      for (int u = 0; u < TD; ++u) {
        if constexpr (!CH) {
          z.q[u][i] = to_f32(masked(q[at + 16 * u], row_mask(ok)));
          z.k[u][i] = to_f32(masked(k[at + 16 * u], row_mask(ok)));
          z.in[u][i] = row[SB * blk + 4 * g + i];
          z.out[u][i] = row[CT + SB * blk + 4 * g + i];
          z.all[u] = row[SB * blk + SB - 1];
        }
      }
    }
    if constexpr (CH) {
#pragma unroll
      for (int u = 0; u < TD; ++u) {
#pragma unroll
        for (int l = 0; l < SB; ++l) {
          const bool ok = l < left;
          const size_t at = (base + (size_t)(SB * blk + (ok ? l : 0)) * H) * DK + d0 + 16 * u;
          z.qc[u][l] = to_f32(masked(q[at], row_mask(ok)));
          z.kc[u][l] = to_f32(masked(k[at], row_mask(ok)));
          const float gate = a.decay[at];
          z.ac[u][l] = ok ? gate : 1.f;
        }
        float p = 1.f;
#pragma unroll
        for (int l = 0; l < SB; ++l) {
          p *= z.ac[u][l];
          if (l >> 2 == g) {
            z.in[u][l & 3] = p;
            z.q[u][l & 3] = z.qc[u][l];
            z.k[u][l & 3] = z.kc[u][l];
          }
        }
        z.all[u] = p;
        p = 1.f;
#pragma unroll
        for (int l = SB - 1; l >= 0; --l) {
          if (l >> 2 == g) z.out[u][l & 3] = p;
          p *= z.ac[u][l];
        }
      }
    }
  };

#pragma unroll
  for (int blk = 0; blk < NB; ++blk) {
    if (blk >= nb) break;
    Rows z;
    rows(z, blk);
    const int left = count - SB * blk;
    const bool valid = m < left;
    const size_t at = (base + (size_t)(SB * blk + (valid ? m : 0)) * H) * DV + 4 * g;
    const size_t wr = ((size_t)cell * CT + SB * blk + m) * DV + 4 * g;
    f32x4 dq[TD], dk[TD];
#pragma unroll
    for (int u = 0; u < TD; ++u) dq[u] = dk[u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < TV; ++t) {
      Quad<float> y, e;
      y.load(a.dy + at + 16 * t);
      y.mask(row_mask(valid));
      if constexpr (DELTA) e.load(a.w.e + wr + 16 * t);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int u = 0; u < TD; ++u) {
          dq[u] = mfma4(y[i], S[t][u][i], dq[u]);
          if constexpr (DELTA) dk[u] = mfma4(e[i], S[t][u][i], dk[u]);
        }
    }
#pragma unroll
    for (int u = 0; u < TD; ++u) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        dq[u][i] *= z.in[u][i];
        dk[u][i] *= -z.in[u][i] * z.b[i];
      }
      if constexpr (!CH) {
        const float4 p4 = *reinterpret_cast<const float4*>(&sp[blk][m * LP + 4 * g]);
        const float p[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) dq[u] = mfma4(p[i], z.k[u][i], dq[u]);
        if constexpr (DELTA) {
          const float4 k4 = *reinterpret_cast<const float4*>(&sk[blk][m * LP + 4 * g]);
          const float kk[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) dk[u] = mfma4(kk[i], z.k[u][i], dk[u]);
        }
      } else {
        // row r: keys j = r, r - 1, .. decayed on the way (column j of G)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 4 * g + i;
          float p = 1.f;
#pragma unroll
          for (int j = SB - 1; j >= 0; --j) {
            const float y = j <= r ? p * z.kc[u][j] : 0.f;
            dq[u][i] += sp[blk][r * LP + j] * y;
            dk[u][i] += sk[blk][r * LP + j] * y;
            if (j <= r) p *= z.ac[u][j];
          }
        }
      }
      dkr[blk][u] = dk[u];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[blk][u][i] = z.q[u][i] * dq[u][i] + (DELTA ? z.k[u][i] * dk[u][i] : 0.f);
        if (4 * g + i < left)
          put(static_cast<TIN*>(a.dq) + (base + (size_t)(SB * blk + 4 * g + i) * H) * DK + d0 + 16 * u,
              dq[u][i]);
      }
    }
    // S <- a_1..a_16 S + (O k)^T w
#pragma unroll
    for (int t = 0; t < TV; ++t) {
      float wv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (DELTA) {
          wv[i] = a.w.r[((size_t)cell * CT + SB * blk + 4 * g + i) * DV + 16 * t + m];
        } else {
          const bool ok = 4 * g + i < left;
          wv[i] = to_f32(masked(v[(base + (size_t)(SB * blk + (ok ? 4 * g + i : 0)) * H) * DV + 16 * t + m],
                                row_mask(ok)));
        }
      }
#pragma unroll
      for (int u = 0; u < TD; ++u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) S[t][u][i] *= z.all[u];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          S[t][u] = mfma4(wv[i], z.out[u][i] * z.k[u][i] * z.b[i], S[t][u]);
      }
    }
  }

  // ---- backwards: the state's gradient, the writers' part of dk, the gates
  const float* G0 = a.w.G + (size_t)cell * DK * DV;
  float carry[TD];
#pragma unroll
  for (int u = 0; u < TD; ++u) carry[u] = 0.f;
#pragma unroll
  for (int t = 0; t < TV; ++t)
#pragma unroll
    for (int u = 0; u < TD; ++u) {
      const f32x4 G =
          *reinterpret_cast<const f32x4*>(G0 + (size_t)(d0 + 16 * u) * DV + 16 * t + 4 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i) carry[u] += S[t][u][i] * G[i];
      S[t][u] = G;
    }
#pragma unroll
  for (int u = 0; u < TD; ++u) carry[u] = xsum32(xsum16(carry[u]));  // rowsum(S_end * G_end)
  if constexpr (!CH) {
    float s = 0.f;
#pragma unroll
    for (int u = 0; u < TD; ++u) s += carry[u];
    s = row_allreduce(s);
    if (lane == 0) send[wave] = s;
  }
#pragma unroll
  for (int blk = NB - 1; blk >= 0; --blk) {
    if (blk >= nb) continue;
    Rows z;
    rows(z, blk);
    const int left = count - SB * blk;
    const bool valid = m < left;
    const size_t at = (base + (size_t)(SB * blk + (valid ? m : 0)) * H) * DV + 4 * g;
    const size_t wr = ((size_t)cell * CT + SB * blk + m) * DV + 4 * g;
    f32x4 dk[TD];
#pragma unroll
    for (int u = 0; u < TD; ++u) dk[u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < TV; ++t) {
      Quad<float> r;
      Quad<TIN> w;
      if constexpr (DELTA) {
        r.load(a.w.r + wr + 16 * t);
      } else {
        w.load(v + at + 16 * t);
        w.mask(row_mask(valid));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int u = 0; u < TD; ++u) {
          if constexpr (DELTA) dk[u] = mfma4(r[i], S[t][u][i], dk[u]);
          else dk[u] = mfma4(w[i], S[t][u][i], dk[u]);
        }
    }
#pragma unroll
    for (int u = 0; u < TD; ++u) {
#pragma unroll
      for (int i = 0; i < 4; ++i) dk[u][i] *= z.out[u][i] * z.b[i];
      if constexpr (!CH) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dk[u] = mfma4(sp[blk][(4 * g + i) * LP + m], z.q[u][i], dk[u]);
          if constexpr (DELTA) dk[u] = mfma4(sk[blk][(4 * g + i) * LP + m], z.k[u][i], dk[u]);
        }
      } else {
        // row j: readers i = j, j + 1, .. (row i of G)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = 4 * g + i;
          float p = 1.f;
#pragma unroll
          for (int r = 0; r < SB; ++r) {
            if (r > j) p *= z.ac[u][r];
            const float y = sp[blk][r * LP + j] * z.qc[u][r] + sk[blk][r * LP + j] * z.kc[u][r];
            dk[u][i] += r >= j ? p * y : 0.f;
          }
        }
      }
      f32x4 s;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[i] = x[blk][u][i] - z.k[u][i] * dk[u][i];
        if (4 * g + i < left)
          put(static_cast<TIN*>(a.dk) + (base + (size_t)(SB * blk + 4 * g + i) * H) * DK + d0 + 16 * u,
              dkr[blk][u][i] + dk[u][i]);
      }
      if constexpr (CH) {
#pragma unroll
        for (int i = 2; i >= 0; --i) s[i] += s[i + 1];
        float after, total;
        above(s[0], lane, g, after, total);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (4 * g + i < left)
            a.dlog[(base + (size_t)(SB * blk + 4 * g + i) * H) * DK + d0 + 16 * u] =
                carry[u] + after + s[i];
        carry[u] += total;
      } else {
        x[blk][u] = s;
      }
    }
    if constexpr (!CH) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float s = 0.f;
#pragma unroll
        for (int u = 0; u < TD; ++u) s += x[blk][u][i];
        s = row_allreduce(s);
        if (m == 0) sx[wave][SB * blk + 4 * g + i] = s;
      }
    }
    if (blk == 0) break;
    // G <- a_1..a_16 G + (I q)^T dy - (I k)^T dr
#pragma unroll
    for (int t = 0; t < TV; ++t) {
      float yv[4], ev[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool ok = 4 * g + i < left;
        yv[i] = masked(a.dy[(base + (size_t)(SB * blk + (ok ? 4 * g + i : 0)) * H) * DV + 16 * t + m],
                       row_mask(ok));
        if constexpr (DELTA) ev[i] = a.w.e[((size_t)cell * CT + SB * blk + 4 * g + i) * DV + 16 * t + m];
      }
#pragma unroll
      for (int u = 0; u < TD; ++u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) S[t][u][i] *= z.all[u];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          S[t][u] = mfma4(yv[i], z.in[u][i] * z.q[u][i], S[t][u]);
          if constexpr (DELTA) S[t][u] = mfma4(ev[i], -z.in[u][i] * z.b[i] * z.k[u][i], S[t][u]);
        }
      }
    }
  }
  if constexpr (!CH) {
    __syncthreads();
    if (wave == 0) {  // suffix sums over the chunk's tokens, lane = token
      float s = 0.f, end = 0.f;
      for (int w = 0; w < W; ++w) {
        s += lane < SB * nb ? sx[w][lane] : 0.f;
        end += send[w];
      }
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const float y = __shfl_down(s, o);
        if (lane + o < 64) s += y;
      }
      if (lane < count) a.dlog[base + (size_t)lane * H] = end + s;
    }
  }
}

}  // namespace ssm
